// hqq_layers_gemm.hip -- the matrix products of the layers with many rows, 16-bit
// inputs and fp32 sums on the matrix cores: C [M, N] = A [M, R] . B [N, R]^T with the
// operators' arithmetic on C while it is in registers, and C = A . B [R, N] for the
// gradients.
//
// A workgroup computes a BM x BN tile of C with WM x WN waves.  Each 64-wide step
// of A and B goes from memory to LDS by DMA (no registers), into S buffers in turn; a
// row's eight 16-byte runs are stored XOR-swizzled by the row's low bits, so that the 16
// rows of an operand read spread over the banks.  The product is formed transposed (the
// rows of B are the instruction's rows): a lane then holds 4 consecutive columns n of one
// row m, which is what the row-wise softmax and the 16-bit stores want.  For the gradients
// the sum runs down the rows of W_hat as it lies there: LDS reads that transpose (4 rows x
// 16 columns among 16 lanes) give the operands, so that no transposed copy of W_hat is
// written (gated backward 2048 x 4096 x 11008, 707 us with one, 647 without).
//
// Bound by the matrix cores, at the clock that the power limit leaves on random data (zeros
// run faster): 2048 x 4096 x 22016 with the gated epilogue takes 287 us, 1.29 PFLOP/s in bf16,
// where torch's product of 8192^3 reaches 1.42 to 1.57.  Its 688 tiles are 2.69 rounds of the
// CUs, so that a tenth of it is the last round's idle part; nothing runs under a workgroup's
// epilogue, and the gated gradient's costs 23 us more (310).  The products of the gradients:
// 2048 x 22016 x 4096 in two splits 1.42 PFLOP/s without their sum, 2048 x 57344 x 8192 1.46.
#include "hqq_layers_epilogue.h"

namespace hqq {
namespace {

// 16 bytes per lane from p into LDS at lds + 16 lane (lds the same in all lanes)
__device__ __forceinline__ void dma16(const void *p, uint4 *lds)
{
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_global_load_lds(p, (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
#endif
}

// ds_read_b64_tr_b16
__device__ __forceinline__ uint2 read_tr(const char *lds)
{
#ifdef __HIP_DEVICE_COMPILE__
    typedef short short4v __attribute__((ext_vector_type(4)));
    const short4v v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) short4v *)const_cast<char *>(lds));
    uint2 u;
    __builtin_memcpy(&u, &v, 8);
    return u;
#else
    return uint2{0, 0};
#endif
}

// The workgroup's barrier, with this wave's LDS accesses complete and at most VM of its
// memory accesses under way.
template <int VM>
__device__ __forceinline__ void tile_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((VM & 15) | 0x0070 | (VM >> 4) << 14);   // vmcnt(VM) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// c += B . A (one 16x16x32 step) with c in accumulation registers, in place.  Written as
// an instruction: from the builtin the compiler gives results registers of their own
// and moves them about, which with 128 sums per lane costs spills in the loop.  It does
// not see an instruction here that needs waiting for: see settle().
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <bool BF>
__device__ __forceinline__ void mfma_into(float4v &c, uint4v B, uint4v A)
{
#ifdef __HIP_DEVICE_COMPILE__
    if constexpr (BF)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(B), "v"(A));
    else
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(B), "v"(A));
#endif
}

// The sums may be read after this: the last matrix instruction's result takes at most
// 18 wait states, and every sum's uses are ordered behind them.
template <int N>
__device__ __forceinline__ void settle(float4v (&c)[N])
{
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_nop 15\n\ts_nop 3");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+a"(c[i]));
#endif
}

// Eight consecutive 16-bit values at p, of which cnt exist (1 .. 8, or more).
__device__ __forceinline__ void store8(uint16_t *p, uint4 v, int cnt)
{
    if (cnt >= 8 && ((uintptr_t)p & 15u) == 0) {
        *reinterpret_cast<uint4 *>(p) = v;
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < cnt)
                p[r] = (uint16_t)(w[r / 2] >> (16 * (r & 1)));
    }
}

__device__ __forceinline__ uint4 load8(const uint16_t *p, int cnt)
{
    if (cnt >= 8 && ((uintptr_t)p & 15u) == 0)
        return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (r < cnt)
            w[r / 2] |= (uint32_t)p[r] << (16 * (r & 1));
    return uint4{w[0], w[1], w[2], w[3]};
}

// What becomes of a wave's part of C: TM x 4 blocks of 16 x 16; acc[u][t][r] of lane l is
// C[m][n] with m = mw + 16 u + l % 16 and n = nw + 16 t + 4 (l / 16) + r.  Gated kinds:
// t = 0, 1 are the gate columns and t = 2, 3 the up columns of the same 32 n.  Values go
// through LDS (4 KB at st for the wave alone), 16 rows at a time, so that memory sees 16
// bytes per lane and whole stretches of a row; they would otherwise be 32-byte pieces of
// 16 rows per instruction.  A row's pitch there is 16 bytes more than its values, against
// bank conflicts.
template <int OUT, int ACT, bool BF, int TM>
__device__ __forceinline__ void epilogue(const GemmArgs &g, const float4v (&acc)[TM][4], int mw, int nw, int lane,
                                         int z, char *st)
{
    const int l16 = lane & 15, l4 = lane >> 4;
    if constexpr (OUT == kOutStore || OUT == kOutSoftGrad) {
        constexpr int P = 144;
        const int width = OUT == kOutStore ? g.N : (int)g.fill;
#pragma unroll
        for (int u = 0; u < TM; ++u) {
            const int m = mw + 16 * u + l16, mc = m < g.M ? m : g.M - 1;
            float f = 1.0f, ref = 0.0f;
            int64_t at = -1;
            bool keep = true;
            if constexpr (OUT == kOutStore) {
                f = row_factor(g.rowf, mc);
            } else {
                const int64_t tgt = g.targets[mc];
                keep = tgt >= 0 && tgt < g.Nall;
                at = tgt - g.n0 - nw;
                ref = g.lse[mc];
                f = BF ? 1.0f : 32768.0f;
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int n = 16 * t + 4 * l4;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (OUT == kOutStore) {
                        v[r] = acc[u][t][r] * f;
                    } else {
                        const float p = exp2_fast((acc[u][t][r] - ref) * kLog2e) - (n + r == at ? 1.0f : 0.0f);
                        v[r] = keep && nw + n + r < g.N ? p * f : 0.0f;
                    }
                }
                *reinterpret_cast<uint2 *>(st + l16 * P + 2 * n) = uint2{out2<BF>(v[0], v[1]), out2<BF>(v[2], v[3])};
            }
            wave_fence();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 8 * i + (lane >> 3), n = nw + 8 * (lane & 7), mr = mw + 16 * u + row;
                const uint4 v = *reinterpret_cast<const uint4 *>(st + row * P + 16 * (lane & 7));
                if (mr < g.M && n < width)
                    store8(g.out + (int64_t)mr * g.ldo + n, v, width - n);
            }
            wave_fence();
        }
    } else if constexpr (OUT == kOutPart) {
        constexpr int P = 144;
#pragma unroll
        for (int u = 0; u < TM; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    *reinterpret_cast<float4v *>(st + l16 * P + 4 * (16 * t + 4 * l4)) = acc[u][2 * h + t];
                wave_fence();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = 8 * i + (lane >> 3), n = nw + 32 * h + 4 * (lane & 7), mr = mw + 16 * u + row;
                    const float4v v = *reinterpret_cast<const float4v *>(st + row * P + 16 * (lane & 7));
                    if (mr < g.M && n < g.N)
                        *reinterpret_cast<float4v *>(g.part + ((int64_t)z * g.M + mr) * g.N + n) = v;
                }
                wave_fence();
            }
    } else if constexpr (OUT == kOutGated || OUT == kOutGatedGrad) {
        constexpr int P = 80;
        constexpr bool GRAD = OUT == kOutGatedGrad;
        char *sg = st, *su = st + 16 * P, *sy = st + 32 * P;
        const float wb = GRAD && g.bound.row ? weight_bound(g.bound) : 0.0f;
        const int row4 = lane >> 2, n4 = nw + 8 * (lane & 3);      // coalesced: 4 lanes per row
        // dY four blocks of rows at a time where the tile is whole: loads behind branches come
        // one by one, and all eight take registers that the sums need
        uint4 y[4];
        auto load_y = [&](int u0) {
            if (mw + 16 * TM <= g.M && nw + 32 <= g.N && g.ldy % 8 == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (u0 + i < TM)
                        y[i] = *reinterpret_cast<const uint4 *>(g.dY + (int64_t)(mw + 16 * (u0 + i) + row4) * g.ldy + n4);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int mr = mw + 16 * (u0 + i) + row4;
                    y[i] = mr < g.M && n4 < g.N ? load8(g.dY + (int64_t)mr * g.ldy + n4, g.N - n4) : uint4{0, 0, 0, 0};
                }
            }
        };
#pragma unroll
        for (int u = 0; u < TM; ++u) {
            const int m = mw + 16 * u + l16, mc = m < g.M ? m : g.M - 1;
            float sc = 1.0f;
            if (GRAD && g.bound.row) {
                float inv;
                sc = grad_scale(g.bound.row[mc], wb, inv);
                if (nw == 0 && l4 == 0 && m < g.M)
                    g.rinv[m] = inv;
            }
            if constexpr (GRAD) {
                if (u % 4 == 0)
                    load_y(u);
                *reinterpret_cast<uint4 *>(sy + row4 * P + 16 * (lane & 3)) = y[u % 4];
                wave_fence();
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int n = 16 * t + 4 * l4;
                float vg[4], vu[4], yv[4];
                if constexpr (GRAD)
                    load4<BF>(sy + l16 * P + 2 * n, yv);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float d;
                    const float f = act_value<ACT>(acc[u][t][r], d);
                    if constexpr (GRAD) {
                        const float ys = yv[r] * sc;
                        const bool in = nw + n + r < g.N;
                        vg[r] = in ? ys * acc[u][t + 2][r] * d : 0.0f;
                        vu[r] = in ? ys * f : 0.0f;
                    } else {
                        vg[r] = f * acc[u][t + 2][r];
                    }
                }
                *reinterpret_cast<uint2 *>(sg + l16 * P + 2 * n) = uint2{out2<BF>(vg[0], vg[1]), out2<BF>(vg[2], vg[3])};
                if constexpr (GRAD)
                    *reinterpret_cast<uint2 *>(su + l16 * P + 2 * n) =
                        uint2{out2<BF>(vu[0], vu[1]), out2<BF>(vu[2], vu[3])};
            }
            wave_fence();
            const int mr = mw + 16 * u + row4, width = GRAD ? (int)g.fill : g.N;
            // (dG and dU in turn by 32 columns, as the weights' rows are)
            uint16_t *o = g.out + (int64_t)mr * g.ldo + (GRAD ? nw + n4 : n4);
            const uint4 v = *reinterpret_cast<const uint4 *>(sg + row4 * P + 16 * (lane & 3));
            if (mr < g.M && n4 < width)
                store8(o, v, width - n4);
            if constexpr (GRAD) {
                const uint4 w = *reinterpret_cast<const uint4 *>(su + row4 * P + 16 * (lane & 3));
                if (mr < g.M && n4 < width)
                    store8(o + 32, w, 8);
            }
            wave_fence();
        }
    } else {   // kOutStats
        // the row's max and sum of exp over this wave's 64 columns, the target left out (a
        // lane's columns, then the four lanes of the row), left at st for the tile's join
#pragma unroll
        for (int u = 0; u < TM; ++u) {
            const int m = mw + 16 * u + l16;
            const bool m_in = m < g.M;
            const int64_t tgt = g.targets[m_in ? m : g.M - 1];
            const int64_t at = tgt >= 0 && tgt < g.Nall ? tgt - g.n0 - nw : -1;
            float mx = -INFINITY, tl = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = 16 * t + 4 * l4 + r;
                    const float v = acc[u][t][r];
                    mx = nw + n < g.N && n != at ? fmaxf(mx, v) : mx;
                    tl = n == at ? v : tl;
                }
            if (m_in && at >= 0 && at < 64 && nw + at < g.N && ((at >> 2) & 3) == l4)
                g.tlogit[m] = tl;
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float ref = stats_ref(mx);
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = 16 * t + 4 * l4 + r;
                    sum += nw + n < g.N && n != at ? exp2_fast((acc[u][t][r] - ref) * kLog2e) : 0.0f;
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (l4 == 0)
                reinterpret_cast<float2 *>(st)[16 * u + l16] = float2{mx, sum};
        }
    }
}

// kOutStats: the (max, sum) of the WN waves that share a row become the tile's; part(w, r):
// wave w's of its row r.
template <int BM, int WM, int WN, typename Part>
__device__ __forceinline__ void join_stats(const GemmArgs &g, int m0, int tile_n, Part &&part)
{
    __syncthreads();
    const int r = threadIdx.x;
    if (r >= BM || m0 + r >= g.M)
        return;
    float2 v[WN];
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < WN; ++w) {
        v[w] = part((r / (BM / WM)) * WN + w, r % (BM / WM));
        mx = fmaxf(mx, v[w].x);
    }
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WN; ++w)
        sum += fabsf(mx) < INFINITY ? v[w].y * exp2_fast((v[w].x - mx) * kLog2e) : v[w].y;
    g.stats[(int64_t)(m0 + r) * g.blocks + tile_n] = float2{mx, sum};
}

// The tile and split of a workgroup.  Workgroups go to the 8 XCDs in turn: each XCD
// gets a contiguous part of the tiles (of one split after the other), in bands of
// kBand tile rows walked column by column, so that the tiles that run on it at one
// time share rows of A and of B in its L2.
constexpr int kBand = 4;

__device__ __forceinline__ void tile_of(const GemmArgs &g, int &tm, int &tn, int &split)
{
    const uint32_t tiles = (uint32_t)(g.tiles_m * g.tiles_n), T = gridDim.x, id = blockIdx.x;
    const uint32_t q = T / 8, r = T % 8, x = id % 8;
    const uint32_t all = x * q + (x < r ? x : r) + id / 8;
    split = (int)(all / tiles);
    const uint32_t t = all - (uint32_t)split * tiles;
    const uint32_t band = t / (uint32_t)(kBand * g.tiles_n), first = band * kBand;
    const uint32_t rows = (uint32_t)g.tiles_m - first < kBand ? (uint32_t)g.tiles_m - first : kBand;
    const uint32_t l = t - first * (uint32_t)g.tiles_n;
    tm = (int)(first + l % rows);
    tn = (int)(l / rows);
}

// A step is two halves of 32 k.  A wave's operands of one half are in registers
// while those of the next are read from LDS under its matrix instructions: the
// second half's from this step's buffers, then, behind the step's one barrier, the
// next step's first half from the next buffers.  That barrier also frees this
// step's buffers, and the DMA of the step S later goes into them under the second
// half, S - 1 whole steps ahead of its use.
template <int OUT, int ACT, bool BF, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(WM * WN * 64) void gemm_kernel(GemmArgs g)
{
    constexpr int NW = WM * WN;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    static_assert(TN == 4, "64 columns per wave: the softmax blocks and the gate / up halves");
    constexpr bool GATED = OUT == kOutGated || OUT == kOutGatedGrad;
    constexpr bool DOWN = OUT == kOutStore || OUT == kOutPart;    // B [R, N]: the sum runs down its rows
    constexpr int BNC = GATED ? BN / 2 : BN;         // columns of the output per tile
    constexpr int IA = BM / 8 / NW, IB = BN / 8 / NW;
    // (arrays of their own: reads of one do not wait for the DMA into another)
    __shared__ uint4 as0[BM * 8], bs0[BN * 8], as1[BM * 8], bs1[BN * 8];
    __shared__ uint4 as2[S > 2 ? BM * 8 : 1], bs2[S > 2 ? BN * 8 : 1], as3[S > 3 ? BM * 8 : 1], bs3[S > 3 ? BN * 8 : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    int tile_m, tile_n, split;
    tile_of(g, tile_m, tile_n, split);
    const int m0 = tile_m * BM, n0 = tile_n * BNC;

    // DMA: wave w moves rows IA * 8 w ..., 8 rows per instruction; lane l fills
    // slot (row 8 i + l / 8, column l % 8), which holds run (l % 8) ^ (row % 8).
    // Rows past the end repeat the last.  The lanes' byte offsets from the tile's
    // first row are formed at each use: kept, they would cost registers.
    const uint32_t run16 = 16 * ((lane & 7) ^ (lane >> 3));
    // DOWN: a step of B is 64 rows of BN columns, RB of them per instruction; a row's
    // 32-byte pieces are XOR-swizzled by its low bits, so that the transposing reads of 16
    // rows spread over the banks.
    constexpr int SB = BN / 8, RB = 64 / SB, MB = BN / 16 - 1;
    int row_a = IA * 8 * wave + (lane >> 3);
    int row_b = DOWN ? IB * RB * wave + lane / SB : IB * 8 * wave + (lane >> 3);
    const int b0 = tile_n * BN;
    const int last_b = DOWN ? (int)g.ldb - 8 : (GATED ? 2 * ((g.N + 31) / 32 * 32) : g.N) - b0 - 1;
    const int last_a = g.M - m0 - 1;
    const char *bb = reinterpret_cast<const char *>(DOWN ? g.B : g.B + (int64_t)b0 * g.ldb);
    uint32_t ldb2 = (uint32_t)(g.ldb * 2);
    const int steps = g.steps;
    const int per = (steps + g.splits - 1) / g.splits;
    const int s0 = split * per;
    const int s1 = s0 + per < steps ? s0 + per : steps;
    // The first segment's fields come with the other arguments; those of a later one, read
    // by its number, are loads that wait for one another.
    int seg = 0, seg_end = g.step0[1];
    const char *ab = reinterpret_cast<const char *>(g.A[0] + (int64_t)m0 * g.lda[0]);   // of the (virtual) step 0
    uint32_t lda2 = (uint32_t)(g.lda[0] * 2);
    auto enter = [&](int s) {          // the segment of step s (not before the current one)
        while (s >= seg_end)
            seg_end = g.step0[++seg + 1];
        ab = reinterpret_cast<const char *>(g.A[seg] + (int64_t)m0 * g.lda[seg] - (int64_t)g.step0[seg] * kStep);
        lda2 = (uint32_t)(g.lda[seg] * 2);
    };
    auto dma_a = [&](int i, int s, uint4 *as) {
        const int r = row_a + 8 * i < last_a ? row_a + 8 * i : last_a;
        dma16(ab + (int64_t)s * (2 * kStep) + ((uint32_t)r * lda2 + run16), as + (IA * wave + i) * 64);
    };
    auto dma_b = [&](int i, int s, uint4 *bs) {
        if constexpr (DOWN) {
            const int r = row_b + RB * i, slot = lane % SB;
            const int c = b0 + 16 * ((slot >> 1) ^ (r & MB)) + 8 * (slot & 1);
            // (columns past the pitch repeat its last; they are not stored)
            dma16(bb + (int64_t)s * kStep * ldb2 + ((uint32_t)r * ldb2 + 2 * (uint32_t)(c < last_b ? c : last_b)),
                  bs + (IB * wave + i) * 64);
        } else {
            const int r = row_b + 8 * i < last_b ? row_b + 8 * i : last_b;
            dma16(bb + (int64_t)s * (2 * kStep) + ((uint32_t)r * ldb2 + run16), bs + (IB * wave + i) * 64);
        }
    };
    auto dma = [&](int s, uint4 *as, uint4 *bs) {
#pragma unroll
        for (int i = 0; i < IA; ++i)
            dma_a(i, s, as);
#pragma unroll
        for (int i = 0; i < IB; ++i)
            dma_b(i, s, bs);
    };
    float4v acc[TM][TN];
#pragma unroll
    for (int u = 0; u < TM; ++u)
#pragma unroll
        for (int t = 0; t < TN; ++t)
            acc[u][t] = float4v{0.f, 0.f, 0.f, 0.f};
    uint4v a[TM], b[TN];
    const int l16 = lane & 15, l4 = lane >> 4, sw = lane & 7;
    auto read_a = [&](int ks, int u, const uint4 *as) {
        return reinterpret_cast<const uint4v *>(as)[(wm * (BM / WM) + 16 * u + l16) * 8 + ((4 * ks + l4) ^ sw)];
    };
    auto read_b = [&](int ks, int t, const uint4 *bs) {
        if constexpr (DOWN) {
            // 8 rows of a column: two reads that transpose 4 rows x 16 columns among 16 lanes
            // (lane i of them reads 8 bytes of row i / 4 and gets column i)
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = 8 * l4 + 4 * q + (l16 >> 2);
                const uint2 v = read_tr(reinterpret_cast<const char *>(bs) + 32 * ks * (2 * BN) + r * (2 * BN) +
                                        (((wn * 4 + t) ^ (r & MB)) * 32 + 8 * (l16 & 3)));
                w[2 * q] = v.x;
                w[2 * q + 1] = v.y;
            }
            return uint4v{w[0], w[1], w[2], w[3]};
        } else {
            return reinterpret_cast<const uint4v *>(bs)[(wn * (BN / WN) + 16 * t + l16) * 8 + ((4 * ks + l4) ^ sw)];
        }
    };
    // One half: TM groups of TN matrix instructions; the reads of the next half's
    // operands (half ks of the given buffers) are spread over all but the last of
    // them, in the order of their use, so that most of them take the registers of
    // operands already used; `more(i)` goes beside group i.
    constexpr int RP = (TM + TN + TM - 2) / (TM - 1);
    auto half = [&](int ks, const uint4 *as, const uint4 *bs, auto &&more) {
        uint4v an[TM], bn[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int r = RP * i; r < RP * (i + 1); ++r) {
                if (r < TN)
                    bn[r] = read_b(ks, r, bs);
                else if (r < TN + TM)
                    an[r - TN] = read_a(ks, r - TN, as);
            }
            more(i);
#pragma unroll
            for (int t = 0; t < TN; ++t)
                mfma_into<BF>(acc[i][t], b[t], a[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int u = 0; u < TM; ++u)
            a[u] = an[u];
#pragma unroll
        for (int t = 0; t < TN; ++t)
            b[t] = bn[t];
    };
    constexpr int DP = (IA + IB + TM - 1) / TM;
    auto step = [&](int s, uint4 *asc, uint4 *bsc, const uint4 *asn, const uint4 *bsn) {
        // past the end the DMA repeats the last step (in bounds, never used)
        const int sn = s + S < s1 ? s + S : s1 - 1;
        if (sn >= seg_end)
            enter(sn);
        // (hides that the pitches do not change: the offsets are not to be kept)
        asm volatile("" : "+s"(lda2), "+s"(ldb2), "+v"(row_a), "+v"(row_b));
        __builtin_amdgcn_sched_barrier(0);
        half(1, asc, bsc, [](int) {});
        tile_barrier<(S - 2) * (IA + IB)>();   // this step's reads are done, the next step has landed
        half(0, asn, bsn, [&](int i) {
#pragma unroll
            for (int j = DP * i; j < DP * (i + 1); ++j) {
                if (j < IA)
                    dma_a(j, sn, asc);
                else if (j < IA + IB)
                    dma_b(j - IA, sn, bsc);
            }
        });
    };
    auto start = [&](int i, uint4 *as, uint4 *bs) {
        const int sn = s0 + i < s1 ? s0 + i : s1 - 1;
        if (sn >= seg_end)
            enter(sn);
        dma(sn, as, bs);
    };
    start(0, as0, bs0);
    start(1, as1, bs1);
    if constexpr (S > 2)
        start(2, as2, bs2);
    if constexpr (S > 3)
        start(3, as3, bs3);
    tile_barrier<(S - 1) * (IA + IB)>();
#pragma unroll
    for (int t = 0; t < TN; ++t)
        b[t] = read_b(0, t, bs0);
#pragma unroll
    for (int u = 0; u < TM; ++u)
        a[u] = read_a(0, u, as0);
    int s = s0;
    for (; s + S <= s1; s += S) {
        step(s, as0, bs0, as1, bs1);
        if constexpr (S == 2) {
            step(s + 1, as1, bs1, as0, bs0);
        } else {
            step(s + 1, as1, bs1, as2, bs2);
            if constexpr (S == 3) {
                step(s + 2, as2, bs2, as0, bs0);
            } else {
                step(s + 2, as2, bs2, as3, bs3);
                step(s + 3, as3, bs3, as0, bs0);
            }
        }
    }
    if (s < s1)
        step(s, as0, bs0, as1, bs1);
    if constexpr (S > 2)
        if (s + 1 < s1)
            step(s + 1, as1, bs1, as2, bs2);
    if constexpr (S > 3)
        if (s + 2 < s1)
            step(s + 2, as2, bs2, as3, bs3);
    tile_barrier<0>();     // no DMA is under way and no operand read: the buffers are free
#pragma unroll
    for (int u = 0; u < TM; ++u)
        settle(acc[u]);
    static_assert(BM * 128 >= NW / 2 * 4096, "4 KB per wave");
    static_assert(S >= 2 && S <= 4, "buffers");
    auto scratch = [&](int w) { return reinterpret_cast<char *>(w < NW / 2 ? as0 : as1) + (w % (NW / 2)) * 4096; };
    char *st = scratch(wave);
    epilogue<OUT, ACT, BF, TM>(g, acc, m0 + wm * (BM / WM), n0 + wn * (BNC / WN), lane, split, st);
    if constexpr (OUT == kOutStats)
        join_stats<BM, WM, WN>(g, m0, tile_n, [&](int w, int r) { return reinterpret_cast<const float2 *>(scratch(w))[r]; });
}

// Tiles (rows x columns, buffers): 256 x 256 (2) and 256 x 128 (3) with 8 waves, 128 x
// 128 (4) with 4 waves, one workgroup per CU, and 64 x 128 (3) with 4 waves, two per CU.
// Their times per 64-wide step in bf16 on MI355X, with the chip full and with at most half
// its workgroups running: 1.50 and 1.25 us, 0.88 and 0.80, 0.52, 0.60 and 0.40, for either
// order of B (in traces of the gradients 1.47 to 1.51 at 125 to 896 steps of 256 x 256, and 1.8
// with the ends counted at 80) (large
// products: 44, 37, 32 and 27 thousand outputs per CU and us; the more buffers, the less
// a step waits for memory: 256 x 128 with two ran 2048 x 4096 x 22016 in 373 us, with three
// in 318).  The tile of the fewest us by rounds of workgroups over the CUs; where that
// leaves CUs idle, the steps are split and a second pass adds the parts (3 us and the
// parts' and the result's bytes at 6 TB/s).
struct Tile {
    int bm, bn, per_cu;
    double us, us_half;
};
constexpr Tile kTiles[] = {{256, 256, 1, 1.50, 1.25}, {256, 128, 1, 0.88, 0.80}, {128, 128, 1, 0.52, 0.52},
                           {64, 128, 2, 0.60, 0.40}};
constexpr int kTileKinds = 4;
constexpr int kCus = 256;
constexpr int kMaxSplits = 32;

double pick_tile(int64_t M, int64_t N, int64_t steps, bool gated, bool may_split, int &tile, int &splits)
{
    double best = 0.0;
    tile = 0;
    splits = 1;
    for (int t = 0; t < kTileKinds; ++t) {
        const Tile &k = kTiles[t];
        const int64_t bn = gated ? k.bn / 2 : k.bn, slots = kCus * k.per_cu;
        const int64_t tiles = (M + k.bm - 1) / k.bm * ((N + bn - 1) / bn);
        for (int sp = 1; sp <= (may_split ? kMaxSplits : 1); ++sp) {
            if (sp > 1 && (steps / sp < 4 || tiles * (sp - 1) >= 4 * slots))
                break;          // a part has a few steps at least; four rounds balance well enough
            const int64_t per = (steps + sp - 1) / sp;
            if ((sp - 1) * per >= steps)
                continue;       // none is empty
            const int64_t rest = tiles * sp % slots;
            const double round = (double)(tiles * sp / slots) * k.us + (rest == 0 ? 0.0 : 2 * rest <= slots ? k.us_half : k.us);
            double us = 3.0 + (double)per * round;
            if (sp > 1)
                us += 3.0 + (double)M * (double)N * (4.0 * sp + 2.0) / 6.0e6;
            if (best == 0.0 || us < best) {
                best = us;
                tile = t;
                splits = sp;
            }
        }
    }
    return best;
}

template <int OUT, int ACT, bool BF, int BM, int BN, int WM, int WN, int S>
hipError_t launch_tile(GemmArgs &g, hipStream_t s)
{
    constexpr bool GATED = OUT == kOutGated || OUT == kOutGatedGrad;
    constexpr int BNC = GATED ? BN / 2 : BN;
    g.tiles_m = (g.M + BM - 1) / BM;
    g.tiles_n = (g.N + BNC - 1) / BNC;
    g.steps = g.step0[g.segs];
    hipLaunchKernelGGL((gemm_kernel<OUT, ACT, BF, BM, BN, WM, WN, S>),
                       dim3((unsigned)(g.tiles_m * g.tiles_n * g.splits)), dim3(WM * WN * 64), 0, s, g);
    return hipGetLastError();
}

template <int OUT, int ACT, bool BF>
hipError_t launch_out(GemmArgs &g, hipStream_t s)
{
    int tile = g.tile, sp;
    if (OUT != kOutStore && OUT != kOutPart)
        pick_tile(g.M, g.N, g.step0[g.segs], OUT == kOutGated || OUT == kOutGatedGrad, false, tile, sp);
    switch (tile) {
    case 0: return launch_tile<OUT, ACT, BF, 256, 256, 2, 4, 2>(g, s);
    case 1: return launch_tile<OUT, ACT, BF, 256, 128, 4, 2, 3>(g, s);
    case 2: return launch_tile<OUT, ACT, BF, 128, 128, 2, 2, 4>(g, s);
    default: return launch_tile<OUT, ACT, BF, 64, 128, 2, 2, 3>(g, s);
    }
}

template <int OUT, bool BF>
hipError_t launch_act(GemmArgs &g, hipStream_t s)
{
    switch (g.act) {
    case HQQ_ACT_SILU: return launch_out<OUT, HQQ_ACT_SILU, BF>(g, s);
    case HQQ_ACT_GELU: return launch_out<OUT, HQQ_ACT_GELU, BF>(g, s);
    default: return launch_out<OUT, HQQ_ACT_GELU_TANH, BF>(g, s);
    }
}

template <bool BF>
hipError_t launch_dtype(GemmOut out, GemmArgs &g, hipStream_t s)
{
    switch (out) {
    case kOutStore: return launch_out<kOutStore, 0, BF>(g, s);
    case kOutPart: return launch_out<kOutPart, 0, BF>(g, s);
    case kOutGated: return launch_act<kOutGated, BF>(g, s);
    case kOutGatedGrad: return launch_act<kOutGatedGrad, BF>(g, s);
    case kOutStats: return launch_out<kOutStats, 0, BF>(g, s);
    default: return launch_out<kOutSoftGrad, 0, BF>(g, s);
    }
}

}  // namespace

hipError_t launch_gemm(GemmOut out, bool bf16, GemmArgs &g, hipStream_t s)
{
    return bf16 ? launch_dtype<true>(out, g, s) : launch_dtype<false>(out, g, s);
}

double gemm_us(int64_t M, int64_t N, int64_t steps)
{
    int tile, splits;
    return pick_tile(M, N, steps, false, false, tile, splits);
}

int64_t gemm_stats_blocks(int64_t M, int64_t N, int64_t steps)
{
    int tile, splits;
    pick_tile(M, N, steps, false, false, tile, splits);
    return (N + kTiles[tile].bn - 1) / kTiles[tile].bn;
}

void gemm_gradient_tile(int64_t M, int64_t N, int64_t steps, int &tile, int &splits)
{
    pick_tile(M, N, steps, false, true, tile, splits);
}

}  // namespace hqq
