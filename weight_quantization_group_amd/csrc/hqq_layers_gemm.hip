// hqq_layers_gemm.hip -- the matrix product of the layers with many rows,
// C [M, N] = A [M, R] . B [N, R]^T in 16-bit inputs and fp32 sums on the matrix
// cores, and the operators' arithmetic on C while it is in registers.
//
// A workgroup computes a BM x BN tile of C with WM x WN waves.  Each 64-wide step
// of A and B goes from memory to LDS by DMA (no registers) into one of two
// buffers while the other is multiplied; a row's eight 16-byte runs are stored
// XOR-swizzled by the row's low bits, so that the 16 rows of an operand read
// spread over the banks.  The product is formed transposed (the rows of B are
// the instruction's rows): a lane then holds 4 consecutive columns n of one row
// m, which is what the row-wise softmax and the 16-bit stores want.
#include "hqq_layers_internal.h"
#include "hqq_linear_dev.h"

namespace hqq {
namespace {

// 16 bytes per lane from p into LDS at lds + 16 lane (lds the same in all lanes)
__device__ __forceinline__ void dma16(const uint16_t *p, uint4 *lds)
{
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_global_load_lds(p, (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
#endif
}

// what a run past the end of a segment of A reads
__device__ const uint4 zero_run = {0, 0, 0, 0};

constexpr float kLog2e = 1.44269504088896340736f;

// 2^x and 1 / x to about an ulp of fp32 (v_exp_f32, v_rcp_f32): the results are
// rounded to 16 bits, or summed over many terms
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// act(g) and, for the backward pass, act'(g).  Each activation is g * p with p in
// (0, 1) formed without cancellation (erfc, and (1 + tanh y) / 2 = 1 / (1 + exp(-2 y))),
// so that its far negative tail keeps its relative precision.
__device__ __forceinline__ float act_value(int act, float g, float &d)
{
    if (act == HQQ_ACT_GELU) {
        const float p = 0.5f * erfcf(g * -0.70710678118654752440f);
        d = p + g * 0.39894228040143267794f * exp2_fast(-0.5f * kLog2e * g * g);
        return g * p;
    }
    // exponent y2 of p = 1 / (1 + exp(-y2)), and its derivative
    float y2 = g, dy2 = 1.0f;
    if (act == HQQ_ACT_GELU_TANH) {
        const float a = 1.59576912160573071176f, b = 0.044715f;   // 2 sqrt(2 / pi)
        y2 = a * (g + b * g * g * g);
        dy2 = a * (1.0f + 3.0f * b * g * g);
    }
    const float e = exp2_fast(-kLog2e * y2);
    const float p = rcp_fast(1.0f + e);
    // p (1 - p) = p^2 e; where e overflows p is 0 and so is the product
    d = p + (e < INFINITY ? g * dy2 * (p * (p * e)) : 0.0f);
    return g * p;
}

__device__ __forceinline__ float from16(uint16_t b, bool bf)
{
    if (bf)
        return __uint_as_float((uint32_t)b << 16);
    _Float16 h;
    __builtin_memcpy(&h, &b, 2);
    return (float)h;
}

// four consecutive 16-bit values at p, of which the first cnt exist
template <bool BF>
__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4], int cnt)
{
    const uint32_t lo = out2<BF>(v[0], v[1]), hi = out2<BF>(v[2], v[3]);
    if (cnt >= 4 && ((uintptr_t)p & 7u) == 0) {
        *reinterpret_cast<uint2 *>(p) = uint2{lo, hi};
    } else {
        const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < cnt)
                p[r] = h[r];
    }
}

template <bool BF>
__device__ __forceinline__ void load4(const uint16_t *p, float (&v)[4], int cnt)
{
    uint16_t h[4] = {0, 0, 0, 0};
    if (cnt >= 4 && ((uintptr_t)p & 7u) == 0) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        h[0] = (uint16_t)u.x; h[1] = (uint16_t)(u.x >> 16); h[2] = (uint16_t)u.y; h[3] = (uint16_t)(u.y >> 16);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < cnt)
                h[r] = p[r];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        v[r] = from16(h[r], BF);
}

__device__ __forceinline__ void tile_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What becomes of a wave's part of C: TM x TN blocks of 16 x 16; acc[u][t][r] of
// lane l is C[m][n] with m = mw + 16 u + l % 16 and n = nw + 16 t + 4 (l / 16) + r.
// Gated kinds: blocks t < TN / 2 are gate columns and t >= TN / 2 the up columns
// of the same n = nw + 16 (t mod TN / 2) + ...
template <int OUT, bool BF, int TM, int TN>
__device__ __forceinline__ void epilogue(const GemmArgs &g, const float4v (&acc)[TM][TN], int mw, int nw, int lane,
                                         int z)
{
    const int l16 = lane & 15, l4 = lane >> 4;
#pragma unroll
    for (int u = 0; u < TM; ++u) {
        const int m = mw + 16 * u + l16;
        const bool m_in = m < g.M;
        if constexpr (OUT == kOutStore || OUT == kOutPart) {
            const float f = OUT == kOutStore && g.rowf && m_in ? g.rowf[m] : 1.0f;
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                const int n = nw + 16 * t + 4 * l4;
                if (m_in && n < g.N) {
                    if constexpr (OUT == kOutStore) {
                        const float v[4] = {acc[u][t][0] * f, acc[u][t][1] * f, acc[u][t][2] * f, acc[u][t][3] * f};
                        store4<BF>(g.out + (int64_t)m * g.ldo + n, v, g.N - n);
                    } else {
                        *reinterpret_cast<float4v *>(g.part + ((int64_t)z * g.M + m) * g.N + n) = acc[u][t];
                    }
                }
            }
        } else if constexpr (OUT == kOutGated) {
#pragma unroll
            for (int t = 0; t < TN / 2; ++t) {
                const int n = nw + 16 * t + 4 * l4;
                if (m_in && n < g.N) {
                    float v[4], d;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[r] = act_value(g.act, acc[u][t][r], d) * acc[u][t + TN / 2][r];
                    store4<BF>(g.out + (int64_t)m * g.ldo + n, v, g.N - n);
                }
            }
        } else if constexpr (OUT == kOutGatedGrad) {
            const float sc = g.rscale && m_in ? g.rscale[m] : 1.0f;
#pragma unroll
            for (int t = 0; t < TN / 2; ++t) {
                const int n = nw + 16 * t + 4 * l4;
                if (m_in && n < g.up_off) {
                    float y[4] = {0.f, 0.f, 0.f, 0.f}, vg[4], vu[4];
                    if (n < g.N)
                        load4<BF>(g.dY + (int64_t)m * g.N + n, y, g.N - n);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float d;
                        const float f = act_value(g.act, acc[u][t][r], d);
                        const float ys = y[r] * sc;
                        vg[r] = n + r < g.N ? ys * acc[u][t + TN / 2][r] * d : 0.0f;
                        vu[r] = n + r < g.N ? ys * f : 0.0f;
                    }
                    uint16_t *o = g.out + (int64_t)m * g.ldo + n;
                    store4<BF>(o, vg, 4);
                    store4<BF>(o + g.up_off, vu, 4);
                }
            }
        } else if constexpr (OUT == kOutStats) {
            // the row's max and sum of exp over this wave's columns, the target
            // left out (a lane's columns, then the four lanes of the row)
            const int64_t tgt = m_in ? g.targets[m] : -1;
            const int64_t at = tgt >= 0 && tgt < g.Nall ? tgt - g.n0 : -1;
            float mx = -INFINITY;
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = nw + 16 * t + 4 * l4 + r;
                    if (n < g.N && n != at)
                        mx = fmaxf(mx, acc[u][t][r]);
                    if (n == at && n < g.N)
                        g.tlogit[m] = acc[u][t][r];
                }
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float ref = mx > -INFINITY ? mx * kLog2e : 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = nw + 16 * t + 4 * l4 + r;
                    sum += n < g.N && n != at ? exp2_fast(__builtin_fmaf(acc[u][t][r], kLog2e, -ref)) : 0.0f;
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (m_in && l4 == 0 && nw < g.N)
                g.stats[(int64_t)m * g.blocks + nw / (16 * TN)] = float2{mx, sum};
        } else if constexpr (OUT == kOutSoftGrad) {
            const int64_t tgt = m_in ? g.targets[m] : -1;
            const bool keep = tgt >= 0 && tgt < g.Nall;
            const int64_t at = tgt - g.n0;
            const float ref = keep ? g.lse[m] : 0.0f;
            const float sc = BF ? 1.0f : 32768.0f;
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                const int n = nw + 16 * t + 4 * l4;
                if (m_in && n < g.ldo) {
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = exp2_fast((acc[u][t][r] - ref) * kLog2e) - (n + r == at ? 1.0f : 0.0f);
                        v[r] = keep && n + r < g.N ? p * sc : 0.0f;
                    }
                    store4<BF>(g.out + (int64_t)m * g.ldo + n, v, 4);
                }
            }
        }
    }
}

template <int OUT, bool BF, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void gemm_kernel(GemmArgs g)
{
    constexpr int NW = WM * WN;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr bool GATED = OUT == kOutGated || OUT == kOutGatedGrad;
    constexpr int BNC = GATED ? BN / 2 : BN;         // columns of the output per tile
    constexpr int IA = BM / 8 / NW, IB = BN / 8 / NW;
    __shared__ uint4 as0[BM * 8], bs0[BN * 8], as1[BM * 8], bs1[BN * 8];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int tile_n = (int)blockIdx.x / g.tiles_m, tile_m = (int)blockIdx.x - tile_n * g.tiles_m;
    const int m0 = tile_m * BM, n0 = tile_n * BNC;

    // DMA: wave w moves rows IA * 8 w ..., 8 rows per instruction; lane l fills
    // slot (row 8 i + l / 8, column l % 8), which holds run (l % 8) ^ (row % 8)
    const int run = (lane & 7) ^ (lane >> 3);
    int arow[IA];
#pragma unroll
    for (int i = 0; i < IA; ++i) {
        const int m = m0 + (IA * wave + i) * 8 + (lane >> 3);
        arow[i] = m < g.M ? m : g.M - 1;
    }
    const uint16_t *bp[IB], *ap[IA];
#pragma unroll
    for (int i = 0; i < IB; ++i) {
        const int r = (IB * wave + i) * 8 + (lane >> 3);
        int64_t row;
        if constexpr (GATED) {
            // a wave's BN / WN rows: half of them gate, half up, of the same n
            constexpr int PW = BN / WN, H = PW / 2;
            const int n = n0 + (r / PW) * H + r % H;
            row = (n < g.N ? n : g.N - 1) + (r % PW >= H ? g.B_up : 0);
        } else {
            const int n = n0 + r;
            row = n < g.N ? n : g.N - 1;
        }
        bp[i] = g.B + row * g.ldb + run * 8;
    }
    const int steps = g.step0[g.segs];
    const int per = (steps + g.splits - 1) / g.splits;
    const int s0 = (int)blockIdx.y * per;
    const int s1 = s0 + per < steps ? s0 + per : steps;
    int seg = 0;
    auto enter = [&](int sg) {
        seg = sg;
#pragma unroll
        for (int i = 0; i < IA; ++i)
            ap[i] = g.A[sg] + (int64_t)arow[i] * g.lda[sg] + run * 8;
    };
    auto dma = [&](int s, uint4 *as, uint4 *bs) {
        while (s >= g.step0[seg + 1])
            enter(seg + 1);
        const int c = (s - g.step0[seg]) * kStep;
        const bool whole = c + kStep <= g.rlen[seg];
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            const uint16_t *p = ap[i] + c;
            if (!whole)
                p = c + 8 * run < g.rlen[seg] ? p : reinterpret_cast<const uint16_t *>(&zero_run);
            dma16(p, &as[(IA * wave + i) * 64]);
        }
#pragma unroll
        for (int i = 0; i < IB; ++i)
            dma16(bp[i] + (int64_t)s * kStep, &bs[(IB * wave + i) * 64]);
    };
    float4v acc[TM][TN];
#pragma unroll
    for (int u = 0; u < TM; ++u)
#pragma unroll
        for (int t = 0; t < TN; ++t)
            acc[u][t] = float4v{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const uint4 *as, const uint4 *bs) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            uint4 a[TM], b[TN];
#pragma unroll
            for (int u = 0; u < TM; ++u) {
                const int r = wm * (BM / WM) + 16 * u + (lane & 15);
                a[u] = as[r * 8 + ((4 * ks + (lane >> 4)) ^ (r & 7))];
            }
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                const int r = wn * (BN / WN) + 16 * t + (lane & 15);
                b[t] = bs[r * 8 + ((4 * ks + (lane >> 4)) ^ (r & 7))];
            }
#pragma unroll
            for (int u = 0; u < TM; ++u)
#pragma unroll
                for (int t = 0; t < TN; ++t)
                    acc[u][t] = mfma<BF>(b[t], a[u], acc[u][t]);
        }
    };
    enter(0);
    dma(s0, as0, bs0);
    for (int s = s0; s < s1; s += 2) {
        tile_barrier();                       // step s has landed; buffer 1 is free
        if (s + 1 < s1)
            dma(s + 1, as1, bs1);
        multiply(as0, bs0);
        if (s + 1 < s1) {
            tile_barrier();
            if (s + 2 < s1)
                dma(s + 2, as0, bs0);
            multiply(as1, bs1);
        }
    }
    epilogue<OUT, BF, TM, TN>(g, acc, m0 + wm * (BM / WM), n0 + wn * (BNC / WN), lane, (int)blockIdx.y);
}

template <int OUT, bool BF>
hipError_t launch_out(GemmArgs &g, hipStream_t s)
{
    constexpr int BM = 128, BN = 128, WM = 2, WN = 2;
    constexpr bool GATED = OUT == kOutGated || OUT == kOutGatedGrad;
    g.tiles_m = (g.M + BM - 1) / BM;
    g.tiles_n = (g.N + (GATED ? BN / 2 : BN) - 1) / (GATED ? BN / 2 : BN);
    hipLaunchKernelGGL((gemm_kernel<OUT, BF, BM, BN, WM, WN>), dim3((unsigned)(g.tiles_m * g.tiles_n), (unsigned)g.splits),
                       dim3(WM * WN * 64), 0, s, g);
    return hipGetLastError();
}

template <bool BF>
hipError_t launch_dtype(GemmOut out, GemmArgs &g, hipStream_t s)
{
    switch (out) {
    case kOutStore: return launch_out<kOutStore, BF>(g, s);
    case kOutPart: return launch_out<kOutPart, BF>(g, s);
    case kOutGated: return launch_out<kOutGated, BF>(g, s);
    case kOutGatedGrad: return launch_out<kOutGatedGrad, BF>(g, s);
    case kOutStats: return launch_out<kOutStats, BF>(g, s);
    default: return launch_out<kOutSoftGrad, BF>(g, s);
    }
}

}  // namespace

hipError_t launch_gemm(GemmOut out, bool bf16, GemmArgs &g, hipStream_t s)
{
    return bf16 ? launch_dtype<true>(out, g, s) : launch_dtype<false>(out, g, s);
}

int gemm_splits(int64_t M, int64_t N, int64_t steps)
{
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    int sp = 1;
    while (sp < 32 && tiles * sp < 512 && steps / (2 * sp) >= 8)
        sp *= 2;
    while ((sp - 1) * ((steps + sp - 1) / sp) >= steps)
        --sp;
    return sp;
}

}  // namespace hqq
