// hqq_layers_skinny.h -- the layers' products for few rows, straight from the
// packed codes: decoding, small batches and short prompts, where the weights'
// bytes and the latency of a launch count and nothing is unpacked to memory.
//
// Forward (skinny_kernel), C [M, N] = X . W_hat^T: a workgroup owns 16 columns
// n (of the gated block: the same 16 of gate and of up, which share the rows
// of X) and its waves split K.  Lane l works on row n = l % 16 and, in each
// 256-wide step, on 64 k, the codes of one group or a few, dequantized in
// registers to the eight operands of eight 16x16x32 MFMAs.  The next step's codes load under the current one's
// arithmetic.  The waves add their sums through LDS, and the operator's
// arithmetic follows there.
//
// Bound by the dequantization's instructions (a table of a group's 16 values and 2.6
// instructions per lookup at 4 bits, about 6 per weight otherwise) and by the launch's ramp: a
// 4096 x 11008 pair, 1 row 4-bit g64 20 us for 56 MB of codes, scales and zeros, 24 rows
// 8-bit g128 39 us for 96 MB; 8 rows of a 4096 x 32000 head 36 us for 82 MB.  VALU
// instructions issue in 54, 43 and 61 % of these kernels' cycles; the waves wait for codes, X or
// LDS in 28, 21 and 22 % of their time, and in 37, 40 and 54 % for their turn to issue.  Four waves per workgroup, eight below 512 workgroups: 5, 6 and 7
// leave the SIMDs uneven and cost up to 37 %.
#pragma once

#include "hqq_layers_epilogue.h"

namespace hqq {
namespace {

constexpr int kSkinnyWaves = 8;      // waves per workgroup, at most

// X in LDS: a row is K / 8 + 1 runs, so that 16 rows fall in different banks
inline int64_t skinny_x_bytes(int64_t rows, int64_t K) { return rows * (K / 8 + 1) * 16; }

// Activations chosen at run time (one element at a time: the code is small).
__device__ __forceinline__ float act_any(int act, float g, float &d)
{
    return act == HQQ_ACT_SILU   ? act_value<HQQ_ACT_SILU>(g, d)
           : act == HQQ_ACT_GELU ? act_value<HQQ_ACT_GELU>(g, d)
                                 : act_value<HQQ_ACT_GELU_TANH>(g, d);
}

// One element C[m][n] (gated: of gate and of up; wb: weight_bound).  For kOutStats the 16 lanes of a
// row hold its 16 columns; all lanes of the wave call.
template <bool BF>
__device__ __forceinline__ void element(GemmOut out, const GemmArgs &g, float wb, float c0, float c1, int m, int n)
{
    const bool m_in = m < g.M;
    if (out == kOutGated) {
        float d;
        if (m_in && n < g.N)
            g.out[(int64_t)m * g.ldo + n] = out1<BF>(act_any(g.act, c0, d) * c1);
    } else if (out == kOutGatedGrad) {
        if (m_in && n < g.fill) {
            float vg = 0.0f, vu = 0.0f;
            if (n < g.N) {
                float d, sc = 1.0f;
                if (g.bound.row) {
                    float inv;
                    sc = grad_scale(g.bound.row[m], wb, inv);
                    if (n == 0)
                        g.rinv[m] = inv;
                }
                const float f = act_any(g.act, c0, d);
                const float y = from16(g.dY[(int64_t)m * g.ldy + n], BF) * sc;
                vg = y * c1 * d;
                vu = y * f;
            }
            uint16_t *o = g.out + (int64_t)m * g.ldo + n;
            o[0] = out1<BF>(vg);
            o[g.up_off] = out1<BF>(vu);
        }
    } else if (out == kOutStats) {
        const int64_t at = m_in ? g.targets[m] : -1;
        if (n == at && n < g.N && m_in)
            g.tlogit[m] = c0;
        const bool in = n < g.N && n != at;
        float mx = in ? c0 : -INFINITY;
#pragma unroll
        for (int o = 1; o < 16; o *= 2)
            mx = fmaxf(mx, __shfl_xor(mx, o));
        float sum = in ? exp2_fast((c0 - stats_ref(mx)) * kLog2e) : 0.0f;
#pragma unroll
        for (int o = 1; o < 16; o *= 2)
            sum += __shfl_xor(sum, o);
        if (m_in && (n & 15) == 0)
            g.stats[(int64_t)m * g.blocks + n / 16] = float2{mx, sum};
    } else {
        const int64_t at = m_in ? g.targets[m] : -1;
        if (m_in && n < g.fill) {
            float v = 0.0f;
            if (at >= 0 && at < g.Nall && n < g.N) {
                const float p = exp2_fast((c0 - g.lse[m]) * kLog2e) - (n == at ? 1.0f : 0.0f);
                v = BF ? p : p * 32768.0f;
            }
            g.out[(int64_t)m * g.ldo + n] = out1<BF>(v);
        }
    }
}

// X where it stays in global memory: a wave fetches its step's rows in two halves (each
// lane quarter's first and second 32 k), 64 bytes or more in a row, and turns them into
// operands through 4 MT KiB of LDS of its own.  (An operand fetched directly touches a
// cache line per lane, and what was fetched is gone from the L1 cache by the next operand:
// 59 against 41 us for the gated block of 24 rows through 4096 x 11008 at 8 bits.)  Run j
// of quarter q of row r lies at 64 j + 16 q + (r ^ (j + 4 q)) of its 16-row block: the
// writes of 8 neighbouring lanes, and the reads, fall into
// different banks.
template <int MT>
struct XHalf {
    uint4 x[4 * MT];
};

template <bool KT, int MT>
__device__ __forceinline__ void load_half(XHalf<MT> &b, const LinearArgs &a, uint32_t k, uint32_t row0, int rows, int lane)
{
    // k: of this lane's run (lane % 16); past K any run, cleared when it is stored
    const uint32_t kk = KT && k >= (uint32_t)a.K ? (uint32_t)a.K - 8 : k;
#pragma unroll
    for (int t = 0; t < 4 * MT; ++t) {
        const int r = lane / 16 + 4 * t < rows ? lane / 16 + 4 * t : rows - 1;
        b.x[t] = *at<uint4>(a.X, 2 * ((row0 + (uint32_t)r) * (uint32_t)a.K + kk));
    }
}

template <bool KT, int MT>
__device__ __forceinline__ void store_half(const XHalf<MT> &b, uint4 *xs, uint32_t in, int lane)
{
    const int q = (lane >> 2) & 3, j = lane & 3;
#pragma unroll
    for (int t = 0; t < 4 * MT; ++t) {
        const int r = lane / 16 + 4 * (t & 3);
        uint4 v = run_order(b.x[t]);
        if constexpr (KT)
            v = and4(v, in);
        xs[(t >> 2) * 256 + 64 * j + 16 * q + (r ^ (j + 4 * q))] = v;
    }
}

// A lane's 64 k of a 256-wide step are two halves of 32.  In groups of 64 and more, at up
// to 4 bits, they lie next to each other in one group, whose scale (and table) serves both;
// else the lane quarters' first halves lie side by side, then their second ones, so that
// the loads of codes and of X cover whole lines (24 rows through 4096 x 11008 8-bit 43.4 ->
// 40.8 us, 32 rows in groups of 16 55 -> 48; 2-bit groups of 64 lose, 27 -> 29).
template <int GPC>
struct Span {
    static constexpr uint32_t lane = GPC == 1 ? 64 : 32;     // from quarter to quarter
    static constexpr uint32_t half = GPC == 1 ? 32 : 128;    // from half to half
};

// Scales of a lane's 64 k
constexpr int groups_of(int nbits, int gs) { return gs >= 64 && nbits < 8 ? 1 : gs >= 32 ? 2 : 64 / gs; }

// Where the halves start; one past K (K % 256 != 0) is moved to the last 32 k, in bounds
// and cleared
template <bool KT, typename S>
__device__ __forceinline__ Chunk halves(uint32_t kbase, int quarter, uint32_t K)
{
    uint32_t k0 = kbase + S::lane * (uint32_t)quarter, kh = k0 + S::half;
    if constexpr (KT) {
        k0 = k0 < K ? k0 : K - 32;
        kh = kh < K ? kh : K - 32;
    }
    return Chunk{k0, kh};
}

// A lane's codes and scales of a step.  A half's 2 or 4 small groups lie next to each
// other, on 8 and 16 bytes (K is a multiple of 32): one load each (fetched one by one,
// the pair of 4096 x 11008 in groups of 16 took 57 us, now 32).
template <int NB, int GPC>
__device__ __forceinline__ void fetch(StepBuf<NB, GPC> &b, const LinearArgs &a, Chunk c, uint32_t nw, uint32_t ng)
{
    if constexpr (GPC <= 2) {
        load_step(b, a, c, nw, ng);
    } else {
        StepBuf<NB, 1> codes;
        load_step(codes, a, c, nw, ng);
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
            b.w[i] = codes.w[i];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t g = 4 * (ng + ((h ? c.kh : c.k0) >> a.gshift));
            if constexpr (GPC == 4) {
                const float2 s = *at<float2>(a.scale, g), z = *at<float2>(a.zero, g);
                b.s[2 * h] = s.x; b.s[2 * h + 1] = s.y;
                b.z[2 * h] = z.x; b.z[2 * h + 1] = z.y;
            } else {
                const float4 s = *at<float4>(a.scale, g), z = *at<float4>(a.zero, g);
                b.s[4 * h] = s.x; b.s[4 * h + 1] = s.y; b.s[4 * h + 2] = s.z; b.s[4 * h + 3] = s.w;
                b.z[4 * h] = z.x; b.z[4 * h + 1] = z.y; b.z[4 * h + 2] = z.z; b.z[4 * h + 3] = z.w;
            }
        }
    }
}

// B operand j (8-k run j of a lane's 64) by direct quotients, in operand order
template <int NB, int GPC, bool BF>
__device__ __forceinline__ uint4 quotients(const StepBuf<NB, GPC> &b, int j)
{
    constexpr uint32_t MASK = (1u << NB) - 1u;
    constexpr int ord[8] = {0, 2, 4, 6, 1, 3, 5, 7};
    const int gi = j * GPC / 8;
    const double R = reciprocal(b.s[gi]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int bit = (8 * j + ord[i]) * NB;
        v[i] = wq((float)((b.w[bit / 32] >> (bit % 32)) & MASK), b.z[gi], R);
    }
    return uint4{out2<BF>(v[0], v[1]), out2<BF>(v[2], v[3]), out2<BF>(v[4], v[5]), out2<BF>(v[6], v[7])};
}

// acc += the operands of half H of a step; a(u, j): operand j of the half, of row block u.
// km clears the weights of a lane whose half lies past K.
template <int H, bool KT, bool BF, int NM, int NB, int MT, int GPC, typename RowRuns>
__device__ __forceinline__ void compute_half(const StepBuf<NB, GPC> (&b)[NM], uint32_t km, float4v (&acc)[NM][MT],
                                             RowRuns &&a)
{
    Tab4 tab[NM];
    if constexpr (NB == 4 && GPC <= 2) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
            tab[m] = make_tab4<BF>(b[m].s[GPC == 1 ? 0 : H], b[m].z[GPC == 1 ? 0 : H]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint4 A[MT];
#pragma unroll
        for (int u = 0; u < MT; ++u)
            A[u] = a(u, j);
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            uint4 B;
            if constexpr (NB == 4 && GPC <= 2)
                B = lookup4(tab[m], b[m].w[4 * H + j]);
            else
                B = quotients<NB, GPC, BF>(b[m], 4 * H + j);
            if constexpr (KT)
                B = and4(B, km);
#pragma unroll
            for (int u = 0; u < MT; ++u)
                acc[m][u] = mfma<BF>(A[u], B, acc[m][u]);
        }
    }
}

// Waves per SIMD that leave the registers for this step's codes and scales and the next's
// (three for the 8-bit pair of 32 rows would spill: 24 rows through 4096 x 11008 43 -> 49 us)
constexpr int waves_per_simd(int nm, int nb, int mt, int gpc)
{
    const int regs = nm * (4 * nb + 4 * gpc) + 20 * mt + 4 * nm * mt;
    return regs <= 72 ? 4 : regs <= 130 ? 3 : 2;
}

// NM: matrices (2: gate and up).  The workgroup's waves split K.
template <int NM, bool KT, int NB, int MT, int GPC, bool XL, bool BF>
__global__ __launch_bounds__(kSkinnyWaves * 64) __attribute__((amdgpu_waves_per_eu(waves_per_simd(NM, NB, MT, GPC)))) void
skinny_kernel(SkinnyArgs s)
{
    using S = Span<GPC>;
    const int WPB = blockDim.x >> 6;
    extern __shared__ uint4 lds[];
    const LinearArgs &a = s.w[0];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane16 = lane & 15, grp = lane >> 4;
    const uint32_t K = (uint32_t)a.K;
    const int64_t n_raw = (int64_t)blockIdx.x * 16 + lane16;
    const uint32_t n = (uint32_t)(n_raw < a.N ? n_raw : a.N - 1);
    const uint32_t nw = n * (uint32_t)a.wpr, ng = n * (uint32_t)a.gpl;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    const int mrows = (int)(a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT);
    const uint32_t xrow = K / 8 + 1;
    uint32_t xr[MT];      // XL; rows past M repeat the last, their outputs are not stored
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const int r = 16 * u + lane16 < mrows ? 16 * u + lane16 : mrows - 1;
        xr[u] = (uint32_t)r * xrow;
    }

    const int n_steps = (int)((K + kStepK - 1) / kStepK);
    const int my = n_steps > wave ? (n_steps - wave + WPB - 1) / WPB : 0;
    auto kbase = [&](int i) { return (uint32_t)(wave + i * WPB) * kStepK; };
    StepBuf<NB, GPC> buf[NM];
    auto load = [&](int i) {
        const Chunk c = halves<KT, S>(kbase(i), grp, K);
#pragma unroll
        for (int j = 0; j < NM; ++j)
            fetch(buf[j], s.w[j], c, nw, ng);
    };
    // the first codes are on their way before X is staged
    if (my > 0)
        load(0);
    if constexpr (XL) {
        const uint32_t runs = K / 8;
        const uint4 *xg = reinterpret_cast<const uint4 *>(a.X + m0 * a.K);
        for (uint32_t c = threadIdx.x; c < (uint32_t)mrows * runs; c += WPB * 64) {
            const uint32_t m = c / runs, r = c - m * runs;
            lds[m * xrow + r] = run_order(xg[c]);
        }
        __syncthreads();
    }
    float4v acc[NM][MT];
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
        for (int u = 0; u < MT; ++u)
            acc[j][u] = float4v{0.f, 0.f, 0.f, 0.f};
    if constexpr (XL) {
        for (int i = 0; i < my; ++i) {
            const Chunk c = halves<KT, S>(kbase(i), grp, K);
            const uint32_t k0 = kbase(i) + S::lane * grp;
            const uint32_t km0 = k0 < K ? 0xffffffffu : 0u;
            const uint32_t km1 = k0 + S::half < K ? 0xffffffffu : 0u;
            StepBuf<NB, GPC> cur[NM];
#pragma unroll
            for (int j = 0; j < NM; ++j)
                cur[j] = buf[j];
            if (i + 1 < my)
                load(i + 1);
            auto runs = [&](uint32_t first, uint32_t km) {
                return [&, first, km](int u, int j) {
                    const uint4 A = lds[xr[u] + first + j];
                    return KT ? and4(A, km) : A;
                };
            };
            compute_half<0, KT, BF>(cur, km0, acc, runs(c.k0 >> 3, km0));
            compute_half<1, KT, BF>(cur, km1, acc, runs(c.kh >> 3, km1));
        }
    } else {
        uint4 *xs = lds + wave * (256 * MT);
        auto run = [&](int u, int j) { return xs[u * 256 + 64 * j + (lane & 48) + ((lane & 15) ^ (j + 4 * grp))]; };
        // the run this lane fetches, of the first half of step i
        auto krun = [&](int i) { return kbase(i) + S::lane * (uint32_t)((lane >> 2) & 3) + 8 * (uint32_t)(lane & 3); };
        XHalf<MT> x;
        if (my > 0)
            load_half<KT>(x, a, krun(0), (uint32_t)m0, mrows, lane);
        for (int i = 0; i < my; ++i) {
            const uint32_t k0 = kbase(i) + S::lane * grp, kr = krun(i);
            StepBuf<NB, GPC> cur[NM];
#pragma unroll
            for (int j = 0; j < NM; ++j)
                cur[j] = buf[j];
            store_half<KT>(x, xs, kr < K ? 0xffffffffu : 0u, lane);
            wave_fence();
            load_half<KT>(x, a, kr + S::half, (uint32_t)m0, mrows, lane);
            if (i + 1 < my)
                load(i + 1);
            compute_half<0, KT, BF>(cur, k0 < K ? 0xffffffffu : 0u, acc, run);
            wave_fence();
            store_half<KT>(x, xs, kr + S::half < K ? 0xffffffffu : 0u, lane);
            wave_fence();
            if (i + 1 < my)
                load_half<KT>(x, a, krun(i + 1), (uint32_t)m0, mrows, lane);
            compute_half<1, KT, BF>(cur, k0 + S::half < K ? 0xffffffffu : 0u, acc, run);
            wave_fence();
        }
    }

    // the waves' sums: red[wave][matrix][4 u + r][lane]
    __syncthreads();
    float *red = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                red[((wave * NM + j) * MT * 4 + u * 4 + r) * 64 + lane] = acc[j][u][r];
    __syncthreads();
    const float wb = s.g.bound.row ? weight_bound(s.g.bound) : 0.0f;
    for (int idx = threadIdx.x; idx < MT * 4 * 64; idx += WPB * 64) {
        const int v = idx >> 6, l = idx & 63;      // one v per wave
        float c[NM];
#pragma unroll
        for (int j = 0; j < NM; ++j) {
            c[j] = 0.0f;
            for (int w = 0; w < WPB; ++w)
                c[j] += red[((w * NM + j) * MT * 4 + v) * 64 + l];
        }
        // sum r of lane l is C[4 (l / 16) + r][l % 16] of m tile u
        const int m = (int)m0 + 16 * (v >> 2) + 4 * (l >> 4) + (v & 3);
        const int nn = (int)blockIdx.x * 16 + (l & 15);
        element<BF>(s.out, s.g, wb, c[0], c[NM - 1], m, nn);
    }
}

template <int NM, int NB, int MT, int GPC, bool XL, bool BF>
hipError_t launch_xl(const SkinnyArgs &s, dim3 grid, int waves, hipStream_t st)
{
    const LinearArgs &a = s.w[0];
    size_t lds = (size_t)waves * NM * MT * 4 * 64 * sizeof(float);
    if (XL) {
        const size_t x = (size_t)skinny_x_bytes(a.M < 16 * MT ? a.M : 16 * MT, a.K);
        lds = x > lds ? x : lds;
    } else {
        const size_t x = (size_t)waves * MT * 4096;
        lds = x > lds ? x : lds;
    }
    if (a.K % kStepK != 0)
        hipLaunchKernelGGL((skinny_kernel<NM, true, NB, MT, GPC, XL, BF>), grid, dim3(waves * 64), lds, st, s);
    else
        hipLaunchKernelGGL((skinny_kernel<NM, false, NB, MT, GPC, XL, BF>), grid, dim3(waves * 64), lds, st, s);
    return hipGetLastError();
}

template <int NM, int NB, int MT, int GPC, bool BF>
hipError_t launch_gpc(const SkinnyArgs &s, hipStream_t st)
{
    const LinearArgs &a = s.w[0];
    const dim3 grid((unsigned)((s.cols + 15) / 16), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
    const int64_t blocks = (int64_t)grid.x * grid.y, steps = (a.K + kStepK - 1) / kStepK;
    const int waves = blocks < 512 && steps > 4 ? 8 : 4;
    // X in LDS as a whole for up to 4 rows, where that leaves the CU 16 waves (4096 x 11008
    // 4-bit pair, 2 rows 22 against 25 us in halves; 8 or 16 rows through 1024 x 2816 to
    // 1024 x 32003 lose 2-12 % by it)
    if constexpr (MT == 1)
        if (a.M <= 4 && skinny_x_bytes(a.M, a.K) <= (waves == 8 ? 64 : 40) * 1024)
            return launch_xl<NM, NB, MT, GPC, true, BF>(s, grid, waves, st);
    return launch_xl<NM, NB, MT, GPC, false, BF>(s, grid, waves, st);
}

template <int NM, int NB, bool BF>
hipError_t launch_mt(const SkinnyArgs &s, hipStream_t st)
{
    const bool one = s.w[0].M <= 16;
    const int gpc = groups_of(NB, s.w[0].gs);
    if constexpr (NB < 8)
        if (gpc == 1)
            return one ? launch_gpc<NM, NB, 1, 1, BF>(s, st) : launch_gpc<NM, NB, 2, 1, BF>(s, st);
    switch (gpc) {
    case 2: return one ? launch_gpc<NM, NB, 1, 2, BF>(s, st) : launch_gpc<NM, NB, 2, 2, BF>(s, st);
    case 4: return one ? launch_gpc<NM, NB, 1, 4, BF>(s, st) : launch_gpc<NM, NB, 2, 4, BF>(s, st);
    default: return one ? launch_gpc<NM, NB, 1, 8, BF>(s, st) : launch_gpc<NM, NB, 2, 8, BF>(s, st);
    }
}

template <int NM>
hipError_t launch_skinny_nm(int nbits, bool bf16, const SkinnyArgs &s, hipStream_t st)
{
    switch (nbits) {
    case 1: return bf16 ? launch_mt<NM, 1, true>(s, st) : launch_mt<NM, 1, false>(s, st);
    case 2: return bf16 ? launch_mt<NM, 2, true>(s, st) : launch_mt<NM, 2, false>(s, st);
    case 4: return bf16 ? launch_mt<NM, 4, true>(s, st) : launch_mt<NM, 4, false>(s, st);
    case 8: return bf16 ? launch_mt<NM, 8, true>(s, st) : launch_mt<NM, 8, false>(s, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace
}  // namespace hqq
