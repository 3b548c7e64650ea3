// hqq_layers_skinny_grad.hip -- C [M, K] = sum_i A_i . W_hat_i for few rows,
// straight from the packed codes.
//
// The sum runs over the rows n of the weights while their codes run along k.  A
// lane takes 8 rows n by 8 consecutive k, dequantizes them, and transposes the
// square in registers (one byte permutation per pair of values; the rest renames
// registers): operand j of its 8 MFMAs is column k = 8 (l % 16) + j of the rows
// 8 (l / 16) .. + 7.  A wave covers 128 k and 32 rows per step; the next step's
// codes load under the current one's arithmetic.  Waves and workgroups split the
// rows; the waves' sums meet in LDS, the workgroups' in a second launch, in a
// fixed order.  Bound by the arithmetic of the dequantization (about 5 instructions per
// weight) and by the latency of two launches: 16 rows through 4096 x 11008 at 4 bits 23.5
// us, of which about 4 are the second; through 4096 x 4096 15, with VALU instructions in a
// third of the first launch's cycles.
#include "hqq_layers_epilogue.h"

namespace hqq {
namespace {

constexpr int kGradWaves = 4;

// 8 consecutive codes of a row
template <int NB>
__device__ __forceinline__ uint2 load_codes(const uint8_t *p)
{
    if constexpr (NB == 8)
        return *reinterpret_cast<const uint2 *>(p);
    else if constexpr (NB == 4)
        return uint2{*reinterpret_cast<const uint32_t *>(p), 0u};
    else if constexpr (NB == 2)
        return uint2{*reinterpret_cast<const uint16_t *>(p), 0u};
    else
        return uint2{*p, 0u};
}

// One step of a lane: the codes of 8 rows, the meta of 8 / SH of them, and its runs of A
template <int NB, int MT, int SH>
struct GradBuf {
    uint2 c[8];
    float s[8 / SH], z[8 / SH];
    uint4 a[MT];
};

// 8 values of A at columns n .. n + 7 of a row; those at or past N are 0
template <bool AL>
__device__ __forceinline__ uint4 load_run(const uint16_t *row, int n, int N)
{
    if (AL && n + 8 <= N)
        return *reinterpret_cast<const uint4 *>(row + n);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = n + 2 * i < N ? row[n + 2 * i] : 0u;
        const uint32_t hi = n + 2 * i + 1 < N ? row[n + 2 * i + 1] : 0u;
        w[i] = lo | hi << 16;
    }
    return uint4{w[0], w[1], w[2], w[3]};
}

// AL: the runs of A are 16-byte aligned.  SH: neighbouring lanes whose 8 k lie in the same
// groups (8 in groups of 64 and more); each fetches and inverts 8 / SH of the 8 scales
template <int NB, int MT, bool BF, bool AL, int SH>
__global__ __launch_bounds__(kGradWaves * 64) __attribute__((amdgpu_waves_per_eu(MT == 1 ? 4 : 3))) void
skinny_grad_kernel(SkinnyGradArgs a)
{
    constexpr uint32_t MASK = (1u << NB) - 1u;
    __shared__ float4v red[kGradWaves / 2][MT * 8][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, l4 = lane >> 4;
    const int kc_raw = (int)blockIdx.x * 128 + 8 * l16;
    const int kc = kc_raw < a.K ? kc_raw : (int)a.K - 8;       // past K: any codes, never stored
    const int m0 = (int)blockIdx.z * 16 * MT;
    const int steps = a.steps;
    const int per = (steps + a.splits - 1) / a.splits;
    const int s0 = (int)blockIdx.y * per, s1 = s0 + per < steps ? s0 + per : steps;

    // The first weight's fields come with the other arguments; those of a later one, read
    // by its number, are loads that wait for one another.
    int j = 0, first = 0, end = a.step0[1], N = a.n[0];
    const uint32_t *packed = a.packed[0];
    const float *scale = a.scale[0], *zero = a.zero[0];
    const uint16_t *A = a.A[0];
    int64_t lda = a.lda[0];
    GradBuf<NB, MT, SH> buf;
    auto load = [&](int s) {
        if (s >= end) {
            while (s >= end)
                end = a.step0[++j + 1];
            first = a.step0[j];
            N = a.n[j];
            packed = a.packed[j];
            scale = a.scale[j];
            zero = a.zero[j];
            A = a.A[j];
            lda = a.lda[j];
        }
        const int n0 = 32 * (s - first) + 8 * l4;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t n = (uint32_t)(n0 + i < N ? n0 + i : N - 1);
            buf.c[i] = load_codes<NB>(at<uint8_t>(packed, n * (uint32_t)a.wpr * 4u + (uint32_t)kc * NB / 8));
        }
#pragma unroll
        for (int i = 0; i < 8 / SH; ++i) {
            const int nr = n0 + SH * i + (l16 & (SH - 1));
            const uint32_t g = (uint32_t)(nr < N ? nr : N - 1) * (uint32_t)a.gpl + ((uint32_t)kc >> a.gshift);
            buf.s[i] = *at<float>(scale, 4 * g);
            buf.z[i] = *at<float>(zero, 4 * g);
        }
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const int m = m0 + 16 * u + l16 < a.M ? m0 + 16 * u + l16 : (int)a.M - 1;
            buf.a[u] = load_run<AL>(A + (int64_t)m * lda, n0, N);
        }
    };
    float4v acc[MT][8];
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int t = 0; t < 8; ++t)
            acc[u][t] = float4v{0.f, 0.f, 0.f, 0.f};
    if (s0 + wave < s1)
        load(s0 + wave);
    for (int s = s0 + wave; s < s1; s += kGradWaves) {
        const GradBuf<NB, MT, SH> cur = buf;
        if (s + kGradWaves < s1)
            load(s + kGradWaves);
        double R[8];
        float Z[8];
        row_meta<SH>(cur.s, cur.z, R, Z);
        uint32_t v[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w[2] = {cur.c[i].x, cur.c[i].y};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int b0 = 2 * t * NB, b1 = b0 + NB;
                v[i][t] = out2<BF>(wq((float)((w[b0 / 32] >> (b0 % 32)) & MASK), Z[i], R[i]),
                                   wq((float)((w[b1 / 32] >> (b1 % 32)) & MASK), Z[i], R[i]));
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const uint32_t sel = t & 1 ? 0x07060302u : 0x05040100u;
            const uint4 B{perm(v[1][t / 2], v[0][t / 2], sel), perm(v[3][t / 2], v[2][t / 2], sel),
                          perm(v[5][t / 2], v[4][t / 2], sel), perm(v[7][t / 2], v[6][t / 2], sel)};
#pragma unroll
            for (int u = 0; u < MT; ++u)
                acc[u][t] = mfma<BF>(cur.a[u], B, acc[u][t]);
        }
    }
    // half of the waves hand their sums to the other half, until one has them all
#pragma unroll
    for (int w = kGradWaves / 2; w > 0; w /= 2) {
        __syncthreads();
        if (wave >= w && wave < 2 * w) {
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    red[wave - w][u * 8 + t][lane] = acc[u][t];
        }
        __syncthreads();
        if (wave < w) {
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    acc[u][t] += red[wave][u * 8 + t][lane];
        }
    }
    if (wave != 0 || kc_raw >= a.K)
        return;
    // acc[u][t][r] is C[16 u + 4 (l / 16) + r][kc + t]
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int m = m0 + 16 * u + 4 * l4 + r;
            if (m >= a.M)
                continue;
            if (a.part) {
                float4v *o = reinterpret_cast<float4v *>(a.part + ((int64_t)blockIdx.y * a.M + m) * a.K + kc);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    o[t] = float4v{acc[u][4 * t][r], acc[u][4 * t + 1][r], acc[u][4 * t + 2][r], acc[u][4 * t + 3][r]};
            } else {
                const float f = row_factor(a.rowf, m);
                *reinterpret_cast<uint4 *>(a.out + (int64_t)m * a.K + kc) =
                    uint4{out2<BF>(acc[u][0][r] * f, acc[u][1][r] * f), out2<BF>(acc[u][2][r] * f, acc[u][3][r] * f),
                          out2<BF>(acc[u][4][r] * f, acc[u][5][r] * f), out2<BF>(acc[u][6][r] * f, acc[u][7][r] * f)};
            }
        }
}

template <int NB, int MT, bool BF, bool AL>
hipError_t launch_sh(const SkinnyGradArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.K + 127) / 128), (unsigned)a.splits, (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
    switch (a.gshift) {
    case 3: hipLaunchKernelGGL((skinny_grad_kernel<NB, MT, BF, AL, 1>), grid, dim3(kGradWaves * 64), 0, s, a); break;
    case 4: hipLaunchKernelGGL((skinny_grad_kernel<NB, MT, BF, AL, 2>), grid, dim3(kGradWaves * 64), 0, s, a); break;
    case 5: hipLaunchKernelGGL((skinny_grad_kernel<NB, MT, BF, AL, 4>), grid, dim3(kGradWaves * 64), 0, s, a); break;
    default: hipLaunchKernelGGL((skinny_grad_kernel<NB, MT, BF, AL, 8>), grid, dim3(kGradWaves * 64), 0, s, a);
    }
    return hipGetLastError();
}

template <int NB, int MT, bool BF>
hipError_t launch_al(const SkinnyGradArgs &a, hipStream_t s)
{
    bool al = true;
    for (int i = 0; i < a.count; ++i)
        al = al && a.lda[i] % 8 == 0;
    return al ? launch_sh<NB, MT, BF, true>(a, s) : launch_sh<NB, MT, BF, false>(a, s);
}

template <int NB, bool BF>
hipError_t launch_mt(const SkinnyGradArgs &a, hipStream_t s)
{
    return a.M <= 16 ? launch_al<NB, 1, BF>(a, s) : launch_al<NB, 2, BF>(a, s);
}

}  // namespace

hipError_t launch_skinny_grad(int nbits, bool bf16, SkinnyGradArgs &a, hipStream_t s)
{
    a.steps = a.step0[a.count];
    switch (nbits) {
    case 1: return bf16 ? launch_mt<1, true>(a, s) : launch_mt<1, false>(a, s);
    case 2: return bf16 ? launch_mt<2, true>(a, s) : launch_mt<2, false>(a, s);
    case 4: return bf16 ? launch_mt<4, true>(a, s) : launch_mt<4, false>(a, s);
    case 8: return bf16 ? launch_mt<8, true>(a, s) : launch_mt<8, false>(a, s);
    default: return hipErrorInvalidValue;
    }
}

// About two workgroups of four waves per CU, each wave with a step at least; no part
// empty.  (Eight waves, or twice the workgroups, cost 5 and 3 % for 16 rows through 4096 x
// 11008 at 4 bits.)
int skinny_grad_splits(int64_t M, int64_t K, int64_t steps)
{
    const int64_t tiles = (K + 127) / 128 * (M <= 16 ? 1 : (M + 31) / 32);
    int64_t sp = (512 + tiles - 1) / tiles;
    const int64_t most = (steps + kGradWaves - 1) / kGradWaves;
    sp = sp < most ? sp : most;
    const int64_t per = (steps + sp - 1) / sp;
    return (int)((steps + per - 1) / per);
}

}  // namespace hqq
