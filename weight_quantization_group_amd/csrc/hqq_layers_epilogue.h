// hqq_layers_epilogue.h -- small device functions of the layers: the reciprocal of
// the dequantization, the activations, loads and stores of runs of 16-bit values.
#pragma once

#include "hqq_layers_internal.h"
#include "hqq_linear_dev.h"

namespace hqq {
namespace {

// 1 / s in fp64 by two Newton steps from v_rcp_f64 (2^-24 or better): within 2^-51.5
// relative, which the exactness of wq needs no more than (a quotient is nowhere nearer
// than 2^-49 to where fp32 rounds the other way); a third of the division's steps.
__device__ __forceinline__ double reciprocal(float s)
{
    const double d = (double)s;
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

// x of lane I of the caller's SH neighbours (lanes SH i .. SH i + SH - 1)
template <int SH, int I>
__device__ __forceinline__ uint32_t from_neighbour(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, (0x1f & ~(SH - 1)) | I << 5);
}

// Z[i] and R[i] = 1 / s of row i of 8: SH neighbouring lanes work on the same rows and in
// one group of each, and lane j of them holds the scales s[k] and zeros z[k] of rows SH k + j.
template <int SH, int I = 0>
__device__ __forceinline__ void share_meta(const float (&z)[8 / SH], const double (&r)[8 / SH], double (&R)[8], float (&Z)[8])
{
    if constexpr (I < 8) {
        if constexpr (SH == 1) {
            R[I] = r[I];
            Z[I] = z[I];
        } else {
            uint32_t w[2], f;
            __builtin_memcpy(w, &r[I / SH], 8);
            __builtin_memcpy(&f, &z[I / SH], 4);
            w[0] = from_neighbour<SH, I % SH>(w[0]);
            w[1] = from_neighbour<SH, I % SH>(w[1]);
            f = from_neighbour<SH, I % SH>(f);
            __builtin_memcpy(&R[I], w, 8);
            __builtin_memcpy(&Z[I], &f, 4);
        }
        share_meta<SH, I + 1>(z, r, R, Z);
    }
}

// the same from the scales
template <int SH>
__device__ __forceinline__ void row_meta(const float (&s)[8 / SH], const float (&z)[8 / SH], double (&R)[8], float (&Z)[8])
{
    double r[8 / SH];
#pragma unroll
    for (int i = 0; i < 8 / SH; ++i)
        r[i] = reciprocal(s[i]);
    share_meta<SH>(z, r, R, Z);
}

// LDS of one wave: written by some lanes and read by others
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

constexpr float kLog2e = 1.44269504088896340736f;

// 2^x and 1 / x to about an ulp of fp32 (v_exp_f32, v_rcp_f32): the results are
// rounded to 16 bits, or summed over many terms
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// act(g) and, for the backward pass, act'(g).  Each activation is g * p with p in
// (0, 1) formed without cancellation (erfc, and (1 + tanh y) / 2 = 1 / (1 + exp(-2 y))),
// so that its far negative tail keeps its relative precision.
template <int ACT>
__device__ __forceinline__ float act_value(float g, float &d)
{
    if constexpr (ACT == HQQ_ACT_GELU) {
        const float p = 0.5f * erfcf(g * -0.70710678118654752440f);
        d = p + g * 0.39894228040143267794f * exp2_fast(-0.5f * kLog2e * g * g);
        return g * p;
    } else {
    // exponent y2 of p = 1 / (1 + exp(-y2)), and its derivative
    float y2 = g, dy2 = 1.0f;
    if constexpr (ACT == HQQ_ACT_GELU_TANH) {
        const float a = 1.59576912160573071176f, b = 0.044715f;   // 2 sqrt(2 / pi)
        y2 = a * (g + b * g * g * g);
        dy2 = a * (1.0f + 3.0f * b * g * g);
    }
    const float e = exp2_fast(-kLog2e * y2);
    const float p = rcp_fast(1.0f + e);
    // p (1 - p) = p^2 e; 0 where e overflows (p is 0), and where e is 0 (dy2 may overflow)
    d = p + (e > 0.0f && e < INFINITY ? g * dy2 * (p * (p * e)) : 0.0f);
    return g * p;
    }
}

// A softmax block of logits is (max, sum of exp(logit - stats_ref(max))).  The reference is
// the maximum where that is finite and 0 elsewhere, so that no inf - inf is formed: a block of
// -inf has the sum 0, one with a +inf the sum +inf, and a NaN among the logits stays in the sum.
__device__ __forceinline__ float stats_ref(float mx) { return fabsf(mx) < INFINITY ? mx : 0.0f; }

__device__ __forceinline__ float row_factor(const RowFactor &r, int64_t m)
{
    if (r.f)
        return r.f[m];
    if (!r.dloss)
        return 1.0f;
    const int64_t t = r.targets[m];
    return t >= 0 && t < r.N ? r.dloss[m] * r.mul : 0.0f;
}

__device__ __forceinline__ float from16(uint16_t b, bool bf)
{
    if (bf)
        return __uint_as_float((uint32_t)b << 16);
    _Float16 h;
    __builtin_memcpy(&h, &b, 2);
    return (float)h;
}

// The largest |W_hat| of the weights, from its parts; all lanes of the wave call.  (Rounding
// keeps the order, so the largest quotient's fp16 value is the largest fp16 value.)
__device__ __forceinline__ float weight_bound(const GradBound &b)
{
    const float4 p = reinterpret_cast<const float4 *>(b.weight)[threadIdx.x & 63];
    float mx = fmaxf(fmaxf(p.x, p.y), fmaxf(p.z, p.w));
#pragma unroll
    for (int o = 1; o < 64; o *= 2)
        mx = fmaxf(mx, __shfl_xor(mx, o));
    return (float)(_Float16)mx;
}
static_assert(kBoundParts == 4 * 64, "four parts per lane");

// The power of two by which a row's dG and dU are multiplied in fp16, and its reciprocal.  With
// b = max |dY| * sum |X| * max |W_hat|, |U| <= sum |X| max |W_hat| and |act(G)| <= |G|, so that
// |dU| <= b and |dG| <= 1.13 b (max |act'|): b is brought to [2^13, 2^14), where nothing
// overflows.  Usual sums of K products stay within 2^8 or so of their bound, which leaves them
// some 20 binades of full precision.  1 where the bound is 0 (so are dG and dU) or not finite
// (b is at least 2^-72 else, and at most 2^65: the exponents below are in range).
__device__ __forceinline__ float grad_scale(float row, float weight, float &inv)
{
    const float b = row * weight;
    const uint32_t e = __float_as_uint(b) >> 23;
    const bool scaled = b > 0.0f && b < INFINITY;
    inv = scaled ? __uint_as_float((e - 13) << 23) : 1.0f;
    return scaled ? __uint_as_float((267 - e) << 23) : 1.0f;
}

// four consecutive 16-bit values at p (8-byte aligned)
template <bool BF>
__device__ __forceinline__ void load4(const char *p, float (&v)[4])
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    v[0] = from16((uint16_t)u.x, BF);
    v[1] = from16((uint16_t)(u.x >> 16), BF);
    v[2] = from16((uint16_t)u.y, BF);
    v[3] = from16((uint16_t)(u.y >> 16), BF);
}

}  // namespace
}  // namespace hqq
