// hqq_linear_dev.h -- device code shared by the kernels that multiply with W_hat
// straight from the packed codes (axis = 1): the exact dequantization, the 4-bit
// code tables, a lane's share of a K step, and the 16x16x32 MFMA.
#pragma once

#include "hqq_internal.h"

namespace hqq {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kLaneK = 64;                // consecutive k per lane per step
constexpr int kStepK = 4 * kLaneK;        // k per wave step
constexpr int kXldsMax = 64 * 1024;       // bytes of X staged in LDS, at most

__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel)
{
    return __builtin_amdgcn_perm(hi, lo, sel);
}

// an 8-k run of X (16-bit values, natural order) in operand order 0,2,4,6,1,3,5,7
__device__ __forceinline__ uint4 run_order(uint4 x)
{
    return uint4{perm(x.y, x.x, 0x05040100u), perm(x.w, x.z, 0x05040100u),
                 perm(x.y, x.x, 0x07060302u), perm(x.w, x.z, 0x07060302u)};
}

typedef float float2v __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));

// two fp32 -> packed fp16 pair, round-to-nearest-even (v_cvt_pk_f16_f32)
__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    const half2v h = __builtin_convertvector(float2v{lo, hi}, half2v);
    uint32_t u;
    __builtin_memcpy(&u, &h, 4);
    return u;
}

typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// two fp32 -> packed pair of the compute dtype (fp16, or BF: bf16), round to
// nearest even (v_cvt_pk_f16_f32 / v_cvt_pk_bf16_f32)
template <bool BF>
__device__ __forceinline__ uint32_t out2(float lo, float hi)
{
    if constexpr (BF) {
        const bf2v h = __builtin_convertvector(float2v{lo, hi}, bf2v);
        uint32_t u;
        __builtin_memcpy(&u, &h, 4);
        return u;
    } else {
        return f16x2(lo, hi);
    }
}

// one fp32 -> 16-bit value of the compute dtype, round to nearest even
template <bool BF>
__device__ __forceinline__ uint16_t out1(float v)
{
    uint16_t u;
    if constexpr (BF) {
        const __bf16 h = (__bf16)v;
        __builtin_memcpy(&u, &h, 2);
    } else {
        const _Float16 h = (_Float16)v;
        __builtin_memcpy(&u, &h, 2);
    }
    return u;
}

// the exact dequantized value of code c (fp32, before the rounding to the
// compute dtype)
__device__ __forceinline__ float wq(float c, float z, double R)
{
    return (float)((double)(c - z) * R);
}

// The 16 values (fp16, or BF: bf16) of a 4-bit group as byte tables: L[q]
// holds the low bytes of codes 4q .. 4q+3, H[q] the high bytes.
struct Tab4 {
    uint32_t L[4], H[4];
};

template <bool BF>
__device__ __forceinline__ Tab4 make_tab4(float s, float z)
{
    const double R = 1.0 / (double)s;
    uint32_t P[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        P[i] = out2<BF>(wq((float)(2 * i), z, R), wq((float)(2 * i + 1), z, R));
    Tab4 t;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        t.L[q] = perm(P[2 * q + 1], P[2 * q], 0x06040200u);
        t.H[q] = perm(P[2 * q + 1], P[2 * q], 0x07050301u);
    }
    return t;
}

// make_tab4 shared by two adjacent lanes that hold the same group: each lane
// evaluates 8 of the 16 values (the even lane codes 0-7, the odd lane codes
// 8-15) and takes the other 8 from its neighbour by a DPP quad permutation
// [1, 0, 3, 2].  The values are those of make_tab4, bit for bit.  Both lanes
// must be active.
template <bool BF>
__device__ __forceinline__ Tab4 make_tab4_pair(float s, float z, bool odd)
{
    const double R = 1.0 / (double)s;
    const float c0 = odd ? 8.0f : 0.0f;
    uint32_t P[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t mine = out2<BF>(wq(c0 + (float)(2 * j), z, R), wq(c0 + (float)(2 * j + 1), z, R));
        const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)mine, 0xB1, 0xF, 0xF, false);
        P[j] = odd ? other : mine;
        P[4 + j] = odd ? mine : other;
    }
    Tab4 t;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        t.L[q] = perm(P[2 * q + 1], P[2 * q], 0x06040200u);
        t.H[q] = perm(P[2 * q + 1], P[2 * q], 0x07050301u);
    }
    return t;
}

// 8 codes of a 4-bit word -> 8 16-bit values in operand order (0,2,4,6,1,3,5,7)
__device__ __forceinline__ uint4 lookup4(const Tab4 &t, uint32_t w)
{
    // byte q of se / so: low 3 bits of the even / odd code of byte q; the
    // masks are 0xff where bit 3 of that code is set (v_perm replicates the
    // sign bit of a byte for selector values 8..11)
    const uint32_t se = w & 0x07070707u, so = (w >> 4) & 0x07070707u;
    const uint32_t me = perm(w << 12, w << 4, 0x090B080Au);
    const uint32_t mo = perm(w << 8, w, 0x090B080Au);
    auto pick = [](uint32_t m, uint32_t a, uint32_t b) { return (m & a) | (~m & b); };
    const uint32_t lo_e = pick(me, perm(t.L[3], t.L[2], se), perm(t.L[1], t.L[0], se));
    const uint32_t hi_e = pick(me, perm(t.H[3], t.H[2], se), perm(t.H[1], t.H[0], se));
    const uint32_t lo_o = pick(mo, perm(t.L[3], t.L[2], so), perm(t.L[1], t.L[0], so));
    const uint32_t hi_o = pick(mo, perm(t.H[3], t.H[2], so), perm(t.H[1], t.H[0], so));
    return uint4{perm(hi_e, lo_e, 0x05010400u), perm(hi_e, lo_e, 0x07030602u),
                 perm(hi_o, lo_o, 0x05010400u), perm(hi_o, lo_o, 0x07030602u)};
}

// Groups whose (scale, zero) a lane needs per step: 1 (gs >= 64), 2 (gs 32,
// one per 32 k) or 8 (gs 8 or 16, one per 8-k run).
constexpr int groups_per_chunk(int gs) { return gs >= 64 ? 1 : gs == 32 ? 2 : 8; }

// One wave step's codes and meta for one lane (its 64-k chunk), and the X
// runs of its m tiles when X is read from global memory.
template <int NB, int GPC>
struct StepBuf {
    uint32_t w[2 * NB];
    float s[GPC], z[GPC];
};

template <int MT>
struct XRuns {
    uint4 x[MT][8];
};

// Where a lane's chunk starts (k0) and where its second 32 k start (kh): k0
// + 32, or k0 again where that is K or beyond (K % 64 == 32; those products
// are masked to zero).  A chunk past K is moved to the last 32 k (in bounds;
// masked to zero as well).  Offsets are 32-bit: the host keeps every array
// below 2^31 bytes, so each load is a uniform base plus a lane offset.
struct Chunk {
    uint32_t k0, kh;
};

template <bool KT>
__device__ __forceinline__ Chunk lane_chunk(uint32_t kbase, int grp, uint32_t K)
{
    uint32_t k0 = kbase + kLaneK * grp;
    if constexpr (KT)
        k0 = k0 < K ? k0 : K - 32;
    const uint32_t kh = KT ? (k0 + 32 < K ? k0 + 32 : k0) : k0 + 32;
    return Chunk{k0, kh};
}

template <typename T>
__device__ __forceinline__ const T *at(const void *base, uint32_t byte_off)
{
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(base) + byte_off);
}

template <int NB, int GPC>
__device__ __forceinline__ void load_step(StepBuf<NB, GPC> &b, const LinearArgs &a, Chunk c,
                                          uint32_t nw, uint32_t ng)
{
    // nw: first word of the lane's row, ng: its first group
    const uint32_t wa = 4 * (nw + c.k0 * NB / 32), wb = 4 * (nw + c.kh * NB / 32);
    if constexpr (NB == 1) {
        b.w[0] = *at<uint32_t>(a.packed, wa);
        b.w[1] = *at<uint32_t>(a.packed, wb);
    } else if constexpr (NB == 2) {
        const uint2 u = *at<uint2>(a.packed, wa);
        const uint2 v = *at<uint2>(a.packed, wb);
        b.w[0] = u.x; b.w[1] = u.y; b.w[2] = v.x; b.w[3] = v.y;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int q = 0; q < NB / 4; ++q) {
                const uint4 v = *at<uint4>(a.packed, (h ? wb : wa) + 16 * q);
                b.w[NB * h + 4 * q + 0] = v.x; b.w[NB * h + 4 * q + 1] = v.y;
                b.w[NB * h + 4 * q + 2] = v.z; b.w[NB * h + 4 * q + 3] = v.w;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < GPC; ++i) {
        const uint32_t kk = GPC == 1 ? c.k0 : GPC == 2 ? (i ? c.kh : c.k0) : (i < 4 ? c.k0 : c.kh) + 8 * (i & 3);
        const uint32_t g = 4 * (ng + (kk >> a.gshift));
        b.s[i] = *at<float>(a.scale, g);
        b.z[i] = *at<float>(a.zero, g);
    }
}

// xr: element index of the first X element of each of the lane's rows
template <int MT>
__device__ __forceinline__ void load_x(XRuns<MT> &b, const LinearArgs &a, Chunk c,
                                       const uint32_t (&xr)[MT])
{
#pragma unroll
    for (int u = 0; u < MT; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            b.x[u][j] = *at<uint4>(a.X, 2 * (xr[u] + c.k0) + 16 * j);
            b.x[u][4 + j] = *at<uint4>(a.X, 2 * (xr[u] + c.kh) + 16 * j);
        }
    }
}

// B operand j (8-k run j of the chunk) by direct quotients, operand order
template <int NB, int GPC, bool BF>
__device__ __forceinline__ uint4 dequant_run(const uint32_t *w, int j, const float *s,
                                             const float *z)
{
    constexpr uint32_t MASK = (1u << NB) - 1u;
    constexpr int ord[8] = {0, 2, 4, 6, 1, 3, 5, 7};
    const int gi = GPC == 1 ? 0 : GPC == 2 ? (j >> 2) : j;
    const double R = 1.0 / (double)s[gi];
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int bit = (8 * j + ord[i]) * NB;
        v[i] = wq((float)((w[bit / 32] >> (bit % 32)) & MASK), z[gi], R);
    }
    return uint4{out2<BF>(v[0], v[1]), out2<BF>(v[2], v[3]), out2<BF>(v[4], v[5]), out2<BF>(v[6], v[7])};
}

__device__ __forceinline__ uint4 and4(uint4 v, uint32_t m)
{
    return uint4{v.x & m, v.y & m, v.z & m, v.w & m};
}

// one 16x16x32 MFMA of the compute dtype (fp16, or BF: bf16), fp32 accumulation
template <bool BF>
__device__ __forceinline__ float4v mfma(uint4 A, uint4 B, float4v c)
{
    if constexpr (BF) {
        bf16x8 a, b;
        __builtin_memcpy(&a, &A, 16);
        __builtin_memcpy(&b, &B, 16);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    } else {
        half8 a, b;
        __builtin_memcpy(&a, &A, 16);
        __builtin_memcpy(&b, &B, 16);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
}

// X staged in LDS: row m of the workgroup's X rows at xs + m * xrow (uint4
// units), runs in operand order; the row pitch is K / 8 + 1 runs so that the
// 16 rows of an operand fall in different banks.
template <bool KT, int NB, int MT, int GPC, bool XL, bool BF>
__device__ __forceinline__ void compute_step(const StepBuf<NB, GPC> &b, const XRuns<XL ? 1 : MT> &xg,
                                             uint32_t km0, uint32_t km1, const uint4 *xs,
                                             const uint32_t (&xm)[MT], Chunk c,
                                             float4v (&acc)[MT])
{
    uint4 B[8];
    if constexpr (NB == 4 && GPC == 1) {
        const Tab4 t = make_tab4<BF>(b.s[0], b.z[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            B[j] = lookup4(t, b.w[j]);
    } else if constexpr (NB == 4 && GPC == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const Tab4 t = make_tab4<BF>(b.s[h], b.z[h]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                B[4 * h + j] = lookup4(t, b.w[4 * h + j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            B[j] = dequant_run<NB, GPC, BF>(b.w, j, b.s, b.z);
    }
    // K % 256 != 0: a lane whose chunk (or its second half) lies past K adds
    // zeros; the operands are cleared with integer masks (a select would
    // become a branch that waits for every load in flight)
    if constexpr (KT) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            B[j] = and4(B[j], j < 4 ? km0 : km1);
    }
    const uint32_t r0 = c.k0 >> 3, r1 = c.kh >> 3;
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint4 A;
            if constexpr (XL)
                A = xs[xm[u] + (j < 4 ? r0 + j : r1 + j - 4)];
            else
                A = run_order(xg.x[u][j]);
            if constexpr (KT)
                A = and4(A, j < 4 ? km0 : km1);
            acc[u] = mfma<BF>(A, B[j], acc[u]);
        }
}

}  // namespace
}  // namespace hqq
