// hqq_cache_attention.h -- attention of one new token over the quantized cache:
// one workgroup takes a run of tokens of one key-value head for 16 query heads.
// Included by hqq_cache_attention_b{2,4,8}.hip, one width each.
//
// Mathematics.  With q scaled by a power of two per row, codes c, and r = 1 / scale:
//   s_t = sum_g r_tg (sum_{d in g} q_d c_td  -  z_tg sum_{d in g} q_d)
//   o_d = sum_t (p_t r_tg) c_td  -  sum_t (p_t r_tg) z_tg        for d in group g
// so the codes go to the matrix units as they are, and scales and zeros meet the
// sums, not the values.  An fp16 subnormal whose bits are the code c is c * 2^-24
// exactly, so a shift and a mask turn a word into operands; a field further up in a half
// word comes out times its place, which is taken back from q (first product) or from the
// output row (second).
//
// Operand layouts (16x16x32): S = K Q^T has a token per row and a head per column, so
// a lane holds 4 tokens of one head; these are the contraction slots of the second
// product O^T = V^T P^T, for which a lane needs exactly its own 8 tokens of the 32:
// the weights never leave their lane.  For V a lane pairs the words of two
// tokens, whose equal fields are neighbours in the contraction.  A group's dims are
// dealt to the rows of whole products (lane m of 16 has gs / 16 consecutive dims),
// as one product has one p_t r_tg per token.
#pragma once

#include "hqq_cache_plan.h"

namespace hqq {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));

__device__ __forceinline__ half8 operand(const uint32_t (&r)[4])
{
    half8 h;
    __builtin_memcpy(&h, r, 16);
    return h;
}

// Field f of both half words of x as fp16 subnormals, times field_factor.  The matrix
// units align the products of a sum by their operands' exponents, and a subnormal counts with
// the least one, so a low field loses bits of the sum.  PRECISE (keys): the fields are brought
// to the upper bits of the 10 that a subnormal has (error of lse at 2 bits 1.5e-6 without);
// values, whose weights have 11 bits, leave them where that saves a shift.
template <int NB, bool PRECISE>
__device__ __forceinline__ uint32_t field(uint32_t x, int f)
{
    if constexpr (NB == 8) {
        return (f ? x >> 8 : x) & 0x00ff00ffu;
    } else if constexpr (NB == 4) {
        if constexpr (PRECISE)
            return (f == 0 ? x << 4 : x >> (4 * f - 4)) & 0x00f000f0u;
        else
            return (f < 2 ? x : x >> 8) & (f % 2 ? 0x00f000f0u : 0x000f000fu);
    } else {
        if constexpr (PRECISE) {
            const int left = 6 - 4 * (f / 2);
            return (left > 0 ? x << left : x >> -left) & (f % 2 ? 0x03000300u : 0x00c000c0u);
        } else {
            return f < 5 ? x & (0x00030003u << (2 * f)) : (x >> 10) & (0x00030003u << (2 * (f - 5)));
        }
    }
}

template <int NB, bool PRECISE>
constexpr float field_factor(int f)
{
    return NB == 8   ? 1.0f
           : NB == 4 ? (PRECISE || f % 2 ? 16.0f : 1.0f)
           : PRECISE ? (f % 2 ? 256.0f : 64.0f)
                     : (float)(1 << (2 * (f < 5 ? f : f - 5)));
}

// How a lane's gs / 4 codes of a token's group stand in the operands of the first
// product: operand u, register r holds codes lo and hi
template <int NB, int GS>
struct KeyOrder {
    static constexpr int kUnits = GS / 32;            // products per group
    static constexpr int kBytes = GS * NB / 32;       // a lane's bytes of a group
    static constexpr bool kHalf = kBytes == 2;        // 8 codes of 2 bits: 4 fields of either half word
    static constexpr int lo(int u, int r)
    {
        return NB == 8   ? 8 * u + 4 * (r / 2) + r % 2
               : NB == 4 ? 8 * u + r
               : kHalf   ? r
                         : 16 * (u / 2) + 4 * (u % 2) + r;
    }
    static constexpr int hi(int u, int r) { return lo(u, r) + (NB == 8 ? 2 : NB == 4 || kHalf ? 4 : 8); }
    static constexpr int field_of(int u, int r) { return NB == 8 ? r % 2 : NB == 4 || kHalf ? r : 4 * (u % 2) + r; }
    static constexpr int word_of(int u, int r) { return NB == 8 ? 2 * u + r / 2 : NB == 4 ? u : u / 2; }
};

// n bytes (2, 4 or whole words) to words
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[(N + 3) / 4], const char *p)
{
    if constexpr (N == 1) {
        w[0] = *(const uint8_t *)p;
    } else if constexpr (N == 2) {
        w[0] = *(const uint16_t *)p;
    } else if constexpr (N == 4) {
        w[0] = *(const uint32_t *)p;
    } else if constexpr (N == 8) {
        const uint2 v = *(const uint2 *)p;
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            const uint4 v = ((const uint4 *)p)[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    }
}

__device__ __forceinline__ float widen16(uint16_t v, bool bf16)
{
    _Float16 h;
    __builtin_memcpy(&h, &v, 2);
    return bf16 ? __uint_as_float((uint32_t)v << 16) : (float)h;
}

// the values of the other half of the wave, and of the other row of 16 in the same half, beside
// this lane's
struct Two {
    float a, b;
};

__device__ __forceinline__ Two halves(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return Two{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

__device__ __forceinline__ Two rows(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return Two{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

// sum, or maximum, over the 4 lanes that share a column
__device__ __forceinline__ float column_sum(float v)
{
    const Two h = halves(v);
    const Two r = rows(h.a + h.b);
    return r.a + r.b;
}

__device__ __forceinline__ float column_max(float v)
{
    const Two h = halves(v);
    const Two r = rows(fmaxf(h.a, h.b));
    return fmaxf(r.a, r.b);
}

__device__ __forceinline__ float power_of_two(int e)      // -126 <= e <= 127
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// a lane's LDS writes are there for the wave's other lanes
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int NB, int GS, int NG>
struct CacheAttention {
    static constexpr int D = GS * NG;
    static constexpr int kRowBytes = D * NB / 8;
    typedef KeyOrder<NB, GS> Keys;
    static constexpr int kValueBits = GS * NB / 16;             // a lane's bits of a token's group
    static constexpr int kValueBytes = kValueBits < 8 ? 1 : kValueBits / 8;
    static constexpr int kValueWords = (kValueBytes + 3) / 4;
    static constexpr int kCodes = GS / 16;                      // ... and codes: products per group
    static constexpr int kMetas = NG <= 2 ? 1 : 2;              // a tile's groups over the lanes
    static constexpr int kPerChunk = kValueBits < 16 ? kCodes : 16 / NB;      // codes of a half word
    static constexpr int kChunks = kValueBits < 16 ? 1 : kValueBits / 16;
    static constexpr int kPitch = D + 4;

    struct alignas(16) Shared {
        union {
            struct {
                uint4 q[NG][Keys::kUnits][64];                  // operands of the first product
                float meta[kCacheWaves][3][NG][kCacheTile];     // r of k, scaled r of v, z of v
            };
            float sums[kCacheWaves][16][kPitch];
        };
        float2 ml[kCacheWaves][16];
    };

    // The tile's two subtiles: each 16 consecutive rows of a page
    struct Where {
        int at;
        int64_t row[2];
        bool there[2];
        bool whole;      // all its tokens count
        bool joined;     // its subtiles are of one page
    };
    // ... and what is loaded of them
    struct Meta {
        float ks[kMetas], kz[kMetas], vs[kMetas], vz[kMetas];
    };
    typedef uint32_t KeyWords[2][NG][(Keys::kBytes + 3) / 4];
    typedef uint32_t ValueWords[8][NG][kValueWords];

    const CacheAttentionArgs &a;
    const int lane, wave, col, quad, head;
    // the segment: tokens [begin, end) of sequence b, of which those from `first` on count
    int b, begin, end, first;

    __device__ __forceinline__ CacheAttention(const CacheAttentionArgs &args)
        : a(args), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), col(lane & 15),
          quad(lane >> 4),
          head(blockIdx.x % args.heads)
    {
    }

    // The pages of 32 of this wave's tiles from tile `at` on: subtile i's in lane i
    __device__ __forceinline__ int pages_from(int at) const
    {
        const int token = at + (lane >> 1) * kCacheStep + (lane & 1) * 16;
        return token < end ? a.table[(int64_t)b * a.table_width + (token >> a.page_shift)] : -1;
    }

    __device__ __forceinline__ Where where(int at, int pages, int tile) const
    {
        Where w;
        w.at = at;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int page = __builtin_amdgcn_readlane(pages, 2 * (tile & 31) + t);
            w.there[t] = page >= 0 && page < a.pages;
            w.row[t] = (((int64_t)(w.there[t] ? page : 0) * a.heads + head) << a.page_shift) +
                       ((at + 16 * t) & a.page_mask);
        }
        w.whole = w.there[0] && w.there[1] && at >= first && at + kCacheTile <= end;
        w.joined = a.page_shift > 4;
        return w;
    }

    __device__ __forceinline__ bool counts(const Where &w, int t, int place) const
    {
        const int token = w.at + 16 * t + place;
        return token >= first && token < end && w.there[t];
    }

    __device__ __forceinline__ void load_keys(const Where &w, KeyWords &kw) const
    {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int g = 0; g < NG; ++g)
                load_words<Keys::kBytes>(kw[t][g], (const char *)a.packed[0] + w.row[t] * kRowBytes + col * kRowBytes +
                                                       g * (GS * NB / 8) + quad * Keys::kBytes);
    }

    __device__ __forceinline__ void load_values(const Where &w, ValueWords &vw) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int g = 0; g < NG; ++g)
                load_words<kValueBytes>(vw[j][g], (const char *)a.packed[1] + w.row[j / 4] * kRowBytes +
                                                      (4 * quad + j % 4) * kRowBytes + g * (GS * NB / 8) +
                                                      (col * kValueBits) / 8);
    }

    // Scales and zeros lie over the lanes as token col and, along the quads, group (and
    // subtile, where the groups leave room)
    static __device__ __forceinline__ int meta_tile(int i, int quad) { return NG <= 2 ? quad / NG : i; }
    static __device__ __forceinline__ int meta_group(int quad) { return NG <= 2 ? quad % NG : quad < NG ? quad : 0; }
    static __device__ __forceinline__ bool meta_there(int i, int quad) { return NG <= 2 ? quad / NG < 2 : quad < NG; }

    __device__ __forceinline__ void load_meta(const Where &w, Meta &m) const
    {
#pragma unroll
        for (int i = 0; i < kMetas; ++i) {
            const int t = meta_tile(i, quad);
            // tokens that do not count: 1 / scale and zero of 0, whatever the page holds there
            m.ks[i] = m.vs[i] = INFINITY;
            m.kz[i] = m.vz[i] = 0.0f;
            const bool in = w.whole || (t ? counts(w, 1, col) : counts(w, 0, col));
            if (meta_there(i, quad) && in) {
                if (w.joined) {          // the tile's rows follow each other: one base for the wave
                    const int64_t base = w.row[0] * NG;
                    const uint32_t from = (16 * t + col) * NG + meta_group(quad);
                    m.ks[i] = (a.scale[0] + base)[from], m.kz[i] = (a.zero[0] + base)[from];
                    m.vs[i] = (a.scale[1] + base)[from], m.vz[i] = (a.zero[1] + base)[from];
                } else {
                    const int64_t from = ((t ? w.row[1] : w.row[0]) + col) * NG + meta_group(quad);
                    m.ks[i] = a.scale[0][from], m.kz[i] = a.zero[0][from];
                    m.vs[i] = a.scale[1][from], m.vz[i] = a.zero[1][from];
                }
            }
        }
    }

    // One segment, from q to the output or the workspace's slot
    __device__ __forceinline__ void segment(Shared &sh, int slot, bool whole_sequence)
    {
        const int row_tile = blockIdx.x / a.heads;
        const int in_group = row_tile * 16 + col;               // this column's q head within the group
        const bool real = in_group < a.G;
        const int q_head = head * a.G + (real ? in_group : 0);

        // ---- the first tile's loads
        const int at0 = begin + wave * kCacheTile;
        const int tiles = at0 < end ? (end - at0 + kCacheStep - 1) / kCacheStep : 0;
        int pages = pages_from(at0);
        KeyWords kw;
        ValueWords vw;
        Meta next_meta;
        Where next = where(at0, pages, 0);
        if (tiles > 0) {
            load_meta(next, next_meta);
            load_keys(next, kw);
            load_values(next, vw);
        }

        // ---- q: operands of the first product (in LDS: 16 to 32 registers; every wave writes the
        // same), and each group's sum
        float q_sum[NG];
        float score_scale;                                      // scores to exponents of 2
        {
            const uint16_t *src = a.Q + b * a.q_batch_stride + q_head * a.q_head_stride + quad * (GS / 4);
            float q[NG][GS / 4];
            float top = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < GS / 4; i += 8) {
                    const uint4 raw = *reinterpret_cast<const uint4 *>(src + g * GS + i);
                    uint16_t h[8];
                    __builtin_memcpy(h, &raw, 16);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        q[g][i + j] = widen16(h[j], a.bf16);
                        top = fmaxf(top, fabsf(q[g][i + j]));
                    }
                }
            top = column_max(top);
            // the largest to [2^14, 2^15): fp16 then holds what is within 2^-20 of it or so whole
            // (the fields' factors take up to 8 bits), and the rest to 2^-31 of it
            int e = top > 0.0f && top < INFINITY ? 14 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
            e = e > 100 ? 100 : e;
            const float f = power_of_two(e);
            score_scale = a.scale_log2 * 0x1p12f * power_of_two(-e);      // 2^12 of the 2^24, see kr
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float sum = 0.0f;
#pragma unroll
                for (int u = 0; u < Keys::kUnits; ++u) {
                    uint32_t q16[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float factor = field_factor<NB, true>(Keys::field_of(u, r));
                        const float inv = f / factor;
                        half2v h;
                        h[0] = (_Float16)(q[g][Keys::lo(u, r)] * inv);
                        h[1] = (_Float16)(q[g][Keys::hi(u, r)] * inv);
                        __builtin_memcpy(&q16[r], &h, 4);
                        sum += ((float)h[0] + (float)h[1]) * (factor * 0x1p-24f);
                    }
                    sh.q[g][u][lane] = uint4{q16[0], q16[1], q16[2], q16[3]};
                }
                q_sum[g] = column_sum(sum);
            }
        }
        // the zeros' part of the scores, -sum_g (r z)_tg q_sum_g, is a product of depth 4 in fp32,
        // with a row's groups (NG <= 2: of both subtiles) along its depth
        float q_zero[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int g = NG <= 2 ? quad - t * NG : quad;
            q_zero[t] = 0.0f;
#pragma unroll
            for (int i = 0; i < NG; ++i)
                q_zero[t] = g == i ? -q_sum[i] : q_zero[t];
        }

        // ---- state: per column, but sums of weights and zeros only over this lane's tokens
        float4v o[NG][kCodes];
        float z_sum[NG], v_unit[NG];
        float m2 = -INFINITY, total = 0.0f;                     // maximum (exponent of 2), sum of weights
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            z_sum[g] = 0.0f;
            v_unit[g] = 0x1p120f;
#pragma unroll
            for (int i = 0; i < kCodes; ++i)
                o[g][i] = float4v{0.f, 0.f, 0.f, 0.f};
        }
        float lane_unit = v_unit[0];                            // of the group whose scales this lane loads
        float (*meta)[NG][kCacheTile] = sh.meta[wave];

        for (int tile = 0; tile < tiles; ++tile) {
            const Where now = next;
            const bool more = tile + 1 < tiles;

            // ---- scales: reciprocals (to 1 ulp), to the layout of the scores through LDS
            float rz[kMetas];                                   // (r z) of k
            float vr[kMetas];
            float raise = 0.0f;
#pragma unroll
            for (int i = 0; i < kMetas; ++i) {
                const float kr = __builtin_amdgcn_rcpf(next_meta.ks[i]) * 0x1p12f;  // the codes' 2^-24 taken back, half here
                vr[i] = __builtin_amdgcn_rcpf(next_meta.vs[i]);
                rz[i] = kr * next_meta.kz[i];
                if (meta_there(i, quad)) {
                    float *to = &meta[0][meta_group(quad)][16 * meta_tile(i, quad) + col];
                    to[0] = kr;
                    to[2 * NG * kCacheTile] = next_meta.vz[i];
                }
                raise = fmaxf(raise, vr[i]);
            }
            // a group's r of v beyond the unit that its weights are held in?
            if (__any(!(raise * lane_unit <= 0x1p15f))) {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float most = 0.0f;
#pragma unroll
                    for (int i = 0; i < kMetas; ++i)
                        most = fmaxf(most, meta_there(i, quad) && meta_group(quad) == g ? vr[i] : 0.0f);
#pragma unroll
                    for (int off = 1; off < 64; off *= 2)
                        most = fmaxf(most, __shfl_xor(most, off));
                    // most * unit in [2^14, 2^15)
                    const int ue = 14 - ((int)(__float_as_uint(most) >> 23) - 127);
                    const float unit = power_of_two(ue < -120 ? -120 : ue > 120 ? 120 : ue);
                    if (unit < v_unit[g]) {
                        const float f = unit / v_unit[g];
                        v_unit[g] = unit;
                        z_sum[g] *= f;
#pragma unroll
                        for (int i = 0; i < kCodes; ++i)
                            o[g][i] *= f;
                    }
                }
                lane_unit = pick(v_unit, meta_group(quad));
            }
#pragma unroll
            for (int i = 0; i < kMetas; ++i)
                if (meta_there(i, quad))
                    meta[1][meta_group(quad)][16 * meta_tile(i, quad) + col] = vr[i] * lane_unit;
            wave_lds_fence();

            // ---- scores
            float4v s[2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
                s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(rz[NG <= 2 ? 0 : t], q_zero[t], float4v{0.f, 0.f, 0.f, 0.f}, 0,
                                                            0, 0);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float4v acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int u = 0; u < Keys::kUnits; ++u) {
                    const uint4 q4 = sh.q[g][u][lane];
                    const uint32_t q16[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        uint32_t regs[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            uint32_t x = kw[t][g][Keys::word_of(u, r)];
                            if constexpr (Keys::kHalf)
                                x = (x & 0xffu) | (x >> 8) << 16;
                            regs[r] = field<NB, true>(x, Keys::field_of(u, r));
                        }
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(regs), operand(q16), acc[t], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float4v r4 = *reinterpret_cast<const float4v *>(&meta[0][g][16 * t + 4 * quad]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        s[t][r] = fmaf(acc[t][r], r4[r], s[t][r]);
                }
            }
            // the keys' registers are free: the next tile's go there while the weights are formed
            if (more) {
                if ((tile & 31) == 31)
                    pages = pages_from(now.at + kCacheStep);
                next = where(now.at + kCacheStep, pages, tile + 1);
                load_meta(next, next_meta);
                load_keys(next, kw);
            }
            if (!now.whole) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (!counts(now, t, 4 * quad + r))
                            s[t][r] = -INFINITY;
            }

            // ---- weights
            float top = s[0][0];
#pragma unroll
            for (int j = 1; j < 8; ++j)
                top = fmaxf(top, s[j / 4][j % 4]);
            const float m_new = fmaxf(m2, column_max(top) * score_scale);
            const float ref = m_new == -INFINITY ? 0.0f : m_new;
            const float alpha = __builtin_amdgcn_exp2f(m2 - ref);
            m2 = m_new;
            if (__any(alpha != 1.0f)) {
                total *= alpha;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    z_sum[g] *= alpha;
#pragma unroll
                    for (int i = 0; i < kCodes; ++i)
                        o[g][i] *= alpha;
                }
            }
            float p[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    p[t][r] = __builtin_amdgcn_exp2f(fmaf(s[t][r], score_scale, -ref));
                    total += p[t][r];
                }

            // ---- the second product
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t w16[4];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float4v r4 = *reinterpret_cast<const float4v *>(&meta[1][g][16 * t + 4 * quad]);
                    const float4v z4 = *reinterpret_cast<const float4v *>(&meta[2][g][16 * t + 4 * quad]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const half2v h = __builtin_convertvector(
                            float2v{p[t][2 * k] * r4[2 * k], p[t][2 * k + 1] * r4[2 * k + 1]}, half2v);
                        // the zeros go with the rounded weights, as the codes do
                        z_sum[g] = fmaf((float)h[0], z4[2 * k], z_sum[g]);
                        z_sum[g] = fmaf((float)h[1], z4[2 * k + 1], z_sum[g]);
                        __builtin_memcpy(&w16[2 * t + k], &h, 4);
                    }
                }
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    uint32_t x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t lo = vw[2 * k][g][c / 2], hi = vw[2 * k + 1][g][c / 2];
                        if constexpr (kValueBits < 32)
                            x[k] = lo | hi << 16;
                        else
                            x[k] = __builtin_amdgcn_perm(hi, lo, c % 2 ? 0x07060302u : 0x05040100u);
                        if constexpr (kValueBits == 4)
                            x[k] >>= 4 * (col & 1);
                    }
#pragma unroll
                    for (int f = 0; f < kPerChunk; ++f) {
                        uint32_t regs[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            regs[k] = field<NB, false>(x[k], f);
                        float4v &acc = o[g][c * kPerChunk + f];
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(regs), operand(w16), acc, 0, 0, 0);
                    }
                }
            }
            if (more)
                load_values(next, vw);
            wave_lds_fence();       // the next tile's scales go where these were
        }

        // ---- the four waves' sums joined
        total = column_sum(total);
#pragma unroll
        for (int g = 0; g < NG; ++g)
            z_sum[g] = column_sum(z_sum[g]);
        if (quad == 0)
            sh.ml[wave][col] = float2{m2, total};
        __syncthreads();            // also: no wave reads scales any more, whose place the sums take
        float m_all = -INFINITY, total_all = 0.0f;
#pragma unroll
        for (int w = 0; w < kCacheWaves; ++w)
            m_all = fmaxf(m_all, sh.ml[w][col].x);
        const float ref = m_all == -INFINITY ? 0.0f : m_all;
#pragma unroll
        for (int w = 0; w < kCacheWaves; ++w)
            total_all += sh.ml[w][col].y * __builtin_amdgcn_exp2f(sh.ml[w][col].x - ref);
        const float own = __builtin_amdgcn_exp2f(m2 - ref);
        if (real) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float back = own / v_unit[g];
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < kCodes; ++i) {
                        const float unit = 0x1p24f / field_factor<NB, false>(i % kPerChunk);
                        sh.sums[wave][col][g * GS + (4 * quad + r) * kCodes + i] =
                            fmaf(o[g][i][r], unit, -z_sum[g]) * back;
                    }
            }
        }
        __syncthreads();
        // 16 threads a head; each takes D / 16 dims, 4 at a time
        const int h = threadIdx.x >> 4, part = threadIdx.x & 15;
        const int g_head = row_tile * 16 + h;
        // m_all and total_all are this lane's column's; its row's are another lane's
        const float m_row = __shfl(m_all, h), total_row = __shfl(total_all, h);
        if (g_head < a.G) {
            const int64_t out_head = head * a.G + g_head;
            const int64_t out_row = (int64_t)b * a.q_heads + out_head;
            const int64_t part_row = (int64_t)slot * a.q_heads + out_head;
            const float inv = cache_inverse(total_row);
#pragma unroll
            for (int d = part * 4; d < D; d += 64) {
                float4v v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < kCacheWaves; ++w)
                    v += *reinterpret_cast<const float4v *>(&sh.sums[w][h][d]);
                if (whole_sequence)
                    *reinterpret_cast<uint2 *>(a.out + out_row * D + d) = cache_round4(v * inv, a.bf16);
                else
                    *reinterpret_cast<float4v *>(a.part + part_row * D + d) = v;
            }
            if (part == 0) {
                if (!whole_sequence)
                    a.part_ml[part_row] = float2{m_row, total_row};
                else if (a.lse)
                    a.lse[out_row] = cache_lse(m_row, total_row);
            }
        }
        __syncthreads();            // the next segment's scales go where the sums were
    }

    static __device__ __forceinline__ float pick(const float (&v)[NG], int g)
    {
        float r = v[0];
#pragma unroll
        for (int i = 1; i < NG; ++i)
            r = g == i ? v[i] : r;
        return r;
    }

    __device__ __forceinline__ void run(Shared &sh)
    {
        const int worker = blockIdx.y;
        int at = 0, start = 0, stop;
        bool cross = false;
        CacheSpan s;
        int slot = 0;
        if (a.workers == 0) {        // a sequence each
            b = worker;
            s = cache_span(a, b);
            stop = s.steps;
        } else {
            const CachePlan plan(a, lane);
            const int64_t from = (int64_t)worker * plan.run;
            if (from > 1 << 30)          // behind the last step
                return;
            at = (int)from;
            stop = at + plan.run;
            cross = plan.cross;
            b = plan.find(a, at, lane, start, s);
            slot = plan.slot(worker, b);
        }
        while (b < a.batch) {
            const int next = start + s.steps, upto = stop < next ? stop : next;
            first = s.first;
            begin = s.base + (at - start) * kCacheStep;
            end = upto < next ? s.base + (upto - start) * kCacheStep : s.length;
            segment(sh, slot, at == start && upto == next);
            if (!cross || upto == stop)
                return;
            at = start = next;
            ++slot;
            if (++b < a.batch)
                s = cache_span(a, b);
        }
    }
};

template <int NB, int GS, int NG>
__global__ __launch_bounds__(64 * kCacheWaves, cache_resident(GS * NG, GS)) void cache_attention_kernel(CacheAttentionArgs a)
{
    __shared__ typename CacheAttention<NB, GS, NG>::Shared sh;
    CacheAttention<NB, GS, NG> attention(a);
    attention.run(sh);
}

template <int NB, int GS, int NG>
hipError_t launch_attention(const CacheAttentionArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)(a.heads * a.row_tiles), (unsigned)(a.workers + a.batch));
    hipLaunchKernelGGL((cache_attention_kernel<NB, GS, NG>), grid, dim3(64 * kCacheWaves), 0, s, a);
    return hipGetLastError();
}

template <int NB>
hipError_t launch_cache_attention(int dim, int gs, const CacheAttentionArgs &a, hipStream_t s)
{
    switch (dim * 1024 + gs) {
    case 64 * 1024 + 32: return launch_attention<NB, 32, 2>(a, s);
    case 64 * 1024 + 64: return launch_attention<NB, 64, 1>(a, s);
    case 96 * 1024 + 32: return launch_attention<NB, 32, 3>(a, s);
    case 128 * 1024 + 32: return launch_attention<NB, 32, 4>(a, s);
    case 128 * 1024 + 64: return launch_attention<NB, 64, 2>(a, s);
    case 128 * 1024 + 128: return launch_attention<NB, 128, 1>(a, s);
    case 192 * 1024 + 64: return launch_attention<NB, 64, 3>(a, s);
    case 256 * 1024 + 64: return launch_attention<NB, 64, 4>(a, s);
    case 256 * 1024 + 128: return launch_attention<NB, 128, 2>(a, s);
    case 256 * 1024 + 256: return launch_attention<NB, 256, 1>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace
}  // namespace hqq
