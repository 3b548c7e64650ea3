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
// a lane holds 4 tokens of each 16 for one head.  These are its contraction slots in the
// second product O^T = V^T P^T, for which it needs just its own tokens: the weights never
// leave their lane.  V's side of it wants 8 tokens of one dim per lane, against rows of dims in
// memory: the transposing LDS reads (of 4 or 8 bits an element; two 2-bit codes count as one
// of 4) hand a lane the codes of its own tokens, in the order of the rows that it names.
//
// A wave takes tiles of 32 tokens, its loads whole lines in 16-byte pieces over the lanes, a tile
// ahead in registers; through LDS they reach the operands' lanes.
//
// What bounds it: the bytes of codes and scales where sequences are long (64 sequences of 8192 tokens,
// 8 heads of 128 dims at 4 bits in groups of 64, 64 q heads: 673 MB in 132 to 137 us, 5 TB/s, of 6.2 that a
// read reaches; its loads alone take 117), with about as much time of vector operations beside them.  A segment
// (a workgroup's part of a sequence) costs about 3 us beside its tiles, which is what short sequences
// pay (32 ragged ones, 32 heads: 344 MB in 78 to 82 us), and a call has a floor of some 9 us of launches.
#pragma once

#include "hqq_cache_plan.h"

#include <type_traits>

namespace hqq {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ half8 operand(const uint32_t (&r)[4])
{
    half8 h;
    __builtin_memcpy(&h, r, 16);
    return h;
}

// Field f of both half words of a word of keys as fp16 subnormals, times key_factor.  The
// matrix units align the products of a sum by their operands' exponents, and a subnormal
// counts with the least one, so a low field loses bits of the sum: they are brought to the
// upper bits of the 10 that a subnormal has (error of lse at 2 bits 1.5e-6 without).
template <int NB>
__device__ __forceinline__ uint32_t key_field(uint32_t x, int f)
{
    if constexpr (NB == 8) {
        return (f ? x >> 8 : x) & 0x00ff00ffu;
    } else if constexpr (NB == 4) {
        return (f == 0 ? x << 4 : x >> (4 * f - 4)) & 0x00f000f0u;
    } else {
        const int left = 6 - 4 * (f / 2);
        return (left > 0 ? x << left : x >> -left) & (f % 2 ? 0x03000300u : 0x00c000c0u);
    }
}

template <int NB>
constexpr float key_factor(int f)
{
    return NB == 8 ? 1.0f : NB == 4 ? 16.0f : f % 2 ? 256.0f : 64.0f;
}

// The same for a lane's values: word x holds 8 tokens of 4 bits (or 4 of 8), field f is tokens f and
// f + 4 (f and f + 2) of it, i the code within 4 bits.  They come out times value_factor.
template <int NB>
__device__ __forceinline__ uint32_t value_field(uint32_t x, int f, int i)
{
    return key_field<NB>(x, NB == 2 ? 2 * f + i : f);
}

template <int NB>
constexpr float value_factor(int i)
{
    return key_factor<NB>(NB == 2 ? i : 0);
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
    if constexpr (N == 2) {
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

template <bool BF>
__device__ __forceinline__ float widen16(uint16_t v)
{
    _Float16 h;
    __builtin_memcpy(&h, &v, 2);
    return BF ? __uint_as_float((uint32_t)v << 16) : (float)h;
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

// the value of the lane CTRL & 15 places on in the row of 16 (0x121 to 0x12f: rotated)
template <int CTRL>
__device__ __forceinline__ float dpp_float(float v)
{
    return __uint_as_float(__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
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

typedef int int2v __attribute__((ext_vector_type(2)));

// 16 rows of 16 4-bit elements (8 rows of 8-bit ones) over 16 lanes, 8 bytes each: lane l gets
// element l of every row
template <int NB>
__device__ __forceinline__ int2v read_transposed(const char *lds)
{
    const auto p = (__attribute__((address_space(3))) int2v *)lds;
    if constexpr (NB == 8)
        return __builtin_amdgcn_ds_read_tr8_b64_v2i32(p);
    else
        return __builtin_amdgcn_ds_read_tr4_b64_v2i32(p);
}

template <int NB, int GS, int NG, bool BF>
struct CacheAttention {
    static constexpr int D = GS * NG;
    static constexpr int kRowBytes = D * NB / 8;
    typedef KeyOrder<NB, GS> Keys;
    static constexpr int kTile = kCacheTile, kStep = kCacheStep;
    static constexpr int kSubs = kTile / 16;                    // subtiles: 16 consecutive rows of a page
    // rows in LDS an odd number of 16-byte pieces apart: 8 of them, at one place each, cover the banks
    static constexpr int kRowPitch = kRowBytes % 32 == 0 ? kRowBytes + 16 : kRowBytes;
    static constexpr int kPieces = (kSubs * kRowBytes + 63) / 64;       // 16-byte pieces per lane and tile
    // a tile's scales over the lanes: token col, and 4 of (subtile, group) along the quads
    static constexpr int kGroups = NG == 3 ? 4 : NG;
    static constexpr int kMetas = (kSubs * kGroups + 3) / 4;
    static constexpr int kPerQuads = 4 / kGroups;               // subtiles along the quads
    // transposed reads, of kCodes dims per lane
    static constexpr int kCodes = NB == 2 ? 2 : 1;
    static constexpr int kBlockDims = 16 * kCodes;
    static constexpr int kBlocks = D / kBlockDims;
    static constexpr int kReadBlocks = NB == 8 ? 1 : 2;         // blocks of a transposed read
    static constexpr int kPitch = D + 4;

    struct alignas(16) Shared {
        union {
            struct {
                uint4v q[NG][Keys::kUnits][64];                 // operands of the first product
                uint4v rows[kCacheWaves][2][kTile * kRowPitch / 16];    // a tile's rows of k and of v
                float meta[kCacheWaves][3][NG][kTile];          // r of k, scaled r of v, z of v
            };
            float sums[kCacheWaves][16][kPitch];
        };
        float2 ml[kCacheWaves][16];
    };

    struct Where {
        int at;
        int there;                                              // bit t: subtile t's page is there
        int64_t row[kSubs];
    };
    struct Loads {
        uint4v k[kPieces], v[kPieces];
        float ks[kMetas], kz[kMetas], vs[kMetas], vz[kMetas];
    };

    const CacheAttentionArgs &a;
    const int lane, wave, col, quad;
    int head, row_tile, worker;
    // the segment: tokens [begin, end) of sequence b, of which those from `first` on count
    int b, begin, end, first;

    __device__ __forceinline__ CacheAttention(const CacheAttentionArgs &args)
        : a(args), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), col(lane & 15),
          quad(lane >> 4)
    {
        // Workgroups go to the 8 XCDs in turn: the heads of one run, whose parts of a page lie
        // together, to one of them
        const uint32_t id = blockIdx.y * gridDim.x + blockIdx.x, turn = id >> 3;
        const uint32_t column = turn % gridDim.x;
        worker = (int)(turn / gridDim.x * 8 + (id & 7));
        head = (int)(column % (uint32_t)a.heads);
        row_tile = (int)(column / (uint32_t)a.heads);
    }

    // The pages of this wave's next 64 subtiles from tile `at` on, one in each lane
    __device__ __forceinline__ int pages_from(int at) const
    {
        const int token = at + lane / kSubs * kStep + lane % kSubs * 16;
        int page = token < end ? a.table[(int64_t)b * a.table_width + (token >> a.page_shift)] : -1;
        // waited for here: tiles that do not come here must not wait for their own loads at its use
        asm volatile("" : "+v"(page));
        return page;
    }

    __device__ __forceinline__ Where where(int at, int pages, int tile) const
    {
        Where w;
        w.at = at;
        w.there = 0;
#pragma unroll
        for (int t = 0; t < kSubs; ++t) {
            const int page = __builtin_amdgcn_readlane(pages, (kSubs * tile + t) & 63);
            const bool there = (uint32_t)page < (uint32_t)a.pages;
            w.there |= there << t;
            w.row[t] = (((int64_t)(there ? page : 0) * a.heads + head) << a.page_shift) + ((at + 16 * t) & a.page_mask);
        }
        return w;
    }

    // whether all the tile's tokens count
    __device__ __forceinline__ bool whole(int at, int there) const
    {
        return there == (1 << kSubs) - 1 && at >= first && at + kTile <= end;
    }

    __device__ __forceinline__ bool counts(int at, int there, int t, int place) const
    {
        const int token = at + 16 * t + place;
        return token >= first && token < end && (there >> t & 1);
    }

    static __device__ __forceinline__ int64_t row_of(const Where &w, int t) { return t ? w.row[1] : w.row[0]; }

    // A lane's i-th piece of a tile; the last lanes may come to the last piece again
    __device__ __forceinline__ int piece(int i) const
    {
        const int x = lane + 64 * i;
        return (kSubs * kRowBytes) % 64 == 0 || x < kSubs * kRowBytes ? x : kSubs * kRowBytes - 1;
    }

    __device__ __forceinline__ int meta_sub(int i) const { return (quad + 4 * i) / kGroups % kSubs; }
    __device__ __forceinline__ int meta_group() const { return quad % kGroups < NG ? quad % kGroups : 0; }

    // All of a tile, nothing under a condition that the lanes do not share: the rows are there
    // whether their tokens count or not
    __device__ __forceinline__ void load(const Where &w, Loads &l) const
    {
        if (a.page_mask >= kTile - 1) {      // the tile's rows follow each other: one base for the wave
            const int64_t base = w.row[0] * NG;
#pragma unroll
            for (int i = 0; i < kMetas; ++i) {
                const uint32_t from = (16 * meta_sub(i) + col) * NG + meta_group();
                l.ks[i] = (a.scale[0] + base)[from], l.kz[i] = (a.zero[0] + base)[from];
                l.vs[i] = (a.scale[1] + base)[from], l.vz[i] = (a.zero[1] + base)[from];
            }
            const uint4v *k = reinterpret_cast<const uint4v *>((const char *)a.packed[0] + w.row[0] * kRowBytes);
            const uint4v *v = reinterpret_cast<const uint4v *>((const char *)a.packed[1] + w.row[0] * kRowBytes);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                l.k[i] = k[piece(i)];
                l.v[i] = v[piece(i)];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kMetas; ++i) {
                const int64_t from = (row_of(w, meta_sub(i)) + col) * NG + meta_group();
                l.ks[i] = a.scale[0][from], l.kz[i] = a.zero[0][from];
                l.vs[i] = a.scale[1][from], l.vz[i] = a.zero[1][from];
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int t = piece(i) / kRowBytes;
                const int64_t from = row_of(w, t) * kRowBytes + (piece(i) - t * kRowBytes) * 16;
                l.k[i] = *reinterpret_cast<const uint4v *>((const char *)a.packed[0] + from);
                l.v[i] = *reinterpret_cast<const uint4v *>((const char *)a.packed[1] + from);
            }
        }
    }

    // A piece's place in LDS
    static __device__ __forceinline__ int piece_place(int x)
    {
        return kRowPitch == kRowBytes ? 16 * x : x / (kRowBytes / 16) * kRowPitch + x % (kRowBytes / 16) * 16;
    }

    // a lane's words of a token's group
    static __device__ __forceinline__ void read_keys(const char *rows, int row, int byte,
                                                     uint32_t (&w)[(Keys::kBytes + 3) / 4])
    {
        constexpr int kPart = Keys::kBytes < 16 ? Keys::kBytes : 16;
#pragma unroll
        for (int i = 0; i < Keys::kBytes / kPart; ++i) {
            uint32_t part[(kPart + 3) / 4];
            load_words<kPart>(part, rows + row * kRowPitch + byte + i * kPart);
#pragma unroll
            for (int k = 0; k < (kPart + 3) / 4; ++k)
                w[i * (kPart / 4) + k] = part[k];
        }
    }

    // One segment, from q to the output or the workspace's slot
    __device__ __forceinline__ void segment(Shared &sh, int slot, bool whole_sequence)
    {
        const int in_group = row_tile * 16 + col;               // this column's q head within the group
        const bool real = in_group < a.G;
        const int q_head = head * a.G + (real ? in_group : 0);

        // ---- the first tile's loads
        const int at0 = begin + wave * kTile;
        const int tiles = at0 < end ? (end - at0 + kStep - 1) / kStep : 0;
        int pages = pages_from(at0);
        Loads l;
        Where next = where(at0, pages, 0);
        if (tiles > 0)
            load(next, l);

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
                    const uint4v raw = *reinterpret_cast<const uint4v *>(src + g * GS + i);
                    uint16_t h[8];
                    __builtin_memcpy(h, &raw, 16);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        q[g][i + j] = widen16<BF>(h[j]);
                        top = fmaxf(top, fabsf(q[g][i + j]));
                    }
                }
            top = column_max(top);
            // the largest to [2^14, 2^15): fp16 then holds what is within 2^-20 of it or so whole
            // (the fields' factors take up to 8 bits), and the rest to 2^-31 of it
            int e = top > 0.0f && top < INFINITY ? 14 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
            e = e > 100 ? 100 : e;
            const float f = power_of_two(e);
            // (2^12 of the 2^24, see kr; below 2^-126 scores of any size are all alike, and 0 times those of
            // tokens that do not count, -infinity, would be NaN)
            score_scale = fmaxf(a.scale_log2 * 0x1p12f * power_of_two(-e), 0x1p-126f);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float sum = 0.0f;
#pragma unroll
                for (int u = 0; u < Keys::kUnits; ++u) {
                    uint32_t q16[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float factor = key_factor<NB>(Keys::field_of(u, r));
                        const float inv = f / factor;
                        half2v h;
                        h[0] = (_Float16)(q[g][Keys::lo(u, r)] * inv);
                        h[1] = (_Float16)(q[g][Keys::hi(u, r)] * inv);
                        __builtin_memcpy(&q16[r], &h, 4);
                        sum += ((float)h[0] + (float)h[1]) * (factor * 0x1p-24f);
                    }
                    sh.q[g][u][lane] = uint4v{q16[0], q16[1], q16[2], q16[3]};
                }
                q_sum[g] = column_sum(sum);
            }
        }
        // the zeros' part of the scores, -sum_g (r z)_tg q_sum_g, is a product of depth 4 in fp32, with the
        // groups of kPerQuads subtiles along its depth
        float q_zero[kPerQuads];
#pragma unroll
        for (int t = 0; t < kPerQuads; ++t) {
            q_zero[t] = 0.0f;
#pragma unroll
            for (int i = 0; i < NG; ++i)
                q_zero[t] = quad == t * kGroups + i ? -q_sum[i] : q_zero[t];
        }

        // ---- state: per column, but sums of weights and zeros only over this lane's tokens
        float4v o[kBlocks][kCodes];
        float z_sum[NG], v_unit[NG];
        float m2 = -INFINITY, total = 0.0f;                     // maximum (exponent of 2), sum of weights
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            z_sum[g] = 0.0f;
            v_unit[g] = 0x1p120f;
        }
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int i = 0; i < kCodes; ++i)
                o[n][i] = float4v{0.f, 0.f, 0.f, 0.f};
        float lane_unit = v_unit[0];                            // of the group whose scales this lane loads
        float (*meta)[NG][kTile] = sh.meta[wave];
        char *k_rows = (char *)sh.rows[wave][0], *v_rows = (char *)sh.rows[wave][1];
        // the row that this lane names to the transposing reads: its quad's tokens in their order
        // (8 bits: 16 dims of each, in two halves; else one block of dims of each and then the next)
        const int named = NB == 8 ? col / 2 : col % 8;
        const int v_row = 16 * (named / 4) + 4 * quad + named % 4;

        // One tile.  The next one's loads leave at its top, when its own are in LDS.  Nothing is loaded
        // under a condition, which would make the waits for older loads wait for these too.
        const auto step = [&](int tile, auto more) {
            const int at = next.at, there = next.there;
            const bool all = whole(at, there);

            // ---- scales: reciprocals (to 1 ulp), to the layout of the scores through LDS
            float rz[kMetas];                                   // (r z) of k
            float vr[kMetas];
            float raise = 0.0f;
            if (!all) {
                // tokens that do not count: 1 / scale and zero of 0, whatever the page holds there
#pragma unroll
                for (int i = 0; i < kMetas; ++i) {
                    const bool in = counts(at, there, meta_sub(i), col);
                    l.ks[i] = in ? l.ks[i] : INFINITY;
                    l.vs[i] = in ? l.vs[i] : INFINITY;
                    l.kz[i] = in ? l.kz[i] : 0.0f;
                    l.vz[i] = in ? l.vz[i] : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < kMetas; ++i) {
                const float kr = __builtin_amdgcn_rcpf(l.ks[i]) * 0x1p12f;  // the codes' 2^-24 taken back, half here
                vr[i] = __builtin_amdgcn_rcpf(l.vs[i]);
                rz[i] = kr * l.kz[i];
                float *to = &meta[0][meta_group()][16 * meta_sub(i) + col];
                to[0] = kr;
                to[2 * NG * kTile] = l.vz[i];
                raise = fmaxf(raise, vr[i]);
            }
            // a group's r of v beyond the unit that its weights are held in?
            if (__any(!(raise * lane_unit <= 0x1p15f))) {
                // the largest of each row of lanes, which hold one group each
                float row_most = raise;
                row_most = fmaxf(row_most, dpp_float<0x128>(row_most));
                row_most = fmaxf(row_most, dpp_float<0x124>(row_most));
                row_most = fmaxf(row_most, dpp_float<0x122>(row_most));
                row_most = fmaxf(row_most, dpp_float<0x121>(row_most));
                float unit[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float most = 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k % kGroups == g)
                            most = fmaxf(most, __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(row_most), 16 * k)));
                    // most * unit in [2^14, 2^15)
                    const int ue = 14 - ((int)(__float_as_uint(most) >> 23) - 127);
                    unit[g] = fminf(v_unit[g], power_of_two(ue < -120 ? -120 : ue > 120 ? 120 : ue));
                    z_sum[g] *= unit[g] / v_unit[g];
                }
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int i = 0; i < kCodes; ++i)
                        o[n][i] *= unit[n * kBlockDims / GS] / v_unit[n * kBlockDims / GS];
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    v_unit[g] = unit[g];
                lane_unit = pick(v_unit, meta_group());
            }
#pragma unroll
            for (int i = 0; i < kMetas; ++i)
                meta[1][meta_group()][16 * meta_sub(i) + col] = vr[i] * lane_unit;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                *reinterpret_cast<uint4v *>(k_rows + piece_place(piece(i))) = l.k[i];
                *reinterpret_cast<uint4v *>(v_rows + piece_place(piece(i))) = l.v[i];
            }
            wave_lds_fence();
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (more) {
                if (((tile + 1) * kSubs & 63) == 0)
                    pages = pages_from(at + kStep);
                next = where(at + kStep, pages, tile + 1);
                load(next, l);
            }

            // ---- scores
            float4v s[kSubs];
#pragma unroll
            for (int t = 0; t < kSubs; ++t)
                s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(rz[t / kPerQuads], q_zero[t % kPerQuads],
                                                            float4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float4v acc[kSubs];
                uint32_t kw[kSubs][(Keys::kBytes + 3) / 4];
#pragma unroll
                for (int t = 0; t < kSubs; ++t) {
                    acc[t] = float4v{0.f, 0.f, 0.f, 0.f};
                    read_keys(k_rows, 16 * t + col, g * (GS * NB / 8) + quad * Keys::kBytes, kw[t]);
                }
#pragma unroll
                for (int u = 0; u < Keys::kUnits; ++u) {
                    const uint4v q4 = sh.q[g][u][lane];
                    const uint32_t q16[4] = {q4[0], q4[1], q4[2], q4[3]};
#pragma unroll
                    for (int t = 0; t < kSubs; ++t) {
                        uint32_t regs[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            uint32_t x = kw[t][Keys::word_of(u, r)];
                            if constexpr (Keys::kHalf)
                                x = (x & 0xffu) | (x >> 8) << 16;
                            regs[r] = key_field<NB>(x, Keys::field_of(u, r));
                        }
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(regs), operand(q16), acc[t], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int t = 0; t < kSubs; ++t) {
                    const float4v r4 = *reinterpret_cast<const float4v *>(&meta[0][g][16 * t + 4 * quad]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        s[t][r] = fmaf(acc[t][r], r4[r], s[t][r]);
                }
            }
            if (!all) {
#pragma unroll
                for (int t = 0; t < kSubs; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (!counts(at, there, t, 4 * quad + r))
                            s[t][r] = -INFINITY;
            }

            // ---- weights
            float top = s[0][0];
#pragma unroll
            for (int j = 1; j < 4 * kSubs; ++j)
                top = fmaxf(top, s[j / 4][j % 4]);
            const float m_new = fmaxf(m2, column_max(top) * score_scale);
            const float ref = m_new == -INFINITY ? 0.0f : m_new;
            const float alpha = __builtin_amdgcn_exp2f(m2 - ref);
            m2 = m_new;
            if (__any(alpha != 1.0f)) {
                total *= alpha;
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    z_sum[g] *= alpha;
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int i = 0; i < kCodes; ++i)
                        o[n][i] *= alpha;
            }
#pragma unroll
            for (int t = 0; t < kSubs; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s[t][r] = __builtin_amdgcn_exp2f(fmaf(s[t][r], score_scale, -ref));
                    total += s[t][r];
                }

            // ---- the second product
            // Weights, paired as value_field pairs tokens.  One operand holds 11 bits of each, a second one the
            // rest: 22 bits, or what is above 2^-39 of the group's largest r so far.  (Without it bf16's outputs too
            // are off by more than their own rounding makes them, 0.00187 of the result beside 0.00181 for one
            // sequence of 131072 tokens; 64 x 8192 tokens 124 us without, 132 with.)
            uint32_t w16[NG][4], rest16[NG][4];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float4v w[2], z4[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    w[t] = s[t] * *reinterpret_cast<const float4v *>(&meta[1][g][16 * t + 4 * quad]);
                    z4[t] = *reinterpret_cast<const float4v *>(&meta[2][g][16 * t + 4 * quad]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // 8 bits: tokens (0, 2) and (1, 3) of either subtile; else the same one of both
                    const int t0 = NB == 8 ? r / 2 : 0, t1 = NB == 8 ? r / 2 : 1;
                    const int r0 = NB == 8 ? r % 2 : r, r1 = NB == 8 ? r % 2 + 2 : r;
                    const float2v both{w[t0][r0], w[t1][r1]};
                    const half2v pair = __builtin_convertvector(both, half2v);
                    __builtin_memcpy(&w16[g][r], &pair, 4);
                    const half2v rest =
                        __builtin_convertvector(float2v{both[0] - (float)pair[0], both[1] - (float)pair[1]}, half2v);
                    __builtin_memcpy(&rest16[g][r], &rest, 4);
                    z_sum[g] = fmaf(both[0], z4[t0][r0], z_sum[g]);
                    z_sum[g] = fmaf(both[1], z4[t1][r1], z_sum[g]);
                }
            }
#pragma unroll
            for (int n = 0; n < kBlocks; n += kReadBlocks) {
                const int block = kReadBlocks == 1 ? n : n + col / 8;       // (96 dims of 2 bits: the last one twice)
                const int byte = NB == 8 ? 16 * n + 8 * (col & 1) : 8 * (block < kBlocks ? block : kBlocks - 1);
                const int2v x = read_transposed<NB>(v_rows + v_row * kRowPitch + byte);
#pragma unroll
                for (int h = 0; h < kReadBlocks && n + h < kBlocks; ++h)
#pragma unroll
                    for (int i = 0; i < kCodes; ++i) {
                        uint32_t regs[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            regs[r] = NB == 8 ? value_field<NB>(x[r / 2], r % 2, 0) : value_field<NB>(x[h], r, i);
                        const int g = (n + h) * kBlockDims / GS;
                        float4v &acc = o[n + h][i];
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(regs), operand(w16[g]), acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(regs), operand(rest16[g]), acc, 0, 0, 0);
                    }
            }
            wave_lds_fence();       // the next tile's rows and scales go where these were
        };
        for (int tile = 0; tile + 1 < tiles; ++tile)
            step(tile, std::true_type{});
        if (tiles > 0)
            step(tiles - 1, std::false_type{});

        // ---- the four waves' sums joined
        total = column_sum(total);
#pragma unroll
        for (int g = 0; g < NG; ++g)
            z_sum[g] = column_sum(z_sum[g]);
        if (quad == 0)
            sh.ml[wave][col] = float2{m2, total};
        __syncthreads();            // also: no wave reads rows or scales any more, whose place the sums take
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
            for (int n = 0; n < kBlocks; ++n) {
                const int g = n * kBlockDims / GS;
                const float back = own / v_unit[g];
                float *to = &sh.sums[wave][col][n * kBlockDims + 4 * quad * kCodes];
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < kCodes; ++i)
                        to[r * kCodes + i] = fmaf(o[n][i][r], 0x1p24f / value_factor<NB>(i), -z_sum[g]) * back;
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
                    *reinterpret_cast<uint2 *>(a.out + out_row * D + d) = cache_round4<BF>(v * inv);
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
        __syncthreads();            // the next segment's rows go where the sums were
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
        int at = 0, start = 0, stop;
        bool cross = false;
        CacheSpan s;
        int slot = 0;
        if (a.workers == 0) {        // a sequence each
            b = worker;
            if (b >= a.batch)
                return;
            s = cache_span(a, b);
            stop = s.steps;
        } else {
            const CachePlan plan(a, lane);
            if (worker >= plan.runs)
                return;
            at = worker * plan.run;  // (below 2^31: of runs that cross there are `workers`)
            stop = at + plan.run;
            cross = plan.cross;
            b = plan.find(a, at, lane, start, s);
            slot = plan.slot(a, worker, b, at == start);
        }
        while (b < a.batch) {
            const int next = start + s.steps, upto = stop < next ? stop : next;
            first = s.first;
            begin = s.base + (at - start) * kStep;
            end = upto < next ? s.base + (upto - start) * kStep : s.length;
            segment(sh, slot, at == start && upto == next);
            if (!cross || upto == stop)
                return;
            at = start = next;
            slot = CachePlan::next_slot(a, slot);
            if (++b < a.batch)
                s = cache_span(a, b);
        }
    }
};

template <int NB, int GS, int NG, bool BF>
__global__ __launch_bounds__(64 * kCacheWaves, cache_resident(NB, GS * NG, GS)) void cache_attention_kernel(CacheAttentionArgs a)
{
    typedef typename CacheAttention<NB, GS, NG, BF>::Shared Shared;
    static_assert(cache_resident(NB, GS * NG, GS) * sizeof(Shared) <= kLdsOfCu);
    __shared__ Shared sh;
    CacheAttention<NB, GS, NG, BF> attention(a);
    attention.run(sh);
}

template <int NB, int GS, int NG, bool BF>
hipError_t launch_attention(const CacheAttentionArgs &a, hipStream_t s)
{
    // runs that keep to their sequences number at most one a sequence more than workers; of more sequences
    // than workers they cross
    const int runs = a.workers + (a.workers && a.batch > a.workers ? 0 : a.batch);
    const dim3 grid((unsigned)(a.heads * a.row_tiles), (unsigned)((runs + 7) / 8 * 8));
    hipLaunchKernelGGL((cache_attention_kernel<NB, GS, NG, BF>), grid, dim3(64 * kCacheWaves), 0, s, a);
    return hipGetLastError();
}

template <int NB, bool BF>
hipError_t launch_cache_attention(int dim, int gs, const CacheAttentionArgs &a, hipStream_t s)
{
    switch (dim * 1024 + gs) {
    case 64 * 1024 + 32: return launch_attention<NB, 32, 2, BF>(a, s);
    case 64 * 1024 + 64: return launch_attention<NB, 64, 1, BF>(a, s);
    case 96 * 1024 + 32: return launch_attention<NB, 32, 3, BF>(a, s);
    case 128 * 1024 + 32: return launch_attention<NB, 32, 4, BF>(a, s);
    case 128 * 1024 + 64: return launch_attention<NB, 64, 2, BF>(a, s);
    case 128 * 1024 + 128: return launch_attention<NB, 128, 1, BF>(a, s);
    case 192 * 1024 + 64: return launch_attention<NB, 64, 3, BF>(a, s);
    case 256 * 1024 + 64: return launch_attention<NB, 64, 4, BF>(a, s);
    case 256 * 1024 + 128: return launch_attention<NB, 128, 2, BF>(a, s);
    case 256 * 1024 + 256: return launch_attention<NB, 256, 1, BF>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace
}  // namespace hqq
