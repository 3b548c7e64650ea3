// hqq_cache_codec.hip -- writing tokens into the quantized key-value cache and
// reading them back.
//
// A lane takes 8 consecutive values of a row (one 16-byte load or store), so a
// group is 4 to 32 neighbouring lanes of one wave; blockIdx.y is the side (k, v).
// Rows go by blocks of 16 tokens, then heads, then the block's tokens: consecutive
// tokens of a head lie together in a page, so that codes and scales move by whole lines,
// where token by token they would by pieces of 8 and 64 bytes.
//
// What bounds them: memory where there are many tokens (write of 4096 tokens of 32 x 128 to 4 bits
// with the values back, 155 MB in 33 us, 4.7 TB/s of the 4.9 of a copy; by tokens 39; read of 32768
// tokens of 8 x 128, 176 MB in 30 us, 5.9 TB/s), else the launch: 3 to 5 us in the kernel, the host's
// side 8 to 9.
#include "hqq_cache_internal.h"

namespace hqq {
namespace {

constexpr int kBlock = 256;

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <bool BF>
__device__ __forceinline__ float widen(uint16_t v)
{
    if constexpr (BF) {
        return __uint_as_float((uint32_t)v << 16);
    } else {
        _Float16 h;
        __builtin_memcpy(&h, &v, 2);
        return (float)h;
    }
}

// one fp32 -> 16-bit value, round to nearest even
template <bool BF>
__device__ __forceinline__ uint16_t narrow(float v)
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

// This lane's row, and its slot's row of the cache (-1: skipped)
template <int D>
struct Place {
    static constexpr int kLanes = D / 8;              // lanes of a row
    static constexpr int kRows = kBlock / kLanes;     // rows of a workgroup
    int chunk;
    int32_t token, head;
    int64_t cache_row;
    bool valid;

    __device__ __forceinline__ Place(const CacheCodecArgs &a, uint32_t group) : Place(a, group, -1)
    {
        if (!valid)
            return;
        const int64_t slot = a.slots[token];
        if (slot >= 0 && slot < a.slot_count)
            cache_row = (((slot >> a.page_shift) * a.heads + head) << a.page_shift) + (slot & a.page_mask);
    }

    // the same again, the cache's row known
    __device__ __forceinline__ Place(const CacheCodecArgs &a, uint32_t group, int64_t known)
    {
        const int local = threadIdx.x / kLanes;
        chunk = threadIdx.x - local * kLanes;
        const uint32_t row = group * kRows + local, line = row / kCacheCodecTokens;
        // line / heads: the factor is rounded up from 2^36 / heads, line * 1023 < 2^36
        const uint32_t block = (uint32_t)((line * a.head_factor) >> 36);
        head = (int32_t)(line - block * (uint32_t)a.heads);
        token = (int32_t)(block * kCacheCodecTokens + row % kCacheCodecTokens);
        valid = local < kRows && token < a.tokens;
        cache_row = known;
    }

    __device__ __forceinline__ int64_t hat_at(const CacheCodecArgs &a) const
    {
        return ((int64_t)token * a.heads + head) * D + chunk * 8;
    }
};

// Whether the quotients (code - zero) / scale, their remainders and 1 / scale stay clear of
// the ends of fp32's range
__device__ __forceinline__ bool moderate(float scale, float zero)
{
    return scale > 0x1p-60f && scale < 0x1p60f && fabsf(zero) < 0x1p60f && (zero == 0.0f || fabsf(zero) > 0x1p-60f);
}

// The values (code - zero) / scale in fp32, rounded once.  Where all the wave's groups are
// moderate, the division is a product with the correctly rounded 1 / scale and two
// corrections by the exact remainder: the first makes the quotient faithful, the second
// correctly rounded (Markstein's theorem), 5 operations for the division's 10.
template <bool BF>
__device__ __forceinline__ uint4v values16(const float (&code)[8], float scale, float zero)
{
    uint16_t v[8];
    if (__all(moderate(scale, zero))) {
        const float inv = 1.0f / scale;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = code[j] - zero;
            float q = x * inv;
            q = fmaf(fmaf(-scale, q, x), inv, q);
            q = fmaf(fmaf(-scale, q, x), inv, q);
            // the quotient is rounded to fp32 first, as the division's is: left to itself the compiler
            // takes the last step and the rounding to fp16 for one operation, with one rounding
            asm("" : "+v"(q));
            v[j] = narrow<BF>(q);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = narrow<BF>((code[j] - zero) / scale);
    }
    uint4v r;
    __builtin_memcpy(&r, v, 16);
    return r;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __uint_as_float(__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}

// The smallest of v over the LANES neighbouring lanes of a group (the largest: of -v): the lanes of
// a pair, of 4, of 8 and of 16 exchanged or mirrored, then rows of 16 swapped
template <int LANES>
__device__ __forceinline__ float group_min(float v)
{
    v = fminf(v, dpp<0xB1>(v));
    v = fminf(v, dpp<0x4E>(v));
    if constexpr (LANES >= 8)
        v = fminf(v, dpp<0x141>(v));
    if constexpr (LANES >= 16)
        v = fminf(v, dpp<0x140>(v));
    if constexpr (LANES >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = fminf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}

// ROWS groups of kRows rows per workgroup, whose loads go out together.  (One in the write: without the
// arrays, the row's place found once, the compiler's order of loads took 33 us of 4096 tokens to 37.)
template <int NB, int D, int GS, bool BF, int ROWS>
__global__ __launch_bounds__(kBlock) void cache_write_kernel(CacheCodecArgs a)
{
    const int side = blockIdx.y;
    uint4 raw[ROWS];
    int64_t cache_row[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const Place<D> p(a, blockIdx.x * ROWS + i);
        cache_row[i] = p.cache_row;
        raw[i] = uint4{0, 0, 0, 0};
        if (p.valid)
            raw[i] = *reinterpret_cast<const uint4 *>(a.x[side] + p.token * a.token_stride[side] +
                                                      p.head * a.head_stride[side] + p.chunk * 8);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const Place<D> p(a, blockIdx.x * ROWS + i, cache_row[i]);
        uint16_t h[8];
        __builtin_memcpy(h, &raw[i], 16);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = widen<BF>(h[j]);
        float lo = x[0], hi = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            lo = fminf(lo, x[j]);
            hi = fmaxf(hi, x[j]);
        }
        lo = group_min<GS / 8>(lo);
        hi = -group_min<GS / 8>(-hi);
        constexpr float qmax = (float)((1 << NB) - 1);
        const float range = hi - lo;
        const float scale = range == 0.0f ? 1.0f : qmax / range;
        const float zero = -(lo * scale);
        float code[8];
        uint64_t bits = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            code[j] = fminf(fmaxf(rintf(fmaf(x[j], scale, zero)), 0.0f), qmax);
            bits |= (uint64_t)(uint32_t)code[j] << (NB * j);
        }
        if (p.cache_row >= 0) {
            char *dst = (char *)a.packed[side] + p.cache_row * (D * NB / 8) + p.chunk * NB;
            if constexpr (NB == 8)
                *reinterpret_cast<uint2 *>(dst) = uint2{(uint32_t)bits, (uint32_t)(bits >> 32)};
            else if constexpr (NB == 4)
                *reinterpret_cast<uint32_t *>(dst) = (uint32_t)bits;
            else
                *reinterpret_cast<uint16_t *>(dst) = (uint16_t)bits;
            if (p.chunk % (GS / 8) == 0) {
                const int64_t g = p.cache_row * (D / GS) + p.chunk / (GS / 8);
                a.scale[side][g] = scale;
                a.zero[side][g] = zero;
            }
        }
        if (a.hat[side]) {
            const uint4v values = values16<BF>(code, scale, zero);
            if (p.valid)
                *reinterpret_cast<uint4v *>(a.hat[side] + p.hat_at(a)) = p.cache_row >= 0 ? values : uint4v{0, 0, 0, 0};
        }
    }
}

template <int NB, int D, int GS, bool BF, int ROWS>
__global__ __launch_bounds__(kBlock) void cache_read_kernel(CacheCodecArgs a)
{
    const int side = blockIdx.y;
    uint64_t bits[ROWS];
    float scale[ROWS], zero[ROWS];
    int64_t cache_row[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const Place<D> p(a, blockIdx.x * ROWS + i);
        cache_row[i] = p.cache_row;
        bits[i] = 0;
        scale[i] = 1.0f;
        zero[i] = 0.0f;
        if (p.cache_row >= 0) {
            const char *src = (const char *)a.packed[side] + p.cache_row * (D * NB / 8) + p.chunk * NB;
            if constexpr (NB == 8) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src);
                bits[i] = (uint64_t)w.y << 32 | w.x;
            } else if constexpr (NB == 4) {
                bits[i] = *reinterpret_cast<const uint32_t *>(src);
            } else {
                bits[i] = *reinterpret_cast<const uint16_t *>(src);
            }
            const int64_t g = p.cache_row * (D / GS) + p.chunk / (GS / 8);
            scale[i] = a.scale[side][g];
            zero[i] = a.zero[side][g];
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const Place<D> p(a, blockIdx.x * ROWS + i, cache_row[i]);
        float code[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            code[j] = (float)(uint32_t)(bits[i] >> (NB * j) & ((1u << NB) - 1));
        const uint4v values = values16<BF>(code, scale[i], zero[i]);
        uint4v *to = reinterpret_cast<uint4v *>(a.hat[side] + p.hat_at(a));
        if (p.valid) {
            if constexpr (ROWS > 1)          // more than the L2s hold: past them
                __builtin_nontemporal_store(values, to);
            else
                *to = values;
        }
    }
}

// Groups of rows per workgroup: the read waits for slots, then codes, and has little to do with
// either, so large ones take several at a time (32768 tokens of 8 x 128 at 4 bits 43 us by 4, 56 by 1,
// 29 by 4 with stores past the caches); the write is no faster so.
constexpr int kReadRows = 4;
constexpr int64_t kReadLarge = 65536;

template <int D, int ROWS>
dim3 grid_of(const CacheCodecArgs &a)
{
    constexpr int kRows = Place<D>::kRows * ROWS;
    return dim3((unsigned)((a.rows + kRows - 1) / kRows), 2);
}

template <int NB, int D, int GS, bool BF>
hipError_t launch(bool write, const CacheCodecArgs &a, hipStream_t s)
{
    if (write)
        hipLaunchKernelGGL((cache_write_kernel<NB, D, GS, BF, 1>), (grid_of<D, 1>(a)), dim3(kBlock), 0, s, a);
    else if (a.rows >= kReadLarge)
        hipLaunchKernelGGL((cache_read_kernel<NB, D, GS, BF, kReadRows>), (grid_of<D, kReadRows>(a)), dim3(kBlock),
                           0, s, a);
    else
        hipLaunchKernelGGL((cache_read_kernel<NB, D, GS, BF, 1>), (grid_of<D, 1>(a)), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

template <int NB, bool BF>
hipError_t launch_format(bool write, int dim, int gs, const CacheCodecArgs &a, hipStream_t s)
{
    switch (dim * 1024 + gs) {
    case 64 * 1024 + 32: return launch<NB, 64, 32, BF>(write, a, s);
    case 64 * 1024 + 64: return launch<NB, 64, 64, BF>(write, a, s);
    case 96 * 1024 + 32: return launch<NB, 96, 32, BF>(write, a, s);
    case 128 * 1024 + 32: return launch<NB, 128, 32, BF>(write, a, s);
    case 128 * 1024 + 64: return launch<NB, 128, 64, BF>(write, a, s);
    case 128 * 1024 + 128: return launch<NB, 128, 128, BF>(write, a, s);
    case 192 * 1024 + 64: return launch<NB, 192, 64, BF>(write, a, s);
    case 256 * 1024 + 64: return launch<NB, 256, 64, BF>(write, a, s);
    case 256 * 1024 + 128: return launch<NB, 256, 128, BF>(write, a, s);
    case 256 * 1024 + 256: return launch<NB, 256, 256, BF>(write, a, s);
    }
    return hipErrorInvalidValue;
}

template <int NB>
hipError_t launch_bits(bool write, int dim, int gs, bool bf16, const CacheCodecArgs &a, hipStream_t s)
{
    return bf16 ? launch_format<NB, true>(write, dim, gs, a, s) : launch_format<NB, false>(write, dim, gs, a, s);
}

hipError_t launch_all(bool write, int nbits, int dim, int gs, bool bf16, const CacheCodecArgs &a, hipStream_t s)
{
    return nbits == 2   ? launch_bits<2>(write, dim, gs, bf16, a, s)
           : nbits == 4 ? launch_bits<4>(write, dim, gs, bf16, a, s)
                        : launch_bits<8>(write, dim, gs, bf16, a, s);
}

}  // namespace

hipError_t launch_cache_write(int nbits, int dim, int group_size, bool bf16, const CacheCodecArgs &a, hipStream_t s)
{
    return launch_all(true, nbits, dim, group_size, bf16, a, s);
}

hipError_t launch_cache_read(int nbits, int dim, int group_size, bool bf16, const CacheCodecArgs &a, hipStream_t s)
{
    return launch_all(false, nbits, dim, group_size, bf16, a, s);
}

}  // namespace hqq
