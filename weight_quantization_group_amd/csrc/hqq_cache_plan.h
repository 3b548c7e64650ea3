// hqq_cache_plan.h -- how an attention call's sequences are shared out over the
// workgroups, found on the device (the lengths are there), and the ends that the
// attention and the join have in common.
//
// The tokens of all sequences, in tiles of 32 and one sequence after the other, are cut
// into `workers` equal runs; workgroup w of a key-value head takes run w, whatever
// sequences it crosses, so that all of them end together however ragged the batch is.  The
// part of a sequence that a run holds is a segment.  Runs and sequences both advance along
// the tiles, so segment (w, b) has slot w + b in the workspace to itself.
#pragma once

#include "hqq_cache_internal.h"

namespace hqq {
namespace {

typedef float float4v __attribute__((ext_vector_type(4)));

struct CacheSpan {
    int first, base, length;   // first token that counts, its tile's first token, the length
    int tiles;                 // tiles from base on, at least one (it writes the output)
};

// A 64-bit value that is the same in all lanes, as such
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ CacheSpan cache_span(const CacheAttentionArgs &a, int b)
{
    const int64_t most = (int64_t)a.table_width << a.page_shift;
    int n = a.lengths[b];
    n = n < 0 ? 0 : n > most ? (int)most : n;
    const int first = a.window > 0 && n > a.window ? n - a.window : 0;
    const int base = first & ~(kCacheTile - 1);
    const int tiles = (n - base + kCacheTile - 1) / kCacheTile;
    return CacheSpan{first, base, n, tiles < 1 ? 1 : tiles};
}

__device__ __forceinline__ int64_t wave_sum(int64_t v)
{
#pragma unroll
    for (int o = 1; o < 64; o *= 2)
        v += __shfl_xor(v, o);
    return v;
}

// Tiles per run: whole workgroup steps, as many as cover all sequences.
__device__ __forceinline__ int64_t cache_run(const CacheAttentionArgs &a, int lane)
{
    int64_t tiles = 0;
    for (int b = lane; b < a.batch; b += 64)
        tiles += cache_span(a, b).tiles;
    tiles = wave_sum(tiles);
    const int64_t per = (tiles + a.workers - 1) / a.workers;
    return uniform((per + kCacheWaves - 1) / kCacheWaves * kCacheWaves);
}

// The sequence that holds tile `at` (batch behind the last), and its first tile
__device__ __forceinline__ int cache_find(const CacheAttentionArgs &a, int64_t at, int lane, int64_t &start)
{
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const int b = b0 + lane;
        const int64_t tiles = b < a.batch ? cache_span(a, b).tiles : 0;
        int64_t upto = tiles;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const int64_t up = __shfl_up(upto, o);
            upto += lane >= o ? up : 0;
        }
        upto += before;
        const uint64_t behind = __ballot(at < upto);
        if (behind) {
            const int src = __ffsll((unsigned long long)behind) - 1;
            start = uniform(__shfl(upto - tiles, src));
            return __builtin_amdgcn_readfirstlane(b0 + src);
        }
        before = __shfl(upto, 63);
    }
    start = 0;
    return a.batch;
}

__device__ __forceinline__ uint2 cache_round4(float4v v, bool bf16)
{
    uint16_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            const __bf16 h = (__bf16)v[i];
            __builtin_memcpy(&u[i], &h, 2);
        } else {
            const _Float16 h = (_Float16)v[i];
            __builtin_memcpy(&u[i], &h, 2);
        }
    }
    uint2 r;
    __builtin_memcpy(&r, u, 8);
    return r;
}

// 1 / total; 0 where nothing counted
__device__ __forceinline__ float cache_inverse(float total) { return total == 0.0f ? 0.0f : 1.0f / total; }

// log(total * 2^m2); -infinity where nothing counted
__device__ __forceinline__ float cache_lse(float m2, float total)
{
    return total == 0.0f ? -INFINITY : (float)((double)m2 * 0.693147180559945309417) + logf(total);
}

}  // namespace
}  // namespace hqq
