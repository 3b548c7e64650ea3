// hqq_cache_plan.h -- how an attention call's sequences are cut into items, found
// on the device (the lengths are there), and the ends that items and join share.
#pragma once

#include "hqq_cache_internal.h"

namespace hqq {
namespace {

// One item: tokens [begin, end) of sequence `batch`, of which those from `first` on count.
struct CacheItem {
    int batch;         // -1: no such item
    int begin, end, first;
    int index;         // the item's place in the workspace
    int count;         // items of the sequence
};

struct CacheSpan {
    int first, base, length;   // first token that counts, its tile's first token, the length
};

__device__ __forceinline__ CacheSpan cache_span(const CacheAttentionArgs &a, int b)
{
    const int64_t most = (int64_t)a.table_width << a.page_shift;
    int n = a.lengths[b];
    n = n < 0 ? 0 : n > most ? (int)most : n;
    const int first = a.window > 0 && n > a.window ? n - a.window : 0;
    return CacheSpan{first, first & ~(kCacheTile - 1), n};
}

__device__ __forceinline__ int wave_inclusive_sum(int v, int lane)
{
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const int up = __shfl_up(v, o);
        v += lane >= o ? up : 0;
    }
    return v;
}

__device__ __forceinline__ int64_t wave_sum(int64_t v)
{
#pragma unroll
    for (int o = 1; o < 64; o *= 2)
        v += __shfl_xor(v, o);
    return v;
}

// Tokens per item: what splits all sequences into about items_per_head items, in whole
// workgroup steps.  A sequence of n tokens has ceil(n / chunk) items, at least one, so all of
// them number at most items_per_head + batch.
__device__ __forceinline__ int cache_chunk(const CacheAttentionArgs &a, int lane)
{
    int64_t tokens = 0;
    for (int b = lane; b < a.batch; b += 64) {
        const CacheSpan s = cache_span(a, b);
        tokens += s.length - s.base;
    }
    tokens = wave_sum(tokens);
    const int64_t per = (tokens + a.items_per_head - 1) / a.items_per_head;
    const int64_t chunk = (per + kCacheStep - 1) / kCacheStep * kCacheStep;
    return chunk < kCacheStep ? kCacheStep : chunk > (1 << 30) ? 1 << 30 : (int)chunk;
}

__device__ __forceinline__ int cache_items(const CacheSpan &s, int chunk)
{
    const int n = s.length - s.base;
    return n <= chunk ? 1 : (int)(((int64_t)n + chunk - 1) / chunk);
}

// Item `index` of a key-value head; every wave finds it by itself.
__device__ __forceinline__ CacheItem cache_item(const CacheAttentionArgs &a, int index)
{
    const int lane = threadIdx.x & 63;
    const int chunk = cache_chunk(a, lane);
    int before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const int b = b0 + lane;
        CacheSpan s{0, 0, 0};
        int n = 0;
        if (b < a.batch) {
            s = cache_span(a, b);
            n = cache_items(s, chunk);
        }
        const int upto = before + wave_inclusive_sum(n, lane);
        const uint64_t mine = __ballot(index < upto);
        if (mine) {
            const int src = __ffsll((unsigned long long)mine) - 1;
            const int count = __shfl(n, src), start = __shfl(upto, src) - count;
            const int base = __shfl(s.base, src), length = __shfl(s.length, src);
            CacheItem it;
            it.batch = __builtin_amdgcn_readfirstlane(b0 + src);
            it.first = __builtin_amdgcn_readfirstlane(__shfl(s.first, src));
            it.count = __builtin_amdgcn_readfirstlane(count);
            it.index = index;
            it.begin = __builtin_amdgcn_readfirstlane(base + (index - start) * chunk);
            it.end = __builtin_amdgcn_readfirstlane(length - it.begin > chunk ? it.begin + chunk : length);
            return it;
        }
        before = __shfl(upto, 63);
    }
    return CacheItem{-1, 0, 0, 0, 0, 0};
}

__device__ __forceinline__ uint2 cache_round4(const float __attribute__((ext_vector_type(4))) v, bool bf16)
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

// log(total * 2^m2); -infinity where nothing counted
__device__ __forceinline__ float cache_lse(float m2, float total)
{
    return total == 0.0f ? -INFINITY : (float)((double)m2 * 0.693147180559945309417) + logf(total);
}

}  // namespace
}  // namespace hqq
