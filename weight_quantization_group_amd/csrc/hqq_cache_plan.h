// hqq_cache_plan.h -- how an attention call's sequences are shared out over the
// workgroups, found on the device (the lengths are there), and the ends that the
// attention and the join have in common.
//
// The tokens of all sequences, in steps of a workgroup and one sequence after the other, are
// cut into runs of equal length, about `workers` of them; workgroup w of a key-value head
// takes run w.  Long runs cross from one sequence to the next, so that all of them end
// together however ragged the batch is, and so do runs of more sequences than runs; other short
// ones do not, as each segment (a run's part of a sequence) has a prologue and an end of its own
// that cost as much as some steps.  (512 sequences of 100 tokens, 64 runs: 54 us across, 68 within.)
#pragma once

#include "hqq_cache_internal.h"

namespace hqq {
namespace {

typedef float float4v __attribute__((ext_vector_type(4)));

struct CacheSpan {
    int first, base, length;   // first token that counts, its tile's first token, the length
    int steps;                 // workgroup steps from base on, at least one (it writes the output)
};

__device__ __forceinline__ CacheSpan cache_span(const CacheAttentionArgs &a, int b)
{
    const int64_t most = (int64_t)a.table_width << a.page_shift;
    int n = a.lengths[b];
    n = n < 0 ? 0 : n > most ? (int)most : n;
    const int first = a.window > 0 && n > a.window ? n - a.window : 0;
    const int base = first & ~(kCacheTile - 1);
    const int steps = (n - base + kCacheStep - 1) / kCacheStep;
    return CacheSpan{first, base, n, steps < 1 ? 1 : steps};
}

// Adds another lane's value: CTRL as in DPP, into the rows of MASK
template <int CTRL, int MASK>
__device__ __forceinline__ int dpp_add(int v)
{
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, MASK, 0xF, false);
}

// Sums of lanes 0 to this one (row shifts by 1, 2, 4 and 8, then the rows' last lanes to the
// rows behind them)
__device__ __forceinline__ int wave_inclusive_sum(int v)
{
    v = dpp_add<0x111, 0xF>(v);
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);
    return dpp_add<0x143, 0xC>(v);
}

__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_inclusive_sum(v), 63); }

// Every wave finds the same plan by itself, lane l holding sequence l's span, or, of many
// sequences, reads the one that cache_plan_kernel left in the workspace.  All steps number at most
// 2^30 + 2^15 (batch * table_width * page_size <= 2^37).  Of runs that cross sequences there are
// `workers`, of others at most `batch` more.
struct CachePlan {
    CacheSpan mine;            // of sequence `lane` (steps 0: there is none)
    int run;                   // steps per run
    int runs;                  // how many there are
    bool cross;

    __device__ __forceinline__ CachePlan() {}

    __device__ __forceinline__ CachePlan(const CacheAttentionArgs &a, int lane)
    {
        if (a.plan) {
            mine = CacheSpan{0, 0, 0, 0};
            run = a.plan[0];
            runs = a.plan[1];
            cross = a.plan[2] != 0;
            return;
        }
        mine = lane < a.batch ? cache_span(a, lane) : CacheSpan{0, 0, 0, 0};
        find_runs(a, [&](int size) {
            int n = runs_of(mine.steps, size);
            for (int b = lane + 64; b < a.batch; b += 64)
                n += runs_of(cache_span(a, b).steps, size);
            return wave_sum(n);
        });
    }

    // sum(size): runs of `size` steps that the sequences take
    template <class Sum>
    __device__ __forceinline__ void find_runs(const CacheAttentionArgs &a, Sum sum)
    {
        const int steps = sum(1);
        run = (steps + a.workers - 1) / a.workers;
        runs = a.workers;
        cross = run > kCacheCross || a.batch > a.workers;
        if (cross)
            return;
        // runs that keep to their sequences are more: lengthened until one round holds them
        runs = sum(run);
        for (int i = 0; i < 3 && runs > a.workers; ++i) {
            run += (run + 3) / 4;
            runs = sum(run);
        }
    }

    static __device__ __forceinline__ int runs_of(int steps, int size)
    {
        return size == 1 ? steps : (uint32_t)(steps + size - 1) / (uint32_t)size;
    }

    // a sequence's steps in the order of runs
    __device__ __forceinline__ int padded(int steps) const { return cross ? steps : runs_of(steps, run) * run; }

    // The workspace's place of run w's segment of sequence b, which is split.  Runs and sequences both advance;
    // of more sequences than runs a run has two places, for what goes on from the run before and for what begins
    // in it and goes on (those between are whole)
    __device__ __forceinline__ int slot(const CacheAttentionArgs &a, int w, int b, bool begins) const
    {
        return a.batch > a.workers ? 2 * w + begins : cross ? w + b : w;
    }

    // the place of the run's next segment
    static __device__ __forceinline__ int next_slot(const CacheAttentionArgs &a, int slot)
    {
        return a.batch > a.workers ? slot | 1 : slot + 1;
    }

    // The sequence that holds step `at`, its first step and span (batch: behind the last)
    __device__ __forceinline__ int find(const CacheAttentionArgs &a, int at, int lane, int &start, CacheSpan &span) const
    {
        start = 0;
        span = CacheSpan{0, 0, 0, 0};
        if (a.plan) {
            const int *starts = a.plan + kCachePlanHead;
            if (at >= starts[a.batch])
                return a.batch;
            // the last sequence that begins at `at` or before, among 64 probes at a time
            int b = 0;
            for (int count = a.batch; count > 1;) {
                const int stride = (count + 63) / 64, i = lane * stride;
                const int n = __popcll(__ballot(i < count && starts[b + (i < count ? i : 0)] <= at)) - 1;
                b += n * stride;
                count = count - n * stride < stride ? count - n * stride : stride;
            }
            start = starts[b];
            span = cache_span(a, b);
            return __builtin_amdgcn_readfirstlane(b);
        }
        int before = 0;
        CacheSpan s = mine;
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            if (b0)
                s = b0 + lane < a.batch ? cache_span(a, b0 + lane) : CacheSpan{0, 0, 0, 0};
            const int steps = padded(s.steps);
            int upto = wave_inclusive_sum(steps);
            upto += before;
            const uint64_t behind = __ballot(at < upto);
            if (behind) {
                const int src = __ffsll((unsigned long long)behind) - 1;
                start = __builtin_amdgcn_readlane(upto - steps, src);
                span.first = __builtin_amdgcn_readlane(s.first, src);
                span.base = __builtin_amdgcn_readlane(s.base, src);
                span.length = __builtin_amdgcn_readlane(s.length, src);
                span.steps = __builtin_amdgcn_readlane(s.steps, src);
                return __builtin_amdgcn_readfirstlane(b0 + src);
            }
            before = __builtin_amdgcn_readlane(upto, 63);
        }
        return a.batch;
    }
};

template <bool BF>
__device__ __forceinline__ uint2 cache_round4(float4v v)
{
    uint16_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF) {
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
