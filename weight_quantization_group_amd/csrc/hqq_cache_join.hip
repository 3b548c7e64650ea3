// hqq_cache_join.hip -- the plan of many sequences, and the join of the segments of those that were
// split over their length: one query head of one sequence per workgroup, or per wave where there are
// enough.
#include "hqq_cache_plan.h"

namespace hqq {
namespace {

constexpr int kJoinBlock = 256;
constexpr int kPlanBlock = 1024;

// One workgroup: the runs, and where each sequence begins in their order
__global__ __launch_bounds__(kPlanBlock) void cache_plan_kernel(CacheAttentionArgs a)
{
    constexpr int kWaves = kPlanBlock / 64;
    __shared__ int sums[2][kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int turn = 0;
    // the workgroup's sum of v, and of the threads before this one
    const auto scan = [&](int v, int &before) {
        const int upto = wave_inclusive_sum(v);
        int (&by_wave)[kWaves] = sums[turn];
        turn ^= 1;                    // (two in turn: one barrier each)
        if (lane == 63)
            by_wave[wave] = upto;
        __syncthreads();
        int all = 0;
        before = upto - v;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            before += w < wave ? by_wave[w] : 0;
            all += by_wave[w];
        }
        return all;
    };
    CachePlan plan;
    plan.find_runs(a, [&](int size) {
        int n = 0, before;
        for (int b = threadIdx.x; b < a.batch; b += kPlanBlock)
            n += CachePlan::runs_of(cache_span(a, b).steps, size);
        return scan(n, before);
    });
    if (threadIdx.x == 0) {
        a.plan[0] = plan.run;
        a.plan[1] = plan.runs;
        a.plan[2] = plan.cross;
    }
    int *starts = a.plan + kCachePlanHead;
    int total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanBlock) {
        const int b = b0 + (int)threadIdx.x;
        int before;
        const int all = scan(b < a.batch ? plan.padded(cache_span(a, b).steps) : 0, before);
        if (b < a.batch)
            starts[b] = total + before;
        total += all;
    }
    if (threadIdx.x == 0)
        starts[a.batch] = total;
}

// WAVES: waves per query head
template <int D, int WAVES>
struct Join {
    static constexpr int kLanes = D / 4;                                    // lanes of a row, 4 dims each
    static constexpr int kAtOnce = kJoinBlock / kLanes / (4 / WAVES);       // segments read at a time
    static constexpr int kHeads = 4 / WAVES;
    typedef float4v Shared[kHeads][kAtOnce][kLanes];

    // Sequence b of `steps` steps (in the order of runs), which begins at step `start`: whole waves, all
    // of the workgroup
    static __device__ __forceinline__ void sequence(const CacheAttentionArgs &a, const CachePlan &plan, int b, int start,
                                                    int steps, Shared &sums)
    {
        const int w0 = start / plan.run, count = (start + steps - 1) / plan.run - w0 + 1;
        if (count == 1)
            return;                   // the one segment wrote the output itself
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int local = wave / WAVES, thread = threadIdx.x - local * WAVES * 64;
        const int head = blockIdx.x * kHeads + local;
        const bool real = head < a.q_heads;
        // Segment i lies `at` places behind these: i or, where a run has two places, the first one's second and
        // the others' first
        const int two = a.batch > a.workers, step = 1 + two;
        const int64_t row0 = (int64_t)(plan.slot(a, w0, b, true) - two) * a.q_heads + (real ? head : 0);
        const float2 *ml = a.part_ml + row0;
        const float *part = a.part + row0 * D;
        float m = -INFINITY;
        for (int i = lane, at = i ? step * i : two; i < count; i += 64, at = step * i)
            m = fmaxf(m, ml[(int64_t)at * a.q_heads].x);
#pragma unroll
        for (int o = 1; o < 64; o *= 2)
            m = fmaxf(m, __shfl_xor(m, o));
        const float ref = m == -INFINITY ? 0.0f : m;
        float total = 0.0f;
        for (int i = lane, at = i ? step * i : two; i < count; i += 64, at = step * i) {
            const float2 v = ml[(int64_t)at * a.q_heads];
            total += v.y * __builtin_amdgcn_exp2f(v.x - ref);
        }
#pragma unroll
        for (int o = 1; o < 64; o *= 2)
            total += __shfl_xor(total, o);
        const int group = thread / kLanes, dims = thread % kLanes;
        float4v v{0.f, 0.f, 0.f, 0.f};
        if (group < kAtOnce) {
#pragma unroll 4
            for (int i = group, at = i ? step * i : two; i < count; i += kAtOnce, at = step * i) {
                const float w = __builtin_amdgcn_exp2f(ml[(int64_t)at * a.q_heads].x - ref);
                v += w * *reinterpret_cast<const float4v *>(part + (int64_t)at * a.q_heads * D + 4 * dims);
            }
            sums[local][group][dims] = v;
        }
        __syncthreads();              // (count is one number for all of the workgroup)
        if (group == 0 && real) {
#pragma unroll
            for (int i = 1; i < kAtOnce; ++i)
                v += sums[local][i][dims];
            const int64_t row = (int64_t)b * a.q_heads + head;
            *reinterpret_cast<uint2 *>(a.out + row * D + 4 * dims) =
                a.bf16 ? cache_round4<true>(v * cache_inverse(total)) : cache_round4<false>(v * cache_inverse(total));
            if (dims == 0 && a.lse)
                a.lse[row] = cache_lse(m, total);
        }
    }
};

// blockIdx.y: a sequence
template <int D, int WAVES>
__global__ __launch_bounds__(kJoinBlock) void cache_join_kernel(CacheAttentionArgs a)
{
    __shared__ typename Join<D, WAVES>::Shared sums;
    const int lane = threadIdx.x & 63, b = blockIdx.y;
    const CachePlan plan(a, lane);
    int start = lane < b ? plan.padded(plan.mine.steps) : 0;
    for (int i = lane + 64; i < b; i += 64)
        start += plan.padded(cache_span(a, i).steps);
    Join<D, WAVES>::sequence(a, plan, b, wave_sum(start), plan.padded(cache_span(a, b).steps), sums);
}

// blockIdx.y: a run; the sequence that begins in it and goes on behind it, if one does
template <int D, int WAVES>
__global__ __launch_bounds__(kJoinBlock) void cache_join_runs_kernel(CacheAttentionArgs a)
{
    __shared__ typename Join<D, WAVES>::Shared sums;
    const CachePlan plan(a, 0);
    for (int w = blockIdx.y; w < plan.runs; w += gridDim.y) {
        const int from = w * plan.run, to = from + plan.run;
        int start;
        CacheSpan span;
        const int b = plan.find(a, to - 1, threadIdx.x & 63, start, span);
        if (b == a.batch || start < from || start + plan.padded(span.steps) <= to)
            continue;
        Join<D, WAVES>::sequence(a, plan, b, start, plan.padded(span.steps), sums);
        __syncthreads();              // the next one's sums go where these were
    }
}

template <int D, int WAVES>
void launch_join(const CacheAttentionArgs &a, hipStream_t s)
{
    const unsigned heads = (unsigned)((a.q_heads + 4 / WAVES - 1) / (4 / WAVES));
    if (a.plan)
        hipLaunchKernelGGL((cache_join_runs_kernel<D, WAVES>), dim3(heads, (unsigned)a.workers), dim3(kJoinBlock), 0, s, a);
    else
        hipLaunchKernelGGL((cache_join_kernel<D, WAVES>), dim3(heads, (unsigned)a.batch), dim3(kJoinBlock), 0, s, a);
}

template <int D>
hipError_t launch_join(const CacheAttentionArgs &a, hipStream_t s)
{
    if ((int64_t)a.q_heads * (a.plan ? a.workers : a.batch) > 1024)
        launch_join<D, 1>(a, s);
    else
        launch_join<D, 4>(a, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_plan(const CacheAttentionArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(cache_plan_kernel, dim3(1), dim3(kPlanBlock), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_cache_join(int dim, const CacheAttentionArgs &a, hipStream_t s)
{
    switch (dim) {
    case 64: return launch_join<64>(a, s);
    case 96: return launch_join<96>(a, s);
    case 128: return launch_join<128>(a, s);
    case 192: return launch_join<192>(a, s);
    case 256: return launch_join<256>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace hqq
