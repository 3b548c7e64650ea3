// hqq_cache_join.hip -- joins the segments of sequences that were split over their
// length: one query head of one sequence per workgroup, or per wave where there are enough.
#include "hqq_cache_plan.h"

namespace hqq {
namespace {

constexpr int kJoinBlock = 256;

// WAVES: waves per query head
template <int D, int WAVES>
__global__ __launch_bounds__(kJoinBlock) void cache_join_kernel(CacheAttentionArgs a)
{
    constexpr int kLanes = D / 4;                           // lanes of a row, 4 dims each
    constexpr int kAtOnce = kJoinBlock / kLanes / (4 / WAVES);   // segments read at a time
    constexpr int kHeads = 4 / WAVES;
    __shared__ float4v sums[kHeads][kAtOnce][kLanes];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int local = wave / WAVES, thread = threadIdx.x - local * WAVES * 64;
    const int head = blockIdx.x * kHeads + local, b = blockIdx.y;
    const CachePlan plan(a, lane);
    int start = lane < b ? plan.padded(plan.mine.steps) : 0;
    for (int i = lane + 64; i < b; i += 64)
        start += plan.padded(cache_span(a, i).steps);
    start = wave_sum(start);
    const int w0 = start / plan.run;
    const int count = (start + plan.padded(cache_span(a, b).steps) - 1) / plan.run - w0 + 1;
    if (count == 1)
        return;                       // the one segment wrote the output itself
    const bool real = head < a.q_heads;
    const int64_t slot = plan.slot(w0, b);
    const float2 *ml = a.part_ml + slot * a.q_heads + (real ? head : 0);
    const float *part = a.part + (slot * a.q_heads + (real ? head : 0)) * D;
    float m = -INFINITY;
    for (int i = lane; i < count; i += 64)
        m = fmaxf(m, ml[(int64_t)i * a.q_heads].x);
#pragma unroll
    for (int o = 1; o < 64; o *= 2)
        m = fmaxf(m, __shfl_xor(m, o));
    const float ref = m == -INFINITY ? 0.0f : m;
    float total = 0.0f;
    for (int i = lane; i < count; i += 64) {
        const float2 v = ml[(int64_t)i * a.q_heads];
        total += v.y * __builtin_amdgcn_exp2f(v.x - ref);
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2)
        total += __shfl_xor(total, o);
    const int group = thread / kLanes, at = thread % kLanes;
    float4v v{0.f, 0.f, 0.f, 0.f};
    if (group < kAtOnce) {
#pragma unroll 4
        for (int i = group; i < count; i += kAtOnce) {
            const float w = __builtin_amdgcn_exp2f(ml[(int64_t)i * a.q_heads].x - ref);
            v += w * *reinterpret_cast<const float4v *>(part + (int64_t)i * a.q_heads * D + 4 * at);
        }
        sums[local][group][at] = v;
    }
    __syncthreads();                  // (count is one number for all of the workgroup)
    if (group != 0 || !real)
        return;
#pragma unroll
    for (int i = 1; i < kAtOnce; ++i)
        v += sums[local][i][at];
    const int64_t row = (int64_t)b * a.q_heads + head;
    *reinterpret_cast<uint2 *>(a.out + row * D + 4 * at) =
        a.bf16 ? cache_round4<true>(v * cache_inverse(total)) : cache_round4<false>(v * cache_inverse(total));
    if (at == 0 && a.lse)
        a.lse[row] = cache_lse(m, total);
}

template <int D>
hipError_t launch_join(const CacheAttentionArgs &a, hipStream_t s)
{
    if ((int64_t)a.q_heads * a.batch > 1024)
        hipLaunchKernelGGL((cache_join_kernel<D, 1>), dim3((unsigned)((a.q_heads + 3) / 4), (unsigned)a.batch),
                           dim3(kJoinBlock), 0, s, a);
    else
        hipLaunchKernelGGL((cache_join_kernel<D, 4>), dim3((unsigned)a.q_heads, (unsigned)a.batch), dim3(kJoinBlock), 0,
                           s, a);
    return hipGetLastError();
}

}  // namespace

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
