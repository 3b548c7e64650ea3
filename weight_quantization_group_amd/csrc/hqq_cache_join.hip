// hqq_cache_join.hip -- joins the items of sequences that were split over their
// length: one workgroup per sequence and query head.
#include "hqq_cache_plan.h"

namespace hqq {
namespace {

typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kJoinBlock = 256;

template <int D>
__global__ __launch_bounds__(kJoinBlock) void cache_join_kernel(CacheAttentionArgs a)
{
    constexpr int kLanes = D / 4, kGroups = kJoinBlock / kLanes;
    __shared__ float4v sums[kGroups][kLanes];
    const int head = blockIdx.x, b = blockIdx.y;
    const int lane = threadIdx.x & 63;
    const int chunk = cache_chunk(a, lane);
    const int count = cache_items(cache_span(a, b), chunk);
    if (count == 1)
        return;                       // the item wrote the output itself
    int64_t before = 0;
    for (int i = lane; i < b; i += 64)
        before += cache_items(cache_span(a, i), chunk);
    before = wave_sum(before);
    const float2 *ml = a.part_ml + before * a.q_heads + head;
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
    const int group = threadIdx.x / kLanes, at = threadIdx.x % kLanes;
    float4v v{0.f, 0.f, 0.f, 0.f};
    if (group < kGroups)
        for (int i = group; i < count; i += kGroups) {
            const float w = __builtin_amdgcn_exp2f(ml[(int64_t)i * a.q_heads].x - ref);
            v += w * *reinterpret_cast<const float4v *>(a.part + ((before + i) * a.q_heads + head) * D + 4 * at);
        }
    if (group < kGroups)
        sums[group][at] = v;
    __syncthreads();
    if (group != 0)
        return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i)
        v += sums[i][at];
    const float inv = total > 0.0f || !(total == total) ? 1.0f / total : 0.0f;
    const int64_t row = (int64_t)b * a.q_heads + head;
    *reinterpret_cast<uint2 *>(a.out + row * D + 4 * at) = cache_round4(v * inv, a.bf16);
    if (at == 0 && a.lse)
        a.lse[row] = cache_lse(m, total);
}

template <int D>
hipError_t launch_join(const CacheAttentionArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((cache_join_kernel<D>), dim3((unsigned)a.q_heads, (unsigned)a.batch), dim3(kJoinBlock), 0, s, a);
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
