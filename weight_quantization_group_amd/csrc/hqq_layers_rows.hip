// hqq_layers_rows.hip -- the small row-wise kernels around the layers' products:
// joining split sums and the softmax blocks, bounds of the rows' gradients.
#include "hqq_layers_epilogue.h"

namespace hqq {
namespace {

constexpr int kRowsBlock = 256;

// Parts of a split product added in a fixed order in fp32; 4 values per lane.  GR: groups
// of lanes that take a share of the parts each and join through LDS: 4 where the values
// alone would leave most of the chip idle (16 parts of 16 x 4096, 4.6 us by one
// group, 3.7 by 4).
template <bool BF, int GR>
__global__ __launch_bounds__(kRowsBlock) void reduce_kernel(ReduceArgs a)
{
    constexpr int kLanes = kRowsBlock / GR;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int64_t i = ((int64_t)blockIdx.x * kLanes + lane) * 4;
    const int64_t total = a.M * a.N;
    const int per = (a.splits + GR - 1) / GR, z0 = group * per, z1 = z0 + per < a.splits ? z0 + per : a.splits;
    float4v v{0.f, 0.f, 0.f, 0.f};
    if (i < total) {
#pragma unroll 8
        for (int z = z0; z < z1; ++z)
            v += *reinterpret_cast<const float4v *>(a.part + z * total + i);
    }
    if constexpr (GR > 1) {
        __shared__ float4v sums[GR - 1][kLanes];
        if (group > 0)
            sums[group - 1][lane] = v;
        __syncthreads();
        if (group > 0)
            return;
#pragma unroll
        for (int r = 0; r < GR - 1; ++r)
            v += sums[r][lane];
    }
    if (i >= total)
        return;
    if (a.acc_in)
        v += *reinterpret_cast<const float4v *>(a.acc_in + i);
    if (a.acc_out) {
        *reinterpret_cast<float4v *>(a.acc_out + i) = v;
        return;
    }
    const float f = row_factor(a.rowf, i / a.N);
    *reinterpret_cast<uint2 *>(a.out + i) = uint2{out2<BF>(v[0] * f, v[1] * f), out2<BF>(v[2] * f, v[3] * f)};
}

template <bool BF>
hipError_t launch_reduce_dtype(const ReduceArgs &a, hipStream_t s)
{
    const int64_t lanes = a.M * a.N / 4;
    if (a.splits >= 8 && lanes <= 256 * kRowsBlock)
        hipLaunchKernelGGL((reduce_kernel<BF, 4>), dim3((unsigned)((lanes + 63) / 64)), dim3(kRowsBlock), 0, s, a);
    else
        hipLaunchKernelGGL((reduce_kernel<BF, 1>), dim3((unsigned)((lanes + kRowsBlock - 1) / kRowsBlock)), dim3(kRowsBlock), 0,
                           s, a);
    return hipGetLastError();
}

// (max, sum) pairs of sums of exponentials; an empty one is (-inf, 0)
__device__ __forceinline__ float2 join(float2 a, float2 b)
{
    const float m = fmaxf(a.x, b.x);
    if (!(fabsf(m) < INFINITY))
        return float2{m, a.y + b.y};     // both empty, or a +inf: see stats_ref
    return float2{m, a.y * expf(a.x - m) + b.y * expf(b.x - m)};
}

// one workgroup per row
__global__ __launch_bounds__(kRowsBlock) void loss_kernel(LossArgs a)
{
    __shared__ float2 parts[kRowsBlock / 64];
    const int64_t m = blockIdx.x;
    float2 s{-INFINITY, 0.0f};
    for (int64_t b = threadIdx.x; b < a.blocks; b += kRowsBlock)
        s = join(s, a.stats[m * a.pitch + b]);
#pragma unroll
    for (int o = 1; o < 64; o *= 2)
        s = join(s, float2{__shfl_xor(s.x, o), __shfl_xor(s.y, o)});
    if ((threadIdx.x & 63) == 0)
        parts[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x != 0)
        return;
#pragma unroll
    for (int w = 1; w < kRowsBlock / 64; ++w)
        s = join(s, parts[w]);
    // lse of the others, then the target joins: with d = lse_others - l_t,
    // loss = log(1 + exp(d)), lse = l_t + loss
    const float others = s.x + logf(s.y);
    const int64_t t = a.targets[m];
    if (t < 0 || t >= a.N) {
        a.loss[m] = 0.0f;
        a.lse[m] = others;
        return;
    }
    const float lt = a.tlogit[m];
    const float d = a.N > 1 ? others - lt : -INFINITY;
    const float tail = log1pf(expf(-fabsf(d)));
    // (lse - l_t of a target of +inf is inf - inf; an infinity that the target and the others
    // share is lse)
    a.loss[m] = lt < INFINITY ? fmaxf(d, 0.0f) + tail : NAN;
    a.lse[m] = others == lt && !(fabsf(lt) < INFINITY) ? lt : (d > 0.0f ? others : lt) + tail;
}

// The workgroup's maximum and sum, in thread 0
__device__ __forceinline__ float2 max_and_sum(float mx, float sum)
{
    __shared__ float2 parts[kRowsBlock / 64];
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        mx = fmaxf(mx, __shfl_xor(mx, o));
        sum += __shfl_xor(sum, o);
    }
    if ((threadIdx.x & 63) == 0)
        parts[threadIdx.x >> 6] = float2{mx, sum};
    __syncthreads();
#pragma unroll
    for (int w = 1; w < kRowsBlock / 64; ++w) {
        mx = fmaxf(mx, parts[w].x);
        sum += parts[w].y;
    }
    return float2{mx, sum};
}

__device__ __forceinline__ float group_bound(float s, float z, float qmax)
{
    return fmaxf(fabsf(z), fabsf(qmax - z)) / fabsf(s);
}

// The first kBoundParts workgroups (if asked for) take the groups of the weights in turn: the
// largest |code - zero| / |scale| is at an end of the codes (used or not: a loose bound costs
// headroom only, of which there is plenty).  One workgroup per row follows; a
// row that is not finite makes the bound so (fp16 magnitudes compare as their bits).  Bound
// by the launch and the meta's bytes: about 5 us of an fp16 backward pass of 1 or 16 rows
// through 4096 x 11008 in groups of 64 (59 and 64 us; bf16, which needs no bound, 54 and 59).
__global__ __launch_bounds__(kRowsBlock) void grad_bound_kernel(BoundArgs a)
{
    const int parts = a.weight ? kBoundParts : 0;
    if ((int)blockIdx.x < parts) {
        float mx = 0.0f;
        const int64_t quads = a.groups / 4, first = (int64_t)blockIdx.x * kRowsBlock + threadIdx.x;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll 4
            for (int64_t i = first; i < quads; i += kBoundParts * kRowsBlock) {
                const float4 s = reinterpret_cast<const float4 *>(a.scale[w])[i];
                const float4 z = reinterpret_cast<const float4 *>(a.zero[w])[i];
                mx = fmaxf(fmaxf(mx, group_bound(s.x, z.x, a.qmax)), group_bound(s.y, z.y, a.qmax));
                mx = fmaxf(fmaxf(mx, group_bound(s.z, z.z, a.qmax)), group_bound(s.w, z.w, a.qmax));
            }
            if (first < a.groups % 4)
                mx = fmaxf(mx, group_bound(a.scale[w][4 * quads + first], a.zero[w][4 * quads + first], a.qmax));
        }
        mx = max_and_sum(mx, 0.0f).x;
        if (threadIdx.x == 0)
            a.weight[blockIdx.x] = mx;
        return;
    }
    const int64_t m = (int64_t)blockIdx.x - parts;
    const uint16_t *y = a.dY + m * a.N, *x = a.X + m * a.K;
    uint32_t top = 0;
    if (a.N % 8 == 0) {
        for (int64_t i = threadIdx.x; i < a.N / 8; i += kRowsBlock) {
            const uint4 v = reinterpret_cast<const uint4 *>(y)[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = w[j] & 0x7fffu, hi = w[j] >> 16 & 0x7fffu, b = lo > hi ? lo : hi;
                top = b > top ? b : top;
            }
        }
    } else {
        for (int64_t i = threadIdx.x; i < a.N; i += kRowsBlock) {
            const uint32_t b = y[i] & 0x7fffu;
            top = b > top ? b : top;
        }
    }
    float sum = 0.0f;
    for (int64_t i = threadIdx.x; i < a.K / 8; i += kRowsBlock) {
        const uint4 v = reinterpret_cast<const uint4 *>(x)[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sum += fabsf(from16((uint16_t)w[j], false)) + fabsf(from16((uint16_t)(w[j] >> 16), false));
    }
    const float2 r = max_and_sum(top >= 0x7c00u ? INFINITY : from16((uint16_t)top, false), sum);
    if (threadIdx.x == 0)
        a.row[m] = r.x * r.y;
}

}  // namespace

hipError_t launch_reduce(bool bf16, const ReduceArgs &a, hipStream_t s)
{
    return bf16 ? launch_reduce_dtype<true>(a, s) : launch_reduce_dtype<false>(a, s);
}

hipError_t launch_loss(const LossArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(loss_kernel, dim3((unsigned)a.M), dim3(kRowsBlock), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_bound(const BoundArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(grad_bound_kernel, dim3((unsigned)(a.M + (a.weight ? kBoundParts : 0))), dim3(kRowsBlock), 0, s, a);
    return hipGetLastError();
}

}  // namespace hqq
