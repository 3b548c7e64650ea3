// hqq_layers_rows.hip -- the small row-wise kernels around the layers' products:
// joining split sums and the softmax blocks, scales of rows.
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
    if (!(m > -INFINITY))
        return float2{m, a.y + b.y};     // both empty (or a NaN, which stays)
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
    a.loss[m] = fmaxf(d, 0.0f) + tail;
    a.lse[m] = (d > 0.0f ? others : lt) + tail;
}

// one workgroup per row; fp16 magnitudes compare as their bits
__global__ __launch_bounds__(kRowsBlock) void row_scale_kernel(const uint16_t *rows, int64_t N, float *scale, float *inv)
{
    __shared__ uint32_t top[kRowsBlock / 64];
    const uint16_t *r = rows + (int64_t)blockIdx.x * N;
    uint32_t mx = 0;
    for (int64_t i = threadIdx.x; i < N; i += kRowsBlock) {
        const uint32_t b = r[i] & 0x7fffu;
        mx = b > mx ? b : mx;
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const uint32_t b = (uint32_t)__shfl_xor((int)mx, o);
        mx = b > mx ? b : mx;
    }
    if ((threadIdx.x & 63) == 0)
        top[threadIdx.x >> 6] = mx;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kRowsBlock / 64; ++w)
            mx = top[w] > mx ? top[w] : mx;
        float f = 1.0f;
        if (mx > 0 && mx < 0x7c00u) {
            _Float16 h;
            const uint16_t b = (uint16_t)mx;
            __builtin_memcpy(&h, &b, 2);
            int e;
            frexpf((float)h, &e);          // max = f * 2^e, f in [1/2, 1)
            f = ldexpf(1.0f, -6 - e);
        }
        scale[blockIdx.x] = f;
        inv[blockIdx.x] = 1.0f / f;
    }
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

hipError_t launch_row_scale(const uint16_t *rows, int64_t M, int64_t N, float *scale, float *inv, hipStream_t s)
{
    hipLaunchKernelGGL(row_scale_kernel, dim3((unsigned)M), dim3(kRowsBlock), 0, s, rows, N, scale, inv);
    return hipGetLastError();
}

}  // namespace hqq
