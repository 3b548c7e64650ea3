// hqq_layers_unpack.hip -- a weight's W_hat, written to the workspace for the products of
// many rows.
//
// W_hat is bit for bit what the dequantize kernel writes (the fp64 product of
// hqq_linear_dev.h in place of the division).  A lane takes one run of 8 consecutive
// k in each of 8 rows n; the 64 lanes of a wave are 8 x 8 such squares and the four
// waves of a workgroup lie side by side along k, so that each row of codes is read,
// and each row of W written, in stretches of 128 bytes or more.  Workgroups go to the
// 8 XCDs in turn; each XCD gets a contiguous part of them, so that the lines of codes,
// scales and zeros that neighbours along k share are fetched into one L2 only.  Bound
// by the bytes: 49 us for the 90 M weights of a 4096 x 11008 pair at 4 bits in groups
// of 64, 180 MB written and 56 read, 4.8 TB/s where a large copy reaches 5.2.  The SH
// lanes of a row that work in one group (8 in groups of 64 and more) fetch and invert the
// scales of 8 / SH rows each and share them; without that the same took 64 us.
#include "hqq_layers_epilogue.h"

namespace hqq {
namespace {

constexpr int kUnpackWaves = 4;

// 16 bytes of a padded copy per lane; the job's workgroups go over it in turn
__device__ void pad_rows(const PadJob &p)
{
    const int64_t runs = (p.N + 63) / 64 * 8, total = p.M * runs;
    for (int64_t i = (int64_t)blockIdx.x * (kUnpackWaves * 64) + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * (kUnpackWaves * 64)) {
        const int64_t m = i / runs, n = (i - m * runs) * 8;
        const uint16_t *src = p.src + m * p.N + n;
        uint32_t w[4];
        if (n + 8 <= p.N && ((uintptr_t)src & 15u) == 0) {
            const uint4 u = *reinterpret_cast<const uint4 *>(src);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = n + 2 * j < p.N ? src[2 * j] : 0u;
                const uint32_t hi = n + 2 * j + 1 < p.N ? src[2 * j + 1] : 0u;
                w[j] = lo | hi << 16;
            }
        }
        *reinterpret_cast<uint4 *>(p.dst + m * p.ldd + n) = uint4{w[0], w[1], w[2], w[3]};
    }
}

// grid: y over the weights, then the copies; x over the largest weight's squares, a
// multiple of 8.  (A flat grid with a table of first workgroups costs loads of arguments
// that wait for one another: 3 us of a
// 26 us gated block, 333 rows through 1056 x 2753.)
template <int NB, bool BF, int SH>
__global__ __launch_bounds__(kUnpackWaves * 64) void unpack_kernel(UnpackArgs a)
{
    constexpr uint32_t MASK = (1u << NB) - 1u;
    const int which = (int)blockIdx.y;
    if (which >= a.count) {
        pad_rows(a.pad[which - a.count]);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int kl = lane & 7, nl = lane >> 3;
    const int64_t an = a.n[which];
    const uint32_t kblocks = (uint32_t)((a.K + 64 * kUnpackWaves - 1) / (64 * kUnpackWaves));
    // this workgroup's place in the order of its XCD
    const uint32_t T = kblocks * (uint32_t)((an + 63) / 64), q = T / 8, rest = T % 8, x = blockIdx.x % 8;
    if (blockIdx.x >= T)
        return;
    const uint32_t id = x * q + (x < rest ? x : rest) + blockIdx.x / 8, nb = id / kblocks;
    const int64_t run = (int64_t)((id - nb * kblocks) * kUnpackWaves + wave) * 8 + kl;   // 8-k run of the row
    const int64_t n0 = (int64_t)nb * 64 + 8 * nl;
    const int64_t runs = a.K / 8;
    const bool k_in = run < runs;
    const int64_t rows = round_up(an, a.pair ? 32 : 64);      // those past n are zeroed
    if (n0 >= rows || run * 8 >= round_up(a.K, 64))
        return;

    const int64_t r = k_in ? run : runs - 1;
    double R[8];
    float Z[8];
    {
        float sc[8 / SH], ze[8 / SH];
#pragma unroll
        for (int i = 0; i < 8 / SH; ++i) {
            const int64_t nr = n0 + SH * i + (kl & (SH - 1)), n = nr < an ? nr : an - 1;
            const int64_t g = n * a.gpl + ((8 * r) >> a.gshift);
            sc[i] = a.scale[which][g];
            ze[i] = a.zero[which][g];
        }
        row_meta<SH>(sc, ze, R, Z);
    }
    uint32_t v[8][4];     // row i: 8 values of the run
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + i < an ? n0 + i : an - 1;
        const uint8_t *p = reinterpret_cast<const uint8_t *>(a.packed[which] + n * a.wpr) + r * NB;
        uint32_t w[2] = {0, 0};
        if constexpr (NB == 8) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x;
            w[1] = u.y;
        } else if constexpr (NB == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else if constexpr (NB == 2) {
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        } else {
            w[0] = *p;
        }
        const bool in = k_in && n0 + i < an;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int b0 = 2 * j * NB, b1 = (2 * j + 1) * NB;
            const float x = wq((float)((w[b0 / 32] >> (b0 % 32)) & MASK), Z[i], R[i]);
            const float y = wq((float)((w[b1 / 32] >> (b1 % 32)) & MASK), Z[i], R[i]);
            v[i][j] = in ? out2<BF>(x, y) : 0u;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (n0 + i < rows) {
            const int64_t n = n0 + i, row = a.pair ? (n >> 5) * 64 + (n & 31) + 32 * which : a.row0[which] + n;
            *reinterpret_cast<uint4 *>(a.W + row * a.ldw + run * 8) = uint4{v[i][0], v[i][1], v[i][2], v[i][3]};
        }
}

template <int NB, bool BF>
hipError_t launch_nb(const UnpackArgs &a, hipStream_t s)
{
    if (a.count + a.pads == 0)
        return hipSuccess;
    int64_t n = a.count ? 0 : 64 * 64;                // copies alone: 64 rows of squares
    for (int i = 0; i < a.count; ++i)
        n = a.n[i] > n ? a.n[i] : n;
    const int64_t squares = (a.K + 64 * kUnpackWaves - 1) / (64 * kUnpackWaves) * ((n + 63) / 64);
    const dim3 grid((unsigned)round_up(squares, 8), (unsigned)(a.count + a.pads));
    switch (a.gshift) {
    case 3: hipLaunchKernelGGL((unpack_kernel<NB, BF, 1>), grid, dim3(kUnpackWaves * 64), 0, s, a); break;
    case 4: hipLaunchKernelGGL((unpack_kernel<NB, BF, 2>), grid, dim3(kUnpackWaves * 64), 0, s, a); break;
    case 5: hipLaunchKernelGGL((unpack_kernel<NB, BF, 4>), grid, dim3(kUnpackWaves * 64), 0, s, a); break;
    default: hipLaunchKernelGGL((unpack_kernel<NB, BF, 8>), grid, dim3(kUnpackWaves * 64), 0, s, a);
    }
    return hipGetLastError();
}

template <bool BF>
hipError_t launch_bits(int nbits, const UnpackArgs &a, hipStream_t s)
{
    switch (nbits) {
    case 1: return launch_nb<1, BF>(a, s);
    case 2: return launch_nb<2, BF>(a, s);
    case 4: return launch_nb<4, BF>(a, s);
    case 8: return launch_nb<8, BF>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_unpack_weight(int nbits, bool bf16, const UnpackArgs &a, hipStream_t s)
{
    return bf16 ? launch_bits<true>(nbits, a, s) : launch_bits<false>(nbits, a, s);
}

}  // namespace hqq
