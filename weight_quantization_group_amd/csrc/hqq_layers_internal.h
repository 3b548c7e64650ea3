// hqq_layers_internal.h -- declarations shared by libhqq_layers.so's own
// translation units.
#pragma once

#include "hqq_internal.h"
#include "hqq_layers.h"

namespace hqq {

constexpr int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Dequantization into the workspace, before a tiled product: weight i's n[i] rows to
// W [rows, K] row-major from row row0[i] on, columns K .. round_up(K, 64) - 1 zeroed, and
// its rows past n[i] up to round_up(n[i], 64) zeroed.  pair: two weights of one n, 32 rows
// of the first (gate) and 32 of the second (up) in turn, to 2 round_up(n, 32) rows.  In the
// same launch, matrices whose rows end inside a 64-wide step are copied with zeros up
// to its end.
constexpr int kMaxSegs = HQQ_MAX_GRADS;

struct PadJob {
    const uint16_t *src;      // [M, N]
    uint16_t *dst;            // [M, round_up(N, 64)], row pitch ldd
    int64_t M, N, ldd;
};

struct UnpackArgs {
    int count, pair;
    const uint32_t *packed[kMaxSegs];   // of the first row
    const float *scale[kMaxSegs], *zero[kMaxSegs];
    int64_t n[kMaxSegs], row0[kMaxSegs];
    int64_t K;
    int64_t wpr, gpl;         // words and groups per row
    int gshift;               // log2 of the group size
    uint16_t *W;
    int64_t ldw;
    int pads;
    PadJob pad[kMaxSegs];
};
static_assert(sizeof(UnpackArgs) <= 4096, "kernel arguments within 4 KiB");
hipError_t launch_unpack_weight(int nbits, bool bf16, const UnpackArgs &a, hipStream_t s);

// The matrix product C [M, N] of 16-bit matrices with fp32 sums, and what becomes of C:
// C = A [M, R] . B [N, R]^T, or, for the gradients (kOutStore, kOutPart), C = A . B [R, N].
// A comes in segments along R, each a matrix of its own of whole 64-wide steps; B is
// an unpacked weight (or several, one below the other).  Where padding meets in a
// step, both are zero.
constexpr int kStep = 64;            // depth of a step
// Row pitch of a matrix in the workspace that the product reads: whole steps and
// 128 bytes more, so that the rows of a tile do not all fall on the same cache
// channels (measured at pitches of 8 KB: 330 us without, 296 us with, for 2048 x
// 22016 x 4096).
constexpr int64_t pitch_for(int64_t depth) { return round_up(depth, kStep) + 64; }

// The factor of a row of the results: f[m] if given; else, if given, a loss's dloss[m]
// times mul where targets[m] is one of N classes, and 0 elsewhere; else 1.
struct RowFactor {
    const float *f, *dloss;
    const int64_t *targets;
    int64_t N;
    float mul;
};

// What bounds a row's |dG| and |dU| in fp16 (null: they are not scaled): row[m] = max |dY[m]|
// * sum |X[m]| and the parts of the largest |quotient| of the weights.
constexpr int kBoundParts = 256;
struct GradBound {
    const float *row, *weight;       // [M], [kBoundParts]
};

enum GemmOut {
    kOutStore,      // out16 = round(rowf * C)
    kOutPart,       // part[z] = C over this split's steps (fp32)
    kOutGated,      // out16 = act(C_gate) * C_up
    kOutGatedGrad,  // dG, dU from C_gate, C_up and dY, in B's order of rows
    kOutStats,      // per row and column tile: max and sum of exp of the logits
    kOutSoftGrad    // exp(C - lse) - onehot(target)
};

struct GemmArgs {
    const uint16_t *A[kMaxSegs];     // segment i: [M, 64 steps], row pitch lda[i] (below 2^23)
    int64_t lda[kMaxSegs];
    int32_t step0[kMaxSegs + 1];     // first step of each segment; step0[segs]: their number
    int segs;
    const uint16_t *B;               // [N, ldb] (gated: [2 round_up(N, 32), ldb]), or [R, ldb]
    int64_t ldb;                     // below 2^23
    int32_t M, N;
    int tile, splits;                // kOutStore, kOutPart: by gemm_gradient_tile
    int tiles_m, tiles_n, steps;     // filled by the launcher
    // outputs
    uint16_t *out;                   // [M, ldo]
    int64_t ldo;
    float *part;                     // kOutPart: [splits, M, N]
    RowFactor rowf;                  // kOutStore
    int act;
    const uint16_t *dY;              // kOutGatedGrad: [M, N]
    GradBound bound;                 // of dG and dU, which are scaled by it
    float *rinv;                     // kOutGatedGrad with a bound: 1 / the scale of each row, written
    int64_t ldy;                     // row pitch of dY
    int64_t up_off;                  // kOutGatedGrad, few rows: dU's first column in out
    int64_t fill;                    // kOutGatedGrad, kOutSoftGrad: columns N .. fill - 1 of out are zeroed
    float2 *stats;                   // kOutStats: (max, sum) of row m and column tile i at [m * blocks + i]
    int64_t blocks;
    float *tlogit;                   // kOutStats: the target's logit, where it is in this piece
    const int64_t *targets;
    const float *lse;
    int64_t n0, Nall;                // first class of this piece, and all classes
};
hipError_t launch_gemm(GemmOut out, bool bf16, GemmArgs &g, hipStream_t s);
// Column tiles of a kOutStats product (at most (N + 127) / 128).
int64_t gemm_stats_blocks(int64_t M, int64_t N, int64_t steps);
// The estimated time of a product that is not split.
double gemm_us(int64_t M, int64_t N, int64_t steps);
// The tile and the splits of the steps (none of them empty) for a kOutStore or kOutPart
// product.
void gemm_gradient_tile(int64_t M, int64_t N, int64_t steps, int &tile, int &splits);

// Few rows, straight from the packed codes (hqq_layers_skinny.h): C [M, N] =
// X . W_hat^T with g's fields for what becomes of it (kOutStats: 16 columns per
// block).  Gated kinds take two weights.
struct SkinnyArgs {
    LinearArgs w[2];      // the weight, or gate and up (X, M, K, wpr, gpl, gs, gshift the same)
    GemmOut out;
    int64_t cols;         // columns to cover: N, or the padded width that out is given
    GemmArgs g;
};
hipError_t launch_skinny(int nbits, bool bf16, const SkinnyArgs &s, hipStream_t st);
hipError_t launch_skinny_pair(int nbits, bool bf16, const SkinnyArgs &s, hipStream_t st);

// Few rows: C [M, K] = sum_i A_i . W_hat_i (hqq_layers_skinny_grad.hip), as
// round(rowf * C) in out, or as the splits' parts [splits, M, K].
struct SkinnyGradArgs {
    int count;
    const uint32_t *packed[kMaxSegs];
    const float *scale[kMaxSegs], *zero[kMaxSegs];
    const uint16_t *A[kMaxSegs];     // [M, n[i]], row pitch lda[i]
    int64_t lda[kMaxSegs];
    int32_t n[kMaxSegs];
    int32_t step0[kMaxSegs + 1];     // first 32-row step of each weight
    int64_t M, K, wpr, gpl;
    int gshift, splits, steps;       // steps: filled by the launcher
    float *part;
    uint16_t *out;
    RowFactor rowf;
};
hipError_t launch_skinny_grad(int nbits, bool bf16, SkinnyGradArgs &a, hipStream_t s);
int skinny_grad_splits(int64_t M, int64_t K, int64_t steps);

// Sum of the parts: v = sum_z part[z] (+ acc_in), then out = round(rowf * v),
// or acc_out = v.  M x N values, N a multiple of 4.
struct ReduceArgs {
    const float *part;
    int splits;
    int64_t M, N;
    const float *acc_in;
    float *acc_out;
    uint16_t *out;
    RowFactor rowf;
};
hipError_t launch_reduce(bool bf16, const ReduceArgs &a, hipStream_t s);

// Cross entropy, the end: the blocks' (max, sum) of each row, then loss and lse.
struct LossArgs {
    const float2 *stats;      // [M, pitch], of which blocks are set
    int64_t pitch, blocks, M, N;
    const float *tlogit;
    const int64_t *targets;
    float *loss, *lse;
};
hipError_t launch_loss(const LossArgs &a, hipStream_t s);

// A GradBound's arrays; weight is null where its parts are there already.
struct BoundArgs {
    const uint16_t *X, *dY;          // [M, K], [M, N], fp16
    int64_t M, K, N;
    float *row;
    const float *scale[2], *zero[2]; // of gate and up, groups of each
    int64_t groups;
    float qmax;
    float *weight;
};
hipError_t launch_grad_bound(const BoundArgs &a, hipStream_t s);

}  // namespace hqq
