// hqq_layers_abi.cpp -- the C ABI of include/hqq_layers.h: argument checks, the
// workspace layouts, and the order of the launches.  No allocation, no state.
#include "hqq_layers_internal.h"

#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <initializer_list>

namespace {

using namespace hqq;

constexpr int64_t kMaxRows = int64_t(1) << 20;
constexpr int64_t kMaxDepth = int64_t(1) << 17;
constexpr int64_t kMaxWidth = int64_t(1) << 22;
constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxBytes = int64_t(1) << 31;
// The backward passes keep 16-bit gradients of this many rows at a time.
constexpr int64_t kRowChunk = 8192;

bool aligned(const void *p, unsigned to) { return p && ((uintptr_t)p & (to - 1)) == 0; }

int log2_group(int gs)
{
    for (int b = 3; b <= 8; ++b)
        if (gs == (1 << b))
            return b;
    return -1;
}

int check_sizes(int64_t M, int64_t K, int64_t N, int nbits, int group_size)
{
    if (!valid_nbits(nbits) || nbits == 3)
        return HQQ_EINVAL_NBITS;
    if (M < 1 || N < 1 || K < 32 || K % 32 != 0 || M > kMaxRows || K > kMaxDepth || N > kMaxWidth ||
        M * N > kMaxElems || N * (K * nbits / 32) * 4 >= kMaxBytes)
        return HQQ_EINVAL_SHAPE;
    if (log2_group(group_size) < 0 || K % group_size != 0)
        return HQQ_EINVAL_GROUP;
    if (N * (K / group_size) * 4 >= kMaxBytes)
        return HQQ_EINVAL_SHAPE;
    return HQQ_OK;
}

// Whether a product runs straight from the codes (which every 32 rows dequantize
// anew) or W_hat is unpacked for the tiled product.  n: all rows of its weights.
// By the rows, and for small weights, which leave the CUs room for the row blocks, by
// blocks of 32 rows times weights.  Crossovers measured on MI355X in bf16 at 1, 2, 4 and
// 8 bits in groups of 8 to 128; rows, codes / unpacked in us at 4 bits (groups of 64, and
// of 16 where they differ):
//              1024 x 2816        1024 x 32003       4096 x 11008       8192 x 28672
//   pair       128 12/15          64 39/53, 96 56/64 64 55/85, 128 94/85 96 391/496, 128 516/503
//   its grad.  64 29/29, 96 32/30 32 61/78, 48 90/80 64 119/120, 96 178/123 64 620/654
//     g16      64 30/30           32 74/96           32 92/127, 48 160/130 64 746/668
//   one grad.  64 13/15, 96 16/15 32 35/33, 48 44/34 64 38/45, 96 58/50 64 162/240, 96 253/228
//     g16                                            32 36/46, 48 50/47 64 219/248
//   head       128 14/19          32 26/34, 48 37/34 64 45/53, 96 65/53 96 251/324, 128 327/320
//   its grad.  96 25/26           32 43/45, 48 57/47 32 52/69, 48 74/70 64 327/435, 96 472/439
// (Large weights leave the last-level cache between unpacking and use; a shallow weight
// makes the few-rows kernels' ends weigh more.)
// HQQ_LAYERS_PATH=codes or =tiled in the environment, read at each call, forces one
// (tests run both), the codes up to the 256 rows beyond which the rule never takes
// them: their kernels address the activations by 32-bit offsets.
enum Product { kPair, kPairGrad, kBackward, kHead, kHeadGrad };

bool straight(Product what, int64_t M, int64_t K, int64_t n, int group_size)
{
    if (M > 256)
        return false;
    if (const char *e = getenv("HQQ_LAYERS_PATH")) {
        if (strcmp(e, "codes") == 0)
            return true;
        if (strcmp(e, "tiled") == 0)
            return false;
    }
    const bool small_groups = group_size < 64, shallow = K < 2048, large = K * n > 200000000;
    int64_t rows = 0, work = 0;           // work: millions of weights times blocks of 32 rows
    switch (what) {
    case kPair: rows = large ? 96 : 64; work = 24; break;
    case kPairGrad: rows = small_groups || shallow ? 32 : 64; work = 12; break;
    case kBackward: rows = !large && (small_groups || shallow) ? 32 : 64; work = 6; break;
    case kHead: rows = large ? 96 : shallow ? 32 : 64; work = 12; break;
    case kHeadGrad: rows = large ? 64 : 32; work = 9; break;
    }
    return M <= rows || (M + 31) / 32 * K * n <= work * 1000000;
}

int check_batch(int64_t M, int64_t K, const int64_t *n, int count, int nbits, int group_size)
{
    int64_t total = 0;
    for (int i = 0; i < count; ++i) {
        if (const int st = check_sizes(M, K, n[i], nbits, group_size))
            return st;
        total += round_up(n[i], kStep);
    }
    return total > 2 * kMaxWidth ? HQQ_EINVAL_SHAPE : HQQ_OK;
}

int check_dtype(int dtype)
{
    return dtype == HQQ_DTYPE_FP16 || dtype == HQQ_DTYPE_BF16 ? HQQ_OK : HQQ_EINVAL_DTYPE;
}

bool weight_ok(const uint32_t *packed, const float *scale, const float *zero)
{
    return aligned(packed, 16) && aligned(scale, 16) && aligned(zero, 16);
}

int check_workspace(const void *ws, int64_t have, int64_t need)
{
    if (have < 0 || (!ws && have > 0) || (ws && !aligned(ws, 16)))
        return HQQ_EINVAL_PTR;
    return have < need ? HQQ_EWORKSPACE : HQQ_OK;
}

// Whether what the call writes (an output, or the workspace) shares memory with something
// that it reads or uses
struct Range {
    const void *p;
    int64_t bytes;
};

bool overlaps(Range out, std::initializer_list<Range> others)
{
    const uintptr_t a = (uintptr_t)out.p;
    for (const Range &o : others) {
        const uintptr_t b = (uintptr_t)o.p;
        if (out.bytes && o.bytes && a < b + (uint64_t)o.bytes && b < a + (uint64_t)out.bytes)
            return true;
    }
    return false;
}

// the same for the arrays of a weight [N, K]
bool overlaps_weight(std::initializer_list<Range> written, const uint32_t *packed, const float *scale, const float *zero,
                     int64_t N, int64_t K, int nbits, int group_size)
{
    const int64_t codes = N * (K * nbits / 32) * 4, meta = N * (K / group_size) * 4;
    for (const Range &r : written)
        if (overlaps(r, {{packed, codes}, {scale, meta}, {zero, meta}}))
            return true;
    return false;
}

bool overlaps_weight(std::initializer_list<Range> written, const hqq_weight &w, int64_t N, int64_t K, int nbits,
                     int group_size)
{
    return overlaps_weight(written, w.packed, w.scale, w.zero, N, K, nbits, group_size);
}

// The workspace as a run of 256-byte aligned arrays; with a null base only
// their sizes count.
struct Carve {
    char *base;
    int64_t at = 0;
    explicit Carve(void *p) : base((char *)p) {}
    template <typename T>
    T *take(int64_t n)
    {
        T *p = base ? reinterpret_cast<T *>(base + at) : nullptr;
        at += round_up(n * (int64_t)sizeof(T), 256);
        return p;
    }
    template <typename T>
    T *take_some(int64_t n)        // null for none
    {
        return n ? take<T>(n) : nullptr;
    }
};

UnpackArgs unpack_args(uint16_t *W, int64_t K, int nbits, int group_size)
{
    UnpackArgs a{};
    a.wpr = K * nbits / 32;
    a.gpl = K / group_size;
    a.K = K;
    a.gshift = log2_group(group_size);
    a.W = W;
    a.ldw = pitch_for(K);
    return a;
}

// rows first .. first + n - 1 of a weight, to W's row `row` (a pair's rows go in turn)
void unpack_rows(UnpackArgs &a, const uint32_t *packed, const float *scale, const float *zero, int64_t first, int64_t n,
                 int64_t row)
{
    const int i = a.count++;
    a.packed[i] = packed + first * a.wpr;
    a.scale[i] = scale + first * a.gpl;
    a.zero[i] = zero + first * a.gpl;
    a.n[i] = n;
    a.row0[i] = row;
}

// floats of partial sums that a product of up to M rows by N columns may need (the
// largest over the row chunks: whole ones and the last); one part is needed only where
// its sums are carried on
int64_t part_floats(int64_t M, int64_t N, int64_t steps, bool carried)
{
    int64_t most = 0;
    for (const int64_t m : {M < kRowChunk ? M : kRowChunk, M % kRowChunk})
        if (m > 0) {
            int tile, splits;
            gemm_gradient_tile(m, N, steps, tile, splits);
            const int64_t f = splits > 1 || carried ? (int64_t)splits * m * N : 0;
            most = f > most ? f : most;
        }
    return most;
}

// A [m, depth] for a product: itself, or where its rows end inside a step (pad: room
// for that) its padded copy, which the unpacking launch makes
const uint16_t *whole_steps(UnpackArgs &a, const uint16_t *A, int64_t m, int64_t depth, uint16_t *pad)
{
    if (!pad)
        return A;
    a.pad[a.pads++] = PadJob{A, pad, m, depth, pitch_for(depth)};
    return pad;
}

int64_t pad_values(int64_t m, int64_t depth) { return depth % kStep ? m * pitch_for(depth) : 0; }

// row pitch of an A that whole_steps has seen
int64_t whole_pitch(int64_t depth) { return depth % kStep ? pitch_for(depth) : depth; }

// one segment of whole steps
void single_segment(GemmArgs &g, const uint16_t *A, int64_t depth, int64_t pitch)
{
    g.A[0] = A;
    g.lda[0] = pitch;
    g.step0[0] = 0;
    g.step0[1] = (int32_t)(depth / kStep);
    g.segs = 1;
    g.splits = 1;
}

// dX [M, K] = rowf * (A . W): in one launch, or by split sums and a second;
// acc: fp32 sums carried between pieces (null: one piece)
hipError_t gradient_product(GemmArgs &g, bool bf16, float *part, float *acc, bool first, bool last, uint16_t *dX,
                            const RowFactor &rowf, hipStream_t s)
{
    const int64_t M = g.M, K = g.N;
    gemm_gradient_tile(M, K, g.step0[g.segs], g.tile, g.splits);
    if (g.splits == 1 && first && last) {
        g.out = dX;
        g.ldo = K;
        g.rowf = rowf;
        return launch_gemm(kOutStore, bf16, g, s);
    }
    g.part = part;
    if (const hipError_t e = launch_gemm(kOutPart, bf16, g, s))
        return e;
    ReduceArgs r{};
    r.part = part;
    r.splits = g.splits;
    r.M = M;
    r.N = K;
    r.acc_in = first ? nullptr : acc;
    r.acc_out = last ? nullptr : acc;
    r.out = dX;
    r.rowf = rowf;
    return launch_reduce(bf16, r, s);
}

LinearArgs linear_args(const uint16_t *X, const hqq_weight &w, int64_t M, int64_t K, int64_t N, int nbits, int group_size)
{
    LinearArgs a{};
    a.X = X;
    a.packed = w.packed;
    a.scale = w.scale;
    a.zero = w.zero;
    a.M = M;
    a.N = N;
    a.K = K;
    a.wpr = K * nbits / 32;
    a.gpl = K / group_size;
    a.gs = group_size;
    a.gshift = log2_group(group_size);
    return a;
}

// the weights and gradients of a few-rows backward product
void add_grad(SkinnyGradArgs &a, const uint32_t *packed, const float *scale, const float *zero, const uint16_t *A,
              int64_t lda, int64_t n)
{
    const int i = a.count++;
    a.packed[i] = packed;
    a.scale[i] = scale;
    a.zero[i] = zero;
    a.A[i] = A;
    a.lda[i] = lda;
    a.n[i] = (int32_t)n;
    a.step0[i + 1] = a.step0[i] + (int32_t)((n + 31) / 32);
}

int64_t sum_of(const int64_t *n, int count)
{
    int64_t t = 0;
    for (int i = 0; i < count; ++i)
        t += n[i];
    return t;
}

// 32-row steps of the widths n
int64_t grad_steps(const int64_t *n, int count)
{
    int64_t t = 0;
    for (int i = 0; i < count; ++i)
        t += (n[i] + 31) / 32;
    return t;
}

int64_t few_part_floats(int64_t M, int64_t K, int64_t steps)
{
    const int sp = skinny_grad_splits(M, K, steps);
    return sp > 1 ? sp * M * K : 0;
}

hipError_t few_rows_gradient(SkinnyGradArgs &a, bool bf16, int nbits, int group_size, int64_t M, int64_t K, float *part,
                             uint16_t *dX, const RowFactor &rowf, hipStream_t s)
{
    a.M = M;
    a.K = K;
    a.wpr = K * nbits / 32;
    a.gpl = K / group_size;
    a.gshift = log2_group(group_size);
    a.splits = skinny_grad_splits(M, K, a.step0[a.count]);
    a.out = dX;
    a.rowf = rowf;
    a.part = a.splits > 1 ? part : nullptr;
    if (const hipError_t e = launch_skinny_grad(nbits, bf16, a, s))
        return e;
    if (a.splits == 1)
        return hipSuccess;
    ReduceArgs r{};
    r.part = part;
    r.splits = a.splits;
    r.M = M;
    r.N = K;
    r.out = dX;
    r.rowf = rowf;
    return launch_reduce(bf16, r, s);
}

// ---------------------------------------------------------------------------
// layouts
// ---------------------------------------------------------------------------

struct GatedLayout {
    uint16_t *W, *X;
    int64_t bytes;
    GatedLayout(void *p, int64_t M, int64_t K, int64_t N, bool few)
    {
        Carve c(p);
        W = X = nullptr;
        if (!few) {
            W = c.take<uint16_t>(2 * round_up(N, 32) * pitch_for(K));
            X = c.take_some<uint16_t>(pad_values(M, K));
        }
        bytes = c.at;
    }
};

struct GatedGradLayout {
    uint16_t *W, *dGU, *X;
    float *row, *weight, *inv, *part;     // row, weight: a GradBound's
    int64_t bytes;
    GatedGradLayout(void *p, int64_t M, int64_t K, int64_t N, bool few)
    {
        const int64_t Np = round_up(N, 32), mc = M < kRowChunk ? M : kRowChunk;
        Carve c(p);
        W = X = nullptr;
        if (!few) {
            W = c.take<uint16_t>(2 * Np * pitch_for(K));
            X = c.take_some<uint16_t>(pad_values(mc, K));
        }
        dGU = c.take<uint16_t>(mc * pitch_for(2 * Np));
        row = c.take<float>(mc);
        weight = c.take<float>(kBoundParts);
        inv = c.take<float>(mc);
        const int64_t n[2] = {N, N};
        part = c.take_some<float>(few ? few_part_floats(M, K, grad_steps(n, 2))
                                      : part_floats(M, K, 2 * Np / kStep, false));
        bytes = c.at;
    }
};

struct BatchGradLayout {
    uint16_t *W, *pad[HQQ_MAX_GRADS];
    float *part;
    int64_t bytes;
    BatchGradLayout(void *p, int64_t M, int64_t K, const int64_t *n, int count, bool few)
    {
        const int64_t mc = M < kRowChunk ? M : kRowChunk;
        Carve c(p);
        W = nullptr;
        if (few) {
            part = c.take_some<float>(few_part_floats(M, K, grad_steps(n, count)));
            bytes = c.at;
            return;
        }
        int64_t rows = 0;
        for (int i = 0; i < count; ++i)
            rows += round_up(n[i], kStep);
        W = c.take<uint16_t>(rows * pitch_for(K));
        for (int i = 0; i < count; ++i)
            pad[i] = c.take_some<uint16_t>(pad_values(mc, n[i]));
        part = c.take_some<float>(part_floats(M, K, rows / kStep, false));
        bytes = c.at;
    }
};

// Classes per piece: W_hat of a piece takes about 128 MiB (the cache behind the L2s has
// 256 MB), `limit` classes at most.  Of the widths from 5/8 to 5/4 of that, the one whose
// products take the least time by the tiles' model: few rows and a deep head leave tens of
// tiles per piece, and a last piece of a few columns costs a whole round of them.  At most
// 65536, so that the tiles of 2^20 rows fit a grid.
int64_t loss_piece(int64_t M, int64_t K, int64_t N, int64_t limit)
{
    int64_t p = (int64_t(64) << 20) / pitch_for(K) / 256 * 256;
    p = p < limit ? p : limit;
    p = p < 4096 ? 4096 : p > 52224 ? 52224 : p;
    if (N <= p)
        return N;
    const int64_t steps = round_up(K, kStep) / kStep;
    const int64_t by = p / 8 / 256 * 256;
    double best = 0.0;
    int64_t piece = p;
    for (int64_t w = p - 3 * by; w <= p + 2 * by; w += by) {
        if (w >= N) {
            w = N;
        }
        double us = (double)(N / w) * gemm_us(M, w, steps);
        if (N % w)
            us += gemm_us(M, N % w, steps);
        if (best == 0.0 || us < best) {
            best = us;
            piece = w;
        }
        if (w == N)
            break;
    }
    return piece;
}

struct LossLayout {
    uint16_t *W, *X;
    float2 *stats;
    float *tlogit;
    int64_t bytes, piece, pitch;      // classes per piece; blocks that a row of stats has room for
    LossLayout(void *p, int64_t M, int64_t K, int64_t N, bool few)
    {
        Carve c(p);
        W = X = nullptr;
        if (!few) {
            piece = loss_piece(M, K, N, N);
            pitch = N / piece * ((piece + 127) / 128) + (N % piece + 127) / 128;
            W = c.take<uint16_t>(round_up(piece, kStep) * pitch_for(K));
            X = c.take_some<uint16_t>(pad_values(M, K));
        } else {
            piece = N;
            pitch = (N + 15) / 16;
        }
        stats = c.take<float2>(M * pitch);
        tlogit = c.take<float>(M);
        bytes = c.at;
    }
};

// of the backward pass: the 16-bit gradients of a piece's logits take at most about 64
// MiB (beside W_hat's in the cache)
int64_t loss_grad_piece(int64_t m, int64_t K, int64_t N)
{
    return loss_piece(m, K, N, (int64_t(32) << 20) / m / 256 * 256);
}

struct LossGradLayout {
    uint16_t *W, *dL, *X;
    float *part, *acc;
    int64_t bytes, piece, ldl;
    LossGradLayout(void *p, int64_t M, int64_t K, int64_t N, bool few)
    {
        const int64_t mc = M < kRowChunk ? M : kRowChunk;
        Carve c(p);
        W = X = nullptr;
        acc = nullptr;
        if (few) {
            piece = N;
            ldl = round_up(N, kStep);
            dL = c.take<uint16_t>(M * ldl);
            part = c.take_some<float>(few_part_floats(M, K, grad_steps(&N, 1)));
            bytes = c.at;
            return;
        }
        piece = loss_grad_piece(mc, K, N);
        ldl = pitch_for(piece);
        W = c.take<uint16_t>(round_up(piece, kStep) * pitch_for(K));
        dL = c.take<uint16_t>(mc * ldl);
        X = c.take_some<uint16_t>(pad_values(mc, K));
        int64_t f = part_floats(M, K, (piece + kStep - 1) / kStep, piece < N);
        const int64_t rest = N % piece;
        if (rest) {
            const int64_t f2 = part_floats(M, K, (rest + kStep - 1) / kStep, true);
            f = f2 > f ? f2 : f;
        }
        part = c.take_some<float>(f);
        acc = c.take<float>(piece < N ? mc * K : 0);
        bytes = c.at;
    }
};

}  // namespace

extern "C" {

const char *hqq_layers_strerror(int status)
{
    switch (status) {
    case HQQ_OK: return "ok";
    case HQQ_EINVAL_NBITS: return "nbits must be 1, 2, 4 or 8";
    case HQQ_EINVAL_GROUP: return "group_size must be 8, 16, 32, 64, 128 or 256 and divide K";
    case HQQ_EINVAL_SHAPE: return "a size is out of range (K a multiple of 32; M, N, count >= 1 and within their limits)";
    case HQQ_EINVAL_PTR: return "a pointer is NULL or misaligned, or an output or the workspace overlaps an input or one another";
    case HQQ_EHIP: return "a HIP kernel launch failed";
    case HQQ_EINVAL_DTYPE: return "dtype must be HQQ_DTYPE_FP16 or HQQ_DTYPE_BF16";
    case HQQ_EINVAL_ACT: return "act must be HQQ_ACT_SILU, HQQ_ACT_GELU or HQQ_ACT_GELU_TANH";
    case HQQ_EWORKSPACE: return "the workspace is smaller than this call needs";
    default: return "unknown status";
    }
}

int64_t hqq_linear_gated_workspace(int64_t M, int64_t K, int64_t N, int nbits, int group_size)
{
    if (const int st = check_sizes(M, K, N, nbits, group_size))
        return st;
    return GatedLayout(nullptr, M, K, N, straight(kPair, M, K, 2 * N, group_size)).bytes;
}

int hqq_linear_gated(const uint16_t *X, int64_t M, int64_t K, const hqq_weight *gate, const hqq_weight *up, int64_t N,
                     int nbits, int group_size, int dtype, int act, uint16_t *Y, void *workspace,
                     int64_t workspace_bytes, void *stream)
{
    if (const int st = check_sizes(M, K, N, nbits, group_size))
        return st;
    if (const int st = check_dtype(dtype))
        return st;
    if (act < HQQ_ACT_SILU || act > HQQ_ACT_GELU_TANH)
        return HQQ_EINVAL_ACT;
    if (!gate || !up || !weight_ok(gate->packed, gate->scale, gate->zero) || !weight_ok(up->packed, up->scale, up->zero) ||
        !aligned(X, 16) || !aligned(Y, 16))
        return HQQ_EINVAL_PTR;
    const bool few = straight(kPair, M, K, 2 * N, group_size);
    const GatedLayout l(workspace, M, K, N, few);
    if (const int st = check_workspace(workspace, workspace_bytes, l.bytes))
        return st;
    const Range rx{X, 2 * M * K}, ry{Y, 2 * M * N}, rw{workspace, l.bytes};
    if (overlaps(ry, {rx, rw}) || overlaps(rw, {rx}) || overlaps_weight({ry, rw}, *gate, N, K, nbits, group_size) ||
        overlaps_weight({ry, rw}, *up, N, K, nbits, group_size))
        return HQQ_EINVAL_PTR;
    const bool bf16 = dtype == HQQ_DTYPE_BF16;
    const hipStream_t s = (hipStream_t)stream;
    if (few) {
        SkinnyArgs f{};
        f.w[0] = linear_args(X, *gate, M, K, N, nbits, group_size);
        f.w[1] = linear_args(X, *up, M, K, N, nbits, group_size);
        f.out = kOutGated;
        f.cols = N;
        f.g.M = (int32_t)M;
        f.g.N = (int32_t)N;
        f.g.out = Y;
        f.g.ldo = N;
        f.g.act = act;
        return launch_skinny(nbits, bf16, f, s) == hipSuccess ? HQQ_OK : HQQ_EHIP;
    }
    UnpackArgs a = unpack_args(l.W, K, nbits, group_size);
    a.pair = 1;
    unpack_rows(a, gate->packed, gate->scale, gate->zero, 0, N, 0);
    unpack_rows(a, up->packed, up->scale, up->zero, 0, N, 0);
    GemmArgs g{};
    single_segment(g, whole_steps(a, X, M, K, l.X), round_up(K, kStep), whole_pitch(K));
    g.B = l.W;
    g.ldb = a.ldw;
    g.M = (int32_t)M;
    g.N = (int32_t)N;
    g.out = Y;
    g.ldo = N;
    g.act = act;
    return launch_unpack_weight(nbits, bf16, a, s) == hipSuccess && launch_gemm(kOutGated, bf16, g, s) == hipSuccess
               ? HQQ_OK
               : HQQ_EHIP;
}

int64_t hqq_linear_gated_backward_workspace(int64_t M, int64_t K, int64_t N, int nbits, int group_size)
{
    if (const int st = check_sizes(M, K, N, nbits, group_size))
        return st;
    return GatedGradLayout(nullptr, M, K, N, straight(kPairGrad, M, K, 2 * N, group_size)).bytes;
}

int hqq_linear_gated_backward(const uint16_t *dY, const uint16_t *X, int64_t M, int64_t K, const hqq_weight *gate,
                              const hqq_weight *up, int64_t N, int nbits, int group_size, int dtype, int act,
                              uint16_t *dX, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (const int st = check_sizes(M, K, N, nbits, group_size))
        return st;
    if (const int st = check_dtype(dtype))
        return st;
    if (act < HQQ_ACT_SILU || act > HQQ_ACT_GELU_TANH)
        return HQQ_EINVAL_ACT;
    if (!gate || !up || !weight_ok(gate->packed, gate->scale, gate->zero) || !weight_ok(up->packed, up->scale, up->zero) ||
        !aligned(X, 16) || !aligned(dY, 16) || !aligned(dX, 16))
        return HQQ_EINVAL_PTR;
    const bool few = straight(kPairGrad, M, K, 2 * N, group_size);
    const GatedGradLayout l(workspace, M, K, N, few);
    if (const int st = check_workspace(workspace, workspace_bytes, l.bytes))
        return st;
    const Range rx{X, 2 * M * K}, ry{dY, 2 * M * N}, rd{dX, 2 * M * K}, rw{workspace, l.bytes};
    if (overlaps(rd, {rx, ry, rw}) || overlaps(rw, {rx, ry}) ||
        overlaps_weight({rd, rw}, *gate, N, K, nbits, group_size) || overlaps_weight({rd, rw}, *up, N, K, nbits, group_size))
        return HQQ_EINVAL_PTR;
    const bool bf16 = dtype == HQQ_DTYPE_BF16;
    const hipStream_t s = (hipStream_t)stream;
    const int64_t Np = round_up(N, 32), ldg = pitch_for(2 * Np);
    // fp16: dG and dU relative to a bound of the row's (bf16 has fp32's range)
    auto bound_rows = [&](int64_t m0, int64_t m) {
        if (bf16)
            return hipSuccess;
        BoundArgs b{X + m0 * K, dY + m0 * N, m, K, N, l.row};
        b.scale[0] = gate->scale;
        b.scale[1] = up->scale;
        b.zero[0] = gate->zero;
        b.zero[1] = up->zero;
        b.groups = N * (K / group_size);
        b.qmax = (float)((1 << nbits) - 1);
        b.weight = m0 == 0 ? l.weight : nullptr;
        return launch_grad_bound(b, s);
    };
    const GradBound bound = bf16 ? GradBound{} : GradBound{l.row, l.weight};
    if (few) {
        if (bound_rows(0, M) != hipSuccess)
            return HQQ_EHIP;
        SkinnyArgs f{};
        f.w[0] = linear_args(X, *gate, M, K, N, nbits, group_size);
        f.w[1] = linear_args(X, *up, M, K, N, nbits, group_size);
        f.out = kOutGatedGrad;
        f.cols = Np;
        f.g.M = (int32_t)M;
        f.g.N = (int32_t)N;
        f.g.out = l.dGU;
        f.g.ldo = ldg;
        f.g.fill = f.g.up_off = Np;
        f.g.act = act;
        f.g.dY = dY;
        f.g.ldy = N;
        f.g.bound = bound;
        f.g.rinv = l.inv;
        SkinnyGradArgs b{};
        add_grad(b, gate->packed, gate->scale, gate->zero, l.dGU, ldg, N);
        add_grad(b, up->packed, up->scale, up->zero, l.dGU + Np, ldg, N);
        return launch_skinny(nbits, bf16, f, s) == hipSuccess &&
                       few_rows_gradient(b, bf16, nbits, group_size, M, K, l.part, dX, RowFactor{bf16 ? nullptr : l.inv}, s) ==
                           hipSuccess
                   ? HQQ_OK
                   : HQQ_EHIP;
    }
    for (int64_t m0 = 0; m0 < M; m0 += kRowChunk) {
        const int64_t m = M - m0 < kRowChunk ? M - m0 : kRowChunk;
        if (bound_rows(m0, m) != hipSuccess)
            return HQQ_EHIP;
        UnpackArgs a = unpack_args(l.W, K, nbits, group_size);
        a.pair = 1;
        if (m0 == 0) {
            unpack_rows(a, gate->packed, gate->scale, gate->zero, 0, N, 0);
            unpack_rows(a, up->packed, up->scale, up->zero, 0, N, 0);
        }
        const uint16_t *x = whole_steps(a, X + m0 * K, m, K, l.X);
        if (launch_unpack_weight(nbits, bf16, a, s) != hipSuccess)
            return HQQ_EHIP;
        GemmArgs g{};
        single_segment(g, x, round_up(K, kStep), whole_pitch(K));
        g.B = l.W;
        g.ldb = a.ldw;
        g.M = (int32_t)m;
        g.N = (int32_t)N;
        g.act = act;
        g.dY = dY + m0 * N;
        g.ldy = N;
        g.bound = bound;
        g.rinv = l.inv;
        g.out = l.dGU;
        g.ldo = ldg;
        g.fill = Np;
        GemmArgs p{};
        single_segment(p, l.dGU, 2 * Np, ldg);
        p.B = l.W;
        p.ldb = a.ldw;
        p.M = (int32_t)m;
        p.N = (int32_t)K;
        if (launch_gemm(kOutGatedGrad, bf16, g, s) != hipSuccess ||
            gradient_product(p, bf16, l.part, nullptr, true, true, dX + m0 * K, RowFactor{bf16 ? nullptr : l.inv}, s) != hipSuccess)
            return HQQ_EHIP;
    }
    return HQQ_OK;
}

int64_t hqq_linear_batch_backward_workspace(int64_t M, int64_t K, const int64_t *n, int count, int nbits, int group_size)
{
    if (count < 1 || count > HQQ_MAX_GRADS)
        return HQQ_EINVAL_SHAPE;
    if (!n)
        return HQQ_EINVAL_PTR;
    if (const int st = check_batch(M, K, n, count, nbits, group_size))
        return st;
    return BatchGradLayout(nullptr, M, K, n, count, straight(kBackward, M, K, sum_of(n, count), group_size)).bytes;
}

int hqq_linear_batch_backward(const hqq_linear_grad *ws, int count, int64_t M, int64_t K, int nbits, int group_size,
                              int dtype, uint16_t *dX, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (count < 1 || count > HQQ_MAX_GRADS)
        return HQQ_EINVAL_SHAPE;
    if (!ws)
        return HQQ_EINVAL_PTR;
    int64_t n[HQQ_MAX_GRADS];
    for (int i = 0; i < count; ++i)
        n[i] = ws[i].N;
    if (const int st = check_batch(M, K, n, count, nbits, group_size))
        return st;
    if (const int st = check_dtype(dtype))
        return st;
    if (!aligned(dX, 16))
        return HQQ_EINVAL_PTR;
    for (int i = 0; i < count; ++i)
        if (!weight_ok(ws[i].packed, ws[i].scale, ws[i].zero) || !aligned(ws[i].dY, 16))
            return HQQ_EINVAL_PTR;
    const bool few = straight(kBackward, M, K, sum_of(n, count), group_size);
    const BatchGradLayout l(workspace, M, K, n, count, few);
    if (const int st = check_workspace(workspace, workspace_bytes, l.bytes))
        return st;
    const Range rd{dX, 2 * M * K}, rw{workspace, l.bytes};
    if (overlaps(rd, {rw}))
        return HQQ_EINVAL_PTR;
    for (int i = 0; i < count; ++i) {
        const Range ry{ws[i].dY, 2 * M * n[i]};
        if (overlaps(rd, {ry}) || overlaps(rw, {ry}) ||
            overlaps_weight({rd, rw}, ws[i].packed, ws[i].scale, ws[i].zero, n[i], K, nbits, group_size))
            return HQQ_EINVAL_PTR;
    }
    const bool bf16 = dtype == HQQ_DTYPE_BF16;
    const hipStream_t s = (hipStream_t)stream;
    if (few) {
        SkinnyGradArgs b{};
        for (int i = 0; i < count; ++i)
            add_grad(b, ws[i].packed, ws[i].scale, ws[i].zero, ws[i].dY, n[i], n[i]);
        return few_rows_gradient(b, bf16, nbits, group_size, M, K, l.part, dX, RowFactor{}, s) == hipSuccess ? HQQ_OK
                                                                                                        : HQQ_EHIP;
    }
    for (int64_t m0 = 0; m0 < M; m0 += kRowChunk) {
        const int64_t m = M - m0 < kRowChunk ? M - m0 : kRowChunk;
        UnpackArgs a = unpack_args(l.W, K, nbits, group_size);
        GemmArgs g{};
        g.segs = count;
        int64_t row = 0;
        for (int i = 0; i < count; ++i) {
            if (m0 == 0)
                unpack_rows(a, ws[i].packed, ws[i].scale, ws[i].zero, 0, n[i], row);
            row += round_up(n[i], kStep);
            g.A[i] = whole_steps(a, ws[i].dY + m0 * n[i], m, n[i], l.pad[i]);
            g.lda[i] = whole_pitch(n[i]);
            g.step0[i + 1] = (int32_t)(row / kStep);
        }
        if (launch_unpack_weight(nbits, bf16, a, s) != hipSuccess)
            return HQQ_EHIP;
        g.B = l.W;
        g.ldb = pitch_for(K);
        g.M = (int32_t)m;
        g.N = (int32_t)K;
        if (gradient_product(g, bf16, l.part, nullptr, true, true, dX + m0 * K, RowFactor{}, s) != hipSuccess)
            return HQQ_EHIP;
    }
    return HQQ_OK;
}

int64_t hqq_linear_cross_entropy_workspace(int64_t M, int64_t K, int64_t N, int nbits, int group_size)
{
    if (const int st = check_sizes(M, K, N, nbits, group_size))
        return st;
    return LossLayout(nullptr, M, K, N, straight(kHead, M, K, N, group_size)).bytes;
}

int hqq_linear_cross_entropy(const uint16_t *X, int64_t M, int64_t K, const hqq_weight *head, int64_t N, int nbits,
                             int group_size, int dtype, const int64_t *targets, float *loss, float *lse, void *workspace,
                             int64_t workspace_bytes, void *stream)
{
    if (const int st = check_sizes(M, K, N, nbits, group_size))
        return st;
    if (const int st = check_dtype(dtype))
        return st;
    if (!head || !weight_ok(head->packed, head->scale, head->zero) || !aligned(X, 16) || !aligned(targets, 8) ||
        !aligned(loss, 4) || !aligned(lse, 4))
        return HQQ_EINVAL_PTR;
    const bool few = straight(kHead, M, K, N, group_size);
    const LossLayout l(workspace, M, K, N, few);
    if (const int st = check_workspace(workspace, workspace_bytes, l.bytes))
        return st;
    const Range rx{X, 2 * M * K}, rt{targets, 8 * M}, ro{loss, 4 * M}, re{lse, 4 * M}, rw{workspace, l.bytes};
    if (overlaps(ro, {rx, rt, re, rw}) || overlaps(re, {rx, rt, rw}) || overlaps(rw, {rx, rt}) ||
        overlaps_weight({ro, re, rw}, *head, N, K, nbits, group_size))
        return HQQ_EINVAL_PTR;
    const bool bf16 = dtype == HQQ_DTYPE_BF16;
    const hipStream_t s = (hipStream_t)stream;
    if (few) {
        SkinnyArgs f{};
        f.w[0] = linear_args(X, *head, M, K, N, nbits, group_size);
        f.out = kOutStats;
        f.cols = N;
        f.g.M = (int32_t)M;
        f.g.N = (int32_t)N;
        f.g.Nall = N;
        f.g.targets = targets;
        f.g.stats = l.stats;
        f.g.blocks = l.pitch;
        f.g.tlogit = l.tlogit;
        const LossArgs e{l.stats, l.pitch, l.pitch, M, N, l.tlogit, targets, loss, lse};
        return launch_skinny(nbits, bf16, f, s) == hipSuccess && launch_loss(e, s) == hipSuccess ? HQQ_OK : HQQ_EHIP;
    }
    int64_t blocks = 0;
    for (int64_t n0 = 0; n0 < N; n0 += l.piece) {
        const int64_t n = N - n0 < l.piece ? N - n0 : l.piece;
        UnpackArgs a = unpack_args(l.W, K, nbits, group_size);
        unpack_rows(a, head->packed, head->scale, head->zero, n0, n, 0);
        if (n0 == 0)
            X = whole_steps(a, X, M, K, l.X);
        GemmArgs g{};
        single_segment(g, X, round_up(K, kStep), whole_pitch(K));
        g.B = l.W;
        g.ldb = a.ldw;
        g.M = (int32_t)M;
        g.N = (int32_t)n;
        g.stats = l.stats + blocks;
        g.blocks = l.pitch;
        g.tlogit = l.tlogit;
        g.targets = targets;
        g.n0 = n0;
        g.Nall = N;
        if (launch_unpack_weight(nbits, bf16, a, s) != hipSuccess || launch_gemm(kOutStats, bf16, g, s) != hipSuccess)
            return HQQ_EHIP;
        blocks += gemm_stats_blocks(M, n, g.step0[1]);
    }
    const LossArgs e{l.stats, l.pitch, blocks, M, N, l.tlogit, targets, loss, lse};
    return launch_loss(e, s) == hipSuccess ? HQQ_OK : HQQ_EHIP;
}

int64_t hqq_linear_cross_entropy_backward_workspace(int64_t M, int64_t K, int64_t N, int nbits, int group_size)
{
    if (const int st = check_sizes(M, K, N, nbits, group_size))
        return st;
    return LossGradLayout(nullptr, M, K, N, straight(kHeadGrad, M, K, N, group_size)).bytes;
}

int hqq_linear_cross_entropy_backward(const float *dloss, const uint16_t *X, int64_t M, int64_t K, const hqq_weight *head,
                                      int64_t N, int nbits, int group_size, int dtype, const int64_t *targets,
                                      const float *lse, uint16_t *dX, void *workspace, int64_t workspace_bytes,
                                      void *stream)
{
    if (const int st = check_sizes(M, K, N, nbits, group_size))
        return st;
    if (const int st = check_dtype(dtype))
        return st;
    if (!head || !weight_ok(head->packed, head->scale, head->zero) || !aligned(X, 16) || !aligned(dX, 16) ||
        !aligned(targets, 8) || !aligned(dloss, 4) || !aligned(lse, 4))
        return HQQ_EINVAL_PTR;
    const bool few = straight(kHeadGrad, M, K, N, group_size);
    const LossGradLayout l(workspace, M, K, N, few);
    if (const int st = check_workspace(workspace, workspace_bytes, l.bytes))
        return st;
    const Range rx{X, 2 * M * K}, rt{targets, 8 * M}, ro{dloss, 4 * M}, re{lse, 4 * M}, rd{dX, 2 * M * K}, rw{workspace, l.bytes};
    if (overlaps(rd, {rx, rt, ro, re, rw}) || overlaps(rw, {rx, rt, ro, re}) ||
        overlaps_weight({rd, rw}, *head, N, K, nbits, group_size))
        return HQQ_EINVAL_PTR;
    const bool bf16 = dtype == HQQ_DTYPE_BF16;
    const hipStream_t s = (hipStream_t)stream;
    const float unit = bf16 ? 1.0f : 1.0f / 32768.0f;     // of the rounded differences
    if (few) {
        SkinnyArgs f{};
        f.w[0] = linear_args(X, *head, M, K, N, nbits, group_size);
        f.out = kOutSoftGrad;
        f.cols = l.ldl;
        f.g.M = (int32_t)M;
        f.g.N = (int32_t)N;
        f.g.Nall = N;
        f.g.targets = targets;
        f.g.lse = lse;
        f.g.out = l.dL;
        f.g.ldo = l.ldl;
        f.g.fill = l.ldl;
        SkinnyGradArgs b{};
        add_grad(b, head->packed, head->scale, head->zero, l.dL, l.ldl, N);
        return launch_skinny(nbits, bf16, f, s) == hipSuccess &&
                       few_rows_gradient(b, bf16, nbits, group_size, M, K, l.part, dX,
                                         RowFactor{nullptr, dloss, targets, N, unit}, s) == hipSuccess
                   ? HQQ_OK
                   : HQQ_EHIP;
    }
    for (int64_t m0 = 0; m0 < M; m0 += kRowChunk) {
        const int64_t m = M - m0 < kRowChunk ? M - m0 : kRowChunk;
        const uint16_t *x = X + m0 * K;
        const RowFactor rowf{nullptr, dloss + m0, targets + m0, N, unit};
        for (int64_t n0 = 0; n0 < N; n0 += l.piece) {
            const int64_t n = N - n0 < l.piece ? N - n0 : l.piece;
            const int64_t fill = round_up(n, kStep), ldl = pitch_for(n);
            UnpackArgs a = unpack_args(l.W, K, nbits, group_size);
            unpack_rows(a, head->packed, head->scale, head->zero, n0, n, 0);
            if (n0 == 0)
                x = whole_steps(a, x, m, K, l.X);
            GemmArgs g{};
            single_segment(g, x, round_up(K, kStep), whole_pitch(K));
            g.B = l.W;
            g.ldb = a.ldw;
            g.M = (int32_t)m;
            g.N = (int32_t)n;
            g.targets = targets + m0;
            g.lse = lse + m0;
            g.n0 = n0;
            g.Nall = N;
            g.out = l.dL;
            g.ldo = ldl;
            g.fill = fill;
            GemmArgs p{};
            single_segment(p, l.dL, fill, ldl);
            p.B = l.W;
            p.ldb = a.ldw;
            p.M = (int32_t)m;
            p.N = (int32_t)K;
            if (launch_unpack_weight(nbits, bf16, a, s) != hipSuccess ||
                launch_gemm(kOutSoftGrad, bf16, g, s) != hipSuccess ||
                gradient_product(p, bf16, l.part, l.acc, n0 == 0, n0 + n == N, dX + m0 * K, rowf, s) != hipSuccess)
                return HQQ_EHIP;
        }
    }
    return HQQ_OK;
}

}  // extern "C"
