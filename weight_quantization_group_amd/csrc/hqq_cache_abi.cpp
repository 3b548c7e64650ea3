// hqq_cache_abi.cpp -- the C ABI of include/hqq_cache.h: argument checks, the
// workspace's layout, and the launches.  No allocation, no state.
#include "hqq_cache_internal.h"

#include <stdint.h>

#include <initializer_list>

namespace {

using namespace hqq;

bool aligned(const void *p, unsigned to) { return p && ((uintptr_t)p & (to - 1)) == 0; }

bool power_of_two(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

int log2_of(int64_t v)
{
    int b = 0;
    while ((int64_t(1) << b) < v)
        ++b;
    return b;
}

int check_layout(const hqq_cache *c)
{
    if (!c)
        return HQQ_EINVAL_PTR;
    if (c->nbits != 2 && c->nbits != 4 && c->nbits != 8)
        return HQQ_EINVAL_NBITS;
    if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 192 && c->dim != 256)
        return HQQ_EINVAL_SHAPE;
    if (!power_of_two(c->group_size) || c->group_size < 32 || c->group_size > 256 || c->dim % c->group_size != 0 ||
        c->dim / c->group_size > 4)
        return HQQ_EINVAL_GROUP;
    if (!power_of_two(c->page_size) || c->page_size < 16 || c->page_size > 1024 || c->pages < 1 ||
        c->pages > INT32_MAX || c->heads < 1 || c->heads > 1024 ||
        c->pages * c->heads > (int64_t(1) << 40) / c->page_size)
        return HQQ_EINVAL_SHAPE;
    return HQQ_OK;
}

int check_cache(const hqq_cache *c)
{
    if (const int st = check_layout(c))
        return st;
    for (const hqq_cache_side &s : {c->k, c->v})
        if (!aligned(s.packed, 16) || !aligned(s.scale, 16) || !aligned(s.zero, 16))
            return HQQ_EINVAL_PTR;
    return HQQ_OK;
}

int check_dtype(int dtype)
{
    return dtype == HQQ_DTYPE_FP16 || dtype == HQQ_DTYPE_BF16 ? HQQ_OK : HQQ_EINVAL_DTYPE;
}

// [tokens, heads] rows of 16-bit values: whole 16-byte loads, whose span fits
struct Rows {
    const uint16_t *data;
    int64_t token_stride, head_stride;
};

int check_rows(const Rows &r, int64_t tokens, int64_t heads)
{
    if (!aligned(r.data, 16))
        return HQQ_EINVAL_PTR;
    constexpr int64_t kMaxStride = int64_t(1) << 40;
    if (r.token_stride < 0 || r.head_stride < 0 || r.token_stride % 8 != 0 || r.head_stride % 8 != 0 ||
        r.token_stride > kMaxStride / tokens || r.head_stride > kMaxStride / heads)
        return HQQ_EINVAL_SHAPE;
    return HQQ_OK;
}

struct Range {
    const void *p;
    int64_t bytes;
};

Range rows_range(const Rows &r, int64_t tokens, int64_t heads, int64_t dim)
{
    return Range{r.data, 2 * ((tokens - 1) * r.token_stride + (heads - 1) * r.head_stride + dim)};
}

bool overlap(Range a, Range b)
{
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.bytes && b.bytes && x < y + (uint64_t)b.bytes && y < x + (uint64_t)a.bytes;
}

// whether what a call writes shares memory with what it reads or otherwise writes
bool written_overlaps(std::initializer_list<Range> written, std::initializer_list<Range> read)
{
    for (auto w = written.begin(); w != written.end(); ++w) {
        for (const Range &r : read)
            if (overlap(*w, r))
                return true;
        for (auto o = written.begin(); o != w; ++o)
            if (overlap(*w, *o))
                return true;
    }
    return false;
}

struct CacheRanges {
    Range kp, ks, kz, vp, vs, vz;
    explicit CacheRanges(const hqq_cache &c)
    {
        const int64_t rows = c.pages * c.heads * c.page_size;
        const int64_t codes = rows * (c.dim * c.nbits / 8), meta = rows * (c.dim / c.group_size) * 4;
        kp = {c.k.packed, codes}, ks = {c.k.scale, meta}, kz = {c.k.zero, meta};
        vp = {c.v.packed, codes}, vs = {c.v.scale, meta}, vz = {c.v.zero, meta};
    }
};

CacheCodecArgs codec_args(const hqq_cache &c, const int64_t *slots, int64_t tokens)
{
    CacheCodecArgs a{};
    for (int i = 0; i < 2; ++i) {
        const hqq_cache_side &s = i ? c.v : c.k;
        a.packed[i] = s.packed;
        a.scale[i] = s.scale;
        a.zero[i] = s.zero;
    }
    a.slots = slots;
    a.slot_count = c.pages * c.page_size;
    a.tokens = (int32_t)tokens;
    a.heads = c.heads;
    a.rows = (int32_t)((tokens + kCacheCodecTokens - 1) / kCacheCodecTokens * kCacheCodecTokens * c.heads);
    a.head_factor = ((uint64_t(1) << 36) + (uint64_t)c.heads - 1) / (uint64_t)c.heads;
    a.page_shift = log2_of(c.page_size);
    a.page_mask = c.page_size - 1;
    return a;
}

int check_tokens(const hqq_cache &c, int64_t tokens)
{
    return tokens < 0 || tokens > (1 << 26) / c.heads ? HQQ_EINVAL_SHAPE : HQQ_OK;
}

int check_batch(const hqq_cache &c, int64_t batch, int64_t q_heads, int64_t table_width)
{
    if (batch < 0 || batch > (1 << 15) || q_heads < 1 || q_heads > (1 << 16) || q_heads % c.heads != 0 ||
        batch * q_heads > (1 << 28) || table_width < 1 || table_width > (1 << 30) / c.page_size ||
        batch * table_width * c.page_size > int64_t(1) << 37)
        return HQQ_EINVAL_SHAPE;
    return HQQ_OK;
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Runs per key-value head and row tile, `columns` of those: as many workgroups as the chip
// holds, or some rounds of them where that divides better.
int32_t workers_for(const hqq_cache &c, int64_t columns)
{
    const int64_t slots = (int64_t)kCus * cache_resident(c.nbits, c.dim, c.group_size);
    int64_t best = slots / columns, rounds = 1;
    for (int64_t r = 2; r <= 4; ++r)
        if (r * slots / columns * rounds > best * r * 11 / 10) {
            best = r * slots / columns;
            rounds = r;
        }
    return (int32_t)(best < 1 ? 1 : best);
}

struct AttentionLayout {
    int32_t row_tiles, workers;      // workers: 0 where no sequence is split
    float *part = nullptr;
    float2 *part_ml = nullptr;
    int32_t *plan = nullptr;
    int64_t bytes = 0;
    AttentionLayout(void *ws, const hqq_cache &c, int64_t batch, int64_t q_heads, int64_t table_width)
    {
        const int64_t G = q_heads / c.heads;
        row_tiles = (int32_t)((G + 15) / 16);
        workers = 0;
        if (batch == 0 || table_width * c.page_size <= kCacheWhole)
            return;
        workers = workers_for(c, c.heads * row_tiles);
        const int64_t segments = workers + (batch < workers ? batch : workers);
        const int64_t sums = round_up(segments * q_heads * c.dim * 4, 256);
        const int64_t meta = round_up(segments * q_heads * 8, 256);
        const bool planned = batch > kCachePlanned;
        bytes = sums + meta + (planned ? round_up((kCachePlanHead + batch + 1) * 4, 256) : 0);
        if (ws) {
            part = (float *)ws;
            part_ml = (float2 *)((char *)ws + sums);
            if (planned)
                plan = (int32_t *)((char *)ws + sums + meta);
        }
    }
};

}  // namespace

extern "C" {

int hqq_cache_write(const hqq_cache *cache, const uint16_t *K, int64_t k_token_stride, int64_t k_head_stride,
                    const uint16_t *V, int64_t v_token_stride, int64_t v_head_stride, int64_t tokens,
                    const int64_t *slots, int dtype, uint16_t *K_hat, uint16_t *V_hat, void *stream)
{
    if (const int st = check_cache(cache))
        return st;
    if (const int st = check_dtype(dtype))
        return st;
    const hqq_cache &c = *cache;
    if (const int st = check_tokens(c, tokens))
        return st;
    if (tokens == 0)
        return HQQ_OK;
    const Rows x[2] = {{K, k_token_stride, k_head_stride}, {V, v_token_stride, v_head_stride}};
    for (const Rows &r : x)
        if (const int st = check_rows(r, tokens, c.heads))
            return st;
    if (!aligned(slots, 8) || !K_hat != !V_hat || (K_hat && (!aligned(K_hat, 16) || !aligned(V_hat, 16))))
        return HQQ_EINVAL_PTR;
    const CacheRanges r(c);
    const int64_t hat = 2 * tokens * c.heads * c.dim;
    if (written_overlaps({r.kp, r.ks, r.kz, r.vp, r.vs, r.vz, {K_hat, hat}, {V_hat, hat}},
                         {rows_range(x[0], tokens, c.heads, c.dim), rows_range(x[1], tokens, c.heads, c.dim),
                          {slots, 8 * tokens}}))
        return HQQ_EINVAL_PTR;
    CacheCodecArgs a = codec_args(c, slots, tokens);
    for (int i = 0; i < 2; ++i) {
        a.x[i] = x[i].data;
        a.token_stride[i] = x[i].token_stride;
        a.head_stride[i] = x[i].head_stride;
    }
    a.hat[0] = K_hat;
    a.hat[1] = V_hat;
    return launch_cache_write(c.nbits, c.dim, c.group_size, dtype == HQQ_DTYPE_BF16, a, (hipStream_t)stream) == hipSuccess
               ? HQQ_OK
               : HQQ_EHIP;
}

int hqq_cache_read(const hqq_cache *cache, const int64_t *slots, int64_t tokens, int dtype, uint16_t *K, uint16_t *V,
                   void *stream)
{
    if (const int st = check_cache(cache))
        return st;
    if (const int st = check_dtype(dtype))
        return st;
    const hqq_cache &c = *cache;
    if (const int st = check_tokens(c, tokens))
        return st;
    if (tokens == 0)
        return HQQ_OK;
    if (!aligned(slots, 8) || !aligned(K, 16) || !aligned(V, 16))
        return HQQ_EINVAL_PTR;
    const CacheRanges r(c);
    const int64_t hat = 2 * tokens * c.heads * c.dim;
    if (written_overlaps({{K, hat}, {V, hat}}, {r.kp, r.ks, r.kz, r.vp, r.vs, r.vz, {slots, 8 * tokens}}))
        return HQQ_EINVAL_PTR;
    CacheCodecArgs a = codec_args(c, slots, tokens);
    a.hat[0] = K;
    a.hat[1] = V;
    return launch_cache_read(c.nbits, c.dim, c.group_size, dtype == HQQ_DTYPE_BF16, a, (hipStream_t)stream) == hipSuccess
               ? HQQ_OK
               : HQQ_EHIP;
}

int64_t hqq_cache_attention_workspace(const hqq_cache *cache, int64_t batch, int64_t q_heads, int64_t table_width)
{
    if (const int st = check_layout(cache))
        return st;
    if (const int st = check_batch(*cache, batch, q_heads, table_width))
        return st;
    return AttentionLayout(nullptr, *cache, batch, q_heads, table_width).bytes;
}

int hqq_cache_attention(const hqq_cache *cache, const uint16_t *Q, int64_t q_batch_stride, int64_t q_head_stride,
                        int64_t batch, int64_t q_heads, const int32_t *table, int64_t table_width,
                        const int32_t *lengths, float softmax_scale, int64_t window, int dtype, uint16_t *out, float *lse,
                        void *workspace, int64_t workspace_bytes, void *stream)
{
    if (const int st = check_cache(cache))
        return st;
    if (const int st = check_dtype(dtype))
        return st;
    const hqq_cache &c = *cache;
    if (const int st = check_batch(c, batch, q_heads, table_width))
        return st;
    if (!(softmax_scale > 0 && softmax_scale <= 0x1p100f) || window < 0)
        return HQQ_EINVAL_PARAM;
    if (batch == 0)
        return HQQ_OK;
    const Rows q{Q, q_batch_stride, q_head_stride};
    if (const int st = check_rows(q, batch, q_heads))
        return st;
    if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(out, 16) || (lse && !aligned(lse, 4)) ||
        workspace_bytes < 0 || (!workspace && workspace_bytes > 0) || (workspace && !aligned(workspace, 16)))
        return HQQ_EINVAL_PTR;
    const AttentionLayout l(workspace, c, batch, q_heads, table_width);
    if (workspace_bytes < l.bytes)
        return HQQ_EWORKSPACE;
    const CacheRanges r(c);
    if (written_overlaps({{out, 2 * batch * q_heads * c.dim}, {lse, 4 * batch * q_heads}, {workspace, l.bytes}},
                         {r.kp, r.ks, r.kz, r.vp, r.vs, r.vz, rows_range(q, batch, q_heads, c.dim),
                          {table, 4 * batch * table_width}, {lengths, 4 * batch}}))
        return HQQ_EINVAL_PTR;
    CacheAttentionArgs a{};
    for (int i = 0; i < 2; ++i) {
        const hqq_cache_side &s = i ? c.v : c.k;
        a.packed[i] = s.packed;
        a.scale[i] = s.scale;
        a.zero[i] = s.zero;
    }
    a.Q = Q;
    a.q_batch_stride = q_batch_stride;
    a.q_head_stride = q_head_stride;
    a.table = table;
    a.lengths = lengths;
    a.out = out;
    a.lse = lse;
    a.part = l.part;
    a.part_ml = l.part_ml;
    a.plan = l.plan;
    a.batch = (int32_t)batch;
    a.q_heads = (int32_t)q_heads;
    a.heads = c.heads;
    a.G = (int32_t)(q_heads / c.heads);
    a.row_tiles = l.row_tiles;
    a.pages = (int32_t)c.pages;
    a.page_shift = log2_of(c.page_size);
    a.page_mask = c.page_size - 1;
    a.table_width = (int32_t)table_width;
    a.window = window > INT32_MAX ? 0 : (int32_t)window;
    a.workers = l.workers;
    a.scale_log2 = softmax_scale * 1.44269504088896340736f;
    a.bf16 = dtype == HQQ_DTYPE_BF16;
    const hipStream_t s = (hipStream_t)stream;
    if (a.plan && launch_cache_plan(a, s) != hipSuccess)
        return HQQ_EHIP;
    const hipError_t e = c.nbits == 2   ? launch_cache_attention_b2(c.dim, c.group_size, a, s)
                         : c.nbits == 4 ? launch_cache_attention_b4(c.dim, c.group_size, a, s)
                                        : launch_cache_attention_b8(c.dim, c.group_size, a, s);
    if (e != hipSuccess)
        return HQQ_EHIP;
    return !l.workers || launch_cache_join(c.dim, a, s) == hipSuccess ? HQQ_OK : HQQ_EHIP;
}

const char *hqq_cache_strerror(int status)
{
    switch (status) {
    case HQQ_OK: return "success";
    case HQQ_EINVAL_NBITS: return "nbits must be 2, 4 or 8";
    case HQQ_EINVAL_GROUP: return "group_size must be 32, 64, 128 or 256 and divide dim into at most 4 groups";
    case HQQ_EINVAL_SHAPE: return "a size or stride is out of range";
    case HQQ_EINVAL_PTR: return "NULL, misaligned or overlapping pointer";
    case HQQ_EINVAL_PARAM: return "softmax_scale must be > 0 and at most 2^100, window >= 0";
    case HQQ_EHIP: return "HIP launch failed";
    case HQQ_EINVAL_DTYPE: return "dtype must be HQQ_DTYPE_FP16 or HQQ_DTYPE_BF16";
    case HQQ_EWORKSPACE: return "workspace smaller than hqq_cache_attention_workspace says";
    }
    return "unknown status";
}

}  // extern "C"
