// hqq_cache_internal.h -- declarations shared by the cache library's own
// translation units.
#pragma once

#include "hqq_cache.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hqq {

// Tokens of a block of rows in the write and read kernels.
constexpr int kCacheCodecTokens = 16;

// Arguments of the write and read kernels, either side's at [0] (k) and [1] (v).
struct CacheCodecArgs {
    uint32_t *packed[2];
    float *scale[2], *zero[2];
    const uint16_t *x[2];            // write: rows of 16-bit values
    int64_t token_stride[2], head_stride[2];
    uint16_t *hat[2];                // read's outputs; write: null, or the values written
    const int64_t *slots;
    int64_t slot_count;              // pages * page_size
    int32_t tokens, heads;
    int32_t rows;                    // heads * tokens, the tokens rounded up to whole blocks
    uint64_t head_factor;            // 2^36 / heads, rounded up
    int32_t page_shift, page_mask;
};

// Attention: all sequences' tokens are cut into about `workers` equal runs per key-value
// head and row tile (hqq_cache_plan.h), or, workers = 0, a workgroup takes a sequence.
struct CacheAttentionArgs {
    const uint32_t *packed[2];
    const float *scale[2], *zero[2];
    const uint16_t *Q;
    int64_t q_batch_stride, q_head_stride;
    const int32_t *table, *lengths;
    uint16_t *out;
    float *lse;                      // may be null
    float *part;                     // [segments, q_heads, dim] sums of split sequences' segments, of which
                                     // there are at most workers + min(workers, batch)
    float2 *part_ml;                 // [segments, q_heads] their maxima and sums of weights
    int32_t *plan;                   // null, or the plan: kCachePlanHead numbers, then where each sequence begins
    int32_t batch, q_heads, heads, G;
    int32_t row_tiles;               // blocks of 16 q heads of a key-value head
    int32_t pages, page_shift, page_mask, table_width;
    int32_t window;                  // 0: none
    int32_t workers;
    float scale_log2;                // softmax_scale * log2(e)
    int32_t bf16;
};

// Tokens that a wave takes at a time, and a workgroup in a step of its waves.
constexpr int kCacheTile = 32;
constexpr int kCacheWaves = 4;
constexpr int kCacheStep = kCacheTile * kCacheWaves;
// Workgroups of the attention kernel that a CU holds at a time: two, eight waves with some 5 KB
// each on their way.  (More in flight is slower, whatever they compute: the loads alone of 64 x
// 8192 tokens over 8 heads of 128 at 4 bits, 117 us by two, 130 by three, 159 by two with tiles of 64
// tokens; with the arithmetic, weights still in one operand, 125 by two, 139 by three, 152 by one.)  One where 8 bits of 256 dims in groups of
// 64 take more than half of a CU's LDS: runs for two would go in two rounds.  (16 sequences of 8192 tokens over 4
// heads 87.5 us by runs for two, 77.5 for one, 16 of 3000 over 16 heads 89.8 and 75, one of 32768 over 4 heads
// 49.7 and 41; of 4 sequences to 2000 tokens 22.3 and 22.7.)
constexpr int cache_resident(int nbits, int dim, int group_size)
{
    return nbits == 8 && dim == 256 && group_size == 64 ? 1 : 2;
}
constexpr int kCus = 256;
constexpr int kLdsOfCu = 160 * 1024;

// Sequences of at most this many tokens are not split: a step more costs a workgroup 1 us, the join's
// launch, a segment's end and the host's part of them 3 to 6.  (4 bits of 128 dims, fp16, whole and split: one
// sequence of 512 tokens over 8 heads 9.3 and 13.4 us, of 768 11.5 and 13.2, of 1024 14.2 and 12.9; over 32 heads
// of 768 12.4 and 13.2, of 1024 14.8 and 13; 64 sequences of 768 over 8 heads 17.7 and 21.4, 200 of 768 over 32
// 192 and 199.  Large batches gain up to 4 % on beyond it, small ones lose.)
constexpr int kCacheWhole = 768;

// Runs of more steps than this cross sequences.
constexpr int kCacheCross = 8;

// Of more sequences than this the plan is found once, by a launch of its own that costs 2.5 us, not by
// every wave, 64 sequences at a time.  (8 heads: 128 sequences of 100, 1024 and 4000 tokens 19.7, 41.7
// and 135 us by every wave, 22.3, 43.8 and 131 by the launch; 512 sequences 181, 170 and 481, and 68,
// 156 and 471.)
constexpr int kCachePlanned = 128;
constexpr int kCachePlanHead = 3;    // steps per run, runs, whether these cross sequences

hipError_t launch_cache_write(int nbits, int dim, int group_size, bool bf16, const CacheCodecArgs &a, hipStream_t s);
hipError_t launch_cache_read(int nbits, int dim, int group_size, bool bf16, const CacheCodecArgs &a, hipStream_t s);
hipError_t launch_cache_attention_b2(int dim, int group_size, const CacheAttentionArgs &a, hipStream_t s);
hipError_t launch_cache_attention_b4(int dim, int group_size, const CacheAttentionArgs &a, hipStream_t s);
hipError_t launch_cache_attention_b8(int dim, int group_size, const CacheAttentionArgs &a, hipStream_t s);
// finds the plan of many sequences
hipError_t launch_cache_plan(const CacheAttentionArgs &a, hipStream_t s);
// joins the segments of split sequences
hipError_t launch_cache_join(int dim, const CacheAttentionArgs &a, hipStream_t s);

}  // namespace hqq
