// Shared declarations of the paged-attention operators (plan, rotary positions
// with the cache write, tree attention).
#pragma once

#include "internal.h"

namespace moe {

// Workspace: a header that the caller zeroes once, then split partials.
// The counters return to zero by themselves: the last block of a group resets
// the one it counted on.
constexpr int kAttnCounters = 960;
struct AttnHeader {
  int32_t err;                       // device error bits (MOE_DEVERR_*)
  int32_t plan_ticket;               // blocks of the running plan that have read *free_head
  int32_t pad[62];
  int32_t counters[kAttnCounters];   // blocks of a split group that have stored their partial
};
static_assert(sizeof(AttnHeader) == MOE_ATTN_HEADER_BYTES, "attention workspace header");

// Split partials: kAttnMaxCtas blocks own two slots of 128 rows each: the rows'
// FP32 output sums ([four columns][row]) and, after all of them, (max, sum).
constexpr int kAttnMaxCtas = 160;
constexpr int kAttnRows = 128;
constexpr int kAttnPartDim = 128;
// A unit's fixed cost beside its key tiles, in tiles: a piece of a run takes 3 to 4
// us beside 0.8 to 1.2 us a tile.  Cost 2, 3, 4, 5 measured on large trees over short
// and long contexts: 110, 97, 92, 92 us; flat for 64 requests of up to 8,000 tokens.
constexpr int kAttnPieceCost = 4;
constexpr size_t kAttnPartSlots = 2 * kAttnMaxCtas;
constexpr size_t kAttnPartBytes = kAttnPartSlots * kAttnRows * (kAttnPartDim + 2) * 4;
constexpr size_t kAttnJoinBytes = kAttnMaxCtas * 16;   // a record a run: what the join kernel adds

struct PlanArgs {
  const int32_t *ctx_len, *new_len, *parents;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* free_head;
  int32_t *free_head_out, *q_start, *kv_len, *positions;
  int64_t* slot_map;
  int32_t* tree_mask;
  AttnHeader* hdr;
  int R, T, n_free, n_pages, max_pages, page_shift, mask_words;
};
cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t s);

// rows of `heads` heads that one launch turns (or, rot 0, copies)
struct RopeRows {
  const void* src;
  void* dst;
  int64_t src_ld, dst_ld;   // row strides, elements; dst_ld unused where dst is the cache
  int heads;
  int rotate, to_cache;
};
struct RopeArgs {
  RopeRows part[3];
  int n_parts;
  const int32_t* positions;
  const uint64_t* table;
  const int64_t* slot_map;
  AttnHeader* hdr;
  int64_t n_slots;
  int64_t page_stride, token_stride, head_stride;
  float scale;
  int T, D, rot, inverse, page_shift;
};
cudaError_t launch_rope(const RopeArgs& a, int dtype, int interleaved, cudaStream_t s);

struct AttnArgs {
  const void* q;
  const void *k, *v;
  const int32_t *q_start, *kv_len, *block_table, *tree_mask;
  void* out;
  float* lse;
  AttnHeader* hdr;
  float* part;              // [slots] of 128 x kAttnPartDim
  float2* part_ml;          // [slots][128 rows] (max, sum)
  int4* joins;              // [runs] (parts or 0, first row, nodes, KV head)
  int64_t q_ld, out_ld, page_stride, token_stride, head_stride;
  float scale;
  int R, T, H, Hkv, G, D, n_pages, max_pages, page_shift, mask_words;
};
// one warp a key range, FP32 arithmetic on the CUDA cores (FP32 layers)
cudaError_t launch_attention_f32(const AttnArgs& a, cudaStream_t s);
// tensor cores (BF16)
cudaError_t launch_attention_bf16(const AttnArgs& a, cudaStream_t s);

}  // namespace moe
