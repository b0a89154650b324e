// Shared declarations of the paged-attention operators (plan, rotary positions
// with the cache write, tree attention, pages that requests share).
#pragma once

#include "internal.h"
#include "meet.h"

namespace moe {

// Workspace: a header that the caller zeroes once, then split partials.
// The counters return to zero by themselves: the last block of a group resets
// the one it counted on.
constexpr int kAttnCounters = 960;
struct AttnHeader {
  int32_t err;                       // device error bits (MOE_DEVERR_*)
  int32_t plan_ticket;               // blocks of the running plan that have read *free_head
  int32_t met[kMeetWords], left;     // blocks of a cooperative launch that came to meetings, that left
  int32_t pad[61 - kMeetWords];
  int32_t counters[kAttnCounters];   // blocks of a split group that have stored their partial
};
static_assert(sizeof(AttnHeader) == MOE_ATTN_HEADER_BYTES, "attention workspace header");

// Split partials: kAttnMaxCtas blocks own two slots of 128 rows each: the rows'
// FP32 output sums ([four columns][row]) and, after all of them, (max, sum).
constexpr int kAttnMaxCtas = 152;          // a GB300's SMs
constexpr int kAttnRows = 128;
constexpr int kAttnTile = 128;             // keys a tile
constexpr int kAttnPartDim = 128;
// A unit's fixed cost beside its key tiles, in tiles: a piece of a run takes 3 to 4
// us beside 0.8 to 1.2 us a tile.  Cost 2, 3, 4, 5 measured on large trees over short
// and long contexts: 110, 97, 92, 92 us; flat for 64 requests of up to 8,000 tokens.
constexpr int kAttnPieceCost = 4;
constexpr int kPrefixMaxRequests = 2048;   // of a call with shared prefixes (and as many groups)
// The kernel for few rows: its runs (warps) at most, rows of a unit, units of a KV head (1 / 2 / 4 of them, us: 128
// requests of up to 8 nodes 137 / 127 / 126, 64 of 2000 own tokens 115 / 125 / 125, of up to 16 nodes 157 / 156 / 192)
// that a request may have.
constexpr int kFewRuns = 2048;
constexpr int kFewRows = 16, kFewBlocks = 2;
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

struct ForkArgs {
  const int32_t *src, *dst, *lengths;
  const int32_t* src_table;
  int32_t *dst_table, *shares;
  const int32_t *free_pages, *free_head;
  int32_t* free_head_out;
  uint8_t *k, *v;
  AttnHeader* hdr;
  int64_t page_stride, token_stride, head_stride;   // bytes
  int n, R, n_free, n_pages, max_pages, page_shift, Hkv, row_bytes, same;   // same: one table
};
cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s);

struct CompactArgs {
  const int32_t *first, *keep_start, *keep, *block_table, *shares;
  int32_t* len_out;
  uint8_t *k, *v;
  AttnHeader* hdr;
  void* scratch;            // of the moves of long lists
  size_t scratch_bytes;
  int64_t page_stride, token_stride, head_stride;   // bytes
  int R, N, n_pages, max_pages, page_shift, Hkv, row_bytes;
};
cudaError_t launch_compact(const CompactArgs& a, cudaStream_t s);

struct ReleaseArgs {
  const int32_t *held_len, *keep_len;
  int32_t *block_table, *shares, *free_pages, *free_head;
  int32_t* counts;          // [blocks] entries freed (scratch)
  int32_t* last;            // [n_pages] the last entry that gives a page back (scratch)
  AttnHeader* hdr;
  int R, n_free, n_pages, max_pages, page_shift;
};
cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t s);

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
  const int32_t* positions;          // [axes][T]
  const uint8_t* axis;               // of each pair; NULL: one axis
  const uint64_t* table;
  const int64_t* slot_map;
  AttnHeader* hdr;
  int64_t n_slots;
  int64_t page_stride, token_stride, head_stride;
  float scale;
  int T, D, rot, inverse, page_shift, n_axes;
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
  // shared prefixes (n_groups 0: none)
  const int32_t *group_start, *prefix_row, *prefix_len;
  int n_groups;
  float* rows_part;         // [prefix or own][KV head][T * G rows][64 or 128]: output sums of whole units
  float2* rows_ml;          // [prefix or own][KV head][T * G rows] their (max, sum)
  int4* parts_of;           // [prefix or own][KV head][T]: where a token's partials are (PartsOf)
  // the kernel for few rows: nodes that it takes (0: none), whether it runs alone
  int few_tokens, few_alone;
  float* few_part;          // [2 kFewRuns slots][16 rows][64 or 128]
  float2* few_ml;           // [slots][16 rows] (max, sum)
  float* pair_part;         // [kAttnPartSlots slots][2 x 128 rows][64 or 128]: units that a run's end cuts
  float2* pair_ml;          // [slots][rows] (max, sum)
};

// A group of requests that share a prefix: its tokens, whole pages of them, are read through one row of the table.
struct PrefixGroup {
  int begin, end, row, pages;
};
// group g, empty and without pages where its entries are no good; *bad is set then
__device__ __forceinline__ PrefixGroup prefix_group(const int32_t* start, const int32_t* row, const int32_t* len, int g,
                                                    int R, int max_pages, int page_shift, int* bad) {
  PrefixGroup p;
  p.begin = start[g];
  p.end = start[g + 1];
  p.row = row[g];
  const int n = len[g];
  p.pages = min(max(n, 0) >> page_shift, max_pages);
  if (p.begin < 0 || p.end < p.begin || p.end > R || p.row < 0 || p.row >= R || n < 0 || n >> page_shift > max_pages) {
    if (bad) *bad = 1;
    p.begin = p.end = p.row = p.pages = 0;
  }
  if (p.end - p.begin < 2) p.pages = 0;        // nobody to share with
  return p;
}
// group of request r: the last that begins at or before it (its end is the caller's to check); -1: none
__device__ __forceinline__ int group_of(const int32_t* start, int n_groups, int r) {
  if (n_groups == 0 || start[0] > r) return -1;
  int lo = 0, hi = n_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}

// one warp a key range, FP32 arithmetic on the CUDA cores (FP32 layers)
cudaError_t launch_attention_f32(const AttnArgs& a, cudaStream_t s);
// tensor cores (BF16)
cudaError_t launch_attention_bf16(const AttnArgs& a, cudaStream_t s);
// the same with shared prefixes
cudaError_t launch_prefix_attention_f32(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_prefix_attention_bf16(const AttnArgs& a, cudaStream_t s);
void few_shape(AttnArgs* a);
cudaError_t launch_attention_few(const AttnArgs& a, cudaStream_t s);

}  // namespace moe
