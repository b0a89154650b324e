// Requests and groups as the attention kernels walk over them.
#pragma once

#include "attn.h"

namespace moe {

// flags of a Req: a group's prefix; own tokens of rows that have a prefix beside them
constexpr int kPrefix = 8, kJoined = 16;

struct Req {
  int q0, n, kv, ctx, tiles, blocks;
  int row, skip, flags;    // (shared prefixes) the table's row, its pages before the first tile; kPrefix or kJoined
};

__device__ __forceinline__ Req request(const AttnArgs& a, int r, int tb, int* bad) {
  Req q;
  q.q0 = min(max(a.q_start[r], 0), a.T);
  const int q1 = min(max(a.q_start[r + 1], q.q0), a.T);
  q.n = q1 - q.q0;
  // a length past the table's row is cut there: its tokens before that stay where they are, nodes among them or not
  const int cap = a.max_pages << a.page_shift;             // at most 2^30
  const int kv = a.kv_len[r];
  q.ctx = min(max(kv, q.n) - q.n, cap);
  q.kv = min(q.ctx + q.n, cap);
  if (bad && (kv < q.n || kv > cap || q.q0 != a.q_start[r])) *bad = 1;
  q.tiles = max((q.kv + kAttnTile - 1) / kAttnTile, 1);
  q.blocks = (q.n + tb - 1) / tb;
  return q;
}

// Shared prefixes: the walk goes over the groups, then over the requests.  A group
// counts as a request whose nodes are all of its requests' rows and whose tokens
// are the prefix, all of them before the nodes; a request of it keeps the tokens
// behind the prefix.
__device__ __forceinline__ Req group_request(const AttnArgs& a, const PrefixGroup& g, int tb) {
  Req q;
  q.q0 = min(max(a.q_start[g.begin], 0), a.T);
  const int q1 = min(max(a.q_start[g.end], q.q0), a.T);
  q.n = g.pages ? q1 - q.q0 : 0;
  q.ctx = q.kv = g.pages << a.page_shift;
  q.tiles = max((q.kv + kAttnTile - 1) / kAttnTile, 1);
  q.blocks = (q.n + tb - 1) / tb;
  q.row = g.row;
  q.skip = 0;
  q.flags = kPrefix;
  return q;
}
// what request q keeps behind a prefix of `pages` pages
__device__ __forceinline__ void behind_prefix(const AttnArgs& a, Req& q, int pages) {
  const int prefix = pages << a.page_shift;    // at most the row's tokens
  if (pages && q.ctx >= prefix) {              // (a shorter context has the prefix in its own row alone)
    q.ctx -= prefix;
    q.kv -= prefix;
    q.tiles = max((q.kv + kAttnTile - 1) / kAttnTile, 1);
    q.skip = pages;
    q.flags = kJoined;
  }
}
__device__ __forceinline__ Req own_request(const AttnArgs& a, int r, int pages, int tb, int* bad) {
  Req q = request(a, r, tb, bad);
  q.row = r;
  q.skip = q.flags = 0;
  behind_prefix(a, q, pages);
  return q;
}
// whether the kernel for few rows takes a step of the walk (else the one of 128-row tiles does)
__device__ __forceinline__ bool few(const AttnArgs& a, const Req& q) {
  return q.n <= a.few_tokens && q.kv <= a.few_keys;
}

// Where the partials of a token's rows of one unit are, by `parts`: 0: nowhere (the
// output is written); 1: whole, by the rows' own numbers; more: that many slots from
// `at` on, of runs of tiles or of the kernel for few rows
struct PartsOf {
  int parts, at, row, flags;                   // row: the token's first row of the unit's tile; kJoined, kFewSlots
};
constexpr int kFewSlots = 1;
static_assert(sizeof(PartsOf) == sizeof(int4), "a record a token");

// the record of a token's rows: of its group's prefix (which 0), of its own tokens (1)
__device__ __forceinline__ PartsOf parts_of(const AttnArgs& a, int which, int h, int tok) {
  const int4 x = __ldcg(&a.parts_of[(int64_t)(which * a.Hkv + h) * a.T + tok]);
  // slots of runs: the first run's second, then the next runs' first ones; of few rows: every kFewBlocks'th
  const int last = x.y + (x.w & kFewSlots ? kFewBlocks * (x.x - 1) : 2 * x.x - 3);
  // (bad row starts leave a token without a unit: what stands there then is not followed)
  const bool good = x.x >= 0 && x.x <= kAttnMaxCtas && x.y >= 0 && x.y < (int)(kAttnPartSlots + kFewCtas * kFewBlocks) && x.z >= 0 &&
                    (x.x < 2 || (x.w & kFewSlots ? last < kFewCtas * kFewBlocks && x.z <= kFewRows - a.G
                                                 : (x.y & 1) && last < (int)kAttnPartSlots && x.z <= 2 * kAttnRows - a.G));
  return good ? PartsOf{x.x, x.y, x.z, x.w} : PartsOf{0, 0, 0, 0};
}
// partial i of a row (number rg of the KV head's T * G, head `head` of its token): its (max, sum) and its columns
template <int DP>
__device__ __forceinline__ void partial(const AttnArgs& a, const PartsOf& p, int which, int h, int rg, int head, int i,
                                        const float2*& ml, const float4*& v) {
  int64_t at;
  if (p.parts == 1) {
    at = (int64_t)(which * a.Hkv + h) * (a.T * a.G) + rg;
    ml = a.rows_ml + at;
    v = reinterpret_cast<const float4*>(a.rows_part);
  } else if (p.flags & kFewSlots) {
    at = (int64_t)(p.at + kFewBlocks * i) * kFewRows + p.row + head;
    ml = a.few_ml + at;
    v = reinterpret_cast<const float4*>(a.few_part);
  } else {
    at = (int64_t)(i == 0 ? p.at : p.at - 1 + 2 * i) * (2 * kAttnRows) + p.row + head;
    ml = a.pair_ml + at;
    v = reinterpret_cast<const float4*>(a.pair_part);
  }
  v += at * (DP / 4);
}

}  // namespace moe
