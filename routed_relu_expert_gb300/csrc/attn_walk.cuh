// Requests and groups as the attention kernels walk over them.
#pragma once

#include "attn.h"

namespace moe {

// For a kernel whose successor hardly depends on it (no other kernel lets its successor start early): its blocks call
// this after their own pdl_wait, so that the successor, which then need not wait to read what came before both, may
// start where they end; it still waits before it ends.
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// flags of a Req: a group's prefix; own tokens of rows that have a prefix beside them
constexpr int kPrefix = 8, kJoined = 16;

struct Req {
  int q0, n, kv, ctx, tiles, blocks;
  int row, skip, flags;    // (shared prefixes) the table's row, its pages before the first tile; kPrefix or kJoined
};

// a request from its row starts and its length
__device__ __forceinline__ Req request_of(const AttnArgs& a, int start, int next, int kv, int tb, int* bad) {
  Req q;
  q.q0 = min(max(start, 0), a.T);
  const int q1 = min(max(next, q.q0), a.T);
  q.n = q1 - q.q0;
  // a length past the table's row is cut there: its tokens before that stay where they are, nodes among them or not
  const int cap = a.max_pages << a.page_shift;             // at most 2^30
  q.ctx = min(max(kv, q.n) - q.n, cap);
  q.kv = min(q.ctx + q.n, cap);
  if (bad && (kv < q.n || kv > cap || q.q0 != start)) *bad = 1;
  q.tiles = max((q.kv + kAttnTile - 1) / kAttnTile, 1);
  q.blocks = (q.n + tb - 1) / tb;
  return q;
}

__device__ __forceinline__ Req request(const AttnArgs& a, int r, int tb, int* bad) {
  return request_of(a, a.q_start[r], a.q_start[r + 1], a.kv_len[r], tb, bad);
}

// Shared prefixes: the walk goes over the groups, then over the requests.  A group
// counts as a request whose nodes are all of its requests' rows and whose tokens
// are the prefix, all of them before the nodes; a request of it keeps the tokens
// behind the prefix.
// Groups whose bounds do not ascend (`mixed`: in one place at least, so that some of them may overlap, and a row
// would have the partials of two) share nothing.
__device__ __forceinline__ Req group_request(const AttnArgs& a, int group, bool mixed, int tb, int* bad) {
  PrefixGroup g = prefix_group(a.group_start, a.prefix_row, a.prefix_len, group, a.R, a.max_pages, a.page_shift, bad);
  if (mixed) g.pages = 0;
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
  return q.n <= a.few_tokens;
}

// pages of each request's group's prefix, into shared memory; `start`: 3 n_groups + 1 words of it for the meanwhile;
// *mixed (in shared memory, too): whether the groups' bounds do not ascend
template <int kThreads>
__device__ __forceinline__ void prefix_pages(const AttnArgs& a, int32_t* start, int* skip, int* mixed) {
  int32_t *rows = start + a.n_groups + 1, *lens = rows + a.n_groups;
  bool descends = false;
  if (a.n_groups)
    for (int g = threadIdx.x; g <= a.n_groups; g += kThreads) {
      const bool group = g < a.n_groups;
      const int at = a.group_start[g], next = group ? a.group_start[g + 1] : at;
      const int row = group ? a.prefix_row[g] : 0, len = group ? a.prefix_len[g] : 0;
      start[g] = at;                           // (all loads come before the stores)
      if (group) {
        rows[g] = row;
        lens[g] = len;
      }
      descends |= next < at;
    }
  descends = __syncthreads_or(descends);
  if (threadIdx.x == 0) *mixed = descends;
  for (int r = threadIdx.x; r < a.R; r += kThreads) {
    const int g = descends ? -1 : group_of(start, a.n_groups, r);
    int pages = 0;
    if (g >= 0) {
      const PrefixGroup p = prefix_group(start, rows, lens, g, a.R, a.max_pages, a.page_shift, nullptr);
      if (r < p.end) pages = p.pages;
    }
    skip[r] = pages;
  }
  __syncthreads();
}

// exclusive prefix of one value a thread over the block; *all: their sum
template <int kThreads>
__device__ __forceinline__ int64_t block_prefix(int64_t mine, int64_t* scan, int64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  int64_t before = x - mine, sum = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t s = scan[w];
    if (w < warp) before += s;
    sum += s;
  }
  *all = sum;
  return before;
}

// Where the partials of a token's rows of one unit are, by `parts`: 0: nowhere (the
// output is written); 1: whole, by the rows' own numbers; more: that many slots, the
// second (`at`) of the run that the unit begins in, then the first one of each run after
// it, of the one kernel or the other
struct PartsOf {
  int parts, at, row, flags;                   // row: the token's first row of the unit's tile; kJoined, kFewSlots
};
constexpr int kFewSlots = 1;
static_assert(sizeof(PartsOf) == sizeof(int4), "a record a token");

// the record of a token's rows: of its group's prefix (which 0), of its own tokens (1)
__device__ __forceinline__ PartsOf parts_of(const AttnArgs& a, int which, int h, int tok) {
  const int4 x = __ldcg(&a.parts_of[(int64_t)(which * a.Hkv + h) * a.T + tok]);
  const bool of_few = x.w & kFewSlots;
  const int slots = of_few ? 2 * kFewRuns : (int)kAttnPartSlots, rows = of_few ? kFewRows : 2 * kAttnRows;
  // (bad row starts leave a token without a unit: what stands there then is not followed)
  const bool good = x.x >= 0 && x.x < slots && x.y >= 0 && x.y < slots && x.z >= 0 &&
                    (x.x < 2 || ((x.y & 1) && x.y + 2 * x.x - 3 < slots && x.z <= rows - a.G));
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
  } else {
    const bool of_few = p.flags & kFewSlots;
    at = (int64_t)(i == 0 ? p.at : p.at - 1 + 2 * i) * (of_few ? kFewRows : 2 * kAttnRows) + p.row + head;
    ml = (of_few ? a.few_ml : a.pair_ml) + at;
    v = reinterpret_cast<const float4*>(of_few ? a.few_part : a.pair_part);
  }
  v += at * (DP / 4);
}

}  // namespace moe
