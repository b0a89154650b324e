// Block tables, slot maps, positions and tree masks of a step, from its
// request lengths (page "NemotronH (Nemotron 3.5 Lightning, Bolt, Super VL)",
// section "Speculation": verify blocks of drafted rows; the paged cache itself
// has no counterpart in the pages).
//
//   held(c) = ceil(c / S);  more_r = held(ctx + n) - held(ctx)
//   base_r = *free_head + sum_{s < r} more_s;  q_start_r = sum_{s < r} n_s
//
// One launch without a grid-wide wait: every block sums all R lengths itself
// (8 R bytes, out of L2 after the first block) and so knows the prefix of its own
// requests; nothing it needs is written by another block.  That cost grows with R
// squared: a token for each of 2048 requests 5 us, 4096 11 us, 16384 95 us.  The one value
// that all blocks read and one writes, *free_head (it may be updated in place),
// is written by the block whose ticket says that every block has read it.
//
// A warp (or, for long requests, all eight warps of a block and several blocks)
// takes a request's nodes, a lane a node.  The bound is the latency of the
// dependent steps (lengths, table entry, slot), not bytes: 3.5 us
// for one request, 4.5 us for 64 with trees of up to 16, 7.7 us for 2048 with trees
// of up to 64 (1.6 MB; 9.7 us with a walk to the root for each node).  Trees of more
// than 64 nodes do walk to the root, a dependent load a level.
#include "attn.h"

#include <algorithm>

namespace moe {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;

struct ReqLen {
  int ctx, n, held, more;
};

__device__ __forceinline__ ReqLen clamp_len(const PlanArgs& a, int ctx, int n, int& bad) {
  ReqLen q;
  if ((ctx | n) < 0) {
    bad |= MOE_DEVERR_CACHE;
    ctx = max(ctx, 0);
    n = max(n, 0);
  }
  if (n > a.T) {                      // cannot have rows for all of them
    bad |= MOE_DEVERR_CACHE;
    n = a.T;
  }
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  if (ctx > cap) {
    bad |= MOE_DEVERR_PAGES;
    ctx = (int)cap;
  }
  const int64_t mask = (1ll << a.page_shift) - 1;
  q.ctx = ctx;
  q.n = n;
  q.held = (int)((ctx + mask) >> a.page_shift);
  int64_t all = ((int64_t)ctx + n + mask) >> a.page_shift;
  if (all > a.max_pages) {
    bad |= MOE_DEVERR_PAGES;
    all = a.max_pages;
  }
  q.more = (int)all - q.held;
  return q;
}

// the block's sums of four values, in every thread
__device__ __forceinline__ void block_sums(int64_t (&v)[4], int64_t (*tmp)[4]) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) tmp[threadIdx.x >> 5][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int64_t s = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) s += tmp[w][i];
    v[i] = s;
  }
}

// parent of node i, -1 where it is not an earlier node
__device__ __forceinline__ int parent_of(const int32_t* par, int i, int& bad) {
  int p = par[i];
  if (p < -1 || p >= i) {
    bad |= MOE_DEVERR_CACHE;
    p = -1;
  }
  return p;
}

// WPR warps a request: 1 (a block has eight requests) or all eight of the block
template <int WPR>
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanArgs a) {
  constexpr int RB = kPlanWarps / WPR;         // requests a block
  pdl_wait();
  __shared__ int64_t tmp[kPlanWarps][4];
  __shared__ int s_ctx[RB], s_n[RB];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r_base = blockIdx.x * RB;
  int bad = 0;

  // totals before this block's requests and over all of them
  int64_t sums[4] = {0, 0, 0, 0};
  for (int r = tid; r < a.R; r += kPlanThreads) {
    const ReqLen q = clamp_len(a, a.ctx_len[r], a.new_len[r], bad);
    sums[0] += q.n;
    sums[1] += q.more;
    if (r < r_base) {
      sums[2] += q.n;
      sums[3] += q.more;
    }
    if (r >= r_base && r < r_base + RB) {
      s_ctx[r - r_base] = q.ctx;
      s_n[r - r_base] = q.n;
    }
  }
  const int head = max(*a.free_head, 0);
  if (*a.free_head < 0) bad |= MOE_DEVERR_CACHE;
  block_sums(sums, tmp);
  const int64_t rows_all = sums[0], more_all = sums[1], rows_before = sums[2], more_before = sums[3];
  if (rows_all > a.T) bad |= MOE_DEVERR_CACHE;
  if (more_all > (int64_t)a.n_free - head) bad |= more_all > 0 ? MOE_DEVERR_PAGES : 0;

  const int rl = warp / WPR, r = r_base + rl;
  if (r < a.R) {
    // prefix over the block's own requests (at most seven before this one)
    int64_t row0 = rows_before, take = head + more_before;
    for (int i = 0; i < rl; ++i) {
      int ignore = 0;
      const ReqLen q = clamp_len(a, s_ctx[i], s_n[i], ignore);
      row0 += q.n;
      take += q.more;
    }
    const ReqLen q = clamp_len(a, s_ctx[rl], s_n[rl], bad);
    const int start = (int)min(row0, (int64_t)a.T);
    const int n = (int)min((int64_t)q.n, (int64_t)a.T - start);
    if (warp % WPR == 0 && blockIdx.y == 0 && lane == 0) {
      a.q_start[r] = start;
      a.kv_len[r] = q.ctx + n;
      if (r == a.R - 1) a.q_start[a.R] = start + n;
    }
    int32_t* table = a.block_table + (int64_t)r * a.max_pages;
    const int lane_r = (warp % WPR) * 32 + lane, lanes = WPR * 32;
    auto fresh = [&](int j) {                  // page of the request's j-th new entry
      const int64_t at = take + j;
      if (at >= a.n_free) return -1;
      const int p = a.free_pages[at];
      if (p < 0 || p >= a.n_pages) {
        bad |= MOE_DEVERR_CACHE;
        return -1;
      }
      return p;
    };
    if (blockIdx.y == 0)
      for (int j = lane_r; j < q.more; j += lanes) table[q.held + j] = fresh(j);

    const int32_t* par = a.parents ? a.parents + start : nullptr;
    const int step = lanes * (int)gridDim.y;
    constexpr int max_doubled = WPR == 1 ? 2 : 1;
    uint32_t first_set = 0;                    // of the request's first 32 nodes
    // every lane of a warp runs every round: the shuffles below need them all
    for (int i0 = lanes * (int)blockIdx.y + (warp % WPR) * 32; i0 < n; i0 += step) {
      const int i = i0 + lane;
      const bool live = i < n;
      if (live) {
        const int64_t at = (int64_t)q.ctx + i;
        const int64_t page_idx = at >> a.page_shift;
        int page = -1;
        if (page_idx < q.held) {               // the partly filled page that the request holds
          page = table[page_idx];
          if (page < 0 || page >= a.n_pages) {
            bad |= MOE_DEVERR_CACHE;
            page = -1;
          }
        } else if (page_idx < a.max_pages) {
          page = fresh((int)(page_idx - q.held));
        }
        a.slot_map[start + i] =
            page < 0 ? -1 : ((int64_t)page << a.page_shift) + (at & ((1ll << a.page_shift) - 1));
        if (!par) a.positions[start + i] = (int)min(at, (int64_t)INT32_MAX);
      }
      if (!par) continue;
      int depth = 0;
      if (n <= 32 * max_doubled && (a.mask_words != 1 || n <= 32)) {
        // trees of up to 32 nodes (64 where one warp has them all): ancestor sets by pointer doubling, five rounds
        // of shuffles a 32 whatever the depth.  Ancestors come before a node, so the first 32 need no others; a node
        // of the second 32 joins its ancestors there with the set of the one of the first that its chain leaves to
        const bool second = i0 > 0;
        const int up = live ? parent_of(par, i, bad) : -1;
        int jump = second ? (up >= 32 ? up - 32 : -1) : up;
        int leave = second && up < 32 ? up : -1;
        uint32_t set = 1u << lane;
#pragma unroll
        for (int round = 0; round < 5; ++round) {
          const uint32_t up_set = __shfl_sync(0xffffffffu, set, jump & 31);
          const int up_jump = __shfl_sync(0xffffffffu, jump, jump & 31);
          const int up_leave = __shfl_sync(0xffffffffu, leave, jump & 31);
          if (jump >= 0) {
            set |= up_set;
            jump = up_jump;
            leave = up_leave;
          }
        }
        const uint32_t below = __shfl_sync(0xffffffffu, first_set, leave & 31);
        const uint32_t low = second ? (leave >= 0 ? below : 0u) : set, high = second ? set : 0u;
        if (!second) first_set = set;
        depth = __popc(low) + __popc(high) - 1;
        if (live && a.tree_mask) {
          int32_t* out = a.tree_mask + (int64_t)(start + i) * a.mask_words;
          out[0] = (int32_t)low;
          if (a.mask_words > 1) out[1] = (int32_t)high;
        }
        // a mask wider than the tree: the warp clears the rest, row by row
        if (a.mask_words > 2)
          for (int j = i0; j < min(i0 + 32, n); ++j) {
            int32_t* out = a.tree_mask + (int64_t)(start + j) * a.mask_words;
            for (int w = 2 + lane; w < a.mask_words; w += 32) out[w] = 0;
          }
      } else if (live) {
        // any size: walk to the root; ancestors descend, so the words of the
        // mask are finished from the last to the first
        int32_t* out = a.tree_mask ? a.tree_mask + (int64_t)(start + i) * a.mask_words : nullptr;
        int word = a.mask_words - 1;
        uint32_t acc = 0;
        int node = i;
        depth = -1;
        while (node >= 0) {
          ++depth;
          const int w = node >> 5;
          if (out && w >= a.mask_words) {
            bad |= MOE_DEVERR_CACHE;
          } else if (out) {
            while (word > w) {
              out[word--] = (int32_t)acc;
              acc = 0;
            }
            acc |= 1u << (node & 31);
          }
          node = parent_of(par, node, bad);
        }
        if (out)
          while (word >= 0) {
            out[word--] = (int32_t)acc;
            acc = 0;
          }
      }
      if (live) a.positions[start + i] = (int)min((int64_t)q.ctx + depth, (int64_t)INT32_MAX);
    }
  }
  if (a.R == 0 && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.q_start[0] = 0;

  // rows past the last node: no token
  const int64_t first = min(rows_all, (int64_t)a.T);
  const int64_t all_threads = (int64_t)gridDim.x * gridDim.y * kPlanThreads;
  for (int64_t i = first + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kPlanThreads + tid; i < a.T;
       i += all_threads) {
    a.positions[i] = 0;
    a.slot_map[i] = -1;
    if (a.tree_mask)
      for (int w = 0; w < a.mask_words; ++w) a.tree_mask[i * a.mask_words + w] = 0;
  }
  if (bad) set_error(&a.hdr->err, bad);
  // block_sums' barrier puts every thread's read of *free_head before this
  if (tid == 0) {
    const int blocks = (int)(gridDim.x * gridDim.y);
    __threadfence();
    if (blocks == 1 || atomicAdd(&a.hdr->plan_ticket, 1) == blocks - 1) {
      a.hdr->plan_ticket = 0;
      *a.free_head_out = (int)min(head + more_all, (int64_t)max(a.n_free, head));
    }
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t s) {
  // long requests (64 rows each on average): a block a request and, past 1024
  // rows a request, several; else a warp a request.  The mean is what the host
  // knows: one long prompt among many single tokens is walked by one warp
  const int64_t per = a.R > 0 ? a.T / a.R : 0;
  if (per >= 64) {
    const unsigned y = (unsigned)std::min<int64_t>(std::max<int64_t>(per / 1024, 1), 32);
    launch_k(paged_plan_kernel<8>, dim3((unsigned)std::max(a.R, 1), y), kPlanThreads, 0, s, a);
  } else {
    launch_k(paged_plan_kernel<1>, dim3((unsigned)std::max<int64_t>(ceil_div(a.R, kPlanWarps), 1)), kPlanThreads, 0,
             s, a);
  }
  return cudaGetLastError();
}

}  // namespace moe
