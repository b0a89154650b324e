// Tree attention over a paged cache on the tensor cores (tcgen05, BF16 rows and
// caches, FP32 scores, softmax and sums).
//
//   S = Q K^T,  p = exp2(c S - m),  l = sum p,  O = sum p V,  out = O / l
//   c = softmax_scale log2(e); m a running upper reference of c S (below)
//
// Rows.  A unit is (request, KV head, block of up to 128 / G nodes): its nodes'
// G query heads are the 128 rows of one MMA tile, so a KV head's keys are read
// once for all of them.
//
// Work.  A unit's keys are tiles of 128.  The tiles of all units, in order, are
// cut into equal runs, one per CTA (one CTA an SM): the lengths are read on the
// device, no call needs them on the host, and with one row block a KV head (single
// tokens, small trees) every SM streams the same number of keys whatever the batch.
// A chain of several blocks (a prompt) is charged all of its request's tiles for each
// of them, though a block sees only those up to its last node: runs over the first
// blocks end early (figures below).  A unit cut by a run's end leaves FP32 partials
// (at most two a CTA) and a second small kernel adds them in run order.
//
// Inside a CTA: warps 8 and 10 bring K and V tiles into a ring by TMA, a box per
// page and 64-wide half (any page size from 8 on; the table's entries are fetched
// two tiles ahead); warp 9 issues the MMAs; warp 11 works the run's pieces out
// ahead and loads their Q; warps 0-3 and 4-7 are two softmax groups, a thread a row
// and half of the tile's keys.  S and P have two buffers each in tensor memory (with
// O they fill it): S runs two tiles ahead, so that the next tile's scores come to a
// thread's registers beside this one's exponentials.  P goes back to tensor memory
// as the A operand of P V; V is the MN-major B operand as it lies.  A row's two
// threads exchange their maxima through shared memory.
//
// The running maximum and sum are the online softmax of Milakov and Gimelshein
// ("Online normalizer calculation for softmax", 2018), but the reference m of a row
// follows its maximum only when that rose by more than 2^8: below that p and the sums
// just grow by at most 2^8, which the division undoes, and O is left alone.
//
// P is rounded to BF16 for the second product (the tensor cores take one 16-bit type
// for both operands, and V is BF16), at most half a step, 2^-8, of each p; l sums p
// before it.  Against 64 bits the outputs are off by 1.7 to 2.3e-3 of their norm where
// P in FP32 gives 1.5 to 1.7e-3, nearly all of that the store's own rounding.
//
// Bound and measures (GB300, 32 heads over 8 KV heads of 128 unless said): HBM
// while a KV head's rows are few: one request of 262,001 tokens with 16 nodes
// 164 to 167 us = 6.4 to 6.6 TB/s, 64 ragged requests of up to 8,000 tokens and trees of
// up to 8 176 to 185 us = 5.7 to 6.0 TB/s (the mean CTA streams at 6.8), of up to 16,000
// tokens with heads of 64 253 us = 4.2 TB/s (a tile's bytes halve, its chain does not).
// With 128 rows a tile's chain (scores ready, exponentials, P stored, maxima exchanged),
// about 1700 cycles where its products need 1024: 32 requests with trees of up to 64 and
// 16 query heads a KV head 88 to 94 us = 715 to 765 TFLOP/s, 2048 rows behind 8192 cached
// tokens 355 us = 870.  Prompts: one of 8192 rows 1672 us = 329 TFLOP/s, four of 2048
// 437 us = 315 (the busiest run has nearly twice the mean work).  The other split
// measured, tiles of 64 keys that the two groups take in turn, each with its own
// reference and O and no exchange, doubles a tile's fixed waits: 143 us for the large
// trees, 203 us for the long request.
//
// Masked places.  Only the tiles that hold nodes or end past the last key look
// at masks; there, V rows past the last key are zeroed in shared memory (P is 0,
// but 0 x NaN is not), and V rows of nodes that are not finite are zeroed too and
// added by hand to the rows that see them.
#include "attn_tc.cuh"
#include "attn_walk.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {

namespace {

using namespace tc;

constexpr int kTile = kAttnTile;               // keys a tile
constexpr int kSoftWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + 4);
constexpr int kLoaders = 2;                    // warps that issue the TMA copies
constexpr int kQueue = 4;                      // pieces worked out ahead

constexpr uint32_t kTmemCols = 512;

template <int DP>
struct Geo {
  static constexpr int NH = DP / 64;                       // 64-wide halves of a head
  static constexpr int SLOT = NH * kHalfBytes;             // a K or V tile
  static constexpr int SLOTS = DP == 128 ? 5 : 10;         // 160 KB in flight
  static constexpr int RING = SLOTS * SLOT;
  // tensor memory columns: S0 S1 (128 each), P0 P1 (64 each, BF16 pairs), O
  static __host__ __device__ constexpr uint32_t s_col(int b) { return 128u * b; }
  static __host__ __device__ constexpr uint32_t p_col(int b) { return 256u + 64u * b; }
  static constexpr uint32_t O = 384;
};

struct Maps {
  CUtensorMap q, k, v;
};

// a run's part of one unit
struct Piece {
  int r, h;                // request, KV head
  int row0, tok0, ntok;    // first row of the block in q; its first node and its nodes
  int ctx, kv;             // tokens before the nodes; all tokens of the table's row (at most ctx + nodes)
  int t0, n;               // first tile and number of tiles (those that a chain's block can see)
  int flags;               // kStarts, kEnds, kLast
  int parts;               // of a unit that starts here and ends in a later run: its runs
};
constexpr int kStarts = 1, kEnds = 2, kLast = 4;

// fixed shared-memory words after the tiles
struct Small {
  uint64_t full[10], empty[10];
  uint64_t piece_full[kQueue], piece_empty[kQueue];
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done[2], o_free, s_free[2], meet, group, drain;
  float top[2][2][kAttnRows];                  // [tile parity][group][row] maxima of the halves
  float sum[2][2][kAttnRows];                  // [piece parity][group][row]
  uint32_t odd[2][2][4];                       // [tile parity][half of the head]: nodes whose V is not finite
  Piece piece[kQueue];
  Req first;                                   // request that the run begins in
  int first_r;
  uint32_t tmem;
  int abort;
  int64_t scan[kThreads / 32];
};

// the barrier of the two softmax warps that share rows (hardware barriers 1 .. 4)
__device__ __forceinline__ void pair_sync(int q) { asm volatile("bar.sync %0, 64;" ::"r"(q + 1) : "memory"); }
__device__ __forceinline__ void pair_arrive(int q) { asm volatile("bar.arrive %0, 64;" ::"r"(q + 1) : "memory"); }

// order of a piece's tiles in the ring: K0, K1, [K2, V0], [K3, V1], ..., V(n-2), V(n-1)
__device__ __forceinline__ int v_item(int j, int n) {
  return j >= n - 2 ? 2 * n - (n - j) : 2 * j + 3;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_kernel(const __grid_constant__ Maps maps, const AttnArgs a, int tb) {
  using X = Geo<DP>;
  constexpr int NS = X::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t q_smem = (raw + 1023u) & ~1023u;
  uint8_t* q_ptr = smem_raw + (q_smem - raw);
  const uint32_t ring = q_smem + X::SLOT;
  uint8_t* ring_ptr = q_ptr + X::SLOT;
  Small& sm = *reinterpret_cast<Small*>(ring_ptr + X::RING);
  int* prefix = reinterpret_cast<int*>(&sm + 1);           // [R + 1]
  volatile int* abort_flag = &sm.abort;
  int32_t* err = &a.hdr->err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(sm.full[s]), kLoaders);
      mbar_init(bar(sm.empty[s]), 1);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(bar(sm.piece_full[i]), 1);
      mbar_init(bar(sm.piece_empty[i]), kSoftWarps + 1 + kLoaders);
    }
    mbar_init(bar(sm.q_full), 1);
    mbar_init(bar(sm.q_empty), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(sm.s_full[w]), 1);
      mbar_init(bar(sm.p_full[w]), kSoftWarps);
      mbar_init(bar(sm.pv_done[w]), 1);
    }
    mbar_init(bar(sm.group), kSoftWarps);
    mbar_init(bar(sm.o_free), kSoftWarps);
    for (int b = 0; b < 2; ++b) mbar_init(bar(sm.s_free[b]), kSoftWarps);
    mbar_init(bar(sm.meet), kSoftWarps);
    mbar_init(bar(sm.drain), 1);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8 && lane < 3) {
    const CUtensorMap* map = lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  // cost before each request: its units' tiles and fixed costs; this CTA's run of the total, and the request that
  // the run begins in (with what its thread has read of it)
  int total, runs, share, extra;
  // run c begins after c shares, the first `extra` of them one longer
  auto run_start = [&](int c) { return c * share + min(c, extra); };
  {
    int bad = 0;
    const int per = (a.R + kThreads - 1) / kThreads, r0 = min((int)threadIdx.x * per, a.R), r1 = min(r0 + per, a.R);
    auto cost = [&](const Req& q) { return (q.tiles + kAttnPieceCost) * q.blocks * a.Hkv; };
    Req q;
    int64_t local = 0;                                     // (one request's cost fits 31 bits; row starts that are no
    for (int r = r0; r < r1; ++r) {                        // prefix sums may not add up to so few)
      q = request(a, r, tb, &bad);
      local += cost(q);
    }
    int64_t x = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) sm.scan[warp] = x;
    __syncthreads();
    int64_t before = x - local, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int64_t s = sm.scan[w];
      if (w < warp) before += s;
      all += s;
    }
    if (all > INT32_MAX) {
      bad = 1;
      all = 0;                                             // nothing is computed
    }
    total = (int)all;
    int run = (int)before;
    runs = min((int)gridDim.x, max(total, 1));
    share = total / runs;
    extra = total - share * runs;
    const int begin = run_start(blockIdx.x);
    for (int r = r0; r < r1; ++r) {
      if (per > 1) q = request(a, r, tb, nullptr);
      prefix[r] = run;
      const int next = run + cost(q);
      if (run <= begin && begin < next) {
        sm.first_r = r;
        sm.first = q;
      }
      run = next;
    }
    if (threadIdx.x == 0) prefix[a.R] = total;
    if (bad && blockIdx.x == 0) set_error(err, MOE_DEVERR_CACHE);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const bool idle = (int)blockIdx.x >= runs;
  const int begin = idle ? 0 : run_start(blockIdx.x), end = idle ? 0 : run_start(blockIdx.x + 1);

  // the next piece of the queue, for every warp but the one that fills it
  int taken = 0;
  auto next = [&](Piece& p) {
    const int e = taken % kQueue;
    if (!wait_warp<4>(bar(sm.piece_full[e]), (uint32_t)(taken / kQueue) & 1u, abort_flag, err)) return false;
    p = sm.piece[e];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(sm.piece_empty[e]));
    ++taken;
    return !(p.flags & kLast);
  };

  if (warp == 11) {
    // ---------------- the run's pieces, worked out ahead of the other warps, and their Q ----------------
    // a unit's cost is kAttnPieceCost, then a tile each
    auto owner = [&](int at) {                             // the run that holds position `at`
      const int longer = (share + 1) * extra;              // positions in the longer runs
      return at < longer ? at / (share + 1) : extra + (at - longer) / share;
    };
    int pos = begin, made = 0, loads = 0;
    bool last = false;
    Req q = sm.first;                                      // (not read where the run is empty)
    int r = sm.first_r, have = r;
    while (!last) {
      Piece p;
      last = pos >= end;
      p.flags = kLast;
      if (!last) {
        while (prefix[r + 1] <= pos) ++r;
        if (have != r) q = request(a, r, tb, nullptr);
        have = r;
        const int per = q.tiles + kAttnPieceCost, u = (pos - prefix[r]) / per, off = pos - prefix[r] - u * per;
        const int len = min(per - off, end - pos), t0 = max(off - kAttnPieceCost, 0);
        int t1 = off + len - kAttnPieceCost;
        const int unit_end = pos - off + per;
        pos += len;
        if (t1 <= t0) continue;                            // the fixed cost alone
        p.r = r;
        p.h = u / q.blocks;
        p.tok0 = (u - p.h * q.blocks) * tb;
        p.ntok = min(tb, q.n - p.tok0);
        p.row0 = q.q0 + p.tok0;
        p.ctx = q.ctx;
        p.kv = q.kv;
        p.t0 = t0;
        p.flags = (t0 == 0 ? kStarts : 0) | (t1 == q.tiles ? kEnds : 0);
        p.parts = p.flags == kStarts ? owner(unit_end - 1) - (int)blockIdx.x + 1 : 0;
        if (!a.tree_mask) t1 = min(t1, (q.ctx + p.tok0 + p.ntok + kTile - 1) / kTile);
        p.n = max(t1 - t0, 0);
      }
      const int e = made % kQueue;
      if (made >= kQueue &&
          !wait_warp<1>(bar(sm.piece_empty[e]), ((uint32_t)(made / kQueue) & 1u) ^ 1u, abort_flag, err))
        break;
      if (lane == 0) {
        sm.piece[e] = p;
        mbar_arrive(bar(sm.piece_full[e]));
      }
      __syncwarp();
      ++made;
      if (last || p.n == 0) continue;
      // Q, once the last S of the piece before is done; K and V of this piece are on their way meanwhile
      if (loads > 0 && !wait_warp<1>(bar(sm.q_empty), (loads & 1) ^ 1, abort_flag, err)) break;
      if (elect_one()) {
        mbar_expect_tx(bar(sm.q_full), (uint32_t)(X::NH * 128 * a.G * tb));
#pragma unroll
        for (int hh = 0; hh < X::NH; ++hh)
          tma_load_3d(q_smem + hh * kHalfBytes, &maps.q, 64 * hh, p.h * a.G, p.row0, bar(sm.q_full));
      }
      __syncwarp();
      ++loads;
    }
    if (*abort_flag && loads > 0) {
      // the copy in flight must land before the CTA leaves
      const uint64_t t0 = globaltimer();
      while (!mbar_try(bar(sm.q_full), (uint32_t)(loads - 1) & 1u) && globaltimer() - t0 < kWaitLimitNs) {
      }
      __syncwarp();
    }
  } else if (warp == 8 || warp == 10) {
    // ---------------- K and V into shared memory ----------------
    // the boxes of a tile (page by page, half by half) are shared between the two loaders
    const int who = warp == 8 ? 0 : 1;
    const int page = 1 << a.page_shift, rows = min(page, kTile);
    const int per_tile = kTile / rows;                     // boxes of a half: lane l < per_tile has box l
    int slot = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (Piece p; ok && next(p);) {
      if (p.n == 0) continue;
      const int32_t* table = a.block_table + (int64_t)p.r * a.max_pages;
      // page of this lane's box of tile j (of the piece); -1: nothing to load
      auto page_of = [&](int j) {
        const int tok = (p.t0 + j) * kTile + lane * rows;
        if (j >= p.n || lane >= per_tile || tok >= p.kv) return -1;
        const int id = table[tok >> a.page_shift];
        if (id >= 0 && id < a.n_pages) return id;
        set_error(err, MOE_DEVERR_CACHE);
        return a.n_pages;                                  // past the last page: TMA fills zeros
      };
      int id[4] = {page_of(0), page_of(1), page_of(2), -1};   // tiles j .. j + 3
      auto load = [&](const CUtensorMap* map, int j, int pid) {
        if (it >= NS) ok = wait_warp<1>(bar(sm.empty[slot]), phase ^ 1u, abort_flag, err);
        if (!ok) return;
        const int boxes = __popc(__ballot_sync(0xffffffffu, pid >= 0));   // lanes 0 .. boxes - 1
        const int off = ((p.t0 + j) * kTile) & (page - 1);                // pages larger than a tile
        const uint32_t b = bar(sm.full[slot]);
        // two halves: one each; one half: every other box
        const int hh = X::NH == 2 ? who : 0, first = X::NH == 2 ? 0 : who, step = X::NH == 2 ? 1 : kLoaders;
        const uint32_t dst = ring + (uint32_t)(slot * X::SLOT + hh * kHalfBytes);
        if (elect_one()) mbar_expect_tx(b, (uint32_t)((boxes - first + step - 1) / step * 128 * rows));
        __syncwarp();
        for (int i = first; i < boxes; i += step) {
          const int pg = __shfl_sync(0xffffffffu, pid, i);
          if (elect_one()) tma_load_4d(dst + (uint32_t)(i * rows * 128), map, 64 * hh, off, p.h, pg, b);
        }
        __syncwarp();
        ++it;
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
      };
      load(&maps.k, 0, id[0]);
      if (ok && p.n > 1) load(&maps.k, 1, id[1]);
      for (int j = 0; j < p.n && ok; ++j) {
        id[3] = page_of(j + 3);
        if (j + 2 < p.n) load(&maps.k, j + 2, id[2]);
        if (ok) load(&maps.v, j, id[0]);
        id[0] = id[1];
        id[1] = id[2];
        id[2] = id[3];
      }
    }
    if (*abort_flag && lane == 0) {
      // copies in flight must land before the CTA leaves
      const uint64_t t0 = globaltimer();
      auto land = [&](uint32_t b, uint32_t parity) {
        while (!mbar_try(b, parity) && globaltimer() - t0 < kWaitLimitNs) {
        }
      };
      for (int s = 0; s < NS; ++s) {
        const int uses = (it - s + NS - 1) / NS;           // times that slot s was filled
        if (it > s) land(bar(sm.full[s]), (uint32_t)(uses - 1) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------- MMA issuer ----------------
    // the whole warp walks and waits; one elected thread issues (a branch on the
    // lane number instead costs 170 to 250 cycles an MMA: the operands then reach
    // the uniform registers that the instruction takes one lane at a time)
    const uint32_t id_s = idesc_f16kind(kAttnRows, kTile, false);
    const uint32_t id_o = idesc_f16kind(kAttnRows, DP, false) | (1u << 16);      // B is MN-major
    int slot = 0, pieces = 0;
    uint32_t phase = 0;
    int tiles = 0;                                       // of all pieces so far; buffer b = tile & 1
    bool ok = true, issued = false;
    auto wait = [&](uint64_t& b, uint32_t parity) {
      ok = ok && wait_warp(bar(b), parity, abort_flag, err);
      return ok;
    };
    auto advance = [&]() {
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    };
    for (Piece p; ok && next(p);) {
      if (p.n == 0) continue;
      if (!wait(sm.q_full, pieces & 1)) break;
      auto scores = [&](int j) {
        const int b = (tiles + j) & 1;
        if (!wait(sm.full[slot], phase)) return;
        // the buffer's last S has been read
        if (tiles + j >= 2 && !wait(sm.s_free[b], (uint32_t)(((tiles + j) >> 1) - 1) & 1u)) return;
        tc_fence_after();
        issued = true;
        if (elect_one()) {
          const uint64_t da = smem_desc_sw128(q_smem), db = smem_desc_sw128(ring + (uint32_t)(slot * X::SLOT));
          const uint32_t d = tmem + X::s_col(b);
#pragma unroll
          for (int hh = 0; hh < X::NH; ++hh)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t step = hh * (kHalfBytes >> 4) + 2 * k;
              tc_mma<1>(d, da + step, db + step, id_s, (hh | k) != 0);
            }
          tc_commit<1>(bar(sm.empty[slot]));
          tc_commit<1>(bar(sm.s_full[b]));
          if (j == p.n - 1) tc_commit<1>(bar(sm.q_empty));
        }
        __syncwarp();
        advance();
      };
      // S runs two tiles ahead of P V
      scores(0);
      if (p.n > 1) scores(1);
      for (int j = 0; j < p.n && ok; ++j) {
        if (j + 2 < p.n) scores(j + 2);
        const int b = (tiles + j) & 1;
        if (!wait(sm.full[slot], phase) || !wait(sm.p_full[b], (uint32_t)((tiles + j) >> 1) & 1u)) break;
        // O of the previous piece has been read
        if (j == 0 && !wait(sm.o_free, (pieces & 1) ^ 1)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t db = v_desc(ring + (uint32_t)(slot * X::SLOT));
          const uint32_t d = tmem + X::O, pa = tmem + X::p_col(b);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k) mma_ts(d, pa + 8u * k, db + 128u * k, id_o, (j | k) ? 1u : 0u);
          tc_commit<1>(bar(sm.empty[slot]));
          tc_commit<1>(bar(sm.pv_done[b]));
        }
        __syncwarp();
        advance();
      }
      tiles += p.n;
      ++pieces;
    }
    if (*abort_flag && issued) {
      if (elect_one()) tc_commit<1>(bar(sm.drain));
      const uint64_t t0 = globaltimer();
      while (!mbar_try(bar(sm.drain), 0u) && globaltimer() - t0 < kWaitLimitNs) {
      }
      __syncwarp();
    }
  } else {
    // ---------------- softmax: warps q and q + 4 share rows 32 q .. 32 q + 31, group w has keys 64 w .. 64 w + 63 ----
    const int w = warp >> 2, qd = warp & 3, row = 32 * qd + lane;
    const uint32_t lane_addr = (uint32_t)(32 * qd) << 16;
    const float c = a.scale * 1.4426950408889634f;
    // rows that belong to no request
    {
      const int live = a.R > 0 ? min(max(a.q_start[a.R], 0), a.T) : 0;
      for (int t = live + blockIdx.x; t < a.T; t += gridDim.x) {
        bf16* o = reinterpret_cast<bf16*>(a.out) + (int64_t)t * a.out_ld;
        for (int i = threadIdx.x * 8; i < a.H * a.D; i += 32 * kSoftWarps * 8)
          *reinterpret_cast<uint4*>(o + i) = make_uint4(0, 0, 0, 0);
        if (a.lse)
          for (int i = threadIdx.x; i < a.H; i += 32 * kSoftWarps) a.lse[(int64_t)t * a.H + i] = -INFINITY;
      }
    }
    int tiles = 0, items = 0, meets = 0, groups = 0, pairs = 0;
    bool ok = true, joins = false;
    auto wait = [&](uint64_t& b, uint32_t parity) {
      ok = wait_warp(bar(b), parity, abort_flag, err);
      return ok;
    };
    auto arrive = [&](uint64_t& b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    const int row_tok = row / a.G, row_head = row - row_tok * a.G;
    for (Piece p; ok && next(p);) {
      const int valid = p.ntok * a.G;
      const bool live_warp = 32 * qd < valid;
      const int node = p.tok0 + row_tok;
      const int32_t* mask = a.tree_mask ? a.tree_mask + (int64_t)(p.row0 + min(row_tok, p.ntok - 1)) * a.mask_words
                                        : nullptr;
      // the mask's first words, ahead of the tiles that need them
      const uint32_t m0 = mask ? (uint32_t)mask[0] : 0u, m1 = mask && a.mask_words > 1 ? (uint32_t)mask[1] : 0u;
      float mc = -INFINITY, l = 0.f;

      float v[64];                             // this thread's scores: half of its row's keys of a tile
      auto ready = [&](int j) { return wait(sm.s_full[(tiles + j) & 1], (uint32_t)((tiles + j) >> 1) & 1u); };
      auto scores_at = [&](int j) { return tmem + lane_addr + X::s_col((tiles + j) & 1) + 64u * w; };
      // tile j's scores arrived and masked, their maximum told to the thread of the other half
      auto look = [&](int j) {
        ld32_wait<0>(v);
        ld32_wait<32>(v);
        tc_fence_before();
        arrive(sm.s_free[(tiles + j) & 1]);
        const int key0 = (p.t0 + j) * kTile;
        if (__builtin_expect(key0 + kTile > p.ctx, 0)) {
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int k0 = key0 + 64 * w + 32 * cc, j0 = k0 - p.ctx;   // first key of the word, as a node
            auto low = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
            uint32_t bits;
            if (!mask) {
              bits = low(node + 1 - j0);
            } else {
              auto word = [&](int i) {
                return i < 0 ? 0xffffffffu : i == 0 ? m0 : i == 1 ? m1 : i < a.mask_words ? (uint32_t)mask[i] : 0u;
              };
              const int wi = j0 >> 5;
              bits = j0 + 32 <= 0 ? 0xffffffffu : __funnelshift_r(word(wi), word(wi + 1), (uint32_t)(j0 & 31));
            }
            bits &= low(p.kv - k0);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(bits >> i & 1u)) v[32 * cc + i] = -INFINITY;
          }
        }
        float t4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int i = 4; i < 60; i += 2) t4[(i >> 1) & 3] = max3(t4[(i >> 1) & 3], v[i], v[i + 1]);
        const float top = max3(max3(t4[0], t4[1], v[60]), max3(t4[2], t4[3], v[61]), fmaxf(v[62], v[63]));
        sm.top[pairs & 1][w][row] = top;
        return top;
      };
      // both halves' maxima: the reference for tile j, O scaled to it where it rose
      auto agree = [&](int j, float top, int gone) {
        if (__any_sync(0xffffffffu, gone)) {
          ok = false;
          return;
        }
        pair_sync(qd);
        top = fmaxf(top, sm.top[pairs & 1][w ^ 1][row]) * c;
        ++pairs;
        const bool raise = top > mc + kRaise || (mc == -INFINITY && top > mc);
        if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
          const float f = raise ? (mc == -INFINITY ? 0.f : ex2(mc - top)) : 1.f;
          if (raise) mc = top;
          l *= f;
          if (j > 0) {
            // this group's columns of O, after the tile before
            const int last = tiles + j - 1;
            if (!wait(sm.pv_done[last & 1], (uint32_t)(last >> 1) & 1u)) return;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < DP / 2; c0 += 32) {
              float o[32];
              const uint32_t addr = tmem + lane_addr + X::O + (uint32_t)(w * (DP / 2) + c0);
              ld32_async<0>(addr, o);
              ld32_wait<0>(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= f;
              st32(addr, o);
            }
            st_wait();
          }
        }
      };
      // 32 probabilities, from the CC'th half of the scores; summed before they are rounded to BF16 (above)
      auto exps = [&](auto CC, int b, float base) {
        constexpr int cc = decltype(CC)::value;
        const uint64_t c2 = pair(c, c), base2 = pair(-base, -base);
        uint64_t sum[2] = {0, 0};
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x, y;
          unpair(fma2(pair(v[32 * cc + 2 * i], v[32 * cc + 2 * i + 1]), c2, base2), x, y);
          x = ex2(x);
          y = ex2(y);
          sum[i & 1] = add2(sum[i & 1], pair(x, y));
          pk[i] = pack_bf16(x, y);
        }
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        st16(tmem + lane_addr + X::p_col(b) + 32u * w + 16u * cc, pk);
      };
      // V rows of tile j past the last key, and nodes' rows that are not finite, become zeros (by halves of the
      // head); the nodes of the second kind (read before P is announced: two tiles on, the words are others)
      auto clean = [&](int j) {
        const int b = (tiles + j) & 1, key0 = (p.t0 + j) * kTile;
        const int item = items + v_item(j, p.n);
        const uint4 none = make_uint4(0, 0, 0, 0);
        if (!wait(sm.full[item % NS], (uint32_t)(item / NS) & 1u)) return none;
        const int key = key0 + row;
        uint4* v0 = reinterpret_cast<uint4*>(ring_ptr + (item % NS) * X::SLOT + w * kHalfBytes + row * 128);
        const bool zero = key >= p.kv;
        bool strange = false;
        if (w < X::NH) {
          if (!zero && key >= p.ctx) {
            uint32_t hit = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 x = v0[i ^ (row & 7)];               // (eight lanes, eight bank groups)
              const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                hit |= ((ws[e] & 0x7F80u) == 0x7F80u) | ((ws[e] & 0x7F800000u) == 0x7F800000u);
            }
            strange = hit != 0;
          }
          if (zero || strange) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v0[i ^ (row & 7)] = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        const uint32_t mine = __ballot_sync(0xffffffffu, strange);
        if (lane == 0) sm.odd[b][w][qd] = mine;
        arrive(sm.group);
        if (!wait(sm.group, groups & 1)) return none;
        ++groups;
        return make_uint4(sm.odd[b][w][0], sm.odd[b][w][1], sm.odd[b][w][2], sm.odd[b][w][3]);
      };
      if (p.n > 0 && ready(0) && !live_warp) arrive(sm.s_free[tiles & 1]);
      if (p.n > 0 && ok && live_warp) {
        tc_fence_after();
        ld32_async<0>(scores_at(0), v);
        ld32_async<32>(scores_at(0) + 32, v);
        agree(0, look(0), *abort_flag);
      }
      for (int j = 0; j < p.n && ok; ++j) {
        // tile j's scores are in v and its reference stands; the next tile's replace them half by half, so that
        // their way from tensor memory runs beside the exponentials
        const int b = (tiles + j) & 1, gone = *abort_flag;
        const bool more = j + 1 < p.n;
        const float base = mc == -INFINITY ? 0.f : mc;
        // P of two tiles ago has been multiplied: that product was issued before the next tile's S, and the commit
        // behind s_full covers all that was issued before it
        if (more && !ready(j + 1)) break;
        if (!more && tiles + j >= 2 && !wait(sm.pv_done[b], (uint32_t)(((tiles + j) >> 1) - 1) & 1u)) break;
        if (live_warp) {
          tc_fence_after();
          exps(std::integral_constant<int, 0>(), b, base);
          if (more) ld32_async<0>(scores_at(j + 1), v);
          exps(std::integral_constant<int, 1>(), b, base);
          if (more) ld32_async<32>(scores_at(j + 1) + 32, v);
        }
        uint4 odd = make_uint4(0, 0, 0, 0);
        if (__builtin_expect((p.t0 + j + 1) * kTile > p.ctx, 0)) odd = clean(j);
        if (!ok) break;
        if (live_warp) {
          st_wait();
          tc_fence_before();
        }
        arrive(sm.p_full[b]);
        if (!live_warp) {
          if (more) arrive(sm.s_free[b ^ 1]);
          continue;
        }
        if (__builtin_expect((odd.x | odd.y | odd.z | odd.w) != 0, 0)) {
          // p v of the nodes whose V is not finite
          if (!wait(sm.pv_done[b], (uint32_t)((tiles + j) >> 1) & 1u)) break;
          tc_fence_after();
          add_odd(a, a.block_table + (int64_t)p.r * a.max_pages, p.h, (p.t0 + j) * kTile, odd, 64 * w, tmem + lane_addr + X::p_col(b),
                  tmem + lane_addr + X::O);
          tc_fence_before();
          __syncwarp();
        }
        if (more) agree(j + 1, look(j + 1), gone);
      }
      tiles += p.n;
      if (!ok) break;

      // ---- the piece's end: write the rows or their partials ----
      items += 2 * p.n;
      float(&sums)[2][kAttnRows] = sm.sum[meets & 1];
      sums[w][row] = l;
      if (p.n > 0 && !wait(sm.pv_done[(tiles - 1) & 1], (uint32_t)((tiles - 1) >> 1) & 1u)) break;
      arrive(sm.meet);
      if (!wait(sm.meet, meets & 1)) break;    // both halves' sums are there (and odd nodes are added)
      ++meets;
      tc_fence_after();
      const bool whole = (p.flags & (kStarts | kEnds)) == (kStarts | kEnds);
      const int slot = 2 * (int)blockIdx.x + (p.flags & kStarts ? 1 : 0);
      if (live_warp) {
        const float sum = sums[0][row] + sums[1][row];
        // a row without a visible key has sum 0 and O = 0 (never written if the piece has no tile)
        const float g = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        const bool mine = row < valid;
        const int64_t tok = p.row0 + row_tok;
        const int head = p.h * a.G + row_head;
        // group w writes half of the head's columns
#pragma unroll
        for (int cc = 0; cc < DP / 64; ++cc) {
          const int c0 = w * (DP / 2) + 32 * cc;
          float o[32];
          if (p.n > 0) {
            ld32_async<0>(tmem + lane_addr + X::O + c0, o);
            ld32_wait<0>(o);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = sum == 0.f ? 0.f : o[i] * g;
          if (whole) {
            // a row's 64 bytes of the chunk as one piece: four lanes exchange 16-byte quarters, so that a store of the
            // warp touches 8 lines and not 32
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                                pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
            transpose4(x, lane);
            bf16* out = reinterpret_cast<bf16*>(a.out) + (int64_t)p.row0 * a.out_ld + (int64_t)p.h * a.G * a.D + c0 +
                        8 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r2 = (row & ~3) + i, t2 = r2 / a.G;
              if (r2 < valid && c0 + 8 * (lane & 3) < a.D)
                *reinterpret_cast<uint4*>(out + t2 * a.out_ld + (int64_t)(r2 - t2 * a.G) * a.D) = x[i];
            }
          } else if (mine) {
            // partials: [four columns][row]
            float* out = a.part + (int64_t)slot * kAttnRows * kAttnPartDim + ((c0 / 4) * kAttnRows + row) * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(out + 4 * i * kAttnRows) =
                  make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (mine && w == 0) {
          if (!whole) a.part_ml[slot * kAttnRows + row] = make_float2(mc, sum);
          else if (a.lse) a.lse[tok * a.H + head] = sum == 0.f ? -INFINITY : (mc + log2f(sum)) * 0.6931471805599453f;
        }
      }
      if (p.parts) {
        if (threadIdx.x == 0) a.joins[blockIdx.x] = make_int4(p.parts, p.row0, p.ntok, p.h);
        joins = true;
      }
      if (p.n > 0) {
        tc_fence_before();
        arrive(sm.o_free);
      }
    }
    // a warp that gave up lets its partner through (which then sees the abort flag before it waits again)
    if (*abort_flag) pair_arrive(qd);
    if (threadIdx.x == 0 && !joins) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Units that a run's end cut: run c's unit that began but did not end in it has
// its partials in slot 2c + 1 (its own) and 2 (c + 1), 2 (c + 2), ... of the runs
// after it.  A lane a row, a warp four columns (the partials are laid out for it),
// parts in ascending order; the block's 32 rows meet in shared
// memory to be written whole.
constexpr int kJoinWarps = kAttnPartDim / 4;
constexpr int kJoinAhead = 4;                  // parts in flight (32 registers: two blocks an SM)
__global__ void __launch_bounds__(32 * kJoinWarps, 2) attention_join_kernel(const AttnArgs a) {
  pdl_wait();
  const int4 u = a.joins[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, valid = u.z * a.G;
  const int row0 = blockIdx.y * 32;
  if (u.x < 2 || row0 >= valid) return;
  __shared__ uint2 s_out[32][kJoinWarps + 1];
  const int row = min(row0 + lane, valid - 1);
  auto slot = [&](int p) { return 2 * ((int)blockIdx.x + p) + (p == 0 ? 1 : 0); };
  const float* part = a.part + (warp * kAttnRows + row) * 4;
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < u.x; p += kJoinAhead) {
    float2 ml[kJoinAhead];
    float4 v[kJoinAhead];
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k) {
      const bool in = p + k < u.x;
      ml[k] = in ? a.part_ml[slot(p + k) * kAttnRows + row] : make_float2(0.f, 0.f);
      v[k] = in ? *reinterpret_cast<const float4*>(part + (int64_t)slot(p + k) * kAttnRows * kAttnPartDim)
                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float t = top;
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k)
      if (ml[k].y != 0.f) t = fmaxf(t, ml[k].x);
    const float g = sum == 0.f ? 0.f : ex2(top - t);
    top = t;
    sum *= g;
    acc = make_float4(acc.x * g, acc.y * g, acc.z * g, acc.w * g);
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k) {
      if (ml[k].y == 0.f) continue;            // no visible key in that part
      const float f = ex2(ml[k].x - top);
      sum = fmaf(ml[k].y, f, sum);
      acc.x = fmaf(v[k].x, f, acc.x);
      acc.y = fmaf(v[k].y, f, acc.y);
      acc.z = fmaf(v[k].z, f, acc.z);
      acc.w = fmaf(v[k].w, f, acc.w);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  s_out[lane][warp] = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse && warp == 0 && row0 + lane < valid)
    a.lse[(int64_t)(u.y + row / a.G) * a.H + u.w * a.G + row % a.G] =
        sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  __syncthreads();
  const int per_row = a.D / 4;                 // warps of the block
  const int r = threadIdx.x / per_row, r2 = row0 + r, c = threadIdx.x - r * per_row;
  if (r2 < valid)
    *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(a.out) + (int64_t)(u.y + r2 / a.G) * a.out_ld +
                              (int64_t)(u.w * a.G + r2 % a.G) * a.D + 4 * c) = s_out[r][c];
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int DP>
cudaError_t launch_dp(const AttnArgs& a, cudaStream_t s) {
  using X = Geo<DP>;
  const int tb = kAttnRows / a.G, page = 1 << a.page_shift;
  Maps maps;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.H, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)(a.T > 1 ? a.q_ld : (int64_t)a.H * a.D) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)tb};
    if (!make_map(&maps.q, a.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)page, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)a.token_stride * 2,
                                   (cuuint64_t)(a.Hkv > 1 ? a.head_stride : a.token_stride) * 2,
                                   (cuuint64_t)a.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min(page, kTile), 1, 1};
    if (!make_map(&maps.k, a.k, 4, dims, strides, box) || !make_map(&maps.v, a.v, 4, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  const size_t smem = 1024 + X::SLOT + X::RING + sizeof(Small) + ((size_t)a.R + 1) * 4;
  static_assert(1024 + X::SLOT + X::RING + sizeof(Small) + 4097 * 4 <= kMaxSmem, "shared memory");
  static PerDeviceOnce once;
  int sms = 0;
  cudaError_t e = once.run(
      [](int& v) {
        v = std::min(num_sms(), kAttnMaxCtas);
        return cudaFuncSetAttribute(attention_tc_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      },
      &sms);
  if (e != cudaSuccess) return e;
  e = launch_k(attention_tc_kernel<DP>, dim3((unsigned)sms), dim3(kThreads), smem, s, maps, a, tb);
  if (e != cudaSuccess) return e;
  return launch_k(attention_join_kernel, dim3((unsigned)sms, (unsigned)ceil_div(std::min(tb, a.T) * a.G, 32)), dim3(32 * (a.D / 4)), 0,
                  s, a);
}

}  // namespace

cudaError_t launch_attention_bf16(const AttnArgs& a, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  return a.D <= 64 ? launch_dp<64>(a, s) : launch_dp<128>(a, s);
}

}  // namespace moe
