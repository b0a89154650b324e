// Attention with shared prefixes on the tensor cores (tcgen05, BF16 rows and caches,
// FP32 scores, softmax and sums), for units of many rows, and the join of all units.
//
//   S = Q K^T,  p = exp2(c S - m),  l = sum p,  O = sum p V,  out = O / l
//
// Units.  A group's prefix is one request whose nodes are all rows of the group; what a
// request has behind the prefix is another (attn_walk.cuh).  A unit is (one of those,
// KV head, block of up to 2 x 128 rows); its keys are tiles of 128, and the tiles of all
// units, in order, are cut into equal runs, one per CTA (one CTA an SM).  Units of a few
// rows go to the kernel of attention_few.cu.  Rows with a prefix and units that a run's
// end cuts leave FP32 partials, which prefix_join_kernel adds in a fixed order.
//
// Inside a CTA two tiles of 128 rows take turns on the tensor cores, each with a softmax
// group of four warps, a thread a row: while one tile's scores are exponentiated, the
// products of the other run, and a tile of K and V is read once for 256 rows.  S and P of
// a tile share their columns of tensor memory (P is written over scores that were read);
// the next S of a tile is issued behind its P V, which has read P when it starts.  The
// scores are read twice, for the maximum and for the exponentials, the first half of
// them kept in registers between.
//
// The softmax is the one of attention_tc.cu: a reference that follows the maximum only
// past 2^8, P in BF16 for the second product (half a step, 2^-8, of each), sums before
// that rounding.  As there, only the tiles that hold nodes or end past the last key look
// at masks, V rows past the last key are zeroed in shared memory, and V rows of nodes that
// are not finite are zeroed and added by hand to the rows that see them.
//
// Bound: a step of two row tiles takes about 3500 cycles where its products need 2048: the
// chain of scores, exponentials and P of the tile whose turn it is.  128 requests of up to 4
// nodes behind 8000 common tokens (32 heads over 8 of 128): 49 us for the prefix's 34 GFLOP, 700
// TFLOP/s (in full row tiles 42 GFLOP, 870); with all keys through this kernel the call, replayed alone, took 104 us, with
// attention_few.cu beside it 88; every request through tree attention reads the prefix 128 times.
#include "attn_tc.cuh"
#include "attn_walk.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {

namespace {

constexpr int kTile = kAttnTile;
constexpr int kSoftWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + 4);
constexpr int kLoaders = 2;                    // warps that issue the TMA copies
constexpr int kQueue = 4;                      // pieces worked out ahead
constexpr uint32_t kTmemCols = 512;
// a unit's fixed cost beside its tiles, in tiles
constexpr int kPieceCost = 4;
constexpr int kMinRun = 6;                     // of a run: with fewer, the SMs are the other kernel's sooner

template <int DP>
struct Geo {
  static constexpr int NH = DP / 64;                       // 64-wide halves of a head
  static constexpr int SLOT = NH * kHalfBytes;             // a K or V tile, or 128 rows of Q
  static constexpr int SLOTS = DP == 128 ? 4 : 10;
  static constexpr int RING = SLOTS * SLOT;
  // tensor memory columns of row tile w: S (128; P as BF16 pairs in its first 64) and O
  static __device__ constexpr uint32_t s_col(int w) { return 128u * w; }
  static __device__ constexpr uint32_t o_col(int w) { return 256u + 128u * w; }
};

struct Maps {
  CUtensorMap q, k, v;
};

// a run's part of one unit
struct Piece {
  int row, skip, h;        // the table's row, its pages before the unit's first tile; KV head
  int row0, tok0, ntok[2]; // first row of the block in q; its first node; nodes of its two row tiles
  int ctx, kv;             // tokens before the nodes; all tokens
  int t0, n;               // first tile and number of tiles (those that a chain's block can see)
  int flags;               // kStarts, kEnds, kLast, kPrefix, kJoined
  int parts;               // of a unit that starts here and ends in a later run: its runs
};
constexpr int kStarts = 1, kEnds = 2, kLast = 4;         // beside kPrefix, kJoined

// fixed shared-memory words after the tiles
struct Small {
  uint64_t full[10], empty[10];
  uint64_t piece_full[kQueue], piece_empty[kQueue];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], warm[2], both, first_alone, drain;
  // nodes whose V is not finite: [both groups at it, or the first alone][special tile's parity][half of the head][32 keys]
  uint32_t odd[2][2][2][4];
  Piece piece[kQueue];
  Req first;                                   // step of the walk that the run begins in
  int first_v;
  int mixed;                                   // the groups' bounds do not ascend
  uint32_t tmem;
  int abort;
  int64_t scan[kThreads / 32];
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_prefix_kernel(const __grid_constant__ Maps maps, const AttnArgs a, int tb) {
  using X = Geo<DP>;
  constexpr int NS = X::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t q_smem = (raw + 1023u) & ~1023u;
  uint8_t* q_ptr = smem_raw + (q_smem - raw);
  const uint32_t ring = q_smem + 2 * X::SLOT;
  uint8_t* ring_ptr = q_ptr + 2 * X::SLOT;
  Small& sm = *reinterpret_cast<Small*>(ring_ptr + X::RING);
  const int groups_n = a.n_groups, walk_n = groups_n + a.R;
  int* prefix = reinterpret_cast<int*>(&sm + 1);           // [walk_n + 1] cost before each step of the walk
  int* skip = prefix + walk_n + 1;                         // [R] pages of the request's group's prefix
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
      mbar_init(bar(sm.p_full[w]), kSoftWarps / 2);
      mbar_init(bar(sm.o_full[w]), 1);
      mbar_init(bar(sm.warm[w]), kSoftWarps / 2);
    }
    mbar_init(bar(sm.both), kSoftWarps);
    mbar_init(bar(sm.first_alone), kSoftWarps / 2);
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
  pdl_release();                               // the kernel for few rows fills the SMs as this one's blocks end
  // a step of the walk, once the pages of the groups' prefixes are in `skip`
  auto at_walk = [&](int v, int* bad) {
    Req q;
    if (v < groups_n)
      q = group_request(a, v, sm.mixed, tb, bad);
    else
      q = own_request(a, v - groups_n, skip[v - groups_n], tb, bad);
    if (few(a, q)) q.blocks = 0;
    return q;
  };
  // cost before each step: its units' tiles and fixed costs; this CTA's run of the total, and the step that
  // the run begins in (with what its thread has read of it)
  int total, runs, share, extra;
  // run c begins after c shares, the first `extra` of them one longer
  auto run_start = [&](int c) { return c * share + min(c, extra); };
  {
    int bad = 0;
    // a thread's first request beside the groups, which lie in the ring's memory meanwhile
    const int per = (walk_n + kThreads - 1) / kThreads, v0 = min((int)threadIdx.x * per, walk_n),
              v1 = min(v0 + per, walk_n);
    Req q;
    const bool ahead = v0 < v1 && v0 >= groups_n;
    if (ahead) q = own_request(a, v0 - groups_n, 0, tb, &bad);
    prefix_pages<kThreads>(a, reinterpret_cast<int32_t*>(ring_ptr), skip, &sm.mixed);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");       // (before TMA writes there)
    auto cost = [&](const Req& q) { return (q.tiles + kPieceCost) * q.blocks * a.Hkv; };
    int64_t local = 0;                                     // (one step's cost fits 31 bits; row starts that are no
    for (int v = v0; v < v1; ++v) {                        // prefix sums may not add up to so few)
      if (v == v0 && ahead) {
        behind_prefix(a, q, skip[v - groups_n]);
        if (few(a, q)) q.blocks = 0;
      } else {
        q = at_walk(v, &bad);
      }
      local += cost(q);
    }
    int64_t all;
    const int64_t before = block_prefix<kThreads>(local, sm.scan, &all);
    if (all > INT32_MAX) {
      bad = 1;
      all = 0;                                             // nothing is computed
    }
    total = (int)all;
    int run = (int)before;
    runs = min((int)gridDim.x, max(total / kMinRun, 1));
    share = total / runs;
    extra = total - share * runs;
    const int begin = run_start(blockIdx.x);
    for (int v = v0; v < v1; ++v) {
      if (per > 1) q = at_walk(v, nullptr);
      prefix[v] = run;
      const int next = run + cost(q);
      if (run <= begin && begin < next) {
        sm.first_v = v;
        sm.first = q;
      }
      run = next;
    }
    if (threadIdx.x == 0) prefix[walk_n] = total;
    if (bad && blockIdx.x == 0) set_error(err, MOE_DEVERR_CACHE);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const bool idle = (int)blockIdx.x >= runs;
  const int begin = idle ? 0 : run_start(blockIdx.x), end = idle ? 0 : run_start(blockIdx.x + 1);
  const int tb1 = tb / 2;                                  // tokens of a row tile

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
    // a unit's cost is kPieceCost, then a tile each
    auto owner = [&](int at) {                             // the run that holds position `at`
      const int longer = (share + 1) * extra;              // positions in the longer runs
      return at < longer ? at / (share + 1) : extra + (at - longer) / share;
    };
    int pos = begin, made = 0, loads = 0;
    bool last = false;
    Req q = sm.first;                                      // (not read where the run is empty)
    int v = sm.first_v, have = v;
    while (!last) {
      Piece p;
      last = pos >= end;
      p.flags = kLast;
      if (!last) {
        while (prefix[v + 1] <= pos) ++v;
        if (have != v) q = at_walk(v, nullptr);
        have = v;
        const int per = q.tiles + kPieceCost, u = (pos - prefix[v]) / per, off = pos - prefix[v] - u * per;
        const int len = min(per - off, end - pos), t0 = max(off - kPieceCost, 0);
        int t1 = off + len - kPieceCost;
        const int unit_end = pos - off + per;
        pos += len;
        if (t1 <= t0) continue;                            // the fixed cost alone
        p.row = q.row;
        p.skip = q.skip;
        p.h = u / q.blocks;
        p.tok0 = (u - p.h * q.blocks) * tb;
        p.ntok[0] = min(tb1, q.n - p.tok0);
        p.ntok[1] = min(tb1, max(q.n - p.tok0 - tb1, 0));
        p.row0 = q.q0 + p.tok0;
        p.ctx = q.ctx;
        p.kv = q.kv;
        p.t0 = t0;
        p.flags = (t0 == 0 ? kStarts : 0) | (t1 == q.tiles ? kEnds : 0);
        p.parts = p.flags == kStarts ? owner(unit_end - 1) - (int)blockIdx.x + 1 : 0;
        p.flags |= q.flags;
        if (!a.tree_mask) t1 = min(t1, (q.ctx + p.tok0 + p.ntok[0] + p.ntok[1] + kTile - 1) / kTile);
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
        const int tiles = p.ntok[1] ? 2 : 1;
        mbar_expect_tx(bar(sm.q_full), (uint32_t)(tiles * X::NH * 128 * a.G * tb1));
        for (int w = 0; w < tiles; ++w)
#pragma unroll
          for (int hh = 0; hh < X::NH; ++hh)
            tma_load_3d(q_smem + w * X::SLOT + hh * kHalfBytes, &maps.q, 64 * hh, p.h * a.G, p.row0 + w * tb1,
                        bar(sm.q_full));
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
    // ---------------- K and V into shared memory: K0, V0, K1, V1, ... ----------------
    // the boxes of a tile (page by page, half by half) are shared between the two loaders
    const int who = warp == 8 ? 0 : 1;
    const int page = 1 << a.page_shift, rows = min(page, kTile);
    const int per_tile = kTile / rows;                     // boxes of a half: lane l < per_tile has box l
    int slot = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (Piece p; ok && next(p);) {
      if (p.n == 0) continue;
      const int32_t* table = a.block_table + (int64_t)p.row * a.max_pages + p.skip;
      // page of this lane's box of tile j (of the piece); -1: nothing to load
      auto page_of = [&](int j) {
        const int tok = (p.t0 + j) * kTile + lane * rows;
        if (j >= p.n || lane >= per_tile || tok >= p.kv) return -1;
        const int id = table[tok >> a.page_shift];
        if (id >= 0 && id < a.n_pages) return id;
        set_error(err, MOE_DEVERR_CACHE);
        return a.n_pages;                                  // past the last page: TMA fills zeros
      };
      int id[3] = {page_of(0), page_of(1), -1};            // tiles j .. j + 2
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
        // (a lane a box: the first tiles of a run are there 3000 cycles sooner than with one lane for all)
        if (lane < boxes && (step == 1 || (lane & 1) == first))
          tma_load_4d(dst + (uint32_t)(lane * rows * 128), map, 64 * hh, off, p.h, pid, b);
        __syncwarp();
        ++it;
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
      };
      for (int j = 0; j < p.n && ok; ++j) {
        id[2] = page_of(j + 2);
        load(&maps.k, j, id[0]);
        if (ok) load(&maps.v, j, id[0]);
        id[0] = id[1];
        id[1] = id[2];
      }
    }
    if (*abort_flag && lane == 0) {
      // copies in flight must land before the CTA leaves
      const uint64_t t0 = globaltimer();
      for (int s = 0; s < NS; ++s) {
        const int uses = (it - s + NS - 1) / NS;           // times that slot s was filled
        if (it > s)
          while (!mbar_try(bar(sm.full[s]), (uint32_t)(uses - 1) & 1u) && globaltimer() - t0 < kWaitLimitNs) {
          }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------- MMA issuer ----------------
    // the whole warp walks and waits; one elected thread issues
    const uint32_t id_s = idesc_f16kind(kAttnRows, kTile, false);
    const uint32_t id_o = idesc_f16kind(kAttnRows, DP, false) | (1u << 16);      // B is MN-major
    int slot = 0, pieces = 0;
    uint32_t phase = 0;
    int tiles[2] = {0, 0};                                 // of all pieces so far, a row tile each
    bool ok = true, issued = false, warm[2] = {false, false};
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
    // S of row tile w from the K tile in slot k; behind it, what it frees
    auto scores = [&](int w, int k, bool free_k, bool free_q) {
      if (!warm[w]) {                                      // (below: the group has written its columns for the last time)
        warm[w] = true;
        if (!wait(sm.warm[w], 0)) return;
        tc_fence_after();
      }
      if (elect_one()) {
        const uint64_t da = smem_desc_sw128(q_smem + (uint32_t)(w * X::SLOT)),
                       db = smem_desc_sw128(ring + (uint32_t)(k * X::SLOT));
        const uint32_t d = tmem + X::s_col(w);
#pragma unroll
        for (int hh = 0; hh < X::NH; ++hh)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t step = hh * (kHalfBytes >> 4) + 2 * i;
            tc_mma<1>(d, da + step, db + step, id_s, (hh | i) != 0);
          }
        tc_commit<1>(bar(sm.s_full[w]));
        if (free_k) tc_commit<1>(bar(sm.empty[k]));
        if (free_q) tc_commit<1>(bar(sm.q_empty));
      }
      __syncwarp();
    };
    for (Piece p; ok && next(p);) {
      if (p.n == 0) continue;
      const bool two = p.ntok[1] > 0;
      if (!wait(sm.q_full, pieces & 1) || !wait(sm.full[slot], phase)) break;
      tc_fence_after();
      issued = true;
      scores(0, slot, !two, !two && p.n == 1);
      if (two) scores(1, slot, true, p.n == 1);
      advance();
      for (int j = 0; j < p.n && ok; ++j) {
        const bool more = j + 1 < p.n, last_s = j + 2 == p.n;
        const int vs = slot;
        const uint32_t v_phase = phase;
        advance();
        const int ks = slot;
        const uint32_t k_phase = phase;
        if (more) advance();
        if (!wait(sm.full[vs], v_phase)) break;
        for (int w = 0; w < (two ? 2 : 1); ++w) {
          // P is there (and O, zeros at a piece's start, is this piece's)
          if (!wait(sm.p_full[w], (uint32_t)(tiles[w] + j) & 1u)) break;
          tc_fence_after();
          const bool last_w = w == 1 || !two;
          if (elect_one()) {
            const uint64_t db = v_desc(ring + (uint32_t)(vs * X::SLOT));
            const uint32_t d = tmem + X::o_col(w), pa = tmem + X::s_col(w);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) mma_ts(d, pa + 8u * k, db + 128u * k, id_o, 1u);
            if (last_w) tc_commit<1>(bar(sm.empty[vs]));
            if (!more) tc_commit<1>(bar(sm.o_full[w]));
          }
          __syncwarp();
          if (more) {
            if (w == 0 && !wait(sm.full[ks], k_phase)) break;
            tc_fence_after();
            scores(w, ks, last_w, last_w && last_s);
          }
        }
      }
      tiles[0] += p.n;
      if (two) tiles[1] += p.n;
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
    // ---------------- softmax: group w (four warps) has row tile w, a thread a row ----------------
    const int w = warp >> 2, qd = warp & 3, row = 32 * qd + lane;
    const uint32_t lane_addr = (uint32_t)(32 * qd) << 16;
    const uint32_t s_addr = tmem + lane_addr + X::s_col(w), o_addr = tmem + lane_addr + X::o_col(w);
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
    int tiles = 0, items = 0, pieces = 0, meets_both = 0, meets_alone = 0;
    bool ok = true, warm = false;
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
      const bool two = p.ntok[1] > 0;
      const int ntok = p.ntok[w], valid = ntok * a.G, row0 = p.row0 + w * tb1;
      const int first_item = items;
      items += 2 * p.n;
      if (ntok == 0) continue;
      const bool live_warp = 32 * qd < valid;
      const int node = p.tok0 + w * tb1 + row_tok;
      float mc = -INFINITY, l = 0.f;
      if (p.n > 0) {
        // the products add to O
        const float zero[32] = {};
#pragma unroll 1
        for (int c0 = 0; c0 < DP; c0 += 32) st32(o_addr + c0, zero);
        st_wait();
      }
      // V rows of tile j past the last key, and nodes' rows that are not finite, become zeros, by halves of the head:
      // one a group, or both the first one's.  Where the nodes of the second kind are noted (the words of a
      // tile are read before the next special one's meeting, those after it have another parity)
      auto clean = [&](int j) -> const uint32_t(*)[4] {
        const int key0 = (p.t0 + j) * kTile, item = first_item + 2 * j + 1;
        if (!wait(sm.full[item % NS], (uint32_t)(item / NS) & 1u)) return nullptr;
        const int met = two ? meets_both++ : meets_alone++;
        uint32_t(*odd)[4] = sm.odd[two ? 0 : 1][met & 1];
        uint8_t* tile = ring_ptr + (item % NS) * X::SLOT;
        const int key = key0 + row;
        const bool zero = key >= p.kv;
        for (int hh = 0; hh < 2; ++hh) {
          if (two && hh != w) continue;        // (a half of the head each)
          bool strange = false;
          if (hh < X::NH) {
            uint4* v0 = reinterpret_cast<uint4*>(tile + hh * kHalfBytes + row * 128);
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
          }
          const uint32_t mine = __ballot_sync(0xffffffffu, strange);
          if (lane == 0) odd[hh][qd] = mine;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        uint64_t& meet = two ? sm.both : sm.first_alone;
        arrive(meet);
        if (!wait(meet, met & 1)) return nullptr;
        uint32_t any = 0;
        for (int i = 0; i < 8; ++i) any |= odd[i >> 2][i & 3];
        return any ? odd : nullptr;
      };
      // Before its first tile a group goes over whatever its columns hold: that fetches the instructions, some 4000
      // cycles' wait, while the first keys are on their way
      const bool warms = !warm && p.n > 0;
      for (int j = warms ? -1 : 0; j < p.n && ok; ++j) {
        if (j >= 0 && !wait(sm.s_full[w], (uint32_t)(tiles + j) & 1u)) break;
        const int key0 = (p.t0 + j) * kTile;
        const bool special = j >= 0 && key0 + kTile > p.ctx;
        const uint32_t(*odd)[4] = nullptr;
        if (__builtin_expect(special, 0)) odd = clean(j);
        if (!ok) break;
        if (live_warp) {
          tc_fence_after();
          uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
          if (__builtin_expect(special, 0)) {
            const int32_t* mask =
                a.tree_mask ? a.tree_mask + (int64_t)(row0 + min(row_tok, ntok - 1)) * a.mask_words : nullptr;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              const int k0 = key0 + 32 * cc, j0 = k0 - p.ctx;    // first key of the word, as a node
              auto low = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
              if (!mask) {
                bits[cc] = low(node + 1 - j0);
              } else {
                auto word = [&](int i) { return i < 0 ? 0xffffffffu : i < a.mask_words ? (uint32_t)mask[i] : 0u; };
                const int wi = j0 >> 5;
                bits[cc] = j0 + 32 <= 0 ? 0xffffffffu : __funnelshift_r(word(wi), word(wi + 1), (uint32_t)(j0 & 31));
              }
              bits[cc] &= low(p.kv - k0);
            }
          }
          auto masked = [&](float (&v)[64], auto O, uint32_t b) {
            constexpr int o = decltype(O)::value;
            if (__builtin_expect(special, 0)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(b >> i & 1u)) v[o + i] = -INFINITY;
            }
          };
          auto largest = [&](float (&v)[64]) {
            float t4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int i = 4; i < 60; i += 2) t4[(i >> 1) & 3] = max3(t4[(i >> 1) & 3], v[i], v[i + 1]);
            return max3(max3(t4[0], t4[1], v[60]), max3(t4[2], t4[3], v[61]), fmaxf(v[62], v[63]));
          };
          constexpr std::integral_constant<int, 0> lo;
          constexpr std::integral_constant<int, 32> hi;
          // the maximum: the second half of the keys, then the first, which stays
          float v[64];
          ld32_async<0>(s_addr + 64, v);
          ld32_async<32>(s_addr + 96, v);
          ld32_wait<0>(v);
          ld32_wait<32>(v);
          masked(v, lo, bits[2]);
          masked(v, hi, bits[3]);
          float top = largest(v);
          ld32_async<0>(s_addr, v);
          ld32_async<32>(s_addr + 32, v);
          ld32_wait<0>(v);
          ld32_wait<32>(v);
          masked(v, lo, bits[0]);
          masked(v, hi, bits[1]);
          top = fmaxf(top, largest(v)) * c;
          const bool raise = top > mc + kRaise || (mc == -INFINITY && top > mc);
          if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
            const float f = raise ? (mc == -INFINITY ? 0.f : ex2(mc - top)) : 1.f;
            if (raise) mc = top;
            l *= f;
            // O, after the tile before: that product was issued before this tile's S
            if (j > 0) {
#pragma unroll 1
              for (int c0 = 0; c0 < DP; c0 += 32) {
                float o[32];
                ld32_async<0>(o_addr + c0, o);
                ld32_wait<0>(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= f;
                st32(o_addr + c0, o);
              }
              st_wait();
            }
          }
          const float base = mc == -INFINITY ? 0.f : mc;
          const uint64_t c2 = pair(c, c), base2 = pair(-base, -base);
          uint64_t sum[2] = {0, 0};
          // 32 probabilities, summed before they are rounded to BF16 (above), over scores that were read
          auto exps = [&](auto O, int cc) {
            constexpr int o = decltype(O)::value;
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x, y;
              unpair(fma2(pair(v[o + 2 * i], v[o + 2 * i + 1]), c2, base2), x, y);
              x = ex2(x);
              y = ex2(y);
              sum[i & 1] = add2(sum[i & 1], pair(x, y));
              pk[i] = pack_bf16(x, y);
            }
            st16(s_addr + 16u * cc, pk);
          };
          exps(lo, 0);
          ld32_async<0>(s_addr + 64, v);
          exps(hi, 1);
          ld32_async<32>(s_addr + 96, v);
          ld32_wait<0>(v);
          masked(v, lo, bits[2]);
          exps(lo, 2);
          ld32_wait<32>(v);
          masked(v, hi, bits[3]);
          exps(hi, 3);
          float s0, s1;
          unpair(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          st_wait();
          if (__builtin_expect(odd != nullptr, 0)) {
            // p v of the nodes whose V is not finite
            const int32_t* table = a.block_table + (int64_t)p.row * a.max_pages + p.skip;
            for (int hh = 0; hh < X::NH; ++hh)
              add_odd(a, table, p.h, key0, make_uint4(odd[hh][0], odd[hh][1], odd[hh][2], odd[hh][3]), 64 * hh, s_addr,
                      o_addr);
            __syncwarp();
          }
        }
        tc_fence_before();
        if (j < 0) {
          mc = -INFINITY;
          l = 0.f;
          warm = true;
          arrive(sm.warm[w]);
          continue;
        }
        arrive(sm.p_full[w]);
      }
      tiles += p.n;
      if (!ok) break;

      // ---- the piece's end: write the rows or their partials ----
      if (p.n > 0) {
        if (!wait(sm.o_full[w], pieces & 1)) break;
        ++pieces;
        tc_fence_after();
      }
      const bool uncut = (p.flags & (kStarts | kEnds)) == (kStarts | kEnds);
      const bool whole = uncut && !(p.flags & (kPrefix | kJoined));
      const int slot = 2 * (int)blockIdx.x + (p.flags & kStarts ? 1 : 0);
      const int64_t side = (p.flags & kPrefix ? 0 : a.Hkv) + p.h;
      // (partials) this row, by the rows' own numbers or in the run's slot
      const int64_t at = uncut ? side * ((int64_t)a.T * a.G) + (int64_t)row0 * a.G + row
                               : (int64_t)slot * (2 * kAttnRows) + w * kAttnRows + row;
      if (live_warp) {
        // a row without a visible key has sum 0 and O = 0 (never written if the piece has no tile)
        const float g = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int c0 = 0; c0 < DP; c0 += 32) {  // (run once a piece: what it costs is fetching its instructions)
          float o[32];
          if (p.n > 0) {
            ld32_async<0>(o_addr + c0, o);
            ld32_wait<0>(o);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i] * g;
          // a row's piece of 64 bytes at a time: four lanes exchange 16-byte quarters, so that a store of the warp
          // touches 8 lines and not 32
          uint4 x[4];
          if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                                pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
            transpose4(x, lane);
            bf16* out = reinterpret_cast<bf16*>(a.out) + (int64_t)row0 * a.out_ld + (int64_t)p.h * a.G * a.D + c0 +
                        8 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r2 = (row & ~3) + i, t2 = r2 / a.G;
              if (r2 < valid && c0 + 8 * (lane & 3) < a.D)
                *reinterpret_cast<uint4*>(out + t2 * a.out_ld + (int64_t)(r2 - t2 * a.G) * a.D) = x[i];
            }
          } else {
            float* out = (uncut ? a.rows_part : a.pair_part) + (at - (row & 3)) * DP + c0 + 4 * (lane & 3);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[i] = make_uint4(__float_as_uint(o[16 * half + 4 * i]), __float_as_uint(o[16 * half + 4 * i + 1]),
                                  __float_as_uint(o[16 * half + 4 * i + 2]), __float_as_uint(o[16 * half + 4 * i + 3]));
              transpose4(x, lane);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if ((row & ~3) + i < valid) *reinterpret_cast<uint4*>(out + i * DP + 16 * half) = x[i];
            }
          }
        }
        if (row < valid) {
          if (!whole) (uncut ? a.rows_ml : a.pair_ml)[at] = make_float2(mc, l);
          else if (a.lse)
            a.lse[(int64_t)(row0 + row_tok) * a.H + p.h * a.G + row_head] =
                l == 0.f ? -INFINITY : (mc + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (p.flags & kStarts && row < ntok)
        a.parts_of[side * a.T + row0 + row] = make_int4(whole ? 0 : uncut ? 1 : p.parts, uncut ? 0 : slot,
                                                        w * kAttnRows + row * a.G, p.flags & kJoined);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// The rows that still have partials: a row's lanes (four columns each) add those of its
// group's prefix, in order, then those of its own tokens.  Where they are stands in parts_of;
// their maxima and sums come a lane each, so that a row waits for one round of them.
// Bound: latency of the record, the pairs and the columns, then HBM and L2; 128 requests (30
// MB of partials) 9.0 us, 17 requests 5.7 us.  Done in the kernel for few rows,
// prefix partials cost it more than this launch.
// kAhead: a row's partials in flight, 16 where all rows are resident at once with as many registers, else 8 (16 / 8, us
// a call: two samples behind 2000 tokens 15.1 / 16.1, 17 requests 20.9 / 21.3, 128 requests 88 / 84).
constexpr int kJoinThreads = 128;
constexpr int kJoinBlocks = 4;                 // an SM, with 16 in flight
template <int DP, int kAhead>
__global__ void __launch_bounds__(kJoinThreads, kAhead == 16 ? kJoinBlocks : 2 * kJoinBlocks)
    prefix_join_kernel(const AttnArgs a) {
  constexpr int L = DP / 4;                    // lanes a row
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int rows_all = a.T * a.G, id = (blockIdx.x * kJoinThreads + threadIdx.x) / L;
  const int h = id / rows_all, rg = id - h * rows_all, tok = rg / a.G, head = rg - tok * a.G;
  PartsOf own = {0, 0, 0, 0}, pre = {0, 0, 0, 0};
  if (h < a.Hkv) {
    const int live = a.R > 0 ? a.q_start[a.R] : 0;
    own = parts_of(a, 1, h, tok);
    pre = parts_of(a, 0, h, tok);
    if (tok >= live) own.parts = 0;
    if (!own.parts || !(own.flags & kJoined)) pre.parts = 0;
  }
  const int n = pre.parts + own.parts, most = __reduce_max_sync(0xffffffffu, n);
  // partial k of the row
  auto locate = [&](int k, const float2*& ml, const float4*& v) {
    const bool first = k < pre.parts;
    partial<DP>(a, first ? pre : own, first ? 0 : 1, h, rg, head, first ? k : k - pre.parts, ml, v);
  };
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < most; k0 += L) {
    float2 mine = make_float2(0.f, 0.f);
    const float2* ml;
    const float4* at;
    float4 v[kAhead];
    auto fetch = [&](int j0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (k0 + j0 + j < n) {
          locate(k0 + j0 + j, ml, at);
          v[j] = at[sub];
        }
    };
    fetch(0);
    if (k0 + sub < n) {
      locate(k0 + sub, ml, at);
      mine = *ml;
    }
    // the factors of these partials, and of what was added before
    const bool there = mine.y != 0.f;          // (no visible key in that part)
    float t = there ? mine.x : -INFINITY;
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off, L));
    t = fmaxf(t, top);
    const float g = sum == 0.f ? 0.f : ex2(top - t), f = there ? ex2(mine.x - t) : 0.f;
    top = t;
    float more = there ? mine.y * f : 0.f;
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) more += __shfl_xor_sync(0xffffffffu, more, off, L);
    sum = fmaf(sum, g, more);
    acc = make_float4(acc.x * g, acc.y * g, acc.z * g, acc.w * g);
    for (int j0 = 0; j0 < L && k0 + j0 < most; j0 += kAhead) {
      if (j0) fetch(j0);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const float fj = __shfl_sync(0xffffffffu, f, j0 + j, L);
        if (fj == 0.f) continue;
        acc.x = fmaf(v[j].x, fj, acc.x);
        acc.y = fmaf(v[j].y, fj, acc.y);
        acc.z = fmaf(v[j].z, fj, acc.z);
        acc.w = fmaf(v[j].w, fj, acc.w);
      }
    }
  }
  if (n == 0) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (4 * sub < a.D)
    *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(a.out) + (int64_t)tok * a.out_ld + ((int64_t)h * a.G + head) * a.D +
                              4 * sub) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse && sub == 0)
    a.lse[(int64_t)tok * a.H + h * a.G + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int DP>
cudaError_t launch_dp(const AttnArgs& a, cudaStream_t s) {
  using X = Geo<DP>;
  const int tb = 2 * (kAttnRows / a.G), page = 1 << a.page_shift;
  const size_t smem = 1024 + 2 * X::SLOT + X::RING + sizeof(Small) + ((size_t)a.n_groups + 2 * (size_t)a.R + 1) * 4;
  static_assert(1024 + 2 * X::SLOT + X::RING + sizeof(Small) + (3 * kPrefixMaxRequests + 1) * 4 <= kMaxSmem, "shared memory");
  static PerDeviceOnce once;
  int sms = 0;
  cudaError_t e = once.run(
      [](int& v) {
        v = std::min(num_sms(), kAttnMaxCtas);
        return cudaFuncSetAttribute(attention_prefix_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      },
      &sms);
  if (e != cudaSuccess) return e;
  if (!a.few_alone) {
    Maps maps;
    {
      const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.H, (cuuint64_t)a.T};
      const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)(a.T > 1 ? a.q_ld : (int64_t)a.H * a.D) * 2};
      const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)(tb / 2)};
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
    e = launch_k(attention_prefix_kernel<DP>, dim3((unsigned)sms), dim3(kThreads), smem, s, maps, a, tb);
    if (e != cudaSuccess) return e;
  }
  if (a.few_tokens) e = launch_attention_few(a, s);
  if (e != cudaSuccess) return e;
  const int64_t lanes = (int64_t)a.T * a.H * (DP / 4);
  const bool one_wave = lanes <= (int64_t)sms * kJoinBlocks * kJoinThreads;
  const auto join = one_wave ? prefix_join_kernel<DP, 16> : prefix_join_kernel<DP, 8>;
  return launch_k(join, dim3((unsigned)ceil_div(lanes, kJoinThreads)), dim3(kJoinThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_prefix_attention_bf16(const AttnArgs& args, cudaStream_t s) {
  if (args.T <= 0) return cudaSuccess;
  AttnArgs a = args;
  few_shape(&a);
  return a.D <= 64 ? launch_dp<64>(a, s) : launch_dp<128>(a, s);
}

}  // namespace moe
