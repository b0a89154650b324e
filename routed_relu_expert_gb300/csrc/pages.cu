// Pages of the cache that requests share: a request's cache continued by others
// (fork), kept tokens moved to the front (compact), pages given back (release).
// No arithmetic; integers and copied bytes.
#include "attn.h"
#include "tc_common.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int held(int64_t tokens, int shift) { return (int)((tokens + (1ll << shift) - 1) >> shift); }

// Blocks of a cooperative launch that wait for one another (meet.h).  The counters return to
// zero by themselves: the last block to leave resets them.  A wait ends after
// tc::kWaitLimitNs, with MOE_DEVERR_TIMEOUT, for all blocks of the meeting.
struct GridMeet {
  AttnHeader* hdr;
  int blocks, arrived = 0, waited = 0;         // meetings that this block came to, that it waited for
  __device__ GridMeet(AttnHeader* h, int n) : hdr(h), blocks(n) {}
  // at the next meeting: what this block has read until here (and, WRITTEN, written) is done for who waits for it.
  // Reads need no fence: they have returned their values.
  template <bool WRITTEN>
  __device__ void arrive() {
    const int number = arrived++;
    __syncthreads();
    if (blocks > 1 && threadIdx.x == 0) {
      if (WRITTEN) __threadfence();
      atomicAdd(&hdr->met[meet_word(number)], 1);
    }
  }
  // until every block has come to the next meeting that this one has not waited for
  __device__ bool wait() {
    const int number = waited++;
    if (blocks == 1) return true;
    __shared__ int good[2];                    // (in turn: a word is written again two waits later)
    if (threadIdx.x == 0) {
      const uint64_t t0 = globaltimer();
      int32_t* word = &hdr->met[meet_word(number)];
      int seen, tries = 0, state;
      while (true) {
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(word) : "memory");
        state = meet_state(seen, number, blocks);
        if (state != kMeetWait) break;
        // (a swap that fails: a block has come meanwhile, or another has given up)
        if ((++tries & 255) == 0 && globaltimer() - t0 > tc::kWaitLimitNs && atomicCAS(word, seen, seen | kMeetGaveUp) == seen)
          set_error(&hdr->err, MOE_DEVERR_TIMEOUT);
      }
      good[number & 1] = state == kMeetMet;
    }
    __syncthreads();
    return good[number & 1];
  }
  __device__ bool operator()() {
    arrive<true>();
    return wait();
  }
  __device__ void leave() {
    __syncthreads();
    if (blocks > 1 && threadIdx.x == 0 && atomicAdd(&hdr->left, 1) == blocks - 1) {
      for (int i = 0; i < kMeetWords; ++i) hdr->met[i] = 0;
      hdr->left = 0;
    }
  }
};

// sum of one value a thread over the block, in every thread
__device__ __forceinline__ int block_sum(int v, int* tmp) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) all += tmp[w];
  return all;
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
// Every block adds up the pages that the forks before its own take, shares its source's
// whole pages and copies a part of the last one's tokens: one launch, no order among blocks.
// Bound: L2 and HBM for many forks, the chain of dependent loads (rows, table, page, tokens)
// for few.  512 forks of 16 prompts of up to 8000 tokens (120 MB of copied tokens): 24.4 us,
// 4.9 TB/s, as with 8 and 32 pieces a thread (64: 26 to 30); one fork 4.0 us.
constexpr int kForkAhead = 4;                  // 16-byte pieces that a thread has in flight
// blockIdx.x: the fork; blockIdx.y: a part of its page's tokens
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkArgs a) {
  pdl_wait();
  __shared__ int tmp[kThreads / 32];
  const int i = blockIdx.x, tid = threadIdx.x;
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  const int page_mask = (1 << a.page_shift) - 1;
  auto valid = [&](int j) {
    const int s = a.src[j], d = a.dst[j], n = a.lengths[j];
    return s >= 0 && s < a.R && d >= 0 && d < a.R && n >= 0 && n <= cap && !(a.same && s == d);
  };
  // new pages of the forks before this one and of all (two counts of at most 4096 in a word); forks that meet
  // this one's rows
  const bool have = i < a.n;                   // (no fork at all: one block, for free_head_out)
  const int s = have ? a.src[i] : 0, d = have ? a.dst[i] : 0;
  int counts = 0, clash = 0;
  for (int j = tid; j < a.n; j += kThreads) {
    const bool good = valid(j);
    const int need = good && (a.lengths[j] & page_mask);
    counts += need << 16 | (j < i ? need : 0);
    if (good && ((j < i && a.dst[j] == d) || (a.same && a.dst[j] == s))) clash = 1;
  }
  const int head = max(*a.free_head, 0);
  int bad = *a.free_head < 0 ? MOE_DEVERR_CACHE : 0;
  clash = __syncthreads_or(clash);
  counts = block_sum(counts, tmp);
  const int before = counts & 0xffff, all = counts >> 16;
  const bool ok = have && valid(i) && !clash;
  if (have && !ok) bad |= MOE_DEVERR_CACHE;
  if (ok) {
    const int len = a.lengths[i], full = len >> a.page_shift, rest = len & page_mask;
    const int32_t* from = a.src_table + (int64_t)s * a.max_pages;
    int32_t* to = a.dst_table + (int64_t)d * a.max_pages;
    if (blockIdx.y == 0)
      for (int c = tid; c < full; c += kThreads) {
        int p = from[c];
        if (p < 0 || p >= a.n_pages) {
          bad |= MOE_DEVERR_CACHE;
          p = -1;
        } else {
          atomicAdd(&a.shares[p], 1);
        }
        to[c] = p;
      }
    if (rest) {
      const int64_t at = (int64_t)head + before;
      int fresh = -1;
      if (at >= a.n_free) {
        bad |= MOE_DEVERR_PAGES;
      } else {
        fresh = a.free_pages[at];
        if (fresh < 0 || fresh >= a.n_pages) {
          bad |= MOE_DEVERR_CACHE;
          fresh = -1;
        }
      }
      if (blockIdx.y == 0 && tid == 0) to[full] = fresh;
      const int old = from[full];
      if (old < 0 || old >= a.n_pages) {
        bad |= MOE_DEVERR_CACHE;
      } else if (fresh >= 0) {
        // 16-byte pieces: [K or V][token][head][piece]
        const int per_head = a.row_bytes >> 4, per_token = per_head * a.Hkv, per_cache = per_token * rest;
        const int step = kThreads * (int)gridDim.y;
        const int64_t move = (int64_t)(fresh - old) * a.page_stride;
        for (int x0 = (int)blockIdx.y * kThreads + tid; x0 < 2 * per_cache; x0 += kForkAhead * step) {
          uint4 d[kForkAhead];
          uint8_t* at[kForkAhead];
#pragma unroll
          for (int i = 0; i < kForkAhead; ++i) {
            const int x = x0 + i * step;
            if (x >= 2 * per_cache) break;
            const int v = x >= per_cache, y = x - v * per_cache, t = y / per_token, z = y - t * per_token;
            const int h = z / per_head, c = z - h * per_head;
            at[i] = (v ? a.v : a.k) + old * a.page_stride + t * a.token_stride + h * a.head_stride + 16 * c;
            d[i] = *reinterpret_cast<const uint4*>(at[i]);
          }
#pragma unroll
          for (int i = 0; i < kForkAhead; ++i)
            if (x0 + i * step < 2 * per_cache) *reinterpret_cast<uint4*>(at[i] + move) = d[i];
        }
      }
    }
  }
  if (bad) set_error(&a.hdr->err, bad);
  // block_sum's barrier puts every thread's read of *free_head before this
  if (tid == 0) {
    const int blocks = (int)(gridDim.x * gridDim.y);
    __threadfence();
    if (blocks == 1 || atomicAdd(&a.hdr->plan_ticket, 1) == blocks - 1) {
      a.hdr->plan_ticket = 0;
      *a.free_head_out = (int)min((int64_t)head + all, (int64_t)max(a.n_free, head));
    }
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
// a move of one token: offsets (bytes) of its first head in a cache, from -1 where it stays
struct Move {
  int64_t from, to;
};

// kept number i of request r (its list is keep[begin ..)): places ascend and lie at or before their sources
__device__ __forceinline__ Move move_of(const CompactArgs& a, int r, int first, int begin, int i, int& bad) {
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  const int page_mask = (1 << a.page_shift) - 1;
  const int node = a.keep[i], place = i - begin;
  if (node < place || (i > begin && a.keep[i - 1] >= node) || (int64_t)first + node >= cap) {
    bad |= MOE_DEVERR_CACHE;
    return {-1, -1};
  }
  if (node == place) return {-1, -1};
  const int32_t* table = a.block_table + (int64_t)r * a.max_pages;
  const int p = table[(first + node) >> a.page_shift], d = table[(first + place) >> a.page_shift];
  if (p < 0 || p >= a.n_pages || d < 0 || d >= a.n_pages || (a.shares && a.shares[d] > 0)) {
    bad |= MOE_DEVERR_CACHE;
    return {-1, -1};
  }
  return {p * a.page_stride + ((first + node) & page_mask) * a.token_stride,
          d * a.page_stride + ((first + place) & page_mask) * a.token_stride};
}
// request r's list, empty where its bounds are no good; its length goes to len_out
__device__ __forceinline__ void list_of(const CompactArgs& a, int r, int& first, int& begin, int& end, int& bad) {
  begin = a.keep_start[r];
  end = a.keep_start[r + 1];
  first = a.first[r];
  if (begin < 0 || end < begin || end > a.N || first < 0) {
    bad |= MOE_DEVERR_CACHE;
    begin = end = 0;
  }
}

// Short lists: a block has a request and kThreads of a token's 16-byte pieces, a thread
// one of them for token after token.  Bound: the chain of dependent loads (list, table,
// tokens), a list's tokens eight at a time; 64 requests that keep 6 of 16 nodes: 2.5 us.
constexpr int kStage = 256;                    // moves worked out at a time
constexpr int kMoveAhead = 8;                  // tokens whose loads a thread has in flight
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  pdl_wait();
  __shared__ Move s_move[kStage];
  const int r = blockIdx.x, tid = threadIdx.x;
  const int per_head = a.row_bytes >> 4, per_token = per_head * a.Hkv;
  const int x = (int)blockIdx.y * kThreads + tid;
  const bool have = x < 2 * per_token;
  const int v = x >= per_token, z = x - v * per_token, h = z / per_head;
  uint8_t* cache = (v ? a.v : a.k) + h * a.head_stride + 16 * (z - h * per_head);
  int bad = 0, first, begin, end;
  list_of(a, r, first, begin, end, bad);
  if (a.len_out && blockIdx.y == 0 && tid == 0) a.len_out[r] = max(first, 0) + end - begin;
  for (int i0 = begin; i0 < end; i0 += kStage) {
    const int n = min(kStage, end - i0);
    __syncthreads();
    if (tid < n) s_move[tid] = move_of(a, r, first, begin, i0 + tid, bad);
    __syncthreads();
    if (!have) continue;
    // (a place is not written before its own and every earlier source is read)
    for (int j0 = 0; j0 < n; j0 += kMoveAhead) {
      uint4 d[kMoveAhead];
#pragma unroll
      for (int j = 0; j < kMoveAhead; ++j)
        if (j0 + j < n && s_move[j0 + j].from >= 0) d[j] = *reinterpret_cast<const uint4*>(cache + s_move[j0 + j].from);
#pragma unroll
      for (int j = 0; j < kMoveAhead; ++j)
        if (j0 + j < n && s_move[j0 + j].from >= 0) *reinterpret_cast<uint4*>(cache + s_move[j0 + j].to) = d[j];
    }
  }
  if (bad) set_error(&a.hdr->err, bad);
}

// Which of the two, replayed alone, us, short / long: lists of 8 on average (512 requests) 8.3 / 14.5, of 16 (64) 6.3 / 10.4,
// of 32 (16) 8.2 / 10.4, of 64 (16) 10.4 / 10.4; one list of 200 22.9 / 10.3, of 4000 407 / 14.4, of 66667 9800 / 103.
// kShortAll: so that one list among short ones cannot take longer than a few hundred us.
constexpr int kShortList = 32, kShortAll = 4096;
// Long lists, in two launches.  The first works the moves out, a thread a token (of all
// requests' lists as one).
__global__ void __launch_bounds__(kThreads) compact_moves_kernel(const CompactArgs a, Move* moves, int i0, int n) {
  pdl_wait();
  const int x = blockIdx.x * kThreads + threadIdx.x;
  int bad = 0, first, begin, end;
  if (i0 == 0)
    for (int r = x; r < a.R; r += gridDim.x * kThreads) {
      list_of(a, r, first, begin, end, bad);
      if (a.len_out) a.len_out[r] = max(first, 0) + end - begin;
    }
  if (x < n) {
    const int i = i0 + x;
    // the last request whose list begins at or before i
    int lo = 0, hi = a.R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.keep_start[mid] <= i) lo = mid; else hi = mid;
    }
    list_of(a, lo, first, begin, end, bad);
    moves[x] = begin <= i && i < end ? move_of(a, lo, first, begin, i, bad) : Move{-1, -1};
  }
  if (bad) set_error(&a.hdr->err, bad);
}

// The second moves the tokens in waves: all blocks read their part of a wave into shared
// memory, meet, and write it; the next two waves' reads are on their way meanwhile, and a
// block comes to the next wave's meeting before it waits for this one's.  Token i of the lists
// goes to a place at or before its source, so what a wave writes lies behind every later
// wave's sources and only its own wave and earlier ones read there.  A thread reads and
// writes its own 16-byte pieces.  Bound: HBM, reads and writes in turn.  66667 of 100001
// tokens of 4 KB (546 MB): 97 us, 5.6 TB/s or 84 % of a plain copy, and 99.5 us the call; 104
// replayed alone (so, with one wave ahead of the writes 126, with one of 104 KB a block 114; more and
// smaller waves, each of which costs half a microsecond beside its bytes: four of 48 KB 112, of 32 KB 125).
constexpr int kWaveThreads = 512;
constexpr int kWaves = 3;                      // in a block's shared memory
constexpr int kWaveAhead = 9;                  // pieces of a thread a wave (72 KB a block)
constexpr size_t kWaveSmem = (size_t)kWaves * kWaveThreads * kWaveAhead * 16;
__global__ void __launch_bounds__(kWaveThreads, 1) compact_wave_kernel(const CompactArgs a, const Move* moves, int n,
                                                                        int groups) {
  extern __shared__ uint4 held_pieces[];       // [wave modulo kWaves][piece][thread]
  GridMeet meet(a.hdr, (int)gridDim.x);
  // a block has one group of a token's pieces: `per` of them, of as many tokens as it has threads for
  const int per_head = a.row_bytes >> 4, per_token = per_head * a.Hkv, pieces = 2 * per_token;
  const int group = blockIdx.x % groups, block = blockIdx.x / groups, blocks = gridDim.x / groups;
  const int per = min(pieces, kWaveThreads), tokens = kWaveThreads / per;
  const int sub = threadIdx.x / per, x = group * per + threadIdx.x - sub * per;
  const bool have = sub < tokens && x < pieces;
  const int v = x >= per_token, z = x - v * per_token, h = z / per_head;
  uint8_t* cache = (v ? a.v : a.k) + h * a.head_stride + 16 * (z - h * per_head);
  const int step = tokens * kWaveAhead;
  const int64_t wave = (int64_t)blocks * step;
  const int waves = (int)((n + wave - 1) / wave);
  // of this thread's pieces of a wave: where they lie (FROM), or go; -1: nothing to move
  auto moves_of = [&](int w, bool from, int64_t (&at)[kWaveAhead]) {
#pragma unroll
    for (int j = 0; j < kWaveAhead; ++j) {
      const int64_t t = w * wave + (int64_t)block * step + sub + (int64_t)j * tokens;
      at[j] = !have || t >= n ? -1 : from ? moves[t].from : moves[t].to;
    }
  };
  auto piece = [&](int w, int j) { return held_pieces + (w % kWaves * kWaveAhead + j) * kWaveThreads + threadIdx.x; };
  int64_t from[kWaveAhead], to[kWaveAhead];
  auto read = [&](int w) {
#pragma unroll
    for (int j = 0; j < kWaveAhead; ++j)
      if (from[j] >= 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(piece(w, j))), "l"(cache + from[j])
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int w = 0; w < kWaves - 1; ++w) {
    moves_of(w, true, from);
    read(w);
  }
  moves_of(kWaves - 1, true, from);
  asm volatile("cp.async.wait_group %0;" ::"n"(kWaves - 2) : "memory");
  meet.arrive<false>();                        // at the meeting of wave 0: it is read
  for (int w = 0; w < waves; ++w) {
    read(w + kWaves - 1);
    moves_of(w + kWaves, true, from);
    moves_of(w, false, to);
    asm volatile("cp.async.wait_group %0;" ::"n"(kWaves - 2) : "memory");
    meet.arrive<false>();                      // of wave w + 1
    if (!meet.wait()) break;                   // for wave w
#pragma unroll
    for (int j = 0; j < kWaveAhead; ++j)
      if (to[j] >= 0) *reinterpret_cast<uint4*>(cache + to[j]) = *piece(w, j);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  meet.leave();
}

// ---------------------------------------------------------------------------
// release
// ---------------------------------------------------------------------------
constexpr int kRelThreads = 1024;
constexpr int kRelWarps = kRelThreads / 32;
// entries of the table for one block to do it alone: a plain launch costs the host 1.5 us less than one of blocks that
// meet, and all of 4000 entries given back the GPU the same 17 us (of 8000: 27 for 17)
constexpr int kRelAlone = 4 * kRelThreads;
constexpr int kRelEntries = kRelThreads;       // of a block, before another one helps (2048: 20.4 for 18.7 us, 4096: 25.6)

// exclusive prefix of one value a thread over the block; *total: their sum
__device__ __forceinline__ int block_scan(int v, int* tmp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = tmp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) y += z;
    }
    tmp[lane] = y;
  }
  __syncthreads();
  const int before = (warp ? tmp[warp - 1] : 0) + x - v;
  *total = tmp[31];
  __syncthreads();
  return before;
}

// All entries that are given back, in the table's order, are cut into equal parts, a
// block each, and a block's into its warps'; lanes take neighbours.  A page's holders go
// down by atomics on whole numbers, whose order does not matter; which of its entries is the last
// in the table, and so gives it back, is a maximum; places in the list come from prefix sums
// of warps, blocks and the grid.  Bound: the latency of the phases and of up to three meetings
// (2 us each).  1024 requests, most of their pages shared by 16: 18.6 us; 64 requests: 5.8 us;
// with one block for everything the 1024 took 142 us.
__global__ void __launch_bounds__(kRelThreads, 1) release_kernel(const ReleaseArgs a) {
  extern __shared__ int prefix[];              // [R + 1] entries before each request
  __shared__ int tmp[32];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)blockIdx.x;
  int bad = 0;
  auto span = [&](int r, int& lo) {
    int now = a.held_len[r], keep = a.keep_len[r];
    if (now < 0 || keep < 0) bad |= MOE_DEVERR_CACHE;
    lo = held(max(keep, 0), a.page_shift);
    return max(min(held(max(now, 0), a.page_shift), a.max_pages) - lo, 0);
  };
  const int old_head = *a.free_head, head = max(old_head, 0);
  if (old_head < 0) bad |= MOE_DEVERR_CACHE;
  int total;
  {
    const int per = (a.R + kRelThreads - 1) / kRelThreads, r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    int mine = 0, lo;
    for (int r = r0; r < r1; ++r) mine += span(r, lo);
    int at = block_scan(mine, tmp, &total);
    for (int r = r0; r < r1; ++r) {
      prefix[r] = at;
      at += span(r, lo);
    }
    if (tid == 0) prefix[a.R] = total;
  }
  // blocks that take part: the same number in each of them
  const int ctas = min((int)gridDim.x, max((int)(((int64_t)total + kRelEntries - 1) / kRelEntries), 1));
  if (rank >= ctas) return;
  GridMeet meet(a.hdr, ctas);
  __syncthreads();
  const int64_t e0 = (int64_t)total * rank / ctas, e1 = (int64_t)total * (rank + 1) / ctas;
  const int begin = (int)(e0 + (e1 - e0) * warp / kRelWarps), end = (int)(e0 + (e1 - e0) * (warp + 1) / kRelWarps);
  int row0 = 0;
  {
    int lo = 0, hi = a.R;                      // the last row with prefix[row] <= the lane's first entry
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= begin + lane) lo = mid; else hi = mid;
    }
    row0 = lo;
  }
  // f(place in the table or -1, page or -1) of each of them, all lanes together; the first ones, which are all where
  // the blocks are not short of SMs, are looked up once
  constexpr int kAhead = 4;
  int r = row0, have = -1, lo = 0;
  auto look = [&](int b, int (&at)[kAhead], int (&p)[kAhead]) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int e = b + 32 * j + lane;
      at[j] = p[j] = -1;
      if (e < end) {
        while (e >= prefix[r + 1]) ++r;
        if (have != r) span(r, lo);
        have = r;
        at[j] = r * a.max_pages + lo + (e - prefix[r]);
        p[j] = a.block_table[at[j]];
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (p[j] < 0 || p[j] >= a.n_pages) {
        if (p[j] != -1) bad |= MOE_DEVERR_CACHE;
        p[j] = -1;
      }
  };
  int at0[kAhead], p0[kAhead];
  look(begin, at0, p0);
  const int r_next = r, have_next = have, lo_next = lo;
  auto walk = [&](auto f) {
    f(at0, p0);
    r = r_next;
    have = have_next;
    lo = lo_next;
    for (int b = begin + 32 * kAhead; b < end; b += 32 * kAhead) {
      int at[kAhead], p[kAhead];
      look(b, at, p);
      f(at, p);
    }
  };
  if (a.shares) {
    walk([&](int (&)[kAhead], int (&p)[kAhead]) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (p[j] >= 0) a.last[p[j]] = -1;
    });
    if (!meet()) return meet.leave();          // (every block does: list and table stay as they are)
    walk([&](int (&at)[kAhead], int (&p)[kAhead]) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (p[j] >= 0) {
          atomicMax(&a.last[p[j]], at[j]);
          atomicSub(&a.shares[p[j]], 1);
        }
    });
    if (!meet()) return meet.leave();
  }
  // freed: no holder is left, and this is the last of the entries that gave it back
  auto freed = [&](int (&at)[kAhead], int (&p)[kAhead], bool (&is)[kAhead], int (&left)[kAhead]) {
    int of[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      left[j] = p[j] >= 0 && a.shares ? __ldcg(&a.shares[p[j]]) : -1;
      of[j] = p[j] >= 0 && a.shares ? __ldcg(&a.last[p[j]]) : at[j];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) is[j] = p[j] >= 0 && left[j] < 0 && of[j] == at[j];
  };
  int count = 0;
  walk([&](int (&at)[kAhead], int (&p)[kAhead]) {
    bool is[kAhead];
    int left[kAhead];
    freed(at, p, is, left);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) count += __popc(__ballot_sync(0xffffffffu, is[j]));
  });
  int own;
  int place = block_scan(lane == 0 ? count : 0, tmp, &own);      // entries freed before this warp's, in its lane 0
  place = __shfl_sync(0xffffffffu, place, 0);
  int all = own;
  if (ctas > 1) {
    if (tid == 0) a.counts[rank] = own;
    if (!meet()) return meet.leave();
    int before = 0, sum = 0;
    for (int c = tid; c < ctas; c += kRelThreads) {
      const int n = __ldcg(&a.counts[c]);
      sum += n;
      if (c < rank) before += n;
    }
    int ignored;
    block_scan(before, tmp, &ignored);
    place += ignored;
    block_scan(sum, tmp, &all);
  }
  if (all > head || head > a.n_free) bad |= MOE_DEVERR_CACHE;    // more than the list gave out
  place += head - all;
  walk([&](int (&at)[kAhead], int (&p)[kAhead]) {
    bool is[kAhead];
    int left[kAhead];
    freed(at, p, is, left);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t set = __ballot_sync(0xffffffffu, is[j]);
      const int to = place + __popc(set & lanemask_lt());
      place += __popc(set);
      if (is[j]) {
        if (to >= 0 && to < a.n_free) a.free_pages[to] = p[j];
        // (another entry of the page reads a count of -1 or 0 and that the last entry is not it: either way not freed)
        if (left[j] < -1) bad |= MOE_DEVERR_CACHE;               // given back more often than it was held
        if (a.shares) a.shares[p[j]] = 0;
      }
      if (at[j] >= 0) a.block_table[at[j]] = -1;
    }
  });
  if (rank == 0 && tid == 0) *a.free_head = max(head - all, 0);
  if (bad) set_error(&a.hdr->err, bad);
  meet.leave();
}

// blocks of a cooperative launch wait for one another
template <typename... KArgs, typename... Args>
cudaError_t launch_cooperative(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                               Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s) {
  const int64_t pieces = 2ll * (a.row_bytes >> 4) * a.Hkv << a.page_shift;
  const unsigned y = (unsigned)std::min<int64_t>(std::max<int64_t>(pieces / (kThreads * 16), 1), 64);
  return launch_k(fork_kernel, dim3((unsigned)std::max(a.n, 1), a.n ? y : 1), kThreads, 0, s, a);
}

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t s) {
  if (a.R <= 0) return cudaSuccess;
  const int64_t pieces = 2ll * (a.row_bytes >> 4) * a.Hkv;
  const int64_t groups = ceil_div(pieces, kWaveThreads);
  static PerDeviceOnce once;
  int sms = 0;
  const cudaError_t e = once.run(
      [](int& v) {
        v = tc::num_sms();
        return cudaFuncSetAttribute(compact_wave_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWaveSmem);
      },
      &sms);
  if (e != cudaSuccess) return e;
  // short lists; and tokens wider than the waves have blocks for (152 x 8 KB)
  if (a.N <= std::min<int64_t>((int64_t)kShortList * a.R, kShortAll) || groups > sms)
    return launch_k(compact_kernel, dim3((unsigned)a.R, (unsigned)ceil_div(pieces, kThreads)), kThreads, 0, s, a);
  Move* moves = reinterpret_cast<Move*>(a.scratch);
  const int most = (int)(a.scratch_bytes / sizeof(Move));
  for (int i0 = 0; i0 < a.N; i0 += most) {
    const int n = std::min(most, a.N - i0);
    cudaError_t e2 = launch_k(compact_moves_kernel, dim3((unsigned)ceil_div(n, kThreads)), kThreads, 0, s, a, moves, i0, n);
    // as many blocks as the list has work for, the same number in every group
    const int64_t step = kWaveThreads / std::min<int64_t>(pieces, kWaveThreads) * kWaveAhead;
    const int64_t blocks = std::min<int64_t>(sms / groups, ceil_div(n, step));
    if (e2 == cudaSuccess)
      e2 = launch_cooperative(compact_wave_kernel, (unsigned)(blocks * groups), kWaveThreads, kWaveSmem, s, a, moves, n,
                              (int)groups);
    if (e2 != cudaSuccess) return e2;
  }
  return cudaSuccess;
}

cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t s) {
  const size_t smem = ((size_t)a.R + 1) * 4;
  static PerDeviceOnce once;
  int sms = 0;
  const cudaError_t e = once.run(
      [](int& v) {
        v = std::min(tc::num_sms(), kAttnMaxCtas);
        return cudaFuncSetAttribute(release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (16384 + 1) * 4);
      },
      &sms);
  if (e != cudaSuccess) return e;
  const unsigned ctas = (unsigned)std::min<int64_t>(ceil_div((int64_t)a.R * a.max_pages, kRelEntries), sms);
  if ((int64_t)a.R * a.max_pages <= kRelAlone) return launch_k(release_kernel, dim3(1), dim3(kRelThreads), smem, s, a);
  return launch_cooperative(release_kernel, ctas, kRelThreads, smem, s, a);
}

}  // namespace moe
