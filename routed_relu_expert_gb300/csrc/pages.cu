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

// sum of one value a thread over the block, in every thread
__device__ __forceinline__ int block_sum(int v, int* tmp) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) all += tmp[w];
  __syncthreads();
  return all;
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
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
  // new pages of the forks before this one and of all; forks that meet this one's rows
  const bool have = i < a.n;                   // (no fork at all: one block, for free_head_out)
  const int s = have ? a.src[i] : 0, d = have ? a.dst[i] : 0;
  int before = 0, all = 0, clash = 0;
  for (int j = tid; j < a.n; j += kThreads) {
    const int need = valid(j) && (a.lengths[j] & page_mask);
    all += need;
    if (j < i) before += need;
    if (valid(j) && ((j < i && a.dst[j] == d) || (a.same && a.dst[j] == s))) clash = 1;
  }
  const int head = max(*a.free_head, 0);
  int bad = *a.free_head < 0 ? MOE_DEVERR_CACHE : 0;
  before = block_sum(before, tmp);
  all = block_sum(all, tmp);
  clash = block_sum(clash, tmp);
  const bool ok = have && valid(i) && clash == 0;
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
        for (int x = (int)blockIdx.y * kThreads + tid; x < 2 * per_cache; x += step) {
          const int v = x >= per_cache, y = x - v * per_cache, t = y / per_token, z = y - t * per_token;
          const int h = z / per_head, c = z - h * per_head;
          uint8_t* cache = v ? a.v : a.k;
          const int64_t off = t * a.token_stride + h * a.head_stride + 16 * c;
          *reinterpret_cast<uint4*>(cache + fresh * a.page_stride + off) =
              *reinterpret_cast<const uint4*>(cache + old * a.page_stride + off);
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
constexpr int kStage = 256;                    // moves worked out at a time

// blockIdx.x: the request; blockIdx.y: kThreads of a token's 16-byte pieces
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  pdl_wait();
  __shared__ int64_t s_from[kStage], s_to[kStage];
  const int r = blockIdx.x, tid = threadIdx.x;
  const int per_head = a.row_bytes >> 4, per_token = per_head * a.Hkv;
  const int x = (int)blockIdx.y * kThreads + tid;
  const bool have = x < 2 * per_token;
  const int v = x >= per_token, z = x - v * per_token, h = z / per_head;
  uint8_t* cache = (v ? a.v : a.k) + h * a.head_stride + 16 * (z - h * per_head);
  int begin = a.keep_start[r], end = a.keep_start[r + 1];
  const int first = a.first[r];
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  int bad = 0;
  if (begin < 0 || end < begin || end > a.N || first < 0) {
    bad = MOE_DEVERR_CACHE;
    begin = end = 0;
  }
  if (a.len_out && blockIdx.y == 0 && tid == 0) a.len_out[r] = max(first, 0) + end - begin;
  const int32_t* table = a.block_table + (int64_t)r * a.max_pages;
  const int page_mask = (1 << a.page_shift) - 1;
  for (int i0 = begin; i0 < end; i0 += kStage) {
    const int n = min(kStage, end - i0);
    __syncthreads();
    if (tid < n) {
      // where kept token i lies and where it goes (-1: it stays)
      const int i = i0 + tid, node = a.keep[i], place = i - begin;
      int64_t from = -1, to = -1;
      if (node < place || (i > begin && a.keep[i - 1] >= node) || (int64_t)first + node >= cap) {
        bad |= MOE_DEVERR_CACHE;
      } else if (node > place) {
        const int p = table[(first + node) >> a.page_shift], d = table[(first + place) >> a.page_shift];
        if (p < 0 || p >= a.n_pages || d < 0 || d >= a.n_pages || (a.shares && a.shares[d] > 0)) {
          bad |= MOE_DEVERR_CACHE;
        } else {
          from = p * a.page_stride + ((first + node) & page_mask) * a.token_stride;
          to = d * a.page_stride + ((first + place) & page_mask) * a.token_stride;
        }
      }
      s_from[tid] = from;
      s_to[tid] = to;
    }
    __syncthreads();
    if (!have) continue;
    // places ascend and lie at or before their sources: a place is written after it was read
    for (int j = 0; j < n; ++j)
      if (s_from[j] >= 0)
        *reinterpret_cast<uint4*>(cache + s_to[j]) = *reinterpret_cast<const uint4*>(cache + s_from[j]);
  }
  if (bad) set_error(&a.hdr->err, bad);
}

// ---------------------------------------------------------------------------
// release
// ---------------------------------------------------------------------------
constexpr int kRelThreads = 1024;
constexpr int kRelMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank_x() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// a word of another CTA's shared memory
__device__ __forceinline__ int remote_int(const int* p, uint32_t rank) {
  uint32_t at;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

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

// one cluster; its CTAs take equal parts of all entries, in the table's order
__global__ void __launch_bounds__(kRelThreads) release_kernel(const ReleaseArgs a) {
  extern __shared__ int prefix[];              // [R + 1] entries before each request
  __shared__ int tmp[32], s_freed;
  pdl_wait();
  const int tid = threadIdx.x, rank = (int)cluster_rank_x(), ctas = (int)gridDim.x;
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
  __syncthreads();
  // this thread's entries: a run of neighbours
  const int64_t e0 = (int64_t)total * rank / ctas, e1 = (int64_t)total * (rank + 1) / ctas;
  const int k = (int)((e1 - e0 + kRelThreads - 1) / kRelThreads);
  const int begin = (int)min(e0 + (int64_t)tid * k, e1), end = (int)min((int64_t)begin + k, e1);
  int row0 = 0;
  if (begin < end) {
    int lo = 0, hi = a.R;                      // the last row with prefix[row] <= begin
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= begin) lo = mid; else hi = mid;
    }
    row0 = lo;
  }
  // f(place in the table, page or -1) of each of them
  auto walk = [&](auto f) {
    int r = row0, lo = 0;
    if (begin < end) span(r, lo);
    for (int e = begin; e < end; ++e) {
      if (e >= prefix[r + 1]) {
        while (e >= prefix[r + 1]) ++r;
        span(r, lo);
      }
      const int at = r * a.max_pages + lo + (e - prefix[r]);
      int p = a.block_table[at];
      if (p < 0 || p >= a.n_pages) {
        if (p != -1) bad |= MOE_DEVERR_CACHE;
        p = -1;
      }
      f(at, p);
    }
  };
  auto meet = [] {
    __syncwarp();
    tc::cluster_sync();
  };
  if (a.shares) {
    walk([&](int, int p) { if (p >= 0) a.last[p] = -1; });
    meet();
    walk([&](int at, int p) {
      if (p < 0) return;
      atomicMax(&a.last[p], at);
      atomicSub(&a.shares[p], 1);
    });
    meet();
  }
  // freed: no holder is left, and this is the last of the entries that gave it back
  auto freed = [&](int at, int p) {
    return p >= 0 && (!a.shares || (__ldcg(&a.shares[p]) < 0 && __ldcg(&a.last[p]) == at));
  };
  int count = 0, own;
  walk([&](int at, int p) { count += freed(at, p); });
  int place = block_scan(count, tmp, &own);
  if (tid == 0) s_freed = own;
  meet();
  int all = 0;
  for (int c = 0; c < ctas; ++c) {
    const int n = c == rank ? own : remote_int(&s_freed, c);
    if (c < rank) place += n;
    all += n;
  }
  if (all > head || head > a.n_free) bad |= MOE_DEVERR_CACHE;   // more than the list gave out
  place += head - all;
  walk([&](int at, int p) {
    if (freed(at, p)) {
      if (place >= 0 && place < a.n_free) a.free_pages[place] = p;
      ++place;
    }
  });
  // every CTA has looked at the counts
  meet();
  walk([&](int at, int p) {
    if (a.shares && freed(at, p)) {
      if (__ldcg(&a.shares[p]) < -1) bad |= MOE_DEVERR_CACHE;   // given back more often than it was held
      a.shares[p] = 0;
    }
    a.block_table[at] = -1;
  });
  if (rank == 0 && tid == 0) *a.free_head = max(head - all, 0);
  if (bad) set_error(&a.hdr->err, bad);
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
  return launch_k(compact_kernel, dim3((unsigned)a.R, (unsigned)ceil_div(pieces, kThreads)), kThreads, 0, s, a);
}

cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t s) {
  const size_t smem = ((size_t)a.R + 1) * 4;
  static PerDeviceOnce once;
  int unused = 0;
  const cudaError_t e = once.run(
      [](int& v) {
        v = 1;
        return cudaFuncSetAttribute(release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (16384 + 1) * 4);
      },
      &unused);
  if (e != cudaSuccess) return e;
  const unsigned ctas = (int64_t)a.R * a.max_pages > 4096 ? kRelMaxCluster : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kRelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, release_kernel, a);
}

}  // namespace moe
