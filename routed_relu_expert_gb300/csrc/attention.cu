// Tree attention over a paged cache on the CUDA cores, FP32 arithmetic
// throughout: the attention of FP32 layers.
//
//   s_k = scale q.k,  m = max s_k,  l = sum exp(s_k - m),  o = sum exp(s_k - m) v_k / l
//
// A block takes one node's row, four of the query heads that share a KV head,
// and one range of keys; its four warps take 32 keys at a time, a lane a key
// for the scores (the lane walks its key's row in 16-byte pieces, the queries
// come from shared memory), a lane a piece of the head for the output.  Running
// maximum and sum per warp, joined over the warps at the end in warp order.
// Keys that the row does not see are never read.
//
// Bound: latency at the sizes it is for (a block takes about 128 keys; eight V rows
// in flight a warp): 3 requests of up to 777 tokens, trees of up to 5, 8 heads over
// 2 KV heads of 64: 13 us, of which 5 are the launch and the join of the splits.
//
// When rows x KV heads x head groups leave SMs idle the keys are split over
// blocks (a rule on the counts alone: the lengths live on the device); each
// stores its (max, sum, output) and the last to arrive adds them in split order,
// so the result does not depend on which one that is.
#include "attn.h"

#include <algorithm>

namespace moe {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = 4;                      // query heads a block
constexpr int kMaxParts = 640;                 // splits of all units together
static_assert((size_t)kMaxParts * kHeads <= kAttnPartSlots * kAttnRows, "partials in the workspace");

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// request of row t: the last r with q_start[r] <= t (rows past q_start[R]: R)
__device__ __forceinline__ int request_of(const int32_t* q_start, int R, int t) {
  if (R == 0 || t >= q_start[R]) return R;
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q_start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// SHARED: the tokens of a group's prefix are read through the group's row of the table (every row of the group by
// itself: the pages come from memory once and from L2 after that).  4 requests of up to 3 nodes behind 600 common
// tokens, 8 heads over 2 of 64: 12.5 us, the latency of one pass over 128 keys a block and of the join of its splits.
template <bool SHARED>
__global__ void __launch_bounds__(kThreads) attention_f32_kernel(const AttnArgs a, int groups, int splits) {
  pdl_wait();
  __shared__ __align__(16) float s_q[kHeads][kAttnPartDim];
  __shared__ __align__(16) float s_o[kWarps][kHeads][kAttnPartDim];
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = blockIdx.x % splits, unit = blockIdx.x / splits;
  const int grp = unit % groups, hk = (unit / groups) % a.Hkv, t = unit / (groups * a.Hkv);
  const int h0 = hk * a.G + grp * kHeads, nh = min(kHeads, a.G - grp * kHeads);
  const int D = a.D;
  const int r = request_of(a.q_start, a.R, t);
  int bad = 0;

  for (int i = tid; i < kHeads * D; i += kThreads) {
    const int h = i / D, d = i - h * D;
    float v = 0.f;
    if (h < nh) {
      v = reinterpret_cast<const float*>(a.q)[(int64_t)t * a.q_ld + (int64_t)(h0 + h) * D + d];
    }
    s_q[h][d] = v;
  }
  // groups whose bounds do not ascend share nothing
  bool mixed = false;
  if (SHARED) {
    for (int g = tid; g < a.n_groups; g += kThreads) mixed |= a.group_start[g + 1] < a.group_start[g];
    mixed = __syncthreads_or(mixed);
  } else {
    __syncthreads();
  }

  float m[kHeads], l[kHeads];
  float4 o[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int dl = lane * 4;                     // this lane's piece of the head
  if (SHARED && blockIdx.x == 0)
    for (int g = tid; g < a.n_groups; g += kThreads) {
      int no_group = 0;
      prefix_group(a.group_start, a.prefix_row, a.prefix_len, g, a.R, a.max_pages, a.page_shift, &no_group);
      if (no_group) bad = MOE_DEVERR_CACHE;
    }
  if (r < a.R) {
    const int q0 = a.q_start[r], n = a.q_start[r + 1] - q0, node = t - q0;
    const int64_t cap = (int64_t)a.max_pages << a.page_shift;
    // a length past the table's row is cut there: its tokens before that stay where they are, nodes among them or not
    const int len = a.kv_len[r];
    if (len < n || len > cap) bad = MOE_DEVERR_CACHE;
    const int ctx = (int)min((int64_t)max(len, n) - n, cap);
    const int kv = (int)min((int64_t)ctx + n, cap);
    const int32_t* table = a.block_table + (int64_t)r * a.max_pages;
    const int32_t* table0 = table;             // of the first `shared` pages
    int shared = 0;
    if (SHARED) {
      const int g = mixed ? -1 : group_of(a.group_start, a.n_groups, r);
      if (g >= 0) {
        const PrefixGroup p = prefix_group(a.group_start, a.prefix_row, a.prefix_len, g, a.R, a.max_pages, a.page_shift,
                                           nullptr);
        if (r < p.end && ctx >= (int64_t)p.pages << a.page_shift) {
          table0 = a.block_table + (int64_t)p.row * a.max_pages;
          shared = p.pages;
        }
      }
    }
    const int32_t* mask = a.tree_mask ? a.tree_mask + (int64_t)t * a.mask_words : nullptr;
    const int tiles = (kv + 31) / 32;
    const int w0 = (int)((int64_t)tiles * split / splits), w1 = (int)((int64_t)tiles * (split + 1) / splits);
    for (int tile = w0 + warp; tile < w1; tile += kWarps) {
      const int key = tile * 32 + lane;
      bool see = key < ctx;
      if (!see && key < kv) {
        const int j = key - ctx;
        if (!mask) see = j <= node;
        else see = (j >> 5) < a.mask_words && ((uint32_t)mask[j >> 5] >> (j & 31) & 1u);
      }
      int64_t at = 0;
      bool zero = false;                       // a page outside the cache reads as zeros
      if (see) {
        const int at_page = key >> a.page_shift;
        const int page = SHARED && at_page < shared ? table0[at_page] : table[at_page];
        zero = page < 0 || page >= a.n_pages;
        if (zero) bad = MOE_DEVERR_CACHE;
        else
          at = (int64_t)page * a.page_stride + (int64_t)(key & ((1 << a.page_shift) - 1)) * a.token_stride +
               (int64_t)hk * a.head_stride;
      }
      float s[kHeads] = {0.f, 0.f, 0.f, 0.f};
      if (see && !zero) {
        const float* kp = reinterpret_cast<const float*>(a.k) + at;
#pragma unroll 8
        for (int d = 0; d < D; d += 4) {
          const float4 kv4 = load4(kp + d);
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const float4 q4 = *reinterpret_cast<const float4*>(&s_q[h][d]);
            s[h] = fmaf(kv4.x, q4.x, s[h]);
            s[h] = fmaf(kv4.y, q4.y, s[h]);
            s[h] = fmaf(kv4.z, q4.z, s[h]);
            s[h] = fmaf(kv4.w, q4.w, s[h]);
          }
        }
      }
      const uint32_t seen = __ballot_sync(0xffffffffu, see), read = __ballot_sync(0xffffffffu, see && !zero);
      if (!seen) continue;
      float p[kHeads];
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        const float x = see ? s[h] * a.scale : -INFINITY;
        float top = x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          const float y = __shfl_xor_sync(0xffffffffu, top, off);
          top = (y > top || y != y) ? y : top;                  // a NaN score stays
        }
        const float m_new = (top > m[h] || top != top) ? top : m[h];
        const float base = m_new == -INFINITY ? 0.f : m_new;    // all scores so far -inf
        const float f = m[h] == -INFINITY ? 0.f : expf(m[h] - base);
        p[h] = see ? expf(x - base) : 0.f;
        float sum = p[h];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l[h] = fmaf(l[h], f, sum);
        m[h] = m_new;
        o[h].x *= f; o[h].y *= f; o[h].z *= f; o[h].w *= f;
      }
      // eight keys' V rows in flight at a time
#pragma unroll
      for (int k0 = 0; k0 < 32; k0 += 8) {
        if (!(read >> k0 & 0xffu)) continue;
        float4 v4[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int64_t va = __shfl_sync(0xffffffffu, at, k0 + k);
          v4[k] = dl < D && (read >> (k0 + k) & 1u) ? load4(reinterpret_cast<const float*>(a.v) + va + dl)
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const float w = __shfl_sync(0xffffffffu, p[h], k0 + k);
            if (!(read >> (k0 + k) & 1u)) continue;
            o[h].x = fmaf(w, v4[k].x, o[h].x);
            o[h].y = fmaf(w, v4[k].y, o[h].y);
            o[h].z = fmaf(w, v4[k].z, o[h].z);
            o[h].w = fmaf(w, v4[k].w, o[h].w);
          }
        }
      }
    }
  }
  if (bad) set_error(&a.hdr->err, bad);

  // join the warps, in warp order
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (dl < D) *reinterpret_cast<float4*>(&s_o[warp][h][dl]) = o[h];
    if (lane == 0) {
      s_m[warp][h] = m[h];
      s_l[warp][h] = l[h];
    }
  }
  __syncthreads();
  auto factor = [](float mine, float top) { return mine == -INFINITY ? 0.f : expf(mine - top); };
  const int64_t slot = (int64_t)unit * splits + split;
  for (int i = tid; i < nh * D; i += kThreads) {
    const int h = i / D, d = i - h * D;
    float top = s_m[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = (s_m[w][h] > top || s_m[w][h] != s_m[w][h]) ? s_m[w][h] : top;
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = factor(s_m[w][h], top);
      sum = fmaf(s_l[w][h], f, sum);
      acc = fmaf(s_o[w][h][d], f, acc);
    }
    if (splits == 1) {
      reinterpret_cast<float*>(a.out)[(int64_t)t * a.out_ld + (int64_t)(h0 + h) * D + d] =
          top == -INFINITY ? 0.f : acc / sum;
      if (a.lse && d == 0) a.lse[(int64_t)t * a.H + h0 + h] = top == -INFINITY ? -INFINITY : top + logf(sum);
    } else {
      a.part[(slot * kHeads + h) * kAttnPartDim + d] = acc;
      if (d == 0) a.part_ml[slot * kHeads + h] = make_float2(top, sum);
    }
  }
  if (splits == 1) return;

  __threadfence();
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(&a.hdr->counters[unit], 1) == splits - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int i = tid; i < nh * D; i += kThreads) {
    const int h = i / D, d = i - h * D;
    const int64_t first = (int64_t)unit * splits;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
    for (int s0 = 0; s0 < splits; s0 += 8) {                 // eight splits' loads in flight
      float2 ml[8];
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool in = s0 + k < splits;
        const int64_t at = (first + s0 + k) * kHeads + h;
        ml[k] = in ? __ldcg(&a.part_ml[at]) : make_float2(-INFINITY, 0.f);
        v[k] = in ? __ldcg(&a.part[at * kAttnPartDim + d]) : 0.f;
      }
      float m_new = top;
#pragma unroll
      for (int k = 0; k < 8; ++k) m_new = (ml[k].x > m_new || ml[k].x != ml[k].x) ? ml[k].x : m_new;
      const float g = factor(top, m_new);
      top = m_new;
      sum *= g;
      acc *= g;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float f = factor(ml[k].x, top);
        sum = fmaf(ml[k].y, f, sum);
        acc = fmaf(v[k], f, acc);
      }
    }
    reinterpret_cast<float*>(a.out)[(int64_t)t * a.out_ld + (int64_t)(h0 + h) * D + d] =
        top == -INFINITY ? 0.f : acc / sum;
    if (a.lse && d == 0) a.lse[(int64_t)t * a.H + h0 + h] = top == -INFINITY ? -INFINITY : top + logf(sum);
  }
  if (tid == 0) a.hdr->counters[unit] = 0;
}

}  // namespace

// Splits: of at least 128 keys each if the tables' rows are full (a tile for each
// of the four warps), at most 32, while the grid is about four blocks an SM at most and
// the workspace holds their counters.
template <bool SHARED>
static cudaError_t launch_f32(const AttnArgs& a, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  const int groups = (a.G + kHeads - 1) / kHeads;
  const int64_t units = (int64_t)a.T * a.Hkv * groups;
  int64_t splits = 1;
  if (units <= kAttnCounters / 4) {
    const int64_t keys = (int64_t)a.max_pages << a.page_shift;
    splits = std::max<int64_t>(1, std::min<int64_t>({32, kMaxParts / units, ceil_div(keys, 128)}));
  }
  launch_k(attention_f32_kernel<SHARED>, dim3((unsigned)(units * splits)), kThreads, 0, s, a, groups, (int)splits);
  return cudaGetLastError();
}

cudaError_t launch_attention_f32(const AttnArgs& a, cudaStream_t s) { return launch_f32<false>(a, s); }
cudaError_t launch_prefix_attention_f32(const AttnArgs& a, cudaStream_t s) { return launch_f32<true>(a, s); }

}  // namespace moe
