// Attention with shared prefixes where a request (or a group) has few rows: up to 32
// of a KV head.  BF16 rows and caches, FP32 scores, softmax and sums.
//
//   S = Q K^T,  p = exp2(c S - m),  l = sum p,  O = sum p V,  out = O / l
//
// The tiles of the tensor-memory kernel have 128 rows, and a piece of a run costs it 3 to
// 4 us beside its tiles: a request with a few rows and a few hundred tokens of
// its own behind the prefix is mostly that cost.  Here a unit (request or group, KV head,
// split of the keys) is a block of four or eight warps that work for themselves: each takes
// 16 keys of every 64 or 128, its own K and V by cp.async into its own stages, its own running
// maximum and sum, products by mma.sync (16 rows, 16 keys); they meet once, at the end.
// Several blocks an SM hide one another's waits.  The arithmetic is the other kernel's:
// probabilities in BF16 for the second product, sums before that rounding, the reference
// follows the maximum only past 2^8.
//
// Where the rows' prefix is the other kernel's and the keys are not split, the warps
// start from the prefix's partials in place of nothing, and the block writes the
// output; else its partials go to the join.
//
// The other kernel lets this one's blocks start as its own ones end; what they need of it,
// the prefix's partials, they wait for once their first keys are on the way.
//
// Bound: HBM, where there are enough units; else the latency of a block (table, keys,
// softmax, the join of the warps).
#include "attn_walk.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int kSub = 16;                       // keys of a warp at a time
constexpr int kStages = 2;                     // 16 keys each, of a warp
constexpr float kRaise = 8.f;                  // log2 units by which a maximum may pass its reference

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 bytes, zeros where `bytes` is 0
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <int DP, int kWarps>
struct Geo {
  static constexpr int CH = DP / 8;                          // 16-byte chunks of a head
  static constexpr int TILE = kSub * DP * 2;                 // 16 keys of K or V
  static constexpr int RING = 2 * kStages * TILE;            // of a warp: K and V of a stage
  static constexpr int ROW = DP + 4;                         // floats of a row in the join (four banks apart)
  static constexpr int SMEM = kWarps * RING > kWarps * kFewRows * ROW * 4 ? kWarps * RING : kWarps * kFewRows * ROW * 4;
};

// kWarps: 4, three blocks an SM; or 8, where there are fewer units than SMs have blocks
template <int DP, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 4 ? 3 : 1) attention_few_kernel(const AttnArgs a) {
  using X = Geo<DP, kWarps>;
  constexpr int kThreads = 32 * kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][kFewRows], s_l[kWarps][kFewRows];
  __shared__ int s_pages, s_merge;
  __shared__ __align__(128) uint4 s_q[kFewRows * X::CH];
  if (a.few_alone) pdl_wait();                 // (else the other kernel has waited, and let this one start)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // eight warps: a block a row block; four: a block takes them one after the other
  constexpr int kApart = kWarps == 8 ? kFewBlocks : 1;
  const int part = blockIdx.x / kApart, rb0 = blockIdx.x - part * kApart;
  const int unit = part / a.few_splits, split = part - unit * a.few_splits;
  const int walk = unit / a.Hkv, h = unit - walk * a.Hkv;
  const int tb = kFewRows / a.G;               // tokens of a row block
  int bad = 0;

  // rows that belong to no request (the other kernel's to clear where it runs too)
  if (a.few_alone) {
    const int live = a.R > 0 ? min(max(a.q_start[a.R], 0), a.T) : 0;
    for (int t = live + blockIdx.x; t < a.T; t += gridDim.x) {
      bf16* o = reinterpret_cast<bf16*>(a.out) + (int64_t)t * a.out_ld;
      for (int i = tid * 8; i < a.H * a.D; i += kThreads * 8) *reinterpret_cast<uint4*>(o + i) = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int i = tid; i < a.H; i += kThreads) a.lse[(int64_t)t * a.H + i] = -INFINITY;
    }
  }

  Req q;
  bool merge = false;                          // the rows' prefix is the other kernel's
  if (walk < a.n_groups) {
    q = group_request(
        a, prefix_group(a.group_start, a.prefix_row, a.prefix_len, walk, a.R, a.max_pages, a.page_shift, &bad), tb);
  } else {
    // the request's group, every thread looking at some
    const int r = walk - a.n_groups;
    if (tid == 0) s_pages = 0;
    q = own_request(a, r, 0, tb, &bad);
    if (a.n_groups > 0) {
      __syncthreads();
      PrefixGroup p;
      bool found = false;
      for (int i = tid; i < a.n_groups; i += kThreads) {
        const PrefixGroup x = prefix_group(a.group_start, a.prefix_row, a.prefix_len, i, a.R, a.max_pages, a.page_shift,
                                           nullptr);
        // (of the groups that begin at or before r the last one counts, whatever its end)
        if (a.group_start[i] <= r && (i + 1 == a.n_groups || a.group_start[i + 1] > r) && r < x.end && x.pages) {
          p = x;
          found = true;
          s_pages = x.pages;
        }
      }
      __syncthreads();
      behind_prefix(a, q, s_pages);
      if (found) s_merge = !few(a, group_request(a, p, tb));     // (read behind the next barrier)
    }
  }
  if (bad && h == 0 && split == 0 && tid == 0) set_error(&a.hdr->err, MOE_DEVERR_CACHE);
  if (rb0 >= q.blocks || !few(a, q)) {
    if (blockIdx.x == 0) pdl_wait();           // this kernel does not end before the other
    return;
  }
  // this block's keys: tiles of 16 a warp, the same number a split
  constexpr int kTile = kSub * kWarps;
  const int tiles = max((q.kv + kTile - 1) / kTile, 1), per = (tiles + a.few_splits - 1) / a.few_splits;
  const int parts = (tiles + per - 1) / per;
  if (split >= parts) {
    if (blockIdx.x == 0) pdl_wait();
    return;
  }
  const int sub0 = split * per * kWarps + warp, sub1 = min((split + 1) * per, tiles) * kWarps;
  const int32_t* table = a.block_table + (int64_t)q.row * a.max_pages + q.skip;
  const bf16 *kc = reinterpret_cast<const bf16*>(a.k) + (int64_t)h * a.head_stride,
             *vc = reinterpret_cast<const bf16*>(a.v) + (int64_t)h * a.head_stride;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * X::RING;
  const uint32_t q_smem = (uint32_t)__cvta_generic_to_shared(s_q);
  const float c = a.scale * 1.4426950408889634f;
  const int g = lane >> 2, t4 = lane & 3;      // the row (and + 8) and the pair of columns that a lane has of a product

  // where key `key` lies in a cache, elements; -1: nowhere
  auto place = [&](int key) -> int64_t {
    if (key >= q.kv) return -1;
    const int pg = table[key >> a.page_shift];
    if (pg < 0 || pg >= a.n_pages) {
      set_error(&a.hdr->err, MOE_DEVERR_CACHE);
      return -1;
    }
    return (int64_t)pg * a.page_stride + (int64_t)(key & ((1 << a.page_shift) - 1)) * a.token_stride;
  };
  // 16 keys into a stage; at: a lane's key (both halves of the warp have all 16)
  auto copy = [&](int stage, int64_t at) {
    constexpr int KEYS = 32 / X::CH;           // keys of a step of the warp
    const uint32_t dst = ring + stage * 2 * X::TILE;
    const int ch = lane % X::CH;
#pragma unroll
    for (int s = 0; s < kSub / KEYS; ++s) {
      const int key = s * KEYS + lane / X::CH;
      const int64_t off = __shfl_sync(0xffffffffu, at, key);
      const int bytes = off >= 0 && ch * 8 < a.D ? 16 : 0;
      const int64_t from = bytes ? off + ch * 8 : 0;
      const uint32_t to = dst + key * DP * 2 + ((ch ^ (key & 7)) << 4);
      copy16(to, kc + from, bytes);
      copy16(to + X::TILE, vc + from, bytes);
    }
    copy_commit();
  };
  // a lane's key of the warp's 16 from `sub` on
  auto keys = [&](int sub) -> int64_t { return sub < sub1 ? place(sub * kSub + (lane & 15)) : -1; };

  for (int rb = rb0; rb < q.blocks; rb += kApart) {
    const int tok0 = q.q0 + rb * tb, ntok = min(tb, q.n - rb * tb), valid = ntok * a.G;
    // Q, read again for every 16 keys (in registers it would cost a block an SM)
    for (int i = tid; i < kFewRows * X::CH; i += kThreads) {
      const int row = i / X::CH, ch = i - row * X::CH, tk = row / a.G;
      const bool in = row < valid && ch * 8 < a.D;
      copy16(q_smem + row * DP * 2 + ((ch ^ (row & 7)) << 4),
             reinterpret_cast<const bf16*>(a.q) +
                 (in ? (int64_t)(tok0 + tk) * a.q_ld + (int64_t)(h * a.G + row - tk * a.G) * a.D + 8 * ch : 0),
             in ? 16 : 0);
    }
    copy_commit();
    int64_t at[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) at[i] = keys(sub0 + i * kWarps);
#pragma unroll
    for (int i = 0; i < kStages; ++i) copy(i, at[i]);
    int64_t next = keys(sub0 + kStages * kWarps);
    copy_wait<kStages>();
    __syncthreads();                           // Q is there, and the word on the prefix
    merge = parts == 1 && q.flags & kJoined && s_merge;
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float mc[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    if (!a.few_alone) pdl_wait();
    if (merge) {
      // a warp starts from every kWarps'th of the prefix's partials
      PartsOf pre[2];
      int hd[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = g + 8 * i, tk = row / a.G;
        hd[i] = row - tk * a.G;
        pre[i] = parts_of(a, 0, h, tok0 + min(tk, ntok - 1));
        if (row >= valid) pre[i].parts = 0;
      }
      float2 x[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (warp < pre[i].parts) {
          const float2* ml;
          const float4* from;
          partial<DP>(a, pre[i], 0, h, tok0 * a.G + g + 8 * i, hd[i], warp, ml, from);
          x[i] = __ldcg(ml);
#pragma unroll
          for (int j = 0; j < DP / 8; ++j) {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(from) + t4 + 4 * j);
            o[j][2 * i] = y.x;
            o[j][2 * i + 1] = y.y;
          }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (x[i].y != 0.f) {                   // (a part without a visible key has zeros)
          mc[i] = x[i].x;
          l[i] = t4 == 0 ? x[i].y : 0.f;       // (the lanes of a row are added up at the end)
        }
#pragma unroll 1
        for (int k = warp + kWarps; k < pre[i].parts; k += kWarps) {
          const float2* ml;
          const float4* from;
          partial<DP>(a, pre[i], 0, h, tok0 * a.G + g + 8 * i, hd[i], k, ml, from);
          const float2 z = __ldcg(ml);
          if (z.y == 0.f) continue;
          const float top = fmaxf(mc[i], z.x), f0 = mc[i] == -INFINITY ? 0.f : ex2(mc[i] - top), f1 = ex2(z.x - top);
          mc[i] = top;
          l[i] = l[i] * f0 + (t4 == 0 ? z.y * f1 : 0.f);
#pragma unroll
          for (int j = 0; j < DP / 8; ++j) {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(from) + t4 + 4 * j);
            o[j][2 * i] = o[j][2 * i] * f0 + y.x * f1;
            o[j][2 * i + 1] = o[j][2 * i + 1] * f0 + y.y * f1;
          }
        }
      }
    }

    int stage = 0;
    for (int sub = sub0; sub < sub1; sub += kWarps) {
      const uint32_t kt = ring + stage * 2 * X::TILE, vt = kt + X::TILE;
      const int k0 = sub * kSub;
      copy_wait<kStages - 1>();
      __syncwarp();
      // scores of 16 rows and 16 keys
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        // matrices: keys 0-7 and 8-15, two chunks each
        const int key = (lane & 7) + ((lane >> 4) << 3), half = lane >> 3 & 1, q_row = lane & 15;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          uint32_t x[4], b[4];
          ldsm4(q_smem + q_row * DP * 2 + (((2 * k + (lane >> 4)) ^ (q_row & 7)) << 4), x);
          ldsm4(kt + key * DP * 2 + (((2 * k + half) ^ (key & 7)) << 4), b);
          mma_bf16_16816(s[0], x[0], x[1], x[2], x[3], b[0], b[1]);
          mma_bf16_16816(s[1], x[0], x[1], x[2], x[3], b[2], b[3]);
        }
      }
      uint32_t odd = 0;                        // keys whose V is not finite, nodes among them alone
      if (k0 + kSub > q.ctx) {
        // what each row sees of the nodes
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = min(g + 8 * i, valid - 1), tk = row / a.G, node = rb * tb + tk;
          const int32_t* mask = a.tree_mask ? a.tree_mask + (int64_t)(tok0 + tk) * a.mask_words : nullptr;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = k0 + 8 * (j >> 1) + 2 * t4 + (j & 1), n = key - q.ctx;
            bool see = key < q.kv;
            if (see && n >= 0) see = !mask ? n <= node : (n >> 5) < a.mask_words && ((uint32_t)mask[n >> 5] >> (n & 31) & 1u);
            if (!see) s[j >> 1][2 * i + (j & 1)] = -INFINITY;
          }
        }
        // lanes 2 i and 2 i + 1: halves of key i's V
        const int key = lane >> 1;
        bool strange = false;
        if (k0 + key >= q.ctx && k0 + key < q.kv)
          for (int i = 0; i < X::CH / 2; ++i) {
            uint32_t w[4];
            const uint32_t from = vt + key * DP * 2 + ((((lane & 1) * (X::CH / 2) + i) ^ (key & 7)) << 4);
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from));
#pragma unroll
            for (int e = 0; e < 4; ++e) strange |= (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
          }
        const uint32_t set = __ballot_sync(0xffffffffu, strange);
        odd = (set | set >> 1) & 0x55555555u;  // bit 2 i: key i
      }
      // the rows' maxima, and O scaled where a reference rises
      float top[2] = {fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])),
                      fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]))};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2)) * c;
      }
      const bool up0 = top[0] > mc[0] + kRaise || (mc[0] == -INFINITY && top[0] > mc[0]);
      const bool up1 = top[1] > mc[1] + kRaise || (mc[1] == -INFINITY && top[1] > mc[1]);
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float f0 = up0 ? (mc[0] == -INFINITY ? 0.f : ex2(mc[0] - top[0])) : 1.f;
        const float f1 = up1 ? (mc[1] == -INFINITY ? 0.f : ex2(mc[1] - top[1])) : 1.f;
        if (up0) mc[0] = top[0];
        if (up1) mc[1] = top[1];
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f0;
          o[i][2] *= f1;
          o[i][3] *= f1;
        }
      }
      const float base[2] = {mc[0] == -INFINITY ? 0.f : mc[0], mc[1] == -INFINITY ? 0.f : mc[1]};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[j][i] = ex2(fmaf(s[j][i], c, -base[i >> 1]));
          l[i >> 1] += s[j][i];
        }
      const uint32_t p[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]), pack_bf16(s[1][0], s[1][1]),
                             pack_bf16(s[1][2], s[1][3])};
      if (__builtin_expect(odd != 0, 0)) {
        // out of the product, and added to the rows that see them
        for (uint32_t left = odd; left; left &= left - 1) {
          const int key = (__ffs(left) - 1) >> 1;
          for (int i = lane; i < X::CH; i += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vt + key * DP * 2 + (i << 4)), "r"(0u) : "memory");
          const int from = (lane & ~3) | ((key & 7) >> 1);
          const uint32_t w0 = __shfl_sync(0xffffffffu, key < 8 ? p[0] : p[2], from);
          const uint32_t w1 = __shfl_sync(0xffffffffu, key < 8 ? p[1] : p[3], from);
          const float p0 = key & 1 ? bf16_hi(w0) : bf16_lo(w0), p1 = key & 1 ? bf16_hi(w1) : bf16_lo(w1);
          const int64_t off = place(k0 + key);
          if (off < 0) continue;
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            const int col = 8 * i + 2 * t4;
            if (col >= a.D) continue;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(vc + off + col);
            if (p0 != 0.f) {
              o[i][0] = fmaf(p0, bf16_lo(w), o[i][0]);
              o[i][1] = fmaf(p0, bf16_hi(w), o[i][1]);
            }
            if (p1 != 0.f) {
              o[i][2] = fmaf(p1, bf16_lo(w), o[i][2]);
              o[i][3] = fmaf(p1, bf16_hi(w), o[i][3]);
            }
          }
        }
        __syncwarp();
      }
      {
        // matrices: chunk 0's two key halves, chunk 1's
        const int key = (lane & 7) + ((lane >> 3 & 1) << 3), half = lane >> 4;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
          uint32_t b[4];
          ldsm4_t(vt + key * DP * 2 + (((2 * i + half) ^ (key & 7)) << 4), b);
          mma_bf16_16816(o[2 * i], p[0], p[1], p[2], p[3], b[0], b[1]);
          mma_bf16_16816(o[2 * i + 1], p[0], p[1], p[2], p[3], b[2], b[3]);
        }
      }
      __syncwarp();                            // the stage is read before it is filled again
      copy(stage, next);
      next = keys(sub + (kStages + 1) * kWarps);
      if (++stage == kStages) stage = 0;
    }

    // ---- the warps' parts, in warp order ----
    copy_wait<0>();
    __syncthreads();
    float* so = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (t4 == 0) {
        s_m[warp][g + 8 * i] = mc[i];
        s_l[warp][g + 8 * i] = l[i];
      }
#pragma unroll
      for (int j = 0; j < DP / 8; ++j)
        *reinterpret_cast<float2*>(so + (warp * kFewRows + g + 8 * i) * X::ROW + 8 * j + 2 * t4) =
            make_float2(o[j][2 * i], o[j][2 * i + 1]);
    }
    __syncthreads();
    constexpr int kCols = kThreads / kFewRows;   // threads of a row: columns 4 (c0 + kCols i)
    constexpr int kPer = DP / 4 / kCols;
    const int row = tid / kCols, c0 = tid - row * kCols, tk = row / a.G, hd = row - tk * a.G, head = h * a.G + hd;
    float top = -INFINITY, sum = 0.f, f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (s_l[w][row] != 0.f) top = fmaxf(top, s_m[w][row]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = s_l[w][row] == 0.f ? 0.f : ex2(s_m[w][row] - top);       // (no visible key in that part)
      if (s_l[w][row] != 0.f) sum = fmaf(s_l[w][row], f[w], sum);
    }
    const int which = q.flags & kPrefix ? 0 : 1;
    const bool whole = parts == 1 && (!q.flags || merge);
    const int slot = part * kFewBlocks + rb;
    const int rows_all = a.T * a.G, rg = tok0 * a.G + row;
    const int64_t side = which * a.Hkv + h;
    if (row < valid) {
      float4 acc[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (f[w] == 0.f) continue;
          const float4 x = *reinterpret_cast<const float4*>(so + (w * kFewRows + row) * X::ROW + 4 * (c0 + kCols * i));
          acc[i].x = fmaf(x.x, f[w], acc[i].x);
          acc[i].y = fmaf(x.y, f[w], acc[i].y);
          acc[i].z = fmaf(x.z, f[w], acc[i].z);
          acc[i].w = fmaf(x.w, f[w], acc[i].w);
        }
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        bf16* out = reinterpret_cast<bf16*>(a.out) + (int64_t)(tok0 + tk) * a.out_ld + (int64_t)head * a.D;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (4 * (c0 + kCols * i) < a.D)
            *reinterpret_cast<uint2*>(out + 4 * (c0 + kCols * i)) =
                make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
        if (a.lse && c0 == 0)
          a.lse[(int64_t)(tok0 + tk) * a.H + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      } else {
        const int64_t at_row = parts == 1 ? side * rows_all + rg : (int64_t)slot * kFewRows + row;
        float4* part = reinterpret_cast<float4*>(parts == 1 ? a.rows_part : a.few_part) + at_row * (DP / 4);
#pragma unroll
        for (int i = 0; i < kPer; ++i) part[c0 + kCols * i] = acc[i];
        if (c0 == 0) (parts == 1 ? a.rows_ml : a.few_ml)[at_row] = make_float2(top, sum);
      }
    }
    if (split == 0 && tid < ntok)
      a.parts_of[side * a.T + tok0 + tid] = make_int4(whole ? 0 : parts, parts > 1 ? slot : 0, tid * a.G,
                                                      (q.flags & kJoined) | (parts > 1 ? kFewSlots : 0));
    __syncthreads();                           // the buffers are the next row block's
  }
}

template <int DP, int kWarps>
cudaError_t launch_dp(const AttnArgs& a, cudaStream_t s) {
  static PerDeviceOnce once;
  int unused = 0;
  const cudaError_t e = once.run(
      [](int& v) {
        v = 1;
        return cudaFuncSetAttribute(attention_few_kernel<DP, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Geo<DP, kWarps>::SMEM);
      },
      &unused);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)(a.n_groups + a.R) * a.Hkv;
  return launch_k(attention_few_kernel<DP, kWarps>, dim3((unsigned)std::max<int64_t>(units * a.few_splits * (kWarps == 8 ? kFewBlocks : 1), 1)),
                  dim3(32 * kWarps), Geo<DP, kWarps>::SMEM, s, a);
}

}  // namespace

// Few units: blocks of eight warps, their keys split while that leaves SMs without one; else blocks of four.
void few_shape(AttnArgs* a) {
  const int64_t units = (int64_t)(a->n_groups + a->R) * a->Hkv, sms = 152;
  if (a->G > kFewRows) return;                 // (a token's rows do not fit a block's 16)
  a->few_tokens = kFewBlocks * (kFewRows / a->G);
  a->few_warps = units < 2 * sms ? 8 : 4;
  a->few_splits = (int)std::min<int64_t>(std::max<int64_t>(sms / std::max<int64_t>(units, 1), 1), kFewMaxSplits);
  a->few_keys = a->few_splits * a->few_warps * kFewKeys;
  a->few_alone = a->T <= a->few_tokens && (int64_t)a->max_pages << a->page_shift <= a->few_keys;
}

cudaError_t launch_attention_few(const AttnArgs& a, cudaStream_t s) {
  if (a.few_warps == 8) return a.D <= 64 ? launch_dp<64, 8>(a, s) : launch_dp<128, 8>(a, s);
  return a.D <= 64 ? launch_dp<64, 4>(a, s) : launch_dp<128, 4>(a, s);
}

}  // namespace moe
