// Attention with shared prefixes where a request (or a group) has few rows: up to 32
// of a KV head.  BF16 rows and caches, FP32 scores, softmax and sums.
//
//   S = Q K^T,  p = exp2(c S - m),  l = sum p,  O = sum p V,  out = O / l
//
// The tiles of the tensor-memory kernel have 128 rows, and a piece of a run costs it 3 to
// 4 us beside its tiles: a request with a few rows and a few hundred tokens of
// its own behind the prefix is mostly that cost.  Here a unit (request or group, KV head,
// split of the keys) is a block of four warps that work for themselves: each takes
// 16 keys of every 64, its own K and V by cp.async into its own buffers, its own running
// maximum and sum, products by mma.sync (16 rows, 16 keys); they meet once, at the end.
// Several blocks an SM hide one another's waits.  The arithmetic is the other kernel's:
// probabilities in BF16 for the second product, sums before that rounding, the reference
// follows the maximum only past 2^8.
//
// Where the rows' prefix was another kernel's and the keys are not split, the
// block adds the prefix's partials itself and writes the output; else the partials
// go to the join.
//
// Bound: HBM, where there are enough units; else the latency of a block (table, keys,
// softmax, the join of the warps).
#include "attn_walk.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSub = 16;                       // keys of a warp at a time
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

template <int DP>
struct Geo {
  static constexpr int CH = DP / 8;                          // 16-byte chunks of a head
  static constexpr int TILE = kSub * DP * 2;                 // 16 keys of K or V
  static constexpr int RING = 3 * TILE;                      // of a warp: K, and V twice
  static constexpr int ROW = DP + 4;                         // floats of a row in the join (four banks apart)
  static constexpr int SMEM = kWarps * RING > kWarps * kFewRows * ROW * 4 ? kWarps * RING : kWarps * kFewRows * ROW * 4;
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 4) attention_few_kernel(const AttnArgs a) {
  using X = Geo<DP>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][kFewRows], s_l[kWarps][kFewRows];
  __shared__ int s_pages, s_merge;
  __shared__ __align__(128) uint4 s_q[kFewRows * X::CH];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / a.few_splits, split = blockIdx.x - unit * a.few_splits;
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
    q = own_request(a, r, 0, tb, &bad);
    if (a.n_groups > 0) {
      if (tid == 0) s_pages = 0;
      __syncthreads();
      for (int i = tid; i < a.n_groups; i += kThreads) {
        const PrefixGroup p = prefix_group(a.group_start, a.prefix_row, a.prefix_len, i, a.R, a.max_pages, a.page_shift,
                                           nullptr);
        // (of the groups that begin at or before r the last one counts, whatever its end)
        if (a.group_start[i] <= r && (i + 1 == a.n_groups || a.group_start[i + 1] > r) && r < p.end && p.pages) {
          s_pages = p.pages;
          s_merge = !few(a, group_request(a, p, tb));
        }
      }
      __syncthreads();
      const int pages = s_pages, prefix = pages << a.page_shift;
      if (pages && q.ctx >= prefix) {          // as own_request
        q.ctx -= prefix;
        q.kv -= prefix;
        q.skip = pages;
        q.flags = kJoined;
        merge = s_merge;
      }
    }
  }
  if (bad && h == 0 && split == 0 && tid == 0) set_error(&a.hdr->err, MOE_DEVERR_CACHE);
  if (q.n == 0 || !few(a, q)) return;
  // this block's keys: tiles of 64, the same number a split
  constexpr int kTile = kSub * kWarps;
  const int tiles = max((q.kv + kTile - 1) / kTile, 1), per = (tiles + a.few_splits - 1) / a.few_splits;
  const int parts = (tiles + per - 1) / per;
  if (split >= parts) return;
  const int sub0 = split * per * kWarps + warp, sub1 = min((split + 1) * per, tiles) * kWarps;
  const int32_t* table = a.block_table + (int64_t)q.row * a.max_pages + q.skip;
  const bf16 *kc = reinterpret_cast<const bf16*>(a.k) + (int64_t)h * a.head_stride,
             *vc = reinterpret_cast<const bf16*>(a.v) + (int64_t)h * a.head_stride;
  const uint32_t kt = (uint32_t)__cvta_generic_to_shared(smem) + warp * X::RING;
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
  // 16 keys of a cache into a buffer; at: a lane's key (both halves of the warp have all 16)
  auto copy = [&](const bf16* cache, uint32_t dst, int64_t at) {
    constexpr int KEYS = 32 / X::CH;           // keys of a step of the warp
    const int ch = lane % X::CH;
#pragma unroll
    for (int s = 0; s < kSub / KEYS; ++s) {
      const int key = s * KEYS + lane / X::CH;
      const int64_t off = __shfl_sync(0xffffffffu, at, key);
      const int bytes = off >= 0 && ch * 8 < a.D ? 16 : 0;
      copy16(dst + key * DP * 2 + ((ch ^ (key & 7)) << 4), cache + (bytes ? off + ch * 8 : 0), bytes);
    }
    copy_commit();
  };

  for (int rb = 0; rb < q.blocks; ++rb) {
    const int tok0 = q.q0 + rb * tb, ntok = min(tb, q.n - rb * tb), valid = ntok * a.G;
    int64_t at = sub0 < sub1 ? place(sub0 * kSub + (lane & 15)) : -1;
    copy(kc, kt, at);
    copy(vc, kt + X::TILE, at);
    at = sub0 + kWarps < sub1 ? place((sub0 + kWarps) * kSub + (lane & 15)) : -1;
    // Q, read again for every 16 keys (in registers it would cost a block an SM)
    __syncthreads();
    for (int i = tid; i < kFewRows * X::CH; i += kThreads) {
      const int row = i / X::CH, ch = i - row * X::CH, tk = row / a.G;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < valid && ch * 8 < a.D)
        x = *reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(a.q) + (int64_t)(tok0 + tk) * a.q_ld +
                                            (int64_t)(h * a.G + row - tk * a.G) * a.D + 8 * ch);
      s_q[row * X::CH + (ch ^ (row & 7))] = x;
    }
    __syncthreads();
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float mc[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    int turn = 0;                              // the V buffer
    for (int sub = sub0; sub < sub1; sub += kWarps) {
      const uint32_t vt = kt + X::TILE * (1 + turn);
      const bool more = sub + kWarps < sub1;
      const int k0 = sub * kSub;
      copy_wait<1>();                          // K of these keys (V may still come)
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
      __syncwarp();                            // K is read: the next keys' K comes into its place
      if (more) {
        copy(kc, kt, at);
        copy(vc, kt + X::TILE * (2 - turn), at);
        at = sub + 2 * kWarps < sub1 ? place((sub + 2 * kWarps) * kSub + (lane & 15)) : -1;
        copy_wait<2>();                        // this turn's V
      } else {
        copy_wait<0>();
      }
      __syncwarp();
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
      __syncwarp();                            // V is read before its buffer is filled again
      turn ^= 1;
    }

    // ---- the four warps' parts, in warp order ----
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
    const int slot = (int)blockIdx.x * kFewBlocks + rb;
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
        if (merge) {
          // the prefix's partials, in order
          const PartsOf pre = parts_of(a, 0, h, tok0 + tk);
          for (int k = 0; k < pre.parts; ++k) {
            const float2* ml;
            const float4* at_v;
            partial<DP>(a, pre, 0, h, rg, hd, k, ml, at_v);
            const float2 x = __ldcg(ml);
            float4 v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = __ldcg(at_v + c0 + kCols * i);
            if (x.y == 0.f) continue;
            const float t = fmaxf(top, x.x), f0 = sum == 0.f ? 0.f : ex2(top - t), f1 = ex2(x.x - t);
            top = t;
            sum = fmaf(sum, f0, x.y * f1);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              acc[i].x = fmaf(acc[i].x, f0, v[i].x * f1);
              acc[i].y = fmaf(acc[i].y, f0, v[i].y * f1);
              acc[i].z = fmaf(acc[i].z, f0, v[i].z * f1);
              acc[i].w = fmaf(acc[i].w, f0, v[i].w * f1);
            }
          }
        }
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

template <int DP>
cudaError_t launch_dp(const AttnArgs& a, cudaStream_t s) {
  static PerDeviceOnce once;
  int unused = 0;
  const cudaError_t e = once.run(
      [](int& v) {
        v = 1;
        return cudaFuncSetAttribute(attention_few_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<DP>::SMEM);
      },
      &unused);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)(a.n_groups + a.R) * a.Hkv;
  return launch_k(attention_few_kernel<DP>, dim3((unsigned)std::max<int64_t>(units * a.few_splits, 1)), kThreads,
                  Geo<DP>::SMEM, s, a);
}

}  // namespace

cudaError_t launch_attention_few(const AttnArgs& a, cudaStream_t s) {
  return a.D <= 64 ? launch_dp<64>(a, s) : launch_dp<128>(a, s);
}

}  // namespace moe
