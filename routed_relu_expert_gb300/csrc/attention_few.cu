// Attention with shared prefixes where a request (or a group) has few rows: up to 32 of
// a KV head, or any number where all of them together have few keys.  BF16 rows and
// caches, FP32 scores, softmax and sums.
//
//   S = Q K^T,  p = exp2(c S - m),  l = sum p,  O = sum p V,  out = O / l
//
// The tiles of the tensor-memory kernel have 128 rows, and a piece of a run costs it 3 to
// 4 us beside its tiles: a request with a few rows and a few hundred tokens of
// its own behind the prefix is mostly that cost.  Here a unit is (request or group, KV
// head, 16 rows), its keys are taken 16 at a time, and the 16-key steps of all units, in
// order, are cut into equal runs, one a warp: every warp has the same work whatever the
// lengths, and waits for no other.  Its K and V come by cp.async into its own two stages;
// products by mma.sync.  Units that a run's end cuts, and rows that have a prefix, leave
// FP32 partials for the join.  The arithmetic is the other kernel's: probabilities in
// BF16 for the second product, sums before that rounding, the reference follows the
// maximum only past 2^8.
//
// The other kernel lets this one's blocks start as its own ones end (they need nothing of it).
//
// Bound: HBM, where there are enough keys; else the latency of a run (lengths, table, keys,
// softmax, the join).  128 requests' 131 MB of own tokens: 38 us beside the other kernel's end,
// about 20 of them the loop (6.5 TB/s), the rest start and partials; two samples behind 500 tokens
// (no other kernel): 10 us, and the join.
#include "attn_walk.cuh"
#include "tc_common.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSub = 16;                       // keys a step
constexpr int kUnitCost = 2;                   // a unit's fixed cost beside its steps, in steps
// steps of a run at least (2 / 3 / 4 / 6, us: two samples behind 500 tokens 12.5 / 12.2 / 13.8 / 14.6, behind 2000 18.8 /
// 16.3 / 17.1 / 16.8); runs of a unit at most (about)
constexpr int kMinRun = 3, kMaxParts = 64;
// blocks an SM (2 / 3: 16 requests behind 500 tokens 14.4 / 15.2, 128 behind 8000 89.4 / 89.5 and with twice the nodes
// 129 / 127); with three stages a warp 14.8 and 91.8
constexpr int kBlocks = 2;
// This kernel takes all rows where every 16 of them together read at most so many bytes of keys and values, by the
// tables' width.  Both ways, graph replay, us: 16 requests behind 500 common tokens 21.9 for 30.1, 64 of them (136 MB)
// 34 for 41, 17 in three groups behind 1500 to 3001 (80 MB) 25.7 for 28.8, 12 behind 2000 (72 MB) 26 for 30; 32 (172
// MB) 35 for 35, 64 (344 MB) 57 for 44, 8 behind 8000 (174 MB) 43 for 33.
constexpr int64_t kFewBytes = 96ll << 20;
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
// 16 bytes, zeros where `bytes` is 0; policy: how long L2 keeps them
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
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
  static constexpr int RING = 4 * TILE;                      // of a warp: two stages of K and V
  static constexpr int SMEM = kWarps * RING;                 // and the walk's words
};

template <int DP>
__global__ void __launch_bounds__(kThreads, kBlocks) attention_few_kernel(const AttnArgs a, int shift) {
  using X = Geo<DP>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int s_most, s_mixed;
  const int walk_n = a.n_groups + a.R;
  int* prefix = reinterpret_cast<int*>(smem + X::SMEM);      // [walk_n + 1] cost before each step of the walk
  int* skip = prefix + walk_n + 1;                           // [R] pages of the request's group's prefix
  if (a.few_alone) pdl_wait();                 // (else the other kernel has waited, and let this one start)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tb = kFewRows / a.G;               // tokens of a unit
  const int grain = kSub << shift;             // keys that count as one step of the cost

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

  // the walk, as the other kernel has it: cost before each step, runs of the total
  auto at_walk = [&](int v, int* bad) {
    Req q = v < a.n_groups ? group_request(a, v, s_mixed, tb, bad)
                           : own_request(a, v - a.n_groups, skip[v - a.n_groups], tb, bad);
    q.tiles = max((q.kv + grain - 1) / grain, 1);
    if (!few(a, q)) q.blocks = 0;
    return q;
  };
  int total, runs, share, extra;
  auto run_start = [&](int c) { return c * share + min(c, extra); };
  {
    int bad = 0;
    if (tid == 0) s_most = 0;
    prefix_pages<kThreads>(a, reinterpret_cast<int32_t*>(smem), skip, &s_mixed);
    const int per = (walk_n + kThreads - 1) / kThreads, v0 = min(tid * per, walk_n), v1 = min(v0 + per, walk_n);
    auto cost = [&](const Req& q) { return (q.tiles + kUnitCost) * q.blocks * a.Hkv; };
    Req q;
    int64_t local = 0;
    int most = 0;
    for (int v = v0; v < v1; ++v) {
      q = at_walk(v, &bad);
      local += cost(q);
      if (q.blocks) most = max(most, q.tiles);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0 && most) atomicMax(&s_most, most);
    int64_t all;
    const int64_t before = block_prefix<kThreads>(local, s_scan, &all);
    if (all > INT32_MAX) {                                 // (row starts that are no prefix sums)
      bad = 1;
      all = 0;
    }
    total = (int)all;
    int at = (int)before;
    for (int v = v0; v < v1; ++v) {
      if (per > 1) q = at_walk(v, nullptr);
      prefix[v] = at;
      at += cost(q);
    }
    if (tid == 0) prefix[walk_n] = total;
    if (bad && blockIdx.x == 0) set_error(&a.hdr->err, MOE_DEVERR_CACHE);
    __syncthreads();
    const int least = max(kMinRun, (s_most + kMaxParts - 1) / kMaxParts);
    runs = min((int)gridDim.x * kWarps, max(total / least, 1));
    share = total / runs;
    extra = total - share * runs;
  }
  // runs go round the blocks first, so that few of them have an SM each
  const int run = blockIdx.x + gridDim.x * warp;
  if (run >= runs || total == 0) {
    if (!a.few_alone && blockIdx.x == 0 && warp == kWarps - 1) pdl_wait();     // this kernel does not end before the other
    return;
  }
  auto owner = [&](int at) {                               // the run that holds position `at`
    const int longer = (share + 1) * extra;                // positions in the longer runs
    return at < longer ? at / (share + 1) : extra + (at - longer) / share;
  };
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * X::RING;
  const float c = a.scale * 1.4426950408889634f;
  const int g = lane >> 2, t4 = lane & 3;      // the row (and + 8) and the pair of columns that a lane has of a product
  const int64_t rows_all = (int64_t)a.T * a.G;

  const int end = run_start(run + 1);
  int v = 0;
  {
    int hi = walk_n;                           // the last step that begins at or before the run
    while (hi - v > 1) {
      const int mid = (v + hi) >> 1;
      if (prefix[mid] <= run_start(run)) v = mid; else hi = mid;
    }
  }
  for (int pos = run_start(run); pos < end;) {
    while (prefix[v + 1] <= pos) ++v;
    const Req q = at_walk(v, nullptr);
    const int per = q.tiles + kUnitCost, u = (pos - prefix[v]) / per, off = pos - prefix[v] - u * per;
    const int len = min(per - off, end - pos), t0 = max(off - kUnitCost, 0), t1 = off + len - kUnitCost;
    const int unit_end = pos - off + per;
    pos += len;
    if (t1 <= t0) continue;                    // the fixed cost alone
    const int h = u / q.blocks, rb = u - h * q.blocks;
    const bool starts = t0 == 0, ends = t1 == q.tiles;
    const int sub0 = t0 << shift, sub1 = min(t1 << shift, max((q.kv + kSub - 1) / kSub, 1));
    const int32_t* table = a.block_table + (int64_t)q.row * a.max_pages + q.skip;
    const bf16 *kc = reinterpret_cast<const bf16*>(a.k) + (int64_t)h * a.head_stride,
               *vc = reinterpret_cast<const bf16*>(a.v) + (int64_t)h * a.head_stride;
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
    // a lane's key of 16
    auto keys = [&](int sub) -> int64_t { return sub < sub1 ? place(sub * kSub + (lane & 15)) : -1; };
    // own tokens are read once and leave L2 before the partials (92 -> 89 us for 128 requests of 250 tokens each)
    uint64_t policy;
    if (q.flags & kPrefix) asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    else asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    // 16 keys into a stage; at: a lane's key (both halves of the warp have all 16)
    auto copy = [&](int stage, int64_t at) {
      constexpr int KEYS = 32 / X::CH;         // keys of a step of the warp
      const uint32_t dst = ring + stage * 2 * X::TILE;
      const int ch = lane % X::CH;
#pragma unroll
      for (int s = 0; s < kSub / KEYS; ++s) {
        const int key = s * KEYS + lane / X::CH;
        const int64_t o = __shfl_sync(0xffffffffu, at, key);
        const int bytes = o >= 0 && ch * 8 < a.D ? 16 : 0;
        const int64_t from = bytes ? o + ch * 8 : 0;
        const uint32_t to = dst + key * DP * 2 + ((ch ^ (key & 7)) << 4);
        copy16(to, kc + from, bytes, policy);
        copy16(to + X::TILE, vc + from, bytes, policy);
      }
      copy_commit();
    };
    const int64_t at0 = keys(sub0), at1 = keys(sub0 + 1);
    copy(0, at0);
    copy(1, at1);
    int64_t at = keys(sub0 + 2);
    const int tok0 = q.q0 + rb * tb, ntok = min(tb, q.n - rb * tb), valid = ntok * a.G;
    // Q as the A operand: rows g and g + 8
    uint32_t qf[DP / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = g + 8 * i, tk = row / a.G;
      const bf16* p = reinterpret_cast<const bf16*>(a.q) + (int64_t)(tok0 + tk) * a.q_ld +
                      (int64_t)(h * a.G + row - tk * a.G) * a.D;
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = 16 * k + 8 * j + 2 * t4;
          qf[k][2 * j + i] = row < valid && col < a.D ? *reinterpret_cast<const uint32_t*>(p + col) : 0u;
        }
    }
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float mc[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    int stage = 0;
    for (int sub = sub0; sub < sub1; ++sub) {
      const uint32_t kt = ring + stage * 2 * X::TILE, vt = kt + X::TILE;
      const int k0 = sub * kSub;
      copy_wait<1>();
      __syncwarp();
      // scores of 16 rows and 16 keys
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        // matrices: keys 0-7 and 8-15, two chunks each
        const int key = (lane & 7) + ((lane >> 4) << 3), half = lane >> 3 & 1;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          uint32_t b[4];
          ldsm4(kt + key * DP * 2 + (((2 * k + half) ^ (key & 7)) << 4), b);
          mma_bf16_16816(s[0], qf[k][0], qf[k][1], qf[k][2], qf[k][3], b[0], b[1]);
          mma_bf16_16816(s[1], qf[k][0], qf[k][1], qf[k][2], qf[k][3], b[2], b[3]);
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
          const int64_t off_v = place(k0 + key);
          if (off_v < 0) continue;
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            const int col = 8 * i + 2 * t4;
            if (col >= a.D) continue;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(vc + off_v + col);
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
      copy(stage, at);
      at = keys(sub + 3);
      stage ^= 1;
    }
    copy_wait<0>();                            // (the next piece's keys come into the same stages)

    // ---- the piece's end: the rows, or their partials ----
    const int which = q.flags & kPrefix ? 0 : 1, slot = 2 * run + (starts ? 1 : 0);
    const bool uncut = starts && ends, whole = uncut && !q.flags;
    const int64_t side = which * a.Hkv + h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = g + 8 * i, tk = row / a.G, head = h * a.G + row - tk * a.G;
      float sum = l[i] + __shfl_xor_sync(0xffffffffu, l[i], 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (row >= valid) continue;
      if (whole) {
        // a row without a visible key has sum 0 and O = 0
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        bf16* out = reinterpret_cast<bf16*>(a.out) + (int64_t)(tok0 + tk) * a.out_ld + (int64_t)head * a.D + 2 * t4;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j)
          if (8 * j < a.D) *reinterpret_cast<uint32_t*>(out + 8 * j) = pack_bf16(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
        if (a.lse && t4 == 0)
          a.lse[(int64_t)(tok0 + tk) * a.H + head] = sum == 0.f ? -INFINITY : (mc[i] + log2f(sum)) * 0.6931471805599453f;
      } else {
        const int64_t at_row = uncut ? side * rows_all + (int64_t)tok0 * a.G + row : (int64_t)slot * kFewRows + row;
        float* to = (uncut ? a.rows_part : a.few_part) + at_row * DP + 2 * t4;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j)
          *reinterpret_cast<float2*>(to + 8 * j) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
        if (t4 == 0) (uncut ? a.rows_ml : a.few_ml)[at_row] = make_float2(mc[i], sum);
      }
    }
    if (starts && lane < ntok)
      a.parts_of[side * a.T + tok0 + lane] =
          make_int4(whole ? 0 : uncut ? 1 : owner(unit_end - 1) - run + 1, uncut ? 0 : slot, lane * a.G,
                    (q.flags & kJoined) | (uncut ? 0 : kFewSlots));
  }
  if (!a.few_alone && blockIdx.x == 0 && warp == kWarps - 1) pdl_wait();       // as above
}

template <int DP>
cudaError_t launch_dp(const AttnArgs& a, cudaStream_t s) {
  using X = Geo<DP>;
  static PerDeviceOnce once;
  int blocks = 0;
  const cudaError_t e = once.run(
      [](int& v) {
        v = std::min(kBlocks * tc::num_sms(), kFewRuns / kWarps);
        return cudaFuncSetAttribute(attention_few_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    X::SMEM + (3 * kPrefixMaxRequests + 1) * 4);
      },
      &blocks);
  if (e != cudaSuccess) return e;
  // keys that count as one step of the cost: 16, or as many more as keep the cost of all units in 31 bits
  const int64_t units = 2ll * (a.n_groups + a.R + ceil_div(a.T, kFewRows / a.G)) * a.Hkv, keys = (int64_t)a.max_pages << a.page_shift;
  int shift = 0;
  while (units * (((keys + (kSub << shift) - 1) >> shift) / kSub + 1 + kUnitCost) >= ((int64_t)1 << 31)) ++shift;
  // no more blocks than the longest tables' rows have runs for
  const int64_t most = units * (keys / kSub + 1 + kUnitCost) / kMinRun + 1;
  return launch_k(attention_few_kernel<DP>, dim3((unsigned)std::min<int64_t>(blocks, most)), dim3(kThreads),
                  X::SMEM + ((size_t)a.n_groups + 2 * a.R + 1) * 4, s, a, shift);
}

}  // namespace

void few_shape(AttnArgs* a) {
  if (a->G > kFewRows) return;                 // (a token's rows do not fit a unit's 16)
  const int tb = kFewRows / a->G;
  a->few_tokens = kFewBlocks * tb;
  // all of them where reading a prefix once for every 16 rows is less than a second kernel costs
  const int64_t keys = (int64_t)ceil_div(a->T, tb) * a->Hkv * ((int64_t)a->max_pages << a->page_shift);
  if (keys <= kFewBytes / (a->D <= 64 ? 256 : 512)) a->few_tokens = std::max(a->few_tokens, a->T);
  a->few_alone = a->T <= a->few_tokens;
}

cudaError_t launch_attention_few(const AttnArgs& a, cudaStream_t s) {
  return a.D <= 64 ? launch_dp<64>(a, s) : launch_dp<128>(a, s);
}

}  // namespace moe
