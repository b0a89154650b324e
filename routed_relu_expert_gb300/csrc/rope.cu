// Rotary positions, alone (with their backward, the inverse rotation) and fused
// with the write of K and V into the paged cache.
//
//   angle = 2 pi frac(pos * F_i / 2^64),  F_i = round(f_i / (2 pi) * 2^64)
//   (a, b) -> (a cos - b sin, a sin + b cos) * rot_scale
//
// The product pos * F_i mod 2^64 is the fraction of a turn exactly, in one
// 64-bit integer multiply, however far the position (an FP32 product of a
// position near 2^20 and a frequency near 1 is off by a twentieth of a
// radian); its upper 32 bits, taken as a signed fraction of a turn in
// [-1/2, 1/2), go to FP32 with a relative error of 2^-24.  Rows are turned in
// FP32 and rounded once, on the store.
//
// Bound: every row is read once and written once.  A thread owns one piece of one
// head (16 bytes, or the two 16-byte pieces that rotate into each other) and walks
// a block's tokens with it: where the piece lies is worked out once, and the loads
// of kRopeAhead tokens are in flight before the first is turned.  The angles of a
// block's tokens are computed once for all of its pieces, into shared memory.
#include "attn.h"

#include <algorithm>

namespace moe {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxTokens = 16;             // tokens a block
constexpr int kRopeAhead = 2;                  // tokens whose loads a thread has in flight
constexpr int kRopeMaxPairs = 64;              // head_dim / 2 at most

template <typename T> struct Vec16;
template <> struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const void* p, float (&v)[4]) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  }
  static __device__ __forceinline__ void store(void* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Vec16<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const void* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
  }
  static __device__ __forceinline__ void store(void* p, const float (&v)[8]) {
    uint4 q;
    q.x = (uint32_t)bf16_bits(v[0]) | ((uint32_t)bf16_bits(v[1]) << 16);
    q.y = (uint32_t)bf16_bits(v[2]) | ((uint32_t)bf16_bits(v[3]) << 16);
    q.z = (uint32_t)bf16_bits(v[4]) | ((uint32_t)bf16_bits(v[5]) << 16);
    q.w = (uint32_t)bf16_bits(v[6]) | ((uint32_t)bf16_bits(v[7]) << 16);
    *reinterpret_cast<uint4*>(p) = q;
  }
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float* p) { *p = v; }
__device__ __forceinline__ void from_f(float v, bf16* p) { *p = __float2bfloat16_rn(v); }

// VECTOR: pairs by 16-byte pieces (the pieces of a and of b are whole); else a
// pair of elements at a time.  tb: tokens a block; blockIdx.y: kRopeThreads
// pieces.
template <typename T, bool INTER, bool VECTOR>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int tb) {
  constexpr int N = Vec16<T>::N;
  pdl_wait();
  __shared__ __align__(16) float2 cs[kRopeMaxTokens * kRopeMaxPairs];
  __shared__ int64_t slot_at[kRopeMaxTokens];   // cache offset of the token's head 0, -1: not cached
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * tb, nt = min(tb, a.T - t0);
  const int half = a.rot / 2;
  // this thread's piece: part, head, and which of the head's pieces (the ones that rotate, then the others)
  const int n_turn = VECTOR ? (INTER ? a.rot / N : a.rot / (2 * N)) : half;
  int at = blockIdx.y * kRopeThreads + tid, part = 0, turns = 0, pieces = 0;
  for (; part < a.n_parts; ++part) {
    turns = a.part[part].rotate ? n_turn : 0;
    const int rot = a.part[part].rotate ? a.rot : 0;
    pieces = turns + (VECTOR ? (a.D - rot) / N : a.D - rot);
    const int all = pieces * a.part[part].heads;
    if (at < all) break;
    at -= all;
  }
  const bool have = part < a.n_parts;
  const int h = have ? at / pieces : 0, k = have ? at - h * pieces : 0;
  const RopeRows r = a.part[have ? part : 0];
  const bool turn = k < turns;
  // first and, where a piece rotates into another, second element
  const int rest = (r.rotate ? a.rot : 0) + (VECTOR ? (k - turns) * N : k - turns);
  const int e0 = !turn ? rest : VECTOR ? k * N : INTER ? 2 * k : k;
  const int e1 = !turn ? e0 : VECTOR ? (INTER ? e0 : half + k * N) : INTER ? 2 * k + 1 : k + half;
  const bool two = e1 != e0;
  const T* src = reinterpret_cast<const T*>(r.src) + (int64_t)t0 * r.src_ld + (int64_t)h * a.D;
  T* dst = reinterpret_cast<T*>(r.dst) + (r.to_cache ? (int64_t)h * a.head_stride
                                                     : (int64_t)t0 * r.dst_ld + (int64_t)h * a.D);

  uint4 x[kRopeAhead], y[kRopeAhead];
  auto fetch = [&](int t, int i) {
    if (!have || t >= nt) return;
    const T* s = src + t * r.src_ld;
    if (VECTOR) {
      x[i] = __ldcs(reinterpret_cast<const uint4*>(s + e0));
      if (!INTER && two) y[i] = __ldcs(reinterpret_cast<const uint4*>(s + e1));
    } else {
      x[i].x = __float_as_uint(to_f(s[e0]));
      if (two) y[i].x = __float_as_uint(to_f(s[e1]));
    }
  };
#pragma unroll
  for (int i = 0; i < kRopeAhead; ++i) fetch(i, i);

  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int t = i / half, p = i - t * half;
    const uint64_t turned = (uint64_t)(int64_t)a.positions[t0 + t] * a.table[p];
    // upper 32 bits, rounded to nearest, as a signed fraction of a half turn
    const int32_t frac = (int32_t)(uint32_t)((turned + 0x80000000ull) >> 32);
    float s, c;
    sincospif((float)frac * 4.656612873077393e-10f, &s, &c);   // 2^-31
    cs[i] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
  }
  if (a.slot_map && tid < nt) {
    const int64_t slot = a.slot_map[t0 + tid];
    int64_t off = -1;
    if (slot >= 0 && slot < a.n_slots)
      off = (slot >> a.page_shift) * a.page_stride + (slot & ((1ll << a.page_shift) - 1)) * a.token_stride;
    else if (slot != -1)
      set_error(&a.hdr->err, MOE_DEVERR_CACHE);
    slot_at[tid] = off;
  }
  __syncthreads();
  if (!have) return;

  for (int tt = 0; tt < nt; tt += kRopeAhead) {
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) {
      const int t = tt + i;
      if (t >= nt) break;
      const uint4 u = x[i], v = y[i];
      fetch(t + kRopeAhead, i);
      T* d = dst;
      if (r.to_cache) {
        if (slot_at[t] < 0) continue;
        d += slot_at[t];
      } else {
        d += t * r.dst_ld;
      }
      if (VECTOR && !turn) {
        *reinterpret_cast<uint4*>(d + e0) = u;
      } else if (VECTOR && INTER) {
        float f[N];
        Vec16<T>::load(&u, f);
#pragma unroll
        for (int p = 0; p < N / 2; ++p) {
          const float2 w = cs[t * half + k * (N / 2) + p];
          const float fa = f[2 * p], fb = f[2 * p + 1];
          f[2 * p] = fa * w.x - fb * w.y;
          f[2 * p + 1] = fa * w.y + fb * w.x;
        }
        Vec16<T>::store(d + e0, f);
      } else if (VECTOR) {
        float f[N], g[N];
        Vec16<T>::load(&u, f);
        Vec16<T>::load(&v, g);
#pragma unroll
        for (int p = 0; p < N; ++p) {
          const float2 w = cs[t * half + k * N + p];
          const float fa = f[p], fb = g[p];
          f[p] = fa * w.x - fb * w.y;
          g[p] = fa * w.y + fb * w.x;
        }
        Vec16<T>::store(d + e0, f);
        Vec16<T>::store(d + e1, g);
      } else {
        const float fa = __uint_as_float(u.x), fb = __uint_as_float(v.x);
        if (turn) {
          const float2 w = cs[t * half + k];
          from_f(fa * w.x - fb * w.y, d + e0);
          from_f(fa * w.y + fb * w.x, d + e1);
        } else {
          from_f(fa, d + e0);
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, int interleaved, cudaStream_t s) {
  constexpr int N = Vec16<T>::N;
  const bool vec = a.rot % (interleaved ? N : 2 * N) == 0;
  int64_t pieces = 0;
  for (int i = 0; i < a.n_parts; ++i) {
    const int rot = a.part[i].rotate ? a.rot : 0;
    pieces += (int64_t)a.part[i].heads * (vec ? (interleaved ? rot / N : rot / (2 * N)) + (a.D - rot) / N : a.D - rot / 2);
  }
  const int64_t chunks = ceil_div(pieces, kRopeThreads);
  if (chunks > 65535) return cudaErrorInvalidValue;
  // tokens a block: what leaves about two waves of eight blocks an SM.  BF16, 16384 tokens, 48 heads of 128, half of
  // the head turned: 16 tokens 76 us, 8 78, 4 85, 2 102; loads 1, 2 and 4 tokens ahead 80, 76 and 88 us
  const int64_t waves = 2 * 8 * 152;
  const int tb = (int)std::min<int64_t>(std::max<int64_t>((int64_t)a.T * chunks / waves, 1), kRopeMaxTokens);
  const dim3 grid((unsigned)ceil_div(a.T, tb), (unsigned)chunks);
  if (interleaved) {
    if (vec) launch_k(rope_kernel<T, true, true>, grid, kRopeThreads, 0, s, a, tb);
    else launch_k(rope_kernel<T, true, false>, grid, kRopeThreads, 0, s, a, tb);
  } else {
    if (vec) launch_k(rope_kernel<T, false, true>, grid, kRopeThreads, 0, s, a, tb);
    else launch_k(rope_kernel<T, false, false>, grid, kRopeThreads, 0, s, a, tb);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, int interleaved, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  return dtype == MOE_DT_F32 ? launch_t<float>(a, interleaved, s) : launch_t<bf16>(a, interleaved, s);
}

}  // namespace moe
