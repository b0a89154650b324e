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
// Bound: every row is read once and written once.  The angles of a token are
// computed once for all of its heads, into shared memory.
#include "attn.h"

#include <algorithm>

namespace moe {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 8;              // tokens a block
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
// pair of elements at a time.  tb: tokens a block.
template <typename T, bool INTER, bool VECTOR>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int tb) {
  pdl_wait();
  __shared__ float2 cs[kRopeMaxTokens * kRopeMaxPairs];
  __shared__ int64_t slot_at[kRopeMaxTokens];   // cache offset of the token's head 0, -1: not cached
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * tb, nt = min(tb, a.T - t0);
  const int half = a.rot / 2;
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int t = i / half, p = i - t * half;
    const uint64_t turns = (uint64_t)(int64_t)a.positions[t0 + t] * a.table[p];
    // upper 32 bits, rounded to nearest, as a signed fraction of a half turn
    const int32_t frac = (int32_t)(uint32_t)((turns + 0x80000000ull) >> 32);
    float s, c;
    sincospif((float)frac * 4.656612873077393e-10f, &s, &c);   // 2^-31
    cs[i] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
  }
  if (a.slot_map && tid < nt) {
    const int64_t slot = a.slot_map[t0 + tid];
    int64_t at = -1;
    if (slot >= 0 && slot < a.n_slots)
      at = (slot >> a.page_shift) * a.page_stride + (slot & ((1ll << a.page_shift) - 1)) * a.token_stride;
    else if (slot != -1)
      set_error(&a.hdr->err, MOE_DEVERR_CACHE);
    slot_at[tid] = at;
  }
  __syncthreads();

  constexpr int N = Vec16<T>::N;
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    if (part >= a.n_parts) break;
    const RopeRows& r = a.part[part];
    const int rot = r.rotate ? a.rot : 0;
    // items of a head: pieces that rotate, then pieces that are copied
    const int turn_items = VECTOR ? (INTER ? rot / N : rot / (2 * N)) : rot / 2;
    const int items = turn_items + (VECTOR ? (a.D - rot) / N : a.D - rot);
    const int per_token = items * r.heads;
    for (int i = tid; i < nt * per_token; i += kRopeThreads) {
      const int t = i / per_token, j = i - t * per_token;
      const int h = j / items, k = j - h * items;
      const T* src = reinterpret_cast<const T*>(r.src) + (int64_t)(t0 + t) * r.src_ld + h * a.D;
      T* dst;
      if (r.to_cache) {
        if (slot_at[t] < 0) continue;
        dst = reinterpret_cast<T*>(r.dst) + slot_at[t] + (int64_t)h * a.head_stride;
      } else {
        dst = reinterpret_cast<T*>(r.dst) + (int64_t)(t0 + t) * r.dst_ld + h * a.D;
      }
      const float2* c = cs + t * half;
      if (VECTOR) {
        if (k >= turn_items) {
          const int e = rot + (k - turn_items) * N;
          *reinterpret_cast<uint4*>(dst + e) = *reinterpret_cast<const uint4*>(src + e);
        } else if (INTER) {
          float v[N];
          Vec16<T>::load(src + k * N, v);
#pragma unroll
          for (int p = 0; p < N / 2; ++p) {
            const float2 w = c[k * (N / 2) + p];
            const float x = v[2 * p], y = v[2 * p + 1];
            v[2 * p] = x * w.x - y * w.y;
            v[2 * p + 1] = x * w.y + y * w.x;
          }
          Vec16<T>::store(dst + k * N, v);
        } else {
          float x[N], y[N];
          Vec16<T>::load(src + k * N, x);
          Vec16<T>::load(src + half + k * N, y);
#pragma unroll
          for (int p = 0; p < N; ++p) {
            const float2 w = c[k * N + p];
            const float u = x[p], v = y[p];
            x[p] = u * w.x - v * w.y;
            y[p] = u * w.y + v * w.x;
          }
          Vec16<T>::store(dst + k * N, x);
          Vec16<T>::store(dst + half + k * N, y);
        }
      } else if (k >= turn_items) {
        dst[rot + k - turn_items] = src[rot + k - turn_items];
      } else {
        const int ea = INTER ? 2 * k : k, eb = INTER ? 2 * k + 1 : k + half;
        const float2 w = c[k];
        const float x = to_f(src[ea]), y = to_f(src[eb]);
        from_f(x * w.x - y * w.y, dst + ea);
        from_f(x * w.y + y * w.x, dst + eb);
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, int interleaved, cudaStream_t s) {
  constexpr int N = Vec16<T>::N;
  const bool vec = a.rot % (interleaved ? N : 2 * N) == 0;
  // one token a block while that leaves SMs idle, else more, so that a block's
  // threads have at least one item each
  int64_t heads = 0;
  for (int i = 0; i < a.n_parts; ++i) heads += a.part[i].heads;
  const int64_t pieces = std::max<int64_t>(heads * a.D / (vec ? N : 1), 1);
  const int tb = (int)std::min<int64_t>(std::max<int64_t>(kRopeThreads / pieces, 1), kRopeMaxTokens);
  const unsigned grid = (unsigned)ceil_div(a.T, tb);
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
