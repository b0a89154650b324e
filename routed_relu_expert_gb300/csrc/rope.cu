// Rotary positions, alone (with their backward, the inverse rotation) and fused
// with the write of K and V into the paged cache.
//
//   angle = 2 pi frac(pos * F_i / 2^64),  F_i = round(f_i / (2 pi) * 2^64)
//   (a, b) -> (a cos - b sin, a sin + b cos) * rot_scale
//
// The product pos * F_i mod 2^64 is the fraction of a turn in one 64-bit integer
// multiply that rounds nothing, however far the position (an FP32 product of a
// position near 2^20 and a frequency near 1 is off by a twentieth of a radian).  What
// the angle is off by: the table's entry, made in FP64, 2^-51 of pos * f / (2 pi) turns
// at most; the cut to the upper 32 bits, a signed fraction of a turn in [-1/2, 1/2),
// 2^-33 turns; their FP32 value, 2^-24 of it.  The cut is absolute: a sine of 1e-7 keeps
// two digits, an error of 1e-9 beside the cosine's of 6e-8.  Rows are turned in FP32 and
// rounded once, on the store.
//
// Bound: every row is read once and written once.  A thread owns one 16-byte piece
// of one head and walks a block's tokens with it: where the piece lies is worked
// out once, and the loads of kRopeAhead tokens are in flight before the first is
// turned.  In the half layout the piece that a piece rotates with belongs to
// another lane of the warp (a warp holds whole heads) and comes by shuffle, so
// that every load and store is of whole lines.  The angles of a block's tokens are
// computed once for all of its pieces, into shared memory.  16384 BF16 tokens of
// 32 + 2 x 8 heads of 128 (403 MB): 73 us with half of the head turned = 5.5 TB/s, 76
// with all of it, 66 with none (a plain cache write), 69 interleaved, 122 where 22 of
// 128 turn: a rotating part that is no whole number of pieces (of pairs of pieces in the
// half layout) goes by single elements, 2-byte loads and stores.
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

// threads of a head whose rotating part does not end on a piece: pairs, single elements, whole pieces
__host__ __device__ __forceinline__ int pieces_of(int D, int rot, int n) {
  const int edge = (rot + n - 1) / n * n;
  return rot / 2 + (edge - rot) + (D - edge) / n;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float* p) { *p = v; }
__device__ __forceinline__ void from_f(float v, bf16* p) { *p = __float2bfloat16_rn(v); }

// VECTOR: 16-byte pieces (the pieces that rotate are whole); else a thread has a
// pair of elements, or one of the elements between the last pair and the next
// 16-byte boundary, or a whole piece behind that.  tb: tokens a block; blockIdx.y: kRopeThreads pieces.
template <typename T, bool INTER, bool VECTOR>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int tb) {
  constexpr int N = Vec16<T>::N;
  constexpr bool SHUFFLE = VECTOR && !INTER;
  pdl_wait();
  __shared__ __align__(16) float2 cs[kRopeMaxTokens * kRopeMaxPairs];
  __shared__ int64_t slot_at[kRopeMaxTokens];   // cache offset of the token's head 0, -1: not cached
  const int tid = threadIdx.x, lane = tid & 31;
  const int t0 = blockIdx.x * tb, nt = min(tb, a.T - t0);
  const int half = a.rot / 2;
  // this thread's piece k of head h of a part (first the pieces that rotate)
  int part = 0, h = 0, k = 0;
  if (SHUFFLE) {
    const int per = a.D / N, heads = 32 / per;             // a warp: whole heads
    const int i = lane / per;
    k = lane - i * per;
    h = (blockIdx.y * (kRopeThreads / 32) + (tid >> 5)) * heads + i;
    if (i >= heads) h = INT32_MAX;
    for (; part < a.n_parts && h >= a.part[part].heads; ++part) h -= a.part[part].heads;
  } else {
    int at = blockIdx.y * kRopeThreads + tid;
    for (; part < a.n_parts; ++part) {
      const int rot = a.part[part].rotate ? a.rot : 0;
      const int per = VECTOR ? a.D / N : pieces_of(a.D, rot, N), all = per * a.part[part].heads;
      if (at < all) {
        h = at / per;
        k = at - h * per;
        break;
      }
      at -= all;
    }
  }
  const bool have = part < a.n_parts;
  const RopeRows r = a.part[have ? part : 0];
  const int rot = r.rotate ? a.rot : 0;
  const bool turn = VECTOR ? k * N < rot : k < rot / 2;
  const int edge = (rot + N - 1) / N * N;                  // first whole piece that does not rotate
  const bool whole = VECTOR || k >= edge - rot / 2;
  // the piece's first element; without VECTOR a pair's two
  const int e0 = VECTOR  ? k * N
                 : turn  ? (INTER ? 2 * k : k)
                 : whole ? edge + (k - (edge - rot / 2)) * N
                         : rot / 2 + k;
  const int e1 = VECTOR || !turn ? e0 : INTER ? 2 * k + 1 : k + half;
  // SHUFFLE: the lane of the other piece, which piece of the angles, and the sign of the sine
  const int n_half = half / N;
  const bool first = k < n_half;
  const int other = lane + (first ? n_half : -n_half), piece = first ? k : k - n_half;
  const float sign = first ? -1.f : 1.f;
  const T* src = reinterpret_cast<const T*>(r.src) + (int64_t)t0 * r.src_ld + (int64_t)(have ? h : 0) * a.D;
  T* dst = reinterpret_cast<T*>(r.dst) + (r.to_cache ? (int64_t)(have ? h : 0) * a.head_stride
                                                     : (int64_t)t0 * r.dst_ld + (int64_t)(have ? h : 0) * a.D);

  uint4 x[kRopeAhead];
  auto fetch = [&](int t, int i) {
    if (!have || t >= nt) return;
    const T* s = src + t * r.src_ld;
    if (whole) {
      x[i] = __ldcs(reinterpret_cast<const uint4*>(s + e0));
    } else {
      x[i].x = __float_as_uint(to_f(s[e0]));
      x[i].y = __float_as_uint(to_f(s[e1]));
    }
  };
#pragma unroll
  for (int i = 0; i < kRopeAhead; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    fetch(i, i);
  }

  // a token's angles lie so that the lanes of a warp, a piece each, read neighbours: [pair of the piece][piece]
  constexpr int M = !VECTOR ? 1 : INTER ? N / 2 : N;         // pairs (or halves of pairs) a piece
  const int n_piece = half / M;
  auto place = [&](int p) { return p % M * n_piece + p / M; };
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int t = i / half, p = i - t * half;
    const uint64_t turned = (uint64_t)(int64_t)a.positions[t0 + t] * a.table[p];
    // upper 32 bits, rounded to nearest, as a signed fraction of a half turn
    const int32_t frac = (int32_t)(uint32_t)((turned + 0x80000000ull) >> 32);
    float s, c;
    sincospif((float)frac * 4.656612873077393e-10f, &s, &c);   // 2^-31
    cs[t * half + place(p)] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
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

  for (int tt = 0; tt < nt; tt += kRopeAhead) {
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) {
      const int t = tt + i;
      if (t >= nt) break;
      const uint4 u = x[i];
      fetch(t + kRopeAhead, i);
      uint4 v;
      if (SHUFFLE) {
        v.x = __shfl_sync(0xffffffffu, u.x, other & 31);
        v.y = __shfl_sync(0xffffffffu, u.y, other & 31);
        v.z = __shfl_sync(0xffffffffu, u.z, other & 31);
        v.w = __shfl_sync(0xffffffffu, u.w, other & 31);
      }
      if (!have) continue;
      T* d = dst;
      if (r.to_cache) {
        if (slot_at[t] < 0) continue;
        d += slot_at[t];
      } else {
        d += t * r.dst_ld;
      }
      if (whole && !turn) {
        *reinterpret_cast<uint4*>(d + e0) = u;
      } else if (VECTOR && INTER) {
        float f[N];
        Vec16<T>::load(&u, f);
#pragma unroll
        for (int p = 0; p < N / 2; ++p) {
          const float2 w = cs[t * half + p * n_piece + k];
          const float fa = f[2 * p], fb = f[2 * p + 1];
          f[2 * p] = fa * w.x - fb * w.y;
          f[2 * p + 1] = fa * w.y + fb * w.x;
        }
        Vec16<T>::store(d + e0, f);
      } else if (VECTOR) {
        // a cos - b sin, or b cos + a sin
        float f[N], g[N];
        Vec16<T>::load(&u, f);
        Vec16<T>::load(&v, g);
#pragma unroll
        for (int p = 0; p < N; ++p) {
          const float2 w = cs[t * half + p * n_piece + piece];
          f[p] = f[p] * w.x + sign * (g[p] * w.y);
        }
        Vec16<T>::store(d + e0, f);
      } else {
        const float fa = __uint_as_float(u.x), fb = __uint_as_float(u.y);
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
  int64_t threads = 0;
  for (int i = 0; i < a.n_parts; ++i)
    threads += (int64_t)a.part[i].heads * (vec ? a.D / N : pieces_of(a.D, a.part[i].rotate ? a.rot : 0, N));
  if (vec && !interleaved) threads = ceil_div(threads / (a.D / N), 32 / (a.D / N)) * 32;   // whole heads a warp
  const int64_t chunks = ceil_div(threads, kRopeThreads);
  if (chunks > 65535) return cudaErrorInvalidValue;
  // tokens a block: what leaves about eight blocks an SM.  BF16, 16384 tokens, 48 heads of 128, half of
  // the head turned: 16 tokens 76 us, 8 78, 4 85, 2 102; loads 1, 2 and 4 tokens ahead 80, 76 and 88 us
  const int64_t blocks = 8 * 152;
  const int tb = (int)std::min<int64_t>(std::max<int64_t>((int64_t)a.T * chunks / blocks, 1), kRopeMaxTokens);
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
