// What the attention kernels on the tensor cores share: PTX, descriptors, waits.
#pragma once

#include "attn.h"
#include "tc_common.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int kHalfBytes = kAttnTile * 128;    // 128 rows of 64 BF16
constexpr float kRaise = 8.f;                  // log2 units by which a maximum may pass its reference
constexpr int kMaxSmem = 232448;

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[tmem] B[shared]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// one thread of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// 32 columns of this thread's lane, without waiting for them
template <int O, int N>
__device__ __forceinline__ void ld32_async(uint32_t taddr, float (&v)[N]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[O + 0]), "=f"(v[O + 1]), "=f"(v[O + 2]), "=f"(v[O + 3]), "=f"(v[O + 4]), "=f"(v[O + 5]),
        "=f"(v[O + 6]), "=f"(v[O + 7]), "=f"(v[O + 8]), "=f"(v[O + 9]), "=f"(v[O + 10]), "=f"(v[O + 11]),
        "=f"(v[O + 12]), "=f"(v[O + 13]), "=f"(v[O + 14]), "=f"(v[O + 15]), "=f"(v[O + 16]), "=f"(v[O + 17]),
        "=f"(v[O + 18]), "=f"(v[O + 19]), "=f"(v[O + 20]), "=f"(v[O + 21]), "=f"(v[O + 22]), "=f"(v[O + 23]),
        "=f"(v[O + 24]), "=f"(v[O + 25]), "=f"(v[O + 26]), "=f"(v[O + 27]), "=f"(v[O + 28]), "=f"(v[O + 29]),
        "=f"(v[O + 30]), "=f"(v[O + 31])
      : "r"(taddr));
}
// waits for this thread's loads; the values pass through it, so that no use of
// them can move above the wait
template <int O, int N>
__device__ __forceinline__ void ld32_wait(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[O + 0]), "+f"(v[O + 1]), "+f"(v[O + 2]), "+f"(v[O + 3]), "+f"(v[O + 4]), "+f"(v[O + 5]),
                 "+f"(v[O + 6]), "+f"(v[O + 7]), "+f"(v[O + 8]), "+f"(v[O + 9]), "+f"(v[O + 10]), "+f"(v[O + 11]),
                 "+f"(v[O + 12]), "+f"(v[O + 13]), "+f"(v[O + 14]), "+f"(v[O + 15]), "+f"(v[O + 16]), "+f"(v[O + 17]),
                 "+f"(v[O + 18]), "+f"(v[O + 19]), "+f"(v[O + 20]), "+f"(v[O + 21]), "+f"(v[O + 22]), "+f"(v[O + 23]),
                 "+f"(v[O + 24]), "+f"(v[O + 25]), "+f"(v[O + 26]), "+f"(v[O + 27]), "+f"(v[O + 28]), "+f"(v[O + 29]),
                 "+f"(v[O + 30]), "+f"(v[O + 31])
               :
               : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
      "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two FP32 values in one instruction (each rounded as by itself), and the larger
// of three: the softmax groups are bound by the instructions that they issue
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The warp's wait for a phase: a few tries that do not suspend the warp (the
// hot waits end within them, and a suspended warp's wake-up is dearer than they
// are), then the bounded wait of the other tensor-core kernels.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool wait_slow(uint32_t b, uint32_t parity, volatile int* abort_flag, int32_t* err) {
  return __all_sync(0xffffffffu, mbar_wait<false, true>(b, parity, abort_flag, err));
}
template <int TRIES = 32>
__device__ __forceinline__ bool wait_warp(uint32_t b, uint32_t parity, volatile int* abort_flag, int32_t* err) {
#pragma unroll 1
  for (int i = 0; i < TRIES; ++i)
    if (__all_sync(0xffffffffu, mbar_test(b, parity))) return true;
  return wait_slow(b, parity, abort_flag, err);
}

// shared-memory descriptor of V as the MN-major B operand: 64 values of a key
// contiguous (one 128-byte swizzle row), 8-key groups 1024 B apart (stride), the
// next 64 values of the head a half further (leading)
__device__ __forceinline__ uint64_t v_desc(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kHalfBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// lane l of four holds x[0..3]; after it, x[i] is what lane i of the four had in x[l]
__device__ __forceinline__ void transpose4(uint4 (&x)[4], int lane) {
  auto swap = [&](uint4& mine, int by) {
    mine.x = __shfl_xor_sync(0xffffffffu, mine.x, by);
    mine.y = __shfl_xor_sync(0xffffffffu, mine.y, by);
    mine.z = __shfl_xor_sync(0xffffffffu, mine.z, by);
    mine.w = __shfl_xor_sync(0xffffffffu, mine.w, by);
  };
  // two by two blocks, then the pairs inside them
#pragma unroll
  for (int by = 2; by > 0; by >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & by) continue;
      uint4 send = lane & by ? x[i] : x[i | by];
      swap(send, by);
      if (lane & by) x[i] = send; else x[i | by] = send;
    }
}

// ---------------------------------------------------------------------------
// nodes whose V is not finite (out of the hot path's registers)
// ---------------------------------------------------------------------------
// O += p V, columns c0 .. c0 + 63 of the head, for the rows that see them (p, read
// back from tensor memory, is 0 where a row does not)
__device__ __noinline__ void add_odd(const AttnArgs& a, const int32_t* table, int h, int key0, uint4 odd, int c0,
                                     uint32_t p_addr, uint32_t o_addr) {
  for (int i = 0; i < kAttnTile; ++i) {
    const uint32_t word = i < 64 ? (i < 32 ? odd.x : odd.y) : (i < 96 ? odd.z : odd.w);
    if (!(word >> (i & 31) & 1u)) continue;
    const int key = key0 + i;
    const int pg = table[key >> a.page_shift];
    if (pg < 0 || pg >= a.n_pages) continue;
    const bf16* vp = reinterpret_cast<const bf16*>(a.v) + (int64_t)pg * a.page_stride +
                     (int64_t)(key & ((1 << a.page_shift) - 1)) * a.token_stride + (int64_t)h * a.head_stride;
    uint32_t x;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(p_addr + (uint32_t)(i >> 1)));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(x) : : "memory");
    const float pi = i & 1 ? bf16_hi(x) : bf16_lo(x);
    for (int c = c0; c < c0 + 64; ++c) {
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(o_addr + (uint32_t)c));
      asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(x) : : "memory");
      if (pi != 0.f && c < a.D) x = __float_as_uint(fmaf(pi, __bfloat162float(vp[c]), __uint_as_float(x)));
      asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(o_addr + (uint32_t)c), "r"(x) : "memory");
      st_wait();
    }
  }
}

// ---------------------------------------------------------------------------
// tensor maps (host)
// ---------------------------------------------------------------------------
// BF16 tensor of up to four dims (the first contiguous), 128-byte swizzled boxes 64 wide
bool make_map(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box) {
  EncodeTiledFn fn = encode_fn();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace moe
