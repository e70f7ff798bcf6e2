// Pieces of the two attention kernels over the 4-bit cache.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace ovl {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%10, %11, %12, %13};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// 8x8 16-bit matrix, row i in lanes 4 i .. 4 i + 3: transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (a, b) as f16 pairs, the rounded part first; a and b become the rest.
__device__ __forceinline__ uint32_t take_f16(float& a, float& b) {
  const uint32_t r = pack_f16(a, b);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
  a -= f.x;
  b -= f.y;
  return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  return mul_f16x2(a, *reinterpret_cast<const __half2*>(&b));
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// (w & MASK) | magic in one LOP3: only one of the two can be an immediate, so
// magic is a register that the compiler cannot see through.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t mask_or(uint32_t w, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(magic));
  return r;
}

// The four pairs of a word's codes in f16.  As they lie, the bits of subnormals:
// code 2^-24 in pairs 0 and 2, 16 code 2^-24 in pairs 1 and 3.
__device__ __forceinline__ void masked_pairs(uint32_t w, uint32_t (&x)[4]) {
  const uint32_t h = w >> 8;
  x[0] = w & 0x000f000fu;
  x[1] = w & 0x00f000f0u;
  x[2] = h & 0x000f000fu;
  x[3] = h & 0x00f000f0u;
}
// Exactly code - 8, from 1024 + code and 1024 + 16 code.  magic: 0x64006400.
__device__ __forceinline__ void signed_pairs(uint32_t w, uint32_t magic, uint32_t (&x)[4]) {
  const uint32_t h = w >> 8;
  x[0] = sub_f16x2(mask_or<0x000f000fu>(w, magic), 0x64086408u);                // - 1032
  x[1] = fma_f16x2(mask_or<0x00f000f0u>(w, magic), 0x2c002c00u, 0xd480d480u);   // / 16 - 72
  x[2] = sub_f16x2(mask_or<0x000f000fu>(h, magic), 0x64086408u);
  x[3] = fma_f16x2(mask_or<0x00f000f0u>(h, magic), 0x2c002c00u, 0xd480d480u);
}

// Adds 1, returns what was there; releases and acquires at the GPU's scope.
__device__ __forceinline__ uint32_t arrive_acq_rel(uint32_t* p) {
  uint32_t v;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// a * b in 64 bits, one instruction.
__device__ __forceinline__ uint64_t wide(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mul.wide.u32 %0, %1, %2;" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float2 halves(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// N consecutive 32-bit words from global memory, in loads of up to 16 bytes.
template <int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t* w) {
  if constexpr (N == 1) {
    w[0] = *static_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *static_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = static_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

}  // namespace ovl
