// Shared by the translation units of what a decoder block computes between its
// projections (ovl_rope_apply, ovl_block_norm_apply, ovl_glu, ovl_moe_forward).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ovl.h"
#include "kv_internal.h"
#include "ptx.cuh"

namespace ovl {

// A tensor of tokens: element c of token t lies at ptr + (t * stride + c) elements.
struct Rows {
  void* ptr;
  uint64_t stride;
  bool bf16;
};

// N consecutive elements of a float32 or bfloat16 array as they lie.  Loading and
// converting are apart, so that a thread's loads are all under way before the first one is
// waited for: a conversion behind its load, in the branch of its type, had them one by one.
template <int N>
struct Raw {
  uint32_t w[N];
};
// From element `at`.  N > 1: its address is a multiple of N elements or of 16 bytes, whichever is less.
template <int N>
__device__ __forceinline__ void load_raw(const void* base, bool bf16, uint64_t at, Raw<N>& r) {
  static_assert(N == 1 || N == 4 || N == 8, "1, 4 or 8 elements");
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if constexpr (N == 1) {
      r.w[0] = *p;
    } else if constexpr (N == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      r.w[0] = v.x, r.w[1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
    }
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(base) + at;
    if constexpr (N == 1) {
      r.w[0] = *p;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + i);
        r.w[i] = v.x, r.w[i + 1] = v.y, r.w[i + 2] = v.z, r.w[i + 3] = v.w;
      }
    }
  }
}
template <int N>
__device__ __forceinline__ void to_f32(const Raw<N>& r, bool bf16, float (&v)[N]) {
  if (bf16) {
    if constexpr (N == 1) {
      v[0] = __uint_as_float(r.w[0] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        v[2 * i] = __uint_as_float(r.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r.w[i]);
  }
}
template <int N>
__device__ __forceinline__ void load_f32(const void* base, bool bf16, uint64_t at, float (&v)[N]) {
  Raw<N> r;
  load_raw(base, bf16, at, r);
  to_f32(r, bf16, v);
}

__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The same way back, rounded to nearest.
template <int N>
__device__ __forceinline__ void store_f32(void* base, bool bf16, uint64_t at, const float (&v)[N]) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if constexpr (N == 1) *p = static_cast<uint16_t>(two_bf16(v[0], v[0]));
    else if constexpr (N == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(two_bf16(v[0], v[1]), two_bf16(v[2], v[3]));
    else
      *reinterpret_cast<uint4*>(p) = make_uint4(two_bf16(v[0], v[1]), two_bf16(v[2], v[3]), two_bf16(v[4], v[5]),
                                                two_bf16(v[6], v[7]));
  } else {
    float* p = static_cast<float*>(base) + at;
    if constexpr (N == 1) {
      *p = v[0];
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  }
}

// act(v) of OVL_ACT_*, in fp32.  1 + erf(u) is written as erfc(-u), which keeps its bits
// where it is small (at v = -5 the sum is off by 4 %); it costs more: 4096 x 14336 in bf16
// 109 us, 84 with the sum.  (1 + tanh u) / 2 is written as 1 / (1 + e^(-2u)).  The approximate
// quotient is 0 for divisors from 2^126 on: silu and gelu_tanh are 0 where they are below
// 2^-119 in size.  (By e^-|v|, with a divisor of 1 to 2, they were not, and 8 % slower.)
__device__ __forceinline__ float activated(float v, uint32_t act) {
  switch (act) {
    case OVL_ACT_SILU: return __fdividef(v, 1.f + expf(-v));
    case OVL_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
    case OVL_ACT_GELU_TANH:
      return __fdividef(v, 1.f + expf(-1.5957691216057308f * fmaf(0.044715f * v * v, v, v)));
    default: return v < 0.f ? 0.f : v;            // a NaN stays one
  }
}

cudaError_t launch_rope(const ovl_rope& rope, uint32_t n_tokens, const int32_t* pos, Rows q, uint32_t q_heads, Rows k,
                        uint32_t k_heads, Rows q_out, Rows k_out, cudaStream_t st);
cudaError_t launch_kv_positions(const KvDev& kv, const int32_t* seqs, const int32_t* off, uint32_t n, uint32_t n_tokens,
                                int32_t* pos, cudaStream_t st);

// Gate of ovl_block_norm_apply; ptr null: ones.
struct Gate {
  Rows rows;
  const int32_t* row;
  uint32_t n;
};
cudaError_t launch_block_norm(const ovl_block_norm& norm, uint32_t n_tokens, Rows x, Rows y, Gate gate, Rows x_out,
                              Rows h, cudaStream_t st);
cudaError_t launch_glu(uint32_t act, uint32_t n_tokens, uint32_t width, Rows gate, Rows up, Rows out, cudaStream_t st);

// A mixture-of-experts call as its kernels take it.
constexpr uint32_t kMoeTokens = 8;       // tokens of one expert that one pass over its weights serves
constexpr uint32_t kMoeRouted = 8;       // tokens of a router CTA
constexpr uint32_t kMoeGroups = (OVL_MOE_MAX_TOKENS + kMoeRouted - 1) / kMoeRouted;
constexpr uint32_t kMoeMaxPairs = OVL_MOE_MAX_TOKENS * OVL_MOE_MAX_TOP;
constexpr uint32_t kMoeMaxUnits = OVL_MOE_MAX_EXPERTS + kMoeMaxPairs / kMoeTokens;
// Up to kMoeTokens pairs of one expert, in 41 bits.
struct MoeUnit {
  uint16_t first_pairs;    // first of its pairs in the order by experts: 11 bits; pairs - 1: 3
  uint16_t expert_groups;  // expert: 9 bits; units of the expert - 1: the lower 7 of 8
  uint16_t group_groups;   // the expert's first unit: 10 bits; the rest of the 8
  static __device__ MoeUnit make(uint32_t expert, uint32_t pairs, uint32_t group, uint32_t groups, uint32_t first) {
    return {static_cast<uint16_t>(first | (pairs - 1) << 11), static_cast<uint16_t>(expert | ((groups - 1) & 127) << 9),
            static_cast<uint16_t>(group | (groups - 1) >> 7 << 10)};
  }
  __device__ uint32_t expert() const { return expert_groups & 511; }
  __device__ uint32_t groups() const { return (expert_groups >> 9 | (group_groups >> 10 << 7)) + 1; }
  __device__ uint32_t group() const { return group_groups & 1023; }
  __device__ uint32_t pairs() const { return (first_pairs >> 11) + 1; }
  __device__ uint32_t first() const { return first_pairs & 2047; }
};
static_assert(OVL_MOE_MAX_EXPERTS <= 512 && kMoeMaxPairs <= 2048 && kMoeTokens <= 8 && kMoeMaxPairs / kMoeTokens <= 256 &&
                  kMoeMaxUnits <= 1024,
              "fields of a unit");
struct MoeDev {
  const uint8_t *gate_qs, *up_qs, *down_qs, *gate_d, *up_d, *down_d;
  const void* router;
  const float* bias;
  uint32_t quant, experts, top, hidden, ffn, act, score, renormalize;
  float scale;
  bool router_bf16, bf16, given;
  uint32_t tokens, pairs;
  Rows x, y;
  const int32_t* given_choice;
  const float* given_weight;
  int32_t* choice_out;
  float* weight_out;
  // workspace
  uint32_t* arrived;       // [kMoeGroups]: router CTAs of each group of 8 tokens; 0 between calls
  float* logits;           // [tokens][experts]
  int32_t* choice;         // [tokens][top] (the caller's stay where they are)
  float* weight;
  float* power;            // [tokens]: 2^e of the largest |x|
  uint16_t* xp;            // [parts][tokens][hidden] bf16, scaled, in the order of the MMA fragments
  uint16_t* hp;            // [parts][pairs][ffn], the same of the activations
  float* part;             // [pairs][hidden]: weighted outputs
};
cudaError_t launch_moe(const MoeDev& m, cudaStream_t st);

}  // namespace ovl
