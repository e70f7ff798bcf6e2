// Attention over the 4-bit cache.
//
// One warp per query token and head walks its sequence's visible tokens with a
// running maximum and sum; lane c of the warp holds channels c, c + 32, ...
#include <math_constants.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace ovl {
namespace {

constexpr int kWarps = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) k_kv_attend(const KvDev kv, const KvQuery a) {
  constexpr int NB = D / 32;
  const uint64_t id = static_cast<uint64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t token = id / a.heads;
  if (token >= a.n_tokens) return;
  const uint32_t h = id % a.heads, kh = h / a.group;
  const uint32_t i = kv_owner(a.off, a.n_seqs, static_cast<int32_t>(token));
  const int32_t s = a.seqs[i], after = a.off[i + 1] - static_cast<int32_t>(token);
  float q[NB], o[NB] = {};
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint64_t at = token * a.q_stride + h * D + 32 * b + lane;
    if constexpr (BF16) q[b] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.q)[at]) << 16);
    else q[b] = static_cast<const float*>(a.q)[at];
  }
  int32_t pos = -1;
  if (static_cast<uint32_t>(s) >= kv.max_seqs || after <= 0) {
    if (lane == 0) kv_latch(kv, OVL_E_ARG);
  } else {
    pos = kv.length[s] - after;
    if (pos >= static_cast<int32_t>(kv.max_pages << kv.page_shift) ||
        static_cast<int32_t>(token) - a.off[i] >= static_cast<int32_t>(a.max_new)) {
      if (lane == 0) kv_latch(kv, OVL_E_SHAPE);
      pos = -1;
    }
  }
  float m = -CUDART_INF_F, l = 0.f;
  for (int32_t j = 0; j <= pos; ++j) {
    if (a.window && j <= pos - static_cast<int32_t>(a.window) && j >= static_cast<int32_t>(a.sinks)) continue;
    const int32_t p = kv.table[static_cast<size_t>(s) * kv.max_pages + (j >> kv.page_shift)];
    if (static_cast<uint32_t>(p) >= kv.n_pages) {
      if (lane == 0) kv_latch(kv, OVL_E_ARG);
      continue;
    }
    const uint32_t slot = j & (kv.page - 1);
    const uint64_t u = kv_unit(kv, p, a.layer, 0, kh);
    const uint8_t* kc = kv.codes + u * kv.unit_codes + slot * (D / 2);
    float x = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t byte = kc[((lane >> 3) * NB + b) * 4 + ((lane & 7) >> 1)];
      const int code = (byte >> (4 * (lane & 1))) & 15;
      x += q[b] * (__half2float(kv.scales[u * kv.unit_scales + slot * NB + b]) * (code - 8));
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
    x *= a.scale;
    const float mn = fmaxf(m, x), f = expf(m - mn), w = expf(x - mn);
    l = l * f + w;
    m = mn;
    const uint64_t uv = kv_unit(kv, p, a.layer, 1, kh);
    const uint8_t* vc = kv.codes + uv * kv.unit_codes + (slot >> 3) * (4 * D) + (slot & 7) * (D / 16);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t c = 32 * b + lane;
      const uint32_t byte = vc[(c & 7) * (D / 2) + (c >> 4)];
      const int code = (byte >> (4 * ((c >> 3) & 1))) & 15;
      o[b] = o[b] * f + w * (__half2float(kv.scales[uv * kv.unit_scales + slot * NB + b]) * (code - 8));
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint64_t at = token * a.out_stride + h * D + 32 * b + lane;
    const float r = l > 0.f ? o[b] / l : 0.f;
    if constexpr (BF16) {
      uint16_t v;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(v) : "f"(r));
      static_cast<uint16_t*>(a.out)[at] = v;
    } else {
      static_cast<float*>(a.out)[at] = r;
    }
  }
}

template <int D>
cudaError_t attend_dim(const KvDev& kv, const KvQuery& a, cudaStream_t st) {
  const uint64_t blocks = (static_cast<uint64_t>(a.n_tokens) * a.heads + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffu) return cudaErrorInvalidConfiguration;
  if (a.bf16) k_kv_attend<D, true><<<static_cast<uint32_t>(blocks), kWarps * 32, 0, st>>>(kv, a);
  else k_kv_attend<D, false><<<static_cast<uint32_t>(blocks), kWarps * 32, 0, st>>>(kv, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attention(const KvDev& kv, const KvQuery& a, cudaStream_t st) {
  switch (kv.dim) {
    case 64: return attend_dim<64>(kv, a, st);
    case 128: return attend_dim<128>(kv, a, st);
    default: return attend_dim<256>(kv, a, st);
  }
}

}  // namespace ovl
