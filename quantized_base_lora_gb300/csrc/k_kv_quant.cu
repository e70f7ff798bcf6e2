// Writing tokens into the 4-bit cache and reading their values back.
//
// A block of 32 channels is held as d * (code - 8), d = f16(max|x| / 8).  Eight
// channels of one token and head (one 32-bit word of codes) belong to one
// thread, so a block's maximum is a reduction over 4 lanes.  A key word is
// stored as it is; value words are transposed 8 x 8 (nibbles against lanes) with
// three exchanges, since a value unit holds every eighth channel.
// Bound by memory: 2 or 4 bytes read and 0.5625 written per element.
#include "kv_internal.h"
#include "ptx.cuh"

namespace ovl {
namespace {

constexpr int kThreads = 256;

// Lane l of 8 holds nibble g of row l at bits 4 g; afterwards lane g holds row
// l's nibble at bits 4 l.
__device__ __forceinline__ uint32_t transpose8(uint32_t x, uint32_t lane) {
#pragma unroll
  for (int s = 4; s; s >>= 1) {
    const uint32_t low = s == 4 ? 0x0000ffffu : s == 2 ? 0x00ff00ffu : 0x0f0f0f0fu;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, s);
    x = (lane & s) ? ((x & ~low) | ((y & ~low) >> (4 * s))) : ((x & low) | ((y & low) << (4 * s)));
  }
  return x;
}

// Byte offset of word j (channels 8 j .. for keys; for values, after the
// transposition, unit j % 8's word j / 8) of a token inside its unit.
template <int D>
__device__ __forceinline__ uint32_t word_offset(bool values, uint32_t slot, uint32_t j) {
  if (!values) return slot * (D / 2) + ((j & 3) * (D / 32) + (j >> 2)) * 4;
  return (slot >> 3) * (4 * D) + (j & 7) * (D / 2) + (slot & 7) * (D / 16) + (j >> 3) * 4;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* base, uint64_t at, float (&x)[8]) {
  if constexpr (BF16) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

// clamp(round_half_away(x / s), -8, 7) + 8, with inv the reciprocal of s rounded
// to nearest (0 where s is 0).  x inv is corrected by one residual step, which
// gives the correctly rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990; s
// has 11 significant bits, so the method's one exception does not occur).  A
// block costs one reciprocal instead of 32 divisions.
__device__ __forceinline__ uint32_t code_of(float x, float s, float inv) {
  x = x == x ? fminf(fmaxf(x, -3.4e38f), 3.4e38f) : 0.f;         // infinities are clipped
  const float q = x * inv;
  float t = fmaf(fmaf(-q, s, x), inv, q);
  t = fminf(fmaxf(t, -8.f), 7.f);
  return static_cast<uint32_t>(__float2int_rz(t + copysignf(0.5f, t)) + 8);
}

// Heads of one thread: the token's place is found once for them and their loads
// are in flight together.  A call with few tokens has them one by one, so that
// its latency is that of one.
constexpr uint32_t kHeadsMany = 4;

template <int D, bool BF16, uint32_t HT>
__global__ void __launch_bounds__(kThreads) k_kv_append(const KvDev kv, uint32_t layer, const int32_t* seqs,
                                                        const int32_t* off, uint32_t n, uint32_t n_tokens,
                                                        const void* k, const void* v, uint64_t ks, uint64_t vs) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr uint32_t kWords = D / 8;
  const uint64_t id = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint32_t j = id % kWords, parts = (kv.heads + HT - 1) / HT;
  const uint64_t th = id / kWords;
  const uint32_t h0 = th % parts * HT;
  const uint64_t token = th / parts;
  const bool values = blockIdx.y != 0;
  const bool live = token < n_tokens;
  float x[HT][8];
#pragma unroll
  for (uint32_t h = 0; h < HT; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[h][i] = 0.f;
    if (live && h0 + h < kv.heads) load8<BF16>(values ? v : k, token * (values ? vs : ks) + (h0 + h) * D + j * 8, x[h]);
  }
  KvPlace at{-1, 0};
  if (live) at = kv_place(kv, seqs, off, n, static_cast<int32_t>(token));
#pragma unroll
  for (uint32_t h = 0; h < HT; ++h) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[h][i]));   // a NaN is no maximum
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const __half d = __float2half_rn(fminf(m * 0.125f, 65504.f));
    const float s = __half2float(d), inv = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= code_of(x[h][i], s, inv) << (4 * i);
    if (values) w = transpose8(w, j & 7);
    if (at.page < 0 || h0 + h >= kv.heads) continue;
    const uint64_t u = kv_unit(kv, at.page, layer, values, h0 + h);
    *reinterpret_cast<uint32_t*>(kv.codes + u * kv.unit_codes + word_offset<D>(values, at.slot, j)) = w;
    if ((j & 3) == 0) kv.scales[u * kv.unit_scales + at.slot * (D / 32) + (j >> 2)] = d;
  }
}

template <int D, uint32_t HT>
__global__ void __launch_bounds__(kThreads) k_kv_read(const KvDev kv, uint32_t layer, const int32_t* seqs,
                                                      const int32_t* off, uint32_t n, uint32_t n_tokens, float* k,
                                                      float* v) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr uint32_t kWords = D / 8;
  const uint64_t id = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint32_t j = id % kWords, parts = (kv.heads + HT - 1) / HT;
  const uint64_t th = id / kWords;
  const uint32_t h0 = th % parts * HT;
  const uint64_t token = th / parts;
  const bool values = blockIdx.y != 0;
  const bool live = token < n_tokens;
  uint32_t w[HT];
  float d[HT];
  KvPlace at{-1, 0};
  if (live) at = kv_place(kv, seqs, off, n, static_cast<int32_t>(token));
#pragma unroll
  for (uint32_t h = 0; h < HT; ++h) {
    w[h] = 0x88888888u;
    d[h] = 0.f;
    if (at.page >= 0 && h0 + h < kv.heads) {
      const uint64_t u = kv_unit(kv, at.page, layer, values, h0 + h);
      w[h] = *reinterpret_cast<const uint32_t*>(kv.codes + u * kv.unit_codes + word_offset<D>(values, at.slot, j));
      d[h] = __half2float(kv.scales[u * kv.unit_scales + at.slot * (D / 32) + (j >> 2)]);
    }
  }
#pragma unroll
  for (uint32_t h = 0; h < HT; ++h) {
    if (values) w[h] = transpose8(w[h], j & 7);
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)                // 2^23 + code, exactly
      o[i] = d[h] * (__uint_as_float(((w[h] >> (4 * i)) & 15u) | 0x4b000000u) - 8388616.f);
    // a pair of lanes swaps halves, so that each store is 32 whole bytes of the pair
    const bool odd = j & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float give = odd ? o[i] : o[i + 4];
      const float take = __shfl_xor_sync(0xffffffffu, give, 1);
      if (odd) o[i] = take;
      else o[i + 4] = take;
    }
    if (!live || h0 + h >= kv.heads) continue;
    float* const p = (values ? v : k) + (token * kv.heads + h0 + h) * D + (j & ~1u) * 8 + (odd ? 4 : 0);
    __stcs(reinterpret_cast<float4*>(p), make_float4(o[0], o[1], o[2], o[3]));
    __stcs(reinterpret_cast<float4*>(p + 8), make_float4(o[4], o[5], o[6], o[7]));
  }
}

// Blocks of a launch, 0 where there are too many.
template <int D, uint32_t HT>
uint32_t blocks_for(const KvDev& kv, uint32_t n_tokens) {
  const uint64_t threads = static_cast<uint64_t>(n_tokens) * ((kv.heads + HT - 1) / HT) * (D / 8);
  const uint64_t blocks = (threads + kThreads - 1) / kThreads;
  return blocks <= 0x7fffffffu ? static_cast<uint32_t>(blocks) : 0u;
}
// Whether one head a thread leaves SMs idle or barely fills them.
template <int D>
bool few_tokens(const KvDev& kv, uint32_t n_tokens) {
  return blocks_for<D, 1>(kv, n_tokens) <= 4 * kv_sm_count();
}

template <int D, bool BF16, uint32_t HT>
cudaError_t append_heads(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                         uint32_t n_tokens, const void* k, const void* v, uint64_t ks, uint64_t vs, cudaStream_t st) {
  const uint32_t blocks = blocks_for<D, HT>(kv, n_tokens);
  if (!blocks) return cudaErrorInvalidConfiguration;
  return launch_chained(k_kv_append<D, BF16, HT>, dim3(blocks, 2), kThreads, 0, st, kv, layer, seqs, off, n, n_tokens, k,
                        v, ks, vs);
}

template <int D>
cudaError_t append_dim(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                       uint32_t n_tokens, const void* k, const void* v, bool bf16, uint64_t ks, uint64_t vs,
                       cudaStream_t st) {
  if (few_tokens<D>(kv, n_tokens))
    return bf16 ? append_heads<D, true, 1>(kv, layer, seqs, off, n, n_tokens, k, v, ks, vs, st)
                : append_heads<D, false, 1>(kv, layer, seqs, off, n, n_tokens, k, v, ks, vs, st);
  return bf16 ? append_heads<D, true, kHeadsMany>(kv, layer, seqs, off, n, n_tokens, k, v, ks, vs, st)
              : append_heads<D, false, kHeadsMany>(kv, layer, seqs, off, n, n_tokens, k, v, ks, vs, st);
}

template <int D, uint32_t HT>
cudaError_t read_heads(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                       uint32_t n_tokens, float* k, float* v, cudaStream_t st) {
  const uint32_t blocks = blocks_for<D, HT>(kv, n_tokens);
  if (!blocks) return cudaErrorInvalidConfiguration;
  return launch_chained(k_kv_read<D, HT>, dim3(blocks, 2), kThreads, 0, st, kv, layer, seqs, off, n, n_tokens, k, v);
}

template <int D>
cudaError_t read_dim(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                     uint32_t n_tokens, float* k, float* v, cudaStream_t st) {
  return few_tokens<D>(kv, n_tokens) ? read_heads<D, 1>(kv, layer, seqs, off, n, n_tokens, k, v, st)
                                     : read_heads<D, kHeadsMany>(kv, layer, seqs, off, n, n_tokens, k, v, st);
}

}  // namespace

cudaError_t launch_kv_append(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                             uint32_t n_tokens, const void* k, const void* v, bool bf16, uint64_t ks, uint64_t vs,
                             cudaStream_t st) {
  switch (kv.dim) {
    case 64: return append_dim<64>(kv, layer, seqs, off, n, n_tokens, k, v, bf16, ks, vs, st);
    case 128: return append_dim<128>(kv, layer, seqs, off, n, n_tokens, k, v, bf16, ks, vs, st);
    default: return append_dim<256>(kv, layer, seqs, off, n, n_tokens, k, v, bf16, ks, vs, st);
  }
}

cudaError_t launch_kv_read(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                           uint32_t n_tokens, float* k, float* v, cudaStream_t st) {
  switch (kv.dim) {
    case 64: return read_dim<64>(kv, layer, seqs, off, n, n_tokens, k, v, st);
    case 128: return read_dim<128>(kv, layer, seqs, off, n, n_tokens, k, v, st);
    default: return read_dim<256>(kv, layer, seqs, off, n, n_tokens, k, v, st);
  }
}

}  // namespace ovl
