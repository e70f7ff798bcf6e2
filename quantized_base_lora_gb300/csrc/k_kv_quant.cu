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

// Read once: marked as streaming, so that what stays in L2 is the cache (101 -> 95 us
// for writing 16 prompts and reading them back).
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, uint64_t at, float (&x)[8]) {
  if constexpr (BF16) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldcs(p), b = __ldcs(p + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

// The codes of 8 channels, each clamp(round_half_away(x / s), -8, 7) + 8, from
// the lowest 4 bits on.  inv: the reciprocal of s rounded to nearest, 0 where s is
// 0.  x inv is corrected by one residual step, which gives the correctly rounded
// quotient (Markstein, IBM J. Res. Dev. 34, 1990; s has 11 significant bits, so
// the method's one exception does not occur): a block costs one reciprocal
// instead of 32 divisions.
template <bool TAME>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float s, float inv) {
  uint32_t w = 0x88888888u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * inv;
    float t = fminf(fmaf(fmaf(-q, s, x[i]), inv, q), 7.f);
    if constexpr (!TAME) t = fmaxf(t, -8.f);       // a tame block's |t| is below 8.01
    w += static_cast<uint32_t>(__float2int_rz(t + copysignf(0.5f, t))) << (4 * i);
  }
  return w;
}

// Heads of one thread: the token's place is found once for them and their loads
// are in flight together.  A call with few tokens has them one by one, so that
// its latency is that of one.  Bound by memory (reads 2 or 4, writes 0.5625 bytes
// a channel) with the arithmetic close behind: most blocks are tame - finite and
// neither so small nor so large that d is subnormal or saturated - and need no
// care for single channels.  Measured: 26600 tokens of 8 heads of 128 in fp32 (218
// MB in, 31 MB out), and reading their values back (218 MB out), 97 us together;
// 162 us with one head a thread and a division a channel, 115 with four heads and
// one reciprocal a block, 101 without the care (two heads 104, eight 122), 95 with
// streaming loads, 97 with a look at the page's readers.  8 tokens: 5 us each, of which
// the launch and seven dependent loads are all.
constexpr uint32_t kHeadsMany = 4;

template <int D, bool BF16, uint32_t HT>
__global__ void __launch_bounds__(kThreads) k_kv_append(const KvDev kv, uint32_t layer, const int32_t* seqs,
                                                        const int32_t* off, uint32_t n, uint32_t n_tokens,
                                                        const void* k, const void* v, uint64_t ks, uint64_t vs) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr uint32_t kWords = D / 8;
  const uint32_t j = threadIdx.x % kWords, h0 = blockIdx.z * HT;
  const uint64_t token = static_cast<uint64_t>(blockIdx.x) * (kThreads / kWords) + threadIdx.x / kWords;
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
  const int32_t readers = at.page >= 0 ? kv.refs[at.page] : 0;      // asked for here, looked at before the stores
  const uint64_t u0 = kv_unit(kv, at.page < 0 ? 0 : at.page, layer, values, h0);
  uint8_t* const codes = kv.codes + u0 * kv.unit_codes + word_offset<D>(values, at.slot, j);
  __half* const scales = kv.scales + u0 * kv.unit_scales + at.slot * (D / 32) + (j >> 2);
#pragma unroll
  for (uint32_t h = 0; h < HT; ++h) {
    float m = 0.f, odd = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[h][i])), odd = fmaf(x[h][i], 0.f, odd);   // odd: NaN or 0
    const bool tame = odd == 0.f && (m == 0.f || (m >= 0x1p-10f && m <= 8.f * 65504.f));
    if (!__all_sync(0xffffffffu, tame)) {
      m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[h][i] = x[h][i] == x[h][i] ? fminf(fmaxf(x[h][i], -8.f * 65504.f), 8.f * 65504.f) : 0.f;
        m = fmaxf(m, fabsf(x[h][i]));
      }
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const __half d = __float2half_rn(m * 0.125f);
    const float s = __half2float(d), inv = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t w;
    if (__all_sync(0xffffffffu, tame)) w = codes_of<true>(x[h], s, inv);
    else w = codes_of<false>(x[h], s, inv);
    if (values) w = transpose8(w, j & 7);
    if (at.page < 0 || readers > 1 || h0 + h >= kv.heads) continue;
    *reinterpret_cast<uint32_t*>(codes + static_cast<uint64_t>(h) * kv.unit_codes) = w;
    if ((j & 3) == 0) scales[static_cast<uint64_t>(h) * kv.unit_scales] = d;
  }
  if (readers > 1) kv_latch(kv, OVL_E_STATE);      // another row's page as well: its tokens would change under it
}

template <int D, uint32_t HT>
__global__ void __launch_bounds__(kThreads) k_kv_read(const KvDev kv, uint32_t layer, const int32_t* seqs,
                                                      const int32_t* off, uint32_t n, uint32_t n_tokens, float* k,
                                                      float* v) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr uint32_t kWords = D / 8;
  const uint32_t j = threadIdx.x % kWords, h0 = blockIdx.z * HT;
  const uint64_t token = static_cast<uint64_t>(blockIdx.x) * (kThreads / kWords) + threadIdx.x / kWords;
  const bool values = blockIdx.y != 0;
  const bool live = token < n_tokens;
  uint32_t w[HT];
  float d[HT];
  KvPlace at{-1, 0};
  if (live) at = kv_place(kv, seqs, off, n, static_cast<int32_t>(token));
  const uint64_t u0 = kv_unit(kv, at.page < 0 ? 0 : at.page, layer, values, h0);
  const uint8_t* const codes = kv.codes + u0 * kv.unit_codes + word_offset<D>(values, at.slot, j);
  const __half* const scales = kv.scales + u0 * kv.unit_scales + at.slot * (D / 32) + (j >> 2);
#pragma unroll
  for (uint32_t h = 0; h < HT; ++h) {
    w[h] = 0x88888888u;
    d[h] = 0.f;
    if (at.page >= 0 && h0 + h < kv.heads) {
      w[h] = *reinterpret_cast<const uint32_t*>(codes + static_cast<uint64_t>(h) * kv.unit_codes);
      d[h] = __half2float(scales[static_cast<uint64_t>(h) * kv.unit_scales]);
    }
  }
  // A pair of lanes has 16 channels; each store of the pair is 32 bytes of them, so
  // a lane takes half of its own word's channels and half of its neighbour's.
  const bool odd = j & 1;
  float* const out = (values ? v : k) + (token * kv.heads + h0) * D + (j & ~1u) * 8 + (odd ? 4 : 0);
#pragma unroll
  for (uint32_t h = 0; h < HT; ++h) {
    if (values) w[h] = transpose8(w[h], j & 7);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, w[h], 1);
    const uint32_t lo = (odd ? other : w[h]) >> (odd ? 16 : 0), hi = (odd ? w[h] : other) >> (odd ? 16 : 0);
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {              // 2^23 + code, exactly
      o[i] = d[h] * (__uint_as_float(((lo >> (4 * i)) & 15u) | 0x4b000000u) - 8388616.f);
      o[i + 4] = d[h] * (__uint_as_float(((hi >> (4 * i)) & 15u) | 0x4b000000u) - 8388616.f);
    }
    if (!live || h0 + h >= kv.heads) continue;
    __stcs(reinterpret_cast<float4*>(out + h * D), make_float4(o[0], o[1], o[2], o[3]));
    __stcs(reinterpret_cast<float4*>(out + h * D + 8), make_float4(o[4], o[5], o[6], o[7]));
  }
}

// The launch's grid: tokens, K | V, heads in groups of HT.
template <int D, uint32_t HT>
dim3 grid_for(const KvDev& kv, uint32_t n_tokens) {
  constexpr uint32_t kTokens = kThreads / (D / 8);
  return dim3((n_tokens + kTokens - 1) / kTokens, 2, (kv.heads + HT - 1) / HT);
}
// Whether one head a thread leaves SMs idle or barely fills them.
template <int D>
bool few_tokens(const KvDev& kv, uint32_t n_tokens) {
  const dim3 g = grid_for<D, 1>(kv, n_tokens);
  return static_cast<uint64_t>(g.x) * g.z <= 4 * sm_count();
}

template <int D, bool BF16, uint32_t HT>
cudaError_t append_heads(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                         uint32_t n_tokens, const void* k, const void* v, uint64_t ks, uint64_t vs, cudaStream_t st) {
  return launch_chained(k_kv_append<D, BF16, HT>, grid_for<D, HT>(kv, n_tokens), kThreads, 0, st, kv, layer, seqs, off, n, n_tokens, k,
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
  return launch_chained(k_kv_read<D, HT>, grid_for<D, HT>(kv, n_tokens), kThreads, 0, st, kv, layer, seqs, off, n, n_tokens, k, v);
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
