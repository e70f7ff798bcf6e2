// The router of a mixture-of-experts layer, the tokens as its products (moe_rows.cuh) take
// them, and the sum of the experts' outputs.
//
// Scores are plain fp32 dot products: a CTA has 8 experts and up to 8 tokens, two warps an
// expert.  The last CTA of 8 tokens chooses their experts, a warp a token.  Beside that,
// further CTAs split the tokens into scaled bf16 parts.  The counters by which the last CTA
// is known are set back by the first product of the same call, whatever they hold: calls
// that ran beside one another against the rules leave nothing behind for later ones.
#include <type_traits>

#include "moe_rows.cuh"

namespace ovl {
namespace {

using namespace moe;
constexpr uint32_t kThreads = 512;
constexpr int kGroup = kMoeRouted;       // tokens of a router CTA, and its experts

// Order-preserving bits of a score; NaN is the least.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return v != v ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// Scores of N tokens from t0 (places behind the last token take it once more) and an
// expert over every other piece of the row, added up over the warp.
template <int N, bool XB, bool RB>
__device__ __forceinline__ void scores(const MoeDev& m, uint32_t expert, uint32_t t0, uint32_t odd, float (&acc)[N]) {
  constexpr int kAhead = N == 1 ? 8 : XB ? 4 : 2;  // pieces in flight
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  const uint64_t row = static_cast<uint64_t>(expert) * m.hidden;
  for (uint32_t c0 = odd * 128 + lane * 4; c0 < m.hidden; c0 += 256 * kAhead) {
    Raw<4> w[kAhead], x[kAhead][N];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const uint32_t c = min(c0 + 256 * a, m.hidden - 4);
      load_raw<4>(m.router, RB, row + c, w[a]);
#pragma unroll
      for (int i = 0; i < N; ++i) load_raw<4>(m.x.ptr, XB, min(t0 + i, m.tokens - 1) * m.x.stride + c, x[a][i]);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (c0 + 256 * a < m.hidden) {
        float u[4], v[4];
        to_f32<4>(w[a], RB, u);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          to_f32<4>(x[a][i], XB, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i] = fmaf(u[j], v[j], acc[i]);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = warp_sum(acc[i]);
}

// The token's top_k experts and their weights, by one warp; 32 kMost experts at most.
template <int kMost>
__device__ void choose(const MoeDev& m, uint32_t token) {
  const uint32_t lane = threadIdx.x & 31;
  const bool softmax = m.score == OVL_MOE_SOFTMAX;
  float z[kMost];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const uint32_t e = i * 32 + lane;
    z[i] = e < m.experts ? __ldcg(&m.logits[static_cast<uint64_t>(token) * m.experts + e]) : -INFINITY;
    if (e < m.experts) top = fmaxf(top, z[i]);
  }
  float inv = 1.f;
  if (softmax) {
#pragma unroll
    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < kMost; ++i)
      if (i * 32 + lane < m.experts) total += expf(z[i] - top);
    inv = 1.f / warp_sum(total);
  }
  // A score times e^-(ref - none): a weight that is divided by the chosen ones' sum goes by
  // the scores' ratios, which the scores themselves have lost once they are below fp32's range.
  // A sigmoid is written as e^min(v, 0) / (1 + e^-|v|), whose divisor is 1 to 2.
  const float none = softmax ? top : 0.f;
  auto score = [&](float v, float ref) {
    return softmax ? expf(v - ref) * inv : expf(fminf(v, 0.f) - ref) / (1.f + expf(-fabsf(v)));
  };
  // Without a bias the choice goes by the logits, which order as the scores do and do not saturate.
  uint32_t key[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const uint32_t e = i * 32 + lane;
    key[i] = 0;
    if (e < m.experts) key[i] = order_of(m.bias ? score(z[i], none) + m.bias[e] : z[i]);
  }
  uint32_t taken = 0, mine = 0;
  float logit = -INFINITY;
  for (uint32_t s = 0; s < m.top; ++s) {
    uint32_t best = 0;
    int at = -1;
#pragma unroll
    for (int i = 0; i < kMost; ++i)
      if (i * 32 + lane < m.experts && !(taken >> i & 1) && (at < 0 || key[i] > best)) best = key[i], at = i;
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, at >= 0 && best == most ? at * 32 + lane : 0xffffffffu);
    float v = 0.f;
    if ((e & 31) == lane) {
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i == static_cast<int>(e / 32)) v = z[i];
      taken |= 1u << (e / 32);
    }
    v = __shfl_sync(0xffffffffu, v, e & 31);
    if (lane == s) mine = e, logit = v;
  }
  float most = logit;                              // of the chosen ones
#pragma unroll
  for (int s = 16; s; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
  float weight = score(logit, m.renormalize ? fminf(most, none) : none);
  if (m.renormalize) weight /= warp_sum(lane < m.top ? weight : 0.f);
  weight *= m.scale;
  if (lane < m.top) {
    const uint32_t p = token * m.top + lane;
    m.choice[p] = static_cast<int32_t>(mine);
    m.weight[p] = weight;
    if (m.choice_out) m.choice_out[p] = static_cast<int32_t>(mine);
    if (m.weight_out) m.weight_out[p] = weight;
  }
}

// A token as scaled bf16 parts, by one CTA.
template <uint32_t Q, int PARTS>
__device__ void split_token(const MoeDev& m, uint32_t token) {
  __shared__ float most[kThreads / 32];
  const uint64_t row = token * m.x.stride;
  float top = 0.f;
  for (uint32_t c = threadIdx.x * 8; c < m.hidden; c += kThreads * 8) {
    float x[8];
    load_f32<8>(m.x.ptr, PARTS == 1, row + c, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (uint32_t w = 0; w < kThreads / 32; ++w) top = fmaxf(top, most[w]);
  // 2^e <= top < 2^(e + 1) within the normal range, whose inverse is a number too
  const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 2), 253) - 127;
  if (threadIdx.x == 0) m.power[token] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  const float once = __uint_as_float(static_cast<uint32_t>((kTokenExponent - e) / 2 + 127) << 23);       // (100 - e) / 2 is -13 .. 112
  const float twice = __uint_as_float(static_cast<uint32_t>(kTokenExponent - e - (kTokenExponent - e) / 2 + 127) << 23);
  for (uint32_t c = threadIdx.x * 8; c < m.hidden; c += kThreads * 8) {
    float x[8];
    load_f32<8>(m.x.ptr, PARTS == 1, row + c, x);
    uint16_t v[8][PARTS];
#pragma unroll
    for (int j = 0; j < 8; ++j) parts_of<PARTS>(x[j] * once * twice * share_of<Q>(j), v[j]);
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      uint16_t* out = m.xp + (static_cast<uint64_t>(q) * m.tokens + token) * m.hidden + (c & ~31u);
      uint32_t w[4];
      if constexpr (Q == OVL_Q8_0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v[2 * j][q] | static_cast<uint32_t>(v[2 * j + 1][q]) << 16;
        *reinterpret_cast<uint2*>(out + place_of<Q>(c & 31)) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(out + place_of<Q>((c & 31) + 4)) = make_uint2(w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v[j][q] | static_cast<uint32_t>(v[j + 4][q]) << 16;
        *reinterpret_cast<uint4*>(out + (c & 31)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

template <bool XB, bool RB>
__global__ void __launch_bounds__(kThreads) k_moe_route(const __grid_constant__ MoeDev m, uint32_t routers) {
  __shared__ uint32_t last;
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x >= routers) {
    const uint32_t token = blockIdx.x - routers;
    if (m.quant == OVL_Q8_0) split_token<OVL_Q8_0, XB ? 1 : 3>(m, token);
    else split_token<OVL_Q4_0, XB ? 1 : 3>(m, token);
    return;
  }
  __shared__ float part[kGroup][kGroup];           // expert, token: of the odd pieces
  const uint32_t wide = (m.experts + kGroup - 1) / kGroup;
  const uint32_t group = blockIdx.x / wide, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t e = warp % kGroup, odd = warp / kGroup;
  const uint32_t expert = blockIdx.x % wide * kGroup + e, t0 = group * kGroup, n = min(m.tokens - t0, kGroup);
  float mine = 0.f;                                // lane i: of token i
  if (expert < m.experts) {
    if (n == 1) {
      float acc[1];
      scores<1, XB, RB>(m, expert, t0, odd, acc);
      mine = acc[0];
    } else {
      float acc[kGroup];
      scores<kGroup, XB, RB>(m, expert, t0, odd, acc);
#pragma unroll
      for (uint32_t i = 0; i < kGroup; ++i)
        if (lane == i) mine = acc[i];
    }
  }
  if (odd && lane < kGroup) part[e][lane] = mine;
  __syncthreads();
  if (!odd && expert < m.experts && lane < n) {
    m.logits[static_cast<uint64_t>(t0 + lane) * m.experts + expert] = mine + part[e][lane];
    if (wide > 1) __threadfence();
  }
  __syncthreads();
  if (wide > 1) {                                  // else all scores are the CTA's own: one token's choice 1 us sooner
    if (threadIdx.x == 0) last = atomicAdd(&m.arrived[group], 1u) + 1 == wide;
    __syncthreads();
    if (!last) return;
    __threadfence();
  }
  if (warp < n) {
    if (m.experts <= 128) choose<4>(m, t0 + warp);
    else choose<OVL_MOE_MAX_EXPERTS / 32>(m, t0 + warp);
  }
}

// y of a token: its experts' weighted outputs, in the order of the choice.
constexpr uint32_t kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) k_moe_sum(const __grid_constant__ MoeDev m) {
  griddep_launch_dependents();
  // The choice was made before the products began: which places have an expert.
  const int32_t* choice = m.given ? m.given_choice : m.choice;
  const uint32_t per = m.hidden / 4;
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kSumThreads + threadIdx.x;
  const uint32_t token = static_cast<uint32_t>(i / per), c = static_cast<uint32_t>(i % per) * 4;
  uint32_t some = 0;
  if (token < m.tokens)
    for (uint32_t s = 0; s < m.top; ++s)
      if (static_cast<uint32_t>(choice[token * m.top + s]) < m.experts) some |= 1u << s;
  griddep_wait();
  if (token >= m.tokens) return;
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (uint32_t s = 0; s < m.top; ++s) {
    if (!(some >> s & 1)) continue;
    float v[4];
    load_f32<4>(m.part, false, static_cast<uint64_t>(token * m.top + s) * m.hidden + c, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += v[j];
  }
  store_f32<4>(m.y.ptr, m.y.bf16, token * m.y.stride + c, y);
}

}  // namespace

cudaError_t launch_moe(const MoeDev& m, cudaStream_t st) {
  const uint32_t wide = (m.experts + kGroup - 1) / kGroup, groups = (m.tokens + kGroup - 1) / kGroup;
  const uint32_t routers = m.given ? 0 : wide * groups;
  const auto route = m.bf16 ? (m.router_bf16 ? k_moe_route<true, true> : k_moe_route<true, false>)
                            : (m.router_bf16 ? k_moe_route<false, true> : k_moe_route<false, false>);
  cudaError_t e = launch_chained(route, dim3(routers + m.tokens), kThreads, 0, st, m, routers);
  if (e == cudaSuccess)
    e = m.quant == OVL_Q8_0 ? launch_products_q8_0(m, st) : m.quant == OVL_Q4_0 ? launch_products_q4_0(m, st) : launch_products_q4_k(m, st);
  if (e != cudaSuccess) return e;
  return launch_chained(k_moe_sum, dim3((m.tokens * (m.hidden / 4) + kSumThreads - 1) / kSumThreads), kSumThreads, 0, st, m);
}

}  // namespace ovl
