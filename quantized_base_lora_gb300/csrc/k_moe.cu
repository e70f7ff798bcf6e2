// The router of a mixture-of-experts layer, what it hands to the experts' products
// (moe_rows.cuh), and the sum of the experts' outputs.
//
// Scores are plain fp32 dot products: a warp has one expert and up to 8 tokens.  The last
// CTA of 8 tokens chooses their experts, a warp a token, and the last of those sorts the
// chosen (token, expert) pairs by expert: the products then read an expert's weights once for all its tokens.
// Beside that, further CTAs split the tokens into the bf16 parts that the products multiply.
#include <type_traits>

#include "moe_rows.cuh"

namespace ovl {
namespace {

using namespace moe;
constexpr int kThreads = 256;
constexpr uint32_t kGroup = 8;           // tokens of a router CTA, experts of it as well: one a warp

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

// logits[token][expert] of up to 8 tokens from t0 and the warp's expert.
__device__ void scores(const MoeDev& m, uint32_t expert, uint32_t t0, uint32_t n) {
  const uint32_t lane = threadIdx.x & 31;
  float acc[kGroup];
#pragma unroll
  for (int i = 0; i < static_cast<int>(kGroup); ++i) acc[i] = 0.f;
  const uint64_t row = static_cast<uint64_t>(expert) * m.hidden;
#pragma unroll 4
  for (uint32_t c = lane * 4; c < m.hidden; c += 128) {
    float w[4];
    load_f32<4>(m.router, m.router_bf16, row + c, w);
#pragma unroll
    for (int i = 0; i < static_cast<int>(kGroup); ++i) {
      if (i >= static_cast<int>(n)) break;
      float x[4];
      load_f32<4>(m.x.ptr, m.x.bf16, (t0 + i) * m.x.stride + c, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i] = fmaf(w[j], x[j], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < static_cast<int>(kGroup); ++i) {
    const float v = warp_sum(acc[i]);
    if (i < static_cast<int>(n) && lane == 0) m.logits[static_cast<uint64_t>(t0 + i) * m.experts + expert] = v;
  }
}

// The token's top_k experts and their weights, by one warp.
__device__ void choose(const MoeDev& m, uint32_t token) {
  constexpr int kMost = OVL_MOE_MAX_EXPERTS / 32;
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
  auto score = [&](float v) { return softmax ? expf(v - top) * inv : 1.f / (1.f + expf(-v)); };
  // Without a bias the choice goes by the logits, which order as the scores do and do not saturate.
  uint32_t key[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const uint32_t e = i * 32 + lane;
    key[i] = 0;
    if (e < m.experts) key[i] = order_of(m.bias ? score(z[i]) + m.bias[e] : z[i]);
  }
  uint32_t taken = 0, mine = 0;
  float weight = 0.f;
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
    if (lane == s) mine = e, weight = score(v);
  }
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

// Pairs sorted by expert, in pair order within one, and cut into units; by one CTA.
__device__ void sort_pairs(const MoeDev& m, bool given) {
  constexpr uint32_t kW = kThreads / 32;
  __shared__ uint32_t count[kW][OVL_MOE_MAX_EXPERTS];
  __shared__ uint32_t sums[2][kW];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (uint32_t i = threadIdx.x; i < kW * OVL_MOE_MAX_EXPERTS; i += kThreads) (&count[0][0])[i] = 0;
  __syncthreads();
  const uint32_t per = (m.pairs + kW * 32 - 1) / (kW * 32);          // rounds of 32 pairs a warp
  const uint32_t first = warp * per * 32;
  auto expert_of = [&](uint32_t p) {
    int32_t e = -1;
    if (p < m.pairs) {
      e = given ? m.given_choice[p] : __ldcg(&m.choice[p]);
      if (static_cast<uint32_t>(e) >= m.experts) e = -1;
    }
    return e;
  };
  for (uint32_t r = 0; r < per; ++r) {
    const uint32_t p = first + r * 32 + lane;
    const int32_t e = expert_of(p);
    if (given && p < m.pairs) {
      m.choice[p] = e;
      m.weight[p] = m.given_weight[p];
      if (m.choice_out) m.choice_out[p] = e;
      if (m.weight_out) m.weight_out[p] = m.given_weight[p];
    }
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && (same & ((1u << lane) - 1)) == 0) count[warp][e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // Thread t has experts 2 t and 2 t + 1: pairs and units before them.
  uint32_t n[2], before_pairs = 0, before_units = 0, pairs = 0, units = 0;
  static_assert(OVL_MOE_MAX_EXPERTS == 2 * kThreads, "two experts a thread");
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t e = 2 * threadIdx.x + i;
    n[i] = 0;
    for (uint32_t w = 0; w < kW; ++w) n[i] += count[w][e];
    pairs += n[i];
    units += (n[i] + kMoeTokens - 1) / kMoeTokens;
  }
  uint32_t a = pairs, b = units;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, a, s), v = __shfl_up_sync(0xffffffffu, b, s);
    if (static_cast<int>(lane) >= s) a += u, b += v;
  }
  if (lane == 31) sums[0][warp] = a, sums[1][warp] = b;
  __syncthreads();
  for (uint32_t w = 0; w < warp; ++w) before_pairs += sums[0][w], before_units += sums[1][w];
  before_pairs += a - pairs;
  before_units += b - units;
  if (threadIdx.x == kThreads - 1) *m.n_units = before_units + units;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t e = 2 * threadIdx.x + i;
    for (uint32_t at = 0; at < n[i]; at += kMoeTokens)
      m.units[before_units++] = MoeUnit{e << 8 | min(n[i] - at, kMoeTokens), before_pairs + at};
    uint32_t at = before_pairs;
    for (uint32_t w = 0; w < kW; ++w) {
      const uint32_t c = count[w][e];
      count[w][e] = at;
      at += c;
    }
    before_pairs += n[i];
  }
  __syncthreads();
  for (uint32_t r = 0; r < per; ++r) {
    const uint32_t p = first + r * 32 + lane;
    const int32_t e = expert_of(p);
    const uint32_t same = __match_any_sync(0xffffffffu, e), below = __popc(same & ((1u << lane) - 1));
    uint32_t at = 0;
    if (e >= 0) at = count[warp][e] + below;
    __syncwarp();
    if (e >= 0 && below == 0) count[warp][e] += __popc(same);
    __syncwarp();
    if (e >= 0) m.order[at] = static_cast<int32_t>(p);
  }
}

// The tokens as bf16 parts, 8 channels a thread.
template <uint32_t Q>
__device__ void split_tokens(const MoeDev& m, uint32_t block) {
  const uint32_t per = m.hidden / 8;
  const uint64_t i = static_cast<uint64_t>(block) * kThreads + threadIdx.x;
  const uint32_t token = static_cast<uint32_t>(i / per), c = static_cast<uint32_t>(i % per) * 8;
  if (token >= m.tokens) return;
  float x[8];
  load_f32<8>(m.x.ptr, m.x.bf16, token * m.x.stride + c, x);
  auto put = [&](auto parts) {
    constexpr int kParts = decltype(parts)::value;
    uint16_t v[8][kParts];
#pragma unroll
    for (int j = 0; j < 8; ++j) parts_of<kParts>(x[j], v[j]);
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = Q == OVL_Q8_0 ? v[2 * j][q] | static_cast<uint32_t>(v[2 * j + 1][q]) << 16 : v[j][q] | static_cast<uint32_t>(v[j + 4][q]) << 16;
      *reinterpret_cast<uint4*>(m.xp + (static_cast<uint64_t>(q) * m.tokens + token) * m.hidden + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  if (m.bf16) put(std::integral_constant<int, 1>{});
  else put(std::integral_constant<int, 3>{});
}

__global__ void __launch_bounds__(kThreads) k_moe_route(const __grid_constant__ MoeDev m, uint32_t routers) {
  __shared__ uint32_t last;
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x >= routers) {
    if (m.quant == OVL_Q8_0) split_tokens<OVL_Q8_0>(m, blockIdx.x - routers);
    else split_tokens<OVL_Q4_0>(m, blockIdx.x - routers);
    return;
  }
  if (m.given) {
    sort_pairs(m, true);
    return;
  }
  const uint32_t wide = (m.experts + kGroup - 1) / kGroup, groups = (m.tokens + kGroup - 1) / kGroup;
  const uint32_t group = blockIdx.x / wide, warp = threadIdx.x / 32;
  const uint32_t expert = blockIdx.x % wide * kGroup + warp, t0 = group * kGroup, n = min(m.tokens - t0, kGroup);
  if (expert < m.experts) scores(m, expert, t0, n);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(&m.arrived[1 + group], 1u) + 1 == wide;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (warp < n) choose(m, t0 + warp);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    m.arrived[1 + group] = 0;
    last = atomicAdd(&m.arrived[0], 1u) + 1 == groups;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (threadIdx.x == 0) m.arrived[0] = 0;
  sort_pairs(m, false);
}

// y of a token: its experts' weighted outputs, in the order of the choice.
__global__ void __launch_bounds__(kThreads) k_moe_sum(const __grid_constant__ MoeDev m) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t per = m.hidden / 4;
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint32_t token = static_cast<uint32_t>(i / per), c = static_cast<uint32_t>(i % per) * 4;
  if (token >= m.tokens) return;
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (uint32_t s = 0; s < m.top; ++s) {
    const uint32_t p = token * m.top + s;
    if (m.choice[p] < 0) continue;
    float v[4];
    load_f32<4>(m.part, false, static_cast<uint64_t>(p) * m.hidden + c, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += v[j];
  }
  store_f32<4>(m.y.ptr, m.y.bf16, token * m.y.stride + c, y);
}

}  // namespace

cudaError_t launch_moe(const MoeDev& m, cudaStream_t st) {
  const uint32_t wide = (m.experts + kGroup - 1) / kGroup, groups = (m.tokens + kGroup - 1) / kGroup;
  const uint32_t routers = m.given ? 1 : wide * groups;
  const uint32_t splitters = (m.tokens * (m.hidden / 8) + kThreads - 1) / kThreads;
  cudaError_t e = launch_chained(k_moe_route, dim3(routers + splitters), kThreads, 0, st, m, routers);
  if (e == cudaSuccess)
    e = m.quant == OVL_Q8_0 ? launch_products_q8_0(m, st) : m.quant == OVL_Q4_0 ? launch_products_q4_0(m, st) : launch_products_q4_k(m, st);
  if (e != cudaSuccess) return e;
  return launch_chained(k_moe_sum, dim3((m.tokens * (m.hidden / 4) + kThreads - 1) / kThreads), kThreads, 0, st, m);
}

}  // namespace ovl
