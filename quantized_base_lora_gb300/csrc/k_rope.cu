// Rotary positions of queries and keys, and the positions of a batch's tokens in a cache.
//
// The pair (a, b) of a token at position p turns by p w: (a cos - b sin, a sin + b cos).
// p w is needed modulo one turn, and at p = 10^6 an fp32 product would be off by 0.03
// radians.  Frequencies are therefore held as turns in 64-bit fixed point: the
// wrap-around of an integer product is the reduction, exactly, and its upper 32 bits
// leave an angle within 2^-32 of a turn.  The nearest quarter turn comes off as an
// integer as well, so that Taylor's series are needed for |angle| <= pi / 4 only, where
// nine terms of both together end below 2e-9.
// Bound by memory: each element is read once and written once.  8192 tokens of 40 heads of
// 128 in bf16 (168 MB): 26 us, 0.95 of the copy bandwidth; 51 us while loads were converted one
// by one, 33 while the frequencies were kernel arguments that each lane read at its own place.
// Where halves or rows begin at odd places, all channels go pair by pair, those that are only
// copied too, and it is bound by instructions: 37 us for 34 of 128 channels of the same heads,
// 60 while places were divided and heads addressed in 64 bits.
#include "block_internal.h"

namespace ovl {
namespace {

constexpr int kThreads = 256;

// cos and sin of `phase` turns (2^-64 each), times `size`.
__device__ __forceinline__ void turned(uint64_t phase, float size, float* cosine, float* sine) {
  const uint32_t hi = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const float a = static_cast<float>(static_cast<int32_t>(hi - (quarter << 30))) * (6.283185307179586f * 0x1p-32f);
  const float z = a * a;
  float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(s, z, 1.f / 120.f);
  s = fmaf(s, z, -1.f / 6.f);
  s = fmaf(s * z, a, a);
  float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(c, z, -1.f / 720.f);
  c = fmaf(c, z, 1.f / 24.f);
  c = fmaf(c, z, -0.5f);
  c = fmaf(c, z, 1.f);
  const float u = (quarter & 1) ? s : c, v = (quarter & 1) ? c : s;
  *cosine = ((quarter + 1) & 2) ? -u * size : u * size;
  *sine = (quarter & 2) ? -v * size : v * size;
}

struct RopeArgs {
  ovl_rope rope;
  const int32_t* pos;
  uint32_t n_tokens, q_heads, heads, slots, chunks;
  Rows q, k, q_out, k_out;
};

// A thread has P pairs of one token (or 2 P channels that are passed through) and
// HT heads, for which the angles' sines are computed once.
template <int P, int HT, bool XB, bool OB>
__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ RopeArgs a) {
  __shared__ uint64_t turn[OVL_ROPE_MAX_DIM / 2];         // as a kernel argument, each lane's place would be read in turn
  griddep_launch_dependents();
  for (uint32_t j = threadIdx.x; j < a.rope.rot_dim / 2; j += kThreads) turn[j] = a.rope.turn[j];
  __syncthreads();
  griddep_wait();
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  uint32_t slot, chunk;
  uint64_t token;
  if (blockIdx.x < (1u << 24)) {                          // i < 2^32
    const uint32_t rest = static_cast<uint32_t>(i) / a.slots;
    slot = static_cast<uint32_t>(i) - rest * a.slots;
    token = rest / a.chunks;
    chunk = rest - static_cast<uint32_t>(token) * a.chunks;
  } else {
    const uint64_t rest = i / a.slots;
    slot = static_cast<uint32_t>(i - rest * a.slots);
    token = rest / a.chunks;
    chunk = static_cast<uint32_t>(rest - token * a.chunks);
  }
  static_assert(kThreads == 256, "2^24 blocks");
  if (token >= a.n_tokens) return;
  const uint32_t first = slot * P, half = a.rope.rot_dim / 2;
  const bool turns = first < half, halves = a.rope.layout == OVL_ROPE_HALF;
  // channels c0 .. and c1 ..: both halves of the pairs, or 2 P consecutive channels
  const uint32_t c0 = turns && halves ? first : 2 * first, c1 = turns && halves ? half + first : c0 + P;
  const int64_t p = a.pos[token];
  // where head 0 of the queries would begin, and of heads counted on into the keys
  auto rows = [&](const Rows& q, const Rows& k, uint32_t size, uint64_t (&at)[2]) {
    at[0] = reinterpret_cast<uint64_t>(q.ptr) + (token * q.stride + c0) * size;
    at[1] = reinterpret_cast<uint64_t>(k.ptr) + (token * k.stride + c0 - static_cast<uint64_t>(a.q_heads) * a.rope.head_dim) * size;
  };
  constexpr uint32_t kIn = XB ? 2 : 4, kOut = OB ? 2 : 4;
  const uint32_t apart = c1 - c0;
  uint64_t in[2], out[2];
  rows(a.q, a.k, kIn, in);
  rows(a.q_out, a.k_out, kOut, out);
  Raw<P> ur[HT], vr[HT];
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    const uint32_t head = chunk * HT + h;
    if (head >= a.heads) break;
    const void* from = reinterpret_cast<const void*>((head < a.q_heads ? in[0] : in[1]) + static_cast<uint64_t>(head) * (a.rope.head_dim * kIn));
    load_raw<P>(from, XB, 0, ur[h]);
    load_raw<P>(from, XB, apart, vr[h]);
  }
  float cosine[P], sine[P];
  if (turns) {
#pragma unroll
    for (int j = 0; j < P; ++j)
      turned(static_cast<uint64_t>(p) * turn[first + j], a.rope.magnitude, &cosine[j], &sine[j]);
  }
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    const uint32_t head = chunk * HT + h;
    if (head >= a.heads) break;
    float u[P], v[P];
    to_f32<P>(ur[h], XB, u);
    to_f32<P>(vr[h], XB, v);
    if (turns) {
      if (halves) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float x = u[j], y = v[j];
          u[j] = x * cosine[j] - y * sine[j];
          v[j] = x * sine[j] + y * cosine[j];
        }
      } else {
        float w[2 * P];
#pragma unroll
        for (int j = 0; j < P; ++j) w[j] = u[j], w[P + j] = v[j];
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float x = w[2 * j], y = w[2 * j + 1];
          w[2 * j] = x * cosine[j] - y * sine[j];
          w[2 * j + 1] = x * sine[j] + y * cosine[j];
        }
#pragma unroll
        for (int j = 0; j < P; ++j) u[j] = w[j], v[j] = w[P + j];
      }
    }
    void* to = reinterpret_cast<void*>((head < a.q_heads ? out[0] : out[1]) + static_cast<uint64_t>(head) * (a.rope.head_dim * kOut));
    store_f32<P>(to, OB, 0, u);
    store_f32<P>(to, OB, apart, v);
  }
}

__global__ void __launch_bounds__(kThreads) k_kv_positions(const KvDev kv, const int32_t* seqs, const int32_t* off,
                                                           uint32_t n, uint32_t n_tokens, int32_t* pos) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t t = blockIdx.x * kThreads + threadIdx.x;
  if (t >= n_tokens) return;
  const uint32_t i = kv_owner(off, n, static_cast<int32_t>(t));
  const int32_t s = seqs[i], after = off[i + 1] - static_cast<int32_t>(t);
  int32_t p = -1;
  if (static_cast<uint32_t>(s) >= kv.max_seqs || after <= 0 || off[i] > static_cast<int32_t>(t)) kv_latch(kv, OVL_E_ARG);
  else p = max(kv.length[s] - after, -1);
  pos[t] = p;
}

bool wide(const Rows& r) {
  const uint64_t lanes = r.bf16 ? 8 : 4;
  return !r.ptr || ((reinterpret_cast<uintptr_t>(r.ptr) & 15) == 0 && r.stride % lanes == 0);
}

template <int P, int HT, bool XB, bool OB>
cudaError_t launch_as(RopeArgs& a, cudaStream_t st) {
  a.slots = a.rope.head_dim / 2 / P;
  a.chunks = (a.heads + HT - 1) / HT;
  const uint64_t threads = static_cast<uint64_t>(a.n_tokens) * a.slots * a.chunks;
  return launch_chained(k_rope<P, HT, XB, OB>, dim3(static_cast<uint32_t>((threads + kThreads - 1) / kThreads)), kThreads, 0,
                        st, a);
}
template <int P, int HT>
cudaError_t launch_of(RopeArgs& a, cudaStream_t st) {
  if (a.q.bf16) return a.q_out.bf16 ? launch_as<P, HT, true, true>(a, st) : launch_as<P, HT, true, false>(a, st);
  return a.q_out.bf16 ? launch_as<P, HT, false, true>(a, st) : launch_as<P, HT, false, false>(a, st);
}

}  // namespace

cudaError_t launch_rope(const ovl_rope& rope, uint32_t n_tokens, const int32_t* pos, Rows q, uint32_t q_heads, Rows k,
                        uint32_t k_heads, Rows q_out, Rows k_out, cudaStream_t st) {
  RopeArgs a{};
  a.rope = rope;
  a.pos = pos;
  a.n_tokens = n_tokens;
  a.q_heads = q_heads;
  a.heads = q_heads + k_heads;
  a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
  const bool vec = rope.rot_dim % 8 == 0 && rope.head_dim % 8 == 0 && wide(q) && wide(k) && wide(q_out) && wide(k_out);
  // One head a thread while that leaves the SMs room for more; four, which share the
  // sines, where there is work for all of them; eight of many heads (8192 tokens of 40 heads
  // of 128: two 38, four 30, eight 27 us; of 12 heads of 96, four 8.4 and eight 9.1; pair by pair
  // 34 of 40 x 128 channels, four 55, eight and sixteen 51).
  const uint64_t singles = static_cast<uint64_t>(n_tokens) * a.heads * rope.head_dim / (vec ? 8 : 2);
  const bool few = singles <= static_cast<uint64_t>(sm_count()) * 2048;
  if (vec) return few ? launch_of<4, 1>(a, st) : a.heads >= 32 ? launch_of<4, 8>(a, st) : launch_of<4, 4>(a, st);
  return few ? launch_of<1, 1>(a, st) : a.heads >= 32 ? launch_of<1, 8>(a, st) : launch_of<1, 4>(a, st);
}

cudaError_t launch_kv_positions(const KvDev& kv, const int32_t* seqs, const int32_t* off, uint32_t n, uint32_t n_tokens,
                                int32_t* pos, cudaStream_t st) {
  return launch_chained(k_kv_positions, dim3((n_tokens + kThreads - 1) / kThreads), kThreads, 0, st, kv, seqs, off, n,
                        n_tokens, pos);
}

}  // namespace ovl
