// The norms around a block with its gate and residual, and the gated activation.
//
//   x' = alpha x + beta gate * post(y),   h = pre(x')
// A row lives in its threads' registers from the first load to the last store, so x and y
// are read once and x' and h written once; a mean and the squares around it are two
// reductions over the registers, not a difference of two large sums.  Places behind the
// row's end hold zeros throughout.  Bound by memory, with the instructions close behind:
// types and the threads of a row are template arguments (63 instructions an element where
// they were not), and a thread has 16 elements where the width allows it.
#include <atomic>

#include "block_internal.h"

namespace ovl {
namespace {

struct NormArgs {
  ovl_block_norm norm;
  uint32_t n_tokens;
  Rows x, y, x_out, h;
  Gate gate;
};

// Sum over the RT threads of a row, each warp's by exchanges, the warps' through shared memory.
template <int RT>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int turn) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if constexpr (RT > 32) {
    constexpr int kWarps = RT / 32;
    const uint32_t warp = threadIdx.x / 32;
    if ((threadIdx.x & 31) == 0) red[turn][warp] = v;
    __syncthreads();
    const float* mine = red[turn] + warp / kWarps * kWarps;
    float part[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (kWarps % 4 == 0) {
#pragma unroll
      for (int w = 0; w < kWarps; w += 4) {
        const float4 f = *reinterpret_cast<const float4*>(mine + w);
        part[0] += f.x, part[1] += f.y, part[2] += f.z, part[3] += f.w;
      }
    } else {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) part[w & 3] += mine[w];
    }
    v = (part[0] + part[1]) + (part[2] + part[3]);
  }
  return v;
}

// v becomes its norm.
template <int VEC, int NV, int RT>
__device__ __forceinline__ void normed(const ovl_norm& n, float (&v)[NV][VEC], uint32_t hidden, float inv, uint32_t c0,
                                       float (*red)[32], int& turn) {
  if (n.kind == OVL_NORM_NONE) return;
  const bool bf16 = n.w_dtype == OVL_BF16;
  if (n.kind == OVL_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += v[i][j];
    const float mean = row_sum<RT>(s, red, turn) * inv;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = c0 + i * RT * VEC < hidden ? v[i][j] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s = fmaf(v[i][j], v[i][j], s);
  // few pieces: asked for before the others of the row are waited for
  constexpr bool kEarly = VEC * NV <= 16;
  Raw<VEC> w[kEarly ? NV : 1];
  if constexpr (kEarly) {
    if (n.weight) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c0 + i * RT * VEC < hidden) load_raw<VEC>(n.weight, bf16, c0 + i * RT * VEC, w[i]);
    }
  }
  const float r = rsqrtf(fmaf(row_sum<RT>(s, red, turn), inv, n.eps));
  turn ^= 1;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = c0 + i * RT * VEC;
    if (c >= hidden) continue;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] *= r;
    float u[VEC];
    if (n.weight) {
      if constexpr (!kEarly) load_raw<VEC>(n.weight, bf16, c, w[0]);
      to_f32<VEC>(w[kEarly ? i : 0], bf16, u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] *= u[j] + n.offset;
    }
    if (n.bias) {
      load_f32<VEC>(n.bias, bf16, c, u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] += u[j];
    }
  }
}

// One tensor's part of a row in shared memory: a thread asks for the pieces that it takes
// itself, so no barrier is needed.  Pieces lie 16 bytes a thread apart.
template <int NV, int RT, bool BF16>
struct Ahead {
  static constexpr uint32_t kBytes = NV * (BF16 ? 1 : 2) * RT * 16;
  static __device__ __forceinline__ void ask(uint8_t* at, const void* row, uint32_t c0, uint32_t hidden) {
    const uint8_t* from = static_cast<const uint8_t*>(row) + c0 * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (c0 + i * RT * 8 >= hidden) break;
      if constexpr (BF16) {
        cp_async16(at + i * RT * 16, from + i * RT * 16);
      } else {
        cp_async16(at + 2 * i * RT * 16, from + i * RT * 32);
        cp_async16(at + (2 * i + 1) * RT * 16, from + i * RT * 32 + 16);
      }
    }
  }
  static __device__ __forceinline__ void take(const uint8_t* at, uint32_t c0, uint32_t hidden, float (&v)[NV][8]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      if (c0 + i * RT * 8 >= hidden) continue;
      Raw<8> r;
      const uint4 a = *reinterpret_cast<const uint4*>(at + (BF16 ? i : 2 * i) * RT * 16);
      r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
      if constexpr (!BF16) {
        const uint4 b = *reinterpret_cast<const uint4*>(at + (2 * i + 1) * RT * 16);
        r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
      }
      to_f32<8>(r, BF16, v[i]);
    }
  }
};

// What is left of a row once x and y are there.  `row`: of the gate; joins: whether there is a y.
template <int VEC, int NV, int RT>
__device__ __forceinline__ void rest_of_row(const NormArgs& a, float (&x)[NV][VEC], float (&z)[NV][VEC], uint64_t token, bool live,
                                            bool x_bf16, bool h_bf16, float inv, uint32_t c0, float (*red)[32], int& turn) {
  const uint32_t hidden = a.norm.hidden;
  uint32_t row = 0;
  bool joins = live && a.y.ptr != nullptr;
  if (joins && a.gate.rows.ptr) {
    row = a.gate.row ? static_cast<uint32_t>(a.gate.row[token]) : a.gate.n == 1 ? 0u : static_cast<uint32_t>(token);
    joins = row < a.gate.n;
  }
  if (a.y.ptr) normed<VEC, NV, RT>(a.norm.post, z, hidden, inv, c0, red, turn);
  const uint64_t g0 = row * a.gate.rows.stride + c0, x0 = token * a.x_out.stride + c0, h0 = token * a.h.stride + c0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = live && c0 + i * RT * VEC < hidden;
    if (joins) {
      if (a.gate.rows.ptr && in) {
        float g[VEC];
        load_f32<VEC>(a.gate.rows.ptr, a.gate.rows.bf16, g0 + i * RT * VEC, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[i][j] = fmaf(a.norm.beta, z[i][j], a.norm.alpha * x[i][j]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[i][j] *= a.norm.alpha;
    }
    if (in && a.x_out.ptr) store_f32<VEC>(a.x_out.ptr, x_bf16, x0 + i * RT * VEC, x[i]);
  }
  if (!a.h.ptr) return;
  normed<VEC, NV, RT>(a.norm.pre, x, hidden, inv, c0, red, turn);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (live && c0 + i * RT * VEC < hidden) store_f32<VEC>(a.h.ptr, h_bf16, h0 + i * RT * VEC, x[i]);
}

// A thread's pieces of a row that begins at `at`; the type is looked at once.
template <int VEC, int NV, int RT>
__device__ __forceinline__ void load_row(const void* base, bool bf16, uint64_t at, const bool (&in)[NV], Raw<VEC> (&r)[NV]) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) load_raw<VEC>(base, true, at + i * RT * VEC, r[i]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) load_raw<VEC>(base, false, at + i * RT * VEC, r[i]);
  }
}
template <int VEC, int NV>
__device__ __forceinline__ void row_f32(const Raw<VEC> (&r)[NV], bool bf16, float (&v)[NV][VEC]) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < NV; ++i) to_f32<VEC>(r[i], true, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) to_f32<VEC>(r[i], false, v[i]);
  }
}

template <int VEC, int NV, int RT>
__device__ __forceinline__ void store_row(void* base, bool bf16, uint64_t at, const bool (&in)[NV], const float (&v)[NV][VEC]) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) store_f32<VEC>(base, true, at + i * RT * VEC, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) store_f32<VEC>(base, false, at + i * RT * VEC, v[i]);
  }
}

// A norm's weights of a thread, ready to multiply with.
template <int VEC, int NV, int RT>
__device__ __forceinline__ void weights_of(const ovl_norm& n, const bool (&in)[NV], uint32_t c0, float (&w)[NV][VEC]) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = 1.f;
  if (n.kind == OVL_NORM_NONE || !n.weight) return;
  Raw<VEC> r[NV] = {};
  load_row<VEC, NV, RT>(n.weight, n.w_dtype == OVL_BF16, c0, in, r);
  row_f32<VEC, NV>(r, n.w_dtype == OVL_BF16, w);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] += n.offset;
}
// And its biases; none are zeros.
template <int VEC, int NV, int RT>
__device__ __forceinline__ void biases_of(const ovl_norm& n, const bool (&in)[NV], uint32_t c0, float (&b)[NV][VEC]) {
  Raw<VEC> r[NV] = {};
  if (n.kind != OVL_NORM_NONE && n.bias) load_row<VEC, NV, RT>(n.bias, n.w_dtype == OVL_BF16, c0, in, r);
  row_f32<VEC, NV>(r, n.w_dtype == OVL_BF16, b);
}

// v becomes its norm, with the weights at hand (KEEP: and the biases `b`).
template <int VEC, int NV, int RT, bool KEEP>
__device__ __forceinline__ void normed_by(const ovl_norm& n, float (&v)[NV][VEC], const float (&w)[NV][VEC],
                                          const float (&b)[KEEP ? NV : 1][VEC], const bool (&in)[NV],
                                          float inv, uint32_t c0, float (*red)[32], int& turn) {
  if (n.kind == OVL_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += v[i][j];
    const float mean = row_sum<RT>(s, red, turn) * inv;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = in[i] ? v[i][j] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s = fmaf(v[i][j], v[i][j], s);
  const float r = rsqrtf(fmaf(row_sum<RT>(s, red, turn), inv, n.eps));
  turn ^= 1;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] = KEEP ? fmaf(v[i][j] * r, w[i][j], b[KEEP ? i : 0][j]) : v[i][j] * r * w[i][j];
  if (!KEEP && n.bias) {
    Raw<VEC> raw[NV] = {};
    float bias[NV][VEC];
    load_row<VEC, NV, RT>(n.bias, n.w_dtype == OVL_BF16, c0, in, raw);
    row_f32<VEC, NV>(raw, n.w_dtype == OVL_BF16, bias);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] += bias[i][j];
  }
}

// RT threads have a row of NV * VEC * RT channels at most; a block has THREADS / RT rows at a
// time and goes on to others.  The weights stay in registers.  SLOTS > 0 (pieces of 16
// bytes): that many rows, the one at work included, are under way in shared memory; else
// the next one in registers, and types are looked at once a row and not XB, YB and HB.
template <int VEC, int NV, int RT, int THREADS, int SLOTS, int BLOCKS, bool XB, bool YB, bool HB>
__global__ void __launch_bounds__(THREADS, BLOCKS) k_block_norm(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[2][32];
  using X = Ahead<NV, RT, XB>;
  using Y = Ahead<NV, RT, YB>;
  constexpr uint32_t kRows = THREADS / RT, kSlot = X::kBytes + Y::kBytes;
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t hidden = a.norm.hidden, c0 = threadIdx.x % RT * VEC;
  const bool xb = SLOTS > 0 ? XB : a.x.bf16, yb = SLOTS > 0 ? YB : a.y.bf16, hb = SLOTS > 0 ? HB : a.h.bf16;
  const float inv = 1.f / static_cast<float>(hidden);
  uint64_t token = static_cast<uint64_t>(blockIdx.x) * kRows + threadIdx.x / RT;
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRows;
  const uint8_t *xp = static_cast<const uint8_t*>(a.x.ptr), *yp = static_cast<const uint8_t*>(a.y.ptr);
  [[maybe_unused]] uint8_t* mine = smem + threadIdx.x / RT * (SLOTS * kSlot) + threadIdx.x % RT * 16;
  [[maybe_unused]] auto ask = [&](uint64_t t, uint32_t slot) {
    if constexpr (SLOTS > 0) {
      if (t < a.n_tokens) {
        if (yp) Y::ask(mine + slot * kSlot + X::kBytes, yp + t * a.y.stride * (YB ? 2 : 4), c0, hidden);
        X::ask(mine + slot * kSlot, xp + t * a.x.stride * (XB ? 2 : 4), c0, hidden);
      }
      cp_async_commit();
    }
  };
#pragma unroll
  for (int i = 0; i < SLOTS - 1; ++i) ask(token + i * step, i);
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = c0 + i * RT * VEC < hidden;
  float wy[NV][VEC], wx[NV][VEC];
  weights_of<VEC, NV, RT>(a.norm.post, in, c0, wy);
  weights_of<VEC, NV, RT>(a.norm.pre, in, c0, wx);
  constexpr bool kKeep = VEC * NV <= 10;                 // where registers are left: the biases too, and gates early
  float by[kKeep ? NV : 1][VEC], bx[kKeep ? NV : 1][VEC];
  if constexpr (kKeep) {
    biases_of<VEC, NV, RT>(a.norm.post, in, c0, by);
    biases_of<VEC, NV, RT>(a.norm.pre, in, c0, bx);
  }
  [[maybe_unused]] Raw<VEC> xr[NV], yr[NV];             // SLOTS = 0: the next row
  [[maybe_unused]] auto load = [&](uint64_t t) {
    const uint64_t x0 = t * a.x.stride + c0, y0 = t * a.y.stride + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) xr[i].w[j] = yr[i].w[j] = 0;
    }
    if (t < a.n_tokens) {
      load_row<VEC, NV, RT>(xp, xb, x0, in, xr);
      if (yp) load_row<VEC, NV, RT>(yp, yb, y0, in, yr);
    }
  };
  if constexpr (SLOTS == 0) load(token);
  auto gate_of = [&](uint64_t t) -> uint32_t {            // the token's row of the gates; none: outside
    if (!a.gate.rows.ptr || t >= a.n_tokens) return 0;
    return a.gate.row ? static_cast<uint32_t>(a.gate.row[t]) : a.gate.n == 1 ? 0u : static_cast<uint32_t>(t);
  };
  uint32_t row_then = gate_of(token);
  uint32_t slot = 0;
  int turn = 0;
  // as many rounds for every thread of the block
  for (uint64_t first = static_cast<uint64_t>(blockIdx.x) * kRows; first < a.n_tokens; first += step, token += step) {
    const bool live = kRows == 1 || token < a.n_tokens;
    float x[NV][VEC], z[NV][VEC];
    if constexpr (SLOTS > 0) {
      ask(token + (SLOTS - 1) * step, slot ? slot - 1 : SLOTS - 1);        // where the last row was
      asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
      Y::take(mine + slot * kSlot + X::kBytes, c0, live && yp ? hidden : 0, z);
      X::take(mine + slot * kSlot, c0, live ? hidden : 0, x);
      slot = slot + 1 == SLOTS ? 0 : slot + 1;
    } else {
      row_f32<VEC, NV>(xr, xb, x);
      row_f32<VEC, NV>(yr, yb, z);
      load(token + step);
    }
    const uint32_t row = row_then;
    row_then = gate_of(token + step);
    const bool gated = live && yp && a.gate.rows.ptr && row < a.gate.n, joins = live && yp && (gated || !a.gate.rows.ptr);
    Raw<VEC> gr[NV] = {};
    const uint64_t g0 = row * a.gate.rows.stride + c0;
    if (kKeep && gated) load_row<VEC, NV, RT>(a.gate.rows.ptr, a.gate.rows.bf16, g0, in, gr);
    if (yp && a.norm.post.kind != OVL_NORM_NONE) normed_by<VEC, NV, RT, kKeep>(a.norm.post, z, wy, by, in, inv, c0, red, turn);
    if (gated) {
      float g[NV][VEC];
      if (!kKeep) load_row<VEC, NV, RT>(a.gate.rows.ptr, a.gate.rows.bf16, g0, in, gr);
      row_f32<VEC, NV>(gr, a.gate.rows.bf16, g);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[i][j] = in[i] ? z[i][j] * g[i][j] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[i][j] = a.norm.alpha * x[i][j] + (joins ? a.norm.beta * z[i][j] : 0.f);
    if (live && a.x_out.ptr) store_row<VEC, NV, RT>(a.x_out.ptr, xb, token * a.x_out.stride + c0, in, x);
    if (!a.h.ptr) continue;
    normed_by<VEC, NV, RT, kKeep>(a.norm.pre, x, wx, bx, in, inv, c0, red, turn);
    if (live) store_row<VEC, NV, RT>(a.h.ptr, hb, token * a.h.stride + c0, in, x);
  }
  if constexpr (SLOTS > 0) cp_async_wait_all();
}

// Wide rows, of any type: a block of RT threads has one at a time.
template <int VEC, int NV, int RT, int BLOCKS>
__global__ void __launch_bounds__(RT, BLOCKS) k_block_norm_any(const __grid_constant__ NormArgs a) {
  __shared__ __align__(16) float red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t hidden = a.norm.hidden, c0 = threadIdx.x * VEC;
  const float inv = 1.f / static_cast<float>(hidden);
  int turn = 0;
  for (uint64_t token = blockIdx.x; token < a.n_tokens; token += gridDim.x) {
    Raw<VEC> xr[NV], yr[NV];
    const uint64_t x0 = token * a.x.stride + c0, y0 = token * a.y.stride + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) xr[i].w[j] = yr[i].w[j] = 0;
      if (c0 + i * RT * VEC < hidden) {
        load_raw<VEC>(a.x.ptr, a.x.bf16, x0 + i * RT * VEC, xr[i]);
        if (a.y.ptr) load_raw<VEC>(a.y.ptr, a.y.bf16, y0 + i * RT * VEC, yr[i]);
      }
    }
    float x[NV][VEC], z[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) to_f32<VEC>(xr[i], a.x.bf16, x[i]), to_f32<VEC>(yr[i], a.y.bf16, z[i]);
    rest_of_row<VEC, NV, RT>(a, x, z, token, true, a.x.bf16, a.h.bf16, inv, c0, red, turn);
  }
}

struct GluArgs {
  uint64_t width;
  uint32_t n_tokens;
  Rows gate, up, out;
};

// Rows that begin at odd addresses, element by element: a thread has PER of them, 256 apart,
// with all loads under way before the first is looked at, and types looked at once for all.
// bf16, 4095 rows of 14335 (352 MB): 86 us with 8, 94 with 4, 82 with 16, 239 with one; 3333 rows of
// 333, fp32 to bf16: 2.7 with 2, 3.0 with 4, 3.4 with one.
template <int PER, uint32_t ACT>
__global__ void __launch_bounds__(256) k_glu_odd(const __grid_constant__ GluArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const uint64_t c = static_cast<uint64_t>(blockIdx.x) * (256 * PER) + threadIdx.x;
  bool in[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) in[i] = c + i * 256 < a.width;
  for (uint64_t t = blockIdx.y; t < a.n_tokens; t += gridDim.y) {
    Raw<1> gr[PER] = {}, ur[PER] = {};
    float g[PER][1], u[PER][1];
    load_row<1, PER, 256>(a.gate.ptr, a.gate.bf16, t * a.gate.stride + c, in, gr);
    load_row<1, PER, 256>(a.up.ptr, a.up.bf16, t * a.up.stride + c, in, ur);
    row_f32<1, PER>(gr, a.gate.bf16, g);
    row_f32<1, PER>(ur, a.up.bf16, u);
#pragma unroll
    for (int i = 0; i < PER; ++i) g[i][0] = activated(g[i][0], ACT) * u[i][0];
    store_row<1, PER, 256>(a.out.ptr, a.out.bf16, t * a.out.stride + c, in, g);
  }
}

template <int VEC, uint32_t ACT>
__global__ void __launch_bounds__(256) k_glu(const __grid_constant__ GluArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const uint64_t c = (static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x) * VEC;
  if (c >= a.width) return;
  for (uint64_t t = blockIdx.y; t < a.n_tokens; t += gridDim.y) {
    Raw<VEC> gr, ur;
    float g[VEC], u[VEC];
    load_raw<VEC>(a.gate.ptr, a.gate.bf16, t * a.gate.stride + c, gr);
    load_raw<VEC>(a.up.ptr, a.up.bf16, t * a.up.stride + c, ur);
    to_f32<VEC>(gr, a.gate.bf16, g);
    to_f32<VEC>(ur, a.up.bf16, u);
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[j] = activated(g[j], ACT) * u[j];
    store_f32<VEC>(a.out.ptr, a.out.bf16, t * a.out.stride + c, g);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool wide(const Rows& r) { return aligned16(r.ptr) && r.stride % (r.bf16 ? 8 : 4) == 0; }

template <int VEC, int NV, int RT, int THREADS, int SLOTS, int BLOCKS, bool XB, bool YB, bool HB>
cudaError_t norm_as(const NormArgs& a, cudaStream_t st) {
  constexpr uint32_t kRows = THREADS / RT, kSmem = kRows * SLOTS * (Ahead<NV, RT, XB>::kBytes + Ahead<NV, RT, YB>::kBytes);
  auto kernel = k_block_norm<VEC, NV, RT, THREADS, SLOTS, BLOCKS, XB, YB, HB>;
  if constexpr (kSmem > 0) {
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kSmem, &allowed);
    if (e != cudaSuccess) return e;
  }
  const uint32_t fit = sm_count() * BLOCKS, want = (a.n_tokens + kRows - 1) / kRows;
  return launch_chained(kernel, dim3(want < fit ? want : fit), THREADS, kSmem, st, a);
}
template <int VEC, int NV, int RT, int THREADS, int SLOTS, int BLOCKS>
cudaError_t norm_of(const NormArgs& a, cudaStream_t st) {
  switch ((a.x.bf16 ? 4 : 0) | (a.y.bf16 ? 2 : 0) | (a.h.bf16 ? 1 : 0)) {
    case 0: return norm_as<VEC, NV, RT, THREADS, SLOTS, BLOCKS, false, false, false>(a, st);
    case 1: return norm_as<VEC, NV, RT, THREADS, SLOTS, BLOCKS, false, false, true>(a, st);
    case 2: return norm_as<VEC, NV, RT, THREADS, SLOTS, BLOCKS, false, true, false>(a, st);
    case 3: return norm_as<VEC, NV, RT, THREADS, SLOTS, BLOCKS, false, true, true>(a, st);
    case 4: return norm_as<VEC, NV, RT, THREADS, SLOTS, BLOCKS, true, false, false>(a, st);
    case 5: return norm_as<VEC, NV, RT, THREADS, SLOTS, BLOCKS, true, false, true>(a, st);
    case 6: return norm_as<VEC, NV, RT, THREADS, SLOTS, BLOCKS, true, true, false>(a, st);
    default: return norm_as<VEC, NV, RT, THREADS, SLOTS, BLOCKS, true, true, true>(a, st);
  }
}
template <int NV, int RT, int THREADS, int BLOCKS>
cudaError_t norm_odd(const NormArgs& a, cudaStream_t st) {
  return norm_as<1, NV, RT, THREADS, 0, BLOCKS, false, false, false>(a, st);
}
template <int VEC, int NV, int RT, int BLOCKS>
cudaError_t norm_any(const NormArgs& a, cudaStream_t st) {
  const uint32_t fit = sm_count() * BLOCKS;
  return launch_chained(k_block_norm_any<VEC, NV, RT, BLOCKS>, dim3(a.n_tokens < fit ? a.n_tokens : fit), RT, 0, st, a);
}

template <int PER>
cudaError_t glu_odd(uint32_t act, const GluArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<uint32_t>((a.width + 256 * PER - 1) / (256 * PER)), a.n_tokens < 65535 ? a.n_tokens : 65535);
  switch (act) {
    case OVL_ACT_SILU: return launch_chained(k_glu_odd<PER, OVL_ACT_SILU>, grid, 256, 0, st, a);
    case OVL_ACT_GELU: return launch_chained(k_glu_odd<PER, OVL_ACT_GELU>, grid, 256, 0, st, a);
    case OVL_ACT_GELU_TANH: return launch_chained(k_glu_odd<PER, OVL_ACT_GELU_TANH>, grid, 256, 0, st, a);
    default: return launch_chained(k_glu_odd<PER, OVL_ACT_RELU>, grid, 256, 0, st, a);
  }
}
template <int VEC>
cudaError_t glu_as(uint32_t act, const GluArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<uint32_t>((a.width + 256 * VEC - 1) / (256 * VEC)), a.n_tokens < 65535 ? a.n_tokens : 65535);
  switch (act) {
    case OVL_ACT_SILU: return launch_chained(k_glu<VEC, OVL_ACT_SILU>, grid, 256, 0, st, a);
    case OVL_ACT_GELU: return launch_chained(k_glu<VEC, OVL_ACT_GELU>, grid, 256, 0, st, a);
    case OVL_ACT_GELU_TANH: return launch_chained(k_glu<VEC, OVL_ACT_GELU_TANH>, grid, 256, 0, st, a);
    default: return launch_chained(k_glu<VEC, OVL_ACT_RELU>, grid, 256, 0, st, a);
  }
}

}  // namespace

cudaError_t launch_block_norm(const ovl_block_norm& norm, uint32_t n_tokens, Rows x, Rows y, Gate gate, Rows x_out,
                              Rows h, cudaStream_t st) {
  NormArgs a{};
  a.norm = norm;
  a.n_tokens = n_tokens;
  a.x = x, a.y = y, a.x_out = x_out, a.h = h;
  a.gate = gate;
  const bool vec = norm.hidden % 8 == 0 && wide(x) && wide(y) && wide(x_out) && wide(h) && wide(gate.rows) &&
                   aligned16(norm.post.weight) && aligned16(norm.post.bias) && aligned16(norm.pre.weight) &&
                   aligned16(norm.pre.bias);
  // 8 channels a piece where rows and widths allow it, 16 a thread, so that the fewest warps
  // share a row; one warp alone needs no barrier.  8192 rows of 4096, x bf16, y fp32, both norms
  // (336 MB): 64 us, 0.79 of the copy bandwidth; with 8 channels a thread and 512 threads 80, three
  // blocks an SM (80 registers) 76, 32 channels and 128 threads 111, and 91 before types and row
  // lengths were template arguments.  20001 rows of 128 like these: a warp a row 9 us, two 22; 5001
  // of 2048: four warps 21.6, eight 27.
  // Element by element for other rows, 5 to 20 channels a thread and types looked at once a row: these
  // are bound by instructions and by the exchanges of a row's sums.  fp32 rows with gates, layer
  // norms and biases: 20001 of 299, a warp a row 19 us (eight warps 87); 3001 of 1155, four
  // warps 12 (eight 15); 2003 of 4095, eight warps 37 (sixteen 67).
  // Rows above 8192 have 32 channels of two tensors a thread in 64 registers, and spill: 952 bytes a
  // thread, odd rows 236.  2048 rows of 16384, x bf16 and y fp32, 196 us (50 of bytes), of 12288 172
  // (38), of 9001 286 (28).
  if (vec) {
    if (norm.hidden <= 256) return norm_of<8, 1, 32, 256, 3, 2>(a, st);
    if (norm.hidden <= 512) return norm_of<8, 2, 32, 256, 3, 2>(a, st);
    if (norm.hidden <= 1024) return norm_of<8, 2, 64, 256, 3, 2>(a, st);
    if (norm.hidden <= 2048) return norm_of<8, 2, 128, 256, 3, 2>(a, st);
    if (norm.hidden <= 4096) return norm_of<8, 2, 256, 256, 3, 2>(a, st);
    if (norm.hidden <= 8192) return norm_of<8, 2, 512, 512, 3, 1>(a, st);
    return norm_any<8, 4, 1024, 1>(a, st);
  }
  if (norm.hidden <= 160) return norm_odd<5, 32, 256, 3>(a, st);
  if (norm.hidden <= 320) return norm_odd<10, 32, 128, 4>(a, st);
  if (norm.hidden <= 640) return norm_odd<20, 32, 128, 3>(a, st);
  if (norm.hidden <= 1280) return norm_odd<10, 128, 128, 4>(a, st);
  if (norm.hidden <= 2048) return norm_odd<16, 128, 128, 4>(a, st);
  if (norm.hidden <= 4096) return norm_odd<16, 256, 256, 2>(a, st);
  if (norm.hidden <= 8192) return norm_odd<16, 512, 512, 1>(a, st);
  return norm_any<1, 32, 1024, 1>(a, st);
}

cudaError_t launch_glu(uint32_t act, uint32_t n_tokens, uint32_t width, Rows gate, Rows up, Rows out, cudaStream_t st) {
  // One long row, if contiguous, has only its end at no multiple of 8; it goes to the kernel for
  // odd rows as a whole then, like rows that begin at any address.
  GluArgs a{width, n_tokens, gate, up, out};
  if (gate.stride == width && up.stride == width && out.stride == width) {     // one long row
    a.width = static_cast<uint64_t>(width) * n_tokens;
    a.n_tokens = 1;
  }
  const bool vec = a.width % 8 == 0 && wide(gate) && wide(up) && wide(out);
  if (vec) return glu_as<8>(act, a, st);
  return a.width > 1024 ? glu_odd<8>(act, a, st) : glu_odd<2>(act, a, st);
}

}  // namespace ovl
