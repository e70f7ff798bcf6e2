// The norms around a block with its gate and residual, and the gated activation.
//
//   x' = alpha x + beta gate * post(y),   h = pre(x')
// A row lives in its threads' registers from the first load to the last store, so x and y
// are read once and x' and h written once; a mean and the squares around it are two
// reductions over the registers, not a difference of two large sums.  Places behind the
// row's end hold zeros throughout.  Bound by memory.
#include "block_internal.h"

namespace ovl {
namespace {

struct NormArgs {
  ovl_block_norm norm;
  uint32_t n_tokens, row_threads;
  Rows x, y, x_out, h;
  Gate gate;
};

// Sum over the threads of a row; `red` has 2 x 32 entries, used in turn.
__device__ __forceinline__ float row_sum(float v, uint32_t row_threads, float (*red)[32], int turn) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if (row_threads == 32) return v;
  const uint32_t warps = row_threads / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (lane == 0) red[turn][warp] = v;
  __syncthreads();
  v = lane < warps ? red[turn][warp / warps * warps + lane] : 0.f;
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

template <int VEC, int NV>
__device__ __forceinline__ void normed(const ovl_norm& n, float (&v)[NV][VEC], uint32_t hidden, uint32_t c0, uint32_t row_threads,
                                       float (*red)[32], int& turn) {
  if (n.kind == OVL_NORM_NONE) return;
  const float inv = 1.f / static_cast<float>(hidden);
  if (n.kind == OVL_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += v[i][j];
    const float mean = row_sum(s, row_threads, red, turn) * inv;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = c0 + i * row_threads * VEC < hidden ? v[i][j] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s = fmaf(v[i][j], v[i][j], s);
  const float r = rsqrtf(fmaf(row_sum(s, row_threads, red, turn), inv, n.eps));
  turn ^= 1;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = c0 + i * row_threads * VEC;
    if (c >= hidden) continue;
    float w[VEC], b[VEC];
    if (n.weight) load_f32<VEC>(n.weight, n.w_dtype == OVL_BF16, c, w);
    if (n.bias) load_f32<VEC>(n.bias, n.w_dtype == OVL_BF16, c, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float z = v[i][j] * r;
      v[i][j] = n.weight ? z * (w[j] + n.offset) : z;
      if (n.bias) v[i][j] += b[j];
    }
  }
}

// A row has row_threads threads (a multiple of 32), each NV pieces of VEC channels;
// a block has blockDim / row_threads rows.
template <int VEC, int NV>
__global__ void __launch_bounds__(1024) k_block_norm(const __grid_constant__ NormArgs a) {
  __shared__ float red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t rt = a.row_threads, hidden = a.norm.hidden;
  const uint64_t token = static_cast<uint64_t>(blockIdx.x) * (blockDim.x / rt) + threadIdx.x / rt;
  const uint32_t c0 = threadIdx.x % rt * VEC;
  const bool live = token < a.n_tokens;
  int turn = 0;
  float x[NV][VEC], z[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = c0 + i * rt * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[i][j] = z[i][j] = 0.f;
    if (live && c < hidden) {
      load_f32<VEC>(a.x.ptr, a.x.bf16, token * a.x.stride + c, x[i]);
      if (a.y.ptr) load_f32<VEC>(a.y.ptr, a.y.bf16, token * a.y.stride + c, z[i]);
    }
  }
  uint32_t row = 0;
  bool joins = live && a.y.ptr != nullptr;
  if (joins && a.gate.rows.ptr) {
    row = a.gate.row ? static_cast<uint32_t>(a.gate.row[token]) : a.gate.n == 1 ? 0u : static_cast<uint32_t>(token);
    joins = row < a.gate.n;
  }
  if (a.y.ptr) normed<VEC, NV>(a.norm.post, z, hidden, c0, rt, red, turn);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = c0 + i * rt * VEC;
    float g[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[j] = a.norm.beta;
    if (joins && a.gate.rows.ptr && c < hidden) {
      load_f32<VEC>(a.gate.rows.ptr, a.gate.rows.bf16, row * a.gate.rows.stride + c, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) g[j] *= a.norm.beta;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      x[i][j] *= a.norm.alpha;
      if (joins) x[i][j] = fmaf(g[j], z[i][j], x[i][j]);
    }
    if (live && c < hidden && a.x_out.ptr) store_f32<VEC>(a.x_out.ptr, a.x_out.bf16, token * a.x_out.stride + c, x[i]);
  }
  if (!a.h.ptr) return;
  normed<VEC, NV>(a.norm.pre, x, hidden, c0, rt, red, turn);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = c0 + i * rt * VEC;
    if (live && c < hidden) store_f32<VEC>(a.h.ptr, a.h.bf16, token * a.h.stride + c, x[i]);
  }
}

struct GluArgs {
  uint64_t width;
  uint32_t n_tokens;
  Rows gate, up, out;
};

template <int VEC, uint32_t ACT>
__global__ void __launch_bounds__(256) k_glu(const __grid_constant__ GluArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const uint64_t c = (static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x) * VEC;
  if (c >= a.width) return;
  for (uint64_t t = blockIdx.y; t < a.n_tokens; t += gridDim.y) {
    float g[VEC], u[VEC];
    load_f32<VEC>(a.gate.ptr, a.gate.bf16, t * a.gate.stride + c, g);
    load_f32<VEC>(a.up.ptr, a.up.bf16, t * a.up.stride + c, u);
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[j] = activated(g[j], ACT) * u[j];
    store_f32<VEC>(a.out.ptr, a.out.bf16, t * a.out.stride + c, g);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool wide(const Rows& r) { return aligned16(r.ptr) && r.stride % (r.bf16 ? 8 : 4) == 0; }

template <int VEC, int NV>
cudaError_t norm_as(NormArgs& a, cudaStream_t st) {
  const uint32_t pieces = (a.norm.hidden + VEC - 1) / VEC, threads = (pieces + NV - 1) / NV;
  a.row_threads = (threads + 31) / 32 * 32;
  if (a.row_threads == 96) a.row_threads = 128;
  const uint32_t block = a.row_threads < 128 ? 128 : a.row_threads, rows = block / a.row_threads;
  return launch_chained(k_block_norm<VEC, NV>, dim3((a.n_tokens + rows - 1) / rows), block, 0, st, a);
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
  if (vec) {
    if (norm.hidden <= 8192) return norm_as<8, 1>(a, st);
    return norm_as<8, 4>(a, st);
  }
  if (norm.hidden <= 4096) return norm_as<1, 4>(a, st);
  return norm_as<1, 32>(a, st);
}

cudaError_t launch_glu(uint32_t act, uint32_t n_tokens, uint32_t width, Rows gate, Rows up, Rows out, cudaStream_t st) {
  GluArgs a{width, n_tokens, gate, up, out};
  if (gate.stride == width && up.stride == width && out.stride == width) {     // one long row
    a.width = static_cast<uint64_t>(width) * n_tokens;
    a.n_tokens = 1;
  }
  const bool vec = a.width % 8 == 0 && wide(gate) && wide(up) && wide(out);
  if (a.n_tokens == 1 && vec) return glu_as<8>(act, a, st);
  return vec ? glu_as<8>(act, a, st) : glu_as<1>(act, a, st);
}

}  // namespace ovl
