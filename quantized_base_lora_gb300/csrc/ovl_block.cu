// The entry points of what a decoder block computes between its projections:
// argument checks and launches.  Nothing is kept between calls.
#include <cmath>
#include <cstring>
#include <string>

#include "block_internal.h"
#include "ovl_internal.h"

namespace ovl {

namespace {

ovl_status fail(ovl_status st, const char* msg) {
  try {
    set_context_free_error(msg);
  } catch (...) {
  }
  return st;
}

ovl_status done(cudaError_t e) {
  if (e == cudaSuccess) return OVL_OK;
  cudaGetLastError();
  return fail(OVL_E_CUDA, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dtype_ok(uint32_t d) { return d == OVL_F32 || d == OVL_BF16; }
uint64_t up256(uint64_t v) { return (v + 255) & ~static_cast<uint64_t>(255); }

constexpr uint64_t kMaxStride = 1ull << 31;      // elements: 2^31 tokens of it stay within 64 bits of bytes

// A tensor argument: `width` elements a token.
ovl_status check_rows(const char* what, const void* p, uint32_t dtype, uint64_t stride, uint64_t width, uint32_t n) {
  if (!p) return fail(OVL_E_ARG, what);
  if (!aligned(p, dtype == OVL_BF16 ? 2 : 4)) return fail(OVL_E_SHAPE, what);
  if ((n > 1 && stride < width) || stride > kMaxStride) return fail(OVL_E_SHAPE, what);
  return OVL_OK;
}
Rows rows_of(const void* p, uint32_t dtype, uint64_t stride) {
  return Rows{const_cast<void*>(p), stride, dtype == OVL_BF16};
}

ovl_status check_norm(const ovl_norm& n) {
  if (n.kind > OVL_NORM_LAYER) return fail(OVL_E_ARG, "unknown norm");
  if (n.kind == OVL_NORM_NONE) return OVL_OK;
  if ((n.weight || n.bias) && !dtype_ok(n.w_dtype)) return fail(OVL_E_ARG, "w_dtype must be OVL_F32 or OVL_BF16");
  if (!std::isfinite(n.eps) || n.eps < 0 || !std::isfinite(n.offset)) return fail(OVL_E_ARG, "eps or offset of a norm");
  const uintptr_t a = n.w_dtype == OVL_BF16 ? 2 : 4;
  if ((n.weight && !aligned(n.weight, a)) || (n.bias && !aligned(n.bias, a)))
    return fail(OVL_E_SHAPE, "weight and bias need their type's alignment");
  return OVL_OK;
}

// Offsets of a mixture of experts' workspace.
struct MoeLayout {
  uint64_t logits, choice, weight, power, xp, hp, part, total;
};
constexpr uint32_t kMoeHead = 256;               // counters of arrivals
static_assert(4 * kMoeGroups <= kMoeHead, "a word for each group of tokens");

ovl_status check_moe_dims(const ovl_moe* m) {
  if (!m) return fail(OVL_E_ARG, "moe is null");
  if (m->quant != OVL_Q8_0 && m->quant != OVL_Q4_0 && m->quant != OVL_Q4_K) return fail(OVL_E_QUANT, "unknown quant");
  if (!m->n_experts || m->n_experts > OVL_MOE_MAX_EXPERTS) return fail(OVL_E_ARG, "n_experts out of range");
  if (!m->top_k || m->top_k > OVL_MOE_MAX_TOP || m->top_k > m->n_experts) return fail(OVL_E_ARG, "top_k out of range");
  const uint32_t unit = m->quant == OVL_Q4_K ? 256 : 32;
  if (!m->hidden || !m->ffn || m->hidden % unit || m->ffn % unit || m->hidden > OVL_MOE_MAX_HIDDEN ||
      m->ffn > OVL_MOE_MAX_HIDDEN)
    return fail(OVL_E_SHAPE, "hidden and ffn must be multiples of the format's block up to OVL_MOE_MAX_HIDDEN");
  if (m->act < OVL_ACT_SILU || m->act > OVL_ACT_RELU) return fail(OVL_E_ARG, "unknown act");
  if (!m->max_tokens || m->max_tokens > OVL_MOE_MAX_TOKENS) return fail(OVL_E_ARG, "max_tokens must be 1..OVL_MOE_MAX_TOKENS");
  return OVL_OK;
}

MoeLayout moe_layout(const ovl_moe* m) {
  MoeLayout l{};
  const uint64_t t = m->max_tokens, p = t * m->top_k;
  l.logits = kMoeHead;
  l.choice = l.logits + up256(4 * t * m->n_experts);
  l.weight = l.choice + up256(4 * p);
  l.power = l.weight + up256(4 * p);
  l.xp = l.power + up256(4 * t);
  l.hp = l.xp + up256(6 * t * m->hidden);
  l.part = l.hp + up256(6 * p * m->ffn);
  l.total = l.part + up256(4 * p * m->hidden);
  return l;
}

}  // namespace
}  // namespace ovl

using namespace ovl;

extern "C" {

ovl_status ovl_rope_plan(uint32_t head_dim, uint32_t rot_dim, uint32_t layout, double base, uint32_t scaling,
                         double factor, uint32_t original, double low, double high, double magnitude, ovl_rope* out) {
  if (!out) return fail(OVL_E_ARG, "out is null");
  if (head_dim < 2 || head_dim > OVL_ROPE_MAX_DIM || head_dim % 2 || rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
    return fail(OVL_E_SHAPE, "head_dim and rot_dim must be even, rot_dim <= head_dim <= OVL_ROPE_MAX_DIM");
  if (layout != OVL_ROPE_HALF && layout != OVL_ROPE_PAIRS) return fail(OVL_E_ARG, "unknown layout");
  if (!(std::isfinite(base) && base > 1)) return fail(OVL_E_ARG, "base must be above 1");
  if (scaling > OVL_ROPE_RAMP) return fail(OVL_E_ARG, "unknown scaling");
  if (scaling != OVL_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1)) return fail(OVL_E_ARG, "factor must be 1 or more");
  const bool bands = scaling == OVL_ROPE_BANDS || scaling == OVL_ROPE_RAMP;
  if (bands && (!original || !std::isfinite(high) || !(low > 0 && low < high)))
    return fail(OVL_E_ARG, "original must be positive and 0 < low < high");
  if (!(std::isfinite(magnitude) && magnitude >= 0)) return fail(OVL_E_ARG, "magnitude must be 0 or more");
  constexpr double kTurn = 6.283185307179586476925;
  ovl_rope r{};
  r.head_dim = head_dim;
  r.rot_dim = rot_dim;
  r.layout = layout;
  r.magnitude = static_cast<float>(magnitude > 0 ? magnitude : scaling == OVL_ROPE_RAMP ? 0.1 * std::log(factor) + 1 : 1);
  if (!std::isfinite(r.magnitude)) return fail(OVL_E_ARG, "magnitude out of range");
  if (scaling == OVL_ROPE_BASE && rot_dim > 2) base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  if (!std::isfinite(base)) return fail(OVL_E_ARG, "base and factor out of range");
  double first = 0, last = 0;
  if (scaling == OVL_ROPE_RAMP) {
    const double per = rot_dim / (2 * std::log(base));
    first = std::fmax(0, std::floor(per * std::log(original / (high * kTurn))));
    last = std::fmin(rot_dim - 1, std::ceil(per * std::log(original / (low * kTurn))));
  }
  for (uint32_t i = 0; i < rot_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == OVL_ROPE_LINEAR) w /= factor;
    if (scaling == OVL_ROPE_BANDS) {
      const double n = original * w / kTurn, s = std::fmin(1, std::fmax(0, (n - low) / (high - low)));
      w = s * w + (1 - s) * w / factor;
    }
    if (scaling == OVL_ROPE_RAMP) {
      const double s = std::fmin(1, std::fmax(0, (i - first) / std::fmax(last - first, 0.001)));
      w = (1 - s) * w + s * w / factor;
    }
    r.turn[i] = static_cast<uint64_t>(std::round(std::ldexp(w / kTurn, 64)));      // w <= 1, so below 2^62
  }
  *out = r;
  return OVL_OK;
}

ovl_status ovl_rope_apply(const ovl_rope* rope, uint32_t n_tokens, const int32_t* pos, const void* q, uint32_t q_heads,
                          uint64_t q_stride, const void* k, uint32_t k_heads, uint64_t k_stride, uint32_t dtype,
                          void* q_out, uint64_t q_out_stride, void* k_out, uint64_t k_out_stride, uint32_t out_dtype,
                          void* stream) {
  if (!rope) return fail(OVL_E_ARG, "rope is null");
  const uint32_t d = rope->head_dim, r = rope->rot_dim;
  if (d < 2 || d > OVL_ROPE_MAX_DIM || d % 2 || r < 2 || r > d || r % 2 ||
      (rope->layout != OVL_ROPE_HALF && rope->layout != OVL_ROPE_PAIRS))
    return fail(OVL_E_SHAPE, "rope was not made by ovl_rope_plan");
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype)) return fail(OVL_E_ARG, "dtypes must be OVL_F32 or OVL_BF16");
  if (!q_heads || q_heads > 65535 || k_heads > 65535) return fail(OVL_E_SHAPE, "q_heads or k_heads out of range");
  if (n_tokens == 0) return OVL_OK;
  if (n_tokens > 0x7fffffffu) return fail(OVL_E_ARG, "too many tokens");
  if (!pos) return fail(OVL_E_ARG, "pos is null");
  if (!aligned(pos, 4)) return fail(OVL_E_SHAPE, "pos needs 4-byte alignment");
  const uint64_t qw = static_cast<uint64_t>(q_heads) * d, kw = static_cast<uint64_t>(k_heads) * d;
  ovl_status st = check_rows("q: null, misaligned or a stride below its heads", q, dtype, q_stride, qw, n_tokens);
  if (st == OVL_OK) st = check_rows("q_out: null, misaligned or a stride below its heads", q_out, out_dtype, q_out_stride, qw, n_tokens);
  if (st == OVL_OK && k_heads) st = check_rows("k: null, misaligned or a stride below its heads", k, dtype, k_stride, kw, n_tokens);
  if (st == OVL_OK && k_heads) st = check_rows("k_out: null, misaligned or a stride below its heads", k_out, out_dtype, k_out_stride, kw, n_tokens);
  if (st != OVL_OK) return st;
  if ((q == q_out && (dtype != out_dtype || (n_tokens > 1 && q_stride != q_out_stride))) ||
      (k_heads && k == k_out && (dtype != out_dtype || (n_tokens > 1 && k_stride != k_out_stride))))
    return fail(OVL_E_SHAPE, "in place, type and stride must agree");
  const Rows none{};
  return done(launch_rope(*rope, n_tokens, pos, rows_of(q, dtype, q_stride), q_heads,
                          k_heads ? rows_of(k, dtype, k_stride) : none, k_heads, rows_of(q_out, out_dtype, q_out_stride),
                          k_heads ? rows_of(k_out, out_dtype, k_out_stride) : none, static_cast<cudaStream_t>(stream)));
}

ovl_status ovl_block_norm_apply(const ovl_block_norm* norm, uint32_t n_tokens, const void* x, uint32_t x_dtype,
                                uint64_t x_stride, const void* y, uint32_t y_dtype, uint64_t y_stride,
                                const void* gate, uint32_t gate_dtype, uint64_t gate_stride, const int32_t* gate_row,
                                uint32_t n_gates, void* x_out, uint64_t x_out_stride, void* h, uint32_t h_dtype,
                                uint64_t h_stride, void* stream) {
  if (!norm) return fail(OVL_E_ARG, "norm is null");
  const uint32_t hidden = norm->hidden;
  if (!hidden || hidden > OVL_NORM_MAX_HIDDEN) return fail(OVL_E_SHAPE, "hidden must be 1..OVL_NORM_MAX_HIDDEN");
  if (!std::isfinite(norm->alpha) || !std::isfinite(norm->beta)) return fail(OVL_E_ARG, "alpha or beta is not finite");
  ovl_status st = check_norm(norm->post);
  if (st == OVL_OK) st = check_norm(norm->pre);
  if (st != OVL_OK) return st;
  if (!dtype_ok(x_dtype) || (y && !dtype_ok(y_dtype)) || (h && !dtype_ok(h_dtype)) || (gate && !dtype_ok(gate_dtype)))
    return fail(OVL_E_ARG, "dtypes must be OVL_F32 or OVL_BF16");
  if ((norm->pre.kind != OVL_NORM_NONE) != (h != nullptr)) return fail(OVL_E_ARG, "h goes with a pre norm");
  if (!x_out && !h) return fail(OVL_E_ARG, "neither x_out nor h is wanted");
  if (n_tokens == 0) return OVL_OK;
  if (n_tokens > 0x7fffffffu) return fail(OVL_E_ARG, "too many tokens");
  st = check_rows("x: null, misaligned or a stride below hidden", x, x_dtype, x_stride, hidden, n_tokens);
  if (st == OVL_OK && y) st = check_rows("y: misaligned or a stride below hidden", y, y_dtype, y_stride, hidden, n_tokens);
  if (st == OVL_OK && x_out) st = check_rows("x_out: misaligned or a stride below hidden", x_out, x_dtype, x_out_stride, hidden, n_tokens);
  if (st == OVL_OK && h) st = check_rows("h: misaligned or a stride below hidden", h, h_dtype, h_stride, hidden, n_tokens);
  if (st == OVL_OK && gate) st = check_rows("gate: misaligned or a stride below hidden", gate, gate_dtype, gate_stride, hidden, n_gates);
  if (st != OVL_OK) return st;
  if (x == x_out && n_tokens > 1 && x_stride != x_out_stride) return fail(OVL_E_SHAPE, "in place, strides must agree");
  if (gate && (!n_gates || n_gates > 0x7fffffffu)) return fail(OVL_E_ARG, "n_gates out of range");
  if (gate && !gate_row && n_gates != 1 && n_gates != n_tokens)
    return fail(OVL_E_SHAPE, "without gate_row there is one gate, or one for each token");
  if (gate_row && !aligned(gate_row, 4)) return fail(OVL_E_SHAPE, "gate_row needs 4-byte alignment");
  Gate g{};
  if (gate) {
    g.rows = rows_of(gate, gate_dtype, gate_stride);
    g.row = gate_row;
    g.n = n_gates;
  }
  const Rows none{};
  return done(launch_block_norm(*norm, n_tokens, rows_of(x, x_dtype, x_stride), y ? rows_of(y, y_dtype, y_stride) : none, g,
                                x_out ? rows_of(x_out, x_dtype, x_out_stride) : none,
                                h ? rows_of(h, h_dtype, h_stride) : none, static_cast<cudaStream_t>(stream)));
}

ovl_status ovl_glu(uint32_t act, uint32_t n_tokens, uint32_t width, const void* gate, uint64_t gate_stride,
                   const void* up, uint64_t up_stride, uint32_t dtype, void* out, uint64_t out_stride,
                   uint32_t out_dtype, void* stream) {
  if (act < OVL_ACT_SILU || act > OVL_ACT_RELU) return fail(OVL_E_ARG, "unknown act");
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype)) return fail(OVL_E_ARG, "dtypes must be OVL_F32 or OVL_BF16");
  if (!width || width > 0x7fffffffu) return fail(OVL_E_SHAPE, "width out of range");
  if (n_tokens == 0) return OVL_OK;
  if (n_tokens > 0x7fffffffu) return fail(OVL_E_ARG, "too many tokens");
  ovl_status st = check_rows("gate: null, misaligned or a stride below width", gate, dtype, gate_stride, width, n_tokens);
  if (st == OVL_OK) st = check_rows("up: null, misaligned or a stride below width", up, dtype, up_stride, width, n_tokens);
  if (st == OVL_OK) st = check_rows("out: null, misaligned or a stride below width", out, out_dtype, out_stride, width, n_tokens);
  if (st != OVL_OK) return st;
  if ((out == gate && (dtype != out_dtype || (n_tokens > 1 && out_stride != gate_stride))) ||
      (out == up && (dtype != out_dtype || (n_tokens > 1 && out_stride != up_stride))))
    return fail(OVL_E_SHAPE, "in place, type and stride must agree");
  return done(launch_glu(act, n_tokens, width, rows_of(gate, dtype, gate_stride), rows_of(up, dtype, up_stride),
                         rows_of(out, out_dtype, out_stride), static_cast<cudaStream_t>(stream)));
}

ovl_status ovl_moe_workspace_bytes(const ovl_moe* moe, size_t* out) {
  if (!out) return fail(OVL_E_ARG, "out is null");
  *out = 0;
  const ovl_status st = check_moe_dims(moe);
  if (st == OVL_OK) *out = static_cast<size_t>(moe_layout(moe).total);
  return st;
}

ovl_status ovl_moe_forward(const ovl_moe* moe, const void* x, uint32_t dtype, uint32_t n_tokens, uint64_t x_stride,
                           const int32_t* choice, const float* weight, int32_t* choice_out, float* weight_out, void* y,
                           uint64_t y_stride, void* stream) {
  ovl_status st = check_moe_dims(moe);
  if (st != OVL_OK) return st;
  if (!dtype_ok(dtype)) return fail(OVL_E_ARG, "dtype must be OVL_F32 or OVL_BF16");
  if (!moe->gate_qs || !moe->gate_d || !moe->up_qs || !moe->up_d || !moe->down_qs || !moe->down_d || !moe->workspace)
    return fail(OVL_E_ARG, "a plane or the workspace is null");
  if (!aligned(moe->gate_qs, 16) || !aligned(moe->gate_d, 16) || !aligned(moe->up_qs, 16) || !aligned(moe->up_d, 16) ||
      !aligned(moe->down_qs, 16) || !aligned(moe->down_d, 16) || !aligned(moe->workspace, 256))
    return fail(OVL_E_SHAPE, "the planes need 16-byte, the workspace 256-byte alignment");
  const MoeLayout l = moe_layout(moe);
  if (moe->workspace_bytes < l.total) return fail(OVL_E_OOM, "the workspace is smaller than ovl_moe_workspace_bytes");
  if (!choice != !weight) return fail(OVL_E_ARG, "choice and weight come together");
  if (choice && (choice_out || weight_out)) return fail(OVL_E_ARG, "choice_out and weight_out are the router's");
  if (!choice) {
    if (!moe->router) return fail(OVL_E_ARG, "neither a router nor a choice is given");
    if (moe->score != OVL_MOE_SOFTMAX && moe->score != OVL_MOE_SIGMOID) return fail(OVL_E_ARG, "unknown score");
    if (!dtype_ok(moe->router_dtype)) return fail(OVL_E_ARG, "router_dtype must be OVL_F32 or OVL_BF16");
    if (!std::isfinite(moe->scale)) return fail(OVL_E_ARG, "scale is not finite");
    if (!aligned(moe->router, 16) || !aligned(moe->bias, 4)) return fail(OVL_E_SHAPE, "router needs 16-byte, bias 4-byte alignment");
  }
  if (!aligned(choice, 4) || !aligned(weight, 4) || !aligned(choice_out, 4) || !aligned(weight_out, 4))
    return fail(OVL_E_SHAPE, "choices and weights need 4-byte alignment");
  if (n_tokens > moe->max_tokens) return fail(OVL_E_ARG, "n_tokens over max_tokens");
  if (n_tokens == 0) return OVL_OK;
  st = check_rows("x: null or a stride below hidden", x, dtype, x_stride, moe->hidden, n_tokens);
  if (st == OVL_OK) st = check_rows("y: null or a stride below hidden", y, dtype, y_stride, moe->hidden, n_tokens);
  if (st != OVL_OK) return st;
  const uint64_t lanes = dtype == OVL_BF16 ? 8 : 4;
  if (!aligned(x, 16) || !aligned(y, 16) || (n_tokens > 1 && (x_stride % lanes || y_stride % lanes)))
    return fail(OVL_E_SHAPE, "x and y need 16-byte rows");
  uint8_t* w = static_cast<uint8_t*>(moe->workspace);
  MoeDev m{};
  m.gate_qs = static_cast<const uint8_t*>(moe->gate_qs), m.gate_d = static_cast<const uint8_t*>(moe->gate_d);
  m.up_qs = static_cast<const uint8_t*>(moe->up_qs), m.up_d = static_cast<const uint8_t*>(moe->up_d);
  m.down_qs = static_cast<const uint8_t*>(moe->down_qs), m.down_d = static_cast<const uint8_t*>(moe->down_d);
  m.router = moe->router;
  m.bias = moe->bias;
  m.quant = moe->quant;
  m.experts = moe->n_experts;
  m.top = moe->top_k;
  m.hidden = moe->hidden;
  m.ffn = moe->ffn;
  m.act = moe->act;
  m.score = moe->score;
  m.renormalize = moe->renormalize;
  m.scale = moe->scale;
  m.router_bf16 = moe->router_dtype == OVL_BF16;
  m.bf16 = dtype == OVL_BF16;
  m.given = choice != nullptr;
  m.tokens = n_tokens;
  m.pairs = n_tokens * moe->top_k;
  m.x = rows_of(x, dtype, n_tokens > 1 ? x_stride : moe->hidden);
  m.y = rows_of(y, dtype, n_tokens > 1 ? y_stride : moe->hidden);
  m.given_choice = choice;
  m.given_weight = weight;
  m.choice_out = choice_out;
  m.weight_out = weight_out;
  m.arrived = reinterpret_cast<uint32_t*>(w);
  m.logits = reinterpret_cast<float*>(w + l.logits);
  m.choice = reinterpret_cast<int32_t*>(w + l.choice);
  m.weight = reinterpret_cast<float*>(w + l.weight);
  m.power = reinterpret_cast<float*>(w + l.power);
  m.xp = reinterpret_cast<uint16_t*>(w + l.xp);
  m.hp = reinterpret_cast<uint16_t*>(w + l.hp);
  m.part = reinterpret_cast<float*>(w + l.part);
  return done(launch_moe(m, static_cast<cudaStream_t>(stream)));
}

ovl_status ovl_packed(uint32_t call, const uint64_t* words, uint32_t n_words, void* stream) {
  if (!words) return fail(OVL_E_ARG, "words is null");
  bool narrow = true;
  auto ptr = [&](uint32_t i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(words[i])); };
  auto num = [&](uint32_t i) {
    narrow &= words[i] < (1ull << 32);
    return static_cast<uint32_t>(words[i]);
  };
  const auto ints = [&](uint32_t i) { return static_cast<const int32_t*>(ptr(i)); };
  switch (call) {
    case OVL_PACKED_ROPE: {
      if (n_words != 15) break;
      const uint32_t n = num(1), qh = num(4), kh = num(7), dt = num(9), od = num(14);
      if (!narrow) break;
      return ovl_rope_apply(static_cast<const ovl_rope*>(ptr(0)), n, ints(2), ptr(3), qh, words[5], ptr(6), kh, words[8], dt,
                            ptr(10), words[11], ptr(12), words[13], od, stream);
    }
    case OVL_PACKED_BLOCK_NORM: {
      if (n_words != 18) break;
      const uint32_t n = num(1), xd = num(3), yd = num(6), gd = num(9), ng = num(12), hd = num(16);
      if (!narrow) break;
      return ovl_block_norm_apply(static_cast<const ovl_block_norm*>(ptr(0)), n, ptr(2), xd, words[4], ptr(5), yd, words[7],
                                  ptr(8), gd, words[10], ints(11), ng, ptr(13), words[14], ptr(15), hd, words[17], stream);
    }
    case OVL_PACKED_GLU: {
      if (n_words != 11) break;
      const uint32_t act = num(0), n = num(1), width = num(2), dt = num(7), od = num(10);
      if (!narrow) break;
      return ovl_glu(act, n, width, ptr(3), words[4], ptr(5), words[6], dt, ptr(8), words[9], od, stream);
    }
    case OVL_PACKED_MOE: {
      if (n_words != 11) break;
      const uint32_t dt = num(2), n = num(3);
      if (!narrow) break;
      return ovl_moe_forward(static_cast<const ovl_moe*>(ptr(0)), ptr(1), dt, n, words[4], ints(5),
                             static_cast<const float*>(ptr(6)), static_cast<int32_t*>(ptr(7)), static_cast<float*>(ptr(8)),
                             ptr(9), words[10], stream);
    }
    default: return fail(OVL_E_ARG, "unknown call");
  }
  return fail(OVL_E_ARG, "not the call's number of words, or a word above 32 bits");
}

}  // extern "C"
