// The entry points of the 4-bit key/value cache: argument checks, the layout of
// the workspace, and the launches.  Nothing is kept between calls.
#include <cmath>
#include <cstring>
#include <string>

#include "block_internal.h"
#include "kv_internal.h"
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

ovl_status cuda_fail(cudaError_t e) {
  cudaGetLastError();
  return fail(OVL_E_CUDA, cudaGetErrorString(e));
}

uint64_t up256(uint64_t v) { return (v + 255) & ~static_cast<uint64_t>(255); }

// Offsets of the workspace's parts.
struct Layout {
  uint64_t joined, fresh, rows, partial, total;
};

ovl_status check_dims(const ovl_kv* kv) {
  if (!kv) return fail(OVL_E_ARG, "kv is null");
  const uint32_t d = kv->head_dim, p = kv->page_tokens;
  if (d != 64 && d != 128 && d != 256) return fail(OVL_E_SHAPE, "head_dim must be 64, 128 or 256");
  if (p != 16 && p != 32 && p != 64 && p != 128 && p != 256)
    return fail(OVL_E_SHAPE, "page_tokens must be 16, 32, 64, 128 or 256");
  if (!kv->n_pages || kv->n_pages > 0x7fffffffu / 16 || !kv->n_layers || kv->n_layers > 65535 || !kv->n_kv_heads ||
      kv->n_kv_heads > 65535)
    return fail(OVL_E_SHAPE, "n_pages, n_layers or n_kv_heads out of range");
  if (static_cast<uint64_t>(kv->n_layers) * kv->n_kv_heads * p * d >= (1ull << 31))
    return fail(OVL_E_SHAPE, "the codes of a page, all layers, must be below 2^31 bytes");
  if (!kv->max_seqs || kv->max_seqs > kKvMaxSeqs) return fail(OVL_E_SHAPE, "max_seqs must be 1..65536");
  if (!kv->max_pages || static_cast<uint64_t>(kv->max_pages) * p > 0x3fffffffu)
    return fail(OVL_E_SHAPE, "max_pages * page_tokens must be 1..2^30 - 1");
  return OVL_OK;
}

Layout layout_of(const ovl_kv* kv) {
  Layout l{};
  l.joined = 256;
  l.fresh = l.joined + up256(4ull * kKvMaxCtas);
  l.rows = l.fresh + up256(sizeof(KvFresh) * static_cast<uint64_t>(kv->n_pages));
  l.partial = l.rows + up256(4ull * kv->max_seqs * kv->max_pages);
  l.total = l.partial + up256(4ull * kKvMaxCtas * 2 * kKvPartialRows * (kv->head_dim + 2));
  return l;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

ovl_status check_kv(const ovl_kv* kv, KvDev* out) {
  ovl_status st = check_dims(kv);
  if (st != OVL_OK) return st;
  if (!kv->codes || !kv->scales || !kv->table || !kv->length || !kv->refs || !kv->workspace)
    return fail(OVL_E_ARG, "a pointer of kv is null");
  if (!aligned(kv->codes, 16) || !aligned(kv->scales, 16) || !aligned(kv->table, 4) || !aligned(kv->length, 4) ||
      !aligned(kv->refs, 4) || !aligned(kv->workspace, 256))
    return fail(OVL_E_SHAPE, "codes and scales need 16-byte, the workspace 256-byte alignment");
  const Layout l = layout_of(kv);
  if (kv->workspace_bytes < l.total) return fail(OVL_E_OOM, "the workspace is smaller than ovl_kv_workspace_bytes");
  uint8_t* w = static_cast<uint8_t*>(kv->workspace);
  KvDev d{};
  d.codes = static_cast<uint8_t*>(kv->codes);
  d.scales = static_cast<__half*>(kv->scales);
  d.table = kv->table;
  d.length = kv->length;
  d.refs = kv->refs;
  d.status = reinterpret_cast<uint32_t*>(w);
  d.n_fresh = reinterpret_cast<uint32_t*>(w + 128);
  d.joined = reinterpret_cast<uint32_t*>(w + l.joined);
  d.fresh = reinterpret_cast<KvFresh*>(w + l.fresh);
  d.rows = reinterpret_cast<int32_t*>(w + l.rows);
  d.partial = reinterpret_cast<float*>(w + l.partial);
  d.n_pages = kv->n_pages;
  d.page = kv->page_tokens;
  while ((1u << d.page_shift) < d.page) ++d.page_shift;
  d.layers = kv->n_layers;
  d.heads = kv->n_kv_heads;
  d.dim = kv->head_dim;
  d.max_seqs = kv->max_seqs;
  d.max_pages = kv->max_pages;
  d.unit_codes = d.page * d.dim / 2;
  d.unit_scales = d.page * d.dim / 32;
  *out = d;
  return OVL_OK;
}

ovl_status check_batch(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n) {
  if (layer >= kv.layers) return fail(OVL_E_ARG, "layer out of range");
  if (n > OVL_KV_MAX_BATCH) return fail(OVL_E_ARG, "n_seqs over OVL_KV_MAX_BATCH");
  if (n && (!seqs || !off)) return fail(OVL_E_ARG, "seqs or tok_off is null");
  return OVL_OK;
}

ovl_status done(cudaError_t e) { return e == cudaSuccess ? OVL_OK : cuda_fail(e); }

ovl_status pages_call(const ovl_kv* kv, KvPages what, const int32_t* src, const int32_t* dst, const int32_t* keep,
                      const int32_t* off, uint32_t n, uint32_t n_keep, void* stream) {
  KvDev d;
  ovl_status st = check_kv(kv, &d);
  if (st != OVL_OK) return st;
  if (n > OVL_KV_MAX_BATCH) return fail(OVL_E_ARG, "more entries than OVL_KV_MAX_BATCH");
  if (n_keep > 0x7fffffffu) return fail(OVL_E_ARG, "too many positions");
  if (n == 0) return OVL_OK;
  const bool two = what == KvPages::kFork || what == KvPages::kCompact;
  if (!src || (two && !dst) || (what == KvPages::kExtend && !off) || (what == KvPages::kCompact && ((n_keep && !keep) || !off)))
    return fail(OVL_E_ARG, "a device array is null");
  return done(launch_kv_pages(d, what, src, dst, keep, off, n, n_keep, static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace ovl

using namespace ovl;

extern "C" {

ovl_status ovl_kv_workspace_bytes(const ovl_kv* kv, size_t* out) {
  if (!out) return fail(OVL_E_ARG, "out is null");
  *out = 0;
  const ovl_status st = check_dims(kv);
  if (st == OVL_OK) *out = static_cast<size_t>(layout_of(kv).total);
  return st;
}

ovl_status ovl_kv_init(const ovl_kv* kv, void* stream) {
  KvDev d;
  const ovl_status st = check_kv(kv, &d);
  if (st != OVL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(d.table, 0xff, 4ull * d.max_seqs * d.max_pages, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(d.length, 0, 4ull * d.max_seqs, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(d.refs, 0, 4ull * d.n_pages, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(kv->workspace, 0, layout_of(kv).total, s);
  return done(e);
}

ovl_status ovl_kv_extend(const ovl_kv* kv, const int32_t* seqs, const int32_t* tok_off, uint32_t n_seqs,
                         void* stream) {
  return pages_call(kv, KvPages::kExtend, seqs, nullptr, nullptr, tok_off, n_seqs, 0, stream);
}

ovl_status ovl_kv_fork(const ovl_kv* kv, const int32_t* src, const int32_t* dst, const int32_t* keep, uint32_t n,
                       void* stream) {
  return pages_call(kv, KvPages::kFork, src, dst, keep, nullptr, n, 0, stream);
}

ovl_status ovl_kv_compact(const ovl_kv* kv, const int32_t* src, const int32_t* dst, const int32_t* keep,
                          const int32_t* keep_off, uint32_t n, uint32_t n_keep, void* stream) {
  return pages_call(kv, KvPages::kCompact, src, dst, keep, keep_off, n, n_keep, stream);
}

ovl_status ovl_kv_release(const ovl_kv* kv, const int32_t* seqs, uint32_t n, void* stream) {
  return pages_call(kv, KvPages::kRelease, seqs, nullptr, nullptr, nullptr, n, 0, stream);
}

ovl_status ovl_kv_append(const ovl_kv* kv, uint32_t layer, const int32_t* seqs, const int32_t* tok_off,
                         uint32_t n_seqs, uint32_t n_tokens, const void* k, const void* v, uint32_t dtype,
                         uint64_t k_stride, uint64_t v_stride, void* stream) {
  KvDev d;
  ovl_status st = check_kv(kv, &d);
  if (st == OVL_OK) st = check_batch(d, layer, seqs, tok_off, n_seqs);
  if (st != OVL_OK) return st;
  if (dtype != OVL_F32 && dtype != OVL_BF16) return fail(OVL_E_ARG, "dtype must be OVL_F32 or OVL_BF16");
  if (n_seqs == 0 || n_tokens == 0) return OVL_OK;
  if (n_tokens > 0x7fffffffu) return fail(OVL_E_ARG, "too many tokens");
  if (!k || !v) return fail(OVL_E_ARG, "k or v is null");
  const uint64_t row = static_cast<uint64_t>(d.heads) * d.dim, lanes = dtype == OVL_BF16 ? 8 : 4;
  if (k_stride < row || v_stride < row || k_stride % lanes || v_stride % lanes || !aligned(k, 16) || !aligned(v, 16))
    return fail(OVL_E_SHAPE, "k and v need 16-byte aligned tokens of n_kv_heads * head_dim elements");
  return done(launch_kv_append(d, layer, seqs, tok_off, n_seqs, n_tokens, k, v, dtype == OVL_BF16, k_stride, v_stride,
                               static_cast<cudaStream_t>(stream)));
}

ovl_status ovl_kv_read(const ovl_kv* kv, uint32_t layer, const int32_t* seqs, const int32_t* tok_off,
                       uint32_t n_seqs, uint32_t n_tokens, float* k_out, float* v_out, void* stream) {
  KvDev d;
  ovl_status st = check_kv(kv, &d);
  if (st == OVL_OK) st = check_batch(d, layer, seqs, tok_off, n_seqs);
  if (st != OVL_OK) return st;
  if (n_seqs == 0 || n_tokens == 0) return OVL_OK;
  if (n_tokens > 0x7fffffffu) return fail(OVL_E_ARG, "too many tokens");
  if (!k_out || !v_out) return fail(OVL_E_ARG, "k_out or v_out is null");
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return fail(OVL_E_SHAPE, "k_out and v_out need 16-byte alignment");
  return done(launch_kv_read(d, layer, seqs, tok_off, n_seqs, n_tokens, k_out, v_out,
                             static_cast<cudaStream_t>(stream)));
}

ovl_status ovl_kv_positions(const ovl_kv* kv, const int32_t* seqs, const int32_t* tok_off, uint32_t n_seqs,
                            uint32_t n_tokens, int32_t* pos, void* stream) {
  KvDev d;
  ovl_status st = check_kv(kv, &d);
  if (st == OVL_OK) st = check_batch(d, 0, seqs, tok_off, n_seqs);
  if (st != OVL_OK) return st;
  if (n_seqs == 0 || n_tokens == 0) return OVL_OK;
  if (n_tokens > 0x7fffffffu) return fail(OVL_E_ARG, "too many tokens");
  if (!pos) return fail(OVL_E_ARG, "pos is null");
  if (!aligned(pos, 4)) return fail(OVL_E_SHAPE, "pos needs 4-byte alignment");
  return done(launch_kv_positions(d, seqs, tok_off, n_seqs, n_tokens, pos, static_cast<cudaStream_t>(stream)));
}

ovl_status ovl_kv_attention(const ovl_kv* kv, uint32_t layer, const int32_t* seqs, const int32_t* tok_off,
                            uint32_t n_seqs, uint32_t n_tokens, uint32_t max_new, const void* q, uint32_t dtype,
                            uint32_t n_heads, uint64_t q_stride, float scale, uint32_t window, uint32_t sinks,
                            void* out, uint64_t out_stride, void* stream) {
  KvDev d;
  ovl_status st = check_kv(kv, &d);
  if (st == OVL_OK) st = check_batch(d, layer, seqs, tok_off, n_seqs);
  if (st != OVL_OK) return st;
  if (dtype != OVL_F32 && dtype != OVL_BF16) return fail(OVL_E_ARG, "dtype must be OVL_F32 or OVL_BF16");
  if (!std::isfinite(scale)) return fail(OVL_E_ARG, "scale is not finite");
  if (!n_heads || n_heads % d.heads) return fail(OVL_E_SHAPE, "n_heads must be a multiple of n_kv_heads");
  if (n_heads / d.heads > 1024) return fail(OVL_E_SHAPE, "more than 1024 query heads to a kv head");
  if (static_cast<uint64_t>(n_heads) * d.dim >= (1ull << 32))      // offsets inside a token are 32-bit
    return fail(OVL_E_SHAPE, "a token's query heads must be below 2^32 elements");
  if (n_seqs == 0 || n_tokens == 0) return OVL_OK;
  if (n_tokens > 0x7fffffffu || !max_new) return fail(OVL_E_ARG, "n_tokens or max_new out of range");
  if (!q || !out) return fail(OVL_E_ARG, "q or out is null");
  const uint64_t row = static_cast<uint64_t>(n_heads) * d.dim, lanes = dtype == OVL_BF16 ? 8 : 4;
  if (q_stride < row || out_stride < row || q_stride % lanes || out_stride % lanes || !aligned(q, 16) ||
      !aligned(out, 16))
    return fail(OVL_E_SHAPE, "q and out need 16-byte aligned tokens of n_heads * head_dim elements");
  KvQuery a{};
  a.seqs = seqs;
  a.off = tok_off;
  a.n_seqs = n_seqs;
  a.n_tokens = n_tokens;
  a.max_new = max_new < n_tokens ? max_new : n_tokens;
  a.layer = layer;
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.heads = n_heads;
  a.group = n_heads / d.heads;
  a.scale = scale;
  // positions stay below 2^30, so larger bounds mean the same
  a.window = window < 0x40000000u ? window : 0u;
  a.sinks = sinks < 0x40000000u ? sinks : 0x40000000u;
  a.bf16 = dtype == OVL_BF16;
  return done(launch_kv_attention(d, a, static_cast<cudaStream_t>(stream)));
}

ovl_status ovl_debug_kv_route(const ovl_kv* kv, uint32_t n_seqs, uint32_t n_tokens, uint32_t max_new, uint32_t dtype,
                              uint32_t n_heads, uint32_t n_sms, uint32_t* out) {
  const ovl_status st = check_dims(kv);
  if (st != OVL_OK) return st;
  if (!out || !n_sms || (dtype != OVL_F32 && dtype != OVL_BF16)) return fail(OVL_E_ARG, "out, n_sms or dtype");
  if (!n_heads || n_heads % kv->n_kv_heads) return fail(OVL_E_SHAPE, "n_heads must be a multiple of n_kv_heads");
  KvDev d{};
  d.dim = kv->head_dim;
  d.heads = kv->n_kv_heads;
  KvQuery a{};
  a.n_seqs = n_seqs;
  a.n_tokens = n_tokens;
  a.max_new = max_new < n_tokens ? max_new : n_tokens;
  a.group = n_heads / kv->n_kv_heads;
  a.bf16 = dtype == OVL_BF16;
  *out = static_cast<uint32_t>(kv_route(d, a, n_sms));
  return OVL_OK;
}

ovl_status ovl_kv_check(const ovl_kv* kv, void* stream) {
  KvDev d;
  const ovl_status st = check_kv(kv, &d);
  if (st != OVL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t code = 0;
  cudaError_t e = cudaMemcpyAsync(&code, d.status, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && code) e = cudaMemsetAsync(d.status, 0, 4, s);
  if (e != cudaSuccess) return cuda_fail(e);
  if (!code) return OVL_OK;
  return fail(-static_cast<ovl_status>(code), "a call on the cache was refused on the device");
}

}  // extern "C"
