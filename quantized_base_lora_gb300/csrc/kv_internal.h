// Shared by the translation units of the 4-bit key/value cache (ovl_kv_*).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/ovl.h"

namespace ovl {

constexpr uint32_t kKvMaxSeqs = 65536;       // rows: a bit each in shared memory of the page kernel
constexpr uint32_t kKvMaxCtas = 640;         // CTAs of an attention launch that may leave partial results
constexpr uint32_t kKvPartialRows = 16;      // query rows of one partial result

// One fresh page of a fork or compaction: where its bytes come from.
struct KvFresh {
  const int32_t* row;   // compaction: the source's row
  int32_t src_page;     // fork: the page to copy
  int32_t dst_page;
  int32_t first, count; // compaction: the page's tokens in the list of positions
};

// A cache as the kernels take it: ovl_kv's pointers, the parts of the
// workspace, and sizes.
struct KvDev {
  uint8_t* codes;
  __half* scales;
  int32_t* table;
  int32_t* length;
  int32_t* refs;
  uint32_t* status;        // workspace: first latched status code, 0 = none
  uint32_t* n_fresh;       // workspace: fresh pages of the last fork or compaction
  uint32_t* joined;        // workspace: arrivals at a split segment, by its first CTA; 0 between calls
  KvFresh* fresh;          // workspace [n_pages]
  int32_t* rows;           // workspace [max_seqs][max_pages]: source rows of in-place compactions
  float* partial;          // workspace: partial attention results
  uint32_t n_pages, page, page_shift, layers, heads, dim, max_seqs, max_pages;
  uint32_t unit_codes;     // bytes of one (page, layer, K|V, head): page * dim / 2
  uint32_t unit_scales;    // binary16 values of the same: page * dim / 32
};

// Byte offset of the codes (element offset of the scales) of one unit.
__host__ __device__ __forceinline__ uint64_t kv_unit(const KvDev& kv, uint32_t page, uint32_t layer, uint32_t which,
                                                     uint32_t head) {
  return ((static_cast<uint64_t>(page) * kv.layers + layer) * 2 + which) * kv.heads + head;
}

__device__ __forceinline__ void kv_latch(const KvDev& kv, int32_t code) {
  atomicCAS(kv.status, 0u, static_cast<uint32_t>(-code));
}

// The sequence of the batch that owns packed token t: the largest i with
// off[i] <= t (off[n] > t).
__device__ __forceinline__ uint32_t kv_owner(const int32_t* off, uint32_t n, int32_t t) {
  uint32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Where a packed token lives, or page = -1 (the reason is latched).
struct KvPlace {
  int32_t page, slot;
};
__device__ __forceinline__ KvPlace kv_place(const KvDev& kv, const int32_t* seqs, const int32_t* off, uint32_t n,
                                            int32_t t) {
  const uint32_t i = kv_owner(off, n, t);
  const int32_t s = seqs[i], after = off[i + 1] - t;
  if (static_cast<uint32_t>(s) >= kv.max_seqs || after <= 0) {
    kv_latch(kv, OVL_E_ARG);
    return {-1, 0};
  }
  const int32_t pos = kv.length[s] - after;
  if (pos < 0 || static_cast<uint32_t>(pos) >= kv.max_pages << kv.page_shift) {
    kv_latch(kv, OVL_E_SHAPE);
    return {-1, 0};
  }
  const int32_t p = kv.table[static_cast<size_t>(s) * kv.max_pages + (pos >> kv.page_shift)];
  if (static_cast<uint32_t>(p) >= kv.n_pages) {
    kv_latch(kv, OVL_E_ARG);
    return {-1, 0};
  }
  return {p, pos & static_cast<int32_t>(kv.page - 1)};
}

// Query tokens of one attention call.
struct KvQuery {
  const int32_t* seqs;
  const int32_t* off;
  uint32_t n_seqs, n_tokens, max_new, layer;
  const void* q;
  void* out;
  uint64_t q_stride, out_stride;   // elements
  uint32_t heads, group;           // query heads; query heads of one kv head
  float scale;
  uint32_t window, sinks;
  bool bf16;
  uint32_t few;                    // rows of a sequence up to which the few-row kernel serves it
};

uint32_t sm_count();             // of the current device (k_fused_gemm.cu)

// Lets f use `bytes` of dynamic shared memory on the current device.  The attribute is
// a device's own: `done` has a bit for each device that has it.
inline cudaError_t allow_smem(const void* f, uint32_t bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t set = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (set == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return set;
}

// Launches f in the stream's programmatic chain: its CTAs may be scheduled while
// the kernel before it still runs, so f calls griddep_wait() before it reads or
// writes anything, and griddep_launch_dependents() as early as that is sound for
// the next one (at once: every kernel here waits first).  What a kernel before it may
// write - any argument, and the whole cache - is therefore read by ordinary loads, never
// through the read-only path (__ldg, const __restrict__), which promises that nothing
// changes while the kernel is resident.
// `cluster`: CTAs of a cluster, along x.
template <class... P, class... A>
cudaError_t launch_clustered(void (*f)(P...), dim3 grid, uint32_t block, uint32_t smem, cudaStream_t st, uint32_t cluster,
                             A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, f, args...);
}
template <class... P, class... A>
cudaError_t launch_chained(void (*f)(P...), dim3 grid, uint32_t block, uint32_t smem, cudaStream_t st, A... args) {
  return launch_clustered(f, grid, block, smem, st, 1, args...);
}

cudaError_t launch_kv_append(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                             uint32_t n_tokens, const void* k, const void* v, bool bf16, uint64_t ks, uint64_t vs,
                             cudaStream_t st);
cudaError_t launch_kv_read(const KvDev& kv, uint32_t layer, const int32_t* seqs, const int32_t* off, uint32_t n,
                           uint32_t n_tokens, float* k, float* v, cudaStream_t st);
cudaError_t launch_kv_attention(const KvDev& kv, const KvQuery& q, cudaStream_t st);
// Which kernels serve a call of these sizes on a device of `sms` SMs: the one for few
// rows alone, or beside it the one for many, in single CTAs or in pairs.
enum class KvRoute : uint32_t { kFewRows, kSingle, kPairs };
KvRoute kv_route(const KvDev& kv, const KvQuery& q, uint32_t sms);
bool kv_in_pairs(const KvDev& kv, const KvQuery& q, uint32_t sms);
cudaError_t launch_kv_prefill(const KvDev& kv, const KvQuery& q, KvRoute route, cudaStream_t st);
enum class KvPages { kExtend, kFork, kCompact, kRelease };
cudaError_t launch_kv_pages(const KvDev& kv, KvPages what, const int32_t* src, const int32_t* dst, const int32_t* keep,
                            const int32_t* off, uint32_t n, uint32_t n_keep, cudaStream_t st);

}  // namespace ovl
