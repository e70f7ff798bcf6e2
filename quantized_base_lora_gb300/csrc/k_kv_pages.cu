// Pages of the 4-bit cache: growing, forking, compacting and releasing rows.
//
// One CTA does the bookkeeping (k_kv_pages): it checks every entry, moves the
// reader counts, finds the lowest-numbered free pages with a scan over refs and
// writes the new table rows, or changes nothing and latches a status.  It leaves
// a list of fresh pages; the copy kernels, launched behind it, fill them.
//
// Fresh pages come from what is free before the call, plus what the pure
// destinations of the same call release.  Pages that an entry releases from its
// own source row (src = dst) are still read by the copy, so they become free
// only afterwards.
//
// Measured: the bookkeeping 7 us for one entry, 9 for 24, 14 for 16 entries with
// 17000 positions to check (cold; a chain of six dependent loads and a dozen
// barriers).  Copying 24 pages of 2.36 MB 16 us, 7 TB/s of reads and writes;
// compacting 16 rows of 8 layers by half 70 us, 4.5 TB/s (5.6 with the sectors of
// values that are read for a part of them).
#include <algorithm>
#include <type_traits>

#include "kv_internal.h"
#include "ptx.cuh"

namespace ovl {
namespace {

constexpr uint32_t kBook = 1024;               // threads of the bookkeeping CTA; entry i belongs to thread i
static_assert(kBook >= OVL_KV_MAX_BATCH, "one entry per thread");
constexpr uint32_t kCopy = 256;

struct BookShared {
  int32_t src[kBook], dst[kBook];
  int32_t before[kBook];      // pages that the destination held
  int32_t whole[kBook];       // leading pages that it keeps or shares
  int32_t length[kBook];      // its new length
  int32_t limit[kBook];       // compaction: the source's length
  uint32_t first[kBook + 1];  // prefix sums of the fresh pages
  int32_t off[kBook + 1];     // compaction: keep_off
  uint32_t is_dst[kKvMaxSeqs / 32];
  uint32_t warp_sum[32];
  uint32_t found;
  int32_t error;
};

// Inclusive scan over the CTA; every thread calls it.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sum) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, s);
    if (lane >= static_cast<uint32_t>(s)) v += o;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = warp_sum[lane];
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, w, s);
      if (lane >= static_cast<uint32_t>(s)) w += o;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  return v + (warp ? warp_sum[warp - 1] : 0u);
}

// The entry that owns position x of a prefix-sum array f[0..n].
template <class T>
__device__ __forceinline__ uint32_t owner_of(const T* f, uint32_t n, T x) {
  uint32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (f[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void add_refs(const KvDev& kv, int32_t page, int32_t by) {
  if (static_cast<uint32_t>(page) < kv.n_pages) atomicAdd(kv.refs + page, by);
}

__global__ void __launch_bounds__(kBook) k_kv_pages(const KvDev kv, KvPages what, const int32_t* src, const int32_t* dst,
                                                    const int32_t* keep, const int32_t* off, uint32_t n, uint32_t n_keep) {
  __shared__ BookShared s;
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const bool two = what == KvPages::kFork || what == KvPages::kCompact;
  const uint32_t page = kv.page, shift = kv.page_shift;
  griddep_launch_dependents();
  for (uint32_t i = t; i < (kv.max_seqs + 31) / 32; i += kBook) s.is_dst[i] = 0;
  griddep_wait();
  if (t == 0) s.error = 0, s.found = 0;
  __syncthreads();

  // ---- the entries, checked
  int32_t from = 0, to = 0;
  if (what == KvPages::kCompact)
    for (uint32_t i = t; i <= n; i += kBook) s.off[i] = off[i];
  if (t < n) {
    from = src[t];
    to = two ? dst[t] : from;
    if (static_cast<uint32_t>(from) >= kv.max_seqs || static_cast<uint32_t>(to) >= kv.max_seqs) {
      atomicCAS(&s.error, 0, OVL_E_ARG);
    } else if (atomicOr(&s.is_dst[to >> 5], 1u << (to & 31)) >> (to & 31) & 1u) {
      atomicCAS(&s.error, 0, OVL_E_DUPLICATE);
    }
  }
  __syncthreads();
  uint32_t need = 0;
  if (t < n && s.error == 0) {
    if (from != to && (s.is_dst[from >> 5] >> (from & 31) & 1u)) atomicCAS(&s.error, 0, OVL_E_DUPLICATE);
    const int32_t have = kv.length[from], held = kv.length[to];
    const int32_t most = static_cast<int32_t>(kv.max_pages << shift);
    const int32_t* row = kv.table + static_cast<size_t>(from) * kv.max_pages;
    int64_t len = 0;
    int32_t whole = 0;
    if (have < 0 || have > most || held < 0 || held > most) {
      atomicCAS(&s.error, 0, OVL_E_ARG);
    } else if (what == KvPages::kExtend) {
      const int32_t more = off[t + 1] - off[t];
      len = static_cast<int64_t>(have) + more;
      if (more < 0) atomicCAS(&s.error, 0, OVL_E_ARG);
      else if (len > most) atomicCAS(&s.error, 0, OVL_E_OOM);
      else {
        whole = (have + page - 1) >> shift;
        need = static_cast<uint32_t>((len + page - 1) >> shift) - whole;
      }
    } else if (what == KvPages::kFork) {
      len = keep ? keep[t] : have;
      if (len < 0 || len > have) {
        atomicCAS(&s.error, 0, OVL_E_ARG);
      } else {
        whole = static_cast<int32_t>(len) >> shift;
        need = (len & (page - 1)) != 0;
        // taken back inside a page that no one else holds: it stays
        if (need && from == to) {
          const int32_t p = row[whole];
          if (static_cast<uint32_t>(p) < kv.n_pages && __ldcg(kv.refs + p) == 1) need = 0, ++whole;
        }
      }
    } else if (what == KvPages::kCompact) {
      len = static_cast<int64_t>(off[t + 1]) - off[t];
      if (len < 0 || off[t] < 0) atomicCAS(&s.error, 0, OVL_E_ARG);
      else if (len > most) atomicCAS(&s.error, 0, OVL_E_OOM);
      else need = static_cast<uint32_t>((len + page - 1) >> shift);
    }
    s.src[t] = from;
    s.dst[t] = to;
    s.before[t] = (held + page - 1) >> shift;
    s.whole[t] = whole;
    s.length[t] = static_cast<int32_t>(len);
    s.limit[t] = have;
  }
  if (t == 0 && what == KvPages::kCompact && (off[0] != 0 || off[n] < 0 || static_cast<uint32_t>(off[n]) > n_keep))
    s.error = OVL_E_ARG;
  __syncthreads();
  const bool sound = s.error == 0;
  __syncthreads();
  if (what == KvPages::kCompact && sound) {
    // the entries follow one another from position 0, so owner_of finds each one
    const int64_t total = s.off[n];
    uint32_t e = 0;                            // the entry of position j: only ever grows
    for (int64_t j0 = t; j0 < total; j0 += 8 * kBook) {
      int32_t p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = j0 + i * kBook < total ? keep[j0 + i * kBook] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t j = j0 + i * kBook;
        if (j >= total) break;
        while (s.off[e + 1] <= j) ++e;
        if (p[i] < 0 || p[i] >= s.limit[e]) s.error = OVL_E_ARG;
      }
    }
    __syncthreads();
  }
  const uint32_t upto = block_scan(t < n ? need : 0u, s.warp_sum);
  if (t < n) s.first[t + 1] = upto;
  if (t == 0) s.first[0] = 0;
  __syncthreads();
  if (s.error != 0) {
    if (t == 0) {
      kv_latch(kv, s.error);
      *kv.n_fresh = 0;
    }
    return;
  }
  const uint32_t total = s.first[n];

  // ---- reader counts before the allocation: what pure destinations held goes,
  // shared pages gain one.  Signed so that the same loop takes it back.
  auto count_readers = [&](int32_t sign) {
    for (uint32_t e = warp; e < n; e += kBook / 32) {
      if (what == KvPages::kExtend || (two && s.src[e] == s.dst[e])) continue;
      const int32_t* old = kv.table + static_cast<size_t>(s.dst[e]) * kv.max_pages;
      for (int32_t c = lane; c < s.before[e]; c += 32) add_refs(kv, old[c], -sign);
      if (what != KvPages::kFork) continue;
      const int32_t* row = kv.table + static_cast<size_t>(s.src[e]) * kv.max_pages;
      for (int32_t c = lane; c < s.whole[e]; c += 32) add_refs(kv, row[c], sign);
    }
    __syncthreads();
  };
  count_readers(1);

  // ---- the lowest-numbered free pages
  for (uint32_t base = 0; base < kv.n_pages && s.found < total; base += kBook * 4) {
    uint32_t free_mask = 0;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t p = base + t * 4 + k;
      if (p < kv.n_pages && __ldcg(kv.refs + p) == 0) free_mask |= 1u << k;
    }
    const uint32_t mine = __popc(free_mask);
    const uint32_t end = block_scan(mine, s.warp_sum);
    const uint32_t had = s.found;
    uint32_t r = had + end - mine;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      if ((free_mask >> k & 1u) && r < total) {
        KvFresh f{};
        f.dst_page = static_cast<int32_t>(base + t * 4 + k);
        const uint32_t e = owner_of(s.first, n, r);
        f.row = kv.table + static_cast<size_t>(s.src[e]) * kv.max_pages;
        if (what == KvPages::kFork) f.src_page = f.row[s.whole[e]];
        if (what == KvPages::kCompact) {
          if (s.src[e] == s.dst[e]) f.row = kv.rows + static_cast<size_t>(e) * kv.max_pages;
          const int32_t at = static_cast<int32_t>((r - s.first[e]) << shift);
          f.first = s.off[e] + at;
          f.count = min(s.length[e] - at, static_cast<int32_t>(page));
        }
        kv.fresh[r++] = f;
      }
    __syncthreads();
    if (t == kBook - 1) s.found = had + end;
    __syncthreads();
  }
  if (s.found < total) {
    count_readers(-1);
    if (t == 0) {
      kv_latch(kv, OVL_E_OOM);
      *kv.n_fresh = 0;
    }
    return;
  }

  // ---- rows that are their own source: what they drop, and for the copy of a
  // compaction where their tokens were
  for (uint32_t e = warp; e < n; e += kBook / 32) {
    if (!two || s.src[e] != s.dst[e]) continue;
    const int32_t* row = kv.table + static_cast<size_t>(s.dst[e]) * kv.max_pages;
    for (int32_t c = lane; c < s.before[e]; c += 32) {
      const int32_t p = row[c];
      if (what == KvPages::kCompact) kv.rows[static_cast<size_t>(e) * kv.max_pages + c] = p;
      if (c >= s.whole[e]) add_refs(kv, p, -1);
    }
  }
  __syncthreads();

  // ---- the new rows
  for (uint32_t e = warp; e < n; e += kBook / 32) {
    const uint32_t fresh = s.first[e + 1] - s.first[e];
    int32_t* row = kv.table + static_cast<size_t>(s.dst[e]) * kv.max_pages;
    const int32_t* shared_row = kv.table + static_cast<size_t>(s.src[e]) * kv.max_pages;
    const int32_t whole = s.whole[e];
    for (int32_t c = lane; c < static_cast<int32_t>(kv.max_pages); c += 32) {
      if (c < whole) {
        if (s.src[e] != s.dst[e]) row[c] = shared_row[c];
      } else if (c < whole + static_cast<int32_t>(fresh)) {
        const int32_t p = kv.fresh[s.first[e] + c - whole].dst_page;
        row[c] = p;
        kv.refs[p] = 1;
      } else {
        row[c] = -1;
      }
    }
    if (lane == 0) kv.length[s.dst[e]] = s.length[e];
  }
  if (t == 0) *kv.n_fresh = two ? total : 0;
}

// Fork: whole pages, every layer.  A page is two contiguous runs; row blockIdx.y
// of the grid copies fresh page blockIdx.y (a fork has at most one an entry).
__global__ void __launch_bounds__(kCopy) k_kv_copy_pages(const KvDev kv) {
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.y >= kv.n_pages) return;
  const uint32_t fresh = *kv.n_fresh;
  const KvFresh f = kv.fresh[blockIdx.y];            // read beside the count, not after it
  if (blockIdx.y >= fresh || static_cast<uint32_t>(f.src_page) >= kv.n_pages) return;
  const uint64_t units = static_cast<uint64_t>(kv.layers) * 2 * kv.heads;
  const uint64_t nc = units * kv.unit_codes / 16, ns = units * kv.unit_scales / 8;
  constexpr uint32_t kEach = 8;
  constexpr uint64_t kChunk = kCopy * kEach;
  auto run = [&](uint4* pool, uint64_t n, uint32_t part, uint32_t parts) {
    const uint4* const a = pool + f.src_page * n;
    uint4* const b = pool + f.dst_page * n;
    for (uint64_t i0 = part * kChunk + threadIdx.x; i0 < n; i0 += parts * kChunk) {
      uint4 v[kEach];
#pragma unroll
      for (uint32_t k = 0; k < kEach; ++k)
        if (i0 + k * kCopy < n) v[k] = __ldcs(a + i0 + k * kCopy);
#pragma unroll
      for (uint32_t k = 0; k < kEach; ++k)
        if (i0 + k * kCopy < n) b[i0 + k * kCopy] = v[k];
    }
  };
  // the scales, an eighth of the codes, are the last ninth of the CTAs'
  const uint32_t last = (gridDim.x + 8) / 9, most = gridDim.x - last;
  if (blockIdx.x < most) run(reinterpret_cast<uint4*>(kv.codes), nc, blockIdx.x, most);
  else run(reinterpret_cast<uint4*>(kv.scales), ns, blockIdx.x - most, last);
}

// One T of every head of a page, kHeads loads in flight: heads are a constant
// distance apart on both sides.
template <class T>
__device__ __forceinline__ void copy_heads(uint8_t* pool, uint64_t from, uint64_t to, uint32_t heads, uint32_t step) {
  constexpr uint32_t kHeads = 4;
  for (uint32_t h = 0; h < heads; h += kHeads) {
    T v[kHeads];
#pragma unroll
    for (uint32_t k = 0; k < kHeads; ++k)
      if (h + k < heads) v[k] = *reinterpret_cast<const T*>(pool + from + static_cast<uint64_t>(h + k) * step);
#pragma unroll
    for (uint32_t k = 0; k < kHeads; ++k)
      if (h + k < heads) *reinterpret_cast<T*>(pool + to + static_cast<uint64_t>(h + k) * step) = v[k];
  }
}

// Compaction: fresh page after fresh page, blockIdx.y's share of the layers of
// each, keys or values by blockIdx.z; the tokens' sources are found once and used
// for all its layers and heads.
// Bound by memory; a value unit is 4 to 16 bytes, so scattered tokens read whole
// sectors of values for a part of them.
template <int D>
__global__ void __launch_bounds__(kCopy, 4) k_kv_gather(const KvDev kv, const int32_t* keep,
                                                        uint32_t layers_each) {
  __shared__ int32_t from_page[256], from_slot[256];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t fresh = *kv.n_fresh, code_step = kv.unit_codes, scale_step = kv.unit_scales * 2;
  const uint32_t which = blockIdx.z, layer0 = blockIdx.y * layers_each, layer1 = min(kv.layers, layer0 + layers_each);
  uint8_t* const scales = reinterpret_cast<uint8_t*>(kv.scales);
  for (uint32_t r = blockIdx.x; r < fresh; r += gridDim.x) {
    const KvFresh f = kv.fresh[r];
    const uint32_t count = f.count;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < count; i += kCopy) {
      const int32_t pos = keep[f.first + i];
      const int32_t p = f.row[pos >> kv.page_shift];
      from_page[i] = static_cast<uint32_t>(p) < kv.n_pages ? p : -1;
      from_slot[i] = pos & static_cast<int32_t>(kv.page - 1);
    }
    __syncthreads();
    using Small = typename std::conditional<D == 64, uint32_t, typename std::conditional<D == 128, uint2, uint4>::type>::type;
    for (uint32_t layer = layer0; layer < layer1; ++layer) {
      const uint64_t to = kv_unit(kv, f.dst_page, layer, which, 0);
      if (which == 0) {                              // 16-byte pieces of rows
        constexpr uint32_t kRow = D / 32;
        for (uint32_t i = threadIdx.x; i < count * kRow; i += kCopy) {
          const int32_t p = from_page[i / kRow];
          if (p < 0) continue;
          copy_heads<uint4>(kv.codes, kv_unit(kv, p, layer, 0, 0) * code_step + from_slot[i / kRow] * (D / 2) + i % kRow * 16,
                            to * code_step + i * 16, kv.heads, code_step);
        }
      } else {                                       // units, in the order in which they are stored
        for (uint32_t i = threadIdx.x; i < ((count + 7) & ~7u) * 8; i += kCopy) {
          const uint32_t tok = (i >> 6) * 8 + (i & 7), g = (i >> 3) & 7;
          if (tok >= count || from_page[tok] < 0) continue;
          const uint32_t slot = from_slot[tok];
          copy_heads<Small>(kv.codes,
                            kv_unit(kv, from_page[tok], layer, 1, 0) * code_step + (slot >> 3) * (4 * D) +
                                (slot & 7) * (D / 16) + g * (D / 2),
                            to * code_step + i * (D / 16), kv.heads, code_step);
        }
      }
      for (uint32_t i = threadIdx.x; i < count; i += kCopy)
        if (from_page[i] >= 0)
          copy_heads<Small>(scales, kv_unit(kv, from_page[i], layer, which, 0) * scale_step + from_slot[i] * (D / 16),
                            to * scale_step + i * (D / 16), kv.heads, scale_step);
    }
  }
}

}  // namespace

cudaError_t launch_kv_pages(const KvDev& kv, KvPages what, const int32_t* src, const int32_t* dst, const int32_t* keep,
                            const int32_t* off, uint32_t n, uint32_t n_keep, cudaStream_t st) {
  const cudaError_t e = launch_chained(k_kv_pages, dim3(1), kBook, 0, st, kv, what, src, dst, keep, off, n, n_keep);
  if (e != cudaSuccess) return e;
  const uint32_t full = sm_count() * 4;           // CTAs resident at a time
  if (what == KvPages::kFork) {
    const uint64_t units = static_cast<uint64_t>(kv.layers) * 2 * kv.heads;
    const uint64_t per_page = (units * kv.unit_codes / 16 + kCopy * 8 - 1) / (kCopy * 8);
    const uint32_t x = static_cast<uint32_t>(
        std::max<uint64_t>(2, std::min<uint64_t>(per_page + (per_page + 7) / 8, (full + n - 1) / n)));
    return launch_chained(k_kv_copy_pages, dim3(x, n), kCopy, 0, st, kv);
  }
  if (what == KvPages::kCompact) {
    // at most this many fresh pages; as many layers to a CTA as leave eight rounds of CTAs
    const uint64_t pages = n_keep / kv.page + n;
    const uint32_t each = static_cast<uint32_t>(
        std::min<uint64_t>(kv.layers, std::max<uint64_t>(1, pages * kv.layers * 2 / (8 * full))));
    const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(pages, 2 * full)), (kv.layers + each - 1) / each, 2);
    switch (kv.dim) {
      case 64: return launch_chained(k_kv_gather<64>, grid, kCopy, 0, st, kv, keep, each);
      case 128: return launch_chained(k_kv_gather<128>, grid, kCopy, 0, st, kv, keep, each);
      default: return launch_chained(k_kv_gather<256>, grid, kCopy, 0, st, kv, keep, each);
    }
  }
  return cudaSuccess;
}

}  // namespace ovl
