// Attention over the 4-bit cache for many query rows to a key (prompts, chunks
// of prompts): bound by the tensor cores.
//
// One CTA takes 256 rows (128 where D = 256) of one sequence and kv head - the
// query heads that share the kv head are rows too - and walks the visible tokens
// in tiles of 128 (64).  Both products are tcgen05 MMAs with f16 operands and
// fp32 accumulators in tensor memory:
//   S = Q K^T   Q and K in shared memory, S in tensor memory
//   O += P V    P over S's own columns in tensor memory, V^T in shared memory
// so the scores never leave the SM.  Most sequences of more than 256 rows of 128
// channels (kv_in_pairs) are taken by pairs of CTAs, clusters of two: each has its own
// 256 rows, converts half of a tile - half of the tokens for K, half of the
// channels for V - and every MMA runs over both CTAs' rows with the two halves as
// its second operand, issued by the first.  Roles, each its own warps:
//   softmax   4 warps for each 128 rows, a thread a row: S -> P in registers, running
//             maximum and sum; O is rescaled in place, only when a row's maximum
//             has grown by more than 2^6 since its reference was set
//   keys, values   4 warps each: 4-bit words from global memory, one mask a pair
//             of codes, times the block's scale, into the MMA's shared layout;
//             two (four) buffers each; the next words are in flight meanwhile
//   issue     one warp for each 128 rows.  The two row tiles run against each
//             other: the MMAs of one overlap the softmax of the other; and P goes
//             over in parts, so that O's MMAs start with the first.
//
// Layout.  A 32-bit key word is 8 consecutive channels of a token, which is one
// 16-byte chunk of the f16 operand; its codes come out in the order 0 4 1 5 2 6 3
// 7, so Q's chunks are stored in that order as well.  A value unit is every eighth
// channel of a token, so 8 tokens' units give whole 16-byte chunks of V^T (8
// tokens of a channel) to one thread.  In both, 8 neighbouring lanes write 8 rows'
// chunks of one column of the 128-byte swizzle: no bank conflicts.
//
// Range.  Keys and values of a tile are multiplied by 2^-E, 2^E above the tile's
// largest scale, before they are rounded to f16 (|x| <= 8); the factor goes back
// into the scores, and into P for the values.  Rows of q are scaled by a power of
// two.  So f16's 11 bits hold whatever the size of the data is; within a tile, they
// hold down to 2^-14 of the largest scale: smaller blocks end in f16's subnormals.
// Keys, values and P are rounded to them (q is exact): the sums' operands are what
// the tensor cores take, and the output keeps 8 bits.
//
// Measured (GB300, 8 kv heads of 128, 32 query heads): 2 x 2048 new tokens over
// 6000 to 8192, 403 us = 967 TFLOP/s, 0.50 of the measured bf16 burst rate (452 us
// without pairs); 4 chunks of up to 777 tokens, 3 kv heads of 64, window 1024, 62 us
// (267 CTAs of 4 to 11 tiles on 152 SMs: two rounds, each with its prologue).
// Bound by the chain from scores to P and back: of 4800 clocks a tile (timed inside,
// which adds some) a softmax warp is busy for 3300 - scores from tensor memory 250,
// their maximum 310, exponentials and packing 2050 for 128 columns a thread - and
// waits 1500 for the next scores; the key warps wait 800 for a free buffer, so it is
// not the conversion, which without pairs it is as well (1300 of 5500 clocks behind
// shared memory, where a tile's operand reads, 192 KB, meet the stores of 64).
// With the softmax left out 352, without the conversions 393, without both 277 (all
// three without pairs).
// On the way there: pairs whose P was released over the cluster 547, whose softmax
// had fewer registers 437, P in two parts 410; one warp role for keys and values
// 492; MMAs issued by one lane of a diverged warp (operands moved to uniform
// registers for each) 507; the scores read twice from tensor memory, in chunks,
// 643; masks tested one by one 1123.  Not adopted: two threads a row (584), scores
// in two buffers of 64 tokens so that they run ahead of the softmax (498: N = 64 MMAs
// read Q twice as often), in pairs one role for keys and values (591).
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "kv_internal.h"
#include "kv_mma.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace ovl {
namespace {

constexpr uint32_t kTmemCols = 512;
// PAIR: CTAs that work on one MMA.
template <int D, int PAIR>
struct Shape {
  static_assert(PAIR == 1 || D == 128, "pairs take 128 channels");
  static constexpr uint32_t kRowTiles = D == 256 ? 1 : 2;      // of 128 rows a CTA
  static constexpr uint32_t kTokens = D == 256 ? 64 : 128;     // of a tile
  static constexpr uint32_t kRows = 128 * kRowTiles;           // of a CTA
  static constexpr uint32_t kQ = 128 * D * 2;                  // bytes of one row tile
  static constexpr uint32_t kBuf = kTokens * D * 2 / PAIR;     // bytes of a CTA's share of a K or V tile
  static constexpr uint32_t kBufs = 2 * PAIR;
  static constexpr uint32_t kSmem = kRowTiles * kQ + 2 * kBufs * kBuf;
  static constexpr uint32_t kParts = 2 * PAIR;                 // in which P goes over; measured 4 : 2 parts, pairs 403 : 410 us,
                                                               // single CTAs (4 x 777 rows of 64) 66 : 62
  static constexpr uint32_t kSoft = 4 * kRowTiles;             // warps
  static constexpr uint32_t kWarps = kSoft + 12;               // softmax, 4 keys, 4 values, 4 issue (1 or 2 of them busy)
  static constexpr uint32_t kThreads = kWarps * 32;
  // Registers a thread, of the launch's 96: 2 x softmax + 2 x conversion + issue = 5 x 96.
  // A pair's CTA converts half a tile and keeps less in hand for it.
  static constexpr int kSoftRegs = PAIR == 2 ? 168 : 160, kCacheRegs = PAIR == 2 ? 56 : 64, kIssueRegs = 32;
  static constexpr uint32_t kOutCol = kRowTiles * kTokens;     // first tensor memory column of O, behind S
  static_assert(kOutCol + kRowTiles * D <= kTmemCols, "S and O fit");
};

struct Bars {
  // waited for by the issuing warps (of a pair: the first CTA's, for both)
  uint64_t q_ready, k_full[4], v_full[4], p_full[2][4];        // p_full: [row tile][part of the tile's tokens]
  uint64_t k_empty[4], v_empty[4], s_full[2], o_done[2];       // arrived at by the MMAs, in each CTA
  uint64_t e_ready[4];                                         // the tile's v_exp is written
  float k_exp[8], v_exp[8];      // 2^E of the last tiles' scales as E
  uint32_t taddr;
};

template <int PAIR>
__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
template <int PAIR>
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// One arrival on `bar` (in both CTAs of a pair) when the MMAs so far are done.
template <int PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (PAIR == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
template <int PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t* where) {
  if constexpr (PAIR == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int PAIR>
__device__ __forceinline__ void tmem_free(uint32_t taddr) {
  if constexpr (PAIR == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmemCols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmemCols) : "memory");
}

__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Loads in flight have landed: the registers may be used from here on.
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void landed(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}

// The lowest n bits, n clamped to 0..32.
__device__ __forceinline__ uint32_t low_bits(int32_t n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// What one CTA's rows see.
struct Tiles {
  uint32_t lead, start, count;
  __device__ __forceinline__ uint32_t token(uint32_t j, uint32_t size) const {
    return (j < lead ? j : j - lead + start) * size;
  }
};

// What the table says of a tile's tokens 32 k + lane, -1 beyond the row's length;
// judged when it is used, a tile later, so that nothing waits for it here.
template <int N>
__device__ __forceinline__ void tile_pages(const KvDev& kv, const int32_t* row, uint32_t length, uint32_t tok,
                                           uint32_t lane, int32_t (&p)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t t = tok + 32 * k + lane;
    p[k] = -1;
    if (t < length) p[k] = row[t >> kv.page_shift];
  }
}

// E of a tile from every lane's scale words: 2^E above the largest scale.
template <int N>
__device__ __forceinline__ int32_t exponent_above(const uint32_t (&w)[N]) {
  uint32_t x = w[0];
#pragma unroll
  for (int i = 1; i < N; ++i) x = __vmaxu2(x, w[i]);
  x = max(x & 0xffffu, x >> 16);
  return static_cast<int32_t>(__reduce_max_sync(0xffffffffu, x) >> 10) - 14;
}

template <int D, int PAIR>
__global__ void __launch_bounds__(Shape<D, PAIR>::kThreads, 1) k_kv_prefill(const KvDev kv, const KvQuery a) {
  using Sh = Shape<D, PAIR>;
  constexpr uint32_t NB = D / 32, KT = Sh::kTokens, RT = Sh::kRowTiles, NBUF = Sh::kBufs;
  extern __shared__ __align__(1024) uint8_t raw[];
  __shared__ Bars bar;
  uint8_t* const sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* const sm_q = sm;
  uint8_t* const sm_k = sm + RT * Sh::kQ;
  uint8_t* const sm_v = sm_k + NBUF * Sh::kBuf;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  griddep_launch_dependents();
  griddep_wait();
  // ---- this CTA's rows; the ones that see most come first in the grid
  const uint32_t rank = PAIR == 2 ? cluster_ctarank() : 0u;
  const uint32_t seq = blockIdx.y, kh = blockIdx.x / PAIR, row_tile = gridDim.z - 1 - blockIdx.z;
  const int32_t o0 = a.off[seq], o1 = a.off[seq + 1];
  if (o0 < 0 || o1 < o0 || static_cast<uint32_t>(o1) > a.n_tokens) return;      // latched by the few-row launch
  const uint32_t tokens = o1 - o0, group = a.group, pair0 = row_tile * (PAIR * Sh::kRows);
  if (tokens * static_cast<uint64_t>(group) <= a.few) return;                   // served by the few-row launch
  const uint32_t served = min(tokens, a.max_new);
  if (row_tile == gridDim.z - 1 && rank == 0 && tokens > served) {                           // latched as well: zeros
    const uint32_t chunks = group * D / 8;
    for (uint64_t i = tid; i < static_cast<uint64_t>(tokens - served) * chunks; i += Sh::kThreads)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (o0 + served + i / chunks) * a.out_stride +
                                static_cast<uint64_t>(kh) * group * D + i % chunks * 8) = make_uint4(0, 0, 0, 0);
  }
  if (pair0 >= served * group) return;
  const uint32_t pair_rows = min(PAIR * Sh::kRows, served * group - pair0);
  // of them this CTA's: the second of a pair may have none and then only shares the work
  const uint32_t r0 = pair0 + rank * Sh::kRows;
  const uint32_t n_rows = pair_rows > rank * Sh::kRows ? min(Sh::kRows, pair_rows - rank * Sh::kRows) : 0u;
  const int32_t seq_row = a.seqs[seq];
  const bool sound = static_cast<uint32_t>(seq_row) < kv.max_seqs;
  int32_t length = sound ? kv.length[seq_row] : 0;
  if (length < 0 || length > static_cast<int32_t>(kv.max_pages << kv.page_shift)) length = 0;
  const int32_t first = length - static_cast<int32_t>(tokens);                  // position of its first new token
  const int32_t* const table_row = kv.table + static_cast<size_t>(sound ? seq_row : 0) * kv.max_pages;
  // the tiles that any of the rows sees
  const uint32_t i_first = pair0 / group, i_last = (pair0 + pair_rows - 1) / group;
  Tiles tl{0, 0, 0};
  const int32_t p_last = length ? first + static_cast<int32_t>(i_last) : -1;
  if (p_last >= 0) {
    if (a.window) {
      tl.start = static_cast<uint32_t>(max(0, first + static_cast<int32_t>(i_first) - static_cast<int32_t>(a.window) + 1)) / KT;
      tl.lead = (a.sinks + KT - 1) / KT;
      if (tl.lead >= tl.start) tl.lead = tl.start = 0;
    }
    tl.count = tl.lead + static_cast<uint32_t>(p_last) / KT + 1 - tl.start;
  }

  if (warp == 0) tmem_alloc<PAIR>(&bar.taddr);
  if (tid == 32) {
    mbar_init(&bar.q_ready, PAIR * Sh::kSoft);
    for (uint32_t i = 0; i < NBUF; ++i) {
      mbar_init(&bar.k_full[i], PAIR * 4);
      mbar_init(&bar.v_full[i], PAIR * 4);
      mbar_init(&bar.k_empty[i], RT);
      mbar_init(&bar.v_empty[i], RT);
      mbar_init(&bar.e_ready[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      for (uint32_t k = 0; k < Sh::kParts; ++k) mbar_init(&bar.p_full[i][k], PAIR * 4);
      mbar_init(&bar.o_done[i], 1);
    }
    mbar_fence_init();
  }
  tc_fence_before();
  __syncwarp();
  if constexpr (PAIR == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t taddr = bar.taddr;
  bool dead = false;                           // a bounded wait ran out
  // A whole warp waits.  After one wait has run out its others return at once: every
  // role walks its loop to the end, so no barrier between warps is left half full.
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (dead) return;
    const bool landed = warp < Sh::kSoft + 8 ? mbar_wait_bounded(b, parity)
                        : PAIR == 2          ? mbar_wait_cluster(b, parity)
                                             : mbar_wait_spin(b, parity);
    if (!__all_sync(0xffffffffu, landed)) {
      dead = true;
      if (lane == 0) kv_latch(kv, OVL_E_DEVICE_TIMEOUT);
    }
  };

  // One arrival at the issuing CTA's barrier, releasing what was written to shared memory.
  auto arrive = [&](uint64_t* b) {
    if constexpr (PAIR == 2) mbar_arrive_remote(cluster_map(b, 0));
    else mbar_arrive(b);
  };
  // The same for P: tensor memory is ordered by its own fence, and a release over the
  // cluster would wait a thousand clocks for memory that no one asks for.
  auto arrive_p = [&](uint64_t* b) {
    if constexpr (PAIR == 2)
      asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_map(b, 0)) : "memory");
    else mbar_arrive(b);
  };

  if (warp < Sh::kSoft) {
    // ================= softmax: one row a thread
    if constexpr (RT == 2) more_registers<Sh::kSoftRegs>();
    const uint32_t x = warp >> 2, r = tid & 127;
    const uint32_t row = r0 + x * 128 + r;
    const bool on = x * 128 + r < n_rows;
    const uint32_t i = row / group;
    float down = 0.f;
    {
      const uint64_t q_at = static_cast<uint64_t>(o0 + i) * a.q_stride + (kh * group + row % group) * D;
      const uint4* const src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (on ? q_at : 0));
      float top = 0.f;
      if (on) {
#pragma unroll 8
        for (uint32_t c = 0; c < D / 8; ++c) {
          const uint4 v = src[c];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
        }
      }
      // 2^ex <= top < 2^(ex + 1), biased; the row goes to [2^9, 2^10), with scale's sign
      const uint32_t ex = min(max(__float_as_uint(top) >> 23, 10u), 253u);
      const float up = copysignf(__uint_as_float((263u - ex) << 23), a.scale);
      down = fabsf(a.scale) * 1.4426950408889634f * __uint_as_float((ex - 9u) << 23);
      uint8_t* const dst = sm_q + x * Sh::kQ + r * 128;
#pragma unroll 8
      for (uint32_t c = 0; c < D / 8; ++c) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (on) v = src[c];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          f[2 * k] = __uint_as_float(w[k] << 16) * up, f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * up;
        *reinterpret_cast<uint4*>(dst + (c >> 3) * (128 * 128) + ((c & 7) ^ (r & 7)) * 16) =
            make_uint4(pack_f16(f[0], f[4]), pack_f16(f[1], f[5]), pack_f16(f[2], f[6]), pack_f16(f[3], f[7]));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive(&bar.q_ready);
    }
    const int32_t last = on && length ? first + static_cast<int32_t>(i) : -1;
    const int32_t from = a.window ? last - static_cast<int32_t>(a.window) + 1 : 0;
    const int32_t sinks = static_cast<int32_t>(a.sinks);
    // Of the rows of this tile: the ones that see least at either end.  A tile without rows
    // goes by the sequence's last one (by the masks, seeing nothing, it took 145 us beside 98).
    const uint32_t y0 = min(r0 + x * 128, pair0 + pair_rows - 1), y1 = min(r0 + x * 128 + 127, pair0 + pair_rows - 1);
    const int32_t all_last = length ? first + static_cast<int32_t>(y0 / group) : -1;
    const int32_t all_from =
        a.window ? first + static_cast<int32_t>(y1 / group) - static_cast<int32_t>(a.window) + 1 : 0;
    const uint32_t lanes = (warp & 3) * 32 << 16;
    const uint32_t s_at = taddr + lanes + x * KT, o_at = taddr + lanes + Sh::kOutCol + x * D;
    float ref = -CUDART_INF_F, l = 0.f;
#pragma unroll 1
    for (uint32_t j = 0; j < tl.count; ++j) {
      const int32_t tok = static_cast<int32_t>(tl.token(j, KT));
      const bool hidden = tok > all_last - static_cast<int32_t>(KT - 1) ||
                          (tok < all_from && tok > sinks - static_cast<int32_t>(KT));
      wait(&bar.e_ready[j % NBUF], (j / NBUF) & 1);
      wait(&bar.s_full[x], j & 1);
      tc_fence_after();
      const float ve = bar.v_exp[j & 7];
      const float kf = down * exp2f(bar.k_exp[j & 7]);
      // Two copies of the code: most tiles are seen whole.
      auto tile = [&](auto with_mask) {
        constexpr bool masked = decltype(with_mask)::value;
        uint32_t seen[KT / 32];
        if constexpr (masked) {
#pragma unroll
          for (uint32_t c = 0; c < KT; c += 32) {
            const int32_t t = tok + static_cast<int32_t>(c);
            seen[c / 32] = low_bits(last + 1 - t) & (~low_bits(from - t) | low_bits(sinks - t));
          }
        }
        uint32_t s[KT];
#pragma unroll
        for (uint32_t c = 0; c < KT; c += 32) tmem_ld32_async(s_at + c, s + c);
        tmem_wait_ld();
        float t4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (uint32_t c = 0; c < KT; c += 32) {
          landed(s + c);
#pragma unroll
          for (uint32_t k = c; k < c + 32; ++k) {
            if constexpr (masked) s[k] = seen[c / 32] & (1u << (k - c)) ? s[k] : 0xff800000u;
            t4[k & 3] = fmaxf(t4[k & 3], __uint_as_float(s[k]));
          }
        }
        const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        // P = 2^(s + ve - ref) <= 2^8, 2^14 where the reference trails
        const float want = top == -CUDART_INF_F ? -CUDART_INF_F : fmaf(top, kf, ve - 8.f);
        const bool grew = want > ref + 6.f;
        if (__any_sync(0xffffffffu, grew)) {
          const float next = fmaxf(ref, want);
          const float f = ref == -CUDART_INF_F ? 0.f : ex2(ref - next);
          ref = next;
          l *= f;
          if (j) {                             // S of this tile was issued behind O of the last
#pragma unroll 1
            for (uint32_t c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(o_at + c, o);
#pragma unroll
              for (uint32_t k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16_async(o_at + c, o);
            }
          }
        }
        const float add = ref == -CUDART_INF_F ? 0.f : ve - ref;
        const uint64_t kf2 = pair(__float_as_uint(kf), __float_as_uint(kf));
        const uint64_t add_2 = pair(__float_as_uint(add), __float_as_uint(add));
        uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
        for (uint32_t c = 0; c < KT; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (uint32_t k = 0; k < 32; k += 2) {
            const float2 e = both(fma2(pair(s[c + k], s[c + k + 1]), kf2, add_2));
            float u = ex2(e.x), v = ex2(e.y);
            if constexpr (masked) {            // -inf times a scale of 0 is no number
              u = seen[c / 32] & (1u << k) ? u : 0.f;
              v = seen[c / 32] & (2u << k) ? v : 0.f;
            }
            const uint64_t w = pair(__float_as_uint(u), __float_as_uint(v));
            if (k & 2) sum1 = add2(sum1, w);
            else sum0 = add2(sum0, w);
            p[k / 2] = pack_f16(u, v);
          }
          tmem_st16_async(s_at + c / 2, p);
          constexpr uint32_t kPart = KT / Sh::kParts;
          if ((c + 32) % kPart == 0 && c + 32 < KT) {   // a part may go ahead
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_p(&bar.p_full[x][c / kPart]);
          }
        }
        const float2 total = both(add2(sum0, sum1));
        l = fmaf(total.x + total.y, exp2f(-ve), l);
      };
      if (hidden) tile(std::true_type{});
      else tile(std::false_type{});
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_p(&bar.p_full[x][Sh::kParts - 1]);
    }
    if (tl.count) wait(&bar.o_done[x], 0);
    tc_fence_after();
    const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
    uint16_t* const to = static_cast<uint16_t*>(a.out) + static_cast<uint64_t>(o0 + i) * a.out_stride +
                         (kh * group + row % group) * D;
#pragma unroll 1
    for (uint32_t c = 0; c < D; c += 32) {
      uint32_t o[32];
      if (tl.count && !dead) {
        tmem_ld32(o_at + c, o);
      } else {
#pragma unroll
        for (uint32_t k = 0; k < 32; ++k) o[k] = 0;
      }
      if (on) {
#pragma unroll
        for (uint32_t k = 0; k < 32; k += 8) {
          uint32_t w[4];
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            const float u = l == 0.f ? 0.f : __uint_as_float(o[k + 2 * e]) * inv;
            const float v = l == 0.f ? 0.f : __uint_as_float(o[k + 2 * e + 1]) * inv;
            w[e] = pack_bf16(u, v);
          }
          *reinterpret_cast<uint4*>(to + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    tc_fence_before();
  } else if (warp < Sh::kSoft + 8) {
    if constexpr (RT == 2) fewer_registers<Sh::kCacheRegs>();
    constexpr int IT = KT / 32;
    constexpr uint32_t NW = NB / 2;            // scale words of a token
    const uint32_t w4 = warp & 3;
    const bool values = warp >= Sh::kSoft + 4;
    const uint64_t unit = kv_unit(kv, 0, a.layer, values, kh);
    const uint32_t page_codes = kv.unit_codes * kv.layers * 2 * kv.heads, page_scales = page_codes / 16;
    const uint8_t* const codes = kv.codes + unit * kv.unit_codes;
    const __half* const scales = kv.scales + unit * kv.unit_scales;
    uint32_t magic;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
    // 2^-e as f16, |e| <= 16: exact, at the far end as a subnormal
    auto down_by = [](int32_t e) { return __half2half2(__float2half_rn(__int_as_float((127 - e) << 23))); };
    int32_t pages[IT];                         // of tokens 32 k + lane of the next tile to load
    uint32_t sc[IT * NW];                      // scales of tokens 32 k + lane; 0 for tokens never written
    auto load_scales = [&](uint32_t tok) {
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const uint32_t t = tok + 32 * k + lane;
        if (static_cast<uint32_t>(pages[k]) >= kv.n_pages) {
          if (t < static_cast<uint32_t>(length)) kv_latch(kv, OVL_E_ARG);
          pages[k] = -1;
        }
#pragma unroll
        for (uint32_t i = 0; i < NW; ++i) sc[k * NW + i] = 0;
        if (pages[k] >= 0) load_words<NW>(scales + wide(pages[k], page_scales) + (t & (kv.page - 1)) * NB, &sc[k * NW]);
      }
    };
    // The exponent above the tile's scales, which are multiplied by 2^-it.
    auto settle = [&] {
      const int32_t e = exponent_above(sc);
      const __half2 down = down_by(e);
#pragma unroll
      for (uint32_t i = 0; i < IT * NW; ++i) sc[i] = mul_f16x2(sc[i], down);
      return e;
    };
    // Words are requested behind the conversion of the ones before, page numbers a tile
    // earlier.
    auto first = [&](auto load) {
      if (tl.count) {
        tile_pages<IT>(kv, table_row, length, tl.token(0, KT), lane, pages);
        load(tl.token(0, KT));
      }
      if (tl.count > 1) tile_pages<IT>(kv, table_row, length, tl.token(1, KT), lane, pages);
    };
    auto next = [&](uint32_t j, auto load) {
      if (j + 1 < tl.count) load(tl.token(j + 1, KT));
      if (j + 2 < tl.count) tile_pages<IT>(kv, table_row, length, tl.token(j + 2, KT), lane, pages);
    };
    if (!values) {
      // ================= keys: tokens 32 k + 8 w4 + lane % 8, words lane / 8 of every block;
      // of a pair each CTA converts half of the tokens
      constexpr int KI = IT / PAIR;
      const uint32_t from = w4 * 8 + (lane & 7), part = lane >> 3;
      uint32_t kw[KI][NB];
      auto load = [&](uint32_t tok) {
        load_scales(tok);
#pragma unroll
        for (int k = 0; k < KI; ++k) {
          const uint32_t u = tok + 32 * (rank * KI + k) + from;
          const int32_t p = __shfl_sync(0xffffffffu, PAIR == 2 && rank ? pages[(PAIR - 1) * KI + k] : pages[k], from);
#pragma unroll
          for (uint32_t i = 0; i < NB; ++i) kw[k][i] = 0x88888888u;
          if (p >= 0) load_words<NB>(codes + wide(p, page_codes) + (u & (kv.page - 1)) * (D / 2) + part * (D / 8), kw[k]);
        }
      };
      first(load);
#pragma unroll 1
      for (uint32_t j = 0; j < tl.count && !dead; ++j) {
        const uint32_t b = j % NBUF;
        const int32_t e = settle();
        if (j >= NBUF) wait(&bar.k_empty[b], (j / NBUF - 1) & 1);
        if (w4 == 0 && lane == 0) bar.k_exp[j & 7] = static_cast<float>(e);
        uint8_t* const buf = sm_k + b * Sh::kBuf + from * 128;
#pragma unroll
        for (int k = 0; k < KI; ++k) {
          uint32_t d[NW];
#pragma unroll
          for (uint32_t i = 0; i < NW; ++i)
            d[i] = __shfl_sync(0xffffffffu, PAIR == 2 && rank ? sc[((PAIR - 1) * KI + k) * NW + i] : sc[k * NW + i], from);
#pragma unroll
          for (uint32_t i = 0; i < NB; ++i) {
            const __half2 d2 = *reinterpret_cast<const __half2*>(&d[i / 2]);
            const __half2 dd = i & 1 ? __high2half2(d2) : __low2half2(d2);
            uint32_t v[4];
            signed_pairs(kw[k][i], magic, v);
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = mul_f16x2(v[x], dd);
            const uint32_t c = 4 * i + part;   // chunk of 8 channels
            *reinterpret_cast<uint4*>(buf + (i >> 1) * (KT / PAIR * 128) + 32 * k * 128 + ((c & 7) ^ (lane & 7)) * 16) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        next(j, load);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&bar.k_full[b]);
      }
    } else {
      // ================= values: the 8 tokens from 32 k_of + 8 (lane / 8), unit lane % 8
      // (D = 256: half of it; of a pair each CTA converts half of the channels)
      constexpr bool kSplit = D == 256 || PAIR == 2;
      constexpr uint32_t WT = D == 64 || PAIR == 2 ? 1 : 2;   // words of a token's unit that a thread takes
      const uint32_t half = PAIR == 2 ? rank : D == 256 ? w4 >> 1 : 0, k_of = D == 256 ? w4 & 1 : w4;
      const uint32_t g = lane & 7, grp = k_of * 4 + (lane >> 3);
      uint32_t vw[8][WT];
      auto load = [&](uint32_t tok) {
        load_scales(tok);
        int32_t mine = pages[0];
#pragma unroll
        for (int k = 1; k < IT; ++k) mine = k_of == static_cast<uint32_t>(k) ? pages[k] : mine;
        const int32_t p = __shfl_sync(0xffffffffu, mine, lane & 24);
#pragma unroll
        for (uint32_t t = 0; t < 8; ++t)
#pragma unroll
          for (uint32_t i = 0; i < WT; ++i) vw[t][i] = 0x88888888u;
        if (p >= 0) {
          const uint8_t* const at = codes + wide(p, page_codes) + ((tok + grp * 8) & (kv.page - 1)) * (D / 2) + g * (D / 2) +
                                    half * (4 * WT);
          if constexpr (kSplit) {
#pragma unroll
            for (uint32_t t = 0; t < 8; ++t) load_words<WT>(at + t * (D / 16), vw[t]);
          } else {
            uint32_t w[8 * WT];
            load_words<8 * WT>(at, w);
#pragma unroll
            for (uint32_t t = 0; t < 8; ++t)
#pragma unroll
              for (uint32_t i = 0; i < WT; ++i) vw[t][i] = w[t * WT + i];
          }
        }
      };
      first(load);
#pragma unroll 1
      for (uint32_t j = 0; j < tl.count && !dead; ++j) {
        const uint32_t b = j % NBUF;
        const int32_t e = settle();
        uint32_t own[WT];                      // lane l: the scales of token 32 k_of + l, this thread's blocks
#pragma unroll
        for (uint32_t i = 0; i < WT; ++i) {
          auto mine = [&](uint32_t k) { return kSplit && half ? sc[k * NW + NW / 2 + i] : sc[k * NW + i]; };
          own[i] = mine(0);
#pragma unroll
          for (int k = 1; k < IT; ++k) own[i] = k_of == static_cast<uint32_t>(k) ? mine(k) : own[i];
        }
        if (j >= NBUF) wait(&bar.v_empty[b], (j / NBUF - 1) & 1);
        if (w4 == 0 && lane == 0) {
          bar.v_exp[j & 7] = static_cast<float>(e);
          mbar_arrive(&bar.e_ready[b]);
        }
        uint8_t* const buf = sm_v + b * Sh::kBuf + (grp >> 3) * (D / PAIR * 128) + ((PAIR == 1 ? half * 128 : 0) + g) * 128 +
                             ((grp & 7) ^ g) * 16;
#pragma unroll
        for (uint32_t w = 0; w < WT; ++w) {
          uint32_t d[8];
#pragma unroll
          for (uint32_t t = 0; t < 8; ++t) d[t] = __shfl_sync(0xffffffffu, own[w], (lane & 24) + t);
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {   // a block of 32 channels: 4 of this thread's each
            const uint32_t pick = h ? 0x7632u : 0x5410u;
            uint32_t v[4][4];                  // [channel][token pair]
#pragma unroll
            for (uint32_t t = 0; t < 4; ++t) {
              uint32_t x[4];
              signed_pairs(__byte_perm(vw[2 * t][w], vw[2 * t + 1][w], pick), magic, x);
              const uint32_t dd = __byte_perm(d[2 * t], d[2 * t + 1], pick);
#pragma unroll
              for (uint32_t c = 0; c < 4; ++c) v[c][t] = mul_f16x2(x[c], dd);
            }
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(buf + (64 * w + 32 * h + 8 * c) * 128) =
                  make_uint4(v[c][0], v[c][1], v[c][2], v[c][3]);
          }
        }
        next(j, load);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&bar.v_full[b]);
      }
    }
  } else {
    // ================= issue: one warp for each row tile
    if constexpr (RT == 2) fewer_registers<Sh::kIssueRegs>();
    // The whole warp walks the loop and one elected thread issues: descriptors stay in
    // uniform registers, which the MMA instruction takes its operands from.
    const uint32_t x = __shfl_sync(0xffffffffu, warp, 0) - Sh::kSoft - 8;
    if (x < RT && rank == 0) {
      constexpr uint32_t kF32 = 1u << 4;       // accumulators; both operands f16
      constexpr uint32_t kQK = kF32 | ((KT >> 3) << 17) | ((PAIR * 128u >> 4) << 24);
      constexpr uint32_t kPV = kF32 | ((D >> 3) << 17) | ((PAIR * 128u >> 4) << 24);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sm_q) + x * Sh::kQ);
      const uint64_t k_desc = sdesc_sw128(smem_u32(sm_k)), v_desc = sdesc_sw128(smem_u32(sm_v));
      const uint32_t s_at = taddr + x * KT, o_at = taddr + Sh::kOutCol + x * D;
      if (tl.count) wait(&bar.q_ready, 0);
#pragma unroll 1
      for (uint32_t j = 0; j < tl.count && !dead; ++j) {
        const uint32_t parity = (j / NBUF) & 1, b = j % NBUF;
        wait(&bar.k_full[b], parity);
        if (dead) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (uint32_t k = 0; k < D / 16; ++k)   // 64 channels a region of 128-byte rows
            umma_f16<PAIR>(s_at, q_desc + (k >> 2) * (128 * 128 / 16) + 2 * (k & 3),
                           k_desc + b * (Sh::kBuf / 16) + (k >> 2) * (KT / PAIR * 128 / 16) + 2 * (k & 3), kQK, k != 0);
          commit<PAIR>(&bar.s_full[x]);
          commit<PAIR>(&bar.k_empty[b]);
        }
        __syncwarp();
        wait(&bar.v_full[b], parity);
#pragma unroll
        for (uint32_t h = 0; h < Sh::kParts; ++h) {
          wait(&bar.p_full[x][h], j & 1);
          if (dead) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (uint32_t k = h * (KT / 16 / Sh::kParts); k < (h + 1) * (KT / 16 / Sh::kParts); ++k)   // 64 tokens a region
              umma_f16_ts<PAIR>(o_at, s_at + 8 * k,
                                v_desc + b * (Sh::kBuf / 16) + (k >> 2) * (D / PAIR * 128 / 16) + 2 * (k & 3), kPV,
                                (j | k) != 0);
            if (h == Sh::kParts - 1) commit<PAIR>(&bar.v_empty[b]);
          }
          __syncwarp();
        }
      }
      // nothing of this CTA may still run when its tensor memory goes: waited for, within the
      // same limit, where another wait has run out as well
      if (tl.count) {
        if (elect_one()) commit<PAIR>(&bar.o_done[x]);
        __syncwarp();
        dead = false;
        wait(&bar.o_done[x], 0);
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  // of a pair, neither leaves while the other's MMAs or arrivals may still reach it
  if constexpr (PAIR == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free<PAIR>(taddr);
}

template <int D, int PAIR>
cudaError_t prefill(const KvDev& kv, const KvQuery& a, cudaStream_t st) {
  using Sh = Shape<D, PAIR>;
  constexpr uint32_t bytes = Sh::kSmem + 1024, rows = PAIR * Sh::kRows;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_kv_prefill<D, PAIR>), bytes, &ready);
  if (e != cudaSuccess) return e;
  const uint64_t tiles = (static_cast<uint64_t>(a.max_new) * a.group + rows - 1) / rows;   // at most 65535: kv_route
  return launch_clustered(k_kv_prefill<D, PAIR>, dim3(PAIR * kv.heads, a.n_seqs, static_cast<uint32_t>(tiles)),
                          Sh::kThreads, bytes, st, PAIR, kv, a);
}

}  // namespace

// Whether pairs serve a call's sequences of 128 channels.  Per token tile a pair's CTA
// takes 97 us / 47 where a single one takes 110 (8 x 4 heads over 6000 tokens), but a
// sequence whose rows end in the pair's first 256 leaves the second CTA without any.
// So pairs serve as long as they need no more rounds of CTAs on the SMs; measured pairs :
// single, 8 x 4 heads, sequences alike within a factor of two: 2 of 2048 rows over
// 6000 tokens 109 : 119 us, 8 of up to 260 108 : 121, 8 of up to 768 210 : 232; but with
// a round more, 32 of up to 260 over 1024 114 : 83, 32 of up to 768 207 : 159.  Over few
// tokens, which the host does not know, a pair's start shows: 8 of 512 rows over 512 29 : 26.
bool kv_in_pairs(const KvDev& kv, const KvQuery& a, uint32_t sms) {
  const uint64_t rows = static_cast<uint64_t>(a.n_tokens) * a.group, most = static_cast<uint64_t>(a.max_new) * a.group;
  if (most <= 256) return false;
  // as many sequences alike as the rows make; short ones beside long ones do not count
  const uint64_t seqs = std::max<uint64_t>(1, std::min<uint64_t>(a.n_seqs, 2 * rows / most));
  const uint64_t each = std::min(most, (rows + seqs - 1) / seqs);
  auto rounds = [&](uint64_t ctas) { return (ctas * seqs * kv.heads + sms - 1) / sms; };
  return rounds((each + 511) / 512 * 2) <= rounds((each + 255) / 256);
}

cudaError_t launch_kv_prefill(const KvDev& kv, const KvQuery& a, KvRoute route, cudaStream_t st) {
  switch (kv.dim) {
    case 64: return prefill<64, 1>(kv, a, st);
    case 128: return route == KvRoute::kPairs ? prefill<128, 2>(kv, a, st) : prefill<128, 1>(kv, a, st);
    default: return prefill<256, 1>(kv, a, st);
  }
}

}  // namespace ovl
