// Attention over the 4-bit cache for few query rows to a key (decode steps,
// drafted tokens): the cache is read once and its bytes are the floor.
//
// Rows.  The query heads that share a kv head, and all new tokens of a sequence,
// are the rows of one small matrix Q [rows][D]; 8 or 16 rows at a time (one or
// two column tiles of an MMA) are a group.  A segment is one (sequence, kv head,
// group); its keys are walked in tiles of 32 tokens.
//
// Mathematics.  With code = c + 8 and one scale d for 32 channels,
//   s_j = sum_b dK_jb (sum_{i in b} c_ji q_i),   o = sum_j p_j dV_jb c_j,
// so the codes go into the MMA as they are: small integers, exact in f16.  Bits
// 4 i and 16 + 4 i of a word are the two halves of a pair.  For keys in bf16 calls
// a mask alone makes operands of them: the bits of a subnormal, code 2^-24 (even
// i) or 16 code 2^-24 (odd i).  Odd channels' q is divided by 16, and the share of
// the 8 in every code, sum_b dK_jb Q_b with Q_b = -8 sum_i q_i over the block, is
// one more MMA (scales against Q, Q in two f16 parts) that the scores start from:
// of the size of the rest, so nothing of the 32-bit sums is lost to it (as
// 1024 + code, from which 1032 sum_i q_i has to be taken, scores were off by 100
// times as much).  Elsewhere the same mask with an exponent gives 1024 + code and
// 1024 + 16 code, and one instruction a pair makes code - 8 of it, exactly.  The
// scale of a key block multiplies its accumulator (fp32); the scale of a value
// block multiplies p, once a block.  Nothing is dequantized in memory.
// S^T = K Q^T has tokens as rows, so its accumulator has to be transposed to
// become the second operand of O^T = V^T P: one movmatrix for 8x8.
//
// Precision.  A row of q is scaled by a power of two into f16's range (undone in
// fp32): exact for bf16 down to 2^-28 of the row's maximum (2^-24 in odd channels),
// and within 2^-23 of each element of an fp32 q as two f16 parts (2^-34 of the
// row's maximum where that is more).  The running reference of the softmax is
// max_j(s_j) + E, E chosen from the tile's largest value scale so that p dV stays
// below 2^15, up to 2^6 of it for a reference that is only moved when it trails by
// more: bf16 calls round p and p dV to f16 (11 bits each, with 2^E moved from dV to
// p where it is not near 1), f32 calls keep p dV as two f16 parts.  A block whose
// scale is below 2^-14 of its tile's largest meets f16's end earlier.
//
// Split.  All tiles of the call, segment after segment, are dealt to the CTAs in
// equal runs, whatever the lengths are (they are known on the device only).  The
// four warps of a CTA take every fourth tile of its run, each with a running
// maximum and sum of its own and a private ring of asynchronous copies, so there is no
// CTA barrier inside a segment.  A segment that is cut by a run's end is joined
// by whichever of its CTAs arrives last: partial results go through memory, in
// the order of the CTAs, so the same call gives the same bits, and no CTA waits.
//
// Measured (GB300, 8 kv heads of 128, 32 query heads, bf16): 16 sequences of
// 60001 to 131072 tokens, 292 us = 5.7 TB/s, 0.85 of the measured copy rate; 32
// sequences of 500 to 8000 tokens, 32 us (0.39: starting, joining and the first
// loads are two thirds of it); 64 sequences, window 2048 and 4 sinks, 44 us
// (0.50).  The copies alone take 241 us of the first, the arithmetic alone
// about 280: a tile of 32 tokens is some 640 instructions of a warp, 128 of them
// the masks that take the codes apart, at 0.6 to 0.7 of the issue slots with
// four warps a scheduler (128 registers).  What brought it there, in order, on
// that case: 489 us with keys in bf16 and two instructions a mask; 356 with f16
// codes and one; 314 with asynchronous copies by the whole warp in place of bulk
// copies by four lanes (whose operands went through uniform registers one lane
// after the other) and a reference that trails; 291 with a shorter loop; 289 with
// rings of two tiles (three: the 32 sequences 33, the windows 45 us); 292 with value
// scales far from 1 seen to.  Not
// adopted: eight warps a CTA (280, but 36 and 49), two (331, 38, 50), the next
// part's first tiles requested before a part is joined (291, 36, 48: registers).
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "kv_internal.h"
#include "kv_mma.cuh"
#include "ptx.cuh"

namespace ovl {
namespace {

constexpr uint32_t kWarps = 4;
constexpr uint32_t kThreads = kWarps * 32;
constexpr uint32_t kTile = 32;               // tokens
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 6.f;                  // log2 by which the running reference may trail the maximum
constexpr int32_t kNear = 6;                 // |log2| of a tile's value scales up to which p and p dV fit f16 as they are
__device__ constexpr float kZero[4] = {0.f, 0.f, 0.f, 0.f};

template <int D>
struct Stage {
  static constexpr uint32_t kCodes = kTile * D / 2;
  static constexpr uint32_t kScales = kTile * (D / 32) * 2;
  static constexpr uint32_t kBytes = 2 * (kCodes + kScales);   // keys, values, key scales, value scales
  static constexpr uint32_t kRing = D == 64 ? 3 : 2;           // deeper: the first tile of a part waits for all
  static constexpr uint32_t kWarpBytes = kRing * kBytes;
};

// N consecutive 32-bit words from shared memory, in loads of up to 16 bytes.
template <int N>
__device__ __forceinline__ void lds(const void* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *static_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *static_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = static_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int32_t e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// w[i mod N] without indexing registers.
template <int N>
__device__ __forceinline__ uint32_t word_of(const uint32_t (&w)[N], uint32_t i) {
  if constexpr (N == 1) return w[0];
  if constexpr (N == 2) return i & 1 ? w[1] : w[0];
  if constexpr (N == 4) {
    const uint32_t a = i & 1 ? w[1] : w[0], b = i & 1 ? w[3] : w[2];
    return i & 2 ? b : a;
  }
}

// Whether a sequence's part of tok_off names tokens of the call.
__device__ __forceinline__ bool owns(const KvQuery& a, int32_t o0, int32_t o1) {
  return o0 >= 0 && o1 >= o0 && static_cast<uint32_t>(o1) <= a.n_tokens;
}

// Zeros for the tokens that no sequence owns (a call padded beyond tok_off's last
// entry, or a tok_off that does not ascend from 0), latched.  One CTA does it behind
// its share of the tiles: looked for in every CTA's scan it cost each call 0.4 us.
__device__ __forceinline__ void zero_strays(const KvDev& kv, const KvQuery& a, uint32_t head_bytes) {
  bool gap = false;
  for (uint32_t i = threadIdx.x; i < a.n_seqs; i += blockDim.x) {
    const int32_t o0 = a.off[i], o1 = a.off[i + 1];
    gap |= !owns(a, o0, o1) || (i == 0 && o0 != 0) || (i + 1 == a.n_seqs && static_cast<uint32_t>(o1) != a.n_tokens);
  }
  if (!__syncthreads_or(gap)) return;
  const uint32_t lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (threadIdx.x == 0) kv_latch(kv, OVL_E_ARG);
  const uint32_t words = head_bytes / 16 * a.heads;
  const uint64_t stride = a.out_stride * (a.bf16 ? 2 : 4);
#pragma unroll 1
  for (uint64_t t = threadIdx.x >> 5; t < a.n_tokens; t += warps) {      // a token a warp
    bool owned = false;
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < a.n_seqs && !owned; i0 += 32) {
      const uint32_t i = i0 + lane;
      bool mine = false;
      if (i < a.n_seqs) {
        const int32_t o0 = a.off[i], o1 = a.off[i + 1];
        mine = owns(a, o0, o1) && static_cast<uint64_t>(o0) <= t && t < static_cast<uint64_t>(o1);
      }
      owned = __any_sync(0xffffffffu, mine);
    }
    if (owned) continue;
    uint4* const to = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + t * stride);
#pragma unroll 1
    for (uint32_t w = lane; w < words; w += 32) to[w] = make_uint4(0, 0, 0, 0);
  }
}

// What the rows of one sequence see, in tiles.
struct Span {
  int32_t length;      // 0 if the row cannot be used
  int32_t first;       // position of its first new token
  uint32_t tokens;     // new tokens
  uint32_t lead;       // leading tiles that hold sinks outside the window
  uint32_t start;      // first tile of the window
  uint32_t tiles;      // lead + tiles of the window; at least 1, so that every row is written
};

__device__ __forceinline__ Span span_of(const KvDev& kv, const KvQuery& a, uint32_t i, bool report) {
  Span s{};
  const int32_t row = a.seqs[i], o0 = a.off[i], o1 = a.off[i + 1];
  if (!owns(a, o0, o1)) {
    if (report) kv_latch(kv, OVL_E_ARG);
    return s;
  }
  s.tokens = o1 - o0;
  s.tiles = 1;
  if (static_cast<uint32_t>(row) >= kv.max_seqs) {
    if (report && s.tokens) kv_latch(kv, OVL_E_ARG);
    if (static_cast<uint64_t>(s.tokens) * a.group > a.few) s.tokens = 0;
    return s;
  }
  const int32_t n = kv.length[row];
  const bool fits = n >= 0 && n <= static_cast<int32_t>(kv.max_pages << kv.page_shift);
  if (report && (!fits || s.tokens > a.max_new)) kv_latch(kv, OVL_E_SHAPE);
  if (static_cast<uint64_t>(s.tokens) * a.group > a.few) {   // the other kernel's
    s.tokens = 0;
    return s;
  }
  if (!fits) return s;
  s.length = n;
  s.first = n - static_cast<int32_t>(s.tokens);
  if (n > 0) {
    if (a.window) {
      s.start = static_cast<uint32_t>(max(0, s.first - static_cast<int32_t>(a.window) + 1)) / kTile;
      s.lead = (a.sinks + kTile - 1) / kTile;
      if (s.lead >= s.start) s.lead = s.start = 0;
    }
    s.tiles = s.lead + (static_cast<uint32_t>(n) + kTile - 1) / kTile - s.start;
  }
  return s;
}

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, (D <= 128 && BF16 && NT == 1) ? 4 : 2)
    k_kv_decode(const KvDev kv, const KvQuery a) {
  using St = Stage<D>;
  constexpr int NB = D / 32;                  // blocks of 32 channels
  constexpr int MT = D / 16;                  // row tiles of O^T
  constexpr int NS = BF16 ? 1 : 2;            // f16 parts of q and of p dV
  constexpr uint32_t kRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* const ring = smem;
  float* const s_m = reinterpret_cast<float*>(smem + kWarps * St::kWarpBytes);   // [kWarps][kRows]
  float* const s_l = s_m + kWarps * kRows;
  uint64_t* const before = reinterpret_cast<uint64_t*>(s_l + kWarps * kRows); // [n_seqs + 1] tiles before a sequence
  __shared__ uint64_t s_warp[kWarps];
  __shared__ uint32_t s_last;

  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rows_group = a.group;        // query heads of a kv head

  griddep_launch_dependents();
  griddep_wait();
  // ---- tiles before every sequence
  uint64_t base = 0;
  for (uint32_t i0 = 0; i0 < a.n_seqs; i0 += kThreads) {
    const uint32_t i = i0 + tid;
    uint64_t w = 0;
    if (i < a.n_seqs) {
      const Span s = span_of(kv, a, i, blockIdx.x == 0);
      w = static_cast<uint64_t>(s.tiles) * kv.heads * ((s.tokens * rows_group + kRows - 1) / kRows);
    }
    uint64_t inc = w;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const uint64_t o = __shfl_up_sync(0xffffffffu, inc, k);
      if (lane >= static_cast<uint32_t>(k)) inc += o;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    uint64_t add = base;
    for (uint32_t k = 0; k < kWarps; ++k) {
      if (k < warp) add += s_warp[k];
      base += s_warp[k];
    }
    if (i < a.n_seqs) before[i] = add + inc - w;
    __syncthreads();
  }
  if (tid == 0) before[a.n_seqs] = base;
  __syncthreads();
  const uint64_t total = base;
  // at least one tile for every warp: shorter runs only add joins
  const uint64_t chunk = max((total + gridDim.x - 1) / gridDim.x, static_cast<uint64_t>(kWarps));
  uint64_t at = min(blockIdx.x * chunk, total);
  const uint64_t end = min(at + chunk, total);

  uint8_t* const my_ring = ring + warp * St::kWarpBytes;
  uint32_t slot = 0;                          // of the ring, in bytes, across segments
  const float scale2 = fabsf(a.scale) * kLog2e;   // the sign goes into q
  uint32_t magic;
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));

  while (at < end) {
    // ---- the segment
    uint32_t lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1;
      if (before[mid] <= at) lo = mid;
      else hi = mid;
    }
    // sequences without new tokens have no tiles: the last one that starts here owns the tile
    const uint32_t seq = lo;
    const Span sp = span_of(kv, a, seq, false);
    const uint64_t local = at - before[seq];
    const uint32_t seg = static_cast<uint32_t>(local / sp.tiles), tile0 = static_cast<uint32_t>(local % sp.tiles);
    const uint32_t tile1 = static_cast<uint32_t>(min(static_cast<uint64_t>(sp.tiles), tile0 + (end - at)));
    const uint64_t seg_begin = at - tile0, seg_end = seg_begin + sp.tiles;
    const uint32_t groups = (sp.tokens * rows_group + kRows - 1) / kRows;
    const uint32_t kh = seg / groups, r0 = (seg % groups) * kRows;
    const uint32_t n_rows = min(kRows, sp.tokens * rows_group - r0);
    const int32_t* const pages = kv.table + static_cast<size_t>(sp.length ? a.seqs[seq] : 0) * kv.max_pages;
    const int32_t token0 = a.off[seq];

    // ---- what this warp's share of the run reads: tiles x0, x0 + 4, ..; page numbers
    // 32 of them ahead
    const uint32_t x0 = tile0 + warp, skip = sp.start - sp.lead;
    auto token_of = [&](uint32_t x) { return (x < sp.lead ? x : x + skip) * kTile; };
    // the page of a tile's first half and, where pages are 16 tokens, of its second
    bool lost = false;                        // a page that is not there: its tokens take no part
    auto page_at = [&](uint32_t tok) -> int32_t {
      if (tok >= static_cast<uint32_t>(sp.length)) return -1;
      const int32_t p = pages[tok >> kv.page_shift];
      if (static_cast<uint32_t>(p) < kv.n_pages) return p;
      kv_latch(kv, OVL_E_ARG);
      lost = true;
      return -1;
    };
    int32_t ids0, ids1;                       // of the next 32 tiles, one a lane
    auto fetch_pages = [&](uint32_t x) {
      x += lane * kWarps;
      ids0 = ids1 = -1;
      if (x < tile1) {
        const uint32_t tok = token_of(x);
        ids0 = page_at(tok);
        ids1 = kv.page == 16 ? page_at(tok + 16) : ids0;
      }
      lost = __any_sync(0xffffffffu, lost);
    };
    fetch_pages(x0);
    // A tile's copies, in runs of 512 bytes by the whole warp: key codes, value
    // codes (16 bytes a lane and run), then both scale arrays together.
    const uint32_t page_codes = kv.unit_codes * kv.layers * 2 * kv.heads;    // a page is below 2^31 bytes
    const uint32_t page_scales = page_codes / 8;
    const uint64_t unit = kv_unit(kv, 0, a.layer, 0, kh);
    const uint8_t* const k_from = kv.codes + unit * kv.unit_codes + lane * 16;
    const uint32_t to_values = kv.heads * kv.unit_codes;
    constexpr uint32_t kScaleLanes = St::kScales / 16 < 16 ? St::kScales / 16 : 16;   // lanes on one array
    const bool v_lane = lane >= kScaleLanes;
    const uint8_t* const s_from = reinterpret_cast<const uint8_t*>(kv.scales) +
                                  (unit + (v_lane ? kv.heads : 0)) * (2 * kv.unit_scales) +
                                  (lane - (v_lane ? kScaleLanes : 0)) * 16;
    const uint32_t s_half = (lane - (v_lane ? kScaleLanes : 0)) * 16 >= St::kScales / 2 &&
                            St::kScales <= 256;                              // this lane's scales are of tokens 16 ..
    const uint32_t my_ring32 = smem_u32(my_ring) + lane * 16;
    const uint32_t s_to = 2 * St::kCodes + (v_lane ? St::kScales - kScaleLanes * 16 : 0);
    auto issue = [&](uint32_t x, uint32_t lane_of, uint32_t dst) {
      const int32_t p0 = __shfl_sync(0xffffffffu, ids0, lane_of);
      constexpr uint32_t kRuns = St::kCodes / 512;
      if (kv.page != 16) {
        if (p0 >= 0) {
          const uint32_t in_page = token_of(x) & (kv.page - 1);
          const uint8_t* const from = k_from + wide(p0, page_codes) + in_page * (D / 2);
          const uint8_t* const from_v = from + to_values;
#pragma unroll
          for (uint32_t i = 0; i < kRuns; ++i) cp16(dst + i * 512, from + i * 512);
#pragma unroll
          for (uint32_t i = 0; i < kRuns; ++i) cp16(dst + St::kCodes + i * 512, from_v + i * 512);
          const uint8_t* const from_s = s_from + wide(p0, page_scales) + in_page * (NB * 2);
          if (lane < 2 * kScaleLanes)
#pragma unroll
            for (uint32_t i = 0; i < (St::kScales + 255) / 256; ++i) cp16(dst + s_to + i * 256, from_s + i * 256);
        }
      } else {
        // two pages of 16 tokens: the halves of every array have a page each
        const int32_t p1 = __shfl_sync(0xffffffffu, ids1, lane_of);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          const int32_t p = h ? p1 : p0;
          if (p < 0) continue;
          const uint8_t* const from = k_from + wide(p, page_codes);
          const uint8_t* const from_v = from + to_values;
          if (kRuns > 1 || lane < 16)
#pragma unroll
            for (uint32_t i = 0; i < (kRuns + 1) / 2; ++i) {
              cp16(dst + h * (St::kCodes / 2) + i * 512, from + i * 512);
              cp16(dst + St::kCodes + h * (St::kCodes / 2) + i * 512, from_v + i * 512);
            }
          const uint8_t* const from_s = s_from + wide(p, page_scales) - (h ? St::kScales / 2 : 0);
          if (lane < 2 * kScaleLanes) {
            if constexpr (St::kScales <= 256) {
              if (s_half == h) cp16(dst + s_to, from_s);
            } else {
              cp16(dst + s_to + h * 256, from_s + h * 256);
            }
          }
        }
      }
    };
    uint32_t ahead = x0, ahead_of = 0;        // the next tile to request, and its number
    {
      uint32_t at_slot = slot;
#pragma unroll 1
      for (; ahead_of < St::kRing; ++ahead_of, ahead += kWarps) {
        if (ahead < tile1) issue(ahead, ahead_of, my_ring32 + at_slot);
        cp_async_commit();
        at_slot = at_slot + St::kBytes == St::kWarpBytes ? 0 : at_slot + St::kBytes;
      }
    }

    // ---- the rows: q as the MMA's second operand, and where each column looks
    uint32_t qf[NT][NS][NB][4];
    uint32_t qs[NT][2];                       // bf16 calls: the share of the codes' 8, B operand against the key scales
    float to_log2[NT][2];                     // scale, log2(e) and the row's power of two
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t r = nt * 8 + g;
      const bool on = r < n_rows;
      const uint32_t row = r0 + (on ? r : 0);
      const uint64_t qa = static_cast<uint64_t>(token0 + row / rows_group) * a.q_stride +
                          (kh * rows_group + row % rows_group) * D;
      float x[NB][8], top = 0.f, sums[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (BF16) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (on) v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + qa + 32 * b + 8 * t);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[b][2 * k] = __uint_as_float(w[k] << 16), x[b][2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
          float4 u = make_float4(0, 0, 0, 0), v = u;
          if (on) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + qa + 32 * b + 8 * t);
            u = p[0], v = p[1];
          }
          x[b][0] = u.x, x[b][1] = u.y, x[b][2] = u.z, x[b][3] = u.w;
          x[b][4] = v.x, x[b][5] = v.y, x[b][6] = v.z, x[b][7] = v.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[b][k]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^ex <= top < 2^(ex + 1), biased; the row is multiplied by 2^(kUp - ex): as far up
      // as f16 goes for a bf16 number, and for two parts so that both keep their small end.
      constexpr uint32_t kUp = BF16 ? 15 : 9;
      const uint32_t ex = min(max(__float_as_uint(top) >> 23, kUp + 1), 254u);
      const float up = copysignf(__uint_as_float((254u + kUp - ex) << 23), a.scale), down = __uint_as_float((ex - kUp) << 23);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float even = 0.f, odd = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float u = x[b][k] * up, v = x[b][k + 4] * up;
          if constexpr (BF16) {
            uint32_t h = pack_f16(u, v);
            const float2 f = halves(h);
            if (k & 1) odd += f.x + f.y, h = pack_f16(f.x * 0.0625f, f.y * 0.0625f);
            else even += f.x + f.y;
            qf[nt][0][b][k] = h;
          } else {
#pragma unroll
            for (int s = 0; s < NS; ++s) qf[nt][s][b][k] = take_f16(u, v);
          }
        }
        if constexpr (BF16) {
          float c = -0x1p-21f * (even + odd);       // -8 2^-24; below 1, since q is below 2^16
          c += __shfl_xor_sync(0xffffffffu, c, 1);
          sums[b] = c + __shfl_xor_sync(0xffffffffu, c, 2);
        }
      }
      qs[nt][0] = qs[nt][1] = 0;
      if constexpr (BF16) {
        // summed index 2 i, 2 i + 1: blocks 2 i, 2 i + 1, first all rounded parts, then all rests
        uint32_t hi[NB / 2], rest[NB / 2];
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
          hi[i] = take_f16(sums[2 * i], sums[2 * i + 1]);
          rest[i] = pack_f16(sums[2 * i], sums[2 * i + 1]);
        }
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
          if (t == i) qs[nt][0] = hi[i];
          if (NB == 8 ? t == i : t == i + NB / 2) qs[nt][NB == 8] = rest[i];
        }
      }
      // the key codes of bf16 calls stand for 2^-24 of themselves; multiplied last, and kept
      // finite, so that sizes of q and scale that make up for one another do so
      constexpr float kCodes = BF16 ? 0x1p24f : 1.f;
      to_log2[nt][0] = fminf(scale2 * __shfl_sync(0xffffffffu, down, 8 * t) * kCodes, 0x1.fffffep127f);
      to_log2[nt][1] = fminf(scale2 * __shfl_sync(0xffffffffu, down, 8 * t + 4) * kCodes, 0x1.fffffep127f);
    }
    // tiles that every row sees whole need no mask
    const uint32_t i0 = r0 / rows_group, i1 = (r0 + n_rows - 1) / rows_group;
    const int32_t all_last = i1 < a.max_new ? sp.first + static_cast<int32_t>(i0) : -1;
    const int32_t all_from = a.window ? sp.first + static_cast<int32_t>(i1) - static_cast<int32_t>(a.window) + 1 : 0;
    const int32_t sinks = static_cast<int32_t>(a.sinks);

    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -CUDART_INF_F;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    // ---- the tiles
#pragma unroll 1
    for (uint32_t x = x0; x < tile1; x += kWarps) {
      const int32_t tok = static_cast<int32_t>(token_of(x));
      cp_async_wait<St::kRing - 1>();
      __syncwarp();
      const uint8_t* const st = my_ring + slot;
      const bool hidden = tok > all_last - static_cast<int32_t>(kTile - 1) || lost ||
                          (tok < all_from && tok > sinks - static_cast<int32_t>(kTile));

      // Two copies of the tile's code: tiles that need no mask take no part of it.  Without
      // the mask it returns false, having changed nothing, if the tile's scales are far from 1.
      auto tile = [&](auto with_mask) {
      constexpr bool masked = decltype(with_mask)::value;
      // scores: tokens 16 sub + g and + 8 against columns 2 t, 2 t + 1
      float s[2][NT][4];
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        uint32_t k0[NB], k1[NB], d0[NB / 2], d1[NB / 2];
        const uint8_t* const kr = st + (16 * sub + g) * (D / 2) + t * (D / 8);
        lds<NB>(kr, k0);
        lds<NB>(kr + 8 * (D / 2), k1);
        const uint8_t* const dr = st + 2 * St::kCodes + (16 * sub + g) * (NB * 2);
        lds<NB / 2>(dr, d0);
        lds<NB / 2>(dr + 8 * NB * 2, d1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[sub][nt][0] = s[sub][nt][1] = s[sub][nt][2] = s[sub][nt][3] = 0.f;
          if constexpr (BF16) {
            // this lane's pair of scales for the sums' index 2 t (and, with 8 blocks, 2 t + 8)
            const uint32_t u0 = word_of<NB / 2>(d0, t), u1 = word_of<NB / 2>(d1, t);
            mma_f16(s[sub][nt], u0, u1, NB == 8 ? u0 : 0u, NB == 8 ? u1 : 0u, qs[nt][0], qs[nt][1], kZero);
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t x[4], y[4];
          if constexpr (BF16) masked_pairs(k0[b], x), masked_pairs(k1[b], y);
          else signed_pairs(k0[b], magic, x), signed_pairs(k1[b], magic, y);
          const float2 e0 = halves(d0[b / 2]), e1 = halves(d1[b / 2]);
          const float f0 = b & 1 ? e0.y : e0.x, f1 = b & 1 ? e1.y : e1.x;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float c[4];
            mma_f16(c, x[0], y[0], x[1], y[1], qf[nt][0][b][0], qf[nt][0][b][1], kZero);
            mma_f16(c, x[2], y[2], x[3], y[3], qf[nt][0][b][2], qf[nt][0][b][3], c);
#pragma unroll
            for (int p = 1; p < NS; ++p) {
              mma_f16(c, x[0], y[0], x[1], y[1], qf[nt][p][b][0], qf[nt][p][b][1], c);
              mma_f16(c, x[2], y[2], x[3], y[3], qf[nt][p][b][2], qf[nt][p][b][3], c);
            }
            s[sub][nt][0] = fmaf(f0, c[0], s[sub][nt][0]);
            s[sub][nt][1] = fmaf(f0, c[1], s[sub][nt][1]);
            s[sub][nt][2] = fmaf(f1, c[2], s[sub][nt][2]);
            s[sub][nt][3] = fmaf(f1, c[3], s[sub][nt][3]);
          }
        }
      }
      // the largest value scale of the tile, 2^(E - 1) <= it < 2^E, and what that
      // leaves for p: p dV < 2^9 (2^15 where the reference trails), and where p itself is
      // rounded to f16, p too
      const uint8_t* const vd = st + 2 * St::kCodes + St::kScales;
      bool held0 = true, held1 = true;        // the tile's halves have a page
      if (masked && lost) {
        auto there = [&](uint32_t t0) {
          return t0 < static_cast<uint32_t>(sp.length) &&
                 static_cast<uint32_t>(pages[t0 >> kv.page_shift]) < kv.n_pages;
        };
        held0 = there(tok), held1 = there(tok + 16);
      }
      auto written = [&](uint32_t j) {        // token j of the tile holds data
        return tok + static_cast<int32_t>(j) < sp.length && (j < 16 ? held0 : held1);
      };
      uint32_t vmax;
      {
        uint32_t v[NB / 2];
        lds<NB / 2>(vd + lane * NB * 2, v);
        vmax = v[0];
#pragma unroll
        for (int i = 1; i < NB / 2; ++i) vmax = __vmaxu2(vmax, v[i]);
        vmax = max(vmax & 0xffffu, vmax >> 16);
      }
      uint32_t seen = 0;                      // a bit for each of this lane's scores
      if constexpr (masked) {
        if (!written(lane)) vmax = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the column's row sees tokens <= last and (>= from or < sinks)
            const uint32_t c = nt * 8 + 2 * t + e, i = (r0 + c) / rows_group;
            const int32_t last = c < n_rows && i < a.max_new && sp.length ? sp.first + static_cast<int32_t>(i) : -1;
            const int32_t from = a.window ? last - static_cast<int32_t>(a.window) + 1 : 0;
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int32_t j = tok + 16 * sub + 8 * h + static_cast<int32_t>(g);
                const bool sees = j <= last && (j >= from || j < sinks) && (sub ? held1 : held0);
                if (sees) seen |= 1u << (nt * 8 + sub * 4 + e + 2 * h);
                else s[sub][nt][e + 2 * h] = -CUDART_INF_F;
              }
          }
      }
      const int32_t top_exp = static_cast<int32_t>(__reduce_max_sync(0xffffffffu, vmax) >> 10) - 14;
      // bf16 calls: with |E| <= kNear p and p dV both have f16's room (11 bits down to 2^-17 of
      // the largest weight); further off, p is multiplied and dV divided by 2^E, in the
      // masked copy.  The other finds out where the reference has to move, which an infinite
      // `above` makes it do (16 sequences of up to 131072 tokens: 288.6 us without the case,
      // 291.9 like this, 297.2 with the factors in both copies).
      const bool far = BF16 && (top_exp > kNear || top_exp < -kNear), shift = masked && far;
      const float above = !masked && far ? CUDART_INF_F : static_cast<float>((BF16 && !far ? max(top_exp, 0) : top_exp) - 9);
      bool grew = false;
      float ref[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(m[nt][e], fmaf(x, to_log2[nt][e], above));
          grew |= x > m[nt][e] + kLag;
          ref[nt][e] = x;
        }
      if (__any_sync(0xffffffffu, grew)) {
        if (!masked && far) return false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = m[nt][e] == -CUDART_INF_F ? 0.f : ex2(m[nt][e] - ref[nt][e]);
            m[nt][e] = ref[nt][e];
            l[nt][e] *= f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[nt][i][e] *= f, o[nt][i][e + 2] *= f;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float r = masked && m[nt][e] == -CUDART_INF_F ? 0.f : m[nt][e];   // nothing seen yet: every weight is 0
          if (shift) r -= static_cast<float>(top_exp);
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& w = s[sub][nt][e + 2 * h];
              w = ex2(fmaf(w, to_log2[nt][e], -r));
              if (masked && !(seen >> (nt * 8 + sub * 4 + e + 2 * h) & 1u)) w = 0.f;   // -inf times a scale of 0
            }
            l[nt][e] = fmaf(s[sub][nt][e] + s[sub][nt][e + 2], shift ? pow2(-top_exp) : 1.f, l[nt][e]);
          }
        }

      // values: channels as rows, tokens 2 t, 2 t + 1 and + 8 of a sub-tile as the summed index
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        uint32_t va[NB], vb[NB], d0[NB / 2], d1[NB / 2];     // [token 2t | 2t + 1][NB / 2 words], first and second 8 tokens
        const uint8_t* const vr = st + St::kCodes + sub * (8 * D) + lane * (D / 8);
        lds<NB>(vr, va);
        lds<NB>(vr + 4 * D, vb);
        const uint8_t* const dr = vd + (16 * sub + g) * (NB * 2);
        lds<NB / 2>(dr, d0);
        lds<NB / 2>(dr + 8 * NB * 2, d1);
        if constexpr (masked) {                         // what was never written may hold any bits
          const bool w0 = written(16 * sub + g), w1 = written(16 * sub + g + 8);
#pragma unroll
          for (int i = 0; i < NB / 2; ++i) d0[i] = w0 ? d0[i] : 0u, d1[i] = w1 ? d1[i] : 0u;
        }
        uint32_t w0[NT], w1[NT];
        if constexpr (BF16) {
          if (shift) {
            const __half2 f = __float2half2_rn(pow2(-top_exp));
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) d0[i] = mul_f16x2(d0[i], f), d1[i] = mul_f16x2(d1[i], f);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            w0[nt] = pack_f16(s[sub][nt][0], s[sub][nt][1]);
            w1[nt] = pack_f16(s[sub][nt][2], s[sub][nt][3]);
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t pick = b & 1 ? 0x7632u : 0x5410u;
          uint32_t x[4], y[4];
          signed_pairs(__byte_perm(va[b / 2], va[NB / 2 + b / 2], pick), magic, x);
          signed_pairs(__byte_perm(vb[b / 2], vb[NB / 2 + b / 2], pick), magic, y);
          const __half2 e0 = *reinterpret_cast<const __half2*>(&d0[b / 2]);
          const __half2 e1 = *reinterpret_cast<const __half2*>(&d1[b / 2]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (BF16) {
              const uint32_t u = transposed(mul_f16x2(w0[nt], b & 1 ? __high2half2(e0) : __low2half2(e0)));
              const uint32_t v = transposed(mul_f16x2(w1[nt], b & 1 ? __high2half2(e1) : __low2half2(e1)));
              mma_f16(o[nt][2 * b], x[0], x[1], y[0], y[1], u, v, o[nt][2 * b]);
              mma_f16(o[nt][2 * b + 1], x[2], x[3], y[2], y[3], u, v, o[nt][2 * b + 1]);
            } else {
              const float f0 = b & 1 ? __high2float(e0) : __low2float(e0);
              const float f1 = b & 1 ? __high2float(e1) : __low2float(e1);
              float a0 = s[sub][nt][0] * f0, a1 = s[sub][nt][1] * f0, b0 = s[sub][nt][2] * f1, b1 = s[sub][nt][3] * f1;
#pragma unroll
              for (int p = 0; p < NS; ++p) {
                const uint32_t u = transposed(take_f16(a0, a1)), v = transposed(take_f16(b0, b1));
                mma_f16(o[nt][2 * b], x[0], x[1], y[0], y[1], u, v, o[nt][2 * b]);
                mma_f16(o[nt][2 * b + 1], x[2], x[3], y[2], y[3], u, v, o[nt][2 * b + 1]);
              }
            }
          }
        }
      }

      return true;
      };
      if (hidden || !tile(std::false_type{})) tile(std::true_type{});

      // this slot is read: refill it
      __syncwarp();
      if (ahead < tile1) {
        if ((ahead_of & 31) == 0) fetch_pages(ahead);
        issue(ahead, ahead_of & 31, my_ring32 + slot);
        ++ahead_of;
        ahead += kWarps;
      }
      cp_async_commit();
      slot = slot + St::kBytes == St::kWarpBytes ? 0 : slot + St::kBytes;
    }

    // ---- the warps' results into shared memory (each over its own ring, which is drained)
    constexpr uint32_t kLd = D + 4;
    float* const mine = reinterpret_cast<float*>(my_ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const uint32_t r = nt * 8 + 2 * t + e;
        if (g == 0) s_m[warp * kRows + r] = m[nt][e], s_l[warp * kRows + r] = x;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          mine[r * kLd + 16 * i + g] = o[nt][i][e];
          mine[r * kLd + 16 * i + 8 + g] = o[nt][i][e + 2];
        }
      }
    __syncthreads();

    const uint32_t c0 = static_cast<uint32_t>(seg_begin / chunk), c1 = static_cast<uint32_t>((seg_end - 1) / chunk);
    const bool whole = c0 == c1;
    constexpr uint32_t kPart = kKvPartialRows * (D + 2);
    auto part_of = [&](uint32_t c) { return kv.partial + (static_cast<size_t>(c) * 2 + (c == c0)) * kPart; };
    auto store = [&](uint32_t r, uint32_t c, float4 v) {
      const uint32_t row = r0 + r;
      const uint64_t to = static_cast<uint64_t>(token0 + row / rows_group) * a.out_stride +
                          (kh * rows_group + row % rows_group) * D + c;
      if constexpr (BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = v;
    };
    for (uint32_t i = tid; i < n_rows * (D / 4); i += kThreads) {
      const uint32_t r = i / (D / 4), c = i % (D / 4) * 4;
      float top = s_m[r];
#pragma unroll
      for (uint32_t w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w * kRows + r]);
      float sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const float zero = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll
      for (uint32_t w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w * kRows + r] - zero);
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring + w * St::kWarpBytes) +
                                                          r * kLd + c);
        sum = fmaf(f, s_l[w * kRows + r], sum);
        v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);   // nothing seen: zeros
        store(r, c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
      } else {
        float* const p = part_of(blockIdx.x);
        __stcg(reinterpret_cast<float4*>(p + r * D + c), v);
        if (c == 0) __stcg(p + kKvPartialRows * D + r, top), __stcg(p + kKvPartialRows * (D + 1) + r, sum);
      }
    }
    if (!whole) {
      // The barrier orders the CTA's stores before its one arrival, which releases
      // them; the last arrival acquires all.
      __syncthreads();
      if (tid == 0) {
        const uint32_t arrived = arrive_acq_rel(kv.joined + c0);
        s_last = arrived == c1 - c0;
        if (s_last) kv.joined[c0] = 0;        // for the next call
      }
      __syncthreads();
      if (s_last) {
        for (uint32_t i = tid; i < n_rows * (D / 4); i += kThreads) {
          const uint32_t r = i / (D / 4), c = i % (D / 4) * 4;
          float top = -CUDART_INF_F;
#pragma unroll 8
          for (uint32_t k = c0; k <= c1; ++k) top = fmaxf(top, __ldcg(part_of(k) + kKvPartialRows * D + r));
          const float zero = top == -CUDART_INF_F ? 0.f : top;
          float sum = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (uint32_t k = c0; k <= c1; ++k) {
            const float* const p = part_of(k);
            const float f = ex2(__ldcg(p + kKvPartialRows * D + r) - zero);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(p + r * D + c));
            sum = fmaf(f, __ldcg(p + kKvPartialRows * (D + 1) + r), sum);
            v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
          }
          const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);   // nothing seen: zeros
          store(r, c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        }
      }
    }
    at += tile1 - tile0;
    __syncthreads();                          // the rings take copies again
  }
  if (blockIdx.x == gridDim.x - 1) zero_strays(kv, a, D * (BF16 ? 2 : 4));
}

template <int D, bool BF16, int NT>
cudaError_t decode(const KvDev& kv, const KvQuery& a, cudaStream_t st) {
  using St = Stage<D>;
  const uint32_t bytes = kWarps * (St::kWarpBytes + 2 * 4 * 8 * NT) + 8 * (a.n_seqs + 1);
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_kv_decode<D, BF16, NT>), 227 * 1024 - 512, &ready);
  if (e != cudaSuccess) return e;
  // resident CTAs of an SM: by shared memory (1 KB of it is the system's) and by the launch bound
  const uint32_t by_smem = 228 * 1024 / (bytes + 1024 + 256), by_regs = D <= 128 && BF16 && NT == 1 ? 4 : 2;
  const uint32_t per_sm = by_smem < by_regs ? by_smem : by_regs;
  uint32_t grid = sm_count() * (per_sm ? per_sm : 1);
  if (grid > kKvMaxCtas) grid = kKvMaxCtas;
  return launch_chained(k_kv_decode<D, BF16, NT>, dim3(grid), kThreads, bytes, st, kv, a);
}

template <int D>
cudaError_t attend_dim(const KvDev& kv, const KvQuery& a, cudaStream_t st) {
  // 16 rows of 256 channels do not fit the registers
  if constexpr (D <= 128) {
    if (static_cast<uint64_t>(a.max_new) * a.group > 8)
      return a.bf16 ? decode<D, true, 2>(kv, a, st) : decode<D, false, 2>(kv, a, st);
  }
  return a.bf16 ? decode<D, true, 1>(kv, a, st) : decode<D, false, 1>(kv, a, st);
}

}  // namespace

// Rows (new tokens x query heads of a kv head) of a sequence up to which this kernel
// serves it where the other is used.
constexpr uint32_t kFew = 48;

KvRoute kv_route(const KvDev& kv, const KvQuery& a, uint32_t sms) {
  // Which kernel.  Measured (bf16, contexts of 1024 to 16384 tokens, 1 to 64 sequences of
  // 3 to 192 new tokens, head_dim 64, 128 and 256): this one takes a constant time for a
  // group of rows and token tile, k_kv_prefill one for a CTA's token tile, whether its
  // rows are full or not; they break even at 4 groups an SM for each round of the
  // other's CTAs (all lengths alike, 16 sequences over 4096 tokens, 8 x 4 heads of 128:
  // 12 new tokens 74 here and 82 us there, 24 new tokens 124 and 85; one sequence over
  // 16384, 192 new tokens: 230 and 262).  f32 calls need the exact products of this one,
  // and so do sequences of more row tiles than the other's grid has.
  const uint64_t rows = static_cast<uint64_t>(a.n_tokens) * a.group, most = static_cast<uint64_t>(a.max_new) * a.group;
  const uint64_t groups = kv.heads * ((rows + (kv.dim == 256 ? 8 : 16) - 1) / (kv.dim == 256 ? 8 : 16));
  const uint64_t large = kv.dim == 256 ? 128 : 256, served = std::min<uint64_t>(a.n_seqs, rows / (kFew + 1));
  const uint64_t ctas = kv.heads * std::max((rows + large - 1) / large, served);
  if (!a.bf16 || most <= kFew || (most + large - 1) / large > 65535 || groups <= 4 * sms * ((ctas + sms - 1) / sms))
    return KvRoute::kFewRows;
  return kv.dim == 128 && kv_in_pairs(kv, a, sms) ? KvRoute::kPairs : KvRoute::kSingle;
}

cudaError_t launch_kv_attention(const KvDev& kv, const KvQuery& call, cudaStream_t st) {
  KvQuery a = call;
  const KvRoute route = kv_route(kv, a, sm_count());
  a.few = route == KvRoute::kFewRows ? 0xffffffffu : kFew;
  cudaError_t e;
  switch (kv.dim) {
    case 64: e = attend_dim<64>(kv, a, st); break;
    case 128: e = attend_dim<128>(kv, a, st); break;
    default: e = attend_dim<256>(kv, a, st); break;
  }
  return e == cudaSuccess && route != KvRoute::kFewRows ? launch_kv_prefill(kv, a, route, st) : e;
}

}  // namespace ovl
