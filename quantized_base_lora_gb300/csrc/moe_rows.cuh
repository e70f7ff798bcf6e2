// The experts' matrix products of a mixture-of-experts layer for a few tokens.
//
//   k_moe_rows<.., false>  act(gate_e x) * (up_e x) of every chosen (token, expert) pair
//   k_moe_rows<.., true>   weight * down_e h of every pair
//
// Each chosen expert's weights are read once for up to kMoeTokens of its tokens, so for a
// few tokens the bound is memory; the arithmetic has to keep out of its way.  A warp has
// 32 rows of an expert (16 gate and 16 up rows of the same outputs, or 32 down rows) and
// streams them in stages of 128 bytes a row through a ring of its own in shared memory,
// by asynchronous copies that need no barrier among warps.  The codes go into
// mma.sync.m16n8k16 as they are, exact in bf16, with 8 tokens as its columns; the products
// of one 32-weight block are summed in fp32 and multiplied by the block's scale there.  A
// tcgen05 MMA has at least 64 rows and its operands in shared or tensor memory, which would
// cost a conversion pass per token and expert; at up to 8 columns the tensor pipe of
// mma.sync is idle most of the time as it is.
//
// Measured (graph of calls, the whole layer): one fp32 token over two q8_0 experts of 4096 x
// 14336 (375 MB) 80 us; one bf16 token over 8 of 128 q4_0 experts of 2048 x 768 (22 MB) 20; 64
// tokens over the same experts (336 MB) 110; 19 over 64 q4_K experts of 2048 x 1280 (240 MB) 76.
// The first product's copies alone take 0.7 of its time, the arithmetic alone as much: 75
// instructions a 1024 weights, half of the issue slots, waits for fixed latencies between
// them.
//
// Inputs are bf16 parts (one: bf16 tokens; three: all 24 bits of fp32 tokens, and of the
// activations of either call) in the order of the fragments: lane t of a quad takes 8
// consecutive channels of a block in one load, stored as the pairs in which a word's codes
// unpack.  Activations of bf16 calls in two parts, 2^-17 of each, took 100 us instead of 111
// over 64 tokens and 69 instead of 76 over 19, and no less over one; but outputs that cancel
// showed it, and one output in about 1500 was rounded otherwise for it.  A
// unit of so few tokens that all their parts find room in the 8 columns has the parts
// beside one another, added up at the end (one fp32 token: a third of the MMAs and loads).
#pragma once
#include <atomic>
#include <type_traits>

#include "block_internal.h"

namespace ovl {
namespace moe {

// Warps of a CTA.  16 have 128 registers each and leave less of the SM to the cache, 12 have
// 168; q4_K holds the most in both, then three parts.  Both products with 12 against 16, the
// whole layer in us:
//                                             q8_0 bf16   fp32       q4_0 bf16   fp32       q4_K bf16   fp32
//   1 token, 2 experts of 4096 x 14336        84.7/78.8   85.7/80.2  62.6/57.7   60.5/60.5  61.9/62.5   66.2/69.9
//   1 token, 8 of 128 experts of 2048 x 768   21.2/21.2   21.8/22.2  19.7/20.7   19.7/22.0  19.6/21.7   20.9/24.2
//   64 tokens over the same                   153/152     183/180    112/109     140/146    120/123     169/181
// The rule is the better one over the three together, for each instance, not in each of them.  (The
// first product of q8_0 in fp32 spills 8 bytes a thread at 16 warps.  With 12 in the second and 16
// in the first, bf16 calls of q4_0 take 56.7, 19.8 and 109.5.)
template <uint32_t Q, int PARTS>
constexpr uint32_t kWarps = Q == OVL_Q4_K || (Q == OVL_Q4_0 && PARTS == 3) ? 12 : 16;
constexpr int kStages = 2;
constexpr uint32_t kRowBytes = 128;                       // of a row in one stage: 8 pieces of 16
constexpr uint32_t kScaleBytes = 20;                      // of a row in one stage: 16, or five words around 16 bytes
constexpr uint32_t kStageBytes = 32 * (kRowBytes + kScaleBytes);
constexpr uint32_t kJoinBytes = kMoeTokens * 32 * 4;      // a warp's sums

// Shared memory of a CTA.  It stays within 175 KB, so that the rest of the SM's 256 KB is
// cache for the inputs, which every warp reads: at 206 KB, 20 to 57 percent of those loads
// hit, and one token over two experts of 14336 took 110 us instead of 90.
template <uint32_t Q, int PARTS>
struct Shape {
  static constexpr uint32_t kTableBytes = Q == OVL_Q4_K ? 2 * 8 * 32 * 4 : 0;         // a warp's scales and minimums of a stage
  static constexpr uint32_t kTables = kWarps<Q, PARTS> * kStages * kStageBytes, kJoins = kTables + kWarps<Q, PARTS> * kTableBytes,
                            kUnits = kJoins + (kWarps<Q, PARTS> - 1) * kJoinBytes, kOrder = kUnits + kMoeMaxUnits * sizeof(MoeUnit),
                            kSmem = kOrder + kMoeMaxPairs * 2;
  static_assert(kStageBytes % 128 == 0, "slots begin on 128 bytes");
  static_assert(kSmem + 64 <= 175 * 1024, "what is left to the cache");
};

__device__ __forceinline__ void cp_async4_if(uint32_t dst, const void* src, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.ca.shared.global [%0], [%1], 4;\n\t}" ::"r"(dst),
               "l"(src), "r"(static_cast<uint32_t>(on))
               : "memory");
}
// OFF: added to the address in shared memory.
template <int BYTES, int OFF>
__device__ __forceinline__ void cp_async_at(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1], 16;" ::"r"(dst), "l"(src), "n"(OFF) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0 + %2], [%1], %3;" ::"r"(dst), "l"(src), "n"(OFF), "n"(BYTES) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float* c) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// 8x8 16-bit matrices of four groups of 8 rows of 16 bytes: lane l gives the address of row
// l and gets word l % 4 of rows l / 4 + 8 i.
__device__ __forceinline__ void load_rows(uint32_t (&w)[4], uint32_t address) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(address)
               : "memory");
}

// A word of codes as bf16 pairs, exactly and without any arithmetic: the integer n <= 255 in
// the low bits of a bf16 is n 2^-133 (below 128 a subnormal, from there on the first
// binade, which goes on in the same steps).
//   4 bits: pair 0 is codes 0 and 4, pair 1 16 times codes 1 and 5, and so on: the inputs
//   of odd channels are stored a 16th as large.
//   8 bits: code + 128; pairs 0 and 1 of a word.
// What the codes are too large by (8 and 128) is, for inputs in one part, a product with the
// same constant in every place, from which the MMAs of the block start: an MMA then cuts its
// sums as for codes of 128, 4 bits more than 4-bit codes need, which bf16 inputs have to
// spare (signed codes gave outputs no nearer to the plain form's, and took 4 % longer).  For
// three parts it is subtracted from every code: the sums then are no larger than they have to
// be, which their 24 bits are needed for, and three parts would be six more MMAs a block.
constexpr int kCodeExponent = 133;
__device__ __forceinline__ void pairs_of_4(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t h = w >> 8;
  p[0] = w & 0x000f000fu, p[1] = w & 0x00f000f0u, p[2] = h & 0x000f000fu, p[3] = h & 0x00f000f0u;
}
__device__ __forceinline__ void pairs_of_8(uint32_t w, uint32_t& p0, uint32_t& p1) {
  w ^= 0x80808080u;
  p0 = __byte_perm(w, 0, 0x4140), p1 = __byte_perm(w, 0, 0x4342);
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Place of channel c of a block of 32 in the order in which lanes take them.
template <uint32_t Q>
__device__ __forceinline__ uint32_t place_of(uint32_t c) {
  if constexpr (Q == OVL_Q8_0) return (c & 12) * 2 + (c >> 4) * 4 + (c & 3);
  else return (c & 24) + ((c & 4) ? 2 * (c & 7) - 7 : 2 * (c & 7));
}
// What its input is multiplied by.
template <uint32_t Q>
__device__ __forceinline__ float share_of(uint32_t c) {
  return Q != OVL_Q8_0 && (c & 1) ? 0.0625f : 1.f;
}

// Inputs are scaled by powers of two, so that the products stay in fp32's range: a token's
// largest |x| to 2^kTokenExponent and up to twice that, with 2^e the power of two below it;
// the activations by 2^(kActExponent - 2 e), since they go with the square of x.  At
// 2^kActExponent, activations 2^77 times and 2^-20 times max|x|^2 are within range, with all of
// the sums' 24 bits.
__host__ __device__ constexpr float pow2(int e) { return e == 0 ? 1.f : e > 0 ? 2.f * pow2(e - 1) : 0.5f * pow2(e + 1); }
constexpr int kTokenExponent = 100;
constexpr int kActExponent = 50;

// v as bf16 parts: the upper bits cut off, exactly, so that three parts are all 24 bits.
// One part is for values that are bf16 as they are.
template <int PARTS>
__device__ __forceinline__ void parts_of(float v, uint16_t (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    if (PARTS == 1) {
      p[i] = static_cast<uint16_t>(two_bf16(v, v));
      break;
    }
    const uint32_t u = v != v ? 0x7fc00000u : __float_as_uint(v) & 0xffff0000u;
    p[i] = static_cast<uint16_t>(u >> 16);
    const float rest = v - __uint_as_float(u);
    v = fabsf(v) <= 3.402823466e38f ? rest : 0.f;        // of an infinity or NaN nothing is left
  }
}

// Where the share of CTA `cta` begins, of n.
__device__ __forceinline__ uint32_t share(uint32_t n, uint32_t cta) {
  return n / gridDim.x * cta + n % gridDim.x * cta / gridDim.x;
}

// The chosen pairs sorted by expert, in pair order within one, and cut into units: by every
// CTA for itself, in shared memory (less work than to wait for one to do it).  An entry of
// the order is token << 4 | place, which saves the divisions behind it.  The CTA's items are
// range[0] .. range[1] - 1, of range[2] units: runs of tiles of equal cost, where a unit
// whose parts do not fit beside one another counts half as much again.
template <uint32_t Q, int PARTS>
__device__ __forceinline__ void sort_pairs(const MoeDev& m, uint8_t* smem, uint32_t tiles, uint32_t (&range)[3]) {
  MoeUnit* units = reinterpret_cast<MoeUnit*>(smem + Shape<Q, PARTS>::kUnits);
  uint16_t* order = reinterpret_cast<uint16_t*>(smem + Shape<Q, PARTS>::kOrder);
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int32_t* choice = m.given ? m.given_choice : m.choice;
  if (m.tokens == 1 && !m.given) {                        // distinct experts with one pair each
    if (threadIdx.x < m.top) {
      // the router's own, and an expert in any case: a workspace that calls raced on may hold anything
      const uint32_t expert = min(static_cast<uint32_t>(choice[threadIdx.x]), m.experts - 1);
      units[threadIdx.x] = MoeUnit::make(expert, 1, threadIdx.x, 1, threadIdx.x);
      order[threadIdx.x] = static_cast<uint16_t>(threadIdx.x);       // place threadIdx.x of token 0
    }
    if (threadIdx.x < 2) range[threadIdx.x] = share(m.top * tiles, blockIdx.x + threadIdx.x);
    if (threadIdx.x == 2) range[2] = m.top;
    __syncthreads();
    return;
  }
  // scratch where the ring will be: pairs of each expert in each warp's share, first pairs,
  // sums, the pairs' experts and their places in their warp's share.  Loops are not unrolled:
  // each line of instructions comes from L2 here.
  uint16_t* count = reinterpret_cast<uint16_t*>(smem);                   // [kWarps][OVL_MOE_MAX_EXPERTS]
  uint16_t* first = count + kWarps<Q, PARTS> * OVL_MOE_MAX_EXPERTS;
  uint32_t* sums = reinterpret_cast<uint32_t*>(first + OVL_MOE_MAX_EXPERTS);      // [3][kWarps]
  uint32_t* expert_rank = sums + 3 * kWarps<Q, PARTS>;              // [kMoeMaxPairs], of a warp's own pairs
  static_assert(kWarps<Q, PARTS> * 32 >= OVL_MOE_MAX_EXPERTS / 2 && OVL_MOE_MAX_TOP <= 16, "two experts a thread; an entry's fields");
  const uint32_t per = (m.pairs + kWarps<Q, PARTS> * 32 - 1) / (kWarps<Q, PARTS> * 32), from = warp * per * 32 + lane;
  const uint32_t own = 2 * threadIdx.x;                   // the thread's experts: own and own + 1
  if (own < m.experts) {
#pragma unroll 1
    for (uint32_t w = 0; w < kWarps<Q, PARTS>; ++w) *reinterpret_cast<uint32_t*>(count + w * OVL_MOE_MAX_EXPERTS + own) = 0;
  }
  __syncthreads();
#pragma unroll 1
  for (uint32_t r = 0; r < per; ++r) {
    const uint32_t p = from + r * 32;
    uint32_t e = p < m.pairs ? static_cast<uint32_t>(choice[p]) : m.experts;
    if (e >= m.experts) e = OVL_MOE_MAX_EXPERTS;          // none
    const uint32_t same = __match_any_sync(0xffffffffu, e), below = __popc(same & ((1u << lane) - 1));
    uint16_t* c = count + warp * OVL_MOE_MAX_EXPERTS + e;
    const bool some = e < OVL_MOE_MAX_EXPERTS;
    if (p < m.pairs) expert_rank[p] = e << 16 | (some ? *c + below : 0);
    __syncwarp();
    if (some && below == 0) *c = static_cast<uint16_t>(*c + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  uint32_t n[2] = {0, 0};                                 // their pairs
  if (own < m.experts) {
#pragma unroll 1
    for (uint32_t w = 0; w < kWarps<Q, PARTS>; ++w) {
      uint32_t* c = reinterpret_cast<uint32_t*>(count + w * OVL_MOE_MAX_EXPERTS + own);
      const uint32_t some = *c;
      *c = n[0] | n[1] << 16;
      n[0] += some & 0xffff, n[1] += some >> 16;
    }
  }
  const uint32_t groups[2] = {(n[0] + kMoeTokens - 1) / kMoeTokens, (n[1] + kMoeTokens - 1) / kMoeTokens};
  auto cost_of = [](uint32_t pairs) { return !pairs ? 0u : pairs * PARTS <= 8 ? 2u : 3u; };
  uint32_t cost[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) cost[j] = n[j] / kMoeTokens * cost_of(kMoeTokens) + cost_of(n[j] % kMoeTokens);
  uint32_t a = n[0] + n[1], b = groups[0] + groups[1], c = cost[0] + cost[1];    // pairs, units and costs up to them
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, a, s), v = __shfl_up_sync(0xffffffffu, b, s), w = __shfl_up_sync(0xffffffffu, c, s);
    if (static_cast<int>(lane) >= s) a += u, b += v, c += w;
  }
  if (lane == 31) sums[warp] = a, sums[kWarps<Q, PARTS> + warp] = b, sums[2 * kWarps<Q, PARTS> + warp] = c;
  __syncthreads();
  uint32_t all = 0, whole = 0;
#pragma unroll 1
  for (uint32_t w = 0; w < kWarps<Q, PARTS>; ++w) {
    if (w < warp) a += sums[w], b += sums[kWarps<Q, PARTS> + w], c += sums[2 * kWarps<Q, PARTS> + w];
    all += sums[kWarps<Q, PARTS> + w], whole += sums[2 * kWarps<Q, PARTS> + w];
  }
  a -= n[0] + n[1], b -= groups[0] + groups[1], c -= cost[0] + cost[1];
  if (threadIdx.x == 0) range[2] = all;
  uint32_t from_cost[2];                                  // below 768 units * 3 * 2048 tiles
#pragma unroll
  for (uint32_t k = 0; k < 2; ++k) {
    from_cost[k] = share(whole * tiles, blockIdx.x + k);
    if (threadIdx.x == 0 && from_cost[k] == whole * tiles) range[k] = all * tiles;
  }
#pragma unroll
  for (uint32_t j = 0; j < 2; ++j) {
    if (own + j < m.experts) first[own + j] = static_cast<uint16_t>(a);
    for (uint32_t i = 0; i < groups[j]; ++i)
      units[b + i] = MoeUnit::make(own + j, min(n[j] - i * kMoeTokens, kMoeTokens), b, groups[j], a + i * kMoeTokens);
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {                    // the first tile that begins there or behind it
      const uint32_t at = from_cost[k] - c * tiles;
      if (from_cost[k] >= c * tiles && at < cost[j] * tiles) range[k] = b * tiles + (at + cost[j] - 1) / cost[j] * groups[j];
    }
    a += n[j], b += groups[j], c += cost[j];
  }
  __syncthreads();
#pragma unroll 1
  for (uint32_t r = 0; r < per; ++r) {
    const uint32_t p = from + r * 32;
    if (p >= m.pairs) break;
    const uint32_t e = expert_rank[p] >> 16, rank = expert_rank[p] & 0xffff;
    const uint32_t token = p / m.top;
    if (e < OVL_MOE_MAX_EXPERTS)
      order[first[e] + count[warp * OVL_MOE_MAX_EXPERTS + e] + rank] = static_cast<uint16_t>(token << 4 | (p - token * m.top));
  }
  __syncthreads();
}

// An item: 32 rows of a unit.  An expert's units lie side by side for each tile, so that its
// weights are in L2 for the second and later ones.
struct Item {
  MoeUnit unit;
  uint32_t tile, place, next;  // tile; the unit's place in its group; the first unit behind the group
  __device__ void find(const MoeUnit* units, uint32_t tiles, uint32_t item) {
    const MoeUnit any = units[item / tiles];
    const uint32_t g = any.group(), n = any.groups(), r = item - g * tiles;
    tile = n == 1 ? r : r / n;
    place = r - tile * n;
    next = g + n;
    unit = units[g + place];
  }
  // The one behind it; none behind the last unit's last.
  __device__ void advance(const MoeUnit* units, uint32_t tiles, uint32_t n_units) {
    const uint32_t n = unit.groups();
    if (++place < n) {
      unit = units[next - n + place];
      return;
    }
    place = 0;
    if (++tile == tiles) {
      tile = 0;
      if (next == n_units) return;
      unit = units[next];
      next += unit.groups();
    } else if (n > 1) {
      unit = units[next - n];
    }
  }
};

// Where a warp's copies are.
struct Cursor {
  const uint8_t* row[2];       // the lane's next piece: of the first and of the last 16 rows
  const uint8_t* scale;        // the lane's row of scales
  uint32_t stage;
  Item item;
};

// DOWN: the second product.  PARTS: of its input.
template <uint32_t Q, bool DOWN, int PARTS>
struct Rows32 {
  static constexpr uint32_t kBlocks = Q == OVL_Q8_0 ? 4 : 8;            // 32-weight blocks of a stage
  static constexpr bool kSigned = PARTS == 3;
  static constexpr int kScales = Q == OVL_Q8_0 ? 8 : 16;                // bytes of a row's scales in a stage

  const MoeDev& m;
  const MoeUnit* units;        // in shared memory
  uint8_t* ring;               // the warp's
  float* table;
  uint32_t lane, k, pitch, scale_pitch, tiles;
  bool scales_aligned;

  __device__ Rows32(const MoeDev& dev, uint8_t* smem)
      : m(dev), units(reinterpret_cast<const MoeUnit*>(smem + Shape<Q, PARTS>::kUnits)) {
    lane = threadIdx.x & 31;
    ring = smem + threadIdx.x / 32 * kStages * kStageBytes;
    table = reinterpret_cast<float*>(smem + Shape<Q, PARTS>::kTables + threadIdx.x / 32 * Shape<Q, PARTS>::kTableBytes);
    k = DOWN ? m.ffn : m.hidden;
    pitch = Q == OVL_Q8_0 ? k : k / 2;
    scale_pitch = k / 16;                                               // 2 bytes a block; 16 bytes of 256 weights
    scales_aligned = scale_pitch % kScales == 0;
    tiles = DOWN ? m.hidden / 32 : m.ffn / 16;
  }

  // To stage `stage` of the cursor's item.
  __device__ void at(Cursor& c, uint32_t stage) const {
    c.stage = stage;
    const uint32_t expert = c.item.unit.expert(), tile = c.item.tile, r = lane / 8;
    const uint64_t piece = lane % 8 * 16 + stage * kRowBytes;
    if constexpr (DOWN) {
      const uint64_t first = static_cast<uint64_t>(expert) * m.hidden + tile * 32;
      c.row[0] = m.down_qs + (first + r) * pitch + piece;
      c.row[1] = c.row[0] + 16ull * pitch;
      c.scale = m.down_d + (first + lane) * scale_pitch + stage * kScales;
    } else {
      const uint64_t first = static_cast<uint64_t>(expert) * m.ffn + tile * 16;
      c.row[0] = m.gate_qs + (first + r) * pitch + piece;
      c.row[1] = m.up_qs + (first + r) * pitch + piece;
      c.scale = (lane < 16 ? m.gate_d : m.up_d) + (first + (lane & 15)) * scale_pitch + stage * kScales;
    }
  }

  // Asks for stage c.stage of the item and goes on to the next.  Piece p of row r lies at
  // piece p ^ (r % 8), so that the 8 rows of a matrix meet different banks.
  __device__ __forceinline__ void fill(Cursor& c, uint32_t slot) const {
    const uint32_t at = smem_u32(ring) + slot * kStageBytes, r = lane / 8, piece = lane % 8;
    if (c.stage * kRowBytes + piece * 16 < pitch) {
      const uint32_t even = at + r * kRowBytes + ((piece ^ r) << 4), odd = even ^ 64;      // rows r + 8 i, r + 4 + 8 i
      const uint8_t *p = c.row[0], *q = c.row[1];
      const uint64_t step = 4 * pitch;
      cp_async_at<16, 0>(even, p);
      cp_async_at<16, 4 * kRowBytes>(odd, p += step);
      cp_async_at<16, 8 * kRowBytes>(even, p += step);
      cp_async_at<16, 12 * kRowBytes>(odd, p += step);
      cp_async_at<16, 16 * kRowBytes>(even, q);
      cp_async_at<16, 20 * kRowBytes>(odd, q += step);
      cp_async_at<16, 24 * kRowBytes>(even, q += step);
      cp_async_at<16, 28 * kRowBytes>(odd, q += step);
    }
    if (Q == OVL_Q4_K || scales_aligned) {
      cp_async_at<kScales, 32 * kRowBytes>(at + lane * kScales, c.scale);
    } else {                                                            // rows of scales begin at any even address
      const uint32_t shift = (lane & 1) * (scale_pitch & 2);            // a tile begins at an even row
      const uint32_t have = min(static_cast<uint32_t>(kScales), scale_pitch - c.stage * kScales) + shift;
#pragma unroll
      for (uint32_t i = 0; i < kScales / 4 + 1; ++i)
        cp_async4_if(at + 32 * kRowBytes + lane * kScaleBytes + 4 * i, c.scale - shift + 4 * i, 4 * i < have);
    }
    c.row[0] += kRowBytes, c.row[1] += kRowBytes, c.scale += kScales;
    ++c.stage;
  }

  // A stage's scales of row r.
  __device__ const uint16_t* scales_of(uint32_t slot, uint32_t r) const {
    const uint8_t* raw = ring + slot * kStageBytes + 32 * kRowBytes;
    return reinterpret_cast<const uint16_t*>(scales_aligned ? raw + r * kScales : raw + r * kScaleBytes + (r & 1) * (scale_pitch & 2));
  }

  // Q4_K: a stage's scales and minimums as fp32: table[block][row % 8][row / 8], minimums behind.
  __device__ void decode(uint32_t slot) const {
    const uint4 h = *reinterpret_cast<const uint4*>(ring + slot * kStageBytes + 32 * kRowBytes + lane * 16);
    const uint32_t place = (lane & 7) * 4 + (lane >> 3);
    const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
    const uint64_t sc = h.y | (static_cast<uint64_t>(h.z & 0xffffu) << 32), mn = (h.z >> 16) | (static_cast<uint64_t>(h.w) << 16);
#pragma unroll
    for (uint32_t b = 0; b < 8; ++b) {
      const float scale = d.x * static_cast<float>(static_cast<uint32_t>(sc >> (6 * b)) & 63u);
      const float least = -d.y * static_cast<float>(static_cast<uint32_t>(mn >> (6 * b)) & 63u);
      table[b * 32 + place] = scale;
      table[(8 + b) * 32 + place] = 0x1p-7f * (kSigned ? fmaf(8.f, scale, least) : least);
    }
  }

  // The inputs of a block: `at` is the lane's byte in the first part.  The blocks behind a
  // row's last one lie in the workspace too.
  template <int P>
  __device__ void inputs(uint32_t at, uint32_t part, uint4 (&v)[P]) const {
    const char* base = reinterpret_cast<const char*>(DOWN ? m.hp : m.xp);
#pragma unroll
    for (int q = 0; q < P; ++q) v[q] = *reinterpret_cast<const uint4*>(base + (at + q * part));
  }

  // One stage's products: acc[half of the rows][fragment] += scale * codes x, x in P parts
  // one behind the other.  `next` holds the inputs of the two blocks to come (for three parts
  // there is no room).
  template <int P>
  static constexpr bool kAhead = P < 3;
  template <int P>
  __device__ __forceinline__ void multiply(uint32_t slot, uint32_t stage, uint32_t x, uint32_t part, uint4 (&next)[2][P],
                                           float (&acc)[2][4]) const {
    const uint32_t first = stage * kBlocks, blocks = min(kBlocks, k / 32 - first);
    if (blocks == kBlocks) {
      // Four blocks a round, not more: instructions come from L2 when a kernel begins, and
      // unrolled over the stage its first microseconds went there.
#pragma unroll 1
      for (uint32_t b = 0; b < kBlocks; b += 4) {
        uint2 packed[4];                         // scales of rows g + 8 i
        if constexpr (Q != OVL_Q4_K) {
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            const uint16_t* s = scales_of(slot, (lane >> 2) + 8 * i) + b;
            if (scales_aligned) packed[i] = *reinterpret_cast<const uint2*>(s);
            else packed[i] = make_uint2(s[0] | static_cast<uint32_t>(s[1]) << 16, s[2] | static_cast<uint32_t>(s[3]) << 16);
          }
        }
#pragma unroll
        for (uint32_t c = 0; c < 4; c += 2) {
          float scale[2][4], least[2][4];
          if constexpr (Q == OVL_Q4_K) {
            from_table(b + c, scale[0], least[0]);
            from_table(b + c + 1, scale[1], least[1]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(c ? &packed[i].y : &packed[i].x));
              scale[0][i] = f.x, scale[1][i] = f.y;
            }
          }
          uint32_t codes[2][kWords][4];
          codes_of(slot, b + c, codes[0]);
          codes_of(slot, b + c + 1, codes[1]);
          multiply_blocks<2, P>(codes, first + b + c, x, part, scale, least, next, acc);
        }
      }
    } else {                                     // the row's last stage
#pragma unroll 1
      for (uint32_t b = 0; b < blocks; ++b) {
        float scale[1][4], least[1][4];
        if constexpr (Q == OVL_Q4_K) {
          from_table(b, scale[0], least[0]);
        } else {
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i)
            scale[0][i] = __half2float(__ushort_as_half(scales_of(slot, (lane >> 2) + 8 * i)[b]));
        }
        uint32_t codes[1][kWords][4];
        codes_of(slot, b, codes[0]);
        multiply_blocks<1, P>(codes, first + b, x, part, scale, least, next, acc);
      }
    }
  }
  __device__ __forceinline__ void from_table(uint32_t b, float (&scale)[4], float (&least)[4]) const {
    const float4 u = *reinterpret_cast<const float4*>(table + b * 32 + (lane >> 2) * 4);
    const float4 v = *reinterpret_cast<const float4*>(table + (8 + b) * 32 + (lane >> 2) * 4);
    scale[0] = u.x, scale[1] = u.y, scale[2] = u.z, scale[3] = u.w;
    least[0] = v.x, least[1] = v.y, least[2] = v.z, least[3] = v.w;
  }

  // The lane's words of block b, rows of both halves.
  static constexpr int kWords = Q == OVL_Q8_0 ? 2 : 1;
  __device__ __forceinline__ void codes_of(uint32_t slot, uint32_t b, uint32_t (&w)[kWords][4]) const {
    const uint32_t row = smem_u32(ring) + slot * kStageBytes + lane * kRowBytes;
#pragma unroll
    for (uint32_t s = 0; s < kWords; ++s) load_rows(w[s], row + (((kWords * b + s) ^ (lane & 7)) << 4));
  }

  // N blocks beside one another, so that their chains of MMAs fill each other's waits.
  template <int N, int P>
  __device__ __forceinline__ void multiply_blocks(const uint32_t (&codes)[N][kWords][4], uint32_t block, uint32_t x, uint32_t part,
                                                  const float (&scale)[N][4], const float (&least)[N][4],
                                                  uint4 (&next)[2][P], float (&acc)[2][4]) const {
    uint4 xs[N][P];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if constexpr (kAhead<P> && N == 2) {
#pragma unroll
        for (int q = 0; q < P; ++q) xs[n][q] = next[n][q];
        inputs(x + (block + 2 + n) * 64, part, next[n]);
      } else {
        inputs(x + (block + n) * 64, part, xs[n]);
      }
    }
    uint32_t a[N][2][2][4];                      // block, half of the rows, k16 step, fragment
#pragma unroll
    for (uint32_t n = 0; n < N; ++n) {
      if constexpr (Q == OVL_Q8_0) {
#pragma unroll
        for (uint32_t s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) pairs_of_8(codes[n][s][i], a[n][i / 2][s][i % 2], a[n][i / 2][s][2 + i % 2]);
      } else {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pairs_of_4(codes[n][0][i], p);
#pragma unroll
          for (int s = 0; s < 2; ++s) a[n][i / 2][s][i % 2] = p[2 * s], a[n][i / 2][s][2 + i % 2] = p[2 * s + 1];
        }
      }
    }
    if constexpr (kSigned) {
      constexpr uint32_t even = Q == OVL_Q8_0 ? 0x00800080u : 0x00080008u, odd = 0x00800080u;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) a[n][i / 8][i / 4 % 2][i % 4] = sub_bf16x2(a[n][i / 8][i / 4 % 2][i % 4], i % 4 < 2 ? even : odd);
    }
    // The block's inputs added up, in every row: times -8, 128 (Q4_K) or -128 2^-133.  (Of a
    // subnormal, the bits in front of its first one are lost to the product: hence not 1.)
    constexpr bool kSum = Q == OVL_Q4_K || !kSigned;
    constexpr uint32_t one = Q == OVL_Q8_0 ? 0x80808080u : Q == OVL_Q4_0 ? 0x80088008u : 0x00800080u;
    constexpr uint32_t odd = Q == OVL_Q8_0 ? one : Q == OVL_Q4_0 ? 0x80808080u : 0x02800280u;
    const uint32_t same[4] = {one, one, odd, odd};
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    float sum[N][4], p[N][2][4];
    // small parts first: the MMAs cut off their sums
#pragma unroll
    for (int q = kSum ? P - 1 : -1; q >= 0; --q)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int n = 0; n < N; ++n)
          mma_bf16(sum[n], same, s ? xs[n][q].z : xs[n][q].x, s ? xs[n][q].w : xs[n][q].y, q == P - 1 && s == 0 ? zero : sum[n]);
#pragma unroll
    for (int q = P - 1; q >= 0; --q)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            mma_bf16(p[n][h], a[n][h][s], s ? xs[n][q].z : xs[n][q].x, s ? xs[n][q].w : xs[n][q].y,
                     q < P - 1 || s ? p[n][h] : Q == OVL_Q4_K || kSigned ? zero : sum[n]);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[h][i] = fmaf(scale[n][2 * h + (i >> 1)], p[n][h][i], acc[h][i]);
          if constexpr (Q == OVL_Q4_K) acc[h][i] = fmaf(least[n][2 * h + (i >> 1)], sum[n][i], acc[h][i]);
        }
  }

  // What an item's sums become.
  // `w`: the lane's pair's weight, power: its token's 2^e.
  __device__ void finish(uint32_t tile, uint32_t n_pairs, int32_t pair, float w, float power, bool beside, float (&acc)[2][4]) const {
    const uint32_t g = lane >> 2, t = lane & 3;
    if (beside) {                                // column c's parts are columns c + n, c + 2 n: the small ones first
      float all[8];
#pragma unroll
      for (int q = PARTS - 1; q >= 0; --q) {
        const uint32_t by = q * n_pairs;         // odd: the other one of a lane's two columns
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t from = (2 * t + (i & 1) + by) & 7;
          const float v = __shfl_sync(0xffffffffu, (by & 1) ? acc[i / 4][(i & 3) ^ 1] : acc[i / 4][i & 3], (lane & 28) + from / 2);
          all[i] = q == PARTS - 1 ? v : all[i] + v;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i / 4][i & 3] = all[i];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t column = 2 * t + j;
      const int32_t p = __shfl_sync(0xffffffffu, pair, column);
      const float weight = __shfl_sync(0xffffffffu, w, column), up = __shfl_sync(0xffffffffu, power, column);
      if (column >= n_pairs) continue;
      if constexpr (DOWN) {
        constexpr float back = pow2(kCodeExponent - kActExponent);
        float* out = m.part + static_cast<uint64_t>(p) * m.hidden + tile * 32 + g;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) out[h * 16 + e * 8] = weight * (acc[h][2 * e + j] * back * up * up);
      } else {
        constexpr int kParts = 3;                // of the second product's input
        constexpr float back = pow2(kCodeExponent - kTokenExponent), scaled = pow2(kActExponent);
        const float down = 1.f / up;             // a power of two
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float gate = activated(acc[0][2 * e + j] * back * up, m.act) * down;
          const uint32_t c = (tile & 1) * 16 + e * 8 + g;
          uint16_t v[kParts];
          parts_of<kParts>(gate * share_of<Q>(c) * (acc[1][2 * e + j] * back) * scaled, v);
          uint16_t* out = m.hp + static_cast<uint64_t>(p) * m.ffn + (tile >> 1) * 32 + place_of<Q>(c);
#pragma unroll
          for (int q = 0; q < kParts; ++q) out[q * static_cast<uint64_t>(m.pairs) * m.ffn] = v[q];
        }
      }
    }
  }
};

template <uint32_t Q, bool DOWN, int PARTS>
__global__ void __launch_bounds__(kWarps<Q, PARTS> * 32, 1) k_moe_rows(const __grid_constant__ MoeDev m) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  // The first product waits for the router before it lets the second start, so that the
  // second may read the router's results and ask for weights before the first has ended.
  __shared__ uint32_t range[3];
  const Rows32<Q, DOWN, PARTS> op(m, smem);
  if constexpr (!DOWN) {
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x < kMoeGroups) m.arrived[threadIdx.x] = 0;     // the next call's routers wait for this one's end
  }
  sort_pairs<Q, PARTS>(m, smem, op.tiles, range);
  const uint16_t* order = reinterpret_cast<const uint16_t*>(smem + Shape<Q, PARTS>::kOrder);
  // Items in runs of equal cost to the CTAs; inside a CTA, their stages in equal runs to the
  // warps.  An item whose stages are divided is finished by the warp that has its first
  // ones, last thing; the others come to it first thing and leave their sums in shared memory.
  const uint32_t begin = range[0], end = range[1];
  const uint32_t stages = (op.pitch + kRowBytes - 1) / kRowBytes, total = (end - begin) * stages;
  auto start_of = [&](uint32_t w) { return total / kWarps<Q, PARTS> * w + total % kWarps<Q, PARTS> * w / kWarps<Q, PARTS>; };
  const uint32_t p0 = start_of(warp), p1 = start_of(warp + 1);
  Cursor c{};
  uint32_t asked = p0, slot_in = 0;
  if (p0 < p1) {
    c.item.find(op.units, op.tiles, begin + p0 / stages);
    op.at(c, p0 % stages);
  }
  Item now = c.item;
  const uint32_t n_units = range[2];
  auto ask = [&]() {
    if (asked < p1) {
      op.fill(c, slot_in);
      if (++asked < p1 && c.stage == stages) {
        c.item.advance(op.units, op.tiles, n_units);
        op.at(c, 0);
      }
    }
    cp_async_commit();
    slot_in = slot_in + 1 == kStages ? 0 : slot_in + 1;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ask();
  if constexpr (DOWN) {
    griddep_wait();
    griddep_launch_dependents();
  }
  const uint32_t part = (DOWN ? m.pairs : m.tokens) * op.k * 2;
  const float* weights = m.given ? m.given_weight : m.weight;
  float* mine = reinterpret_cast<float*>(smem + Shape<Q, PARTS>::kJoins) + (static_cast<int>(warp) - 1) * static_cast<int>(kJoinBytes / 4) + lane;    // not of warp 0
  uint32_t slot = 0;
  bool divided = false, beside = false;                   // whether others have stages of the last item; parts in columns
  uint32_t n_pairs = 0, s0 = p0 % stages;
  int32_t pair = 0;
  float w = 0.f, power = 1.f, acc[2][4];
  uint32_t p = p0;
  while (p < p1) {
    const uint32_t s1 = min(stages, s0 + (p1 - p));
    p += s1 - s0;
    n_pairs = now.unit.pairs();
    // the lane's pair; places behind the last repeat it, and no one reads their sums
    const uint32_t entry = order[now.unit.first() + min(lane, n_pairs - 1)];
    pair = static_cast<int32_t>((entry >> 4) * m.top + (entry & 15));
    beside = PARTS > 1 && n_pairs * PARTS <= 8;
    const uint32_t column = lane >> 2;
    uint32_t which = 0;
#pragma unroll
    for (int q = 1; q < PARTS; ++q) which += beside && column >= q * n_pairs;
    const uint32_t source = static_cast<uint32_t>(__shfl_sync(0xffffffffu, DOWN ? pair : static_cast<int32_t>(entry >> 4), column - which * n_pairs));
    const uint32_t x = source * op.k * 2 + which * part + (lane & 3) * 16;               // bytes, below 2^32
    if constexpr (DOWN) w = weights[pair];
    power = m.power[entry >> 4];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i / 4][i % 4] = 0.f;
    auto stages_in = [&](auto parts) {
      constexpr int P = decltype(parts)::value;
      uint4 next[2][P];
      if constexpr (op.template kAhead<P>) {
        op.template inputs<P>(x + s0 * op.kBlocks * 64, part, next[0]);
        op.template inputs<P>(x + (s0 * op.kBlocks + 1) * 64, part, next[1]);
      }
      for (uint32_t s = s0; s < s1; ++s) {
        cp_async_wait<kStages - 2>();
        __syncwarp();                                     // everyone's copies are there, and everyone is done with the stage before
        ask();
        if constexpr (Q == OVL_Q4_K) {
          op.decode(slot);
          __syncwarp();
        }
        op.template multiply<P>(slot, s, x, part, next, acc);
        slot = slot + 1 == kStages ? 0 : slot + 1;
      }
    };
    if (beside || PARTS == 1) stages_in(std::integral_constant<int, 1>{});
    else stages_in(std::integral_constant<int, PARTS>{});
    if (s0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[i * 32] = acc[i / 4][i % 4];
    } else if (s1 < stages) {
      divided = true;
      break;
    } else {
      op.finish(now.tile, n_pairs, pair, w, power, beside, acc);
    }
    s0 = 0;
    now.advance(op.units, op.tiles, n_units);
  }
  __syncthreads();
  if (divided) {
    const uint32_t behind = p - p % stages + stages;      // where the item ends: p is inside it
    for (uint32_t o = warp + 1; o < kWarps<Q, PARTS> && start_of(o) < behind; ++o) {
      if (start_of(o) == start_of(o + 1)) continue;
      const float* theirs = mine + kJoinBytes / 4 * (o - warp);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i / 4][i % 4] += theirs[i * 32];
    }
    op.finish(now.tile, n_pairs, pair, w, power, beside, acc);
  }
  cp_async_wait<0>();
}

template <uint32_t Q, bool DOWN, int PARTS>
cudaError_t launch_rows(const MoeDev& m, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_moe_rows<Q, DOWN, PARTS>), Shape<Q, PARTS>::kSmem, &allowed);
  if (e != cudaSuccess) return e;
  return launch_chained(k_moe_rows<Q, DOWN, PARTS>, dim3(sm_count()), kWarps<Q, PARTS> * 32, Shape<Q, PARTS>::kSmem, st, m);
}

// Both products, one behind the other.
template <uint32_t Q>
cudaError_t launch_products(const MoeDev& m, cudaStream_t st) {
  cudaError_t e = m.bf16 ? launch_rows<Q, false, 1>(m, st) : launch_rows<Q, false, 3>(m, st);
  if (e == cudaSuccess) e = launch_rows<Q, true, 3>(m, st);
  return e;
}

// One translation unit for each format.
cudaError_t launch_products_q8_0(const MoeDev& m, cudaStream_t st);
cudaError_t launch_products_q4_0(const MoeDev& m, cudaStream_t st);
cudaError_t launch_products_q4_k(const MoeDev& m, cudaStream_t st);

}  // namespace moe
}  // namespace ovl
