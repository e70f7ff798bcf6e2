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
// Inputs are bf16 parts (one: bf16 tokens; two: activations of bf16 calls; three: all 24
// bits of fp32) in the order of the fragments: lane t of a quad takes 8 consecutive
// channels of a block in one load, stored as the pairs in which a word's codes unpack.
#pragma once
#include <atomic>
#include <type_traits>

#include "block_internal.h"

namespace ovl {
namespace moe {

constexpr int kWarps = 8;
constexpr int kStages = 4;
constexpr uint32_t kRowBytes = 128;                       // of a row in one stage
constexpr uint32_t kScaleBytes = 20;                      // of a row in one stage: 16, or five words around 16 bytes
constexpr uint32_t kStageBytes = 32 * (kRowBytes + kScaleBytes);
constexpr uint32_t kTableBytes = 2 * 8 * 32 * 4;          // a warp's scales (and minimums) of a stage
constexpr uint32_t kJoinBytes = 32 * 32 * 4;              // a warp's sums
constexpr uint32_t kSmem = kWarps * (kStages * kStageBytes + kTableBytes + kJoinBytes);

__device__ __forceinline__ void cp_async4_if(uint32_t dst, const void* src, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.ca.shared.global [%0], [%1], 4;\n\t}" ::"r"(dst),
               "l"(src), "r"(static_cast<uint32_t>(on))
               : "memory");
}
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
               "l"(src), "r"(static_cast<uint32_t>(on))
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight consecutive codes of a row as four bf16 pairs, exactly.
//   4 bits: 0x4300 | c is 128 + c in bf16; pair i is codes i and i + 4 of the word.
//   8 bits: with the sign bit s and the other seven m, 0x4300 | m is 128 + m and 0x4300 |
//   s is 128 or 256: their difference is m - s.  Pair i is codes 2 i and 2 i + 1.
template <uint32_t Q>
__device__ __forceinline__ void pairs_of(uint2 w, uint32_t (&p)[4]) {
  if constexpr (Q == OVL_Q8_0) {
    const uint32_t b[4] = {__byte_perm(w.x, 0, 0x4140), __byte_perm(w.x, 0, 0x4342), __byte_perm(w.y, 0, 0x4140),
                           __byte_perm(w.y, 0, 0x4342)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = sub_bf16x2((b[i] & 0x007f007fu) | 0x43004300u, (b[i] & 0x00800080u) | 0x43004300u);
  } else {
    const uint32_t zero = Q == OVL_Q4_K ? 0x43004300u : 0x43084308u;      // 128, or 128 + 8
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = sub_bf16x2(((w.x >> (4 * i)) & 0x000f000fu) | 0x43004300u, zero);
  }
}
// Place of channel c of a group of 8 in the order of the pairs.
template <uint32_t Q>
__device__ __forceinline__ uint32_t pair_place(uint32_t c) {
  return Q == OVL_Q8_0 ? c : c < 4 ? 2 * c : 2 * c - 7;
}

// v as bf16 parts: the upper bits cut off, exactly, so that three parts are all 24 bits.
// The last of two is rounded to nearest instead.
template <int PARTS>
__device__ __forceinline__ void parts_of(float v, uint16_t (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    if (PARTS < 3 && i == PARTS - 1) {
      p[i] = static_cast<uint16_t>(two_bf16(v, v));
      break;
    }
    const uint32_t u = v != v ? 0x7fc00000u : __float_as_uint(v) & 0xffff0000u;
    p[i] = static_cast<uint16_t>(u >> 16);
    const float rest = v - __uint_as_float(u);
    v = fabsf(v) <= 3.402823466e38f ? rest : 0.f;        // of an infinity or NaN nothing is left
  }
}

// Where a warp's copies are: an item (32 rows of a unit) and the stage inside it.
struct Cursor {
  const uint8_t* row[2];       // the lane's first row and piece: of the first and of the last 16 rows
  const uint8_t* scale;        // the lane's row of scales
  uint32_t item, stage;
};

// DOWN: the second product.  PARTS: of its input.
template <uint32_t Q, bool DOWN, int PARTS>
struct Rows32 {
  static constexpr uint32_t kBlocks = Q == OVL_Q8_0 ? 4 : 8;            // 32-weight blocks of a stage
  static constexpr uint32_t kScales = Q == OVL_Q8_0 ? 8 : 16;           // bytes of a row's scales in a stage

  const MoeDev& m;
  uint8_t* ring;               // the warp's
  float* table;
  uint32_t lane, k, pitch, scale_pitch, tiles;
  bool scales_aligned;

  __device__ Rows32(const MoeDev& dev, uint8_t* r, float* t) : m(dev), ring(r), table(t) {
    lane = threadIdx.x & 31;
    k = DOWN ? m.ffn : m.hidden;
    pitch = Q == OVL_Q8_0 ? k : k / 2;
    scale_pitch = k / 16;                                               // 2 bytes a block; 16 bytes of 256 weights
    scales_aligned = scale_pitch % kScales == 0;
    tiles = DOWN ? m.hidden / 32 : m.ffn / 16;
  }

  __device__ void at(Cursor& c, uint32_t item, uint32_t stage) const {
    c.item = item;
    c.stage = stage;
    const uint32_t unit = item / tiles, tile = item % tiles, expert = m.units[unit].expert_n >> 8;
    const uint32_t r = lane >> 3;
    const uint64_t piece = (lane & 7) * 16;
    if constexpr (DOWN) {
      const uint64_t first = static_cast<uint64_t>(expert) * m.hidden + tile * 32;
      c.row[0] = m.down_qs + (first + r) * pitch + piece;
      c.row[1] = c.row[0] + 16ull * pitch;
      c.scale = m.down_d + (first + lane) * scale_pitch;
    } else {
      const uint64_t first = static_cast<uint64_t>(expert) * m.ffn + tile * 16;
      c.row[0] = m.gate_qs + (first + r) * pitch + piece;
      c.row[1] = m.up_qs + (first + r) * pitch + piece;
      c.scale = (lane < 16 ? m.gate_d : m.up_d) + (first + (lane & 15)) * scale_pitch;
    }
  }

  // Asks for stage c.stage of the item.  Piece p of row r lies at piece p ^ swizzle(r), so
  // that the 8 rows of a fragment load meet different banks.
  __device__ void fill(const Cursor& c, uint32_t slot) const {
    const uint32_t dst = smem_u32(ring + slot * kStageBytes);
    const uint32_t r0 = lane >> 3, piece = lane & 7;
    const bool on = c.stage * kRowBytes + piece * 16 < pitch;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t r = r0 + 4 * i, swizzle = Q == OVL_Q8_0 ? (r & 3) << 1 : r & 7;
      const uint8_t* src = c.row[i / 4] + static_cast<uint64_t>(4 * (i & 3)) * pitch + c.stage * kRowBytes;
      cp_async16_if(dst + r * kRowBytes + ((piece ^ swizzle) << 4), src, on);
    }
    const uint32_t raw = dst + 32 * kRowBytes;
    const uint8_t* s = c.scale + c.stage * kScales;
    if (Q == OVL_Q4_K || scales_aligned) {
      if constexpr (kScales == 16) {
        cp_async16_if(raw + lane * 16, s, true);
      } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(raw + lane * 8), "l"(s) : "memory");
      }
    } else {                                                            // rows of scales begin at any even address
      const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s)) & 2;
      const uint32_t have = min(kScales, scale_pitch - c.stage * kScales) + shift;
#pragma unroll
      for (uint32_t i = 0; i < kScales / 4 + 1; ++i) cp_async4_if(raw + lane * kScaleBytes + 4 * i, s - shift + 4 * i, 4 * i < have);
    }
  }

  // A stage's scales as fp32: table[block][row], and for Q4_K the minimums behind them.
  __device__ void decode(uint32_t slot, uint32_t stage, const uint8_t* scale_row) const {
    const uint8_t* raw = ring + slot * kStageBytes + 32 * kRowBytes;
    if constexpr (Q == OVL_Q4_K) {
      const uint4 h = *reinterpret_cast<const uint4*>(raw + lane * 16);
      const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
      const uint64_t sc = h.y | (static_cast<uint64_t>(h.z & 0xffffu) << 32), mn = (h.z >> 16) | (static_cast<uint64_t>(h.w) << 16);
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        table[b * 32 + lane] = d.x * static_cast<float>(static_cast<uint32_t>(sc >> (6 * b)) & 63u);
        table[256 + b * 32 + lane] = -d.y * static_cast<float>(static_cast<uint32_t>(mn >> (6 * b)) & 63u);
      }
    } else {
      const __half* s;
      if (scales_aligned) s = reinterpret_cast<const __half*>(raw + lane * kScales);
      else s = reinterpret_cast<const __half*>(raw + lane * kScaleBytes +
                                               (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(scale_row + stage * kScales)) & 2));
#pragma unroll
      for (uint32_t b = 0; b < kBlocks; ++b) table[b * 32 + lane] = __half2float(s[b]);
    }
  }

  // One stage's products: acc[half of the rows][8 tokens each][fragment] += scale * codes x.
  template <int NT>
  __device__ void multiply(uint32_t slot, uint32_t stage, const uint16_t* const (&x)[NT], uint64_t part,
                           float (&acc)[2][NT][4]) const {
    const uint8_t* rows = ring + slot * kStageBytes;
    const uint32_t g = lane >> 2, t = lane & 3;
    const uint32_t blocks = min(kBlocks, k / 32 - stage * kBlocks);
#pragma unroll 2
    for (uint32_t b = 0; b < blocks; ++b) {
      uint4 xs[NT][PARTS];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
          xs[n][q] = x[n] ? *reinterpret_cast<const uint4*>(x[n] + q * part + (stage * kBlocks + b) * 32) : make_uint4(0, 0, 0, 0);
      uint32_t a[2][2][4];                       // half, k16 step, fragment
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t r = h * 16 + e * 8 + g;
          uint2 w;
          if constexpr (Q == OVL_Q8_0) {
            const uint32_t piece = (2 * b + (t >> 1)) ^ ((r & 3) << 1);
            w = *reinterpret_cast<const uint2*>(rows + r * kRowBytes + piece * 16 + (t & 1) * 8);
          } else {
            w.x = *reinterpret_cast<const uint32_t*>(rows + r * kRowBytes + ((b ^ (r & 7)) << 4) + t * 4);
            w.y = 0;
          }
          if (e == 0) pairs_of<Q>(w, lo);
          else pairs_of<Q>(w, hi);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) a[h][s][0] = lo[2 * s], a[h][s][1] = hi[2 * s], a[h][s][2] = lo[2 * s + 1], a[h][s][3] = hi[2 * s + 1];
      }
      float scale[4], least[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        scale[r] = table[b * 32 + r * 8 + g];
        if constexpr (Q == OVL_Q4_K) least[r] = table[256 + b * 32 + r * 8 + g];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (Q == OVL_Q4_K) {           // the block's inputs summed up, in every row: codes of one
          const uint32_t one[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
          for (int q = PARTS - 1; q >= 0; --q) {
            mma_bf16(sum, one, xs[n][q].x, xs[n][q].y);
            mma_bf16(sum, one, xs[n][q].z, xs[n][q].w);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float p[4] = {0.f, 0.f, 0.f, 0.f};     // small parts first: the MMAs cut off their sums
#pragma unroll
          for (int q = PARTS - 1; q >= 0; --q) {
            mma_bf16(p, a[h][0], xs[n][q].x, xs[n][q].y);
            mma_bf16(p, a[h][1], xs[n][q].z, xs[n][q].w);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[h][n][i] = fmaf(scale[2 * h + (i >> 1)], p[i], acc[h][n][i]);
            if constexpr (Q == OVL_Q4_K) acc[h][n][i] = fmaf(least[2 * h + (i >> 1)], sum[i], acc[h][n][i]);
          }
        }
      }
    }
  }

  // What an item's sums become.
  template <int NT>
  __device__ void finish(uint32_t item, uint32_t n_pairs, int32_t pair, const float (&acc)[2][NT][4]) const {
    const uint32_t tile = item % tiles, g = lane >> 2, t = lane & 3;
    const float w = DOWN && lane < n_pairs ? m.weight[pair] : 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t column = n * 8 + 2 * t + j;
        const int32_t p = __shfl_sync(0xffffffffu, pair, column);
        const float weight = __shfl_sync(0xffffffffu, w, column);
        if (column >= n_pairs) continue;
        if constexpr (DOWN) {
          float* out = m.part + static_cast<uint64_t>(p) * m.hidden + tile * 32 + g;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) out[h * 16 + e * 8] = weight * acc[h][n][2 * e + j];
        } else {
          constexpr int kParts = PARTS == 1 ? 2 : 3;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint16_t v[kParts];
            parts_of<kParts>(activated(acc[0][n][2 * e + j], m.act) * acc[1][n][2 * e + j], v);
            uint16_t* out = m.hp + static_cast<uint64_t>(p) * m.ffn + tile * 16 + e * 8 + pair_place<Q>(g);
#pragma unroll
            for (int q = 0; q < kParts; ++q) out[q * static_cast<uint64_t>(m.pairs) * m.ffn] = v[q];
          }
        }
      }
    }
  }
};

template <uint32_t Q, bool DOWN, int PARTS>
__global__ void __launch_bounds__(kWarps * 32, 1) k_moe_rows(const __grid_constant__ MoeDev m) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  float* table = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes + warp * kTableBytes);
  float* join = reinterpret_cast<float*>(smem + kWarps * (kStages * kStageBytes + kTableBytes));
  // The first product waits for the router before it lets the second start, so that the
  // second may read the router's results and ask for weights before the first has ended.
  if constexpr (!DOWN) {
    griddep_wait();
    griddep_launch_dependents();
  }
  const Rows32<Q, DOWN, PARTS> op(m, ring, table);
  // Items in equal runs to the CTAs.  Where a CTA has fewer items than warps, `split`
  // warps share an item's stages and add up through shared memory.
  const uint64_t items = static_cast<uint64_t>(*m.n_units) * op.tiles;
  const uint32_t begin = static_cast<uint32_t>(items * blockIdx.x / gridDim.x), end = static_cast<uint32_t>(items * (blockIdx.x + 1) / gridDim.x);
  const uint32_t most = static_cast<uint32_t>((items + gridDim.x - 1) / gridDim.x);
  const uint32_t stages = (op.pitch + kRowBytes - 1) / kRowBytes;
  uint32_t split = kWarps;
  while (split > 1 && (most * split > kWarps || split > stages)) split /= 2;
  const uint32_t slots = kWarps / split, sub = warp % split;
  const uint32_t s0 = stages * sub / split, s1 = stages * (sub + 1) / split;
  const uint32_t rounds = (end - begin + slots - 1) / slots;
  Cursor c{};
  uint32_t ahead = 0;                                     // round of the copies
  c.item = begin + warp / split;
  if (c.item < end) op.at(c, c.item, s0);
  uint32_t slot_in = 0;
  auto ask = [&]() {
    if (c.item < end) {
      op.fill(c, slot_in);
      if (++c.stage == s1) {
        ++ahead;
        c.item += slots;
        if (c.item < end) op.at(c, c.item, s0);
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
  uint32_t slot = 0;
  auto run = [&](auto tokens, uint32_t item, uint32_t n_pairs, int32_t pair) {
    constexpr int NT = decltype(tokens)::value;
    const uint16_t* x[NT];
    const uint64_t part = static_cast<uint64_t>(DOWN ? m.pairs : m.tokens) * op.k;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t column = n * 8 + (lane >> 2);
      const uint32_t p = static_cast<uint32_t>(__shfl_sync(0xffffffffu, pair, column));
      x[n] = column < n_pairs ? (DOWN ? m.hp + static_cast<uint64_t>(p) * op.k : m.xp + static_cast<uint64_t>(p / m.top) * op.k) + (lane & 3) * 8
                              : nullptr;
    }
    float acc[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[h][n][i] = 0.f;
    const uint32_t tile = item % op.tiles, expert = m.units[item / op.tiles].expert_n >> 8;
    const uint8_t* scale_row;
    if constexpr (DOWN) scale_row = m.down_d + (static_cast<uint64_t>(expert) * m.hidden + tile * 32 + lane) * op.scale_pitch;
    else scale_row = (lane < 16 ? m.gate_d : m.up_d) + (static_cast<uint64_t>(expert) * m.ffn + tile * 16 + (lane & 15)) * op.scale_pitch;
    for (uint32_t s = s0; s < s1; ++s) {
      cp_async_wait<kStages - 2>();
      __syncwarp();                                       // everyone's copies are there, and everyone is done with the stage before
      ask();
      op.decode(slot, s, scale_row);
      __syncwarp();
      op.template multiply<NT>(slot, s, x, part, acc);
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
    if (split > 1) {
      float* mine = join + warp * 1024 + lane;
      if (sub) {
#pragma unroll
        for (int i = 0; i < 8 * NT; ++i) mine[i * 32] = acc[i / (4 * NT)][i / 4 % NT][i % 4];
      }
      named_bar(1 + warp / split, split * 32);
      if (!sub) {
        for (uint32_t o = 1; o < split; ++o)
#pragma unroll
          for (int i = 0; i < 8 * NT; ++i) acc[i / (4 * NT)][i / 4 % NT][i % 4] += mine[o * 1024 + i * 32];
      }
      named_bar(1 + warp / split, split * 32);
    }
    if (!sub) op.template finish<NT>(item, n_pairs, pair, acc);
  };
  for (uint32_t r = 0; r < rounds; ++r) {
    const uint32_t item = begin + r * slots + warp / split;
    if (item >= end) break;                               // the same for the warps of an item
    const MoeUnit u = m.units[item / op.tiles];
    const uint32_t n_pairs = u.expert_n & 255;
    const int32_t pair = lane < n_pairs ? m.order[u.first + lane] : 0;
    if (n_pairs <= 8) run(std::integral_constant<int, 1>{}, item, n_pairs, pair);
    else if (n_pairs <= 16) run(std::integral_constant<int, 2>{}, item, n_pairs, pair);
    else run(std::integral_constant<int, 4>{}, item, n_pairs, pair);
  }
  cp_async_wait<0>();
}

template <uint32_t Q, bool DOWN, int PARTS>
cudaError_t launch_rows(const MoeDev& m, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_moe_rows<Q, DOWN, PARTS>), kSmem, &allowed);
  if (e != cudaSuccess) return e;
  return launch_chained(k_moe_rows<Q, DOWN, PARTS>, dim3(sm_count()), kWarps * 32, kSmem, st, m);
}

// Both products, one behind the other.
template <uint32_t Q>
cudaError_t launch_products(const MoeDev& m, cudaStream_t st) {
  cudaError_t e = m.bf16 ? launch_rows<Q, false, 1>(m, st) : launch_rows<Q, false, 3>(m, st);
  if (e == cudaSuccess) e = m.bf16 ? launch_rows<Q, true, 2>(m, st) : launch_rows<Q, true, 3>(m, st);
  return e;
}

// One translation unit for each format.
cudaError_t launch_products_q8_0(const MoeDev& m, cudaStream_t st);
cudaError_t launch_products_q4_0(const MoeDev& m, cudaStream_t st);
cudaError_t launch_products_q4_k(const MoeDev& m, cudaStream_t st);

}  // namespace moe
}  // namespace ovl
