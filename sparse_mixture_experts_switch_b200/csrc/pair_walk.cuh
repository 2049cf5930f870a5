// Walk of CTA pairs over tiles of "output features x one expert's tokens", with
// the tokens as the MMA's flexible N, and the pieces that the drains of such
// tiles share (one feature a lane, 32 tokens a chunk).
#pragma once

#include "q8.cuh"

namespace smoe {

constexpr int kQTok = 256;                             // most tokens of a tile

struct WalkParams {
  int N;                     // experts
  int ntiles_f;              // 256-feature tiles of an expert
  int64_t C;
  const int* counts;
  int parts;                 // of the sum: items are tile * parts + part
};

__device__ __forceinline__ int kept_tokens(const WalkParams& p, int e) {
  const int64_t c = __ldg(p.counts + e);
  return static_cast<int>(c < 0 ? 0 : (c < p.C ? c : p.C));
}
// Token tiles of an expert, of at most 2^shift tokens each.
__device__ __forceinline__ int token_tiles(int kept, int shift) {
  return (kept + (1 << shift) - 1) >> shift;
}

// Per expert its kept tokens, and the exclusive prefix of its tiles (token tiles x
// feature tiles); one warp.  The tiles take up to 256 tokens, or 128 where
// even then every pair has one tile at most: a tile of 128 tokens takes about 300
// cycles for a block of the sum, one of 256 takes 512 (8-bit FFN of 300 tokens, one
// expert of 2048 x 4096: 26.8 against 29.0 us; where it makes two rounds of tiles out
// of one it loses, 38.3 against 34.8).  kept[N] holds the shift.
static __device__ void tiles_prefix_warp(const WalkParams& p, int npairs, int* pts, int* kept) {
  const int lane = threadIdx.x & 31;
  const int per = (p.N + 31) / 32;
  int s = 0, s128 = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < p.N) {
      const int k = kept_tokens(p, e);
      kept[e] = k;
      s += token_tiles(k, 8) * p.ntiles_f;
      s128 += token_tiles(k, 7) * p.ntiles_f;
    }
  }
  const int shift = __reduce_add_sync(0xffffffffu, s128) * p.parts <= npairs ? 7 : 8;
  if (shift == 7) s = s128;
  if (lane == 0) kept[p.N] = shift;
  int inc = s;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  int run = inc - s;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < p.N) {
      pts[e] = run;
      run += token_tiles(kept[e], shift) * p.ntiles_f;
    }
  }
  if (lane == 31) pts[p.N] = inc;
}

struct RowTile {
  int e;        // expert
  int t0;       // first token slot of the tile within the expert
  int nv;       // its tokens (1..256)
  int nmma;     // the MMA's N: nv rounded up to 16
  int f0;       // first output feature of the pair tile
};

__device__ __forceinline__ int small_div(int a, int b) {      // b is 1 or 2 most of the time
  return b == 1 ? a : (b == 2 ? a >> 1 : a / b);
}

// Stages of one part of a sum of `stages`.
struct StageRange {
  int begin, end;
};
__device__ __forceinline__ StageRange part_stages(int part, int parts, int stages) {
  if (parts == 1) return {0, stages};
  return {part * stages / parts, (part + 1) * stages / parts};
}

// Tiles in the order of a pair's walk (tile numbers that only grow).  An
// expert's token tiles vary fastest, so pairs running side by side share the
// weight tile.  A product that reads what the one before it wrote takes the list
// from its end (kForward false): the last experts' rows, written last, are the
// ones still in L2.  The walk
// remembers its expert and looks 32 on at a time, one a lane, so all of a warp's
// lanes call it together (one lane going from expert to expert took 1000 cycles
// where the tiles of 8 lie between a pair's next two).
template <bool kForward>
struct RowWalk {
  const WalkParams& p;
  const int *pts, *kept;
  int e;
  __device__ __forceinline__ RowWalk(const WalkParams& p_, const int* pts_, const int* kept_)
      : p(p_), pts(pts_), kept(kept_), e(kForward ? 0 : p_.N - 1) {}
  __device__ __forceinline__ RowTile at(int tile) {
    const int lane = threadIdx.x & 31;
    if (!kForward) tile = pts[p.N] - 1 - tile;
    int n;
    do {                                     // (the prefix never falls)
      const int i = kForward ? e + 1 + lane : e - lane;
      n = __popc(__ballot_sync(0xffffffffu, kForward ? i <= p.N && pts[i] <= tile
                                                     : i >= 0 && pts[i] > tile));
      e += kForward ? n : -n;
    } while (n == 32);
    RowTile t;
    t.e = e;
    const int k = kept[e];
    const int nt = token_tiles(k, kept[p.N]);
    const int local = tile - pts[e];
    const int mf = small_div(local, nt);
    const int size = (small_div(k + nt - 1, nt) + 15) & ~15;
    t.t0 = (local - mf * nt) * size;
    t.nv = k - t.t0 < size ? k - t.t0 : size;
    t.nmma = (t.nv + 15) & ~15;
    t.f0 = mf * 256;
    return t;
  }
};

// Rows of the token boxes: the smallest of eight that holds half a tile (what a
// box brings beyond it costs shared-memory bandwidth).
constexpr int kRowBoxes = 8;
struct RowMaps {
  CUtensorMap w;
  CUtensorMap tok[kRowBoxes];
};
__host__ __device__ constexpr uint32_t box_rows(int box) {
  return box < 3 ? 8u << box : (box == 3 ? 64u : 16u * box + 16u);   // 8 16 32 64 80 96 112 128
}
__device__ __forceinline__ int box_of(int half) {
  return half <= 8 ? 0 : (half <= 16 ? 1 : (half <= 32 ? 2 : (half <= 64 ? 3 : (half - 1) >> 4)));
}

// relu of four fp32 values as e4m3 codes (NaN stays NaN), `a` in the lowest byte.
__device__ __forceinline__ uint32_t relu_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.relu.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.relu.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The larger of two bf16 numbers, twice; of a number and NaN the number.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The larger of two numbers; NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Lane j: the maximum over the warp of token j, from 16 registers of two tokens
// each (token 2 i in the low half of m[i]), all bf16 numbers (NaN only where all are); the
// result in the upper half.  Five exchanges halve the tokens that a lane still
// follows: 16 shuffles (a warp reduction per token, 32 of two cycles of the whole
// SM each, took 310-940 cycles of a chunk's drain).
__device__ __forceinline__ uint32_t warp_token_max(uint32_t (&m)[16], int lane) {
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1) {                 // lane bit 2 n picks the upper half
    const bool up = (lane & (2 * n)) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const uint32_t keep = up ? m[i + n] : m[i];
      const uint32_t send = up ? m[i] : m[i + n];
      m[i] = max_bf16x2(keep, __shfl_xor_sync(0xffffffffu, send, 2 * n));
    }
  }
  const uint32_t p = max_bf16x2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
  return (lane & 1) ? p & 0xFFFF0000u : p << 16;
}

// Words w of tokens 4k .. 4k + 3 (one byte each, a feature a lane) as four
// features of token 4k + lane % 4: the transpose of four lanes' words.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t w, int lane) {
  const uint32_t t1 = __shfl_xor_sync(0xffffffffu, w, 1);
  const uint32_t x = (lane & 1) ? __byte_perm(t1, w, 0x7351) : __byte_perm(w, t1, 0x6240);
  const uint32_t t2 = __shfl_xor_sync(0xffffffffu, x, 2);
  return (lane & 2) ? __byte_perm(t2, x, 0x7632) : __byte_perm(x, t2, 0x5410);
}
// Rows of 128 codes of 32 tokens in shared memory, 32 codes from each of four
// warps, in 16-byte pieces swizzled by the token (no two lanes of a store meet in a
// bank).  Where lane `lane` of warp q has four features of token tok + lane % 4 ...
__device__ __forceinline__ uint32_t row_word(uint32_t rows, int tok, int q, int lane) {
  const int piece = (q * 2 + (lane >> 4)) ^ ((lane & 3) << 1);
  return rows + static_cast<uint32_t>((tok + (lane & 3)) * 128 + piece * 16 + (lane & 12));
}
// ... and the four warps' stores of the first jn of them to rows row0 .. of out
// [.., cols], columns col .. col + 127 (those below cols): 4 rows x 128 bytes each.
__device__ __forceinline__ void store_rows(uint32_t rows, uint8_t* out, int64_t row0, int jn,
                                           int col, int cols, int q, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int rr = 8 * q + 4 * i + (lane >> 3), c = lane & 7;
    if (rr < jn && col + c * 16 < cols)
      *reinterpret_cast<float4*>(out + (row0 + rr) * cols + col + c * 16) =
          ld_shared_v4(rows + static_cast<uint32_t>(rr * 128 + ((c ^ ((rr & 3) << 1)) << 4)));
  }
}
// Tokens j and j + 1 of this feature (16 bits each) as two features of token
// j + lane % 2.
__device__ __forceinline__ uint32_t transpose_halves(uint32_t w, int lane) {
  const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 1);
  return (lane & 1) ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
}
// Bits of token `lane` over the warp's features as this feature's bits over the
// 32 tokens.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
  const uint32_t masks[5] = {0x0000FFFFu, 0x00FF00FFu, 0x0F0F0F0Fu, 0x33333333u, 0x55555555u};
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int s = 16 >> i;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, s);
    x = (lane & s) ? (x & ~masks[i]) | ((y & ~masks[i]) >> s)
                   : (x & masks[i]) | ((y & masks[i]) << s);
  }
  return x;
}

}  // namespace smoe
