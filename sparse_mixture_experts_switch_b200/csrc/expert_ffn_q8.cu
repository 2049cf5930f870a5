// The experts' ReLU FFNs on 8-bit rows and weights (format: q8.cuh):
//
//   h = relu(x W1_e^T),  (hq, hs) = 8-bit rows of h,  y = h W2_e^T (bf16)
//
//   D[r, f] = sum over blocks k of 2^(sa[r, k] + sw[f / 128, k]) sum_j a[r, k, j] w[f, k, j]
//
// The tensor core applies the scales itself: tcgen05.mma.kind::mxf8f6f4 with
// block_scale multiplies each 32-deep step by one e8m0 scale of each operand
// row, which it reads from TMEM.  A scale here covers 128 columns, so the four
// 32-deep steps of a block use the same byte (the descriptor's scale-factor id
// picks one byte of a row's 32-bit word): one word of a row is the scales of
// 512 columns, exactly four consecutive bytes of the row-major scale array.
// Products and sums are fp32 in TMEM.
//
// One persistent kernel for both products: tile = 128 slots x BN columns, K in
// blocks of 128 bytes through a ring of TMA stages.
//   * warp 0 loads the row and weight tiles by TMA (128-byte swizzle);
//   * warp 2 brings the scales: for each 512 columns the 128 rows' words, laid
//     out as tcgen05.cp wants them (row r at lane r % 32, word r / 32), and one
//     word for each 128 weight rows, repeated;
//   * warp 1 copies the scales to TMEM (tcgen05.cp) and issues the MMAs;
//   * warps 4-11 drain the accumulator, one row and up to 128 columns a
//     thread, all of them in registers at once, so that the accumulator is
//     handed back before they are converted and stored: a hidden row's block of
//     128 columns is then a thread's own (ReLU, maximum, scale, 8 bits).
// BN = 256 has one accumulator of 256 columns (two would leave TMEM no room
// for the scales); its 8 drain warps take the two column halves side by side.
// BN = 128 and 64 have two accumulators, four drain warps each.
#include <cstring>

#include "q8.cuh"
#include "gemm_common.cuh"

namespace smoe {

namespace {

constexpr int kQK = 128;                               // K block: 128 codes
constexpr uint32_t kQABytes = 128 * kQK;               // 16 KB
constexpr int kQThreads = 384;
constexpr int kQDrainWarps = 8;
constexpr int kSfSlots = 4;                            // ring of scale groups (512 columns each)
constexpr uint32_t kSfBytes = 3 * 512;                 // rows, weight rows 0-127, 128-255
constexpr uint32_t kSfTmem = 256;                      // TMEM columns 256 + 16 slot
constexpr uint32_t kQStageOut = 2048;                  // per drain warp: 32 rows x 64 bytes
constexpr uint32_t kQTmemCols = 512;

template <int BN>
struct Q8Tile {
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr uint32_t kBBytes = BN * kQK;
  static constexpr uint32_t kStageBytes = kQABytes + kBBytes;
  static constexpr int kAccs = BN == 256 ? 1 : 2;
  static constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + kQDrainWarps * kQStageOut +
                                    kSfSlots * kSfBytes + 512;   // + mts [N + 1]
};

struct Q8Params {
  int N, n_out, K, ntiles_n;
  int64_t C;
  int kblk;                  // scale bytes of a row: ceil(K / 128)
  int nblk_w;                // weight blocks along n_out: ceil(n_out / 128)
  const int* counts;
  const uint8_t* as;         // [N*C, kblk]
  const uint8_t* ws;         // [N, nblk_w, kblk]
  uint8_t* hq;               // hidden: [N*C, n_out]
  uint8_t* hs;               // hidden: [N*C, nblk_w]
  __nv_bfloat16* y;          // else: [N*C, n_out]
  DevErr* err;
  long long spin;
};

// D (+)= scaled A x scaled B^T; one thread.
__device__ __forceinline__ void umma_q8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 rows x 16 bytes of shared memory (512 consecutive bytes) to 4 TMEM columns,
// repeated in the four lane quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Descriptor of such a block: no swizzle, 8 rows of 16 bytes are 128
// consecutive bytes, the next 8 follow.
__device__ __forceinline__ uint64_t scales_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

// e4m3 x e4m3 with e8m0 block scales -> fp32, both operands K-major; the byte
// of the scale words is added per block (bits 4-5 for B, 29-30 for A).
__host__ __device__ constexpr uint32_t idesc_q8(int M, int N) {
  return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_byte(uint32_t b) { return (b << 4) | (b << 29); }

__device__ __forceinline__ int64_t kept_q8(const Q8Params& p, int e) {
  const int64_t c = p.counts[e];
  return c < 0 ? 0 : (c < p.C ? c : p.C);
}

// Exclusive prefix of the experts' 128-row tiles, one warp.
__device__ void tiles_prefix_warp(const Q8Params& p, int* mts) {
  const int lane = threadIdx.x & 31;
  const int per = (p.N + 31) / 32;
  int s = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < p.N) s += static_cast<int>((kept_q8(p, e) + 127) >> 7);
  }
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
      mts[e] = run;
      run += static_cast<int>((kept_q8(p, e) + 127) >> 7);
    }
  }
  if (lane == 31) mts[p.N] = inc;
}

// Scale bytes 4g .. 4g + 3 of a row of `kblk` bytes (past its end: 2^0).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int g, int kblk) {
  if ((kblk & 3) == 0) return __ldg(reinterpret_cast<const uint32_t*>(row) + g);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = 4 * g + i;
    const uint32_t v = b < kblk ? __ldg(row + b) : 127u;
    w |= v << (8 * i);
  }
  return w;
}

template <int BN, bool kHidden>
__global__ void __launch_bounds__(kQThreads, 1)
    expert_gemm_q8_kernel(const __grid_constant__ CUtensorMap tmap_a,
                          const __grid_constant__ CUtensorMap tmap_b,
                          const __grid_constant__ CUtensorMap tmap_out, Q8Params p) {
  using L = Q8Tile<BN>;
  constexpr int kStages = L::kStages;
  constexpr int kAccs = L::kAccs;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* stage_out = smem + kStages * L::kStageBytes;
  uint8_t* sf = stage_out + kQDrainWarps * kQStageOut;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf + kSfSlots * kSfBytes);
  uint64_t* empty = full + kStages;
  uint64_t* sfull = empty + kStages;
  uint64_t* sempty = sfull + kSfSlots;
  uint64_t* tfull = sempty + kSfSlots;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* mts = reinterpret_cast<int*>(sf + kSfSlots * kSfBytes + 512);     // [N + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long lim = p.spin;
  const int kblocks = (p.K + kQK - 1) / kQK;

  if (warp == 0) tiles_prefix_warp(p, mts);
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kAccs == 1 ? 256 : 128);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int total = mts[p.N] * p.ntiles_n;
  if (static_cast<int>(blockIdx.x) >= total) return;     // uniform for the block
  if (warp == 1) {
    tmem_alloc(tmem_holder, kQTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------- TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tmap_a);
      tma_prefetch_desc(&tmap_b);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued_mask = 0, issued_phase = 0;
      for (int tile = blockIdx.x; tile < total && !*abort_flag; tile += gridDim.x) {
        int e, m, n;
        decode_tile(tile, mts, p.N, p.ntiles_n, e, m, n);
        const int row = static_cast<int>(static_cast<int64_t>(e) * p.C + m * 128);
        bool ok = true;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, lim)) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmProducer, tile);
            *abort_flag = 1;
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * L::kStageBytes;
          mbar_arrive_expect_tx(&full[stage], L::kStageBytes);
          tma_load_2d(sa, &tmap_a, &full[stage], kb * kQK, row);
          tma_load_3d(sa + kQABytes, &tmap_b, &full[stage], kb * kQK, n * BN, e);
          issued_mask |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
      }
      // Never leave with copies in flight into this CTA's shared memory.
      for (int s = 0; s < kStages; ++s)
        if (((issued_mask >> s) & 1u) &&
            !mbar_wait(&full[s], (issued_phase >> s) & 1u, kDefaultSpinCycles))
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereDrain, s);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------- scales
    int slot = 0;
    uint32_t phase = 0;
    const int groups = (kblocks + 3) / 4;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      int e, m, n;
      decode_tile(tile, mts, p.N, p.ntiles_n, e, m, n);
      const int64_t kept = kept_q8(p, e);
      const uint8_t* arow[4];
      bool aon[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = static_cast<int64_t>(m) * 128 + 32 * j + lane;
        aon[j] = r < kept;
        arow[j] = p.as + (static_cast<int64_t>(e) * p.C + (aon[j] ? r : 0)) * p.kblk;
      }
      const int b0 = n * BN / 128;
      const int b1 = b0 + 1 < p.nblk_w ? b0 + 1 : p.nblk_w - 1;
      const uint8_t* w0 = p.ws + (static_cast<int64_t>(e) * p.nblk_w + b0) * p.kblk;
      const uint8_t* w1 = p.ws + (static_cast<int64_t>(e) * p.nblk_w + b1) * p.kblk;
      bool ok = true;
      for (int g = 0; g < groups; ++g) {
        uint32_t a[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = aon[j] ? scale_word(arow[j], g, p.kblk) : 0x7F7F7F7Fu;
        const uint32_t u0 = scale_word(w0, g, p.kblk);
        const uint32_t u1 = BN > 128 ? scale_word(w1, g, p.kblk) : 0u;
        int w_ok = 1;
        if (lane == 0) w_ok = mbar_wait(&sempty[slot], phase ^ 1u, lim) ? 1 : 0;
        w_ok = __shfl_sync(0xffffffffu, w_ok, 0);
        if (!w_ok) {
          if (lane == 0) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmProducer, tile);
            *abort_flag = 1;
          }
          ok = false;
          break;
        }
        const uint32_t dst = smem_u32(sf + slot * kSfBytes) + lane * 16;
        st_shared_v4u(dst, a[0], a[1], a[2], a[3]);
        st_shared_v4u(dst + 512, u0, u0, u0, u0);
        if (BN > 128) st_shared_v4u(dst + 1024, u1, u1, u1, u1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[slot]);
        if (++slot == kSfSlots) { slot = 0; phase ^= 1u; }
      }
      if (!ok) break;
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_q8(128, BN);
      int stage = 0, slot = 0;
      uint32_t phase = 0, sphase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      uint32_t sfa = 0;
      bool any = false;
      for (int tile = blockIdx.x; tile < total && !*abort_flag; tile += gridDim.x) {
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, lim)) {
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmMma, tile);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        bool ok = true;
        for (int kb = 0; kb < kblocks; ++kb) {
          if ((kb & 3) == 0) {
            if (!mbar_wait(&sfull[slot], sphase, lim)) {
              ok = false;
            } else {
              tc_fence_after();
              sfa = tmem_base + kSfTmem + 16u * slot;
              const uint32_t src = smem_u32(sf + slot * kSfBytes);
              tmem_cp_scales(sfa, scales_desc(src));
              tmem_cp_scales(sfa + 4, scales_desc(src + 512));
              if (BN > 128) tmem_cp_scales(sfa + 8, scales_desc(src + 1024));
              any = true;
              umma_commit(&sempty[slot]);
              if (++slot == kSfSlots) { slot = 0; sphase ^= 1u; }
            }
          }
          if (!ok || !mbar_wait(&full[stage], phase, lim)) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmMma, tile);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * L::kStageBytes);
          const uint32_t sb = sa + kQABytes;
          const uint32_t id = idesc | idesc_byte(static_cast<uint32_t>(kb & 3));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_q8(d_tmem, sw128_kmajor_desc(sa + k * 32), sw128_kmajor_desc(sb + k * 32), id, sfa,
                    sfa + 4, (kb | k) != 0 ? 1u : 0u);
          any = true;
          umma_commit(&empty[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&tfull[acc]);
        if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
      }
      if (any && *abort_flag) {
        umma_commit(drain);
        if (!mbar_wait(drain, 0, kDefaultSpinCycles))
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereDrain, -1);
      }
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------- drain warps
    constexpr int kCols = BN < 128 ? BN : 128;            // columns of a thread
    const int q = warp & 3;
    const int half = (warp - 4) >> 2;                     // column half, or accumulator
    const uint32_t stg = smem_u32(stage_out + (warp - 4) * kQStageOut);
    const uint32_t swz = static_cast<uint32_t>((lane >> 1) & 3);
    if (lane == 0) tma_prefetch_desc(&tmap_out);
    const int acc = kAccs == 1 ? 0 : half;
    uint32_t acc_phase = 0;
    int turn = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      if (kAccs == 2 && (turn++ & 1) != half) continue;   // the other accumulator's tile
      const bool ok = __all_sync(0xffffffffu, mbar_wait_sleepy(&tfull[acc], acc_phase, lim));
      if (!ok) {
        if (lane == 0) {
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmEpilogue, tile);
          *abort_flag = 1;
        }
        break;
      }
      acc_phase ^= 1u;
      tc_fence_after();
      int e, m, n;
      decode_tile(tile, mts, p.N, p.ntiles_n, e, m, n);
      const int64_t kept = kept_q8(p, e);
      const int64_t rbase = static_cast<int64_t>(m) * 128 + q * 32;
      const int col0 = n * BN + (kAccs == 1 ? half * 128 : 0);
      const int left = p.n_out - col0;
      const int ncols = left < kCols ? left : kCols;      // 64, 128, or none
      const bool work = rbase < kept && ncols > 0;        // warp-uniform
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(kAccs == 1 ? half * 128 : acc * BN);
      // hidden: the values, after the ReLU; else packed bf16 pairs
      float f[kHidden ? kCols : 1];
      uint32_t pk[kHidden ? kCols / 4 : kCols / 2];
      if (work) {
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t v[32];
          tmem_ld32_issue(taddr + c * 32, v);
          tmem_ld_wait(v);
          if (kHidden) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              f[kHidden ? 32 * c + j : 0] = fmaxf(__uint_as_float(v[j]), 0.f);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              pk[16 * c + j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
      if (!work) continue;
      const int64_t row = static_cast<int64_t>(e) * p.C + rbase + lane;
      const bool valid = rbase + lane < kept;
      const bool bulk = rbase + 32 <= kept;
      if (kHidden) {
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          if (j >= 64 && ncols <= 64) f[kHidden ? j : 0] = 0.f;     // past the last column
          a = fmaxf(a, f[kHidden ? j : 0]);
        }
        const int ex = q8_exponent(a);
        const float is = q8_inv_scale(ex);
#pragma unroll
        for (int j = 0; j < kCols / 4; ++j) {
          const float* g = f + (kHidden ? 4 * j : 0);
          pk[j] = kHidden ? pack_e4m3x4(g[0] * is, g[1] * is, g[2] * is, g[3] * is) : 0u;
        }
        if (valid) p.hs[row * p.nblk_w + col0 / 128] = static_cast<uint8_t>(q8_scale_byte(ex));
        if (bulk) {
#pragma unroll
          for (int b = 0; b < kCols / 64; ++b) {
            if (b * 64 >= ncols) break;
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              st_shared_v4u(stg + lane * 64 + ((static_cast<uint32_t>(k) ^ swz) << 4),
                            pk[16 * b + 4 * k], pk[16 * b + 4 * k + 1], pk[16 * b + 4 * k + 2],
                            pk[16 * b + 4 * k + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmap_out, stg, col0 + b * 64, static_cast<int>(row));
              bulk_commit();
            }
          }
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(p.hq + row * p.n_out + col0);
#pragma unroll
          for (int k = 0; k < kCols / 16; ++k)
            if (k * 16 < ncols)
              dst[k] = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
      } else {
        if (bulk) {
#pragma unroll
          for (int b = 0; b < kCols / 32; ++b) {
            if (b * 32 >= ncols) break;
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              st_shared_v4u(stg + lane * 64 + ((static_cast<uint32_t>(k) ^ swz) << 4),
                            pk[16 * b + 4 * k], pk[16 * b + 4 * k + 1], pk[16 * b + 4 * k + 2],
                            pk[16 * b + 4 * k + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmap_out, stg, col0 + b * 32, static_cast<int>(row));
              bulk_commit();
            }
          }
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(p.y + row * p.n_out + col0);
#pragma unroll
          for (int k = 0; k < kCols / 8; ++k)
            if (k * 8 < ncols)
              dst[k] = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
      }
    }
    if (lane == 0) bulk_wait_all();        // boxes stored from shared memory are written
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, kQTmemCols);
}

// ------------------------------------------------------------------- host

bool encode_u8(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
               const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  PFN_encodeTiled enc = get_encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t strides[2] = {dims[0], dims[0] * dims[1]};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of one product: [rows, K] codes, boxes of 128 rows x 128 codes.
bool map_rows(CUtensorMap* m, const void* base, int64_t rows, int K) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint32_t box[2] = {kQK, 128};
  return encode_u8(m, base, 2, dims, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Weights [N][n_out][K]: boxes of bn rows x 128 codes of one expert (zeros
// past its last row).
bool map_weights(CUtensorMap* m, const void* base, int N, int n_out, int K, int bn) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(n_out),
                              static_cast<cuuint64_t>(N)};
  const cuuint32_t box[3] = {kQK, static_cast<cuuint32_t>(bn), 1};
  return encode_u8(m, base, 3, dims, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Hidden rows as the first product's output: boxes of 32 rows x 64 codes.
bool map_hidden_out(CUtensorMap* m, const void* base, int64_t rows, int F) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(F), static_cast<cuuint64_t>(rows)};
  const cuuint32_t box[2] = {64, 32};
  return encode_u8(m, base, 2, dims, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int BN, bool kHidden>
cudaError_t run_q8(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to,
                   const Q8Params& p, int num_sms, cudaStream_t st) {
  const size_t smem = Q8Tile<BN>::kSmem + sizeof(int) * (p.N + 1);
  static size_t smem_set[64] = {};
  cudaError_t e = ensure_smem_limit(
      reinterpret_cast<const void*>(&expert_gemm_q8_kernel<BN, kHidden>), smem, smem_set);
  if (e != cudaSuccess) return e;
  expert_gemm_q8_kernel<BN, kHidden><<<num_sms, kQThreads, smem, st>>>(ta, tb, to, p);
  return cudaGetLastError();
}

// Columns of a tile: 256 (each weight byte feeds 128 rows, each row byte 256
// columns) unless that gives fewer tiles than SMs, when narrower tiles spread
// the weights' reads over more of them.
int tile_columns(int64_t mtiles, int n_out, int num_sms, int least) {
  int bn = 256;
  while (bn > least && mtiles * ((n_out + bn - 1) / bn) < num_sms) bn /= 2;
  return bn;
}

}  // namespace

cudaError_t launch_expert_ffn_q8(const FfnQ8Args& a, cudaStream_t st) {
  const int64_t slots = static_cast<int64_t>(a.N) * a.C;
  // most row tiles that the batch can fill (the counts are on the device)
  const int64_t per_expert = static_cast<int64_t>(a.N) * ((a.C + 127) / 128);
  const int64_t mtiles = a.A < per_expert ? a.A : per_expert;
  const int bn1 = tile_columns(mtiles, a.F, a.num_sms, 128);
  const int bn2 = tile_columns(mtiles, a.d, a.num_sms, 64);
  CUtensorMap ta1, tb1, to1, ta2, tb2, to2;
  bool ok = map_rows(&ta1, a.xq, slots, a.d);
  ok = ok && map_weights(&tb1, a.w1q, a.N, a.F, a.d, bn1);
  ok = ok && map_hidden_out(&to1, a.hq, slots, a.F);
  ok = ok && map_rows(&ta2, a.hq, slots, a.F);
  ok = ok && map_weights(&tb2, a.w2q, a.N, a.d, a.F, bn2);
  ok = ok && make_tmap_bf16_2d(&to2, a.y, a.d, slots, 32, 32, true);
  if (!ok) return cudaErrorInvalidValue;

  Q8Params p{};
  p.N = a.N;
  p.n_out = a.F;
  p.K = a.d;
  p.ntiles_n = (a.F + bn1 - 1) / bn1;
  p.C = a.C;
  p.kblk = static_cast<int>(q8_blocks(a.d));
  p.nblk_w = static_cast<int>(q8_blocks(a.F));
  p.counts = a.counts;
  p.as = a.xs;
  p.ws = a.w1s;
  p.hq = a.hq;
  p.hs = a.hs;
  p.err = a.err;
  p.spin = a.spin;
  cudaError_t e = bn1 == 256 ? run_q8<256, true>(ta1, tb1, to1, p, a.num_sms, st)
                             : run_q8<128, true>(ta1, tb1, to1, p, a.num_sms, st);
  if (e != cudaSuccess) return e;
  p.n_out = a.d;
  p.K = a.F;
  p.ntiles_n = (a.d + bn2 - 1) / bn2;
  p.kblk = static_cast<int>(q8_blocks(a.F));
  p.nblk_w = static_cast<int>(q8_blocks(a.d));
  p.as = a.hs;
  p.ws = a.w2s;
  p.hq = nullptr;
  p.hs = nullptr;
  p.y = static_cast<__nv_bfloat16*>(a.y);
  if (bn2 == 256) return run_q8<256, false>(ta2, tb2, to2, p, a.num_sms, st);
  if (bn2 == 128) return run_q8<128, false>(ta2, tb2, to2, p, a.num_sms, st);
  return run_q8<64, false>(ta2, tb2, to2, p, a.num_sms, st);
}

}  // namespace smoe
