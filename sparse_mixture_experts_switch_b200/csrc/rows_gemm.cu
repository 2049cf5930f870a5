// Grouped bf16 products over experts' rows for the FFNs that keep 8-bit
// checkpoints and for their backward pass:
//
//   D[f, t] = sum_k W_e[f, k] R[t, k]   for the kept rows t of expert e
//
//   kRowsHidden  h = relu(x W1_e^T): bf16 rows, and the same rows in 8 bits
//                (format: q8.cuh) for the backward;
//   kRowsStore   y = h W2_e^T, or dx = da W1_e;
//   kRowsMask    da = (dy W2_e) where h > 0 (a bit per value).
//
// Sums are fp32 in TMEM; each result is rounded once, to bf16.  So is da, the operand
// of the two products behind it: kept in two bf16 terms it would double the bytes
// and the MMAs of both.  It costs a factor of the square root of two in the error of
// dx and dw1 (2.3e-3 of the norm against 1.7e-3, the rounding of the result alone),
// as in the layer's own backward pass.  Hidden values near a border between two bf16
// numbers may fall to either side with the order of the fp32 sum.
//
// The walk, the roles and the reasons are those of the 8-bit products
// (expert_ffn_q8.cu): CTA pairs, the weights as the MMA's M (256 features a
// tile), up to 256 of an expert's tokens as its N, warp-uniform issue loops, two
// loading warps, stages of eight MMAs (two blocks of 64 columns).  Measured,
// each product alone, 25278 kept tokens, 128 experts of 1024 x 4096 (1.07 GB of
// weights): hidden 238 us (1.4 GB with both forms of the rows), out 225 (1.3 GB),
// da 220, dx 213: 88 to 96% of the copy rate, bound by memory.  Two
// accumulators of 256 columns fill the TMEM.  The weights are read as they lie:
// [f][k] (K-major) in the forward, [k][f] (M-major) in the backward, where one
// 4-D box brings 64 rows x 2 x 64 features in the order that the MN-major
// descriptor wants.
#include <cstring>

#include "pair_walk.cuh"
#include "rows_gemm.cuh"

namespace smoe {

namespace {

constexpr int kRK = 64;                                // K block: 64 bf16 = 128 bytes
constexpr int kRStages = 3;                            // of two K blocks
constexpr uint32_t kRWBytes = 128 * kRK * 2;           // 16 KB: 128 features of a block
constexpr uint32_t kRTokBytes = 128 * kRK * 2;         // 16 KB: up to 128 token rows
constexpr uint32_t kRStageBytes = 2 * (kRWBytes + kRTokBytes);   // W, W, tokens, tokens
constexpr int kRHalves = 4;                            // drain warps per lane quarter
constexpr int kRDrainWarps = 4 * kRHalves;
constexpr int kRThreads = 128 + 32 * kRDrainWarps;
constexpr uint32_t kRIsBytes = kRHalves * 128;         // hidden, per four warps: 32 tokens' 2^-e
constexpr uint32_t kRRedBytes = kRHalves * 4 * 128;    // hidden: maxima [half][quarter][32]
constexpr uint32_t kRRowBytes = 32 * 128;              // hidden: 32 tokens x 128 codes of four warps
constexpr uint32_t kRSmem = 1024 + kRStages * kRStageBytes + kRIsBytes + kRRedBytes +
                            kRHalves * kRRowBytes + 256;   // + pts, kept
static_assert(kRSmem + 8 * (1024 + 1) <= 232448, "a CTA's shared memory");

struct RowsParams {
  WalkParams walk;
  int n_out, K;
  __nv_bfloat16* out;        // [N*C, n_out]
  uint8_t* hq;               // hidden: [N*C, n_out]
  uint8_t* hs;               //   [N*C, ceil(n_out / 128)]
  const uint32_t* mask;      // mask: [N*C, n_out / 32] bits
  float* part;               // partial sums [parts][N*C][n_out], where there are parts
  DevErr* err;
  long long spin;
};

__device__ __forceinline__ uint32_t relu_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.relu.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// kParts: a tile's sum goes in parts (split_sum.cu).
template <int kMode, bool kWMN, bool kForward, bool kParts>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kRThreads, 1)
    rows_gemm_kernel(const __grid_constant__ RowMaps maps, RowsParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  float* is_all = reinterpret_cast<float*>(smem + kRStages * kRStageBytes);
  float* red = is_all + kRIsBytes / 4;
  uint8_t* rows_out = reinterpret_cast<uint8_t*>(red) + kRRedBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(rows_out + kRHalves * kRRowBytes);
  uint64_t* empty = full + kRStages;        // full: leader, both CTAs' bytes; empty: local
  uint64_t* tfull = empty + kRStages;       // local: accumulator ready
  uint64_t* tempty = tfull + 2;             // leader: accumulator drained
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* pts = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + 256);   // [N + 1]
  int* kept = pts + p.walk.N + 1;                      // [N + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(cluster_count_x());
  const long long lim = p.spin;
  const int kblocks = p.K / kRK;
  const int kstages = (kblocks + 1) / 2;

  if (warp == 0) tiles_prefix_warp(p.walk, ncl, pts, kept);
  pdl_launch_dependents();
  if (threadIdx.x == 32) {
    for (int s = 0; s < kRStages; ++s) {
      mbar_init(&full[s], 2);               // the leader's two loading warps
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kRDrainWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int parts = kParts ? p.walk.parts : 1;
  const int total = pts[p.walk.N] * parts;  // items
  if (cid >= total) {                       // same decision in both CTAs of the pair
    pdl_wait_prerequisites();
    return;
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                           // the peer's barriers exist before any remote use
  tc_fence_after();
  pdl_wait_prerequisites();                 // the rows are there (the counts are the caller's)
  const uint32_t tmem_base = *tmem_holder;
  const uint32_t full_lead = map_to_rank(smem_u32(full), 0);
  const uint32_t tempty_lead = map_to_rank(smem_u32(tempty), 0);
  RowWalk<kForward> walk(p.walk, pts, kept);

  if (warp == 0 || warp == 2) {
    // ------------------------------ TMA: warp 0 the weights, warp 2 the tokens
    const bool tokens = warp == 2;
    if (elect_one()) tma_prefetch_desc(tokens ? &maps.tok[kRowBoxes - 1] : &maps.w);
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued_mask = 0, issued_phase = 0;
    for (int item = cid; item < total; item += ncl) {
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      const int tile = small_div(item, parts);
      const StageRange range = part_stages(item - tile * parts, parts, kstages);
      const RowTile t = walk.at(tile);
      const int half = t.nmma >> 1;
      const int box = box_of(half);
      const CUtensorMap* map = tokens ? &maps.tok[box] : &maps.w;
      const int row = tokens ? static_cast<int>(static_cast<int64_t>(t.e) * p.walk.C + t.t0 +
                                                static_cast<int>(rank) * half)
                             : t.f0 + static_cast<int>(rank) * 128;
      const uint32_t bytes = tokens ? box_rows(box) * kRK * 2 : kRWBytes;
      bool ok = true;
      for (int ks = range.begin; ks < range.end; ++ks) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, lim))) {
          if (lane == 0) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmProducer, tile);
            *abort_flag = 1;
          }
          ok = false;
          break;
        }
        const int nb = kblocks - 2 * ks < 2 ? 1 : 2;
        uint8_t* dst = smem + stage * kRStageBytes + (tokens ? 2 * kRWBytes : 0u);
        const uint32_t bar = full_lead + 8u * stage;
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * nb * bytes);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (b >= nb) break;
            const int k = (2 * ks + b) * kRK;
            if (tokens) tma_load_2d_pair(dst + b * kRTokBytes, map, bar, k, row);
            else if (kWMN) tma_load_4d_pair(dst + b * kRWBytes, map, bar, 0, k, row >> 6, t.e);
            else tma_load_3d_pair(dst + b * kRWBytes, map, bar, k, row, t.e);
          }
        }
        issued_mask |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == kRStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
    }
    // Both CTAs' bytes land on the leader's barriers: the leader waits for
    // every issued stage before the final cluster barrier.  (A stage that only
    // one of the two warps had issued before a failure does not complete: its
    // bytes are then waited for by the limit alone.)
    if (leader && lane == 0) {
      for (int s = 0; s < kRStages; ++s)
        if (((issued_mask >> s) & 1u) &&
            !mbar_wait_cluster(&full[s], (issued_phase >> s) & 1u, kCopyDrainCycles))
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereDrain, s);
    }
    settle_copies(abort_flag);
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer (leader)
    if (leader) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool any = false;
      const uint32_t smem0 = smem_u32(smem);
      // a 16-deep step in descriptor units of 16 bytes: 32 bytes along a K-major
      // row, 16 rows of 128 bytes in an M-major tile
      constexpr uint32_t kWStep = kWMN ? 128u : 2u;
      for (int item = cid; item < total; item += ncl) {
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        const int tile = small_div(item, parts);
        const StageRange range = part_stages(item - tile * parts, parts, kstages);
        const uint32_t idesc = idesc_bf16_f32_major(256, walk.at(tile).nmma, kWMN, false);
        bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, lim));
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kQTok);
        for (int ks = range.begin; ok && ks < range.end; ++ks) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, lim));
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = smem0 + stage * kRStageBytes;
          const uint64_t wd = kWMN ? sw128_mnmajor_desc(at, 8192u) : sw128_kmajor_desc(at);
          const uint64_t td = sw128_kmajor_desc(at + 2 * kRWBytes);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_pair(d_tmem, wd + kWStep * k, td + 2 * k, idesc,
                             ks != range.begin || k != 0 ? 1u : 0u);
            if (2 * ks + 1 < kblocks) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_bf16_pair(d_tmem, wd + (kRWBytes >> 4) + kWStep * k,
                               td + (kRTokBytes >> 4) + 2 * k, idesc, 1u);
            }
            umma_commit_pair(&empty[stage], 0x3);
          }
          any = true;
          if (++stage == kRStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) {
          if (lane == 0) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmMma, tile);
            *abort_flag = 1;
          }
          break;
        }
        if (elect_one()) umma_commit_pair(&tfull[acc], 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      __syncwarp();
      if (any && __any_sync(0xffffffffu, *abort_flag)) {
        if (elect_one()) umma_commit_pair(drain, 0x1);
        if (!__all_sync(0xffffffffu, mbar_wait(drain, 0, kDefaultSpinCycles)) && lane == 0)
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereDrain, -1);
      }
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------- drain warps
    // Quarter q of the CTA's 128 features (one a lane); the kRHalves warps of a
    // quarter take the chunks of 32 tokens in turn, from another one on in each
    // tile (tiles of one chunk then drain side by side).
    const int q = warp & 3;
    const int h = (warp - 4) >> 2;
    float* isv = is_all + h * 32;                      // hidden: tokens' 2^-e
    float* r = red + h * 128;                          // hidden: [quarter][32]
    const int64_t nblk = q8_blocks(p.n_out);
    int acc = 0;
    uint32_t acc_phase = 0;
    int first = h;                                     // the warp's first chunk of a tile
    // The accumulator goes back once the warp's last chunk is in registers.  Relaxed:
    // only TMEM loads, which have been waited for, are handed over (a release would
    // hold the warp until its rows' stores had reached memory).
    auto hand_back = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive_relaxed(&tempty[b]);
        else mbar_arrive_remote_relaxed(tempty_lead + 8u * b);
      }
    };
    for (int item = cid; item < total; item += ncl) {
      const int tile = small_div(item, parts);
      bool ok = __all_sync(0xffffffffu, mbar_wait_sleepy(&tfull[acc], acc_phase, lim));
      if (kMode == kRowsHidden) ok = all_of_barrier(ok, 1 + h);   // they meet below: go on together
      if (!ok) {
        if (lane == 0) {
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmEpilogue, tile);
          *abort_flag = 1;
        }
        break;
      }
      tc_fence_after();
      const RowTile t = walk.at(tile);
      const int fc = t.f0 + static_cast<int>(rank) * 128;          // the CTA's first feature
      const int fb = fc + q * 32;                                  // the warp's
      const bool on = fb < p.n_out;                                // warp-uniform
      const int nch = (t.nv + 31) >> 5;
      const int64_t row0 = static_cast<int64_t>(t.e) * p.walk.C + t.t0;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(acc * kQTok);
      if (first >= nch) hand_back(acc);
      for (int c = first; c < nch; c += kRHalves) {
        const int j0 = c * 32;
        const int jn = t.nv - j0 < 32 ? t.nv - j0 : 32;            // tokens of the chunk
        uint32_t bits = 0;
        if (kMode == kRowsMask && !kParts && on && lane < jn)
          bits = p.mask[(row0 + j0 + lane) * (p.n_out >> 5) + (fb >> 5)];
        uint32_t v[32];
        tmem_ld32_issue(taddr + static_cast<uint32_t>(j0), v);
        tmem_ld_wait(v);
        if (c + kRHalves >= nch) hand_back(acc);
        if (kParts) {
          // the part's sums, 32 features of a token a store; rows_join finishes them
          if (on) {
            float* dst = p.part + ((item - tile * parts) * (p.walk.N * p.walk.C) + row0 + j0) *
                                      p.n_out + fb + lane;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < jn) dst[static_cast<int64_t>(j) * p.n_out] = __uint_as_float(v[j]);
          }
          continue;
        }
        if (kMode == kRowsMask) {
          bits = transpose_bits(bits, lane);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = (bits >> j) & 1u ? v[j] : 0u;
        }
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float lo = __uint_as_float(v[2 * i]), hi = __uint_as_float(v[2 * i + 1]);
          pk[i] = kMode == kRowsHidden ? relu_bf16x2(lo, hi) : pack_bf16x2(lo, hi);
        }
        if (on) {
          // two features of a token a lane, 2 tokens x 64 bytes a store
          __nv_bfloat16* dst =
              p.out + (row0 + j0 + (lane & 1)) * p.n_out + fb + (lane & ~1);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t z = transpose_halves(pk[j / 2], lane);
            if (j + (lane & 1) < jn)
              *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * p.n_out) = z;
          }
        }
        if (kMode != kRowsHidden) continue;
        // 8 bits: the token's maximum over the CTA's 128 features (without those that
        // are NaN; zero where all are)
        uint32_t m[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i] = pk[i];
        r[q * 32 + lane] = __uint_as_float(warp_token_max(m, lane));
        named_bar_sync(1 + h, 128);
        const float a = fmaxf(fmaxf(r[lane], r[32 + lane]), fmaxf(r[64 + lane], r[96 + lane]));
        const int ex = q8_exponent(fmaxf(a, 0.f));
        // (what the four warps share is written after this chunk's first barrier, read
        // before its second or the next chunk's first; expert_ffn_q8.cu has the rows' layout)
        isv[lane] = q8_inv_scale(ex);
        __syncwarp();
        const uint32_t rows = smem_u32(rows_out) + h * kRRowBytes;
        if (on) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (4 * k >= jn) break;
            const float4 s = reinterpret_cast<const float4*>(isv)[k];
            // what is above zero stays above zero, NaN stays NaN
            const float x0 = bf16_lo(pk[2 * k]), x1 = bf16_hi(pk[2 * k]);
            const float x2 = bf16_lo(pk[2 * k + 1]), x3 = bf16_hi(pk[2 * k + 1]);
            const uint32_t w = relu_e4m3x4(max_nan(x0 * s.x, x0 > 0.f ? kQ8Least : 0.f),
                                           max_nan(x1 * s.y, x1 > 0.f ? kQ8Least : 0.f),
                                           max_nan(x2 * s.z, x2 > 0.f ? kQ8Least : 0.f),
                                           max_nan(x3 * s.w, x3 > 0.f ? kQ8Least : 0.f));
            st_shared_u32(row_word(rows, 4 * k, q, lane), transpose_bytes(w, lane));
          }
        }
        named_bar_sync(1 + h, 128);
        store_rows(rows, p.hq, row0 + j0, jn, fc, p.n_out, q, lane);
        if (q == 0 && on && lane < jn)
          p.hs[(row0 + j0 + lane) * nblk + (fc >> 7)] = static_cast<uint8_t>(q8_scale_byte(ex));
      }
      first = (first + 1) % kRHalves;
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                          // no CTA leaves while its peer may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

template <int kMode, bool kWMN, bool kForward, bool kParts>
cudaError_t run_rows_parts(const RowsGemmArgs& a, cudaStream_t st) {
  const int64_t slots = static_cast<int64_t>(a.N) * a.C;
  RowMaps maps;
  bool ok = kWMN ? make_tmap_mn_major(&maps.w, a.w, a.n_out, a.K, a.N)
                 : make_tmap_bf16_3d(&maps.w, a.w, a.K, a.n_out, a.N, kRK, 128);
  for (int i = 0; i < kRowBoxes; ++i)
    ok = ok && make_tmap_bf16_2d(&maps.tok[i], a.rows, a.K, slots, kRK, box_rows(i));
  if (!ok) return cudaErrorInvalidValue;
  RowsParams p{};
  p.walk.N = a.N;
  p.walk.C = a.C;
  p.walk.counts = a.counts;
  p.walk.ntiles_f = (a.n_out + 255) / 256;
  p.n_out = a.n_out;
  p.K = a.K;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.hq = a.hq;
  p.hs = a.hs;
  p.mask = a.mask;
  p.err = a.err;
  p.spin = a.spin;
  p.walk.parts = a.parts;
  p.part = a.part;
  const size_t smem = kRSmem + sizeof(int) * (2 * a.N + 2);
  static size_t smem_set[64] = {};
  cudaError_t e = ensure_smem_limit(
      reinterpret_cast<const void*>(&rows_gemm_kernel<kMode, kWMN, kForward, kParts>), smem, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_dependent(rows_gemm_kernel<kMode, kWMN, kForward, kParts>, (a.num_sms / 2) * 2,
                       kRThreads, smem, st, maps, p);
  if (e != cudaSuccess || !kParts) return e;
  JoinArgs j{};
  j.parts = a.parts;
  j.N = a.N;
  j.C = a.C;
  j.n_out = a.n_out;
  j.counts = a.counts;
  j.part = a.part;
  j.out = a.out;
  j.hq = a.hq;
  j.hs = a.hs;
  j.mask = a.mask;
  j.num_sms = a.num_sms;
  return launch_rows_join(kMode, j, st);
}

template <int kMode, bool kWMN, bool kForward>
cudaError_t run_rows(const RowsGemmArgs& a, cudaStream_t st) {
  return a.parts > 1 ? run_rows_parts<kMode, kWMN, kForward, true>(a, st)
                     : run_rows_parts<kMode, kWMN, kForward, false>(a, st);
}

}  // namespace

// bf16 [outer][k][m] (m contiguous, a multiple of 64) as MN-major operand tiles:
// one box is 64 k rows of 2 x 64 consecutive m, each 64 a swizzled 128-byte row.
bool make_tmap_mn_major(CUtensorMap* map, const void* base, int64_t m, int64_t k, int64_t outer) {
  PFN_encodeTiled enc = get_encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(m / 64),
                              static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(m) * 2, 128,
                                 static_cast<cuuint64_t>(m) * static_cast<cuuint64_t>(k) * 2};
  const cuuint32_t box[4] = {64, 64, 2, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_rows_hidden(const RowsGemmArgs& a, cudaStream_t st) {
  return run_rows<kRowsHidden, false, true>(a, st);
}
cudaError_t launch_rows_out(const RowsGemmArgs& a, cudaStream_t st) {
  return run_rows<kRowsStore, false, false>(a, st);
}
cudaError_t launch_rows_da(const RowsGemmArgs& a, cudaStream_t st) {
  return run_rows<kRowsMask, true, true>(a, st);
}
cudaError_t launch_rows_dx(const RowsGemmArgs& a, cudaStream_t st) {
  return run_rows<kRowsStore, true, false>(a, st);
}

}  // namespace smoe
