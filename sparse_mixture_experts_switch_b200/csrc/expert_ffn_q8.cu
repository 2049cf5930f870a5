// The experts' ReLU FFNs on 8-bit rows and weights (format: q8.cuh):
//
//   h = relu(x W1_e^T),  (hq, hs) = 8-bit rows of h,  y = h W2_e^T (bf16)
//
//   D[f, t] = sum over blocks k of 2^(sw[f / 128, k] + sa[t, k]) sum_j w[f, k, j] a[t, k, j]
//
// The tensor core applies the scales itself: tcgen05.mma.kind::mxf8f6f4 with
// block_scale multiplies each 32-deep step by one e8m0 scale of each operand
// row, which it reads from TMEM.  A scale here covers 128 columns, so the four
// 32-deep steps of a block use the same byte (the descriptor's scale-factor id
// picks one byte of a row's 32-bit word): one word of a row is the scales of
// 512 columns, exactly four consecutive bytes of the row-major scale array.
// Products and sums are fp32 in TMEM.
//
// One persistent kernel on CTA pairs for both products, with the weights as the
// MMA's M and the tokens as its flexible N: a tile is 256 output features x up
// to 256 of one expert's tokens (the expert's tokens are split evenly, in steps
// of 16, so few columns are padding).  CTA r of a pair holds features 128 r ..
// 128 r + 127 and loads half of the tokens.  Two accumulators share the 448
// TMEM columns that the scales leave (acc_column).
//   * warp 0 loads the weights and warp 2 the tokens by TMA, 256 bytes deep (two
//     boxes in the 128-byte swizzle), through a ring of three stages;
//   * warp 3 brings the scales of each 512 columns, laid out as tcgen05.cp wants
//     them (row r at lane r % 32, word r / 32; both CTAs need every token's),
//     from arrays of words [512 columns][slot] that the gather and the first
//     product's drain write (a tile's rows are then consecutive);
//   * warp 1 of the leader copies the scales to TMEM and issues the MMAs;
//   * warps 4-19 drain: one feature a lane, 32 tokens at a time.  For the
//     hidden rows a token's scale is over the CTA's 128 features, that is 32
//     lanes of four warps: a warp maximum per token, then one exchange through
//     shared memory.
//
// At these tile sizes (a 32-deep MMA takes N / 2 cycles) the issuing warps set
// the pace as easily as the tensor core: a TMA issue takes about 200 cycles and
// a stage of four MMAs about 510 when one lane of a divergent warp issues them,
// 160 and 350 when the whole warp runs the loop and an elected lane issues
// (addresses then live in uniform registers), and a stage's waits and commit
// are another 150: hence warp-uniform loops, two loading warps, and stages of
// eight MMAs.
//
// Measured, each product alone: 25278 kept tokens, 128 experts of 1024 x 4096,
// 126 us (weights 537 MB, hidden rows 107 MB) and 116 us (671 MB in all); 16
// experts of 4096 x 10240 with 3148 tokens 141 and 152 us.  There the weights'
// stream (103 us at the copy rate) and shared memory (operands in and out at 128
// bytes a cycle: about 470 cycles for a block of 104 tokens a CTA, the MMAs 416)
// are close to each other; calls back to back run into the power limit.
#include <cstring>

#include "pair_walk.cuh"
#include "rows_gemm.cuh"

namespace smoe {

namespace {

constexpr int kQK = 128;                               // K block: 128 codes
constexpr int kQStages = 3;                            // of two K blocks
constexpr uint32_t kQWBytes = 128 * kQK;               // 16 KB: 128 weight rows of a block
constexpr uint32_t kQTokBytes = kQTok / 2 * kQK;       // 16 KB: up to 128 token rows
constexpr uint32_t kQStageBytes = 2 * (kQWBytes + kQTokBytes);   // W, W, tokens, tokens
constexpr int kQHalves = 4;                            // drain warps per lane quarter
constexpr int kQDrainWarps = 4 * kQHalves;
constexpr int kQThreads = 128 + 32 * kQDrainWarps;
constexpr int kSfSlots = 4;                            // ring of scale groups (512 columns each)
constexpr int kSfTmemSlots = 4;
constexpr uint32_t kSfBytes = 3 * 512;                 // weight rows, tokens 0-127, 128-255
constexpr uint32_t kSfTmem = 448;                      // TMEM columns 448 + 16 i, i < 4
constexpr uint32_t kQStageOut = 128;                   // hidden, per four warps: 32 tokens' 2^-e
constexpr uint32_t kQRedBytes = kQHalves * 4 * 128;    // hidden: maxima [half][quarter][32]
constexpr uint32_t kQRowBytes = 32 * 128;              // hidden: 32 tokens x 128 codes of four warps
constexpr uint32_t kQBarBytes = 512;
constexpr uint32_t kQTmemCols = 512;
constexpr uint32_t kQSmem = 1024 + kQStages * kQStageBytes + kQHalves * kQStageOut +
                            kSfSlots * kSfBytes + kQRedBytes + kQHalves * kQRowBytes +
                            kQBarBytes;                // + pts, kept
static_assert(kQSmem + 8 * (1024 + 1) <= 232448, "a CTA's shared memory");

struct Q8Params {
  WalkParams walk;
  int n_out, K;
  int kblk;                  // scale bytes of a weight row: ceil(K / 128)
  int nblk_w;                // weight blocks along n_out: ceil(n_out / 128)
  int64_t slots;             // N*C
  const uint32_t* as;        // scale words of the rows [ceil(K / 512)][N*C]
  const uint8_t* ws;         // [N, nblk_w, kblk]
  uint8_t* hq;               // hidden: [N*C, n_out]
  uint8_t* hs;               // hidden: scale words [ceil(n_out / 512)][N*C], by bytes
  __nv_bfloat16* y;          // else: [N*C, n_out]
  float* part;               // partial sums [parts][N*C][n_out], where there are parts
  DevErr* err;
  long long spin;
};

// D (+)= scaled A x scaled B^T over both CTAs; one thread of the leader.
__device__ __forceinline__ void umma_q8_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 rows x 16 bytes of each CTA's shared memory (512 consecutive bytes) to 4
// columns of its TMEM, repeated in the four lane quarters.
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
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

// First TMEM column of a tile's accumulator: even tiles grow from column 0, odd
// ones end at the scales (column 448).  Two tiles in a row overlap where their
// columns sum to more than 448, by 64 columns at most.
__device__ __forceinline__ uint32_t acc_column(int acc, int nmma) {
  return acc == 0 ? 0u : kSfTmem - static_cast<uint32_t>(nmma);
}

__device__ __forceinline__ void cp_async4_s(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// kParts: a tile's sum goes in parts (split_sum.cu).
template <bool kHidden, bool kParts>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kQThreads, 1)
    expert_gemm_q8_kernel(const __grid_constant__ RowMaps maps, Q8Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* stage_out = smem + kQStages * kQStageBytes;
  uint8_t* sf = stage_out + kQHalves * kQStageOut;
  float* red = reinterpret_cast<float*>(sf + kSfSlots * kSfBytes);
  uint8_t* rows_out = reinterpret_cast<uint8_t*>(red) + kQRedBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(rows_out + kQHalves * kQRowBytes);
  uint64_t* empty = full + kQStages;        // full: leader, both CTAs' bytes; empty: local
  uint64_t* sfull = empty + kQStages;       // scales in shared memory (leader: both CTAs')
  uint64_t* sempty = sfull + kSfSlots;      // local: copied to TMEM
  uint64_t* tfull = sempty + kSfSlots;      // local: accumulator ready
  uint64_t* tempty = tfull + 2;             // leader: accumulator drained
  uint64_t* tover = tempty + 2;             // leader: the columns that the next tile may need
  uint64_t* drain = tover + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* pts = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + kQBarBytes);   // [N + 1]
  int* kept = pts + p.walk.N + 1;                      // [N + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(cluster_count_x());
  const long long lim = p.spin;
  const int kblocks = (p.K + kQK - 1) / kQK;

  if (warp == 0) tiles_prefix_warp(p.walk, ncl, pts, kept);
  pdl_launch_dependents();
  if (threadIdx.x == 32) {
    for (int s = 0; s < kQStages; ++s) {
      mbar_init(&full[s], 2);               // the leader's two loading warps
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      // 32 asynchronous copies' arrivals and the warp's; the leader's also takes
      // the follower's relay
      mbar_init(&sfull[s], leader ? 34 : 33);
      mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kQDrainWarps);
      mbar_init(&tover[b], 2 * kQDrainWarps);
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
    tmem_alloc_pair(tmem_holder, kQTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                           // the peer's barriers exist before any remote use
  tc_fence_after();
  pdl_wait_prerequisites();                 // the rows are there (the counts are the caller's)
  const uint32_t tmem_base = *tmem_holder;
  const uint32_t full_lead = map_to_rank(smem_u32(full), 0);
  const uint32_t sfull_lead = map_to_rank(smem_u32(sfull), 0);
  const uint32_t tempty_lead = map_to_rank(smem_u32(tempty), 0);
  const uint32_t tover_lead = map_to_rank(smem_u32(tover), 0);

  RowWalk<kHidden> walk(p.walk, pts, kept);
  const int kstages = (kblocks + 1) / 2;
  const int groups = (kblocks + 3) / 4;     // of scales: two stages each; parts are of whole groups
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
      const StageRange range = part_stages(item - tile * parts, parts, groups);
      const int ks1 = 2 * range.end < kstages ? 2 * range.end : kstages;
      const RowTile t = walk.at(tile);
      const int half = t.nmma >> 1;
      const int box = box_of(half);
      const CUtensorMap* map = tokens ? &maps.tok[box] : &maps.w;
      const int row = tokens ? static_cast<int>(static_cast<int64_t>(t.e) * p.walk.C + t.t0 +
                                                static_cast<int>(rank) * half)
                             : t.f0 + static_cast<int>(rank) * 128;
      const uint32_t bytes = tokens ? box_rows(box) * kQK : kQWBytes;
      const uint32_t step = tokens ? kQTokBytes : kQWBytes;
      bool ok = true;
      for (int ks = 2 * range.begin; ks < ks1; ++ks) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, lim))) {
          if (lane == 0) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmProducer, tile);
            *abort_flag = 1;
          }
          ok = false;
          break;
        }
        const int nb = kblocks - 2 * ks < 2 ? 1 : 2;
        uint8_t* dst = smem + stage * kQStageBytes + (tokens ? 2 * kQWBytes : 0u);
        const uint32_t bar = full_lead + 8u * stage;
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * nb * bytes);
          if (tokens) {
            tma_load_2d_pair(dst, map, bar, 2 * ks * kQK, row);
            if (nb == 2) tma_load_2d_pair(dst + step, map, bar, (2 * ks + 1) * kQK, row);
          } else {
            tma_load_3d_pair(dst, map, bar, 2 * ks * kQK, row, t.e);
            if (nb == 2) tma_load_3d_pair(dst + step, map, bar, (2 * ks + 1) * kQK, row, t.e);
          }
        }
        issued_mask |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == kQStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
    }
    // Both CTAs' bytes land on the leader's barriers: the leader waits for
    // every issued stage before the final cluster barrier.  (A stage that only
    // one of the two warps had issued before a failure does not complete: its
    // bytes are then waited for by the limit alone.)
    if (leader && lane == 0) {
      for (int s = 0; s < kQStages; ++s)
        if (((issued_mask >> s) & 1u) &&
            !mbar_wait_cluster(&full[s], (issued_phase >> s) & 1u, kCopyDrainCycles))
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereDrain, s);
    }
    settle_copies(abort_flag);
  } else if (warp == 3) {
    // ------------------------------------------------------------- scales
    // Groups of 512 columns by asynchronous copies, as far ahead as the ring
    // goes (a group is consumed in about the time that one load takes).  The
    // copies arrive on the group's barrier by themselves; the proxy fence between
    // them and tcgen05.cp is left to warps with no copies of their own in flight,
    // since it waits for all of a thread's.
    const bool words = (p.kblk & 3) == 0;
    int item = cid, g = 0;
    RowTile t{};
    StageRange range{};
    const uint8_t* wrow = nullptr;
    uint32_t wb[4] = {};
    auto enter = [&]() {
      const int tile = small_div(item, parts);
      range = part_stages(item - tile * parts, parts, groups);
      g = range.begin;
      t = walk.at(tile);
      int b = (t.f0 >> 7) + static_cast<int>(rank);
      if (b >= p.nblk_w) b = p.nblk_w - 1;             // features past the end: zero rows
      wrow = p.ws + (static_cast<int64_t>(t.e) * p.nblk_w + b) * p.kblk;
    };
    // the weight rows' bytes where their word is not aligned, asked for a group
    // ahead (past the row's end: its last one)
    auto ask = [&]() {
      if (words || item >= total) return;
      const int left = p.kblk - 4 * g;
#pragma unroll
      for (int k = 0; k < 4; ++k) wb[k] = __ldg(wrow + 4 * g + (k < left ? k : left - 1));
    };
    int slot = 0;
    uint32_t phase = 0;
    enter();
    ask();
    while (item < total) {
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      if (!__all_sync(0xffffffffu, mbar_wait(&sempty[slot], phase ^ 1u, lim))) {
        if (lane == 0) {
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmProducer, item);
          *abort_flag = 1;
        }
        break;
      }
      const uint32_t dst = smem_u32(sf + slot * kSfBytes) + lane * 16;
      const uint32_t* src =
          p.as + static_cast<int64_t>(g) * p.slots + static_cast<int64_t>(t.e) * p.walk.C + t.t0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {                    // rows past the last: any scale
        const int r = 32 * j + lane;
        cp_async4_s(dst + 512 + (j >> 2) * 512 + (j & 3) * 4, src + (r < t.nv ? r : 0));
      }
      // the weight rows' word, four times a lane
      if (words) {
#pragma unroll
        for (int j = 0; j < 4; ++j) cp_async4_s(dst + j * 4, wrow + 4 * g);
        cp_async_mbar_arrive_noinc(&sfull[slot]);
        if (lane == 0) mbar_arrive_relaxed(&sfull[slot]);
      } else {
        cp_async_mbar_arrive_noinc(&sfull[slot]);
        const uint32_t u = wb[0] | wb[1] << 8 | wb[2] << 16 | wb[3] << 24;
        st_shared_v4u(dst, u, u, u, u);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[slot]);
      }
      if (++slot == kSfSlots) { slot = 0; phase ^= 1u; }
      if (++g == range.end) {
        item += ncl;
        if (item < total) enter();
      }
      ask();
    }
    cp_async_wait_all();                               // none in flight behind this
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer (leader)
    if (leader) {
      int stage = 0, slot = 0, tslot = 0;
      uint32_t phase = 0, sphase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      uint32_t sfa = 0;
      int last_nmma = 0;
      bool any = false;
      const uint32_t smem0 = smem_u32(smem), sf0 = smem_u32(sf);
      for (int item = cid; item < total; item += ncl) {
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        const int tile = small_div(item, parts);
        const StageRange range = part_stages(item - tile * parts, parts, groups);
        const int ks0 = 2 * range.begin;
        const int ks1 = 2 * range.end < kstages ? 2 * range.end : kstages;
        const int nmma = walk.at(tile).nmma;
        const uint32_t idesc = idesc_q8(256, nmma);
        // The accumulator's last tile is drained.  Its tover was arrived at before its
        // tempty, but relaxed and on another barrier, so that is waited for too: the
        // wait below for the next phase of the same barrier (one parity bit) is then
        // never met by the phase before it.
        bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, lim) &&
                                              mbar_wait_cluster(&tover[acc], acc_phase ^ 1u, lim));
        // columns that the last tile has too: its drain takes those first
        if (ok && nmma + last_nmma > static_cast<int>(kSfTmem))
          ok = __all_sync(0xffffffffu,
                          mbar_wait_cluster(&tover[acc ^ 1], acc == 0 ? acc_phase ^ 1u : acc_phase, lim));
        last_nmma = nmma;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc_column(acc, nmma);
        for (int ks = ks0; ok && ks < ks1; ++ks) {
          if ((ks & 1) == 0) {                         // the scales of the next 4 K blocks
            ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sfull[slot], sphase, lim));
            if (!ok) break;
            fence_proxy_async_smem();                  // this CTA's scales -> tcgen05.cp
            tc_fence_after();
            sfa = tmem_base + kSfTmem + 16u * tslot;
            tslot = (tslot + 1) % kSfTmemSlots;   // (copies and MMAs run in order)
            const uint32_t src = sf0 + slot * kSfBytes;
            if (elect_one()) {
              tmem_cp_scales_pair(sfa, scales_desc(src));
              tmem_cp_scales_pair(sfa + 4, scales_desc(src + 512));
              if (nmma > 128) tmem_cp_scales_pair(sfa + 8, scales_desc(src + 1024));
              umma_commit_pair(&sempty[slot], 0x3);
            }
            any = true;
            if (++slot == kSfSlots) { slot = 0; sphase ^= 1u; }
          }
          ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, lim));
          if (!ok) break;
          tc_fence_after();
          const uint64_t wd = sw128_kmajor_desc(smem0 + stage * kQStageBytes);
          const uint64_t td = sw128_kmajor_desc(smem0 + stage * kQStageBytes + 2 * kQWBytes);
          const uint32_t id = idesc | idesc_byte(2u * (ks & 1));
          if (elect_one()) {
            // descriptors count 16 bytes: a 32-deep step is 2 of them
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_q8_pair(d_tmem, wd + 2 * k, td + 2 * k, id, sfa, sfa + 4,
                           ks != ks0 || k != 0 ? 1u : 0u);
            if (2 * ks + 1 < kblocks) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_q8_pair(d_tmem, wd + (kQWBytes >> 4) + 2 * k, td + (kQTokBytes >> 4) + 2 * k,
                             id + idesc_byte(1), sfa, sfa + 4, 1u);
            }
            umma_commit_pair(&empty[stage], 0x3);
          }
          any = true;
          if (++stage == kQStages) { stage = 0; phase ^= 1u; }
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
    } else {
      // -------------------------- follower: relay its scales to the leader
      int slot = 0;
      uint32_t phase = 0;
      for (int item = cid; item < total; item += ncl) {
        bool ok = !__any_sync(0xffffffffu, *abort_flag);
        const int tile = small_div(item, parts);
        const StageRange range = part_stages(item - tile * parts, parts, groups);
        for (int g = range.begin; ok && g < range.end; ++g) {
          ok = __all_sync(0xffffffffu, mbar_wait(&sfull[slot], phase, lim));
          if (!ok) {
            if (lane == 0) {
              report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmProducer, tile);
              *abort_flag = 1;
            }
            break;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(sfull_lead + 8u * slot);
          if (++slot == kSfSlots) { slot = 0; phase ^= 1u; }
        }
        if (!ok) break;
      }
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------- drain warps
    // Quarter q of the CTA's 128 features (one a lane); the kQHalves warps of a
    // quarter take the chunks of 32 tokens in turn (from another one on in each
    // tile: tiles of one chunk then drain side by side), first those whose columns
    // the next tile may need.
    const int q = warp & 3;
    const int h = (warp - 4) >> 2;
    float* isv = reinterpret_cast<float*>(stage_out) + h * 32;   // tokens' 2^-e
    float* r = red + h * 128;                          // [quarter][32]
    int acc = 0;
    uint32_t acc_phase = 0;
    int first = h;                                     // the warp's first chunk of a tile
    // relaxed: only TMEM loads, which have been waited for, are handed over (a
    // release would hold the warp until its rows' stores had reached memory)
    auto arrive_lead = [&](uint64_t* bar, uint32_t lead, int b) {
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive_relaxed(&bar[b]);
        else mbar_arrive_remote_relaxed(lead + 8u * b);
      }
    };
    for (int item = cid; item < total; item += ncl) {
      const int tile = small_div(item, parts);
      bool ok = __all_sync(0xffffffffu, mbar_wait_sleepy(&tfull[acc], acc_phase, lim));
      if (kHidden) ok = all_of_barrier(ok, 1 + h);   // they meet below: go on together
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
                             acc_column(acc, t.nmma);
      if (first >= 2 || first >= nch) arrive_lead(tover, tover_lead, acc);   // none of those
      if (first >= nch) {
        tc_fence_before();
        arrive_lead(tempty, tempty_lead, acc);
      }
      for (int i = first; i < nch; i += kQHalves) {
        const int c = acc == 0 ? nch - 1 - i : i;
        uint32_t v[32];
        tmem_ld32_issue(taddr + static_cast<uint32_t>(c * 32), v);
        tmem_ld_wait(v);
        if (i < 2 || i + kQHalves >= nch) tc_fence_before();
        if (i < 2) arrive_lead(tover, tover_lead, acc);            // at most 64 columns overlap
        if (i + kQHalves >= nch) arrive_lead(tempty, tempty_lead, acc);   // the warp's last
        const int j0 = c * 32;
        const int jn = t.nv - j0 < 32 ? t.nv - j0 : 32;            // tokens of the chunk
        if (kParts) {
          // the part's sums, 32 features of a token a store; rows_join finishes them
          if (on) {
            float* dst = p.part + ((item - tile * parts) * p.slots + row0 + j0) * p.n_out + fb + lane;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < jn) dst[static_cast<int64_t>(j) * p.n_out] = __uint_as_float(v[j]);
          }
          continue;
        }
        if (kHidden) {
          // the maximum as an upper bound with the same scale: the upper 16 bits of
          // the fp32 number, rounded up (a scale changes where the significand passes
          // 1.75, a border that 16 bits hold; what is below zero becomes 0, the ReLU,
          // and so does NaN, which does not count)
          uint32_t m[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            m[i] = max_bf16x2(__byte_perm(v[2 * i] + 0xFFFFu, v[2 * i + 1] + 0xFFFFu, 0x7632), 0u);
          const float mine = __uint_as_float(warp_token_max(m, lane));
          r[q * 32 + lane] = mine;
          named_bar_sync(1 + h, 128);
          const float a = fmaxf(fmaxf(r[lane], r[32 + lane]), fmaxf(r[64 + lane], r[96 + lane]));
          const int ex = q8_exponent(a);
          // the token's 2^-e to every lane (the four warps write the same; what they
          // share is written after this chunk's first barrier, read before its second
          // or the next chunk's first)
          isv[lane] = q8_inv_scale(ex);
          __syncwarp();
          // codes of tokens 4k .. 4k + 3 of this feature in a word; a transpose of
          // four lanes' words makes it four features of token 4k + lane % 4, and the
          // four warps' words meet in shared memory as rows (with stores of 4 tokens x
          // 32 bytes straight from the warps the first product at Large's shape took
          // 141 us against 126)
          const uint32_t rows = smem_u32(rows_out) + h * kQRowBytes;
          if (on) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (4 * k >= jn) break;
              const float4 sc = reinterpret_cast<const float4*>(isv)[k];
              const uint32_t w = relu_e4m3x4(
                  __uint_as_float(v[4 * k]) * sc.x, __uint_as_float(v[4 * k + 1]) * sc.y,
                  __uint_as_float(v[4 * k + 2]) * sc.z, __uint_as_float(v[4 * k + 3]) * sc.w);
              st_shared_u32(row_word(rows, 4 * k, q, lane), transpose_bytes(w, lane));
            }
          }
          named_bar_sync(1 + h, 128);
          store_rows(rows, p.hq, row0 + j0, jn, fc, p.n_out, q, lane);
          if (q == 0 && on && lane < jn)
            p.hs[(static_cast<int64_t>(fc >> 9) * p.slots + row0 + j0 + lane) * 4 + ((fc >> 7) & 3)] =
                static_cast<uint8_t>(q8_scale_byte(ex));
        } else if (on) {
          // tokens j and j + 1 of this feature in a word; exchanged with the next
          // lane it is two features of one token, and a store writes 2 tokens x 64
          // bytes
          __nv_bfloat16* dst = p.y + (row0 + j0 + (lane & 1)) * p.n_out + fb + (lane & ~1);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t w = pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
            const uint32_t z = transpose_halves(w, lane);
            if (j + (lane & 1) < jn)
              *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * p.n_out) = z;
          }
        }
      }
      first = (first + 1) % kQHalves;
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                          // no CTA leaves while its peer may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kQTmemCols);
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

// Rows of one product [rows, K]: boxes of `box` rows x 128 codes.
bool map_rows(CUtensorMap* m, const void* base, int64_t rows, int K, uint32_t box) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint32_t b[2] = {kQK, box};
  return encode_u8(m, base, 2, dims, b, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Weights [N][n_out][K]: boxes of 128 rows x 128 codes of one expert (zeros
// past its last row).
bool map_weights(CUtensorMap* m, const void* base, int N, int n_out, int K) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(n_out),
                              static_cast<cuuint64_t>(N)};
  const cuuint32_t b[3] = {kQK, 128, 1};
  return encode_u8(m, base, 3, dims, b, CU_TENSOR_MAP_SWIZZLE_128B);
}
template <bool kHidden, bool kParts>
cudaError_t run_q8_parts(const void* rows, const void* weights, const Q8Params& p, int num_sms,
                   cudaStream_t st) {
  const int64_t slots = static_cast<int64_t>(p.walk.N) * p.walk.C;
  RowMaps maps;
  bool ok = map_weights(&maps.w, weights, p.walk.N, p.n_out, p.K);
  for (int i = 0; i < kRowBoxes; ++i)
    ok = ok && map_rows(&maps.tok[i], rows, slots, p.K, box_rows(i));
  if (!ok) return cudaErrorInvalidValue;
  const size_t smem = kQSmem + sizeof(int) * (2 * p.walk.N + 2);
  static size_t smem_set[64] = {};
  cudaError_t e = ensure_smem_limit(
      reinterpret_cast<const void*>(&expert_gemm_q8_kernel<kHidden, kParts>), smem, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_dependent(expert_gemm_q8_kernel<kHidden, kParts>, (num_sms / 2) * 2, kQThreads, smem,
                       st, maps, p);
  if (e != cudaSuccess || !kParts) return e;
  JoinArgs j{};
  j.parts = p.walk.parts;
  j.N = p.walk.N;
  j.C = p.walk.C;
  j.n_out = p.n_out;
  j.counts = p.walk.counts;
  j.part = p.part;
  j.out = p.y;
  j.hq = p.hq;
  j.hs = p.hs;
  j.num_sms = num_sms;
  return launch_rows_join(kHidden ? kRowsHiddenQ8 : kRowsStore, j, st);
}

template <bool kHidden>
cudaError_t run_q8(const void* rows, const void* weights, const Q8Params& p, int num_sms,
                   cudaStream_t st) {
  return p.walk.parts > 1 ? run_q8_parts<kHidden, true>(rows, weights, p, num_sms, st)
                          : run_q8_parts<kHidden, false>(rows, weights, p, num_sms, st);
}

}  // namespace

cudaError_t launch_expert_ffn_q8(const FfnQ8Args& a, cudaStream_t st) {
  const int64_t slots = static_cast<int64_t>(a.N) * a.C;
  Q8Params p{};
  p.walk.N = a.N;
  p.n_out = a.F;
  p.K = a.d;
  p.walk.ntiles_f = (a.F + 255) / 256;
  p.walk.C = a.C;
  p.kblk = static_cast<int>(q8_blocks(a.d));
  p.nblk_w = static_cast<int>(q8_blocks(a.F));
  p.walk.counts = a.counts;
  p.slots = slots;
  p.as = a.xw;
  p.ws = a.w1s;
  p.hq = a.hq;
  p.hs = reinterpret_cast<uint8_t*>(a.hw);
  p.err = a.err;
  p.spin = a.spin;
  p.walk.parts = a.parts1;
  p.part = a.part;
  cudaError_t e = run_q8<true>(a.xq, a.w1q, p, a.num_sms, st);
  if (e != cudaSuccess) return e;
  p.n_out = a.d;
  p.K = a.F;
  p.walk.ntiles_f = (a.d + 255) / 256;
  p.kblk = static_cast<int>(q8_blocks(a.F));
  p.nblk_w = static_cast<int>(q8_blocks(a.d));
  p.walk.parts = a.parts2;
  p.as = a.hw;
  p.ws = a.w2s;
  p.hq = nullptr;
  p.hs = nullptr;
  p.y = static_cast<__nv_bfloat16*>(a.y);
  return run_q8<false>(a.hq, a.w2q, p, a.num_sms, st);
}

}  // namespace smoe
