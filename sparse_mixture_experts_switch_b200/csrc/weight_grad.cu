// Weight gradients of the expert FFNs' backward pass from 8-bit checkpoints:
//
//   dw[e][m, n] = sum over the kept rows r of expert e of a[r, m] b[r, n]
//
// of two such gradients (of both weights) in one launch.
//
// A product with a short sum (an expert's few hundred rows) and a large result:
// bound by writing dw.  One persistent kernel on CTA pairs, 256 x 256 tiles; both
// operands lie with m or n contiguous and are used as they lie (MN-major tiles,
// 64 rows deep, one 4-D box of 64 rows x 2 x 64 columns per operand and CTA).
//   * warps 0 and 2 load A and B through a ring of five stages, warp 1 of the
//     leader issues (warp-uniform loops: expert_ffn_q8.cu says why);
//   * 16 drain warps: 32 result rows x 64 columns each, in bf16 through a
//     128-byte-swizzled box that one TMA store writes (it clips at the edges).
// The last stage of an expert's rows may hold rows of no token, with anything in
// them: such a stage arrives on a barrier of its own CTA, warp 3 zeroes those rows
// of both operands in shared memory, and only then hands the stage to the leader.
//
// Measured alone, 128 experts of 1024 x 4096, 25278 kept rows, both gradients (2.15
// GB written, 0.5 read): 534 us, 565 without the fetch of later tiles into L2; the
// same stores without any rows take 411 us (5.2 TB/s).  Stores by the drain warps'
// own instructions instead of TMA boxes took 550.  Launches of the same build on the
// same buffers' sizes range from 534 to 625 us (26163 rows), so compare medians.
#include <cstring>

#include "rows_gemm.cuh"

namespace smoe {

namespace {

constexpr int kGK = 64;                                // rows of a stage
constexpr int kGStages = 5;
constexpr int kGAhead = 2;                             // tiles of a pair between prefetch and load
constexpr uint32_t kGOpBytes = 128 * kGK * 2;          // 16 KB: 64 rows x 128 columns
constexpr uint32_t kGStageBytes = 2 * kGOpBytes;
constexpr int kGDrainWarps = 16;
constexpr int kGThreads = 128 + 32 * kGDrainWarps;
constexpr uint32_t kGBoxBytes = 32 * 128;              // 32 rows x 64 bf16
constexpr uint32_t kGSmem = 1024 + kGStages * kGStageBytes + kGDrainWarps * kGBoxBytes + 256;
static_assert(kGSmem <= 232448, "a CTA's shared memory");

struct GradMaps {
  CUtensorMap a[2], b[2], out[2];
};
struct GradParams {
  int N;
  int M[2], Nn[2], tm[2], tn[2];   // tm, tn: 256-wide tiles
  int total[2];                    // items of the first gradient, of both
  int parts;                       // items of a tile: most parts of its sum
  float* part;                     // partial sums [2][parts][N][M][Nn]
  int64_t C;
  const int* counts;
  DevErr* err;
  long long spin;
};

struct GradTile {
  int g, e, m0, n0, kept;
  int part, parts;     // of the sum; an item with part >= parts is none
  int kb0, kb1;        // its stages
};

// Item t, part t % parts of tile t / parts.  Tiles: first the tiles of gradient 0, then those of gradient 1; an expert's m
// tiles vary fastest, then its n tiles.
template <bool kParts>
__device__ __forceinline__ GradTile grad_tile(const GradParams& p, int t) {
  GradTile r;
  r.g = t < p.total[0] ? 0 : 1;
  if (r.g) t -= p.total[0];
  r.part = 0;
  if (kParts) {
    const int tile = t / p.parts;
    r.part = t - tile * p.parts;
    t = tile;
  }
  const int tm = r.g ? p.tm[1] : p.tm[0];
  const int per = tm * (r.g ? p.tn[1] : p.tn[0]);
  r.e = t / per;
  const int local = t - r.e * per;
  const int n = local / tm;
  r.n0 = n * 256;
  r.m0 = (local - n * tm) * 256;
  const int64_t c = __ldg(p.counts + r.e);
  r.kept = static_cast<int>(c < 0 ? 0 : (c < p.C ? c : p.C));
  const int kblocks = (r.kept + kGK - 1) / kGK;
  r.parts = kParts ? grad_tile_parts(kblocks, p.parts) : 1;
  r.kb0 = kParts ? r.part * kblocks / r.parts : 0;
  r.kb1 = kParts ? (r.part + 1) * kblocks / r.parts : kblocks;
  return r;
}

template <bool kParts>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
    weight_grad_kernel(const __grid_constant__ GradMaps maps, GradParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* stage_out = smem + kGStages * kGStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(stage_out + kGDrainWarps * kGBoxBytes);
  uint64_t* empty = full + kGStages;        // full: leader; empty: local
  uint64_t* tail = empty + kGStages;        // local: a ragged stage's bytes
  uint64_t* tfull = tail + kGStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(cluster_count_x());
  const long long lim = p.spin;
  const int total = p.total[1];
  pdl_launch_dependents();
  if (cid >= total) {                       // same decision in both CTAs of the pair
    pdl_wait_prerequisites();
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGStages; ++s) {
      mbar_init(&full[s], 2);               // the two loading warps, or the two CTAs' warp 3
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 2);               // the CTA's two loading warps
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kGDrainWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                           // the peer's barriers exist before any remote use
  tc_fence_after();
  pdl_wait_prerequisites();                 // both operands are there
  const uint32_t tmem_base = *tmem_holder;
  const uint32_t full_lead = map_to_rank(smem_u32(full), 0);
  const uint32_t tail_own = map_to_rank(smem_u32(tail), rank);
  const uint32_t tempty_lead = map_to_rank(smem_u32(tempty), 0);

  if (warp == 0 || warp == 2) {
    // ------------------------------------------- TMA: warp 0 A, warp 2 B
    const bool is_b = warp == 2;
    const CUtensorMap* map0 = is_b ? maps.b : maps.a;
    if (elect_one()) tma_prefetch_desc(map0);
    int stage = 0;
    uint32_t phase = 0;
    uint32_t full_mask = 0, tail_mask = 0, full_phase = 0, tail_phase = 0;
    uint32_t tail_now = 0;                  // phase of each tail barrier's next use
    for (int tile = cid; tile < total; tile += ncl) {
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      const GradTile t = grad_tile<kParts>(p, tile);
      if (kParts && t.part >= t.parts) continue;
      const CUtensorMap* map = map0 + t.g;
      const int x = (is_b ? t.n0 : t.m0) + static_cast<int>(rank) * 128;
      bool ok = true;
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, lim))) {
          if (lane == 0) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmProducer, tile);
            *abort_flag = 1;
          }
          ok = false;
          break;
        }
        uint8_t* dst = smem + stage * kGStageBytes + (is_b ? kGOpBytes : 0u);
        const bool ragged = (kb + 1) * kGK > t.kept;
        if (elect_one()) {
          if (ragged) {
            mbar_arrive_expect_tx(&tail[stage], kGOpBytes);
            tma_load_4d_pair(dst, map, tail_own + 8u * stage, 0, kb * kGK, x >> 6, t.e);
          } else {
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kGOpBytes);
            tma_load_4d_pair(dst, map, full_lead + 8u * stage, 0, kb * kGK, x >> 6, t.e);
          }
        }
        if (ragged) {
          tail_mask |= 1u << stage;
          tail_phase = (tail_phase & ~(1u << stage)) | (tail_now & (1u << stage));
          tail_now ^= 1u << stage;
          full_mask &= ~(1u << stage);      // (its last loaded stage has been used up)
        } else {
          full_mask |= 1u << stage;
          full_phase = (full_phase & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == kGStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      // the operands of a later tile into L2: of the tiles that share one, the
      // first asks for it
      const int ahead = tile + kGAhead * ncl;
      if (ahead < total) {
        const GradTile u = grad_tile<kParts>(p, ahead);
        if (u.part < u.parts && (is_b ? u.m0 : u.n0) == 0 && elect_one()) {
          const int xu = ((is_b ? u.n0 : u.m0) + static_cast<int>(rank) * 128) >> 6;
          for (int kb = u.kb0; kb < u.kb1; ++kb)
            tma_prefetch_l2_4d(map0 + u.g, 0, kb * kGK, xu, u.e);
        }
      }
    }
    // Never leave with copies in flight into the pair's shared memory: ragged
    // stages on this CTA's barriers, the others on the leader's.  (After a failure
    // a barrier may miss the other warp's arrival and be waited for by the limit.)
    if (lane == 0) {
      for (int s = 0; s < kGStages; ++s) {
        if (((tail_mask >> s) & 1u) && !mbar_wait(&tail[s], (tail_phase >> s) & 1u, kCopyDrainCycles))
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereDrain, s);
        if (leader && ((full_mask >> s) & 1u) &&
            !mbar_wait_cluster(&full[s], (full_phase >> s) & 1u, kCopyDrainCycles))
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereDrain, s);
      }
    }
    settle_copies(abort_flag);
  } else if (warp == 3) {
    // ----------------------------------------- ragged stages: rows of no token
    int stage = 0;
    uint32_t tail_now = 0;
    for (int tile = cid; tile < total; tile += ncl) {
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      const GradTile t = grad_tile<kParts>(p, tile);
      if (kParts && t.part >= t.parts) continue;
      const int rows = t.kept % kGK;
      if (rows != 0 && t.part == t.parts - 1) {        // the expert's last stage
        const int s = (stage + t.kb1 - t.kb0 - 1) % kGStages;
        if (!__all_sync(0xffffffffu, mbar_wait(&tail[s], (tail_now >> s) & 1u, lim))) {
          if (lane == 0) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmProducer, tile);
            *abort_flag = 1;
          }
          break;
        }
        tail_now ^= 1u << s;
        // four boxes of 64 rows x 128 bytes: rows on from `rows` to zero
        const uint32_t at = smem_u32(smem + s * kGStageBytes);
        const int n = (kGK - rows) * 8;              // 16-byte pieces of a box
        for (int i = lane; i < n; i += 32) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            st_shared_v4u(at + b * 8192u + static_cast<uint32_t>(rows * 128 + i * 16), 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&full[s]);
          else mbar_arrive_remote(full_lead + 8u * s);
        }
      }
      stage = (stage + t.kb1 - t.kb0) % kGStages;
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer (leader)
    if (leader) {
      constexpr uint32_t idesc = idesc_bf16_f32_major(256, 256, true, true);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool any = false;
      const uint32_t smem0 = smem_u32(smem);
      for (int tile = cid; tile < total; tile += ncl) {
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        const GradTile t = grad_tile<kParts>(p, tile);
        if (kParts && t.part >= t.parts) continue;
        bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, lim));
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
        for (int kb = t.kb0; ok && kb < t.kb1; ++kb) {
          ok = __all_sync(0xffffffffu, (kb + 1) * kGK > t.kept
                                           ? mbar_wait_cluster(&full[stage], phase, lim)
                                           : mbar_wait(&full[stage], phase, lim));
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = smem0 + stage * kGStageBytes;
          const uint64_t ad = sw128_mnmajor_desc(at, 8192u);
          const uint64_t bd = sw128_mnmajor_desc(at + kGOpBytes, 8192u);
          if (elect_one()) {
            // a 16-deep step: 16 rows of 128 bytes, in descriptor units of 16 bytes
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_pair(d_tmem, ad + 128 * k, bd + 128 * k, idesc,
                             kb != t.kb0 || k != 0 ? 1u : 0u);
            umma_commit_pair(&empty[stage], 0x3);
          }
          any = true;
          if (++stage == kGStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) {
          if (lane == 0) {
            report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmMma, tile);
            *abort_flag = 1;
          }
          break;
        }
        if (elect_one()) umma_commit_pair(&tfull[acc], 0x3);   // also without rows (zeros written)
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
  } else {
    // --------------------------------------------------------- drain warps
    const int q = warp & 3;                 // TMEM lane quarter: 32 result rows
    const int cg = (warp - 4) >> 2;         // 64 of the tile's columns
    const uint32_t box = smem_u32(stage_out + (warp - 4) * kGBoxBytes);
    const uint32_t swz = static_cast<uint32_t>(lane & 7);
    if (lane == 0) tma_prefetch_desc(&maps.out[0]);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = cid; tile < total; tile += ncl) {
      const GradTile t = grad_tile<kParts>(p, tile);
      if (kParts && t.part >= t.parts) continue;
      const bool ok = __all_sync(0xffffffffu, mbar_wait_sleepy(&tfull[acc], acc_phase, lim));
      if (!ok) {
        if (lane == 0) {
          report_error(p.err, SWITCH_ERR_TIMEOUT, kWhereGemmEpilogue, tile);
          *abort_flag = 1;
        }
        break;
      }
      tc_fence_after();
      const int m = t.m0 + static_cast<int>(rank) * 128 + q * 32;
      const int n = t.n0 + cg * 64;
      const bool on = m < p.M[t.g] && n < p.Nn[t.g];   // warp-uniform: the box begins inside dw
      if (kParts) {
        // the part's sums in fp32: 32 columns at a time through the box, four rows
        // of 128 bytes a store; grad_join finishes them
        const int64_t nn = p.Nn[t.g];
        float* dst = p.part +
                     ((static_cast<int64_t>(t.g * p.parts + t.part) * p.N + t.e) * p.M[t.g] + m) * nn + n;
#pragma unroll
        for (int b = 0; b < 64; b += 32) {
          uint32_t v[32];
          if (on && t.kb1 > t.kb0) {
            tmem_ld32_issue(tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>(acc * 256 + cg * 64 + b), v);
            tmem_ld_wait(v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          if (!on) continue;
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4u(box + lane * 128 + ((static_cast<uint32_t>(k) ^ swz) << 4), v[4 * k],
                          v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = 4 * k + (lane >> 3);
            *reinterpret_cast<float4*>(dst + row * nn + b + 4 * (lane & 7)) =
                ld_shared_v4(box + row * 128 + ((lane ^ row) & 7) * 16);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive_relaxed(&tempty[acc]);
          else mbar_arrive_remote_relaxed(tempty_lead + 8u * acc);
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
        continue;
      }
      uint32_t pk[32];
      if (on) {
        if (t.kb1 > t.kb0) {
          uint32_t v[32], u[32];
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                 static_cast<uint32_t>(acc * 256 + cg * 64);
          tmem_ld32_issue(taddr, v);
          tmem_ld32_issue(taddr + 32, u);
          tmem_ld_wait(v);
          tmem_ld_wait(u);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            pk[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            pk[16 + i] = pack_bf16x2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) pk[i] = 0u;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive_relaxed(&tempty[acc]);
        else mbar_arrive_remote_relaxed(tempty_lead + 8u * acc);
      }
      if (on) {
        if (lane == 0) bulk_wait_read<0>();          // the last box has left the buffer
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          st_shared_v4u(box + lane * 128 + ((static_cast<uint32_t>(k) ^ swz) << 4), pk[4 * k],
                        pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&maps.out[t.g], box, n, m, t.e);
          bulk_commit();
        }
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) bulk_wait_all();         // boxes stored from shared memory are written
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                           // no CTA leaves while its peer may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

template <bool kParts>
cudaError_t run_grads(const GradMaps& maps, const GradParams& p, int num_sms, cudaStream_t st) {
  static size_t smem_set[64] = {};
  const cudaError_t e = ensure_smem_limit(
      reinterpret_cast<const void*>(&weight_grad_kernel<kParts>), kGSmem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_dependent(weight_grad_kernel<kParts>, (num_sms / 2) * 2, kGThreads, kGSmem, st, maps,
                          p);
}

}  // namespace

cudaError_t launch_weight_grads(const WeightGradArgs& a, cudaStream_t st) {
  GradMaps maps;
  GradParams p{};
  p.N = a.N;
  p.C = a.C;
  p.counts = a.counts;
  p.err = a.err;
  p.spin = a.spin;
  p.parts = a.parts;
  p.part = a.part;
  int64_t total = 0;
  for (int g = 0; g < 2; ++g) {
    bool ok = make_tmap_mn_major(&maps.a[g], a.a[g], a.M[g], a.C, a.N);
    ok = ok && make_tmap_mn_major(&maps.b[g], a.b[g], a.Nn[g], a.C, a.N);
    ok = ok && make_tmap_bf16_3d(&maps.out[g], a.dw[g], a.Nn[g], a.M[g], a.N, 64, 32);
    if (!ok) return cudaErrorInvalidValue;
    p.M[g] = a.M[g];
    p.Nn[g] = a.Nn[g];
    p.tm[g] = (a.M[g] + 255) / 256;
    p.tn[g] = (a.Nn[g] + 255) / 256;
    total += static_cast<int64_t>(a.N) * p.tm[g] * p.tn[g] * a.parts;
    if (total > INT32_MAX) return cudaErrorInvalidValue;
    p.total[g] = static_cast<int>(total);
  }
  if (a.parts == 1) return run_grads<false>(maps, p, a.num_sms, st);
  const cudaError_t e = run_grads<true>(maps, p, a.num_sms, st);
  return e != cudaSuccess ? e : launch_grad_join(a, st);
}

}  // namespace smoe
