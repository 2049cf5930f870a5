// The 8-bit expert FFNs (expert_ffn_q8.cu) for the few tokens of a decoding step.
// Every weight byte is then used for a handful of products, so the two products
// are streams of weights, bound by memory and its latency: no tiles in shared
// memory and no TMEM, but weight rows loaded straight into the registers of
// warp-level MMAs (m16n8k32, e4m3, fp32 sums): 16 features x 8 tokens a warp (an
// expert whose slots the caller gave more rows, tokens named more than once, takes
// them eight at a time).
//
// A lane loads 16 consecutive bytes of a row, so a quad reads 64 and the order of
// the columns inside an MMA differs from memory's: a sum does not mind, as long
// as the tokens' rows are loaded the same way.  Four MMAs make a block of 128
// columns, whose sum is then scaled by 2^(sw + sa) and added in fp32.
//
//   * first product: an item is the 128 features of one scale block, 16 a warp; it
//     reads the tokens' rows through slot_token (no gather) and quantises its
//     hidden block;
//   * second product: an item is 16 features, the columns over 8 warps.  It is
//     launched early (programmatic dependent launch) and has its first weights in
//     flight before it waits for the hidden rows.
// Two CTAs an SM walk over the items of the experts that hold tokens, each with
// the next item's weights in flight while the present one's sums are joined.
//
// Measured, calls back to back: 8 tokens of 8 of 128 experts of 1024 x 4096 (67
// MB of weights, 10.3 us at the copy rate) 24.3 us, one token of one expert (8.4
// MB) 14.4 us: two launches and three dependent loads each before the first MMA.
#include "q8.cuh"

namespace smoe {

namespace {

constexpr int kDepth = 4;                    // column blocks of weights in flight per warp

struct FewParams {
  int N, n_out, K;
  int64_t C, T;
  const int* counts;
  const int* slot_token;     // first product: token of a slot, or null (rows by slot)
  const uint8_t* rows;       // tokens' (or slots') rows [.., K]
  const uint8_t* rs;         // their scales [.., ceil(K / 128)]
  const uint8_t* w;          // [N, n_out, K]
  const uint8_t* wsc;        // [N, ceil(n_out / 128), ceil(K / 128)]
  uint8_t* hq;               // first product: [N*C, n_out]
  uint8_t* hs;               //   [N*C, ceil(n_out / 128)]
  __nv_bfloat16* y;          // second: [N*C, n_out]
  DevErr* err;
};

__device__ __forceinline__ void mma_e4m3(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^(byte - 127) of a scale byte 1 .. 254.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// RG groups of 16 features x S warps over the columns.
template <bool kHidden, int RG, int S>
__global__ void __launch_bounds__(RG * S * 32, 2) few_gemm_kernel(FewParams p) {
  constexpr int kRows = RG * 16;
  __shared__ float red[S][8][kRows + 4];         // [warp over columns][token][feature]
  __shared__ int64_t row_of[8];
  __shared__ int n_hit;
  __shared__ int16_t hit[1024];                  // the experts that hold tokens
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = warp % RG, s = warp / RG;
  const int g = lane >> 2, t = lane & 3;
  if (warp == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.N; e0 += 256) {      // eight loads in flight
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = e0 + 32 * i + lane < p.N ? p.counts[e0 + 32 * i + lane] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t m = __ballot_sync(0xffffffffu, c[i] > 0);
        if (c[i] > 0) hit[n + __popc(m & ((1u << lane) - 1u))] = static_cast<int16_t>(e0 + 32 * i + lane);
        n += __popc(m);
      }
    }
    if (lane == 0) n_hit = n;
  }
  if (kHidden) pdl_launch_dependents();
  __syncthreads();
  const int tiles = (p.n_out + kRows - 1) / kRows;
  const int total = n_hit * tiles;
  const int kb_n = static_cast<int>(q8_blocks(p.K));
  const int64_t nblk = q8_blocks(p.n_out);
  const uint4 zero = make_uint4(0, 0, 0, 0);

  // this lane's two weight rows of an item (rows past the last: any)
  const uint8_t *w0 = nullptr, *w1 = nullptr;
  auto enter = [&](int item) {
    const int e = hit[item / tiles];
    const int fr = (item % tiles) * kRows + rg * 16 + g;
    const uint8_t* base = p.w + static_cast<int64_t>(e) * p.n_out * p.K + t * 16;
    w0 = base + static_cast<int64_t>(fr < p.n_out ? fr : 0) * p.K;
    w1 = base + static_cast<int64_t>(fr + 8 < p.n_out ? fr + 8 : 0) * p.K;
  };
  // weights of column block kb: two rows, two halves of 64 columns
  auto load_w = [&](int kb, uint4* a) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool on = kb * 128 + h * 64 < p.K;
      a[2 * h] = on ? ldg_stream(w0 + kb * 128 + h * 64) : zero;
      a[2 * h + 1] = on ? ldg_stream(w1 + kb * 128 + h * 64) : zero;
    }
  };
  uint4 a[kDepth][4];
  auto load_first = [&]() {
#pragma unroll
    for (int u = 0; u < kDepth; ++u)
      if (s + u * S < kb_n) load_w(s + u * S, a[u]);
  };
  int item = blockIdx.x;
  if (item < total) {
    enter(item);
    load_first();
  }
  if (!kHidden) pdl_wait_prerequisites();         // the hidden rows are there

  while (item < total) {
    const int e = hit[item / tiles];
    const int f0 = (item % tiles) * kRows;
    const int64_t cnt = p.counts[e];
    const int kept = static_cast<int>(cnt < p.C ? cnt : p.C);
    const uint8_t* wsrow = p.wsc + (e * nblk + (f0 >> 7)) * kb_n;
    const int next = item + static_cast<int>(gridDim.x);
    for (int tok0 = 0; tok0 < kept; tok0 += 8) {
      const int nt = kept - tok0 < 8 ? kept - tok0 : 8;
      const int64_t slot0 = static_cast<int64_t>(e) * p.C + tok0;
      if (threadIdx.x < 8) {
        int64_t r = -1;
        if (threadIdx.x < nt) {
          r = slot0 + threadIdx.x;
          if (kHidden && p.slot_token != nullptr) {
            const int64_t tk = p.slot_token[r];
            const bool bad = tk < 0 || tk >= p.T;
            if (bad) report_error(p.err, SWITCH_ERR_DEVICE_BOUNDS, kWhereDispatch, r);
            r = bad ? -1 : tk;
          }
        }
        row_of[threadIdx.x] = r;
      }
      __syncthreads();                            // (also: the last sums have been read)
      const int64_t rb = row_of[g];               // B column g: a token's row
      const uint8_t* xrow = p.rows + (rb < 0 ? 0 : rb) * p.K + t * 16;
      const int64_t r0 = row_of[2 * t], r1 = row_of[2 * t + 1];   // the accumulators' tokens
      const uint8_t* s0 = p.rs + (r0 < 0 ? 0 : r0) * kb_n;
      const uint8_t* s1 = p.rs + (r1 < 0 ? 0 : r1) * kb_n;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int kb = s; kb < kb_n; kb += kDepth * S) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
          const int k = kb + u * S;
          if (k >= kb_n) break;                   // warp-uniform
          uint4 b[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            b[h] = rb >= 0 && k * 128 + h * 64 < p.K
                       ? *reinterpret_cast<const uint4*>(xrow + k * 128 + h * 64)
                       : zero;
          const float sw = scale_of(__ldg(wsrow + k));
          const float sa0 = r0 < 0 ? 1.f : scale_of(s0[k]);     // (no token: a zero row)
          const float sa1 = r1 < 0 ? 1.f : scale_of(s1[k]);
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 x = a[u][2 * h], z = a[u][2 * h + 1];
            mma_e4m3(c, x.x, z.x, x.y, z.y, b[h].x, b[h].y);
            mma_e4m3(c, x.z, z.z, x.w, z.w, b[h].z, b[h].w);
          }
          if (k + kDepth * S < kb_n) load_w(k + kDepth * S, a[u]);
          // the scales' product first: a power of two, where a block's sum (2^-18 to
          // 2^25 in size) times one scale alone may leave fp32's range
          const float f0 = sw * sa0, f1 = sw * sa1;
          sum[0] = fmaf(c[0], f0, sum[0]);
          sum[1] = fmaf(c[1], f1, sum[1]);
          sum[2] = fmaf(c[2], f0, sum[2]);
          sum[3] = fmaf(c[3], f1, sum[3]);
        }
      }
      // the next weights on their way before the sums meet: this expert's again
      // for more tokens (from L2 now), or the next item's
      if (tok0 + 8 < kept) {
        load_first();
      } else if (next < total) {
        enter(next);
        load_first();
      }
      const int f = rg * 16 + g;
      red[s][2 * t][f] = sum[0];
      red[s][2 * t + 1][f] = sum[1];
      red[s][2 * t][f + 8] = sum[2];
      red[s][2 * t + 1][f + 8] = sum[3];
      __syncthreads();
      if (kHidden) {
        // a warp per token: ReLU, the block's scale, 4 codes a lane
        for (int tok = warp; tok < nt; tok += RG * S) {
          const int fo = f0 + 4 * lane;
          const bool on = fo < p.n_out;           // n_out is a multiple of 64
          float v[4], m = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = 0.f;
#pragma unroll
            for (int j = 0; j < S; ++j) x += red[j][tok][4 * lane + i];
            v[i] = on && !(x <= 0.f) ? x : 0.f;  // ReLU; NaN stays NaN
            m = fmaxf(m, v[i]);                  // (and does not count)
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int ex = q8_exponent(m);
          const float is = q8_inv_scale(ex);
          if (on)
            *reinterpret_cast<uint32_t*>(p.hq + (slot0 + tok) * p.n_out + fo) =
                pack_e4m3x4(v[0] * is, v[1] * is, v[2] * is, v[3] * is);
          if (lane == 0)
            p.hs[(slot0 + tok) * nblk + (f0 >> 7)] = static_cast<uint8_t>(q8_scale_byte(ex));
        }
      } else {
        for (int i = threadIdx.x; i < nt * kRows / 2; i += RG * S * 32) {
          const int tok = i / (kRows / 2), fo = (i % (kRows / 2)) * 2;
          float x = 0.f, y = 0.f;
#pragma unroll
          for (int j = 0; j < S; ++j) {
            x += red[j][tok][fo];
            y += red[j][tok][fo + 1];
          }
          if (f0 + fo < p.n_out)
            *reinterpret_cast<uint32_t*>(p.y + (slot0 + tok) * p.n_out + f0 + fo) = pack_bf16x2(x, y);
        }
      }
    }
    item = next;
  }
}

}  // namespace

cudaError_t launch_expert_ffn_q8_few(const FfnQ8Args& a, cudaStream_t st) {
  // at most min(rows, N) experts hold tokens; two CTAs an SM
  const int64_t experts = a.A < a.N ? a.A : a.N;
  auto grid = [&](int tiles) {
    const int64_t items = experts * tiles, most = 2 * a.num_sms;
    return static_cast<unsigned>(items < most ? items : most);
  };
  FewParams p{};
  p.N = a.N;
  p.n_out = a.F;
  p.K = a.d;
  p.C = a.C;
  p.T = a.T;
  p.counts = a.counts;
  p.slot_token = a.slot_token;
  p.rows = a.xq;
  p.rs = a.xs;
  p.w = a.w1q;
  p.wsc = a.w1s;
  p.hq = a.hq;
  p.hs = reinterpret_cast<uint8_t*>(a.hw);
  p.err = a.err;
  few_gemm_kernel<true, 8, 1><<<grid((a.F + 127) / 128), 256, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  FewParams p2 = p;
  p2.n_out = a.d;
  p2.K = a.F;
  p2.slot_token = nullptr;
  p2.rows = a.hq;
  p2.rs = p.hs;
  p2.w = a.w2q;
  p2.wsc = a.w2s;
  p2.y = static_cast<__nv_bfloat16*>(a.y);
  return launch_dependent(few_gemm_kernel<false, 1, 8>, static_cast<int>(grid((a.d + 15) / 16)), 256,
                          0, st, p2);
}

}  // namespace smoe
