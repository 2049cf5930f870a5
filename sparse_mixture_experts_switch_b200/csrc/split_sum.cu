// Long sums in parts.  A product with few tiles (one feature tile of a few experts'
// tokens, say, with thousands of columns to sum) would keep a few CTA pairs busy
// for the whole sum.  Its tiles then become several items each, one per part of
// the sum (whole stages; expert_ffn_q8.cu, rows_gemm.cu, weight_grad.cu), which
// leave fp32 sums in scratch, and a second launch adds a value's parts, always in
// their order, and does what the product's drain otherwise does.  No pair waits for
// another, and no sum depends on who finishes first.
//
// When (parts_of in rows_gemm.cuh): every item has a CTA pair of its own (by the
// most tiles that the sizes allow), a part has six stages at least, and what is
// saved, 0.28 us for each stage that a pair no longer takes, is more than the second
// launch (3 us with its margin) and the way of the sums through L2 (2 MB a us, there
// and back).  Measured, whole calls, in parts against without: 8-bit FFN of 718 tokens,
// one expert of 64 x 9472, 31.1 and 39.2 us; backward of 146 tokens, two experts of 960
// x 7744, 64 and 82; of 30000 tokens, one expert of 256 x 256, 78 and 179; but of 512
// tokens, one expert of 1024 x 4096 (10 MB of sums for 32 stages), 47.6 and 45.0, and
// of 3000, two experts of 256 x 1024, 38.4 and 33.6: those stay whole.  Of 260 drawn
// sizes (1 to 32768 tokens, widths from 64) 27 have a sum in parts: against the same
// sums whole 20 of them gain 5 to 37%, none loses.  Where the workspace has no room
// for all parts, there are as many as it holds, or the sum stays whole.
#include "rows_gemm.cuh"

namespace smoe {

namespace {

constexpr int kJoinThreads = 256;

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ uint32_t relu_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.relu.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// What a ReLU leaves orders as its bits; NaN does not count.
__device__ __forceinline__ int relu_bits(float v) { return max(__float_as_int(fmaxf(v, 0.f)), 0); }

// Kept rows, a warp for each 128 columns of one, four a lane.
template <int kMode>
__global__ void __launch_bounds__(kJoinThreads) rows_join_kernel(JoinArgs p) {
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int nblk = static_cast<int>(q8_blocks(p.n_out));
  const int64_t slots = p.N * p.C;
  const int64_t stride = slots * p.n_out;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kJoinThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
       i < slots * nblk; i += step) {
    const int64_t r = i / nblk;
    const int b = static_cast<int>(i - r * nblk);
    const int64_t e = r / p.C;
    if (r - e * p.C >= p.counts[e]) continue;
    const int col = b * 128 + lane * 4;
    const bool on = col < p.n_out;                     // (n_out is a multiple of 64)
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      const float* src = p.part + r * p.n_out + col;
      s = __ldcg(reinterpret_cast<const float4*>(src));
#pragma unroll 4
      for (int k = 1; k < p.parts; ++k)
        s = add4(s, __ldcg(reinterpret_cast<const float4*>(src + k * stride)));
    }
    uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + r * p.n_out + col);
    if (kMode == kRowsStore) {
      if (on) *out = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    } else if (kMode == kRowsMask) {
      if (!on) continue;
      const uint32_t w = p.mask[r * (p.n_out >> 5) + (col >> 5)] >> (col & 31);
      *out = make_uint2(pack_bf16x2(w & 1u ? s.x : 0.f, w & 2u ? s.y : 0.f),
                        pack_bf16x2(w & 4u ? s.z : 0.f, w & 8u ? s.w : 0.f));
    } else {
      int most;
      if (kMode == kRowsHidden) {
        const uint2 h = make_uint2(relu_pack(s.x, s.y), relu_pack(s.z, s.w));
        if (on) *out = h;
        s = make_float4(bf16_lo(h.x), bf16_hi(h.x), bf16_lo(h.y), bf16_hi(h.y));
      }
      most = max(max(relu_bits(s.x), relu_bits(s.y)), max(relu_bits(s.z), relu_bits(s.w)));
      const int ex = q8_exponent(__int_as_float(__reduce_max_sync(0xffffffffu, most)));
      if (!on) continue;
      const float is = q8_inv_scale(ex);
      float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float least = kMode == kRowsHidden && f[j] > 0.f ? kQ8Least : 0.f;
        // ReLU; for a checkpoint what is above zero stays above zero.  NaN stays NaN.
        f[j] = f[j] != f[j] ? f[j] : fmaxf(f[j] * is, least);
      }
      *reinterpret_cast<uint32_t*>(p.hq + r * p.n_out + col) = pack_e4m3x4(f[0], f[1], f[2], f[3]);
      if (lane == 0) {
        if (kMode == kRowsHidden) p.hs[r * nblk + b] = static_cast<uint8_t>(q8_scale_byte(ex));
        else p.hs[((b >> 2) * slots + r) * 4 + (b & 3)] = static_cast<uint8_t>(q8_scale_byte(ex));
      }
    }
  }
}

// A thread per eight values of either gradient.
__global__ void __launch_bounds__(kJoinThreads) grad_join_kernel(WeightGradArgs p) {
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int64_t per = static_cast<int64_t>(p.M[0]) * p.Nn[0];        // of an expert; both alike
  const int64_t all = p.N * per;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kJoinThreads * 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x) * 8; i < 2 * all;
       i += step) {
    const int g = i < all ? 0 : 1;
    const int64_t at = g ? i - all : i;
    const int64_t c = p.counts[at / per];
    const int kept = static_cast<int>(c < 0 ? 0 : (c < p.C ? c : p.C));
    const int parts = grad_tile_parts((kept + 63) / 64, p.parts);
    const float4* src = reinterpret_cast<const float4*>(p.part + g * p.parts * all + at);
    float4 a = __ldcg(src), b = __ldcg(src + 1);
#pragma unroll 4
    for (int k = 1; k < parts; ++k) {
      a = add4(a, __ldcg(src + k * (all / 4)));
      b = add4(b, __ldcg(src + k * (all / 4) + 1));
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g ? p.dw[1] : p.dw[0]) + at) =
        make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                   pack_bf16x2(b.z, b.w));
  }
}

int join_grid(int64_t blocks, int num_sms) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, num_sms * 8)));
}

}  // namespace

cudaError_t launch_rows_join(int mode, const JoinArgs& a, cudaStream_t st) {
  const int grid = join_grid((a.N * a.C * q8_blocks(a.n_out) + 7) / 8, a.num_sms);
  switch (mode) {
    case kRowsHidden:
      return launch_dependent(rows_join_kernel<kRowsHidden>, grid, kJoinThreads, 0, st, a);
    case kRowsMask:
      return launch_dependent(rows_join_kernel<kRowsMask>, grid, kJoinThreads, 0, st, a);
    case kRowsHiddenQ8:
      return launch_dependent(rows_join_kernel<kRowsHiddenQ8>, grid, kJoinThreads, 0, st, a);
    default:
      return launch_dependent(rows_join_kernel<kRowsStore>, grid, kJoinThreads, 0, st, a);
  }
}

cudaError_t launch_grad_join(const WeightGradArgs& a, cudaStream_t st) {
  const int64_t all = 2 * static_cast<int64_t>(a.N) * a.M[0] * a.Nn[0];
  return launch_dependent(grad_join_kernel, join_grid((all / 8 + kJoinThreads - 1) / kJoinThreads,
                                                      a.num_sms),
                          kJoinThreads, 0, st, a);
}

}  // namespace smoe
