// Kernels that make, unpack and move 8-bit block rows (format: q8.cuh).  All
// are one pass over memory: a warp takes a row, 8 bf16 (or 16 codes) a lane,
// and 16 neighbouring lanes hold one block of 128 columns.  Measured alone at 25278
// rows: unpacking 4096 columns with their bits and 1024 columns 62 us (388 MB, 6.2
// TB/s), copying and quantising 1024 columns 23 us (129 MB), moving 1024 codes 14 us
// (52 MB).  Weights, calls back to back: both of 128 experts of 1024 x 4096 625 us (3.2
// GB: 493 at the copy rate), of 16 of 4096 x 10240 790 (4.0 GB: 617).
#include "q8.cuh"

namespace smoe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int64_t kept_of(const int* counts, int64_t C, int64_t e) {
  const int64_t c = counts[e];
  return c < 0 ? 0 : (c < C ? c : C);
}

// The token of kept slot r; one outside [0, T) is reported and gives a row of
// zeros.
__device__ __forceinline__ int64_t slot_row(const int* slot_token, int64_t r, int64_t T,
                                            DevErr* err) {
  const int64_t t = slot_token[r];
  if (t >= 0 && t < T) return t;
  report_error(err, SWITCH_ERR_DEVICE_BOUNDS, kWhereDispatch, r);
  return -1;
}

// One warp per row.
template <bool kPositive>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(
    int64_t rows, int cols, const uint4* __restrict__ src, const int* __restrict__ counts,
    int64_t C, const int* __restrict__ slot_token, int64_t T, uint4* __restrict__ copy,
    uint8_t* __restrict__ q, uint8_t* __restrict__ s, DevErr* err) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nv = cols / 8;
  const int nv_up = (nv + 31) / 32 * 32;
  const int64_t nblk = q8_blocks(cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
       r += step) {
    if (counts != nullptr) {
      const int64_t e = r / C, i = r - e * C;
      const int64_t kept = kept_of(counts, C, e);
      if (i >= kept) {
        if (copy != nullptr && i < (kept + 63) / 64 * 64)
          for (int v = lane; v < nv; v += 32) copy[r * nv + v] = make_uint4(0, 0, 0, 0);
        continue;
      }
    }
    const int64_t t = slot_token != nullptr ? slot_row(slot_token, r, T, err) : r;
    for (int v = lane; v < nv_up; v += 32) {
      const bool on = v < nv;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (on && t >= 0) u = __ldg(src + t * nv + v);
      if (on && copy != nullptr) copy[r * nv + v] = u;
      float f[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                    bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(f[j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      if (!on) continue;
      const int e = q8_exponent(a);
      const float is = q8_inv_scale(e);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool pos = kPositive && f[j] > 0.f;
        f[j] *= is;
        if (pos) f[j] = fmaxf(f[j], 0.001953125f);     // 2^-9, the smallest code above zero
      }
      reinterpret_cast<uint2*>(q + r * cols)[v] =
          make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
      if (v % 16 == 0) s[r * nblk + v / 16] = static_cast<uint8_t>(q8_scale_byte(e));
    }
  }
}

// 0x80 in each byte that holds a code above zero.
__device__ __forceinline__ uint32_t positive_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & ~w & 0x80808080u;
}
// The four flags as bits 0 .. 3.
__device__ __forceinline__ uint32_t flag_bits(uint32_t f) {
  return ((f >> 7) * 0x01020408u) >> 24;
}

// One set of rows per blockIdx.y.  kPad: zero rows up to the next multiple of 64;
// else the kept rows' bits where there is a mask.
template <bool kPad>
__global__ void __launch_bounds__(kThreads) unpack_rows_kernel(int64_t rows,
                                                              const int* __restrict__ counts,
                                                              int64_t C, UnpackSet s0,
                                                              UnpackSet s1) {
  pdl_launch_dependents();
  const UnpackSet u = blockIdx.y == 0 ? s0 : s1;
  const int lane = threadIdx.x & 31;
  const int nv = u.cols / 8;
  const int64_t nblk = q8_blocks(u.cols);
  auto* out = static_cast<uint4*>(u.out);
  auto* mask = reinterpret_cast<uint8_t*>(u.mask);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
       r += step) {
    const int64_t e = r / C, i = r - e * C;
    const int64_t kept = kept_of(counts, C, e);
    if (i >= kept) {
      if (kPad && i < (kept + 63) / 64 * 64)
        for (int v = lane; v < nv; v += 32) out[r * nv + v] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint2* row = reinterpret_cast<const uint2*>(u.q + r * u.cols);
    for (int v = lane; v < nv; v += 32) {
      const uint2 w = __ldg(row + v);
      out[r * nv + v] = q8_decode8(w, __ldg(u.s + r * nblk + v / 16));
      if (!kPad && mask != nullptr)
        mask[r * nv + v] = static_cast<uint8_t>(flag_bits(positive_codes(w.x)) |
                                                flag_bits(positive_codes(w.y)) << 4);
    }
  }
}

__global__ void __launch_bounds__(kThreads) gather_rows_q8_kernel(
    int64_t slots, int cols, const int* __restrict__ slot_token, const uint8_t* __restrict__ xq,
    const uint8_t* __restrict__ xs, const int* __restrict__ counts, int64_t C, int64_t T,
    uint8_t* __restrict__ q, uint32_t* __restrict__ xw, int hcols, uint32_t* __restrict__ hw,
    DevErr* err) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nv = cols / 16;
  const int nblk = static_cast<int>(q8_blocks(cols));
  const int hblk = static_cast<int>(q8_blocks(hcols));
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < slots;
       r += step) {
    const int64_t e = r / C;
    if (r - e * C >= kept_of(counts, C, e)) continue;
    int64_t t = r;
    if (q != nullptr) {
      t = slot_row(slot_token, r, T, err);
      const uint4* row = reinterpret_cast<const uint4*>(xq + t * cols);
      uint4* dst = reinterpret_cast<uint4*>(q + r * cols);
      for (int v = lane; v < nv; v += 32) dst[v] = t >= 0 ? __ldg(row + v) : make_uint4(0, 0, 0, 0);
    }
    for (int g = lane; g * 4 < nblk; g += 32) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = 4 * g + i;
        const uint32_t v = (t >= 0 && b < nblk) ? __ldg(xs + t * nblk + b) : 127u;
        w |= v << (8 * i);
      }
      xw[static_cast<int64_t>(g) * slots + r] = w;
    }
    // the first product's drain writes hw's bytes one by one: the rest of the
    // last word here
    if ((hblk & 3) != 0 && lane == 0) hw[static_cast<int64_t>(hblk >> 2) * slots + r] = 0x7F7F7F7Fu;
  }
}

// One block per 128 x 128 block of a weight matrix: 16 lanes hold a row's 128
// columns, 16 rows at a time, kept in registers between the maximum and the
// conversion.
__global__ void __launch_bounds__(kThreads) quantize_weights_kernel(int rows, int cols,
                                                                   const uint4* __restrict__ w,
                                                                   uint8_t* __restrict__ q,
                                                                   uint8_t* __restrict__ s) {
  __shared__ float red[kWarps];
  const int bc = static_cast<int>(q8_blocks(cols)), br = static_cast<int>(q8_blocks(rows));
  const int64_t b = blockIdx.x;
  const int64_t per = static_cast<int64_t>(bc) * br;
  const int64_t n = b / per;
  const int r0 = static_cast<int>((b % per) / bc) * kQBlock;
  const int c0 = static_cast<int>(b % bc) * kQBlock + static_cast<int>(threadIdx.x & 15) * 8;
  uint4 u[8];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + i * 16 + static_cast<int>(threadIdx.x >> 4);
    u[i] = make_uint4(0, 0, 0, 0);
    if (r < rows && c0 < cols) u[i] = __ldg(w + ((n * rows + r) * cols + c0) / 8);
    const uint32_t p[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) a = fmaxf(a, fmaxf(fabsf(bf16_lo(p[j])), fabsf(bf16_hi(p[j]))));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) a = fmaxf(a, red[i]);
  const int e = q8_exponent(a);
  const float is = q8_inv_scale(e);
  if (threadIdx.x == 0) s[b] = static_cast<uint8_t>(q8_scale_byte(e));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + i * 16 + static_cast<int>(threadIdx.x >> 4);
    if (r < rows && c0 < cols)
      *reinterpret_cast<uint2*>(q + (n * rows + r) * cols + c0) = make_uint2(
          pack_e4m3x4(bf16_lo(u[i].x) * is, bf16_hi(u[i].x) * is, bf16_lo(u[i].y) * is,
                      bf16_hi(u[i].y) * is),
          pack_e4m3x4(bf16_lo(u[i].z) * is, bf16_hi(u[i].z) * is, bf16_lo(u[i].w) * is,
                      bf16_hi(u[i].w) * is));
  }
}

int row_blocks(int64_t rows) {
  const int64_t b = (rows + kWarps - 1) / kWarps;
  return static_cast<int>(b < 148 * 16 ? b : 148 * 16);
}

}  // namespace

cudaError_t launch_quantize_rows(int64_t rows, int cols, const void* src, const int* counts,
                                 int64_t C, const int* slot_token, int64_t T, void* copy,
                                 bool positive, uint8_t* q, uint8_t* s, DevErr* err,
                                 cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const auto* u = static_cast<const uint4*>(src);
  auto* c = static_cast<uint4*>(copy);
  if (positive)
    quantize_rows_kernel<true><<<row_blocks(rows), kThreads, 0, st>>>(rows, cols, u, counts, C,
                                                                      slot_token, T, c, q, s, err);
  else
    quantize_rows_kernel<false><<<row_blocks(rows), kThreads, 0, st>>>(rows, cols, u, counts, C,
                                                                       slot_token, T, c, q, s, err);
  return cudaGetLastError();
}

cudaError_t launch_unpack_rows(int64_t rows, const int* counts, int64_t C, bool pad,
                               const UnpackSet* sets, int n, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(row_blocks(rows)), static_cast<unsigned>(n));
  const UnpackSet& last = sets[n - 1];
  if (pad)
    unpack_rows_kernel<true><<<grid, kThreads, 0, st>>>(rows, counts, C, sets[0], last);
  else
    unpack_rows_kernel<false><<<grid, kThreads, 0, st>>>(rows, counts, C, sets[0], last);
  return cudaGetLastError();
}

cudaError_t launch_gather_rows_q8(int64_t slots, int cols, const int* slot_token,
                                  const uint8_t* xq, const uint8_t* xs, const int* counts,
                                  int64_t C, int64_t T, uint8_t* q, uint32_t* xw, int hcols,
                                  uint32_t* hw, DevErr* err, cudaStream_t st) {
  if (slots == 0) return cudaSuccess;
  gather_rows_q8_kernel<<<row_blocks(slots), kThreads, 0, st>>>(
      slots, cols, slot_token, xq, xs, counts, C, T, q, xw, hcols, hw, err);
  return cudaGetLastError();
}

cudaError_t launch_quantize_weights(int64_t n, int rows, int cols, const void* w, uint8_t* q,
                                    uint8_t* s, cudaStream_t st) {
  const int64_t blocks = n * q8_blocks(rows) * q8_blocks(cols);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  quantize_weights_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(
      rows, cols, static_cast<const uint4*>(w), q, s);
  return cudaGetLastError();
}

}  // namespace smoe
