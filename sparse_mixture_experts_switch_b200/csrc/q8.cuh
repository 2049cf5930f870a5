// 8-bit block rows: e4m3 values with one power-of-two scale (an e8m0 byte,
// value 2^(byte - 127)) for each 128 consecutive columns of a row, or for
// each 128 x 128 block of a weight matrix.  Device helpers and the launch
// wrappers of the kernels that make, copy and read such rows.
//
// The scale of a block is the smallest power of two s >= 2^-100 with
// max |v| <= 448 s (448 is the largest e4m3 value), so no value saturates;
// a power of two loses none of e4m3's relative precision, makes the values
// q * s exact in bf16 (4 significant bits), and is the form in which the
// tensor core takes block scales.
#pragma once

#include "kernels.cuh"

namespace smoe {

constexpr int kQBlock = 128;           // columns (and weight rows) of one scale
constexpr int kScaleMinExp = -100;     // also the exponent of an all-zero block

__host__ __device__ constexpr int64_t q8_blocks(int64_t cols) {
  return (cols + kQBlock - 1) / kQBlock;
}

// Exponent e of a block's scale 2^e from its largest magnitude: 448 is
// 1.75 x 2^8, so e is amax's own exponent - 8, plus one if amax's significand
// is above 1.75.  (A NaN or infinite amax gives 120 or 121, never an index.)
__device__ __forceinline__ int q8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7FFFFFFFu;
  const int e = static_cast<int>(u >> 23) - 135 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kScaleMinExp ? kScaleMinExp : e;
}
__device__ __forceinline__ uint32_t q8_scale_byte(int e) { return static_cast<uint32_t>(e + 127); }
// 2^-e for -100 <= e <= 121: a normal fp32 number.
__device__ __forceinline__ float q8_inv_scale(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// Four fp32 values to four e4m3 codes (round to nearest, ties to even); `a`
// in the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Two e4m3 codes (the low 16 bits of `q`) times a bf16x2 factor m, where the
// value's scale is m * 2^-120.  The code's exponent and mantissa bits, moved
// to their places in a bf16, stand for the e4m3 value times 2^-120 (bias 127
// against 7; e4m3's subnormals become bf16's), so one exact product with the
// rebias and the scale together gives the value: exact wherever the result is
// a bf16 (4 significant bits).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t q, uint32_t m) {
  const uint32_t w = __byte_perm(q, 0, 0x1404);            // codes in the upper bytes
  const uint32_t v = (w & 0x80008000u) | ((w & 0x7F007F00u) >> 4);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(m));
  return r;
}
// The factor for a scale byte: 2^(byte - 127 + 120).  Bytes 27 .. 134 (scales
// to 2^7, magnitudes to 57344) give a normal bf16; a larger scale needs the
// two-step product below.
__device__ __forceinline__ uint32_t q8_factor(uint32_t byte) {
  const uint32_t h = (byte + 120u) << 7;
  return h | (h << 16);
}
constexpr uint32_t kQ8OneStepMax = 134;

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight codes (two words) of one block to eight bf16.
__device__ __forceinline__ uint4 q8_decode8(uint2 q, uint32_t byte) {
  const bool two = byte > kQ8OneStepMax;
  const uint32_t m = q8_factor(two ? 127u : byte);
  uint4 o = make_uint4(e4m3x2_to_bf16x2(q.x & 0xFFFFu, m), e4m3x2_to_bf16x2(q.x >> 16, m),
                       e4m3x2_to_bf16x2(q.y & 0xFFFFu, m), e4m3x2_to_bf16x2(q.y >> 16, m));
  if (two) {                          // the plain value first, then its scale (a bf16 power of two)
    const uint32_t s = byte << 7;
    const uint32_t ss = s | (s << 16);
    o = make_uint4(mul_bf16x2(o.x, ss), mul_bf16x2(o.y, ss), mul_bf16x2(o.z, ss),
                   mul_bf16x2(o.w, ss));
  }
  return o;
}

// ---------------------------------------------------------------- launches

// Launch as a programmatic dependent of the kernel before it on the stream: it
// may take its place while that one ends, and waits (pdl_wait_prerequisites,
// before anything that depends on earlier kernels of the same call, and before
// leaving) until it and all before it are complete.  Never the first kernel of
// a call: what the caller ran before is then complete.  What an earlier kernel of the
// call wrote is read by plain loads (or TMA), not through the read-only path, whose
// loads the compiler may take to before the wait.
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), int grid, int block, size_t smem,
                                    cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Residual norm (norm.cu).
struct NormArgs {
  int64_t T;
  int d;
  bool bf16;
  const void* x;
  const void* residual;      // or null
  const float* gain;         // or null (ones)
  float eps;
  void* z;                   // or null
  void* y;                   // or null
  uint8_t* yq;               // or null
  uint8_t* ys;               // with yq
  float* rstd;               // or null
  int num_sms;
};
cudaError_t launch_residual_norm(const NormArgs& a, cudaStream_t st);

struct NormBwdArgs {
  int64_t T;
  int d;
  bool bf16;
  const void* z;
  const float* gain;         // or null
  const float* rstd;
  const void* dy;
  const void* dsum;          // or null
  void* dx;                  // or null
  float* dgain;              // or null
  float* part;               // [kNormParts][d] scratch
  int num_sms;
};
constexpr int kNormParts = 296;        // rows of partial gain gradients (2 per SM of a B200)
cudaError_t launch_residual_norm_backward(const NormBwdArgs& a, cudaStream_t st);

// Quantises rows [rows, cols] bf16 (rows_q8.cu).  counts: rows are the slots
// of N experts of C each and only min(counts[e], C) of expert e are made,
// the rest of q and s is not touched; null: every row.  slot_token: row s is
// src[slot_token[s]] (a token outside [0, T) is reported in err) and, with `copy`, is also written there in bf16 (with
// zeros up to the next multiple of 64 rows).  positive: a value above zero
// never rounds to zero.
cudaError_t launch_quantize_rows(int64_t rows, int cols, const void* src, const int* counts,
                                 int64_t C, const int* slot_token, int64_t T, void* copy,
                                 bool positive, uint8_t* q, uint8_t* s, DevErr* err,
                                 cudaStream_t st);
// bf16 rows from one or two sets of 8-bit rows of expert slots (kept rows only).
// pad: also zeros in the rows up to the next multiple of 64 (or C); else, with a
// mask, a bit per value, set where the code is above zero [rows, cols / 32].
struct UnpackSet {
  int cols;
  const uint8_t *q, *s;
  void* out;
  uint32_t* mask;
};
cudaError_t launch_unpack_rows(int64_t rows, const int* counts, int64_t C, bool pad,
                               const UnpackSet* sets, int n, cudaStream_t st);
// 8-bit rows into the slots of their experts (kept slots only; q null: the
// rows are there already, xq and xs are the slots'), their scales as words
// xw [ceil(cols / 512)][slots] (four blocks' bytes, 2^0 past the row's end),
// and the bytes of hw [ceil(hcols / 512)][slots] past hcols' blocks as 2^0.
cudaError_t launch_gather_rows_q8(int64_t slots, int cols, const int* slot_token,
                                  const uint8_t* xq, const uint8_t* xs, const int* counts,
                                  int64_t C, int64_t T, uint8_t* q, uint32_t* xw, int hcols,
                                  uint32_t* hw, DevErr* err, cudaStream_t st);
// Weights [n, rows, cols] bf16 to e4m3 with a scale for each 128 x 128 block.
cudaError_t launch_quantize_weights(int64_t n, int rows, int cols, const void* w, uint8_t* q,
                                    uint8_t* s, cudaStream_t st);

// The experts' FFNs on 8-bit rows and weights (expert_ffn_q8.cu).
struct FfnQ8Args {
  int64_t A, T;              // most kept rows, tokens
  int d, F, N;
  int64_t C;
  const uint8_t* xq;         // [N*C, d]; few: [T, d], or by slots with slot_token null
  const uint32_t* xw;        // scale words of its rows [ceil(d / 512)][N*C]
  const uint8_t* xs;         // few: its scales [.., ceil(d / 128)]
  const int* slot_token;     // few
  const int* counts;
  const uint8_t *w1q, *w1s, *w2q, *w2s;
  uint8_t* hq;               // [N*C, F] scratch
  uint32_t* hw;              // scale words [ceil(F / 512)][N*C] scratch
  void* y;                   // [N*C, d] bf16
  int parts1, parts2;        // of the products' sums (sum_parts)
  float* part;               // scratch for them
  DevErr* err;
  long long spin;
  int num_sms;
};
cudaError_t launch_expert_ffn_q8(const FfnQ8Args& a, cudaStream_t st);
// The same for few rows, by and large kFewTokens assignments (expert_ffn_q8_few.cu):
// reads the tokens' rows through slot_token itself; hw holds row-major scale
// bytes.  Measured against the tensor-core tiles, experts of 1024 x 4096: 8
// assignments of 128 experts 24.3 against 33.6 us, of one expert 14.4 against
// 21.9; 16 of one expert 25.1 against 22.4, 64 of 64 experts 94.7 against 77.6
// (converting the codes for warp-level MMAs then sets the pace).
constexpr int kFewTokens = 8;
cudaError_t launch_expert_ffn_q8_few(const FfnQ8Args& a, cudaStream_t st);

}  // namespace smoe
