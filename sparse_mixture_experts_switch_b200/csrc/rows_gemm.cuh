// Products of the expert FFNs with 8-bit checkpoints and of their backward pass:
// over experts' rows (rows_gemm.cu), and of rows' transposes (weight_grad.cu).
#pragma once

#include <algorithm>
#include <cmath>

#include "backward.cuh"
#include "q8.cuh"

namespace smoe {

enum RowsMode : int {
  kRowsHidden = 0, kRowsStore = 1, kRowsMask = 2,
  kRowsHiddenQ8 = 3,         // split_sum.cu: the hidden rows of the 8-bit FFN
};

constexpr float kQ8Least = 0.001953125f;               // 2^-9, the smallest e4m3 value
// Limit of a failed kernel's last wait for copies in flight (about 20 ms; a load
// takes microseconds).
constexpr long long kCopyDrainCycles = 40000000LL;

// After a failure the two CTAs of a pair may have issued different stages, and
// the leader's barriers then do not tell of all of them: the loading warps stay
// for a time in which every copy in flight lands (0.2 ms).
__device__ __forceinline__ void settle_copies(const volatile int* abort_flag) {
  if (*abort_flag == 0) return;
  const long long t0 = clock64();
  while (clock64() - t0 < 400000) {
  }
}

// ok of all 128 threads of named barrier `id`.
__device__ __forceinline__ bool all_of_barrier(bool ok, int id) {
  int r;
  asm volatile(
      "{\n .reg .pred p, r;\n setp.ne.b32 p, %1, 0;\n"
      " barrier.cta.red.and.pred r, %2, 128, p;\n selp.u32 %0, 1, 0, r;\n}\n"
      : "=r"(r)
      : "r"(ok ? 1 : 0), "r"(id)
      : "memory");
  return r != 0;
}

// Long sums with few tiles in parts (split_sum.cu says when and why).
constexpr int kSplitPairs = 74;             // CTA pairs of a B200
constexpr int kPartStages = 6;              // fewest stages of a part
constexpr int64_t kSplitBytes = 24 << 20;   // most scratch
// Parts of sums of `stages` stages: at most `most`, and so many that the stages
// saved are worth the most against `bytes` of scratch a part, if they are worth it.
inline int parts_of(int64_t stages, int64_t most, double bytes) {
  most = std::min(most, stages / kPartStages);
  if (most < 2) return 1;
  constexpr double kStageUs = 0.28, kBytesPerUs = 2e6, kLaunchUs = 3;
  const double best = std::sqrt(kStageUs * kBytesPerUs * static_cast<double>(stages) / bytes);
  const int64_t s = best < 2 ? 2 : (best < static_cast<double>(most) ? static_cast<int64_t>(best) : most);
  const double sd = static_cast<double>(s);
  const double gain = kStageUs * static_cast<double>(stages) * (1 - 1 / sd) - sd * bytes / kBytesPerUs;
  return gain > kLaunchUs ? static_cast<int>(s) : 1;
}
// A product over experts' rows: n_out results of the kept rows (A at most), `stages`
// stages of 128 bf16 or 256 codes each; scratch of at most `room` bytes.
inline int sum_parts(int64_t N, int64_t C, int64_t A, int64_t n_out, int64_t stages, size_t room) {
  if (A <= 0 || C <= 0) return 1;
  const int64_t tiles = std::min(std::min(N, A) + A / 256, N * ((C + 255) / 256)) *
                        ((n_out + 255) / 256);
  const int64_t most = static_cast<int64_t>(std::min<size_t>(room, kSplitBytes));
  return parts_of(stages, std::min(kSplitPairs / tiles, most / (4 * N * C * n_out)),
                  4.0 * static_cast<double>(std::min(A, N * C)) * static_cast<double>(n_out));
}
// Most parts of the weight gradients' sums over an expert's rows (by an even share of
// the batch's A assignments; sums of more rows take no more parts), and those of an
// expert with `stages` stages (64 rows each).
inline int grad_parts(int64_t N, int64_t C, int64_t A, int64_t d, int64_t F, size_t room) {
  const int64_t tiles = 2 * N * ((d + 255) / 256) * ((F + 255) / 256);
  if (tiles > kSplitPairs) return 1;
  const int64_t most = static_cast<int64_t>(std::min<size_t>(room, kSplitBytes));
  return parts_of((std::min(C, A / N) + 63) / 64, std::min(kSplitPairs / tiles, most / (8 * N * d * F)),
                  8.0 * static_cast<double>(N * d * F));
}
__host__ __device__ inline int grad_tile_parts(int stages, int most) {
  const int s = stages / kPartStages;
  return s < 1 ? 1 : (s < most ? s : most);
}

struct JoinArgs {
  int parts, N, n_out;
  int64_t C;
  const int* counts;
  const float* part;         // [parts][N*C][n_out]
  void* out;                 // [N*C, n_out] bf16
  uint8_t *hq, *hs;          // hidden: the rows in 8 bits
  const uint32_t* mask;
  int num_sms;
};
cudaError_t launch_rows_join(int mode, const JoinArgs& a, cudaStream_t st);

struct RowsGemmArgs {
  int N, n_out, K;
  int64_t C;
  const int* counts;
  const void* rows;          // [N*C, K] bf16
  const void* w;             // bf16: [N, n_out, K], or [N, K, n_out] (da, dx)
  void* out;                 // [N*C, n_out] bf16, kept rows only
  uint8_t *hq, *hs;          // hidden: the rows in 8 bits too
  const uint32_t* mask;      // da: bits [N*C, n_out / 32]
  int parts;                 // of the sum (sum_parts; split_sum.cu)
  float* part;               // scratch [parts][N*C][n_out] for more than one
  DevErr* err;
  long long spin;
  int num_sms;
};
cudaError_t launch_rows_hidden(const RowsGemmArgs& a, cudaStream_t st);   // relu(rows w^T)
cudaError_t launch_rows_out(const RowsGemmArgs& a, cudaStream_t st);      // rows w^T
cudaError_t launch_rows_da(const RowsGemmArgs& a, cudaStream_t st);       // (rows w) where mask
cudaError_t launch_rows_dx(const RowsGemmArgs& a, cudaStream_t st);       // rows w

// dw[g][e] [M, Nn] = a[g][e]^T b[g][e] over the kept rows of expert e (zeros
// without any), for two gradients g; a [N*C, M], b [N*C, Nn] bf16, what lies
// behind the kept rows is not used.
struct WeightGradArgs {
  int N;
  int M[2], Nn[2];
  int64_t C;
  const int* counts;
  const void *a[2], *b[2];
  void* dw[2];
  int parts;                 // most parts of a sum (grad_parts)
  float* part;               // scratch [2][parts][N][M][Nn] for more than one
  DevErr* err;
  long long spin;
  int num_sms;
};
cudaError_t launch_weight_grads(const WeightGradArgs& a, cudaStream_t st);
cudaError_t launch_grad_join(const WeightGradArgs& a, cudaStream_t st);

// bf16 [outer][k][m] as MN-major operand tiles (rows_gemm.cu).
bool make_tmap_mn_major(CUtensorMap* map, const void* base, int64_t m, int64_t k, int64_t outer);

}  // namespace smoe
