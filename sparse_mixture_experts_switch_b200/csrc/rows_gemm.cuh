// Products of the expert FFNs with 8-bit checkpoints and of their backward pass:
// over experts' rows (rows_gemm.cu), and of rows' transposes (weight_grad.cu).
#pragma once

#include "backward.cuh"
#include "q8.cuh"

namespace smoe {

enum RowsMode : int { kRowsHidden = 0, kRowsStore = 1, kRowsMask = 2 };

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

struct RowsGemmArgs {
  int N, n_out, K;
  int64_t C;
  const int* counts;
  const void* rows;          // [N*C, K] bf16
  const void* w;             // bf16: [N, n_out, K], or [N, K, n_out] (da, dx)
  void* out;                 // [N*C, n_out] bf16, kept rows only
  uint8_t *hq, *hs;          // hidden: the rows in 8 bits too
  const uint32_t* mask;      // da: bits [N*C, n_out / 32]
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
  DevErr* err;
  long long spin;
  int num_sms;
};
cudaError_t launch_weight_grads(const WeightGradArgs& a, cudaStream_t st);

// bf16 [outer][k][m] as MN-major operand tiles (rows_gemm.cu).
bool make_tmap_mn_major(CUtensorMap* map, const void* base, int64_t m, int64_t k, int64_t outer);

}  // namespace smoe
