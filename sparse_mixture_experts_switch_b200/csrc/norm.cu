// Root-mean-square norm in front of the layer, with the residual's addition
// and an 8-bit output, and its backward pass.
//
//   z = x + residual (rounded once to the rows' type),
//   rstd = 1 / sqrt(mean(z^2) + eps),   y = z rstd gain
//
// y leaves in the rows' type, as e4m3 rows with a power-of-two scale for each
// 128 columns (q8.cuh), or both; backward, with t = dy gain:
//
//   dx = rstd t - z rstd^3 mean(t z) (+ dsum),   dgain = sum over rows of dy z rstd
//
// Both are bound by memory: every row is read once into registers and leaves
// from there.  A row belongs to W warps (1, 2, 4 or 8: the fewest that hold it
// in V 16-byte vectors a lane); the lanes that hold one block of 128 columns
// are 16 neighbours (bf16) or one warp (fp32), so a block's scale takes four or
// five shuffles.  Wider rows are read twice by 256 threads.  Sums are fp32.
//
// Measured on 32768 x 1024 bf16 (calls back to back): forward with residual, both
// outputs and the sum, V = 2 and eight blocks an SM in turn 52.4 us, V = 4 and two
// blocks 53.4, three blocks of 80 registers (spilling) 61 (302 MB: 46.3 at the
// copy rate); backward with its second gradient, V = 4 and two resident blocks an
// SM 55.5 us, four blocks queued 61.8, V = 2 62.2 (268 MB: 41.1).  Short launches wait
// on latency: 5003 x 772 fp32 forward (31 MB: 4.7 us) 10.3 us, as 193 vectors fill 256
// lane slots and each of 1184 blocks, 592 resident, takes two or three pairs of rows
// with a barrier in each; 517 x 4096 fp32 backward (25 MB: 3.9) 12.5 us, as a block loads
// its second row after the first one's barrier, and dgain's reduction follows.  Wide rows,
// bf16: 4096 x 8256 forward 76.8 us (304 MB: 46.6), backward 93.8 (203 MB: 31.1; z and dy
// are read three times), 4096 x 20480 170 and 176 (116, 77).
#include "q8.cuh"

namespace smoe {

namespace {

constexpr int kNormThreads = 256;

template <bool kBf16>
struct Row;
template <>
struct Row<true> {
  static constexpr int kPer = 8;         // values in 16 bytes
  static __device__ __forceinline__ void get(const uint4& u, float* v) {
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Row<false> {
  static constexpr int kPer = 4;
  static __device__ __forceinline__ void get(const uint4& u, float* v) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};

template <int kPer>
__device__ __forceinline__ void load_gain(const float* gain, int col, float* g) {
  if (gain == nullptr) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) g[j] = 1.f;
    return;
  }
#pragma unroll
  for (int j = 0; j < kPer; j += 4) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(gain + col + j));
    g[j] = u.x; g[j + 1] = u.y; g[j + 2] = u.z; g[j + 3] = u.w;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the W warps that share a row.  W > 1: every warp of the block
// calls it the same number of times; `red` holds two sets that alternate
// with `flip`, so one barrier a call is enough (a warp can be at most one
// call ahead of the slowest reader).
template <int W>
__device__ __forceinline__ float row_sum(float v, float (*red)[kNormThreads / 32], int warp,
                                         int& flip) {
  v = warp_sum(v);
  if (W == 1) return v;
  float* r = red[flip];
  flip ^= 1;
  if ((threadIdx.x & 31) == 0) r[warp] = v;
  __syncthreads();
  const int w0 = warp / W * W;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) s += r[w0 + i];
  return s;
}

// One vector of y (fp32) as 8-bit codes and, from the block's first lane, its
// scale byte.  Called by whole warps; `on`: this lane has a vector.
template <bool kBf16>
__device__ __forceinline__ void store_q8(const float* y, bool on, int vec, uint8_t* qrow,
                                         uint8_t* srow) {
  constexpr int kPer = Row<kBf16>::kPer;
  constexpr int kLanes = kQBlock / kPer;            // 16 or 32 lanes hold a block
  float a = 0.f;
  if (on) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) a = fmaxf(a, fabsf(y[j]));
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (!on) return;
  const int e = q8_exponent(a);
  const float is = q8_inv_scale(e);
  if (kPer == 8) {
    reinterpret_cast<uint2*>(qrow)[vec] =
        make_uint2(pack_e4m3x4(y[0] * is, y[1] * is, y[2] * is, y[3] * is),
                   pack_e4m3x4(y[4] * is, y[5] * is, y[6] * is, y[7] * is));
  } else {
    reinterpret_cast<uint32_t*>(qrow)[vec] =
        pack_e4m3x4(y[0] * is, y[1] * is, y[2] * is, y[3] * is);
  }
  if (vec % kLanes == 0) srow[vec / kLanes] = static_cast<uint8_t>(q8_scale_byte(e));
}

// ------------------------------------------------------------------ forward

template <bool kBf16, int W, int V>
__global__ void __launch_bounds__(kNormThreads, 8 / V) residual_norm_kernel(NormArgs a) {
  using R = Row<kBf16>;
  constexpr int kPer = R::kPer;
  constexpr int kRows = kNormThreads / 32 / W;        // rows of a block at a time
  __shared__ float red[2][kNormThreads / 32];
  int flip = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nv = a.d / kPer;
  const int v0 = (warp % W) * 32 + lane;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const int64_t nblk = q8_blocks(a.d);
  // block-uniform trip count (the sums of W > 1 are block barriers)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < a.T;
       r0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t r = r0 + warp / W;
    const bool row_on = r < a.T;
    const int64_t off = r * nv;
    uint4 ux[V], ur[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = v0 + i * 32 * W;
      if (row_on && v < nv) {
        ux[i] = reinterpret_cast<const uint4*>(a.x)[off + v];
        if (a.residual != nullptr) ur[i] = reinterpret_cast<const uint4*>(a.residual)[off + v];
      }
    }
    float z[V][kPer];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = v0 + i * 32 * W;
      if (row_on && v < nv) {
        R::get(ux[i], z[i]);
        if (a.residual != nullptr) {
          float t[kPer];
          R::get(ur[i], t);
#pragma unroll
          for (int j = 0; j < kPer; ++j) z[i][j] += t[j];
          const uint4 uz = R::put(z[i]);
          if (a.z != nullptr) reinterpret_cast<uint4*>(a.z)[off + v] = uz;
          R::get(uz, z[i]);                          // the norm is that of the rounded sum
        } else if (a.z != nullptr) {
          reinterpret_cast<uint4*>(a.z)[off + v] = ux[i];
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) ss = fmaf(z[i][j], z[i][j], ss);
      }
    }
    ss = row_sum<W>(ss, red, warp, flip);
    const float rstd = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
    if (a.rstd != nullptr && row_on && v0 == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = v0 + i * 32 * W;
      const bool on = row_on && v < nv;
      float y[kPer];
      if (on) {
        float g[kPer];
        load_gain<kPer>(a.gain, v * kPer, g);
#pragma unroll
        for (int j = 0; j < kPer; ++j) y[j] = z[i][j] * rstd * g[j];
        if (a.y != nullptr) reinterpret_cast<uint4*>(a.y)[off + v] = R::put(y);
      }
      if (a.yq != nullptr)
        store_q8<kBf16>(y, on, v, a.yq + r * a.d, a.ys + r * nblk);
    }
  }
}

// Rows that four vectors a lane do not hold: one block a row, read twice (a
// thread reads back only vectors that it wrote itself).
template <bool kBf16>
__global__ void __launch_bounds__(kNormThreads) residual_norm_wide_kernel(NormArgs a) {
  using R = Row<kBf16>;
  constexpr int kPer = R::kPer;
  constexpr int W = kNormThreads / 32;
  __shared__ float red[2][W];
  int flip = 0;
  const int warp = threadIdx.x >> 5;
  const int nv = a.d / kPer;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const int64_t nblk = q8_blocks(a.d);
  const int nv_up = (nv + kNormThreads - 1) / kNormThreads * kNormThreads;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x) {
    const int64_t off = r * nv;
    auto sum_of = [&](int v, float* z) {
      const uint4 u = reinterpret_cast<const uint4*>(a.x)[off + v];
      R::get(u, z);
      if (a.residual != nullptr) {
        float t[kPer];
        R::get(reinterpret_cast<const uint4*>(a.residual)[off + v], t);
#pragma unroll
        for (int j = 0; j < kPer; ++j) z[j] += t[j];
        R::get(R::put(z), z);
      }
    };
    float ss = 0.f;
    for (int v = threadIdx.x; v < nv; v += kNormThreads) {
      float z[kPer];
      sum_of(v, z);
      if (a.z != nullptr) reinterpret_cast<uint4*>(a.z)[off + v] = R::put(z);
#pragma unroll
      for (int j = 0; j < kPer; ++j) ss = fmaf(z[j], z[j], ss);
    }
    ss = row_sum<W>(ss, red, warp, flip);
    const float rstd = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[r] = rstd;
    for (int v = threadIdx.x; v < nv_up; v += kNormThreads) {
      const bool on = v < nv;
      float y[kPer];
      if (on) {
        float z[kPer], g[kPer];
        if (a.z != nullptr)
          R::get(reinterpret_cast<const uint4*>(a.z)[off + v], z);
        else
          sum_of(v, z);
        load_gain<kPer>(a.gain, v * kPer, g);
#pragma unroll
        for (int j = 0; j < kPer; ++j) y[j] = z[j] * rstd * g[j];
        if (a.y != nullptr) reinterpret_cast<uint4*>(a.y)[off + v] = R::put(y);
      }
      if (a.yq != nullptr)
        store_q8<kBf16>(y, on, v, a.yq + r * a.d, a.ys + r * nblk);
    }
  }
}

// ----------------------------------------------------------------- backward

// dx of the block's rows, and the block's sum of dy z rstd per column into
// part[blockIdx.x] (every block writes its row of `part`; a block's rows are
// fixed by the launch, so the sums are the same in every run).
template <bool kBf16, int W, int V>
__global__ void __launch_bounds__(kNormThreads, 2) residual_norm_bwd_kernel(NormBwdArgs a) {
  using R = Row<kBf16>;
  constexpr int kPer = R::kPer;
  constexpr int kRows = kNormThreads / 32 / W;
  __shared__ float red[2][kNormThreads / 32];
  __shared__ float dg[kRows > 1 ? W * 32 * V * kPer : 1];
  int flip = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nv = a.d / kPer;
  const int v0 = (warp % W) * 32 + lane;
  const float inv_d = 1.f / static_cast<float>(a.d);
  float acc[V][kPer];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < kPer; ++j) acc[i][j] = 0.f;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < a.T;
       r0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t r = r0 + warp / W;
    const bool row_on = r < a.T;
    const int64_t off = r * nv;
    uint4 uz[V], uy[V], us[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = v0 + i * 32 * W;
      if (row_on && v < nv) {
        uz[i] = reinterpret_cast<const uint4*>(a.z)[off + v];
        uy[i] = reinterpret_cast<const uint4*>(a.dy)[off + v];
        if (a.dsum != nullptr) us[i] = reinterpret_cast<const uint4*>(a.dsum)[off + v];
      }
    }
    const float rstd = row_on ? a.rstd[r] : 0.f;
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = v0 + i * 32 * W;
      if (row_on && v < nv) {
        float z[kPer], y[kPer], g[kPer];
        R::get(uz[i], z);
        R::get(uy[i], y);
        load_gain<kPer>(a.gain, v * kPer, g);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float p = y[j] * z[j];
          c = fmaf(p, g[j], c);
          acc[i][j] = fmaf(p, rstd, acc[i][j]);
        }
      }
    }
    c = row_sum<W>(c, red, warp, flip);
    const float k = c * inv_d * rstd * rstd * rstd;
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = v0 + i * 32 * W;
        if (row_on && v < nv) {
          float z[kPer], y[kPer], g[kPer], o[kPer];
          R::get(uz[i], z);
          R::get(uy[i], y);
          load_gain<kPer>(a.gain, v * kPer, g);
          if (a.dsum != nullptr) {
            R::get(us[i], o);
          } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) o[j] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < kPer; ++j) o[j] += fmaf(y[j] * g[j], rstd, -z[j] * k);
          reinterpret_cast<uint4*>(a.dx)[off + v] = R::put(o);
        }
      }
    }
  }
  if (a.dgain == nullptr) return;
  pdl_launch_dependents();               // the reduction may get into place
  // the block's rows side by side are added in row order through shared memory
  for (int k = 0; k < kRows; ++k) {
    if (warp / W == k) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = v0 + i * 32 * W;
        if (v >= nv) continue;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int col = v * kPer + j;
          if (kRows == 1) {
            a.part[static_cast<int64_t>(blockIdx.x) * a.d + col] = acc[i][j];
          } else if (k == 0) {
            dg[col] = acc[i][j];
          } else {
            dg[col] += acc[i][j];
          }
        }
      }
    }
    if (kRows > 1) __syncthreads();
  }
  if (kRows > 1)
    for (int col = threadIdx.x; col < a.d; col += kNormThreads)
      a.part[static_cast<int64_t>(blockIdx.x) * a.d + col] = dg[col];
}

// Wide rows: dx with one block a row, read twice.
template <bool kBf16>
__global__ void __launch_bounds__(kNormThreads) residual_norm_bwd_wide_kernel(NormBwdArgs a) {
  using R = Row<kBf16>;
  constexpr int kPer = R::kPer;
  constexpr int W = kNormThreads / 32;
  __shared__ float red[2][W];
  int flip = 0;
  const int warp = threadIdx.x >> 5;
  const int nv = a.d / kPer;
  const float inv_d = 1.f / static_cast<float>(a.d);
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x) {
    const int64_t off = r * nv;
    const float rstd = a.rstd[r];
    float c = 0.f;
    for (int v = threadIdx.x; v < nv; v += kNormThreads) {
      float z[kPer], y[kPer], g[kPer];
      R::get(reinterpret_cast<const uint4*>(a.z)[off + v], z);
      R::get(reinterpret_cast<const uint4*>(a.dy)[off + v], y);
      load_gain<kPer>(a.gain, v * kPer, g);
#pragma unroll
      for (int j = 0; j < kPer; ++j) c = fmaf(y[j] * z[j], g[j], c);
    }
    c = row_sum<W>(c, red, warp, flip);
    const float k = c * inv_d * rstd * rstd * rstd;
    for (int v = threadIdx.x; v < nv; v += kNormThreads) {
      float z[kPer], y[kPer], g[kPer], o[kPer];
      R::get(reinterpret_cast<const uint4*>(a.z)[off + v], z);
      R::get(reinterpret_cast<const uint4*>(a.dy)[off + v], y);
      load_gain<kPer>(a.gain, v * kPer, g);
      if (a.dsum != nullptr) {
        R::get(reinterpret_cast<const uint4*>(a.dsum)[off + v], o);
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[j] += fmaf(y[j] * g[j], rstd, -z[j] * k);
      reinterpret_cast<uint4*>(a.dx)[off + v] = R::put(o);
    }
  }
}

// Wide rows: column sums of dy z rstd over the rows blockIdx.y, + gridDim.y, ...; runs
// of 64 rows are summed by themselves and then added (one running sum's error would
// grow with the rows: 170 2^-24 over 1024 equal terms of 0.7, so 12).
template <bool kBf16>
__global__ void __launch_bounds__(kNormThreads) gain_columns_kernel(NormBwdArgs a) {
  using R = Row<kBf16>;
  constexpr int kPer = R::kPer;
  const int nv = a.d / kPer;
  const int v = blockIdx.x * kNormThreads + threadIdx.x;
  if (v >= nv) return;
  float acc[kPer], run[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) acc[j] = run[j] = 0.f;
  int n = 0;
  for (int64_t r = blockIdx.y; r < a.T; r += gridDim.y) {
    float z[kPer], y[kPer];
    R::get(reinterpret_cast<const uint4*>(a.z)[r * nv + v], z);
    R::get(reinterpret_cast<const uint4*>(a.dy)[r * nv + v], y);
    const float rstd = a.rstd[r];
#pragma unroll
    for (int j = 0; j < kPer; ++j) run[j] = fmaf(y[j] * z[j], rstd, run[j]);
    if (++n == 64) {
      n = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        acc[j] += run[j];
        run[j] = 0.f;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    a.part[static_cast<int64_t>(blockIdx.y) * a.d + v * kPer + j] = acc[j] + run[j];
}

// dgain[c] = sum of the nparts rows of `part`: a block takes 32 columns, each of
// its 32 warps every 32nd part (eight loads in flight, added in order), and the
// warps' sums meet in a fixed tree.
__global__ void __launch_bounds__(1024) gain_reduce_kernel(int nparts, int d,
                                                           const float* part, float* dgain) {
  __shared__ float s[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  pdl_wait_prerequisites();
  if (c < d) {
    for (int p0 = warp; p0 < nparts; p0 += 8 * 32) {
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = p0 + 32 * i;
        u[i] = q < nparts ? part[static_cast<int64_t>(q) * d + c] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v += u[i];
    }
  }
  s[warp][lane] = v;
  __syncthreads();
  // a warp a column: its 32 sums in a fixed tree
  const float t = warp_sum(s[lane][warp]);
  if (lane == 0 && blockIdx.x * 32 + warp < d) dgain[blockIdx.x * 32 + warp] = t;
}

// Warps of a row: the fewest whose lanes hold it in `vecs` vectors; 0: none do.
int warps_per_row(int d, bool bf16, int vecs) {
  const int nv = d / (bf16 ? 8 : 4);
  for (int w = 1; w <= kNormThreads / 32; w *= 2)
    if (nv <= 32 * vecs * w) return w;
  return 0;
}

template <bool kBf16>
cudaError_t run_forward(const NormArgs& a, cudaStream_t st) {
  const int w = warps_per_row(a.d, kBf16, 2);
  const int rows = w ? kNormThreads / 32 / w : 1;
  int64_t blocks = (a.T + rows - 1) / rows;
  const int64_t most = static_cast<int64_t>(a.num_sms) * 8;
  if (blocks > most) blocks = most;
  const int g = static_cast<int>(blocks);
  switch (w) {
    case 1: residual_norm_kernel<kBf16, 1, 2><<<g, kNormThreads, 0, st>>>(a); break;
    case 2: residual_norm_kernel<kBf16, 2, 2><<<g, kNormThreads, 0, st>>>(a); break;
    case 4: residual_norm_kernel<kBf16, 4, 2><<<g, kNormThreads, 0, st>>>(a); break;
    case 8: residual_norm_kernel<kBf16, 8, 2><<<g, kNormThreads, 0, st>>>(a); break;
    default:
      if (warps_per_row(a.d, kBf16, 4) == 8)
        residual_norm_kernel<kBf16, 8, 4><<<g, kNormThreads, 0, st>>>(a);
      else
        residual_norm_wide_kernel<kBf16><<<g, kNormThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <bool kBf16>
cudaError_t run_backward(const NormBwdArgs& a, cudaStream_t st) {
  const int w = warps_per_row(a.d, kBf16, 4);
  const int rows = w ? kNormThreads / 32 / w : 1;
  int64_t blocks = (a.T + rows - 1) / rows;
  int64_t most = static_cast<int64_t>(a.num_sms) * 2;      // resident at once
  if (most > kNormParts) most = kNormParts;
  if (blocks > most) blocks = most;
  const int g = static_cast<int>(blocks);
  int nparts = g;
  switch (w) {
    case 1: residual_norm_bwd_kernel<kBf16, 1, 4><<<g, kNormThreads, 0, st>>>(a); break;
    case 2: residual_norm_bwd_kernel<kBf16, 2, 4><<<g, kNormThreads, 0, st>>>(a); break;
    case 4: residual_norm_bwd_kernel<kBf16, 4, 4><<<g, kNormThreads, 0, st>>>(a); break;
    case 8: residual_norm_bwd_kernel<kBf16, 8, 4><<<g, kNormThreads, 0, st>>>(a); break;
    default: {
      // the gain's sums first: dx may be dy's own buffer
      if (a.dgain != nullptr) {
        const int nv = a.d / Row<kBf16>::kPer;
        nparts = static_cast<int>(a.T < 64 ? a.T : 64);
        const dim3 grid(static_cast<unsigned>((nv + kNormThreads - 1) / kNormThreads),
                        static_cast<unsigned>(nparts));
        gain_columns_kernel<kBf16><<<grid, kNormThreads, 0, st>>>(a);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
      }
      if (a.dx != nullptr) {
        int64_t wide = a.T;
        if (wide > static_cast<int64_t>(a.num_sms) * 16) wide = static_cast<int64_t>(a.num_sms) * 16;
        residual_norm_bwd_wide_kernel<kBf16><<<static_cast<int>(wide), kNormThreads, 0, st>>>(a);
      }
    }
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.dgain == nullptr) return e;
  return launch_dependent(gain_reduce_kernel, (a.d + 31) / 32, 1024, 0, st, nparts, a.d, a.part,
                          a.dgain);
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs& a, cudaStream_t st) {
  return a.bf16 ? run_forward<true>(a, st) : run_forward<false>(a, st);
}

cudaError_t launch_residual_norm_backward(const NormBwdArgs& a, cudaStream_t st) {
  return a.bf16 ? run_backward<true>(a, st) : run_backward<false>(a, st);
}

}  // namespace smoe
