// LayerNorm around the row-typed FFN: the forward pass with the residual add
// of the sub-layer before it, and the backward pass with the sums over the
// rows that the affine weights' gradients need.
//
//   forward   s = x + delta (stored, rounded to x's type);  mu = mean(s),
//             r = 1 / sqrt(mean((s - mu)^2) + eps);  y = (s - mu) r gamma + beta
//   backward  xh = (s - mu) r,  g = dy gamma,
//             dx = dS + r (g - mean(g) - xh mean(g xh)),
//             dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Both are bound by HBM: about ten operations an element against 6 to 16
// bytes.  So a row is read once and kept in registers: the mean and the
// variance are two passes over registers (the variance is that of the
// deviations, so a large common offset costs no digits), and every tensor
// crosses HBM once.  All sums are float32.
#include <hip/hip_runtime.h>

#include "aa_device.h"
#include "aa_internal.h"

namespace aa {
namespace {

constexpr int kVec = 4;   // consecutive features of one lane and chunk

// Four features at any element alignment: rows of an odd width start at any
// address, and the memory system takes 8- and 16-byte accesses at every
// alignment, so one path serves all widths.
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x4_u __attribute__((ext_vector_type(4), aligned(2)));

template <typename T> struct Vec4;
template <> struct Vec4<float> { typedef f32x4_u type; };
template <> struct Vec4<__bf16> { typedef bf16x4_u type; };

// v[0..3] = p[0..3], of which only the first n exist (the rest are zero).
template <typename T>
__device__ inline void load_chunk(const T* p, int64_t n, float* v) {
  if (n >= kVec) {
    const typename Vec4<T>::type t = *reinterpret_cast<const typename Vec4<T>::type*>(p);
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = float(t[e]);
  } else {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = e < n ? float(p[e]) : 0.0f;
  }
}

template <typename T>
__device__ inline void store_chunk(T* p, int64_t n, const float* v) {
  if (n >= kVec) {
    typename Vec4<T>::type t;
#pragma unroll
    for (int e = 0; e < kVec; ++e) t[e] = T(v[e]);
    *reinterpret_cast<typename Vec4<T>::type*>(p) = t;
  } else {
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (e < n) p[e] = T(v[e]);
  }
}

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s, kWave);
  return v;
}

// Sum over the WPR waves of a row (all waves of the workgroup when WPR > 1);
// every lane gets it.  Each of a kernel's two call sites has WPR floats of its
// own in `slot`: a site's next write comes behind the other site's barrier,
// which every wave reaches after this site's reads.
template <int WPR>
__device__ inline float row_sum(float v, float* slot) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) slot[wave] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) v += slot[w];
  }
  return v;
}

struct NormFwdParams {
  const void* X;
  const void* delta;   // or nullptr
  const float* gamma;  // or nullptr: ones
  const float* beta;   // or nullptr: zeros
  void* S;             // with delta
  void* Y;
  float* mean;         // or nullptr
  float* rstd;
  int64_t M, d;
  float eps;
  int32_t delta_f32;
};

// One row per WPR waves; NC chunks of 64 * WPR * kVec features.
template <typename TX, typename TY, int WPR, int NC>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void norm_fwd_kernel(NormFwdParams p) {
  constexpr int kRowsPerWg = WPR == 1 ? 4 : 1;
  __shared__ float slots[2 * WPR];
  const int wave = threadIdx.x / kWave;
  const int lane_in_row = WPR == 1 ? threadIdx.x & (kWave - 1) : threadIdx.x;
  const float d = float(p.d);
  for (int64_t row = int64_t(blockIdx.x) * kRowsPerWg + (WPR == 1 ? wave : 0); row < p.M;
       row += int64_t(gridDim.x) * kRowsPerWg) {
    const int64_t base = row * p.d;
    float x[NC][kVec];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = int64_t(c * 64 * WPR + lane_in_row) * kVec;
      load_chunk(static_cast<const TX*>(p.X) + base + col, p.d - col, x[c]);
    }
    if (p.delta) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int64_t col = int64_t(c * 64 * WPR + lane_in_row) * kVec;
        float t[kVec];
        if (p.delta_f32) load_chunk(static_cast<const float*>(p.delta) + base + col, p.d - col, t);
        else load_chunk(static_cast<const __bf16*>(p.delta) + base + col, p.d - col, t);
        // the norm is that of the stored sum (rounded to x's type): the
        // backward pass reads it from S
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[c][e] = float(TX(x[c][e] + t[e]));
        store_chunk(static_cast<TX*>(p.S) + base + col, p.d - col, x[c]);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) sum += (x[c][0] + x[c][1]) + (x[c][2] + x[c][3]);
    const float mean = row_sum<WPR>(sum, slots) / d;
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = int64_t(c * 64 * WPR + lane_in_row) * kVec;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        x[c][e] -= mean;
        sq += col + e < p.d ? x[c][e] * x[c][e] : 0.0f;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<WPR>(sq, slots + WPR) / d + p.eps);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = int64_t(c * 64 * WPR + lane_in_row) * kVec;
      float g[kVec] = {1.0f, 1.0f, 1.0f, 1.0f}, b[kVec] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (p.gamma) load_chunk(p.gamma + col, p.d - col, g);
      if (p.beta) load_chunk(p.beta + col, p.d - col, b);
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[c][e] = x[c][e] * rstd * g[e] + b[e];
      store_chunk(static_cast<TY*>(p.Y) + base + col, p.d - col, x[c]);
    }
    if (p.mean && lane_in_row == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
  }
}

struct NormBwdParams {
  const void* X;
  const void* dY;
  const float* gamma;  // or nullptr
  const float* mean;
  const float* rstd;
  const void* dS;      // or nullptr
  void* dX;
  float* part;         // [gridDim.x][2][d]: sums of dy xh and of dy over the workgroup's rows, or nullptr
  int64_t M, d;
};

// Same split as the forward kernel.  A wave meets the same features in every
// row, so the weights' gradients gather in its registers; the waves of a
// workgroup add theirs in order through LDS and the workgroup writes one
// partial row, which norm_bwd_reduce_kernel sums: no atomics, so the result
// does not depend on the order of execution.
template <typename TX, typename TY, int WPR, int NC>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void norm_bwd_kernel(NormBwdParams p) {
  constexpr int kRowsPerWg = WPR == 1 ? 4 : 1;
  __shared__ float slots[2 * WPR];
  extern __shared__ float sums[];   // WPR == 1: [2][d]
  const int wave = threadIdx.x / kWave;
  const int lane_in_row = WPR == 1 ? threadIdx.x & (kWave - 1) : threadIdx.x;
  const float d = float(p.d);
  float dg[NC][kVec], db[NC][kVec];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < kVec; ++e) dg[c][e] = db[c][e] = 0.0f;
  for (int64_t row = int64_t(blockIdx.x) * kRowsPerWg + (WPR == 1 ? wave : 0); row < p.M;
       row += int64_t(gridDim.x) * kRowsPerWg) {
    const int64_t base = row * p.d;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float xh[NC][kVec], g[NC][kVec];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = int64_t(c * 64 * WPR + lane_in_row) * kVec;
      load_chunk(static_cast<const TX*>(p.X) + base + col, p.d - col, xh[c]);
      load_chunk(static_cast<const TY*>(p.dY) + base + col, p.d - col, g[c]);
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = int64_t(c * 64 * WPR + lane_in_row) * kVec;
      float gm[kVec] = {1.0f, 1.0f, 1.0f, 1.0f};
      if (p.gamma) load_chunk(p.gamma + col, p.d - col, gm);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        // behind the row's end dy is zero, so xh only has to be finite there
        xh[c][e] = col + e < p.d ? (xh[c][e] - mean) * rstd : 0.0f;
        dg[c][e] += g[c][e] * xh[c][e];
        db[c][e] += g[c][e];
        g[c][e] *= gm[e];
        s1 += g[c][e];
        s2 += g[c][e] * xh[c][e];
      }
    }
    s1 = row_sum<WPR>(s1, slots) / d;
    s2 = row_sum<WPR>(s2, slots + WPR) / d;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = int64_t(c * 64 * WPR + lane_in_row) * kVec;
      float r[kVec] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (p.dS) load_chunk(static_cast<const TX*>(p.dS) + base + col, p.d - col, r);
#pragma unroll
      for (int e = 0; e < kVec; ++e) r[e] += rstd * (g[c][e] - s1 - xh[c][e] * s2);
      store_chunk(static_cast<TX*>(p.dX) + base + col, p.d - col, r);
    }
  }
  if (!p.part) return;
  float* out = p.part + int64_t(blockIdx.x) * 2 * p.d;
  if constexpr (WPR == 1) {
    for (int w = 0; w < 4; ++w) {
      if (wave == w) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int64_t col = int64_t(c * 64 + lane_in_row) * kVec;
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            if (col + e >= p.d) break;
            sums[col + e] = (w ? sums[col + e] : 0.0f) + dg[c][e];
            sums[p.d + col + e] = (w ? sums[p.d + col + e] : 0.0f) + db[c][e];
          }
        }
      }
      __syncthreads();
    }
    for (int64_t i = threadIdx.x; i < 2 * p.d; i += blockDim.x) out[i] = sums[i];
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = int64_t(c * 64 * WPR + lane_in_row) * kVec;
      store_chunk(out + col, p.d - col, dg[c]);
      store_chunk(out + p.d + col, p.d - col, db[c]);
    }
  }
}

// dgamma, dbeta = sums of the G partial rows; 64 columns a workgroup, its 16
// waves take the rows in turn and join in LDS, in a fixed order.
__global__ __launch_bounds__(1024) void norm_bwd_reduce_kernel(const float* part, int G, int64_t d, float* dgamma,
                                                               float* dbeta) {
  __shared__ float red[16][kWave];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int64_t col = int64_t(blockIdx.x) * kWave + lane;   // of 2 d
  float acc = 0.0f;
  if (col < 2 * d) {
#pragma unroll 4
    for (int g = wave; g < G; g += 16) acc += part[int64_t(g) * 2 * d + col];
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && col < 2 * d) {
#pragma unroll
    for (int w = 1; w < 16; ++w) acc += red[w][lane];
    float* out = col < d ? dgamma : dbeta;
    if (out) out[col < d ? col : col - d] = acc;
  }
}

// Rows are dealt to at most this many workgroups of 256 threads (or 4 times
// fewer of 1024).
int64_t fwd_grid(int64_t M, int wpr) {
  const int64_t rows_per_wg = wpr == 1 ? 4 : 1;
  const int64_t wgs = (M + rows_per_wg - 1) / rows_per_wg;
  const int64_t cap = int64_t(device_cu_count()) * (wpr == 16 ? 2 : 8);
  if (wgs <= cap) return wgs;
  const int64_t rounds = (wgs + cap - 1) / cap;   // every workgroup the same number of rows
  return (wgs + rounds - 1) / rounds;
}

constexpr int kBwdMaxGrid = 512;
int64_t bwd_grid(int64_t M, int64_t d) {
  const int64_t rows_per_wg = d <= 2048 ? 4 : 1;
  const int64_t wgs = (M + rows_per_wg - 1) / rows_per_wg;
  const int64_t rounds = (wgs + kBwdMaxGrid - 1) / kBwdMaxGrid;
  return rounds ? (wgs + rounds - 1) / rounds : 0;
}

// Calls f with the split of a row of d features: waves per row, chunks.
#define AA_NORM_SPLIT(d, CALL)          \
  do {                                  \
    if ((d) <= 256) CALL(1, 1);         \
    else if ((d) <= 512) CALL(1, 2);    \
    else if ((d) <= 768) CALL(1, 3);    \
    else if ((d) <= 1024) CALL(1, 4);   \
    else if ((d) <= 2048) CALL(1, 8);   \
    else if ((d) <= 4096) CALL(4, 4);   \
    else if ((d) <= 8192) CALL(4, 8);   \
    else CALL(16, 8);                   \
  } while (0)

template <typename TX, typename TY>
void launch_fwd(const NormFwdParams& p, hipStream_t stream) {
#define AA_CALL(WPR, NC)                                                                            \
  launch((norm_fwd_kernel<TX, TY, WPR, NC>), dim3(uint32_t(fwd_grid(p.M, WPR))), dim3(WPR == 1 ? 256 : WPR * 64), 0u, \
         stream, p)
  AA_NORM_SPLIT(p.d, AA_CALL);
#undef AA_CALL
}

template <typename TX, typename TY>
void launch_bwd(const NormBwdParams& p, hipStream_t stream) {
  const uint32_t grid = uint32_t(bwd_grid(p.M, p.d));
#define AA_CALL(WPR, NC)                                                                              \
  launch((norm_bwd_kernel<TX, TY, WPR, NC>), dim3(grid), dim3(WPR == 1 ? 256 : WPR * 64),             \
         uint32_t(WPR == 1 && p.part ? 8 * p.d : 0), stream, p)
  AA_NORM_SPLIT(p.d, AA_CALL);
#undef AA_CALL
}

}  // namespace

aa_status_t launch_norm_fwd(const NormFwdCall& c, hipStream_t stream) {
  const NormFwdParams p{c.X, c.delta, c.gamma, c.beta, c.S, c.Y, c.mean, c.rstd, c.M, c.d, c.eps,
                        c.delta_dtype == AA_F32 ? 1 : 0};
  if (c.x_dtype == AA_F32) {
    if (c.y_dtype == AA_F32) launch_fwd<float, float>(p, stream);
    else launch_fwd<float, __bf16>(p, stream);
  } else {
    if (c.y_dtype == AA_F32) launch_fwd<__bf16, float>(p, stream);
    else launch_fwd<__bf16, __bf16>(p, stream);
  }
  return after_launch(stream, "norm_fwd_kernel");
}

size_t norm_bwd_workspace_bytes(int64_t M, int64_t d) { return size_t(bwd_grid(M, d)) * 2 * size_t(d) * 4; }

aa_status_t launch_norm_bwd(const NormBwdCall& c, hipStream_t stream) {
  const bool sums = c.dgamma || c.dbeta;
  const NormBwdParams p{c.X, c.dY, c.gamma, c.mean, c.rstd, c.dS, c.dX, sums ? c.workspace : nullptr, c.M, c.d};
  if (c.M > 0) {
    if (c.x_dtype == AA_F32) {
      if (c.dy_dtype == AA_F32) launch_bwd<float, float>(p, stream);
      else launch_bwd<float, __bf16>(p, stream);
    } else {
      if (c.dy_dtype == AA_F32) launch_bwd<__bf16, float>(p, stream);
      else launch_bwd<__bf16, __bf16>(p, stream);
    }
    const aa_status_t st = after_launch(stream, "norm_bwd_kernel");
    if (st != AA_OK || !sums) return st;
  }
  if (!sums) return AA_OK;
  launch(norm_bwd_reduce_kernel, dim3(uint32_t((2 * c.d + kWave - 1) / kWave)), dim3(1024), 0u, stream,
         static_cast<const float*>(c.workspace), int(bwd_grid(c.M, c.d)), c.d, c.dgamma, c.dbeta);
  return after_launch(stream, "norm_bwd_reduce_kernel");
}

}  // namespace aa
