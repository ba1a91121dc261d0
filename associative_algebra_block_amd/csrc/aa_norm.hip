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
// crosses HBM once.  All sums are float32.  12288 rows of 768 with a residual
// operand (132 MB) take 21 us forward and 29.4 us backward (its kernels traced
// alone 25.5 and 5.2), where a copy of as many bytes takes 27; one row takes 2.8
// us, which a launch costs anyhow.  Times below are of whole calls that follow one
// another, backward ones with both weights' gradients.
#include <hip/hip_runtime.h>

#include <algorithm>

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

// Where a lane's features lie in a row: NC chunks of four, a row's lanes after
// one another, and behind the last whole chunk up to three features, one for
// each of the row's first lanes.
struct Place {
  int lane, lanes;   // of the row
  int whole, d;      // features in whole chunks, all features
  __device__ int col(int c) const { return (c * lanes + lane) * kVec; }
  __device__ bool has(int c) const { return col(c) < whole; }
  __device__ bool has_tail() const { return lane < d - whole; }
};

// A lane's part of a row as it lies in memory: the loads go out together, and
// nothing is converted before all of them are on their way.
template <typename T, int NC>
struct RawRow {
  typename Vec4<T>::type v[NC];
  T tail;
  __device__ void load(const T* row, const Place& at) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      v[c] = typename Vec4<T>::type{T(0.0f), T(0.0f), T(0.0f), T(0.0f)};
      if (at.has(c)) v[c] = *reinterpret_cast<const typename Vec4<T>::type*>(row + at.col(c));
    }
    tail = T(0.0f);
    if (at.has_tail()) tail = row[at.whole + at.lane];
  }
};

// The same in float32; features that the lane does not have are zero.
template <int NC>
struct Row {
  float v[NC][kVec], tail;
  template <typename T>
  __device__ void set(const RawRow<T, NC>& r) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[c][e] = float(r.v[c][e]);
    tail = float(r.tail);
  }
  template <typename T>
  __device__ void load(const T* row, const Place& at) {
    RawRow<T, NC> r;
    r.load(row, at);
    set(r);
  }
  __device__ void fill(float x) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[c][e] = x;
    tail = x;
  }
  template <bool NT = false, typename T>
  __device__ void store(T* row, const Place& at) const {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (at.has(c)) {
        typename Vec4<T>::type t;
#pragma unroll
        for (int e = 0; e < kVec; ++e) t[e] = T(v[c][e]);
        auto* dst = reinterpret_cast<typename Vec4<T>::type*>(row + at.col(c));
        if constexpr (NT) __builtin_nontemporal_store(t, dst);
        else *dst = t;
      }
    if (at.has_tail()) row[at.whole + at.lane] = T(tail);
  }
  template <typename T>
  __device__ void store(T* row, const Place& at, int nt) const {
    if (nt) store<true>(row, at);
    else store(row, at);
  }
  // f(chunk, element) -> void over all of a lane's features; chunk NC is the tail
  template <typename F>
  __device__ static void each(F f) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < kVec; ++e) f(c, e);
    f(NC, 0);
  }
  __device__ float& operator()(int c, int e) { return c < NC ? v[c][e] : tail; }
  __device__ float operator()(int c, int e) const { return c < NC ? v[c][e] : tail; }
};

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
  int32_t nt;          // outputs go past the caches
};

// One row per WPR waves; NC chunks of 64 * WPR * kVec features.
template <typename TX, typename TY, int WPR, int NC>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void norm_fwd_kernel(NormFwdParams p) {
  constexpr int kRowsPerWg = WPR == 1 ? 4 : 1;
  __shared__ float slots[2 * WPR];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);   // uniform: row addresses stay scalar
  const Place at = {int(WPR == 1 ? threadIdx.x & (kWave - 1) : threadIdx.x), 64 * WPR, int(p.d) & ~(kVec - 1),
                    int(p.d)};
  const float d = float(at.d);
  for (int64_t row = int64_t(blockIdx.x) * kRowsPerWg + (WPR == 1 ? wave : 0); row < p.M;
       row += int64_t(gridDim.x) * kRowsPerWg) {
    const int64_t base = row * p.d;
    Row<NC> x;
    if (p.delta) {
      // the norm is that of the stored sum (rounded to x's type): the
      // backward pass reads it from S
      RawRow<TX, NC> rx;
      rx.load(static_cast<const TX*>(p.X) + base, at);
      Row<NC> t;
      if (p.delta_f32) t.load(static_cast<const float*>(p.delta) + base, at);
      else t.load(static_cast<const __bf16*>(p.delta) + base, at);
      x.set(rx);
      Row<NC>::each([&](int c, int e) { x(c, e) = float(TX(x(c, e) + t(c, e))); });
      x.store(static_cast<TX*>(p.S) + base, at, p.nt);
    } else {
      x.load(static_cast<const TX*>(p.X) + base, at);
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) sum += (x.v[c][0] + x.v[c][1]) + (x.v[c][2] + x.v[c][3]);
    const float mean = row_sum<WPR>(sum + x.tail, slots) / d;
    float sq = 0.0f;
    Row<NC>::each([&](int c, int e) {
      const bool mine = c < NC ? at.has(c) : at.has_tail();
      x(c, e) = mine ? x(c, e) - mean : 0.0f;
      sq += x(c, e) * x(c, e);
    });
    const float rstd = 1.0f / sqrtf(row_sum<WPR>(sq, slots + WPR) / d + p.eps);
    Row<NC> g, b;
    g.fill(1.0f);
    b.fill(0.0f);
    if (p.gamma) g.load(p.gamma, at);
    if (p.beta) b.load(p.beta, at);
    Row<NC>::each([&](int c, int e) { x(c, e) = x(c, e) * rstd * g(c, e) + b(c, e); });
    x.store(static_cast<TY*>(p.Y) + base, at, p.nt);
    if (p.mean && at.lane == 0) {
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
  float* sum_xh;       // sums of dy xh and of dy over a workgroup's rows: of workgroup w at 2 d w (nullptr: not wanted)
  float* sum_1;
  int64_t M, d;
  int32_t nt;          // dX goes past the caches
};

// Same split as the forward kernel, with kBwdWaves rows a workgroup at one wave
// a row.  A wave meets the same features in every row, so the weights'
// gradients gather in its registers; the waves of a workgroup add theirs in
// order through LDS and the workgroup writes one partial row, which
// norm_bwd_reduce_kernel sums (of a single workgroup it is the result): no
// atomics, so the result does not depend on the order of execution.
constexpr int kBwdWaves = 4;
template <typename TX, typename TY, int WPR, int NC>
__global__ __launch_bounds__(WPR == 1 ? kBwdWaves * 64 : WPR * 64, WPR == 1 && NC <= 3 ? 4 : 1)
void norm_bwd_kernel(NormBwdParams p) {
  constexpr int kRowsPerWg = WPR == 1 ? kBwdWaves : 1;
  constexpr bool kAhead = WPR > 1 && NC <= 4;   // the next row is on its way while this one is reduced
  __shared__ float slots[2 * WPR];
  extern __shared__ float sums[];   // WPR == 1: [2][d]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);   // uniform: row addresses stay scalar
  const Place at = {int(WPR == 1 ? threadIdx.x & (kWave - 1) : threadIdx.x), 64 * WPR, int(p.d) & ~(kVec - 1),
                    int(p.d)};
  const float d = float(at.d);
  Row<NC> dg, db;
  dg.fill(0.0f);
  db.fill(0.0f);
  const int64_t step = int64_t(gridDim.x) * kRowsPerWg;
  int64_t row = int64_t(blockIdx.x) * kRowsPerWg + (WPR == 1 ? wave : 0);
  RawRow<TX, NC> rx;
  RawRow<TY, NC> ry;
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t r) {
    rx.load(static_cast<const TX*>(p.X) + r * p.d, at);
    ry.load(static_cast<const TY*>(p.dY) + r * p.d, at);
    mean = p.mean[r];
    rstd = p.rstd[r];
  };
  if (kAhead && row < p.M) fetch(row);
  for (; row < p.M; row += step) {
    if (!kAhead) fetch(row);
    RawRow<TX, NC> rs;
    Row<NC> xh, g, gm;
    gm.fill(1.0f);
    if (p.gamma) gm.load(p.gamma, at);
    if (p.dS) rs.load(static_cast<const TX*>(p.dS) + row * p.d, at);   // needed last
    xh.set(rx);
    g.set(ry);
    const float r_mean = mean, r_rstd = rstd;
    if (kAhead && row + step < p.M) fetch(row + step);
    float s1 = 0.0f, s2 = 0.0f;
    Row<NC>::each([&](int c, int e) {
      // features that are not there have dy = 0; xh only has to be finite
      const bool mine = c < NC ? at.has(c) : at.has_tail();
      xh(c, e) = mine ? (xh(c, e) - r_mean) * r_rstd : 0.0f;
      dg(c, e) += g(c, e) * xh(c, e);
      db(c, e) += g(c, e);
      g(c, e) *= gm(c, e);
      s1 += g(c, e);
      s2 += g(c, e) * xh(c, e);
    });
    s1 = row_sum<WPR>(s1, slots) / d;
    s2 = row_sum<WPR>(s2, slots + WPR) / d;
    Row<NC> res;
    res.fill(0.0f);
    if (p.dS) res.set(rs);
    Row<NC>::each([&](int c, int e) { res(c, e) += r_rstd * (g(c, e) - s1 - xh(c, e) * s2); });
    res.store(static_cast<TX*>(p.dX) + row * p.d, at, p.nt);
  }
  if (!p.sum_xh && !p.sum_1) return;
  float* out_xh = p.sum_xh ? p.sum_xh + int64_t(blockIdx.x) * 2 * p.d : nullptr;
  float* out_1 = p.sum_1 ? p.sum_1 + int64_t(blockIdx.x) * 2 * p.d : nullptr;
  if constexpr (WPR == 1) {
    for (int w = 0; w < kBwdWaves; ++w) {
      if (wave == w) {
        Row<NC>::each([&](int c, int e) {
          const bool mine = c < NC ? at.has(c) : at.has_tail();
          const int col = c < NC ? at.col(c) + e : at.whole + at.lane;
          if (mine) {
            sums[col] = (w ? sums[col] : 0.0f) + dg(c, e);
            sums[at.d + col] = (w ? sums[at.d + col] : 0.0f) + db(c, e);
          }
        });
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < at.d; i += blockDim.x) {
      if (out_xh) out_xh[i] = sums[i];
      if (out_1) out_1[i] = sums[at.d + i];
    }
  } else {
    if (out_xh) dg.store(out_xh, at);
    if (out_1) db.store(out_1, at);
  }
}

// dgamma, dbeta = sums of the G partial rows.  A workgroup takes 16 columns, so
// that 768 features give 96 workgroups: its 64 groups of 16 lanes take the rows
// in turn and join in LDS, in a fixed order.
constexpr int kCols = 16, kRowGroups = 1024 / kCols;
__global__ __launch_bounds__(1024) void norm_bwd_reduce_kernel(const float* part, int G, int64_t d, float* dgamma,
                                                               float* dbeta) {
  __shared__ float red[kRowGroups][kCols];
  const int c = threadIdx.x % kCols, group = threadIdx.x / kCols;
  const int64_t col = int64_t(blockIdx.x) * kCols + c;   // of 2 d
  float acc = 0.0f;
  if (col < 2 * d) {
#pragma unroll 8
    for (int g = group; g < G; g += kRowGroups) acc += part[int64_t(g) * 2 * d + col];
  }
  red[group][c] = acc;
  __syncthreads();
  if (threadIdx.x < kWave) {   // four partial columns a lane column
    acc = 0.0f;
#pragma unroll
    for (int g = 0; g < kRowGroups / 4; ++g) acc += red[group * (kRowGroups / 4) + g][c];
    acc += __shfl_xor(acc, kCols, kWave);
    acc += __shfl_xor(acc, 2 * kCols, kWave);
    float* out = col < d ? dgamma : dbeta;
    if (group == 0 && col < 2 * d && out) out[col < d ? col : col - d] = acc;
  }
}

// Rows are dealt to at most 16 workgroups a compute unit.  With half as many,
// which still fill it, the rows of a wave follow one another and the second
// one's loads wait for the first one's stores: 22.2 against 21.1 us for 12288
// rows of 768; with twice as many 21.1.
int64_t fwd_grid(int64_t M, int wpr) {
  const int64_t rows_per_wg = wpr == 1 ? 4 : 1;
  const int64_t wgs = (M + rows_per_wg - 1) / rows_per_wg;
  const int64_t cap = int64_t(device_cu_count()) * 16;
  const int64_t rounds = (wgs + cap - 1) / cap;   // every workgroup the same number of rows
  return (wgs + rounds - 1) / rounds;
}

// Outputs that no L2 can hold until the next kernel reads them (the eight of
// 4 MB together) are stored past the caches: 12288 rows of 768 take 21.0 against
// 27.9 us forward and 29.5 against 32.8 us backward; norm, FFN (Q2 x Q2, 1536
// wide) and norm take 108.0 and 107.4.  Smaller ones are left where the next
// kernel may find them: norm, FFN (q = 16, 768 wide) and norm of 2048 rows of 2048
// take 36.0 us past the caches and 36.5 through them, of 4096 rows 63.6 and 62.9.
constexpr int64_t kL2Bytes = int64_t(32) << 20;
int32_t past_caches(int64_t values, int64_t bytes_each) { return values * bytes_each > kL2Bytes ? 1 : 0; }
int64_t size_of(aa_dtype_t t) { return t == AA_F32 ? 4 : 2; }

// Workgroups of the backward kernel, each of which writes 2 d partial sums.
// One wave a row: 512 (12288 float32 rows of 768 with dS take 34.0, 29.4 and
// 31.3 us with 256, 512 and 1024).  Wider rows: at least eight a workgroup from
// 256 on (1000 rows of 2048 take 14.2 us with 256 and 17.2 with 512, whose sums
// take longer to write and join than the rows), and not so many that the rows in
// flight, 4 MB, outgrow the L2s: 4600 float32 rows of 2048 take 29.8, 23.5 and
// 24.7 us with 256, 512 and 1024; 8000 bf16 rows 48.0, 37.8 and 33.4; 10000 rows
// of 4096 with 256 and 512: 76 and 85 in float32, 76 and 64 in bf16.
int64_t bwd_grid(int64_t M, int64_t d, int64_t size) {
  const bool narrow = d <= 1024;
  const int64_t wgs = narrow ? (M + kBwdWaves - 1) / kBwdWaves : M;
  const int64_t fit = std::min<int64_t>(std::max<int64_t>((int64_t(4) << 20) / (d * size), 256), 1024);
  const int64_t cap = narrow ? 512 : std::min<int64_t>(fit, std::max<int64_t>(M / 8, 256));
  const int64_t rounds = (wgs + cap - 1) / cap;
  return rounds ? (wgs + rounds - 1) / rounds : 0;
}

// Calls CALL(waves per row, chunks) for a row of d features.  Up to 1024 one
// wave a row, no barrier: 12288 float32 rows of 768 take 21.1 us forward and 29.4
// backward, with four waves 23.0 and 33.4 at the best (64 rows: 3.5 and 3.2
// forward).  Beyond, 8 to 32 features a lane (float32 rows forward with a float32
// residual operand):
//   2048 (4608 float32 rows)  4 x 8 features 21.9, 8 x 4 23.5, 1 x 32 21.8 us
//                             forward, which one wave loses with few rows (64:
//                             3.6, 3.5 and 4.6 us)
//   4096 (2048 bf16 rows)     4 x 16 11.2, 8 x 8 12.4 us forward; backward, where
//                             a lane holds three rows, the other way round (2300
//                             float32 rows: 25.6 and 23.1)
//   8192 (1152 float32 rows)  4 x 32 23.2, 8 x 16 22.5 us forward, 40 and 35
//                             backward
//   16384 (576 float32 rows)  8 x 32 26.5, 16 x 16 26.2 us forward, 55 and 123
//                             backward (a wave of 16 has registers for half a row)
#define AA_NORM_SPLIT(d, CALL, SPLIT4096) \
  do {                                    \
    if ((d) <= 256) CALL(1, 1);           \
    else if ((d) <= 512) CALL(1, 2);      \
    else if ((d) <= 768) CALL(1, 3);      \
    else if ((d) <= 1024) CALL(1, 4);     \
    else if ((d) <= 2048) CALL(4, 2);     \
    else if ((d) <= 4096) SPLIT4096;      \
    else if ((d) <= 8192) CALL(8, 4);     \
    else CALL(8, 8);                      \
  } while (0)

template <typename TX, typename TY>
void launch_fwd(const NormFwdParams& p, hipStream_t stream) {
#define AA_CALL(WPR, NC)                                                                            \
  launch((norm_fwd_kernel<TX, TY, WPR, NC>), dim3(uint32_t(fwd_grid(p.M, WPR))), dim3(WPR == 1 ? 256 : WPR * 64), 0u, \
         stream, p)
  AA_NORM_SPLIT(p.d, AA_CALL, AA_CALL(4, 4));
#undef AA_CALL
}

template <typename TX, typename TY>
void launch_bwd(const NormBwdParams& p, hipStream_t stream) {
  const uint32_t grid = uint32_t(bwd_grid(p.M, p.d, sizeof(TX)));
#define AA_CALL(WPR, NC)                                                                              \
  launch((norm_bwd_kernel<TX, TY, WPR, NC>), dim3(grid), dim3(WPR == 1 ? kBwdWaves * 64 : WPR * 64),  \
         uint32_t(WPR == 1 && (p.sum_xh || p.sum_1) ? 8 * p.d : 0), stream, p)
  AA_NORM_SPLIT(p.d, AA_CALL, AA_CALL(8, 2));
#undef AA_CALL
}

}  // namespace

aa_status_t launch_norm_fwd(const NormFwdCall& c, hipStream_t stream) {
  const NormFwdParams p{c.X, c.delta, c.gamma, c.beta, c.S, c.Y, c.mean, c.rstd, c.M, c.d, c.eps,
                        c.delta_dtype == AA_F32 ? 1 : 0,
                        past_caches(c.M * c.d, size_of(c.y_dtype) + (c.S ? size_of(c.x_dtype) : 0))};
  if (c.x_dtype == AA_F32) {
    if (c.y_dtype == AA_F32) launch_fwd<float, float>(p, stream);
    else launch_fwd<float, __bf16>(p, stream);
  } else {
    if (c.y_dtype == AA_F32) launch_fwd<__bf16, float>(p, stream);
    else launch_fwd<__bf16, __bf16>(p, stream);
  }
  return after_launch(stream, "norm_fwd_kernel");
}

// For either type: bf16 rows have the larger grid.
size_t norm_bwd_workspace_bytes(int64_t M, int64_t d) { return size_t(bwd_grid(M, d, 2)) * 2 * size_t(d) * 4; }

aa_status_t launch_norm_bwd(const NormBwdCall& c, hipStream_t stream) {
  const bool sums = c.dgamma || c.dbeta;
  // a single workgroup's sums are the result
  const int64_t grid = bwd_grid(c.M, c.d, size_of(c.x_dtype));
  const bool direct = grid == 1;
  const NormBwdParams p{c.X, c.dY, c.gamma, c.mean, c.rstd, c.dS, c.dX,
                        direct ? c.dgamma : sums ? c.workspace : nullptr,
                        direct ? c.dbeta : sums ? c.workspace + c.d : nullptr, c.M, c.d,
                        past_caches(c.M * c.d, size_of(c.x_dtype))};
  if (c.M > 0) {
    if (c.x_dtype == AA_F32) {
      if (c.dy_dtype == AA_F32) launch_bwd<float, float>(p, stream);
      else launch_bwd<float, __bf16>(p, stream);
    } else {
      if (c.dy_dtype == AA_F32) launch_bwd<__bf16, float>(p, stream);
      else launch_bwd<__bf16, __bf16>(p, stream);
    }
    const aa_status_t st = after_launch(stream, "norm_bwd_kernel");
    if (st != AA_OK || !sums || direct) return st;
  }
  if (!sums) return AA_OK;
  launch(norm_bwd_reduce_kernel, dim3(uint32_t((2 * c.d + kCols - 1) / kCols)), dim3(1024), 0u, stream,
         static_cast<const float*>(c.workspace), int(grid), c.d, c.dgamma, c.dbeta);
  return after_launch(stream, "norm_bwd_reduce_kernel");
}

}  // namespace aa
