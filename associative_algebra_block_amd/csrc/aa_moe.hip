// A mixture-of-experts layer for a few tokens, whose experts are row-typed
// SwiGLU FFNs.
//
//   r = x Wr^T (one logit an expert);  the top_k largest are chosen, ties to
//   the lower index;  w = softmax of r over all experts, or over the chosen;
//   y = sum over the chosen e of w_e ((silu(x * Wg_e) (x * Wu_e)) * Wd_e)
//
// where * is the row-typed product of the token's type: under Q_q a token
// touches 2 q - 1 of an expert's q^2 blocks of each matrix.  What bounds the
// call is reading those blocks (9.1 MB for one token of the 2048 -> 768
// experts at q = 16 with 8 chosen) at a latency that few tokens do not hide,
// so every kernel spreads its loads over as many waves as there are 16-column
// strips and issues them before the first use.
//
// Three launches: the logits; gate and up of every (token, expert) pair; the
// down projection with the weighted sum.  The choice itself is no launch: each
// workgroup of the second ranks the logits of its token (E^2 comparisons in
// parallel) for the one expert it needs.  The logits are float64: products of
// bf16 values are exact and their sum all but exact, so the order of summation
// never decides between two experts.  The hidden activation stays float32.
#include <hip/hip_runtime.h>

#include "aa_device.h"
#include "aa_internal.h"

namespace aa {
namespace {

constexpr int kPerThread = kMoeMaxExperts / 256;   // experts that one thread of a workgroup ranks

struct MoeParams {
  const __bf16* X;       // [M][D]
  const __bf16* Wr;      // [E][D]
  const __bf16* Wg;      // [E] packed D x F
  const __bf16* Wu;
  const __bf16* Wd;      // [E] packed F x D
  void* Y;               // [M][D]
  int32_t* experts;      // [M][top_k], or nullptr
  float* weights;
  double* logits;        // workspace: [M][E]
  float* h;              // [M][top_k][F]
  int32_t* chosen;       // [M][top_k]
  float* share;          // [M][top_k]
  const int32_t* types;  // or nullptr: by position
  int64_t M, D, F, off, period;
  int32_t E, top_k, q, law, normalize, y_f32;
};

// The row type of token t; rows of a type outside [0, q) are left alone.
__device__ inline int row_type(const MoeParams& p, int64_t t) {
  if (p.types) return p.types[t];
  int64_t pos = p.off + t;
  if (p.period) pos %= p.period;
  return int(pos % p.q);
}

__device__ inline float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ inline float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// One wave per (token, expert); four waves a workgroup.
__global__ __launch_bounds__(256) void moe_router_kernel(MoeParams p) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = blockIdx.y;
  if (e >= p.E) return;
  const __bf16* x = p.X + t * p.D;
  const __bf16* w = p.Wr + e * p.D;
  double acc = 0.0;
#pragma unroll 4
  for (int64_t c = lane * 8; c < p.D; c += 512) {
    const u32x4_t a = *reinterpret_cast<const u32x4_t*>(x + c);
    const u32x4_t b = *reinterpret_cast<const u32x4_t*>(w + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // a product of two bf16 is exact in float32
      acc += double(lo_f(a[j]) * lo_f(b[j]));
      acc += double(hi_f(a[j]) * hi_f(b[j]));
    }
  }
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) acc += __shfl_xor(acc, s, 64);
  if (lane == 0) p.logits[t * p.E + e] = acc;
}

// a comes before b in the choice (NaN first, so that it is not lost).
__device__ inline bool before(double a, int ia, double b, int ib) {
  const bool na = a != a, nb = b != b;
  if (na || nb) return na && (!nb || ia < ib);
  return a > b || (a == b && ia < ib);
}

// acc[m] += this lane's part of x_g . (columns of a strip) over the input
// groups of one leaf, for NM matrices of one layout.  A lane holds run `lane`
// of every 32-row slab: 8 rows of one column.  off: element offset of the
// expert; x: the token's row.
template <int NM, typename TX>
__device__ inline void strip_dot(const __bf16* const* W, int64_t off, const TX* x, const int* groups, int n_groups,
                                 int k, int q, int bi, int64_t block, int strip, int lane, float* acc) {
  constexpr int U = 8;   // steps whose loads are in flight together
  const int slabs = (bi + 31) / 32;
  const int steps = n_groups * slabs;
  const int64_t in_strip = int64_t(strip) * bi * 16;
  for (int s0 = 0; s0 < steps; s0 += U) {
    u32x4_t w[U][NM];
    float xv[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u;
#pragma unroll
      for (int m = 0; m < NM; ++m) w[u][m] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) xv[u][e] = 0.0f;
      if (s < steps) {
        const int gi = s / slabs, slab = s - gi * slabs;
        const int grp = groups[gi];
        // the last slab of an odd multiple of 16 rows has half the runs
        if (slab * 32 + (lane >> 4) * 8 < bi) {
          const int64_t at = off + (int64_t(grp) * q + k) * block + in_strip + slab * 512 + lane * 8;
#pragma unroll
          for (int m = 0; m < NM; ++m) w[u][m] = *reinterpret_cast<const u32x4_t*>(W[m] + at);
          const TX* src = x + int64_t(grp) * bi + slab * 32 + (lane >> 4) * 8;
          if constexpr (sizeof(TX) == 2) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(src);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              xv[u][2 * j] = lo_f(v[j]);
              xv[u][2 * j + 1] = hi_f(v[j]);
            }
          } else {
            const f32x4_t a = reinterpret_cast<const f32x4_t*>(src)[0], b = reinterpret_cast<const f32x4_t*>(src)[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              xv[u][j] = a[j];
              xv[u][4 + j] = b[j];
            }
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[m] = fmaf(lo_f(w[u][m][j]), xv[u][2 * j], acc[m]);
          acc[m] = fmaf(hi_f(w[u][m][j]), xv[u][2 * j + 1], acc[m]);
        }
  }
}

__device__ inline float quad_sum(float v) {   // over the four lanes of a column
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Gate, up and SiLU: one wave per 16 hidden columns of one (token, rank).
__global__ __launch_bounds__(256) void moe_up_kernel(MoeParams p) {
  extern __shared__ double s_logit[];   // [E]
  __shared__ int s_expert, s_first;
  __shared__ float s_red[4];
  const int64_t pair = blockIdx.y;
  const int64_t t = pair / p.top_k;
  const int rank = int(pair - t * p.top_k);
  const int tau = row_type(p, t);
  if (tau < 0 || tau >= p.q) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < p.E; e += 256) s_logit[e] = p.logits[t * p.E + e];
  __syncthreads();
  int place[kPerThread];   // this thread's experts' places in the choice
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int e = threadIdx.x + 256 * i;
    place[i] = p.E;
    if (e >= p.E) continue;
    const double v = s_logit[e];
    int r = 0;
    for (int o = 0; o < p.E; ++o) r += before(s_logit[o], o, v, e) ? 1 : 0;
    place[i] = r;
    if (r == rank) s_expert = e;
    if (r == 0) s_first = e;
  }
  __syncthreads();
  const int expert = s_expert;
  if (blockIdx.x == 0) {   // this pair's weight, for the next kernel and the caller
    const double top = s_logit[s_first];
    float mine[kPerThread], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int e = threadIdx.x + 256 * i;
      mine[i] = e < p.E ? expf(float(s_logit[e] - top)) : 0.0f;
      if (!p.normalize || place[i] < p.top_k) sum += mine[i];
    }
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s, 64);
    if (lane == 0) s_red[wave] = sum;
    __syncthreads();
    sum = (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (place[i] == rank) {
        const float w = mine[i] / sum;
        p.chosen[pair] = expert;
        p.share[pair] = w;
        if (p.experts) p.experts[pair] = expert;
        if (p.weights) p.weights[pair] = w;
      }
  }
  const int bi = int(p.D / p.q), bo = int(p.F / p.q);
  const int strips = bo / 16;
  const int s = blockIdx.x * 4 + wave;   // strip of the whole hidden row
  if (s >= p.q * strips) return;
  const int k = s / strips, strip = s - k * strips;
  int groups[4];
  const int ng = device_leaf_groups(p.law, tau, k, groups);
  const __bf16* W[2] = {p.Wg, p.Wu};
  float acc[2] = {0.0f, 0.0f};
  strip_dot<2>(W, int64_t(expert) * p.D * p.F, p.X + t * p.D, groups, ng, k, p.q, bi, int64_t(bi) * bo, strip, lane,
               acc);
  const float g = quad_sum(acc[0]), u = quad_sum(acc[1]);
  if (lane < 16) p.h[pair * p.F + int64_t(k) * bo + strip * 16 + lane] = g / (1.0f + expf(-g)) * u;
}

// Down projection and weighted sum: a workgroup per 16 output columns of a
// token; its waves take the chosen experts in turn and join in a fixed order.
__global__ __launch_bounds__(256) void moe_down_kernel(MoeParams p) {
  __shared__ float s_part[4][16];
  const int64_t t = blockIdx.y;
  const int tau = row_type(p, t);
  if (tau < 0 || tau >= p.q) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bi = int(p.F / p.q), bo = int(p.D / p.q);
  const int strips = bo / 16;
  const int k = blockIdx.x / strips, strip = blockIdx.x - k * strips;
  int groups[4];
  const int ng = device_leaf_groups(p.law, tau, k, groups);
  const __bf16* W[1] = {p.Wd};
  float y = 0.0f;
  for (int a = wave; a < p.top_k; a += 4) {
    const int64_t pair = t * p.top_k + a;
    float acc[1] = {0.0f};
    strip_dot<1>(W, int64_t(p.chosen[pair]) * p.D * p.F, p.h + pair * p.F, groups, ng, k, p.q, bi,
                 int64_t(bi) * bo, strip, lane, acc);
    y = fmaf(p.share[pair], acc[0], y);
  }
  y = quad_sum(y);
  if (lane < 16) s_part[wave][lane] = y;
  __syncthreads();
  if (threadIdx.x < 16) {
    const int c = threadIdx.x;
    y = (s_part[0][c] + s_part[1][c]) + (s_part[2][c] + s_part[3][c]);
    const int64_t at = t * p.D + int64_t(k) * bo + strip * 16 + c;
    if (p.y_f32) static_cast<float*>(p.Y)[at] = y;
    else static_cast<__bf16*>(p.Y)[at] = (__bf16)y;
  }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

struct MoeSpace {
  size_t logits, h, chosen, share, bytes;
};
MoeSpace space(const aa_plan_s& up, int E, int top_k, int64_t M) {
  MoeSpace s;
  const size_t pairs = size_t(M) * size_t(top_k);
  s.logits = 0;
  s.h = up256(size_t(M) * size_t(E) * 8);
  s.chosen = s.h + up256(pairs * size_t(up.d_out) * 4);
  s.share = s.chosen + up256(pairs * 4);
  s.bytes = s.share + up256(pairs * 4);
  return s;
}

}  // namespace

size_t moe_workspace_bytes(const aa_plan_s& up, int n_experts, int top_k, int64_t M) {
  return M < 1 ? 0 : space(up, n_experts, top_k, M).bytes;
}

aa_status_t launch_moe(const aa_plan_s& up, const aa_plan_s& down, const MoeCall& c, hipStream_t stream) {
  const MoeSpace sp = space(up, c.n_experts, c.top_k, c.M);
  char* ws = static_cast<char*>(c.workspace);
  MoeParams p{};
  p.X = static_cast<const __bf16*>(c.X);
  p.Wr = static_cast<const __bf16*>(c.Wr);
  p.Wg = static_cast<const __bf16*>(c.Wg);
  p.Wu = static_cast<const __bf16*>(c.Wu);
  p.Wd = static_cast<const __bf16*>(c.Wd);
  p.Y = c.Y;
  p.experts = c.experts;
  p.weights = c.weights;
  p.logits = reinterpret_cast<double*>(ws + sp.logits);
  p.h = reinterpret_cast<float*>(ws + sp.h);
  p.chosen = reinterpret_cast<int32_t*>(ws + sp.chosen);
  p.share = reinterpret_cast<float*>(ws + sp.share);
  p.types = c.row_types;
  p.M = c.M;
  p.D = up.d_in;
  p.F = up.d_out;
  p.period = up.period;
  p.off = c.pos_offset % (up.period ? up.period : up.q);
  p.E = c.n_experts;
  p.top_k = c.top_k;
  p.q = up.q;
  p.law = up.law;
  p.normalize = c.normalize;
  p.y_f32 = down.out_dtype == AA_F32;
  const uint32_t M = uint32_t(c.M), pairs = M * uint32_t(c.top_k);
  launch(moe_router_kernel, dim3((p.E + 3) / 4, M), dim3(256), 0u, stream, p);
  aa_status_t st = after_launch(stream, "moe_router_kernel");
  if (st != AA_OK) return st;
  launch(moe_up_kernel, dim3(uint32_t((p.F / 16 + 3) / 4), pairs), dim3(256), uint32_t(p.E * 8), stream, p);
  st = after_launch(stream, "moe_up_kernel");
  if (st != AA_OK) return st;
  launch(moe_down_kernel, dim3(uint32_t(p.D / 16), M), dim3(256), 0u, stream, p);
  return after_launch(stream, "moe_down_kernel");
}

}  // namespace aa
