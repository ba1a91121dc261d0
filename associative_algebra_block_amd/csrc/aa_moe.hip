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
// strips and issues them before the first use.  One token takes 3.0 + 5.8 + 4.0
// us (logits, gate and up, down), each within a few us of an empty launch;
// sixteen, 120 MB, 4.6 + 17.8 + 11.6 us: 4 TB/s over the last two, where a plain
// read of as much reaches 6.8.  The choice in front of gate and up's loads, the
// tails and the down projection's half slabs (every second step of its 48-row
// blocks fetches 512 bytes instead of 1024) take the rest.
//
// Three launches: the logits; gate and up of every (token, expert) pair; the
// down projection with the weighted sum.  The choice itself is no launch: each
// workgroup of the second ranks the logits of its token (E^2 comparisons in
// parallel) for the one expert it needs.  The logits are float64: products of
// bf16 values are exact and their sum all but exact, so the order of summation
// never decides between two experts.  The hidden activation stays float32.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "aa_device.h"
#include "aa_internal.h"
#include "aa_rules.h"

namespace aa {
namespace {

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
  int64_t D, F;
  int32_t E, top_k, q, law, normalize, y_f32;
  int32_t off;           // position of token 0, modulo q
  uint32_t parts, pairs; // workgroups of a pair, (token, expert) pairs: the second kernel
};

// The row type of token t; rows of a type outside [0, q) are left alone.  A
// period is a multiple of q, so it does not change the type of a position.
__device__ inline int row_type(const MoeParams& p, int t) {
  return p.types ? p.types[t] : int(uint32_t(p.off + t) % uint32_t(p.q));
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
    for (int j = 0; j < 4; ++j) {   // float64 holds every product of two bf16, float32 not the largest and smallest
      acc = fma(double(lo_f(a[j])), double(lo_f(b[j])), acc);
      acc = fma(double(hi_f(a[j])), double(hi_f(b[j])), acc);
    }
  }
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) acc += __shfl_xor(acc, s, 64);
  if (lane == 0) p.logits[t * p.E + e] = acc;
}

// The order of the choice as that of unsigned integers: larger logits have
// larger keys, -0 and 0 the same one, NaN (which must not get lost) the largest.
__device__ inline uint64_t choice_key(double v) {
  const uint64_t b = uint64_t(__double_as_longlong(v + 0.0));
  if (v != v) return ~uint64_t(0);
  return b >> 63 ? ~b : b | uint64_t(1) << 63;
}

// The input groups of a leaf, two to a register: an array that a loop's counter
// indexes would be kept in memory.
struct Groups {
  uint64_t lo, hi;
  int n;
};
__device__ inline Groups leaf_groups_of(int law, int i, int k) {
  int g[4] = {0, 0, 0, 0};
  Groups r;
  r.n = device_leaf_groups(law, i, k, g);
  r.lo = uint32_t(g[0]) | uint64_t(uint32_t(g[1])) << 32;
  r.hi = uint32_t(g[2]) | uint64_t(uint32_t(g[3])) << 32;
  return r;
}

// acc[m] += the steps begin .. end - 1 of the sum of one strip of 16 columns of
// output group k, for NM matrices of one layout.  The steps run over the chosen
// experts (a: its element offset expert_at(a), its factor share(a), activations
// at x + a * x_stride), the leaf's input groups and the 32-row slabs of a
// group's block; a lane holds run `lane` of a slab, 8 rows of one column.
//
// Lane i works out where step i lies, once for 64 steps, and the wave reads it
// back a step at a time: done by the scalar unit the addresses took longer than
// the loads.  U steps' loads go out without a branch or a use between them (8,
// or 4 with two matrices: at 8 those take 115 registers and fewer waves fit,
// 36.1 against 33.3 us for a call of 16 tokens); a step behind the end loads the last
// one's data again and is left out of the sum, as are the lanes behind the half
// slab that ends a block of an odd multiple of 16 rows.
template <int NM, typename TX, typename FAt, typename FShare>
__device__ inline void strip_dot(const __bf16* const* W, FAt expert_at, const TX* x, int x_stride, FShare share,
                                 Groups groups, int k, int q, int bi, int64_t block, int strip, int lane, int begin,
                                 int end, float* acc) {
  constexpr int U = NM == 2 ? 4 : 8;
  constexpr int kXRegs = sizeof(TX) / 2;   // 16-byte pieces of 8 activations
  const int slabs = (bi + 31) / 32, per_expert = groups.n * slabs;
  const int row = (lane >> 4) * 8;
  for (int s0 = begin; s0 < end; s0 += 64) {
    const int s = min(s0 + lane, end - 1);
    const int a = s / per_expert, in_expert = s - a * per_expert;
    const int g = in_expert / slabs, slab = in_expert - g * slabs;
    const int grp = int((g & 2 ? groups.hi : groups.lo) >> (32 * (g & 1)));
    const int64_t at = expert_at(a) + (int64_t(grp) * q + k) * block + int64_t(strip) * bi * 16 + slab * 512;
    const int at_lo = int(at), at_hi = int(at >> 32);
    const int x_at = a * x_stride + grp * bi + slab * 32;
    const int full = slab * 32 + 32 <= bi;
    const int sh = __float_as_int(share(a));
    const int n = min(end - s0, 64);
    for (int u0 = 0; u0 < n; u0 += U) {
      u32x4_t w[U][NM], xv[U][kXRegs];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t w_at = int64_t(uint64_t(uint32_t(__builtin_amdgcn_readlane(at_lo, u0 + u))) |
                                     uint64_t(uint32_t(__builtin_amdgcn_readlane(at_hi, u0 + u))) << 32);
        const bool whole = __builtin_amdgcn_readlane(full, u0 + u) != 0;
#pragma unroll
        for (int m = 0; m < NM; ++m)
          w[u][m] = *reinterpret_cast<const u32x4_t*>(W[m] + w_at + (whole ? lane : lane & 31) * 8);
        const TX* src = x + __builtin_amdgcn_readlane(x_at, u0 + u) + (whole ? row : row & 15);
#pragma unroll
        for (int i = 0; i < kXRegs; ++i) xv[u][i] = reinterpret_cast<const u32x4_t*>(src)[i];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u0 + u >= n) break;
        const bool ok = lane < 32 || __builtin_amdgcn_readlane(full, u0 + u) != 0;
        const float factor = __int_as_float(__builtin_amdgcn_readlane(sh, u0 + u));
        float xf[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (kXRegs == 1) {
            xf[2 * j] = lo_f(xv[u][0][j]);
            xf[2 * j + 1] = hi_f(xv[u][0][j]);
          } else {
            xf[j] = __uint_as_float(xv[u][0][j]);
            xf[4 + j] = __uint_as_float(xv[u][1][j]);
          }
        }
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          float part = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            part = fmaf(lo_f(w[u][m][j]), xf[2 * j], part);
            part = fmaf(hi_f(w[u][m][j]), xf[2 * j + 1], part);
          }
          acc[m] += ok ? part * factor : 0.0f;
        }
      }
    }
  }
}

__device__ inline float quad_sum(float v) {   // over the four lanes of a column
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// How many experts come before expert e in the choice, where `per` neighbouring
// lanes share an expert and take the others in turn, four at a time; keys in LDS,
// zeros behind the last.  By the keys' upper halves alone (exact == false)
// experts that agree in them get the same place, which the caller sees: two such
// logits differ by less than 2^-20 of themselves.
constexpr int kUpWaves = kMoeUpWaves, kUpThreads = 64 * kUpWaves;
static_assert(kUpThreads >= kMoeMaxExperts, "a thread for every expert");
template <bool exact>
__device__ inline int place_of(const uint64_t* keys, const uint32_t* upper, int E, int e, int per) {
  const int part = threadIdx.x & (per - 1);
  const uint64_t mine = keys[e];
  const uint32_t mine_upper = uint32_t(mine >> 32);
  int r = 0;
#pragma unroll 4
  for (int o = 4 * part; o < E; o += 4 * per) {
    if constexpr (exact) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r += keys[o + j] > mine || (keys[o + j] == mine && o + j < e) ? 1 : 0;
    } else {
      const u32x4_t u = *reinterpret_cast<const u32x4_t*>(upper + o);
#pragma unroll
      for (int j = 0; j < 4; ++j) r += u[j] > mine_upper ? 1 : 0;
    }
  }
  for (int s = 1; s < per; s *= 2) r += __shfl_xor(r, s, 64);
  return r;
}

// Gate, up and SiLU of one (token, rank): WS waves per 16 hidden columns, which
// share the sum's parts and join in LDS.
template <int WS>
__global__ __launch_bounds__(kUpThreads) void moe_up_kernel(MoeParams p) {
  __shared__ uint64_t s_key[kMoeMaxExperts];
  __shared__ __align__(16) uint32_t s_upper[kMoeMaxExperts];
  __shared__ int s_place[kMoeMaxExperts];
  __shared__ int s_expert, s_hits[3];
  __shared__ uint64_t s_top;
  __shared__ float s_red[kUpWaves], s_part[kUpWaves][2][16];
  // Workgroup `part` of a pair.  Consecutive workgroups go to the eight dies in
  // turn: where a pair has a multiple of eight, those of a strip lie on one die,
  // and pairs that share an expert meet there.  Where it has not, a row of the
  // grid is eight pairs, and each die takes all workgroups of an eighth of the
  // parts (q = 2, 2048 -> 768, 16 tokens: 55 against 61 us; 640 -> 1440, 7 tokens,
  // 42 pairs: 35 against 37; with 16 parts, where both do it, 82 against 78).
  uint32_t part = blockIdx.x, pair = blockIdx.y;
  if (gridDim.x != p.parts) {
    const uint32_t place = blockIdx.x % 8 * p.parts + blockIdx.x / 8;
    part = place / 8;
    pair = blockIdx.y * 8 + place % 8;
    if (pair >= p.pairs) return;
  }
  const int64_t t = pair / uint32_t(p.top_k);
  const int rank = int(pair) - int(t) * p.top_k;
  const int tau = row_type(p, int(t));
  if (tau < 0 || tau >= p.q) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // This workgroup ranks all experts for itself.  The comparisons of upper
  // halves are a fifth of the exact ones' work (which took 7 of 30 us with 16
  // tokens and 128 experts) and nearly always decide; where the first place,
  // this workgroup's or the border of the choice is shared, all are compared.
  // The ranking takes 2 us of a call; where every wave searched the keys for its
  // expert bit by bit, one token took 1.2 us longer.
  {
    const int e = threadIdx.x;
    const uint64_t key = e < p.E ? choice_key(p.logits[t * p.E + e]) : 0;
    s_key[e] = key;
    s_upper[e] = uint32_t(key >> 32);
    if (e < 3) s_hits[e] = 0;
  }
  __syncthreads();
  const int per = p.E <= 64 ? 8 : p.E <= 128 ? 4 : p.E <= 256 ? 2 : 1;
  const int e = threadIdx.x / uint32_t(per);
  const bool first = (threadIdx.x & (per - 1)) == 0 && e < p.E;
  auto settle = [&](int place) {   // the experts at this workgroup's place and at the first
    if (first) s_place[e] = place;
    if (first && place == 0) s_top = s_key[e], atomicAdd(&s_hits[0], 1);
    if (first && place == rank) s_expert = e, atomicAdd(&s_hits[1], 1);
    const int chosen = __popcll(__ballot(first && place < p.top_k));
    if (lane == 0 && chosen) atomicAdd(&s_hits[2], chosen);
    __syncthreads();
  };
  settle(place_of<false>(s_key, s_upper, p.E, e, per));
  if (s_hits[0] != 1 || s_hits[1] != 1 || s_hits[2] != p.top_k) {   // the same for all threads
    const int place = place_of<true>(s_key, s_upper, p.E, e, per);
    __syncthreads();                                                // the counts have been read
    settle(place);
  }
  const int expert = __builtin_amdgcn_readfirstlane(s_expert);
  // This pair's weight, for the next kernel and the caller.  In a workgroup of its
  // own it takes 0.3 us less for one token, but with one workgroup more a pair
  // those that read the same strip of an expert no longer fall on the same die
  // (80 tokens of 8 Q2 x Q2 experts, 768 -> 2048, 2 chosen: 106 instead of 77 us).
  if (part == 0) {
    const uint64_t top_key = s_top;
    const double top = top_key == ~uint64_t(0) ? double(NAN)
                       : __longlong_as_double((long long)(top_key >> 63 ? top_key ^ uint64_t(1) << 63 : ~top_key));
    float sum = 0.0f, mine = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += kUpThreads) {
      const float x = expf(float(p.logits[t * p.E + e] - top));
      if (!p.normalize || s_place[e] < p.top_k) sum += x;
      if (e == expert) mine = x;
    }
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s, 64);
    if (lane == 0) s_red[wave] = sum;
    __syncthreads();
    sum = s_red[0];
#pragma unroll
    for (int v = 1; v < kUpWaves; ++v) sum += s_red[v];
    if (threadIdx.x == (expert & (kUpThreads - 1))) {
      const float w = mine / sum;
      p.chosen[pair] = expert;
      p.share[pair] = w;
      if (p.experts) p.experts[pair] = expert;
      if (p.weights) p.weights[pair] = w;
    }
  }

  const int bi = int(uint32_t(p.D) / uint32_t(p.q)), bo = int(uint32_t(p.F) / uint32_t(p.q));
  const int strips = bo / 16;
  const int s = int(part) * (kUpWaves / WS) + wave / WS;   // strip of the whole hidden row
  const bool live = s < p.q * strips;
  const int k = s / strips, strip = s - k * strips;
  float acc[2] = {0.0f, 0.0f};
  if (live) {
    const Groups groups = leaf_groups_of(p.law, tau, k);
    const __bf16* W[2] = {p.Wg, p.Wu};
    const int64_t base = int64_t(expert) * p.D * p.F;
    const int steps = groups.n * ((bi + 31) / 32), w = wave % WS;
    strip_dot<2>(W, [&](int) { return base; }, p.X + t * p.D, 0, [](int) { return 1.0f; }, groups, k, p.q, bi,
                 int64_t(bi) * bo, strip, lane, w * steps / WS, (w + 1) * steps / WS, acc);
  }
  float g = quad_sum(acc[0]), u = quad_sum(acc[1]);
  if constexpr (WS > 1) {
    if (lane < 16) {
      s_part[wave][0][lane] = g;
      s_part[wave][1][lane] = u;
    }
    __syncthreads();
    if (wave % WS != 0) return;
#pragma unroll
    for (int v = 1; v < WS; ++v) {
      g += s_part[wave + v][0][lane & 15];
      u += s_part[wave + v][1][lane & 15];
    }
  }
  if (live && lane < 16) p.h[int64_t(pair) * p.F + int64_t(k) * bo + strip * 16 + lane] = g / (1.0f + expf(-g)) * u;
}

// Down projection and weighted sum: a workgroup per NS strips of 16 output
// columns of a token (NS = 2: neighbours of one output group, which share the
// loads of the hidden activation; the last of an odd number is alone).  Its NW
// waves share the parts of the sum over the chosen experts and join in a fixed
// order.
template <int NS, int NW>
__global__ __launch_bounds__(64 * NW) void moe_down_kernel(MoeParams p) {
  __shared__ float s_part[NW][NS][16];
  const int64_t t = blockIdx.y;
  const int tau = row_type(p, int(t));
  if (tau < 0 || tau >= p.q) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int bi = int(uint32_t(p.F) / uint32_t(p.q)), bo = int(uint32_t(p.D) / uint32_t(p.q));
  const int strips = bo / 16, parts = (strips + NS - 1) / NS;
  const int k = blockIdx.x / parts, strip = (blockIdx.x - k * parts) * NS;
  const bool both = strip + 1 < strips;
  const Groups groups = leaf_groups_of(p.law, tau, k);
  const __bf16* W[NS];
  W[0] = p.Wd;
  if constexpr (NS == 2) W[1] = p.Wd + (both ? int64_t(bi) * 16 : 0);
  const int32_t* chosen = p.chosen + t * p.top_k;
  const float* weight = p.share + t * p.top_k;
  const int steps = p.top_k * groups.n * ((bi + 31) / 32);
  float acc[NS] = {};
  // the place is held inside the weights even where a caller lets another call
  // or kernel write the workspace meanwhile: wrong values then, but no fault
  const uint32_t last_expert = uint32_t(p.E - 1);
  auto expert_at = [&](int a) { return int64_t(min(uint32_t(chosen[a]), last_expert)) * p.D * p.F; };
  strip_dot<NS>(W, expert_at, p.h + t * p.top_k * p.F, int(p.F),
                [&](int a) { return weight[a]; }, groups, k, p.q, bi, int64_t(bi) * bo, strip, lane, wave * steps / NW,
                (wave + 1) * steps / NW, acc);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const float y = quad_sum(acc[i]);
    if (lane < 16) s_part[wave][i][lane] = y;
  }
  __syncthreads();
  const int i = threadIdx.x / 16, c = threadIdx.x & 15;
  if (i < NS && strip + i < strips) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w += 4)
      v += (s_part[w][i][c] + s_part[w + 1][i][c]) + (s_part[w + 2][i][c] + s_part[w + 3][i][c]);
    const int64_t at = t * p.D + int64_t(k) * bo + (strip + i) * 16 + c;
    if (p.y_f32) static_cast<float*>(p.Y)[at] = v;
    else static_cast<__bf16*>(p.Y)[at] = (__bf16)v;
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
  p.D = up.d_in;
  p.F = up.d_out;
  p.off = int32_t(c.pos_offset % up.q);
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
  const MoeRule rule = moe_rule(up.law == AA_LAW_Q2XQ2, p.q, p.D, p.F, p.top_k, c.M);
  const dim3 block(kUpThreads);
  p.parts = rule.up_parts;
  p.pairs = pairs;
  const dim3 grid = rule.rows_of_eight ? dim3(8 * p.parts, (pairs + 7) / 8) : dim3(p.parts, pairs);
  if (rule.up_waves == 8) launch((moe_up_kernel<8>), grid, block, 0u, stream, p);
  else if (rule.up_waves == 4) launch((moe_up_kernel<4>), grid, block, 0u, stream, p);
  else if (rule.up_waves == 2) launch((moe_up_kernel<2>), grid, block, 0u, stream, p);
  else launch((moe_up_kernel<1>), grid, block, 0u, stream, p);
  st = after_launch(stream, "moe_up_kernel");
  if (st != AA_OK) return st;
  const uint32_t out_strips = uint32_t(p.D / 16), q = uint32_t(p.q);
  const dim3 down_grid((out_strips / q + rule.down_strips - 1) / rule.down_strips * q, M);
  const dim3 down_block(64 * rule.down_waves);
  if (rule.down_strips == 2 && rule.down_waves == 4) launch((moe_down_kernel<2, 4>), down_grid, down_block, 0u, stream, p);
  else if (rule.down_strips == 2) launch((moe_down_kernel<2, 8>), down_grid, down_block, 0u, stream, p);
  else if (rule.down_waves == 4) launch((moe_down_kernel<1, 4>), down_grid, down_block, 0u, stream, p);
  else launch((moe_down_kernel<1, 16>), down_grid, down_block, 0u, stream, p);
  return after_launch(stream, "moe_down_kernel");
}

}  // namespace aa
