// Attention of one new token per sequence over a paged key-value cache, and
// the append that writes new tokens into the cache.
//
//   s_j = scale q . k_j  (0 <= j < length),  p = softmax(s),  o = sum_j p_j v_j
//
// The cache is bf16: pages of `page` positions (a power of two), keys as
// [page id][kv head][position][feature], values as [page id][kv head][feature]
// [position].  With the values transposed, both products find 16 bytes of a
// fragment together:
//   S^T (keys x heads)  = K (16 keys x 32 features) . Q^T
//   O^T (features x heads) += V^T (16 features x 32 keys) . P^T
// The key order inside a product is free, so the 32 keys of a step are dealt
// to the two S^T fragments such that the lane that holds a probability is the
// lane that needs it for the second product: lane (head n, group g) gets keys
// 8 g + 4 t + i in element i of fragment t, and feeds keys 8 g .. 8 g + 7.
//
// The cache crosses HBM once and that bounds the call: 2 G operations a loaded
// value (G query heads share a kv head) are far below the matrix rate even
// where only one of a fragment's 16 head columns is in use.  The matrix slack
// pays for exactness: float32 queries go in as three bf16 terms, the
// probabilities as two (three for float32 outputs), so neither is rounded to
// bf16.
//
// Loads of fragments straight from the cache (16 rows of 64 bytes each) reached
// 5.3 TB/s on 32 sequences of 1000 to 8192 positions (8 kv heads of 128, pages
// of 16, 603 MB); loads of whole kilobytes straight into LDS, read back as
// fragments, reach 6.0 (100 us), where a plain read of as much reaches 6.8.
// One sequence of 131001 positions in pages of 64: 89.8 us, 6.0 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "aa_device.h"
#include "aa_internal.h"
#include "aa_rules.h"

namespace aa {
namespace {

constexpr int kKeys = 32;        // keys of one step of a wave
constexpr int kAttnWaves = 4;
constexpr int kMinTiles = 4;     // steps of a part that a sequence is split into at the least, one a wave
constexpr int kFullTiles = 32;   // steps that repay a workgroup's start and join where others wait for the place
constexpr int kMaxSplit = 256;
constexpr float kLog2e = 1.4426950408889634f;

typedef float f32x8_u __attribute__((ext_vector_type(8), aligned(4)));
typedef __bf16 bf16x8_u __attribute__((ext_vector_type(8), aligned(2)));

// Eight values at the alignment of one.
__device__ inline f32x8_u load8(const float* p) { return *reinterpret_cast<const f32x8_u*>(p); }
__device__ inline f32x8_u load8(const __bf16* p) {
  return __builtin_convertvector(*reinterpret_cast<const bf16x8_u*>(p), f32x8_u);
}

struct AttnParams {
  const void* Q;
  const __bf16* K;
  const __bf16* V;
  const int32_t* table;
  const int32_t* lens;
  void* O;
  float* part;       // [B H][nsplit][D], unnormalised
  float* ml;         // [B H][nsplit][2]: running maximum (log2 scale) and sum
  int64_t ldq, n_pages, max_pages;
  int32_t B, H, Hkv, G, D, head_tiles, page_shift, nsplit, min_tiles, o_f32;
  float scale;
};

// The tiles of a sequence that part s of at most nsplit takes; 32 bits hold
// every count (a length is an int32).
struct TileRange {
  int begin, end;
};
__device__ inline TileRange split_tiles(int len, int nsplit, int min_tiles, int s, int* used) {
  const uint32_t tiles = (uint32_t(len) + kKeys - 1) / kKeys;
  const uint32_t per = max((tiles + nsplit - 1) / uint32_t(nsplit), uint32_t(min_tiles));
  *used = int((tiles + per - 1) / per);
  return {int(min(s * per, tiles)), int(min((s + 1) * per, tiles))};
}

// 16 bytes from each lane's own address to dst + 16 lane (dst is the same for
// the whole wave); NT: past the caches.
typedef __attribute__((address_space(3))) void* lds_ptr_t;
template <bool NT>
__device__ inline void dma16(const __bf16* src, unsigned char* dst) {
  __builtin_amdgcn_global_load_lds(src, (lds_ptr_t)dst, 16, 0, NT ? 2 : 0);
}
// Until all but the last N memory operations of the wave have landed.
template <int N>
__device__ inline void wait_vm() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x0f70 | (N >> 4) << 14);
  __builtin_amdgcn_sched_barrier(0);
}
// v[i] = 16 bytes of LDS at byte address at[i].  As one block with its wait: a
// plain LDS read behind loads into LDS makes the compiler wait for all of them,
// the next step's too.
__device__ inline void read_lds2(const uint32_t* at, u32x4_t* v) {
  asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(v[0]), "=&v"(v[1])
               : "v"(at[0]), "v"(at[1])
               : "memory");
}
__device__ inline uint32_t lds_address(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p));
}

template <bool B> struct Bool {
  static constexpr bool value = B;
};

// x = hi + mid + lo exactly to 24 bits, each a bf16.  lead is x, or x held within
// bf16's range: bf16 rounds the largest float32 values up to infinity, and the
// largest bf16 leaves 16 digits of them as a rounding does.
constexpr float kMaxBf16 = 0x1.fep127f;
__device__ inline void split3(float x, float lead, __bf16* t) {
  t[0] = (__bf16)lead;
  float r = x - float(t[0]);
  t[1] = (__bf16)r;
  t[2] = (__bf16)(r - float(t[1]));
}

__device__ inline bf16x8_t as_frag(u32x4_t v) { return __builtin_bit_cast(bf16x8_t, v); }
__device__ inline f32x4_t mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Two workgroups a unit up to DC = 5, whose LDS just fits twice (47 short sequences
// of 12 heads of 160: 11.3 us instead of 16.5 with one; long ones of float32
// queries, which spill ten registers, take 1 % longer).
//
// DC: 32-wide feature chunks (D <= 32 DC).  NQ: bf16 terms of a query; NP: of
// a probability.
template <int DC, typename TQ, int NP>
__global__ __launch_bounds__(kAttnWaves * 64, DC <= 5 ? 2 : 1) void attn_decode_kernel(AttnParams p) {
  constexpr int NQ = sizeof(TQ) == 4 ? 3 : 1;
  constexpr int DT = 2 * DC;             // 16-wide feature tiles of the output
  constexpr int kRow = 16 * DT + 4;      // floats of one head's row in LDS
  constexpr int kStage = 2048 * DT;      // a wave's keys and values of one step, and in the end its sums
  constexpr int kSums = kAttnWaves * 16 * kRow * 4;   // bytes
  __shared__ __align__(16) unsigned char s_stage[kAttnWaves * kStage];   // all of it: DC = 5 just fits twice
  static_assert(kSums + kAttnWaves * 16 * 2 * 4 <= kAttnWaves * kStage, "the waves' sums overlie the keys and values");
  float(*s_acc)[16][kRow] = reinterpret_cast<float(*)[16][kRow]>(s_stage);
  float(*s_ml)[16][2] = reinterpret_cast<float(*)[16][2]>(s_stage + kSums);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  // parts outermost: consecutive workgroups go to different dies, and the parts
  // that only long sequences have spread over all of them (with the parts
  // innermost, eight of them tied each part to one die, a fifth slower)
  uint32_t w = blockIdx.x;
  const int ht = int(w % uint32_t(p.head_tiles));
  w /= uint32_t(p.head_tiles);
  const int hkv = int(w % uint32_t(p.Hkv));
  w /= uint32_t(p.Hkv);
  const int b = int(w % uint32_t(p.B)), split = int(w / uint32_t(p.B));
  const int heads = min(16, p.G - 16 * ht);              // query heads of this workgroup
  const int head0 = hkv * p.G + 16 * ht;

  int len = p.lens[b];
  bool bad = len < 0 || len > (p.max_pages << p.page_shift);
  if (bad) len = 0;
  int used;
  const TileRange r = split_tiles(len, p.nsplit, p.min_tiles, split, &used);
  if (split >= max(used, 1)) return;

  // queries: lane n holds features 32 c + 8 g .. + 7 of head n
  bf16x8_t q[NQ][DC];
  {
    f32x8_u raw[DC];
#pragma unroll
    for (int c = 0; c < DC; ++c) {
      const int f = 32 * c + 8 * g;
      raw[c] = f32x8_u{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (n < heads && f < p.D)
        raw[c] = load8(static_cast<const TQ*>(p.Q) + b * p.ldq + int64_t(head0 + n) * p.D + f);
    }
#pragma unroll
    for (int c = 0; c < DC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        __bf16 t[3];
        // an infinite or NaN query gives NaN with any keys, here by its lower terms
        const float x = raw[c][e];
        split3(x, NQ > 1 ? __builtin_amdgcn_fmed3f(x, -kMaxBf16, kMaxBf16) : x, t);
#pragma unroll
        for (int k = 0; k < NQ; ++k) q[k][c][e] = t[k];
      }
  }

  f32x4_t acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  const float c2 = p.scale * kLog2e;
  const int last = len - 1;
  const int page_mask = (1 << p.page_shift) - 1;
  const int64_t page_elems = int64_t(p.D) << p.page_shift;   // of one head's page
  const int32_t* row = p.table + b * p.max_pages;

  // A step's 32 positions are two halves of 16, which lie in one page or in two.
  // A missing second half reads the first one's place: what lies behind the end
  // of a sequence is read as it comes, its scores masked and its values zeroed.
  // The ids are read by lanes 0 and 32: a scalar load would hold up the LDS
  // operations behind it.
  auto read_ids = [&](int tile) { return row[min(tile * kKeys + 16 * (lane >> 5), last) >> p.page_shift]; };
  struct Halves {
    int64_t first, second;   // element offsets of the pages
  };
  auto halves_of = [&](int ids) {
    const int id0 = __builtin_amdgcn_readlane(ids, 0), id1 = __builtin_amdgcn_readlane(ids, 32);
    const bool wrong = id0 < 0 || id0 >= p.n_pages || id1 < 0 || id1 >= p.n_pages;
    bad |= wrong;
    Halves h;
    h.first = (int64_t(wrong ? 0 : id0) * p.Hkv + hkv) * page_elems;
    h.second = (int64_t(wrong ? 0 : id1) * p.Hkv + hkv) * page_elems;
    return h;
  };

  // Memory straight to the wave's own LDS, 1 KiB in a row for each load: slot
  // 64 i + lane of load i takes one piece of 16 bytes (slots behind the last
  // piece take that one again).  The keys' whole lines are fetched past the
  // caches (nontemporal), as a long or large cache is read but once: the ragged
  // batch of the head comment takes 108 us with its append and join, with keys
  // through the caches 113.5, the long sequence 98 and 106.  Where tiles of heads
  // or sequences read the same keys, and where the whole cache is small, it costs
  // a little: 8 sequences of 8000 with 40 heads on one kv head 31.5 us against
  // 29.5, 16 of 8000 on the same pages 46.4 and 44.5.  The values are fetched past
  // the caches from pages of up to 32 positions; from larger ones a feature's 64
  // bytes are half a line, whose other half a neighbour wave wants.
  const int R = p.D / 8;              // pieces of a key
  const bool small = p.page_shift == 4;
  unsigned char* kmine = s_stage + wave * kStage;
  unsigned char* vmine = kmine + 1024 * DT;
  // Slot (key, x) of the keys holds piece x - r modulo R, where r is the key's
  // row in its fragment: the 16 rows of a fragment then lie in different banks.
  const uint32_t by_row = (65536u + R - 1) / uint32_t(R);   // y / R = y * by_row >> 16 for all y < 33 R
  int koff[DT];                       // offset of this lane's piece of load i, from the page of its half
#pragma unroll
  for (int i = 0; i < DT; ++i) {
    const int slot = min(64 * i + lane, 32 * R - 1);
    const int key = int(uint32_t(slot) * by_row >> 16);
    const int y = slot - key * R + 32 * R - (((key >> 3) << 2) | (key & 3));
    koff[i] = key * p.D + 8 * (y - int(uint32_t(y) * by_row >> 16) * R);
  }
  auto load_k = [&](int tile, const Halves& h) {
    const __bf16* k0 = p.K + h.first + int64_t((tile * kKeys) & page_mask) * p.D;
    const __bf16* k1 = p.K + h.second + int64_t((tile * kKeys + 16) & page_mask) * p.D - 16 * p.D;
#pragma unroll
    for (int i = 0; i < DT; ++i) dma16<true>((koff[i] < 16 * p.D ? k0 : k1) + koff[i], kmine + 1024 * i);
  };
  // Values: [half][feature][16] from pages of 16, else [feature][32], the pieces
  // of a feature turned by its row in the fragment for the banks' sake.
  auto load_wide = [&](auto nt, int tile, const Halves& h) {
    const __bf16* v0 = p.V + h.first + ((tile * kKeys) & page_mask);
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      const int slot = min(64 * i + lane, 4 * p.D - 1);
      dma16<nt.value>(v0 + (int64_t(slot >> 2) << p.page_shift) + ((slot - (slot >> 4)) & 3) * 8, vmine + 1024 * i);
    }
  };
  auto load_v = [&](int tile, const Halves& h) {
    if (small) {
      const __bf16* v0 = p.V + h.first;
      const __bf16* v1 = p.V + h.second - 16 * p.D;
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        const int slot = min(64 * i + lane, 4 * p.D - 1);
        const int half = slot < 2 * p.D ? 0 : 1, d = (slot - half * 2 * p.D) >> 1;
        dma16<true>((half ? v1 : v0) + (slot ^ ((d >> 3) & 1)) * 8, vmine + 1024 * i);
      }
    } else if (p.page_shift == 5) {
      load_wide(Bool<true>(), tile, h);
    } else {
      load_wide(Bool<false>(), tile, h);
    }
  };
  uint32_t kslot[2 * DC];             // LDS address of this lane's piece of chunk c in fragment t: row n there is
#pragma unroll
  for (int c = 0; c < DC; ++c) {      // key 8 (n / 4) + 4 t + n mod 4
    const int piece = min(4 * c + g, R - 1), y = piece + n;
    kslot[c] = lds_address(kmine) + ((8 * (n >> 2) + (n & 3)) * R + y - int(uint32_t(y) * by_row >> 16) * R) * 16;
    kslot[DC + c] = kslot[c] + 64 * R;
  }
  const uint32_t vfrag = lds_address(vmine) + (small ? (g >> 1) * 32 * p.D + n * 32 + ((g ^ (n >> 3)) & 1) * 16
                                                     : n * 64 + ((g + (n >> 2)) & 3) * 16);
  const int vstep = small ? 512 : 1024;   // bytes from 16 features to the next

  // The next step's keys are on their way as soon as this one's have left LDS,
  // its values likewise, and the page ids a step before that.  Every step issues
  // the ids, DT loads of keys and DT of values in this order, so a count says
  // which have landed.
  int tile = r.begin + wave;
  int ids = 0;
  auto step = [&](auto more) {
    const int next = tile + kAttnWaves;
    wait_vm<DT>();                    // keys (behind them: this step's values)
    f32x4_t s[2], lo[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) s[t] = lo[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 2 * DC; j += 2) {   // pieces j and j + 1 of [fragment][chunk]
      u32x4_t kf[2];
      read_lds2(kslot + j, kf);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = (j + x) / DC, c = (j + x) % DC;
        // features behind D: zero (a zero query alone would turn an infinite key into a NaN)
        if (c == DC - 1 && 4 * c + g >= R) kf[x] = u32x4_t{0u, 0u, 0u, 0u};
        s[t] = mfma(as_frag(kf[x]), q[0][c], s[t]);
#pragma unroll
        for (int i = NQ - 1; i >= 1; --i) lo[t] = mfma(as_frag(kf[x]), q[i][c], lo[t]);
      }
    }
    if constexpr (NQ > 1) {
      // an infinite key: the leading term has the query's sign, the others need not
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] = __builtin_isfinite(s[t][i]) ? s[t][i] + lo[t][i] : s[t][i];
    }
    Halves now = {0, 0};
    if constexpr (more.value) {
      now = halves_of(ids);
      ids = read_ids(min(next + kAttnWaves, r.end - 1));
      load_k(next, now);
    }
    const int left = len - (tile * kKeys + 8 * g);          // positions of this lane's 8 that count
    float mx = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[t][i] = 4 * t + i < left ? s[t][i] * c2 : -INFINITY;
        mx = fmaxf(mx, s[t][i]);
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    const float m_new = fmaxf(m, mx);
    const float mu = m_new == -INFINITY ? 0.0f : m_new;          // all scores -inf so far: their weights are 0
    const float alpha = __builtin_amdgcn_exp2f(m - mu);
    m = m_new;
    float sum = 0.0f;
    bf16x8_t pf[NP];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(s[t][i] - mu);
        sum += e;
        __bf16 term[3];
        split3(e, e, term);
#pragma unroll
        for (int k = 0; k < NP; ++k) pf[k][4 * t + i] = term[k];
      }
    l = l * alpha + sum;
    // what lies behind the end may be anything, NaN included, and 0 . NaN is no zero
    uint32_t keep[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) keep[j] = (2 * j < left ? 0xffffu : 0u) | (2 * j + 1 < left ? 0xffff0000u : 0u);
    const bool tail = len - tile * kKeys < kKeys;
    wait_vm<more.value ? DT + 1 : 0>();   // values (behind them: ids and the next keys)
    if (__any(alpha != 1.0f)) {   // the maximum moves in few steps but the first
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] *= alpha;
    }
#pragma unroll
    for (int d = 0; d < DT; d += 2) {
      const uint32_t at[2] = {vfrag + d * vstep, vfrag + (d + 1) * vstep};
      u32x4_t v[2];
      read_lds2(at, v);       // rows behind D hold anything and are not stored
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (tail) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[x][j] &= keep[j];
        }
#pragma unroll
        for (int k = NP - 1; k >= 0; --k) acc[d + x] = mfma(as_frag(v[x]), pf[k], acc[d + x]);
      }
    }
    if constexpr (more.value) {
      load_v(next, now);
    }
  };
  if (tile < r.end) {
    const int first_ids = read_ids(tile);
    ids = read_ids(min(tile + kAttnWaves, r.end - 1));
    const Halves first = halves_of(first_ids);
    load_k(tile, first);
    load_v(tile, first);
    for (; tile + kAttnWaves < r.end; tile += kAttnWaves) step(Bool<true>());
    step(Bool<false>());
  }

  // join the waves: lane (n, g) holds features 16 d + 4 g .. + 3 of head n
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  if (__any(bad)) l = NAN;   // a page outside the cache: the result is no number
  __syncthreads();   // the sums of one wave overlie what another may still read
  if (g == 0) {
    s_ml[wave][n][0] = m;
    s_ml[wave][n][1] = l;
  }
#pragma unroll
  for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4_t*>(&s_acc[wave][n][16 * d + 4 * g]) = acc[d];
  __syncthreads();
  for (int i = threadIdx.x; i < heads * p.D; i += kAttnWaves * 64) {
    const int hn = i / p.D, f = i - hn * p.D;
    float mm = s_ml[0][hn][0];
#pragma unroll
    for (int v = 1; v < kAttnWaves; ++v) mm = fmaxf(mm, s_ml[v][hn][0]);
    const float mu = mm == -INFINITY ? 0.0f : mm;
    float ll = 0.0f, o = 0.0f;
#pragma unroll
    for (int v = 0; v < kAttnWaves; ++v) {
      const float e = __builtin_amdgcn_exp2f(s_ml[v][hn][0] - mu);
      ll += e * s_ml[v][hn][1];
      o += e * s_acc[v][hn][f];
    }
    const int64_t out = int64_t(b) * p.H + head0 + hn;
    if (p.nsplit == 1) {
      o = p.lens[b] == 0 ? 0.0f : o / ll;   // no position: zeros
      if (p.o_f32) static_cast<float*>(p.O)[out * p.D + f] = o;
      else static_cast<__bf16*>(p.O)[out * p.D + f] = (__bf16)o;
    } else {
      const int64_t at = out * p.nsplit + split;
      p.part[at * p.D + f] = o;
      if (f == 0) {
        p.ml[2 * at] = mm;
        p.ml[2 * at + 1] = ll;
      }
    }
  }
}

// Joins the splits of one (sequence, head): a thread per split for the maximum
// and the sum, then the threads as groups of `lanes` (a power of two that holds
// a row in pieces of four features) that take the splits in turn and join in
// LDS, all in a fixed order.  One wave that took the splits in turn needed
// 17.7 us for 32 heads of 128 splits, each load behind the last; this takes 4.8.
__global__ __launch_bounds__(kMaxSplit) void attn_join_kernel(AttnParams p, int lanes) {
  __shared__ float s_w[kMaxSplit], s_red[2][kMaxSplit / 64];
  __shared__ float s_o[kMaxSplit * 4];
  const int64_t out = blockIdx.x;
  const int b = int(blockIdx.x / uint32_t(p.H));
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t length = p.lens[b];
  int len = length;
  if (len < 0 || len > (p.max_pages << p.page_shift)) len = 0;   // split 0 wrote a NaN
  int used;
  split_tiles(len, p.nsplit, p.min_tiles, 0, &used);
  used = max(used, 1);
  const float* ml = p.ml + 2 * out * p.nsplit;
  const float m = tid < used ? ml[2 * tid] : -INFINITY;
  const float l = tid < used ? ml[2 * tid + 1] : 0.0f;
  float mm = m;
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) mm = fmaxf(mm, __shfl_xor(mm, x, 64));
  if (lane == 0) s_red[0][wave] = mm;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kMaxSplit / 64; ++v) mm = fmaxf(mm, s_red[0][v]);
  const float w = __builtin_amdgcn_exp2f(m - (mm == -INFINITY ? 0.0f : mm));
  s_w[tid] = w;
  float sum = tid < used ? w * l : 0.0f;
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) sum += __shfl_xor(sum, x, 64);
  if (lane == 0) s_red[1][wave] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int v = 0; v < kMaxSplit / 64; ++v) sum += s_red[1][v];

  const int groups = kMaxSplit / lanes, group = tid / lanes, f = 4 * (tid & (lanes - 1));
  f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (f < p.D) {
    const float* part = p.part + out * p.nsplit * p.D + f;
#pragma unroll 8
    for (int s = group; s < used; s += groups) o += *reinterpret_cast<const f32x4_t*>(part + int64_t(s) * p.D) * s_w[s];
  }
  *reinterpret_cast<f32x4_t*>(&s_o[4 * tid]) = o;   // [group][4 lanes]
  __syncthreads();
  if (tid < p.D) {
    float v = 0.0f;
    for (int g = 0; g < min(groups, used); ++g) v += s_o[4 * lanes * g + tid];
    v = length == 0 ? 0.0f : v / sum;
    if (p.o_f32) static_cast<float*>(p.O)[out * p.D + tid] = v;
    else static_cast<__bf16*>(p.O)[out * p.D + tid] = (__bf16)v;
  }
}

struct AppendParams {
  const void* K;
  const void* V;
  __bf16* Kp;
  __bf16* Vp;
  const int32_t* table;
  const int32_t* seq;   // or nullptr: token t belongs to sequence t
  const int32_t* pos;
  int64_t ldk, ldv, n, n_seqs, n_pages, max_pages, total;
  int32_t Hkv, D, page_shift;
};

// Where token t goes: the element offset of head h in its page, or -1, and the
// position in the page.
struct Slot {
  int64_t head;
  int32_t slot;
};
__device__ inline Slot slot_of(const AppendParams& p, int64_t t, int h) {
  const int64_t s = p.seq ? p.seq[t] : t, pos = p.pos[t];
  if (s < 0 || s >= p.n_seqs || pos < 0 || (pos >> p.page_shift) >= p.max_pages) return {-1, 0};
  const int64_t page = p.table[s * p.max_pages + (pos >> p.page_shift)];
  if (page < 0 || page >= p.n_pages) return {-1, 0};
  return {(page * p.Hkv + h) * (int64_t(p.D) << p.page_shift), int32_t(pos & ((int64_t(1) << p.page_shift) - 1))};
}

// A few tokens: one thread per 8 features of one token and head, bound by
// latency.  Small workgroups spread the scattered stores of the values over more
// units (32 tokens of 8 heads of 128: 2.7 us, in workgroups of 256 3.5).
constexpr int kAppendThreads = 64;
template <typename T>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendParams p) {
  const int chunks = p.D / 8;
  const int64_t stride = int64_t(gridDim.x) * kAppendThreads;
  for (int64_t i = int64_t(blockIdx.x) * kAppendThreads + threadIdx.x; i < p.total; i += stride) {
    const int c = int(i % chunks);
    const int64_t th = i / chunks;
    const int h = int(th % p.Hkv);
    const int64_t t = th / p.Hkv;
    // the token's values do not wait for its place
    const f32x8_u k = load8(static_cast<const T*>(p.K) + t * p.ldk + int64_t(h) * p.D + 8 * c);
    const f32x8_u v = load8(static_cast<const T*>(p.V) + t * p.ldv + int64_t(h) * p.D + 8 * c);
    const Slot at = slot_of(p, t, h);
    if (at.head < 0) continue;
    *reinterpret_cast<bf16x8_u*>(p.Kp + at.head + int64_t(at.slot) * p.D + 8 * c) = __builtin_convertvector(k, bf16x8_u);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      p.Vp[at.head + (int64_t(8 * c + e) << p.page_shift) + at.slot] = (__bf16)v[e];
  }
}

// Many tokens, as a prompt has them: a workgroup takes 64 tokens of one head and
// turns their values in LDS, so that 8 tokens at successive positions of a page
// leave as 16 bytes a feature and 64 as whole lines; others leave one by one.
// Rows of D + 2 values put the 64 reads of a wave (8 tokens apart, 8 features)
// into different banks.
template <typename T>
__global__ __launch_bounds__(kTurnThreads) void kv_append_turn_kernel(AppendParams p) {
  typedef __bf16 bf16x8_4 __attribute__((ext_vector_type(8), aligned(4)));
  extern __shared__ __align__(16) __bf16 s_v[];   // [64][D + 2]
  __shared__ int64_t s_head[kTurnTokens];
  __shared__ int32_t s_slot[kTurnTokens], s_run[kTurnTokens / 8];
  const int64_t t0 = int64_t(blockIdx.x) * kTurnTokens;
  const int h = blockIdx.y, chunks = p.D / 8, stride = p.D + 2;
  if (threadIdx.x < kTurnTokens) {
    Slot at = {-1, 0};
    if (t0 + threadIdx.x < p.n) at = slot_of(p, t0 + threadIdx.x, h);
    s_head[threadIdx.x] = at.head;
    s_slot[threadIdx.x] = at.slot;
  }
  __syncthreads();
  if (threadIdx.x < kTurnTokens / 8) {
    const int first = threadIdx.x * 8;
    bool run = s_head[first] >= 0;
    for (int j = 1; j < 8; ++j) run &= s_head[first + j] == s_head[first] && s_slot[first + j] == s_slot[first] + j;
    s_run[threadIdx.x] = run;
  }
  for (int i = threadIdx.x; i < kTurnTokens * chunks; i += kTurnThreads) {
    const int token = i / chunks, c = i - token * chunks;
    if (s_head[token] < 0) continue;
    const int64_t t = t0 + token;
    const f32x8_u k = load8(static_cast<const T*>(p.K) + t * p.ldk + int64_t(h) * p.D + 8 * c);
    const f32x8_u v = load8(static_cast<const T*>(p.V) + t * p.ldv + int64_t(h) * p.D + 8 * c);
    *reinterpret_cast<bf16x8_u*>(p.Kp + s_head[token] + int64_t(s_slot[token]) * p.D + 8 * c) =
        __builtin_convertvector(k, bf16x8_u);
    *reinterpret_cast<bf16x8_4*>(s_v + token * stride + 8 * c) = __builtin_convertvector(v, bf16x8_4);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * p.D; i += kTurnThreads) {
    const int g = i & 7, d = i >> 3;
    const __bf16* src = s_v + 8 * g * stride + d;
    __bf16* dst = p.Vp + (int64_t(d) << p.page_shift);
    if (s_run[g]) {
      bf16x8_u v;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = src[j * stride];
      *reinterpret_cast<bf16x8_u*>(dst + s_head[8 * g] + s_slot[8 * g]) = v;
    } else {
      for (int j = 0; j < 8; ++j)
        if (s_head[8 * g + j] >= 0) dst[s_head[8 * g + j] + s_slot[8 * g + j]] = src[j * stride];
    }
  }
}

int page_shift_of(int page) { return __builtin_ctz(unsigned(page)); }
int head_tiles_of(int G) { return (G + 15) / 16; }

template <int DC>
void launch_attn_dc(const AttnParams& p, bool q_f32, uint32_t grid, hipStream_t stream) {
  const dim3 g(grid), blk(kAttnWaves * 64);
  if (q_f32) {
    if (p.o_f32) launch((attn_decode_kernel<DC, float, 3>), g, blk, 0u, stream, p);
    else launch((attn_decode_kernel<DC, float, 2>), g, blk, 0u, stream, p);
  } else {
    if (p.o_f32) launch((attn_decode_kernel<DC, __bf16, 3>), g, blk, 0u, stream, p);
    else launch((attn_decode_kernel<DC, __bf16, 2>), g, blk, 0u, stream, p);
  }
}

}  // namespace

// Parts that one (sequence, kv head, head tile) is split into at most: what
// gives every compute unit a workgroup when every page of the table is in use,
// as long as each part keeps kMinTiles steps; of narrow heads, whose small steps
// are bound by latency, as many workgroups as fit, in parts of twice as many
// steps.  More, up to eight workgroups a unit in parts of kFullTiles steps, even
// out long sequences of different lengths.  A
// shorter sequence takes parts of the same size, kFullTiles at most, and then
// fewer of them (split_tiles).  Measured with 32 query and 8 kv heads of 128
// (us): one sequence of 8000 in 16, 32, 64 parts 14.4, 12.3, 12.3; two of up to
// 8000 in 8, 16, 32 parts 20.7, 15.9, 17.2; 32 of up to 2000 in 1, 2, 8 parts
// 31.9, 35.3, 40.0 (31 of 100 with one of 2000 in 1 and 8: 27.1 and 19.0); 32 of
// 1000 to 8192 in 4 and 8 parts 102.8 and 100.3; one of 2000 in parts of at least
// 4 and 8 steps 9.3 and 11.0.  32 heads of 24, eight sequences of up to 1500 in
// 1, 2, 4, 8 parts: 13.8, 14.5, 13.7, 13.4; four: 13.8, 11.9, 10.4, 10.4.
// All of these fill their tables.  In a wider table a part is at least the
// table's steps over its parts (min_tiles), so short sequences get few of them:
// one sequence of 2000 takes 9.4 us in a table of 2048 positions and 18.6 in one
// of 32768, one of 8192 14.7 and 19.6, four of 2000 13.8 and 19.7; with 32 heads
// of 24, one of 200 takes 4.9 us in a table of 256 and 7.7, with a join, in one of
// 1536.
int attn_nsplit(int64_t n_seqs, int H, int Hkv, int D, int64_t max_pages, int page) {
  const int64_t rows = std::max<int64_t>(n_seqs * Hkv * head_tiles_of(H / Hkv), 1);
  const int64_t tiles = (max_pages * page + kKeys - 1) / kKeys;
  if (tiles <= 4 * kMinTiles) return 1;   // 400 positions: 10.3 us, in two parts and a join 10.7
  const int64_t units = device_cu_count(), per_unit = D <= 32 ? 8 : D <= 64 ? 4 : 1;
  auto parts = [&](int64_t wgs_per_unit, int64_t steps) {   // rounded up: parts of at most `steps`
    return std::min((wgs_per_unit * units + rows - 1) / rows, (tiles + steps - 1) / steps);
  };
  const int64_t fill = std::max(parts(1, kMinTiles), parts(per_unit, 2 * kMinTiles));
  const int64_t even = tiles < 4 * kFullTiles ? 1 : parts(8, kFullTiles);
  return int(std::max<int64_t>(1, std::min<int64_t>(std::max(fill, even), kMaxSplit)));
}

size_t attn_workspace_bytes(int64_t n_seqs, int H, int Hkv, int D, int page, int64_t max_pages) {
  const int ns = attn_nsplit(n_seqs, H, Hkv, D, max_pages, page);
  return ns == 1 ? 0 : size_t(n_seqs) * size_t(H) * size_t(ns) * size_t(D + 2) * 4;
}

aa_status_t launch_attn_decode(const AttnCall& c, hipStream_t stream) {
  AttnParams p{};
  p.Q = c.Q;
  p.K = static_cast<const __bf16*>(c.k_pages);
  p.V = static_cast<const __bf16*>(c.v_pages);
  p.table = c.page_table;
  p.lens = c.lengths;
  p.O = c.O;
  p.ldq = c.ldq;
  p.n_pages = c.n_pages;
  p.max_pages = c.max_pages;
  p.B = int(c.n_seqs);
  p.H = c.n_heads;
  p.Hkv = c.n_kv_heads;
  p.G = c.n_heads / c.n_kv_heads;
  p.D = c.head_dim;
  p.head_tiles = head_tiles_of(p.G);
  p.page_shift = page_shift_of(c.page_size);
  p.nsplit = attn_nsplit(c.n_seqs, c.n_heads, c.n_kv_heads, c.head_dim, c.max_pages, c.page_size);
  const int64_t tiles = (c.max_pages * c.page_size + kKeys - 1) / kKeys;
  p.min_tiles = int(std::min<int64_t>(std::max<int64_t>(tiles / p.nsplit, kMinTiles), kFullTiles));
  p.o_f32 = c.o_dtype == AA_F32;
  p.scale = c.scale;
  p.part = static_cast<float*>(c.workspace);
  p.ml = p.part ? p.part + int64_t(p.B) * p.H * p.nsplit * p.D : nullptr;
  const uint32_t grid = uint32_t(c.n_seqs * c.n_kv_heads * p.head_tiles * p.nsplit);
  const bool q_f32 = c.q_dtype == AA_F32;
  switch ((p.D + 31) / 32) {
    case 1: launch_attn_dc<1>(p, q_f32, grid, stream); break;
    case 2: launch_attn_dc<2>(p, q_f32, grid, stream); break;
    case 3: launch_attn_dc<3>(p, q_f32, grid, stream); break;
    case 4: launch_attn_dc<4>(p, q_f32, grid, stream); break;
    case 5: launch_attn_dc<5>(p, q_f32, grid, stream); break;
    case 6: launch_attn_dc<6>(p, q_f32, grid, stream); break;
    case 7: launch_attn_dc<7>(p, q_f32, grid, stream); break;
    default: launch_attn_dc<8>(p, q_f32, grid, stream); break;
  }
  aa_status_t st = after_launch(stream, "attn_decode_kernel");
  if (st != AA_OK || p.nsplit == 1) return st;
  int lanes = 2;
  while (4 * lanes < p.D) lanes *= 2;
  launch(attn_join_kernel, dim3(uint32_t(int64_t(p.B) * p.H)), dim3(kMaxSplit), 0u, stream, p, lanes);
  return after_launch(stream, "attn_join_kernel");
}

aa_status_t launch_kv_append(const AppendCall& c, hipStream_t stream) {
  AppendParams p{c.K,     c.V,        static_cast<__bf16*>(c.k_pages), static_cast<__bf16*>(c.v_pages),
                 c.page_table, c.seq, c.pos, c.ldk, c.ldv, c.n, c.n_seqs, c.n_pages, c.max_pages,
                 c.n * c.n_kv_heads * (c.head_dim / 8), c.n_kv_heads, c.head_dim, page_shift_of(c.page_size)};
  if (append_turns(p.n, p.D)) {
    const dim3 grid(uint32_t(append_turn_workgroups(p.n)), uint32_t(p.Hkv));
    const uint32_t lds = uint32_t(kTurnTokens * (p.D + 2) * 2);
    if (c.in_dtype == AA_F32) launch((kv_append_turn_kernel<float>), grid, dim3(kTurnThreads), lds, stream, p);
    else launch((kv_append_turn_kernel<__bf16>), grid, dim3(kTurnThreads), lds, stream, p);
    return after_launch(stream, "kv_append_turn_kernel");
  }
  const int64_t wgs =
      std::min<int64_t>((p.total + kAppendThreads - 1) / kAppendThreads, int64_t(device_cu_count()) * 32);
  if (c.in_dtype == AA_F32) launch((kv_append_kernel<float>), dim3(uint32_t(wgs)), dim3(kAppendThreads), 0u, stream, p);
  else launch((kv_append_kernel<__bf16>), dim3(uint32_t(wgs)), dim3(kAppendThreads), 0u, stream, p);
  return after_launch(stream, "kv_append_kernel");
}

}  // namespace aa
