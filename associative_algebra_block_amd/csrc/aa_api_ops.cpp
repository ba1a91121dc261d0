// Entry points of the operators around the row-typed FFN (LayerNorm, paged
// decode attention, the mixture-of-experts layer): host-side argument checks,
// then the launches.  Every check happens before anything is enqueued, so a
// call that fails leaves the stream untouched.
#include <math.h>
#include <stdint.h>

#include <string>

#include "aa_checks.h"
#include "aa_internal.h"

using aa::check_dtype;
using aa::check_opt_ptr;
using aa::check_ptr;
using aa::elem_size;
using aa::fail;
using aa::overlaps;

namespace {

aa_status_t check_norm(int64_t M, int64_t d, const char* fn) {
  if (M < 0) return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": M is negative");
  if (M >= (int64_t(1) << 31)) return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": M of 2^31 rows or more");
  if (d < 1) return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": d is less than 1");
  if (d > aa::kNormMaxWidth) return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": rows wider than 16384 features");
  return AA_OK;
}

// Sizes of a paged cache and its table.
aa_status_t check_cache(int64_t n_pages, int32_t page_size, int32_t n_kv_heads, int32_t head_dim, int64_t n_seqs,
                        int64_t max_pages, const char* fn) {
  constexpr int64_t kMax = int64_t(1) << 31;
  if (n_pages < 1 || n_kv_heads < 1 || head_dim < 1 || n_seqs < 0 || max_pages < 1)
    return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": a negative or zero size");
  if (page_size < 16 || page_size > 4096 || (page_size & (page_size - 1)))
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": page_size is not a power of two from 16 to 4096");
  if (head_dim % 8 || head_dim > 256)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": head_dim is not a multiple of 8 up to 256");
  if (n_pages >= kMax || n_seqs >= kMax || max_pages >= kMax || n_kv_heads > 1024)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": more than 1024 kv heads, or 2^31 pages or sequences");
  return AA_OK;
}

// An operand read by elements of `align` bytes.
aa_status_t check_elems(const void* p, size_t align, const char* what, const char* fn) {
  if (!p) return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": " + what + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": " + what + " is not aligned to its elements");
  return AA_OK;
}

// Bytes that rows of `width` elements at a stride of ld span.
size_t rows_bytes(int64_t rows, int64_t ld, int64_t width, aa_dtype_t t) {
  return rows < 1 ? 0 : (size_t(rows - 1) * size_t(ld) + size_t(width)) * elem_size(t);
}

aa_status_t check_ld(int64_t ld, int64_t width, const char* what, const char* fn) {
  if (ld < width) return fail(AA_ERR_SHAPE, std::string(fn) + ": " + what + " is smaller than a row");
  if (ld >= int64_t(1) << 31) return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": " + what + " of 2^31 or more");
  return AA_OK;
}

// A range of memory that a call reads or writes.  in_place: the index of the
// output that this operand is, where the call replaces it in place.
struct Range {
  const void* p;
  size_t bytes;
  const char* name;
  int in_place = -1;
};

// No output may overlap another operand; the outputs are the operands from
// first_out on.  Empty and absent ranges overlap nothing.
template <int N>
aa_status_t check_disjoint(const Range (&all)[N], int first_out, const char* fn) {
  for (int i = first_out; i < N; ++i)
    for (int j = 0; j < N; ++j) {
      if (j == i || all[j].in_place == i || !all[i].p || !all[j].p || !all[i].bytes || !all[j].bytes) continue;
      if (overlaps(all[i].p, all[i].bytes, all[j].p, all[j].bytes))
        return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": " + all[i].name + " overlaps " + all[j].name);
    }
  return AA_OK;
}

}  // namespace

extern "C" {

aa_status_t aa_layernorm_fwd(const void* X, const void* delta, const float* gamma, const float* beta, void* S,
                             void* Y, float* mean, float* rstd, int64_t M, int64_t d, float eps,
                             aa_dtype_t x_dtype, aa_dtype_t delta_dtype, aa_dtype_t y_dtype, hipStream_t stream) {
  aa::clear_error();
  static const char* fn = "aa_layernorm_fwd";
  aa_status_t st;
  if ((st = check_norm(M, d, fn)) != AA_OK) return st;
  if ((st = check_dtype(x_dtype, "x_dtype", fn)) != AA_OK) return st;
  if ((st = check_dtype(delta_dtype, "delta_dtype", fn)) != AA_OK) return st;
  if ((st = check_dtype(y_dtype, "y_dtype", fn)) != AA_OK) return st;
  if (!(eps >= 0.0f) || !isfinite(eps))
    return fail(AA_ERR_INVALID_ARG, "aa_layernorm_fwd: eps is negative or not finite");
  if (!delta != !S) return fail(AA_ERR_INVALID_ARG, "aa_layernorm_fwd: delta and S come together");
  if (!mean != !rstd) return fail(AA_ERR_INVALID_ARG, "aa_layernorm_fwd: mean and rstd come together");
  if (M == 0) return AA_OK;
  if ((st = check_ptr(X, "X", fn)) != AA_OK) return st;
  if ((st = check_ptr(Y, "Y", fn)) != AA_OK) return st;
  if ((st = check_opt_ptr(delta, "delta", fn)) != AA_OK) return st;
  if ((st = check_opt_ptr(S, "S", fn)) != AA_OK) return st;
  if ((st = check_opt_ptr(gamma, "gamma", fn)) != AA_OK) return st;
  if ((st = check_opt_ptr(beta, "beta", fn)) != AA_OK) return st;
  if ((st = check_opt_ptr(mean, "mean", fn)) != AA_OK) return st;
  if ((st = check_opt_ptr(rstd, "rstd", fn)) != AA_OK) return st;
  const size_t n = size_t(M) * size_t(d), row = size_t(d) * 4;
  const Range in[] = {{X, n * elem_size(x_dtype), "X", S == X ? 4 : -1},   // the sum may replace X in place
                      {delta, n * elem_size(delta_dtype), "delta"},
                      {gamma, row, "gamma"},
                      {beta, row, "beta"},
                      {S, n * elem_size(x_dtype), "S"},
                      {Y, n * elem_size(y_dtype), "Y"},
                      {mean, size_t(M) * 4, "mean"},
                      {rstd, size_t(M) * 4, "rstd"}};
  if ((st = check_disjoint(in, 4, fn)) != AA_OK) return st;
  return aa::launch_norm_fwd({X, delta, gamma, beta, S, Y, mean, rstd, M, d, eps, x_dtype, delta_dtype, y_dtype},
                             stream);
}

aa_status_t aa_layernorm_bwd_workspace(int64_t M, int64_t d, size_t* bytes) {
  aa::clear_error();
  aa_status_t st;
  if ((st = check_norm(M, d, "aa_layernorm_bwd_workspace")) != AA_OK) return st;
  if (bytes) *bytes = aa::norm_bwd_workspace_bytes(M, d);
  return AA_OK;
}

aa_status_t aa_layernorm_bwd(const void* X, const void* dY, const float* gamma, const float* mean, const float* rstd,
                             const void* dS, void* dX, float* dgamma, float* dbeta, int64_t M, int64_t d,
                             aa_dtype_t x_dtype, aa_dtype_t dy_dtype, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
  aa::clear_error();
  static const char* fn = "aa_layernorm_bwd";
  aa_status_t st;
  if ((st = check_norm(M, d, fn)) != AA_OK) return st;
  if ((st = check_dtype(x_dtype, "x_dtype", fn)) != AA_OK) return st;
  if ((st = check_dtype(dy_dtype, "dy_dtype", fn)) != AA_OK) return st;
  if ((st = check_opt_ptr(dgamma, "dgamma", fn)) != AA_OK) return st;
  if ((st = check_opt_ptr(dbeta, "dbeta", fn)) != AA_OK) return st;
  const size_t row = size_t(d) * 4, need = dgamma || dbeta ? aa::norm_bwd_workspace_bytes(M, d) : 0;
  if (M > 0) {
    if ((st = check_ptr(X, "X", fn)) != AA_OK) return st;
    if ((st = check_ptr(dY, "dY", fn)) != AA_OK) return st;
    if ((st = check_ptr(mean, "mean", fn)) != AA_OK) return st;
    if ((st = check_ptr(rstd, "rstd", fn)) != AA_OK) return st;
    if ((st = check_ptr(dX, "dX", fn)) != AA_OK) return st;
    if ((st = check_opt_ptr(gamma, "gamma", fn)) != AA_OK) return st;
    if ((st = check_opt_ptr(dS, "dS", fn)) != AA_OK) return st;
    if (workspace_bytes < need)
      return fail(AA_ERR_INVALID_ARG, "aa_layernorm_bwd: workspace smaller than aa_layernorm_bwd_workspace reports");
    if (need > 0 && (st = check_ptr(workspace, "workspace", fn)) != AA_OK) return st;
  }
  const size_t n = size_t(M) * size_t(d);
  const Range in[] = {{X, n * elem_size(x_dtype), "X"},
                      {dY, n * elem_size(dy_dtype), "dY"},
                      {gamma, row, "gamma"},
                      {mean, size_t(M) * 4, "mean"},
                      {rstd, size_t(M) * 4, "rstd"},
                      {dS, n * elem_size(x_dtype), "dS", dS == dX ? 6 : -1},   // dX may replace dS in place
                      {dX, n * elem_size(x_dtype), "dX"},
                      {dgamma, row, "dgamma"},
                      {dbeta, row, "dbeta"},
                      {workspace, need, "workspace"}};
  if ((st = check_disjoint(in, 6, fn)) != AA_OK) return st;
  return aa::launch_norm_bwd({X, dY, gamma, mean, rstd, dS, dX, dgamma, dbeta, M, d, x_dtype, dy_dtype,
                              static_cast<float*>(workspace)},
                             stream);
}

aa_status_t aa_kv_append(const void* K, const void* V, int64_t ldk, int64_t ldv, aa_dtype_t in_dtype, void* k_pages,
                         void* v_pages, int64_t n_pages, int32_t page_size, int32_t n_kv_heads, int32_t head_dim,
                         const int32_t* page_table, int64_t n_seqs, int64_t max_pages, const int32_t* seq,
                         const int32_t* pos, int64_t n, hipStream_t stream) {
  aa::clear_error();
  static const char* fn = "aa_kv_append";
  aa_status_t st;
  if ((st = check_dtype(in_dtype, "in_dtype", fn)) != AA_OK) return st;
  if ((st = check_cache(n_pages, page_size, n_kv_heads, head_dim, n_seqs, max_pages, fn)) != AA_OK) return st;
  if (n < 0) return fail(AA_ERR_INVALID_ARG, "aa_kv_append: n is negative");
  if (n >= int64_t(1) << 31) return fail(AA_ERR_UNSUPPORTED, "aa_kv_append: 2^31 tokens or more");
  if (!seq && n > n_seqs) return fail(AA_ERR_SHAPE, "aa_kv_append: more tokens than sequences and no seq");
  const int64_t width = int64_t(n_kv_heads) * head_dim;
  if ((st = check_ld(ldk, width, "ldk", fn)) != AA_OK) return st;
  if ((st = check_ld(ldv, width, "ldv", fn)) != AA_OK) return st;
  if (n == 0) return AA_OK;
  if ((st = check_elems(K, elem_size(in_dtype), "K", fn)) != AA_OK) return st;
  if ((st = check_elems(V, elem_size(in_dtype), "V", fn)) != AA_OK) return st;
  if ((st = check_ptr(k_pages, "k_pages", fn)) != AA_OK) return st;
  if ((st = check_ptr(v_pages, "v_pages", fn)) != AA_OK) return st;
  if ((st = check_elems(page_table, 4, "page_table", fn)) != AA_OK) return st;
  if (seq && (st = check_elems(seq, 4, "seq", fn)) != AA_OK) return st;
  if ((st = check_elems(pos, 4, "pos", fn)) != AA_OK) return st;
  const size_t cache = size_t(n_pages) * size_t(page_size) * size_t(width) * 2;
  const Range in[] = {{K, rows_bytes(n, ldk, width, in_dtype), "K"},
                      {V, rows_bytes(n, ldv, width, in_dtype), "V"},
                      {page_table, size_t(n_seqs) * size_t(max_pages) * 4, "page_table"},
                      {seq, size_t(n) * 4, "seq"},
                      {pos, size_t(n) * 4, "pos"},
                      {k_pages, cache, "k_pages"},
                      {v_pages, cache, "v_pages"}};
  if ((st = check_disjoint(in, 5, fn)) != AA_OK) return st;
  return aa::launch_kv_append({K, V, ldk, ldv, in_dtype, k_pages, v_pages, n_pages, page_size, n_kv_heads, head_dim,
                               page_table, n_seqs, max_pages, seq, pos, n},
                              stream);
}

// Head counts and the number of rows of the attention calls.
static aa_status_t check_heads(int64_t n_seqs, int32_t n_heads, int32_t n_kv_heads, const char* fn) {
  if (n_heads < 1) return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": n_heads is less than 1");
  if (n_heads % n_kv_heads)
    return fail(AA_ERR_SHAPE, std::string(fn) + ": n_kv_heads does not divide n_heads");
  if (n_seqs * n_heads >= int64_t(1) << 23)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": 2^23 query heads or more over all sequences");
  return AA_OK;
}

aa_status_t aa_attn_decode_workspace(int64_t n_seqs, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                     int32_t page_size, int64_t max_pages, size_t* bytes) {
  aa::clear_error();
  static const char* fn = "aa_attn_decode_workspace";
  aa_status_t st;
  if ((st = check_cache(1, page_size, n_kv_heads, head_dim, n_seqs, max_pages, fn)) != AA_OK) return st;
  if ((st = check_heads(n_seqs, n_heads, n_kv_heads, fn)) != AA_OK) return st;
  if (bytes) *bytes = aa::attn_workspace_bytes(n_seqs, n_heads, n_kv_heads, head_dim, page_size, max_pages);
  return AA_OK;
}

aa_status_t aa_attn_decode(const void* Q, int64_t ldq, aa_dtype_t q_dtype, const void* k_pages, const void* v_pages,
                           int64_t n_pages, int32_t page_size, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                           const int32_t* page_table, int64_t n_seqs, int64_t max_pages, const int32_t* lengths,
                           float scale, void* O, aa_dtype_t o_dtype, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  aa::clear_error();
  static const char* fn = "aa_attn_decode";
  aa_status_t st;
  if ((st = check_dtype(q_dtype, "q_dtype", fn)) != AA_OK) return st;
  if ((st = check_dtype(o_dtype, "o_dtype", fn)) != AA_OK) return st;
  if ((st = check_cache(n_pages, page_size, n_kv_heads, head_dim, n_seqs, max_pages, fn)) != AA_OK) return st;
  if ((st = check_heads(n_seqs, n_heads, n_kv_heads, fn)) != AA_OK) return st;
  // the kernel takes scores to base 2, whose factor must be finite too
  if (!(fabsf(scale) <= 0x1p127f)) return fail(AA_ERR_INVALID_ARG, "aa_attn_decode: scale is not finite or beyond 2^127");
  const int64_t width = int64_t(n_heads) * head_dim;
  if ((st = check_ld(ldq, width, "ldq", fn)) != AA_OK) return st;
  if (n_seqs == 0) return AA_OK;
  if ((st = check_elems(Q, elem_size(q_dtype), "Q", fn)) != AA_OK) return st;
  if ((st = check_ptr(k_pages, "k_pages", fn)) != AA_OK) return st;
  if ((st = check_ptr(v_pages, "v_pages", fn)) != AA_OK) return st;
  if ((st = check_elems(page_table, 4, "page_table", fn)) != AA_OK) return st;
  if ((st = check_elems(lengths, 4, "lengths", fn)) != AA_OK) return st;
  if ((st = check_ptr(O, "O", fn)) != AA_OK) return st;
  const size_t need = aa::attn_workspace_bytes(n_seqs, n_heads, n_kv_heads, head_dim, page_size, max_pages);
  if (workspace_bytes < need)
    return fail(AA_ERR_INVALID_ARG, "aa_attn_decode: workspace smaller than aa_attn_decode_workspace reports");
  if (need > 0 && (st = check_ptr(workspace, "workspace", fn)) != AA_OK) return st;
  const size_t cache = size_t(n_pages) * size_t(page_size) * size_t(n_kv_heads) * size_t(head_dim) * 2;
  const Range in[] = {{Q, rows_bytes(n_seqs, ldq, width, q_dtype), "Q"},
                      {k_pages, cache, "k_pages"},
                      {v_pages, cache, "v_pages"},
                      {page_table, size_t(n_seqs) * size_t(max_pages) * 4, "page_table"},
                      {lengths, size_t(n_seqs) * 4, "lengths"},
                      {O, size_t(n_seqs) * size_t(width) * elem_size(o_dtype), "O"},
                      {workspace, need, "workspace"}};
  if ((st = check_disjoint(in, 5, fn)) != AA_OK) return st;
  return aa::launch_attn_decode({Q, ldq, q_dtype, k_pages, v_pages, n_pages, page_size, n_heads, n_kv_heads, head_dim,
                                 page_table, n_seqs, max_pages, lengths, scale, O, o_dtype, workspace},
                                stream);
}

// Plans and sizes of the mixture-of-experts calls.
static aa_status_t check_moe(aa_plan_t up, aa_plan_t down, int32_t n_experts, int32_t top_k, int64_t M,
                             const char* fn) {
  if (!up || !down) return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": plan is NULL");
  if (up->law != down->law || up->q != down->q)
    return fail(AA_ERR_SHAPE, std::string(fn) + ": up and down plans use different laws or q");
  if (up->type_kind != down->type_kind || up->period != down->period)
    return fail(AA_ERR_SHAPE, std::string(fn) + ": up and down plans use different type maps");
  if (up->d_out != down->d_in || up->d_in != down->d_out)
    return fail(AA_ERR_SHAPE, std::string(fn) + ": up must map D -> F and down F -> D");
  if (up->in_dtype != AA_BF16 || down->in_dtype != AA_BF16)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": experts need bf16 operands");
  if (up->law == AA_LAW_DIGRAPH)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": digraph plans have no expert kernels");
  if (up->layout_version != 1 || down->layout_version != 1)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": blocks that are not multiples of 16 have no expert kernels");
  if (up->type_kind == AA_TYPES_BLOCK_ROWS)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": block-row typing has no expert kernels");
  if (up->d_in >= int64_t(1) << 24 || up->d_out >= int64_t(1) << 24)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": widths of 2^24 or more");
  if (n_experts < 1 || top_k < 1)
    return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": n_experts or top_k is less than 1");
  if (top_k > n_experts) return fail(AA_ERR_SHAPE, std::string(fn) + ": top_k exceeds n_experts");
  if (n_experts > aa::kMoeMaxExperts || top_k > aa::kMoeMaxTopK)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": more than 512 experts, or more than 64 chosen");
  if (M < 0) return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": M is negative");
  if (M > aa::kMoeMaxPairs / top_k)
    return fail(AA_ERR_UNSUPPORTED, std::string(fn) + ": more than 65535 (token, expert) pairs");
  return AA_OK;
}

aa_status_t aa_moe_ffn_workspace(aa_plan_t up, aa_plan_t down, int32_t n_experts, int32_t top_k, int64_t M,
                                 size_t* bytes) {
  aa::clear_error();
  aa_status_t st;
  if ((st = check_moe(up, down, n_experts, top_k, M, "aa_moe_ffn_workspace")) != AA_OK) return st;
  if (bytes) *bytes = aa::moe_workspace_bytes(*up, n_experts, top_k, M);
  return AA_OK;
}

aa_status_t aa_moe_ffn_fwd(aa_plan_t up, aa_plan_t down, const void* X, const void* Wr, int32_t n_experts,
                           int32_t top_k, int32_t normalize, const void* Wg_packed, const void* Wu_packed,
                           const void* Wd_packed, void* Y, int32_t* experts, float* weights, int64_t M,
                           int64_t pos_offset, const int32_t* row_types, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  aa::clear_error();
  static const char* fn = "aa_moe_ffn_fwd";
  aa_status_t st;
  if ((st = check_moe(up, down, n_experts, top_k, M, fn)) != AA_OK) return st;
  if (pos_offset < 0) return fail(AA_ERR_INVALID_ARG, "aa_moe_ffn_fwd: pos_offset is negative");
  if (up->type_kind == AA_TYPES_EXPLICIT) {
    if (!row_types && M > 0) return fail(AA_ERR_INVALID_ARG, "aa_moe_ffn_fwd: explicit type map needs row_types");
  } else if (row_types) {
    return fail(AA_ERR_INVALID_ARG, "aa_moe_ffn_fwd: row_types given for a plan without an explicit type map");
  }
  if (M == 0) return AA_OK;
  if (row_types && (st = check_elems(row_types, 4, "row_types", fn)) != AA_OK) return st;
  if ((st = check_ptr(X, "X", fn)) != AA_OK) return st;
  if ((st = check_ptr(Wr, "Wr", fn)) != AA_OK) return st;
  if ((st = check_ptr(Wg_packed, "Wg_packed", fn)) != AA_OK) return st;
  if ((st = check_ptr(Wu_packed, "Wu_packed", fn)) != AA_OK) return st;
  if ((st = check_ptr(Wd_packed, "Wd_packed", fn)) != AA_OK) return st;
  if ((st = check_ptr(Y, "Y", fn)) != AA_OK) return st;
  if (experts && (st = check_elems(experts, 4, "experts", fn)) != AA_OK) return st;
  if (weights && (st = check_elems(weights, 4, "weights", fn)) != AA_OK) return st;
  const size_t need = aa::moe_workspace_bytes(*up, n_experts, top_k, M);
  if (workspace_bytes < need)
    return fail(AA_ERR_INVALID_ARG, "aa_moe_ffn_fwd: workspace smaller than aa_moe_ffn_workspace reports");
  if ((st = check_ptr(workspace, "workspace", fn)) != AA_OK) return st;
  const size_t E = size_t(n_experts), wb = E * size_t(up->d_in) * size_t(up->d_out) * 2, pairs = size_t(M) * top_k * 4;
  const Range in[] = {{X, size_t(M) * size_t(up->d_in) * 2, "X"},
                      {Wr, E * size_t(up->d_in) * 2, "Wr"},
                      {Wg_packed, wb, "Wg_packed"},
                      {Wu_packed, wb, "Wu_packed"},
                      {Wd_packed, wb, "Wd_packed"},
                      {row_types, size_t(M) * 4, "row_types"},
                      {Y, size_t(M) * size_t(up->d_in) * elem_size(down->out_dtype), "Y"},
                      {experts, pairs, "experts"},
                      {weights, pairs, "weights"},
                      {workspace, need, "workspace"}};
  if ((st = check_disjoint(in, 6, fn)) != AA_OK) return st;
  return aa::launch_moe(*up, *down,
                        {X, Wr, n_experts, top_k, normalize, Wg_packed, Wu_packed, Wd_packed, Y, experts, weights, M,
                         pos_offset, row_types, workspace},
                        stream);
}

}  // extern "C"
