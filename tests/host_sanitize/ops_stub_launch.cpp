// Stand-ins for the launchers behind the LayerNorm, paged-attention and
// mixture-of-experts entry points, for the host-only build under the
// sanitizers: each records that it was reached and launches nothing.
#include "aa_internal.h"

namespace aa {

int g_launches = 0;

aa_status_t launch_norm_fwd(const NormFwdCall&, hipStream_t) {
  ++g_launches;
  return AA_OK;
}
size_t norm_bwd_workspace_bytes(int64_t M, int64_t d) { return M > 0 ? size_t(d) * 8 : 0; }
aa_status_t launch_norm_bwd(const NormBwdCall&, hipStream_t) {
  ++g_launches;
  return AA_OK;
}
size_t attn_workspace_bytes(int64_t n_seqs, int n_heads, int, int head_dim, int, int64_t) {
  return size_t(n_seqs) * n_heads * (head_dim + 2) * 4;
}
aa_status_t launch_attn_decode(const AttnCall&, hipStream_t) {
  ++g_launches;
  return AA_OK;
}
aa_status_t launch_kv_append(const AppendCall&, hipStream_t) {
  ++g_launches;
  return AA_OK;
}
size_t moe_workspace_bytes(const aa_plan_s& up, int n_experts, int top_k, int64_t M) {
  return size_t(M) * (size_t(n_experts) * 8 + size_t(top_k) * up.d_out * 4);
}
aa_status_t launch_moe(const aa_plan_s&, const aa_plan_s&, const MoeCall&, hipStream_t) {
  ++g_launches;
  return AA_OK;
}

}  // namespace aa
