// C-ABI entry points between an attention block's projections: the norm of each head with the rotation
// by position, and causal attention over packed sequences. Everything is checked on the host before
// anything is enqueued.
#include <cmath>

#include "api_util.h"

using namespace lora;

namespace {

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 256;
constexpr int64_t kMaxPositions = int64_t(1) << 24;
constexpr int32_t kMaxHeads = 1 << 13;
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int32_t kMaxSeqs = 1 << 24;
constexpr int64_t kMaxLd = int64_t(1) << 32;

// `ld` with 0 standing for `width` elements; < 0: the status to return
int64_t stride_of(int64_t ld, int64_t width, int64_t align) {
  if (ld == 0) return width;
  if (ld < width) return -LORA_ERR_INVALID;
  if (ld % align) return -LORA_ERR_ALIGN;
  if (ld > kMaxLd) return -LORA_ERR_UNSUPPORTED;
  return ld;
}

// The tensors' strides, checked; x: q, k; y: outputs.
int check_rope(const lora_rope_desc* d, int64_t T, int64_t n_pos, RopeArgs& a) {
  if (!d || T < 0 || n_pos < 1 || d->q_heads < 1 || d->k_heads < 0 || d->head_dim <= 0) return LORA_ERR_INVALID;
  if (d->dtype != LORA_F32 && d->dtype != LORA_BF16) return LORA_ERR_INVALID;
  if (d->layout != LORA_ROPE_HALVES && d->layout != LORA_ROPE_PAIRS) return LORA_ERR_INVALID;
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return LORA_ERR_INVALID;
  if ((d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) || d->q_heads > kMaxHeads ||
      d->k_heads > kMaxHeads - d->q_heads || T >= kMaxTokens || n_pos > kMaxPositions)
    return LORA_ERR_UNSUPPORTED;
  const int64_t ld[2][2] = {{d->ld_q, d->ld_k}, {d->ld_yq, d->ld_yk}};
  a.heads[0] = d->q_heads;
  a.heads[1] = d->k_heads;
  for (int s = 0; s < 2; ++s) {
    for (int y = 0; y < 2; ++y) {
      const int64_t v = s && !a.heads[1] ? 0
                                         : stride_of(ld[y][s], (int64_t)a.heads[s] * d->head_dim,
                                                     d->dtype == LORA_BF16 ? 8 : 4);
      if (v < 0) return (int)-v;
      (y ? a.ld_y : a.ld_x)[s] = v;
    }
  }
  a.T = T; a.n_pos = n_pos; a.dim = d->head_dim; a.dtype = d->dtype;
  a.pairs = d->layout == LORA_ROPE_PAIRS; a.eps = d->eps;
  return LORA_OK;
}

int check_attn(const lora_attn_desc* d, int64_t T, AttnArgs& a) {
  if (!d || T < 0 || d->q_heads < 1 || d->kv_heads < 1 || d->head_dim <= 0) return LORA_ERR_INVALID;
  if (d->q_heads % d->kv_heads) return LORA_ERR_INVALID;
  if (d->dtype < LORA_F32 || d->dtype > LORA_BF16_BLK8) return LORA_ERR_INVALID;
  if (!(d->scale > 0.f) || !std::isfinite(d->scale)) return LORA_ERR_INVALID;
  const int64_t wq = (int64_t)d->q_heads * d->head_dim, wk = (int64_t)d->kv_heads * d->head_dim;
  if (d->dtype != LORA_BF16 || (d->head_dim != 64 && d->head_dim != 128) || wq > kMaxWidth || T >= kMaxTokens)
    return LORA_ERR_UNSUPPORTED;
  const int64_t v[4] = {stride_of(d->ld_q, wq, 8), stride_of(d->ld_k, wk, 8), stride_of(d->ld_v, wk, 8),
                        stride_of(d->ld_o, wq, 8)};
  for (int64_t s : v)
    if (s < 0) return (int)-s;
  a.T = T; a.q_heads = d->q_heads; a.kv_heads = d->kv_heads; a.dim = d->head_dim; a.scale = d->scale;
  a.ld_q = v[0]; a.ld_k = v[1]; a.ld_v = v[2]; a.ld_o = v[3];
  return LORA_OK;
}

int check_seqs(int64_t T, int32_t n_seq) {
  if (T < 0 || n_seq < 1) return LORA_ERR_INVALID;
  if (T >= kMaxTokens || n_seq > kMaxSeqs) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

}  // namespace

extern "C" {

int lora_rope_table(int64_t n_pos, int32_t head_dim, const double* inv_freq, float* table, void* stream) {
  if (n_pos < 1 || head_dim <= 0 || !inv_freq || !table) return LORA_ERR_INVALID;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || n_pos > kMaxPositions) return LORA_ERR_UNSUPPORTED;
  if (!al16(inv_freq) || !al16(table)) return LORA_ERR_ALIGN;
  clear_stale();
  return cuda_status(launch_rope_table(n_pos, head_dim, inv_freq, table, (cudaStream_t)stream));
}

int lora_rope_forward(const lora_rope_desc* d, int64_t T, const void* Q, const void* K, const float* gamma_q,
                      const float* gamma_k, const int32_t* pos, const float* table, int64_t n_pos, void* YQ,
                      void* YK, void* stream) {
  RopeArgs a{};
  const int rc = check_rope(d, T, n_pos, a);
  if (rc) return rc;
  if (!Q || !YQ || !pos || !table || (d->k_heads && (!K || !YK)) || !gamma_q != !gamma_k) return LORA_ERR_INVALID;
  if (!al16(Q) || !al16(K) || !al16(gamma_q) || !al16(gamma_k) || !al16(pos) || !al16(table) || !al16(YQ) || !al16(YK))
    return LORA_ERR_ALIGN;
  if (T == 0) return LORA_OK;
  clear_stale();
  a.x[0] = Q; a.x[1] = K; a.y[0] = YQ; a.y[1] = YK;
  a.gamma[0] = gamma_q; a.gamma[1] = gamma_k; a.pos = pos; a.table = table;
  return cuda_status(launch_rope(a, false, (cudaStream_t)stream));
}

size_t lora_rope_backward_workspace_size(const lora_rope_desc* d, int64_t T) {
  RopeArgs a{};
  if (check_rope(d, T, 1, a) != LORA_OK) return 0;
  return (size_t)kRopeMostCtas * 2 * d->head_dim * sizeof(float) + kWsAlign;
}

int lora_rope_backward(const lora_rope_desc* d, int64_t T, const void* Q, const void* K, const float* gamma_q,
                       const float* gamma_k, const int32_t* pos, const float* table, int64_t n_pos,
                       const void* dYQ, const void* dYK, void* dQ, void* dK, float* dgamma_q, float* dgamma_k,
                       void* ws, size_t ws_bytes, void* stream) {
  RopeArgs a{};
  const int rc = check_rope(d, T, n_pos, a);
  if (rc) return rc;
  if (!gamma_q != !gamma_k || (gamma_q && (!Q || (d->k_heads && !K))) || (!gamma_q && (dgamma_q || dgamma_k)))
    return LORA_ERR_INVALID;
  if (!pos || !table || !dYQ || !dQ || (d->k_heads && (!dYK || !dK)) || !ws) return LORA_ERR_INVALID;
  if (!al16(Q) || !al16(K) || !al16(gamma_q) || !al16(gamma_k) || !al16(pos) || !al16(table) || !al16(dYQ) ||
      !al16(dYK) || !al16(dQ) || !al16(dK) || !al16(dgamma_q) || !al16(dgamma_k) || !al16(ws))
    return LORA_ERR_ALIGN;
  if (ws_bytes < lora_rope_backward_workspace_size(d, T)) return LORA_ERR_WORKSPACE;
  if (T == 0) return LORA_OK;
  clear_stale();
  a.x[0] = Q; a.x[1] = K; a.y[0] = dQ; a.y[1] = dK; a.dy[0] = dYQ; a.dy[1] = dYK;
  a.gamma[0] = gamma_q; a.gamma[1] = gamma_k; a.dgamma[0] = dgamma_q; a.dgamma[1] = dgamma_k;
  a.pos = pos; a.table = table;
  a.part = Carve(ws).take<float>(1);
  return cuda_status(launch_rope(a, true, (cudaStream_t)stream));
}

size_t lora_attn_plan_size(int64_t T, int32_t n_seq) {
  if (check_seqs(T, n_seq) != LORA_OK) return 0;
  return attn_plan(T, n_seq, nullptr).bytes + kWsAlign;
}

int lora_attn_plan_build(int64_t T, int32_t n_seq, const int32_t* d_seq_start, void* plan, size_t plan_bytes,
                         void* stream) {
  const int rc = check_seqs(T, n_seq);
  if (rc) return rc;
  if (!d_seq_start || !plan) return LORA_ERR_INVALID;
  if (!al16(plan) || (reinterpret_cast<uintptr_t>(d_seq_start) & 3u)) return LORA_ERR_ALIGN;
  if (plan_bytes < lora_attn_plan_size(T, n_seq)) return LORA_ERR_WORKSPACE;
  clear_stale();
  return cuda_status(launch_attn_plan(T, n_seq, d_seq_start, attn_plan(T, n_seq, plan), (cudaStream_t)stream));
}

int lora_attn_forward(const lora_attn_desc* d, int64_t T, int32_t n_seq, const void* plan, const void* Q,
                      const void* K, const void* V, void* O, float* lse, void* stream) {
  AttnArgs a{};
  int rc = check_attn(d, T, a);
  if (!rc) rc = check_seqs(T, n_seq);
  if (rc) return rc;
  if (!plan || !Q || !K || !V || !O || !lse) return LORA_ERR_INVALID;
  if (!al16(plan) || !al16(Q) || !al16(K) || !al16(V) || !al16(O) || !al16(lse)) return LORA_ERR_ALIGN;
  if (T == 0) return LORA_OK;
  clear_stale();
  a.plan = attn_plan(T, n_seq, const_cast<void*>(plan));
  a.Q = Q; a.K = K; a.V = V; a.O = O; a.lse = lse;
  return cuda_status(launch_attn_forward(a, (cudaStream_t)stream));
}

size_t lora_attn_backward_workspace_size(const lora_attn_desc* d, int64_t T) {
  AttnArgs a{};
  if (check_attn(d, T, a) != LORA_OK) return 0;
  return (size_t)T * d->q_heads * sizeof(float) + 2 * kWsAlign;
}

int lora_attn_backward(const lora_attn_desc* d, int64_t T, int32_t n_seq, const void* plan, const void* Q,
                       const void* K, const void* V, const void* O, const float* lse, const void* dO, void* dQ,
                       void* dK, void* dV, void* ws, size_t ws_bytes, void* stream) {
  AttnArgs a{};
  int rc = check_attn(d, T, a);
  if (!rc) rc = check_seqs(T, n_seq);
  if (rc) return rc;
  if (!plan || !Q || !K || !V || !O || !lse || !dO || !dQ || !dK || !dV || !ws) return LORA_ERR_INVALID;
  if (!al16(plan) || !al16(Q) || !al16(K) || !al16(V) || !al16(O) || !al16(lse) || !al16(dO) || !al16(dQ) ||
      !al16(dK) || !al16(dV) || !al16(ws))
    return LORA_ERR_ALIGN;
  if (ws_bytes < lora_attn_backward_workspace_size(d, T)) return LORA_ERR_WORKSPACE;
  if (T == 0) return LORA_OK;
  clear_stale();
  a.plan = attn_plan(T, n_seq, const_cast<void*>(plan));
  a.Q = Q; a.K = K; a.V = V; a.O = const_cast<void*>(O); a.lse = const_cast<float*>(lse); a.dO = dO;
  a.dQ = dQ; a.dK = dK; a.dV = dV;
  Carve c(ws);
  a.ready = c.take<int32_t>(1);
  a.delta = c.take<float>(1);
  return cuda_status(launch_attn_backward(a, (cudaStream_t)stream));
}

}  // extern "C"
