// C-ABI entry points around the adapted linear: the block-scaled E4M3 frozen product, layer norm,
// the orthogonalised update. Everything is checked on the host before anything is enqueued.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "api_util.h"

using namespace lora;

namespace {

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 256;
constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxElements = int64_t(1) << 40;   // 2^30 blocks of 256 vectors at the least

int check_product(int64_t T, int64_t out_dim, int64_t in_dim) {
  if (T < 0 || out_dim <= 0 || in_dim <= 0) return LORA_ERR_INVALID;
  if (out_dim % 16 || in_dim % 16) return LORA_ERR_ALIGN;
  if (T >= kMaxTokens || out_dim > kMaxDim || in_dim > kMaxDim) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

struct ProductWs {
  uint8_t* codes;
  float* scales;
  size_t bytes;
};

ProductWs product_carve(int64_t T, int64_t K, void* ws) {
  ProductWs w;
  Carve c(ws);
  w.codes = c.take<uint8_t>((size_t)T * K);
  w.scales = c.take<float>((size_t)block_scales_ld(T) * ((K + LORA_SCALE_BLOCK - 1) / LORA_SCALE_BLOCK));
  w.bytes = c.off + kWsAlign;
  return w;
}

int check_norm(const lora_norm_desc* d, int64_t T) {
  if (!d || T < 0 || d->dim <= 0) return LORA_ERR_INVALID;
  if (d->kind != LORA_NORM_LAYER && d->kind != LORA_NORM_RMS) return LORA_ERR_INVALID;
  if (d->dtype != LORA_F32 && d->dtype != LORA_BF16) return LORA_ERR_INVALID;
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return LORA_ERR_INVALID;
  if (d->dim % 8) return LORA_ERR_ALIGN;
  if (d->dim > LORA_NORM_MAX_DIM || T >= kMaxTokens) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

// The matrices of an update, checked; `groups` may be null (the workspace's size alone).
int check_mats(int32_t n_mats, const lora_mat* mats, const GroupTab* groups) {
  if (n_mats < 0 || (n_mats > 0 && !mats)) return LORA_ERR_INVALID;
  bool sorted = true;
  for (int32_t i = 0; i < n_mats; ++i) {
    const lora_mat& e = mats[i];
    if (e.offset < 0 || e.rows <= 0 || e.cols <= 0 || e.group < 0) return LORA_ERR_INVALID;
    if (e.kind != LORA_KIND_A && e.kind != LORA_KIND_B) return LORA_ERR_INVALID;
    const int64_t s = std::min(e.rows, e.cols), n = std::max(e.rows, e.cols);
    if (s > LORA_MAX_RANK || s % 4 || n > kMaxDim) return LORA_ERR_UNSUPPORTED;
    if (e.offset % 4 || n % 4) return LORA_ERR_ALIGN;
    if (e.offset > INT64_MAX - s * n) return LORA_ERR_INVALID;
    if (groups) {
      if (e.group >= groups->n) return LORA_ERR_INVALID;
      const int64_t lo = groups->offset[e.group], hi = lo + groups->count[e.group];
      if (e.offset < lo || e.offset + s * n > hi) return LORA_ERR_INVALID;
    }
    if (i && e.offset < mats[i - 1].offset + mats[i - 1].rows * mats[i - 1].cols) sorted = false;
  }
  if (!sorted) {   // not in ascending, disjoint order as given: sort a copy and look again
    std::vector<std::pair<int64_t, int64_t>> r(n_mats);
    for (int32_t i = 0; i < n_mats; ++i)
      r[i] = {mats[i].offset, mats[i].offset + mats[i].rows * mats[i].cols};
    std::sort(r.begin(), r.end());
    for (int32_t i = 1; i < n_mats; ++i)
      if (r[i].first < r[i - 1].second) return LORA_ERR_INVALID;
  }
  return LORA_OK;
}

// The matrices in the order of their launches: by kernel (smaller side at most 16, each of its own,
// or above) and falling length. A launch takes a run of equal keys; a kernel's matrices have one
// cluster size, so that those of a call share one launch.
struct MuonOrder {
  int32_t at;      // index into the caller's table
  int32_t key;     // cluster size and smaller side (0: above 16)
  MuonMat m;
};

std::vector<MuonOrder> muon_order(int32_t n_mats, const lora_mat* mats) {
  std::vector<MuonOrder> v(n_mats);
  int cluster[17] = {};
  for (int32_t i = 0; i < n_mats; ++i) {
    const lora_mat& e = mats[i];
    MuonMat& t = v[i].m;
    t = MuonMat{};
    t.offset = e.offset;
    t.tall = e.rows > e.cols;
    t.s = (int32_t)std::min(e.rows, e.cols);
    t.n = std::max(e.rows, e.cols);
    t.group = e.group;
    v[i].at = i;
    v[i].key = t.s <= 16 ? t.s : 0;
    if (v[i].key) cluster[v[i].key] = std::max(cluster[v[i].key], muon_cluster_simt(t, n_mats));
  }
  std::stable_sort(v.begin(), v.end(), [](const MuonOrder& a, const MuonOrder& b) {
    return a.key != b.key ? a.key < b.key : a.m.n > b.m.n;
  });
  std::vector<int64_t> n;   // of the tensor cores' matrices, which come first
  for (int32_t i = 0; i < n_mats && v[i].key == 0; ++i) n.push_back(v[i].m.n);
  if (!n.empty()) cluster[0] = muon_cluster_tc(n.data(), (int)n.size());
  for (MuonOrder& e : v) e.key += 32 * cluster[e.key];
  return v;
}

int32_t muon_run(const std::vector<MuonOrder>& v, int32_t at) {   // matrices of the launch at `at`
  int32_t n = 1;
  while (n < kMuonMatsPerLaunch && at + n < (int32_t)v.size() && v[at + n].key == v[at].key) ++n;
  return n;
}

// f(), or `bad` where the host's memory runs out: no exception leaves a C entry point.
template <typename R, typename F>
R no_throw(R bad, F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return bad;
  }
}

size_t muon_workspace(int32_t n_mats, const lora_mat* mats) {
  if (check_mats(n_mats, mats, nullptr) != LORA_OK) return 0;
  // the launches run one after the other and share the room for tiles that do not fit on chip
  const std::vector<MuonOrder> v = muon_order(n_mats, mats);
  size_t most = 0;
  for (int32_t at = 0; at < n_mats;) {
    const int32_t n = muon_run(v, at);
    most = std::max(most, muon_spill_bytes(v[at].m, v[at].key / 32, n));
    at += n;
  }
  return most + kWsAlign;
}

int muon_step(float* params, float* grads, float* m, int32_t n_groups, const lora_group* groups,
              int32_t n_mats, const lora_mat* mats, const lora_muon_hp* hp, const double* d_scale_norm,
              const int32_t* d_status, int32_t zero_grads, void* ws, size_t ws_bytes, void* stream) {
  if (!hp) return LORA_ERR_INVALID;
  if (!(hp->momentum >= 0.0 && hp->momentum < 1.0) || !std::isfinite(hp->weight_decay) ||
      !std::isfinite(hp->plus_ratio) || !std::isfinite(hp->coef[0]) ||
      !std::isfinite(hp->coef[1]) || !std::isfinite(hp->coef[2]) || hp->steps < 1 ||
      hp->steps > 8 || (hp->nesterov != 0 && hp->nesterov != 1) ||
      (hp->adjust != LORA_MUON_ADJUST_ASPECT && hp->adjust != LORA_MUON_ADJUST_RMS))
    return LORA_ERR_INVALID;
  GroupTab g;
  int rc = build_groups(n_groups, groups, g, nullptr);
  if (rc) return rc;
  if ((rc = check_mats(n_mats, mats, &g))) return rc;
  if (!params || !grads || !m || !d_scale_norm || !d_status || !ws) return LORA_ERR_INVALID;
  if (!al16(params) || !al16(grads) || !al16(m) || !al16(ws) ||
      (reinterpret_cast<uintptr_t>(d_scale_norm) & 7u) ||
      (reinterpret_cast<uintptr_t>(d_status) & 3u))
    return LORA_ERR_ALIGN;
  if (ws_bytes < muon_workspace(n_mats, mats)) return LORA_ERR_WORKSPACE;
  clear_stale();
  MuonK k;
  k.mu = (float)hp->momentum;
  k.a = (float)hp->coef[0]; k.b = (float)hp->coef[1]; k.c = (float)hp->coef[2];
  k.steps = hp->steps; k.nesterov = hp->nesterov;
  MuonTab tab;
  const std::vector<MuonOrder> v = muon_order(n_mats, mats);
  for (int32_t at = 0; at < n_mats;) {
    tab.n = muon_run(v, at);
    for (int32_t i = 0; i < tab.n; ++i) {
      const lora_mat& e = mats[v[at + i].at];
      MuonMat& t = tab.m[i];
      t = v[at + i].m;
      const double lr = g.lr[e.group];
      const double adj = hp->adjust == LORA_MUON_ADJUST_RMS
                             ? 0.2 * std::sqrt((double)t.n)
                             : std::sqrt(std::max(1.0, (double)e.rows / (double)e.cols));
      t.lr = (float)lr;
      t.decay = e.kind == LORA_KIND_A ? (float)hp->weight_decay : 0.f;
      t.step = (float)(lr * adj * (e.kind == LORA_KIND_B ? hp->plus_ratio : 1.0));
    }
    LORA_TRY(launch_muon(params, grads, m, tab, k, d_scale_norm, d_status, zero_grads != 0,
                         v[at].key / 32, Carve(ws).take<char>(1), (cudaStream_t)stream));
    at += tab.n;
  }
  return LORA_OK;
}

}  // namespace

extern "C" {

size_t lora_block_product_workspace_size(int64_t T, int64_t out_dim, int64_t in_dim,
                                         int32_t transposed) {
  if (check_product(T, out_dim, in_dim) != LORA_OK) return 0;
  return product_carve(T, transposed ? out_dim : in_dim, nullptr).bytes;
}

int lora_block_product(int64_t T, int64_t out_dim, int64_t in_dim, const void* X,
                       const uint8_t* W8, const float* sw, void* Y, int32_t transposed, void* ws,
                       size_t ws_bytes, void* stream) {
  int rc = check_product(T, out_dim, in_dim);
  if (rc) return rc;
  if (!X || !W8 || !sw || !Y || !ws) return LORA_ERR_INVALID;
  if (!al16(X) || !al16(W8) || !al16(sw) || !al16(Y) || !al16(ws)) return LORA_ERR_ALIGN;
  const ProductWs w = product_carve(T, transposed ? out_dim : in_dim, ws);
  if (ws_bytes < w.bytes) return LORA_ERR_WORKSPACE;
  if (T == 0) return LORA_OK;
  clear_stale();
  BlockProductArgs a{};
  a.T = T; a.out_dim = out_dim; a.in_dim = in_dim;
  a.W8 = W8; a.sw = sw; a.transposed = transposed != 0; a.Y = Y;
  a.codes = w.codes; a.scales = w.scales; a.ld_scales = block_scales_ld(T);
  a.X = X;
  return cuda_status(launch_block_product(a, (cudaStream_t)stream, 0));
}

int lora_block_quantize_weight(const void* W, int64_t out_dim, int64_t in_dim, uint8_t* W8,
                               float* sw, void* stream) {
  int rc = check_product(0, out_dim, in_dim);
  if (rc) return rc;
  if (!W || !W8 || !sw) return LORA_ERR_INVALID;
  if (!al16(W) || !al16(W8) || !al16(sw)) return LORA_ERR_ALIGN;
  clear_stale();
  return cuda_status(launch_block_quant_weight(W, out_dim, in_dim, W8, sw, (cudaStream_t)stream));
}

int lora_block_quantize(const void* src, int64_t rows, int64_t K, uint8_t* codes, float* scales,
                        void* stream) {
  if (rows < 0 || K <= 0 || !src || !codes || !scales) return LORA_ERR_INVALID;
  if (K % 16 || !al16(src) || !al16(codes) || !al16(scales)) return LORA_ERR_ALIGN;
  if (K > kMaxDim || rows >= kMaxTokens) return LORA_ERR_UNSUPPORTED;
  clear_stale();
  return cuda_status(launch_block_quant(src, rows, K, codes, scales,
                                        (K + LORA_SCALE_BLOCK - 1) / LORA_SCALE_BLOCK, 1,
                                        (cudaStream_t)stream));
}

int lora_norm_forward(const lora_norm_desc* d, int64_t T, const void* X, const float* gamma,
                      const float* beta, void* Y, float* stats, void* stream) {
  int rc = check_norm(d, T);
  if (rc) return rc;
  if (!X || !gamma || !Y || !stats || (beta && d->kind == LORA_NORM_RMS)) return LORA_ERR_INVALID;
  if (!al16(X) || !al16(gamma) || !al16(beta) || !al16(Y) || !al16(stats)) return LORA_ERR_ALIGN;
  if (T == 0) return LORA_OK;
  clear_stale();
  NormArgs a{};
  a.T = T; a.dim = d->dim; a.dtype = d->dtype; a.rms = d->kind == LORA_NORM_RMS; a.eps = d->eps;
  a.X = X; a.gamma = gamma; a.beta = beta; a.Y = Y; a.stats = stats;
  return cuda_status(launch_norm_forward(a, (cudaStream_t)stream));
}

size_t lora_norm_backward_workspace_size(const lora_norm_desc* d, int64_t T) {
  if (check_norm(d, T) != LORA_OK) return 0;
  return (size_t)norm_bwd_parts(d->dim, d->dtype, T) * 2 * d->dim * sizeof(float) + kWsAlign;
}

int lora_norm_backward(const lora_norm_desc* d, int64_t T, const void* X, const float* gamma,
                       const void* dY, const float* stats, const void* dX_add, void* dX,
                       float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_norm(d, T);
  if (rc) return rc;
  if (!X || !gamma || !dY || !stats || !ws) return LORA_ERR_INVALID;
  if ((!dX && !dgamma && !dbeta) || (dX_add && !dX) || (dbeta && d->kind == LORA_NORM_RMS))
    return LORA_ERR_INVALID;
  if (!al16(X) || !al16(gamma) || !al16(dY) || !al16(stats) || !al16(dX_add) || !al16(dX) ||
      !al16(dgamma) || !al16(dbeta) || !al16(ws))
    return LORA_ERR_ALIGN;
  if (ws_bytes < lora_norm_backward_workspace_size(d, T)) return LORA_ERR_WORKSPACE;
  if (T == 0) return LORA_OK;
  clear_stale();
  NormArgs a{};
  a.T = T; a.dim = d->dim; a.dtype = d->dtype; a.rms = d->kind == LORA_NORM_RMS;
  a.X = X; a.gamma = gamma; a.dY = dY; a.stats = const_cast<float*>(stats);
  a.dX_add = dX_add; a.dX = dX; a.dgamma = dgamma; a.dbeta = dbeta;
  a.part = Carve(ws).take<float>(1);
  return cuda_status(launch_norm_backward(a, (cudaStream_t)stream));
}

int lora_sum(int32_t n, const void* const* src, int64_t count, int32_t dtype, void* dst, void* stream) {
  if (n < 1 || !src || count < 0 || !dst || (dtype != LORA_F32 && dtype != LORA_BF16)) return LORA_ERR_INVALID;
  if (n > LORA_SUM_MAX || count >= kMaxElements) return LORA_ERR_UNSUPPORTED;
  SumArgs a{};
  for (int32_t k = 0; k < n; ++k) {
    if (!src[k]) return LORA_ERR_INVALID;
    if (!al16(src[k])) return LORA_ERR_ALIGN;
    a.src[k] = src[k];
  }
  if (!al16(dst) || count % 8) return LORA_ERR_ALIGN;
  if (count == 0) return LORA_OK;
  clear_stale();
  a.n = n; a.count = count; a.dtype = dtype; a.dst = dst;
  return cuda_status(launch_sum(a, (cudaStream_t)stream));
}

size_t lora_muon_workspace_size(int32_t n_mats, const lora_mat* mats) {
  return no_throw(size_t(0), [&] { return muon_workspace(n_mats, mats); });
}

int lora_muon_step(float* params, float* grads, float* m, int32_t n_groups,
                   const lora_group* groups, int32_t n_mats, const lora_mat* mats,
                   const lora_muon_hp* hp, const double* d_scale_norm, const int32_t* d_status,
                   int32_t zero_grads, void* ws, size_t ws_bytes, void* stream) {
  // the host's tables are made before anything is enqueued
  return no_throw<int>(LORA_ERR_UNSUPPORTED, [&] {
    return muon_step(params, grads, m, n_groups, groups, n_mats, mats, hp, d_scale_norm, d_status,
                     zero_grads, ws, ws_bytes, stream);
  });
}

}  // extern "C"
