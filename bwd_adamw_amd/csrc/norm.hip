// Entry points of the row norms (include/lora.h: lora_norm_forward,
// lora_norm_backward) and the choice of their kernels.
#include <math.h>
#include <string.h>

#include <cmath>

#include "host.hpp"
#include "launch.hpp"
#include "norm.hpp"

using namespace lora;
using namespace lora::host;

namespace {

// Lanes a row and 4-element groups a lane, by the width that they hold: one
// group a lane up to a wave's 256 elements, two or four in one wave up to 1024,
// then three to five in two, four or eight waves, so that the backward's five
// arrays of them stay in registers beside the loads in flight.  Past 10240
// elements eight waves hold eight groups each, the most that a block takes: of
// the backward's kernels those of four float32 gradients and of element loads
// spill there (44 and 68 bytes a lane), none elsewhere.
#define LORA_NORM_SHAPES(X) \
  X(16, 1) X(32, 1) X(64, 1) X(64, 2) X(64, 4) X(128, 3) X(128, 4) X(128, 5) X(256, 4) X(256, 5) \
  X(512, 4) X(512, 5) X(512, 8)
constexpr int64_t kNormMaxDim = 512 * 8 * 4;

int norm_tpr(int64_t dim) {
#define LORA_NORM_TPR(TPR_, V_) if (dim <= TPR_ * V_ * 4) return TPR_;
  LORA_NORM_SHAPES(LORA_NORM_TPR)
#undef LORA_NORM_TPR
  return 0;
}

struct NormGrid {
  int64_t blocks, rpb;
};
NormGrid norm_grid(int64_t rows, int64_t dim, int64_t cap) {
  const int tpr = norm_tpr(dim), nt = norm_threads(tpr), r = nt / tpr;
  const int64_t want = clampi(cdiv(rows, r), 1, cap * 256 / nt);
  const int64_t rpb = rup(cdiv(rows, want), r);
  return {cdiv(rows, rpb), rpb};
}
// Forward: eight blocks of 256 threads a CU at most.  Backward: two, since
// each block leaves a partial of dgamma and dbeta (4096 x 2560 float32: two
// partials of 10 KB a CU against 820 KB of rows).
constexpr int64_t kFwdBlocks = 8 * kCUs, kBwdBlocks = 2 * kCUs;

int check_norm(const lora_norm* n) {
  if (!n) return LORA_E_INVALID;
  if (n->rows <= 0 || n->dim <= 0 || n->dim > kNormMaxDim || n->ldx < n->dim || n->ldy < n->dim)
    return LORA_E_SHAPE;
  if (n->kind != LORA_NORM_LAYER && n->kind != LORA_NORM_RMS) return LORA_E_INVALID;
  if (n->dtype != LORA_F32 && n->dtype != LORA_BF16) return LORA_E_DTYPE;
  if (!(n->eps >= 0.0f) || !std::isfinite(n->eps)) return LORA_E_INVALID;
  if (((uintptr_t)n->gamma | (uintptr_t)n->beta) & 3u) return LORA_E_ALIGN;
  return LORA_OK;
}

bool al_elem(const lora_norm* n, const void* p) {
  return ((uintptr_t)p & (n->dtype == LORA_F32 ? 3u : 1u)) == 0;
}
// Rows that 4-element accesses can address (16 bytes of float32, 8 of bf16).
bool vec_rows(const lora_norm* n, const void* p, int64_t ld) {
  return ld % 4 == 0 && ((uintptr_t)p & (n->dtype == LORA_F32 ? 15u : 7u)) == 0;
}
bool vec_vector(const float* p) { return al16(p); }   // NULL included

NormArgs norm_args(const lora_norm* n, const void* X, const NormGrid& g) {
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.X = X;
  a.gamma = n->gamma;
  a.beta = n->kind == LORA_NORM_LAYER ? n->beta : nullptr;
  a.rows = n->rows;
  a.ldx = n->ldx;
  a.ldy = n->ldy;
  a.rpb = g.rpb;
  a.dim = (int)n->dim;
  a.layer = n->kind == LORA_NORM_LAYER;
  a.eps = n->eps;
  a.fdim = (float)n->dim;
  return a;
}

template <typename T, bool VEC>
void launch_fwd(const NormArgs& a, dim3 grid, hipStream_t st, const prof::Scope& ps) {
#define LORA_NORM_FWD(TPR_, V_)                                                          \
  if (a.dim <= TPR_ * V_ * 4) {                                                          \
    launch_n(norm_fwd_kernel<T, TPR_, V_, VEC>, grid, norm_threads(TPR_), st, ps, a);     \
    return;                                                                              \
  }
  LORA_NORM_SHAPES(LORA_NORM_FWD)
#undef LORA_NORM_FWD
}

template <typename T, bool VEC, int NDY>
void launch_bwd(const NormArgs& a, dim3 grid, hipStream_t st, const prof::Scope& ps) {
#define LORA_NORM_BWD(TPR_, V_)                                                          \
  if (a.dim <= TPR_ * V_ * 4) {                                                          \
    launch_n(norm_bwd_kernel<T, TPR_, V_, VEC, NDY>, grid, norm_threads(TPR_), st, ps, a); \
    return;                                                                              \
  }
  LORA_NORM_SHAPES(LORA_NORM_BWD)
#undef LORA_NORM_BWD
}
template <typename T>
void launch_bwd_n(bool vec, const NormArgs& a, dim3 grid, hipStream_t st, const prof::Scope& ps) {
  if (!vec) return launch_bwd<T, false, 0>(a, grid, st, ps);
  switch (a.ndy) {
    case 1: return launch_bwd<T, true, 1>(a, grid, st, ps);
    case 2: return launch_bwd<T, true, 2>(a, grid, st, ps);
    case 3: return launch_bwd<T, true, 3>(a, grid, st, ps);
    default: return launch_bwd<T, true, 4>(a, grid, st, ps);
  }
}

}  // namespace

extern "C" {

int lora_norm_forward(const lora_norm* norm, const void* X, void* Y, float* stats, void* stream) {
  const int rc = check_norm(norm);
  if (rc) return rc;
  if (!X || !Y) return LORA_E_INVALID;
  if (!al_elem(norm, X) || !al_elem(norm, Y) || ((uintptr_t)stats & 7u)) return LORA_E_ALIGN;
  const NormGrid g = norm_grid(norm->rows, norm->dim, kFwdBlocks);
  NormArgs a = norm_args(norm, X, g);
  a.out = Y;
  a.stats = stats;
  const bool vec = norm->dim % 4 == 0 && vec_rows(norm, X, norm->ldx) &&
                   vec_rows(norm, Y, norm->ldy) && vec_vector(a.gamma) && vec_vector(a.beta);
  const double e = norm->dtype == LORA_F32 ? 4.0 : 2.0;
  prof::Scope ps("norm_fwd", norm->rows, norm->dim, norm->kind, 8.0 * norm->rows * norm->dim,
                 2.0 * e * norm->rows * norm->dim + 8.0 * norm->rows + 8.0 * norm->dim);
  const dim3 grid((unsigned)g.blocks);
  hipStream_t st = (hipStream_t)stream;
  if (norm->dtype == LORA_F32) {
    if (vec) launch_fwd<float, true>(a, grid, st, ps);
    else launch_fwd<float, false>(a, grid, st, ps);
  } else {
    if (vec) launch_fwd<uint16_t, true>(a, grid, st, ps);
    else launch_fwd<uint16_t, false>(a, grid, st, ps);
  }
  return hip_status();
}

size_t lora_norm_workspace_bytes(const lora_norm* norm) {
  if (check_norm(norm) != LORA_OK) return 0;
  const NormGrid g = norm_grid(norm->rows, norm->dim, kBwdBlocks);
  return g.blocks > 1 ? (size_t)(g.blocks * 2 * norm->dim) * sizeof(float) : 0;
}

int lora_norm_backward(const lora_norm* norm, const void* X, int n_dy, const void* const* dY,
                       const float* stats, void* dX, float* dgamma, float* dbeta, int accumulate,
                       void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_norm(norm);
  if (rc) return rc;
  if (!X || !stats || !dY || n_dy < 1 || n_dy > LORA_MAX_GROUP) return LORA_E_INVALID;
  if (!dX && !dgamma && !dbeta) return LORA_E_INVALID;
  if (dbeta && norm->kind != LORA_NORM_LAYER) return LORA_E_INVALID;
  if (!al_elem(norm, X) || (dX && !al_elem(norm, dX)) || ((uintptr_t)stats & 7u) ||
      (((uintptr_t)dgamma | (uintptr_t)dbeta) & 3u))
    return LORA_E_ALIGN;
  for (int i = 0; i < n_dy; ++i) {
    if (!dY[i]) return LORA_E_INVALID;
    if (!al_elem(norm, dY[i])) return LORA_E_ALIGN;
  }
  const bool sums = dgamma || dbeta;
  const size_t need = sums ? lora_norm_workspace_bytes(norm) : 0;
  if (need && (!ws || ws_bytes < need || ((uintptr_t)ws & 15u))) return LORA_E_WORKSPACE;
  const NormGrid g = norm_grid(norm->rows, norm->dim, kBwdBlocks);
  NormArgs a = norm_args(norm, X, g);
  bool vec = norm->dim % 4 == 0 && vec_rows(norm, X, norm->ldx) && vec_vector(a.gamma) &&
             (!dX || vec_rows(norm, dX, norm->ldx));
  for (int i = 0; i < n_dy; ++i) {
    a.dY[i] = dY[i];
    vec = vec && vec_rows(norm, dY[i], norm->ldy);
  }
  a.ndy = n_dy;
  a.out = dX;
  a.stats = const_cast<float*>(stats);
  a.part = (float*)ws;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.accumulate = accumulate ? 1 : 0;
  const double e = norm->dtype == LORA_F32 ? 4.0 : 2.0;
  hipStream_t st = (hipStream_t)stream;
  {
    prof::Scope ps("norm_bwd", norm->rows, norm->dim, n_dy, 14.0 * norm->rows * norm->dim,
                   e * norm->rows * norm->dim * (1 + n_dy + (dX ? 1 : 0)) + 8.0 * norm->rows +
                       (sums ? 8.0 * g.blocks * norm->dim : 0.0));
    const dim3 grid((unsigned)g.blocks);
    if (norm->dtype == LORA_F32) launch_bwd_n<float>(vec, a, grid, st, ps);
    else launch_bwd_n<uint16_t>(vec, a, grid, st, ps);
  }
  if (sums && g.blocks > 1) {
    prof::Scope ps("norm_finish", g.blocks, norm->dim, 1, 0.0, 8.0 * g.blocks * norm->dim);
    launch_n(norm_finish_kernel, dim3((unsigned)cdiv(norm->dim, 32), dbeta ? 2u : 1u), 1024u, st, ps,
             (const float*)ws, (int)g.blocks, (int)norm->dim, dgamma, dbeta, a.accumulate);
  }
  return hip_status();
}

}  // extern "C"
