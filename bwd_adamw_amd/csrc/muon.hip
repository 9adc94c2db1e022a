// Entry points of the orthogonalised update (include/lora.h:
// lora_orthogonalize, lora_muon_step) and the plan of their launches.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "host.hpp"
#include "launch.hpp"
#include "muon.hpp"

using namespace lora;
using namespace lora::host;

static_assert(LORA_MAX_RUNS == MUON_MAX_RUNS, "matrix runs of one call");

namespace {

// Short side, padded to the fragments' 16.
int muon_rp(int64_t r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
int64_t tiles(int rp) { return (int64_t)(rp / 16) * (rp / 16 + 1) / 2; }

struct Class {          // the runs of one padded short side
  MuonArgs a;
  int64_t blocks, mats;
  double elems, flops;
  bool vec;
  size_t part, poly, mem, bytes;
  bool small;
};

int check_runs(const lora_matrix_run* runs, int n) {
  if (!runs || n < 1 || n > LORA_MAX_RUNS) return LORA_E_INVALID;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    const lora_matrix_run& r = runs[i];
    if (r.rows <= 0 || r.cols <= 0 || r.count <= 0 || std::min(r.rows, r.cols) > 128 ||
        std::max(r.rows, r.cols) > (1ll << 22) || r.count > (1 << 20))
      return LORA_E_SHAPE;
    if (r.offset < 0 || (r.count > 1 && r.stride < r.rows * r.cols)) return LORA_E_INVALID;
    if (r.kind != 0 && r.kind != 1) return LORA_E_INVALID;
    total += r.count;
  }
  return total > (1 << 20) ? LORA_E_SHAPE : LORA_OK;
}

int check_hparams(const lora_muon_hparams* h) {
  if (!h) return LORA_E_INVALID;
  if (h->steps < 1 || h->steps > 10) return LORA_E_INVALID;
  if (h->adjust != LORA_MUON_SHAPE && h->adjust != LORA_MUON_RMS) return LORA_E_INVALID;
  if (!(h->eps >= 0.0) || !(h->momentum >= 0.0 && h->momentum < 1.0)) return LORA_E_INVALID;
  for (double v : {h->lr, h->weight_decay, h->plus_ratio, h->eps, h->a, h->b, h->c})
    if (!std::isfinite(v)) return LORA_E_INVALID;
  return LORA_OK;
}

// Blocks: one round of what the CUs hold when there are matrices enough for
// it, each over a range of whole 64-index tiles, at least two (more blocks
// would shorten the other launches less than they lengthen the sums of their
// partials: 36 x [64, 2560], 20 ranges instead of 14: 82 -> 90 us).
int64_t muon_blocks(int rp) { return kCUs * (rp == 128 ? muon_per_cu<128>() : muon_per_cu<64>()); }
constexpr int64_t kMuonMinLen = 128;

// Short sides up to 16 with long sides up to this run whole in one block: one
// CU's float64 MFMA takes 3.3 us for each 1024 of them (both products), which
// from about here on costs more than the launch saved.
constexpr int64_t kMuonSmallLen = 512;

bool plan_class(const lora_matrix_run* runs, int n, int rp, const lora_muon_hparams* h, Class& c) {
  memset(&c, 0, sizeof(c));
  c.vec = true;
  c.small = rp == 16;
  for (int i = 0; i < n; ++i)
    if (muon_rp(std::min(runs[i].rows, runs[i].cols)) == rp) c.mats += runs[i].count;
  if (!c.mats) return false;
  const int64_t want = std::max<int64_t>(1, muon_blocks(rp) / c.mats);
  int64_t mat = 0, blk = 0;
  for (int i = 0; i < n; ++i) {
    const lora_matrix_run& s = runs[i];
    if (muon_rp(std::min(s.rows, s.cols)) != rp) continue;
    MuonRun& r = c.a.run[c.a.nruns++];
    const int64_t L = std::max(s.rows, s.cols), R = std::min(s.rows, s.cols);
    const int64_t sp = clampi(want, 1, cdiv(L, kMuonMinLen));
    r.offset = s.offset;
    r.stride = s.stride;
    r.rows = (int32_t)s.rows;
    r.cols = (int32_t)s.cols;
    r.count = (int32_t)s.count;
    r.len = (int32_t)rup(cdiv(L, sp), 64);
    r.splits = (int32_t)cdiv(L, r.len);
    r.mat0 = (int32_t)mat;
    r.blk0 = (int32_t)blk;
    mat += s.count;
    blk += s.count * r.splits;
    if (h) {
      const double f = h->adjust == LORA_MUON_RMS ? 0.2 * sqrt((double)L)
                                                  : sqrt(std::max(1.0, (double)s.rows / s.cols));
      r.rate = (float)(h->lr * f * (s.kind == 1 ? h->plus_ratio : 1.0));
      r.decay = s.kind == 0 ? (float)(h->lr * h->weight_decay) : 0.0f;
    }
    c.small = c.small && L <= kMuonSmallLen;
    c.elems += (double)s.count * s.rows * s.cols;
    c.flops += (double)s.count * s.rows * s.cols * R;
    c.vec = c.vec && s.cols % 4 == 0 && s.offset % 4 == 0 && (s.count == 1 || s.stride % 4 == 0);
  }
  c.blocks = blk;
  size_t off = 0;
  c.part = off;
  off += (size_t)rup(blk * tiles(rp) * 64 * 32, 256);
  c.poly = off;
  if (rp > 16) off += (size_t)rup(mat * rp * rp * 8, 256);
  c.mem = off;
  if (rp == 128) off += (size_t)(mat * PolyMem<128>::BYTES);
  c.bytes = off;
  return true;
}

template <int RP, bool VEC, bool MUON>
void launch_class(const Class& c, char* ws, hipStream_t st) {
  const double e = 4.0 * c.elems, part = 32.0 * 64 * tiles(RP) * c.blocks;
  if constexpr (RP == 16) {
    if (c.small) {
      prof::Scope ps("muon_small", c.mats, RP, c.a.steps, 3.0 * c.flops, (MUON ? 5 : 2) * e);
      launch_n(muon_small_kernel<RP, VEC, MUON>, dim3((unsigned)c.mats), 1024u, st, ps, c.a);
      return;
    }
  }
  if constexpr (RP == 128 && MUON) {
    prof::Scope ps("muon_momentum", c.mats, RP, c.blocks, 0.0, 3 * e);
    launch(muon_momentum_kernel<VEC>, dim3((unsigned)c.blocks), st, ps, c.a);
  }
  {
    prof::Scope ps("muon_gram", c.mats, RP, c.blocks, c.flops, (MUON ? 3 : 1) * e + part);
    launch(muon_gram_kernel<RP, VEC, MUON>, dim3((unsigned)c.blocks), st, ps, c.a);
  }
  if constexpr (RP == 128) {
    char* mem = ws + c.mem;
    {
      prof::Scope ps("muon_assemble", c.mats, RP, c.blocks, 0.0, part);
      launch(muon_assemble_kernel<RP>, dim3((unsigned)(c.mats * tiles(RP) / 4)), st, ps, c.a, mem);
    }
    for (int k = 0; k < c.a.steps; ++k) {
      const bool last = k + 1 == c.a.steps;
      for (int phase = 0; phase < 3; ++phase) {
        if (last && (phase == 2 || (phase == 1 && k == 0))) continue;
        const int64_t n = c.mats * tiles(RP) * (phase == 1 && k > 0 && !last ? 2 : 1);
        prof::Scope ps("muon_product", c.mats, RP, phase, 2.0 * 256 * RP * n, 24.0 * 256 * n);
        launch(muon_product_kernel<RP>, dim3((unsigned)(n / 4)), st, ps, c.a, mem, phase, k);
      }
    }
  } else if constexpr (RP > 16) {   // at 16 the apply pass iterates it
    prof::Scope ps("muon_poly", c.mats, RP, c.a.steps, 8.0 * c.a.steps * c.mats * RP * RP * RP,
                   part + 8.0 * c.mats * RP * RP);
    launch_n(muon_poly_kernel<RP>, dim3((unsigned)c.mats), 64u * poly_nw<RP>(), st, ps, c.a);
  }
  prof::Scope ps("muon_apply", c.mats, RP, c.blocks, 2.0 * c.flops,
                 (MUON ? 4 : 2) * e + 8.0 * c.blocks * RP * RP);
  launch(muon_apply_kernel<RP, VEC, MUON>, dim3((unsigned)c.blocks), st, ps, c.a);
}
template <bool MUON>
void launch_rp(int rp, const Class& c, char* ws, hipStream_t st) {
#define LORA_MUON_RP(RP_)                                       \
  if (rp == RP_) {                                              \
    if (c.vec) launch_class<RP_, true, MUON>(c, ws, st);        \
    else launch_class<RP_, false, MUON>(c, ws, st);             \
  }
  LORA_MUON_RP(16) LORA_MUON_RP(32) LORA_MUON_RP(64) LORA_MUON_RP(128)
#undef LORA_MUON_RP
}

int run_all(const lora_matrix_run* runs, int n, const lora_muon_hparams* h, const float* G,
            float* M, float* P, const float* d_scale, void* ws, size_t ws_bytes, void* stream) {
  const size_t need = lora_muon_workspace_bytes(runs, n);
  if (!ws || ws_bytes < need) return LORA_E_WORKSPACE;
  if (!al16(ws)) return LORA_E_ALIGN;
  for (int rp = 16; rp <= 128; rp *= 2) {
    Class c;
    if (!plan_class(runs, n, rp, h, c)) continue;
    c.a.G = G;
    c.a.M = M;
    c.a.P = P;
    c.a.d_scale = d_scale;
    c.a.part = (double*)((char*)ws + c.part);
    c.a.poly = (double*)((char*)ws + c.poly);
    c.a.mu = (float)h->momentum;
    c.a.nesterov = h->nesterov ? 1 : 0;
    c.a.steps = h->steps;
    c.a.eps = h->eps;
    c.a.a = h->a;
    c.a.b = h->b;
    c.a.c = h->c;
    if (M) launch_rp<true>(rp, c, (char*)ws, (hipStream_t)stream);
    else launch_rp<false>(rp, c, (char*)ws, (hipStream_t)stream);
  }
  return hip_status();
}

}  // namespace

extern "C" {

size_t lora_muon_workspace_bytes(const lora_matrix_run* runs, int n) {
  if (check_runs(runs, n) != LORA_OK) return 0;
  size_t most = 0;   // the classes run one after another
  for (int rp = 16; rp <= 128; rp *= 2) {
    Class c;
    if (plan_class(runs, n, rp, nullptr, c)) most = std::max(most, c.bytes);
  }
  return most;
}

int lora_orthogonalize(const float* G, float* O, const lora_matrix_run* runs, int n,
                       const lora_muon_hparams* hp, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_runs(runs, n);
  if (!rc) rc = check_hparams(hp);
  if (rc) return rc;
  if (!G || !O) return LORA_E_INVALID;
  if (!al16(G) || !al16(O)) return LORA_E_ALIGN;
  return run_all(runs, n, hp, G, nullptr, O, nullptr, ws, ws_bytes, stream);
}

int lora_muon_step(float* params, const float* grads, float* m, const lora_matrix_run* runs, int n,
                   const lora_muon_hparams* hp, const float* d_scale, void* ws, size_t ws_bytes,
                   void* stream) {
  int rc = check_runs(runs, n);
  if (!rc) rc = check_hparams(hp);
  if (rc) return rc;
  if (!params || !grads || !m || !d_scale) return LORA_E_INVALID;
  if (!al16(params) || !al16(grads) || !al16(m)) return LORA_E_ALIGN;
  if ((uintptr_t)d_scale & 3u) return LORA_E_ALIGN;
  return run_all(runs, n, hp, grads, m, params, d_scale, ws, ws_bytes, stream);
}

}  // extern "C"
