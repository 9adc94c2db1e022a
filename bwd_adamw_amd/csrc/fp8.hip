// Entry points of the 8-bit block-scaled products (include/lora.h:
// lora_fp8_quantize, lora_fp8_product) and the plan of their launches.
#include <string.h>

#include <algorithm>

#include "fp8.hpp"
#include "host.hpp"
#include "launch.hpp"

using namespace lora;
using namespace lora::host;

namespace {

// Tiles: tokens, columns, wave grid, stages in LDS (130, 66 and 63 KB of
// them), blocks a CU holds, and the time of one contraction step of a CU's
// resident blocks and of a block's ends, in microseconds, fitted to all three
// on the Qwen3-4B-shaped products at 512 to 4096 tokens.  4096 tokens of
// [2560 -> 4096] forward: 71, 82 and 129 us; 512 of them 35, 29 and 19; 1000
// of [2056 -> 1368] 30, 25 and 16.
struct Fp8Cfg {
  int bm, bn, per_cu;
  double step, ends;
};
#define LORA_FP8_CFGS(X)                          \
  X(0, 256, 256, 2, 4, 2, 1, 2.9, 16.0)           \
  X(1, 128, 128, 2, 2, 2, 2, 1.88, 4.5)           \
  X(2, 32, 128, 1, 4, 3, 2, 0.73, 4.7)
constexpr Fp8Cfg kCfg[] = {
#define LORA_FP8_ROW(i, bm, bn, wm, wn, ns, pc, st, en) {bm, bn, pc, st, en},
    LORA_FP8_CFGS(LORA_FP8_ROW)
#undef LORA_FP8_ROW
};

constexpr int kNCfg = sizeof(kCfg) / sizeof(kCfg[0]);

struct Fp8Plan {
  int cfg, per, nsplit;
  double t;          // microseconds
};
// Rounds of a CU's blocks: all but the first start under the last one's end.
double round_time(const Fp8Cfg& c, int64_t rounds, int steps) {
  return c.ends + rounds * (steps * c.step) + (rounds - 1) * 1.0;
}
// most: the largest number of splits.
Fp8Plan plan(int64_t M, int64_t Nc, int nk, int most = 16) {
  Fp8Plan best = {0, nk, 1, 1e30};
  for (int i = 0; i < kNCfg; ++i) {
    const Fp8Cfg& c = kCfg[i];
    const int64_t tiles = cdiv(M, c.bm) * cdiv(Nc, c.bn);
    for (int want = 1; want <= std::min(nk, most); ++want) {
      const int per = (int)cdiv(nk, want), n = (int)cdiv(nk, per);
      if (n != want) continue;
      double t = round_time(c, cdiv(tiles * n, kCUs * c.per_cu), per);
      // Split partials: written, read, and summed by a launch of its own.
      if (n > 1) t += 2.5 + 4.0 * M * Nc * (1.6 * n) / 5e6;
      if (t < best.t) best = {i, per, n, t};
    }
  }
  return best;
}

// Columns that run first, as whole rounds of the largest tile, when the rest
// in a launch of their own is faster than a last, partly filled round (4096
// tokens of [2560 -> 9728]: two rounds and 1536 columns instead of three
// rounds, 192 -> 173 us); 0: all in one.
int64_t whole_rounds(const Fp8Plan& g, int64_t M, int64_t Nc, int nk) {
  const Fp8Cfg& c = kCfg[0];
  const int64_t ntm = cdiv(M, c.bm), full = ntm * cdiv(Nc, c.bn) / kCUs;
  const int64_t cols = full * kCUs / ntm * c.bn;
  if (g.nsplit != 1 || full < 1 || cols >= Nc) return 0;
  const double two = round_time(c, full, nk) + plan(M, Nc - cols, nk, 1).t + 3.0;
  return two < g.t ? cols : 0;
}

template <bool DX, int OUT>
void launch_gemm(int cfg, const Fp8Args& a, dim3 grid, hipStream_t st, const prof::Scope& ps) {
#define LORA_FP8_LAUNCH(i, bm, bn, wm, wn, ns, pc, s_, e_) \
  if (cfg == i)                                            \
    return launch_n(fp8_gemm_kernel<bm, bn, wm, wn, ns, DX, OUT>, grid, 64u * wm * wn, st, ps, a);
  LORA_FP8_CFGS(LORA_FP8_LAUNCH)
#undef LORA_FP8_LAUNCH
}

int check_fp8(const lora_fp8_operand* x, int64_t N, int64_t K, int dx) {
  if (!x) return LORA_E_INVALID;
  if (x->rows <= 0 || x->cols <= 0 || N <= 0 || K <= 0) return LORA_E_SHAPE;
  if (x->cols != (dx ? N : K)) return LORA_E_SHAPE;
  if (!lora_fp8_weight_layout(N, K, nullptr) ||
      !lora_fp8_operand_layout(x->rows, x->cols, nullptr))
    return LORA_E_SHAPE;
  return LORA_OK;
}

// Few tokens, forward: up to one tile of 16 run without stages or splits, in
// one launch.  [2560 -> 9728]: 16 tokens 9.5 us, where 17 take 10.7 on the
// 32-token tile with its split sums; one token 6.6.
constexpr int64_t kFewTokens = 16;
bool few(int64_t M, bool dx) { return !dx && M <= kFewTokens; }

// Everything but the output and the split of a product.
Fp8Args product_args(const void* x, int64_t rows, const void* W, int64_t N, int64_t K, bool dx) {
  Fp8Args a;
  memset(&a, 0, sizeof(a));
  a.M = rows;
  a.Nc = a.ldc = dx ? K : N;
  a.nk = (int)cdiv(dx ? N : K, 128);
  a.ldq = (int64_t)a.nk * 128;
  a.lde = rup(rows, 128);
  a.Q = (const uint8_t*)x;
  a.E = a.Q + rup(rows * a.ldq, 256);
  a.ldw = rup(K, 128);
  a.W = (const uint8_t*)W;
  a.S = (const float*)(a.W + rup(N, 128) * a.ldw);
  a.lds_ = a.ldw / 128;
  return a;
}

void quantize(const void* X, int dtype, int64_t ldx, int64_t rows, int64_t cols, void* data,
              hipStream_t st) {
  Fp8QuantArgs a;
  a.X = X;
  a.Q = (uint8_t*)data;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldq = rup(cols, 128);
  a.lde = rup(rows, 128);
  a.E = a.Q + rup(rows * a.ldq, 256);
  const int64_t unit = dtype == LORA_F32 ? 4 : 8;   // elements of a 16-byte load
  const bool vec = al16(X) && ldx % unit == 0 && cols % unit == 0;
  const double e = dtype == LORA_F32 ? 4.0 : 2.0;
  prof::Scope ps("fp8_quant", rows, cols, 1, 3.0 * rows * cols, (e + 1.0) * rows * cols);
  const dim3 grid((unsigned)cdiv(rows * (a.ldq / 128), 16));
  if (dtype == LORA_F32) {
    if (vec) launch(fp8_quant_kernel<float, true>, grid, st, ps, a);
    else launch(fp8_quant_kernel<float, false>, grid, st, ps, a);
  } else {
    if (vec) launch(fp8_quant_kernel<uint16_t, true>, grid, st, ps, a);
    else launch(fp8_quant_kernel<uint16_t, false>, grid, st, ps, a);
  }
}

}  // namespace

namespace lora {

size_t fp8_operand_bytes(int64_t rows, int64_t cols) {
  return lora_fp8_operand_layout(rows, cols, nullptr);
}

void fp8_launch_quantize(const float* X, int64_t rows, int64_t cols, void* data, hipStream_t st) {
  quantize(X, LORA_F32, cols, rows, cols, data, st);
}

void fp8_launch_lora_product(const void* x, int64_t rows, const void* W, int64_t N, int64_t K,
                             bool dx, const Fp8Lora& l, float* out, float* out2, hipStream_t st) {
  Fp8Args a = product_args(x, rows, W, N, K, dx);
  // One block sums the whole contraction: the LoRA term joins it there.
  const Fp8Plan g = plan(a.M, a.Nc, a.nk, 1);
  a.per = a.nk;
  a.nsplit = 1;
  a.C = out;
  a.C2 = out2;
  a.lora = l;
  const Fp8Cfg& c = kCfg[g.cfg];
  const int64_t Kc = dx ? N : K;
  prof::Scope ps(dx ? "fp8_gemm_dx" : "fp8_gemm_fwd", a.M, a.Nc, Kc,
                 2.0 * a.M * a.Nc * (Kc + l.r),
                 (double)a.M * a.ldq + (double)N * K + 4.0 * a.M * a.Nc * (out2 ? 2 : 1));
  const dim3 grid((unsigned)(cdiv(a.M, c.bm) * cdiv(a.Nc, c.bn)));
  if (dx) launch_gemm<true, 3>(g.cfg, a, grid, st, ps);
  else launch_gemm<false, 3>(g.cfg, a, grid, st, ps);
}

}  // namespace lora

extern "C" {

size_t lora_fp8_weight_layout(int64_t out_dim, int64_t in_dim, size_t* scale_offset) {
  if (out_dim <= 0 || in_dim <= 0 || out_dim > (1 << 30) || in_dim > (1 << 30)) return 0;
  const int64_t np = rup(out_dim, 128), kp = rup(in_dim, 128);
  if (np * kp >= (1ll << 31)) return 0;
  if (scale_offset) *scale_offset = (size_t)(np * kp);
  return (size_t)(np * kp + (np / 128) * (kp / 128) * 4);
}

size_t lora_fp8_operand_layout(int64_t rows, int64_t cols, size_t* scale_offset) {
  if (rows <= 0 || cols <= 0 || cols > (1 << 22) || rows > (1 << 30)) return 0;
  // The exponents are addressed with 32-bit offsets.
  if (rup(rows, 128) * cdiv(cols, 128) >= (1ll << 31)) return 0;
  const size_t q = (size_t)(rows * rup(cols, 128));
  const size_t off = (size_t)rup((int64_t)q, 256);
  if (scale_offset) *scale_offset = off;
  return off + (size_t)rup(rup(rows, 128) * cdiv(cols, 128), 256);
}

int lora_fp8_quantize(const void* X, int dtype, int64_t ldx, const lora_fp8_operand* out,
                      void* stream) {
  if (!out) return LORA_E_INVALID;
  if (!lora_fp8_operand_layout(out->rows, out->cols, nullptr) || ldx < out->cols) return LORA_E_SHAPE;
  if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_E_DTYPE;
  if (!X || !out->data) return LORA_E_INVALID;
  if (!al16(out->data) || ((uintptr_t)X & (dtype == LORA_F32 ? 3u : 1u))) return LORA_E_ALIGN;
  if (cdiv(out->rows * (rup(out->cols, 128) / 128), 16) > 0x7fffffffll) return LORA_E_SHAPE;
  quantize(X, dtype, ldx, out->rows, out->cols, out->data, (hipStream_t)stream);
  return hip_status();
}

size_t lora_fp8_product_workspace_bytes(const lora_fp8_operand* x, int64_t out_dim, int64_t in_dim,
                                        int dx) {
  if (check_fp8(x, out_dim, in_dim, dx) != LORA_OK) return 0;
  const int64_t Nc = dx ? in_dim : out_dim;
  if (few(x->rows, dx)) return 0;
  const Fp8Plan g = plan(x->rows, Nc, (int)cdiv(x->cols, 128));
  return g.nsplit > 1 ? sizeof(float) * (size_t)(g.nsplit * x->rows * Nc) : 0;
}

int lora_fp8_product(const lora_fp8_operand* x, const void* W, int64_t out_dim, int64_t in_dim,
                     int dx, void* out, int out_dtype, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_fp8(x, out_dim, in_dim, dx);
  if (rc) return rc;
  if (out_dtype != LORA_F32 && out_dtype != LORA_BF16) return LORA_E_DTYPE;
  if (!x->data || !W || !out) return LORA_E_INVALID;
  if (!al16(x->data) || !al16(W) || !al16(out)) return LORA_E_ALIGN;
  Fp8Args a = product_args(x->data, x->rows, W, out_dim, in_dim, dx != 0);
  if (few(a.M, dx)) {
    a.C = out;
    const bool bf = out_dtype == LORA_BF16;
    prof::Scope ps("fp8_few_fwd", a.M, a.Nc, x->cols, 2.0 * a.M * a.Nc * x->cols,
                   (double)a.M * a.ldq + (double)out_dim * in_dim + (bf ? 2.0 : 4.0) * a.M * a.Nc);
    const dim3 grid((unsigned)cdiv(a.Nc, 16));
    hipStream_t st = (hipStream_t)stream;
    if (bf) launch_n(fp8_few_kernel<true>, grid, 512u, st, ps, a);
    else launch_n(fp8_few_kernel<false>, grid, 512u, st, ps, a);
    return hip_status();
  }
  const Fp8Plan g = plan(a.M, a.Nc, a.nk);
  const size_t need = lora_fp8_product_workspace_bytes(x, out_dim, in_dim, dx);
  if (need && (!ws || ws_bytes < need || !al16(ws))) return LORA_E_WORKSPACE;
  a.C = out;
  a.part = (float*)ws;
  a.per = g.per;
  a.nsplit = g.nsplit;
  if (cdiv(a.M, 32) * cdiv(a.Nc, 128) > 0x7fffffffll / g.nsplit) return LORA_E_SHAPE;
  hipStream_t st = (hipStream_t)stream;
  const double eo = out_dtype == LORA_F32 ? 4.0 : 2.0;
  const int o = g.nsplit > 1 ? 2 : out_dtype == LORA_BF16 ? 1 : 0;
  auto product = [&](const Fp8Args& q, int cfg) {
    const Fp8Cfg& c = kCfg[cfg];
    prof::Scope ps(dx ? "fp8_gemm_dx" : "fp8_gemm_fwd", q.M, q.Nc, x->cols, 2.0 * q.M * q.Nc * x->cols,
                   (double)q.M * q.ldq + (double)q.Nc * x->cols +
                       (g.nsplit > 1 ? 4.0 * g.nsplit : eo) * q.M * q.Nc);
    const dim3 grid((unsigned)(cdiv(q.M, c.bm) * cdiv(q.Nc, c.bn) * q.nsplit));
    if (dx) {
      if (o == 0) launch_gemm<true, 0>(cfg, q, grid, st, ps);
      else if (o == 1) launch_gemm<true, 1>(cfg, q, grid, st, ps);
      else launch_gemm<true, 2>(cfg, q, grid, st, ps);
    } else {
      if (o == 0) launch_gemm<false, 0>(cfg, q, grid, st, ps);
      else if (o == 1) launch_gemm<false, 1>(cfg, q, grid, st, ps);
      else launch_gemm<false, 2>(cfg, q, grid, st, ps);
    }
  };
  const int64_t first = whole_rounds(g, a.M, a.Nc, a.nk);
  if (first) {
    Fp8Args q = a;
    q.Nc = first;
    product(q, 0);
    q.Nc = a.Nc - first;
    q.W += dx ? first : first * a.ldw;
    q.S += dx ? first / 128 : first / 128 * a.lds_;
    q.C = (char*)a.C + (size_t)(eo * first);
    product(q, plan(q.M, q.Nc, q.nk, 1).cfg);
  } else {
    product(a, g.cfg);
  }
  if (g.nsplit > 1) {
    const int64_t n = a.M * a.Nc;
    prof::Scope ps("fp8_reduce", a.M, a.Nc, g.nsplit, 0.0, (4.0 * g.nsplit + eo) * n);
    const dim3 rg((unsigned)cdiv(n, 1024));
    if (out_dtype == LORA_BF16) launch(fp8_reduce_kernel<true>, rg, st, ps, (const float*)ws, n, g.nsplit, out);
    else launch(fp8_reduce_kernel<false>, rg, st, ps, (const float*)ws, n, g.nsplit, out);
  }
  return hip_status();
}

}  // extern "C"
