// Newton-Schulz orthogonalisation of matrices with one short side, and the
// momentum update that uses it.
//
// With X_0 = u / (||u||_F + eps) and R the short side, a step is
//   X_{k+1} = Q_k X_k,  Q_k = a I + b G_k + c G_k^2,  G_k = X_k X_k^T  (R x R).
// Every Q_k is a polynomial of G_0, so all of them commute and
//   X_n = P X_0,  P = Q_{n-1} ... Q_0,   G_{k+1} = Q_k G_k Q_k:
// the iteration needs the data only for G_0 and for the last product.  (A
// tall matrix is the transpose: G_0 = X^T X, X_n = X P.)  Three launches:
//   gram   u from the gradient and the momentum (which it updates), and the
//          upper half of u u^T by blocks of columns; reads g, m, writes m
//   poly   one block a matrix (at R > 64 a launch a product): sums the blocks'
//          partials in order, takes the norm from the trace, iterates Q and G,
//          leaves P; up to R 16 the apply blocks do it themselves
//   apply  P u and the parameter update; reads g, m, p, writes p
// against the 2 n passes over X of the iteration as written.
//
// The products run on float64 MFMA (16x16x4).  P reaches a^n (485 for the
// usual a and five steps) where a singular value is small, and an error e of
// G_0 there becomes P e X: with float32 sums of G a spectrum wider than 1e3
// would lose all but three digits.  In float64 the results are as accurate as
// the float32 data, and up to R = 64 the two passes still cost less MFMA time
// (2 R flops an element in the second, 5/8 of that in the first by symmetry)
// than memory time; at 128 about as much.  Measured for 72 x [9728, 64]: gram
// 110 us (543 MB, 4.9 TB/s), poly 38, apply 155 (724 MB, 4.7 TB/s); wide
// matrices, whose rows are read in 64-byte pieces, 20 % slower.
//
// Fragments: a 16x16x4 operand is row l % 16 and contraction index l / 16 of
// lane l, the same for both sides of a symmetric product, so one load serves
// both.  Which element a lane calls its "row" and which contraction index a
// lane group takes is free as long as the sides agree: wide matrices take
// four neighbouring columns a lane (16-byte loads), tall ones RP / 16
// neighbouring columns a lane as RP / 16 fragments.  The result's row is
// 4 v + l / 16 for value v (not 4 (l / 16) + v as in float32).
#pragma once
#include "common.hpp"

namespace lora {

typedef double f64x4 __attribute__((ext_vector_type(4)));
LORA_DEV f64x4 mfma16x16x4_f64(double a, double b, f64x4 c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

constexpr int MUON_MAX_RUNS = 32;
struct MuonRun {
  int64_t offset, stride;    // first matrix, elements between matrices
  int32_t rows, cols, count;
  int32_t splits;            // blocks a matrix (gram and apply)
  int32_t len;               // long-side length of a block's range
  int32_t mat0;              // index of its first matrix among the call's
  int32_t blk0;              // first block
  float rate, decay;         // lr factor, lr weight decay
};
struct MuonArgs {
  MuonRun run[MUON_MAX_RUNS];
  int nruns;
  const float* G;        // gradient arena
  float* M;              // momentum arena (NULL: orthogonalise G alone)
  float* P;              // parameter arena, or the result of an orthogonalisation
  const float* d_scale;  // or NULL
  double* part;          // [block][tiles][64][4]
  double* poly;          // [matrix][RP][RP], RP above 16
  float mu;
  int nesterov;
  int steps;
  double eps, a, b, c;
};

// The run that block (or, by `mats`, matrix) index b falls in.
LORA_DEV int muon_find(const MuonArgs& p, int b, bool mats) {
  int r = 0;
  for (int i = 1; i < p.nruns; ++i)
    if ((mats ? p.run[i].mat0 : p.run[i].blk0) <= b) r = i;
  return __builtin_amdgcn_readfirstlane(r);
}

LORA_DEV bool muon_vetoed(const MuonArgs& p) {
  return p.d_scale && !(fabsf(*p.d_scale) <= 3.402823466e38f);
}

// N (1, 2 or 4) neighbouring values at element `at` of a matrix (under 2^30
// elements: a scalar base and a 32-bit byte offset), of which the first n
// exist; the others hold values of the matrix's first elements, for the caller
// to mask when it uses them (maskn).  Every load is unconditional and nothing
// looks at its result here: a guarded load becomes a branch, at whose end the
// compiler waits for all loads in flight, and a select waits at once.
template <bool VEC, int N>
LORA_DEV void ldn(float* v, const float* base, uint32_t at, int n) {
  auto addr = [&](uint32_t i) {
    return reinterpret_cast<const float*>(reinterpret_cast<const char*>(base) + 4u * i);
  };
  if constexpr (VEC && N == 4) {
    const f32x4 t = *reinterpret_cast<const f32x4*>(addr(n > 0 ? at : 0));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[e];
  } else if constexpr (VEC && N == 2) {
    const f32x2 t = *reinterpret_cast<const f32x2*>(addr(n > 0 ? at : 0));
    v[0] = t[0];
    v[1] = t[1];
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = *addr(e < n ? at + e : 0);
  }
}
template <bool VEC, int N>
LORA_DEV float maskn(float v, int e, int n) {
  return (VEC && N > 1 ? n > 0 : e < n) ? v : 0.0f;
}
template <bool VEC, int N>
LORA_DEV void stn(const float* v, float* base, uint32_t at, int n) {
  float* p = reinterpret_cast<float*>(reinterpret_cast<char*>(base) + 4u * at);
  if constexpr (VEC && N == 4) {
    if (n > 0) *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  } else if constexpr (VEC && N == 2) {
    if (n > 0) *reinterpret_cast<f32x2*>(p) = f32x2{v[0], v[1]};
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < n) p[e] = v[e];
  }
}

// u of one element, from the gradient and the momentum after its update.
LORA_DEV float muon_u(const MuonArgs& p, float g, float m) {
  return p.nesterov ? fmaf(p.mu, m, g) : m;
}

// A chunk of the long side as gram reads it: NK contraction steps of four
// indices, one per lane group, for each of the F fragments.
template <int RP, bool WIDE, bool VEC, bool MUON>
struct GramChunk {
  static constexpr int F = RP / 16;
  static constexpr int NK = RP >= 64 ? 4 : 8;   // 16 or 32 long-side indices, as registers allow
  static constexpr int LEN = 4 * NK;
  float g[F][NK], m[MUON ? F : 1][MUON ? NK : 1];

  // Each access: fragment f (wide) or group of Q fragments (tall).
  static constexpr int Q = WIDE ? 4 : (F > 4 ? 4 : F);

  template <typename Fn>
  LORA_DEV static void each(const MuonRun& r, int k0, int k1, int lane, Fn fn) {
    const int c = lane & 15, h = lane >> 4;
    if constexpr (WIDE) {
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int q = 0; q < NK / 4; ++q) {
          const int row = 16 * f + c;
          const int k = k0 + 16 * q + 4 * h;
          fn(f, 4 * q, (uint32_t)row * (uint32_t)r.cols + (uint32_t)k,
             row < r.rows && k < k1 ? min(4, k1 - k) : 0);
        }
    } else {
#pragma unroll
      for (int s = 0; s < NK; ++s)
#pragma unroll
        for (int f = 0; f < F; f += Q) {
          const int k = k0 + 4 * s + h;
          const int col = F * c + f;
          fn(f, s, (uint32_t)k * (uint32_t)r.cols + (uint32_t)col, k < k1 && col < r.cols ? min(Q, r.cols - col) : 0);
        }
    }
  }
  LORA_DEV void load(const MuonArgs& p, const MuonRun& r, int64_t base, int k0, int k1, int lane) {
    each(r, k0, k1, lane, [&](int f, int s, uint32_t at, int n) {
      float v[Q];
      ldn<VEC, Q>(v, p.G + base, at, n);
#pragma unroll
      for (int e = 0; e < Q; ++e) (WIDE ? g[f][s + e] : g[f + e][s]) = v[e];
      if constexpr (MUON) {
        ldn<VEC, Q>(v, p.M + base, at, n);
#pragma unroll
        for (int e = 0; e < Q; ++e) (WIDE ? m[f][s + e] : m[f + e][s]) = v[e];
      }
    });
  }
  // The momentum's update (done before this kernel where waves share their
  // chunks, RP 128); g becomes u, zero where there is no element.
  LORA_DEV void update(const MuonArgs& p, const MuonRun& r, int64_t base, int k0, int k1, int lane,
                       float sc) {
    each(r, k0, k1, lane, [&](int f, int s, uint32_t at, int n) {
      float mv[Q];
#pragma unroll
      for (int e = 0; e < Q; ++e) {
        float& x = WIDE ? g[f][s + e] : g[f + e][s];
        if constexpr (MUON) {
          const float gs = x * sc, mo = WIDE ? m[f][s + e] : m[f + e][s];
          mv[e] = RP < 128 ? fmaf(p.mu, mo, gs) : mo;
          x = muon_u(p, gs, mv[e]);
        }
        x = maskn<VEC, Q>(x, e, n);
      }
      if constexpr (MUON && RP < 128) stn<VEC, Q>(mv, p.M + base, at, n);
    });
  }
};

template <int RP>
constexpr int muon_tiles() {
  return (RP / 16) * (RP / 16 + 1) / 2;
}

// Upper tile index -> (row tile, column tile), rows first.
template <int RP>
LORA_DEV void muon_tile(int i, int& t, int& u) {
  t = 0;
  int n = RP / 16;
  while (i >= n) {
    i -= n;
    --n;
    ++t;
  }
  u = t + i;
}

// Blocks of four waves a CU, which their registers (and at 128 LDS) are held to.
template <int RP>
constexpr int muon_per_cu() {
  return RP == 128 ? 1 : 2;
}

// Parts that the waves of a block split the result's tiles into: at RP 128
// the 36 upper tiles (288 registers) are shared by two waves a chunk.
template <int RP>
constexpr int muon_parts() {
  return RP == 128 ? 2 : 1;
}
template <int RP>
constexpr int muon_part_tiles() {
  return muon_tiles<RP>() / muon_parts<RP>();
}

// PART's tiles (i % parts == PART) over the chunks of wave kw of KW.
template <int RP, bool WIDE, bool VEC, bool MUON, int PART, int KW>
LORA_DEV void gram_range(const MuonArgs& p, const MuonRun& r, int64_t base, int k0, int k1, int kw,
                         float sc, f64x4 (&acc)[muon_part_tiles<RP>()]) {
  typedef GramChunk<RP, WIDE, VEC, MUON> Chunk;
  constexpr int F = Chunk::F, NP = muon_parts<RP>();
  const int lane = threadIdx.x & 63;
  auto use = [&](Chunk& x, int k) {
    x.update(p, r, base, k, k1, lane, sc);
#pragma unroll
    for (int s = 0; s < Chunk::NK; ++s) {
      double d[F];
#pragma unroll
      for (int f = 0; f < F; ++f) d[f] = (double)x.g[f][s];
      int i = 0;
#pragma unroll
      for (int t = 0; t < F; ++t)
#pragma unroll
        for (int u = t; u < F; ++u, ++i)
          if (i % NP == PART) acc[i / NP] = mfma16x16x4_f64(d[t], d[u], acc[i / NP]);
    }
  };
  // Two chunks take turns: one's loads are in flight while the other is used.
  constexpr int STEP = KW * Chunk::LEN;
  Chunk x, y;
  int k = k0 + kw * Chunk::LEN;
  if (k >= k1) return;
  x.load(p, r, base, k, k1, lane);
  for (;;) {
    if (k + STEP < k1) y.load(p, r, base, k + STEP, k1, lane);
    __builtin_amdgcn_sched_barrier(0);
    use(x, k);
    if ((k += STEP) >= k1) break;
    if (k + STEP < k1) x.load(p, r, base, k + STEP, k1, lane);
    __builtin_amdgcn_sched_barrier(0);
    use(y, k);
    if ((k += STEP) >= k1) break;
  }
}

// RP 128 reads each chunk in two waves, so the momentum is updated ahead of
// it: m <- mu m + g' of one block's range.
template <bool VEC>
__global__ __launch_bounds__(256) void muon_momentum_kernel(MuonArgs p) {
  if (muon_vetoed(p)) return;
  const float sc = *p.d_scale;
  const MuonRun& r = p.run[muon_find(p, blockIdx.x, false)];
  const int rel = blockIdx.x - r.blk0, mat = rel / r.splits, sp = rel % r.splits;
  const uint32_t n = (uint32_t)r.rows * (uint32_t)r.cols;
  const uint32_t per = (n / r.splits + 1024) / 1024 * 1024;
  const uint32_t e0 = sp * per, e1 = min(n, e0 + per);
  const int64_t base = r.offset + mat * r.stride;
  for (uint32_t e = e0 + 4 * threadIdx.x; e < e1; e += 1024) {
    const int k = (int)min(4u, e1 - e);
    float g[4], m[4];
    ldn<VEC, 4>(g, p.G + base, e, k);
    ldn<VEC, 4>(m, p.M + base, e, k);
#pragma unroll
    for (int q = 0; q < 4; ++q) m[q] = fmaf(p.mu, m[q], g[q] * sc);
    stn<VEC, 4>(m, p.M + base, e, k);
  }
}

// The Gram matrix of one block's range of a matrix, its upper tiles in `sum`
// (the waves' sums, in wave order).  W waves.
template <int RP, bool VEC, bool MUON, int W>
LORA_DEV void gram_block(const MuonArgs& p, const MuonRun& r, int64_t base, int k0, int k1, float sc,
                         f64x4* sum) {
  constexpr int NP = muon_parts<RP>(), NA = muon_part_tiles<RP>(), KW = W / NP;
  f64x4 acc[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) acc[i] = f64x4{0, 0, 0, 0};
  const bool wide = r.rows <= r.cols;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = wave % NP, kw = wave / NP;
  if (part == 0) {
    if (wide) gram_range<RP, true, VEC, MUON, 0, KW>(p, r, base, k0, k1, kw, sc, acc);
    else gram_range<RP, false, VEC, MUON, 0, KW>(p, r, base, k0, k1, kw, sc, acc);
  } else {
    if (wide) gram_range<RP, true, VEC, MUON, NP - 1, KW>(p, r, base, k0, k1, kw, sc, acc);
    else gram_range<RP, false, VEC, MUON, NP - 1, KW>(p, r, base, k0, k1, kw, sc, acc);
  }
  for (int w = 0; w < KW; ++w) {
    if (kw == w) {
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        f64x4& s = sum[(i * NP + part) * 64 + lane];
        s = w ? s + acc[i] : acc[i];
      }
    }
    __syncthreads();
  }
}

template <int RP, bool VEC, bool MUON>
__global__ __launch_bounds__(256, muon_per_cu<RP>()) void muon_gram_kernel(MuonArgs p) {
  constexpr int NT = muon_tiles<RP>();
  __shared__ f64x4 sum[NT * 64];
  if (muon_vetoed(p)) return;
  const float sc = p.d_scale ? *p.d_scale : 1.0f;
  const MuonRun& r = p.run[muon_find(p, blockIdx.x, false)];
  const int rel = blockIdx.x - r.blk0, mat = rel / r.splits, sp = rel % r.splits;
  const int k0 = sp * r.len, k1 = min(max(r.rows, r.cols), k0 + r.len);
  gram_block<RP, VEC, MUON, 4>(p, r, r.offset + mat * r.stride, k0, k1, sc, sum);
  f64x4* out = reinterpret_cast<f64x4*>(p.part) + (int64_t)blockIdx.x * NT * 64;
  for (int i = threadIdx.x; i < NT * 64; i += 256) out[i] = sum[i];
}

// ------------------------------------------------------------------- poly
// Symmetric RP x RP matrices as 16 x 16 tiles in the layout that the matrix
// instruction leaves a result in: value v of lane l is element (4 v + l / 16,
// l % 16).  That is also its B operand of step v, and, the matrix being
// symmetric, tile (w, t) is the A operand of step v for tile (t, w): a product
// of two such matrices needs no rearrangement, only 16-byte LDS reads.
//
// The iteration takes 4 products a step (G^2, Q P, Q G, Q (Q G); the first
// and last step fewer), 17 in all for five steps, and is bound by float64 MFMA
// (32 to 35 ns an instruction and SIMD, measured).  Up to RP 64 one CU runs it
// whole, all matrices in LDS (128 KB at 64), with only the upper tiles
// computed, 5/8 of them at 64; stores mirror them.  At RP 128 that would be
// 160 us of one CU's MFMA (275 us measured): there each product is a launch
// with a wave for every upper tile (muon_product_kernel), 15 for five steps.
template <int RP>
struct PolyLds {
  static constexpr int F = RP / 16, NM = F == 1 ? 1 : 4;
  f64x4 a[NM][F * F * 64];   // tile (w, t) at (w F + t) 64
  double diag[RP];
};
// Waves of poly_waves, and its barriers.
template <int RP>
constexpr int poly_nw() {
  return RP == 16 ? 1 : RP == 32 ? 4 : 8;   // RP up to 64
}
constexpr int POLY16_SYNCS = 2;   // at RP 16, for waves that only join them

// s = the n values at `in`, stride apart, in order; eight loads at a time, all
// of them unconditional (past the last one it is read again, and not added).
LORA_DEV void sum_tiles(f64x4& s, const f64x4* in, int stride, int n) {
  s = f64x4{0, 0, 0, 0};
  for (int q = 0; q < n; q += 8) {
    f64x4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = in[(int64_t)min(q + u, n - 1) * stride];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (q + u < n) s += v[u];
  }
}

// Tile (t, u) of A B.
template <int F>
LORA_DEV f64x4 sym_tile(const f64x4* A, const f64x4* B, int t, int u, int lane) {
  f64x4 d = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < F; ++w) {
    const f64x4 x = A[(w * F + t) * 64 + lane], y = B[(w * F + u) * 64 + lane];
#pragma unroll
    for (int s = 0; s < 4; ++s) d = mfma16x16x4_f64(x[s], y[s], d);
  }
  return d;
}
template <int F>
LORA_DEV void sym_store(f64x4* M, int t, int u, f64x4 d, int lane) {
  M[(t * F + u) * 64 + lane] = d;
  if (t == u) return;
  const int c = lane & 15, h = lane >> 4;
  double* m = reinterpret_cast<double*>(M + ((u * F + t) * 64 + (c & 3) * 16 + h)) + (c >> 2);
#pragma unroll
  for (int v = 0; v < 4; ++v) m[16 * v] = d[v];
}

// One matrix: G from the upper tiles in `in` (`splits` sets of them, added in
// order), P / norm left in `out` [RP][RP], rows ldp apart.  Called by the
// first poly_nw waves of a block; `sync` is the block's barrier.
template <int RP, typename Sync>
LORA_DEV void poly_waves(const MuonArgs& p, bool wide, const f64x4* in, int splits, PolyLds<RP>& m,
                         double* out, int ldp, Sync sync) {
  constexpr int F = RP / 16, NT = muon_tiles<RP>(), NW = poly_nw<RP>();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, h = lane >> 4;
  double* const flat = reinterpret_cast<double*>(m.a[0]);
  auto at = [&](int i, int j) -> double& {
    return flat[(((i >> 4) * F + (j >> 4)) * 64 + (i & 3) * 16 + (j & 15)) * 4 + ((i >> 2) & 3)];
  };
  // A tall matrix's fragment f holds columns F c + f.
  for (int i = wave; i < NT; i += NW) {
    f64x4 s;
    sum_tiles(s, in + i * 64 + lane, NT * 64, splits);
    int t, w;
    muon_tile<RP>(i, t, w);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int rc = 4 * v + h;
      const int row = wide ? 16 * t + rc : F * rc + t, col = wide ? 16 * w + c : F * c + w;
      at(row, col) = s[v];
      at(col, row) = s[v];
    }
  }
  sync();
  for (int i = threadIdx.x; i < RP; i += 64 * NW) m.diag[i] = at(i, i);
  sync();
  double tr = 0.0;
#pragma unroll 16
  for (int i = 0; i < RP; ++i) tr += m.diag[i];
  const double norm = sqrt(tr) + p.eps;
  const double inv = norm > 0.0 || norm != norm ? 1.0 / norm : 0.0;   // a NaN stays one
  // G is kept unscaled in LDS until the first step reads it.
  const double inv2 = inv * inv;
  auto poly = [&](f64x4 s, f64x4 g, bool diag) {   // a I + b G + c G^2
#pragma unroll
    for (int v = 0; v < 4; ++v)
      s[v] = p.c * s[v] + p.b * g[v] + (diag && 4 * v + h == c ? p.a : 0.0);
    return s;
  };

  if constexpr (PolyLds<RP>::NM == 4) {
    f64x4 *G = m.a[0], *Q = m.a[1], *P = m.a[2], *T = m.a[3];
    constexpr int PER = (NT + NW - 1) / NW;
    auto emit = [&](int t, int u, f64x4 d) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = 16 * t + 4 * v + h, col = 16 * u + c;
        out[row * ldp + col] = d[v] * inv;
        out[col * ldp + row] = d[v] * inv;
      }
    };
    for (int k = 0; k < p.steps; ++k) {
      const bool last = k + 1 == p.steps;
      // The first step's G is unscaled: G^2 takes inv2 twice.
      const double g1 = k == 0 ? inv2 : 1.0, g2 = g1 * g1;
      for (int i = wave; i < NT; i += NW) {
        int t, u;
        muon_tile<RP>(i, t, u);
        const f64x4 d = poly(sym_tile<F>(G, G, t, u, lane) * g2, G[(t * F + u) * 64 + lane] * g1, t == u);
        sym_store<F>(Q, t, u, d, lane);
        if (k == 0) sym_store<F>(P, t, u, d, lane);
        if (k == 0 && last) emit(t, u, d);
      }
      sync();
      f64x4 d[PER];
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int i = wave + NW * q;
        if (k > 0 && i < NT) {
          int t, u;
          muon_tile<RP>(i, t, u);
          d[q] = sym_tile<F>(Q, P, t, u, lane);
          if (last) emit(t, u, d[q]);
        }
      }
      if (last) {
        sync();
        break;
      }
      for (int i = NW - 1 - wave; i < NT; i += NW) {   // the other way round: waves share evenly
        int t, u;
        muon_tile<RP>(i, t, u);
        sym_store<F>(T, t, u, sym_tile<F>(Q, G, t, u, lane) * g1, lane);
      }
      sync();
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int i = wave + NW * q;
        if (k > 0 && i < NT) {
          int t, u;
          muon_tile<RP>(i, t, u);
          sym_store<F>(P, t, u, d[q], lane);
        }
      }
      for (int i = wave; i < NT; i += NW) {
        int t, u;
        muon_tile<RP>(i, t, u);
        sym_store<F>(G, t, u, sym_tile<F>(Q, T, t, u, lane), lane);
      }
      sync();
    }
  } else {
    f64x4 G = m.a[0][lane] * inv2, P = G;
    auto mul = [](f64x4 A, f64x4 B) {
      f64x4 d = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 4; ++s) d = mfma16x16x4_f64(A[s], B[s], d);
      return d;
    };
    for (int k = 0; k < p.steps; ++k) {
      const f64x4 Q = poly(mul(G, G), G, true);
      P = k == 0 ? Q : mul(Q, P);
      if (k + 1 < p.steps) G = mul(Q, mul(Q, G));
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) out[(4 * v + h) * ldp + c] = P[v] * inv;
  }
}

template <int RP>
__global__ __launch_bounds__(64 * poly_nw<RP>()) void muon_poly_kernel(MuonArgs p) {
  __shared__ PolyLds<RP> m;
  if (muon_vetoed(p)) return;
  const MuonRun& r = p.run[muon_find(p, blockIdx.x, true)];
  const int mat = blockIdx.x - r.mat0;
  const f64x4* in = reinterpret_cast<const f64x4*>(p.part) +
                    ((int64_t)r.blk0 + (int64_t)mat * r.splits) * muon_tiles<RP>() * 64;
  poly_waves<RP>(p, r.rows <= r.cols, in, r.splits, m, p.poly + (int64_t)blockIdx.x * RP * RP, RP,
                 [] { __syncthreads(); });
}

// RP 128: five matrices a mat in device memory, in the tiles of PolyLds.
template <int RP>
struct PolyMem {
  static constexpr int F = RP / 16, SZ = F * F * 64;   // f64x4 a matrix
  static constexpr int64_t BYTES = 5ll * SZ * 32 + 256;
  f64x4* p;
  LORA_DEV PolyMem(char* base, int mat) : p(reinterpret_cast<f64x4*>(base + mat * BYTES)) {}
  LORA_DEV f64x4* G() const { return p; }
  LORA_DEV f64x4* Q() const { return p + SZ; }
  LORA_DEV f64x4* T() const { return p + 2 * SZ; }
  LORA_DEV f64x4* P(int k) const { return p + (3 + (k & 1)) * SZ; }   // after step k
  LORA_DEV double& inv() const { return *reinterpret_cast<double*>(p + 5 * SZ); }
};

// G from the blocks' partials, a wave an upper tile.
template <int RP>
__global__ __launch_bounds__(256) void muon_assemble_kernel(MuonArgs p, char* mem) {
  constexpr int F = RP / 16, NT = muon_tiles<RP>();
  static_assert(NT % 4 == 0, "whole blocks a matrix");
  if (muon_vetoed(p)) return;
  const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int mi = wave / NT, i = wave % NT, lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const MuonRun& r = p.run[muon_find(p, mi, true)];
  const bool wide = r.rows <= r.cols;
  const f64x4* in = reinterpret_cast<const f64x4*>(p.part) +
                    ((int64_t)r.blk0 + (int64_t)(mi - r.mat0) * r.splits) * NT * 64 + i * 64 + lane;
  f64x4 s;
  sum_tiles(s, in, NT * 64, r.splits);
  double* flat = reinterpret_cast<double*>(PolyMem<RP>(mem, mi).G());
  auto at = [&](int i, int j) -> double& {
    return flat[(((i >> 4) * F + (j >> 4)) * 64 + (i & 3) * 16 + (j & 15)) * 4 + ((i >> 2) & 3)];
  };
  int t, w;
  muon_tile<RP>(i, t, w);
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int rc = 4 * v + h;
    const int row = wide ? 16 * t + rc : F * rc + t, col = wide ? 16 * w + c : F * c + w;
    at(row, col) = s[v];
    at(col, row) = s[v];
  }
}

// One product of step k, a wave an upper tile.  phase 0: Q = a I + b G + c G^2
// (and P at k 0); 1: T = Q G, and after them P <- Q P for k > 0 (the last step:
// P alone); 2: G = Q T.  The last P goes to p.poly, divided by the norm.
template <int RP>
__global__ __launch_bounds__(256) void muon_product_kernel(MuonArgs p, char* mem, int phase, int k) {
  constexpr int F = RP / 16, NT = muon_tiles<RP>();
  static_assert(NT % 4 == 0, "whole blocks a matrix");
  if (muon_vetoed(p)) return;
  const bool last = k + 1 == p.steps, both = phase == 1 && k > 0 && !last;
  const int jobs = both ? 2 * NT : NT;
  const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int mat = wave / jobs, job = wave % jobs, lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  int t, u;
  muon_tile<RP>(job % NT, t, u);
  const PolyMem<RP> m(mem, mat);
  double inv;
  if (phase == 0 && k == 0) {   // the norm, from G's trace
    double tr = 0.0;
#pragma unroll
    for (int i = lane; i < RP; i += 64)
      tr += reinterpret_cast<const double*>(
          m.G() + (i >> 4) * (F + 1) * 64 + (i & 3) * 16 + (i & 15))[(i >> 2) & 3];
    const double norm = sqrt(wave_sum(tr)) + p.eps;
    inv = norm > 0.0 || norm != norm ? 1.0 / norm : 0.0;   // a NaN stays one
    if (job == 0 && lane == 0) m.inv() = inv;
  } else {
    inv = m.inv();
  }
  const double g1 = k == 0 ? inv * inv : 1.0;
  const bool is_p = phase == 1 && (last || job >= NT);
  f64x4* out;
  f64x4 d;
  if (phase == 0) {
    d = sym_tile<F>(m.G(), m.G(), t, u, lane);
    const f64x4 g = m.G()[(t * F + u) * 64 + lane];
#pragma unroll
    for (int v = 0; v < 4; ++v)
      d[v] = p.c * (g1 * g1) * d[v] + p.b * g1 * g[v] + (t == u && 4 * v + h == c ? p.a : 0.0);
    out = m.Q();
  } else {
    d = sym_tile<F>(m.Q(), phase == 2 ? m.T() : is_p ? m.P(k - 1) : m.G(), t, u, lane);
    if (phase == 1 && !is_p) d *= g1;
    out = phase == 2 ? m.G() : is_p ? m.P(k) : m.T();
  }
  sym_store<F>(out, t, u, d, lane);
  if (phase == 0 && k == 0) sym_store<F>(m.P(0), t, u, d, lane);
  if (last && (is_p || (phase == 0 && k == 0))) {
    double* poly = p.poly + (int64_t)mat * RP * RP;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 16 * t + 4 * v + h, col = 16 * u + c;
      poly[row * RP + col] = d[v] * inv;
      poly[col * RP + row] = d[v] * inv;
    }
  }
}

// ------------------------------------------------------------------ apply
// One wave's share: E groups of 16 long-side indices times P, or at RP 128
// times one half of P's rows (the waves pair up, each with half the result).
template <int RP, bool WIDE, bool VEC, bool MUON>
struct ApplyChunk {
  static constexpr int F = RP / 16, E = RP >= 64 ? 2 : 4;
  static constexpr int NS = WIDE ? RP / 4 : E * F, N = WIDE ? E : 4;
  float g[NS][N], m[MUON ? NS : 1][MUON ? N : 1];

  // Access i.  Wide: row 4 i + h, E columns from k + E c.  Tall: row
  // k + 16 (i / F) + c, four columns from 16 (i % F) + 4 h.
  template <typename Fn>
  LORA_DEV static void each(const MuonRun& r, int k, int k1, int lane, Fn fn) {
    const int c = lane & 15, h = lane >> 4;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int row = WIDE ? 4 * i + h : k + 16 * (i / F) + c;
      const int col = WIDE ? k + E * c : 16 * (i % F) + 4 * h;
      const bool in = WIDE ? row < r.rows && col < k1 : row < k1 && col < r.cols;
      fn(i, (uint32_t)row * (uint32_t)r.cols + (uint32_t)col,
         in ? min(N, (WIDE ? k1 : r.cols) - col) : 0);
    }
  }
  LORA_DEV void load(const MuonArgs& p, const MuonRun& r, int64_t base, int k, int k1, int lane) {
    each(r, k, k1, lane, [&](int i, uint32_t at, int n) {
      ldn<VEC, N>(g[i], p.G + base, at, n);
      if constexpr (MUON) ldn<VEC, N>(m[i], p.M + base, at, n);
    });
  }
  LORA_DEV void to_u(const MuonArgs& p, const MuonRun& r, int k, int k1, int lane, float sc,
                     float (&x)[NS][N]) {
    each(r, k, k1, lane, [&](int i, uint32_t, int n) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float u = g[i][e];
        if constexpr (MUON) u = muon_u(p, u * sc, m[i][e]);
        x[i][e] = maskn<VEC, N>(u, e, n);
      }
    });
  }
};

// `ready` makes P ready (with a barrier) while the first chunk arrives.
template <int RP, bool WIDE, bool VEC, bool MUON, int W, typename Ready>
LORA_DEV void apply_range(const MuonArgs& p, const MuonRun& r, const double* P, int64_t base, int k0,
                          int k1, float sc, Ready ready) {
  typedef ApplyChunk<RP, WIDE, VEC, MUON> Chunk;
  constexpr int F = RP / 16, E = Chunk::E, LDP = RP + 4, NP = muon_parts<RP>(), FP = F / NP;
  constexpr int NO = WIDE ? FP * 4 : E * FP, N = Chunk::N, STEP = (W / NP) * 16 * E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, h = lane >> 4;
  const int t0 = (wave % NP) * FP;
  // Result i of a lane.  Wide: tile t0 + i / 4, row value i % 4, E columns.
  // Tall: token group i / FP, tile t0 + i % FP, four columns.
  auto results = [&](int k, auto fn) {
#pragma unroll
    for (int i = 0; i < NO; ++i) {
      const int row = WIDE ? 16 * (t0 + i / 4) + 4 * (i % 4) + h : k + 16 * (i / FP) + c;
      const int col = WIDE ? k + E * c : 16 * (t0 + i % FP) + 4 * h;
      const bool in = WIDE ? row < r.rows && col < k1 : row < k1 && col < r.cols;
      fn(i, (uint32_t)row * (uint32_t)r.cols + (uint32_t)col,
         in ? min(N, (WIDE ? k1 : r.cols) - col) : 0);
    }
  };
  // From the range's end to its start: what the gram pass read last is still
  // in the last-level cache (256 MB).
  const int kw = k0 + (wave / NP) * 16 * E;
  int k = kw + (k1 - 1 - kw + STEP) / STEP * STEP - STEP;   // below kw: no chunk
  Chunk q;
  if (k >= kw) q.load(p, r, base, k, k1, lane);
  __builtin_amdgcn_sched_barrier(0);
  ready();
  for (; k >= kw; k -= STEP) {
    float x[Chunk::NS][N], w[MUON ? NO : 1][MUON ? N : 1];
    q.to_u(p, r, k, k1, lane, sc, x);
    // This chunk's parameters and the next chunk arrive during the products.
    if constexpr (MUON)
      results(k, [&](int i, uint32_t at, int n) { ldn<VEC, N>(w[i], p.P + base, at, n); });
    if (k - STEP >= kw) q.load(p, r, base, k - STEP, k1, lane);
    __builtin_amdgcn_sched_barrier(0);
    f64x4 acc[FP][E];
#pragma unroll
    for (int t = 0; t < FP; ++t)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[t][e] = f64x4{0, 0, 0, 0};
    // Tall: P's rows permuted so that a lane's four results are neighbours.
    const int j = WIDE ? c : 4 * (c & 3) + (c >> 2);
#pragma unroll
    for (int s = 0; s < RP / 4; ++s) {
#pragma unroll
      for (int t = 0; t < FP; ++t) {
        const double a = P[(16 * (t0 + t) + j) * LDP + (WIDE ? 4 * s + h : 16 * (s / 4) + 4 * h + s % 4)];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const double b = WIDE ? (double)x[s][e] : (double)x[e * F + s / 4][s % 4];
          acc[t][e] = mfma16x16x4_f64(a, b, acc[t][e]);
        }
      }
      // Keeps the reads of P from all being hoisted to the top (RP^2 / 64
      // doubles a lane).
      if (s % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
    results(k, [&](int i, uint32_t at, int n) {
      float o[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        o[e] = (float)(WIDE ? acc[i / 4][e % E][i % 4] : acc[i % FP][i / FP][e]);
        if constexpr (MUON) o[e] = w[i][e] - r.rate * o[e] - r.decay * w[i][e];
      }
      stn<VEC, N>(o, p.P + base, at, n);
    });
  }
}

template <int RP, bool VEC, bool MUON>
__global__ __launch_bounds__(256, muon_per_cu<RP>()) void muon_apply_kernel(MuonArgs p) {
  constexpr int LDP = RP + 4;
  __shared__ __align__(16) double P[RP * LDP];
  if (muon_vetoed(p)) return;
  const float sc = p.d_scale ? *p.d_scale : 1.0f;
  const MuonRun& r = p.run[muon_find(p, blockIdx.x, false)];
  const int rel = blockIdx.x - r.blk0, mat = rel / r.splits, sp = rel % r.splits;
  const bool wide = r.rows <= r.cols;
  auto ready = [&] {
    if constexpr (RP == 16) {
      // The polynomial of a 16 x 16 matrix is 2 us of one wave: every block
      // iterates its own, under its first chunk's loads, which saves a launch
      // (22 x [8, 2048]: 16.8 -> 13.2 us).
      __shared__ PolyLds<RP> m;
      const f64x4* in = reinterpret_cast<const f64x4*>(p.part) +
                        ((int64_t)r.blk0 + (int64_t)mat * r.splits) * muon_tiles<RP>() * 64;
      auto sync = [] { __syncthreads(); };
      if (threadIdx.x < 64) {
        poly_waves<RP>(p, wide, in, r.splits, m, P, LDP, sync);
      } else {
        for (int i = 0; i < POLY16_SYNCS; ++i) sync();
      }
    } else {
      typedef double f64x2 __attribute__((ext_vector_type(2)));
      const f64x2* src = reinterpret_cast<const f64x2*>(p.poly + (int64_t)(r.mat0 + mat) * RP * RP);
#pragma unroll
      for (int i = 2 * threadIdx.x; i < RP * RP; i += 512)
        *reinterpret_cast<f64x2*>(P + (i / RP) * LDP + i % RP) = src[i / 2];
    }
    __syncthreads();
  };
  const int k0 = sp * r.len, k1 = min(max(r.rows, r.cols), k0 + r.len);
  const int64_t base = r.offset + mat * r.stride;
  if (wide) apply_range<RP, true, VEC, MUON, 4>(p, r, P, base, k0, k1, sc, ready);
  else apply_range<RP, false, VEC, MUON, 4>(p, r, P, base, k0, k1, sc, ready);
}

// All three steps of a small matrix in one block (sixteen waves): one launch
// instead of two, with its second pass over the matrix in the CU's reach.
template <int RP, bool VEC, bool MUON>
__global__ __launch_bounds__(1024) void muon_small_kernel(MuonArgs p) {
  static_assert(RP == 16, "POLY16_SYNCS");
  constexpr int LDP = RP + 4, NT = muon_tiles<RP>();
  __shared__ f64x4 sum[NT * 64];
  __shared__ PolyLds<RP> m;
  __shared__ double P[RP * LDP];
  if (muon_vetoed(p)) return;
  const float sc = p.d_scale ? *p.d_scale : 1.0f;
  const MuonRun& r = p.run[muon_find(p, blockIdx.x, true)];
  const int64_t base = r.offset + (int64_t)(blockIdx.x - r.mat0) * r.stride;
  const int L = max(r.rows, r.cols);
  const bool wide = r.rows <= r.cols;
  gram_block<RP, VEC, MUON, 16>(p, r, base, 0, L, sc, sum);
  // The first waves iterate; the others only join the barriers.
  auto sync = [] { __syncthreads(); };
  if ((int)threadIdx.x < 64 * poly_nw<RP>()) {
    poly_waves<RP>(p, wide, sum, 1, m, P, LDP, sync);
  } else {
    for (int i = 0; i < POLY16_SYNCS; ++i) sync();
  }
  __syncthreads();   // P, and the momentum that other waves wrote
  if (wide) apply_range<RP, true, VEC, MUON, 16>(p, r, P, base, 0, L, sc, [] {});
  else apply_range<RP, false, VEC, MUON, 16>(p, r, P, base, 0, L, sc, [] {});
}

}  // namespace lora
