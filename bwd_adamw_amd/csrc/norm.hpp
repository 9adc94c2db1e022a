// Layer norm and RMS norm over the rows of X, forward and backward.
//
//   mean = sum x / K (RMS: 0),  rstd = 1 / sqrt(sum (x - mean)^2 / K + eps)
//   xh = (x - mean) rstd,       y = xh gamma + beta
//   g = dy gamma,  dx = rstd (g - [layer] mean_k g - xh mean_k(g xh))
//   dgamma = sum_t dy xh,       dbeta = sum_t dy
//
// Both directions are bound by memory: a row is read once into registers
// (so the variance is of the centred values, in a second pass over registers
// rather than memory), reduced, and written once.  TPR lanes hold a row, V
// groups of 4 elements each: a whole wave or less for narrow rows, whose
// sums then need no LDS, several waves for wide ones.  A block keeps gamma
// (and beta) in registers while it walks its rows.
//
// The backward sums its one to four gradients of y as it loads them, so the
// projections' separate dX never meet in memory.  Each lane also holds the
// running dgamma and dbeta of its columns (float32, over its rows of one
// block, at most rows / 256 and one more); they leave as one partial per block,
// which norm_finish_kernel adds in block order in double.  One block writes the
// result itself.
//
// Measured (a plain copy moves 5.1 TB/s from HBM): 4096 rows of 2560 float32,
// forward 13.5 us (84 MB, part of it from the last-level cache); backward of
// three gradients 39.8 us (210 MB, 5.3 TB/s) and 4.7 for the sums of the
// partials; 1537 x 4100 bf16, one gradient, 18.7 and 5.4 us (38 MB and 25 MB
// of partials: few rows for the width).
#pragma once
#include <type_traits>

#include "common.hpp"

namespace lora {

struct NormArgs {
  const void* X;          // [rows, ldx]
  const void* dY[4];      // [rows, ldy], bwd
  void* out;              // fwd Y [rows, ldy]; bwd dX [rows, ldx] or NULL
  const float* gamma;     // [dim] or NULL (1)
  const float* beta;      // [dim] or NULL (0)
  float* stats;           // [rows][2] mean, rstd (fwd: written or NULL; bwd: read)
  float* part;            // bwd, more than one block: [blocks][2][dim]
  float* dgamma;          // bwd, or NULL
  float* dbeta;           // bwd, or NULL
  int64_t rows, ldx, ldy;
  int64_t rpb;            // rows per block
  int dim;
  int layer;              // 1 layer norm, 0 RMS norm
  int accumulate;         // add to dgamma and dbeta
  int ndy;                // gradients of y (element loads; else NDY)
  float eps, fdim;
};

template <typename T>
LORA_DEV float load1(const T* p) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float*>(p);
  else return bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(p));
}
template <typename T>
LORA_DEV f32x4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const f32x4*>(p);
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    return f32x4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u),
                 __uint_as_float(v[1] << 16), __uint_as_float(v[1] & 0xffff0000u)};
  }
}
// Float32 as it is, bf16 rounded to nearest even: the one rounding of the result.
template <typename T>
LORA_DEV void store1(T* p, float v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float*>(p) = v;
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)f32_to_bf16_bits(v);
}
template <typename T>
LORA_DEV void store4(T* p, f32x4 v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4*>(p) = v;
  else *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

constexpr int norm_threads(int tpr) { return tpr > 256 ? tpr : 256; }

// Sum of a and b over the TPR lanes of a row; every lane gets both.  `buf`
// alternates between calls, so that one barrier a call suffices: a wave can
// only write a buffer again after the barrier of the call between, which
// every reader of its old contents has passed.
template <int TPR>
LORA_DEV void row_sum(float& a, float& b, float (*red)[8][2], int& buf) {
  constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    const int wave = threadIdx.x >> 6, g = wave / NW, lane = threadIdx.x & 63;
    if (lane == 0) {
      red[buf][wave][0] = a;
      red[buf][wave][1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      a += red[buf][g * NW + w][0];
      b += red[buf][g * NW + w][1];
    }
    buf ^= 1;
  }
}

// The column of element e of a lane's group i: four neighbours where rows
// allow 4-element accesses (VEC), else lane-contiguous single elements.
template <int TPR, bool VEC>
LORA_DEV int norm_col(int i, int e, int t) {
  return VEC ? (i * TPR + t) * 4 + e : (i * 4 + e) * TPR + t;
}

template <typename T, int TPR, int V, bool VEC>
LORA_DEV void norm_load(f32x4 (&v)[V], const T* row, int dim, int t) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (VEC) {
      const int c = norm_col<TPR, true>(i, 0, t);
      v[i] = c < dim ? load4(row + c) : f32x4{0, 0, 0, 0};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = norm_col<TPR, false>(i, e, t);
        v[i][e] = c < dim ? load1(row + c) : 0.0f;
      }
    }
  }
}
template <typename T, int TPR, int V, bool VEC>
LORA_DEV void norm_store(T* row, const f32x4 (&v)[V], int dim, int t) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (VEC) {
      const int c = norm_col<TPR, true>(i, 0, t);
      if (c < dim) store4(row + c, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = norm_col<TPR, false>(i, e, t);
        if (c < dim) store1(row + c, v[i][e]);
      }
    }
  }
}
template <int TPR, int V, bool VEC>
LORA_DEV void norm_vector(f32x4 (&v)[V], const float* p, float none, int dim, int t) {
  if (p) {
    norm_load<float, TPR, V, VEC>(v, p, dim, t);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = f32x4{none, none, none, none};
  }
}

// Block: 256 / TPR rows at a time (TPR lanes each), rows [b rpb, (b+1) rpb).
template <typename T, int TPR, int V, bool VEC>
__global__ __launch_bounds__(norm_threads(TPR)) void norm_fwd_kernel(NormArgs p) {
  constexpr int R = norm_threads(TPR) / TPR;
  __shared__ float red[2][8][2];
  const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
  const int64_t r0 = (int64_t)blockIdx.x * p.rpb, r1 = min(p.rows, r0 + p.rpb);
  f32x4 ga[V], be[V];
  norm_vector<TPR, V, VEC>(ga, p.gamma, 1.0f, p.dim, t);
  norm_vector<TPR, V, VEC>(be, p.beta, 0.0f, p.dim, t);
  int buf = 0;
  for (int64_t base = r0; base < r1; base += R) {
    // Lanes past the last row repeat it (they take part in the barriers).
    const int64_t row = min(base + g, r1 - 1);
    const bool mine = base + g < r1;
    f32x4 x[V];
    norm_load<T, TPR, V, VEC>(x, (const T*)p.X + row * p.ldx, p.dim, t);
    float s = 0.0f, u = 0.0f, mean = 0.0f;
    if (p.layer) {
#pragma unroll
      for (int i = 0; i < V; ++i) s += (x[i][0] + x[i][1]) + (x[i][2] + x[i][3]);
      row_sum<TPR>(s, u, red, buf);
      mean = s / p.fdim;   // a division: one rounding after the sum's
    }
    s = u = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float d = norm_col<TPR, VEC>(i, e, t) < p.dim ? x[i][e] - mean : 0.0f;
        x[i][e] = d;
        s += d * d;
      }
    row_sum<TPR>(s, u, red, buf);
    const float rstd = 1.0f / sqrtf(s / p.fdim + p.eps);
    if (!mine) continue;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = x[i][e] * rstd * ga[i][e] + be[i][e];
    norm_store<T, TPR, V, VEC>((T*)p.out + row * p.ldy, x, p.dim, t);
    if (p.stats && t == 0) *reinterpret_cast<f32x2*>(p.stats + 2 * row) = f32x2{mean, rstd};
  }
}

// A row's operands as loaded: x and NDY gradients of y (0: the sum of p.ndy of
// them, read element by element one after another).
template <typename T, int TPR, int V, bool VEC, int NDY>
struct NormRow {
  typedef std::conditional_t<sizeof(T) == 4, f32x4, u32x2> Raw;
  static constexpr int N = NDY ? NDY : 1;
  static constexpr bool AHEAD = VEC && (1 + N) * V * (int)sizeof(T) <= 24;
  std::conditional_t<VEC, Raw, f32x4> x[V], d[N][V];
  f32x2 stats;

  // Unconditional loads (columns past dim repeat the first ones; their dy is
  // masked in dy()): a guarded load is waited for at the end of its branch.
  LORA_DEV void load(const NormArgs& p, int64_t row, int t) {
    const T* xr = (const T*)p.X + row * p.ldx;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        int c = norm_col<TPR, true>(i, 0, t);
        c = c < p.dim ? c : 0;
        x[i] = *reinterpret_cast<const Raw*>(xr + c);
#pragma unroll
        for (int n = 0; n < N; ++n)
          d[n][i] = *reinterpret_cast<const Raw*>((const T*)p.dY[n] + row * p.ldy + c);
      }
    } else {
      norm_load<T, TPR, V, false>(x, xr, p.dim, t);
      norm_load<T, TPR, V, false>(d[0], (const T*)p.dY[0] + row * p.ldy, p.dim, t);
      for (int n = 1; n < p.ndy; ++n) {
        const void* q = n == 1 ? p.dY[1] : n == 2 ? p.dY[2] : p.dY[3];
        f32x4 e[V];
        norm_load<T, TPR, V, false>(e, (const T*)q + row * p.ldy, p.dim, t);
#pragma unroll
        for (int i = 0; i < V; ++i) d[0][i] += e[i];
      }
    }
    stats = *reinterpret_cast<const f32x2*>(p.stats + 2 * row);
  }
  template <typename R>
  LORA_DEV static f32x4 value(R r) {
    if constexpr (sizeof(R) == 16) return r;
    else return f32x4{__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u),
                      __uint_as_float(r[1] << 16), __uint_as_float(r[1] & 0xffff0000u)};
  }
  LORA_DEV f32x4 dy(int i, bool in) const {
    f32x4 s = value(d[0][i]);
#pragma unroll
    for (int n = 1; n < N; ++n) s += value(d[n][i]);
    return in ? s : f32x4{0, 0, 0, 0};
  }
};

template <typename T, int TPR, int V, bool VEC, int NDY>
__global__ __launch_bounds__(norm_threads(TPR)) void norm_bwd_kernel(NormArgs p) {
  constexpr int NT = norm_threads(TPR), R = NT / TPR, COLS = TPR * V * 4;
  __shared__ float red[2][8][2];
  __shared__ float comb[R > 1 ? R * COLS : 1];
  const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
  const int64_t r0 = (int64_t)blockIdx.x * p.rpb, r1 = min(p.rows, r0 + p.rpb);
  f32x4 ga[V], dg[V], db[V];
  norm_vector<TPR, V, VEC>(ga, p.gamma, 1.0f, p.dim, t);
#pragma unroll
  for (int i = 0; i < V; ++i) dg[i] = db[i] = f32x4{0, 0, 0, 0};
  int buf = 0;
  typedef NormRow<T, TPR, V, VEC, NDY> Row;
  auto use = [&](const Row& q, int64_t base) {
    const bool mine = base + g < r1;
    const float mean = q.stats[0], rstd = q.stats[1];
    // Columns past dim hold dy = 0 and drop out of every sum.
    f32x4 x[V], dy[V];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = Row::value(q.x[i]);
      dy[i] = q.dy(i, mine && (!VEC || norm_col<TPR, true>(i, 0, t) < p.dim));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float xh = (x[i][e] - mean) * rstd, d = dy[i][e];
        x[i][e] = xh;
        dg[i][e] += d * xh;
        db[i][e] += d;
        dy[i][e] = d * ga[i][e];
        s1 += dy[i][e];
        s2 += dy[i][e] * xh;
      }
    }
    if (!p.out) return;   // the same for every lane
    row_sum<TPR>(s1, s2, red, buf);
    s1 = p.layer ? s1 / p.fdim : 0.0f;
    s2 /= p.fdim;
    if (!mine) return;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = rstd * (dy[i][e] - s1 - x[i][e] * s2);
    norm_store<T, TPR, V, VEC>((T*)p.out + (base + g) * p.ldx, x, p.dim, t);
  };
  // Lanes past the last row repeat it.  Where a row is a few registers the
  // next one loads while one is used (1537 x 4100 bf16, one gradient: 27 -> 19
  // us); with more, the waves that fit fewer registers hide as much (4096 x
  // 2560 float32, three gradients: 44 us against 40).
  auto at = [&](int64_t base) { return min(base + g, r1 - 1); };
  int64_t base = r0;
  if constexpr (Row::AHEAD) {
    Row a, b;
    a.load(p, at(base), t);
    for (;;) {
      if (base + R < r1) b.load(p, at(base + R), t);
      __builtin_amdgcn_sched_barrier(0);
      use(a, base);
      if ((base += R) >= r1) break;
      if (base + R < r1) a.load(p, at(base + R), t);
      __builtin_amdgcn_sched_barrier(0);
      use(b, base);
      if ((base += R) >= r1) break;
    }
  } else {
    for (; base < r1; base += R) {
      Row a;
      a.load(p, at(base), t);
      use(a, base);
    }
  }
  if (!p.dgamma && !p.dbeta) return;
  // Sum the block's R row groups in group order, gamma then beta.
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k == 0 ? !p.dgamma : !p.dbeta) continue;
    f32x4(&acc)[V] = k == 0 ? dg : db;
    if constexpr (R > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) comb[g * COLS + norm_col<TPR, VEC>(i, e, t)] = acc[i][e];
      __syncthreads();
    }
    float* dst = k == 0 ? p.dgamma : p.dbeta;
    const bool last = gridDim.x == 1;
    if (!last) dst = p.part + ((int64_t)blockIdx.x * 2 + k) * p.dim;
    const bool add = last && p.accumulate;
    if constexpr (R > 1) {
      for (int c = threadIdx.x; c < p.dim; c += NT) {
        float s = comb[c];
#pragma unroll 4
        for (int q = 1; q < R; ++q) s += comb[q * COLS + c];
        dst[c] = add ? dst[c] + s : s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = norm_col<TPR, VEC>(i, e, t);
          if (c < p.dim) dst[c] = add ? dst[c] + acc[i][e] : acc[i][e];
        }
    }
  }
}

// dgamma / dbeta from the blocks' partials: a block takes 32 columns of one
// of the two, 32 threads a column (each every 32nd partial, in order), in
// double.
__global__ __launch_bounds__(1024) void norm_finish_kernel(const float* __restrict__ part, int parts,
                                                           int dim, float* dgamma, float* dbeta,
                                                           int accumulate) {
  __shared__ double red[32][33];
  const int cx = threadIdx.x & 31, py = threadIdx.x >> 5;
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (!out) return;
  const int c = blockIdx.x * 32 + cx;
  double s = 0.0;
  if (c < dim) {
    const float* q = part + (int64_t)blockIdx.y * dim + c;
#pragma unroll 8
    for (int i = py; i < parts; i += 32) s += (double)q[(int64_t)i * 2 * dim];
  }
  red[py][cx] = s;
  __syncthreads();
  if (py == 0 && c < dim) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += red[i][cx];
    out[c] = (float)(accumulate ? (double)out[c] + s : s);
  }
}

}  // namespace lora
