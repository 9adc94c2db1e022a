// Norm and rotation of heads, forward and backward.
//
//   z = x rstd gamma,  rstd = 1 / sqrt(sum x^2 / D + eps)   (or z = x)
//   y_a = z_a cos - z_b sin,  y_b = z_b cos + z_a sin for each pair (a, b),
//   the angle being the token's position times the pair's frequency
//   dz = the rotation by the negative angle of dy,  dgamma = sum dz xh,
//   dx = rstd (g - xh mean(g xh)),  xh = x rstd,  g = dz gamma
//
// Bound by memory: a head is read once into the registers of LPH lanes (eight
// values each, so that both members of a pair are in one lane and only the
// norm's sum crosses lanes) and written once; rstd is computed again in the
// backward, which reads x anyway.  A wave takes several heads of one token and
// computes the token's angles once for all of them.
//
// Angles: position times frequency passes 2 pi many times at far positions, so
// the product and its reduction to half a turn either way are float64; sine and
// cosine are float32 functions of the remainder.
//
// Measured (a plain copy moves 5.1 TB/s from HBM): 4096 tokens of 32 and 8 heads of
// 128, float32 to bf16, 26 us (126 MB, 4.8 TB/s); backward of 2048 in float32, 24.5
// us (126 MB, 5.1 TB/s) and 3.9 for gamma's sums; one token 4.3 (latency).
#pragma once
#include "common.hpp"

namespace lora {

struct HeadsOne {
  const void* X;
  const void* dY;         // backward
  void* out;              // Y or dX
  const float* gamma;     // [dim] or NULL (1)
  const double* freqs;    // [rot / 2]
  float* dgamma;          // backward, or NULL
  float* part;            // backward, more than one block: [blocks][dim]
  int64_t ldx, hx, ldy, hy;
  int32_t heads, dim, rot, norm, inter, xbf, ybf;
  int32_t ranges, iters;  // ranges of a token's heads, and each one's steps of 64 / LPH heads
  float eps, fdim;
};
struct HeadsArgs {
  HeadsOne one[4];
  const int32_t* pos;     // [tokens]
  int64_t tokens;
  int32_t accumulate;
};

// The eight columns of lane t.  VEC: two groups of four neighbours; else four
// pairs LPH apart.  Either way values k and 4 + k are a pair, but for
// neighbours (INTER) in VEC's order, where 2 k and 2 k + 1 are.
template <int LPH, bool VEC>
struct HeadCols {
  int a, b, t, rot, dim;
  bool near;
  LORA_DEV HeadCols(const HeadsOne& p, int t_) : t(t_), rot(p.rot), dim(p.dim) {
    near = p.inter || 8 * t >= rot;   // neighbouring columns: interleaved pairs, or not rotated
    a = near ? 8 * t : 4 * t;
    b = near ? 8 * t + 4 : rot / 2 + 4 * t;
  }
  LORA_DEV int pair(int k) const { return VEC ? 4 * t + k : t + LPH * k; }
  LORA_DEV bool turned(int k) const { return 2 * pair(k) < rot; }
  LORA_DEV int col(const HeadsOne& p, int e) const {
    if constexpr (VEC) return e < 4 ? a + e : b + e - 4;
    const int q = pair(e & 3);
    return p.inter || 2 * q >= rot ? 2 * q + (e >> 2) : q + (e >> 2) * (rot / 2);
  }
};

template <typename T, int LPH, bool VEC>
LORA_DEV void heads_load(f32x4 (&v)[2], const T* g, const HeadsOne& p, const HeadCols<LPH, VEC>& c) {
  if constexpr (VEC) {
    const bool in = 8 * c.t < p.dim;
    v[0] = load4(g + (in ? c.a : 0));
    v[1] = load4(g + (in ? c.b : 0));
    if (!in) v[0] = v[1] = f32x4{0, 0, 0, 0};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = c.col(p, e);
      v[e >> 2][e & 3] = k < p.dim ? load1(g + k) : 0.0f;
    }
  }
}
template <typename T, int LPH, bool VEC>
LORA_DEV void heads_store(T* g, const f32x4 (&v)[2], const HeadsOne& p, const HeadCols<LPH, VEC>& c) {
  if constexpr (VEC) {
    if (8 * c.t < p.dim) {
      store4(g + c.a, v[0]);
      store4(g + c.b, v[1]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = c.col(p, e);
      if (k < p.dim) store1(g + k, v[e >> 2][e & 3]);
    }
  }
}

template <int LPH>
LORA_DEV float head_sum(float x) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

struct HeadAngles {
  double turns[4];   // turns a position
  float co[4], si[4];
  template <int LPH, bool VEC>
  LORA_DEV void init(const HeadsOne& p, const HeadCols<LPH, VEC>& c) {
#pragma unroll
    for (int k = 0; k < 4; ++k) turns[k] = c.turned(k) ? p.freqs[c.pair(k)] * 0.15915494309189535 : 0.0;
  }
  LORA_DEV void at(int pos) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const double x = (double)pos * turns[k];
      sincospif(2.0f * (float)(x - rint(x)), &si[k], &co[k]);
    }
  }
};
// v turned by the angles (sign 1) or back (-1).
template <int LPH, bool VEC>
LORA_DEV void heads_turn(f32x4 (&v)[2], const HeadAngles& an, float sign, const HeadsOne& p,
                         const HeadCols<LPH, VEC>& c) {
  auto turn = [&](float& a, float& b, int k) {
    const float s = sign * an.si[k], x = a * an.co[k] - b * s, y = b * an.co[k] + a * s;
    a = c.turned(k) ? x : a;
    b = c.turned(k) ? y : b;
  };
  if (VEC && p.inter) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a = v[k >> 1][2 * (k & 1)], b = v[k >> 1][2 * (k & 1) + 1];
      turn(a, b, k);
      v[k >> 1][2 * (k & 1)] = a;
      v[k >> 1][2 * (k & 1) + 1] = b;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a = v[0][k], b = v[1][k];
      turn(a, b, k);
      v[0][k] = a;
      v[1][k] = b;
    }
  }
}

// Waves of the grid take (token, range of heads) in turn.
template <typename TX, typename TY, int LPH, bool VEC>
LORA_DEV void heads_fwd_body(const HeadsArgs& p, const HeadsOne& d) {
  constexpr int HPI = 64 / LPH;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const HeadCols<LPH, VEC> c(d, lane % LPH);
  HeadAngles an;
  an.init(d, c);
  f32x4 ga[2];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = c.col(d, e);
    ga[e >> 2][e & 3] = d.gamma && k < d.dim ? d.gamma[k] : 1.0f;
  }
  const int64_t tasks = p.tokens * d.ranges;
  for (int64_t task = (int64_t)blockIdx.x * 4 + wave; task < tasks; task += (int64_t)gridDim.x * 4) {
    const int64_t tok = task / d.ranges;
    const int r = (int)(task % d.ranges);
    if (d.rot) an.at(p.pos[tok]);
    const TX* x = (const TX*)d.X + tok * d.ldx;
    TY* y = (TY*)d.out + tok * d.ldy;
    for (int j = 0; j < d.iters; ++j) {
      const int head = (r * d.iters + j) * HPI + lane / LPH;
      const int hc = min(head, d.heads - 1);   // lanes past the last head repeat it
      f32x4 v[2];
      heads_load<TX, LPH, VEC>(v, x + hc * d.hx, d, c);
      if (d.norm) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          s += (v[q][0] * v[q][0] + v[q][1] * v[q][1]) + (v[q][2] * v[q][2] + v[q][3] * v[q][3]);
        const float rstd = 1.0f / sqrtf(head_sum<LPH>(s) / d.fdim + d.eps);
        v[0] = v[0] * rstd * ga[0];
        v[1] = v[1] * rstd * ga[1];
      }
      if (d.rot) heads_turn<LPH, VEC>(v, an, 1.0f, d, c);
      if (head < d.heads) heads_store<TY, LPH, VEC>(y + head * d.hy, v, d, c);
    }
  }
}

template <typename TX, typename TY, int LPH, bool VEC>
LORA_DEV void heads_bwd_body(const HeadsArgs& p, const HeadsOne& d, float (*red)[LPH * 8]) {
  constexpr int HPI = 64 / LPH;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const HeadCols<LPH, VEC> c(d, lane % LPH);
  HeadAngles an;
  an.init(d, c);
  f32x4 ga[2], dg[2] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = c.col(d, e);
    ga[e >> 2][e & 3] = d.gamma && k < d.dim ? d.gamma[k] : 1.0f;
  }
  const int64_t tasks = p.tokens * d.ranges;
  for (int64_t task = (int64_t)blockIdx.x * 4 + wave; task < tasks; task += (int64_t)gridDim.x * 4) {
    const int64_t tok = task / d.ranges;
    const int r = (int)(task % d.ranges);
    if (d.rot) an.at(p.pos[tok]);
    for (int j = 0; j < d.iters; ++j) {
      const int head = (r * d.iters + j) * HPI + lane / LPH;
      const int hc = min(head, d.heads - 1);
      f32x4 g[2], x[2];
      heads_load<TY, LPH, VEC>(g, (const TY*)d.dY + tok * d.ldy + hc * d.hy, d, c);
      if (d.norm) heads_load<TX, LPH, VEC>(x, (const TX*)d.X + tok * d.ldx + hc * d.hx, d, c);
      if (d.rot) heads_turn<LPH, VEC>(g, an, -1.0f, d, c);
      if (d.norm) {
        float s = 0.0f, u = 0.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          s += (x[q][0] * x[q][0] + x[q][1] * x[q][1]) + (x[q][2] * x[q][2] + x[q][3] * x[q][3]);
        const float rstd = 1.0f / sqrtf(head_sum<LPH>(s) / d.fdim + d.eps);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          x[q] *= rstd;
          if (head < d.heads) dg[q] += g[q] * x[q];
          g[q] *= ga[q];
          u += (g[q][0] * x[q][0] + g[q][1] * x[q][1]) + (g[q][2] * x[q][2] + g[q][3] * x[q][3]);
        }
        u = head_sum<LPH>(u) / d.fdim;
#pragma unroll
        for (int q = 0; q < 2; ++q) g[q] = (g[q] - x[q] * u) * rstd;
      }
      if (d.out && head < d.heads)
        heads_store<TX, LPH, VEC>((TX*)d.out + tok * d.ldx + head * d.hx, g, d, c);
    }
  }
  if (!d.dgamma) return;
  // The wave's heads, then the block's waves, in order.
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float s = dg[e >> 2][e & 3];
#pragma unroll
    for (int o = LPH; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    const int k = c.col(d, e);
    if (lane < LPH && k < d.dim) red[wave][k] = s;
  }
  __syncthreads();
  const bool last = gridDim.x == 1;
  for (int k = threadIdx.x; k < d.dim; k += 256) {
    const float s = (red[0][k] + red[1][k]) + (red[2][k] + red[3][k]);
    if (last) d.dgamma[k] = p.accumulate ? d.dgamma[k] + s : s;
    else d.part[(int64_t)blockIdx.x * d.dim + k] = s;
  }
}

template <int LPH, bool VEC>
__global__ __launch_bounds__(256) void heads_fwd_kernel(HeadsArgs p) {
  const HeadsOne d = p.one[blockIdx.y];
  if (d.xbf) {
    if (d.ybf) heads_fwd_body<uint16_t, uint16_t, LPH, VEC>(p, d);
    else heads_fwd_body<uint16_t, float, LPH, VEC>(p, d);
  } else {
    if (d.ybf) heads_fwd_body<float, uint16_t, LPH, VEC>(p, d);
    else heads_fwd_body<float, float, LPH, VEC>(p, d);
  }
}
template <int LPH, bool VEC>
__global__ __launch_bounds__(256) void heads_bwd_kernel(HeadsArgs p) {
  __shared__ float red[4][LPH * 8];
  const HeadsOne d = p.one[blockIdx.y];
  if (d.xbf) {
    if (d.ybf) heads_bwd_body<uint16_t, uint16_t, LPH, VEC>(p, d, red);
    else heads_bwd_body<uint16_t, float, LPH, VEC>(p, d, red);
  } else {
    if (d.ybf) heads_bwd_body<float, uint16_t, LPH, VEC>(p, d, red);
    else heads_bwd_body<float, float, LPH, VEC>(p, d, red);
  }
}

// dgamma from the blocks' partials: a block takes 32 columns, 32 threads a
// column (each every 32nd partial, in order), in double.
__global__ __launch_bounds__(1024) void heads_finish_kernel(HeadsArgs p, int parts) {
  __shared__ double red[32][33];
  const HeadsOne d = p.one[blockIdx.y];
  if (!d.dgamma) return;
  const int cx = threadIdx.x & 31, py = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
  double s = 0.0;
  if (c < d.dim) {
    // Sixteen loads at a time (past the last partial it is read again and not
    // added): 512 partials are one round trip, 6.1 -> 3.4 us.
    for (int i = py; i < parts; i += 16 * 32) {
      float v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = d.part[(int64_t)min(i + 32 * k, parts - 1) * d.dim + c];
#pragma unroll
      for (int k = 0; k < 16; ++k) s += i + 32 * k < parts ? (double)v[k] : 0.0;
    }
  }
  red[py][cx] = s;
  __syncthreads();
  if (py == 0 && c < d.dim) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += red[i][cx];
    d.dgamma[c] = (float)(p.accumulate ? (double)d.dgamma[c] + s : s);
  }
}

}  // namespace lora
