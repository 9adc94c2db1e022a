// Attention over packed sequences, softmax(scale Q K^T) V per sequence and
// head, forward and backward.
//
// Rows.  The query heads that share a key head are taken together: row m of a
// sequence and key head is query token m / G of head kvh G + m % G, G = heads /
// kv_heads.  A tile of rows then reads its keys once for all G heads, a causal
// tile spans few tokens, and single tokens fill G rows of a tile.  Row tiles
// are numbered over the whole batch without a list: sequence i's start at
// offset_i G / BM + i (rounded down), which leaves room for its ragged last one.
//
// Registers.  Every product is 32x32 on the matrix cores (bf16: 16 terms an
// instruction, float32: 2), and the softmax never leaves registers: a wave
// computes S^T = K Q^T, so that a lane holds 16 keys of one row (its maximum
// and sum are its own and its other half's), and the same registers, rounded
// to bf16, are the B operand of O^T = V^T P^T; only the order in which a lane
// half holds its keys matters, and V^T's operand follows it (read transposed
// from LDS).  The backward's two passes do the same: dQ as S^T, dK and dV as S
// with the keys across lanes.
#pragma once
#include <type_traits>

#include "common.hpp"

namespace lora {

struct AttnArgs {
  const void *Q, *K, *V;        // T
  void* O;                      // OT (backward: read)
  const void* dO;               // OT
  void *dQ, *dK, *dV;           // OT
  float* lse;                   // [heads][q_tokens], forward: may be NULL
  float* delta;                 // [heads][q_tokens] (workspace of the backward)
  const int32_t *qo, *ko, *kl;  // offsets [seqs + 1] and lengths [seqs] or NULL
  int64_t ldq, hq, ldk, hk, ldv, hv, ldo, ho;
  int64_t q_tokens, k_tokens;
  int32_t seqs, kv, group, dim, causal, tiles;
  float scale, c;               // c = scale log2 e
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Element types: bf16 operands are held as 8 values in a u32x4, float32 ones
// as 4 in an f32x4; a fragment covers FK contraction indices over both halves.
template <typename T>
struct Frag;
template <>
struct Frag<uint16_t> {
  typedef u32x4 V;
  static constexpr int E = 8, FK = 16;
  LORA_DEV static f32x16 mma(V a, V b, f32x16 c) { return mfma32x32x16_bf16(a, b, c); }
};
template <>
struct Frag<float> {
  typedef f32x4 V;
  static constexpr int E = 4, FK = 8;
  LORA_DEV static f32x16 mma(V a, V b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = mfma32x32x2(a[e], b[e], c);
    return c;
  }
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
// Two values to bf16, to nearest even (one instruction).
LORA_DEV uint32_t cvt_bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2_t));
}

// 16-byte chunk c of row `row` of an LDS tile [rows][DP] is stored at chunk
// c ^ attn_swz(row) of the row.  Operands with the rows across lanes are read
// 16 bytes a lane: 16 neighbouring rows then touch all 64 banks once.  The
// transpose reads of bf16 (4 rows x 64 bytes for a pair of 16-lane groups) need
// the chunks' upper bits to differ between those four rows.
template <typename T, int DP>
LORA_DEV int attn_swz(int row) {
  if constexpr (sizeof(T) == 4) return row & 15;
  else if constexpr (DP == 128) return ((row & 3) << 2) ^ ((row >> 2) & 3);
  else return ((row & 2) << 1) ^ ((row >> 2) & 3);
}

// Operand with rows across lanes: row r0 + l % 32, fragment s of its values.
template <typename T, int DP>
LORA_DEV typename Frag<T>::V lds_rows(const T* tile, int row, int s, int half) {
  constexpr int CPR = DP * (int)sizeof(T) / 16;
  static_assert(CPR >= 8, "");
  return *reinterpret_cast<const typename Frag<T>::V*>(
      reinterpret_cast<const char*>(tile) + row * (DP * (int)sizeof(T)) + ((2 * s + half) ^ attn_swz<T, DP>(row)) * 16);
}

typedef short attn_s4 __attribute__((ext_vector_type(4)));
// Operand with columns (d) across lanes and the contraction over rows, in the
// order of a product's result: lane half h's values v = 8 u .. 8 u + 7 are rows
// 16 u + 4 h + 0..3 and 16 u + 8 + 4 h + 0..3 of the 32 from r0.
template <int DP>
LORA_DEV u32x4 lds_cols(const uint16_t* tile, int r0, int u, int d0, int lane) {
  const int i = lane & 15, g = lane >> 4;
  const int row = r0 + 16 * u + 4 * (g >> 1) + (i >> 2);
  const int col = d0 + 16 * (g & 1) + 4 * (i & 3);
  auto at = [&](int r) {
    return (__attribute__((address_space(3))) attn_s4*)(
        (__attribute__((address_space(3))) const char*)tile + r * (DP * 2) +
        (((col >> 3) ^ attn_swz<uint16_t, DP>(r)) << 4) + ((col & 4) << 1));
  };
  const attn_s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(row));
  const attn_s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(row + 8));
  const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
  return u32x4{a[0], a[1], b[0], b[1]};
}
template <int DP>
LORA_DEV float lds_cols(const float* tile, int r0, int v, int d0, int lane) {
  const int row = r0 + row32(v, lane), col = d0 + (lane & 31);
  return *reinterpret_cast<const float*>(reinterpret_cast<const char*>(tile) + row * (DP * 4) +
                                         (((col >> 2) ^ attn_swz<float, DP>(row)) << 4) + ((col & 3) << 2));
}

// acc[dt] += tile[r0 .. r0 + 31][dt]^T x, x a product's result with the same 32
// rows down its registers: the products over keys (forward, dQ) or rows (dK, dV).
template <typename T, int DP>
LORA_DEV void mma_cols(f32x16 (&acc)[DP / 32], const T* tile, int r0, const f32x16& x, int lane) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      u32x4 b;
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = cvt_bf16x2(x[8 * u + 2 * e], x[8 * u + 2 * e + 1]);
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt)
        acc[dt] = mfma32x32x16_bf16(lds_cols<DP>(tile, r0, u, 32 * dt, lane), b, acc[dt]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v)
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt)
        acc[dt] = mfma32x32x2(lds_cols<DP>(tile, r0, v, 32 * dt, lane), x[v], acc[dt]);
  }
}

// acc += rows of the tile times the register operand f (both along DP).
template <typename T, int DP>
LORA_DEV f32x16 mma_rows(const T* tile, int row, const typename Frag<T>::V (&f)[DP / Frag<T>::FK], int half) {
  f32x16 acc = {};
#pragma unroll
  for (int s = 0; s < DP / Frag<T>::FK; ++s)
    acc = Frag<T>::mma(lds_rows<T, DP>(tile, row, s, half), f[s], acc);
  return acc;
}

// The other half's value of the same row.
LORA_DEV float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// ---------------------------------------------------------------------------
// Sequences.  Offsets are clamped to the buffers, so that no value of theirs
// leads outside; tiles past a sequence's end do nothing.
// ---------------------------------------------------------------------------
struct AttnSeq {
  int q0, lq, k0, lk;   // first row and length, queries and keys
};
LORA_DEV AttnSeq attn_seq(const AttnArgs& p, int i) {
  const int tq = (int)p.q_tokens, tk = (int)p.k_tokens;
  AttnSeq s;
  s.q0 = min(max(p.qo[i], 0), tq);
  s.lq = min(max(p.qo[i + 1], s.q0), tq) - s.q0;
  s.k0 = min(max(p.ko[i], 0), tk);
  s.lk = min(max(p.ko[i + 1], s.k0), tk) - s.k0;
  if (p.kl) s.lk = min(max(p.kl[i], 0), s.lk);
  return s;
}
// The sequence of tile t, where sequence i's tiles start at off_i mul / B + i.
LORA_DEV int attn_find(const int32_t* off, int seqs, int64_t most, int mul, int B, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = seqs;
  while (n > 1) {
    const int step = (n + 63) >> 6, i = lane * step;
    bool in = false;
    if (i < n) in = min(max((int64_t)off[lo + i], (int64_t)0), most) * mul / B + lo + i <= t;
    const int before = max((int)__popcll(__ballot(in)) - 1, 0) * step;
    lo += before;
    n = min(step, n - before);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}
LORA_DEV int attn_first(const int32_t* off, int64_t most, int mul, int B, int i) {
  return (int)(min(max((int64_t)off[i], (int64_t)0), most) * mul / B) + i;
}
// Keys that query token i of the sequence sees.
LORA_DEV int attn_limit(const AttnArgs& p, const AttnSeq& s, int i) {
  return p.causal ? min(max(i + s.lk - s.lq + 1, 0), s.lk) : s.lk;
}

template <typename T, typename OT>
LORA_DEV typename Frag<T>::V frag_of(const OT* g) {
  if constexpr (std::is_same_v<T, OT>) {
    return *reinterpret_cast<const typename Frag<T>::V*>(g);
  } else {   // float32 rounded to bf16
    const f32x4 a = *reinterpret_cast<const f32x4*>(g), b = *reinterpret_cast<const f32x4*>(g + 4);
    return u32x4{cvt_bf16x2(a[0], a[1]), cvt_bf16x2(a[2], a[3]), cvt_bf16x2(b[0], b[1]), cvt_bf16x2(b[2], b[3])};
  }
}
// A row's register operand: fragment s holds values FK s + E half ...
template <typename T, int DP, typename OT>
LORA_DEV void load_frags(typename Frag<T>::V (&f)[DP / Frag<T>::FK], const OT* row, int dim, int half) {
#pragma unroll
  for (int s = 0; s < DP / Frag<T>::FK; ++s) {
    const int d = Frag<T>::FK * s + Frag<T>::E * half;
    f[s] = d < dim ? frag_of<T>(row + d) : typename Frag<T>::V{};
  }
}

// Rows of memory into an LDS tile [ROWS][DP]; `at(r)` gives row r's address or
// NULL (zeros).  Values past dim are zero.
template <typename T, int DP, int ROWS, int NT, typename OT, typename F>
LORA_DEV void stage_rows(T* tile, int dim, F at) {
  constexpr int CPR = DP * (int)sizeof(T) / 16, E = Frag<T>::E;
#pragma unroll
  for (int c = threadIdx.x; c < ROWS * CPR; c += NT) {
    const int row = c / CPR, ch = c % CPR;
    const OT* g = at(row);
    const typename Frag<T>::V v = g && ch * E < dim ? frag_of<T>(g + ch * E) : typename Frag<T>::V{};
    *reinterpret_cast<typename Frag<T>::V*>(reinterpret_cast<char*>(tile) + row * (DP * (int)sizeof(T)) +
                                            (ch ^ attn_swz<T, DP>(row)) * 16) = v;
  }
}

// Four neighbouring results of one row.
template <typename OT>
LORA_DEV void store_4(OT* g, float a, float b, float c, float d) {
  if constexpr (sizeof(OT) == 4) *reinterpret_cast<f32x4*>(g) = f32x4{a, b, c, d};
  else *reinterpret_cast<u32x2*>(g) = u32x2{cvt_bf16x2(a, b), cvt_bf16x2(c, d)};
}
// acc^T [d][row] times f to the row at g.
template <int DP, typename OT>
LORA_DEV void store_row(OT* g, const f32x16 (&acc)[DP / 32], float f, int dim, int half) {
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int d = 32 * dt + 8 * q + 4 * half;
      if (d < dim)
        store_4(g + d, acc[dt][4 * q] * f, acc[dt][4 * q + 1] * f, acc[dt][4 * q + 2] * f, acc[dt][4 * q + 3] * f);
    }
}

// ---------------------------------------------------------------------------
// Forward.  A block's RW waves hold 32 rows each.
// ---------------------------------------------------------------------------
template <typename T, typename OT, int DP, int RW, int KT>
__global__ __launch_bounds__(64 * RW) void attn_fwd_kernel(AttnArgs p) {
  constexpr int NT = 64 * RW, BM = 32 * RW, BN = 32 * KT, KS = DP / Frag<T>::FK, DT = DP / 32;
  typedef typename Frag<T>::V V;
  __shared__ __attribute__((aligned(16))) T Ks[BN * DP];
  __shared__ __attribute__((aligned(16))) T Vs[BN * DP];
  const int kvh = (int)(blockIdx.x % p.kv), t = p.tiles - 1 - (int)(blockIdx.x / p.kv);
  const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
  const int i = attn_find(p.qo, p.seqs, p.q_tokens, p.group, BM, t);
  const AttnSeq sq = attn_seq(p, i);
  const int m0 = (t - attn_first(p.qo, p.q_tokens, p.group, BM, i)) * BM, rows = sq.lq * p.group;
  if (m0 < 0 || m0 >= rows) return;
  // This lane's row (lanes past the last one repeat it) and the keys it sees.
  const int m = m0 + 32 * wave + (lane & 31), mc = min(m, rows - 1);
  const int tok = mc / p.group, head = kvh * p.group + mc % p.group;
  const int lim = attn_limit(p, sq, tok);
  const int most = attn_limit(p, sq, (min(m0 + BM, rows) - 1) / p.group);        // of the block's rows
  const int least = attn_limit(p, sq, min(m0 + 32 * wave, rows - 1) / p.group);  // of the wave's
  V qf[KS];
  load_frags<T, DP>(qf, (const T*)p.Q + (sq.q0 + tok) * p.ldq + head * p.hq, p.dim, half);
  f32x16 o[DT] = {};
  float mx = -INFINITY, m2 = 0.0f, l = 0.0f;   // maximum, maximum times c (0: none yet), this half's sum
  const T* Kg = (const T*)p.K + sq.k0 * p.ldk + kvh * p.hk;
  const T* Vg = (const T*)p.V + sq.k0 * p.ldv + kvh * p.hv;
  for (int kb = 0; kb < most; kb += BN) {
    __syncthreads();
    stage_rows<T, DP, BN, NT, T>(Ks, p.dim, [&](int r) { return kb + r < sq.lk ? Kg + (kb + r) * p.ldk : nullptr; });
    stage_rows<T, DP, BN, NT, T>(Vs, p.dim, [&](int r) { return kb + r < sq.lk ? Vg + (kb + r) * p.ldv : nullptr; });
    __syncthreads();
    f32x16 s[KT];
    float top = mx;
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      s[j] = mma_rows<T, DP>(Ks, 32 * j + (lane & 31), qf, half);
      if (kb + BN > least) {
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (kb + 32 * j + row32(v, lane) >= lim) s[j][v] = -INFINITY;
      }
#pragma unroll
      for (int v = 0; v < 16; ++v) top = fmaxf(top, s[j][v]);
    }
    top = fmaxf(top, other_half(top));
    const float now = top == -INFINITY ? 0.0f : top * p.c;
    const float old = mx == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m2 - now);
    mx = top;
    m2 = now;
    l *= old;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[dt] *= old;
#pragma unroll
    for (int j = 0; j < KT; ++j) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        s[j][v] = __builtin_amdgcn_exp2f(fmaf(s[j][v], p.c, -now));
        l += s[j][v];
      }
      mma_cols<T, DP>(o, Vs, 32 * j, s[j], lane);
    }
  }
  l += other_half(l);
  if (m >= rows) return;
  store_row<DP>((OT*)p.O + (sq.q0 + tok) * p.ldo + head * p.ho, o, l == 0.0f ? 0.0f : 1.0f / l, p.dim, half);
  if (p.lse && half == 0)
    p.lse[head * p.q_tokens + sq.q0 + tok] = l == 0.0f ? -INFINITY : (m2 + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---------------------------------------------------------------------------
// Backward, with delta = do . o and p = exp(s - lse):
//   ds = p (dp - delta),  dp = do v^T;  dq = scale ds k;  dk = scale ds^T q,
//   dv = p^T do.
// Two passes, each of which owns what it writes: a pass over keys for each row
// tile (dQ, and delta for the second) and one over rows for each key tile (dK,
// dV).  S and dP are computed in both: 7 products where one pass would take 5,
// but dQ would then be summed over key tiles in memory, in no fixed order.
// ---------------------------------------------------------------------------
template <typename T, typename OT, int DP, int RW>
__global__ __launch_bounds__(64 * RW) void attn_dq_kernel(AttnArgs p) {
  constexpr int NT = 64 * RW, BM = 32 * RW, BN = 32, KS = DP / Frag<T>::FK, DT = DP / 32;
  typedef typename Frag<T>::V V;
  __shared__ __attribute__((aligned(16))) T Ks[BN * DP];
  __shared__ __attribute__((aligned(16))) T Vs[BN * DP];
  const int kvh = (int)(blockIdx.x % p.kv), t = p.tiles - 1 - (int)(blockIdx.x / p.kv);
  const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
  const int i = attn_find(p.qo, p.seqs, p.q_tokens, p.group, BM, t);
  const AttnSeq sq = attn_seq(p, i);
  const int m0 = (t - attn_first(p.qo, p.q_tokens, p.group, BM, i)) * BM, rows = sq.lq * p.group;
  if (m0 < 0 || m0 >= rows) return;
  const int m = m0 + 32 * wave + (lane & 31), mc = min(m, rows - 1);
  const int tok = mc / p.group, head = kvh * p.group + mc % p.group;
  const int lim = attn_limit(p, sq, tok);
  const int most = attn_limit(p, sq, (min(m0 + BM, rows) - 1) / p.group);
  const int least = attn_limit(p, sq, min(m0 + 32 * wave, rows - 1) / p.group);
  V qf[KS], df[KS];
  load_frags<T, DP>(qf, (const T*)p.Q + (sq.q0 + tok) * p.ldq + head * p.hq, p.dim, half);
  const OT* dor = (const OT*)p.dO + (sq.q0 + tok) * p.ldo + head * p.ho;
  const OT* orow = (const OT*)p.O + (sq.q0 + tok) * p.ldo + head * p.ho;
  load_frags<T, DP>(df, dor, p.dim, half);
  float delta = 0.0f;
  for (int d = 4 * half; d < p.dim; d += 8) {
    f32x4 a, b;
    if constexpr (sizeof(OT) == 4) {
      a = *reinterpret_cast<const f32x4*>(dor + d);
      b = *reinterpret_cast<const f32x4*>(orow + d);
    } else {
      const u32x2 x = *reinterpret_cast<const u32x2*>(dor + d), y = *reinterpret_cast<const u32x2*>(orow + d);
      a = f32x4{__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u), __uint_as_float(x[1] << 16),
                __uint_as_float(x[1] & 0xffff0000u)};
      b = f32x4{__uint_as_float(y[0] << 16), __uint_as_float(y[0] & 0xffff0000u), __uint_as_float(y[1] << 16),
                __uint_as_float(y[1] & 0xffff0000u)};
    }
    delta += (a[0] * b[0] + a[1] * b[1]) + (a[2] * b[2] + a[3] * b[3]);
  }
  delta += other_half(delta);
  const int64_t at = head * p.q_tokens + sq.q0 + tok;
  if (half == 0 && m < rows) p.delta[at] = delta;
  const float lse2 = p.lse[at] * kLog2e;
  f32x16 dq[DT] = {};
  const T* Kg = (const T*)p.K + sq.k0 * p.ldk + kvh * p.hk;
  const T* Vg = (const T*)p.V + sq.k0 * p.ldv + kvh * p.hv;
  for (int kb = 0; kb < most; kb += BN) {
    __syncthreads();
    stage_rows<T, DP, BN, NT, T>(Ks, p.dim, [&](int r) { return kb + r < sq.lk ? Kg + (kb + r) * p.ldk : nullptr; });
    stage_rows<T, DP, BN, NT, T>(Vs, p.dim, [&](int r) { return kb + r < sq.lk ? Vg + (kb + r) * p.ldv : nullptr; });
    __syncthreads();
    f32x16 s = mma_rows<T, DP>(Ks, lane & 31, qf, half);
    const f32x16 dp = mma_rows<T, DP>(Vs, lane & 31, df, half);
#pragma unroll
    for (int v = 0; v < 16; ++v) s[v] = __builtin_amdgcn_exp2f(fmaf(s[v], p.c, -lse2)) * (dp[v] - delta);
    if (kb + BN > least) {   // after the products: what a masked score gives must not count
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if (kb + row32(v, lane) >= lim) s[v] = 0.0f;
    }
    mma_cols<T, DP>(dq, Ks, 0, s, lane);
  }
  if (m >= rows) return;
  store_row<DP>((OT*)p.dQ + (sq.q0 + tok) * p.ldq + head * p.hq, dq, p.scale, p.dim, half);
}

// dK and dV of 32 keys a wave, over all rows that see them.
template <typename T, typename OT, int DP, int KW>
__global__ __launch_bounds__(64 * KW) void attn_dkv_kernel(AttnArgs p) {
  constexpr int NT = 64 * KW, BK = 32 * KW, BQ = 32, KS = DP / Frag<T>::FK, DT = DP / 32;
  typedef typename Frag<T>::V V;
  __shared__ __attribute__((aligned(16))) T Qs[BQ * DP];
  __shared__ __attribute__((aligned(16))) T Ds[BQ * DP];
  __shared__ __attribute__((aligned(16))) float ls[BQ], des[BQ];
  __shared__ int lims[BQ];
  const int kvh = (int)(blockIdx.x % p.kv), t = (int)(blockIdx.x / p.kv);
  const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
  const int i = attn_find(p.ko, p.seqs, p.k_tokens, 1, BK, t);
  const AttnSeq sq = attn_seq(p, i);
  const int k0 = (t - attn_first(p.ko, p.k_tokens, 1, BK, i)) * BK, rows = sq.lq * p.group;
  if (k0 < 0 || k0 >= sq.lk) return;
  const int key = k0 + 32 * wave + (lane & 31), kc = min(key, sq.lk - 1);
  V kf[KS], vf[KS];
  load_frags<T, DP>(kf, (const T*)p.K + (sq.k0 + kc) * p.ldk + kvh * p.hk, p.dim, half);
  load_frags<T, DP>(vf, (const T*)p.V + (sq.k0 + kc) * p.ldv + kvh * p.hv, p.dim, half);
  f32x16 dk[DT] = {}, dv[DT] = {};
  // The first row that sees one of the block's keys.
  const int first = p.causal ? max(k0 - (sq.lk - sq.lq), 0) * p.group : 0;
  for (int mb = first / BQ * BQ; mb < rows; mb += BQ) {
    __syncthreads();
    auto row = [&](int r, int64_t ld, int64_t h) {
      const int m = mb + r;
      return (sq.q0 + m / p.group) * ld + (kvh * p.group + m % p.group) * h;
    };
    stage_rows<T, DP, BQ, NT, T>(Qs, p.dim, [&](int r) {
      return mb + r < rows ? (const T*)p.Q + row(r, p.ldq, p.hq) : nullptr;
    });
    stage_rows<T, DP, BQ, NT, OT>(Ds, p.dim, [&](int r) {
      return mb + r < rows ? (const OT*)p.dO + row(r, p.ldo, p.ho) : nullptr;
    });
    if (threadIdx.x < BQ) {
      const int m = mb + threadIdx.x;
      const bool in = m < rows;
      const int64_t at = in ? row(threadIdx.x, 1, p.q_tokens) : 0;
      ls[threadIdx.x] = in ? p.lse[at] * kLog2e : 0.0f;
      des[threadIdx.x] = in ? p.delta[at] : 0.0f;
      lims[threadIdx.x] = in ? attn_limit(p, sq, m / p.group) : 0;
    }
    __syncthreads();
    f32x16 s = mma_rows<T, DP>(Qs, lane & 31, kf, half);
    f32x16 ds = mma_rows<T, DP>(Ds, lane & 31, vf, half);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int r = row32(v, lane);
      const bool in = key < lims[r];
      s[v] = in ? __builtin_amdgcn_exp2f(fmaf(s[v], p.c, -ls[r])) : 0.0f;
      ds[v] = in ? s[v] * (ds[v] - des[r]) : 0.0f;
    }
    mma_cols<T, DP>(dv, Ds, 0, s, lane);
    mma_cols<T, DP>(dk, Qs, 0, ds, lane);
  }
  if (key >= sq.lk) return;
  store_row<DP>((OT*)p.dK + (sq.k0 + key) * p.ldk + kvh * p.hk, dk, p.scale, p.dim, half);
  store_row<DP>((OT*)p.dV + (sq.k0 + key) * p.ldv + kvh * p.hv, dv, 1.0f, p.dim, half);
}

}  // namespace lora
