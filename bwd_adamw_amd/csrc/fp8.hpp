// 8-bit frozen products with a scale for each block of 128, and the rounding
// of their activations.
//
//   forward  Y[t][n]  = sum_b 2^e[t][b] w[n/128][b] (q[t] . Wq[n])_b
//   dX       dX[t][k] = sum_b 2^e[t][b] w[b][k/128] (q[t] . Wq[:, k])_b
//
// where b runs over the 128-wide blocks of the contraction, q and 2^e are the
// activations' e4m3 values and scales (fp8_quant_kernel) and Wq, w those of
// W, read in its own [N, K] layout in both directions.  All 128 products of a
// block share both scales: four MFMAs sum a block of a 16 x 16 tile, and one
// float32 FMA per result adds it with W's scale.
//
// Accuracy: the values are widened to bf16, which holds every e4m3 value (and
// its product with a power of two) exactly, and multiplied by bf16 MFMA, whose
// products are exact and whose sums are float32.  The 8-bit MFMAs take half
// the time (4096 tokens of [2560 -> 4096]: 43 us against 75), but each aligns
// the products of a block to their largest and drops what lies about 2^-14
// below it: a result off by 1.3e-5 to 2.6e-5 on ordinary data, and by all of it
// where large products cancel.
//
// Tile: BM tokens x BN columns, contraction step 128 = one scale block.  Both
// operands go to LDS by direct-to-LDS loads, NS stages deep, as rows of 128
// bytes (dX's W: 128 rows of BN bytes) whose 16-byte chunks are XOR-swizzled
// by row, so that the fragment reads (16 rows at one chunk) and the loads
// touch every bank once.  A fragment is 32 bytes a lane: row l % 16, chunks
// l / 16 and l / 16 + 4; the order of the contraction within a block is free
// as long as both operands use the same one.  dX reads W transposed with
// ds_read_b64_tr_b8: even lanes of a group address the first eight columns of
// a 16-wide tile in eight rows, odd lanes the other eight, which gives lane c
// column c in those rows.
//
// Rate: the 256 x 256 tile runs 4096 tokens of [2560 -> 4096], one full round,
// at 1.15 PFLOP/s (75 us), of [9728 -> 4096] at 1.38; a step takes 2.9 us
// against the 2.2 that its MFMAs need at the 1.95 PFLOP/s they reach alone.  The
// rest is the vector unit's work (192 widenings and 128 FMAs a wave and step
// for 128 MFMAs, two thirds of their time beside them), of which each step's
// start, W's widening, stands alone in all waves.  Rounding moves 4 + 1 bytes a
// value at 5 TB/s (4096 x 2560: 10.5 us).
#pragma once
#include <utility>

#include "common.hpp"
#include "fp8_launch.hpp"

namespace lora {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Args {
  const uint8_t* Q;      // activations [rows, ldq] e4m3, whole 128-blocks
  const uint8_t* E;      // their scales, biased exponents [nk, lde] (fp8_scale_at)
  const uint8_t* W;      // [Np, Kp] e4m3
  const float* S;        // [Np/128, Kp/128]
  void* C;               // [M, Nc] float32 or bf16
  float* part;           // [nsplit][M][Nc] when nsplit > 1
  int64_t M, Nc;
  int64_t ldc;           // elements between rows of C
  int64_t ldq, lde, ldw, lds_;   // bytes a row of Q, W and a block of E; floats a row of S
  int nk;                // contraction steps
  int per;               // steps of a split
  int nsplit;
  Fp8Lora lora;          // OUT 3
  float* C2;             // OUT 3: a second copy of the result, or NULL
};

// Place of token t's exponent within a contraction block's lde of them: of
// each 128 tokens, the eight that a lane's row of eight tiles needs (t % 16
// equal) are neighbours, so that a lane reads them at once.
LORA_HD inline int64_t fp8_scale_at(int64_t t) {
  return (t & ~(int64_t)127) + (t & 15) * 8 + ((t >> 4) & 7);
}

// The 32 values of a fragment times a power of two, as four bf16 operands:
// e4m3 has four significant bits, bf16 eight.
struct Wide {
  bf16x8 k[4];
};
LORA_DEV Wide widen(i32x8 f, float p2) {
  Wide o;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t v[4];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      v[2 * w] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[2 * q + w], p2, false));
      v[2 * w + 1] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[2 * q + w], p2, true));
    }
    o.k[q] = __builtin_bit_cast(bf16x8, u32x4{v[0], v[1], v[2], v[3]});
  }
  return o;
}
LORA_DEV f32x4 mfma16x16x32_bf16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// A token's scale 2^(e - 127) and W's: as much of the first as keeps every
// value and product a normal number goes into the token's operand (2^-100 to
// 2^100), the rest (1 for blocks of 1e-28 to 5e32) into the factor of the sum.
struct TokenScale {
  float x, sum;
  LORA_DEV TokenScale(int e, float w) {
    const int in = min(max(e, 27), 227);
    x = __uint_as_float((uint32_t)in << 23);
    sum = ldexpf(w, e - in);
  }
};
template <int J>
LORA_DEV TokenScale scale_at(const u32x2& ex, float w) {
  return TokenScale((int)((ex[J / 4] >> (8 * (J % 4))) & 0xffu), w);
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <typename F, int... J>
LORA_DEV void unrolled_(F f, std::integer_sequence<int, J...>) {
  (f(std::integral_constant<int, J>{}), ...);
}
template <int N, typename F>
LORA_DEV void unrolled(F f) {
  unrolled_(f, std::make_integer_sequence<int, N>{});
}

// LDS bytes that no load in flight writes (restrict): without that the
// compiler waits for every direct-to-LDS load before each read.
LORA_DEV i32x8 frag_rows(const lds_u8* __restrict__ p, int lo, int hi) {
  const u32x4 a = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(p + lo);
  const u32x4 b = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(p + hi);
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}
LORA_DEV u32x2 lds_pair(const lds_u8* __restrict__ p, int at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x2*>(p + at);
}
// Four transpose reads: rows +0, +8, +64, +72 of the lane's base.
LORA_DEV i32x8 frag_cols(const lds_u8* __restrict__ p, int row_bytes) {
  typedef int v2 __attribute__((ext_vector_type(2)));
  i32x8 r;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const v2 t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (__attribute__((address_space(3))) v2*)(p + ((q >> 1) * 64 + (q & 1) * 8) * row_bytes));
    r[2 * q] = t[0];
    r[2 * q + 1] = t[1];
  }
  return r;
}

LORA_DEV uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2_t));
}

// Eight neighbours of a row of n float32 values (a multiple of 4 of them) from
// index k, as bf16 (zero past the row).
LORA_DEV u32x4 row_bf16(const float* row, int64_t k, int64_t n, float mul) {
  f32x4 v[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const bool in = k + 4 * q < n;
    const f32x4 x = *reinterpret_cast<const f32x4*>(row + (in ? k + 4 * q : 0)) * mul;
    v[q] = in ? x : f32x4{0, 0, 0, 0};   // not a product with 0: x may be infinite
  }
  return u32x4{pack2(v[0][0], v[0][1]), pack2(v[0][2], v[0][3]), pack2(v[1][0], v[1][1]),
               pack2(v[1][2], v[1][3])};
}
// Eight values of a column, ld apart.
LORA_DEV u32x4 col_bf16(const float* col, int64_t k, int64_t n, int64_t ld) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool in = k + e < n;
    const float x = col[(in ? k + e : 0) * ld];   // unconditional: no wait in between
    v[e] = in ? x : 0.0f;
  }
  return u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
}

// OUT: 0 float32, 1 bf16 (round to nearest even), 2 float32 partials, 3
// float32 with the LoRA term, whose factors are rounded to bf16 as in the
// products over a bf16 W.
template <int BM, int BN, int WM, int WN, int NS, bool DX, int OUT>
__global__ __launch_bounds__(64 * WM * WN) void fp8_gemm_kernel(Fp8Args p) {
#if defined(__HIP_DEVICE_COMPILE__)   // the host pass has no use for the body
  constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int XB = BM * 128, WB = BN * 128, STAGE = XB + WB + 1024;   // X, W, exponents
  constexpr int XL = XB / 1024 / NW, WL = WB / 1024 / NW;   // loads a wave and stage
  static_assert(XB % (1024 * NW) == 0 && WB % (1024 * NW) == 0, "whole loads per wave");
  static_assert(TM >= 1 && TN >= 1 && (BN / WN) <= 128 && 128 % (BN / WN) == 0, "one W scale a wave");
  __shared__ __align__(1024) uint8_t smem[NS * STAGE];
  lds_u8* lds = (lds_u8*)smem;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int64_t ntm = (p.M + BM - 1) / BM, ntn = (p.Nc + BN - 1) / BN;
  const int64_t g = xcd_tile(blockIdx.x, ntm * ntn * p.nsplit);
  const int split = __builtin_amdgcn_readfirstlane((int)(g / (ntm * ntn)));
  int64_t tm, tn;
  grouped_tile(g % (ntm * ntn), ntm, ntn, tm, tn);
  tm = __builtin_amdgcn_readfirstlane((int)tm);
  tn = __builtin_amdgcn_readfirstlane((int)tn);
  const int64_t m0 = tm * BM, n0 = tn * BN;
  const int kb0 = split * p.per, nk = min(p.per, p.nk - kb0);
  const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);

  // Resources at the tile's first row.  Rows of the tile past the operand's
  // end repeat its last one (W has whole 128-blocks, but a 256-wide tile may
  // pass them): their results are not stored.
  const int64_t xbytes = (p.M - m0) * p.ldq;
  const __amdgpu_buffer_rsrc_t rX = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.Q + m0 * p.ldq), (short)0, (int)(xbytes > 0x7fffffffll ? 0x7fffffff : xbytes), 0x00020000);
  const int64_t wrows = (DX ? (int64_t)p.nk * 128 : (p.Nc + 127) / 128 * 128) - (DX ? 0 : n0);
  const int64_t wbytes = wrows * p.ldw - (DX ? n0 : 0);
  const __amdgpu_buffer_rsrc_t rW = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.W + (DX ? n0 : n0 * p.ldw)), (short)0,
      (int)(wbytes > 0x7fffffffll ? 0x7fffffff : wbytes), 0x00020000);
  uint32_t vx[XL], vw[WL];
#pragma unroll
  for (int q = 0; q < XL; ++q) {
    const int row = 8 * (wave * XL + q) + (lane >> 3);
    vx[q] = (uint32_t)(min((int64_t)row, p.M - 1 - m0) * p.ldq) + 16 * ((lane & 7) ^ (row & 7));
  }
#pragma unroll
  for (int q = 0; q < WL; ++q) {
    if constexpr (DX) {
      constexpr int CPR = BN / 16;
      const int slot = 64 * (wave * WL + q) + lane, row = slot / CPR, ch = (slot % CPR) ^ (row & 7);
      // Columns past the last 128-block: the tile's first ones instead.
      vw[q] = (uint32_t)(row * p.ldw) + (n0 + 16 * ch < (p.Nc + 127) / 128 * 128 ? 16 * ch : 0);
    } else {
      const int row = 8 * (wave * WL + q) + (lane >> 3);
      vw[q] = (uint32_t)(min((int64_t)row, wrows - 1) * p.ldw) + 16 * ((lane & 7) ^ (row & 7));
    }
  }
  // Exponents: the (up to two) whole groups of 128 tokens that hold the tile.
  const int64_t mg = m0 & ~(int64_t)127;
  const __amdgpu_buffer_rsrc_t rE = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.E + mg), (short)0, (int)((int64_t)p.nk * p.lde - mg), 0x00020000);
  const uint32_t ve = (uint32_t)min((int64_t)4 * lane, p.lde - mg - 4);
  auto dma = [&](int k, int buf) {
    const int kk = kb0 + min(k, nk - 1);
    const int sx = kk * 128;
    const uint32_t sw = DX ? (uint32_t)kk * 128u * (uint32_t)p.ldw : (uint32_t)kk * 128u;
    uint8_t* b = smem + buf * STAGE;
#pragma unroll
    for (int q = 0; q < XL; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rX, (__attribute__((address_space(3))) void*)(b + 1024 * (wave * XL + q)), 16, vx[q], sx, 0, 0);
#pragma unroll
    for (int q = 0; q < WL; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rW, (__attribute__((address_space(3))) void*)(b + XB + 1024 * (wave * WL + q)), 16, vw[q],
          (int)sw, 0, 0);
    if (wave == 0)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rE, (__attribute__((address_space(3))) void*)(b + XB + WB), 4, ve, (int)(kk * p.lde), 0, 0);
  };
  const int64_t sblk = (n0 + wn) / 128;
  const float* sp = p.S + min(sblk, (p.Nc - 1) / 128) * (DX ? 1 : p.lds_);
  // (constant address space: a scalar load, off the vector memory counter)
  typedef const __attribute__((address_space(4))) float* const_f32;
  auto wscale = [&](int k) {
    const int kk = kb0 + min(k, nk - 1);
    return ((const_f32)sp)[DX ? (int64_t)kk * p.lds_ : (int64_t)kk];
  };

  // Fragment addresses within a stage.
  int xo[2], wo[2];
  xo[0] = c * 128 + 16 * (h ^ (c & 7));
  xo[1] = c * 128 + 16 * ((h + 4) ^ (c & 7));
  const int mrow = c >> 1;   // dX: the lane's row of eight, and half of a chunk
  wo[0] = DX ? (16 * h + mrow) * BN + 8 * (c & 1) : xo[0];
  wo[1] = xo[1];

  // Exponents of this wave's TM token tiles, tile j in byte j.
  const int eo = (int)(m0 + wm - mg);
  auto exponents = [&](const lds_u8* e) {
    const u32x2 w = lds_pair(e, (eo & ~127) + 8 * c);
    if constexpr (TM == 8) return w;
    const uint64_t all = ((uint64_t)w[1] << 32) | w[0];
    return u32x2{(uint32_t)(all >> (8 * ((eo >> 4) & 7))), 0u};
  };
  static_assert(TM == 8 || TM <= 4, "exponents of a wave in one word, or in two whole ones");

  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

#pragma unroll
  for (int s = 0; s < NS - 1; ++s) dma(s, s);
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  int cur = 0;
  float sw = wscale(0);
  for (int k = 0; k < nk; ++k) {
    const int nxt = cur == 0 ? NS - 1 : cur - 1;   // (cur + NS - 1) % NS
    dma(k + NS - 1, nxt);
    const lds_u8* X = lds + cur * STAGE + wm * 128;
    const lds_u8* W = lds + cur * STAGE + XB;
    const u32x2 ex = exponents(W + WB);
    Wide w[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      if constexpr (DX) {
        const int ch = (wn >> 4) + i;
        w[i] = widen(frag_cols(W + wo[0] + 16 * ((ch & ~7) | ((ch ^ mrow) & 7)), BN), 1.0f);
      } else {
        w[i] = widen(frag_rows(W + (wn + 16 * i) * 128, wo[0], wo[1]), 1.0f);
      }
    }
    // A wave whose MFMAs are ready goes before one that widens: the two waves
    // of a SIMD of the 256-wide tile part by it (dX of 4096 x [4096 -> 2560]:
    // 80 -> 75 us).  The 128-wide tile's two blocks are apart already (82 -> 84).
    unrolled<TM>([&](auto J_) {
      constexpr int J = decltype(J_)::value;
      const TokenScale ts = scale_at<J>(ex, sw);
      const Wide x = widen(frag_rows(X + 16 * J * 128, xo[0], xo[1]), ts.x);
      f32x4 d[TN];
      if constexpr (TM == 8) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < TN; ++i)
          d[i] = mfma16x16x32_bf16(w[i].k[q], x.k[q], q ? d[i] : f32x4{0, 0, 0, 0});
      if constexpr (TM == 8) __builtin_amdgcn_s_setprio(0);
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][J][v] = fmaf(d[i][v], ts.sum, acc[i][J][v]);
    });
    sw = wscale(k + 1);
    // Stage k + 1 is in once only the later stages' loads remain.
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * (XL + WL)) : "memory");
    cur = cur + 1 == NS ? 0 : cur + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // Tile (i, j) holds columns n0 + wn + 16 i + 4 h + v of token 16 j + c.
  const int64_t nb = n0 + wn;
  if constexpr (OUT == 3) {
    const Fp8Lora& l = p.lora;
    int64_t t[TM];
    uint32_t keep[TM];   // dX: mask bits of the lane's 4 TN results a token
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      t[j] = min(m0 + wm + 16 * j + c, p.M - 1);
      keep[j] = 0xffffffffu;
      if (DX && l.drop.on) {
        const uint64_t row = drop_row(l.drop, t[j]);
        keep[j] = 0;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            keep[j] |= (uint32_t)drop_keep(l.drop, row, nb + 16 * i + 4 * h + v) << (4 * i + v);
      }
    }
    const float mul = DX && l.drop.on ? l.drop.keep : 1.0f;
    for (int64_t k = 0; k < l.r; k += 32) {
      bf16x8 b[TN], u[TM];
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int64_t n = min(nb + 16 * i + c, p.Nc - 1);
        b[i] = __builtin_bit_cast(bf16x8, DX ? col_bf16(l.lb + n, k + 8 * h, l.r, p.Nc)
                                             : row_bf16(l.lb + n * l.r, k + 8 * h, l.r, 1.0f));
      }
#pragma unroll
      for (int j = 0; j < TM; ++j)
        u[j] = __builtin_bit_cast(bf16x8, row_bf16(l.lu + t[j] * l.r, k + 8 * h, l.r, l.ls * mul));
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int i = 0; i < TN; ++i) {
          if constexpr (DX) {
            const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[i], u[j], f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] += (keep[j] >> (4 * i + v)) & 1 ? d[v] : 0.0f;
          } else {
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[i], u[j], acc[i][j], 0, 0, 0);
          }
        }
    }
  }
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t t = m0 + wm + 16 * j + c;
    const bool in = t < p.M;
    if constexpr (OUT == 1) {
      uint16_t* row = (uint16_t*)p.C + (in ? t : 0) * p.ldc;
      if (TN % 2 == 0 && p.ldc % 8 == 0) {
        // Tiles i and i + 1 swap between neighbouring lane groups, so that a
        // lane stores eight columns of one of them.
#pragma unroll
        for (int i = 0; i + 1 < TN; i += 2) {
          uint32_t a[2], b[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t x = pack2(acc[i][j][2 * q], acc[i][j][2 * q + 1]);
            const uint32_t y = pack2(acc[i + 1][j][2 * q], acc[i + 1][j][2 * q + 1]);
            const u32x2 s = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x, y, false, false));
            a[q] = s[0];
            b[q] = s[1];
          }
          const int64_t n = nb + 16 * (i + (h & 1)) + 8 * (h >> 1);
          if (in && n < p.Nc) *reinterpret_cast<u32x4*>(row + n) = u32x4{a[0], a[1], b[0], b[1]};
        }
      } else {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int64_t n = nb + 16 * i + 4 * h + v;
            if (in && n < p.Nc) row[n] = (uint16_t)f32_to_bf16_bits(acc[i][j][v]);
          }
      }
    } else {
      float* row = OUT == 2 ? p.part + ((int64_t)split * p.M + (in ? t : 0)) * p.Nc
                            : (float*)p.C + (in ? t : 0) * p.ldc;
      float* row2 = OUT == 3 && p.C2 ? p.C2 + (in ? t : 0) * p.Nc : nullptr;
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int64_t n = nb + 16 * i + 4 * h;
        if ((OUT == 2 ? p.Nc : p.ldc) % 4 == 0) {
          if (in && n < p.Nc) *reinterpret_cast<f32x4*>(row + n) = acc[i][j];
          if (row2 && in && n < p.Nc) *reinterpret_cast<f32x4*>(row2 + n) = acc[i][j];
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (in && n + v < p.Nc) row[n + v] = acc[i][j][v];
        }
      }
    }
  }
#endif
}

// Forward for up to 16 tokens (serving's single one, the shortest chunks):
// bound by W's bytes and by latency, so no LDS stages and no second launch.  A
// block takes 16 columns; its eight waves take every eighth contraction step,
// with the next two steps' fragments loading straight into registers, and
// their sums meet in LDS in wave order.  W's rows are read in 64-byte pieces,
// two of a step making whole lines.  One token of [2560 -> 4096]: 5.3 us for
// 10.5 MB (2.0 TB/s, with the launch).
template <bool BF16>
__global__ __launch_bounds__(512) void fp8_few_kernel(Fp8Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = 8;
  __shared__ f32x4 sum[NW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const uint8_t* wrow = p.W + (n0 + c) * p.ldw + 16 * h;   // W has whole 128-blocks
  const int64_t tc = min((int64_t)c, p.M - 1);
  const uint8_t* xrow = p.Q + tc * p.ldq + 16 * h;
  const uint8_t* erow = p.E + fp8_scale_at(tc);
  const float* sp = p.S + (n0 / 128) * p.lds_;
  struct Step {
    u32x4 w[2], x[2];
    int e;
    float s;
  };
  auto load = [&](Step& f, int k) {
    const int64_t kk = min(k, p.nk - 1);   // past the end: the last step again, not added
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f.w[q] = *reinterpret_cast<const u32x4*>(wrow + 128 * kk + 64 * q);
      f.x[q] = *reinterpret_cast<const u32x4*>(xrow + 128 * kk + 64 * q);
    }
    f.e = erow[kk * p.lde];
    f.s = sp[kk];
  };
  f32x4 acc = {0, 0, 0, 0};
  auto frag = [](const u32x4(&v)[2]) {
    return i32x8{(int)v[0][0], (int)v[0][1], (int)v[0][2], (int)v[0][3],
                 (int)v[1][0], (int)v[1][1], (int)v[1][2], (int)v[1][3]};
  };
  auto add = [&](const Step& f) {
    const TokenScale ts(f.e, f.s);
    const Wide w = widen(frag(f.w), 1.0f), x = widen(frag(f.x), ts.x);
    f32x4 d = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) d = mfma16x16x32_bf16(w.k[q], x.k[q], d);
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = fmaf(d[v], ts.sum, acc[v]);
  };
  Step a, b, d;
  int k = wave;
  load(a, k);
  load(b, k + NW);
  while (k < p.nk) {   // three steps take turns
    load(d, k + 2 * NW);
    add(a);
    if ((k += NW) >= p.nk) break;
    load(a, k + 2 * NW);
    add(b);
    if ((k += NW) >= p.nk) break;
    load(b, k + 2 * NW);
    add(d);
    k += NW;
  }
  sum[wave][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  f32x4 r = sum[0][lane];
#pragma unroll
  for (int w = 1; w < NW; ++w) r += sum[w][lane];
  const int64_t n = n0 + 4 * h;
  if (c >= p.M) return;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (n + v < p.Nc) {
      if constexpr (BF16) ((uint16_t*)p.C)[c * p.Nc + n + v] = (uint16_t)f32_to_bf16_bits(r[v]);
      else ((float*)p.C)[c * p.Nc + n + v] = r[v];
    }
#endif
}

// The splits' partials in split order.
template <bool BF16>
__global__ __launch_bounds__(256) void fp8_reduce_kernel(const float* __restrict__ part, int64_t n,
                                                         int nsplit, void* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  if (n % 4 == 0) {
    const f32x4 s = sum_parts4(part, n, nsplit, i);
    if constexpr (BF16) *reinterpret_cast<u32x2*>((uint16_t*)out + i) = u32x2{pack2(s[0], s[1]), pack2(s[2], s[3])};
    else *reinterpret_cast<f32x4*>((float*)out + i) = s;
  } else {
    for (int64_t e = i; e < min(n, i + 4); ++e) {
      const float s = sum_parts1(part, n, nsplit, e);
      if constexpr (BF16) ((uint16_t*)out)[e] = (uint16_t)f32_to_bf16_bits(s);
      else ((float*)out)[e] = s;
    }
  }
}

// ------------------------------------------------------------------ rounding
struct Fp8QuantArgs {
  const void* X;         // [rows, ldx]
  uint8_t* Q;            // [rows, ldq], ldq a multiple of 128
  uint8_t* E;            // [ldq / 128, lde], lde = rows rounded up to 128
  int64_t rows, cols, ldx, ldq, lde;
};

// The biased exponent of the smallest power of two 2^e with amax <= 448 2^e
// (448 = 1.75 2^8 is the largest e4m3 value), at least 2^-127.
LORA_DEV int fp8_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int ex = (int)(u >> 23);   // amax = 1.m 2^(ex - 127); 0 for subnormals
  const int e = ex - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(0, min(254, e));
}

// A block of 128 in 16 lanes of eight; four blocks a wave.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void fp8_quant_kernel(Fp8QuantArgs p) {
  const int lane = threadIdx.x & 15;
  const int64_t nb = p.ldq / 128;
  const int64_t id = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (id >= p.rows * nb) return;   // whole groups of 16 lanes
  const int64_t row = id / nb, b = id % nb, col = b * 128 + 8 * lane;
  const T* src = (const T*)p.X + row * p.ldx + col;
  float x[8];
  if constexpr (VEC && sizeof(T) == 4) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const f32x4 v = col + 4 * q < p.cols ? *reinterpret_cast<const f32x4*>(src + 4 * q) : f32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * q + e] = v[e];
    }
  } else if constexpr (VEC) {
    const u32x4 v = col < p.cols ? *reinterpret_cast<const u32x4*>(src) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(v[e] << 16);
      x[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (sizeof(T) == 4) x[e] = col + e < p.cols ? (float)src[e] : 0.0f;
      else x[e] = col + e < p.cols ? bf16_bits_to_f32(src[e]) : 0.0f;
    }
  }
  float amax = 0.0f;
  bool bad = false;   // a NaN or an infinity
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    amax = fmaxf(amax, fabsf(x[e]));
    bad = bad || !(fabsf(x[e]) <= 3.402823466e38f);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
  const int e = fp8_exp(amax);
  u32x2 q;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = ldexpf(x[4 * i + k], 127 - e);
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], r, true);
    q[i] = (uint32_t)r;
  }
  if (bad) {   // e4m3 has no infinity: both become its NaN
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (!(fabsf(x[k]) <= 3.402823466e38f)) q[k >> 2] |= 0x7fu << (8 * (k & 3));
  }
  *reinterpret_cast<u32x2*>(p.Q + row * p.ldq + col) = q;
  if (lane == 0) p.E[b * p.lde + fp8_scale_at(row)] = (uint8_t)e;
}

}  // namespace lora
