// Few-token product with a 4-bit group weight: y[t][n] = sum_k x[t][k] W[n][k].
//
//   sum_k x W = sum_groups ( s sum_k x c + m sum_k x )
//
// The inner sums are MFMA 16x16x32 products: A = x (16 tokens), B = the
// codes of 16 rows n as 16-bit floats OFF + c (u4_common.h), accumulated
// over one group and then scaled in fp32.  sum_k x is a product of the same
// x operand with ones, so a group adds
//   acc += s d + (m - OFF s) X,   d = sum x (OFF + c), X = sum x.
//
// Bound by HBM on the codes at few tokens.  A block owns 16 R rows and all
// of K: its W waves split K, keep fp32 sums and add them in wave order
// through LDS at the end, so nothing is left for a second launch and every
// run gives the same bits.  R is chosen so that the blocks fill the chip in
// whole rounds: x is read by every block, and a last round of few blocks
// costs as much as a full one.
//
// A wave walks units of 256 elements (128 with four token tiles).  Of a unit
// x becomes operands in registers once, then the block's row tiles follow.
// Codes, pairs and x are read in the order of memory, with neighbouring
// lanes on neighbouring 16 bytes, and brought into operand order (lane l:
// row l % 16, a quarter l / 16 of each group) through the wave's own LDS:
// lanes that each read a row of their own cost the address unit a cycle
// each, 64 for an instruction, and took 24 us where this takes 14 (M 16,
// N 8192, K 8192, groups of 128; a copy of the same bytes takes 7.6).  The
// pairs of a unit are one load: read group by group they were as many
// requests as the codes.
//
// Measured (graph replays, weights from HBM; in brackets a copy of the same
// bytes): M 1, 4096 x 4096, groups of 64: 4.8 us (2.0); M 1, 8192 x 8192:
// 10.5 (7.9); M 4, 22016 x 8192: 25 (21.3); M 16, 8192 x 8192: 14.4 (7.6);
// M 61, 11008 x 4096, groups of 32: 25 (6.3).  Neither of the last two is
// bound by one unit.  While its two waves are there, a SIMD's vector
// instructions take 40 % of the time (M 16) and 39 % (M 61), its matrix core 13
// and 21 %, the LDS that the block's eight waves share 34 and 40 %, and a wave
// waits for 45 and 33 % of it: two waves a SIMD are too few to hide one behind
// the others, and every block reads all of x, at M 16 twice the codes' bytes.

#include "launch.h"
#include "u4_common.h"

namespace qlora {
namespace {

// A wave's own LDS.  x is staged before the codes of a unit are, 16 tokens
// and 128 elements at a time, so both have the same place.
template <int G, int NT>
struct Stage {
  static constexpr int kUnit = NT < 4 ? 256 : 128;  // elements of K taken at a time
  static constexpr int kPieces = kUnit / 32;  // 16-byte pieces of a row's codes
  static constexpr int kPairs = kUnit / G;    // pairs of a row
  struct Codes {
    u32x4_t c[16][kPieces];
    uint32_t p[16][kPairs];
  };
  union {
    Codes w;
    u32x4_t x[16][16];
  };
  f32x4_t X[kPairs][4 * NT];  // sums of x over the unit's groups
};

template <class DT, int G, int NT, int XQ, int TI, int W>
__global__ __launch_bounds__(64 * W) void linear_u4_kernel(
    const uint8_t* __restrict__ codes, const uint32_t* __restrict__ pairs,
    const uint16_t* __restrict__ x, int64_t ldx, uint16_t* __restrict__ y, int64_t ldy, int64_t M,
    int64_t N, int64_t K, int R) {
  using S = Stage<G, NT>;
  constexpr int U = S::kUnit;
  constexpr int C = G / 32;         // products per group
  constexpr int XS = U / 32;        // products per unit
  constexpr int XP = U / 128;       // pieces of x per unit
  constexpr int LPR = S::kPieces;   // lanes per row of codes
  constexpr int NC = LPR / 4;       // loads of codes per tile
  constexpr int NP = (S::kPairs + 3) / 4;  // loads of pairs per tile
  __shared__ S stage[W];
  extern __shared__ f32x4_t sums[];  // [W][R * NT][64]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R), m0 = (int64_t)blockIdx.y * (16 * NT);
  const int groups = (int)(K / G), units = (int)((K + U - 1) / U);
  const int u0 = (int)((int64_t)units * wave / W), u1 = (int)((int64_t)units * (wave + 1) / W);
  S& st = stage[wave];
  f32x4_t* acc = sums + (int64_t)wave * R * NT * 64 + lane;

  // Fetching: neighbouring lanes take neighbouring 16-byte pieces of a row.
  // The buffers end with the block's last row and token, and what is read
  // past the end is zero; past the end of a row is the next one, whose values
  // meet no group.  Every lane's offsets are worked out once: a load costs an
  // addition.
  const int cr = lane / LPR, cs = lane % LPR;  // codes: row of 64 / LPR, piece
  const int pr = lane >> 2, ps = lane & 3;     // pairs: row, pair of four
  const int xr = lane >> 4, xs = lane & 15;    // x: token of four, piece
  const uint32_t krow = (uint32_t)(K / 2), prow = (uint32_t)groups * 4;
  const uint32_t xrow = (uint32_t)ldx * 2;
  const uint32_t rows = (uint32_t)min(N - n0, (int64_t)(16 * R));
  const uint32_t toks = (uint32_t)min(M - m0, (int64_t)(16 * NT));
  const auto cbuf = make_rsrc(codes + n0 * (K / 2), rows * krow);
  const auto pbuf = make_rsrc(pairs + n0 * groups, rows * prow);
  const auto xbuf = make_rsrc(x + m0 * ldx, (toks - 1) * xrow + (uint32_t)K * 2);
  const uint32_t co = cr * krow + cs * 16, po = pr * prow + ps * 4, xo0 = xr * xrow + xs * 16;

  u32x4_t cv[NC];
  uint32_t pv[NP];
  auto load_w = [&](int u, int r) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      cv[i] = buffer_load16(cbuf, co + ((16 * r + (64 / LPR) * i) * krow + u * (U / 2)));
#pragma unroll
    for (int i = 0; i < NP; ++i)
      pv[i] = __builtin_amdgcn_raw_buffer_load_b32(
          pbuf, (int)(po + (16 * r * prow + (u * S::kPairs + 4 * i) * 4)), 0, 0);
  };
  // The pieces' places are exchanged within a row so that the 16 rows of an
  // operand read lie in different banks.
  auto place = [](int row, int piece) {
    return LPR == 8 ? piece ^ (row >> 1) : piece ^ (row >> 2);
  };
  auto store_w = [&] {
    wave_exchange();  // the place's last reads: of x, or of the tile before
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int row = (64 / LPR) * i + cr;
      st.w.c[row][place(row, cs)] = cv[i];
    }
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (4 * i + ps < S::kPairs) st.w.p[pr][4 * i + ps] = pv[i];
    wave_exchange();
  };

  const u32x4_t ones = {U4Mfma<DT>::kOne, U4Mfma<DT>::kOne, U4Mfma<DT>::kOne, U4Mfma<DT>::kOne};
  u32x4_t xo[XS][NT];  // x of the unit as operands
  u32x4_t xv[XP][XQ];  // x of the next unit: four tokens each
  auto load_x = [&](int u) {
#pragma unroll
    for (int q = 0; q < XP; ++q)
#pragma unroll
      for (int t = 0; t < XQ; ++t)
        xv[q][t] = buffer_load16(xbuf, xo0 + (4 * t * xrow + u * U * 2 + 256 * q));
  };
  auto order_x = [&] {
    wave_exchange();  // the last tile's reads
#pragma unroll
    for (int q = 0; q < XP; ++q) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * t + i < XQ) st.x[4 * i + xr][xs ^ (4 * i + xr)] = xv[q][4 * t + i];
        wave_exchange();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // product 4 q + c: of group g of the piece the lane's quarter
          const int g = c / C, e = c % C;
          xo[4 * q + c][t] = u4_order8(st.x[lr][(g * (G / 8) + lg * C + e) ^ lr]);
        }
        wave_exchange();
      }
    }
    // a group's sums: the product with ones, whose columns are all alike
#pragma unroll
    for (int g = 0; g < S::kPairs; ++g)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4_t s = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < C; ++c) s = DT::mfma16(xo[g * C + c][t], ones, s);
        if (lr == 0) st.X[g][4 * t + lg] = s;
      }
  };

  // one tile of 16 rows over one unit
  auto work = [&](int u, int r, bool first, bool all) {
    uint32_t cw[S::kPairs][C], pair[S::kPairs];
#pragma unroll
    for (int g = 0; g < S::kPairs; ++g) {
      // the lane's G / 8 bytes of row lr
      const int byte = g * (G / 2) + lg * (G / 8);
      __builtin_memcpy(cw[g],
                       __builtin_assume_aligned(reinterpret_cast<const uint8_t*>(
                                                    &st.w.c[lr][place(lr, byte >> 4)]) +
                                                    (byte & 15),
                                                4 * C),
                       4 * C);
      pair[g] = st.w.p[lr][g];
    }
    f32x4_t a[NT], d[S::kPairs][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) a[t] = first ? f32x4_t{0, 0, 0, 0} : acc[(r * NT + t) * 64];
#pragma unroll
    for (int g = 0; g < S::kPairs; ++g)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const u32x4_t b = u4_expand8<U4Mfma<DT>>(cw[g][c]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          d[g][t] = DT::mfma16(xo[g * C + c][t], b, c ? d[g][t] : f32x4_t{0, 0, 0, 0});
      }
    // (m - OFF s) X: where a unit has four groups or more and there are more
    // tokens than 16, as an fp32 product whose k-slots are four groups (lane:
    // group 4 e + l / 16), for the vector instructions bound the kernel there
    // (N 11008, K 4096, groups of 32: M 61 28.0 us without, 24.9 with; M 32
    // 23.0 and 20.0).  With fewer groups slots are empty and it is slower (M 61,
    // groups of 128: 20.8 us without, 21.9 with).
    constexpr bool kSlots = NT > 1 && S::kPairs >= 4;
    if constexpr (kSlots) {
#pragma unroll
      for (int e = 0; e < S::kPairs / 4; ++e) {
        const int g = 4 * e + lg;
        const bool valid = all || u * S::kPairs + g < groups;
        const uint32_t w = st.w.p[lr][g];
        const float m = valid ? fmaf(-U4Mfma<DT>::kOff, u4_s(w), u4_m(w)) : 0.0f;
        const float* X = reinterpret_cast<const float*>(st.X[g]) + lr;
#pragma unroll
        for (int t = 0; t < NT; ++t)
          a[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(valid ? X[16 * t] : 0.0f, m, a[t], 0, 0, 0);
      }
    }
#pragma unroll
    for (int g = 0; g < S::kPairs; ++g) {
      if (!all && u * S::kPairs + g >= groups) break;
      const float s = u4_s(pair[g]), m = fmaf(-U4Mfma<DT>::kOff, s, u4_m(pair[g]));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4_t X = {0, 0, 0, 0};
        if constexpr (!kSlots) X = st.X[g][4 * t + lg];
#pragma unroll
        for (int i = 0; i < TI; ++i)
          a[t][i] = fmaf(s, d[g][t][i], kSlots ? a[t][i] : fmaf(m, X[i], a[t][i]));
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[(r * NT + t) * 64] = a[t];
  };

  // A wave's stage is its own, so it needs no barrier of the block.
  // The next tile's codes and the next unit's x are on their way during a
  // tile's work.
  if (u0 < u1) {
    load_x(u0);
    load_w(u0, 0);
    for (int u = u0; u < u1; ++u) {
      order_x();
      if (u + 1 < u1) load_x(u + 1);
      for (int r = 0; r < R; ++r) {
        store_w();
        if (r + 1 < R)
          load_w(u, r + 1);
        else if (u + 1 < u1)
          load_w(u + 1, 0);
        if ((u + 1) * U <= (int)K)
          work(u, r, u == u0, true);
        else
          work(u, r, u == u0, false);
      }
    }
  } else {
    for (int r = 0; r < R * NT; ++r) acc[r * 64] = f32x4_t{0, 0, 0, 0};
  }
  __syncthreads();
  // sum i of lane l of tile (r, t) is token 16 t + 4 (l / 16) + i, row
  // 16 r + l % 16: neighbouring threads take neighbouring rows of one token
  const float* red = reinterpret_cast<const float*>(sums);
  for (int o = threadIdx.x; o < R * NT * 256; o += 64 * W) {
    const int n = o & 15, tok = (o >> 4) & 15, tile = o >> 8;
    const int r = tile / NT, t = tile - r * NT;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < W; ++q)
      v += red[((q * R * NT + tile) * 64 + (tok >> 2) * 16 + n) * 4 + (tok & 3)];
    const int64_t row = n0 + 16 * r + n, m = m0 + 16 * t + tok;
    if (row < N && m < M) y[m * ldy + row] = DT::cvt(v);
  }
}

template <class DT, int G, int NT, int XQ, int TI, int W, int CAP>
void go(const uint8_t* codes, const uint32_t* pairs, const uint16_t* x, int64_t ldx, uint16_t* y,
        int64_t ldy, int64_t M, int64_t N, int64_t K, int R, hipStream_t s) {
  static_assert(W * (sizeof(Stage<G, NT>) + CAP * NT * 1024) <= 160 * 1024, "LDS of a CU");
  const dim3 grid((unsigned)((N + 16 * R - 1) / (16 * R)), (unsigned)((M + 16 * NT - 1) / (16 * NT)));
  linear_u4_kernel<DT, G, NT, XQ, TI, W><<<grid, 64 * W, (size_t)W * R * NT * 1024, s>>>(
      codes, pairs, x, ldx, y, ldy, M, N, K, R);
}

// Row tiles per block: as few rounds of the chip as `cap` tiles of LDS allow,
// and these filled (`slots` blocks run at once).
int tiles_per_block(int64_t N, int slots, int cap) {
  const int64_t tiles = (N + 15) / 16, per = (int64_t)slots * cap;
  const int64_t rounds = (tiles + per - 1) / per;
  return (int)((tiles + slots * rounds - 1) / (slots * rounds));
}

template <class DT, int G>
void pick(const uint8_t* codes, const uint32_t* pairs, const uint16_t* x, int64_t ldx, uint16_t* y,
          int64_t ldy, int64_t M, int64_t N, int64_t K, hipStream_t s) {
#define QLORA_U4_GO(NT, XQ, TI, W, CAP, PER_CU)                                              \
  return go<DT, G, NT, XQ, TI, W, CAP>(codes, pairs, x, ldx, y, ldy, M, N, K,             \
                                       tiles_per_block(N, 256 * (PER_CU), CAP), s)
  const int64_t units = (K + 255) / 256;
  if (M <= 4) {
    // 16 waves a block (one block per CU) where each still has a unit and
    // three row tiles a block hold all rows; else 8 (two per CU), or 4 for a
    // short K.  N 8192, K 8192, M 1: 10.5 us against 12.5 with 8 waves;
    // N 22016: 24.3 against 21.1; N 2048, K 1024: 4.1, 3.3 with 8, 2.8 with 4.
    // Groups of 32 need the registers of 8 waves (N 4096, M 2: 7.1 against 5.9).
    if constexpr (G > 32) {
      if (units >= 16 && N <= 16 * 256 * 3) {
        if (M == 1) QLORA_U4_GO(1, 1, 1, 16, 3, 1);
        QLORA_U4_GO(1, 1, 4, 16, 3, 1);
      }
    }
    if (M == 1) {
      if (units >= 8) QLORA_U4_GO(1, 1, 1, 8, 4, 2);
      QLORA_U4_GO(1, 1, 1, 4, 4, 4);
    }
    if (units >= 8) QLORA_U4_GO(1, 1, 4, 8, 4, 2);
    QLORA_U4_GO(1, 1, 4, 4, 4, 4);
  }
  // more tokens: x is most of what a block reads, so a block keeps as many
  // rows as it can (M 16, N 22016, K 8192: 27.6 us with six tiles, 32.1 with
  // three).  With groups of 32 the variant for 17 to 32 tokens has all 256
  // registers and 28 more in scratch memory, some of them in the loop over K
  // (N 11008, K 4096, M 32: 20.0 us).
  if (M <= 16) QLORA_U4_GO(1, 4, 4, 8, 8, 1);
  if (M <= 32) QLORA_U4_GO(2, 8, 4, 8, 6, 1);
  QLORA_U4_GO(4, 16, 4, 8, 3, 1);
#undef QLORA_U4_GO
}

}  // namespace

hipError_t launch_linear_u4(const uint8_t* codes, const uint32_t* pairs, int group,
                            const uint16_t* x, int64_t ldx, uint16_t* y, int64_t ldy, int64_t M,
                            int64_t N, int64_t K, bool f16, hipStream_t s) {
  auto by_group = [&](auto dt) {
    using DT = decltype(dt);
    if (group == 32)
      pick<DT, 32>(codes, pairs, x, ldx, y, ldy, M, N, K, s);
    else if (group == 64)
      pick<DT, 64>(codes, pairs, x, ldx, y, ldy, M, N, K, s);
    else
      pick<DT, 128>(codes, pairs, x, ldx, y, ldy, M, N, K, s);
  };
  if (f16)
    by_group(F16T{});
  else
    by_group(Bf16T{});
  return hipGetLastError();
}

}  // namespace qlora
