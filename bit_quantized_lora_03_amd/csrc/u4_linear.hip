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
// Bound by HBM on the codes.  A block owns 16 R rows and all of K: its W
// waves split the groups, keep fp32 sums in registers and add them in wave
// order through LDS at the end, so nothing is left for a second launch and
// every run gives the same bits.  Lane l holds row l % 16 of a tile and, of
// each group, the quarter l / 16: x, codes and pair come straight from
// global memory in the operand's layout, without LDS.

#include "launch.h"
#include "u4_common.h"

namespace qlora {
namespace {

template <int G>
struct CodeLoad;  // G / 32 words of codes per lane and group
template <>
struct CodeLoad<32> {
  uint32_t w[1];
  __device__ __forceinline__ void load(const uint8_t* p) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
};
template <>
struct CodeLoad<64> {
  uint32_t w[2];
  __device__ __forceinline__ void load(const uint8_t* p) {
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p);
    w[0] = v[0];
    w[1] = v[1];
  }
};
template <>
struct CodeLoad<128> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const uint8_t* p) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
  }
};

template <class DT, int G, int NT, int R, int W>
__global__ __launch_bounds__(64 * W) void linear_u4_kernel(
    const uint8_t* __restrict__ codes, const uint32_t* __restrict__ pairs,
    const uint16_t* __restrict__ x, int64_t ldx, uint16_t* __restrict__ y, int64_t ldy, int64_t M,
    int64_t N, int64_t K) {
  constexpr int C = G / 32;                  // MFMA steps per group
  constexpr int P = G == 32 ? 8 : G == 64 ? 4 : 2;  // groups loaded together
  __shared__ float red[W][R * NT][64][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R), m0 = (int64_t)blockIdx.y * (16 * NT);
  const int groups = (int)(K / G);
  const int g0 = (int)((int64_t)groups * wave / W), g1 = (int)((int64_t)groups * (wave + 1) / W);

  // rows and tokens past the end repeat the last one; their sums are dropped
  const uint8_t* cp[R];
  const uint32_t* pp[R];
  const uint16_t* xp[NT];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t n = min(n0 + 16 * r + lr, N - 1);
    cp[r] = codes + n * (K / 2) + lg * (G / 8);
    pp[r] = pairs + n * groups;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
    xp[t] = x + min(m0 + 16 * t + lr, M - 1) * ldx + lg * (G / 4);

  f32x4_t acc[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};
  const u32x4_t ones = {U4Mfma<DT>::kOne, U4Mfma<DT>::kOne, U4Mfma<DT>::kOne, U4Mfma<DT>::kOne};

  auto group = [&](const CodeLoad<G>(&cw)[R], const uint32_t(&pr)[R], const u32x4_t(&xv)[C][NT]) {
    f32x4_t X[NT];
    u32x4_t xo[C][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      X[t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        xo[c][t] = u4_order8(xv[c][t]);
        X[t] = DT::mfma16(xo[c][t], ones, X[t]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f32x4_t d[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) d[t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const u32x4_t b = u4_expand8<DT>(cw[r].w[c]);
#pragma unroll
        for (int t = 0; t < NT; ++t) d[t] = DT::mfma16(xo[c][t], b, d[t]);
      }
      const float s = u4_s(pr[r]), m = fmaf(-U4Mfma<DT>::kOff, s, u4_m(pr[r]));
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[r][t][i] = fmaf(s, d[t][i], fmaf(m, X[t][i], acc[r][t][i]));
    }
  };

  int g = g0;
  for (; g + P <= g1; g += P) {
    CodeLoad<G> cw[P][R];
    uint32_t pr[P][R];
    u32x4_t xv[P][C][NT];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int r = 0; r < R; ++r) cw[p][r].load(cp[r] + (int64_t)(g + p) * (G / 2));
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int r = 0; r < R; ++r) pr[p][r] = pp[r][g + p];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          xv[p][c][t] = *reinterpret_cast<const u32x4_t*>(xp[t] + (int64_t)(g + p) * G + 8 * c);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) group(cw[p], pr[p], xv[p]);
  }
  for (; g < g1; ++g) {
    CodeLoad<G> cw[R];
    uint32_t pr[R];
    u32x4_t xv[C][NT];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      cw[r].load(cp[r] + (int64_t)g * (G / 2));
      pr[r] = pp[r][g];
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        xv[c][t] = *reinterpret_cast<const u32x4_t*>(xp[t] + (int64_t)g * G + 8 * c);
    group(cw, pr, xv);
  }

#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<f32x4_t*>(red[wave][r * NT + t][lane]) = acc[r][t];
  __syncthreads();
  // sum i of lane l of tile (r, t) is token 16 t + 4 (l / 16) + i, row
  // 16 r + l % 16: neighbouring threads take neighbouring rows of one token
  for (int o = threadIdx.x; o < R * NT * 256; o += 64 * W) {
    const int n = o & 15, tok = (o >> 4) & 15, tile = o >> 8;
    const int r = tile / NT, t = tile - r * NT;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < W; ++q) v += red[q][tile][(tok >> 2) * 16 + n][tok & 3];
    const int64_t row = n0 + 16 * r + n, m = m0 + 16 * t + tok;
    if (row < N && m < M) y[m * ldy + row] = DT::cvt(v);
  }
}

template <class DT, int G, int NT, int R, int W>
void go(const uint8_t* codes, const uint32_t* pairs, const uint16_t* x, int64_t ldx, uint16_t* y,
        int64_t ldy, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  const dim3 grid((unsigned)((N + 16 * R - 1) / (16 * R)), (unsigned)((M + 16 * NT - 1) / (16 * NT)));
  linear_u4_kernel<DT, G, NT, R, W><<<grid, 64 * W, 0, s>>>(codes, pairs, x, ldx, y, ldy, M, N, K);
}

template <class DT, int G>
void pick(const uint8_t* codes, const uint32_t* pairs, const uint16_t* x, int64_t ldx, uint16_t* y,
          int64_t ldy, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  if (M <= 16)
    go<DT, G, 1, 1, 16>(codes, pairs, x, ldx, y, ldy, M, N, K, s);
  else if (M <= 32)
    go<DT, G, 2, 1, 8>(codes, pairs, x, ldx, y, ldy, M, N, K, s);
  else
    go<DT, G, 4, 1, 8>(codes, pairs, x, ldx, y, ldy, M, N, K, s);
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
