// Products of 8-bit tokens with 8-bit weights (i8_common.h):
//
//   y[m][n] = sx[m] sw[n] sum_k x[m][k] W[n][k]
//
// and, with a second weight U, act(g) u of the two products g and u.  The sums
// are int32 in the matrix cores and exact: K is at most 2^17 - 128, so no sum
// of products of two codes passes 2^31.  So a split over k in any order gives
// the same bits, and a result is rounded where it is scaled (three roundings to
// fp32) and once to 16 bits.

#include "i8_common.h"
#include "launch.h"

namespace qlora {
namespace {

// Few tokens: up to 16, or 32 where a block for each 16 rows fills the chip
// once.  16 tokens, N and K 8192: 12.8 us against 15.7 with the form for many;
// 32 tokens, K 4096: 6.9 against 7.7 at N 4096, 15.3 against 10.7 at N 11008.
bool few(int64_t M, int64_t N) { return M <= 16 || (M <= 32 && N <= 4096); }

__device__ __forceinline__ i32x4_t mfma16(u32x4_t a, u32x4_t b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a),
                                               __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// Four neighbouring outputs of a token, n .. n + 3 of which N has some.
template <class DT>
__device__ __forceinline__ void store4(uint16_t* row, int64_t n, int64_t N, bool whole,
                                       const float (&v)[4]) {
  const u32x2_t o = {DT::pack2(v[0], v[1]), DT::pack2(v[2], v[3])};
  if (whole) {
    *reinterpret_cast<u32x2_t*>(row + n) = o;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < N) row[n + j] = (uint16_t)(o[j / 2] >> (16 * (j & 1)));
  }
}

// Few tokens: a block owns 16 R rows of each of the G weights and all of K,
// its W waves split K, and their sums meet in LDS.  A weight's operands come
// straight from memory, 1024 bytes in a run; x is read by every block, from
// the caches.
template <class DT, int G, int R, int T, int W>
__global__ __launch_bounds__(64 * W) void few_i8_kernel(I8LinearArg p) {
  constexpr int U = 4;  // steps of 64 columns in flight
  __shared__ i32x4_t part[W][G * R * T][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t Kp = i8_padded(p.K), n_tiles = (p.N + 15) / 16;
  const int64_t tile0 = (int64_t)blockIdx.x * R, m0 = (int64_t)blockIdx.y * (16 * T);
  const uint32_t panel = 16 * (uint32_t)Kp;
  const int steps = (int)(Kp / 64);
  const int s0 = steps * wave / W, s1 = steps * (wave + 1) / W;
  // rows and tokens that are not there read as zeros
  const uint32_t rows = (uint32_t)min(n_tiles - tile0, (int64_t)R);
  const uint32_t toks = (uint32_t)min(p.M - m0, (int64_t)(16 * T));
  __amdgpu_buffer_rsrc_t wbuf[G];
#pragma unroll
  for (int g = 0; g < G; ++g) wbuf[g] = make_rsrc(p.tiles[g] + tile0 * panel, rows * panel);
  const auto xbuf = make_rsrc(p.codes + m0 * Kp, toks * (uint32_t)Kp);
  const uint32_t wo = lane * 16, xo = lr * (uint32_t)Kp + lg * 16;

  i32x4_t acc[G][R][T];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[g][r][t] = i32x4_t{0, 0, 0, 0};
  auto run = [&](int s, auto count) {
    constexpr int C = decltype(count)::value;
    u32x4_t w[C][G][R], x[C][T];
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r)
          w[c][g][r] = buffer_load16(wbuf[g], wo + r * panel + (uint32_t)(s + c) * kI8Tile);
#pragma unroll
      for (int t = 0; t < T; ++t)
        x[c][t] = buffer_load16(xbuf, xo + 16 * t * (uint32_t)Kp + (uint32_t)(s + c) * 64);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < T; ++t) acc[g][r][t] = mfma16(w[c][g][r], x[c][t], acc[g][r][t]);
  };
  int s = s0;
  for (; s + U <= s1; s += U) run(s, std::integral_constant<int, U>());
  for (; s < s1; ++s) run(s, std::integral_constant<int, 1>());

#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t) part[wave][(g * R + r) * T + t][lane] = acc[g][r][t];
  __syncthreads();
  // lane l of tile (r, t) has token 16 t + l % 16 and rows 16 r + 4 (l / 16) ..
  const bool vec = ((uintptr_t)p.y & 7) == 0 && p.ldy % 4 == 0;
  for (int o = threadIdx.x; o < R * T * 64; o += 64 * W) {
    const int l = o & 63, r = (o >> 6) / T, t = (o >> 6) - r * T;
    i32x4_t sum[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      sum[g] = i32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < W; ++q) sum[g] += part[q][(g * R + r) * T + t][l];
    }
    const int64_t n = 16 * (tile0 + r) + 4 * (l >> 4), m = m0 + 16 * t + (l & 15);
    if (m >= p.M || n >= p.N) continue;
    const float sx = p.xscale[m];
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = n + j < p.N ? n + j : p.N - 1;
      v[j] = i8_scaled(sum[0][j], p.wscale[0][row], sx);
      if constexpr (G == 2) v[j] = i8_gated(v[j], i8_scaled(sum[1][j], p.wscale[1][row], sx), p.act);
    }
    store4<DT>(p.y + m * p.ldy, n, p.N, vec && n + 4 <= p.N, v);
  }
}

template <class DT, int G, int R, int T, int W>
void go_few(const I8LinearArg& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 16 * R - 1) / (16 * R)), (unsigned)((p.M + 16 * T - 1) / (16 * T)));
  few_i8_kernel<DT, G, R, T, W><<<grid, 64 * W, 0, s>>>(p);
}

template <class DT, int G>
void pick(const I8LinearArg& p, hipStream_t s) {
  if (p.M <= 16) return go_few<DT, G, 1, 1, 8>(p, s);
  return go_few<DT, G, 1, 2, 8>(p, s);
}

}  // namespace

hipError_t launch_linear_i8(const I8LinearArg& p, bool f16, hipStream_t s) {
  if (!few(p.M, p.N)) return launch_gemm_i8(p, f16, s);
  if (p.tiles[1]) {
    if (f16)
      pick<F16T, 2>(p, s);
    else
      pick<Bf16T, 2>(p, s);
  } else {
    if (f16)
      pick<F16T, 1>(p, s);
    else
      pick<Bf16T, 1>(p, s);
  }
  return hipGetLastError();
}

}  // namespace qlora
