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
// once.  16 tokens, N and K 8192: 12.6 us against 15.7 with the form for many;
// 32 tokens, K 4096: 6.7 against 7.7 at N 4096, 15.3 against 10.7 at N 11008.
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

constexpr int W = 8;  // waves of a block

// Few tokens (16 T): a block owns 16 rows of each of the G weights and all of K,
// its waves split K, and their sums meet in LDS.  A weight's operands come
// straight from memory, 1024 bytes in a run; x is read by every block, from
// the caches.
//
// Bound by HBM on the weights: 1 token of 4096 x 4096 takes 3.7 us in a replayed
// graph (a copy of the bytes 3.3), 16 of 8192 x 8192 12.6 (13.1, but part stays
// in the last-level cache), 4 of a gated 11008 x 4096 17.4 (17.5), 4 of 22016 x
// 8192 27.4.  Blocks of 32 or 64 rows read x less often and fill the chip less
// evenly: 16 of 8192 x 8192 15.1 and 16.0 us, 16 of 11008 x 4096 9.4 and 11.9
// against 9.8.
template <class DT, int G, int T>
__global__ __launch_bounds__(64 * W) void few_i8_kernel(I8LinearArg p) {
  constexpr int U = 4;  // steps of 64 columns in flight
  __shared__ i32x4_t part[W][G * T][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t Kp = i8_padded(p.K), n0 = (int64_t)blockIdx.x * 16;
  const uint32_t panel = 16 * (uint32_t)Kp;
  const int steps = (int)(Kp / 64);
  const int s0 = steps * wave / W, s1 = steps * (wave + 1) / W;
  // tokens that are not there read as zeros
  __amdgpu_buffer_rsrc_t wbuf[G];
#pragma unroll
  for (int g = 0; g < G; ++g)
    wbuf[g] = make_rsrc(p.tiles[g] + (int64_t)blockIdx.x * panel, panel);
  const auto xbuf = make_rsrc(p.codes, (uint32_t)p.M * (uint32_t)Kp);
  const uint32_t wo = lane * 16, xo = lr * (uint32_t)Kp + lg * 16;

  i32x4_t acc[G][T];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[g][t] = i32x4_t{0, 0, 0, 0};
  auto run = [&](int s, auto count) {
    constexpr int C = decltype(count)::value;
    u32x4_t w[C][G], x[C][T];
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        w[c][g] = buffer_load16(wbuf[g], wo + (uint32_t)(s + c) * kI8Tile);
#pragma unroll
      for (int t = 0; t < T; ++t)
        x[c][t] = buffer_load16(xbuf, xo + 16 * t * (uint32_t)Kp + (uint32_t)(s + c) * 64);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[g][t] = mfma16(w[c][g], x[c][t], acc[g][t]);
  };
  int s = s0;
  for (; s + U <= s1; s += U) run(s, std::integral_constant<int, U>());
  for (; s < s1; ++s) run(s, std::integral_constant<int, 1>());

#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int t = 0; t < T; ++t) part[wave][g * T + t][lane] = acc[g][t];
  __syncthreads();
  // lane l of tile t has token 16 t + l % 16 and rows 4 (l / 16) and on
  const int l = threadIdx.x & 63, t = threadIdx.x >> 6;
  if (t >= T) return;
  i32x4_t sum[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    sum[g] = i32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < W; ++q) sum[g] += part[q][g * T + t][l];
  }
  const int64_t n = n0 + 4 * (l >> 4), m = 16 * t + (l & 15);
  if (m >= p.M || n >= p.N) return;
  const bool vec = ((uintptr_t)p.y & 7) == 0 && p.ldy % 4 == 0;
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

template <class DT, int G>
void pick(const I8LinearArg& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 15) / 16));
  if (p.M <= 16)
    few_i8_kernel<DT, G, 1><<<grid, 64 * W, 0, s>>>(p);
  else
    few_i8_kernel<DT, G, 2><<<grid, 64 * W, 0, s>>>(p);
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
