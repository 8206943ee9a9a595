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

// Small tiles: a block owns 16 R rows of each of the G weights, 16 T tokens and
// all of K, its waves split K, and their sums meet in LDS.  A weight's operands
// come straight from memory, 1024 bytes in a run.  Tokens come in rows of 128
// bytes and pass through the wave's own LDS: read in the operands' order, 16
// bytes of each of 16 rows side by side, they took four times as long (64
// tokens, N 677, K 7232 6.5 us where this takes 4.3; 16 of 4096 x 4096 4.6 and
// 3.7; 256 of 1024 x 8192 11.6 and 7.6).
//
// Bound by HBM on the weights where tokens are few: 1 token of 4096 x 4096 takes
// 3.4 us in a replayed graph (a copy of the bytes 3.3), 16 of 8192 x 8192 11.9
// (13.1, but part stays in the last-level cache), 4 of a gated 11008 x 4096 15.3
// (17.5), 4 of 22016 x 8192 26.9; else by what a CU takes in of its tile (32 of
// 4096 x 4096 4.3; 256 of 1024 x K, a block of 32 x 32 on each CU, 4.3 at K 2048
// and 7.5 at 8192: 123 GB/s a CU, 31 TB/s for all, from L2).  Neither two tiles of
// K in flight nor loads ahead of the exchange through LDS gained anything.
template <class DT, int G, int T, int R>
__global__ __launch_bounds__(64 * W) void few_i8_kernel(I8LinearArg p) {
  constexpr int KT = 128;                               // columns at a time
  constexpr int kX = 16 * T * KT, kSum = 1024 * G * T * R;  // bytes of a wave
  constexpr int kWave = kX > kSum ? kX : kSum;
  __shared__ __attribute__((aligned(16))) uint8_t lds[W * kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  uint32_t mt, nt;
  i8_tile_of(blockIdx.x, gridDim.x, (uint32_t)((p.M + 16 * T - 1) / (16 * T)),
             (uint32_t)((p.N + 16 * R - 1) / (16 * R)), 1024 / (16 * T), mt, nt);
  const int64_t Kp = i8_padded(p.K), n0 = (int64_t)nt * (16 * R), m0 = (int64_t)mt * (16 * T);
  const uint32_t panel = 16 * (uint32_t)Kp;
  const int tiles = (int)(Kp / KT);
  const int k0 = tiles * wave / W, k1 = tiles * (wave + 1) / W;
  // rows of panels and tokens that are not there read as zeros
  const uint32_t held = (uint32_t)min((p.N + 15) / 16 - (int64_t)nt * R, (int64_t)R) * panel;
  __amdgpu_buffer_rsrc_t wbuf[G];
#pragma unroll
  for (int g = 0; g < G; ++g) wbuf[g] = make_rsrc(p.tiles[g] + (int64_t)nt * R * panel, held);
  const auto xbuf = make_rsrc(p.codes + m0 * Kp,
                              (uint32_t)min(p.M - m0, (int64_t)16 * T) * (uint32_t)Kp);
  const uint32_t wo = lane * 16, xo = (lane >> 3) * (uint32_t)Kp + (lane & 7) * 16;
  uint8_t* const mine = lds + wave * kWave;
  // where piece c of a token is: 16 neighbouring tokens' in different banks
  auto place = [&](int tok, int c) {
    return reinterpret_cast<u32x4_t*>(mine + tok * KT + 16 * (c ^ ((tok >> 1) & 7)));
  };

  i32x4_t acc[G][R][T];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[g][r][t] = i32x4_t{0, 0, 0, 0};
  for (int k = k0; k < k1; ++k) {
    u32x4_t w[2][G][R], x[2 * T];
#pragma unroll
    for (int i = 0; i < 2 * T; ++i)
      x[i] = buffer_load16(xbuf, xo + 8 * i * (uint32_t)Kp + (uint32_t)k * KT);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r)
          w[h][g][r] = buffer_load16(wbuf[g], wo + r * panel + (uint32_t)(2 * k + h) * kI8Tile);
#pragma unroll
    for (int i = 0; i < 2 * T; ++i) *place(8 * i + (lane >> 3), lane & 7) = x[i];
    wave_exchange();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const u32x4_t v = *place(16 * t + lr, 4 * h + lg);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int r = 0; r < R; ++r) acc[g][r][t] = mfma16(w[h][g][r], v, acc[g][r][t]);
      }
    wave_exchange();
  }

  auto sums = [&](int of, int g, int r, int t, int l) {
    return reinterpret_cast<i32x4_t*>(lds + of * kWave + ((g * R + r) * T + t) * 1024 + l * 16);
  };
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t) *sums(wave, g, r, t, lane) = acc[g][r][t];
  __syncthreads();
  // a wave joins the sums of 16 tokens and 16 rows: lane l has token l % 16 and
  // rows 4 (l / 16) and on
  static_assert(T * R <= W, "a wave joins one tile");
  if (wave >= T * R) return;
  const int t = wave % T, r = wave / T;
  i32x4_t sum[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    sum[g] = i32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < W; ++q) sum[g] += *sums(q, g, r, t, lane);
  }
  const int64_t n = n0 + 16 * r + 4 * lg, m = m0 + 16 * t + lr;
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

// Which form and tile.  A call of B blocks and k tiles of 128 columns takes
//
//   start + max(ceil(B / 256) alone k, B / 256 (busy k + end))   us
//
// with what a tile of K takes in the CU that has most blocks, or in all of them
// when they have many, and what a block's outputs take; fitted together, for the
// choice (one alone is no rate), to 560 calls (1 to 4000 tokens, 16 to 22016
// rows, K to 11008), each timed in every form.  In
// 440 other calls the chosen one is within 0.4 % of the best in the mean and 20 %
// in the worst (1428 tokens of 11008 x 320).  Without 16 x 16 calls take 5 to 7 %
// more in the mean, without any other form 0.7 to 4 %.  256 tokens of 1024 x 8192
// take 7.3 us in 32 x 32, 12.2 in 16 x 16 and 13.4 in 32 x 128; 61 of 11008 x
// 4096 10.5 in 32 x 128 and 12.0 in 32 x 32; 501 of 4096 x 4096 12.5 in 64 x 128,
// 15.7 in 128 x 128 and 18.8 in 64 x 32; 1000 of 8192 x 8192 85, 64, 120 and 60
// in the large tiles, smallest first.  A tile of 256 x 256 gained 2 % at 8192^3
// and nothing at 4096 x 22016 x 8192; splitting K over blocks, with a join in a
// second launch, gained 3 % in the latter's last round and lost on other large
// calls; a join in the same launch is not tried, nor any at 65 to 1200 tokens, where
// calls are 1.1 to 5 times their floor (256 of 1024 x 4096 5.4 us, floor 1.1).
struct Form {
  int tm, tn;
  float start, alone, busy, end;
};
constexpr int kSmall = 4;  // of them are this file's
constexpr Form kPlain[] = {
    {16, 16, 2.63f, 0.0313f, 0.0393f, 0.146f}, {32, 16, 2.84f, 0.0404f, 0.0562f, 0.137f},
    {32, 32, 2.86f, 0.0787f, 0.0841f, 0.232f}, {64, 32, 3.31f, 0.1167f, 0.1170f, 0.703f},
    {32, 128, 3.12f, 0.201f, 0.147f, 1.05f},   {64, 128, 3.66f, 0.255f, 0.316f, 0.954f},
    {128, 128, 3.98f, 0.371f, 0.1715f, 3.44f}, {128, 256, 5.74f, 0.618f, 0.2965f, 5.03f}};
constexpr Form kGated[] = {
    {16, 16, 2.98f, 0.0267f, 0.0688f, 0.158f}, {32, 16, 3.47f, 0.0544f, 0.0947f, 0.156f},
    {32, 32, 3.44f, 0.1428f, 0.1413f, 0.490f}, {64, 32, 4.05f, 0.1462f, 0.2336f, 1.336f},
    {32, 128, 4.20f, 0.300f, 0.337f, 0.851f},  {64, 128, 4.47f, 0.494f, 0.4436f, 1.726f},
    {128, 128, 6.78f, 0.590f, 0.3834f, 3.71f}};
template <int C>
int best_of(const Form (&forms)[C], const I8LinearArg& p) {
  const float k = (float)(i8_padded(p.K) / 128);
  int best = C - 1;
  float least = 0.0f;
  for (int i = C - 1; i >= 0; --i) {
    const Form& f = forms[i];
    const int64_t blocks = ((p.M + f.tm - 1) / f.tm) * ((p.N + f.tn - 1) / f.tn);
    // (a launch holds below 2^32 threads, which the large tiles keep to)
    if (i < kSmall && blocks >= (int64_t{1} << 22)) continue;
    const float most = (float)((blocks + 255) / 256) * f.alone * k;
    const float all = (float)blocks / 256.0f * (f.busy * k + f.end);
    const float time = f.start + (most > all ? most : all);
    if (i == C - 1 || time < least) best = i, least = time;
  }
  return best;
}

template <class DT, int G, int T, int R>
void go(const I8LinearArg& p, hipStream_t s) {
  const int64_t blocks = ((p.M + 16 * T - 1) / (16 * T)) * ((p.N + 16 * R - 1) / (16 * R));
  few_i8_kernel<DT, G, T, R><<<dim3((unsigned)blocks), 64 * W, 0, s>>>(p);
}
template <class DT, int G>
void pick(const I8LinearArg& p, int form, hipStream_t s) {
  switch (form) {
    case 0: return go<DT, G, 1, 1>(p, s);
    case 1: return go<DT, G, 2, 1>(p, s);
    case 2: return go<DT, G, 2, 2>(p, s);
    default: return go<DT, G, 4, 2>(p, s);
  }
}

}  // namespace

hipError_t launch_linear_i8(const I8LinearArg& p, bool f16, hipStream_t s) {
  const int form = p.tiles[1] ? best_of(kGated, p) : best_of(kPlain, p);
  if (form >= kSmall) return launch_gemm_i8(p, form - kSmall, f16, s);
  if (p.tiles[1]) {
    if (f16)
      pick<F16T, 2>(p, form, s);
    else
      pick<Bf16T, 2>(p, form, s);
  } else {
    if (f16)
      pick<F16T, 1>(p, form, s);
    else
      pick<Bf16T, 1>(p, form, s);
  }
  return hipGetLastError();
}

}  // namespace qlora
