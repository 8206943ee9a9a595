// A weight in the 8-bit row format and its tiles (i8_common.h): the quantiser
// of fp32 rows and what they stand for.
//
// Bound by HBM: 4 bytes of a value in, one out.  A row of up to 32768 values
// stays in registers between the search for its largest magnitude and its
// codes, 64 values a lane: one, two, four or eight waves have a row, and a block
// eight waves (sixteen for the longest rows; with sixteen for all, one block a
// CU, 11008 x 4096 took 55.6 us).  Longer rows are read twice, a wave a row.
// Codes go through LDS into the tiles' order, 8 or 16 KiB at a time, so stores
// are runs of a block's rows.
//
// Measured: 11008 x 4096 42 us, 22016 x 8192 181 (902 MB, 5.0 TB/s; a large copy
// 5.16), 4096 x 11008 54, 8192 x 28672 355; reading the first two back 22 and 117.

#include "i8_common.h"
#include "launch.h"

namespace qlora {
namespace {

constexpr int kCols = 1024;         // columns of a panel at a time
constexpr int kLdsRow = kCols + 16;  // bytes: the rows' pieces in different banks

__device__ __forceinline__ f32x4_t load4(const float* p, int64_t k, int64_t K) {
  f32x4_t v = {0, 0, 0, 0};
  if (k + 4 <= K) {
    __builtin_memcpy(&v, p + k, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k + j < K) v[j] = p[k + j];
  }
  return v;
}

__global__ __launch_bounds__(1024) void quantize_i8_kernel(const float* __restrict__ w, int64_t N,
                                                           int64_t K, int8_t* __restrict__ tiles,
                                                           float* __restrict__ scales) {
  __shared__ __attribute__((aligned(16))) int8_t lds[16 * kLdsRow];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 16 + wave, Kp = i8_padded(K);
  const bool row = n < N;
  const float* src = w + (row ? n : 0) * K;
  uint32_t top = 0;
  if (row)
    for (int64_t k = 4 * lane; k < K; k += 256) {
      const f32x4_t v = load4(src, k, K);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
  const I8Row code = i8_row(__uint_as_float(top), 1.0, top < 0x7F800000u);
  if (row && lane == 0) scales[n] = code.s;
  int8_t* dst = tiles + (int64_t)blockIdx.x * 16 * Kp;
  for (int64_t k0 = 0; k0 < Kp; k0 += kCols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = k0 + 256 * i + 4 * lane;
      uint32_t c = 0;
      if (row && k < K) {
        const f32x4_t v = load4(src, k, K);
#pragma unroll
        for (int j = 0; j < 4; ++j) c |= ((uint32_t)i8_code(code, v[j]) & 0xFFu) << (8 * j);
      }
      *reinterpret_cast<uint32_t*>(&lds[wave * kLdsRow + 256 * i + 4 * lane]) = c;
    }
    __syncthreads();
    // thread t has piece (t % 64) / 16 of row t % 16 of tile t / 64
    const int t = threadIdx.x, col = 64 * (t >> 6) + 16 * ((t >> 4) & 3);
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(&lds[(t & 15) * kLdsRow + col]);
    if (k0 + col < Kp) *reinterpret_cast<u32x4_t*>(dst + 16 * k0 + 16 * t) = v;
    __syncthreads();
  }
}

// W: waves of the block, WR: of a row.
template <int W, int WR>
__global__ __launch_bounds__(64 * W) void quantize_rows_i8_kernel(const float* __restrict__ w,
                                                                int N, int K,
                                                                int8_t* __restrict__ tiles,
                                                                float* __restrict__ scales) {
  constexpr int R = W / WR;             // rows of the block
  constexpr int COLS = 1024 * WR;       // columns at a time
  constexpr int LD = COLS + 16;         // bytes of a row in LDS
  __shared__ __attribute__((aligned(16))) int8_t lds[2][R * LD];
  __shared__ uint32_t tops[W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = wave / WR, part = wave % WR;
  const int n = blockIdx.x * R + r, Kp = (int)i8_padded(K);
  const bool row = n < N;
  const float* src = w + (int64_t)(row ? n : N - 1) * K;
  f32x4_t v[16];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = load4(src, (i * WR + part) * 256 + 4 * lane, K);
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
  if constexpr (WR > 1) {
    if (lane == 0) tops[wave] = top;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < WR; ++q) top = max(top, tops[r * WR + q]);
  }
  const I8Row code = i8_row(__uint_as_float(top), 1.0, top < 0x7F800000u);
  if (row && lane == 0 && part == 0) scales[n] = code.s;
  int8_t* dst = tiles + (int64_t)(blockIdx.x / (16 / R)) * 16 * Kp + (blockIdx.x % (16 / R)) * (16 * R);
  // thread t stores 16 columns of row t % R
  const int t = threadIdx.x, tr = t % R, piece = t / R;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (g * COLS >= Kp) break;
    int8_t* at = &lds[g & 1][r * LD + part * 256 + 4 * lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c |= ((uint32_t)i8_code(code, v[4 * g + i][j]) & 0xFFu) << (8 * j);
      *reinterpret_cast<uint32_t*>(at + i * (256 * WR)) = row ? c : 0u;
    }
    __syncthreads();
    const int col = g * COLS + 16 * piece;
    if (col < Kp)
      *reinterpret_cast<u32x4_t*>(dst + (col >> 6) * kI8Tile + ((col >> 4) & 3) * 256 + 16 * tr) =
          *reinterpret_cast<const u32x4_t*>(&lds[g & 1][tr * LD + 16 * piece]);
  }
}

// A wave has a row of the panel, a lane 8 columns of it: the sixteen waves read
// the lines of a tile together.
template <class DT>
__global__ __launch_bounds__(1024) void dequantize_i8_kernel(const int8_t* __restrict__ tiles,
                                                             const float* __restrict__ scales,
                                                             int64_t N, int64_t K,
                                                             uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 16 + wave;
  if (n >= N) return;
  const float s = scales[n];
  const int8_t* src = tiles + (int64_t)blockIdx.x * 16 * i8_padded(K) + 16 * wave;
  uint16_t* dst = out + n * K;
  for (int k = 8 * lane; k < (int)K; k += 512) {
    const u32x2_t c = *reinterpret_cast<const u32x2_t*>(src + (int64_t)(k >> 6) * kI8Tile +
                                                        ((k >> 4) & 3) * 256 + (k & 8));
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = c[j / 2] >> (16 * (j & 1));
      v[j] = DT::pack2(i8_value((int8_t)b, s), i8_value((int8_t)(b >> 8), s));
    }
    store_piece(dst, k, (int)K, v);
  }
}

}  // namespace

hipError_t launch_quantize_i8(const float* w, int64_t N, int64_t K, int8_t* tiles, float* scales,
                              hipStream_t s) {
  const unsigned panels = (unsigned)((N + 15) / 16);
  if (K <= 4096)
    quantize_rows_i8_kernel<8, 1><<<dim3(2 * panels), 512, 0, s>>>(w, (int)N, (int)K, tiles, scales);
  else if (K <= 8192)
    quantize_rows_i8_kernel<8, 2><<<dim3(4 * panels), 512, 0, s>>>(w, (int)N, (int)K, tiles, scales);
  else if (K <= 16384)
    quantize_rows_i8_kernel<8, 4><<<dim3(8 * panels), 512, 0, s>>>(w, (int)N, (int)K, tiles, scales);
  else if (K <= 32768)
    quantize_rows_i8_kernel<16, 8><<<dim3(8 * panels), 1024, 0, s>>>(w, (int)N, (int)K, tiles, scales);
  else
    quantize_i8_kernel<<<dim3(panels), 1024, 0, s>>>(w, N, K, tiles, scales);
  return hipGetLastError();
}

hipError_t launch_dequantize_i8(const int8_t* tiles, const float* scales, int64_t N, int64_t K,
                                uint16_t* out, bool f16, hipStream_t s) {
  const dim3 grid((unsigned)((N + 15) / 16));
  if (f16)
    dequantize_i8_kernel<F16T><<<grid, 1024, 0, s>>>(tiles, scales, N, K, out);
  else
    dequantize_i8_kernel<Bf16T><<<grid, 1024, 0, s>>>(tiles, scales, N, K, out);
  return hipGetLastError();
}

}  // namespace qlora
