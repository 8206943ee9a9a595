// Tokens in the 8-bit row format (i8_common.h): the quantiser, the norm that
// writes them, and what they stand for.
//
// The norm: h = x + residual, rounded to 16 bits and kept as the new residual
// stream; t = h w; y = t / sqrt(mean h^2 + eps) is what is coded.  The root is
// common to a row, so codes are rint(127 t / max |t|) whatever it is, and only
// the scale, max |t| / (127 root), has it: one pass collects max |t| and the
// sum of h^2 together, and no code depends on how the root was rounded.
//
// Bound by HBM.  A row stays in registers between the two passes, so each
// input is read once.  A row of up to 2048 values belongs to one wave (no
// barrier; where rows are few, of up to 512 values), longer ones to four, eight
// or sixteen.  Sums, maxima and quotients are fp64: with a product of two 16-bit
// floats exact in it nothing overflows, and its share is small beside the
// memory's.
//
// Measured: 4096 tokens of 8192 20 us, with the norm and a residual 46 (5.1 TB/s;
// a large copy 5.16); 2047 of 11008 16.1 and 37, of 22016 27 and 72; one of 4096
// 2.5 and 3.6 in a replayed graph.  4096 of 65536 155 and 460 (4.1 TB/s), of 130944
// 336 and 940 (4.0); of 65544, where half of the lanes' pieces are empty, 222 and
// 679 (2.8).

#include <type_traits>

#include "i8_common.h"
#include "launch.h"

namespace qlora {
namespace {

template <int W>
constexpr int rows_threads() { return W == 1 ? 256 : 64 * W; }

__device__ __forceinline__ double lane_xor(double v, int m) { return __shfl_xor(v, m); }

// DT: type of x.  W: waves of a row.  CH: pieces of 8 values a lane.
template <class DT, int W, int CH, bool NORM>
__global__ __launch_bounds__(rows_threads<W>()) void rows_i8_kernel(I8RowsArg p) {
  constexpr int T = 64 * W;                       // lanes of a row
  constexpr int ROWS = rows_threads<W>() / T;     // rows of a block
  constexpr uint32_t kInf = std::is_same<DT, F16T>::value ? 0x7C00u : 0x7F80u;
  __shared__ double part[W][3];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = W == 1 ? lane : threadIdx.x;
  const int K = (int)p.K, Kp = (int)i8_padded(K);
  // at most four pieces' loads are ahead of their use, or long rows spill (with
  // the norm, those past 65536 values do all the same: 14 registers, 60 bytes a
  // lane)
  auto fence = [](int i) {
    if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
  };
  const int64_t row = (int64_t)blockIdx.x * ROWS + (W == 1 ? wave : 0);
  if (row >= p.M) return;
  // The norm's weight: up to four pieces a lane are asked for with x and held
  // (one token of 4096 3.9 -> 3.6 us, of 8192 5.4 -> 4.9; 2047 of 4096 17.3 ->
  // 15.8), more are read anew for each pass.  Either way it is opaque to the last
  // pass, or its values and products would be kept as fp64 and spilled.
  constexpr bool kHeld = NORM && CH <= 4;
  const uint16_t* pw = p.w;
  asm volatile("" : "+s"(pw));
  u32x4_t h[CH];
  const uint16_t* x = p.x + row * p.ldx;
#pragma unroll
  for (int i = 0; i < CH; ++i) h[i] = load_piece(x, 8 * (i * T + at), K);
  u32x4_t held[kHeld ? CH : 1];
  if constexpr (kHeld) {
#pragma unroll
    for (int i = 0; i < CH; ++i) held[i] = load_piece(pw, 8 * (i * T + at), K);
  }
  auto weight = [&](int i) {
    if constexpr (kHeld)
      return held[i];
    else
      return load_piece(pw, 8 * (i * T + at), K);
  };
  // One wave sums its pieces of 64 lanes apart and joins them as four waves do, so
  // a row's bits do not depend on which of them has it.
  constexpr int NS = W == 1 ? CH : 1;
  double a = 0.0, sum = 0.0, s[NS] = {};
  uint32_t top = 0;
  bool ok = true;
  if constexpr (NORM) {
    if (p.res) {
      const uint16_t* r = p.res + row * p.ldr;
      uint16_t* o = p.h + row * p.ldh;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int k = 8 * (i * T + at);
        const u32x4_t v = load_piece(r, k, K);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[i][j] = DT::pack2(
              DT::tof((uint16_t)half_of(h[i], 2 * j)) + DT::tof((uint16_t)half_of(v, 2 * j)),
              DT::tof((uint16_t)half_of(h[i], 2 * j + 1)) +
                  DT::tof((uint16_t)half_of(v, 2 * j + 1)));
        store_piece(o, k, K, h[i]);
        fence(i);
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const u32x4_t w = weight(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double v = DT::tof((uint16_t)half_of(h[i], j));
        const double t = fabs(v * DT::tof((uint16_t)half_of(w, j)));
        s[i % NS] = __builtin_fma(v, v, s[i % NS]);
        a = fmax(a, t);
        ok = ok && t <= 1e300;
      }
      fence(i);
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
      a = fmax(a, lane_xor(a, m));
#pragma unroll
      for (int i = 0; i < NS; ++i) s[i] += lane_xor(s[i], m);
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) sum += s[i];
    ok = __all(ok);
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, half_of(h[i], j) & 0x7FFFu);
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
  }
  if constexpr (W > 1) {
    if (lane == 0) {
      part[wave][0] = NORM ? a : (double)top;
      part[wave][1] = sum;
      part[wave][2] = ok ? 0.0 : 1.0;
    }
    __syncthreads();
    a = 0.0, sum = 0.0;
#pragma unroll
    for (int q = 0; q < W; ++q) {
      a = fmax(a, part[q][0]);
      sum += part[q][1];
      ok = ok && part[q][2] == 0.0;
    }
    top = NORM ? 0u : (uint32_t)a;
  }
  double times = 1.0;
  if constexpr (NORM) {
    times = 1.0 / sqrt(sum / (double)K + p.eps);
  } else {
    ok = top < kInf;
    a = DT::tof((uint16_t)top);
  }
  const I8Row code = i8_row(a, times, ok);
  if (at == 0) p.scales[row] = code.s;
  int8_t* o = p.codes + row * Kp;
  asm volatile("" : "+s"(pw));
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k = 8 * (i * T + at);
    u32x4_t w;
    if constexpr (NORM) {
      asm volatile("" : "+v"(h[i]));
      if constexpr (kHeld) asm volatile("" : "+v"(held[i]));
      w = weight(i);
    }
    u32x2_t c = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      double v = DT::tof((uint16_t)half_of(h[i], j));
      if constexpr (NORM) v *= DT::tof((uint16_t)half_of(w, j));
      c[j / 4] |= ((uint32_t)i8_code(code, v) & 0xFFu) << (8 * (j & 3));
    }
    if (k < Kp) *reinterpret_cast<u32x2_t*>(o + k) = c;
    fence(i);
  }
}

template <class DT, bool NORM>
void go_rows(const I8RowsArg& p, hipStream_t s) {
  // a launch holds below 2^32 threads: 2^21 rows at a time
  auto run = [&](auto kernel, int threads, int rows) {
    constexpr int64_t kMost = int64_t{1} << 21;
    for (int64_t at = 0; at < p.M; at += kMost) {
      I8RowsArg q = p;
      q.M = p.M - at < kMost ? p.M - at : kMost;
      q.x += at * p.ldx;
      if (p.res) {
        q.res += at * p.ldr;
        q.h += at * p.ldh;
      }
      q.codes += at * i8_padded(p.K);
      q.scales += at;
      kernel<<<dim3((unsigned)((q.M + rows - 1) / rows)), threads, 0, s>>>(q);
    }
  };
  const int64_t pieces = i8_padded(p.K) / 8;
#define QLORA_I8_ROWS(W, CH) \
  if (pieces <= 64 * (W) * (CH)) \
    return run(rows_i8_kernel<DT, W, CH, NORM>, rows_threads<W>(), (W) == 1 ? 4 : 1)
  // as many pieces a lane as a row has use for: with powers of two alone 2047
  // rows of 11008 took 17.5 us where they take 16.1.  More waves and fewer pieces
  // where the norm would hold too much: 2047 of 11008 36 to 38 us, 41 with four
  // waves of six pieces (without the norm 16.9 and 16.0); of 22016 72 us, and 27
  // without it, 97 and 31 with sixteen waves of three, which leave a CU one row.
  QLORA_I8_ROWS(1, 1);
  // few rows of up to 2048 values are done sooner by four waves (one of 2048 2.6
  // -> 2.2 us, with the norm 4.3 -> 3.1; 512 3.2 -> 3.0 and 5.3 -> 4.4; 1024 3.5
  // -> 3.9 and 5.9 -> 6.2)
  if (p.M <= 512) {
    QLORA_I8_ROWS(4, 1);
  }
  QLORA_I8_ROWS(1, 2);
  QLORA_I8_ROWS(1, 3);
  QLORA_I8_ROWS(1, 4);
  QLORA_I8_ROWS(4, 2);
  QLORA_I8_ROWS(4, 3);
  QLORA_I8_ROWS(4, 4);
  if constexpr (NORM) {
    QLORA_I8_ROWS(8, 3);
    QLORA_I8_ROWS(8, 4);
  } else {
    QLORA_I8_ROWS(4, 5);
    QLORA_I8_ROWS(4, 6);
    QLORA_I8_ROWS(4, 8);
  }
  QLORA_I8_ROWS(8, 5);
  QLORA_I8_ROWS(8, 6);
  QLORA_I8_ROWS(8, 8);
  QLORA_I8_ROWS(16, 6);
  QLORA_I8_ROWS(16, 8);
  QLORA_I8_ROWS(16, 16);
#undef QLORA_I8_ROWS
}

// Eight values a lane; lanes run over the rows' pieces.
template <class DT>
__global__ __launch_bounds__(256) void values_i8_kernel(const int8_t* __restrict__ codes,
                                                        const float* __restrict__ scales,
                                                        int64_t M, int64_t K,
                                                        uint16_t* __restrict__ out) {
  const int64_t Kp = i8_padded(K), per = (K + 7) / 8, n = M * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int k = 8 * (int)(i - row * per);
    const u32x2_t c = *reinterpret_cast<const u32x2_t*>(codes + row * Kp + k);
    const float s = scales[row];
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = c[j / 2] >> (16 * (j & 1));
      v[j] = DT::pack2(i8_value((int8_t)w, s), i8_value((int8_t)(w >> 8), s));
    }
    store_piece(out + row * K, k, (int)K, v);
  }
}

}  // namespace

hipError_t launch_rows_i8(const I8RowsArg& p, bool f16, hipStream_t s) {
  if (p.w) {
    if (f16)
      go_rows<F16T, true>(p, s);
    else
      go_rows<Bf16T, true>(p, s);
  } else {
    if (f16)
      go_rows<F16T, false>(p, s);
    else
      go_rows<Bf16T, false>(p, s);
  }
  return hipGetLastError();
}

hipError_t launch_values_i8(const int8_t* codes, const float* scales, int64_t M, int64_t K,
                            uint16_t* out, bool f16, hipStream_t s) {
  const int64_t n = M * ((K + 7) / 8), blocks = (n + 255) / 256, most = int64_t{1} << 22;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  if (f16)
    values_i8_kernel<F16T><<<grid, 256, 0, s>>>(codes, scales, M, K, out);
  else
    values_i8_kernel<Bf16T><<<grid, 256, 0, s>>>(codes, scales, M, K, out);
  return hipGetLastError();
}

}  // namespace qlora
