// Quantiser and dequantiser of the 4-bit group format (u4_common.h).
//
// Both are bound by HBM: the quantiser reads 4 bytes per value and writes
// 0.5 + 4 / G.  A lane takes four neighbouring values (one 16-byte load, so
// a wave reads 1 KiB without gaps), a group is G / 4 neighbouring lanes, and
// its minimum and maximum are joined with DPP steps.  A wave has kBatch
// loads in flight before it works on the first.
//
// Measured: quantising 4096 x 4096 in groups of 64 takes 17.7 us (76 MB, 4.3
// TB/s) and 22016 x 8192 in groups of 128 168 to 193 us (817 MB, 171 us at
// the rate of a large copy); dequantising the same takes 8 and 67 us (43 and
// 457 MB, so much of them stays in the last-level cache).

#include "launch.h"
#include "u4_common.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;

template <int G>
__global__ __launch_bounds__(kThreads) void quantize_u4_kernel(const float* __restrict__ w,
                                                               int64_t n,
                                                               uint8_t* __restrict__ codes,
                                                               uint32_t* __restrict__ pairs) {
  constexpr int LANES = G / 4;
  const int64_t base = (int64_t)blockIdx.x * (kThreads * 4 * kBatch) + threadIdx.x * 4;
  f32x4_t v[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int64_t e = base + b * (kThreads * 4);
    v[b] = e < n ? *reinterpret_cast<const f32x4_t*>(w + e) : f32x4_t{0, 0, 0, 0};
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    // n is a multiple of G, so a group is inside or outside as a whole
    const int64_t e = base + b * (kThreads * 4);
    float lo = fminf(fminf(v[b][0], v[b][1]), fminf(v[b][2], v[b][3]));
    float hi = fmaxf(fmaxf(v[b][0], v[b][1]), fmaxf(v[b][2], v[b][3]));
    bool fin = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) fin = fin && fabsf(v[b][i]) <= 3.4028235e38f;
    lanes_minmax<LANES>(lo, hi);
    const U4Coder u = u4_coder<float>(lo, hi, lanes_all<LANES>(fin));
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c |= u4_code(u, v[b][i], v[b][i] - u.m) << (4 * i);
    if (e < n) {
      *reinterpret_cast<uint16_t*>(codes + e / 2) = (uint16_t)c;
      if (e % G == 0) pairs[e / G] = u.pair;
    }
  }
}

// 8 values per lane: a 4-byte load, the pair, and a 16-byte store.
template <class DT>
__global__ __launch_bounds__(kThreads) void dequantize_u4_kernel(
    const uint32_t* __restrict__ codes, const uint32_t* __restrict__ pairs, int64_t words,
    int words_log2, u32x4_t* __restrict__ out) {
  const int64_t base = (int64_t)blockIdx.x * (kThreads * kBatch) + threadIdx.x;
  uint32_t w[kBatch], p[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int64_t i = base + b * kThreads;
    w[b] = i < words ? codes[i] : 0;
    p[b] = i < words ? pairs[i >> words_log2] : 0;
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int64_t i = base + b * kThreads;
    float v[8];
    u4_values8(w[b], p[b], v);
    if (i < words)
      out[i] = u32x4_t{DT::pack2(v[0], v[1]), DT::pack2(v[2], v[3]), DT::pack2(v[4], v[5]),
                       DT::pack2(v[6], v[7])};
  }
}

}  // namespace

hipError_t launch_quantize_u4(const float* w, int64_t n, int group, uint8_t* codes,
                              uint32_t* pairs, hipStream_t s) {
  const int64_t per = kThreads * 4 * kBatch;
  const dim3 grid((unsigned)((n + per - 1) / per));
  if (group == 32)
    quantize_u4_kernel<32><<<grid, kThreads, 0, s>>>(w, n, codes, pairs);
  else if (group == 64)
    quantize_u4_kernel<64><<<grid, kThreads, 0, s>>>(w, n, codes, pairs);
  else
    quantize_u4_kernel<128><<<grid, kThreads, 0, s>>>(w, n, codes, pairs);
  return hipGetLastError();
}

hipError_t launch_dequantize_u4(const uint8_t* codes, const uint32_t* pairs, int64_t n, int group,
                                uint16_t* out, bool f16, hipStream_t s) {
  const int64_t words = n / 8, per = kThreads * kBatch;
  const dim3 grid((unsigned)((words + per - 1) / per));
  const int lg = group == 32 ? 2 : group == 64 ? 3 : 4;
  const auto* c = reinterpret_cast<const uint32_t*>(codes);
  auto* o = reinterpret_cast<u32x4_t*>(out);
  if (f16)
    dequantize_u4_kernel<F16T><<<grid, kThreads, 0, s>>>(c, pairs, words, lg, o);
  else
    dequantize_u4_kernel<Bf16T><<<grid, kThreads, 0, s>>>(c, pairs, words, lg, o);
  return hipGetLastError();
}

}  // namespace qlora
