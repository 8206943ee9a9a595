// Rows of the 4-bit paged cache: appending rotated keys and values, and
// reading rows back.
//
// The cache holds, for keys and for values, codes [pages][kv heads]
// [page size][head_dim / 2] and pairs [pages][kv heads][page size]: one
// group of the 4-bit format (u4_common.h) per token and head.
//
// Both kernels move little data per token and are bound by latency at a
// decode step and by HBM at a prefill.  A head's vector is D / 8
// neighbouring lanes with 8 values each, every vector of a call is
// independent, and a token's sequence comes from the grid (y), so no lane
// searches for it.

#include "kv4_common.h"
#include "launch.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

// One 16-bit head vector: where this lane's two runs of four values start.
// The rotated pairs lie in one lane: (i, i + rot / 2) with runs at 4 l and
// rot / 2 + 4 l, or neighbours (interleaved, and past the rotated part)
// with one run of 8.
struct Runs {
  int a, b;
};
__device__ __forceinline__ Runs lane_runs(int l, int rot, int interleaved) {
  const int rl = rot >> 3;  // lanes that rotate
  if (l < rl && !interleaved) return {4 * l, (rot >> 1) + 4 * l};
  return {8 * l, 8 * l + 4};
}

template <class DT>
__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[8], int at) {
  const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[at + i] = DT::tof((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
}

// Positions and places are worked out per vector; rotation and encoding run
// in fp64 (half the fp32 rate on this chip, and a few operations a value):
// a product of a 16-bit value and an fp32 cosine is exact there and the
// rotated value rounded once, so codes at a border come out as defined.
template <class DT, int D>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(Kv4CacheArg c, Kv4BatchArg bt,
                                                              Kv4AppendArg a) {
  constexpr int LPV = D / 8, VPB = kThreads / LPV;
  const int l = threadIdx.x % LPV;
  const int64_t v = (int64_t)blockIdx.x * VPB + threadIdx.x / LPV;
  const int heads = a.q_heads + 2 * c.kv_heads;
  const int b = blockIdx.y;
  const Kv4Seq sq = kv4_seq(bt, b);
  const int64_t i = v / heads;
  int h = (int)(v - i * heads);
  if (i >= sq.n) return;
  const int64_t row = sq.row0 + i, pos = sq.pos0 + i;
  const bool is_q = h < a.q_heads;
  if (!is_q) h -= a.q_heads;
  const bool is_v = !is_q && h >= c.kv_heads;
  if (is_v) h -= c.kv_heads;

  const int rot = is_v ? 0 : a.rot;
  const Runs r = lane_runs(l, rot, a.interleaved);
  const uint16_t* src = is_q ? a.q + row * a.q_ts + h * a.q_hs
                             : is_v ? a.v + row * a.v_ts + h * a.v_hs
                                    : a.k + row * a.k_ts + h * a.k_hs;
  float x[8];
  load4<DT>(src + r.a, x, 0);
  load4<DT>(src + r.b, x, 4);
  double d[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] = x[j];
  // no angle for this position: the query becomes NaN, nothing is stored
  const bool known = a.rot == 0 ? pos >= 0 : (pos >= 0 && pos < a.table_rows);
  if (l < (rot >> 3) && known) {
    const float* t = a.cos_sin + pos * rot;
    const int first = 4 * l;  // of the lane's four angles
    const f32x4_t co = *reinterpret_cast<const f32x4_t*>(t + first);
    const f32x4_t si = *reinterpret_cast<const f32x4_t*>(t + (rot >> 1) + first);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p0 = a.interleaved ? 2 * j : j, p1 = a.interleaved ? 2 * j + 1 : j + 4;
      const double u = d[p0], w = d[p1], cj = co[j], sj = si[j];
      d[p0] = fma(-w, sj, u * cj);
      d[p1] = fma(u, sj, w * cj);
    }
  }
  if (is_q) {
    if (!known) {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = __builtin_nan("");
    }
    uint16_t* o = a.q_out + (row * a.q_heads + h) * D;
    *reinterpret_cast<u32x2_t*>(o + r.a) =
        u32x2_t{DT::pack2((float)d[0], (float)d[1]), DT::pack2((float)d[2], (float)d[3])};
    *reinterpret_cast<u32x2_t*>(o + r.b) =
        u32x2_t{DT::pack2((float)d[4], (float)d[5]), DT::pack2((float)d[6], (float)d[7])};
    return;
  }
  double lo = d[0], hi = d[0];
  bool fin = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = d[j] < lo ? d[j] : lo;
    hi = d[j] > hi ? d[j] : hi;
    fin = fin && fabs(d[j]) <= 1e300;
  }
  lanes_minmax<LPV>(lo, hi);
  const U4Coder u = u4_coder(lo, hi, lanes_all<LPV>(fin));
  uint32_t ca = 0, cb = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    ca |= u4_code(u, d[j], (float)(d[j] - (double)u.m)) << (4 * j);
    cb |= u4_code(u, d[j + 4], (float)(d[j + 4] - (double)u.m)) << (4 * j);
  }
  const int64_t slot = known ? kv4_slot(c, bt, b, pos, h) : -1;
  if (slot < 0) return;
  uint8_t* codes = (is_v ? c.v_codes : c.k_codes) + slot * (D / 2);
  *reinterpret_cast<uint16_t*>(codes + r.a / 2) = (uint16_t)ca;
  *reinterpret_cast<uint16_t*>(codes + r.b / 2) = (uint16_t)cb;
  if (l == 0) (is_v ? c.v_pairs : c.k_pairs)[slot] = u.pair;
}

template <class DT, int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4CacheArg c, Kv4BatchArg bt,
                                                            uint16_t* __restrict__ k_out,
                                                            uint16_t* __restrict__ v_out) {
  constexpr int LPV = D / 8, VPB = kThreads / LPV;
  const int l = threadIdx.x % LPV;
  const int64_t v = (int64_t)blockIdx.x * VPB + threadIdx.x / LPV;
  const int b = blockIdx.y;
  const Kv4Seq sq = kv4_seq(bt, b);
  const int64_t i = v / (2 * c.kv_heads);
  int h = (int)(v - i * 2 * c.kv_heads);
  if (i >= sq.n) return;
  const bool is_v = h >= c.kv_heads;
  if (is_v) h -= c.kv_heads;
  const int64_t slot = sq.pos0 + i >= 0 ? kv4_slot(c, bt, b, sq.pos0 + i, h) : -1;
  float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (slot >= 0) {
    const uint8_t* codes = (is_v ? c.v_codes : c.k_codes) + slot * (D / 2);
    u4_values8(reinterpret_cast<const uint32_t*>(codes)[l], (is_v ? c.v_pairs : c.k_pairs)[slot],
               f);
  }
  uint16_t* o = (is_v ? v_out : k_out) + ((sq.row0 + i) * c.kv_heads + h) * D + 8 * l;
  *reinterpret_cast<u32x4_t*>(o) = u32x4_t{DT::pack2(f[0], f[1]), DT::pack2(f[2], f[3]),
                                           DT::pack2(f[4], f[5]), DT::pack2(f[6], f[7])};
}

template <class F>
void by_dim(int D, F f) {
  if (D == 64)
    f(std::integral_constant<int, 64>{});
  else if (D == 128)
    f(std::integral_constant<int, 128>{});
  else
    f(std::integral_constant<int, 256>{});
}

}  // namespace

hipError_t launch_kv4_append(const Kv4CacheArg& c, const Kv4BatchArg& b, const Kv4AppendArg& a,
                             bool f16, hipStream_t s) {
  by_dim(c.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const int64_t vpb = kThreads / (D / 8), n = (int64_t)b.max_q * (a.q_heads + 2 * c.kv_heads);
    const dim3 grid((unsigned)((n + vpb - 1) / vpb), (unsigned)b.seqs);
    if (f16)
      kv4_append_kernel<F16T, D><<<grid, kThreads, 0, s>>>(c, b, a);
    else
      kv4_append_kernel<Bf16T, D><<<grid, kThreads, 0, s>>>(c, b, a);
  });
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4CacheArg& c, const Kv4BatchArg& b, uint16_t* k_out,
                           uint16_t* v_out, bool f16, hipStream_t s) {
  by_dim(c.head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const int64_t vpb = kThreads / (D / 8), n = (int64_t)b.max_q * 2 * c.kv_heads;
    const dim3 grid((unsigned)((n + vpb - 1) / vpb), (unsigned)b.seqs);
    if (f16)
      kv4_read_kernel<F16T, D><<<grid, kThreads, 0, s>>>(c, b, k_out, v_out);
    else
      kv4_read_kernel<Bf16T, D><<<grid, kThreads, 0, s>>>(c, b, k_out, v_out);
  });
  return hipGetLastError();
}

}  // namespace qlora
