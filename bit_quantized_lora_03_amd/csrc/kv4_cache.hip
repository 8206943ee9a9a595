// Rows of the 4-bit paged cache: appending rotated keys and values, and
// reading rows back.
//
// The cache holds, for keys and for values, codes [pages][kv heads]
// [page size][head_dim / 2] and pairs [pages][kv heads][page size]: one
// group of the 4-bit format (u4_common.h) per token and head.
//
// Both are bound by latency at a decode step and by HBM at a prefill.  A
// head's vector is D / 8 neighbouring lanes with 8 values each, every vector
// of a call is independent, and a token's sequence comes from the grid (y), so
// no lane searches for it.  Several vectors for each lane, asked for together,
// were no faster (43 against 40 us).
//
// Measured: 64 new tokens of 32 + 2 x 8 heads, D 128, bf16: 4.0 us, the read
// 3.0; 6600 tokens of them, fp16: 40 us (a copy of the same bytes takes 30),
// the read 9.5.

#include "kv4_common.h"
#include "launch.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

// One head vector is D / 8 lanes.  A lane has two runs of four values, which
// start at a and b: where it rotates pairs (i, i + rot / 2), at 4 l and
// rot / 2 + 4 l, so that it has both of a pair; else (no rotation, rotation
// of neighbours, and past the rotated part) they are one run of 8.
struct Runs {
  int a, b;
};
__device__ __forceinline__ Runs lane_runs(int l, int rot, bool halves) {
  if (halves && l < rot >> 3) return {4 * l, (rot >> 1) + 4 * l};
  return {8 * l, 8 * l + 4};
}

template <class DT>
__device__ __forceinline__ void unpack4(u32x2_t w, float (&v)[8], int at) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[at + i] = DT::tof((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
}

// Codes and pair of a head vector of T (fp32: as loaded; fp64: rotated), into
// its place in the cache.
template <int D, class T>
__device__ __forceinline__ void encode(const T (&v)[8], Runs r, bool halves, int l, int64_t slot,
                                       uint8_t* codes, uint32_t* pairs) {
  T lo = v[0], hi = v[0];
  bool fin = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = v[j] < lo ? v[j] : lo;
    hi = v[j] > hi ? v[j] : hi;
    fin = fin && fabs(v[j]) <= (T)3.4028234663852886e38;
  }
  lanes_minmax<D / 8>(lo, hi);
  const U4Coder u = u4_coder<T>(lo, hi, lanes_all<D / 8>(fin));
  uint32_t ca = 0, cb = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    ca |= u4_code(u, v[j], (float)(v[j] - (T)u.m)) << (4 * j);
    cb |= u4_code(u, v[j + 4], (float)(v[j + 4] - (T)u.m)) << (4 * j);
  }
  if (slot < 0) return;
  uint8_t* c = codes + slot * (D / 2);
  if (!halves) {
    *reinterpret_cast<uint32_t*>(c + r.a / 2) = ca | cb << 16;
  } else {
    *reinterpret_cast<uint16_t*>(c + r.a / 2) = (uint16_t)ca;
    *reinterpret_cast<uint16_t*>(c + r.b / 2) = (uint16_t)cb;
  }
  if (l == 0) pairs[slot] = u.pair;
}

// Rotation runs in fp64 (a few operations a value at fp32's rate): a product
// of a 16-bit value and an fp32 cosine is exact there and the rotated value
// is rounded once, so codes at a border come out as defined.
template <class DT, int D>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(Kv4CacheArg c, Kv4BatchArg bt,
                                                              Kv4AppendArg a) {
  constexpr int LPV = D / 8, VPB = kThreads / LPV;
  const int l = threadIdx.x % LPV;
  const uint32_t v = blockIdx.x * VPB + threadIdx.x / LPV;
  const uint32_t heads = a.q_heads + 2 * c.kv_heads;
  const int b = blockIdx.y;
  const Kv4Seq sq = kv4_seq(bt, b);
  const int i = v / heads;
  int h = v - i * heads;
  if (i >= sq.n) return;
  const int64_t row = sq.row0 + i, pos = sq.pos0 + i;
  const bool is_q = h < a.q_heads;
  if (!is_q) h -= a.q_heads;
  const bool is_v = !is_q && h >= c.kv_heads;
  if (is_v) h -= c.kv_heads;

  const int rot = is_v ? 0 : a.rot;
  const bool halves = rot > 0 && !a.interleaved;
  const Runs r = lane_runs(l, rot, halves);
  const uint16_t* src = is_q   ? a.q + row * a.q_ts + h * a.q_hs
                        : is_v ? a.v + row * a.v_ts + h * a.v_hs
                               : a.k + row * a.k_ts + h * a.k_hs;
  float x[8];
  if (!halves) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(src + r.a);
    unpack4<DT>(u32x2_t{w[0], w[1]}, x, 0);
    unpack4<DT>(u32x2_t{w[2], w[3]}, x, 4);
  } else {
    unpack4<DT>(*reinterpret_cast<const u32x2_t*>(src + r.a), x, 0);
    unpack4<DT>(*reinterpret_cast<const u32x2_t*>(src + r.b), x, 4);
  }
  // no angle for this position: the query becomes NaN, nothing is stored
  const bool known = pos >= 0 && (a.rot == 0 || pos < a.table_rows);
  if (is_v) {
    encode<D, float>(x, r, false, l, known ? kv4_slot(c, bt, b, pos, h) : -1, c.v_codes, c.v_pairs);
    return;
  }
  double d[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] = x[j];
  if (l < (rot >> 3) && known) {
    const float* t = a.cos_sin + pos * rot + 4 * l;  // the lane's four angles
    const f32x4_t co = *reinterpret_cast<const f32x4_t*>(t);
    const f32x4_t si = *reinterpret_cast<const f32x4_t*>(t + (rot >> 1));
    auto turn = [&](double& p, double& q, int j) {
      const double u = p, w = q;
      p = fma(-w, (double)si[j], u * (double)co[j]);
      q = fma(u, (double)si[j], w * (double)co[j]);
    };
    if (halves) {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn(d[j], d[j + 4], j);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn(d[2 * j], d[2 * j + 1], j);
    }
  }
  if (!is_q) {
    encode<D, double>(d, r, halves, l, known ? kv4_slot(c, bt, b, pos, h) : -1, c.k_codes,
                      c.k_pairs);
    return;
  }
  // by way of fp32, which the compiler may not see: it knows no instruction
  // from fp64 to fp16 and writes 35 for each value instead of two
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = known ? (float)d[j] : __builtin_nanf("");
    asm("" : "+v"(x[j]));
  }
  uint16_t* o = a.q_out + (row * a.q_heads + h) * D;
  const u32x2_t oa = {DT::pack2(x[0], x[1]), DT::pack2(x[2], x[3])};
  const u32x2_t ob = {DT::pack2(x[4], x[5]), DT::pack2(x[6], x[7])};
  if (!halves) {
    *reinterpret_cast<u32x4_t*>(o + r.a) = u32x4_t{oa[0], oa[1], ob[0], ob[1]};
  } else {
    *reinterpret_cast<u32x2_t*>(o + r.a) = oa;
    *reinterpret_cast<u32x2_t*>(o + r.b) = ob;
  }
}

template <class DT, int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4CacheArg c, Kv4BatchArg bt,
                                                            uint16_t* __restrict__ k_out,
                                                            uint16_t* __restrict__ v_out) {
  constexpr int LPV = D / 8, VPB = kThreads / LPV;
  const int l = threadIdx.x % LPV;
  const uint32_t v = blockIdx.x * VPB + threadIdx.x / LPV, heads = 2 * c.kv_heads;
  const int b = blockIdx.y;
  const Kv4Seq sq = kv4_seq(bt, b);
  const int i = v / heads;
  int h = v - i * heads;
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
