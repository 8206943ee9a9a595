// The 8-bit row format: a row (a token, or an output channel of a weight)
// with the largest magnitude a has the fp32 scale s = a / 127 and codes
// rint(127 v / a), halves to even; a value is s times its code.  Rows are
// stored with K rounded up to kI8Pad columns, zeros behind K, so no kernel
// has a tail along K.
//
// Tokens are rows in memory.  A weight is stored in tiles of 16 rows and 64
// columns in the order in which the matrix instructions take them: [N / 16]
// [K / 64][4][16][16], sixteen rows' first 16 bytes, then their next.  Lane l
// of a wave that multiplies 16 rows takes row l % 16 and piece l / 16, so its
// 64 pieces are one run of 1024 bytes.
#pragma once

#include "device_common.h"

namespace qlora {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kI8Pad = 128;   // columns
constexpr int kI8Tile = 1024;  // bytes: 16 rows, 64 columns
__host__ __device__ __forceinline__ int64_t i8_padded(int64_t K) {
  return (K + kI8Pad - 1) & ~(int64_t)(kI8Pad - 1);
}

// How a row is coded.  The quotient 127 v / a decides borders exactly: it
// differs from h / 2, h odd, by |254 v - h a| / (h a) of it, and with v = V 2^e
// and a = A 2^f the difference is a multiple of 2^f (then 1 / (h A) at least) or
// an even one of 2^e (1 / (127 V)).  V and A are below 2^24, or 2^22 as products
// of two 16-bit floats, and h is at most 253, so a quotient that is no half is
// more than 2^-32 of itself away from any (2^-30); some come that close.  A half
// comes out as it is: q below is the quotient rounded once (r is off by an ulp at
// most, and one correction in exact arithmetic follows).
struct I8Row {
  double a, r;  // r = 1 / a, or 0 for a row of zeros
  float s;
  bool ok;      // without NaN and infinity; otherwise s is NaN and codes are 0
};
// `times` is a factor of the scale that the codes do not have (a norm's).
__device__ __forceinline__ I8Row i8_row(double a, double times, bool ok) {
  I8Row o;
  const float s = (float)(a * times / 127.0);
  o.ok = ok && s <= 3.4028235e38f;
  o.s = o.ok ? s : __uint_as_float(0x7fc00000u);
  o.a = a;
  o.r = a > 0.0 ? 1.0 / a : 0.0;
  return o;
}
__device__ __forceinline__ int i8_code(const I8Row& w, double v) {
  const double t = 127.0 * v;
  const double q0 = t * w.r;
  const double q = __builtin_fma(__builtin_fma(-q0, w.a, t), w.r, q0);
  return w.ok ? (int)__builtin_rint(q) : 0;
}

// What a code stands for, a sum of products of codes, and a gated value: each
// product is rounded to fp32.  (The compiler makes one instruction with one
// rounding of the last and a conversion to fp16 where it sees both, also with
// contraction off, so it is not let to: a gated value in fp16 depended on the
// kernel, so on the number of tokens.)
__device__ __forceinline__ float i8_value(int8_t c, float s) {
  float v = (float)c * s;
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ float i8_scaled(int32_t sum, float sw, float sx) {
  float v = (float)sum * sw * sx;
  asm("" : "+v"(v));
  return v;
}

constexpr int kI8Silu = 0, kI8Gelu = 1;
// act(g) u.  Both forms are g / (1 + exp(-z)): z = g, or for gelu's tanh form
// z = 2 sqrt(2 / pi) (g + 0.044715 g^3).
__device__ __forceinline__ float i8_gated(float g, float u, int act) {
  const float z = act == kI8Silu ? g : 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
  float v = g * __builtin_amdgcn_rcpf(1.0f + __expf(-z)) * u;
  asm("" : "+v"(v));
  return v;
}

// The tile of a block.  Blocks go to the eight XCDs in turn; neighbouring ranks
// are made to be on one, whose L2 then holds what they share.  Ranks walk bands
// of 1024 tokens, a column of tiles of the band at a time.
__device__ __forceinline__ void i8_tile_of(uint32_t id, uint32_t total, uint32_t m_tiles,
                                           uint32_t n_tiles, uint32_t band, uint32_t& m,
                                           uint32_t& n) {
  const uint32_t xcd = id % 8, per = total / 8, extra = total % 8;
  const uint32_t rank = xcd * per + min(xcd, extra) + id / 8;
  const uint32_t span = band * n_tiles, g = rank / span, w = rank - g * span;
  const uint32_t gm = min(m_tiles - band * g, band);
  n = w / gm;
  m = band * g + (w - n * gm);
}

// Eight neighbouring 16-bit floats of a row that ends at K; rows may start at
// any multiple of 2 bytes.
__device__ __forceinline__ u32x4_t load_piece(const uint16_t* p, int k, int K) {
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (k + 8 <= K) {
    __builtin_memcpy(&v, p + k, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < K) v[j / 2] |= (uint32_t)p[k + j] << (16 * (j & 1));
  }
  return v;
}
__device__ __forceinline__ void store_piece(uint16_t* p, int k, int K, u32x4_t v) {
  if (k + 8 <= K) {
    __builtin_memcpy(p + k, &v, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < K) p[k + j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ uint32_t half_of(u32x4_t v, int j) {
  return (v[j / 2] >> (16 * (j & 1))) & 0xFFFFu;
}

}  // namespace qlora
