// The 4-bit group format: a group of G values holds a code c in 0..15 for
// each and one pair (s, m) of bf16; a value is m + s c.  Codes are packed
// two per byte, the even element in the low nibble; a pair is one 32-bit
// word, s in the low half.
#pragma once

#include "device_common.h"

namespace qlora {

// ---- encoding --------------------------------------------------------------
// m = the group's minimum rounded down to bf16, s = (maximum - m) / 15
// rounded up to bf16, c = rint((v - m) / s) with ties to even (0 where s is
// 0), all as computed in fp64.  Rounding m down and s up keeps every
// (v - m) / s inside [0, 15], so no code is clipped and a value is off by at
// most s / 2.  A group that holds a NaN or an infinity, or whose m or s
// passes bf16's range, gets m = s = NaN and codes 0: whatever reads it is
// NaN too.

// The largest bf16 value not above x, as fp32 bits.
__device__ __forceinline__ uint32_t bf16_down(float x) {
  const uint32_t b = __float_as_uint(x), low = b & 0xFFFFu;
  return b - low + ((low && (b >> 31)) ? 0x10000u : 0u);
}
__device__ __forceinline__ uint32_t bf16_down(double x) { return bf16_down(__double2float_rd(x)); }
// (hi - m) / 15 rounded up to bf16, as fp32 bits.  The fp32 quotient is within
// 2^-22 of the exact one, so it tells which bf16 values lie around it unless
// its low 16 bits are next to 0; then the division is done in fp64.
__device__ __forceinline__ uint32_t u4_step(double range) {
  uint32_t b = __float_as_uint((float)range * (1.0f / 15.0f));
  const uint32_t low = b & 0xFFFFu;
  if (low - 8u >= 0xFFF0u || b < 0x01000000u) {
    b = __float_as_uint(__double2float_ru(range / 15.0));
    return b - (b & 0xFFFFu) + ((b & 0xFFFFu) ? 0x10000u : 0u);
  }
  return b - low + 0x10000u;
}

struct U4Coder {
  float s, m;
  float inv;    // fp32 1 / s, or 0 where the exact quotient has to be taken
  uint32_t pair;
};

// finite: every value of the group is finite.  T: the values' type, fp32 or
// fp64.
template <class T>
__device__ __forceinline__ U4Coder u4_coder(T lo, T hi, bool finite) {
  U4Coder u;
  u.m = __uint_as_float(bf16_down(lo));
  u.s = __uint_as_float(u4_step((double)hi - (double)u.m));
  // also false for an infinite or NaN m or s
  finite = finite && fabsf(u.m) <= 3.4e38f && fabsf(u.s) <= 3.4e38f;
  if (!finite) u.s = u.m = __uint_as_float(0x7FC00000u);
  // below 2^-100 the fp32 reciprocal nears its range: take the exact path
  u.inv = u.s > 0x1p-100f ? __builtin_amdgcn_rcpf(u.s) : 0.0f;
  u.pair = (__float_as_uint(u.s) >> 16) | (__float_as_uint(u.m) & 0xFFFF0000u);
  return u;
}

// rint((v - m) / s), t = fp32(v - m).  The fp32 quotient t * inv is within
// 15 * 2^-22 (t and the product are rounded once, inv is good to a unit in the
// last place) of the exact one, so it decides the code wherever it lies further than 1e-4 from a
// half; the few others (about one in 5000) divide in fp64.
__device__ __forceinline__ uint32_t u4_code(const U4Coder& u, double v, float t) {
  const float q = t * u.inv;
  float c = rintf(q);
  if (!(fabsf(q - c) < 0.4999f) || u.inv == 0.0f)
    c = u.s > 0.0f ? (float)rint((v - (double)u.m) / (double)u.s) : 0.0f;
  return (uint32_t)fminf(fmaxf(c, 0.0f), 15.0f);  // a NaN becomes 0
}

// ---- decoding --------------------------------------------------------------
// Products read the codes as 16-bit floats OFF + c, formed by putting the
// code into the mantissa of a constant: two codes per v_and_or_b32 and no
// conversion.  The offset leaves through sum(x (OFF + c)) - OFF sum(x),
// which costs bits of the fp32 sum: 7 at OFF = 128, where bf16's mantissa
// ends at the code's last bit, 4 at OFF = 16, with the code at the
// mantissa's top and one more shift for 8 codes.  Results that are rounded
// to bf16 take 128; fp16 ones, and scores, which become exponents, 16.  The
// attention's values, fp16 operands for both types of results, take 64, the
// smallest without the additional shift.
// The pairs of a word are (element j, element j + 4), j = 0..3.
// (x & mask) | bits.  With both constant the compiler takes two instructions;
// a constant whose origin it does not see sits in a register and takes one
// (v_and_or_b32).  The empty statement is no instruction: one written out in
// assembly would not be seen as a vector instruction whose result a following
// MFMA has to wait for.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  asm("" : "+v"(bits));
  return (x & mask) | bits;
}
template <uint32_t BITS, int SHIFT>
struct U4Bits {  // the code SHIFT bits up in the 16-bit constant BITS
  static __device__ __forceinline__ uint32_t pair(uint32_t w, int j) {
    const int sh = SHIFT - 4 * j;
    return and_or(sh > 0 ? w << sh : w >> -sh, 0x000F000Fu << SHIFT, BITS << 16 | BITS);
  }
};
template <class DT>
struct U4Mfma;  // products whose sums are rounded to DT
template <>
struct U4Mfma<Bf16T> : U4Bits<0x4300, 0> {
  static constexpr float kOff = 128.0f;
  static constexpr uint32_t kOne = 0x3F803F80u;  // two ones
};
template <>
struct U4Mfma<F16T> : U4Bits<0x4C00, 6> {
  static constexpr float kOff = 16.0f;
  static constexpr uint32_t kOne = 0x3C003C00u;
};
template <class DT>
struct U4Score;  // products with an operand in DT whose sums are scores
template <>
struct U4Score<Bf16T> : U4Bits<0x4180, 3> {
  static constexpr float kOff = 16.0f;
};
template <>
struct U4Score<F16T> : U4Mfma<F16T> {};
struct U4Value : U4Bits<0x5400, 4> {  // with fp16 weights of the attention's values
  static constexpr float kOff = 64.0f;
  static constexpr uint32_t kOne = 0x3C003C00u;
};
// The 8 codes of a word as MFMA operand, in the order 0 4 1 5 2 6 3 7.
template <class OP>
__device__ __forceinline__ u32x4_t u4_expand8(uint32_t w) {
  return u32x4_t{OP::pair(w, 0), OP::pair(w, 1), OP::pair(w, 2), OP::pair(w, 3)};
}
// Eight 16-bit values in the same order.
__device__ __forceinline__ u32x4_t u4_order8(u32x4_t v) {
  return u32x4_t{perm(v[2], v[0], 0x05040100u), perm(v[2], v[0], 0x07060302u),
                 perm(v[3], v[1], 0x05040100u), perm(v[3], v[1], 0x07060302u)};
}
__device__ __forceinline__ float u4_s(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float u4_m(uint32_t pair) {
  return __uint_as_float(pair & 0xFFFF0000u);
}
// The 8 codes of a word as values m + s c (one rounding, to fp32).
__device__ __forceinline__ void u4_values8(uint32_t w, uint32_t pair, float (&v)[8]) {
  const float s = u4_s(pair), m = u4_m(pair);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fmaf(s, (float)((w >> (4 * i)) & 15u), m);
}

// Stands between LDS writes of a wave's lanes and reads of the same place by
// its other lanes.  The hardware does one wave's LDS operations in order, so
// it is no instruction; it keeps the compiler, which sees one lane, from
// moving them past each other.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- reductions over 8, 16 or 32 neighbouring lanes ------------------------
// Each step brings every lane the value of a lane that holds the other half
// of the lanes combined so far.
template <int STEP>
__device__ __forceinline__ float lane_other(float v) {
  const int i = __float_as_int(v);
  if constexpr (STEP == 1) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0xB1, 15, 15, true));   // quad 1 0 3 2
  if constexpr (STEP == 2) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x4E, 15, 15, true));   // quad 2 3 0 1
  if constexpr (STEP == 4) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x141, 15, 15, true));  // mirrored in 8
  if constexpr (STEP == 8) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x140, 15, 15, true));  // mirrored in 16
  return __shfl_xor(v, STEP);
}
template <int STEP>
__device__ __forceinline__ double lane_other(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __float_as_uint(lane_other<STEP>(__uint_as_float((uint32_t)b)));
  const uint32_t hi = __float_as_uint(lane_other<STEP>(__uint_as_float((uint32_t)(b >> 32))));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int LANES, class T>
__device__ __forceinline__ void lanes_minmax(T& lo, T& hi) {
  auto step = [&](T a, T b) {
    lo = a < lo ? a : lo;
    hi = b > hi ? b : hi;
  };
  if constexpr (LANES > 1) step(lane_other<1>(lo), lane_other<1>(hi));
  if constexpr (LANES > 2) step(lane_other<2>(lo), lane_other<2>(hi));
  if constexpr (LANES > 4) step(lane_other<4>(lo), lane_other<4>(hi));
  if constexpr (LANES > 8) step(lane_other<8>(lo), lane_other<8>(hi));
  if constexpr (LANES > 16) step(lane_other<16>(lo), lane_other<16>(hi));
}
// Whether `ok` holds in all of the LANES aligned lanes that the caller is in.
template <int LANES>
__device__ __forceinline__ bool lanes_all(bool ok) {
  const uint64_t bad = __ballot(!ok);
  const int first = (threadIdx.x & 63) & ~(LANES - 1);
  constexpr uint64_t kMask = LANES == 64 ? ~0ull : (1ull << (LANES & 63)) - 1;
  return ((bad >> first) & kMask) == 0;
}

}  // namespace qlora
