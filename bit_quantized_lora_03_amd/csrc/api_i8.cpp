// C ABI of the 8-bit row format, its products and the norm that writes it:
// argument validation and dispatch.  As in api.cpp every argument is checked
// before the first HIP call and no C++ exception crosses the ABI.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/qlora.h"
#include "i8_common.h"
#include "launch.h"

namespace {

// No sum of K products of two codes (-128 among them, which no quantiser
// writes) passes 2^31.
constexpr int64_t kMaxK = (int64_t{1} << 17) - qlora::kI8Pad;
// A launch holds below 2^32 threads along x: the quantiser's 1024 for 2 rows.
constexpr int64_t kMaxN = (int64_t{1} << 23) - 64;
constexpr int64_t kMaxM = int64_t{1} << 30;
// Tokens of a product: their scales have 32-bit offsets.
constexpr int64_t kMaxLinearM = int64_t{1} << 28;
constexpr int64_t kMaxStride = (int64_t{1} << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
int hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_EHIP; }

struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// Whether an output overlaps an input or another output.
template <int O, int I>
bool clash(const Range (&out)[O], const Range (&in)[I]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (overlap(out[o], in[i])) return true;
    for (int q = o + 1; q < O; ++q)
      if (overlap(out[o], out[q])) return true;
  }
  return false;
}
size_t rows_bytes(int64_t M, int64_t ld, int64_t K) {
  return ((size_t)(M - 1) * (size_t)ld + (size_t)K) * 2;
}
size_t tile_bytes(int64_t N, int64_t K) {
  return (size_t)((N + 15) / 16) * 16 * (size_t)qlora::i8_padded(K);
}
size_t code_bytes(int64_t M, int64_t K) { return (size_t)M * (size_t)qlora::i8_padded(K); }

int check_size(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0) return QLORA_EINVAL;
  return N > kMaxN || K > kMaxK ? QLORA_ESHAPE : QLORA_OK;
}
int check_weight(const qlora_i8_weight* w) {
  if (!w || !w->tiles || !w->scales) return QLORA_EINVAL;
  const int st = check_size(w->N, w->K);
  if (st != QLORA_OK) return st;
  return aligned(w->tiles, 16) && aligned(w->scales, 4) ? QLORA_OK : QLORA_EALIGN;
}
// codes and scales of M tokens (M = 0: none of either is looked at)
int check_tokens(const int8_t* codes, const float* scales, int64_t M, int64_t K) {
  if (M < 0 || K <= 0) return QLORA_EINVAL;
  if (M > kMaxM || K > kMaxK) return QLORA_ESHAPE;
  if (M == 0) return QLORA_OK;
  if (!codes || !scales) return QLORA_EINVAL;
  return aligned(codes, 16) && aligned(scales, 4) ? QLORA_OK : QLORA_EALIGN;
}
int check_tokens(const qlora_i8_tokens* t) {
  return t ? check_tokens(t->codes, t->scales, t->M, t->K) : QLORA_EINVAL;
}
// rows of 16-bit floats, ld apart
int check_rows(const uint16_t* p, int64_t ld, int64_t K) {
  if (!p || ld < K) return QLORA_EINVAL;
  if (ld > kMaxStride) return QLORA_ESHAPE;
  return aligned(p, 2) ? QLORA_OK : QLORA_EALIGN;
}

int dequantize_weight(const qlora_i8_weight* w, uint16_t* out, void* stream, bool f16) {
  try {
    const int st = check_weight(w);
    if (st != QLORA_OK) return st;
    if (!out) return QLORA_EINVAL;
    if (!aligned(out, 2)) return QLORA_EALIGN;
    if (clash<1, 2>({{out, (size_t)w->N * w->K * 2}},
                    {{w->tiles, tile_bytes(w->N, w->K)}, {w->scales, (size_t)w->N * 4}}))
      return QLORA_EINVAL;
    return hip_status(
        qlora::launch_dequantize_i8(w->tiles, w->scales, w->N, w->K, out, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int quantize_tokens(const uint16_t* x, int64_t ldx, int64_t M, int64_t K, int8_t* codes,
                    float* scales, void* stream, bool f16) {
  try {
    int st = check_tokens(codes, scales, M, K);
    if (st != QLORA_OK || M == 0) return st;
    if ((st = check_rows(x, ldx, K)) != QLORA_OK) return st;
    if (clash<2, 1>({{codes, code_bytes(M, K)}, {scales, (size_t)M * 4}},
                    {{x, rows_bytes(M, ldx, K)}}))
      return QLORA_EINVAL;
    const qlora::I8RowsArg p{x, nullptr, nullptr, nullptr, ldx, 0, 0, M, K, 0.0, codes, scales};
    return hip_status(qlora::launch_rows_i8(p, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int dequantize_tokens(const qlora_i8_tokens* t, uint16_t* out, void* stream, bool f16) {
  try {
    const int st = check_tokens(t);
    if (st != QLORA_OK || t->M == 0) return st;
    if (!out) return QLORA_EINVAL;
    if (!aligned(out, 2)) return QLORA_EALIGN;
    if (clash<1, 2>({{out, (size_t)t->M * t->K * 2}},
                    {{t->codes, code_bytes(t->M, t->K)}, {t->scales, (size_t)t->M * 4}}))
      return QLORA_EINVAL;
    return hip_status(
        qlora::launch_values_i8(t->codes, t->scales, t->M, t->K, out, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int norm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
         const uint16_t* weight, double eps, int64_t M, int64_t K, uint16_t* h, int64_t ldh,
         int8_t* codes, float* scales, void* stream, bool f16) {
  try {
    int st = check_tokens(codes, scales, M, K);
    if (st != QLORA_OK) return st;
    if (!(eps >= 0.0) || !std::isfinite(eps)) return QLORA_EINVAL;
    if (!residual != !h) return QLORA_EINVAL;
    if (M == 0) return QLORA_OK;
    if ((st = check_rows(x, ldx, K)) != QLORA_OK) return st;
    if ((st = check_rows(weight, K, K)) != QLORA_OK) return st;
    if (residual) {
      if ((st = check_rows(residual, ldr, K)) != QLORA_OK) return st;
      if ((st = check_rows(h, ldh, K)) != QLORA_OK) return st;
    }
    const Range rx{x, rows_bytes(M, ldx, K)}, rw{weight, (size_t)K * 2},
        rr{residual, residual ? rows_bytes(M, ldr, K) : 0},
        rh{h, h ? rows_bytes(M, ldh, K) : 0};
    const Range rc{codes, code_bytes(M, K)}, rs{scales, (size_t)M * 4};
    if (clash<2, 4>({rc, rs}, {rx, rw, rr, rh}) || overlap(rh, rw)) return QLORA_EINVAL;
    // h may be x or the residual, row for row
    if (overlap(rh, rx) && !(h == x && (ldh == ldx || M == 1))) return QLORA_EINVAL;
    if (overlap(rh, rr) && !(h == residual && (ldh == ldr || M == 1))) return QLORA_EINVAL;
    const qlora::I8RowsArg p{x, residual, weight, h, ldx, ldr, ldh, M, K, eps, codes, scales};
    return hip_status(qlora::launch_rows_i8(p, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int linear(const qlora_i8_weight* w, const qlora_i8_weight* up, bool gated, int32_t act,
           const qlora_i8_tokens* x, uint16_t* y, int64_t ldy, void* stream, bool f16) {
  try {
    int st = check_weight(w);
    if (st != QLORA_OK) return st;
    if (gated) {
      if ((st = check_weight(up)) != QLORA_OK) return st;
      if (up->N != w->N || up->K != w->K) return QLORA_EINVAL;
      if (act != QLORA_ACT_SILU && act != QLORA_ACT_GELU) return QLORA_ENOTSUP;
    }
    if ((st = check_tokens(x)) != QLORA_OK) return st;
    if (x->K != w->K) return QLORA_EINVAL;
    if (x->M == 0) return QLORA_OK;
    if (!y || ldy < w->N) return QLORA_EINVAL;
    // a grid of large tiles has at most two blocks, of 256 threads, for each 64 x 64
    // outputs, one of small tiles is taken below 2^22 blocks of 512
    if (ldy > kMaxStride || x->M > kMaxLinearM ||
        ((x->M + 63) / 64) * ((w->N + 63) / 64) >= (int64_t{1} << 22))
      return QLORA_ESHAPE;
    if (!aligned(y, 2)) return QLORA_EALIGN;
    const size_t tb = tile_bytes(w->N, w->K), sb = (size_t)w->N * 4;
    if (clash<1, 6>({{y, rows_bytes(x->M, ldy, w->N)}},
                    {{w->tiles, tb},
                     {w->scales, sb},
                     {gated ? up->tiles : nullptr, tb},
                     {gated ? up->scales : nullptr, sb},
                     {x->codes, code_bytes(x->M, x->K)},
                     {x->scales, (size_t)x->M * 4}}))
      return QLORA_EINVAL;
    const qlora::I8LinearArg p{{w->tiles, gated ? up->tiles : nullptr},
                               {w->scales, gated ? up->scales : nullptr},
                               x->codes,
                               x->scales,
                               y,
                               ldy,
                               x->M,
                               w->N,
                               w->K,
                               act};
    return hip_status(qlora::launch_linear_i8(p, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

}  // namespace

extern "C" {

int qlora_quantize_i8(const float* w, int64_t N, int64_t K, int8_t* tiles, float* scales,
                      void* stream) {
  try {
    const int st = check_size(N, K);
    if (st != QLORA_OK) return st;
    if (!w || !tiles || !scales) return QLORA_EINVAL;
    if (!aligned(w, 4) || !aligned(tiles, 16) || !aligned(scales, 4)) return QLORA_EALIGN;
    if (clash<2, 1>({{tiles, tile_bytes(N, K)}, {scales, (size_t)N * 4}},
                    {{w, (size_t)N * K * 4}}))
      return QLORA_EINVAL;
    return hip_status(qlora::launch_quantize_i8(w, N, K, tiles, scales, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int qlora_dequantize_i8(const qlora_i8_weight* w, uint16_t* out, void* stream) {
  return dequantize_weight(w, out, stream, false);
}
int qlora_dequantize_i8_f16(const qlora_i8_weight* w, uint16_t* out, void* stream) {
  return dequantize_weight(w, out, stream, true);
}

int qlora_quantize_tokens_i8(const uint16_t* x, int64_t ldx, int64_t M, int64_t K, int8_t* codes,
                             float* scales, void* stream) {
  return quantize_tokens(x, ldx, M, K, codes, scales, stream, false);
}
int qlora_quantize_tokens_i8_f16(const uint16_t* x, int64_t ldx, int64_t M, int64_t K,
                                 int8_t* codes, float* scales, void* stream) {
  return quantize_tokens(x, ldx, M, K, codes, scales, stream, true);
}

int qlora_dequantize_tokens_i8(const qlora_i8_tokens* t, uint16_t* out, void* stream) {
  return dequantize_tokens(t, out, stream, false);
}
int qlora_dequantize_tokens_i8_f16(const qlora_i8_tokens* t, uint16_t* out, void* stream) {
  return dequantize_tokens(t, out, stream, true);
}

int qlora_rms_norm_i8(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
                      const uint16_t* weight, double eps, int64_t M, int64_t K, uint16_t* h,
                      int64_t ldh, int8_t* codes, float* scales, void* stream) {
  return norm(x, ldx, residual, ldr, weight, eps, M, K, h, ldh, codes, scales, stream, false);
}
int qlora_rms_norm_i8_f16(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
                          const uint16_t* weight, double eps, int64_t M, int64_t K, uint16_t* h,
                          int64_t ldh, int8_t* codes, float* scales, void* stream) {
  return norm(x, ldx, residual, ldr, weight, eps, M, K, h, ldh, codes, scales, stream, true);
}

int qlora_linear_i8_fwd(const qlora_i8_weight* w, const qlora_i8_tokens* x, uint16_t* y,
                        int64_t ldy, void* stream) {
  return linear(w, nullptr, false, 0, x, y, ldy, stream, false);
}
int qlora_linear_i8_fwd_f16(const qlora_i8_weight* w, const qlora_i8_tokens* x, uint16_t* y,
                            int64_t ldy, void* stream) {
  return linear(w, nullptr, false, 0, x, y, ldy, stream, true);
}

int qlora_gated_i8_fwd(const qlora_i8_weight* gate, const qlora_i8_weight* up, int32_t act,
                       const qlora_i8_tokens* x, uint16_t* y, int64_t ldy, void* stream) {
  return linear(gate, up, true, act, x, y, ldy, stream, false);
}
int qlora_gated_i8_fwd_f16(const qlora_i8_weight* gate, const qlora_i8_weight* up, int32_t act,
                           const qlora_i8_tokens* x, uint16_t* y, int64_t ldy, void* stream) {
  return linear(gate, up, true, act, x, y, ldy, stream, true);
}

}  // extern "C"
