// C ABI of the 4-bit group format and of the 4-bit paged cache: argument
// validation and dispatch.  As in api.cpp every argument is checked before
// the first HIP call and no C++ exception crosses the ABI.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/qlora.h"
#include "launch.h"

namespace {

constexpr int64_t kMaxRows = int64_t{1} << 30;
// The product's kernel reads 128 rows of codes and 64 of x with 32-bit offsets.
constexpr int64_t kMaxK = int64_t{1} << 23;
constexpr int64_t kMaxGrid = (int64_t{1} << 31) - 1;
// A launch holds below 2^32 threads along x.  Of a product they are at most
// 512 for 3 tiles of 16 rows; of a head vector a lane for 8 values; of the
// attention 256 for a tile of 16 query rows; of the quantiser 256 for 4096
// values and of the dequantiser 256 for 8192.
constexpr int64_t kMaxN = int64_t{1} << 28;
constexpr int64_t kMaxVectorValues = int64_t{1} << 34;
constexpr int64_t kMaxQueryRows = int64_t{1} << 27;
constexpr int64_t kMaxBlocks = (int64_t{1} << 24) - 1;  // of 256 threads
constexpr int64_t kMaxQuantized = kMaxBlocks * 4096, kMaxDequantized = kMaxBlocks * 8192;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
int hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_EHIP; }

bool group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }

const uint32_t* words(const uint16_t* p) { return reinterpret_cast<const uint32_t*>(p); }
uint32_t* words(uint16_t* p) { return reinterpret_cast<uint32_t*>(p); }

struct Range {
  const void* p;
  size_t n;
};
// Whether an output overlaps an input or another output.
template <int O, int I>
bool clash(const Range (&out)[O], const Range (&in)[I]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (overlap(out[o].p, out[o].n, in[i].p, in[i].n)) return true;
    for (int q = o + 1; q < O; ++q)
      if (overlap(out[o].p, out[o].n, out[q].p, out[q].n)) return true;
  }
  return false;
}

int check_u4(const qlora_u4_weight* w) {
  if (!w || !w->codes || !w->pairs) return QLORA_EINVAL;
  if (w->N <= 0 || w->K <= 0) return QLORA_EINVAL;
  if (!group_ok(w->group)) return QLORA_ENOTSUP;
  if (w->K % w->group || w->K > kMaxK || w->N >= kMaxN) return QLORA_ESHAPE;
  if (!aligned(w->codes, 16) || !aligned(w->pairs, 16)) return QLORA_EALIGN;
  return QLORA_OK;
}

int dequantize(const qlora_u4_weight* w, uint16_t* out, void* stream, bool f16) {
  try {
    const int st = check_u4(w);
    if (st != QLORA_OK) return st;
    if (!out) return QLORA_EINVAL;
    if (!aligned(out, 16)) return QLORA_EALIGN;
    const size_t n = (size_t)w->N * w->K;
    if (n > (size_t)kMaxDequantized) return QLORA_ESHAPE;
    if (clash<1, 2>({{out, n * 2}}, {{w->codes, n / 2}, {w->pairs, n / w->group * 4}}))
      return QLORA_EINVAL;
    return hip_status(qlora::launch_dequantize_u4(w->codes, words(w->pairs), (int64_t)n, w->group,
                                                  out, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int linear(const qlora_u4_weight* w, const uint16_t* x, int64_t ldx, int64_t M, uint16_t* y,
           int64_t ldy, void* stream, bool f16) {
  try {
    const int st = check_u4(w);
    if (st != QLORA_OK) return st;
    if (M < 0) return QLORA_EINVAL;
    if (M == 0) return QLORA_OK;
    if (!x || !y || ldx < w->K || ldy < w->N) return QLORA_EINVAL;
    if (M > 65535 * 16 || ldx > kMaxK || ldy >= kMaxGrid) return QLORA_ESHAPE;
    if (!aligned(x, 16) || ldx % 8 || !aligned(y, 2)) return QLORA_EALIGN;
    const size_t n = (size_t)w->N * w->K;
    if (clash<1, 3>({{y, ((size_t)(M - 1) * ldy + w->N) * 2}},
                    {{w->codes, n / 2},
                     {w->pairs, n / w->group * 4},
                     {x, ((size_t)(M - 1) * ldx + w->K) * 2}}))
      return QLORA_EINVAL;
    return hip_status(qlora::launch_linear_u4(w->codes, words(w->pairs), w->group, x, ldx, y, ldy,
                                              M, w->N, w->K, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int check_cache(const qlora_kv4_cache* c, qlora::Kv4CacheArg* o) {
  if (!c || !c->k_codes || !c->k_pairs || !c->v_codes || !c->v_pairs) return QLORA_EINVAL;
  if (c->pages <= 0 || c->kv_heads <= 0) return QLORA_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QLORA_ENOTSUP;
  int lg = 4;
  while (lg < 10 && (1 << lg) != c->page_size) ++lg;
  if ((1 << lg) != c->page_size) return QLORA_ENOTSUP;
  if (c->pages > kMaxGrid || c->kv_heads > 4096) return QLORA_ESHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_pairs, 16) || !aligned(c->v_codes, 16) ||
      !aligned(c->v_pairs, 16))
    return QLORA_EALIGN;
  *o = {c->k_codes, words(c->k_pairs), c->v_codes, words(c->v_pairs),
        c->pages,   lg,                c->kv_heads, c->head_dim};
  return QLORA_OK;
}
size_t code_bytes(const qlora_kv4_cache* c) {
  return (size_t)c->pages * c->kv_heads * c->page_size * (c->head_dim / 2);
}
size_t pair_bytes(const qlora_kv4_cache* c) {
  return (size_t)c->pages * c->kv_heads * c->page_size * 4;
}

int check_batch(const qlora_kv4_batch* b, const qlora_kv4_cache* c, qlora::Kv4BatchArg* o) {
  if (!b) return QLORA_EINVAL;
  if (b->seqs < 0 || b->rows < 0 || b->max_q < 0 || b->table_width < 0) return QLORA_EINVAL;
  if (b->seqs > 65535 || b->rows > kMaxRows || b->max_q > kMaxRows ||
      (int64_t)b->table_width * c->page_size > kMaxRows)
    return QLORA_ESHAPE;
  if (b->seqs > 0 && b->rows > 0 && b->max_q > 0) {
    if (!b->cu_q || !b->seq_lens || (!b->block_table && b->table_width > 0)) return QLORA_EINVAL;
    if (!aligned(b->cu_q, 4) || !aligned(b->seq_lens, 4) || !aligned(b->block_table, 4))
      return QLORA_EALIGN;
  }
  *o = {b->cu_q, b->seq_lens, b->block_table, b->rows, b->seqs, b->table_width, b->max_q};
  return QLORA_OK;
}
bool no_rows(const qlora_kv4_batch* b) { return b->seqs == 0 || b->rows == 0 || b->max_q == 0; }

// A strided tensor of T rows and `heads` heads of D: QLORA_OK and its extent
// in bytes.
int check_rows(const uint16_t* p, int64_t ts, int64_t hs, int64_t T, int heads, int D,
               size_t* bytes) {
  if (!p || ts < 0 || hs < 0) return QLORA_EINVAL;
  if (!aligned(p, 16) || ts % 8 || hs % 8) return QLORA_EALIGN;
  if (ts > kMaxGrid || hs > kMaxGrid) return QLORA_ESHAPE;
  *bytes = ((size_t)(T - 1) * ts + (size_t)(heads - 1) * hs + D) * 2;
  return QLORA_OK;
}

int append(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch, const uint16_t* k,
           int64_t k_ts, int64_t k_hs, const uint16_t* v, int64_t v_ts, int64_t v_hs,
           const uint16_t* q, int64_t q_ts, int64_t q_hs, int32_t q_heads, const float* cos_sin,
           int64_t table_rows, int32_t rot, int32_t interleaved, uint16_t* q_out, void* stream,
           bool f16) {
  try {
    qlora::Kv4CacheArg c;
    qlora::Kv4BatchArg b;
    int st = check_cache(cache, &c);
    if (st != QLORA_OK) return st;
    if ((st = check_batch(batch, cache, &b)) != QLORA_OK) return st;
    if (q_heads < 0 || rot < 0 || table_rows < 0) return QLORA_EINVAL;
    if (q_heads > 65536) return QLORA_ESHAPE;
    if (rot > c.head_dim || rot % 8) return QLORA_ESHAPE;
    if (rot > 0 && (!cos_sin || table_rows == 0)) return QLORA_EINVAL;
    if (rot > 0 && !aligned(cos_sin, 16)) return QLORA_EALIGN;
    if (rot > 0 && table_rows > kMaxRows) return QLORA_ESHAPE;
    if (no_rows(batch)) return QLORA_OK;
    size_t nk = 0, nv = 0, nq = 0;
    if ((st = check_rows(k, k_ts, k_hs, b.rows, c.kv_heads, c.head_dim, &nk)) != QLORA_OK)
      return st;
    if ((st = check_rows(v, v_ts, v_hs, b.rows, c.kv_heads, c.head_dim, &nv)) != QLORA_OK)
      return st;
    if (q_heads > 0) {
      if ((st = check_rows(q, q_ts, q_hs, b.rows, q_heads, c.head_dim, &nq)) != QLORA_OK) return st;
      if (!q_out) return QLORA_EINVAL;
      if (!aligned(q_out, 16)) return QLORA_EALIGN;
    }
    if ((int64_t)b.max_q * (q_heads + 2 * c.kv_heads) > kMaxVectorValues / c.head_dim)
      return QLORA_ESHAPE;
    const size_t cb = code_bytes(cache), pb = pair_bytes(cache);
    if (clash<5, 7>({{c.k_codes, cb},
                     {c.v_codes, cb},
                     {c.k_pairs, pb},
                     {c.v_pairs, pb},
                     {q_heads > 0 ? q_out : nullptr, (size_t)b.rows * q_heads * c.head_dim * 2}},
                    {{k, nk},
                     {v, nv},
                     {q_heads > 0 ? q : nullptr, nq},
                     {rot > 0 ? cos_sin : nullptr, (size_t)table_rows * rot * 4},
                     {b.cu_q, (size_t)(b.seqs + 1) * 4},
                     {b.seq_lens, (size_t)b.seqs * 4},
                     {b.block_table, (size_t)b.seqs * b.table_width * 4}}))
      return QLORA_EINVAL;
    const qlora::Kv4AppendArg a{q,    k,       v,          q_ts,    q_hs, k_ts,        k_hs, v_ts,
                                v_hs, cos_sin, table_rows, q_heads, rot,  interleaved, q_out};
    return hip_status(qlora::launch_kv4_append(c, b, a, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int read(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch, uint16_t* k_out,
         uint16_t* v_out, void* stream, bool f16) {
  try {
    qlora::Kv4CacheArg c;
    qlora::Kv4BatchArg b;
    int st = check_cache(cache, &c);
    if (st != QLORA_OK) return st;
    if ((st = check_batch(batch, cache, &b)) != QLORA_OK) return st;
    if (no_rows(batch)) return QLORA_OK;
    if (!k_out || !v_out) return QLORA_EINVAL;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return QLORA_EALIGN;
    if ((int64_t)b.max_q * 2 * c.kv_heads > kMaxVectorValues / c.head_dim) return QLORA_ESHAPE;
    const size_t cb = code_bytes(cache), pb = pair_bytes(cache),
                 no = (size_t)b.rows * c.kv_heads * c.head_dim * 2;
    if (clash<2, 7>({{k_out, no}, {v_out, no}},
                    {{c.k_codes, cb},
                     {c.v_codes, cb},
                     {c.k_pairs, pb},
                     {c.v_pairs, pb},
                     {b.cu_q, (size_t)(b.seqs + 1) * 4},
                     {b.seq_lens, (size_t)b.seqs * 4},
                     {b.block_table, (size_t)b.seqs * b.table_width * 4}}))
      return QLORA_EINVAL;
    return hip_status(qlora::launch_kv4_read(c, b, k_out, v_out, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

// The shape part of the attention call, shared with the workspace query.
int attn_plan(int64_t seqs, int64_t max_q, int64_t max_len, int32_t q_heads, int32_t kv_heads,
              int32_t head_dim, int32_t window, qlora::Kv4AttnPlan* p) {
  if (seqs < 0 || max_q < 0 || max_len < 0 || q_heads <= 0 || kv_heads <= 0 || window < 0)
    return QLORA_EINVAL;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return QLORA_ENOTSUP;
  if (seqs > 65535 || max_q > kMaxRows || max_len > kMaxRows || kv_heads > 4096 ||
      q_heads > 65536 || q_heads % kv_heads)
    return QLORA_ESHAPE;
  if (max_q * (q_heads / kv_heads) > kMaxQueryRows) return QLORA_ESHAPE;
  *p = qlora::kv4_attn_plan(seqs, max_q, max_len, q_heads, kv_heads, head_dim, window);
  return QLORA_OK;
}

int attention(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch, const uint16_t* q,
              int64_t q_ts, int64_t q_hs, int32_t q_heads, float scale, int32_t causal,
              int32_t window, int64_t max_len, uint16_t* out, float* lse, void* workspace,
              size_t ws_bytes, void* stream, bool f16) {
  try {
    qlora::Kv4CacheArg c;
    qlora::Kv4BatchArg b;
    qlora::Kv4AttnPlan p;
    int st = check_cache(cache, &c);
    if (st != QLORA_OK) return st;
    if ((st = check_batch(batch, cache, &b)) != QLORA_OK) return st;
    if (!std::isfinite(scale)) return QLORA_EINVAL;
    if ((st = attn_plan(b.seqs, b.max_q, max_len, q_heads, c.kv_heads, c.head_dim, window, &p)) !=
        QLORA_OK)
      return st;
    if (no_rows(batch)) return QLORA_OK;
    size_t nq = 0;
    if ((st = check_rows(q, q_ts, q_hs, b.rows, q_heads, c.head_dim, &nq)) != QLORA_OK) return st;
    if (!out) return QLORA_EINVAL;
    if (!aligned(out, 16) || !aligned(lse, 4)) return QLORA_EALIGN;
    const size_t need = qlora::kv4_attn_workspace(p, b.seqs, c.kv_heads, c.head_dim);
    if (need > 0) {
      if (!workspace || ws_bytes < need) return QLORA_EWORKSPACE;
      if (!aligned(workspace, 256)) return QLORA_EALIGN;
    }
    const size_t cb = code_bytes(cache), pb = pair_bytes(cache);
    if (clash<3, 8>({{out, (size_t)b.rows * q_heads * c.head_dim * 2},
                     {lse, (size_t)b.rows * q_heads * 4},
                     {need > 0 ? workspace : nullptr, need}},
                    {{q, nq},
                     {c.k_codes, cb},
                     {c.v_codes, cb},
                     {c.k_pairs, pb},
                     {c.v_pairs, pb},
                     {b.cu_q, (size_t)(b.seqs + 1) * 4},
                     {b.seq_lens, (size_t)b.seqs * 4},
                     {b.block_table, (size_t)b.seqs * b.table_width * 4}}))
      return QLORA_EINVAL;
    const qlora::Kv4AttnArg a{q,      q_ts,   q_hs, q_heads,
                              scale,  causal, window,
                              (int64_t)b.table_width * cache->page_size, out, lse};
    float* ws = need > 0 ? static_cast<float*>(workspace) : nullptr;
    return hip_status(qlora::launch_kv4_attention(c, b, a, p, ws, f16, as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

}  // namespace

extern "C" {

int qlora_quantize_u4(const float* w, int64_t n_elems, int32_t group, uint8_t* codes,
                      uint16_t* pairs, void* stream) {
  try {
    if (n_elems < 0) return QLORA_EINVAL;
    if (!group_ok(group)) return QLORA_ENOTSUP;
    if (n_elems % group || n_elems > kMaxQuantized) return QLORA_ESHAPE;
    if (n_elems == 0) return QLORA_OK;
    if (!w || !codes || !pairs) return QLORA_EINVAL;
    if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(pairs, 16)) return QLORA_EALIGN;
    const size_t n = (size_t)n_elems;
    if (clash<2, 1>({{codes, n / 2}, {pairs, n / group * 4}}, {{w, n * 4}})) return QLORA_EINVAL;
    return hip_status(
        qlora::launch_quantize_u4(w, n_elems, group, codes, words(pairs), as_stream(stream)));
  } catch (...) {
    return QLORA_EHIP;
  }
}

int qlora_dequantize_u4(const qlora_u4_weight* w, uint16_t* out, void* stream) {
  return dequantize(w, out, stream, false);
}
int qlora_dequantize_u4_f16(const qlora_u4_weight* w, uint16_t* out, void* stream) {
  return dequantize(w, out, stream, true);
}

int qlora_linear_u4_fwd(const qlora_u4_weight* w, const uint16_t* x, int64_t ldx, int64_t M,
                        uint16_t* y, int64_t ldy, void* stream) {
  return linear(w, x, ldx, M, y, ldy, stream, false);
}
int qlora_linear_u4_fwd_f16(const qlora_u4_weight* w, const uint16_t* x, int64_t ldx, int64_t M,
                            uint16_t* y, int64_t ldy, void* stream) {
  return linear(w, x, ldx, M, y, ldy, stream, true);
}

int qlora_kv4_append(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch, const uint16_t* k,
                     int64_t k_ts, int64_t k_hs, const uint16_t* v, int64_t v_ts, int64_t v_hs,
                     const uint16_t* q, int64_t q_ts, int64_t q_hs, int32_t q_heads,
                     const float* cos_sin, int64_t table_rows, int32_t rot, int32_t interleaved,
                     uint16_t* q_out, void* stream) {
  return append(cache, batch, k, k_ts, k_hs, v, v_ts, v_hs, q, q_ts, q_hs, q_heads, cos_sin,
                table_rows, rot, interleaved, q_out, stream, false);
}
int qlora_kv4_append_f16(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch,
                         const uint16_t* k, int64_t k_ts, int64_t k_hs, const uint16_t* v,
                         int64_t v_ts, int64_t v_hs, const uint16_t* q, int64_t q_ts, int64_t q_hs,
                         int32_t q_heads, const float* cos_sin, int64_t table_rows, int32_t rot,
                         int32_t interleaved, uint16_t* q_out, void* stream) {
  return append(cache, batch, k, k_ts, k_hs, v, v_ts, v_hs, q, q_ts, q_hs, q_heads, cos_sin,
                table_rows, rot, interleaved, q_out, stream, true);
}

int qlora_kv4_read(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch, uint16_t* k_out,
                   uint16_t* v_out, void* stream) {
  return read(cache, batch, k_out, v_out, stream, false);
}
int qlora_kv4_read_f16(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch, uint16_t* k_out,
                       uint16_t* v_out, void* stream) {
  return read(cache, batch, k_out, v_out, stream, true);
}

size_t qlora_kv4_attention_workspace_bytes(int64_t seqs, int64_t max_q, int64_t max_len,
                                           int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                           int32_t window) {
  try {
    qlora::Kv4AttnPlan p;
    if (attn_plan(seqs, max_q, max_len, q_heads, kv_heads, head_dim, window, &p) != QLORA_OK)
      return 0;
    return qlora::kv4_attn_workspace(p, seqs, kv_heads, head_dim);
  } catch (...) {
    return 0;
  }
}

int qlora_kv4_attention(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch,
                        const uint16_t* q, int64_t q_ts, int64_t q_hs, int32_t q_heads,
                        float scale, int32_t causal, int32_t window, int64_t max_len,
                        uint16_t* out, float* lse, void* workspace, size_t ws_bytes,
                        void* stream) {
  return attention(cache, batch, q, q_ts, q_hs, q_heads, scale, causal, window, max_len, out, lse,
                   workspace, ws_bytes, stream, false);
}
int qlora_kv4_attention_f16(const qlora_kv4_cache* cache, const qlora_kv4_batch* batch,
                            const uint16_t* q, int64_t q_ts, int64_t q_hs, int32_t q_heads,
                            float scale, int32_t causal, int32_t window, int64_t max_len,
                            uint16_t* out, float* lse, void* workspace, size_t ws_bytes,
                            void* stream) {
  return attention(cache, batch, q, q_ts, q_hs, q_heads, scale, causal, window, max_len, out, lse,
                   workspace, ws_bytes, stream, true);
}

}  // extern "C"
