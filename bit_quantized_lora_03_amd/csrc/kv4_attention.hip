// Attention of a ragged batch over the 4-bit paged cache.
//
// For one query row with scores z_t = scale (s_t q.c_t + m_t sum q) over the
// codes c_t and the pair (s_t, m_t) of key t, and p_t = 2^(z_t log2 e - M):
//   o_d = (sum_t p_t s'_t c'_td + sum_t p_t m'_t) / sum_t p_t
// with the values' codes c' and pairs (s', m').  The pairs never meet the
// codes: scores are scaled after the product, and s'_t goes into p_t.
//
// Bound by HBM on the cache at few rows.  The query rows of one KV head (its
// group of query heads times the sequence's new tokens) are the 16 columns
// of MFMA 16x16x32 products:
//   scores: A = 16 keys, B = q.  Lane l reads key l % 16 and the quarter
//     l / 16 of its codes, which are contiguous, and expands a word into 8
//     operand values; q was put into that order once.
//   values: A = V^T, B = p s'.  Lane l has, from the score tiles of two
//     neighbouring 16-key halves, the 8 keys 4 (l / 16) + i of both, which
//     are this product's 8 k-slots as they stand; it reads D / 16
//     neighbouring codes of each of these keys, and a v_perm for two keys
//     brings them where two codes of one channel form an operand word.  So
//     the transposition costs one instruction per 8 codes, and neither
//     product goes through LDS.
// Codes enter as OFF + c.  Of the values' sums (OFF + 8) sum(p s') is taken
// off again, from a product with ones, so it has the same rounded p s', and
// 8 s' joins m' in the fp32 sum: what rounding p s' does is then multiplied
// by c' - 8 and not by c' (error of the outputs 2.7 times smaller).
//
// A wave walks 32 keys a step with the next step's loads in flight.  The
// running maximum is only moved when a score passes it by 2^kSlack: p stays
// below 2^kSlack, far inside fp32 and bf16, and the accumulators are hardly
// ever rescaled.  Four waves of a block interleave their steps and join in
// LDS; long axes are cut into chunks whose partial results a second kernel
// joins in chunk order (no atomics: every run gives the same bits).

#include "kv4_common.h"
#include "launch.h"

namespace qlora {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;
constexpr float kSlack = 8.0f;
constexpr float kMid = 8.0f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// The keys of a tile of query rows: [lo, hi), lo a multiple of 32, cut into
// n chunks of `chunk` keys.
struct Span {
  int lo, hi, chunk, n;
  int i0, i1;  // first and last query token of the tile
};
__device__ __forceinline__ Span kv4_span(const Kv4Seq& sq, const Kv4AttnArg& a, int group,
                                         int r0, int tile, int chunk, int splits) {
  Span s;
  const int last = (int)sq.n * group - 1;
  s.i0 = r0 / group;
  s.i1 = min(r0 + tile - 1, last) / group;
  // the table's last key bounds what can be read
  int64_t hi = min(sq.len, a.table_keys), lo = 0;
  if (a.causal) hi = min(hi, sq.pos0 + s.i1 + 1);
  if (a.window > 0) lo = max(lo, sq.pos0 + s.i0 - a.window + 1);
  s.hi = (int)max(hi, (int64_t)0);
  s.lo = (int)(lo & ~(int64_t)(kStep - 1));
  const int keys = max(s.hi - s.lo, 0);
  // a sequence longer than the call was planned for takes larger chunks
  const int need = (keys + splits - 1) / splits;
  s.chunk = max(chunk, (need + kStep - 1) / kStep * kStep);
  s.n = (keys + s.chunk - 1) / s.chunk;
  return s;
}

// A step's codes and pairs of keys and values, in the lane's places.
template <int D>
struct StepData {
  static constexpr int KW = D / 32;                 // words of key codes per half
  static constexpr int VW = D == 64 ? 1 : D / 128;  // words of value codes per key
  uint32_t k[2][KW];
  uint32_t v[2][4][VW];
  u32x4_t kp[2], vp[2];
};
// Where the two halves of a step lie (the same for the wave).
struct StepAt {
  int64_t slot[2];
  bool ok[2];
};
// Lane offsets of a step's loads.
struct LaneOffsets {
  uint32_t k, v, p;
};

__device__ __forceinline__ StepAt locate(const Kv4CacheArg& c, const int32_t* table, int width,
                                         int head, int t, int hi) {
  StepAt a;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int th = t + 16 * h, e = th >> c.page_log2;
    int page = th < hi && e < width ? table[e] : -1;
    a.ok[h] = page >= 0 && page < c.pages;
    page = a.ok[h] ? page : 0;
    a.slot[h] =
        (((int64_t)page * c.kv_heads + head) << c.page_log2) + (th & ((1 << c.page_log2) - 1));
  }
  return a;
}
template <class T>
__device__ __forceinline__ T load_at(const void* base, uint32_t off) {
  return *reinterpret_cast<const T*>(static_cast<const uint8_t*>(base) + off);
}
template <int D>
__device__ __forceinline__ void load_keys(StepData<D>& s, const Kv4CacheArg& c, const StepAt& a,
                                          const LaneOffsets& lo) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* kc = c.k_codes + a.slot[h] * (D / 2);
    if constexpr (D == 64) {
      const u32x2_t w = load_at<u32x2_t>(kc, lo.k);
      s.k[h][0] = w[0];
      s.k[h][1] = w[1];
    } else {
#pragma unroll
      for (int q = 0; q < D / 128; ++q) {
        const u32x4_t w = load_at<u32x4_t>(kc, lo.k + 16u * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) s.k[h][4 * q + i] = w[i];
      }
    }
    s.kp[h] = load_at<u32x4_t>(c.k_pairs + a.slot[h], lo.p);
  }
}
template <int D>
__device__ __forceinline__ void load_values(StepData<D>& s, const Kv4CacheArg& c, const StepAt& a,
                                            const LaneOffsets& lo) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* vc = c.v_codes + a.slot[h] * (D / 2);
    s.vp[h] = load_at<u32x4_t>(c.v_pairs + a.slot[h], lo.p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t off = lo.v + (uint32_t)(i * (D / 2));
      if constexpr (D == 64) {
        s.v[h][i][0] = load_at<uint16_t>(vc, off);
      } else if constexpr (D == 128) {
        s.v[h][i][0] = load_at<uint32_t>(vc, off);
      } else {
        const u32x2_t w = load_at<u32x2_t>(vc, off);
        s.v[h][i][0] = w[0];
        s.v[h][i][1] = w[1];
      }
    }
  }
}

// Sum over the four lanes l % 16 + 16 g of a column.
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

template <class DT, int D, int NT>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 2 : 3) void kv4_attention_kernel(
    Kv4CacheArg c, Kv4BatchArg bt, Kv4AttnArg a, int chunk, int splits, int tiles,
    float* __restrict__ part_o, float* __restrict__ part_ml) {
  constexpr int KC = D / 32;  // score products per half
  constexpr int VC = D / 16;  // value products, and codes per lane and key
  // fp16 keeps what p s' loses in bf16 (whose range it needs) as a second
  // operand; bf16 results are rounded to the operand's precision anyway
  constexpr bool kSplitP = std::is_same_v<DT, F16T>;
  constexpr float kOffK = U4Score<DT>::kOff, kOffV = U4Mfma<Bf16T>::kOff + kMid;
  constexpr int OS = D + 4;
  __shared__ float o_lds[kWaves][16][OS];
  __shared__ float m_lds[kWaves][16 * NT], l_lds[kWaves][16 * NT];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int b = blockIdx.z, head = blockIdx.y;
  const int tile = blockIdx.x / splits, split = blockIdx.x - tile * splits;
  const int group = a.q_heads / c.kv_heads;
  const Kv4Seq sq = kv4_seq(bt, b);
  const int r0 = tile * (16 * NT), rows = (int)(sq.n * group);
  if (r0 >= rows) return;
  const Span sp = kv4_span(sq, a, group, r0, 16 * NT, chunk, splits);
  if (split > 0 && split >= sp.n) return;
  const int t0 = sp.lo + split * sp.chunk, t1 = min(t0 + sp.chunk, sp.hi);

  // this lane's query rows (past the last: the last again, not stored)
  u32x4_t q[NT][KC];
  float qsum[NT];
  int row_lo[NT], row_n[NT];
  const u32x4_t ones = {U4Mfma<DT>::kOne, U4Mfma<DT>::kOne, U4Mfma<DT>::kOne, U4Mfma<DT>::kOne};
  // a negative scale turns the queries' signs, so that the largest product is
  // the largest score
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = min(r0 + 16 * n + lr, rows - 1), i = r / group;
    const uint16_t* p =
        a.q + (sq.row0 + i) * a.q_ts + (int64_t)(head * group + r - i * group) * a.q_hs;
    f32x4_t qs = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      q[n][k] = u4_order8(*reinterpret_cast<const u32x4_t*>(p + lg * (D / 4) + 8 * k)) ^ flip;
      qs = DT::mfma16(ones, q[n][k], qs);
    }
    qsum[n] = qs[0];
    const int64_t pos = sq.pos0 + i;
    const int64_t rhi = max(a.causal ? min(sq.len, pos + 1) : sq.len, (int64_t)0);
    const int64_t rlo = a.window > 0 ? max(pos - a.window + 1, (int64_t)0) : 0;
    row_lo[n] = (int)rlo;
    row_n[n] = (int)max(rhi - rlo, (int64_t)0);
  }
  // keys that every row of the tile sees
  const int all_lo = a.window > 0 ? (int)max(sq.pos0 + sp.i1 - a.window + 1, (int64_t)0) : 0;
  const int all_hi = (int)max(a.causal ? min(sq.len, sq.pos0 + sp.i0 + 1) : sq.len, (int64_t)0);

  f32x4_t o[NT][VC], po[NT];
  float m[NT], mu[NT], l[NT], cs[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int j = 0; j < VC; ++j) o[n][j] = f32x4_t{0, 0, 0, 0};
    po[n] = f32x4_t{0, 0, 0, 0};
    m[n] = -INFINITY;  // running maximum of the products q.k
    mu[n] = 0.0f;      // the same in log2 units, 0 while it is -inf
    l[n] = cs[n] = 0.0f;
  }
  const float c1 = fabsf(a.scale) * kLog2e;
  const float slack = fminf(kSlack / c1, 3e38f);  // any product is within it where the scale is 0
  const LaneOffsets lane_at = {(uint32_t)(lr * (D / 2) + lg * (D / 8)),
                               (uint32_t)(4 * lg * (D / 2) + lr * (D / 32)), 16u * lg};
  const u32x4_t onesv = {U4Mfma<Bf16T>::kOne, U4Mfma<Bf16T>::kOne, U4Mfma<Bf16T>::kOne,
                         U4Mfma<Bf16T>::kOne};
  const int32_t* table = bt.block_table + (int64_t)b * bt.table_width;

  // one step; the next one's keys are asked for once these are used, and its
  // values likewise, so one set of registers serves both
  auto step = [&](StepData<D>& s, const StepAt& at, const StepAt& next, bool more, int t) {
    const bool masked = !(at.ok[0] && at.ok[1]) || t < all_lo || t + kStep > all_hi;
    // scores
    f32x4_t z[NT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int n = 0; n < NT; ++n) z[n][h] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const u32x4_t kk = u4_expand8<U4Score<DT>>(s.k[h][k]);
#pragma unroll
        for (int n = 0; n < NT; ++n) z[n][h] = DT::mfma16(kk, q[n][k], z[n][h]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ks = u4_s(s.kp[h][i]);
        const float km = fmaf(-kOffK, ks, u4_m(s.kp[h][i]));
#pragma unroll
        for (int n = 0; n < NT; ++n) z[n][h][i] = fmaf(ks, z[n][h][i], km * qsum[n]);
      }
    }
    if (more) load_keys<D>(s, c, next, lane_at);
    u32x4_t pb[NT], pl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t vis = 0xFF;
      if (masked) {
        vis = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool v = at.ok[h] &&
                           (uint32_t)(t + 16 * h + 4 * lg + i - row_lo[n]) < (uint32_t)row_n[n];
            z[n][h][i] = v ? z[n][h][i] : -INFINITY;
            vis |= (v ? 1u : 0u) << (4 * h + i);
          }
      }
      float top = fmaxf(fmaxf(fmaxf(z[n][0][0], z[n][0][1]), fmaxf(z[n][0][2], z[n][0][3])),
                        fmaxf(fmaxf(z[n][1][0], z[n][1][1]), fmaxf(z[n][1][2], z[n][1][3])));
      if (__any(top > m[n] + slack)) {
        top = fmaxf(column_max(top), m[n]);
        const float was = m[n] == -INFINITY ? -INFINITY : mu[n];
        m[n] = top;
        mu[n] = top == -INFINITY ? 0.0f : top * c1;
        const float f = exp2f(was - mu[n]);
#pragma unroll
        for (int j = 0; j < VC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][j][i] *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) po[n][i] *= f;
        l[n] *= f;
        cs[n] *= f;
      }
      float ps[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float p = __builtin_amdgcn_exp2f(fmaf(z[n][h][i], c1, -mu[n]));
          float vs = u4_s(s.vp[h][i]), vm = fmaf(kMid, vs, u4_m(s.vp[h][i]));
          if (masked) {  // whatever a hidden key's pair holds is not read
            const bool v = vis >> (4 * h + i) & 1;
            vs = v ? vs : 0.0f;
            vm = v ? vm : 0.0f;
            p = v ? p : 0.0f;  // -inf times a scale of 0
          }
          l[n] += p;
          ps[h][i] = p * vs;
          cs[n] = fmaf(p, vm, cs[n]);
        }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float u0 = ps[w >> 1][2 * (w & 1)], u1 = ps[w >> 1][2 * (w & 1) + 1];
        pb[n][w] = Bf16T::pack2(u0, u1);
        if constexpr (kSplitP)
          pl[n][w] = Bf16T::pack2(u0 - __uint_as_float(pb[n][w] << 16),
                                  u1 - __uint_as_float(pb[n][w] & 0xFFFF0000u));
      }
      po[n] = Bf16T::mfma16(onesv, pb[n], po[n]);
      if constexpr (kSplitP) po[n] = Bf16T::mfma16(onesv, pl[n], po[n]);
    }
    // values: word w of the operand holds keys 2 w, 2 w + 1 of the lane's 8
#pragma unroll
    for (int half = 0; half < VC / 4; ++half) {  // four channels of the lane
      uint32_t x[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t u0 = s.v[w >> 1][2 * (w & 1)][half >> 1],
                       u1 = s.v[w >> 1][2 * (w & 1) + 1][half >> 1];
        x[w] = half & 1 ? perm(u1, u0, 0x07060302u) : perm(u1, u0, 0x05040100u);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4_t vv = {U4Mfma<Bf16T>::pair(x[0], j), U4Mfma<Bf16T>::pair(x[1], j),
                            U4Mfma<Bf16T>::pair(x[2], j), U4Mfma<Bf16T>::pair(x[3], j)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][4 * half + j] = Bf16T::mfma16(vv, pb[n], o[n][4 * half + j]);
          if constexpr (kSplitP) o[n][4 * half + j] = Bf16T::mfma16(vv, pl[n], o[n][4 * half + j]);
        }
      }
    }
    if (more) load_values<D>(s, c, next, lane_at);
  };

  constexpr int kStride = kStep * kWaves;
  int t = t0 + kStep * wave;
  if (t < t1) {
    auto find = [&](int at) { return locate(c, table, bt.table_width, head, at, sp.hi); };
    StepData<D> s;
    StepAt at = find(t);
    load_keys<D>(s, c, at, lane_at);
    load_values<D>(s, c, at, lane_at);
    for (; t < t1; t += kStride) {
      const bool more = t + kStride < t1;
      const StepAt next = find(more ? t + kStride : t);
      step(s, at, next, more, t);
      at = next;
    }
  }

  // join the four waves, their maxima in log2 units
#pragma unroll
  for (int n = 0; n < NT; ++n) m[n] = m[n] == -INFINITY ? m[n] : mu[n];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] = column_sum(l[n]);
    cs[n] = column_sum(cs[n]);
    if (lg == 0) {
      m_lds[wave][16 * n + lr] = m[n];
      l_lds[wave][16 * n + lr] = l[n];
    }
  }
  __syncthreads();
  const bool whole = sp.n <= 1;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, m_lds[w][16 * n + lr]);
    const float f = m[n] == -INFINITY ? 0.0f : exp2f(m[n] - top);
    const float add = fmaf(-kOffV, po[n][0], cs[n]);
    if (n > 0) __syncthreads();  // the last tile's sums have been read
    // lane: channels lg D / 4 + i VC + j of row lr
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < VC; j += 4) {
        f32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (o[n][j + e][i] + add) * f;
        *reinterpret_cast<f32x4_t*>(&o_lds[wave][lr][lg * (D / 4) + i * VC + j]) = v;
      }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * (D / 4); e += 64 * kWaves) {
      const int rr = e / (D / 4), d = 4 * (e - rr * (D / 4)), r = r0 + 16 * n + rr;
      if (r >= rows) continue;
      float mm = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, m_lds[w][16 * n + rr]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float mw = m_lds[w][16 * n + rr];
        // a sum without a maximum is 0, or NaN where every score was
        sum = fmaf(l_lds[w][16 * n + rr], mw == -INFINITY ? 0.0f : exp2f(mw - mm), sum);
      }
      f32x4_t v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4_t*>(&o_lds[w][rr][d]);
      if (whole) {
        const int i = r / group, hq = head * group + r - i * group;
        const int64_t at = (sq.row0 + i) * a.q_heads + hq;
        // no visible key: zeros
        const bool none = mm == -INFINITY && sum == 0.0f;
        v = none ? f32x4_t{0, 0, 0, 0} : v * (1.0f / sum);
        *reinterpret_cast<u32x2_t*>(a.out + at * D + d) =
            u32x2_t{DT::pack2(v[0], v[1]), DT::pack2(v[2], v[3])};
        if (a.lse && d == 0) a.lse[at] = none ? -INFINITY : (mm + log2f(sum)) * kLn2;
      } else {
        const int64_t at =
            ((((int64_t)b * c.kv_heads + head) * tiles + tile) * splits + split) * (16 * NT) +
            16 * n + rr;
        *reinterpret_cast<f32x4_t*>(part_o + at * D + d) = v;
        if (d == 0) {
          part_ml[2 * at] = mm;
          part_ml[2 * at + 1] = sum;
        }
      }
    }
  }
}

// Joins the chunks of the query rows: a row is D / 4 lanes times J shares of
// its chunks, 256 / (D / 4) / J rows a block.
constexpr int kJoinThreads = 256;
template <class DT, int D, int J>
__global__ __launch_bounds__(kJoinThreads) void kv4_join_kernel(
    Kv4CacheArg c, Kv4BatchArg bt, Kv4AttnArg a, int tile_rows, int chunk, int splits, int tiles,
    const float* __restrict__ part_o, const float* __restrict__ part_ml) {
  constexpr int LPV = D / 4, RPB = kJoinThreads / LPV / J;
  __shared__ f32x4_t o_lds[RPB][J][LPV];
  __shared__ float l_lds[RPB][J], m_lds[RPB][J];
  const int b = blockIdx.z, head = blockIdx.y;
  const int group = a.q_heads / c.kv_heads;
  const Kv4Seq sq = kv4_seq(bt, b);
  const int d = threadIdx.x % LPV, j = threadIdx.x / LPV % J, rb = threadIdx.x / LPV / J;
  const int r = blockIdx.x * RPB + rb, rows = (int)(sq.n * group);
  const int tile = r / tile_rows, rr = r - tile * tile_rows;
  f32x4_t v = {0, 0, 0, 0};
  float sum = 0.0f, top = -INFINITY;  // of this share
  bool mine = r < rows;
  if (mine) {
    const Span sp = kv4_span(sq, a, group, tile * tile_rows, tile_rows, chunk, splits);
    mine = sp.n > 1;  // with one chunk it is already written
    if (mine) {
      const int64_t base =
          (((int64_t)b * c.kv_heads + head) * tiles + tile) * splits * tile_rows + rr;
      for (int s = j; s < sp.n; s += J)
        top = fmaxf(top, part_ml[2 * (base + (int64_t)s * tile_rows)]);
      for (int s = j; s < sp.n; s += J) {
        const int64_t at = base + (int64_t)s * tile_rows;
        const float ms = part_ml[2 * at], f = ms == -INFINITY ? 0.0f : exp2f(ms - top);
        sum = fmaf(part_ml[2 * at + 1], f, sum);
        v += *reinterpret_cast<const f32x4_t*>(part_o + at * D + 4 * d) * f;
      }
    }
  }
  if constexpr (J > 1) {
    o_lds[rb][j][d] = v;
    if (d == 0) {
      l_lds[rb][j] = sum;
      m_lds[rb][j] = top;
    }
    __syncthreads();
    if (j > 0) return;
#pragma unroll
    for (int w = 1; w < J; ++w) top = fmaxf(top, m_lds[rb][w]);
    v = f32x4_t{0, 0, 0, 0};
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < J; ++w) {
      const float mw = m_lds[rb][w], f = mw == -INFINITY ? 0.0f : exp2f(mw - top);
      v += o_lds[rb][w][d] * f;
      sum = fmaf(l_lds[rb][w], f, sum);
    }
  }
  if (!mine) return;
  const int i = r / group, hq = head * group + r - i * group;
  const int64_t at = (sq.row0 + i) * a.q_heads + hq;
  const bool none = top == -INFINITY && sum == 0.0f;
  v = none ? f32x4_t{0, 0, 0, 0} : v * (1.0f / sum);
  *reinterpret_cast<u32x2_t*>(a.out + at * D + 4 * d) =
      u32x2_t{DT::pack2(v[0], v[1]), DT::pack2(v[2], v[3])};
  if (a.lse && d == 0) a.lse[at] = none ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <class DT, int D>
void go(const Kv4CacheArg& c, const Kv4BatchArg& b, const Kv4AttnArg& a, const Kv4AttnPlan& p,
        float* ws, hipStream_t s) {
  const int64_t parts = (int64_t)b.seqs * c.kv_heads * p.tiles * p.splits * p.tile;
  float* ml = ws ? ws + parts * D : nullptr;
  const dim3 grid((unsigned)(p.splits * p.tiles), (unsigned)c.kv_heads, (unsigned)b.seqs);
  kv4_attention_kernel<DT, D, 1>
      <<<grid, 64 * kWaves, 0, s>>>(c, b, a, p.chunk, p.splits, p.tiles, ws, ml);
  if (p.splits > 1) {
    const int64_t rows = (int64_t)b.max_q * (a.q_heads / c.kv_heads);
    auto join = [&](auto jc) {
      constexpr int J = decltype(jc)::value, RPB = kJoinThreads / (D / 4) / J;
      const dim3 jgrid((unsigned)((rows + RPB - 1) / RPB), (unsigned)c.kv_heads, (unsigned)b.seqs);
      kv4_join_kernel<DT, D, J><<<jgrid, kJoinThreads, 0, s>>>(c, b, a, p.tile, p.chunk, p.splits,
                                                               p.tiles, ws, ml);
    };
    if (p.splits <= 8)
      join(std::integral_constant<int, 1>{});
    else
      join(std::integral_constant<int, kJoinThreads / (D / 4)>{});
  }
}

}  // namespace

Kv4AttnPlan kv4_attn_plan(int64_t seqs, int64_t max_q, int64_t max_len, int q_heads, int kv_heads,
                          int head_dim, int window) {
  Kv4AttnPlan p;
  p.tile = 16;
  const int64_t rows = max_q * (q_heads / kv_heads);
  p.tiles = (int)((rows + p.tile - 1) / p.tile);
  int64_t keys = max_len;
  // a tile's window starts up to 31 keys early
  if (window > 0 && window + max_q + kStep < keys) keys = window + max_q + kStep;
  const int64_t want = 4096, base = seqs * kv_heads * p.tiles;
  const int64_t per = kStep * kWaves;
  int64_t chunk = (keys * base + want - 1) / want;
  chunk = (chunk + per - 1) / per * per;
  if (chunk < 2 * per) chunk = 2 * per;
  p.splits = (int)((keys + chunk - 1) / chunk);
  if (p.splits < 1) p.splits = 1;
  if (p.splits == 1) chunk = (keys + per - 1) / per * per;
  p.chunk = (int)chunk;
  return p;
}

size_t kv4_attn_workspace(const Kv4AttnPlan& p, int64_t seqs, int kv_heads, int head_dim) {
  if (p.splits <= 1) return 0;
  return (size_t)seqs * kv_heads * p.tiles * p.splits * p.tile * (head_dim + 2) * sizeof(float);
}

hipError_t launch_kv4_attention(const Kv4CacheArg& c, const Kv4BatchArg& b, const Kv4AttnArg& a,
                                const Kv4AttnPlan& p, float* workspace, bool f16, hipStream_t s) {
  auto by_dim = [&](auto dt) {
    using DT = decltype(dt);
    if (c.head_dim == 64)
      go<DT, 64>(c, b, a, p, workspace, s);
    else if (c.head_dim == 128)
      go<DT, 128>(c, b, a, p, workspace, s);
    else
      go<DT, 256>(c, b, a, p, workspace, s);
  };
  if (f16)
    by_dim(F16T{});
  else
    by_dim(Bf16T{});
  return hipGetLastError();
}

}  // namespace qlora
