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
//   scores: A = 16 keys, B = q.  Lane l has key l % 16 and the quarter l / 16
//     of its codes, and expands a word into 8 operand values; q was put into
//     that order once.
//   values: A = V^T, B = p s'.  Lane l has, from the score tiles of two
//     neighbouring 16-key halves, the 8 keys 4 (l / 16) + i of both, which
//     are this product's 8 k-slots as they stand; it takes D / 16
//     neighbouring codes of each of these keys, and a v_perm for two keys
//     brings them where two codes of one channel form an operand word, so the
//     transposition costs one instruction per 8 codes.
// Codes enter as OFF + c.  Of the values' sums (OFF + 8) sum(p s') is taken
// off again, from a product with ones, so it has the same rounded p s', and
// 8 s' joins m' in the fp32 sum: what rounding p s' does is then multiplied
// by c' - 8 and not by c'.
// p s' is an fp16 operand (half a step is 2^-11): as a bf16 one (2^-8) it took
// bf16 outputs 2.4e-3 from the 64-bit result; now they are 1.7e-3 off, as the
// exact result rounded is (64 ragged sequences 103 us with either, many rows 3
// to 6 % slower).  fp16 outputs take a second operand for what the first loses
// (2^-22).  fp16's range is narrow, so M follows the row's largest p s' and
// not its largest p (kUp below): what is small in fp16 is small beside the
// largest share of the result, whatever the steps are.
//
// A wave walks 32 keys a step.  Keys, values and pairs come to its own LDS by
// DMA two steps ahead (one at D = 256): a step's 4.3 KiB (D 128) in 8
// instructions and no registers.  M is a whole number that is only moved when
// some p s' passes 2^kMost, then far enough for it to grow 2^8 times, so the
// accumulators are hardly ever rescaled, and exactly.  Four waves of a block
// interleave their steps and join in LDS; long axes are cut into chunks whose
// partial results a second kernel joins in chunk order (no atomics: every run
// gives the same bits).
//
// Measured (calls from Python that follow each other; in brackets a copy of
// the same bytes): 64 ragged sequences up to 8192 keys, 32 heads on 8, D 128,
// bf16: 98 us (80), the join 5 of it; 2 x 131071 keys, 64 heads on 8, fp16: 65
// (48), the join 7; one sequence of 777, 16 heads, D 64: 9.6 in a replayed
// graph, two launches and their first loads.  A step's 290 vector instructions
// (130 for expanding the codes) keep the vector units busy for half of the
// time at 64 sequences; what is left is the start of a block, four dependent
// loads long, and the ragged ends.  Many rows: 3 x 251 rows of 16 heads on 4, D
// 256, window 4096: 101 us, 0.38 PFLOP/s; 440 vector instructions for 33 MFMAs
// a step, which take 83 % of the time while a SIMD has its two waves and 53 %
// of all of it, for 756 blocks are one and a half rounds.

#include <algorithm>

#include "kv4_common.h"
#include "launch.h"

namespace qlora {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = kKv4Step;
constexpr float kMid = 8.0f;
// M is the row's largest z log2 e + log2 s', rounded up, less kUp: its largest
// p s' is 2^kUp, 2^20 times the smallest normal fp16 number, and moves M again
// when it would pass 2^kMost, inside fp16.  With small steps M stays at the
// largest z log2 e less kUnder, so that sums of p stay inside fp32.
constexpr float kUp = 6.0f, kMost = 14.0f, kUnder = 40.0f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// A wave's LDS: a ring of stages, each with one step's keys, values (32 rows
// of D / 2 bytes) and their pairs (16 words each: keys of both halves, values
// of both).  The 16-byte pieces of a row are exchanged so that neither the
// 16 rows of a key operand nor the 4 keys of a value read share banks.
template <int D>
struct Ring {
  static constexpr int kCodes = 16 * D, kStage = 2 * kCodes + 256;
  static constexpr int kPieces = D / 32, kRowsPerBanks = 512 / D;
  static constexpr int kHalfLoads = D == 256 ? 2 : 1;  // DMA instructions for a half's keys
  static constexpr int kAll = 4 * kHalfLoads + 4;      // ... and for a step
  // Two stages in flight beside the one in use; at D = 256 one, so that two
  // blocks fit a CU.
  static constexpr int kStages = D == 256 ? 2 : 3;
  static __device__ __forceinline__ uint32_t place(uint32_t row, uint32_t piece) {
    return row * (D / 2) + ((piece ^ (row / kRowsPerBanks)) & (kPieces - 1)) * 16;
  }
};
// The pages of a step's two halves as the block table has them (-1: none).
// The table is read through the constant address space: by scalar loads.
typedef const __attribute__((address_space(4))) int32_t* TablePtr;
struct StepPages {
  int page[2];
};
__device__ __forceinline__ StepPages look_up(const Kv4CacheArg& c, TablePtr table, int width,
                                             int t, int hi) {
  StepPages p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int th = t + 16 * h, e = th >> c.page_log2;
    p.page[h] = th < hi && e < width ? table[e] : -1;
  }
  return p;
}
// Which halves have a page, as bits.
__device__ __forceinline__ uint32_t there(const Kv4CacheArg& c, const StepPages& p) {
  const uint32_t pages = (uint32_t)c.pages;
  return ((uint32_t)p.page[0] < pages ? 1u : 0u) | ((uint32_t)p.page[1] < pages ? 2u : 0u);
}

// 16 (4) bytes a lane from a buffer straight to LDS, lane after lane.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t from, uint32_t off, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16,
                                           off, 0, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t from, uint32_t off, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 4,
                                           off, 0, 0, 0);
}
// s_waitcnt immediate: at most `vm` vector-memory operations outstanding.
constexpr int wait_vm(int vm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (15 << 8); }

// One step's keys, values and pairs into a stage, straight to LDS: lane l of
// a load brings its 16 bytes l (4 of the pairs).  Each half's 16 rows are a
// buffer of their own.  A half without a page brings page 0's.
template <int D>
__device__ __forceinline__ void fetch(const Kv4CacheArg& c, const StepPages& p, uint32_t have,
                                      int head, int t, uint8_t* to, int lane) {
  using R = Ring<D>;
  // the lane's piece of a KiB (or of the half's 512 bytes at D = 64)
  uint32_t off[R::kHalfLoads];
#pragma unroll
  for (int i = 0; i < R::kHalfLoads; ++i) {
    const uint32_t row = (1024u * i + 16u * lane) / (D / 2);
    const uint32_t piece = (lane ^ row / R::kRowsPerBanks) & (R::kPieces - 1);
    off[i] = row * (D / 2) + piece * 16;
  }
  constexpr int kHalf = 8 * D;  // bytes of a half's codes
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int page = have >> h & 1 ? p.page[h] : 0;
    const int64_t slot = (((int64_t)page * c.kv_heads + head) << c.page_log2) +
                         ((t + 16 * h) & ((1 << c.page_log2) - 1));
    const __amdgpu_buffer_rsrc_t kc = make_rsrc(c.k_codes + slot * (D / 2), kHalf);
    const __amdgpu_buffer_rsrc_t vc = make_rsrc(c.v_codes + slot * (D / 2), kHalf);
    const __amdgpu_buffer_rsrc_t kp = make_rsrc(c.k_pairs + slot, 64);
    const __amdgpu_buffer_rsrc_t vp = make_rsrc(c.v_pairs + slot, 64);
    if (D > 64 || lane < 32) {
#pragma unroll
      for (int i = 0; i < R::kHalfLoads; ++i) {
        dma16(kc, off[i], to + h * kHalf + 1024 * i);
        dma16(vc, off[i], to + R::kCodes + h * kHalf + 1024 * i);
      }
    }
    if (lane < 16) {
      dma4(kp, 4 * lane, to + 2 * R::kCodes + 64 * h);
      dma4(vp, 4 * lane, to + 2 * R::kCodes + 128 + 64 * h);
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

// ln(2^m sum); the sum's exponent is added to m as it is, so that what p was
// counted from costs no bits.
__device__ __forceinline__ float log_sum(float m, float sum) {
  int e;
  const float f = frexpf(sum, &e);
  return (m + (float)e + log2f(f)) * kLn2;
}

template <class DT, int D, int NT>
__global__ __launch_bounds__(64 * kWaves, D * NT >= 256 ? 2 : 3) void kv4_attention_kernel(
    Kv4CacheArg c, Kv4BatchArg bt, Kv4AttnArg a, int chunk, int splits, int tiles,
    float* __restrict__ part_o, float* __restrict__ part_ml) {
  constexpr int KC = D / 32;  // score products per half
  constexpr int VC = D / 16;  // value products, and codes per lane and key
  constexpr int VW = D == 64 ? 1 : D / 128;  // words of these
  // what an fp16 operand loses of p s' is a second one for fp16 results; bf16
  // results are rounded to an eighth of its precision
  constexpr bool kSplitP = std::is_same_v<DT, F16T>;
  constexpr float kOffK = U4Score<DT>::kOff, kOffV = U4Value::kOff + kMid;
  constexpr int OS = D + 4;
  using R = Ring<D>;
  // the rings, and after the walk the place of the waves' sums
  union Shared {
    uint8_t ring[kWaves][R::kStages * R::kStage];
    float o[kWaves][16][OS];
  };
  __shared__ __attribute__((aligned(16))) Shared lds;
  __shared__ float m_lds[kWaves][16 * NT], l_lds[kWaves][16 * NT];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int b = blockIdx.z, head = blockIdx.y;
  // Neighbouring blocks go to the eight XCDs in turn, and late chunks have less
  // to do or nothing; so which block has which chunk turns from one tile, head
  // and sequence to the next.  (With an even number of chunks: 48 ragged
  // sequences up to 8000 keys, four chunks: 71 us, 81 without; 4 x 251 rows of
  // D 256 in two: 147 and 192.)
  const int tile = blockIdx.x / splits;
  const int split = (blockIdx.x + tile + head + b) % splits;
  const int group = a.q_heads / c.kv_heads;
  const Kv4Seq sq = kv4_seq(bt, b);
  const int r0 = tile * (16 * NT), rows = (int)(sq.n * group);
  if (r0 >= rows) return;
  const Span sp = kv4_span(sq, a, group, r0, 16 * NT, chunk, splits);
  if (split > 0 && split >= sp.n) return;
  const int t0 = sp.begin(split), t1 = sp.end(split);

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
  float gate[NT], mu[NT], l[NT], cs[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int j = 0; j < VC; ++j) o[n][j] = f32x4_t{0, 0, 0, 0};
    po[n] = f32x4_t{0, 0, 0, 0};
    mu[n] = 0.0f;         // M, 0 while nothing has been seen
    gate[n] = -INFINITY;  // M + kMost, -inf while nothing has been seen
    l[n] = cs[n] = 0.0f;
  }
  // never 0, which would make a hidden score, -inf, NaN; 2^-100 is as good
  const float c1 = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f);
  // where the lane reads its part of a stage
  uint32_t koff[D == 256 ? 2 : 1], voff[4];
  if constexpr (D == 64) {
    koff[0] = R::place(lr, lg >> 1) + 8 * (lg & 1);
  } else {
#pragma unroll
    for (int e = 0; e < D / 128; ++e) koff[e] = R::place(lr, lg * (D / 128) + e);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    voff[i] = R::kCodes + R::place(4 * lg + i, lr * (D / 32) / 16) + lr * (D / 32) % 16;
  const u32x4_t onesv = {U4Value::kOne, U4Value::kOne, U4Value::kOne, U4Value::kOne};
  const TablePtr table = (TablePtr)(bt.block_table + (int64_t)b * bt.table_width);

  // one step on the stage at s; have: which of its halves have a page
  auto step = [&](const uint8_t* s, uint32_t have, int t) __attribute__((always_inline)) {
    // some row of the tile does not see some key of the step
    const bool masked = have != 3 || t < all_lo || t + kStep > all_hi;
    // scores
    f32x4_t z[NT][2];
    const auto* pairs = reinterpret_cast<const u32x4_t*>(s + 2 * R::kCodes) + lg;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t kw[KC];
      if constexpr (D == 64) {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(s + koff[0] + h * (8 * D));
        kw[0] = w[0];
        kw[1] = w[1];
      } else {
#pragma unroll
        for (int e = 0; e < D / 128; ++e) {
          const u32x4_t w = *reinterpret_cast<const u32x4_t*>(s + koff[e] + h * (8 * D));
#pragma unroll
          for (int i = 0; i < 4; ++i) kw[4 * e + i] = w[i];
        }
      }
      const u32x4_t kp = pairs[4 * h];
#pragma unroll
      for (int n = 0; n < NT; ++n) z[n][h] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const u32x4_t kk = u4_expand8<U4Score<DT>>(kw[k]);
#pragma unroll
        for (int n = 0; n < NT; ++n) z[n][h] = DT::mfma16(kk, q[n][k], z[n][h]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ks = u4_s(kp[i]), km = fmaf(-kOffK, ks, u4_m(kp[i]));
#pragma unroll
        for (int n = 0; n < NT; ++n) z[n][h][i] = fmaf(ks, z[n][h][i], km * qsum[n]);
      }
    }
    const u32x4_t vp0[2] = {pairs[8], pairs[12]};
    u32x4_t pb[NT], pl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      u32x4_t vp[2] = {vp0[0], vp0[1]};
      if (masked) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool v = (have >> h & 1) &&
                           (uint32_t)(t + 16 * h + 4 * lg + i - row_lo[n]) < (uint32_t)row_n[n];
            z[n][h][i] = v ? z[n][h][i] : -INFINITY;
            vp[h][i] = v ? vp[h][i] : 0;  // whatever a hidden key's pair holds
          }
      }
      float top = fmaxf(fmaxf(fmaxf(z[n][0][0], z[n][0][1]), fmaxf(z[n][0][2], z[n][0][3])),
                        fmaxf(fmaxf(z[n][1][0], z[n][1][1]), fmaxf(z[n][1][2], z[n][1][3])));
      float vs[2][4], most = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vs[h][i] = u4_s(vp[h][i]);
          most = fmaxf(most, fabsf(vs[h][i]));
        }
      // the lane's largest p and s' bound its products
      if (__any(fmaf(top, c1, fmaxf(__builtin_amdgcn_logf(most), kMost - kUnder)) > gate[n])) {
        float r = -INFINITY;  // the largest z log2 e + log2 s'
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            r = fmaxf(r, fmaf(z[n][h][i], c1, __builtin_amdgcn_logf(fabsf(vs[h][i]))));
        r = column_max(r);
        top = column_max(top) * c1;
        // a row that has seen nothing stays so, and one whose products do not
        // pass has its M
        const bool move = fmaxf(r, top + (kMost - kUnder)) > gate[n];
        const float to = fmaxf(ceilf(r) - kUp, ceilf(top) - kUnder);
        const float f = !move                  ? 1.0f
                        : gate[n] == -INFINITY ? 0.0f
                                               : exp2f(mu[n] - to);
        mu[n] = move ? to : mu[n];
        gate[n] = move ? to + kMost : gate[n];
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
          const float p = __builtin_amdgcn_exp2f(fmaf(z[n][h][i], c1, -mu[n]));
          l[n] += p;
          ps[h][i] = p * vs[h][i];
          cs[n] = fmaf(p, fmaf(kMid, vs[h][i], u4_m(vp[h][i])), cs[n]);
        }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float u0 = ps[w >> 1][2 * (w & 1)], u1 = ps[w >> 1][2 * (w & 1) + 1];
        pb[n][w] = F16T::pack2(u0, u1);
        if constexpr (kSplitP)
          pl[n][w] = F16T::pack2(u0 - F16T::tof((uint16_t)pb[n][w]),
                                 u1 - F16T::tof((uint16_t)(pb[n][w] >> 16)));
      }
      po[n] = F16T::mfma16(onesv, pb[n], po[n]);
      if constexpr (kSplitP) po[n] = F16T::mfma16(onesv, pl[n], po[n]);
    }
    // values: word w of the operand holds keys 2 w, 2 w + 1 of the lane's 8
    uint32_t vw[2][4][VW];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = s + voff[i] + h * (8 * D);
        if constexpr (D == 64) {
          vw[h][i][0] = *reinterpret_cast<const uint16_t*>(p);
        } else if constexpr (D == 128) {
          vw[h][i][0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
          const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
          vw[h][i][0] = w[0];
          vw[h][i][1] = w[1];
        }
      }
#pragma unroll
    for (int half = 0; half < VC / 4; ++half) {  // four channels of the lane
      uint32_t x[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t u0 = vw[w >> 1][2 * (w & 1)][half >> 1],
                       u1 = vw[w >> 1][2 * (w & 1) + 1][half >> 1];
        x[w] = half & 1 ? perm(u1, u0, 0x07060302u) : perm(u1, u0, 0x05040100u);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4_t vv = {U4Value::pair(x[0], j), U4Value::pair(x[1], j),
                            U4Value::pair(x[2], j), U4Value::pair(x[3], j)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][4 * half + j] = F16T::mfma16(vv, pb[n], o[n][4 * half + j]);
          if constexpr (kSplitP) o[n][4 * half + j] = F16T::mfma16(vv, pl[n], o[n][4 * half + j]);
        }
      }
    }
  };

  constexpr int kStride = kStep * kWaves;
  const int first = t0 + kStep * wave;
  if (first < t1) {
    // One iteration: asks for the stage kAhead steps ahead, waits until this
    // step's stage is there (loads return in order, so the number that may be
    // outstanding says so) and works on it.  The stage read and the one being
    // filled are distinct, which the restrict pointers say: the compiler
    // leaves the DMA in flight across the reads.  The stage that is filled was
    // read in the iteration before, whose reads have returned.  The walk
    // starts kAhead steps early, without work, so that there is one place
    // that asks: a second would not be known to be distinct.
    constexpr int kAhead = R::kStages - 1;
    auto pages_of = [&](int at) { return look_up(c, table, bt.table_width, at, sp.hi); };
    StepPages pg = pages_of(first);
    uint32_t have = 0;  // two bits for each step that is in flight, this one's lowest
    auto iteration = [&](const uint8_t* __restrict__ rd, uint8_t* __restrict__ fill, int t)
                         __attribute__((always_inline)) {
      const int at = t + kAhead * kStride;
      if (at < t1) {
        const uint32_t h = there(c, pg);
        have |= h << (2 * kAhead);
        fetch<D>(c, pg, h, head, at, fill, lane);
        pg = pages_of(at + kStride);  // for the next time
        __builtin_amdgcn_s_waitcnt(wait_vm(kAhead * R::kAll));
      } else if (kAhead == 2 && t + kStride < t1) {
        __builtin_amdgcn_s_waitcnt(wait_vm(R::kAll));
      } else {
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
      }
      __builtin_amdgcn_sched_barrier(0);
      if (t >= first) step(rd, have & 3, t);
      __builtin_amdgcn_sched_barrier(0);
      have >>= 2;
    };
    uint8_t *const S0 = lds.ring[wave], *const S1 = S0 + R::kStage,
            *const S2 = S0 + kAhead * R::kStage;
    // a copy for each place in the ring: with the stages at constant offsets
    // the compiler knows the age of the DMA that a read has to wait for
    int t = first - kAhead * kStride;
    for (;;) {
      iteration(S1, S0, t);
      if ((t += kStride) >= t1) break;
      if constexpr (R::kStages == 3) {
        iteration(S2, S1, t);
        if ((t += kStride) >= t1) break;
      }
      iteration(S0, S2, t);
      if ((t += kStride) >= t1) break;
    }
  }

  // join the four waves
  float m[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) m[n] = gate[n] == -INFINITY ? -INFINITY : mu[n];
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
        *reinterpret_cast<f32x4_t*>(&lds.o[wave][lr][lg * (D / 4) + i * VC + j]) = v;
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
      for (int w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4_t*>(&lds.o[w][rr][d]);
      if (whole) {
        const int i = r / group, hq = head * group + r - i * group;
        const int64_t at = (sq.row0 + i) * a.q_heads + hq;
        // no visible key: zeros
        const bool none = mm == -INFINITY && sum == 0.0f;
        v = none ? f32x4_t{0, 0, 0, 0} : v * (1.0f / sum);
        *reinterpret_cast<u32x2_t*>(a.out + at * D + d) =
            u32x2_t{DT::pack2(v[0], v[1]), DT::pack2(v[2], v[3])};
        if (a.lse && d == 0) a.lse[at] = none ? -INFINITY : log_sum(mm, sum);
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
#pragma unroll 4
      for (int s = j; s < sp.n; s += J)
        top = fmaxf(top, part_ml[2 * (base + (int64_t)s * tile_rows)]);
#pragma unroll 4
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
  if (a.lse && d == 0) a.lse[at] = none ? -INFINITY : log_sum(top, sum);
}

template <class DT, int D>
void go(const Kv4CacheArg& c, const Kv4BatchArg& b, const Kv4AttnArg& a, const Kv4AttnPlan& p,
        float* ws, hipStream_t s) {
  const int64_t parts = (int64_t)b.seqs * c.kv_heads * p.tiles * p.splits * p.tile;
  float* ml = ws ? ws + parts * D : nullptr;
  const dim3 grid((unsigned)(p.splits * p.tiles), (unsigned)c.kv_heads, (unsigned)b.seqs);
  auto walk = [&](auto nt) {
    kv4_attention_kernel<DT, D, decltype(nt)::value>
        <<<grid, 64 * kWaves, 0, s>>>(c, b, a, p.chunk, p.splits, p.tiles, ws, ml);
  };
  if (p.tile == 16) walk(std::integral_constant<int, 1>{});
  if constexpr (D == 128)
    if (p.tile == 32) walk(std::integral_constant<int, 2>{});
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
  const int64_t rows = max_q * (q_heads / kv_heads);
  // Two column tiles share a step's decoding where there are rows for them
  // (2 x 1000 rows of 32 heads on 8, D 128: 123 us against 144; at 20 rows, of
  // which the second tile has 4, 52 against 47; at D = 64, where decoding is
  // less of the work, 80 against 60, and D = 256 lacks the registers).
  p.tile = head_dim == 128 && rows >= 64 ? 32 : 16;
  p.tiles = (int)((rows + p.tile - 1) / p.tile);
  int64_t keys = max_len;
  // a tile's window starts up to 31 keys early
  if (window > 0 && window + max_q + kStep < keys) keys = window + max_q + kStep;
  // As many chunks as make 1536 blocks, so that the short sequences of a
  // ragged batch do not leave the chip idle, of at least two steps for each
  // wave: 64 ragged sequences up to 8192, 8 heads: 101 us, with 768 blocks
  // wanted 109, with 3840 117.  Full tiles of rows, whose partial results are
  // more of the work, as make 768: 3 x 251 rows, window 4096, D 256: 106 us
  // with one chunk, 126 with two; 700 rows on 8000 keys, D 128: 200 and 207.
  // Both are what measured best and not whole rounds: a CU has room for five
  // blocks at D 64, three at D 128 and two at D 256 and with two column tiles.
  // The number of chunks is rounded to the nearest: a last chunk of few keys
  // costs all the partial results (3 x 500 rows, 1512 blocks: 205 us with a
  // second chunk, 126 without).  Every sequence is taken to have max_q rows:
  // beside one long prompt the others' keys are not cut.
  const int64_t want = rows >= 64 ? 768 : 1536;
  constexpr int64_t kPer = kStep * kWaves;
  const int64_t base = std::max<int64_t>(seqs * kv_heads * p.tiles, 1);
  const int64_t n = std::max<int64_t>((want + base / 2) / base, 1);
  int64_t chunk = (keys + n - 1) / n;
  chunk = (chunk + kPer - 1) / kPer * kPer;
  if (chunk < 2 * kPer) chunk = 2 * kPer;
  p.splits = chunk >= keys ? 1 : (int)((keys + chunk - 1) / chunk);
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
