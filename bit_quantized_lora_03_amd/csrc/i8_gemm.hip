// Products of 8-bit tokens with 8-bit weights for many tokens (i8_linear.hip
// has the formula and the form for few).
//
// Bound by the matrix cores.  A block of four waves has a tile of 128 NI
// weight rows and 32 JT tokens; wave w has 32 NI of the rows against all the
// tokens, NI x JT accumulators of the 32 x 32 x 32 instruction.  With two
// weights (G = 2) accumulator 0 is of the gate's rows and 1 of the same rows of
// the other, so a lane has both sums of an output.  K goes by in tiles of 128
// columns.
//
// Weights come from memory into registers as operands (their tiles are in that
// order, so a load is runs of 512 bytes) and never pass through LDS.  A tile
// of K's operands are loaded two tiles ahead, into the registers that the tile
// before last has left, step by step.  Tokens, which the waves share, reach LDS
// by DMA, in a ring of four stages filled three tiles ahead, so one barrier a
// tile is enough.  A stage's rows are 128 bytes, eight pieces; a piece lies at
// its number ^ (row / 2) % 8, so the 16 rows that a read serves in a cycle lie
// in different banks.

#include "i8_common.h"
#include "launch.h"

namespace qlora {
namespace {

constexpr int KT = 128;     // columns of a tile
constexpr int kStages = 4;  // of the tokens' ring

// Until at most `vm` vector-memory operations of the wave are outstanding, and
// no LDS operation.
constexpr int wait_imm(int vm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4); }

__device__ __forceinline__ i32x16_t mfma32(u32x4_t a, u32x4_t b, i32x16_t c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a),
                                               __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// act(g) u.  Both forms are g / (1 + exp(-z)): z = g, or for gelu's tanh form
// z = 2 sqrt(2 / pi) (g + 0.044715 g^3).
__device__ __forceinline__ float gated(float g, float u, int act) {
  const float z = act == kI8Silu ? g : 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-z)) * u;
}

// The share of K and of the output that a block has.  The first `full` blocks
// have a whole tile each; the tail_q tiles behind them are split tail_s ways
// over K, and their sums go to the workspace.
struct Part {
  int m, n;  // tile
  int tail;  // of the tail's tiles, or -1
  int z, nz;
};
// Neighbouring ranks are on one XCD, whose L2 then holds what they share
// (blocks go to the eight XCDs in turn).
__device__ __forceinline__ uint32_t xcd_rank(uint32_t id, uint32_t total) {
  const uint32_t xcd = id % 8, per = total / 8, extra = total % 8;
  return xcd * per + (xcd < extra ? xcd : extra) + id / 8;
}
// Ranks walk groups of four rows of tiles, a column of the group at a time.
__device__ __forceinline__ void tile_at(uint32_t rank, uint32_t m_tiles, uint32_t n_tiles, int& m,
                                        int& n) {
  const uint32_t span = 4 * n_tiles, g = rank / span, w = rank - g * span;
  const uint32_t gm = min(m_tiles - 4 * g, 4u);
  n = (int)(w / gm);
  m = (int)(4 * g + (w - (uint32_t)n * gm));
}
__device__ __forceinline__ Part part_of(uint32_t id, uint32_t m_tiles, uint32_t n_tiles,
                                        const I8GemmPlan& p) {
  Part o;
  uint32_t rank;
  if (id < (uint32_t)p.full) {
    rank = xcd_rank(id, p.full);
    o.tail = -1;
    o.z = 0;
    o.nz = 1;
  } else {
    const uint32_t r = xcd_rank(id - p.full, p.tail_q * p.tail_s);
    o.z = (int)(r / p.tail_q);
    o.nz = p.tail_s;
    o.tail = (int)(r - o.z * p.tail_q);
    rank = p.full + o.tail;
  }
  tile_at(rank, m_tiles, n_tiles, o.m, o.n);
  return o;
}

struct GemmArg {
  I8LinearArg a;
  I8GemmPlan plan;
  i32x4_t* part;  // [tail_s][tail_q][wave][JT][NI][4][64]
};

// A wave's outputs: RO rows from n0 on of the 32 J tokens from m0 on.  All of
// them are scaled into the wave's LDS first, and go out from there in a loop,
// in runs of a token's row: done for 32 tokens at a time, with a wait between
// each write and read and code for every one, it took 10 us a tile of 256 x
// 256, a tenth of the time at K 8192.
template <class DT, int NI, int G, int J>
struct Outputs {
  static constexpr int RO = G == 2 ? 32 : 32 * NI;
  static constexpr int PR = RO / 8;              // 16-byte pieces of a token
  static constexpr int kBytes = 32 * J * RO * 2;  // of LDS
  // where piece c of a token is: 16 neighbouring tokens' in different banks
  static __device__ int place(int tok, int c) {
    return tok * PR + (c ^ (PR == 8 ? (tok >> 1) & 7 : (tok >> 2) & 3));
  }

  template <class Acc>
  static __device__ void run(const Acc& acc, const I8LinearArg& p, int64_t n0, int64_t m0,
                             uint8_t* lds, int lane) {
    const int lr = lane & 31, lg = lane >> 5;
    f32x4_t sw[NI][4];  // the lane's rows; past N and M: zero
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const auto ws = make_rsrc(p.wscale[G == 2 ? i : 0], (uint32_t)(p.N * 4));
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sw[i][q] = __builtin_bit_cast(
            f32x4_t, buffer_load16(ws, (uint32_t)(n0 + (G == 2 ? 0 : 32 * i) + 8 * q + 4 * lg) * 4));
    }
    float sx[J];
    const auto xs = make_rsrc(p.xscale, (uint32_t)(p.M * 4));
#pragma unroll
    for (int j = 0; j < J; ++j)
      sx[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          xs, (int)((uint32_t)(m0 + 32 * j + lr) * 4), 0, 0));
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < (G == 2 ? 1 : NI); ++i) {
        // (as wholes up to here, or the compiler copies all sums out of the
        // accumulators' registers before the first is used, and spills)
        i32x16_t a = acc[j][i], b = acc[j][G - 1];
        asm volatile("" : "+a"(a));
        if constexpr (G == 2) asm volatile("" : "+a"(b));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = i8_scaled(a[4 * q + e], sw[i][q][e], sx[j]);
            if constexpr (G == 2) v[e] = gated(v[e], i8_scaled(b[4 * q + e], sw[1][q][e], sx[j]), p.act);
          }
          *reinterpret_cast<u32x2_t*>(lds + 16 * place(32 * j + lr, 4 * i + q) + 8 * lg) =
              u32x2_t{DT::pack2(v[0], v[1]), DT::pack2(v[2], v[3])};
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    wave_exchange();
    const int c = lane % PR, t0 = lane / PR;
    uint16_t* y = p.y + (m0 + t0) * p.ldy + n0 + 8 * c;
    const int64_t step = 64 / PR * p.ldy;
    if (((uintptr_t)p.y & 15) == 0 && p.ldy % 8 == 0 && m0 + 32 * J <= p.M && n0 + RO <= p.N) {
#pragma unroll 4
      for (int t = 0; t < J * PR / 2; ++t, y += step)
        *reinterpret_cast<u32x4_t*>(y) =
            *reinterpret_cast<const u32x4_t*>(lds + 16 * place(t0 + 64 / PR * t, c));
    } else {
#pragma nounroll
      for (int t = 0; t < J * PR / 2; ++t, y += step) {
        const u32x4_t v =
            *reinterpret_cast<const u32x4_t*>(lds + 16 * place(t0 + 64 / PR * t, c));
        if (m0 + t0 + 64 / PR * t < p.M)
          store_piece(y, 0, (int)min(p.N - n0 - 8 * c, (int64_t)8), v);
      }
    }
  }
};

template <class DT, int NI, int JT, int G>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, JT == 8 ? 1 : 2)))
void gemm_i8_kernel(GemmArg g) {
  using S = Outputs<DT, NI, G, JT>;
  constexpr int TM = 32 * JT, RO = S::RO, TN = 4 * RO;
  constexpr int XR = JT;               // DMA instructions of a wave a tile
  constexpr int LC = 4 * NI;           // loads of weights a tile
  constexpr int XST = TM * KT;         // bytes of a stage
  constexpr int SLOTS = NI * JT;       // matrix instructions a step
  constexpr int DP = 4 * SLOTS / XR;   // of these from one DMA to the next
  __shared__ __attribute__((aligned(16))) uint8_t lds[kStages * XST > 4 * S::kBytes ? kStages * XST : 4 * S::kBytes];
  const I8LinearArg& p = g.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 31, lg = lane >> 5;
  const int64_t Kp = i8_padded(p.K), n_panels = (p.N + 15) / 16;
  const uint32_t m_tiles = (uint32_t)((p.M + TM - 1) / TM), n_tiles = (uint32_t)((p.N + TN - 1) / TN);
  const Part w = part_of(blockIdx.x, m_tiles, n_tiles, g.plan);
  const int64_t m0 = (int64_t)w.m * TM, n0 = (int64_t)w.n * TN;
  const int nkt = (int)(Kp / KT), pairs = (nkt + 1) / 2;
  const int kt0 = 2 * (int)((uint32_t)(pairs * w.z) / w.nz),
            kt1 = min(nkt, 2 * (int)((uint32_t)(pairs * (w.z + 1)) / w.nz));

  // Operands of a weight: lane l has row l % 32 and 16 columns of a step of
  // 32.  Panels past the end read as zeros (the range check covers the lane's
  // offset, which has the panel; the tile of K is in the scalar one).
  const uint32_t panel = 16 * (uint32_t)Kp;
  const int64_t left = n_panels - n0 / 16;
  const uint32_t held = (uint32_t)min(left, (int64_t)(TN / 16)) * panel;
  const int8_t* const w0 = p.tiles[0] + (n0 / 16) * panel;
  const int8_t* const w1 = p.tiles[G - 1] + (n0 / 16) * panel;
  uint32_t wo[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
    wo[i] = (wave * (RO / 16) + (G == 2 ? 0 : 2 * i) + (lr >> 4)) * panel + lg * 256 + (lr & 15) * 16;
  // Tiles are worked on in pairs; weights of one past the last are zeros (a
  // buffer of no bytes).
  auto load_w = [&](int kt, int i, int kk) -> u32x4_t {
    const auto buf = make_rsrc(G == 2 && i == 1 ? w1 : w0, kt < kt1 ? held : 0);
    return buffer_load16(buf, wo[i] + (kk >> 1) * 1024 + (kk & 1) * 512,
                         (uint32_t)kt * (2 * kI8Tile));
  };
  // Tokens: DMA q of the wave fills the 1 KiB from row 8 (XR wave + q) on,
  // lane l the 16 bytes at 16 l: row l / 8, place l % 8.
  const auto xbuf = make_rsrc(p.codes + m0 * Kp,
                              (uint32_t)min(p.M - m0, (int64_t)TM) * (uint32_t)Kp);
  uint32_t xo[2];
#pragma unroll
  for (int odd = 0; odd < 2; ++odd)
    xo[odd] = (8 * XR * wave + (lane >> 3)) * (uint32_t)Kp +
              16 * ((lane & 7) ^ ((4 * odd + (lane >> 4)) & 7));
  auto dma_x = [&](uint8_t* stage, int kt, int q) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        xbuf, (__attribute__((address_space(3))) void*)(stage + 1024 * (XR * wave + q)), 16,
        xo[(XR * wave + q) & 1] + q * 8 * (uint32_t)Kp, (uint32_t)kt * KT, 0, 0);
  };
  auto read_x = [&](const uint8_t* stage, int kk, int j) -> u32x4_t {
    const int row = 32 * j + lr;
    return *reinterpret_cast<const u32x4_t*>(stage + row * KT +
                                             16 * ((2 * kk + lg) ^ ((row >> 1) & 7)));
  };

  i32x16_t acc[JT][NI];
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[j][i][v] = 0;

  if (kt0 < kt1) {
    const int last = kt1 - 1;
    auto cl = [&](int kt) { return kt < last ? kt : last; };
    u32x4_t W[2][4][NI], X[2][JT];
    // x of the first two tiles, weights of the first, then as in the loop
#pragma unroll
    for (int q = 0; q < XR; ++q) dma_x(lds, kt0, q);
#pragma unroll
    for (int q = 0; q < XR; ++q) dma_x(lds + XST, cl(kt0 + 1), q);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < NI; ++i) W[0][kk][i] = load_w(kt0, i, kk);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < XR; ++q) dma_x(lds + 2 * XST, cl(kt0 + 2), q);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < NI; ++i) W[1][kk][i] = load_w(kt0 + 1, i, kk);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_imm(XR + 2 * LC));
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int j = 0; j < JT; ++j) X[0][j] = read_x(lds, 0, j);

    // A matrix instruction holds the wave's issue only until the matrix core
    // takes it, so each is followed by a share of the other work and a fence.
    // The stages are restrict pointers: the compiler then leaves the DMA in
    // flight across the reads.  Its end is awaited by hand.
    auto iteration = [&](int kt, auto phase, uint8_t* __restrict__ now, uint8_t* __restrict__ next,
                         uint8_t* __restrict__ fill) {
      constexpr int ph = decltype(phase)::value;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          const int j = s / NI, i = s % NI;
          acc[j][i] = mfma32(W[ph][kk][i], X[kk & 1][j], acc[j][i]);
          if (i == NI - 1)
            X[(kk + 1) & 1][j] = kk < 3 ? read_x(now, kk + 1, j) : read_x(next, 0, j);
          const int slot = SLOTS * kk + s;
          if (slot % DP == DP - 1) dma_x(fill, cl(kt + 3), slot / DP);
          // the registers of the step before are free
          if (kk > 0 && s % (SLOTS / NI) == SLOTS / NI / 2 - 1)
            W[ph][kk - 1][s / (SLOTS / NI)] = load_w(kt + 2, s / (SLOTS / NI), kk - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) W[ph][3][i] = load_w(kt + 2, i, 3);
      __builtin_amdgcn_sched_barrier(0);
      // x of tile kt + 2: all that the last iteration asked for but its last
      // weights
      __builtin_amdgcn_s_waitcnt(wait_imm(XR + LC + NI));
      __builtin_amdgcn_s_barrier();
    };
    int stage = 0, kt = kt0;
    auto at = [&](int d) { return lds + ((stage + d) & (kStages - 1)) * XST; };
    for (; kt < kt1; kt += 2, stage += 2) {
      iteration(kt, std::integral_constant<int, 0>(), at(0), at(1), at(3));
      iteration(kt + 1, std::integral_constant<int, 1>(), at(1), at(2), at(4));
    }
    // what was asked for past the end is still on its way to LDS
    __builtin_amdgcn_s_waitcnt(wait_imm(0));
  }
  __syncthreads();
  if (w.tail >= 0) {
    i32x4_t* o = g.part +
                 ((int64_t)(w.z * g.plan.tail_q + w.tail) * 4 + wave) * (JT * NI * 4 * 64) + lane;
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        i32x16_t a = acc[j][i];
        asm volatile("" : "+a"(a));
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[((j * NI + i) * 4 + q) * 64] =
              i32x4_t{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
      }
  } else {
    S::run(acc, p, n0 + wave * RO, m0, lds + wave * S::kBytes, lane);
  }
}

// The tail's sums over its splits: a wave has 32 tokens of a wave's tile.
template <class DT, int NI, int JT, int G>
__global__ __launch_bounds__(256) void join_i8_kernel(GemmArg g) {
  using S = Outputs<DT, NI, G, 1>;
  constexpr int TM = 32 * JT, RO = S::RO, TN = 4 * RO;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * S::kBytes];
  const I8LinearArg& p = g.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t piece = blockIdx.x * 4 + wave;  // [tail][wave][j]
  const int owner = piece / JT % 4, j = piece % JT;
  int m, n;
  tile_at((uint32_t)g.plan.full + piece / (4 * JT), (uint32_t)((p.M + TM - 1) / TM),
          (uint32_t)((p.N + TN - 1) / TN), m, n);
  const int64_t n0 = (int64_t)n * TN + owner * RO, m0 = (int64_t)m * TM + 32 * j;
  if (n0 >= p.N || m0 >= p.M) return;
  const int64_t stride = (int64_t)g.plan.tail_q * 4 * JT * NI * 4 * 64;
  const i32x4_t* src = g.part + (int64_t)piece * (NI * 4 * 64) + lane;
  i32x16_t acc[1][NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[0][i][v] = 0;
  for (int z = 0; z < g.plan.tail_s; ++z, src += stride)
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x4_t v = src[(i * 4 + q) * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][i][4 * q + e] += v[e];
      }
  S::run(acc, p, n0, m0, lds + wave * S::kBytes, lane);
}

template <class DT, int NI, int JT, int G>
void go(const GemmArg& g, hipStream_t s) {
  const int64_t blocks = g.plan.full + (int64_t)g.plan.tail_q * g.plan.tail_s;
  gemm_i8_kernel<DT, NI, JT, G><<<dim3((unsigned)blocks), 256, 0, s>>>(g);
  if (g.plan.tail_q > 0)
    join_i8_kernel<DT, NI, JT, G><<<dim3((unsigned)(g.plan.tail_q * JT)), 256, 0, s>>>(g);
}

template <class DT, int G>
void pick(const GemmArg& g, hipStream_t s) {
  const I8GemmPlan& p = g.plan;
  if (G == 2 || p.tn == 256) {
    if (p.tm == 256) return go<DT, 2, 8, G>(g, s);
    if (p.tm == 128) return go<DT, 2, 4, G>(g, s);
    return go<DT, 2, 2, G>(g, s);
  }
  if constexpr (G == 1) {
    if (p.tm == 128) return go<DT, 1, 4, G>(g, s);
    return go<DT, 1, 2, G>(g, s);
  }
}

}  // namespace

I8GemmPlan gemm_i8_plan(int64_t M, int64_t N, int64_t K, bool gated) {
  const int64_t nkt = i8_padded(K) / KT;
  I8GemmPlan best{};
  double best_t = 1e300;
  for (int tm = 256; tm >= 128; tm /= 2) {
    const int tn = gated ? 128 : 256;
    const int64_t tiles = ((M + tm - 1) / tm) * ((N + tn - 1) / tn);
    const double tile_t = (tm == 256 ? 1.0 : 0.6) * nkt;
    I8GemmPlan p{tm, tn, (int)tiles, 0, 1};
    const int64_t q = tiles % 256;
    double t = (double)((tiles + 255) / 256) * tile_t;
    if (q > 0) {
      int64_t s = 256 / q;
      if (s > nkt / 2) s = nkt / 2;
      if (s > 16) s = 16;
      if (s >= 2) {
        p.full = (int)(tiles - q);
        p.tail_q = (int)q;
        p.tail_s = (int)s;
        t = ((double)(tiles / 256) + 1.0 / s) * tile_t + 4 + (double)(s * q * tm) / 16384;
      }
    }
    if (t < best_t) {
      best_t = t;
      best = p;
    }
  }
  return best;
}

size_t gemm_i8_workspace(const I8GemmPlan& p, bool gated) {
  return (size_t)p.tail_q * (p.tail_q ? p.tail_s : 0) * p.tm * p.tn * (gated ? 2 : 1) * 4;
}

hipError_t launch_gemm_i8(const I8LinearArg& p, const I8GemmPlan& plan, int32_t* workspace,
                          bool f16, hipStream_t s) {
  const GemmArg g{p, plan, reinterpret_cast<i32x4_t*>(workspace)};
  if (p.tiles[1]) {
    if (f16)
      pick<F16T, 2>(g, s);
    else
      pick<Bf16T, 2>(g, s);
  } else {
    if (f16)
      pick<F16T, 1>(g, s);
    else
      pick<Bf16T, 1>(g, s);
  }
  return hipGetLastError();
}

}  // namespace qlora
