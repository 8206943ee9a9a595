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

// A wave's outputs of 32 tokens: RO rows from n0 on of the tokens from m0 on.
// Through the wave's LDS, so that stores are runs of a token's row.
template <class DT, int NI, int G>
struct Slice {
  static constexpr int RO = G == 2 ? 32 : 32 * NI;
  static constexpr int LD = RO * 2 + 16;  // bytes of a token in LDS
  static constexpr int kBytes = 32 * LD;
  f32x4_t sw[NI][4];  // the lane's rows
  __amdgpu_buffer_rsrc_t xs;

  __device__ void scales(const I8LinearArg& p, int64_t n0, int lane) {
    xs = make_rsrc(p.xscale, (uint32_t)(p.M * 4));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const auto ws = make_rsrc(p.wscale[G == 2 ? i : 0], (uint32_t)(p.N * 4));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + (G == 2 ? 0 : 32 * i) + 8 * q + 4 * (lane >> 5);
        // past N: zero
        sw[i][q] = __builtin_bit_cast(f32x4_t, buffer_load16(ws, (uint32_t)(n * 4)));
      }
    }
  }
  __device__ void store(const i32x16_t (&acc)[NI], const I8LinearArg& p, int64_t n0, int64_t m0,
                        uint8_t* lds, int lane) {
    const int lr = lane & 31, lg = lane >> 5;
    const float sx = __uint_as_float(
        __builtin_amdgcn_raw_buffer_load_b32(xs, (int)((m0 + lr) * 4), 0, 0));
#pragma unroll
    for (int i = 0; i < (G == 2 ? 1 : NI); ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = i8_scaled(acc[i][4 * q + j], sw[i][q][j], sx);
          if constexpr (G == 2)
            v[j] = gated(v[j], i8_scaled(acc[1][4 * q + j], sw[1][q][j], sx), p.act);
        }
        *reinterpret_cast<u32x2_t*>(lds + lr * LD + (32 * i + 8 * q + 4 * lg) * 2) =
            u32x2_t{DT::pack2(v[0], v[1]), DT::pack2(v[2], v[3])};
      }
    wave_exchange();
    constexpr int PR = RO / 8;  // 16-byte pieces of a token
    const bool whole = ((uintptr_t)p.y & 15) == 0 && p.ldy % 8 == 0;
#pragma unroll
    for (int t = 0; t < 32 * PR / 64; ++t) {
      const int tok = (64 * t + lane) / PR, c = lane % PR;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(lds + tok * LD + 16 * c);
      const int64_t m = m0 + tok, n = n0 + 8 * c;
      if (m < p.M && n < p.N) {
        uint16_t* y = p.y + m * p.ldy + n;
        if (whole && n + 8 <= p.N) {
          *reinterpret_cast<u32x4_t*>(y) = v;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (n + j < p.N) y[j] = (uint16_t)half_of(v, j);
        }
      }
    }
    wave_exchange();
  }
};

template <class DT, int NI, int JT, int G>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_i8_kernel(GemmArg g) {
  using S = Slice<DT, NI, G>;
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
  const int nkt = (int)(Kp / KT);
  const int kt0 = (int)((uint32_t)(nkt * w.z) / w.nz), kt1 = (int)((uint32_t)(nkt * (w.z + 1)) / w.nz);

  // Operands of a weight: lane l has row l % 32 and 16 columns of a step of
  // 32.  Panels past the end read as zeros (the range check covers the lane's
  // offset, which has the panel; the tile of K is in the scalar one).
  const uint32_t panel = 16 * (uint32_t)Kp;
  const int64_t left = n_panels - n0 / 16;
  const uint32_t held = (uint32_t)min(left, (int64_t)(TN / 16)) * panel;
  const auto wbuf0 = make_rsrc(p.tiles[0] + (n0 / 16) * panel, held);
  const auto wbuf1 = make_rsrc(p.tiles[G - 1] + (n0 / 16) * panel, held);
  uint32_t wo[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
    wo[i] = (wave * (RO / 16) + (G == 2 ? 0 : 2 * i) + (lr >> 4)) * panel + lg * 256 + (lr & 15) * 16;
  auto load_w = [&](int kt, int i, int kk) -> u32x4_t {
    return buffer_load16(G == 2 && i == 1 ? wbuf1 : wbuf0, wo[i] + (kk >> 1) * 1024 + (kk & 1) * 512,
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
      for (int i = 0; i < NI; ++i) W[1][kk][i] = load_w(cl(kt0 + 1), i, kk);
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
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < NI; ++i) W[ph][kk][i] = load_w(cl(kt + 2), i, kk);
      __builtin_amdgcn_sched_barrier(0);
      // x of tile kt + 2, which the last iteration asked for before its weights
      __builtin_amdgcn_s_waitcnt(wait_imm(XR + 2 * LC));
      __builtin_amdgcn_s_barrier();
    };
    int stage = 0, kt = kt0;
    auto at = [&](int d) { return lds + ((stage + d) & (kStages - 1)) * XST; };
    for (; kt + 2 <= kt1; kt += 2, stage += 2) {
      iteration(kt, std::integral_constant<int, 0>(), at(0), at(1), at(3));
      iteration(kt + 1, std::integral_constant<int, 1>(), at(1), at(2), at(4));
    }
    if (kt < kt1) iteration(kt, std::integral_constant<int, 0>(), at(0), at(1), at(3));
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
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[((j * NI + i) * 4 + q) * 64] = i32x4_t{acc[j][i][4 * q], acc[j][i][4 * q + 1],
                                                   acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
  } else {
    S out;
    out.scales(p, n0 + wave * RO, lane);
    uint8_t* scratch = lds + wave * S::kBytes;
#pragma unroll
    for (int j = 0; j < JT; ++j) out.store(acc[j], p, n0 + wave * RO, m0 + 32 * j, scratch, lane);
  }
}

// The tail's sums over its splits: a wave has 32 tokens of a wave's tile.
template <class DT, int NI, int JT, int G>
__global__ __launch_bounds__(256) void join_i8_kernel(GemmArg g) {
  using S = Slice<DT, NI, G>;
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
  S out;
  out.scales(p, n0, lane);
  const int64_t stride = (int64_t)g.plan.tail_q * 4 * JT * NI * 4 * 64;
  const i32x4_t* src = g.part + (int64_t)piece * (NI * 4 * 64) + lane;
  i32x16_t acc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[i][v] = 0;
  for (int z = 0; z < g.plan.tail_s; ++z, src += stride)
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x4_t v = src[(i * 4 + q) * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][4 * q + e] += v[e];
      }
  out.store(acc, p, n0, m0, lds + wave * S::kBytes, lane);
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
  if (g.plan.tm == 256)
    go<DT, 2, 8, G>(g, s);
  else
    go<DT, 2, 4, G>(g, s);
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
