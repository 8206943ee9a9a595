// Products of 8-bit tokens with 8-bit weights in large tiles (i8_linear.hip has
// the formula, the form in small ones and the choice).
//
// A block of four waves has a tile of 128 NI weight rows and 32 JT tokens; wave
// w has 32 NI of the rows against all the tokens, NI x JT accumulators of the
// 32 x 32 x 32 instruction.  With two weights (G = 2) accumulator 0 is of the
// gate's rows and 1 of the same rows of the other, so a lane has both sums of an
// output.  K goes by in tiles of 128 columns.
//
// Weights come from memory into registers as operands (their tiles are in that
// order, so a load is runs of 512 bytes) and never pass through LDS.  A tile
// of K's operands are loaded two tiles ahead, into the registers that the tile
// before last has left, step by step.  Tokens, which the waves share, reach LDS
// by DMA, in a ring of four to eight stages filled as far ahead, so one barrier
// a tile is enough.  A stage's rows are 128 bytes, eight pieces; a piece lies at
// its number ^ (row / 2) % 8, so the 16 rows that a read serves in a cycle lie
// in different banks.
//
// Large calls are bound by the chip's power: the matrix cores are busy for 80 %
// of the cycles in 128 x 256 (4096 tokens of 22016 x 8192) and for 64 % in the
// gated 128 x 128 (2047 of 11008 x 4096), on a full chip whose clock is then 1.3
// and 1.7 GHz instead of 2.35.  Once a run is under way 8192^3 takes 419 to 449 us
// by the codes, 2450 to 2620 TOPS (the library's int8 product of the same codes
// 439 to 447); 4096 tokens of 22016 x 8192 585 to 618 us (715 to 726); gated, 2047
// of 11008 x 4096, 159 to 174.  501 tokens of 4096 x K, a block of 64 x 128 on each
// CU, take 7.9 us at K 2048, 12.5 at 4096 and 22.6 at 8192: 80 GB/s a CU, 20 TB/s
// for all.  That is not L2's limit, which gives the small tiles 31; what holds it is
// not known.  61 of 11008 x 4096 (10.2) are bound by the weight's way from behind L2.

#include "i8_common.h"
#include "launch.h"

namespace qlora {
namespace {

constexpr int KT = 128;  // columns of a tile

// Until at most `vm` vector-memory operations of the wave are outstanding, and
// no LDS operation.
constexpr int wait_imm(int vm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4); }

__device__ __forceinline__ i32x16_t mfma32(u32x4_t a, u32x4_t b, i32x16_t c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a),
                                               __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// A wave's outputs: RO rows from n0 on of the 32 J tokens from m0 on.  All of
// them are scaled into the wave's LDS first, and go out from there in a loop,
// in runs of a token's row: done for 32 tokens at a time, with a wait between
// each write and read and code for every one, it took 10 us a tile of 256 x 256
// (the largest when this was measured, now gone), a tenth of the time at K 8192.
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
            if constexpr (G == 2) v[e] = i8_gated(v[e], i8_scaled(b[4 * q + e], sw[1][q][e], sx[j]), p.act);
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

// Up to four blocks of the small tiles on a CU: 2048 tokens of 8192 x 128 take
// 16.5 us, 17.7 with two, gated 785 of 10016 x 333 18.9 and 20.7.
template <class DT, int NI, int JT, int G>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, JT <= 2 ? 4 : 2)))
void gemm_i8_kernel(I8LinearArg p) {
  using S = Outputs<DT, NI, G, JT>;
  constexpr int TM = 32 * JT, RO = S::RO, TN = 4 * RO;
  // Stages of the tokens' ring: more for the small tiles, whose work covers less
  // of a load's way (32 x 128: 64 tokens, N and K 8192 take 19.0 us with four,
  // 16.5 with eight; 64 x 128: 501 tokens, N and K 4096 13.3 with four, 12.7 with
  // six; 128 x 128 loses with six).
  constexpr int ST = JT == 1 ? 8 : JT == 2 ? 6 : 4;
  constexpr int WD = 2;                // tiles of K whose weights are held or on their way
  constexpr int XR = JT;               // DMA instructions of a wave a tile
  constexpr int LC = 4 * NI;           // loads of weights a tile
  constexpr int XST = TM * KT;         // bytes of a stage
  constexpr int SLOTS = NI * JT;       // matrix instructions a step
  constexpr int DP = 4 * SLOTS / XR;   // of these from one DMA to the next
  constexpr int kRing = ST * XST, kOut = 4 * S::kBytes;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing > kOut ? kRing : kOut];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 31, lg = lane >> 5;
  const int64_t Kp = i8_padded(p.K), n_panels = (p.N + 15) / 16;
  uint32_t mt, nt;
  i8_tile_of(blockIdx.x, gridDim.x, (uint32_t)((p.M + TM - 1) / TM),
             (uint32_t)((p.N + TN - 1) / TN), 1024 / TM, mt, nt);
  const int64_t m0 = (int64_t)mt * TM, n0 = (int64_t)nt * TN;
  // x of tile kt + 2 has to be there at the end of iteration kt, and is when
  // no more operations are outstanding than came behind it: those of ST - 3
  // iterations and the last weights of its own, or in the first iterations
  // those of the prologue.
  constexpr int kSteady = (ST - 3) * (XR + LC) + NI, kFirst = (ST - 3) * XR + WD * LC;
  constexpr int kWait = kSteady < kFirst ? kSteady : kFirst;
  static_assert(kWait < 64 && ST >= 4, "outstanding operations of a wave");
  const int nkt = (int)(Kp / KT);

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
  // Weights of tiles past the last are zeros (a buffer of no bytes).
  auto load_w = [&](int kt, int i, int kk) -> u32x4_t {
    const auto buf = make_rsrc(G == 2 && i == 1 ? w1 : w0, kt < nkt ? held : 0);
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

  {
    auto cl = [&](int kt) { return kt < nkt ? kt : nkt - 1; };
    u32x4_t W[WD][4][NI], X[2][JT];
    auto load_tile = [&](int kt, int at) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < NI; ++i) W[at][kk][i] = load_w(kt, i, kk);
      __builtin_amdgcn_sched_barrier(0);
    };
    auto dma_tile = [&](int kt, int at) {
#pragma unroll
      for (int q = 0; q < XR; ++q) dma_x(lds + at * XST, cl(kt), q);
      __builtin_amdgcn_sched_barrier(0);
    };
    // x of the first two tiles, weights of the first, then the rest
    dma_tile(0, 0);
    dma_tile(1, 1);
    load_tile(0, 0);
#pragma unroll
    for (int d = 2; d < ST - 1; ++d) dma_tile(d, d);
#pragma unroll
    for (int d = 1; d < WD; ++d) load_tile(d, d);
    __builtin_amdgcn_s_waitcnt(wait_imm((ST - 3) * XR + WD * LC));
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
          if (slot % DP == DP - 1) dma_x(fill, cl(kt + ST - 1), slot / DP);
          // the registers of the step before are free
          if (kk > 0 && s % JT == (JT - 1) / 2)
            W[ph][kk - 1][s / JT] = load_w(kt + WD, s / JT, kk - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) W[ph][3][i] = load_w(kt + WD, i, 3);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_imm(kWait));
      __builtin_amdgcn_s_barrier();
    };
    int stage = 0;
    auto at = [&](int d) { return lds + (stage + d < ST ? stage + d : stage + d - ST) * XST; };
    auto step = [&](int kt, auto phase) {
      iteration(kt, phase, at(0), at(1), at(ST - 1));
      stage = stage + 1 < ST ? stage + 1 : 0;
    };
    for (int kt = 0; kt < nkt; kt += WD) {
      step(kt, std::integral_constant<int, 0>());
      step(kt + 1, std::integral_constant<int, 1>());
    }
    // what was asked for past the end is still on its way to LDS
    __builtin_amdgcn_s_waitcnt(wait_imm(0));
  }
  __syncthreads();
  S::run(acc, p, n0 + wave * RO, m0, lds + wave * S::kBytes, lane);
}

template <class DT, int NI, int JT, int G>
void go(const I8LinearArg& p, hipStream_t s) {
  constexpr int TM = 32 * JT, TN = G == 2 ? 128 : 128 * NI;
  const int64_t blocks = ((p.M + TM - 1) / TM) * ((p.N + TN - 1) / TN);
  gemm_i8_kernel<DT, NI, JT, G><<<dim3((unsigned)blocks), 256, 0, s>>>(p);
}

template <class DT, int G>
void pick(const I8LinearArg& p, int tile, hipStream_t s) {
  if constexpr (G == 2) {
    switch (tile) {
      case 0: return go<DT, 2, 1, 2>(p, s);
      case 1: return go<DT, 2, 2, 2>(p, s);
      default: return go<DT, 2, 4, 2>(p, s);
    }
  } else {
    switch (tile) {
      case 0: return go<DT, 1, 1, 1>(p, s);
      case 1: return go<DT, 1, 2, 1>(p, s);
      case 2: return go<DT, 1, 4, 1>(p, s);
      default: return go<DT, 2, 4, 1>(p, s);
    }
  }
}

}  // namespace

hipError_t launch_gemm_i8(const I8LinearArg& p, int tile, bool f16, hipStream_t s) {
  if (p.tiles[1]) {
    if (f16)
      pick<F16T, 2>(p, tile, s);
    else
      pick<Bf16T, 2>(p, tile, s);
  } else {
    if (f16)
      pick<F16T, 1>(p, tile, s);
    else
      pick<Bf16T, 1>(p, tile, s);
  }
  return hipGetLastError();
}

}  // namespace qlora
