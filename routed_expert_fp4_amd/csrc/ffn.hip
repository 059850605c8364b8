// libroutedfp4, the gated feed-forward block with dense weights:
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) * u                              (forward)
//   du = dh act(g),  dg = dh u act'(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x                      (backward)
//
// act is SiLU, g sigmoid(g), or GELU's tanh form, g sigmoid(2 sqrt(2/pi) (g + 0.044715 g^3)).
// Sums are fp32; h is formed of them and rounded once.  dg and du of 16-bit tensors
// meet the matrix cores again in two terms of that type, so that a gradient carries
// the rounding of its result and no other that counts.
//
// Kernels:
//   k_ffew      up to 32 tokens: bound by the stream of both weight matrices;
//               a workgroup takes eight rows of each, its waves ranges of columns
//   k_fgemm     more tokens, and the three products of the backward pass: one
//               tiled matrix product, whose operands lie along the sum's axis or
//               across it; g and u of the same rows and tokens are in the same lane
//   k_fjoin     adds ranges of the sum's axis, where tiles alone are too few
//   k_fact      dg and du as operands; in fp16 under a power of two, for which
//               k_fmost finds their largest
//   k_fpack     tensors whose rows are not at multiples of 16 bytes, into ones
//               that are
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include <type_traits>

#include "dense.h"

namespace rf4 {
namespace {

// sigmoid(z) and sigmoid(-z), both to fp32's precision down to its smallest
__device__ __forceinline__ void sigmoids(float z, float& s, float& c) {
  const float e = expf(-fabsf(z)), r = 1.0f / (1.0f + e);
  s = z < 0.0f ? e * r : r;
  c = z < 0.0f ? r : e * r;
}
// The argument of the sigmoid is g (k1 + k3 g^2): SiLU (1, 0), GELU's tanh form 2
// sqrt(2 / pi) (1, 0.044715).
struct Act { float k1, k3; };
inline Act act_constants(int act) {
  return act == MOE_ACT_SILU ? Act{1.0f, 0.0f} : Act{1.5957691216057308f, (float)(1.5957691216057308 * 0.044715)};
}
// k3 g^2, and 0 for SiLU whatever g is: 0 times an infinity is NaN
__device__ __forceinline__ float cubic(const Act& k, float g) { return k.k3 != 0.0f ? k.k3 * g * g : 0.0f; }
// act(g) and its slope; where the sigmoid is gone they are 0, however large g
__device__ __forceinline__ float act_of(const Act& k, float g) {
  float s, c;
  sigmoids(g * (k.k1 + cubic(k, g)), s, c);
  return s > 0.0f ? g * s : 0.0f * s;
}
__device__ __forceinline__ void act_slope(const Act& k, float g, float& a, float& d) {
  const float q = cubic(k, g);
  float s, c;
  sigmoids(g * (k.k1 + q), s, c);
  const float slope = k.k1 + 3.0f * q, e = s * c;
  a = s > 0.0f ? g * s : 0.0f * s;
  d = s + (e > 0.0f ? g * slope * e : 0.0f * e);
}

struct FArgs {
  int C, H, I;
  Act act;
  const uint8_t *x, *wg, *wu;
  int64_t x_pitch, wg_pitch, wu_pitch;                    // bytes, throughout
  uint8_t *h, *gate, *up;
  int64_t h_pitch, gate_pitch, up_pitch;
  // the product's operands and sizes (k_fgemm)
  const uint8_t *a0, *a1, *b0, *b1;
  int64_t a_pitch, b0_pitch, b1_pitch;
  int M, N, K;                                            // of one phase of the sum
  int mblocks, nblocks, steps, per_split, splits;         // steps of 128 bytes over all phases
  uint8_t *o0, *o1;
  int64_t o0_pitch, o1_pitch;
  int accumulate, out_f32;
  float* part;                                            // [splits][M][N] fp32
  const float* unscale;                                   // fp16 gradients: undoes dg's and du's power of two
};

// ---------------------------------------------------------------------------
// Few tokens
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void store_elem(uint8_t* p, float v) {
  if constexpr (DT == MOE_DT_F32) *reinterpret_cast<float*>(p) = v;
  else *reinterpret_cast<uint16_t*>(p) = round16<DT>(v);
}
template <int DT>
__device__ __forceinline__ float load_elem(const uint8_t* p) {
  if constexpr (DT == MOE_DT_F32) return *reinterpret_cast<const float*>(p);
  const uint16_t b = *reinterpret_cast<const uint16_t*>(p);
  if constexpr (DT == MOE_DT_BF16) return __uint_as_float((uint32_t)b << 16);
  return (float)__builtin_bit_cast(_Float16, b);
}

template <int DT>
__device__ __forceinline__ void put_gated(const FArgs& a, int c, int i, float g, float u) {
  constexpr int B = kBytes<DT>;
  store_elem<DT>(a.h + c * a.h_pitch + (int64_t)i * B, act_of(a.act, g) * u);
  if (a.gate) {
    store_elem<DT>(a.gate + c * a.gate_pitch + (int64_t)i * B, g);
    store_elem<DT>(a.up + c * a.up_pitch + (int64_t)i * B, u);
  }
}

// Bound by the weights' stream: one bf16 token x 7168 x 1536 9.8 us for 44 MB (4.5 TB/s,
// the launch included), 16 tokens x 7168 x 4096 27.2 for 117 (4.3).  Eight rows of each
// matrix are a 16-row operand; sixteen of each would leave half the workgroups.
constexpr int kFewWG = 512, kFewWaves = kFewWG / 64;
template <int DT, int TT>
__global__ __launch_bounds__(kFewWG) void k_ffew(FArgs a) {
  constexpr int B = kBytes<DT>;
  __shared__ float s_red[kFewWaves][TT][64][4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane & 15, quarter = lane >> 4;
  const int i0 = 8 * blockIdx.x;
  // first operand: rows 0 .. 7 of the gate, then of the up matrix (past the last: it again)
  const int i = i0 + (row & 7) < a.I ? i0 + (row & 7) : a.I - 1;
  const uint8_t* w = row < 8 ? a.wg + i * a.wg_pitch : a.wu + i * a.wu_pitch;
  const uint8_t* x[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int c = 16 * t + row;
    x[t] = a.x + (c < a.C ? c : a.C - 1) * a.x_pitch;
  }
  float4v acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = float4v(0.0f);
  // 128 columns to a wave at a time, the next on their way while these are multiplied
  // (by turns in two sets of registers: a copy would wait for them)
  constexpr int S = 4, U = 32 * S;
  struct Turn { Eight<DT> w[S], x[S][TT]; };
  auto load = [&](int c, Turn& u) {
#pragma unroll
    for (int q = 0; q < S; ++q) u.w[q] = load8<DT>(w + (int64_t)(c + 32 * q + 8 * quarter) * B);
#pragma unroll
    for (int q = 0; q < S; ++q)
#pragma unroll
      for (int t = 0; t < TT; ++t) u.x[q][t] = load8<DT>(x[t] + (int64_t)(c + 32 * q + 8 * quarter) * B);
  };
  auto multiply = [&](const Turn& u) {
#pragma unroll
    for (int q = 0; q < S; ++q)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] = mma8<DT>(u.w[q], u.x[q][t], acc[t]);
  };
  constexpr int kStep = U * kFewWaves;
  const int whole = a.H / U * U;
  Turn even, odd;
  int c = U * wave;
  if (c < whole) load(c, even);
  for (; c < whole; c += 2 * kStep) {
    if (c + kStep < whole) load(c + kStep, odd);
    __builtin_amdgcn_sched_barrier(0);
    multiply(even);
    if (c + kStep >= whole) break;
    if (c + 2 * kStep < whole) load(c + 2 * kStep, even);
    __builtin_amdgcn_sched_barrier(0);
    multiply(odd);
  }
  if (whole < a.H && whole / U % kFewWaves == wave) {
    // a row's last columns, zeros behind them
    for (int k = whole + 8 * quarter, q = 0; q < S && whole + 32 * q < a.H; ++q, k += 32) {
      const Eight<DT> e = load8_of<DT>(w, k, a.H);
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] = mma8<DT>(e, load8_of<DT>(x[t], k, a.H), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) s_red[wave][t][lane][e] = acc[t][e];
  __syncthreads();
  // 16 tokens x 8 rows to a token tile: thread (row of eight, token); register e
  // of lane l is weight row 4 (l / 16) + e, token l % 16
  for (int k = tid; k < TT * 128; k += kFewWG) {
    const int t = k >> 7, n = k & 7, c = (k >> 3) & 15;
    const int token = 16 * t + c;
    if (token >= a.C || i0 + n >= a.I) continue;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) {
      g += s_red[v][t][16 * (n >> 2) + c][n & 3];
      u += s_red[v][t][16 * (2 + (n >> 2)) + c][n & 3];
    }
    put_gated<DT>(a, token, i0 + n, g, u);
  }
}

// ---------------------------------------------------------------------------
// The tiled product
// ---------------------------------------------------------------------------
// A step takes 128 bytes along the sum's axis of an operand whose rows lie along
// it (64 elements of 16 bits, 32 of fp32): LDS holds its rows one after the
// other, the 16-byte unit u of row m at u ^ (m / 2 & 7) (16 rows that are read
// together fill the 256 bytes of the banks).  An operand that lies across the axis
// has that many of its rows in LDS, units exchanged too, and is read with the
// transposing LDS loads; fp32 is read element by element.  Both are loaded into LDS
// directly, one step ahead.
// dg and du in 16 bits are two terms (hi, then lo) by turns of 32 elements of a row: a
// step is 128 bytes of 32 positions, quarters hi and lo of one 16, then of the other, and
// the second operand's fragments, half as many, serve both.
// First launches in bf16 x 7168 x 4096: 2048 tokens 200 us (1.2 PFLOP/s), matrix cores
// busy for 60% of the cycles; 4096 tokens' dx 760 and weights' gradients 763, 1.26 PFLOP/s
// of both terms, 57% and 59% (in one term, rounded to the type, 449 and 448).
enum { kFwd, kDx, kDw };
template <int DT, int MODE>
constexpr int kTerms = DT != MOE_DT_F32 && MODE != kFwd ? 2 : 1;
// two stages, or the results
template <int DT, int MODE, int BM, int BN>
constexpr int kGemmLds = [] {
  constexpr int stages = 2 * (BM * 128 + BN * 128 / kTerms<DT, MODE>), results = BM * ((MODE == kFwd ? BN / 2 : BN) * 2 + 16);
  return DT == MOE_DT_F32 || stages > results ? stages : results;
}();

// 16 bytes a lane into LDS, at `at` + 16 lane, by inline assembly: behind the
// compiler's own form it lets every transposing LDS read wait for all of them.  They
// have no register to write but m0, which holds the LDS address, and are waited for
// before the barrier that opens them.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p);
}
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>((uintptr_t)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ void load_lds(const uint8_t* base, uint32_t off, const uint8_t* at) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(uniform(base)), "s"(lds_address(at)) : "m0", "memory");
}
__device__ __forceinline__ void load_lds(const uint8_t* p, const uint8_t* at) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(p), "s"(lds_address(at)) : "m0", "memory");
}
__device__ const uint32_t __attribute__((aligned(16))) kZeros[4] = {0, 0, 0, 0};

typedef short short4v __attribute__((ext_vector_type(4)));
template <int DT>
__device__ __forceinline__ float16v mma32(uint4v a, uint4v b, float16v c) {
  if constexpr (DT == MOE_DT_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  } else if constexpr (DT == MOE_DT_BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
  }
}

// The exchange of units in row k (mod 4) of an operand that lies across, `units` to a
// row: the 64 bytes that a transposing load takes of each of four rows fill the 256
// bytes of the banks.
template <int DT>
__device__ __forceinline__ int across_swap(int k, int units) {
  return DT == MOE_DT_F32 ? 0 : units >= 16 ? 4 * (k & 3) : 4 * (k >> 1 & 1);
}

// 32 rows (or columns) from `m` on, quarter ks of a step: lane l holds row l % 32
// and the eight (fp32: four) elements 2 ks + l / 32 of the step
template <int DT, bool ALONG, int ROWS>
__device__ __forceinline__ uint4v fragment(const uint8_t* s, int m, int ks, int lane) {
  if constexpr (ALONG) {
    const int row = m + (lane & 31), unit = 2 * ks + (lane >> 5);
    return *reinterpret_cast<const uint4v*>(s + row * 128 + ((unit ^ ((lane >> 1) & 7)) * 16));
  } else if constexpr (DT == MOE_DT_F32) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(s) + (8 * ks + 4 * (lane >> 5)) * ROWS + m + (lane & 31);
    return uint4v{p[0], p[ROWS], p[2 * ROWS], p[3 * ROWS]};
  } else {
    // a transposing load gives lane i of 16 element i of four rows, of which lane
    // i reads elements 4 (i % 4) .. of row i / 4
    const int g = lane >> 4, i = lane & 15, k = 16 * ks + 8 * (g >> 1) + (i >> 2);
    const int unit = (m >> 3) + 2 * (g & 1) + ((i >> 1) & 1);
    const uint8_t* p = s + k * (ROWS * 2) + ((unit ^ across_swap<DT>(i >> 2, ROWS / 8)) * 16) + (i & 1) * 8;
    const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v*)p);
    const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v*)(p + 4 * ROWS * 2));
    typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
    const uint2v l = __builtin_bit_cast(uint2v, lo), h = __builtin_bit_cast(uint2v, hi);
    return uint4v{l[0], l[1], h[0], h[1]};
  }
}

template <int DT, int MODE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_fgemm(FArgs a) {
  constexpr int TERMS = kTerms<DT, MODE>;
  constexpr int B = kBytes<DT>, WG = 64 * WM * WN, E = 128 / B / TERMS;   // positions of a step
  constexpr bool AL = MODE != kDw, BL = MODE == kFwd;                // rows along the sum's axis
  constexpr int MT = BM / WM / 32, NT = BN / WN / 32, NH = NT / 2;   // row and column tiles of a wave
  constexpr int kA = BM * 128, kB = BN * 128 / TERMS, kStage = kA + kB;
  constexpr int LA = kA / 16 / WG, LB = kB / 16 / WG;
  extern __shared__ __align__(1024) uint8_t s_ab[];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  // workgroups b, b + 8, .. run on one XCD: consecutive tiles each, eight blocks
  // of rows by all blocks of columns at a time, so that an XCD's tiles share both
  const int total = a.mblocks * a.nblocks, xcd = blockIdx.x & 7, rem = total & 7;
  const int tile = xcd * (total >> 3) + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const int group = tile / (8 * a.nblocks), in = tile - group * 8 * a.nblocks;
  const int rows = a.mblocks - 8 * group < 8 ? a.mblocks - 8 * group : 8;
  const int mb = 8 * group + in % rows, nb = in / rows;
  // kDw: the blocks of rows are dWg's, then dWu's
  const int half_blocks = MODE == kDw ? a.mblocks / 2 : a.mblocks;
  const bool second = MODE == kDw && mb >= half_blocks;
  const int m0 = (MODE == kDw && second ? mb - half_blocks : mb) * BM;
  const int n0 = MODE == kFwd ? nb * (BN / 2) : nb * BN;
  const int s0 = blockIdx.y * a.per_split, s1 = s0 + a.per_split < a.steps ? s0 + a.per_split : a.steps;
  const int phase = MODE == kDx ? a.steps / 2 : a.steps;             // steps of one phase

  // This thread's units of a step as offsets from the step's (scalar) bases; rows
  // and columns past the last are the last again, whose sums are not used.
  constexpr int UA = BM * B / 16, UB = BN * B / 16;                  // units of a row that lies across
  uint32_t oa[LA], ob[LB];
  auto unit_along = [&](int u) { return (u & 7) ^ ((u >> 4) & 7); };
  auto unit_across = [&](int u, int n) { return (u % n) ^ across_swap<DT>(u / n, n); };
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int u = i * WG + tid;
    if constexpr (AL) {
      const int r = u >> 3, most = a.M - 1 - m0;
      oa[i] = (uint32_t)((r < most ? r : most) * (uint32_t)a.a_pitch + unit_along(u) * 16);
    } else {
      const int most = (a.M * B + 15) / 16 - 1 - m0 * B / 16, n = unit_across(u, UA);
      const int w = n < most ? n : most, r = u / UA;
      oa[i] = (uint32_t)(r % E) * (uint32_t)a.a_pitch + (TERMS == 2 ? (w >> 2) * 128 + r / E * 64 + (w & 3) * 16 : w * 16);
    }
  }
  // (dx: those of the phase's matrix, whose rows may be another pitch apart)
  bool two_now = MODE == kDx && s0 >= phase;
  auto offsets_b = [&] {
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int u = i * WG + tid, most = (a.N * B + 15) / 16 - 1 - n0 * B / 16, n = unit_across(u, UB);
      ob[i] = (uint32_t)(u / UB) * (uint32_t)(two_now ? a.b1_pitch : a.b0_pitch) + (n < most ? n : most) * 16;
    }
  };
  if constexpr (!BL) offsets_b();
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int u = i * WG + tid;
    if constexpr (BL) {
      const int r = (u >> 3) & (BN / 2 - 1), most = a.N - 1 - n0;
      ob[i] = (uint32_t)(r < most ? r : most) * (uint32_t)(i < LB / 2 ? a.b0_pitch : a.b1_pitch) + unit_along(u) * 16;
    }
  }
  const uint8_t* a0 = (second ? a.a1 : a.a0) + (AL ? m0 * a.a_pitch : (int64_t)m0 * (B * TERMS));
  const uint8_t* b0 = a.b0 + (BL ? n0 * a.b0_pitch : (int64_t)n0 * B);
  const uint8_t* b1 = MODE == kFwd ? a.b1 + n0 * a.b1_pitch : a.b1 + (int64_t)n0 * B;
  // where a step's operands lie
  struct From { const uint8_t *pa, *pb, *pu; int k0; };
  auto from = [&](int s) {
    const bool two = MODE == kDx && s >= phase;
    const int k0 = (two ? s - phase : s) * E;
    if constexpr (MODE == kDx) {
      if (two != two_now) {
        two_now = two;
        offsets_b();
      }
    }
    return From{AL ? a0 + (two ? a.a1 - a.a0 : 0) + (int64_t)k0 * (B * TERMS) : a0 + k0 * a.a_pitch,
                BL ? b0 + (int64_t)k0 * B : two ? b1 + k0 * a.b1_pitch : b0 + k0 * a.b0_pitch, b1 + (int64_t)k0 * B, k0};
  };
  auto stage_one = [&](const From& f, const uint8_t* to, int i) {
    if (i < LA) load_lds(f.pa, oa[i], to + (i * WG + wave * 64) * 16);
    else load_lds(BL && i - LA >= LB / 2 ? f.pu : f.pb, ob[i - LA], to + kA + ((i - LA) * WG + wave * 64) * 16);
  };
  auto stage = [&](int s, const uint8_t* to) {
    const From f = from(s);
    const int k0 = f.k0;
    if (k0 + E <= a.K) {
#pragma unroll
      for (int i = 0; i < LA + LB; ++i) stage_one(f, to, i);
    } else {
      // zeros past the sum's end (rows of two terms hold them themselves)
      auto load = [&](const uint8_t* base, uint32_t off, bool ok, const uint8_t* at) {
        load_lds(ok ? base + off : reinterpret_cast<const uint8_t*>(kZeros), at);
      };
#pragma unroll
      for (int i = 0; i < LA; ++i) {
        const int u = i * WG + tid;
        load(f.pa, oa[i], k0 + (!AL ? u / UA % E : TERMS == 2 ? 0 : unit_along(u) * (16 / B)) < a.K, to + (i * WG + wave * 64) * 16);
      }
#pragma unroll
      for (int i = 0; i < LB; ++i) {
        const int u = i * WG + tid;
        load(BL && i >= LB / 2 ? f.pu : f.pb, ob[i], k0 + (BL ? unit_along(u) * (16 / B) : u / UB) < a.K,
             to + kA + (i * WG + wave * 64) * 16);
      }
    }
  };

  float16v acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = float16v(0.0f);
  // the column tiles of a wave: forward, NH of the gate's and the same of up's
  auto column = [&](int j) {
    return MODE == kFwd ? 32 * (NH * wn + j % NH) + (j / NH) * (BN / 2) : 32 * (NT * wn + j);
  };
  uint4v fa[2][MT], fb[2][NT];
  auto second_of = [](int k) { return TERMS == 2 ? k >> 1 : k; };    // quarter k's of the second operand
  auto read = [&](const uint8_t* t, int k) {
    if (TERMS == 1 || !(k & 1)) {
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[second_of(k) & 1][j] = fragment<DT, BL, BN>(t + kA, column(j), second_of(k), lane);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
      fa[k & 1][i] = fragment<DT, AL, BM>(t, wm * (BM / WM) + 32 * i, TERMS == 2 ? 2 * (k & 1) + (k >> 1) : k, lane);
  };
  // a quarter's products, and loads n0 .. n1 - 1 of a step to come between them: a
  // matrix instruction leaves the time for one
  From f = {};
  bool more = false;
  auto product = [&](int k, int n0, int n1, const uint8_t* to) {
    int n = n0;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        acc[i][j] = mma32<DT>(fa[k & 1][i], fb[second_of(k) & 1][j], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
        const int upto = n0 + (n1 - n0) * (i * NT + j + 1) / (MT * NT);
#pragma unroll
        for (; n < upto; ++n)
          if (more) stage_one(f, to, n);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  // this wave's loads into LDS and reads from it are complete, and so every wave's
  auto meet = [&] {
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);                    // lgkmcnt(0) too, in the compiler's own count
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
  };
  // A step is four quarters.  A quarter's operands are read during the one before;
  // the move to the next step comes before the last quarter's products, so that
  // they cover it: by then this step is read, and its buffer is free for the step
  // after the next, whose loads go out between those products (spread over three
  // quarters they came too late: 4096 tokens x 7168 x 4096, dx of one term 473 us against 430).
  stage(s0, s_ab);
  meet();
  read(s_ab, 0);
  if (s0 + 1 < s1) stage(s0 + 1, s_ab + kStage);
  // nothing is on its way when the loop begins, scalar loads among it: they would
  // make every wait in it one for all LDS reads
  __builtin_amdgcn_s_waitcnt(0x0070);
  __builtin_amdgcn_sched_barrier(0);
  int buf = 0;
  for (int s = s0; s < s1; ++s) {
    const uint8_t *t = s_ab + buf * kStage, *next = s_ab + (buf ^ 1) * kStage;
    read(t, 1);
    __builtin_amdgcn_sched_barrier(0);
    product(0, 0, 0, t);
    read(t, 2);
    __builtin_amdgcn_sched_barrier(0);
    product(1, 0, 0, t);
    read(t, 3);
    __builtin_amdgcn_sched_barrier(0);
    product(2, 0, 0, t);
    meet();
    read(next, 0);                                         // behind the last step: read, and not used
    __builtin_amdgcn_sched_barrier(0);
    f = from(s + 2);
    more = s + 2 < s1 && f.k0 + E <= a.K;
    if (!more && s + 2 < s1) stage(s + 2, t);
    product(3, 0, LA + LB, t);
    buf ^= 1;
  }

  if constexpr (DT == MOE_DT_F16 && TERMS == 2) {
    const float un = *a.unscale;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] *= un;
  }
  // register r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
  auto row_of = [&](int i, int r) { return wm * (BM / WM) + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3); };
  if constexpr (B == 2) {
    if (a.splits == 1 && !a.accumulate && !a.out_f32) {
      // The results through LDS, so that rows are stored 16 bytes a lane: as they lie
      // in registers a store holds 64 bytes of two rows.  Forward: h, then g and u.
      constexpr int WN0 = MODE == kFwd ? BN / 2 : BN, kPitch = WN0 * 2 + 16;   // bytes of a row; 16 more spread the banks
      static_assert(BM * kPitch <= kGemmLds<DT, MODE, BM, BN> && 2 * kStage <= kGemmLds<DT, MODE, BM, BN>, "the results fit the LDS");
      auto through = [&](uint8_t* out, int64_t pitch, auto value) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int j = 0; j < (MODE == kFwd ? NH : NT); ++j)
              *reinterpret_cast<uint16_t*>(s_ab + row_of(i, r) * kPitch + (column(j) + (lane & 31)) * 2) = round16<DT>(value(i, j, r));
        __syncthreads();
        constexpr int per = WN0 / 8;                         // lanes to a row
        for (int k = tid; k < BM * per; k += WG) {
          const int m = k / per, n = k % per * 8;
          if (m0 + m >= a.M) break;
          store16_some<DT>(out + (m0 + m) * pitch + (int64_t)(n0 + n) * 2,
                           *reinterpret_cast<const uint4v*>(s_ab + m * kPitch + n * 2), a.N - n0 - n);
        }
      };
      if constexpr (MODE == kFwd) {
        through(a.h, a.h_pitch, [&](int i, int j, int r) { return act_of(a.act, acc[i][j][r]) * acc[i][j + NH][r]; });
        if (a.gate) {
          through(a.gate, a.gate_pitch, [&](int i, int j, int r) { return acc[i][j][r]; });
          through(a.up, a.up_pitch, [&](int i, int j, int r) { return acc[i][j + NH][r]; });
        }
      } else {
        through(second ? a.o1 : a.o0, second ? a.o1_pitch : a.o0_pitch, [&](int i, int j, int r) { return acc[i][j][r]; });
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int m = m0 + row_of(i, r);
      if (m >= a.M) continue;
      if constexpr (MODE == kFwd) {
#pragma unroll
        for (int j = 0; j < NH; ++j) {
          const int n = n0 + column(j) + (lane & 31);
          if (n >= a.N) continue;
          if (a.splits > 1) {
            float* o = a.part + ((int64_t)blockIdx.y * a.M + m) * 2 * a.N + n;
            o[0] = acc[i][j][r];
            o[a.N] = acc[i][j + NH][r];
          } else {
            put_gated<DT>(a, m, n, acc[i][j][r], acc[i][j + NH][r]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int n = n0 + column(j) + (lane & 31);
          if (n >= a.N) continue;
          const float v = acc[i][j][r];
          if (MODE == kDx && a.splits > 1) {
            a.part[((int64_t)blockIdx.y * a.M + m) * a.N + n] = v;
          } else if (MODE == kDw && a.out_f32) {
            float* o = reinterpret_cast<float*>((second ? a.o1 : a.o0) + m * (second ? a.o1_pitch : a.o0_pitch)) + n;
            *o = a.accumulate ? *o + v : v;
          } else {
            uint8_t* o = (second ? a.o1 : a.o0) + m * (second ? a.o1_pitch : a.o0_pitch) + (int64_t)n * B;
            store_elem<DT>(o, a.accumulate ? load_elem<DT>(o) + v : v);
          }
        }
      }
    }
}

// The ranges of the sum's axis, added in order, then what the tile would have done.
template <int DT, int MODE>
__global__ __launch_bounds__(256) void k_fjoin(FArgs a) {
  const int64_t n = (int64_t)a.M * a.N, step = MODE == kFwd ? 2 * n : n;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
    const int64_t m = e / a.N;
    const int k = (int)(e - m * a.N);
    if constexpr (MODE == kFwd) {
      const float* p = a.part + m * 2 * a.N + k;
      float g = 0.0f, u = 0.0f;
      for (int s = 0; s < a.splits; ++s) {
        g += p[s * step];
        u += p[s * step + a.N];
      }
      put_gated<DT>(a, (int)m, k, g, u);
    } else {
      float v = 0.0f;
      for (int s = 0; s < a.splits; ++s) v += a.part[s * step + e];
      uint8_t* o = a.o0 + m * a.o0_pitch + (int64_t)k * kBytes<DT>;
      store_elem<DT>(o, a.accumulate ? load_elem<DT>(o) + v : v);
    }
  }
}

// ---------------------------------------------------------------------------
// dg and du, and packing
// ---------------------------------------------------------------------------
constexpr int kMostParts = 1024;
struct GArgs {
  int C, I;
  Act act;
  const uint8_t *gate, *up, *dh;
  int64_t gate_pitch, up_pitch, dh_pitch;
  uint8_t *dg, *du;                                       // rows of `units` eights, in 16 bits of two terms
  int64_t pitch;
  int units;
  float* most;                                            // fp16: [kMostParts], then what undoes the scale
  int parts;
};
// Columns i .. i + 7 of a token's dg and du, zeros past the last.
template <int DT>
__device__ __forceinline__ void gate_grads(const GArgs& a, int64_t c, int i, float (&dg)[8], float (&du)[8]) {
  constexpr int B = kBytes<DT>;
  const uint8_t *pg = a.gate + c * a.gate_pitch, *pu = a.up + c * a.up_pitch, *pd = a.dh + c * a.dh_pitch;
  Eight<DT> g, u, d;
  if (a.units * 8 == a.I) {             // one branch for the three, which are then on their way together
    g = load8<DT>(pg + (int64_t)i * B);
    u = load8<DT>(pu + (int64_t)i * B);
    d = load8<DT>(pd + (int64_t)i * B);
  } else {
    g = load8_of<DT>(pg, i, a.I);
    u = load8_of<DT>(pu, i, a.I);
    d = load8_of<DT>(pd, i, a.I);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float act, slope;
    act_slope(a.act, get8<DT>(g, j), act, slope);
    const float t = get8<DT>(d, j);
    du[j] = t * act;
    dg[j] = t * get8<DT>(u, j) * slope;
  }
}

// The largest finite magnitude of dg and du (fp16), a part of them to a workgroup: 4096 x
// 4096 33.7 us with four workgroups a CU, 52.6 with one.
__device__ __forceinline__ uint32_t most_of(uint32_t v, uint32_t* s) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, d, 64);
    v = o > v ? o : v;
  }
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) v = s[w] > v ? s[w] : v;
  return v;
}
__global__ __launch_bounds__(256) void k_fmost(GArgs a) {
  __shared__ uint32_t s_most[4];
  const int64_t n = (int64_t)a.C * a.units;
  uint32_t most = 0;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
    const int64_t c = e / a.units;
    float dg[8], du[8];
    gate_grads<MOE_DT_F16>(a, c, 8 * (int)(e - c * a.units), dg, du);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t x = __float_as_uint(dg[j]) & 0x7FFFFFFFu, y = __float_as_uint(du[j]) & 0x7FFFFFFFu;
      if (x < 0x7F800000u) most = x > most ? x : most;
      if (y < 0x7F800000u) most = y > most ? y : most;
    }
  }
  most = most_of(most, s_most);
  if (threadIdx.x == 0) a.most[blockIdx.x] = __uint_as_float(most);
}

// dg and du as operands; past the last column zeros, the sum over I runs on whole steps.
// In 16 bits a value is two terms, itself rounded and what is left rounded: 2^-17 of it
// is lost in bf16.  In fp16 both are under the power of two that puts the call's largest
// finite value at 2^14 or more and below 2^15 (2^-23 of a value is lost, or 2^-39 of the
// largest), so that neither an infinity nor a zero comes of its range.  Bound by memory:
// 4096 x 4096 in bf16 40.8 us for 235 MB (5.8 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void k_fact(GArgs a) {
  constexpr int B = kBytes<DT>;
  __shared__ uint32_t s_most[4];
  float m = 1.0f;
  if constexpr (DT == MOE_DT_F16) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kMostParts; i += 256) {
      const int k = i + (int)threadIdx.x;
      const uint32_t v = __float_as_uint(a.most[k < a.parts ? k : 0]);
      most = v > most ? v : most;
    }
    most = most_of(most, s_most);
    int e = most ? 14 - ((int)(most >> 23) - 127) : 0;
    e = e > 126 ? 126 : e;
    m = __uint_as_float((uint32_t)(127 + e) << 23);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.most[kMostParts] = __uint_as_float((uint32_t)(127 - e) << 23);
  }
  const int64_t n = (int64_t)a.C * a.units;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
    const int64_t c = e / a.units;
    const int i = 8 * (int)(e - c * a.units);
    float dg[8], du[8];
    gate_grads<DT>(a, c, i, dg, du);
    auto put = [&](uint8_t* row, float (&v)[8]) {
      if constexpr (DT == MOE_DT_F32) {
        store8<DT>(row + (int64_t)i * B, put8<DT>(v));
      } else {
        uint8_t* p = row + (i >> 5) * 128 + (i & 31) * 2;
        float lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= m;
        const Eight<DT> hi = put8<DT>(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float h = get8<DT>(hi, j);
          lo[j] = fabsf(h) < INFINITY ? v[j] - h : 0.0f;   // not finite: its own first term
        }
        store8<DT>(p, hi);
        store8<DT>(p + 64, put8<DT>(lo));
      }
    };
    put(a.dg + c * a.pitch, dg);
    put(a.du + c * a.pitch, du);
  }
}

struct Pack {
  const uint8_t* in;
  int64_t in_pitch, rows;
  uint8_t* out;
};
struct KArgs {
  Pack t[3];
  int cols, units;
};
// rows of `cols` elements into rows of `units` eights, zeros behind them
template <int DT>
__global__ __launch_bounds__(256) void k_fpack(KArgs a) {
  constexpr int B = kBytes<DT>;
  const Pack& p = a.t[blockIdx.y];
  const int64_t n = p.rows * a.units;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
    const int64_t r = e / a.units;
    const int k = 8 * (int)(e - r * a.units);
    store8<DT>(p.out + e * 8 * B, load8_of<DT>(p.in + r * p.in_pitch, k, a.cols));
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int kFewTokens = 32;

moe_status ffn_status(const moe_ffn* f) {
  if (!f) return MOE_ERR_INVALID_ARG;
  if (!dense_dtype_ok(f->dtype) || (f->act != MOE_ACT_SILU && f->act != MOE_ACT_GELU) || f->hidden < 1 ||
      f->hidden > MOE_MAX_QUANT_COLS || f->inter < 1 || f->inter > MOE_MAX_QUANT_COLS)
    return MOE_ERR_UNSUPPORTED;
  const int64_t s = dense_size(f->dtype);
  moe_status st = rows_status(Rows{f->w_gate, f->gate_pitch, f->hidden, f->inter, s});
  return st != MOE_OK ? st : rows_status(Rows{f->w_up, f->up_pitch, f->hidden, f->inter, s});
}

// rows that can be loaded into LDS 16 bytes at a time, in whole units, 256 of them
// by 32-bit offsets
bool whole_units(const void* p, int64_t pitch, int64_t rows, int64_t cols, int64_t s) {
  return (uintptr_t)p % 16 == 0 && (rows == 1 || (pitch * s % 16 == 0 && pitch * s <= (1 << 23))) && cols * s % 16 == 0;
}

// How a product is tiled and split.
struct Tiling { int bm, bn, mblocks, nblocks, steps, splits, per_split; };
Tiling tiling(int mode, int64_t M, int64_t N, int64_t K, int64_t s) {
  Tiling t;
  const int e = (int)(s == 2 && mode != kFwd ? 32 : 128 / s);       // positions of a step
  auto blocks = [&](int bm, int bn) {
    t.bm = bm; t.bn = bn;
    t.mblocks = (int)((M + bm - 1) / bm) * (mode == kDw ? 2 : 1);
    const int n = mode == kFwd ? bn / 2 : bn;
    t.nblocks = (int)((N + n - 1) / n);
    return (int64_t)t.mblocks * t.nblocks;
  };
  // 256 x 256 where its tiles, one a CU, come near the number of CUs; 64 x 128 for up
  // to 64 rows, for few tiles, and where the sum's axis is not split
  int64_t n = blocks(256, 256);
  if (n < 192) n = blocks(128, 128);
  if (t.bm == 128 && (M <= 64 || n < 64 || (mode == kDw && n < 256))) n = blocks(64, 128);
  t.steps = (int)((K + e - 1) / e) * (mode == kDx ? 2 : 1);
  t.splits = 1;
  t.per_split = t.steps;
  if (t.bm < 256 && mode != kDw) {
    // ranges of four steps at least, as many workgroups as the CUs hold
    int64_t q = (t.bm == 64 ? 768 : 512) / n, most = t.steps / 4;
    q = q < most ? q : most;
    if (q > 1) {
      t.per_split = (int)((t.steps + q - 1) / q);
      t.splits = (t.steps + t.per_split - 1) / t.per_split;
    }
  }
  return t;
}

struct FfnWs { size_t x, wg, wu, dg, du, most, part, total; int64_t hp, ip; };
FfnWs ffn_ws_for(const moe_ffn* f, int C, bool bwd) {
  const int64_t s = dense_size(f->dtype), H = f->hidden, I = f->inter;
  FfnWs w = {};
  w.hp = (H + 7) / 8 * 8 * s;
  w.ip = s == 2 ? (I + 31) / 32 * 128 : (I + 7) / 8 * 8 * s;
  size_t o = 0;
  if (!bwd && C <= kFewTokens) {
    w.total = 0;                        // k_ffew takes everything as it is
    return w;
  }
  // x's own alignment is not known here: room for it and for weights that need it
  w.x = o; o = align256(o + (size_t)C * w.hp);
  w.wg = o; o = align256(o + (whole_units(f->w_gate, f->gate_pitch, I, H, s) ? 0 : (size_t)I * w.hp));
  w.wu = o; o = align256(o + (whole_units(f->w_up, f->up_pitch, I, H, s) ? 0 : (size_t)I * w.hp));
  w.dg = o; o = align256(o + (bwd ? (size_t)C * w.ip : 0));
  w.du = o; o = align256(o + (bwd ? (size_t)C * w.ip : 0));
  w.most = o; o = align256(o + (bwd && f->dtype == MOE_DT_F16 ? (kMostParts + 1) * sizeof(float) : 0));
  w.part = o;
  const Tiling t = bwd ? tiling(kDx, C, H, I, s) : tiling(kFwd, C, I, H, s);
  if (t.splits > 1) o = align256(o + (size_t)t.splits * C * (bwd ? H : 2 * I) * sizeof(float));
  w.total = o;
  return w;
}
// The most that any number of tokens up to C needs: partial results come and go
// with the ranges, which depend on tiles of 64 tokens.
size_t ffn_workspace(const moe_ffn* f, int C, bool bwd) {
  size_t most = 256;
  for (int c = C;; c = (c - 1) / 64 * 64) {
    const size_t a = ffn_ws_for(f, c, false).total, b = bwd ? ffn_ws_for(f, c, true).total : 0;
    most = a > most ? a : most;
    most = b > most ? b : most;
    if (c <= 64) break;
  }
  return most;
}

template <int DT, int MODE, int BM, int BN, int WM, int WN>
moe_status launch_gemm_t(const FArgs& a, dim3 grid, hipStream_t st) {
  constexpr int lds = kGemmLds<DT, MODE, BM, BN>;
  auto k = k_fgemm<DT, MODE, BM, BN, WM, WN>;
  if (lds > 65536 && hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize,
                                         lds) != hipSuccess)
    return MOE_ERR_DEVICE;
  hipLaunchKernelGGL(k, grid, dim3(64 * WM * WN), lds, st, a);
  return MOE_OK;
}
template <int DT, int MODE>
moe_status launch_product(FArgs a, hipStream_t st) {
  const Tiling t = tiling(MODE, a.M, a.N, a.K, kBytes<DT>);
  a.mblocks = t.mblocks; a.nblocks = t.nblocks;
  a.steps = t.steps; a.splits = t.splits; a.per_split = t.per_split;
  const dim3 grid((unsigned)(t.mblocks * t.nblocks), (unsigned)t.splits);
  const moe_status s = t.bm == 256   ? launch_gemm_t<DT, MODE, 256, 256, 2, 4>(a, grid, st)
                       : t.bm == 128 ? launch_gemm_t<DT, MODE, 128, 128, 2, 2>(a, grid, st)
                                     : launch_gemm_t<DT, MODE, 64, 128, 2, 2>(a, grid, st);
  if (s != MOE_OK) return s;
  if constexpr (MODE != kDw) {
    if (t.splits > 1) {
      const int64_t n = ((int64_t)a.M * a.N + 255) / 256;
      hipLaunchKernelGGL((k_fjoin<DT, MODE>), dim3((unsigned)(n < 65536 ? n : 65536)), dim3(256), 0, st, a);
    }
  }
  return MOE_OK;
}

unsigned fill_grid(int64_t n) {
  n = (n + 255) / 256;
  return (unsigned)(n < 65536 ? n : 65536);
}

// x and the weights as the matrix kernel takes them: themselves, or packed.
template <int DT>
void operands(const moe_ffn* f, FArgs& a, const FfnWs& w, uint8_t* w8, bool weights, bool need_x, hipStream_t st) {
  const int64_t s = kBytes<DT>;
  KArgs k = {};
  int n = 0;
  int64_t most = 0;
  k.cols = a.H;
  k.units = (a.H + 7) / 8;
  auto pack = [&](const uint8_t*& p, int64_t& pitch, int64_t rows, size_t at) {
    if (whole_units(p, pitch / s, rows, a.H, s)) return;
    k.t[n++] = Pack{p, pitch, rows, w8 + at};
    most = rows > most ? rows : most;
    p = w8 + at;
    pitch = w.hp;
  };
  if (need_x) pack(a.x, a.x_pitch, a.C, w.x);
  if (weights) {
    pack(a.wg, a.wg_pitch, a.I, w.wg);
    pack(a.wu, a.wu_pitch, a.I, w.wu);
  }
  if (n) hipLaunchKernelGGL((k_fpack<DT>), dim3(fill_grid(most * k.units), (unsigned)n), dim3(256), 0, st, k);
}

template <int DT>
moe_status ffn_forward(const moe_ffn* f, FArgs a, const FfnWs& w, uint8_t* w8, hipStream_t st) {
  if (a.C <= kFewTokens) {
    const dim3 grid((unsigned)((a.I + 7) / 8));
    if (a.C <= 16) hipLaunchKernelGGL((k_ffew<DT, 1>), grid, dim3(kFewWG), 0, st, a);
    else hipLaunchKernelGGL((k_ffew<DT, 2>), grid, dim3(kFewWG), 0, st, a);
    return MOE_OK;
  }
  operands<DT>(f, a, w, w8, true, true, st);
  a.a0 = a.x; a.a_pitch = a.x_pitch;
  a.b0 = a.wg; a.b0_pitch = a.wg_pitch; a.b1 = a.wu; a.b1_pitch = a.wu_pitch;
  a.M = a.C; a.N = a.I; a.K = a.H * kBytes<DT> % 16 ? (a.H + 7) / 8 * 8 : a.H;   // packed rows end in zeros
  a.part = reinterpret_cast<float*>(w8 + w.part);
  return launch_product<DT, kFwd>(a, st);
}

template <int DT>
moe_status ffn_backward(const moe_ffn* f, FArgs a, GArgs g, uint8_t* dx, int64_t dx_pitch, uint8_t* dwg,
                        int64_t dwg_pitch, uint8_t* dwu, int64_t dwu_pitch, int out_f32, int accumulate, const FfnWs& w,
                        uint8_t* w8, hipStream_t st) {
  g.dg = w8 + w.dg; g.du = w8 + w.du;
  g.pitch = w.ip;
  g.units = DT == MOE_DT_F32 ? (a.I + 7) / 8 : (a.I + 31) / 32 * 4;
  if constexpr (DT == MOE_DT_F16) {
    g.most = reinterpret_cast<float*>(w8 + w.most);
    const unsigned most = fill_grid((int64_t)a.C * g.units);
    g.parts = most < kMostParts ? (int)most : kMostParts;
    hipLaunchKernelGGL(k_fmost, dim3((unsigned)g.parts), dim3(256), 0, st, g);
    a.unscale = g.most + kMostParts;
  }
  hipLaunchKernelGGL((k_fact<DT>), dim3(fill_grid((int64_t)a.C * g.units)), dim3(256), 0, st, g);
  operands<DT>(f, a, w, w8, dx != nullptr, dwg != nullptr, st);
  a.part = reinterpret_cast<float*>(w8 + w.part);
  a.accumulate = accumulate;
  a.a0 = g.dg; a.a1 = g.du; a.a_pitch = w.ip;
  if (dx) {
    FArgs p = a;
    p.b0 = a.wg; p.b0_pitch = a.wg_pitch; p.b1 = a.wu; p.b1_pitch = a.wu_pitch;
    p.M = a.C; p.N = a.H; p.K = a.I;
    p.o0 = dx; p.o0_pitch = dx_pitch;
    const moe_status s = launch_product<DT, kDx>(p, st);
    if (s != MOE_OK) return s;
  }
  if (dwg) {
    FArgs p = a;
    p.b0 = a.x; p.b0_pitch = a.x_pitch;
    p.M = a.I; p.N = a.H; p.K = a.C;
    p.o0 = dwg; p.o0_pitch = dwg_pitch; p.o1 = dwu; p.o1_pitch = dwu_pitch;
    p.out_f32 = out_f32;
    return launch_product<DT, kDw>(p, st);
  }
  return MOE_OK;
}

void ffn_args(const moe_ffn* f, const void* x, int64_t x_pitch, int C, FArgs& a) {
  const int64_t s = dense_size(f->dtype);
  a.C = C; a.H = f->hidden; a.I = f->inter; a.act = act_constants(f->act);
  a.x = static_cast<const uint8_t*>(x); a.x_pitch = x_pitch * s;
  a.wg = static_cast<const uint8_t*>(f->w_gate); a.wg_pitch = f->gate_pitch * s;
  a.wu = static_cast<const uint8_t*>(f->w_up); a.wu_pitch = f->up_pitch * s;
}

}  // namespace
}  // namespace rf4

using namespace rf4;

extern "C" {

size_t moe_ffn_workspace_size(const moe_ffn* f, int32_t C) {
  if (ffn_status(f) != MOE_OK || C < 1 || C > MOE_MAX_FFN_TOKENS) return 0;
  return ffn_workspace(f, C, true);
}

size_t moe_ffn_fwd_workspace_size(const moe_ffn* f, int32_t C) {
  if (ffn_status(f) != MOE_OK || C < 1 || C > MOE_MAX_FFN_TOKENS) return 0;
  return ffn_workspace(f, C, false);
}

moe_status moe_ffn_fwd(const moe_ffn* f, const void* x, int64_t x_pitch, int32_t C, void* h, int64_t h_pitch, void* gate,
                       int64_t gate_pitch, void* up, int64_t up_pitch, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = ffn_status(f);
  if (st != MOE_OK) return st;
  if (C < 1 || C > MOE_MAX_FFN_TOKENS) return MOE_ERR_UNSUPPORTED;
  const int64_t s = dense_size(f->dtype);
  const Rows rx = {x, x_pitch, f->hidden, C, s}, rh = {h, h_pitch, f->inter, C, s};
  const Rows rg = {gate, gate_pitch, f->inter, C, s}, ru = {up, up_pitch, f->inter, C, s};
  const Rows w0 = {f->w_gate, f->gate_pitch, f->hidden, f->inter, s}, w1 = {f->w_up, f->up_pitch, f->hidden, f->inter, s};
  if (!gate != !up) return MOE_ERR_INVALID_ARG;
  if ((st = rows_status(rx)) != MOE_OK || (st = rows_status(rh)) != MOE_OK) return st;
  if (gate && ((st = rows_status(rg)) != MOE_OK || (st = rows_status(ru)) != MOE_OK)) return st;
  const Rows outs[] = {rh, rg, ru, span(ws, (int64_t)ws_bytes)}, ins[] = {rx, w0, w1};
  if (any_share(outs, ins) || any_share({outs[3]}, {rh, rg, ru})) return MOE_ERR_INVALID_ARG;
  if (share(rh, rg) || share(rh, ru) || share(rg, ru)) return MOE_ERR_INVALID_ARG;
  const FfnWs w = ffn_ws_for(f, C, false);
  if (!ws || (uintptr_t)ws % 256 || ws_bytes < w.total) return MOE_ERR_WORKSPACE;
  FArgs a = {};
  ffn_args(f, x, x_pitch, C, a);
  a.h = static_cast<uint8_t*>(h); a.h_pitch = h_pitch * s;
  a.gate = static_cast<uint8_t*>(gate); a.gate_pitch = gate_pitch * s;
  a.up = static_cast<uint8_t*>(up); a.up_pitch = up_pitch * s;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  hipStream_t q = reinterpret_cast<hipStream_t>(stream);
  st = f->dtype == MOE_DT_F32    ? ffn_forward<MOE_DT_F32>(f, a, w, w8, q)
       : f->dtype == MOE_DT_BF16 ? ffn_forward<MOE_DT_BF16>(f, a, w, w8, q)
                                 : ffn_forward<MOE_DT_F16>(f, a, w, w8, q);
  if (st != MOE_OK) return st;
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

moe_status moe_ffn_bwd(const moe_ffn* f, const void* x, int64_t x_pitch, const void* gate, int64_t gate_pitch,
                       const void* up, int64_t up_pitch, const void* dh, int64_t dh_pitch, int32_t C, void* dx,
                       int64_t dx_pitch, int32_t grad_dtype, void* dw_gate, int64_t dw_gate_pitch, void* dw_up,
                       int64_t dw_up_pitch, int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = ffn_status(f);
  if (st != MOE_OK) return st;
  if (C < 1 || C > MOE_MAX_FFN_TOKENS) return MOE_ERR_UNSUPPORTED;
  if (!dw_gate != !dw_up || (!dx && !dw_gate)) return MOE_ERR_INVALID_ARG;
  if (dw_gate && grad_dtype != f->dtype && grad_dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
  const int64_t s = dense_size(f->dtype), H = f->hidden, I = f->inter;
  const int64_t gs = dw_gate ? dense_size(grad_dtype) : s;
  const Rows rx = {dw_gate ? x : nullptr, x_pitch, H, C, s}, rg = {gate, gate_pitch, I, C, s}, ru = {up, up_pitch, I, C, s};
  const Rows rh = {dh, dh_pitch, I, C, s}, rd = {dx, dx_pitch, H, C, s};
  const Rows w0 = {f->w_gate, f->gate_pitch, H, I, s}, w1 = {f->w_up, f->up_pitch, H, I, s};
  const Rows g0 = {dw_gate, dw_gate_pitch, H, I, gs}, g1 = {dw_up, dw_up_pitch, H, I, gs};
  for (const Rows& r : {rg, ru, rh})
    if ((st = rows_status(r)) != MOE_OK) return st;
  if (dx && (st = rows_status(rd)) != MOE_OK) return st;
  if (dw_gate && ((st = rows_status(rx)) != MOE_OK || (st = rows_status(g0)) != MOE_OK || (st = rows_status(g1)) != MOE_OK))
    return st;
  const Rows outs[] = {rd, g0, g1, span(ws, (int64_t)ws_bytes)}, ins[] = {rx, rg, ru, rh, w0, w1};
  if (any_share(outs, ins) || any_share({outs[3]}, {rd, g0, g1})) return MOE_ERR_INVALID_ARG;
  if (share(rd, g0) || share(rd, g1) || share(g0, g1)) return MOE_ERR_INVALID_ARG;
  const FfnWs w = ffn_ws_for(f, C, true);
  if (!ws || (uintptr_t)ws % 256 || ws_bytes < w.total) return MOE_ERR_WORKSPACE;
  FArgs a = {};
  ffn_args(f, x, x_pitch, C, a);
  GArgs g = {};
  g.C = C; g.I = f->inter; g.act = act_constants(f->act);
  g.gate = static_cast<const uint8_t*>(gate); g.gate_pitch = gate_pitch * s;
  g.up = static_cast<const uint8_t*>(up); g.up_pitch = up_pitch * s;
  g.dh = static_cast<const uint8_t*>(dh); g.dh_pitch = dh_pitch * s;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  hipStream_t q = reinterpret_cast<hipStream_t>(stream);
  auto go = [&](auto dt) {
    return ffn_backward<decltype(dt)::value>(f, a, g, static_cast<uint8_t*>(dx), dx_pitch * s, static_cast<uint8_t*>(dw_gate),
                                             dw_gate_pitch * gs, static_cast<uint8_t*>(dw_up), dw_up_pitch * gs,
                                             grad_dtype == MOE_DT_F32, accumulate, w, w8, q);
  };
  st = f->dtype == MOE_DT_F32    ? go(std::integral_constant<int, MOE_DT_F32>())
       : f->dtype == MOE_DT_BF16 ? go(std::integral_constant<int, MOE_DT_BF16>())
                                 : go(std::integral_constant<int, MOE_DT_F16>());
  if (st != MOE_OK) return st;
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // extern "C"
