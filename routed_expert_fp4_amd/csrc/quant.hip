// libroutedfp4, dense matrices in 4-bit codes with group scales:
//
//   y[c][n] = sum_k x[c][k] W[n][k],   W[n][k] = s[n][g] (q[n][k] - z[n][g]),  g = k / G
//           = sum_g s[n][g] * ( sum_{k in g} x[c][k] (q[n][k] - z[n][g]) )
//
// The inner sums run on the fp16 matrix cores (16x16x32): q - z is an integer
// of at most 8 bits, exact in fp16, and x enters as fp16 terms, so every
// product is exact and only fp32 sums round; the group's scale multiplies its
// fp32 sum.  fp16 x is taken as it is.  bf16 x (8 bits) is one fp16 term under
// a power of two per token that puts the token's largest value below 2^15:
// exact down to 2^-28 of that value, and off by at most 2^-38 of it below.
// fp32 x is two such terms (22 bits): a third would make half as many matrix
// instructions again, for an error that fp32 sums cover (7168 columns against 64
// bits: 1e-7, a library's fp32 product 7e-7).
//
// Codes become fp16 without conversions: a nibble OR-ed into the fp16 1024 is
// 1024 + q, one in the next four bits of the fp16 64 is 64 + q, and one packed
// subtraction each takes 1024 + z or 64 + z away exactly: 9 instructions for 8
// codes.  That leaves x's columns in the order 0 4 1 5 2 6 3 7, in which its
// terms are laid out too.
//
// Lane l of a wave holds, of a 16-row tile, row l % 16 and one 16-byte unit
// (32 columns) of each 128-column chunk, unit l / 16.  Groups of 128 or more
// columns (G % 128 == 0) then need no exchange: product j of a chunk takes
// dword j of every unit.  For G 32 and 64 a 4x4 transpose over the lane
// quarters (four permlane swaps) first gives product j the whole of unit j,
// so that its sum lies inside one group.
//
// Kernels:
//   k_qone     one token: bound by reading the codes; its terms are made in LDS
//              by every workgroup, whose waves split the rows, the columns of
//              a row tile, or both
//   k_qfew     2 .. 16 tokens: workgroups take rows x column slices, make the
//              slice's terms in LDS and stream its codes; the last of a group
//              of rows to finish adds the ranges of slices
//   k_qterms   x to fp16 terms in the workspace, in the operand order
//   k_qgemm    17 and more tokens: workgroup tiles of tokens x rows, x's terms
//              through LDS (loaded there directly, three buffers), the codes
//              from memory to registers; k_qreduce adds split column ranges
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <limits.h>

#include "common.h"

namespace rf4 {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

constexpr int kQChunk = 128;          // columns per chunk: 64 bytes of a row's codes
constexpr int kQWG = 512;             // threads of the stream and matrix kernels
constexpr int kQWaves = kQWG / 64;
constexpr int kQTermBytes = 4096;     // terms of 16 tokens x 128 columns
constexpr int kQStageBytes = 49152;   // LDS for one token's terms

struct QArgs {
  const uint8_t* codes;
  int64_t code_pitch;
  const uint8_t* scales;
  int64_t scale_pitch;                // bytes
  const uint8_t* zeros;
  int64_t zero_pitch;
  int zero_step;                      // 0 where one byte (8) serves every group
  int scale_bf16;                     // 16-bit scales: bf16, else fp16
  int scales_vec;                     // G 32, 64: a chunk's scales and zero points can be loaded together
  int N, K;
  int units;                          // 16-byte units of a row
  int nch;                            // chunks of a row
  int ng;                             // groups of a row
  int gshift;                         // G 32, 64: log2 G
  uint32_t gmul;                      // G >= 128: group of chunk c = (c * gmul) >> 20
  const void* x;
  int64_t x_pitch;
  int x_dt, x_vec;                    // x_vec: rows are 16-byte aligned
  int C;
  void* y;
  int64_t y_pitch;
  int y_vec;                          // rows of y are aligned to four of its elements
  int accumulate;
  float* inv;                         // [C]: takes the terms' power of two out again; a token
                                      // that is not finite: -1 (its terms are not scaled)
  uint8_t* terms;                     // [P][C / 16][nch][16 blocks][16 tokens][16 bytes]
  float* part;                        // [splits][C][N]
  uint32_t* tickets;                  // few tokens: arrivals per group of rows, left at zero
  int ks, spt;                        // one token: 2^ks waves to a row tile, steps per tile
  int splits, per_split;              // matrix kernel: column ranges, chunks in each
  int row_groups;                     // one token: groups of row tiles; matrix kernel: row tiles
};

__device__ const uint8_t kEight[16] = {8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8};

// Token t of a 16-token tile is row 4 (t % 4) + t / 4 of the first operand, so
// that up to 4 tokens need one result register (row 4 (l / 16) + r is register
// r of lane l), up to 8 two.
__device__ __forceinline__ int token_row(int t) { return 4 * (t & 3) + (t >> 2); }
__device__ __forceinline__ int row_token(int r) { return (r >> 2) + 4 * (r & 3); }

// ---------------------------------------------------------------------------
// Codes
// ---------------------------------------------------------------------------
// A wave's view of the codes, scales and zero points of the rows from n0 on:
// buffer loads whose row and unit are a per-lane offset, and whose tile and
// chunk are a scalar one.  Offsets past the last row's last unit read zeros.
struct View {
  __amdgpu_buffer_rsrc_t codes, scales, zeros;
  uint32_t vc, vs, vz;      // per-lane offsets: row (and, for codes, unit)
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t qview(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

template <int SS>
__device__ __forceinline__ View view_rows(const QArgs& a, int n0, int rows, int row, int quarter) {
  View v;
  int left = a.N - n0 < rows ? a.N - n0 : rows;
  if (left < 1) { left = 1; n0 = a.N - 1; }
  v.codes = qview(a.codes + (int64_t)n0 * a.code_pitch, (int64_t)(left - 1) * a.code_pitch + 16 * a.units);
  v.scales = qview(a.scales + (int64_t)n0 * a.scale_pitch, (int64_t)(left - 1) * a.scale_pitch + SS * a.ng);
  v.zeros = a.zeros ? qview(a.zeros + (int64_t)n0 * a.zero_pitch, (int64_t)(left - 1) * a.zero_pitch + a.ng)
                    : qview(kEight, sizeof(kEight));
  v.vc = (uint32_t)(row * a.code_pitch) + 16u * quarter;
  v.vs = (uint32_t)(row * a.scale_pitch);
  v.vz = (uint32_t)(row * a.zero_pitch);
  return v;
}

constexpr uint32_t kOutside = 0x80000000u;   // an offset past every view of 16 rows

// N (up to 4) of a wave's chunks, c, c + step, ...: codes, and as stored the
// scales and zero points of all of them, for which a lane reads not its own
// unit's but those of chunk number `quarter` (G >= 128: one; TR: of the
// chunk's four units).  A load of one scale per row touches a cache line per
// row, and the lines are gone by the row's next chunk; so each is touched once
// for four chunks.
template <int N, bool TR>
struct Quad {
  static constexpr int S = TR ? 4 : 1;
  uint4v q[N];
  uint32_t s[S], z[S];
};

// Units past the last column read what lies there (a code is finite, and x is
// zero); their scale is 0, since what lies behind a row of scales may be no
// number, and the last group's may be infinite.  Chunks from nch on (or live false) are not read.
// The loads are always issued, so that the count of loads in flight is the
// same on every path and a wait for one step's codes leaves the next step's in
// flight.
// Codes are not loaded as non-temporal, though a call reads them once: 64 bytes
// of a row are half a cache line, and the other half is the next chunk's (65536
// x 7168, one token: 58.5 us non-temporal, 52.6 not).
template <int N, bool TR, int SS>
__device__ __forceinline__ void load_quad(const QArgs& a, const View& v, int c, int step, int quarter, bool live,
                                          Quad<N, TR>& u) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int ci = c + step * i;
    u.q[i] = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(
        v.codes, (int)(v.vc | (live && ci < a.nch ? 0u : kOutside)), 64 * ci, 0));
  }
  int cq = c + step * (quarter < N ? quarter : N - 1);
  cq = cq < a.nch ? cq : a.nch - 1;
  const uint32_t out = live ? 0u : kOutside;
  if (TR && a.scales_vec) {
    // the chunk's four (G 32) or two scales and zero points in one load each
    // (the zero points' first: what follows waits for the scales)
    if (a.gshift == 5) {
      const int os = (int)((v.vs + 4 * SS * cq) | out);
      const uint32_t z = __builtin_amdgcn_raw_buffer_load_b32(v.zeros, (int)((v.vz + 4 * a.zero_step * cq) | out), 0, 0);
      if (SS == 4) {
        const auto s = __builtin_amdgcn_raw_buffer_load_b128(v.scales, os, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < Quad<N, TR>::S; ++e) u.s[e] = s[e];
      } else {
        const auto s = __builtin_amdgcn_raw_buffer_load_b64(v.scales, os, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < Quad<N, TR>::S; ++e) u.s[e] = (e & 1) ? s[e >> 1] >> 16 : s[e >> 1] & 0xFFFFu;
      }
#pragma unroll
      for (int e = 0; e < Quad<N, TR>::S; ++e) u.z[e] = (z >> (8 * e)) & 0xFFu;
    } else {
      const int os = (int)((v.vs + 2 * SS * cq) | out);
      const uint32_t z = __builtin_amdgcn_raw_buffer_load_b16(v.zeros, (int)((v.vz + 2 * a.zero_step * cq) | out), 0, 0);
      if (SS == 4) {
        const auto s = __builtin_amdgcn_raw_buffer_load_b64(v.scales, os, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < Quad<N, TR>::S; ++e) u.s[e] = s[e >> 1];
      } else {
        const uint32_t s = __builtin_amdgcn_raw_buffer_load_b32(v.scales, os, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < Quad<N, TR>::S; ++e) u.s[e] = e >> 1 ? s >> 16 : s & 0xFFFFu;
      }
#pragma unroll
      for (int e = 0; e < Quad<N, TR>::S; ++e) u.z[e] = e >> 1 ? z >> 8 : z & 0xFFu;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < Quad<N, TR>::S; ++e) {
    int g = TR ? (4 * cq + e) >> (a.gshift - 5) : (int)(((uint32_t)cq * a.gmul) >> 20);
    const uint32_t skip = TR && 4 * cq + e >= a.units ? kOutside : out;
    if (SS == 4) u.s[e] = __builtin_amdgcn_raw_buffer_load_b32(v.scales, (int)((v.vs + SS * g) | skip), 0, 0);
    else u.s[e] = __builtin_amdgcn_raw_buffer_load_b16(v.scales, (int)((v.vs + SS * g) | skip), 0, 0);
    u.z[e] = __builtin_amdgcn_raw_buffer_load_b8(v.zeros, (int)((v.vz + a.zero_step * g) | skip), 0, 0);
  }
}

template <int SS>
__device__ __forceinline__ float scale_of(int bf16, uint32_t s) {
  if (SS == 4) return __uint_as_float(s);
  // both readings and a mask: a branch would cost more
  const uint32_t h = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)s));
  const uint32_t b = bf16 ? 0xFFFFFFFFu : 0u;
  return __uint_as_float(((s << 16) & b) | (h & ~b));
}

__device__ __forceinline__ half2v as_half2(uint32_t v) { return __builtin_bit_cast(half2v, v); }

// zero points as the fp16 pair (1024 + z, 64 + z)
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
  const _Float16 h = (_Float16)(float)(64u + z);
  return (0x6400u | z) | ((uint32_t)__builtin_bit_cast(uint16_t, h) << 16);
}

// The unpacking constants, one pair in scalar and one in vector registers: an
// AND-OR takes at most one scalar and no literal, and the compiler, left to
// itself, uses literals and two instructions.
struct Magic {
  uint32_t m0, m1, k1024, k64;
};
__device__ __forceinline__ Magic magic() {
  Magic k;
  asm("s_mov_b32 %0, 0x000f000f" : "=s"(k.m0));
  asm("s_mov_b32 %0, 0x00f000f0" : "=s"(k.m1));
  asm("v_mov_b32 %0, 0x64006400" : "=v"(k.k1024));
  asm("v_mov_b32 %0, 0x54005400" : "=v"(k.k64));
  return k;
}

// eight codes as q - z in the column order 0 4 1 5 2 6 3 7
__device__ __forceinline__ half8 unpack8(const Magic& k, uint32_t d, uint32_t zp) {
  const half2v z = as_half2(zp);
  const half2v z0 = {z[0], z[0]}, z1 = {z[1], z[1]};
  const uint32_t e = d >> 8;
  const half2v t0 = as_half2((d & k.m0) | k.k1024) - z0;
  const half2v t1 = as_half2((d & k.m1) | k.k64) - z1;
  const half2v t2 = as_half2((e & k.m0) | k.k1024) - z0;
  const half2v t3 = as_half2((e & k.m1) | k.k64) - z1;
  return half8{t0[0], t0[1], t1[0], t1[1], t2[0], t2[1], t3[0], t3[1]};
}

__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0]; b = r[1];
}
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0]; b = r[1];
}
// d[j] of lane quarter q <- d[q] of lane quarter j
__device__ __forceinline__ void transpose4(uint32_t (&d)[4]) {
  swap16(d[0], d[1]);
  swap16(d[2], d[3]);
  swap32(d[0], d[2]);
  swap32(d[1], d[3]);
}
// v of quarter j, in every quarter, as o[j]
__device__ __forceinline__ void spread4(uint32_t v, uint32_t (&o)[4]) {
  o[0] = v; o[2] = v;
  swap32(o[0], o[2]);
  o[1] = o[0]; o[3] = o[2];
  swap16(o[0], o[1]);
  swap16(o[2], o[3]);
}

// The scales and zero pairs of a quad: of chunk i in s[i], z[i], for TR those
// of the lane's own unit.
template <int N, bool TR, int SS>
__device__ __forceinline__ void quad_scales(const QArgs& a, const Quad<N, TR>& u, uint32_t (&s)[4], uint32_t (&z)[4]) {
  if (TR) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] = __float_as_uint(scale_of<SS>(a.scale_bf16, u.s[e]));
      z[e] = zero_pair(u.z[e]);
    }
    transpose4(s);
    transpose4(z);
  } else {
    spread4(__float_as_uint(scale_of<SS>(a.scale_bf16, u.s[0])), s);
    spread4(zero_pair(u.z[0]), z);
  }
}

__device__ __forceinline__ float4v mma(half8 x, half8 w, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w, c, 0, 0, 0);
}

// The block (of 8 columns, 16 in a chunk) that product j takes in quarter q.
template <bool TR>
__device__ __forceinline__ int block_of(int j, int q) { return TR ? 4 * j + q : 4 * q + j; }

// ---------------------------------------------------------------------------
// Activations as fp16 terms
// ---------------------------------------------------------------------------
// The power of two that takes a token's largest |x| (fp32 bits) below 2^15,
// within fp32's normal range, and its inverse.  Infinity or NaN: 1.
__device__ __forceinline__ void term_scale(uint32_t maxbits, float& m, float& inv) {
  int e = 14 - ((int)(maxbits >> 23) - 127);
  if (maxbits >= 0x7F800000u) e = 0;
  e = e > 126 ? 126 : e;
  m = __uint_as_float((uint32_t)(127 + e) << 23);
  inv = __uint_as_float((uint32_t)(127 - e) << 23);
}

// v (scaled) as hi + lo.  A token with an infinity or NaN is not scaled: its
// finite values are held within fp16's range (its results are infinite or NaN
// whatever they are), and the infinity itself has no second term.
template <bool FINITE>
__device__ __forceinline__ void split_term(float v, _Float16& hi, _Float16& lo) {
  if (!FINITE && fabsf(v) < INFINITY) v = fminf(fmaxf(v, -65504.0f), 65504.0f);
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
  if (!FINITE && !(fabsf(v) < INFINITY)) lo = (_Float16)0.0f;
}

// Eight columns of a row of x as stored (0 past the last column), through a
// buffer view of x whose loads outside it give zeros: 16 bytes at a time
// (load8v) where every row starts 16-byte aligned, else element by element.
template <int DT>
struct Raw { uint4v v[DT == MOE_DT_F32 ? 2 : 1]; };

template <int DT>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t x_view(const QArgs& a, int t, int rows) {
  constexpr int B = DT == MOE_DT_F32 ? 4 : 2;
  return qview(static_cast<const uint8_t*>(a.x) + (int64_t)t * a.x_pitch * B, ((rows - 1) * a.x_pitch + a.K) * B);
}
template <int DT>
__device__ __forceinline__ void load8e(const QArgs& a, __amdgpu_buffer_rsrc_t x, uint32_t row, int k, bool live,
                                       Raw<DT>& r) {
  constexpr int B = DT == MOE_DT_F32 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t o = live && k + i < a.K ? row + (uint32_t)((k + i) * B) : kOutside;
    if (DT == MOE_DT_F32) {
      r.v[i >> 2][i & 3] = __builtin_amdgcn_raw_buffer_load_b32(x, (int)o, 0, 0);
    } else {
      const uint32_t h = __builtin_amdgcn_raw_buffer_load_b16(x, (int)o, 0, 0);
      r.v[0][i >> 1] = (i & 1) ? r.v[0][i >> 1] | (h << 16) : h;
    }
  }
}
template <int DT>
__device__ __forceinline__ void load8v(const QArgs& a, __amdgpu_buffer_rsrc_t x, uint32_t row, int k, bool live,
                                       Raw<DT>& r) {
  constexpr int B = DT == MOE_DT_F32 ? 4 : 2;
  const uint32_t o = live && k + 8 <= a.K ? row + (uint32_t)(k * B) : kOutside;
#pragma unroll
  for (int i = 0; i < B / 2; ++i)
    r.v[i] = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(x, (int)(o + 16 * i), 0, 0));
  if (live && k < a.K && k + 8 > a.K) load8e<DT>(a, x, row, k, live, r);   // a row's last columns
}
template <int DT>
__device__ __forceinline__ void load8(const QArgs& a, __amdgpu_buffer_rsrc_t x, uint32_t row, int k, bool live,
                                      Raw<DT>& r) {
  if (a.x_vec) load8v<DT>(a, x, row, k, live, r);
  else load8e<DT>(a, x, row, k, live, r);
}

template <int DT>
__device__ __forceinline__ float raw_f32(const Raw<DT>& r, int i) {
  if (DT == MOE_DT_F32) return __uint_as_float(r.v[i >> 2][i & 3]);
  const uint32_t w = r.v[0][i >> 1];
  return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);        // bf16
}

// The largest |x| so far as fp32 bits (NaN above infinity above the rest).
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint32_t raw_max(const Raw<DT>& r, uint32_t m) {
  if (DT == MOE_DT_BF16) {
    // pairs of bf16: their bits rise with |x|
    ushort2v p = __builtin_bit_cast(ushort2v, r.v[0][0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i)
      p = __builtin_elementwise_max(p, __builtin_bit_cast(ushort2v, r.v[0][i] & 0x7FFF7FFFu));
    const uint32_t b = (uint32_t)(p[0] > p[1] ? p[0] : p[1]) << 16;
    return b > m ? b : m;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(raw_f32<DT>(r, i)) & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
  return m;
}

// The block's terms in the operand order.  Tokens that are not finite are set
// apart by a branch of the wave: selecting in every element cost as much as the
// split itself.
template <int DT, bool FINITE>
__device__ __forceinline__ void make_terms_of(const Raw<DT>& r, float m, half8& hi, half8& lo) {
  constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
  if (DT == MOE_DT_BF16 && FINITE) {
    // two at a time, toward zero: exact wherever fp16 is normal
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto h = __builtin_amdgcn_cvt_pkrtz(raw_f32<DT>(r, i) * m, raw_f32<DT>(r, i + 4) * m);
      hi[2 * i] = h[0];
      hi[2 * i + 1] = h[1];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = order[i];
    if (DT == MOE_DT_F16) {
      const uint32_t w = r.v[0][k >> 1];
      hi[i] = __builtin_bit_cast(_Float16, (uint16_t)((k & 1) ? w >> 16 : w));
    } else {
      _Float16 h, l;
      split_term<FINITE>(raw_f32<DT>(r, k) * m, h, l);
      hi[i] = h;
      if (DT == MOE_DT_F32) lo[i] = l;
    }
  }
}
template <int DT>
__device__ __forceinline__ void make_terms(const Raw<DT>& r, float m, bool finite, half8& hi, half8& lo) {
  if (DT == MOE_DT_F16 || __ballot(!finite) == 0) make_terms_of<DT, true>(r, m, hi, lo);
  else make_terms_of<DT, false>(r, m, hi, lo);
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, m, 64);
    v = o > v ? o : v;
  }
  return v;
}

// Four tokens whose operand rows are next to each other (t, t + 4, t + 8,
// t + 12 of a tile), so that four lanes write 64 contiguous bytes: their
// largest values, then their terms.  NB blocks of 8 columns a thread (0: any
// number): the rows, up to 8192 or 16384 columns, stay in registers between the
// two, else they are read twice (2048 tokens x 7168 in fp32: 12 us more; 64
// unaligned tokens x 10001: 11.6 us, 9.0 in registers).
constexpr int kTermWG = 1024, kTermBlocks = kTermWG / 4;
template <int DT, int NB>
__global__ __launch_bounds__(kTermWG) void k_qterms(QArgs a) {
  constexpr int B = DT == MOE_DT_F32 ? 4 : 2;
  constexpr bool FITS = NB > 0;
  __shared__ uint32_t s_max[kTermWG / 64][4];
  const int tid = threadIdx.x, lane = tid & 63, k = tid & 3;
  const int t0 = blockIdx.x / 4 * 16, t = t0 + blockIdx.x % 4 + 4 * k;
  const bool live = t < a.C;
  const int nblk = a.nch * (kQChunk / 8);
  const __amdgpu_buffer_rsrc_t x = x_view<DT>(a, t0, a.C - t0 < 16 ? a.C - t0 : 16);
  const uint32_t row = (uint32_t)((t - t0) * (int)a.x_pitch * B);
  float m = 1.0f, inv = 1.0f;
  bool finite = true;
  Raw<DT> r[FITS ? NB : 1];
  if (FITS) {
#pragma unroll
    for (int i = 0; i < NB; ++i) load8<DT>(a, x, row, 8 * ((tid >> 2) + kTermBlocks * i), live, r[i]);
  }
  if (DT != MOE_DT_F16) {
    uint32_t mx = 0;
    if (FITS) {
#pragma unroll
      for (int i = 0; i < NB; ++i) mx = raw_max<DT>(r[i], mx);
    } else {
      for (int b = tid >> 2; b < nblk; b += kTermBlocks) {
        load8<DT>(a, x, row, 8 * b, live, r[0]);
        mx = raw_max<DT>(r[0], mx);
      }
    }
#pragma unroll
    for (int w = 4; w < 64; w <<= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)mx, w, 64);
      mx = o > mx ? o : mx;
    }
    if (lane < 4) s_max[tid >> 6][lane] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTermWG / 64; ++w) mx = s_max[w][k] > mx ? s_max[w][k] : mx;
    term_scale(mx, m, inv);
    finite = mx < 0x7F800000u;
  }
  if (!live) return;
  if (tid < 4) a.inv[t] = finite ? inv : -1.0f;
  const int ct = (a.C + 15) / 16;
  const int64_t plane = (int64_t)ct * a.nch * kQTermBytes;
  uint8_t* out = a.terms + (int64_t)(t >> 4) * a.nch * kQTermBytes + token_row(t & 15) * 16;
  auto write = [&](int b, const Raw<DT>& v) {
    half8 hi, lo;
    make_terms<DT>(v, m, finite, hi, lo);
    *reinterpret_cast<half8*>(out + (int64_t)b * 256) = hi;
    if (DT == MOE_DT_F32) *reinterpret_cast<half8*>(out + plane + (int64_t)b * 256) = lo;
  };
  if (FITS) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int b = (tid >> 2) + kTermBlocks * i;
      if (b < nblk) write(b, r[i]);
    }
  } else {
    for (int b = tid >> 2; b < nblk; b += kTermBlocks) {
      load8<DT>(a, x, row, 8 * b, live, r[0]);
      write(b, r[0]);
    }
  }
}

// ---------------------------------------------------------------------------
// Results
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void put(const QArgs& a, int t, int n, float v) {
  const int64_t i = (int64_t)t * a.y_pitch + n;
  if (DT == MOE_DT_F32) {
    float* y = static_cast<float*>(a.y) + i;
    *y = a.accumulate ? *y + v : v;
  } else if (DT == MOE_DT_BF16) {
    __hip_bfloat16* y = static_cast<__hip_bfloat16*>(a.y) + i;
    *y = __float2bfloat16(a.accumulate ? __bfloat162float(*y) + v : v);
  } else {
    __half* y = static_cast<__half*>(a.y) + i;
    *y = __float2half(a.accumulate ? __half2float(*y) + v : v);
  }
}
__device__ __forceinline__ void put(const QArgs& a, int t, int n, float v) {
  if (a.x_dt == MOE_DT_F32) put<MOE_DT_F32>(a, t, n, v);
  else if (a.x_dt == MOE_DT_BF16) put<MOE_DT_BF16>(a, t, n, v);
  else put<MOE_DT_F16>(a, t, n, v);
}

// Four results of a token, rows n .. n + 3 (n % 4 == 0).
template <int DT>
__device__ __forceinline__ void put4(const QArgs& a, int t, int n, float4 v) {
  if (a.y_vec && n + 3 < a.N && !a.accumulate) {
    const int64_t i = (int64_t)t * a.y_pitch + n;
    if (DT == MOE_DT_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.y) + i) = v;
    } else if (DT == MOE_DT_BF16) {
      const __hip_bfloat16 h[4] = {__float2bfloat16(v.x), __float2bfloat16(v.y), __float2bfloat16(v.z),
                                   __float2bfloat16(v.w)};
      __builtin_memcpy(__builtin_assume_aligned(static_cast<__hip_bfloat16*>(a.y) + i, 8), h, 8);
    } else {
      const __half h[4] = {__float2half(v.x), __float2half(v.y), __float2half(v.z), __float2half(v.w)};
      __builtin_memcpy(__builtin_assume_aligned(static_cast<__half*>(a.y) + i, 8), h, 8);
    }
    return;
  }
  const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) put<DT>(a, t, n + i, e[i]);
}
__device__ __forceinline__ void put4(const QArgs& a, int t, int n, float4 v) {
  if (a.x_dt == MOE_DT_F32) put4<MOE_DT_F32>(a, t, n, v);
  else if (a.x_dt == MOE_DT_BF16) put4<MOE_DT_BF16>(a, t, n, v);
  else put4<MOE_DT_F16>(a, t, n, v);
}

// ---------------------------------------------------------------------------
// Results beyond the scaled sums' range
// ---------------------------------------------------------------------------
// The sums are scaled while their activations are raised to just below 2^15, and
// the token's power of two is taken out last.  Very small activations (raised by
// up to 2^126) against very large scales so leave fp32's range with a result
// inside it.  Every kernel looks at its results, and where one of a finite token
// is not finite this forms its columns k0 (a chunk's first) to k1 - 1 anew, in 64
// bits: fp32 inputs neither overflow nor vanish there, and what is still infinite
// or NaN comes of infinite scales or of a sum past fp32.  Folding the power into
// the scale instead would lose small scales, and doing so per token would cost a
// product per result and group.
//
// The arguments are read from the kernel's own argument segment (every kernel has
// QArgs first), by a pointer that the compiler cannot see through: kept in scalar
// registers over the whole kernel for this they took those of its loop.
typedef const __attribute__((address_space(4))) QArgs* QArgsPtr;
__device__ __forceinline__ QArgsPtr args_again() {
  QArgsPtr a = (QArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  return a;
}
__device__ __forceinline__ double readlane_f64(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, readlane_u64(u, l));
}
// Result (t, n), the same in every lane that is active, by all of these together:
// one column after the other a lane took 0.5 ms for 7168 of them.
template <int DT, bool TR, int SS>
__device__ __forceinline__ float sum_in_f64(int t, int n, int k0, int k1) {
  const QArgsPtr a = args_again();
  const uint8_t* code = a->codes + (int64_t)n * a->code_pitch;
  const uint8_t* scale = a->scales + (int64_t)n * a->scale_pitch;
  const uint8_t* zero = a->zeros ? a->zeros + (int64_t)n * a->zero_pitch : nullptr;
  const int64_t row = (int64_t)t * a->x_pitch;
  const bool wide = DT == 0 ? a->x_dt == MOE_DT_F32 : DT == MOE_DT_F32;
  k1 = k1 < a->K ? k1 : a->K;
  const uint64_t on = __ballot(1);
  const int lanes = __popcll(on), rank = __popcll(on & ((1ull << (threadIdx.x & 63)) - 1ull));
  auto total = [&](double v) {                             // in the order of the lanes
    double sum = 0.0;
    for (uint64_t m = on; m; m &= m - 1) sum += readlane_f64(v, __ffsll((long long)m) - 1);
    return sum;
  };
  auto group = [&](int k) { return TR ? k >> a->gshift : (int)(((uint32_t)(k / kQChunk) * a->gmul) >> 20); };
  auto scale_at = [&](int k) {
    const int g = group(k);
    const uint32_t s = SS == 4 ? reinterpret_cast<const uint32_t*>(scale)[g] : reinterpret_cast<const uint16_t*>(scale)[g];
    return scale_of<SS>(a->scale_bf16, s);
  };
  auto eight = [&](int k, int end) {                       // columns k .. k + 7, one group
    const uint32_t q = *reinterpret_cast<const uint32_t*>(code + k / 2);   // up to the end of a 16-byte unit
    const int z = zero ? zero[group(k)] : 8;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = row + (k + i < end ? k + i : end - 1);
      const float x = wide ? static_cast<const float*>(a->x)[at]
                           : __uint_as_float((uint32_t)static_cast<const uint16_t*>(a->x)[at] << 16);
      if (k + i < end) sum += (double)x * (double)((int)((q >> (4 * i)) & 15u) - z);
    }
    return sum;
  };
  double y = 0.0;
  // infinite and NaN scales first, each times its group's sum (of a chunk, in
  // groups of several): beside them the other groups make no difference
  bool only = false;
  const int step = TR ? 1 << a->gshift : kQChunk;
#pragma unroll 1
  for (int base = k0; base < k1; base += step * lanes) {
    const int k = base + step * rank;
    const float s = k < k1 ? scale_at(k) : 0.0f;
#pragma unroll 1
    for (uint64_t m = __ballot(!(fabsf(s) < INFINITY)); m; m &= m - 1) {
      const int l = __ffsll((long long)m) - 1, kb = __builtin_amdgcn_readlane(k, l);
      const int end = kb + step < k1 ? kb + step : k1;
      double sum = 0.0;
#pragma unroll 1
      for (int c = kb + 8 * rank; c < end; c += 8 * lanes) sum += eight(c, end);
      y += (double)__int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), l)) * total(sum);
      only = true;
      if (y != y) return (float)y;
    }
  }
  if (only) return (float)y;
#pragma unroll 1
  for (int k = k0 + 8 * rank; k < k1; k += 8 * lanes) y += (double)scale_at(k) * eight(k, k1);
  return (float)total(y);
}
// v unless it has left the range (`spoilt`: the token is not finite; asked only
// then).  fp16 activations are not raised: theirs stays.  DT 0: as the call says.
// The branch is the wave's: one scalar test where nothing has.
template <int DT, bool TR, int SS, class F>
__device__ __forceinline__ float in_range(float v, F spoilt, int t, int n, int k0, int k1) {
  if (DT == MOE_DT_F16) return v;
  const bool left = !(fabsf(v) < INFINITY);
  if (__builtin_expect(__ballot(left) != 0, 0)) {
#pragma unroll 1
    for (uint64_t m = __ballot(left && !spoilt()); m; m &= m - 1) {
      const int l = __ffsll((long long)m) - 1;
      const float y = sum_in_f64<DT, TR, SS>(__builtin_amdgcn_readlane(t, l), __builtin_amdgcn_readlane(n, l), k0, k1);
      if ((int)(threadIdx.x & 63) == l) v = y;
    }
  }
  return v;
}

// ---------------------------------------------------------------------------
// One unit's four products
// ---------------------------------------------------------------------------
// acc[r] += a chunk's scaled sums; frag(p, j) gives x's term p of product j.
// The terms' sums are chains of their own: none waits for the other.
template <int P, int NR, bool TR, class F>
__device__ __forceinline__ void multiply(const Magic& mg, uint4v q, uint32_t s, uint32_t z, F frag, float (&acc)[NR]) {
  uint32_t d[4] = {q[0], q[1], q[2], q[3]}, sj[4], zj[4];
  if (TR) {
    transpose4(d);
    spread4(s, sj);
    spread4(z, zj);
  }
  float4v sum[P];
#pragma unroll
  for (int p = 0; p < P; ++p) sum[p] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const half8 b = unpack8(mg, d[j], TR ? zj[j] : z);
#pragma unroll
    for (int p = 0; p < P; ++p) sum[p] = mma(frag(p, j), b, TR ? float4v{0.0f, 0.0f, 0.0f, 0.0f} : sum[p]);
    if (TR || j == 3) {
      const float f = __uint_as_float(TR ? sj[j] : s);
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[r] += f * (P == 2 ? sum[0][r] + sum[P - 1][r] : sum[0][r]);
    }
  }
}

// ---------------------------------------------------------------------------
// One token
// ---------------------------------------------------------------------------
// The workgroup makes the token's terms in LDS ([P][blocks] of 16 bytes) while
// the first codes are on their way (x's loads are issued before theirs: loads
// complete in order).  It takes kQWaves >> ks tiles of 16 rows at a time, 2^ks
// waves to a tile; a wave walks its tile's chunks kw, kw + 2^ks, ... in steps
// of eight, each quad's next step loaded as soon as it is multiplied, on into
// the next tile.  Short code matters here as much as bytes: a call for a few
// thousand rows lasts about as long as fetching a straight-line kernel does.
// 65536 x 7168: 49 us, 4.9 TB/s, bound by that read; 3584 x 7168: 7.7 us, bound
// by latencies (launch, x, terms, one step of codes, the waves' sum).
template <int DT, bool TR, int SS>
__global__ __launch_bounds__(kQWG, 2) void k_qone(QArgs a) {
  constexpr int P = DT == MOE_DT_F32 ? 2 : 1;
  constexpr int NB = kQStageBytes / (16 * P) / kQWG;      // blocks per thread at most
  extern __shared__ __align__(16) uint8_t s_x[];
  __shared__ float s_red[2][kQWaves * 16];
  __shared__ uint32_t s_max[kQWaves];
  // the wave's number through readfirstlane: its tiles and chunks are scalars
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int row = lane & 15, quarter = lane >> 4;
  const int ks = a.ks, wk = 1 << ks, kw = wave & (wk - 1), tw = wave >> ks, tiles = kQWaves >> ks;
  const int nblk = a.nch * (kQChunk / 8);

  Raw<DT> raw[NB];
  const __amdgpu_buffer_rsrc_t xv = x_view<DT>(a, 0, 1);
  if (a.x_vec) {
#pragma unroll
    for (int i = 0; i < NB; ++i) load8v<DT>(a, xv, 0, 8 * (tid + kQWG * i), true, raw[i]);
  }
  __builtin_amdgcn_sched_barrier(0);

  // the codes of one step: step ld_i of the workgroup's ld_g-th tile group
  int ld_g = blockIdx.x, ld_i = 0;
  View v = view_rows<SS>(a, (ld_g * tiles + tw) * 16, 16, row, quarter);
  Quad<4, TR> u[2];
  auto load = [&](int k) {
    load_quad<4, TR, SS>(a, v, kw + ((8 * ld_i + 4 * k) << ks), wk, quarter, ld_g < a.row_groups, u[k]);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto advance = [&]() {
    if (++ld_i == a.spt) {
      ld_i = 0;
      ld_g += gridDim.x;
      v = view_rows<SS>(a, (ld_g * tiles + tw) * 16, 16, row, quarter);
    }
  };
  const Magic mg = magic();
  load(0);
  load(1);
  advance();

  float m = 1.0f, inv = 1.0f;
  bool finite = true;
  if (DT != MOE_DT_F16) {
    uint32_t mx = 0;
    if (a.x_vec) {
#pragma unroll
      for (int i = 0; i < NB; ++i) mx = raw_max<DT>(raw[i], mx);
    } else {
      for (int b = tid; b < nblk; b += kQWG) {
        load8e<DT>(a, xv, 0, 8 * b, true, raw[0]);
        mx = raw_max<DT>(raw[0], mx);
      }
    }
    mx = wave_umax(mx);
    if (lane == 0) s_max[wave] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQWaves; ++w) mx = s_max[w] > mx ? s_max[w] : mx;
    term_scale(mx, m, inv);
    finite = mx < 0x7F800000u;
    inv = finite ? inv : -inv;                            // its sign is kept for the results
  }
  auto write = [&](int b, const Raw<DT>& r) {
    half8 hi, lo;
    make_terms<DT>(r, m, finite, hi, lo);
    *reinterpret_cast<half8*>(s_x + 16 * b) = hi;
    if (P == 2) *reinterpret_cast<half8*>(s_x + 16 * (nblk + b)) = lo;
  };
  if (a.x_vec) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (tid + kQWG * i < nblk) write(tid + kQWG * i, raw[i]);
  } else {
    for (int b = tid; b < nblk; b += kQWG) {
      load8e<DT>(a, xv, 0, 8 * b, true, raw[0]);
      write(b, raw[0]);
    }
  }
  __syncthreads();

  int parity = 0;
  // bit i: this thread's result in the workgroup's i-th tile group left the range
  // (at most 64 of them: 2^22 rows over 512 workgroups of 128)
  uint64_t left = 0, bit = 1;
  for (int cg = blockIdx.x; cg < a.row_groups; cg += gridDim.x, bit <<= 1) {
    float acc[1] = {0.0f};
    for (int ci = 0; ci < a.spt; ++ci) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t sc[4], zp[4];
        quad_scales<4, TR, SS>(a, u[k], sc, zp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = kw + ((8 * ci + 4 * k + i) << ks);
          if (c >= a.nch) continue;
          const uint8_t* xc = s_x + c * (2 * kQChunk) + (TR ? 1 : 4) * 16 * quarter;
          multiply<P, 1, TR>(mg, u[k].q[i], sc[i], zp[i], [&](int p, int j) {
            return *reinterpret_cast<const half8*>(xc + 16 * (p * nblk + (TR ? 4 : 1) * j));
          }, acc);
        }
        load(k);
      }
      advance();
    }
    // the tile is done: the waves that split its columns add up, in order
    float* red = s_red[parity];
    parity ^= 1;
    if (lane < 16) red[wave * 16 + lane] = acc[0];
    if (ks) __syncthreads();
    const int tile = ks ? tid >> 4 : tw;
    const int n = (cg * tiles + tile) * 16 + (tid & 15);
    if ((ks ? tid < tiles * 16 : lane < 16) && n < a.N) {
      float s = 0.0f;
      for (int w = 0; w < wk; ++w) s += red[((tile << ks) + w) * 16 + (tid & 15)];
      s *= fabsf(inv);
      if (DT != MOE_DT_F16 && !(fabsf(s) < INFINITY) && inv > 0.0f) left |= bit;
      else put<DT>(a, 0, n, s);
    }
  }
  if (DT == MOE_DT_F16 || __ballot(left != 0) == 0) return;
  // behind the loop, whose scalars this code would spill
  const QArgsPtr b = args_again();
  for (int cg = blockIdx.x; cg < b->row_groups; cg += gridDim.x, left >>= 1) {
    const int n = (cg * (kQWaves >> b->ks) + (b->ks ? tid >> 4 : tid >> 6)) * 16 + (tid & 15);
#pragma unroll 1
    for (uint64_t m = __ballot(left & 1); m; m &= m - 1) {
      const int l = __ffsll((long long)m) - 1;
      const float s = sum_in_f64<DT, TR, SS>(0, __builtin_amdgcn_readlane(n, l), 0, INT_MAX);
      QArgs c;
      c.y = b->y; c.y_pitch = b->y_pitch; c.accumulate = b->accumulate;
      if (lane == l) put<DT>(c, 0, n, s);
    }
  }
}

// ---------------------------------------------------------------------------
// 2 .. 16 tokens
// ---------------------------------------------------------------------------
// Workgroup (rows, range): kQWaves / WK tiles of 16 rows, a range of column
// slices of kQSlice chunks.  For each slice the workgroup makes the tokens'
// terms in LDS, under a power of two per token and slice; its waves then walk
// the slice's codes (WK waves share a tile's chunks), the next slice's loaded
// as soon as these are used.  Small matrices take a larger WK (and with eight as
// long a slice as 64 KB of terms hold): more workgroups, each with less to do
// after its loads have arrived.  7 tokens, bf16, 7168 x 3584 in groups of 32:
// 11.6 us, of which unpacking and transposing are 3.3, and latencies (x, terms,
// the ranges added one load after the other) most of the rest.
// Calls of up to 8 tokens and eight waves to a row tile are for two workgroups a
// CU: four waves to a SIMD (8 tokens x 16384 x 4096, fp32: 25.3 us with three).
constexpr int few_slice(int P, int TOK, int WK) { return WK == 8 ? 65536 / (P * TOK * 2 * kQChunk) : 8; }

template <int DT, int TOK, int WK, bool TR, int SS>
__global__ __launch_bounds__(kQWG, WK == 8 || TOK == 8 ? 4 : 2) void k_qfew(QArgs a) {
  constexpr int P = DT == MOE_DT_F32 ? 2 : 1;
  constexpr int NR = TOK / 4;
  constexpr int kQSlice = few_slice(P, TOK, WK), kQSliceCols = kQSlice * kQChunk;
  constexpr int NB = TOK * kQSliceCols / 8 / kQWG;        // blocks of x per thread
  constexpr int kBlocks = kQSliceCols / 8;
  constexpr int B = DT == MOE_DT_F32 ? 4 : 2;
  constexpr int NU = kQSlice / WK, NQ = NU > 4 ? 4 : NU, QN = NU / NQ;   // a wave's chunks, as quads
  extern __shared__ __align__(16) uint8_t s_x[];          // [P][blocks][TOK] of 16 bytes
  __shared__ uint32_t s_max[kQWaves][TOK];
  __shared__ bool s_spoilt[TOK];                          // tokens that are not finite in these slices
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int row = lane & 15, quarter = lane >> 4;
  const int kw = wave % WK;
  const int n0 = (blockIdx.x * (kQWaves / WK) + wave / WK) * 16;
  const int s0 = blockIdx.y * a.per_split;
  const int nsl = (a.nch + kQSlice - 1) / kQSlice;
  const int s1 = s0 + a.per_split < nsl ? s0 + a.per_split : nsl;
  const int t = tid % TOK;                                // this thread's token
  const __amdgpu_buffer_rsrc_t xv = x_view<DT>(a, 0, a.C);
  const View v = view_rows<SS>(a, n0, 16, row, quarter);

  Raw<DT> raw[NB];
  auto load_x = [&](int s) {
    const uint32_t xrow = (uint32_t)(t * (int)a.x_pitch * B);
    const int k = s * kQSliceCols + 8 * (tid / TOK);
    if (a.x_vec) {
#pragma unroll
      for (int i = 0; i < NB; ++i) load8v<DT>(a, xv, xrow, k + 8 * (kQWG / TOK) * i, t < a.C && s < s1, raw[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NB; ++i) load8e<DT>(a, xv, xrow, k + 8 * (kQWG / TOK) * i, t < a.C && s < s1, raw[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const Magic mg = magic();
  Quad<NQ, TR> u[QN];
  auto load = [&](int s, int k) {
    load_quad<NQ, TR, SS>(a, v, s * kQSlice + kw + WK * NQ * k, WK, quarter, s < s1, u[k]);
    __builtin_amdgcn_sched_barrier(0);
  };
  load_x(s0);
#pragma unroll
  for (int k = 0; k < QN; ++k) load(s0, k);

  // the token of operand row `row`; rows beyond TOK tokens repeat one
  const uint8_t* frag0 = s_x + 16 * (TOK == 8 ? (row >> 2) + 4 * (row & 1) : row_token(row)) +
                         16 * TOK * (TR ? 1 : 4) * quarter;
  bool spoilt = false;
  float sum[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) sum[r] = 0.0f;
  for (int s = s0; s < s1; ++s) {
    float m = 1.0f, inv[NR];
    bool finite = true;
    uint32_t mx = 0;
    if (DT != MOE_DT_F16) {
#pragma unroll
      for (int i = 0; i < NB; ++i) mx = raw_max<DT>(raw[i], mx);
#pragma unroll
      for (int w = TOK; w < 64; w <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)mx, w, 64);
        mx = o > mx ? o : mx;
      }
      if (lane < TOK) s_max[wave][lane] = mx;
    }
    __syncthreads();                                      // and all are done with the last slice's terms
    if (DT != MOE_DT_F16) {
#pragma unroll
      for (int w = 0; w < kQWaves; ++w) mx = s_max[w][t] > mx ? s_max[w][t] : mx;
      float unused;
      term_scale(mx, m, unused);
      finite = mx < 0x7F800000u;
      spoilt |= !finite;
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      inv[r] = 1.0f;
      if (DT != MOE_DT_F16) {
        uint32_t q = 0;
#pragma unroll
        for (int w = 0; w < kQWaves; ++w) q = s_max[w][4 * r + quarter] > q ? s_max[w][4 * r + quarter] : q;
        float unused;
        term_scale(q, unused, inv[r]);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      half8 hi, lo;
      make_terms<DT>(raw[i], m, finite, hi, lo);
      uint8_t* o = s_x + 16 * (size_t)(tid + kQWG * i);
      *reinterpret_cast<half8*>(o) = hi;
      if (P == 2) *reinterpret_cast<half8*>(o + 16 * kBlocks * TOK) = lo;
    }
    if (s + 1 < s1) load_x(s + 1);
    __syncthreads();
    float acc[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[r] = 0.0f;
#pragma unroll
    for (int k = 0; k < QN; ++k) {
      uint32_t sc[4], zp[4];
      quad_scales<NQ, TR, SS>(a, u[k], sc, zp);
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int c = kw + WK * (NQ * k + i);             // in the slice
        if (s * kQSlice + c >= a.nch) continue;
        const uint8_t* xc = frag0 + c * (16 * TOK * (kQChunk / 8));
        multiply<P, NR, TR>(mg, u[k].q[i], sc[i], zp[i], [&](int p, int j) {
          return *reinterpret_cast<const half8*>(xc + 16 * TOK * (p * kBlocks + (TR ? 4 : 1) * j));
        }, acc);
      }
      load(s + 1, k);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) sum[r] += inv[r] * acc[r];
  }
  if (tid < TOK) s_spoilt[tid] = spoilt;
  if (WK == 1) __syncthreads();
  const int k0 = s0 * kQSliceCols, k1 = s1 * kQSliceCols;
  auto out = [&](int r, int n, float val) {               // of token 4 r + quarter
    const int tok = 4 * r + quarter;
    if (tok >= a.C || n >= a.N) return;
    val = in_range<DT, TR, SS>(val, [&] { return s_spoilt[tok]; }, tok, n, k0, k1);
    if (a.splits > 1) store_coherent(a.part + ((int64_t)blockIdx.y * a.C + tok) * a.N + n, val);
    else put<DT>(a, tok, n, val);
  };
  if (WK == 1) {
#pragma unroll
    for (int r = 0; r < NR; ++r) out(r, n0 + row, sum[r]);
  } else {
    // the waves that shared a tile's chunks add up, in order
    float* red = reinterpret_cast<float*>(s_x);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NR; ++r) red[(wave * NR + r) * 64 + lane] = sum[r];
    __syncthreads();
    for (int i = tid; i < kQWaves / WK * NR * 64; i += kQWG) {
      const int r = (i >> 6) % NR, tile = (i >> 6) / NR;  // i % 64 is the lane
      float val = 0.0f;
#pragma unroll
      for (int w = 0; w < WK; ++w) val += red[((tile * WK + w) * NR + r) * 64 + lane];
      out(r, (blockIdx.x * (kQWaves / WK) + tile) * 16 + row, val);
    }
  }
  // the last of the rows' workgroups to arrive adds their ranges up, in order
  // (a launch of its own for that took 2 us and the gap before it)
  if (a.splits == 1) return;
  __shared__ int s_last;
  uint32_t* ticket = a.tickets + blockIdx.x;
  if (!last_to_arrive(ticket, (uint32_t)a.splits, &s_last)) return;
  if (tid == 0) reset_ticket(ticket);
  constexpr int kRows = 16 * kQWaves / WK;
  const __amdgpu_buffer_rsrc_t pv = coherent_view(a.part, (uint32_t)a.splits * a.C * a.N * 4u);
  for (int i = tid; i < a.C * kRows; i += kQWG) {
    const int tok = i / kRows, n = blockIdx.x * kRows + i % kRows;
    if (n >= a.N) continue;
    float val = 0.0f;
    for (int s = 0; s < a.splits; ++s) val += coherent_ld(pv, 4u * (uint32_t)((s * a.C + tok) * a.N + n));
    put<DT>(a, tok, n, val);
  }
}

// ---------------------------------------------------------------------------
// Matrix kernel: 17 and more tokens
// ---------------------------------------------------------------------------
// Products of 32 tokens x 32 rows x 16 columns.  A workgroup's waves are WT
// along the tokens and the rest along the rows, each with TW x RT such tiles.
// In LDS: a ring of three buffers, each a chunk's terms (as they lie in the
// workspace) and codes (64 bytes of each row), which loads go to directly, two
// to three chunks ahead of the products; and two tables of (scale, zero pair),
// each for every row of four chunks (G >= 128: one group a chunk) or of a
// chunk's four units.  The tables are there because a load of one scale per
// row touches a cache line per row: taken chunk by chunk and wave by wave those
// lines were more traffic than terms and codes together.  2048 tokens x 3584 x
// 7168, bf16, in groups of 128: a call takes 120 us one behind the other, of which
// the terms are about 11, so 0.97 PFLOP/s (a large library fp16 product reaches
// 1.4); under a profiler, with the kernels apart, 121 to 148.  The matrix cores
// are busy for 40% of that time and the vector units for 43% (unpacking), and a
// wave waits for 31% of its own: neither bounds it alone (see the waits below; 224
// workgroups on 256 CUs).
template <int P, int WT, int TW, int RT>
struct GemmTile {
  static constexpr int WR = kQWaves / WT, TM = WT * TW * 2, rows = WR * RT * 32;
  static constexpr int terms = P * TM * kQTermBytes, codes = rows * 64, buffer = terms + codes;
  static constexpr int ring = 3;
  static constexpr int loads = buffer / 1024 / kQWaves;    // LDS loads per wave and chunk
  static constexpr int entries = rows * 4 / kQWG;          // table entries per thread
  static constexpr int table = rows * 4 * 8;               // bytes
  static constexpr int lds = ring * buffer + 2 * table;
};

typedef float float16v __attribute__((ext_vector_type(16)));

// UG: units (of 32 columns) to a group for G 32 and 64, else 0.
template <int P, int WT, int TW, int RT, int UG, int SS>
__global__ __launch_bounds__(kQWG, 2) void k_qgemm(QArgs a) {
  using G = GemmTile<P, WT, TW, RT>;
  constexpr bool TR = UG > 0;
  constexpr int kGroupSteps = TR ? 2 * UG : 8;             // steps of 16 columns to a scale
  constexpr int WR = G::WR, TM = G::TM;
  extern __shared__ __align__(16) uint8_t s_x[];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int row = lane & 31, half = lane >> 5;
  const int wt = wave / WR, wr = wave % WR;
  // workgroups b, b + 8, ... run on one XCD: a run of consecutive tiles (rows
  // fastest) each, so that an XCD's L2 serves few token tiles and all rows
  const int total = gridDim.x, xcd = blockIdx.x & 7, rem = total & 7;
  const int tile = xcd * (total >> 3) + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const int tg = tile / a.row_groups, rg = tile - tg * a.row_groups;
  const int ct = (a.C + 15) / 16;
  const int c0 = blockIdx.y * a.per_split;
  const int c1 = c0 + a.per_split < a.nch ? c0 + a.per_split : a.nch;
  const int nw = rg * G::rows;                             // the workgroup's rows

  // this thread's table entries: row tr, units or chunks te, te + 1, ...
  constexpr int kPer = 4 / G::entries;
  const int tr = tid / kPer, te = tid % kPer * G::entries;
  const View v = view_rows<SS>(a, nw, G::rows, tr, 0);
  uint32_t ts[G::entries], tz[G::entries], ns[G::entries], nz[G::entries];
  // block kb's into ns, nz (live false: nothing is read)
  auto load_table = [&](int kb, bool live) {
#pragma unroll
    for (int e = 0; e < G::entries; ++e) {
      int g;
      if (TR) {
        const int u = 4 * (kb < c1 ? kb : c1 - 1) + te + e;
        g = u >> (a.gshift - 5);
      } else {
        const int c = 4 * kb + te + e;
        g = (int)(((uint32_t)(c < a.nch ? c : a.nch - 1) * a.gmul) >> 20);
      }
      // past the last group (units past the last column): a scale of 0.  A view
      // of 256 rows may pass 2^31 bytes, but not this offset
      constexpr uint32_t nowhere = 0xFFFFFFFCu;
      const bool there = live && (!TR || g < a.ng);
      const int os = (int)(there ? v.vs + SS * g : nowhere), oz = (int)(there ? v.vz + a.zero_step * g : nowhere);
      if (SS == 4) ns[e] = __builtin_amdgcn_raw_buffer_load_b32(v.scales, os, 0, 0);
      else ns[e] = __builtin_amdgcn_raw_buffer_load_b16(v.scales, os, 0, 0);
      nz[e] = __builtin_amdgcn_raw_buffer_load_b8(v.zeros, oz, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto take_table = [&](bool yes) {
#pragma unroll
    for (int e = 0; e < G::entries; ++e) {
      ts[e] = yes ? ns[e] : ts[e];
      tz[e] = yes ? nz[e] : tz[e];
    }
  };
  auto write_table = [&](int kb) {
    uint8_t* t = s_x + G::ring * G::buffer + (kb & 1) * G::table;
#pragma unroll
    for (int e = 0; e < G::entries; ++e)
      *reinterpret_cast<uint2*>(t + ((te + e) * G::rows + tr) * 8) =
          make_uint2(__float_as_uint(scale_of<SS>(a.scale_bf16, ts[e])), zero_pair(tz[e]));
  };
  // At every chunk c (just opened): the next block's table is written (a
  // block's four chunks write the same, without a branch), and at a block's
  // last chunk the table after it is loaded, to be taken at the next chunk.
  // The table being written was last read a block ago.
  auto step_table = [&](int c) {
    const int kb = TR ? c : c >> 2;
    take_table(TR || (c & 3) == 0);
    write_table(kb + 1);
    load_table(kb + 2, TR || (c & 3) == 3);
  };

  // pieces of 1 KB: the terms' (term, token tile, quarter of it), then the
  // codes' (16 rows each); scalar bases and 32-bit lane offsets
  uint32_t vrow[G::codes / 1024 / kQWaves];
#pragma unroll
  for (int i = 0; i < G::codes / 1024 / kQWaves; ++i) {
    const int n = nw + 16 * (kQWaves * i + wave) + (lane >> 2);
    vrow[i] = (uint32_t)((n < a.N ? n : a.N - 1) - nw) * (uint32_t)a.code_pitch;
  }
  const uint8_t* cbase = a.codes + (int64_t)nw * a.code_pitch;
  constexpr int kTermPieces = G::terms / 1024 / kQWaves, kPieces = G::loads;
  const uint8_t* tbase[kTermPieces];                       // chunk 0's pieces
#pragma unroll
  for (int k = 0; k < kTermPieces; ++k) {
    const int i = k * kQWaves + wave;
    int t = tg * TM + (i >> 2) % TM;
    t = t < ct ? t : ct - 1;
    tbase[k] = a.terms + ((int64_t)(i / (4 * TM) * ct + t) * a.nch) * kQTermBytes + (i & 3) * 1024;
  }
  auto stage_piece = [&](int c, int buf, int k) {
    if (k < kTermPieces) {
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(tbase[k] + (uint32_t)c * (uint32_t)kQTermBytes +
                                                          (uint32_t)(lane * 16)),
          (__attribute__((address_space(3))) void*)(s_x + buf * G::buffer + (k * kQWaves + wave) * 1024), 16, 0, 0);
    } else {
      const int i = k - kTermPieces;
      int u = 4 * c + (lane & 3);
      u = u < a.units ? u : a.units - 1;                   // x is zero past the last column
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(cbase + (vrow[i] + 16u * (uint32_t)u)),
          (__attribute__((address_space(3))) void*)(s_x + buf * G::buffer + G::terms +
                                                    (kQWaves * i + wave) * 1024),
          16, 0, 0);
    }
  };
  auto stage = [&](int c, int buf) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) stage_piece(c, buf, k);
  };

  const Magic mg = magic();
  auto clamped = [&](int c) { return c < c1 ? c : c1 - 1; };
  // The pipeline.  A chunk is eight steps of 16 columns; during a step's matrix
  // instructions the terms of the step two on are read from LDS and the next
  // step's codes unpacked, and where a group's sums are complete (after the chunk, or for
  // TR after each group's units of two steps) the step after scales them into acc, so
  // that vector instructions lie between the matrix instructions of the same
  // wave (the waves of a workgroup run in step: what each does in phases, none
  // overlaps).  The move to the next chunk comes before the last two steps: this
  // chunk's LDS reads are complete by then, so one barrier both frees its
  // buffer for the chunk three on and, each wave having waited for its own
  // loads, opens the next chunk's.  Loads complete in order, and the barrier lets
  // the newest (one chunk's LDS loads) stay in flight; past the last chunk the
  // last is loaded again, so that their number is the same everywhere.  As compiled
  // they do not stay there for long: the LDS reads behind the barrier are taken to
  // depend on the loads into LDS and wait for all of them, and the next chunk's
  // first step waits for the table's loads; groups of 32 and 64 wait so two or
  // three times more in the middle of a chunk, and for groups of 64 the larger tile
  // of one term keeps a few registers in scratch memory.
  float16v acc[TW][RT], d[TW][RT];
  half8 x[4][TW][P], b[RT];                                // step s's terms in x[s & 3]
  uint32_t w[RT][2][4];                                    // codes: unit 2 u + half (TR: swapped, see codes_of)
  uint2 sz[2][RT];                                         // (scale, zero pair): TR group & 1, else [0]
  float sp[RT];                                            // scales of the sums in d
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    sp[i] = 0.0f;
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      acc[t][i] = float16v(0.0f);
      d[t][i] = float16v(0.0f);
    }
  }
  int buf = 0;
  const uint8_t* tables = s_x + G::ring * G::buffer + (wr * RT * 32 + row) * 8;
  // The block of 8 columns that a step takes in this half of the wave: TR
  // step s is half of unit s / 2; else dword s % 4 of units 2 (s / 4) + half.
  auto read = [&](int s) {
    const uint8_t* xs = s_x + buf * G::buffer + (2 * wt * TW + (row >> 4)) * kQTermBytes + (row & 15) * 16 +
                        (TR ? half : 4 * half) * 256;
    const int block = TR ? 2 * s : 8 * (s >> 2) + (s & 3);
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
      for (int p = 0; p < P; ++p)
        x[s & 3][t][p] = *reinterpret_cast<const half8*>(xs + (p * TM + 2 * t) * kQTermBytes + block * 256);
  };
  auto read_scales = [&](int c, int u) {
    const uint8_t* t = tables + ((TR ? c : c >> 2) & 1) * G::table + (TR ? u : c & 3) * G::rows * 8;
#pragma unroll
    for (int i = 0; i < RT; ++i) sz[TR ? u / (kGroupSteps / 2) & 1 : 0][i] = *reinterpret_cast<const uint2*>(t + 32 * 8 * i);
  };
  // every wave's loads of buffer `buf` are complete, and so are its reads of
  // the one before (a plain barrier: __syncthreads would wait for all loads)
  auto open = [&](int c) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(G::loads) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
    const uint8_t* q = s_x + buf * G::buffer + G::terms + (wr * RT * 32 + row) * 64 + half * 16;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint4v v4 = *reinterpret_cast<const uint4v*>(q + i * 2048 + u * 32);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[i][u][k] = v4[k];
      }
    read_scales(c, 0);
    read(0);
  };
  // TR: dwords 0 and 1 of unit 2 u come to lie in the two halves of w[u][0]
  // and those of unit 2 u + 1 in w[u][1] (2 and 3 likewise)
  auto codes_of = [&](int i) {
    if (TR) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        swap32(w[i][u][0], w[i][u][1]);
        swap32(w[i][u][2], w[i][u][3]);
      }
    }
  };
  auto code = [&](int s, int i) { return TR ? w[i][s >> 2][2 * (s & 1) + ((s >> 1) & 1)] : w[i][s >> 2][s & 3]; };
  auto unpack = [&](int s, int i) { b[i] = unpack8(mg, code(s, i), sz[TR ? s / kGroupSteps & 1 : 0][i].y); };
  const int k0 = TR ? c0 : c0 >> 2;
  load_table(k0, true);
  take_table(true);
  load_table(k0 + 1, true);
  stage(c0, 0);
  stage(clamped(c0 + 1), 1);
  write_table(k0);
  take_table(true);
  write_table(k0 + 1);
  open(c0);
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    codes_of(i);
    unpack(0, i);
  }
  __builtin_amdgcn_sched_barrier(0);
  read(1);
  load_table(k0 + 2, TR || (c0 & 3) == 3);
  // the matrix instructions of row tile i in step s
  auto product = [&](int s, int i) {
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      if (s % kGroupSteps == 0) {
        acc[t][i] += sp[i] * d[t][i];
        d[t][i] = float16v(0.0f);
      }
#pragma unroll
      for (int p = 0; p < P; ++p)
        d[t][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[s & 3][t][p], b[i], d[t][i], 0, 0, 0);
    }
    if (s % kGroupSteps == 0) sp[i] = __uint_as_float(sz[TR ? s / kGroupSteps & 1 : 0][i].x);
  };
  // The loads of the chunk two on are issued one by one between the products:
  // together, right after the barrier, they kept both waves of a SIMD from
  // their products for a quarter of the chunk.
  for (int c = c0; c < c1; ++c) {
    const int c2 = clamped(c + 2), free = buf == 0 ? 2 : buf - 1;
    uint32_t code7[RT], z7[RT];
#pragma unroll
    for (int s = 0; s < 6; ++s) {
      read(s + 2);
#pragma unroll
      for (int k = s * kPieces / 6; k < (s + 1) * kPieces / 6; ++k) stage_piece(c2, free, k);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        product(s, i);
        unpack(s + 1, i);
      }
      if (TR && s % kGroupSteps == kGroupSteps - 2) read_scales(c, s / 2 + 1);
      // a matrix instruction, then a few vector ones and an LDS read
#pragma unroll
      for (int k = 0; k < TW * RT * P; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      code7[i] = code(7, i);
      z7[i] = sz[TR ? 1 : 0][i].y;
    }
    buf = buf == 2 ? 0 : buf + 1;
    open(c + 1);
    // two steps left: the next chunk's codes are on their way from LDS
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      product(6, i);
      b[i] = unpack8(mg, code7[i], z7[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    read(1);
#pragma unroll
    for (int i = 0; i < RT; ++i) product(7, i);
    step_table(c + 1);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      codes_of(i);
      unpack(0, i);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int t = 0; t < TW; ++t) acc[t][i] += sp[i] * d[t][i];
  // no load into LDS may be in flight when the workgroup gives its LDS up
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");

  // The results through LDS, so that a wave stores a token's consecutive rows
  // (as they lie in registers, a store held two tokens' 32 rows each, and 64 of
  // them took a tenth of the kernel).  Register r of a product is its row
  // 8 (r / 4) + 4 half + r % 4.
  constexpr int kPitch = G::rows + 32;
  static_assert(kPitch * TM * 16 * 4 <= G::lds, "the results fit the LDS");
  float* res = reinterpret_cast<float*>(s_x);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < TW; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int m = 8 * (r >> 2) + 4 * half + (r & 3);
      const int tok = 16 * (2 * (wt * TW + t) + (m >> 4)) + row_token(m & 15);
#pragma unroll
      for (int i = 0; i < RT; ++i) res[tok * kPitch + (wr * RT + i) * 32 + row] = acc[t][i][r];
    }
  __syncthreads();
  for (int k = wave; k < TM * 16; k += kQWaves) {
    const int tok = tg * TM * 16 + k, c = 4 * lane;
    if (tok >= a.C) break;
    if (c >= G::rows) continue;
    const float inv = a.inv[tok];
    float4 v = *reinterpret_cast<const float4*>(res + k * kPitch + c);
    const float up = fabsf(inv);
    v.x *= up; v.y *= up; v.z *= up; v.w *= up;
    const int n = nw + c;
    // infinite or NaN among them
    if (__builtin_expect(__ballot(0.0f * v.x + 0.0f * v.y + 0.0f * v.z + 0.0f * v.w != 0.0f) != 0, 0)) {
      const int k0 = c0 * kQChunk, k1 = c1 * kQChunk;
#pragma unroll 1
      for (int i = 0; i < 4 && n + i < a.N; ++i) {
        const float e = in_range<0, TR, SS>(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w,
                                         [&] { return inv < 0.0f || a.x_dt == MOE_DT_F16; }, tok, n + i, k0, k1);
        v = make_float4(i == 0 ? e : v.x, i == 1 ? e : v.y, i == 2 ? e : v.z, i == 3 ? e : v.w);
      }
    }
    if (a.splits > 1) {
      float* o = a.part + ((int64_t)blockIdx.y * a.C + tok) * a.N + n;
      if (a.N % 4 == 0 && n < a.N) {
        *reinterpret_cast<float4*>(o) = v;
      } else {
        const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < a.N) o[i] = e[i];
      }
    } else {
      put4(a, tok, n, v);
    }
  }
}

__global__ __launch_bounds__(256) void k_qreduce(QArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = (int64_t)a.C * a.N;
  if (i >= n) return;
  // eight ranges in flight, added in order (500 x 100 results of 19 ranges: 6.6
  // us one by one, 4.2)
  float v = 0.0f;
  int s = 0;
  for (; s + 8 <= a.splits; s += 8) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = a.part[(s + j) * n + i];
#pragma unroll
    for (int j = 0; j < 8; ++j) v += q[j];
  }
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = s + j < a.splits ? a.part[(s + j) * n + i] : 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) v += q[j];
  put(a, (int)(i / a.N), (int)(i % a.N), v);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int64_t kMaxPitch = 1 << 22, kMaxRow = 1 << 24;
bool dtype_ok(int d) { return d == MOE_DT_F32 || d == MOE_DT_BF16 || d == MOE_DT_F16; }
int64_t dtype_size(int d) { return d == MOE_DT_F32 ? 4 : 2; }

moe_status matrix_status(const moe_quant_matrix* m) {
  if (!m || !m->codes || !m->scales) return MOE_ERR_INVALID_ARG;
  if (m->rows < 1 || m->rows > MOE_MAX_QUANT_ROWS || m->cols < 1 || m->cols > MOE_MAX_QUANT_COLS)
    return MOE_ERR_UNSUPPORTED;
  if (m->group != 32 && m->group != 64 && (m->group < 128 || m->group % 128)) return MOE_ERR_UNSUPPORTED;
  if (!dtype_ok(m->scale_dtype)) return MOE_ERR_UNSUPPORTED;
  const int64_t ng = ((int64_t)m->cols + m->group - 1) / m->group;
  if ((uintptr_t)m->codes % 16 || m->code_pitch % 16 || m->code_pitch < ((int64_t)m->cols + 1) / 2)
    return MOE_ERR_INVALID_ARG;
  if (m->scale_pitch < ng || (uintptr_t)m->scales % dtype_size(m->scale_dtype)) return MOE_ERR_INVALID_ARG;
  if (m->zeros && m->zero_pitch < ng) return MOE_ERR_INVALID_ARG;
  // a workgroup's rows (256 at most, of up to 2^24 bytes) are addressed by
  // 32-bit offsets, and so are 16 rows of x
  if (m->code_pitch > kMaxPitch || m->scale_pitch > kMaxPitch || (m->zeros && m->zero_pitch > kMaxPitch))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// How a call runs: one rule on its sizes.
enum { kOne, kFew, kMany };
constexpr size_t kTicketBytes = 256 * sizeof(uint32_t);
struct QPlan {
  int P, nch, ct;                      // terms, chunks, token tiles
  int path;
  bool wide;                           // the larger matrix tile
  int wk;                              // few tokens: waves to a row tile
  int row_groups, tok_groups, splits, per_split;
  size_t inv, terms, part, total;
};

QPlan quant_plan(const moe_quant_matrix* m, int dtype, int C) {
  QPlan p = {};
  p.P = dtype == MOE_DT_F32 ? 2 : 1;
  p.nch = (m->cols + kQChunk - 1) / kQChunk;
  p.ct = (C + 15) / 16;
  p.splits = 1;
  p.tok_groups = 1;
  p.per_split = p.nch;
  p.path = C == 1 && (int64_t)p.nch * kQChunk * 2 * p.P <= kQStageBytes ? kOne
           : C <= MOE_MAX_DECODE_TOKENS ? kFew : kMany;
  if (p.path == kFew) {
    // the fewest waves to a row tile that give every CU a workgroup, eight only
    // up to a workgroup of 16 rows a CU: a workgroup of fewer rows makes the same
    // terms for less (us with one, two, eight: 7 tokens, bf16, 7168 x 3584 14.7,
    // 13.0, 13.1; 16384 x 4096 15.3, 16.4, 19.7; 2 tokens, 14917 x 832 6.7, 5.8,
    // 13.4; 4 tokens, 3000 x 2000 13.4, 10.6, 8.7; 6000 x 2000 9.9, 8.2, 9.2; 16
    // tokens, fp32, 1001 x 4099 23.8, 17.7, 16.8)
    const int tok = C <= 8 ? 8 : 16;
    int nsl = 1, s = 1;
    for (p.wk = 1;; p.wk = p.wk == 1 ? 2 : 8) {
      const int rows = 16 * kQWaves / p.wk, slice = few_slice(p.P, tok, p.wk);
      nsl = (p.nch + slice - 1) / slice;
      p.row_groups = (m->rows + rows - 1) / rows;
      if (p.wk == 8 || (int64_t)p.row_groups * nsl >= 256 || (p.wk == 2 && m->rows > 4096)) break;
    }
    // ranges of slices: two workgroups a CU (7 tokens, bf16, 7168 x 3584: 12.9
    // us in four ranges, 13.8 in two; 16, fp32, 1001 x 4099: 17.0 in five, 20.6
    // in three); for more than 8 tokens in slices of several chunks a wave one,
    // whose partial results are half as many (16, fp32, 3584 x 7168: 17.0 in
    // four, 20.9 in seven)
    s = (tok == 8 || p.wk == 8 ? 512 : 256) / p.row_groups;
    s = s < 1 ? 1 : s > nsl ? nsl : s;
    p.per_split = (nsl + s - 1) / s;
    p.splits = (nsl + p.per_split - 1) / p.per_split;
  } else if (p.path == kMany) {
    // the larger tile (256 rows, and tokens whose terms fit the LDS ring): with
    // two terms where its workgroups, one a CU, fill half the CUs (us without,
    // with it, 7168 columns: 512 tokens x 3584, 112 workgroups, 85, 89; 1024
    // tokens, 224, 141, 113); with one, whose smaller tile runs two workgroups a
    // CU and so is the faster as long as all of those run at once, where they do
    // not (3136 columns: 1024 tokens x 4096, 512 small ones, 49.7, 55.0; 1100
    // tokens, 576, 67.9, 56.6)
    const int wide_tokens = p.P == 2 ? 64 : 128;
    const int64_t wide = (int64_t)((C + wide_tokens - 1) / wide_tokens) * ((m->rows + 255) / 256);
    const int64_t narrow = (int64_t)((C + 63) / 64) * ((m->rows + 127) / 128);
    p.wide = C > 64 && (p.P == 2 ? wide >= 128 : narrow > 512);
    p.tok_groups = p.wide ? (C + wide_tokens - 1) / wide_tokens : (C + 63) / 64;
    p.row_groups = p.wide ? (m->rows + 255) / 256 : (m->rows + 127) / 128;
    const int64_t wgs = (int64_t)p.tok_groups * p.row_groups;
    if (!p.wide && wgs < 256) {
      // column ranges: a workgroup a CU as long as a range keeps four chunks;
      // with one term, where two workgroups fit a CU, two as long as it keeps
      // twelve (us in 1, 2, 4, 7 ranges, 3584 x 7168: fp32, 128 tokens, 56
      // workgroups, 63.7, 43.1, 32.8, 39.2; 200 tokens, 112 of them, 64.9, 47.1,
      // 51.9, 66.5; bf16, 128 tokens 54.1, 36.7, 27.3, 28.4; 256 tokens in 2, 4, 9
      // ranges 40.0, 37.5, 45.1)
      const int64_t once = 256 / wgs < p.nch / 4 ? 256 / wgs : p.nch / 4;
      const int64_t twice = p.P == 2 ? 0 : 512 / wgs < p.nch / 12 ? 512 / wgs : p.nch / 12;
      const int s = (int)(once > twice ? once : twice);
      if (s > 1) {
        p.per_split = (p.nch + s - 1) / s;
        p.splits = (p.nch + p.per_split - 1) / p.per_split;
      }
    }
  }
  // the tickets come first in every plan (ranges are only split for up to 256
  // groups of rows), so that calls of other shapes leave them at zero
  size_t o = kTicketBytes;
  p.inv = o; o = align256(o + (p.path == kMany ? (size_t)C * sizeof(float) : 0));
  p.terms = o; o = align256(o + (p.path == kMany ? (size_t)p.P * p.ct * p.nch * kQTermBytes : 0));
  p.part = o; o = align256(o + (p.splits > 1 ? (size_t)p.splits * C * m->rows * sizeof(float) : 0));
  p.total = o;
  return p;
}

// The most that any number of tokens up to C needs.  A plan's partial results come
// and go with its ranges, so fewer tokens may need more than C (bf16, 7168 x 3584:
// 256 tokens 16.5 MB, 257 2 MB).  From 17 tokens on tile and ranges depend on the
// tiles of 64 tokens alone, so that among equal ones the most tokens need the most.
size_t quant_workspace(const moe_quant_matrix* m, int dtype, int C) {
  size_t most = quant_plan(m, dtype, C).total;
  for (int c = 1; c < C; c = c < MOE_MAX_DECODE_TOKENS ? c + 1 : c / 64 * 64 + 64) {
    const size_t n = quant_plan(m, dtype, c).total;
    most = n > most ? n : most;
  }
  return most;
}

template <int DT>
void launch_one(const QArgs& a, bool tr, int ss, int grid, size_t lds, hipStream_t st) {
  if (tr) {
    if (ss == 4) hipLaunchKernelGGL((k_qone<DT, true, 4>), dim3(grid), dim3(kQWG), lds, st, a);
    else hipLaunchKernelGGL((k_qone<DT, true, 2>), dim3(grid), dim3(kQWG), lds, st, a);
  } else {
    if (ss == 4) hipLaunchKernelGGL((k_qone<DT, false, 4>), dim3(grid), dim3(kQWG), lds, st, a);
    else hipLaunchKernelGGL((k_qone<DT, false, 2>), dim3(grid), dim3(kQWG), lds, st, a);
  }
}

template <int DT, int TOK, int WK, bool TR, int SS>
moe_status launch_few_t(const QArgs& a, dim3 grid, hipStream_t st) {
  constexpr int P = DT == MOE_DT_F32 ? 2 : 1, lds = P * 2 * few_slice(P, TOK, WK) * kQChunk * TOK;
  auto k = k_qfew<DT, TOK, WK, TR, SS>;
  if (lds + 1024 > 65536 && hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                                hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
    return MOE_ERR_DEVICE;
  hipLaunchKernelGGL(k, grid, dim3(kQWG), lds, st, a);
  return MOE_OK;
}
template <int DT, int TOK, int WK>
moe_status launch_few_w(const QArgs& a, bool tr, int ss, dim3 grid, hipStream_t st) {
  if (tr) return ss == 4 ? launch_few_t<DT, TOK, WK, true, 4>(a, grid, st) : launch_few_t<DT, TOK, WK, true, 2>(a, grid, st);
  return ss == 4 ? launch_few_t<DT, TOK, WK, false, 4>(a, grid, st) : launch_few_t<DT, TOK, WK, false, 2>(a, grid, st);
}
template <int DT, int TOK>
moe_status launch_few(const QArgs& a, bool tr, int ss, int wk, dim3 grid, hipStream_t st) {
  if (wk == 1) return launch_few_w<DT, TOK, 1>(a, tr, ss, grid, st);
  if (wk == 2) return launch_few_w<DT, TOK, 2>(a, tr, ss, grid, st);
  return launch_few_w<DT, TOK, 8>(a, tr, ss, grid, st);
}

template <int P, int WT, int TW, int RT, int UG, int SS>
moe_status launch_gemm_t(const QArgs& a, dim3 grid, hipStream_t st) {
  constexpr int lds = GemmTile<P, WT, TW, RT>::lds;
  auto k = k_qgemm<P, WT, TW, RT, UG, SS>;
  if (lds > 65536 && hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize,
                                         lds) != hipSuccess)
    return MOE_ERR_DEVICE;
  hipLaunchKernelGGL(k, grid, dim3(kQWG), lds, st, a);
  return MOE_OK;
}

template <int P, int WT, int TW, int RT, int UG>
moe_status launch_gemm_u(const QArgs& a, int ss, dim3 grid, hipStream_t st) {
  return ss == 4 ? launch_gemm_t<P, WT, TW, RT, UG, 4>(a, grid, st) : launch_gemm_t<P, WT, TW, RT, UG, 2>(a, grid, st);
}
template <int P, int WT, int TW, int RT>
moe_status launch_gemm(const QArgs& a, bool tr, int ss, dim3 grid, hipStream_t st) {
  if (!tr) return launch_gemm_u<P, WT, TW, RT, 0>(a, ss, grid, st);
  return a.gshift == 5 ? launch_gemm_u<P, WT, TW, RT, 1>(a, ss, grid, st) : launch_gemm_u<P, WT, TW, RT, 2>(a, ss, grid, st);
}

template <int DT>
moe_status launch_quant(QArgs a, const QPlan& p, bool tr, int ss, hipStream_t st) {
  constexpr int P = DT == MOE_DT_F32 ? 2 : 1;
  moe_status s = MOE_OK;
  if (p.path == kOne) {
    // waves to a row tile: the power of two that comes nearest to eight waves
    // a CU (us with 1, 2, 4, 8 waves: fp32, 3584 x 7168 25.9, 16.5, 11.2, 9.0;
    // 7168 x 3584 15.7, 10.8, 8.5, 9.3; 16384 x 7168 26.5, 18.2, 17.9, 17.7;
    // bf16, 65536 x 7168 50.8, 54.0, 52.6, 56.2); tiles walked by a resident
    // grid, whose terms are made once (65536 x 7168: 50.5 us from 512 workgroups,
    // 51.3 from 8192)
    const int nt = (a.N + 15) / 16;
    a.ks = 3;
    while (a.ks > 0 && ((int64_t)nt << (a.ks - 1)) >= 1536) --a.ks;
    a.row_groups = (nt + (kQWaves >> a.ks) - 1) / (kQWaves >> a.ks);
    a.spt = (((a.nch + (1 << a.ks) - 1) >> a.ks) + 7) / 8;
    launch_one<DT>(a, tr, ss, a.row_groups < 512 ? a.row_groups : 512, (size_t)p.nch * kQChunk * 2 * P, st);
  } else if (p.path == kFew) {
    const dim3 grid((unsigned)p.row_groups, (unsigned)p.splits);
    s = a.C <= 8 ? launch_few<DT, 8>(a, tr, ss, p.wk, grid, st) : launch_few<DT, 16>(a, tr, ss, p.wk, grid, st);
  } else {
    const dim3 tgrid((unsigned)p.ct * 4);
    constexpr int kTermChunks = kTermBlocks * 8 / kQChunk;         // of one block a thread
    if (p.nch <= 4 * kTermChunks) hipLaunchKernelGGL((k_qterms<DT, 4>), tgrid, dim3(kTermWG), 0, st, a);
    else if (p.nch <= 8 * kTermChunks) hipLaunchKernelGGL((k_qterms<DT, 8>), tgrid, dim3(kTermWG), 0, st, a);
    else hipLaunchKernelGGL((k_qterms<DT, 0>), tgrid, dim3(kTermWG), 0, st, a);
    a.row_groups = p.row_groups;
    const dim3 grid((unsigned)(p.row_groups * p.tok_groups), (unsigned)p.splits);
    s = !p.wide ? launch_gemm<P, 2, 1, 1>(a, tr, ss, grid, st)
        : P == 2 ? launch_gemm<2, 1, 2, 1>(a, tr, ss, grid, st) : launch_gemm<1, 2, 2, 2>(a, tr, ss, grid, st);
  }
  if (s != MOE_OK) return s;
  if (p.path == kMany && p.splits > 1)
    hipLaunchKernelGGL(k_qreduce, dim3((unsigned)(((int64_t)a.C * a.N + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // namespace
}  // namespace rf4

using namespace rf4;

extern "C" {

size_t moe_quant_workspace_size(const moe_quant_matrix* m, int32_t dtype, int32_t C) {
  if (matrix_status(m) != MOE_OK || !dtype_ok(dtype) || C < 1 || C > MOE_MAX_TOKENS) return 0;
  return quant_workspace(m, dtype, C);
}

moe_status moe_quant_linear(const moe_quant_matrix* m, int32_t dtype, const void* x,
                            int64_t x_pitch, int32_t C, void* y, int64_t y_pitch,
                            int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  const moe_status ms = matrix_status(m);
  if (ms != MOE_OK) return ms;
  if (!x || !y) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || C < 1 || C > MOE_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
  const int64_t xs = dtype_size(dtype), ss = dtype_size(m->scale_dtype);
  if (x_pitch > kMaxRow || y_pitch > kMaxRow) return MOE_ERR_UNSUPPORTED;
  if (x_pitch < m->cols || y_pitch < m->rows || (uintptr_t)x % xs || (uintptr_t)y % xs)
    return MOE_ERR_INVALID_ARG;
  if (rows_overlap(x, m->cols * xs, x_pitch * xs, y, m->rows * xs, y_pitch * xs, C)) return MOE_ERR_INVALID_ARG;
  const QPlan p = quant_plan(m, dtype, C);
  if (!ws || (uintptr_t)ws % 256 || ws_bytes < p.total) return MOE_ERR_WORKSPACE;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  QArgs a = {};
  a.codes = static_cast<const uint8_t*>(m->codes); a.code_pitch = m->code_pitch;
  a.scales = static_cast<const uint8_t*>(m->scales); a.scale_pitch = m->scale_pitch * ss;
  a.scale_bf16 = m->scale_dtype == MOE_DT_BF16;
  a.zeros = m->zeros;
  a.zero_pitch = m->zeros ? m->zero_pitch : 0;
  a.zero_step = m->zeros ? 1 : 0;
  a.N = m->rows; a.K = m->cols;
  a.units = (m->cols + 31) / 32; a.nch = p.nch;
  a.ng = (int)(((int64_t)m->cols + m->group - 1) / m->group);
  const bool tr = m->group < 128;
  // whole chunks, and rows of scales and zero points at multiples of 4 bytes
  a.scales_vec = m->cols % kQChunk == 0 && (uintptr_t)m->scales % 4 == 0 && a.scale_pitch % 4 == 0 &&
                 (uintptr_t)m->zeros % 4 == 0 && a.zero_pitch % 4 == 0;
  a.gshift = m->group == 32 ? 5 : 6;
  // groups of whole chunks: c < 2^10 chunks over gc chunks a group; the
  // product's error c / 2^20 stays under the 1 / gc to the next quotient
  const int gc = tr ? 1 : m->group / kQChunk < p.nch ? m->group / kQChunk : p.nch;
  a.gmul = (1u << 20) / (uint32_t)gc + 1u;
  a.x = x; a.x_pitch = x_pitch; a.x_dt = dtype;
  a.x_vec = (uintptr_t)x % 16 == 0 && (C == 1 || x_pitch * xs % 16 == 0);
  a.C = C; a.y = y; a.y_pitch = y_pitch; a.accumulate = accumulate;
  a.y_vec = (uintptr_t)y % (4 * xs) == 0 && y_pitch % 4 == 0;
  a.inv = reinterpret_cast<float*>(w8 + p.inv);
  a.terms = w8 + p.terms;
  a.part = reinterpret_cast<float*>(w8 + p.part);
  a.tickets = reinterpret_cast<uint32_t*>(w8);
  a.splits = p.splits; a.per_split = p.per_split;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == MOE_DT_F32) return launch_quant<MOE_DT_F32>(a, p, tr, (int)ss, st);
  if (dtype == MOE_DT_BF16) return launch_quant<MOE_DT_BF16>(a, p, tr, (int)ss, st);
  return launch_quant<MOE_DT_F16>(a, p, tr, (int)ss, st);
}

}  // extern "C"
