// Internal header of libroutedfp4: what the dense operators in 16 and 32 bits
// (adapter.hip, ffn.hip) share: eight elements of a row at a time, the counter
// generator of dropout, and checks of arguments.  Not part of the C ABI.
#pragma once

#include "common.h"

namespace rf4 {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <int DT>
constexpr int kBytes = DT == MOE_DT_F32 ? 4 : 2;

// Eight consecutive elements of a row, as stored.
template <int DT>
struct Eight { uint4v v[DT == MOE_DT_F32 ? 2 : 1]; };

// 16 bytes at any address that is aligned to its elements (global accesses
// need no more on this device).
typedef uint4v uint4u __attribute__((aligned(2)));
__device__ __forceinline__ uint4v load16(const void* p) { return *static_cast<const uint4u*>(p); }
__device__ __forceinline__ void store16(void* p, uint4v v) { *static_cast<uint4u*>(p) = v; }

template <int DT>
__device__ __forceinline__ Eight<DT> load8(const void* p) {
  Eight<DT> e;
  e.v[0] = load16(p);
  if constexpr (DT == MOE_DT_F32) e.v[1] = load16(static_cast<const uint8_t*>(p) + 16);
  return e;
}
// the first `n` of them (n may be 0 or less, or more than 8), zeros for the others:
// one by one from the last, in a loop that stays one (unrolled at every use, it was
// most of the kernels' code)
template <int DT>
__device__ __forceinline__ Eight<DT> load8_some(const void* p, int n) {
  if (n >= 8) return load8<DT>(p);
  Eight<DT> e = {};
#pragma unroll 1
  for (int i = n - 1; i >= 0; --i) {
    if constexpr (DT == MOE_DT_F32) {
#pragma unroll
      for (int k = 7; k > 0; --k) e.v[k >> 2][k & 3] = e.v[(k - 1) >> 2][(k - 1) & 3];
      e.v[0][0] = static_cast<const uint32_t*>(p)[i];
    } else {
#pragma unroll
      for (int k = 3; k > 0; --k) e.v[0][k] = (e.v[0][k] << 16) | (e.v[0][k - 1] >> 16);
      e.v[0][0] = (e.v[0][0] << 16) | static_cast<const uint16_t*>(p)[i];
    }
  }
  return e;
}
// The same by one load, for n >= 0 and where eight elements may be read.
template <int DT>
__device__ __forceinline__ Eight<DT> load8_first(const void* p, int n) {
  Eight<DT> e = load8<DT>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == MOE_DT_F32) e.v[i >> 2][i & 3] = i < n ? e.v[i >> 2][i & 3] : 0u;
    else if (!(i & 1)) e.v[0][i >> 1] &= (i < n ? 0xFFFFu : 0u) | (i + 1 < n ? 0xFFFF0000u : 0u);
  }
  return e;
}

template <int DT>
__device__ __forceinline__ float get8(const Eight<DT>& e, int i) {
  if constexpr (DT == MOE_DT_F32) return __uint_as_float(e.v[i >> 2][i & 3]);
  const uint32_t w = e.v[0][i >> 1];
  if constexpr (DT == MOE_DT_BF16) return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)((i & 1) ? w >> 16 : w));
}
// one rounding to the nearest, ties to even
template <int DT>
__device__ __forceinline__ uint16_t round16(float f) {
  if constexpr (DT == MOE_DT_BF16) return __builtin_bit_cast(uint16_t, (__bf16)f);
  return __builtin_bit_cast(uint16_t, (_Float16)f);
}
template <int DT>
__device__ __forceinline__ Eight<DT> put8(const float (&f)[8]) {
  Eight<DT> e;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == MOE_DT_F32) e.v[i >> 2][i & 3] = __float_as_uint(f[i]);
    else if (i & 1) e.v[0][i >> 1] |= (uint32_t)round16<DT>(f[i]) << 16;
    else e.v[0][i >> 1] = round16<DT>(f[i]);
  }
  return e;
}
template <int DT>
__device__ __forceinline__ void store8(void* p, const Eight<DT>& e) {
  store16(p, e.v[0]);
  if constexpr (DT == MOE_DT_F32) store16(static_cast<uint8_t*>(p) + 16, e.v[1]);
}
template <int DT>
__device__ __forceinline__ void store8_some(void* p, const Eight<DT>& e, int n) {
  if (n >= 8) { store8<DT>(p, e); return; }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < n) {
      if constexpr (DT == MOE_DT_F32) static_cast<uint32_t*>(p)[i] = e.v[i >> 2][i & 3];
      else static_cast<uint16_t*>(p)[i] = (uint16_t)(e.v[0][i >> 1] >> (16 * (i & 1)));
    }
  }
}

// 16 bytes' worth of them: eight of 16 bits, four of fp32
template <int DT>
__device__ __forceinline__ Eight<DT> first_of(uint4v v) {
  Eight<DT> e = {};
  e.v[0] = v;
  return e;
}
template <int DT, int N>
__device__ __forceinline__ uint4v pack16(const float (&f)[N]) {
  static_assert(N * kBytes<DT> == 16, "16 bytes");
  uint4v v;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (DT == MOE_DT_F32) v[i] = __float_as_uint(f[i]);
    else if (i & 1) v[i >> 1] |= (uint32_t)round16<DT>(f[i]) << 16;
    else v[i >> 1] = round16<DT>(f[i]);
  }
  return v;
}
// Elements k .. k + 7 of a row of `cols`, zeros behind its end: the load ends with
// the row, and what came too early is shifted out.  No element outside the row is
// read, and lanes at a row's end load like the others.
template <int DT>
__device__ __forceinline__ Eight<DT> load8_of(const uint8_t* row, int k, int cols) {
  if (cols < 8) return load8_some<DT>(row + (int64_t)k * kBytes<DT>, cols - k);
  const int over = k + 8 - cols, s = over < 0 ? 0 : over > 8 ? 8 : over;   // elements to shift out
  Eight<DT> e = load8<DT>(row + (int64_t)(k + 8 < cols ? k : cols - 8) * kBytes<DT>);
  constexpr int N = DT == MOE_DT_F32 ? 8 : 4;                              // words
  uint32_t w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = e.v[i >> 2][i & 3];
#pragma unroll
  for (int b = N / 2; b >= 1; b /= 2) {                                    // by b words
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = s & (DT == MOE_DT_F32 ? b : 2 * b) ? (i + b < N ? w[i + b] : 0u) : w[i];
  }
  if constexpr (DT != MOE_DT_F32) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = s & 1 ? (w[i] >> 16) | (i + 1 < N ? w[i + 1] << 16 : 0u) : w[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) e.v[i >> 2][i & 3] = s >= 8 ? 0u : w[i];
  return e;
}
// load8_of of 16 bytes: eight elements of 16 bits, four of fp32.
template <int DT>
__device__ __forceinline__ uint4v load16_of(const uint8_t* row, int k, int cols) {
  if constexpr (DT != MOE_DT_F32) return load8_of<DT>(row, k, cols).v[0];
  uint4v w = uint4v(0u);
  if (cols < 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k + i < cols) w[i] = reinterpret_cast<const uint32_t*>(row)[k + i];
    return w;
  }
  const int over = k + 4 - cols, s = over < 0 ? 0 : over > 4 ? 4 : over;
  w = load16(row + (int64_t)(k + 4 < cols ? k : cols - 4) * 4);
  if (s & 2) w = uint4v{w[2], w[3], 0u, 0u};
  if (s & 1) w = uint4v{w[1], w[2], w[3], 0u};
  return s >= 4 ? uint4v(0u) : w;
}
template <int DT>
__device__ __forceinline__ void store16_some(void* p, uint4v v, int n) {
  if (n >= 16 / kBytes<DT>) { store16(p, v); return; }
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    if constexpr (DT == MOE_DT_F32) {
      static_cast<uint32_t*>(p)[i] = v[0];
#pragma unroll
      for (int k = 0; k < 3; ++k) v[k] = v[k + 1];
    } else {
      static_cast<uint16_t*>(p)[i] = (uint16_t)v[0];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = (v[k] >> 16) | (k < 3 ? v[k + 1] << 16 : 0u);
    }
  }
}

__device__ __forceinline__ float4v mma_f16(uint4v a, uint4v b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
__device__ __forceinline__ float4v mma_bf16(uint4v a, uint4v b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// 16x16x32 of operands whose lane holds row l % 16 and eight columns 8 (l / 16)
// .. of a step of 32: in fp32 eight products of four columns, one of each quarter
template <int DT>
__device__ __forceinline__ float4v mma8(const Eight<DT>& a, const Eight<DT>& b, float4v c) {
  if constexpr (DT == MOE_DT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(get8<DT>(a, i), get8<DT>(b, i), c, 0, 0, 0);
    return c;
  } else if constexpr (DT == MOE_DT_BF16) {
    return mma_bf16(a.v[0], b.v[0], c);
  } else {
    return mma_f16(a.v[0], b.v[0], c);
  }
}

// ---------------------------------------------------------------------------
// Dropout's counter generator
// ---------------------------------------------------------------------------
// Philox 4x32, ten rounds (Salmon, Moraes, Dror, Shaw: Parallel random numbers:
// as easy as 1, 2, 3; SC 2011): the key is the seed, the counter is (offset,
// column / 8, row), and its 128 bits are the 16-bit numbers of eight columns.
// Ten rounds are 20 products of 32 x 32 bits; a number of 16 bits per element
// halves them against 32, and a probability is taken to a multiple of 2^-16.
struct Dropout {
  uint32_t drop;            // dropped where the number is below: 0 (none) .. 65536 (all)
  float scale;              // 1 / (1 - drop / 65536), or 0
  const uint64_t* rng;      // seed, offset
};

struct Counter { uint32_t k0, k1, o0, o1; };
__device__ __forceinline__ Counter counter_of(const uint64_t* rng) {
  const uint64_t s = rng[0], o = rng[1];
  Counter c;
  c.k0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)s);
  c.k1 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(s >> 32));
  c.o0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)o);
  c.o1 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(o >> 32));
  return c;
}
// one instruction, which the compiler does not find
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) { return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96); }
__device__ __forceinline__ uint4v philox(const Counter& c, uint32_t block, uint32_t row) {
  uint32_t w0 = c.o0, w1 = c.o1, w2 = block, w3 = row, k0 = c.k0, k1 = c.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = (uint64_t)w0 * 0xD2511F53u, q = (uint64_t)w2 * 0xCD9E8D57u;
    w0 = xor3((uint32_t)(q >> 32), w1, k0);
    w1 = (uint32_t)q;
    w2 = xor3((uint32_t)(p >> 32), w3, k1);
    w3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return uint4v{w0, w1, w2, w3};
}
// Elements that are dropped become zeros, whatever they are.
template <int DT>
__device__ __forceinline__ Eight<DT> drop8(Eight<DT> e, const Dropout& d, const Counter& c, int col, uint32_t row) {
  const uint4v w = philox(c, (uint32_t)col >> 3, row);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (w[i] & 0xFFFFu) >= d.drop, hi = (w[i] >> 16) >= d.drop;
    if constexpr (DT == MOE_DT_F32) {
      e.v[i >> 1][2 * (i & 1)] = lo ? e.v[i >> 1][2 * (i & 1)] : 0u;
      e.v[i >> 1][2 * (i & 1) + 1] = hi ? e.v[i >> 1][2 * (i & 1) + 1] : 0u;
    } else {
      e.v[0][i] &= (lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
    }
  }
  return e;
}
// The same of 16 bytes from column `col` on: of fp32, half of a block of eight.
template <int DT>
__device__ __forceinline__ uint4v drop16(uint4v v, const Dropout& d, const Counter& c, int col, uint32_t row) {
  if constexpr (DT != MOE_DT_F32) {
    return drop8<DT>(first_of<DT>(v), d, c, col, row).v[0];
  } else {
    const uint4v w = philox(c, (uint32_t)col >> 3, row);
    const bool up = col & 4;
    const uint32_t w0 = up ? w[2] : w[0], w1 = up ? w[3] : w[1];
    return uint4v{(w0 & 0xFFFFu) >= d.drop ? v[0] : 0u, (w0 >> 16) >= d.drop ? v[1] : 0u,
                  (w1 & 0xFFFFu) >= d.drop ? v[2] : 0u, (w1 >> 16) >= d.drop ? v[3] : 0u};
  }
}
__device__ __forceinline__ void drop8f(float (&f)[8], const Dropout& d, const Counter& c, int col, uint32_t row) {
  const uint4v w = philox(c, (uint32_t)col >> 3, row);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu;
    f[i] = h >= d.drop ? f[i] * d.scale : 0.0f;
  }
}
// N = 8, or 4: half of a block
template <int N>
__device__ __forceinline__ void drop_some(float (&f)[N], const Dropout& d, const Counter& c, int col, uint32_t row) {
  if constexpr (N == 8) {
    drop8f(f, d, c, col, row);
  } else {
    uint4v v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i] * d.scale);
    v = drop16<MOE_DT_F32>(v, d, c, col, row);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
}

// ---------------------------------------------------------------------------
// Checks of arguments
// ---------------------------------------------------------------------------
inline bool dense_dtype_ok(int d) { return d == MOE_DT_F32 || d == MOE_DT_BF16 || d == MOE_DT_F16; }
inline int64_t dense_size(int d) { return d == MOE_DT_F32 ? 4 : 2; }
constexpr int64_t kMaxRowPitch = 1 << 24;

// A matrix of n rows of `cols` elements, `pitch` elements apart.
struct Rows {
  const void* p;
  int64_t pitch, cols, n, size;
};
inline moe_status rows_status(const Rows& r) {
  if (!r.p || (uintptr_t)r.p % (uintptr_t)r.size || (r.n > 1 && r.pitch < r.cols)) return MOE_ERR_INVALID_ARG;
  return r.n > 1 && r.pitch > kMaxRowPitch ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
// whether they share a byte; NULL shares none
inline bool share(const Rows& a, const Rows& b) {
  if (!a.p || !b.p) return false;
  if (a.n == b.n) return rows_overlap(a.p, a.cols * a.size, a.pitch * a.size, b.p, b.cols * b.size, b.pitch * b.size, a.n);
  return overlap(a.p, ((a.n - 1) * a.pitch + a.cols) * a.size, b.p, ((b.n - 1) * b.pitch + b.cols) * b.size);
}
inline Rows span(const void* p, int64_t bytes) { return Rows{p, bytes, bytes, 1, 1}; }
// whether something that is written shares a byte with something else
template <size_t A, size_t B>
inline bool any_share(const Rows (&outs)[A], const Rows (&others)[B]) {
  for (const Rows& o : outs)
    for (const Rows& i : others)
      if (share(o, i)) return true;
  return false;
}
// the same rows of one matrix
inline bool same(const Rows& a, const Rows& b) { return a.p == b.p && (a.n == 1 || a.pitch == b.pitch); }

// p in [0, 1], and a seed where something may be dropped
inline moe_status dropout_of(double p, const uint64_t* rng, Dropout& d) {
  if (!(p >= 0.0 && p <= 1.0)) return MOE_ERR_INVALID_ARG;
  d.drop = (uint32_t)__builtin_llrint(p * 65536.0);
  d.scale = d.drop < 65536u ? (float)(65536.0 / (65536.0 - (double)d.drop)) : 0.0f;
  d.rng = rng;
  return d.drop && (!rng || (uintptr_t)rng % 8) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

}  // namespace rf4
