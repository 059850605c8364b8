// libroutedfp4, low-rank adapters of many requests beside a shared projection:
//
//   t_c = A_a drop(x_c)          [r]      a = the token's adapter
//   y_c = base_c + s_a B_a t_c   [N]
// and, for the gradients,
//   u_c = s_a B_a^T dy_c         [r]
//   dx_c = base_c + drop'(A_a^T u_c),   dA_a = sum_c u_c drop(x_c)^T,   dB_a = s_a sum_c dy_c t_c^T
//
// A rank is small (1 .. 128), so every product is bound by reading x, dy and the
// adapters and by writing y and dx as long as the matrix cores are fed; t and u
// stay in fp32.  Where t or u is an operand it enters as three bf16 pieces that
// sum to it exactly (24 bits), where a 16-bit tensor meets them it is one bf16
// (bf16) or two (fp16: 11 bits as 8 + 3), so every product is exact and only the
// fp32 sums round.  The first product (x by A, dy by B) takes both sides as
// stored, fp16 on the fp16 matrix cores.  fp32 tensors use the fp32 ones.
//
// Tokens are taken in the order of a plan: sorted by adapter, in tiles of one
// adapter's tokens (16, or 64 in large batches), and for the gradients of A and
// B in chunks.
//
// Kernels:
//   k_aplan     the plan: a counting sort by one workgroup
//   k_ashrink   t or u: a tile's tokens by a range of columns; partial sums
//   k_aexpand   y or dx: a tile's tokens by a range of columns; adds the partial
//               sums up first and keeps them (t for the caller, u for the next)
//   k_aouter    dA and dB of a chunk's tokens, 128 columns to a workgroup
//   k_areduce   adds the chunks up
//   k_aturn     B by rank for u's product
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include <type_traits>

#include "dense.h"

namespace rf4 {
namespace {

constexpr int kAWG = 256;              // threads, 4 waves
constexpr int kPlanWG = 512;
constexpr int kPlanMagic = 0x41504C4E;

// ---------------------------------------------------------------------------
// The plan
// ---------------------------------------------------------------------------
// A batch of more tokens has tiles of 64: a tile's columns of A and B are read
// once for all of its tokens.
inline int plan_tile(int C) { return C > 1024 ? 64 : 16; }
// Tokens to a chunk: four chunks in a batch, 256 .. 2048 tokens each.
inline int plan_chunk(int C) {
  int q = 256;
  while (q < 2048 && q * 4 < C) q *= 2;
  return q;
}
struct PlanLayout { int64_t perm, tiles, chunks, first, total; int max_tiles, max_chunks; };   // in int32
inline PlanLayout plan_layout(int C, int n) {
  PlanLayout p;
  const int t = plan_tile(C), q = plan_chunk(C), most = C < n ? C : n;
  p.max_tiles = C / t + most + 1;       // every adapter's last may be partial, and the idle tokens'
  p.max_chunks = C / q + most;
  p.perm = 16;
  p.tiles = p.perm + (C + 3) / 4 * 4;
  p.chunks = p.tiles + 4 * (int64_t)p.max_tiles;
  p.first = p.chunks + 4 * (int64_t)p.max_chunks;
  p.total = p.first + n + 1;
  return p;
}

struct PArgs {
  const int32_t* who;
  int C, n, tile, chunk;
  int32_t* plan;
  PlanLayout at;
};

// One workgroup: eight waves take an eighth of the tokens each, count them by
// adapter (adapter n: none), and after a scan over (adapter, wave) place them in
// order, so that tokens of one adapter stay in the batch's order.
__global__ __launch_bounds__(kPlanWG) void k_aplan(PArgs a) {
  constexpr int W = kPlanWG / 64, M = MOE_MAX_ADAPTERS + 1;
  __shared__ int s_count[W][M];
  __shared__ int s_first[M + 1], s_tile[M + 1], s_chunk[M + 1];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n1 = a.n + 1;
  for (int i = tid; i < W * M; i += kPlanWG) s_count[i / M][i % M] = 0;
  __syncthreads();
  const int per = ((a.C + W - 1) / W + 63) / 64 * 64;
  const int lo = wave * per < a.C ? wave * per : a.C, hi = lo + per < a.C ? lo + per : a.C;
  auto adapter = [&](int c) {
    const int v = a.who[c];
    return v >= 0 && v < a.n ? v : a.n;
  };
  for (int c = lo + lane; c < hi; c += 64) atomicAdd(&s_count[wave][adapter(c)], 1);
  __syncthreads();
  if (wave == 0) {
    int f = 0, t = 0, q = 0;
    for (int i = 0; i < n1; i += 64) {
      const int e = i + lane;
      int c = 0;
      if (e < n1)
        for (int w = 0; w < W; ++w) c += s_count[w][e];
      const int ct = (c + a.tile - 1) / a.tile, cq = e < a.n ? (c + a.chunk - 1) / a.chunk : 0;
      const int sf = wave_incl_scan(c), st = wave_incl_scan(ct), sq = wave_incl_scan(cq);
      if (e < n1) {
        s_first[e] = f + sf - c;
        s_tile[e] = t + st - ct;
        s_chunk[e] = q + sq - cq;
      }
      f += __shfl(sf, 63, 64);
      t += __shfl(st, 63, 64);
      q += __shfl(sq, 63, 64);
    }
    if (lane == 0) {
      s_first[n1] = f;
      s_tile[n1] = t;
      s_chunk[n1] = q;
      a.plan[0] = kPlanMagic;
      a.plan[1] = a.C;
      a.plan[2] = a.n;
      a.plan[3] = t;
      a.plan[4] = q;
    }
  }
  __syncthreads();
  for (int e = tid; e < n1; e += kPlanWG) {
    int at = s_first[e];
    for (int w = 0; w < W; ++w) {
      const int c = s_count[w][e];
      s_count[w][e] = at;
      at += c;
    }
    a.plan[a.at.first + e] = s_chunk[e];   // adapter n: the number of chunks
  }
  for (int e = wave; e < n1; e += W) {
    const int first = s_first[e], count = s_first[e + 1] - first, who = e < a.n ? e : -1;
    for (int i = lane; i < s_tile[e + 1] - s_tile[e]; i += 64) {
      const int left = count - i * a.tile;
      *reinterpret_cast<int4*>(a.plan + a.at.tiles + 4 * (int64_t)(s_tile[e] + i)) =
          make_int4(who, first + i * a.tile, left < a.tile ? left : a.tile, 0);
    }
    for (int i = lane; i < s_chunk[e + 1] - s_chunk[e]; i += 64) {
      const int left = count - i * a.chunk;
      *reinterpret_cast<int4*>(a.plan + a.at.chunks + 4 * (int64_t)(s_chunk[e] + i)) =
          make_int4(who, first + i * a.chunk, left < a.chunk ? left : a.chunk, 0);
    }
  }
  __syncthreads();
  for (int c0 = lo; c0 < hi; c0 += 64) {
    const int c = c0 + lane;
    const int v = c < hi ? adapter(c) : -1;
    uint64_t todo = __ballot(c < hi);
    int pos = 0;
    while (todo) {
      const int leader = __ffsll((long long)todo) - 1;
      const int lv = __builtin_amdgcn_readlane(v, leader);
      const uint64_t mine = __ballot(v == lv);
      const int base = s_count[wave][lv];
      if (v == lv) pos = base + __popcll(mine & ((1ull << lane) - 1ull));
      wave_lds_fence();
      if (lane == leader) s_count[wave][lv] = base + __popcll(mine);
      wave_lds_fence();
      todo &= ~mine;
    }
    if (c < hi) a.plan[a.at.perm + pos] = c;
  }
}

// ---------------------------------------------------------------------------
// Pieces of operands
// ---------------------------------------------------------------------------
// v as three bf16 that sum to it exactly, each the truncation of what is left.
// An infinity or NaN is its own first piece and has no others.
__device__ __forceinline__ void pieces3(float v, uint32_t& a, uint32_t& b, uint32_t& c) {
  a = __float_as_uint(v) & 0xFFFF0000u;
  const float r = v - __uint_as_float(a);
  b = __float_as_uint(r) & 0xFFFF0000u;
  const float s = r - __uint_as_float(b);
  c = __float_as_uint(s);
  if ((a & 0x7F800000u) == 0x7F800000u) {
    if (v != v) a = 0x7FC00000u;           // a NaN whose truncation would be an infinity
    b = 0;
    c = 0;
  }
}
__device__ __forceinline__ uint32_t high_pair(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }

// An operand tile of a 16-bit tensor in bf16 pieces: one for bf16, two for fp16.
template <int DT>
constexpr int kPieces = DT == MOE_DT_F16 ? 2 : 1;
template <int DT>
__device__ __forceinline__ void pieces(uint4v v, uint4v (&p)[kPieces<DT>]) {
  if constexpr (DT == MOE_DT_F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f0 = (float)__builtin_bit_cast(_Float16, (uint16_t)v[i]);
      const float f1 = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[i] >> 16));
      const uint32_t a0 = __float_as_uint(f0) & 0xFFFF0000u, a1 = __float_as_uint(f1) & 0xFFFF0000u;
      // the rest of an infinity or NaN is left out (a NaN of 11 bits keeps one in its first 8: it is quiet)
      const uint32_t b0 = __float_as_uint(f0 - __uint_as_float(a0)), b1 = __float_as_uint(f1 - __uint_as_float(a1));
      p[0][i] = high_pair(a0, a1);
      p[1][i] = high_pair((a0 & 0x7F800000u) == 0x7F800000u ? 0u : b0, (a1 & 0x7F800000u) == 0x7F800000u ? 0u : b1);
    }
  } else {
    p[0] = v;
  }
}

// c += (the sum of small's pieces) * (the sum of big's): the products of the
// two lowest, below 2^-24 of the whole, are left out
template <int DT>
__device__ __forceinline__ float4v mma_pieces(const uint4v (&s)[3], const uint4v (&b)[kPieces<DT>], float4v c) {
#pragma unroll
  for (int j = kPieces<DT> - 1; j >= 0; --j)
#pragma unroll
    for (int i = 2 - j; i >= 0; --i) c = mma_bf16(s[i], b[j], c);
  return c;
}

// Eight rows of eight elements, transposed: out[i] is element i of every row.
__device__ __forceinline__ void turn8(const uint4v (&in)[8], uint4v (&out)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      out[i][k] = __builtin_amdgcn_perm(in[2 * k + 1][i >> 1], in[2 * k][i >> 1], (i & 1) ? 0x07060302u : 0x05040100u);
}

struct Tile { int who, first, count; };
__device__ __forceinline__ bool plan_entry(const int32_t* plan, int C, int n, int slot, int64_t list, int i, Tile& t) {
  // a plan of another batch: nothing is done
  if (plan[0] != kPlanMagic || plan[1] != C || plan[2] != n || i >= plan[slot]) return false;
  const int4 v = *reinterpret_cast<const int4*>(plan + list + 4 * (int64_t)i);
  t = Tile{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y), __builtin_amdgcn_readfirstlane(v.z)};
  return true;
}

struct AArgs {
  const int32_t* plan;
  PlanLayout at;
  int C, n, r;
  // shrink: in [C][cols] by w [n][r][cols]; expand: out [C][cols] from w [n][cols][r] or (BWD) [n][r][cols];
  // outer: in [C][cols] by small [C][r]
  int cols;
  const uint8_t* in;
  int64_t in_pitch;                     // pitches and strides in bytes
  const uint8_t* w;
  int64_t w_stride, w_pitch;
  const uint8_t* base;
  int64_t base_pitch;
  uint8_t* out;
  int64_t out_pitch;
  const float* scales;
  float* part;                          // shrink, expand: [splits][C][r] in the plan's order
  int splits, per_split;                // column ranges, columns in each (multiple of 256)
  float* keep;                          // expand: the finished sums [C][r] by token, or NULL
  const float* small;                   // outer: [C][r] by token
  float* sums;                          // outer: [chunks][r][cols]
  Dropout drop;
};

// ---------------------------------------------------------------------------
// t = x A^T over a range of columns
// ---------------------------------------------------------------------------
template <int DT, int NT, int TT, bool DROP>
__global__ __launch_bounds__(kAWG) void k_ashrink(AArgs a) {
  constexpr int B = kBytes<DT>, T = 16 * TT;
  __shared__ float s_red[2][T][NT * 16];
  Tile t;
  if (!plan_entry(a.plan, a.C, a.n, 3, a.at.tiles, blockIdx.x, t) || t.who < 0) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane & 15, quarter = lane >> 4;
  Counter ctr = {};
  if constexpr (DROP) ctr = counter_of(a.drop.rng);
  const uint8_t *xr[TT], *ar[NT];
  int token[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int k = 16 * i + row;
    token[i] = a.plan[a.at.perm + t.first + (k < t.count ? k : t.count - 1)];
    xr[i] = a.in + token[i] * a.in_pitch;
  }
  // rows past the last repeat it: their sums are not used
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int k = 16 * j + row;
    ar[j] = a.w + t.who * a.w_stride + (k < a.r ? k : a.r - 1) * a.w_pitch;
  }
  float4v acc[TT][NT];
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = float4v(0.0f);
  const int c0 = blockIdx.y * a.per_split, c1 = c0 + a.per_split < a.cols ? c0 + a.per_split : a.cols;
  auto step = [&](int c, bool whole) {
    Eight<DT> x[TT], w[NT];
    const int k = c + 8 * quarter;
#pragma unroll
    for (int i = 0; i < TT; ++i) x[i] = whole ? load8<DT>(xr[i] + k * B) : load8_some<DT>(xr[i] + k * B, a.cols - k);
#pragma unroll
    for (int j = 0; j < NT; ++j) w[j] = whole ? load8<DT>(ar[j] + k * B) : load8_some<DT>(ar[j] + k * B, a.cols - k);
    if constexpr (DROP) {
#pragma unroll
      for (int i = 0; i < TT; ++i) x[i] = drop8<DT>(x[i], a.drop, ctr, k, (uint32_t)token[i]);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mma8<DT>(x[i], w[j], acc[i][j]);
  };
  // 64 columns to a wave: whole lines of 16-bit rows
  for (int c = c0 + 64 * wave; c < c1; c += 256) {
    if (c + 64 <= a.cols) {
      step(c, true);
      step(c + 32, true);
    } else {
      step(c, false);
      if (c + 32 < a.cols) step(c + 32, false);
    }
  }
  // the four waves' sums, in a fixed order
  auto put = [&](int s) {
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_red[s][16 * i + 4 * quarter + e][16 * j + row] = acc[i][j][e];
  };
  auto add = [&](int s) {
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] += s_red[s][16 * i + 4 * quarter + e][16 * j + row];
  };
  if (wave >= 2) put(wave - 2);
  __syncthreads();
  if (wave < 2) add(wave);
  __syncthreads();
  if (wave == 1) put(0);
  __syncthreads();
  if (wave == 0) {
    add(0);
    float* o = a.part + ((int64_t)blockIdx.y * a.C + t.first) * a.r;
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 16 * i + 4 * quarter + e;
        if (k >= t.count) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (16 * j + row < a.r) o[(int64_t)k * a.r + 16 * j + row] = acc[i][j][e];
      }
  }
}

// ---------------------------------------------------------------------------
// y = base + s B t, dx = base + drop'(A^T u)
// ---------------------------------------------------------------------------
// A wave's lane l holds, of 128 columns, eight consecutive ones 8 (l % 16) ..:
// as tile i of eight those 8 (l % 16) + i, so that B's and A's rows are read,
// and y's written, 16 bytes (of 16-bit types) at a time.
template <int DT, int TT, bool BWD, bool DROP>
__global__ __launch_bounds__(kAWG) void k_aexpand(AArgs a) {
  constexpr int B = kBytes<DT>, T = 16 * TT, P = DT == MOE_DT_F32 ? 1 : 3;
  // the sums as pieces, [piece][rank / 8][token][8]
  extern __shared__ __align__(16) uint8_t s_t[];
  Tile t;
  if (!plan_entry(a.plan, a.C, a.n, 3, a.at.tiles, blockIdx.x, t)) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane & 15, quarter = lane >> 4;
  const int kt = (a.r + 31) / 32, r32 = 32 * kt;
  const bool idle = t.who < 0;
  const float s = idle ? 0.0f : a.scales ? a.scales[t.who] : 1.0f;
  for (int e = tid; e < T * r32; e += kAWG) {
    const int k = e / r32, j = e - k * r32;
    float v = 0.0f;
    if (!idle && k < t.count && j < a.r) {
      const float* p = a.part + (int64_t)(t.first + k) * a.r + j;
      const int64_t step = (int64_t)a.C * a.r;
      int q = 0;
      for (; q + 8 <= a.splits; q += 8) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = p[(q + i) * step];
#pragma unroll
        for (int i = 0; i < 8; ++i) v += w[i];
      }
      for (; q < a.splits; ++q) v += p[q * step];
    }
    // forward: t, then times s_a; backward: u
    v *= BWD ? s : a.drop.scale;
    if (a.keep && blockIdx.y == 0 && k < t.count && j < a.r) a.keep[(int64_t)a.plan[a.at.perm + t.first + k] * a.r + j] = v;
    if (!BWD) v *= s;
    const int at = ((j >> 3) * T + k) * 8 + (j & 7);
    if constexpr (DT == MOE_DT_F32) {
      reinterpret_cast<float*>(s_t)[at] = v;
    } else {
      uint32_t p0, p1, p2;
      pieces3(v, p0, p1, p2);
      uint16_t* o = reinterpret_cast<uint16_t*>(s_t);
      o[at] = p0 >> 16;
      o[at + T * r32] = p1 >> 16;
      o[at + 2 * T * r32] = p2 >> 16;
    }
  }
  __syncthreads();
  Counter ctr = {};
  if constexpr (DROP) ctr = counter_of(a.drop.rng);
  const uint8_t* w = a.w + (idle ? 0 : t.who) * a.w_stride;
  for (int c0 = 128 * (blockIdx.y * 4 + wave); c0 < a.cols; c0 += 512 * gridDim.y) {
    float4v acc[TT][8];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = float4v(0.0f);
    const int c = c0 + 8 * row;
    if (!idle) {
      for (int k = 0; k < kt; ++k) {
        const int j0 = 32 * k + 8 * quarter;
        Eight<DT> f[8];                 // tile i: column c + i, rank j0 .. j0 + 7
        if constexpr (!BWD) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int n = c + i < a.cols ? c + i : a.cols - 1;
            f[i] = load8_some<DT>(w + n * a.w_pitch + j0 * B, a.r - j0);
          }
        } else {
          Eight<DT> g[8];               // rank j0 + i, columns c .. c + 7
#pragma unroll
          for (int i = 0; i < 8; ++i)
            g[i] = j0 + i < a.r ? load8_some<DT>(w + (j0 + i) * a.w_pitch + c * B, a.cols - c) : zero8<DT>();
          if constexpr (DT == MOE_DT_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int e = 0; e < 8; ++e) f[i].v[e >> 2][e & 3] = g[e].v[i >> 2][i & 3];
          } else {
            uint4v gi[8], fo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) gi[i] = g[i].v[0];
            turn8(gi, fo);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i].v[0] = fo[i];
          }
        }
        if constexpr (DT == MOE_DT_F32) {
#pragma unroll
          for (int i = 0; i < TT; ++i) {
            Eight<DT> u = *reinterpret_cast<const Eight<DT>*>(s_t + (((4 * k + quarter) * T + 16 * i + row) * 8) * 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = mma8<DT>(u, f[j], acc[i][j]);
          }
        } else {
          uint4v u[TT][3];
#pragma unroll
          for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int p = 0; p < P; ++p)
              u[i][p] = *reinterpret_cast<const uint4v*>(s_t + (p * T * r32 + ((4 * k + quarter) * T + 16 * i + row) * 8) * 2);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4v b[kPieces<DT>];
            pieces<DT>(f[j].v[0], b);
#pragma unroll
            for (int i = 0; i < TT; ++i) acc[i][j] = mma_pieces<DT>(u[i], b, acc[i][j]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 16 * i + 4 * quarter + e;
        if (k >= t.count || c >= a.cols) continue;
        const int token = a.plan[a.at.perm + t.first + k];
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = acc[i][j][e];
        if constexpr (BWD && DROP) drop8f(v, a.drop, ctr, c, (uint32_t)token);
        if (a.base) {
          const Eight<DT> b = load8_some<DT>(a.base + token * a.base_pitch + (int64_t)c * B, a.cols - c);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = idle ? get8<DT>(b, j) : v[j] + get8<DT>(b, j);
        }
        store8_some<DT>(a.out + token * a.out_pitch + (int64_t)c * B, put8<DT>(v), a.cols - c);
      }
  }
}

// ---------------------------------------------------------------------------
// sums[j][col] = sum over a chunk's tokens of small[token][j] in[token][col]
// ---------------------------------------------------------------------------
template <int DT, int NT, bool DROP>
__global__ __launch_bounds__(kAWG) void k_aouter(AArgs a) {
  constexpr int B = kBytes<DT>;
  __shared__ float s_red[2][NT * 16][132];
  Tile t;
  if (!plan_entry(a.plan, a.C, a.n, 4, a.at.chunks, blockIdx.y, t)) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane & 15, quarter = lane >> 4;
  const int c = 128 * blockIdx.x + 8 * row, r0 = 64 * blockIdx.z;
  Counter ctr = {};
  if constexpr (DROP) ctr = counter_of(a.drop.rng);
  float4v acc[NT][8];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = float4v(0.0f);
  const int32_t* perm = a.plan + a.at.perm + t.first;
  for (int k0 = 32 * wave; k0 < t.count; k0 += 128) {
    int token[8];
    bool in[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + 8 * quarter + i;
      in[i] = k < t.count;
      token[i] = perm[in[i] ? k : 0];
    }
    Eight<DT> g[8];                     // tokens k0 + 8 quarter + i, columns c .. c + 7
#pragma unroll
    for (int i = 0; i < 8; ++i)
      g[i] = in[i] ? load8_some<DT>(a.in + token[i] * a.in_pitch + (int64_t)c * B, a.cols - c) : zero8<DT>();
    float sm[NT][8];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = r0 + 16 * j + row;
        sm[j][i] = in[i] && k < a.r ? a.small[(int64_t)token[i] * a.r + k] : 0.0f;
      }
    if constexpr (DROP) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = drop8<DT>(g[i], a.drop, ctr, c, (uint32_t)token[i]);
    }
    if constexpr (DT == MOE_DT_F32) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(sm[j][e], get8<DT>(g[e], i), acc[j][i], 0, 0, 0);
    } else {
      uint4v gi[8], f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) gi[i] = g[i].v[0];
      turn8(gi, f);
      uint4v u[NT][3];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[2][3];
          pieces3(sm[j][2 * i], p[0][0], p[0][1], p[0][2]);
          pieces3(sm[j][2 * i + 1], p[1][0], p[1][1], p[1][2]);
#pragma unroll
          for (int q = 0; q < 3; ++q) u[j][q][i] = high_pair(p[0][q], p[1][q]);
        }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4v b[kPieces<DT>];
        pieces<DT>(f[i], b);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j][i] = mma_pieces<DT>(u[j], b, acc[j][i]);
      }
    }
  }
  auto put = [&](int s) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 8; ++i) s_red[s][16 * j + 4 * quarter + e][8 * row + i] = acc[j][i][e];
  };
  auto add = [&](int s) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i][e] += s_red[s][16 * j + 4 * quarter + e][8 * row + i];
  };
  if (wave >= 2) put(wave - 2);
  __syncthreads();
  if (wave < 2) add(wave);
  __syncthreads();
  if (wave == 1) put(0);
  __syncthreads();
  if (wave == 0) {
    add(0);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = r0 + 16 * j + 4 * quarter + e;
        if (k >= a.r || c >= a.cols) continue;
        float* o = a.sums + ((int64_t)blockIdx.y * a.r + k) * a.cols + c;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = acc[j][i][e];
        store8_some<MOE_DT_F32>(o, put8<MOE_DT_F32>(v), a.cols - c);
      }
  }
}

struct RArgs {
  const int32_t* plan;
  PlanLayout at;
  int C, n, r, cols;
  const float* sums;                    // [chunks][r][cols]
  float* out;                           // [n][r][cols], or [n][cols][r] (turned)
  const float* scales;                  // a factor by adapter, or NULL
  float factor;
  int accumulate;
};

// Adds an adapter's chunks in order; an adapter without tokens has zeros.
template <bool TURN>
__global__ __launch_bounds__(256) void k_areduce(RArgs a) {
  const int32_t* plan = a.plan;
  if (plan[0] != kPlanMagic || plan[1] != a.C || plan[2] != a.n) return;
  for (int who = blockIdx.y; who < a.n; who += gridDim.y) {
    const int q0 = plan[a.at.first + who], q1 = plan[a.at.first + who + 1];
    if (a.accumulate && q0 == q1) continue;
    const float f = a.scales ? a.scales[who] * a.factor : a.factor;
    const int64_t n = (int64_t)a.r * a.cols;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
      // e runs over the sums' order, or (TURN) over the output's
      const int64_t at = TURN ? (e % a.r) * a.cols + e / a.r : e;
      float v = 0.0f;
      for (int q = q0; q < q1; ++q) v += a.sums[(int64_t)q * n + at];
      float* o = a.out + (int64_t)who * n + e;
      v *= f;
      *o = a.accumulate ? *o + v : v;
    }
  }
}

struct TArgs {
  const int32_t* plan;
  PlanLayout at;
  int C, n, r, rows;
  const uint8_t* b;                     // [n][rows][r]
  int64_t b_stride, b_pitch;
  uint8_t* out;                         // [n][r][rows], dense, rows padded to `pitch` bytes
  int64_t out_stride, pitch;
};

// B [rows][r] of the adapters that have tokens to [r][rows]: 64 rows to a workgroup.
template <int B>
__global__ __launch_bounds__(256) void k_aturn(TArgs a) {
  typedef typename std::conditional<B == 4, uint32_t, uint16_t>::type E;
  __shared__ E s[64][MOE_MAX_RANK + 2];
  const int32_t* plan = a.plan;
  if (plan[0] != kPlanMagic || plan[1] != a.C || plan[2] != a.n) return;
  for (int who = blockIdx.y; who < a.n; who += gridDim.y) {
    if (plan[a.at.first + who] == plan[a.at.first + who + 1]) continue;
    const int n0 = 64 * blockIdx.x;
    for (int e = threadIdx.x; e < 64 * a.r; e += 256) {
      const int k = e / a.r, j = e - k * a.r;
      if (n0 + k < a.rows)
        s[k][j] = reinterpret_cast<const E*>(a.b + who * a.b_stride + (n0 + k) * a.b_pitch)[j];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * a.r; e += 256) {
      const int j = e >> 6, k = e & 63;
      if (n0 + k < a.rows) reinterpret_cast<E*>(a.out + who * a.out_stride + j * a.pitch)[n0 + k] = s[k][j];
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
moe_status adapter_status(const moe_adapter_bank* b) {
  if (!b) return MOE_ERR_INVALID_ARG;
  if (!dense_dtype_ok(b->dtype) || b->adapters < 1 || b->adapters > MOE_MAX_ADAPTERS || b->rank < 1 ||
      b->rank > MOE_MAX_RANK || b->cols < 1 || b->cols > MOE_MAX_QUANT_COLS || b->rows < 1 ||
      b->rows > MOE_MAX_QUANT_COLS)
    return MOE_ERR_UNSUPPORTED;
  const int64_t s = dense_size(b->dtype);
  const Rows ra = {b->a, b->a_pitch, b->cols, b->rank, s}, rb = {b->b, b->b_pitch, b->rank, b->rows, s};
  moe_status st = rows_status(ra);
  if (st == MOE_OK) st = rows_status(rb);
  if (st != MOE_OK) return st;
  if (b->adapters > 1 && (b->a_stride < (b->rank - 1) * b->a_pitch + b->cols ||
                          b->b_stride < (b->rows - 1) * b->b_pitch + b->rank))
    return MOE_ERR_INVALID_ARG;
  if (b->adapters > 1 && (b->a_stride > ((int64_t)1 << 40) || b->b_stride > ((int64_t)1 << 40))) return MOE_ERR_UNSUPPORTED;
  return (uintptr_t)b->scales % 4 ? MOE_ERR_INVALID_ARG : MOE_OK;
}

// Column ranges of the first product: about two workgroups a CU, a range of 512
// columns at least.
struct Split { int splits, per; };
Split shrink_split(int tiles, int cols) {
  int s = 512 / tiles, most = (cols + 511) / 512;
  s = s < most ? s : most;
  s = s < 1 ? 1 : s;
  Split p;
  p.per = ((cols + s - 1) / s + 255) / 256 * 256;
  p.splits = (cols + p.per - 1) / p.per;
  return p;
}

// The workspace: bounds that hold for every number of tokens up to C, so that it
// serves fewer too.  With ranges (512 / tiles, tiles > C / 64) the partial sums are
// those of 512 * 64 tokens at most, and there are four chunks a batch, or one to
// 2048 tokens, besides every adapter's last.
struct AdapterWs { size_t part, u, turned, suma, sumb, total; int64_t turn_pitch, turn_stride; };
AdapterWs adapter_ws(const moe_adapter_bank* b, int C) {
  const int64_t s = dense_size(b->dtype);
  const int64_t most = ((b->cols > b->rows ? b->cols : b->rows) + 511) / 512;
  const int64_t rows = C * most < 512 * 64 ? C * most : C > 512 * 64 ? C : 512 * 64;
  const int64_t four = C / 256 < 4 ? C / 256 : 4, chunks = (C / 2048 > four ? C / 2048 : four) + (C < b->adapters ? C : b->adapters);
  AdapterWs w;
  size_t o = 0;
  w.part = o; o = align256(o + (size_t)rows * b->rank * sizeof(float));
  w.u = o; o = align256(o + (size_t)C * b->rank * sizeof(float));
  w.turn_pitch = (b->rows * s + 15) / 16 * 16;
  w.turn_stride = w.turn_pitch * b->rank;
  w.turned = o; o = align256(o + (size_t)b->adapters * w.turn_stride);
  w.suma = o; o = align256(o + (size_t)chunks * b->rank * b->cols * sizeof(float));
  w.sumb = o; o = align256(o + (size_t)chunks * b->rank * b->rows * sizeof(float));
  w.total = o;
  return w;
}

template <int DT, int TT, bool DROP>
void launch_shrink_t(const AArgs& a, int tiles, hipStream_t st) {
  const dim3 grid((unsigned)tiles, (unsigned)a.splits);
  if (a.r <= 16) hipLaunchKernelGGL((k_ashrink<DT, 1, TT, DROP>), grid, dim3(kAWG), 0, st, a);
  else if (a.r <= 32) hipLaunchKernelGGL((k_ashrink<DT, 2, TT, DROP>), grid, dim3(kAWG), 0, st, a);
  else if (a.r <= 64) hipLaunchKernelGGL((k_ashrink<DT, 4, TT, DROP>), grid, dim3(kAWG), 0, st, a);
  else hipLaunchKernelGGL((k_ashrink<DT, 8, TT, DROP>), grid, dim3(kAWG), 0, st, a);
}
template <int DT>
void launch_shrink(const AArgs& a, int tiles, bool drop, hipStream_t st) {
  if (plan_tile(a.C) == 16) {
    if (drop) launch_shrink_t<DT, 1, true>(a, tiles, st);
    else launch_shrink_t<DT, 1, false>(a, tiles, st);
  } else {
    if (drop) launch_shrink_t<DT, 4, true>(a, tiles, st);
    else launch_shrink_t<DT, 4, false>(a, tiles, st);
  }
}

template <int DT, bool BWD>
void launch_expand(const AArgs& a, int tiles, bool drop, hipStream_t st) {
  // blocks of 128 columns, one or more to a wave, about two workgroups a CU
  const int blocks = a.cols > 0 ? (a.cols + 511) / 512 : 1;
  int y = 512 / tiles;
  y = y < 1 ? 1 : y > blocks ? blocks : y;
  const dim3 grid((unsigned)tiles, (unsigned)y);
  const int T = plan_tile(a.C), r32 = (a.r + 31) / 32 * 32;
  const size_t lds = (size_t)T * r32 * (DT == MOE_DT_F32 ? 4 : 6);
  if (T == 16) {
    if (drop) hipLaunchKernelGGL((k_aexpand<DT, 1, BWD, true>), grid, dim3(kAWG), lds, st, a);
    else hipLaunchKernelGGL((k_aexpand<DT, 1, BWD, false>), grid, dim3(kAWG), lds, st, a);
  } else {
    if (drop) hipLaunchKernelGGL((k_aexpand<DT, 4, BWD, true>), grid, dim3(kAWG), lds, st, a);
    else hipLaunchKernelGGL((k_aexpand<DT, 4, BWD, false>), grid, dim3(kAWG), lds, st, a);
  }
}

template <int DT, bool DROP>
void launch_outer_t(const AArgs& a, int chunks, hipStream_t st) {
  const dim3 grid((unsigned)((a.cols + 127) / 128), (unsigned)chunks, (unsigned)((a.r + 63) / 64));
  if (a.r <= 16) hipLaunchKernelGGL((k_aouter<DT, 1, DROP>), grid, dim3(kAWG), 0, st, a);
  else if (a.r <= 32) hipLaunchKernelGGL((k_aouter<DT, 2, DROP>), grid, dim3(kAWG), 0, st, a);
  else hipLaunchKernelGGL((k_aouter<DT, 4, DROP>), grid, dim3(kAWG), 0, st, a);
}
template <int DT>
void launch_outer(const AArgs& a, int chunks, bool drop, hipStream_t st) {
  if (drop) launch_outer_t<DT, true>(a, chunks, st);
  else launch_outer_t<DT, false>(a, chunks, st);
}

template <bool TURN>
void launch_reduce(const RArgs& a, hipStream_t st) {
  const int64_t n = (int64_t)a.r * a.cols;
  const unsigned x = (unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
  hipLaunchKernelGGL((k_areduce<TURN>), dim3(x, (unsigned)a.n), dim3(256), 0, st, a);
}

// fn(dtype constant)
template <typename F>
void by_dtype(int dtype, F fn) {
  if (dtype == MOE_DT_F32) fn(std::integral_constant<int, MOE_DT_F32>());
  else if (dtype == MOE_DT_BF16) fn(std::integral_constant<int, MOE_DT_BF16>());
  else fn(std::integral_constant<int, MOE_DT_F16>());
}

// The bank's tensors, the plan and the seed, which no output may overlap.
struct Reads { Rows r[5]; };
Reads adapter_reads(const moe_adapter_bank* b, const void* plan, size_t plan_bytes, const uint64_t* rng) {
  const int64_t s = dense_size(b->dtype), n = b->adapters - 1;
  return Reads{{span(b->a, (n * b->a_stride + (b->rank - 1) * b->a_pitch + b->cols) * s),
                span(b->b, (n * b->b_stride + (b->rows - 1) * b->b_pitch + b->rank) * s),
                span(b->scales, 4 * (int64_t)b->adapters), span(plan, (int64_t)plan_bytes), span(rng, 16)}};
}

// The checks that both directions make, and the arguments that they share.
struct Call {
  AArgs a;
  PlanLayout at;
  AdapterWs ws;
  uint8_t* w8;
  int64_t s;
};
moe_status adapter_call(const moe_adapter_bank* b, const void* plan, size_t plan_bytes, int32_t C, double p,
                        const uint64_t* rng, void* ws, size_t ws_bytes, Call& c) {
  moe_status st = dropout_of(p, rng, c.a.drop);
  if (st != MOE_OK) return st;
  c.at = plan_layout(C, b->adapters);
  if (!plan || (uintptr_t)plan % 256 || plan_bytes < (size_t)c.at.total * sizeof(int32_t)) return MOE_ERR_WORKSPACE;
  c.ws = adapter_ws(b, C);
  if (!ws || (uintptr_t)ws % 256 || ws_bytes < c.ws.total) return MOE_ERR_WORKSPACE;
  c.s = dense_size(b->dtype);
  c.w8 = static_cast<uint8_t*>(ws);
  c.a.plan = static_cast<const int32_t*>(plan);
  c.a.at = c.at;
  c.a.C = C; c.a.n = b->adapters; c.a.r = b->rank;
  c.a.scales = b->scales;
  c.a.part = reinterpret_cast<float*>(c.w8 + c.ws.part);
  return MOE_OK;
}

}  // namespace
}  // namespace rf4

using namespace rf4;

extern "C" {

size_t moe_adapter_plan_size(int32_t C, int32_t adapters) {
  if (C < 1 || C > MOE_MAX_BATCH_TOKENS || adapters < 1 || adapters > MOE_MAX_ADAPTERS) return 0;
  return align256((size_t)plan_layout(C, adapters).total * sizeof(int32_t));
}

moe_status moe_adapter_plan(const int32_t* token_adapter, int32_t C, int32_t adapters, void* plan, size_t plan_bytes,
                            void* stream) {
  if (C < 1 || C > MOE_MAX_BATCH_TOKENS || adapters < 1 || adapters > MOE_MAX_ADAPTERS) return MOE_ERR_UNSUPPORTED;
  if (!token_adapter || (uintptr_t)token_adapter % 4) return MOE_ERR_INVALID_ARG;
  PArgs a;
  a.at = plan_layout(C, adapters);
  if (!plan || (uintptr_t)plan % 256 || plan_bytes < (size_t)a.at.total * sizeof(int32_t)) return MOE_ERR_WORKSPACE;
  if (overlap(token_adapter, 4 * (int64_t)C, plan, 4 * a.at.total)) return MOE_ERR_INVALID_ARG;
  a.who = token_adapter;
  a.C = C; a.n = adapters;
  a.tile = plan_tile(C); a.chunk = plan_chunk(C);
  a.plan = static_cast<int32_t*>(plan);
  hipLaunchKernelGGL(k_aplan, dim3(1), dim3(kPlanWG), 0, reinterpret_cast<hipStream_t>(stream), a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

size_t moe_adapter_workspace_size(const moe_adapter_bank* b, int32_t C) {
  if (adapter_status(b) != MOE_OK || C < 1 || C > MOE_MAX_BATCH_TOKENS) return 0;
  return adapter_ws(b, C).total;
}

moe_status moe_adapter_fwd(const moe_adapter_bank* b, const void* plan, size_t plan_bytes, const void* x,
                           int64_t x_pitch, int32_t C, const void* base, int64_t base_pitch, void* y, int64_t y_pitch,
                           float* hidden, double p, const uint64_t* rng, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = adapter_status(b);
  if (st != MOE_OK) return st;
  if (C < 1 || C > MOE_MAX_BATCH_TOKENS) return MOE_ERR_UNSUPPORTED;
  const int64_t s = dense_size(b->dtype);
  const Rows rx = {x, x_pitch, b->cols, C, s}, rb = {base, base_pitch, b->rows, C, s}, ry = {y, y_pitch, b->rows, C, s};
  const Rows rh = {hidden, b->rank, b->rank, C, 4};
  if ((st = rows_status(rx)) != MOE_OK || (st = rows_status(ry)) != MOE_OK) return st;
  if (base && (st = rows_status(rb)) != MOE_OK) return st;
  if (hidden && (st = rows_status(rh)) != MOE_OK) return st;
  if (share(rx, ry) || (share(rb, ry) && !same(rb, ry)) || share(rh, ry) || share(rh, rx) || share(rh, rb))
    return MOE_ERR_INVALID_ARG;
  const Rows outs[] = {ry, rh, span(ws, (int64_t)ws_bytes)};
  const Rows tensors[] = {rx, ry, rb, rh};
  if (any_share(outs, adapter_reads(b, plan, plan_bytes, p > 0 ? rng : nullptr).r) || any_share({outs[2]}, tensors)) return MOE_ERR_INVALID_ARG;
  Call c = {};
  if ((st = adapter_call(b, plan, plan_bytes, C, p, rng, ws, ws_bytes, c)) != MOE_OK) return st;
  hipStream_t q = reinterpret_cast<hipStream_t>(stream);
  by_dtype(b->dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    AArgs a = c.a;
    const Split f = shrink_split(c.at.max_tiles, b->cols);
    a.splits = f.splits; a.per_split = f.per;
    a.cols = b->cols;
    a.in = static_cast<const uint8_t*>(x); a.in_pitch = x_pitch * s;
    a.w = static_cast<const uint8_t*>(b->a); a.w_stride = b->a_stride * s; a.w_pitch = b->a_pitch * s;
    launch_shrink<DT>(a, c.at.max_tiles, a.drop.drop != 0, q);
    a.cols = b->rows;
    a.w = static_cast<const uint8_t*>(b->b); a.w_stride = b->b_stride * s; a.w_pitch = b->b_pitch * s;
    a.base = static_cast<const uint8_t*>(base); a.base_pitch = base_pitch * s;
    a.out = static_cast<uint8_t*>(y); a.out_pitch = y_pitch * s;
    a.keep = hidden;
    launch_expand<DT, false>(a, c.at.max_tiles, false, q);
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

moe_status moe_adapter_bwd(const moe_adapter_bank* b, const void* plan, size_t plan_bytes, const void* x,
                           int64_t x_pitch, const float* hidden, const void* dy, int64_t dy_pitch, int32_t C,
                           const void* base, int64_t base_pitch, void* dx, int64_t dx_pitch, float* da, float* db,
                           int32_t accumulate, double p, const uint64_t* rng, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = adapter_status(b);
  if (st != MOE_OK) return st;
  if (C < 1 || C > MOE_MAX_BATCH_TOKENS) return MOE_ERR_UNSUPPORTED;
  const int64_t s = dense_size(b->dtype), r = b->rank;
  const Rows rx = {x, x_pitch, b->cols, C, s}, rd = {dy, dy_pitch, b->rows, C, s};
  const Rows rb = {base, base_pitch, b->cols, C, s}, rg = {dx, dx_pitch, b->cols, C, s};
  const Rows rh = {hidden, r, r, C, 4};
  const Rows ga = {da, r * b->cols, r * b->cols, b->adapters, 4}, gb = {db, r * b->rows, r * b->rows, b->adapters, 4};
  if (!dx && !da && !db) return MOE_ERR_INVALID_ARG;
  if ((st = rows_status(rd)) != MOE_OK) return st;
  if (dx && (st = rows_status(rg)) != MOE_OK) return st;
  if (dx && base && (st = rows_status(rb)) != MOE_OK) return st;
  if (da && (st = rows_status(rx)) != MOE_OK) return st;
  if (db && (st = rows_status(rh)) != MOE_OK) return st;
  if ((uintptr_t)da % 4 || (uintptr_t)db % 4) return MOE_ERR_INVALID_ARG;
  const Rows outs[] = {rg, ga, gb, span(ws, (int64_t)ws_bytes)};
  const Rows ins[] = {rd, da ? rx : Rows{}, db ? rh : Rows{}};
  const Rows grads[] = {rg, ga, gb, dx ? rb : Rows{}};
  if (any_share(outs, ins) || any_share({outs[3]}, grads) ||
      any_share(outs, adapter_reads(b, plan, plan_bytes, p > 0 ? rng : nullptr).r))
    return MOE_ERR_INVALID_ARG;
  if (share(rg, ga) || share(rg, gb) || share(ga, gb)) return MOE_ERR_INVALID_ARG;
  if (dx && base && ((share(rb, rg) && !same(rb, rg)) || share(rb, ga) || share(rb, gb))) return MOE_ERR_INVALID_ARG;
  Call c = {};
  if ((st = adapter_call(b, plan, plan_bytes, C, p, rng, ws, ws_bytes, c)) != MOE_OK) return st;
  hipStream_t q = reinterpret_cast<hipStream_t>(stream);
  const bool drop = c.a.drop.drop != 0;
  float* u = reinterpret_cast<float*>(c.w8 + c.ws.u);
  by_dtype(b->dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    AArgs a = c.a;
    if (dx || da) {
      TArgs t = {};
      t.plan = a.plan; t.at = c.at;
      t.C = C; t.n = b->adapters; t.r = b->rank; t.rows = b->rows;
      t.b = static_cast<const uint8_t*>(b->b); t.b_stride = b->b_stride * s; t.b_pitch = b->b_pitch * s;
      t.out = c.w8 + c.ws.turned; t.out_stride = c.ws.turn_stride; t.pitch = c.ws.turn_pitch;
      hipLaunchKernelGGL((k_aturn<kBytes<DT>>), dim3((unsigned)((b->rows + 63) / 64), (unsigned)b->adapters), dim3(256), 0,
                         q, t);
      const Split f = shrink_split(c.at.max_tiles, b->rows);
      a.splits = f.splits; a.per_split = f.per;
      a.cols = b->rows;
      a.in = static_cast<const uint8_t*>(dy); a.in_pitch = dy_pitch * s;
      a.w = t.out; a.w_stride = t.out_stride; a.w_pitch = t.pitch;
      launch_shrink<DT>(a, c.at.max_tiles, false, q);
      a.cols = b->cols;
      a.w = static_cast<const uint8_t*>(b->a); a.w_stride = b->a_stride * s; a.w_pitch = b->a_pitch * s;
      a.base = dx ? static_cast<const uint8_t*>(base) : nullptr; a.base_pitch = base_pitch * s;
      a.out = static_cast<uint8_t*>(dx); a.out_pitch = dx_pitch * s;
      a.keep = u;
      if (!dx) a.cols = 0;              // u alone
      launch_expand<DT, true>(a, c.at.max_tiles, drop, q);
    }
    if (da) {
      a.cols = b->cols;
      a.in = static_cast<const uint8_t*>(x); a.in_pitch = x_pitch * s;
      a.small = u;
      a.sums = reinterpret_cast<float*>(c.w8 + c.ws.suma);
      launch_outer<DT>(a, c.at.max_chunks, drop, q);
    }
    if (db) {
      a.cols = b->rows;
      a.in = static_cast<const uint8_t*>(dy); a.in_pitch = dy_pitch * s;
      a.small = hidden;
      a.sums = reinterpret_cast<float*>(c.w8 + c.ws.sumb);
      launch_outer<DT>(a, c.at.max_chunks, false, q);
    }
  });
  RArgs r2 = {};
  r2.plan = c.a.plan; r2.at = c.at;
  r2.C = C; r2.n = b->adapters; r2.r = b->rank;
  r2.accumulate = accumulate;
  if (da) {
    r2.cols = b->cols;
    r2.sums = reinterpret_cast<const float*>(c.w8 + c.ws.suma);
    r2.out = da;
    r2.factor = c.a.drop.scale;
    launch_reduce<false>(r2, q);
  }
  if (db) {
    r2.cols = b->rows;
    r2.sums = reinterpret_cast<const float*>(c.w8 + c.ws.sumb);
    r2.out = db;
    r2.factor = 1.0f;
    r2.scales = b->scales;
    launch_reduce<true>(r2, q);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // extern "C"
