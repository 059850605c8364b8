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
// stay in fp32.  The first product (x by A, dy by B) takes both sides as stored,
// fp16 on the fp16 matrix cores; fp32 tensors use the fp32 ones throughout: exact
// products, fp32 sums.  Beside 16-bit tensors t and u are operands in pieces:
//   bf16   three bf16 that sum to them exactly (24 bits): exact products again
//   fp16   y and dx: two fp16 terms under a power of two per token, that lose 2^-23
//          of a value, or 2^-39 of the token's largest (a rank whose t is that far
//          below the others' loses its bits, which a large B shows in y);
//          dA and dB: the three bf16, by the two that an fp16 element is (11 bits as
//          8 + 3), without the product of the lowest two, below 2^-22 of the whole
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
//   k_apieces   t and u laid out as operands
//   k_aouter    dA and dB of a chunk's tokens, 128 columns (fp32: 64) to a workgroup
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
// Tokens to a chunk: eight chunks in a batch, 256 .. 2048 tokens each.
inline int plan_chunk(int C) {
  int q = 256;
  while (q < 2048 && q * 8 < C) q *= 2;
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

// One workgroup, since tokens keep their order without any exchange between workgroups:
// 64 tokens of 24 adapters 5.6 us, 8192 of 4 16; a batch's once, for all projections.  Its
// time is the last loop's, over the adapters among 64 tokens: 8192 of 48 56 us.
// Eight waves take an eighth of the tokens each, count them by
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
// (What is left of an infinity or NaN is NaN.)
__device__ __forceinline__ void pieces3(float v, uint32_t& a, uint32_t& b, uint32_t& c) {
  a = __float_as_uint(v) & 0xFFFF0000u;
  const float r = v - __uint_as_float(a);
  b = __float_as_uint(r) & 0xFFFF0000u;
  c = __float_as_uint(r - __uint_as_float(b));
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
      const uint32_t b0 = __float_as_uint(f0 - __uint_as_float(a0)), b1 = __float_as_uint(f1 - __uint_as_float(a1));
      p[0][i] = high_pair(a0, a1);
      p[1][i] = high_pair(b0, b1);       // of an infinity: NaN
    }
  } else {
    p[0] = v;
  }
}

// c += (the sum of small's pieces) * (the sum of big's).  Of fp16's six products that of
// the two lowest pieces is left out: they are truncations, below 2^-15 of a value and at
// most 7 2^-10 of an fp16 element, so 2^-22.2 of their product at most, of its sign.
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
// Entry i of a list (i < its room in the plan, whatever the plan says); false where
// the plan has no such entry or is of another batch: then nothing is done.
__device__ __forceinline__ bool plan_entry(const int32_t* plan, int C, int n, int slot, int64_t list, int i, Tile& t) {
  const int4 h = *reinterpret_cast<const int4*>(plan), v = *reinterpret_cast<const int4*>(plan + list + 4 * (int64_t)i);
  const int most = slot == 3 ? h.w : plan[4];
  t = Tile{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y), __builtin_amdgcn_readfirstlane(v.z)};
  return h.x == kPlanMagic && h.y == C && h.z == n && i < most;
}

// Tiles of 16 columns that a wave takes in k_aexpand and k_aouter: a lane has that
// many consecutive ones, 16 bytes.
template <int DT>
constexpr int kTiles = DT == MOE_DT_F32 ? 4 : 8;

__device__ const uint32_t __attribute__((aligned(16))) kZeroRow[8] = {};

struct AArgs {
  const int32_t* plan;
  PlanLayout at;
  int C, n, r;
  // shrink: in [C][cols] by w [n][r][cols]; expand: out [C][cols] from w [n][cols][r] or (BWD) [n][r][cols]
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
  float* part;                          // [splits][C][r] in the plan's order
  int splits, per_split;                // column ranges, columns in each (multiple of 256)
  float* keep;                          // expand: the finished sums [C][r] by token, or NULL
  int column_parts;                     // expand: workgroups to a tile
  Dropout drop;
};

// ---------------------------------------------------------------------------
// t = x A^T over a range of columns
// ---------------------------------------------------------------------------
// A workgroup has a tile's tokens, 64 ranks at most and a range of columns, of which
// its waves take 32 in turn; a wave loads the next columns before it multiplies the
// last.  Bound by x and, once a tile, A: 4096 bf16 tokens x 7168 of 8 adapters of rank 64
// 23.8 us, 118 MB together.  (64 at a time, whole lines of 16-bit rows, took more
// registers than two waves a SIMD have: 8192 fp16 tokens x 3584, rank 64, with dropout
// 36 us against 28.  fp32 with dropout, tiles of 64 tokens and more than 32 ranks takes
// more than half of a SIMD's registers, one wave.)
template <int DT, int NT, int TT, bool DROP>
__global__ __launch_bounds__(kAWG) void k_ashrink(AArgs a) {
  constexpr int B = kBytes<DT>, T = 16 * TT, S = 1, U = 32 * S;   // steps and columns of a wave's turn
  __shared__ float s_red[2][T][NT * 16];
  Tile t;
  if (!plan_entry(a.plan, a.C, a.n, 3, a.at.tiles, blockIdx.x, t) || t.who < 0) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane & 15, quarter = lane >> 4;
  const int r0 = 64 * blockIdx.z, ranks = a.r - r0 < 64 ? a.r - r0 : 64;
  Counter ctr = {};
  if constexpr (DROP) ctr = counter_of(a.drop.rng);
  const uint8_t *xr[TT], *ar[NT];
  int token[TT];
  // rows past the last repeat it: their sums are not used
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int k = 16 * i + row;
    token[i] = a.plan[a.at.perm + t.first + (k < t.count ? k : t.count - 1)];
    xr[i] = a.in + token[i] * a.in_pitch + 8 * quarter * B;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int k = 16 * j + row;
    ar[j] = a.w + t.who * a.w_stride + (r0 + (k < ranks ? k : ranks - 1)) * a.w_pitch + 8 * quarter * B;
  }
  float4v acc[TT][NT];
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = float4v(0.0f);
  const int c0 = blockIdx.y * a.per_split, c1 = c0 + a.per_split < a.cols ? c0 + a.per_split : a.cols;
  struct Turn { Eight<DT> x[S][TT], w[S][NT]; };
  auto load = [&](int c, Turn& u) {
#pragma unroll
    for (int q = 0; q < S; ++q) {
#pragma unroll
      for (int i = 0; i < TT; ++i) u.x[q][i] = load8<DT>(xr[i] + (int64_t)(c + 32 * q) * B);
#pragma unroll
      for (int j = 0; j < NT; ++j) u.w[q][j] = load8<DT>(ar[j] + (int64_t)(c + 32 * q) * B);
    }
  };
  auto multiply = [&](int c, Turn& u, int q) {
    if constexpr (DROP) {
#pragma unroll
      for (int i = 0; i < TT; ++i) u.x[q][i] = drop8<DT>(u.x[q][i], a.drop, ctr, c + 32 * q + 8 * quarter, (uint32_t)token[i]);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mma8<DT>(u.x[q][i], u.w[q][j], acc[i][j]);
  };
  const int whole = c1 - (c1 - c0) % U;      // whole turns end here
  int c = c0 + U * wave;
  Turn u, v;
  if (c < whole) load(c, u);
  for (; c < whole; c += 4 * U) {
    if (c + 4 * U < whole) load(c + 4 * U, v);
#pragma unroll
    for (int q = 0; q < S; ++q) multiply(c, u, q);
    u = v;
  }
  if (whole < c1 && (whole - c0) / U % 4 == wave) {
    // a row's last columns, zeros behind them
    for (int q = 0; q < S && whole + 32 * q < c1; ++q) {
      const int k = whole + 32 * q;
#pragma unroll
      for (int i = 0; i < TT; ++i) u.x[0][i] = load8_of<DT>(xr[i] - 8 * quarter * B, k + 8 * quarter, c1);
#pragma unroll
      for (int j = 0; j < NT; ++j) u.w[0][j] = load8_of<DT>(ar[j] - 8 * quarter * B, k + 8 * quarter, c1);
      multiply(k, u, 0);
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
    float* o = a.part + ((int64_t)blockIdx.y * a.C + t.first) * a.r + r0;
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 16 * i + 4 * quarter + e;
        if (k >= t.count) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (16 * j + row < ranks) o[(int64_t)k * a.r + 16 * j + row] = acc[i][j][e];
      }
  }
}

// ---------------------------------------------------------------------------
// y = base + s B t, dx = base + drop'(A^T u)
// ---------------------------------------------------------------------------
// A wave's lane l holds, of 128 (fp32: 64) columns, eight (four) consecutive ones from
// 8 (l % 16) on: as tile i those 8 (l % 16) + i, so that B's and A's rows are read,
// and y's written, 16 bytes at a time.  The columns' rows of B (or columns of A)
// stay in registers for all of the tile's tokens, 16 at a time.
// Bound by latency, then by base and y: 4096 bf16 tokens x 3584, rank 64, 25.7 us for 58
// MB, all workgroups at once; 8192 fp16 x 7168 70 us for 235 MB, 3.3 TB/s.
// Registers: ranks above 64 take more than half of a SIMD's, one wave; dx of ranks 33 to 64
// with dropout in 16 bits keeps two waves and puts 28 bytes a lane into scratch (8192 x
// 3584: 47 us).
// For fp16, t and u are two fp16 terms under a power of two per token that puts the
// token's largest at 2^14 or more and below 2^15: the first leaves half a step of 11 bits,
// the second half a step of that, 2^-23 of a value, or half of fp16's smallest, 2^-39 of
// the largest; for bf16 three bf16 pieces, exact.
//
// sum += the partial sums of a tile's tokens tid / 16 + 16 i, ranks 32 q + 2 (tid % 16)
// and the next, over all ranges in order, U of them at a time.
template <int SUBS, int KT, int U>
__device__ __forceinline__ void add_ranges(const AArgs& a, const Tile& t, float (&sum)[4][KT][2], int tid) {
  const int row = tid & 15;
  const int64_t range = (int64_t)a.C * a.r;
  const float* p = a.part + (int64_t)t.first * a.r;
  uint32_t at[SUBS][KT][2];
#pragma unroll
  for (int i = 0; i < SUBS; ++i) {
    const int k = (tid >> 4) + 16 * i;
#pragma unroll
    for (int q = 0; q < KT; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 32 * q + 2 * row + e;
        at[i][q][e] = (uint32_t)((k < t.count ? k : t.count - 1) * a.r + (j < a.r ? j : a.r - 1));
      }
  }
  for (int x = 0; x < a.splits; x += U) {
    float w[U][SUBS][KT][2];
#pragma unroll
    for (int y = 0; y < U; ++y) {
      const float* f = p + (x + y < a.splits ? x + y : x) * range;
#pragma unroll
      for (int i = 0; i < SUBS; ++i)
#pragma unroll
        for (int q = 0; q < KT; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) w[y][i][q][e] = f[at[i][q][e]];
    }
#pragma unroll
    for (int y = 0; y < U; ++y) {
      if (x + y >= a.splits) break;
#pragma unroll
      for (int i = 0; i < SUBS; ++i)
#pragma unroll
        for (int q = 0; q < KT; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) sum[i][q][e] += w[y][i][q][e];
    }
  }
}

template <int DT, int KT, bool BWD, bool DROP>
__global__ __launch_bounds__(kAWG, KT <= 2 ? 2 : 1) void k_aexpand(AArgs a) {
  constexpr int B = kBytes<DT>, NTL = kTiles<DT>, W = 16 * NTL, P = DT == MOE_DT_F32 ? 1 : DT == MOE_DT_F16 ? 2 : 3;
  // the sums as operands, [piece][rank / 8][token][8], and the tokens
  extern __shared__ __align__(16) uint8_t s_t[];
  __shared__ int s_token[64];
  __shared__ float s_inv[64];
  // workgroups b, b + 8, .. run on one XCD: those of one tile, which read the same
  // partial sums, follow each other on one
  const int run = blockIdx.x >> 3, part = run % a.column_parts, tile = run / a.column_parts * 8 + (blockIdx.x & 7);
  Tile t;
  if (tile >= a.at.max_tiles || !plan_entry(a.plan, a.C, a.n, 3, a.at.tiles, tile, t)) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = lane & 15, quarter = lane >> 4;
  const int subs = (t.count + 15) / 16, T = 16 * subs;
  const bool idle = t.who < 0;
  const float s = idle ? 0.0f : a.scales ? a.scales[t.who] : 1.0f;
  const uint8_t* w = a.w + (idle ? 0 : t.who) * a.w_stride;
  Eight<DT> f[KT][NTL];                 // tile i of rank 32 k + 8 quarter .. + 7: column c + i
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(kZeroRow);     // ranks past the last
  // (One branch for all of a set of loads, here and below: a branch at each would keep
  // them from being on their way together.)
  auto operands = [&](int c0) {
    const int c = c0 + NTL * row;
    if constexpr (!BWD) {
      auto column = [&](int i) { return w + (c + i < a.cols ? c + i : a.cols - 1) * a.w_pitch; };
      if (a.r % 8 == 0) {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const int j0 = 32 * k + 8 * quarter;
#pragma unroll
          for (int i = 0; i < NTL; ++i) f[k][i] = load8<DT>(j0 < a.r ? column(i) + j0 * B : zeros);
        }
      } else if (a.r > 8) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int i = 0; i < NTL; ++i) f[k][i] = load8_of<DT>(column(i), 32 * k + 8 * quarter, a.r);
      } else if (c0 + W + 7 <= a.cols) {
        // what a load takes behind a row's end, seven elements at most, lies in the matrix:
        // seven rows of one element at least follow these columns'
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const int j0 = 32 * k + 8 * quarter;
#pragma unroll
          for (int i = 0; i < NTL; ++i) f[k][i] = load8_first<DT>(j0 < a.r ? column(i) + j0 * B : zeros, a.r - j0);
        }
      } else {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const int j0 = 32 * k + 8 * quarter;
#pragma unroll
          for (int i = 0; i < NTL; ++i) f[k][i] = load8_some<DT>(column(i) + j0 * B, a.r - j0);
        }
      }
    } else {
      uint4v g[KT][8];                  // rank 32 k + 8 quarter + i, columns c ..
      auto rank = [&](int j) { return w + j * a.w_pitch + (int64_t)c * B; };
      if (c0 + W <= a.cols) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = 32 * k + 8 * quarter + i;
            g[k][i] = load16(j < a.r ? rank(j) : zeros);
          }
      } else {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = 32 * k + 8 * quarter + i;
            g[k][i] = load16_of<DT>(w + (j < a.r ? j : a.r - 1) * a.w_pitch, j < a.r ? c : a.cols, a.cols);
          }
      }
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        if constexpr (DT == MOE_DT_F32) {
#pragma unroll
          for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) f[k][i].v[e >> 2][e & 3] = g[k][e][i];
        } else {
          uint4v o[8];
          turn8(g[k], o);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[k][i].v[0] = o[i];
        }
      }
    }
  };
  int c0 = W * (part * 4 + wave);
  const int step = 4 * W * a.column_parts;
  // base's rows of 16 tokens, loaded while those before are multiplied; the first
  // before anything else
  uint4v old[4], next[4];
  auto base_rows = [&](const int (&token)[4], int c0) {
    const int c = c0 + NTL * row;
    if (c0 + W <= a.cols) {
#pragma unroll
      for (int e = 0; e < 4; ++e) next[e] = load16(a.base + token[e] * a.base_pitch + (int64_t)c * B);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) next[e] = load16_of<DT>(a.base + token[e] * a.base_pitch, c, a.cols);
    }
  };
  if (a.base && c0 < a.cols) {
    int token[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) token[e] = a.plan[a.at.perm + t.first + (4 * quarter + e < t.count ? 4 * quarter + e : t.count - 1)];
    base_rows(token, c0);
  }
  if (!idle && c0 < a.cols) operands(c0);
  // t (or u) of the tile: 16 lanes to a token, two ranks a lane and 32
  if (tid < T) s_token[tid] = a.plan[a.at.perm + t.first + (tid < t.count ? tid : t.count - 1)];
  float sum[4][KT][2];                  // of tokens tid / 16 + 16 i
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < KT; ++q) sum[i][q][0] = sum[i][q][1] = 0.0f;
  if (!idle) {
    // as many ranges' loads on their way together as 64 registers hold
    if (subs == 1) add_ranges<1, KT, 16 / KT>(a, t, sum, tid);
    else add_ranges<4, KT, 8 / KT>(a, t, sum, tid);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= subs) break;
    const int k = (tid >> 4) + 16 * i;
    float v[KT][2];
#pragma unroll
    for (int q = 0; q < KT; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // forward: t, then times s_a; backward: u
        const bool live = k < t.count && 32 * q + 2 * row + e < a.r;
        v[q][e] = live ? sum[i][q][e] * (BWD ? s : a.drop.scale) : 0.0f;
      }
    if (a.keep && part == 0 && k < t.count) {
      float* o = a.keep + (int64_t)a.plan[a.at.perm + t.first + k] * a.r;
#pragma unroll
      for (int q = 0; q < KT; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (32 * q + 2 * row + e < a.r) o[32 * q + 2 * row + e] = v[q][e];
    }
    float m = 1.0f;
    if constexpr (DT == MOE_DT_F16) {
      uint32_t most = 0;
#pragma unroll
      for (int q = 0; q < KT; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!BWD) v[q][e] *= s;
          const uint32_t b = __float_as_uint(v[q][e]) & 0x7FFFFFFFu;
          most = b > most ? b : most;
        }
#pragma unroll
      for (int d = 8; d >= 1; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)most, d, 16);
        most = o > most ? o : most;
      }
      // the power of two that takes it below 2^15, within fp32's normal range
      int e = 14 - ((int)(most >> 23) - 127);
      if (most >= 0x7F800000u) e = 0;
      e = e > 126 ? 126 : e;
      m = __uint_as_float((uint32_t)(127 + e) << 23);
      if (row == 0) s_inv[k] = __uint_as_float((uint32_t)(127 - e) << 23);
    } else if constexpr (!BWD) {
#pragma unroll
      for (int q = 0; q < KT; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) v[q][e] *= s;
    }
#pragma unroll
    for (int q = 0; q < KT; ++q) {
      const int at = (((32 * q + 2 * row) >> 3) * T + k) * 8 + ((2 * row) & 7), piece = 32 * KT * T;
      if constexpr (DT == MOE_DT_F32) {
        *reinterpret_cast<float2*>(s_t + at * 4) = make_float2(v[q][0], v[q][1]);
      } else {
        uint32_t p[2][3] = {};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (DT == MOE_DT_F16) {
            // not finite: its own first term, and the finite ones beside it in range
            float z = v[q][e] * m;
            const bool fine = fabsf(z) < INFINITY;
            if (fine) z = fminf(fmaxf(z, -65504.0f), 65504.0f);
            const _Float16 h = (_Float16)z;
            p[e][0] = (uint32_t)__builtin_bit_cast(uint16_t, h) << 16;
            p[e][1] = fine ? (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)(z - (float)h)) << 16 : 0u;
          } else {
            pieces3(v[q][e], p[e][0], p[e][1], p[e][2]);
          }
        }
#pragma unroll
        for (int x = 0; x < P; ++x) *reinterpret_cast<uint32_t*>(s_t + (x * piece + at) * 2) = high_pair(p[0][x], p[1][x]);
      }
    }
  }
  __syncthreads();
  Counter ctr = {};
  if constexpr (DROP) ctr = counter_of(a.drop.rng);
  for (; c0 < a.cols; c0 += step) {
    const int c = c0 + NTL * row, left = a.cols - c;
    const bool whole = c0 + W <= a.cols;
    for (int sub = 0; sub < subs; ++sub) {
#pragma unroll
      for (int e = 0; e < 4; ++e) old[e] = next[e];
      // the next 16 tokens', or the next columns' first
      const bool last = sub + 1 == subs;
      if (a.base && (!last || c0 + step < a.cols)) {
        int token[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) token[e] = s_token[(last ? 0 : 16 * (sub + 1)) + 4 * quarter + e];
        base_rows(token, last ? c0 + step : c0);
      }
      float4v acc[NTL];
#pragma unroll
      for (int i = 0; i < NTL; ++i) acc[i] = float4v(0.0f);
      if (!idle) {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const int at = ((4 * k + quarter) * T + 16 * sub + row) * 8;
          if constexpr (DT == MOE_DT_F32) {
            const Eight<DT> u = *reinterpret_cast<const Eight<DT>*>(s_t + at * 4);
#pragma unroll
            for (int i = 0; i < NTL; ++i) acc[i] = mma8<DT>(u, f[k][i], acc[i]);
          } else {
            uint4v u[P];
#pragma unroll
            for (int p = 0; p < P; ++p) u[p] = *reinterpret_cast<const uint4v*>(s_t + (p * 32 * KT * T + at) * 2);
#pragma unroll
            for (int p = P - 1; p >= 0; --p)
#pragma unroll
              for (int i = 0; i < NTL; ++i) acc[i] = DT == MOE_DT_F16 ? mma_f16(u[p], f[k][i].v[0], acc[i]) : mma_bf16(u[p], f[k][i].v[0], acc[i]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 16 * sub + 4 * quarter + e, token = s_token[k];
        const float inv = DT == MOE_DT_F16 ? s_inv[k] : 1.0f;
        float v[NTL];
#pragma unroll
        for (int i = 0; i < NTL; ++i) v[i] = DT == MOE_DT_F16 ? acc[i][e] * inv : acc[i][e];
        if constexpr (BWD && DROP) drop_some<NTL>(v, a.drop, ctr, c, (uint32_t)token);
        if (a.base) {
          const Eight<DT> b = first_of<DT>(old[e]);
#pragma unroll
          for (int i = 0; i < NTL; ++i) v[i] = idle ? get8<DT>(b, i) : v[i] + get8<DT>(b, i);
        }
        if (k < t.count) {
          uint8_t* o = a.out + token * a.out_pitch + (int64_t)c * B;
          const uint4v q = pack16<DT>(v);
          if (whole) store16(o, q);
          else store16_some<DT>(o, q, left);
        }
      }
    }
    if (!idle && c0 + step < a.cols) operands(c0 + step);
  }
}

// ---------------------------------------------------------------------------
// sums[j][col] = sum over a chunk's tokens of small[token][j] in[token][col]
// ---------------------------------------------------------------------------
// dA (x by u) and dB (dy by t) in one launch.  A workgroup has 128 (fp32: 64) columns
// of a chunk; of its eight waves RH share the ranks, 16 NT each (32 at most: two waves
// to a SIMD), and the others the tokens, 32 at a time, whose rows are transposed in
// registers.  Bound by vector work at rank 64 (pieces of fp16, the generator): 8192 fp16
// tokens x (3584 + 7168) with dropout 110 us; 2048 bf16 x (7168 + 3584), rank 16, 19.
// (Four waves with 64 ranks each, which read and drop x once and not
// twice: 8192 fp16 tokens, rank 64, 122 us against 109.)
// u and t are needed by every workgroup of a chunk: k_apieces lays them out once as
// the first operand, [32 tokens][16 ranks][piece][lane], three bf16 pieces, or the
// two halves of eight fp32.
struct Outer {
  const uint8_t* in;                    // [C][cols]
  int64_t in_pitch;
  const float* small;                   // [C][r] by token
  uint8_t* pieces;                      // small laid out
  float* sums;                          // [chunks][r][cols]
  int cols, blocks;                     // of columns
};
struct OArgs {
  const int32_t* plan;
  PlanLayout at;
  int C, n, r;
  Outer da, db;                         // blocks 0: not asked for
  Dropout drop;                         // of da's input
};
template <int DT>
constexpr int kParts = DT == MOE_DT_F32 ? 2 : 3;
// The 32 tokens from step s of chunk q on have a place of their own: chunks start
// anywhere, and each may end in a partial step: C / 32 + chunks + 1 places in all.
__device__ __forceinline__ int64_t step_place(const Tile& t, int q, int s) { return t.first / 32 + q + s; }

template <int DT>
__global__ __launch_bounds__(256) void k_apieces(OArgs a) {
  const Outer& o = blockIdx.z == 0 && a.da.blocks ? a.da : a.db;
  Tile t;
  if (!plan_entry(a.plan, a.C, a.n, 4, a.at.chunks, blockIdx.y, t)) return;
  const int lane = threadIdx.x & 63, row = lane & 15, quarter = lane >> 4, s = blockIdx.x, tiles = (a.r + 15) / 16;
  if (32 * s >= t.count) return;
  int token[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = 32 * s + 8 * quarter + i;
    token[i] = a.plan[a.at.perm + t.first + (k < t.count ? k : t.count - 1)];
  }
  for (int j = threadIdx.x >> 6; j < tiles; j += 4) {
    const int rank = 16 * j + row;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = o.small[(int64_t)token[i] * a.r + (rank < a.r ? rank : a.r - 1)];
    // tokens behind the last, and ranks, are zeros
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * s + 8 * quarter + i >= t.count || rank >= a.r) v[i] = 0.0f;
    uint4v* out = reinterpret_cast<uint4v*>(o.pieces) + ((step_place(t, blockIdx.y, s) * tiles + j) * kParts<DT>) * 64 + lane;
    if constexpr (DT == MOE_DT_F32) {
      out[0] = uint4v{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      out[64] = uint4v{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else {
      uint4v m[3];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t p[2][3];
        pieces3(v[2 * i], p[0][0], p[0][1], p[0][2]);
        pieces3(v[2 * i + 1], p[1][0], p[1][1], p[1][2]);
#pragma unroll
        for (int q = 0; q < 3; ++q) m[q][i] = high_pair(p[0][q], p[1][q]);
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) out[64 * q] = m[q];
    }
  }
}

constexpr int kOWaves = 8;
template <int DT, int NT, int RH, bool DROP>
__global__ __launch_bounds__(64 * kOWaves, 2) void k_aouter(OArgs a) {
  constexpr int B = kBytes<DT>, NTL = kTiles<DT>, W = 16 * NTL, TG = kOWaves / RH, R = 16 * NT, P = kParts<DT>;
  extern __shared__ __align__(16) uint8_t s_o[];
  int* s_token = reinterpret_cast<int*>(s_o);                       // [2048], then the sums
  float* s_red = reinterpret_cast<float*>(s_o);                     // [TG / 2][RH][R][W + 4]
  Tile t;
  if (!plan_entry(a.plan, a.C, a.n, 4, a.at.chunks, blockIdx.y, t)) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int row = lane & 15, quarter = lane >> 4;
  const bool second = (int)blockIdx.x >= a.da.blocks;
  const Outer& o = second ? a.db : a.da;
  const int c0 = W * (blockIdx.x - (second ? a.da.blocks : 0)), c = c0 + NTL * row, left = o.cols - c;
  const bool whole = c0 + W <= o.cols, drops = DROP && !second;
  const int rh = wave % RH, tg = wave / RH, r0 = R * rh, tiles = (a.r + 15) / 16;
  Counter ctr = {};
  if constexpr (DROP) ctr = counter_of(a.drop.rng);
  // the tokens, the last again behind it up to whole steps
  const int steps = (t.count + 31) / 32;
  for (int i = tid; i < 32 * steps; i += 64 * kOWaves) s_token[i] = a.plan[a.at.perm + t.first + (i < t.count ? i : t.count - 1)];
  __syncthreads();
  float4v acc[NT][NTL];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NTL; ++j) acc[i][j] = float4v(0.0f);
  const uint4v* small = reinterpret_cast<const uint4v*>(o.pieces) + step_place(t, blockIdx.y, 0) * tiles * P * 64;
  struct Turn { uint4v g[8]; };
  uint4v m[NT][P];
  auto load = [&](int s, Turn& u) {
    const uint8_t* p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = o.in + s_token[32 * s + 8 * quarter + i] * o.in_pitch + (int64_t)c * B;
    if (whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u.g[i] = load16(p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) u.g[i] = load16_of<DT>(p[i] - (int64_t)c * B, c, o.cols);
    }
  };
  // (loaded as they are needed: a step ahead they take the registers of a second wave)
  auto small_of = [&](int s) {
    // (tiles past the last: the last again, whose sums are not used)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int k = r0 / 16 + j < tiles ? r0 / 16 + j : tiles - 1;
#pragma unroll
      for (int q = 0; q < P; ++q) m[j][q] = small[((int64_t)s * tiles + k) * (P * 64) + 64 * q + lane];
    }
  };
  auto multiply = [&](int s, Turn& u) {
    if (32 * s + 32 > t.count) {        // tokens behind the last add nothing
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (32 * s + 8 * quarter + i >= t.count) u.g[i] = uint4v(0u);
    }
    if (drops) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u.g[i] = drop16<DT>(u.g[i], a.drop, ctr, c, (uint32_t)s_token[32 * s + 8 * quarter + i]);
    }
    if constexpr (DT == MOE_DT_F32) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(m[j][e >> 2][e & 3]), __uint_as_float(u.g[e][i]),
                                                             acc[j][i], 0, 0, 0);
    } else {
      uint4v f[8];
      turn8(u.g, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4v b[kPieces<DT>];
        pieces<DT>(f[i], b);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j][i] = mma_pieces<DT>(m[j], b, acc[j][i]);
      }
    }
  };
  // (two sets by turns: a copy would wait for what is on its way)
  Turn even, odd;
  if (tg < steps) load(tg, even);
  for (int s = tg; s < steps; s += 2 * TG) {
    small_of(s);
    if (s + TG < steps) load(s + TG, odd);
    __builtin_amdgcn_sched_barrier(0);
    multiply(s, even);
    __builtin_amdgcn_sched_barrier(0);
    if (s + TG >= steps) break;
    small_of(s + TG);
    if (s + 2 * TG < steps) load(s + 2 * TG, even);
    __builtin_amdgcn_sched_barrier(0);
    multiply(s + TG, odd);
    __builtin_amdgcn_sched_barrier(0);
  }
  // the sums of the waves that share the tokens, in a fixed order
  float* mine = s_red + rh * R * (W + 4);
  constexpr int slot = RH * R * (W + 4);
#pragma unroll
  for (int h = TG / 2; h >= 1; h /= 2) {
    __syncthreads();
    if (tg >= h && tg < 2 * h) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < NTL; ++i) mine[(tg - h) * slot + (16 * j + 4 * quarter + e) * (W + 4) + NTL * row + i] = acc[j][i][e];
    }
    __syncthreads();
    if (tg < h) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < NTL; ++i) acc[j][i][e] += mine[tg * slot + (16 * j + 4 * quarter + e) * (W + 4) + NTL * row + i];
    }
  }
  if (tg == 0) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = r0 + 16 * j + 4 * quarter + e;
        if (k >= a.r) continue;
        float* p = o.sums + ((int64_t)blockIdx.y * a.r + k) * o.cols + c;
#pragma unroll
        for (int h = 0; h < NTL; h += 4) {
          const float q[4] = {acc[j][h][e], acc[j][h + 1][e], acc[j][h + 2][e], acc[j][h + 3][e]};
          if (whole) store16(p + h, pack16<MOE_DT_F32>(q));
          else store16_some<MOE_DT_F32>(p + h, pack16<MOE_DT_F32>(q), left - h);
        }
      }
  }
}

struct RArgs {
  const int32_t* plan;
  PlanLayout at;
  int C, n, r, accumulate;
  int ca, cb;                           // columns of dA, of dB; 0: not asked for
  int64_t xa;                           // workgroups of dA's
  const float *sa, *sb;                 // [chunks][r][columns]
  float *da, *db;                       // [n][r][ca], [n][cb][r]
  const float* scales;                  // dB's factor by adapter, or NULL
  float factor;                         // dA's
};

// Adds an adapter's chunks in order; an adapter without tokens has zeros.  dB is
// transposed on the way: a thread has a column's four ranks.  Bound by latency: 6.6 us
// for one adapter of rank 16 by 7168 + 3584 in eight chunks, 13.4 for four of rank 64.
__global__ __launch_bounds__(256) void k_areduce(RArgs a) {
  const int32_t* plan = a.plan;
  if (plan[0] != kPlanMagic || plan[1] != a.C || plan[2] != a.n) return;
  const bool second = blockIdx.x >= a.xa;
  const int64_t x = (int64_t)(second ? blockIdx.x - a.xa : blockIdx.x) * 256 + threadIdx.x;
  const int who = blockIdx.y;
  const int q0 = plan[a.at.first + who], q1 = plan[a.at.first + who + 1];
  if (a.accumulate && q0 == q1) return;
  const int cols = second ? a.cb : a.ca;
  const int64_t n = (int64_t)a.r * cols;
  const float f = second ? (a.scales ? a.scales[who] : 1.0f) : a.factor;
  // four elements: of a row of dA's sums, or (dB) of four rows, at one column
  const int64_t at = second ? (x / cols) * 4 * cols + x % cols : 4 * x, step = second ? cols : 1;
  if (second ? x / cols * 4 >= a.r : at >= n) return;
  const int most = second ? a.r - (int)(x / cols) * 4 : n - at < 4 ? (int)(n - at) : 4;
  float v[4] = {};
  const float* s = (second ? a.sb : a.sa) + at;
  // four chunks on their way together
  for (int q = q0; q < q1; q += 4) {
    float w[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* p = s + (q + k < q1 ? q + k : q0) * n;
      if (!second && most >= 4) {
        const uint4v x4 = load16(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[k][i] = __uint_as_float(x4[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[k][i] = p[i < most ? i * step : 0];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += q + k < q1 ? w[k][i] : 0.0f;
  }
  float* o = second ? a.db + who * n + x % cols * a.r + x / cols * 4 : a.da + who * n + at;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = q0 == q1 ? 0.0f : v[i] * f;   // no tokens: zeros, whatever an unused adapter's scale is
    if (a.accumulate && i < most) v[i] += o[i];
  }
  store16_some<MOE_DT_F32>(o, pack16<MOE_DT_F32>(v), most);
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

// B [rows][r] of the adapters that have tokens to [r][rows]: 64 rows by eight ranks
// to a wave at a time.
template <int DT>
__global__ __launch_bounds__(256) void k_aturn(TArgs a) {
  constexpr int B = kBytes<DT>;
  typedef typename std::conditional<B == 4, uint32_t, uint16_t>::type E;
  const int32_t* plan = a.plan;
  if (plan[0] != kPlanMagic || plan[1] != a.C || plan[2] != a.n) return;
  const int who = blockIdx.y, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (plan[a.at.first + who] == plan[a.at.first + who + 1]) return;
  const int n = 64 * blockIdx.x + lane;
  if (n >= a.rows) return;
  const uint8_t* b = a.b + who * a.b_stride + n * a.b_pitch;
  E* o = reinterpret_cast<E*>(a.out + who * a.out_stride) + n;
  for (int j = 8 * wave; j < a.r; j += 32) {
    const Eight<DT> v = load8_of<DT>(b, j, a.r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (j + i >= a.r) break;
      E* p = reinterpret_cast<E*>(reinterpret_cast<uint8_t*>(o) + (j + i) * a.pitch);
      if constexpr (B == 4) *p = v.v[i >> 2][i & 3];
      else *p = (uint16_t)(v.v[0][i >> 1] >> (16 * (i & 1)));
    }
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
// serves fewer too.  With ranges (512 / tiles, tiles > C / 64) the partial sums, the
// first part and all that the forward pass uses, are those of 512 * 64 tokens at most,
// and there are eight chunks a batch, or one to 2048 tokens, besides every adapter's last.
size_t partial_sums(int C, int64_t cols, int rank) {
  const int64_t most = (cols + 511) / 512, rows = C * most < 512 * 64 ? C * most : C > 512 * 64 ? C : 512 * 64;
  return align256((size_t)rows * rank * sizeof(float));
}
struct AdapterWs { size_t part, u, turned, suma, sumb, pieces, piece_bytes, total; int64_t turn_pitch, turn_stride; };
AdapterWs adapter_ws(const moe_adapter_bank* b, int C) {
  const int64_t s = dense_size(b->dtype);
  const int64_t few = C / 256 < 8 ? C / 256 : 8, chunks = (C / 2048 > few ? C / 2048 : few) + (C < b->adapters ? C : b->adapters);
  AdapterWs w;
  size_t o = 0;
  w.part = o; o += partial_sums(C, b->cols > b->rows ? b->cols : b->rows, b->rank);
  w.u = o; o = align256(o + (size_t)C * b->rank * sizeof(float));
  w.turn_pitch = (b->rows * s + 15) / 16 * 16;
  w.turn_stride = w.turn_pitch * b->rank;
  w.turned = o; o = align256(o + (size_t)b->adapters * w.turn_stride);
  w.suma = o; o = align256(o + (size_t)chunks * b->rank * b->cols * sizeof(float));
  w.sumb = o; o = align256(o + (size_t)chunks * b->rank * b->rows * sizeof(float));
  w.piece_bytes = align256((size_t)(C / 32 + chunks + 1) * ((b->rank + 15) / 16) * (s == 4 ? 2 : 3) * 1024);
  w.pieces = o; o += 2 * w.piece_bytes;
  w.total = o;
  return w;
}

template <int DT, int TT, bool DROP>
void launch_shrink_t(const AArgs& a, int tiles, hipStream_t st) {
  const dim3 grid((unsigned)tiles, (unsigned)a.splits, (unsigned)((a.r + 63) / 64));
  if (a.r <= 16) hipLaunchKernelGGL((k_ashrink<DT, 1, TT, DROP>), grid, dim3(kAWG), 0, st, a);
  else if (a.r <= 32) hipLaunchKernelGGL((k_ashrink<DT, 2, TT, DROP>), grid, dim3(kAWG), 0, st, a);
  else hipLaunchKernelGGL((k_ashrink<DT, 4, TT, DROP>), grid, dim3(kAWG), 0, st, a);
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

template <int DT, bool BWD, bool DROP>
void launch_expand(AArgs a, int tiles, hipStream_t st) {
  // a wave's columns once, or again where that makes more than four workgroups a CU
  const int per = 64 * kTiles<DT>, blocks = a.cols > 0 ? (a.cols + per - 1) / per : 1;
  int y = 1024 / tiles;
  y = y < 1 ? 1 : y > blocks ? blocks : y;
  a.column_parts = y;
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8 * y));
  const int kt = a.r <= 32 ? 1 : a.r <= 64 ? 2 : 4;
  const size_t lds = (size_t)plan_tile(a.C) * 32 * kt * (DT == MOE_DT_F32 ? 4 : DT == MOE_DT_F16 ? 4 : 6);
  if (kt == 1) hipLaunchKernelGGL((k_aexpand<DT, 1, BWD, DROP>), grid, dim3(kAWG), lds, st, a);
  else if (kt == 2) hipLaunchKernelGGL((k_aexpand<DT, 2, BWD, DROP>), grid, dim3(kAWG), lds, st, a);
  else hipLaunchKernelGGL((k_aexpand<DT, 4, BWD, DROP>), grid, dim3(kAWG), lds, st, a);
}

template <int DT, int NT, int RH, bool DROP>
moe_status launch_outer_t(const OArgs& a, int chunks, hipStream_t st) {
  constexpr int W = 16 * kTiles<DT>, sums = kOWaves / 2 * 16 * NT * (W + 4) * 4, lds = sums > 8192 ? sums : 8192;
  auto k = k_aouter<DT, NT, RH, DROP>;
  if (lds > 65536 && hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize,
                                         lds) != hipSuccess)
    return MOE_ERR_DEVICE;
  hipLaunchKernelGGL(k, dim3((unsigned)(a.da.blocks + a.db.blocks), (unsigned)chunks), dim3(64 * kOWaves), lds, st, a);
  return MOE_OK;
}
template <int DT, bool DROP>
moe_status launch_outer(const OArgs& a, int chunks, hipStream_t st) {
  if (a.r <= 16) return launch_outer_t<DT, 1, 1, DROP>(a, chunks, st);
  if (a.r <= 32) return launch_outer_t<DT, 2, 1, DROP>(a, chunks, st);
  if (a.r <= 64) return launch_outer_t<DT, 2, 2, DROP>(a, chunks, st);
  return launch_outer_t<DT, 2, 4, DROP>(a, chunks, st);
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

// The checks that both directions make, and the arguments that they share; `need`: the
// workspace's bytes.
struct Call {
  AArgs a;
  PlanLayout at;
  AdapterWs ws;
  uint8_t* w8;
  int64_t s;
};
moe_status adapter_call(const moe_adapter_bank* b, const void* plan, size_t plan_bytes, int32_t C, double p,
                        const uint64_t* rng, void* ws, size_t ws_bytes, size_t need, Call& c) {
  moe_status st = dropout_of(p, rng, c.a.drop);
  if (st != MOE_OK) return st;
  c.at = plan_layout(C, b->adapters);
  if (!plan || (uintptr_t)plan % 256 || plan_bytes < (size_t)c.at.total * sizeof(int32_t)) return MOE_ERR_WORKSPACE;
  c.ws = adapter_ws(b, C);
  if (!ws || (uintptr_t)ws % 256 || ws_bytes < need) return MOE_ERR_WORKSPACE;
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

size_t moe_adapter_fwd_workspace_size(const moe_adapter_bank* b, int32_t C) {
  if (adapter_status(b) != MOE_OK || C < 1 || C > MOE_MAX_BATCH_TOKENS) return 0;
  return partial_sums(C, b->cols, b->rank);
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
  const bool forward = ws_bytes & MOE_WS_FORWARD;
  ws_bytes &= ~MOE_WS_FORWARD;
  const Rows outs[] = {ry, rh, span(ws, (int64_t)ws_bytes)};
  const Rows tensors[] = {rx, ry, rb, rh};
  if (any_share(outs, adapter_reads(b, plan, plan_bytes, p > 0 ? rng : nullptr).r) || any_share({outs[2]}, tensors)) return MOE_ERR_INVALID_ARG;
  Call c = {};
  const size_t need = forward ? partial_sums(C, b->cols, b->rank) : adapter_ws(b, C).total;
  if ((st = adapter_call(b, plan, plan_bytes, C, p, rng, ws, ws_bytes, need, c)) != MOE_OK) return st;
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
    launch_expand<DT, false, false>(a, c.at.max_tiles, q);
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
  if (ws_bytes & MOE_WS_FORWARD) return MOE_ERR_WORKSPACE;
  const Rows outs[] = {rg, ga, gb, span(ws, (int64_t)ws_bytes)};
  const Rows ins[] = {rd, da ? rx : Rows{}, db ? rh : Rows{}};
  const Rows grads[] = {rg, ga, gb, dx ? rb : Rows{}};
  if (any_share(outs, ins) || any_share({outs[3]}, grads) ||
      any_share(outs, adapter_reads(b, plan, plan_bytes, p > 0 ? rng : nullptr).r))
    return MOE_ERR_INVALID_ARG;
  if (share(rg, ga) || share(rg, gb) || share(ga, gb)) return MOE_ERR_INVALID_ARG;
  if (dx && base && ((share(rb, rg) && !same(rb, rg)) || share(rb, ga) || share(rb, gb))) return MOE_ERR_INVALID_ARG;
  Call c = {};
  if ((st = adapter_call(b, plan, plan_bytes, C, p, rng, ws, ws_bytes, adapter_ws(b, C).total, c)) != MOE_OK) return st;
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
      hipLaunchKernelGGL((k_aturn<DT>), dim3((unsigned)((b->rows + 63) / 64), (unsigned)b->adapters), dim3(256), 0,
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
      if (drop) launch_expand<DT, true, true>(a, c.at.max_tiles, q);
      else launch_expand<DT, true, false>(a, c.at.max_tiles, q);
    }
    if (da || db) {
      OArgs o = {};
      o.plan = a.plan; o.at = c.at;
      o.C = C; o.n = b->adapters; o.r = b->rank;
      o.drop = a.drop;
      constexpr int W = 16 * kTiles<DT>;
      if (da) o.da = Outer{static_cast<const uint8_t*>(x), x_pitch * s, u, c.w8 + c.ws.pieces, reinterpret_cast<float*>(c.w8 + c.ws.suma), b->cols, (b->cols + W - 1) / W};
      if (db) o.db = Outer{static_cast<const uint8_t*>(dy), dy_pitch * s, hidden, c.w8 + c.ws.pieces + c.ws.piece_bytes, reinterpret_cast<float*>(c.w8 + c.ws.sumb), b->rows, (b->rows + W - 1) / W};
      const unsigned steps = (unsigned)(plan_chunk(C) / 32);
      hipLaunchKernelGGL((k_apieces<DT>), dim3(steps, (unsigned)c.at.max_chunks, da && db ? 2 : 1), dim3(256), 0, q, o);
      st = drop && da ? launch_outer<DT, true>(o, c.at.max_chunks, q) : launch_outer<DT, false>(o, c.at.max_chunks, q);
    }
  });
  if (st != MOE_OK) return st;
  if (da || db) {
    RArgs r2 = {};
    r2.plan = c.a.plan; r2.at = c.at;
    r2.C = C; r2.n = b->adapters; r2.r = b->rank;
    r2.accumulate = accumulate;
    r2.ca = da ? b->cols : 0; r2.cb = db ? b->rows : 0;
    r2.sa = reinterpret_cast<const float*>(c.w8 + c.ws.suma); r2.sb = reinterpret_cast<const float*>(c.w8 + c.ws.sumb);
    r2.da = da; r2.db = db;
    r2.scales = b->scales;
    r2.factor = c.a.drop.scale;
    r2.xa = ((r * r2.ca + 3) / 4 + 255) / 256;
    const int64_t xb = ((r + 3) / 4 * r2.cb + 255) / 256;
    hipLaunchKernelGGL(k_areduce, dim3((unsigned)(r2.xa + xb), (unsigned)b->adapters), dim3(256), 0, q, r2);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // extern "C"
