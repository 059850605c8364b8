// libroutedfp4, router load: per-expert counts of a selection, the balance
// loss over it with its gradient, and the gradient of the renormalised
// routing weights.
//
//   p_t    = a token's logits as shares over the experts (normalised sigmoid,
//            or softmax)
//   P[s]   = mean of p_t over the T_s tokens of sequence s
//   f[s]   = E counts[s] / (k T_s)
//   loss   = alpha / S * sum_s f[s] . P[s]
//   dl_e   = p_e (g_e - p . g) (* sigmoid(-l_e)),  g = dloss alpha / (S T_s) f[s]
//
// A row of up to 1024 logits lies in one wave's registers (16 a lane), so each
// pass over the logits reads it once.  A share costs one exponential and one
// reciprocal (hardware, 1 unit each), so that arithmetic stays below the memory
// time.  65536 tokens x 448, packed, with padding: the backward pass is bound by
// reading and writing C*E floats (38.5 us, 6.1 TB/s, logits partly from the last
// level of cache); the forward pass reads the same logits in 38 us, 3.1 TB/s: its
// waves wait for 73% of their time, each workgroup for its search, its offsets, its
// counts and the sum over its waves, around eight tokens a wave.
//
// A slot or part has at most 2^20 tokens of k <= 32 choices: i / k of its i-th
// choice is the high word of i * kmul, kmul = 2^32 / k + 1, whose error
// i / 2^32 stays under 1 / k.
//
// Kernels:
//   k_bal_part    a slot of up to TB tokens of one sequence: the slot's sums
//                 of shares, its counts and its number of tokens; a small
//                 batch is one slot, whose workgroup goes on to the loss
//   k_bal_final   per sequence and 64 experts: the slots added in order, the
//                 loss from the last workgroup to arrive
//   k_bal_bwd     a few consecutive tokens per wave
//   k_count       counts without logits: a workgroup per sequence, or several
//   k_count_fill / k_count_slots   counts of large packed batches, in slots
//   k_route_bwd   two, four or eight tokens per wave
#include "common.h"

namespace rf4 {
namespace {

constexpr int kPartWG = 512;          // eight waves share a slot's tokens
constexpr int kPartWaves = kPartWG / 64;
constexpr int kBalWG = 256;           // backward kernels: four waves
constexpr int kBalWaves = kBalWG / 64;
constexpr int kOneSlot = 32;          // tokens up to which a single sequence is one slot

// Sequence bounds from the device offsets, clipped to the batch so that no
// content of seq_off makes a kernel leave its tensors.
__device__ __forceinline__ int seq_at(const int32_t* off, int i, int S, int C) {
  const int v = off ? off[i] : (i < S ? 0 : C);
  return v < 0 ? 0 : v > C ? C : v;
}

// The largest i in [0, n) whose key is at most x, keys rising and key(0) <= x:
// 64 candidates a step, one per lane, since a binary search waits for memory
// once per halving (65535 sequences take three steps).  Whatever the keys are,
// the result lies in [0, n).
template <class K>
__device__ __forceinline__ int wave_search(int n, int x, K key) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int64_t i = (int64_t)lane * step;
    const int c = __popcll(__ballot(i < n && key(lo + (int)i) <= x));
    const int k = c > 1 ? (c - 1) * step : 0;
    lo += k;
    n = n - k < step ? n - k : step;
  }
  return lo;
}

// The sequence that token t lies in (the last one that starts at or before
// t, so empty ones are passed over), or -1.
__device__ __forceinline__ int seq_of(const int32_t* off, int t, int S, int C) {
  if (!off) return 0;
  const int s = wave_search(S + 1, t, [&](int i) { return seq_at(off, i, S, C); });
  return s < S && seq_at(off, s, S, C) <= t ? s : -1;
}

// Tokens per slot, a power of two, so that a sequence's first slot is a shift:
// 8 (one a wave) while that makes a slot a CU, then up to 32 (8192 tokens x 896,
// both passes, with 8, 16, 32, 64: 38.8, 37.1, 32.6, 36.4 us), then as many as
// keep the slots at 1024, whose partial sums (a row of E per slot) stay a small
// share of the logits read (65536 x 448 with 16, 32, 64, 128: 103.6, 96.2, 95.1,
// 93.4 us).  One slot for up to 32 tokens, whose workgroup writes the loss (16
// tokens: 11.1 us in one slot, 13.7 in two; 32: 13.9 and 13.8; 64: 19.2 and
// 14.0).
__host__ __device__ inline int slot_limit(int s) { return s < 5 ? 256 : 1024; }
__host__ __device__ inline int slot_shift(int C, int S) {
  if (S == 1 && C <= kOneSlot) return 5;
  int s = 3;
  while (s < 10 && (C >> s) > slot_limit(s)) ++s;
  return s;
}
// Slots of sequence s: from (off[s] >> shift) + s, one per TB tokens.  The
// next sequence's first slot is at least that many further on, so slots need
// no prefix sum over the sequences.
__host__ __device__ inline int num_slots(int C, int S) { return (C >> slot_shift(C, S)) + S; }
// The most slots of a batch of up to C tokens, which a workspace is sized by: they
// fall where the slots grow (32799 tokens are 1024 full slots, 32800 are 512).
inline int most_slots(int C, int S) {
  int n = num_slots(C, S);
  for (int s = 3; s < 10; ++s) {
    const int last = ((slot_limit(s) + 1) << s) - 1;       // the most tokens in slots of 2^s
    if (last < C && num_slots(last, S) > n) n = num_slots(last, S);
  }
  return n;
}

// Tickets of k_bal_final, each in a cache line of its own: one for up to twice
// kTickets workgroups; for more, kTickets that they share out among them and one
// for the last of each, since they take turns at one word (both passes, 896
// experts: 47 sequences, 658 workgroups, 21.7 us with one ticket, 17.9 with 65; 8
// sequences, 112 workgroups, 16.6 and 17.1).
constexpr int kTickets = 64, kTicketStride = 64;

struct BalWs {
  size_t ctrl, psum, pcnt, ptok, dots, total;
};
inline int expert_blocks(int E) { return (E + 63) / 64; }
inline BalWs bal_ws(int C, int E, int S) {
  BalWs W;
  size_t o = 0;
  const size_t n = (size_t)most_slots(C, S);
  W.ctrl = o; o = align256(o + (1 + kTickets) * kTicketStride * sizeof(uint32_t));
  W.psum = o; o = align256(o + n * E * sizeof(float));
  W.pcnt = o; o = align256(o + n * E * sizeof(uint16_t));
  W.ptok = o; o = align256(o + n * sizeof(int32_t));
  W.dots = o; o = align256(o + (size_t)S * expert_blocks(E) * sizeof(float));
  W.total = o;
  return W;
}

struct BalArgs {
  const float* logits;
  const int32_t* idx;
  const int32_t* off;
  const uint8_t* mask;
  int C, k, E, S;
  int32_t* counts;
  int32_t* tokens;
  float* probs;
  float* loss;
  float alpha;
  // workspace
  uint32_t* ticket;
  float* psum;
  uint16_t* pcnt;
  int32_t* ptok;
  float* dots;
  // backward
  const float* grad;
  float* dlogits;
  int accumulate;
  int per;             // tokens per wave
  uint32_t kmul;       // see above
  int shift;           // slot_shift
  bool one;            // one slot holds the batch
  bool vec_counts;     // and rows of counts
  bool vec;            // rows of logits (and dlogits) are 16-byte aligned
};

// Reductions over the wave with DPP row shifts and row broadcasts (six adds;
// through LDS permutes they took half of a row's time); every lane gets lane
// 63's result.  Lanes a shift leaves without a source take the identity.
template <int CTRL, int RMASK>
__device__ __forceinline__ float dpp(float id, float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(id), __float_as_int(x), CTRL, RMASK, 0xF, false));
}
__device__ __forceinline__ float lane63(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0x111, 0xF>(0.0f, v);
  v += dpp<0x112, 0xF>(0.0f, v);
  v += dpp<0x114, 0xF>(0.0f, v);
  v += dpp<0x118, 0xF>(0.0f, v);
  v += dpp<0x142, 0xA>(0.0f, v);
  v += dpp<0x143, 0xC>(0.0f, v);
  return lane63(v);
}
__device__ __forceinline__ float row_max(float v) {
  constexpr float lo = -INFINITY;
  v = fmaxf(v, dpp<0x111, 0xF>(lo, v));
  v = fmaxf(v, dpp<0x112, 0xF>(lo, v));
  v = fmaxf(v, dpp<0x114, 0xF>(lo, v));
  v = fmaxf(v, dpp<0x118, 0xF>(lo, v));
  v = fmaxf(v, dpp<0x142, 0xA>(lo, v));
  v = fmaxf(v, dpp<0x143, 0xC>(lo, v));
  return lane63(v);
}

// e^x by the hardware's 2^y: y = x log2(e) is rounded, and what the rounding
// (and log2(e) as an fp32 number) leaves out enters as a factor 1 + r ln 2.
// x <= 0 or NaN here; -inf gives 0.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 1.44269502162933349609f, kLog2eLo = 1.92596299112661746887e-8f;
  constexpr float kLn2 = 0.69314718055994530942f;
  x = x < -200.0f ? -200.0f : x;           // 0 already; keeps the remainder finite
  const float y = x * kLog2e;
  const float r = fmaf(x, kLog2eLo, fmaf(x, kLog2e, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return fmaf(e, r * kLn2, e);
}

// A row of E logits over a wave: lane l holds experts 4 (l + 64 j) + c in
// v[4 j + c]; past E: fill.  vec: every row is 16-byte aligned (E % 4 == 0 and
// an aligned base); a slice of logits may start anywhere.
template <int NJ>
__device__ __forceinline__ void load_row(const float* row, int E, bool vec, float fill, float (&v)[4 * NJ]) {
  const int lane = threadIdx.x & 63;
  if (vec) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = 4 * (lane + 64 * j);
      float4 q = make_float4(fill, fill, fill, fill);
      if (e < E) q = *reinterpret_cast<const float4*>(row + e);
      v[4 * j] = q.x; v[4 * j + 1] = q.y; v[4 * j + 2] = q.z; v[4 * j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = 4 * (lane + 64 * j) + c;
        v[4 * j + c] = e < E ? row[e] : fill;
      }
  }
}

// sigmoid(l) and sigmoid(-l)
__device__ __forceinline__ void sigmoids(float l, float& s, float& neg) {
  const float u = exp_neg(-fabsf(l));
  const float r = __builtin_amdgcn_rcpf(1.0f + u);
  const float ur = u * r;
  s = l >= 0.0f ? r : ur;
  neg = l >= 0.0f ? ur : r;
}

// A row's scores in place of its logits, and their sum; for the sigmoid score
// also sigmoid(-l).  Where the whole row lies far below zero the sigmoids
// underflow; the scores are then sigmoid(l) e^-m, m the largest logit, which is
// e^(l - m) / (1 + e^l).  A row of -inf has scores 0.
template <int NJ, bool SIG>
__device__ __forceinline__ float scores(float (&v)[4 * NJ], float (&neg)[4 * NJ]) {
  float z = 0.0f;
  if (SIG) {
    float l[4 * NJ];
#pragma unroll
    for (int i = 0; i < 4 * NJ; ++i) {
      l[i] = v[i];
      sigmoids(l[i], v[i], neg[i]);
      z += v[i];
    }
    z = row_sum(z);
    if (!(z < 1e-18f)) return z;            // NaN too
#pragma unroll
    for (int i = 0; i < 4 * NJ; ++i) v[i] = l[i];
  }
  float m = v[0];
#pragma unroll
  for (int i = 1; i < 4 * NJ; ++i) m = fmaxf(m, v[i]);
  m = row_max(m);
  m = m == -INFINITY ? 0.0f : m;            // a row of -inf: every score is e^-inf
  z = 0.0f;
#pragma unroll
  for (int i = 0; i < 4 * NJ; ++i) {
    v[i] = exp_neg(v[i] - m);
    if (SIG) v[i] *= neg[i];                // 1 / (1 + e^l)
    z += v[i];
  }
  return row_sum(z);
}

// The sum over a workgroup, its waves' sums in order.
__device__ __forceinline__ float block_sum(float d, float* s_p, int waves) {
  const int tid = threadIdx.x;
  d = row_sum(d);
  if ((tid & 63) == 0) s_p[tid >> 6] = d;
  __syncthreads();
  float v = 0.0f;
  for (int w = 0; w < waves; ++w) v += s_p[w];
  return v;
}

template <int NJ, bool SIG>
__global__ __launch_bounds__(kPartWG) void k_bal_part(BalArgs a) {
  __shared__ float s_sum[kPartWaves][256 * NJ];
  __shared__ uint32_t s_cnt[256 * NJ];
  __shared__ float s_p[kPartWaves];
  __shared__ int s_tok;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  constexpr int threads = kPartWG, waves = kPartWaves;
  const int E = a.E, slot = blockIdx.x, sh = a.shift;
  // the sequence whose slots this one is among: largest s with
  // (off[s] >> sh) + s <= slot
  const int lo = wave_search(a.S, slot, [&](int i) { return (seq_at(a.off, i, a.S, a.C) >> sh) + i; });
  const int b = seq_at(a.off, lo, a.S, a.C), end = seq_at(a.off, lo + 1, a.S, a.C);
  const int first = slot - ((b >> sh) + lo);
  const int64_t t0 = b + ((int64_t)first << sh);
  if (first < 0 || t0 >= end) return;
  const int n = end - t0 < (1 << sh) ? (int)(end - t0) : (1 << sh);

  for (int e = tid; e < 256 * NJ; e += threads) s_cnt[e] = 0u;
  if (tid == 0) s_tok = 0;
  __syncthreads();
  // sums of shares: each wave its tokens in order, then the waves in order
  float acc[4 * NJ];
#pragma unroll
  for (int i = 0; i < 4 * NJ; ++i) acc[i] = 0.0f;
  int live = 0;
  // 64 of the wave's tokens at a time: which are live, in one load of the
  // mask; two tokens' rows are loaded while the two before are worked on
  for (int base = wave; base < n || base == wave; base += 64 * waves) {
    const int mine = base + waves * lane;
    uint64_t left = __ballot(mine < n && (!a.mask || a.mask[t0 + mine] != 0));
    live += __popcll(left);
    const float* row0 = a.logits + (t0 + base) * E;
    float next[2][4 * NJ];
    auto take = [&](float (&v)[4 * NJ]) {      // the row of the lowest token left, which leaves
      if (!left) return;
      load_row<NJ>(row0 + (int64_t)waves * (__ffsll((long long)left) - 1) * E, E, a.vec, -INFINITY, v);
      left &= left - 1;
    };
    int todo = __popcll(left);
    take(next[0]);
    take(next[1]);
    if (base == wave) {
      // counts, while the first rows are on their way (integers: any order
      // gives the same)
      for (int i = tid; i < n * a.k; i += threads) {
        const int e = a.idx[t0 * a.k + i];
        const bool on = !a.mask || a.mask[t0 + (a.k == 1 ? i : (int)__umulhi((uint32_t)i, a.kmul))] != 0;
        if (on && e >= 0 && e < E) atomicAdd(&s_cnt[e], 1u);
      }
    }
    for (; todo > 0; todo -= 2) {
      float v[2][4 * NJ], neg[4 * NJ];
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) { v[0][i] = next[0][i]; v[1][i] = next[1][i]; }
      take(next[0]);
      take(next[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && todo == 1) break;
        const float z = scores<NJ, SIG>(v[h], neg);
        const float iz = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
        for (int i = 0; i < 4 * NJ; ++i) acc[i] = fmaf(v[h][i], iz, acc[i]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    *reinterpret_cast<float4*>(&s_sum[wave][4 * (lane + 64 * j)]) =
        make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
  if (lane == 0 && live) atomicAdd(&s_tok, live);
  __syncthreads();
  const int tok = s_tok;
  const float it = tok > 0 ? 1.0f / (float)tok : 0.0f;
  float d = 0.0f;
  for (int e = tid; e < E; e += threads) {
    float p = s_sum[0][e];
    for (int w = 1; w < waves; ++w) p += s_sum[w][e];
    const int c = (int)s_cnt[e];
    if (a.one) {
      const float P = p * it;
      a.probs[e] = P;
      a.counts[e] = c;
      d += (float)c * it * ((float)E / (float)a.k) * P;
    } else {
      a.psum[(size_t)slot * E + e] = p;
      a.pcnt[(size_t)slot * E + e] = (uint16_t)c;         // at most 1024 tokens * 32 slots
    }
  }
  if (!a.one) {
    if (tid == 0) a.ptok[slot] = tok;
    return;
  }
  d = block_sum(d, s_p, waves);
  if (tid == 0) {
    a.tokens[0] = tok;
    a.loss[0] = a.alpha * d;
  }
}

// Experts 64 x .. 64 x + 63 of sequence y: 16 threads per expert add every
// 16th slot, eight of them in flight, then their sums in order.
constexpr int kFinWG = 1024, kFinRows = kFinWG / 64;
__global__ __launch_bounds__(kFinWG) void k_bal_final(BalArgs a) {
  __shared__ float s_p[kFinWG];
  __shared__ int s_c[kFinWG];
  __shared__ float s_t[kFinRows];
  __shared__ int s_flag;
  const int tid = threadIdx.x, le = tid & 63, row = tid >> 6;
  const int s = blockIdx.y, e = blockIdx.x * 64 + le, E = a.E;
  const int sh = a.shift, total = num_slots(a.C, a.S);
  const int b = seq_at(a.off, s, a.S, a.C), end = seq_at(a.off, s + 1, a.S, a.C);
  const int len = end > b ? end - b : 0;
  const int j0 = (b >> sh) + s;
  int n = (len + (1 << sh) - 1) >> sh;
  if (n > total - j0) n = total - j0;
  const int ec = e < E ? e : E - 1;
  const float* ps = a.psum + (size_t)j0 * E + ec;
  const uint16_t* pc = a.pcnt + (size_t)j0 * E + ec;
  float p = 0.0f, live = 0.0f;
  int c = 0;
  for (int j = tid; j < n; j += kFinWG) live += (float)a.ptok[j0 + j];
  int j = row;
  for (; j + 7 * kFinRows < n; j += 8 * kFinRows) {
    float q[8];
    int k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = ps[(size_t)(j + i * kFinRows) * E];
      k[i] = pc[(size_t)(j + i * kFinRows) * E];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) { p += q[i]; c += k[i]; }
  }
  for (; j < n; j += kFinRows) {
    p += ps[(size_t)j * E];
    c += pc[(size_t)j * E];
  }
  s_p[tid] = p; s_c[tid] = c;
  // at most 2^20 tokens: exact in fp32
  const int t = (int)block_sum(live, s_t, kFinRows);
  if (row == 0) {
#pragma unroll
    for (int r = 1; r < kFinRows; ++r) {
      p += s_p[64 * r + le];
      c += s_c[64 * r + le];
    }
    const float it = t > 0 ? 1.0f / (float)t : 0.0f;
    const float P = p * it;
    const float f = (float)c * it * ((float)E / (float)a.k);
    if (e < E) {
      a.probs[(size_t)s * E + e] = P;
      a.counts[(size_t)s * E + e] = c;
    }
    const float d = row_sum(e < E ? f * P : 0.0f);
    if (le == 0) {
      if (blockIdx.x == 0) a.tokens[s] = t;
      store_coherent(a.dots + (size_t)s * gridDim.x + blockIdx.x, d);
    }
  }
  const uint32_t nb = gridDim.x * gridDim.y;
  uint32_t arrive = nb;
  if (nb > 2 * kTickets) {
    const uint32_t t = (blockIdx.y * gridDim.x + blockIdx.x) % kTickets;
    uint32_t* ticket = a.ticket + (1 + t) * kTicketStride;
    if (!last_to_arrive(ticket, (nb - t + kTickets - 1) / kTickets, &s_flag)) return;
    if (tid == 0) reset_ticket(ticket);
    arrive = kTickets;
  }
  if (!last_to_arrive(a.ticket, arrive, &s_flag)) return;
  if (tid == 0) reset_ticket(a.ticket);
  const __amdgpu_buffer_rsrc_t v = coherent_view(a.dots, nb * 4u);
  float d = 0.0f;
  for (uint32_t i = tid; i < nb; i += 8 * kFinWG) {       // past the last: zeros
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = coherent_ld(v, 4u * (i + j * kFinWG));
#pragma unroll
    for (int j = 0; j < 8; ++j) d += q[j];
  }
  d = block_sum(d, s_p, kFinRows);
  if (tid == 0) a.loss[0] = a.alpha / (float)a.S * d;
}

// Each wave takes a.per consecutive tokens; g (the sequence's counts, scaled)
// stays in registers from one token of a sequence to the next.
template <int NJ, bool SIG>
__global__ __launch_bounds__(kBalWG) void k_bal_bwd(BalArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int E = a.E;
  const int64_t base = ((int64_t)blockIdx.x * kBalWaves + wave) * a.per;
  int end = -1;                              // of the sequence whose g is loaded
  float g[4 * NJ], next[4 * NJ];
#pragma unroll
  for (int i = 0; i < 4 * NJ; ++i) g[i] = 0.0f;
  // which of the tokens are live, in one load of the mask; a live token's row
  // is loaded while the one before it is worked on
  const uint64_t live = __ballot(lane < a.per && base + lane < a.C && (!a.mask || a.mask[base + lane] != 0));
  if (live & 1) load_row<NJ>(a.logits + base * E, E, a.vec, -INFINITY, next);
  for (int k = 0; k < a.per && base + k < a.C; ++k) {
    const int64_t t = base + k;
    float v[4 * NJ], neg[4 * NJ];
#pragma unroll
    for (int i = 0; i < 4 * NJ; ++i) v[i] = next[i];
    if (live >> k >> 1 & 1) load_row<NJ>(a.logits + (t + 1) * E, E, a.vec, -INFINITY, next);
    if (t >= end) {
      const int s = seq_of(a.off, (int)t, a.S, a.C);
      const int e1 = s < 0 ? -1 : seq_at(a.off, s + 1, a.S, a.C);
      if (t >= e1) continue;                 // outside every sequence
      end = e1;
      const int n = a.tokens[s];
      const float it = n > 0 ? 1.0f / (float)n : 0.0f;
      const float w = a.grad[0] * (a.alpha / (float)a.S) * it * it * ((float)E / (float)a.k);
      load_row<NJ>(reinterpret_cast<const float*>(a.counts) + (size_t)s * E, E, a.vec_counts, 0.0f, g);
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) g[i] = w * (float)__float_as_int(g[i]);      // 0.0f is the integer 0
    }
    if (!(live >> k & 1)) {
      if (a.accumulate) continue;
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) v[i] = 0.0f;
    } else {
      const float z = scores<NJ, SIG>(v, neg);
      const float iz = z == 0.0f ? 0.0f : 1.0f / z;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) {
        v[i] *= iz;
        dot = fmaf(v[i], g[i], dot);
      }
      dot = row_sum(dot);
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) {
        v[i] *= g[i] - dot;
        if (SIG) v[i] *= neg[i];
      }
    }
    float* out = a.dlogits + t * E;
    if (a.vec) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = 4 * (lane + 64 * j);
        if (e >= E) continue;
        float4 d = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        float4* o = reinterpret_cast<float4*>(out + e);
        if (a.accumulate) {
          const float4 old = *o;
          d.x += old.x; d.y += old.y; d.z += old.z; d.w += old.w;
        }
        *o = d;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) {
        const int e = 4 * (lane + 64 * (i >> 2)) + (i & 3);
        if (e < E) out[e] = a.accumulate ? out[e] + v[i] : v[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Counts without logits
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_count_fill(int32_t* counts, int32_t* tokens, int64_t n, int S) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) counts[i] = 0;
  if (tokens && i < S) tokens[i] = 0;
}

// A workgroup's tokens t0 .. t1 - 1 (k times their number at most 2^25): their
// choices into s_cnt, the live ones into s_tok (where tok).  Four choices a thread
// are loaded together without a mask; with one, as compiled, each waits for its
// mask byte.
constexpr int kCntWG = 1024;
__device__ __forceinline__ void count_tokens(const int32_t* idx, const uint8_t* mask, int t0, int t1, int k, uint32_t kmul,
                                             int E, bool tok, int32_t* s_cnt, int32_t* s_tok) {
  const int tid = threadIdx.x, threads = blockDim.x;
  for (int e = tid; e < E; e += threads) s_cnt[e] = 0;
  if (tid == 0) *s_tok = 0;
  const int n = (t1 - t0) * k;
  const int32_t* at = idx + (int64_t)t0 * k;
  __syncthreads();
  for (int i0 = tid; i0 < n; i0 += 4 * threads) {
    int e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * threads;
      e[j] = i < n ? at[i] : -1;
      if (mask && i < n && !mask[t0 + (int)(k == 1 ? (uint32_t)i : __umulhi((uint32_t)i, kmul))]) e[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e[j] >= 0 && e[j] < E) atomicAdd(&s_cnt[e[j]], 1);
  }
  if (tok) {
    int live = 0;
    for (int t = t0 + tid; t < t1; t += threads) live += mask ? mask[t] != 0 : 1;
    if (live) atomicAdd(s_tok, live);
  }
  __syncthreads();
}
// The workgroup's counts added to a row by atomics (integers: any order gives
// the same).
__device__ __forceinline__ void add_counts(const int32_t* s_cnt, int s_tok, int E, int32_t* row, int32_t* tok) {
  const int tid = threadIdx.x, threads = blockDim.x;
  for (int e = tid; e < E; e += threads)
    if (s_cnt[e]) atomicAdd(&row[e], s_cnt[e]);
  if (tok && tid == 0 && s_tok) atomicAdd(tok, s_tok);
}

// Workgroup (s, j): the j-th of gridDim.x parts of sequence s.  One part:
// the row is written (or added to) as a whole.
__global__ __launch_bounds__(kCntWG) void k_count(const int32_t* idx, const int32_t* off, const uint8_t* mask,
                                                  int C, int k, uint32_t kmul, int E, int S, int32_t* counts,
                                                  int32_t* tokens, int accumulate) {
  __shared__ int32_t s_cnt[MOE_MAX_EXPERTS];
  __shared__ int32_t s_tok;
  const int tid = threadIdx.x, threads = blockDim.x, s = blockIdx.y, parts = gridDim.x;
  const int b = seq_at(off, s, S, C), end = seq_at(off, s + 1, S, C);
  const int len = end > b ? end - b : 0;
  const int per = (len + parts - 1) / parts;
  const int t0 = b + ((int64_t)per * blockIdx.x < len ? per * (int)blockIdx.x : len);
  const int t1 = t0 + per < b + len ? t0 + per : b + len;
  count_tokens(idx, mask, t0, t1, k, kmul, E, tokens != nullptr, s_cnt, &s_tok);
  int32_t* row = counts + (size_t)s * E;
  if (parts > 1) {
    add_counts(s_cnt, s_tok, E, row, tokens ? tokens + s : nullptr);
    return;
  }
  for (int e = tid; e < E; e += threads) row[e] = accumulate ? row[e] + s_cnt[e] : s_cnt[e];
  if (tokens && tid == 0) tokens[s] = accumulate ? tokens[s] + s_tok : s_tok;
}

// Slots of up to 2^sh tokens of one sequence, numbered as k_bal_part numbers
// its own: however uneven the sequences are, no workgroup has more than a slot.
// A slot that holds all of its sequence writes the row (zeroed before, unless the
// call accumulates) without atomics.  65536 tokens x 16 of 896 experts, 61
// sequences, with a mask: 7.2 us (and 1.9 for the zero fill), a chain of latencies:
// search, offsets, choices behind their mask bytes, atomics.
__global__ __launch_bounds__(kCntWG) void k_count_slots(const int32_t* idx, const int32_t* off, const uint8_t* mask,
                                                        int C, int k, uint32_t kmul, int E, int S, int sh,
                                                        int32_t* counts, int32_t* tokens, int accumulate) {
  __shared__ int32_t s_cnt[MOE_MAX_EXPERTS];
  __shared__ int32_t s_tok;
  const int slot = blockIdx.x;
  const int s = wave_search(S, slot, [&](int i) { return (seq_at(off, i, S, C) >> sh) + i; });
  const int b = seq_at(off, s, S, C), end = seq_at(off, s + 1, S, C);
  const int first = slot - ((b >> sh) + s);
  const int64_t t0 = b + ((int64_t)first << sh);
  if (first < 0 || t0 >= end) return;
  const int t1 = end - t0 < (1 << sh) ? end : (int)t0 + (1 << sh);
  count_tokens(idx, mask, (int)t0, t1, k, kmul, E, tokens != nullptr, s_cnt, &s_tok);
  int32_t* row = counts + (size_t)s * E;
  if (t0 > b || t1 < end) {
    add_counts(s_cnt, s_tok, E, row, tokens ? tokens + s : nullptr);
    return;
  }
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    if (s_cnt[e]) row[e] = accumulate ? row[e] + s_cnt[e] : s_cnt[e];
  if (tokens && threadIdx.x == 0) tokens[s] = accumulate ? tokens[s] + s_tok : s_tok;
}

// ---------------------------------------------------------------------------
// Gradient of the routing weights
// ---------------------------------------------------------------------------
// Sum and maximum over the KP lanes of a group, in every lane of it: DPP
// permutes inside 4, 8 and 16 lanes, one LDS permute across 16.
template <int KP, class F>
__device__ __forceinline__ float group_reduce(float v, F f) {
  v = f(v, dpp<0xB1, 0xF>(0.0f, v));         // lanes 1 0 3 2
  v = f(v, dpp<0x4E, 0xF>(0.0f, v));         // lanes 2 3 0 1
  v = f(v, dpp<0x141, 0xF>(0.0f, v));        // mirrored in 8
  if (KP >= 16) v = f(v, dpp<0x140, 0xF>(0.0f, v));   // mirrored in 16
  if (KP >= 32) v = f(v, __shfl_xor(v, 16, 64));
  return v;
}

// KP lanes (k rounded up to 8, 16 or 32) per token, so that a wave has 64 / KP
// tokens' loads and sums in flight together; then their rows, one after the
// other through a row of zeros in LDS that each token's values are put into
// and taken out of again.  Bound by writing the rows (40001 x 448: 17 to 23 us,
// 3.1 to 4.2 TB/s).
template <int KP>
__global__ __launch_bounds__(kBalWG) void k_route_bwd(const float* logits, const int32_t* idx,
                                                      const float* dw, int C, int k, int E,
                                                      const uint8_t* mask, float* dlogits, int accumulate,
                                                      bool vec) {
  constexpr int TPW = 64 / KP;
  __shared__ __align__(16) float s_row[kBalWaves][MOE_MAX_EXPERTS];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, slot = lane % KP;
  const int64_t t0 = ((int64_t)blockIdx.x * kBalWaves + wave) * TPW, t = t0 + lane / KP;
  if (t0 >= C) return;                      // whole waves: no barrier below
  float* srow = s_row[wave];
  if (!accumulate) {
    for (int i = 4 * lane; i < E; i += 256) *reinterpret_cast<float4*>(srow + i) = make_float4(0, 0, 0, 0);
  }
  int e = -1;
  float l = -INFINITY, d = 0.0f;
  if (t < C && slot < k && (!mask || mask[t] != 0)) {
    e = idx[t * k + slot];
    if (e < 0 || e >= E) e = -1;
    if (e >= 0) {
      l = logits[t * E + e];
      d = dw[t * k + slot];
    }
  }
  auto add = [](float x, float y) { return x + y; };
  auto larger = [](float x, float y) { return fmaxf(x, y); };
  float sg, neg;
  sigmoids(l, sg, neg);
  const float m = group_reduce<KP>(l, larger);
  if (m < -40.0f) sg = l == -INFINITY ? 0.0f : exp_neg(l - m) * neg;       // the sigmoids underflow
  if (e < 0) sg = 0.0f;
  const float z = group_reduce<KP>(sg, add);
  const float w = z == 0.0f ? 0.0f : sg / z;
  const float dot = group_reduce<KP>(e >= 0 ? w * d : 0.0f, add);
  const float dl = e >= 0 ? w * neg * (d - dot) : 0.0f;
  // slots that name one expert: the first adds them up, in slot order
  float mine = 0.0f;
  bool first = e >= 0;
  for (int s = 0; s < k; ++s) {
    const int es = __shfl(e, s, KP);
    const float ds = __shfl(dl, s, KP);
    if (es == e) {
      if (s < slot) first = false;
      mine += ds;
    }
  }
  if (accumulate) {
    if (first) dlogits[t * E + e] += mine;
    return;
  }
  wave_lds_fence();
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    if (t0 + i >= C) return;
    const bool here = first && lane / KP == i;
    if (here) srow[e] = mine;
    wave_lds_fence();
    float* out = dlogits + (t0 + i) * E;
    if (vec) {
      for (int c = 4 * lane; c < E; c += 256)
        *reinterpret_cast<float4*>(out + c) = *reinterpret_cast<const float4*>(srow + c);
    } else {
      for (int c = lane; c < E; c += 64) out[c] = srow[c];
    }
    wave_lds_fence();
    if (here) srow[e] = 0.0f;
  }
}

uint32_t division(int k) { return k == 1 ? 0u : (uint32_t)((1ull << 32) / (unsigned)k) + 1u; }
bool batch_ok(int C, int k, int E) {
  return C >= 1 && C <= MOE_MAX_BATCH_TOKENS && E >= 1 && E <= MOE_MAX_EXPERTS && k >= 1 &&
         k <= MOE_MAX_TOPK && k <= E;
}
bool seq_ok(const int32_t* off, int S) { return S >= 1 && S <= MOE_MAX_SEQUENCES && (off || S == 1); }
bool aligned4(const void* p) { return (uintptr_t)p % 4 == 0; }

moe_status launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE; }

#define RF4_BY_ROW(KERNEL, E, SIG, GRID, WG, ST, ...)                                              \
  do {                                                                                             \
    const int nj_ = ((E) + 255) / 256;                                                             \
    if (SIG) {                                                                                     \
      if (nj_ == 1) hipLaunchKernelGGL((KERNEL<1, true>), GRID, dim3(WG), 0, ST, __VA_ARGS__);     \
      else if (nj_ == 2) hipLaunchKernelGGL((KERNEL<2, true>), GRID, dim3(WG), 0, ST, __VA_ARGS__);\
      else if (nj_ == 3) hipLaunchKernelGGL((KERNEL<3, true>), GRID, dim3(WG), 0, ST, __VA_ARGS__);\
      else hipLaunchKernelGGL((KERNEL<4, true>), GRID, dim3(WG), 0, ST, __VA_ARGS__);              \
    } else {                                                                                       \
      if (nj_ == 1) hipLaunchKernelGGL((KERNEL<1, false>), GRID, dim3(WG), 0, ST, __VA_ARGS__);    \
      else if (nj_ == 2) hipLaunchKernelGGL((KERNEL<2, false>), GRID, dim3(WG), 0, ST, __VA_ARGS__);\
      else if (nj_ == 3) hipLaunchKernelGGL((KERNEL<3, false>), GRID, dim3(WG), 0, ST, __VA_ARGS__);\
      else hipLaunchKernelGGL((KERNEL<4, false>), GRID, dim3(WG), 0, ST, __VA_ARGS__);             \
    }                                                                                              \
  } while (0)

}  // namespace
}  // namespace rf4

using namespace rf4;

extern "C" {

moe_status moe_expert_counts(const int32_t* topk_idx, int32_t C, int32_t k, int32_t E,
                             const int32_t* seq_off, int32_t S, const uint8_t* token_mask,
                             int32_t* counts, int32_t* tokens, int32_t accumulate, void* stream) {
  if (!topk_idx || !counts) return MOE_ERR_INVALID_ARG;
  if (!aligned4(topk_idx) || !aligned4(counts) || !aligned4(tokens) || !aligned4(seq_off))
    return MOE_ERR_INVALID_ARG;
  if (!batch_ok(C, k, E) || S < 1 || S > MOE_MAX_SEQUENCES) return MOE_ERR_UNSUPPORTED;
  if (!seq_ok(seq_off, S)) return MOE_ERR_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t choices = (int64_t)C * k;
  // How long a sequence is only the device knows, so the rule is on the choices of
  // the whole batch.  Up to 65536 of them, one workgroup per sequence, which writes
  // its row without zero fill or atomics: at worst one sequence has them all (us,
  // even sequences and all in one, here and in slots: 16 of 4096 choices 5.5, 12.2
  // and 7.4, 7.6; 1000 of 64 5.0, 22.5 and 8.2, 10.1).  More are shared out in slots
  // (128 of 8192 here 6.0, 145.6, in slots 9.1, 12.1), about 256 of at least 2048
  // choices (61 sequences, 2^20 choices: 9.0, in 512 slots 10.4); one sequence in
  // parts, which need no search (2^20 choices: 10.5 in 64, 11.8 in 256).
  const bool slots = S > 1 && choices > 65536;
  int64_t parts = 1;
  if (S == 1 && choices > 8192) {
    parts = (choices + 2047) / 2048;
    if (parts > 64) parts = 64;
  }
  if ((slots || parts > 1) && !accumulate) {
    const int64_t n = (int64_t)S * E;
    hipLaunchKernelGGL(k_count_fill, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, counts, tokens, n, S);
  }
  if (slots) {
    int sh = 0;
    while (((int64_t)k << sh) < 2048 || (C >> sh) > 256) ++sh;
    // workgroups as large as lets all of them run at once (1000 sequences of 524
    // choices: 9.1 us with 256 threads, 18.0 with 1024; 16 of 8192: 8.2 and 7.7)
    const int wgs = (C >> sh) + S, wg = wgs <= 512 ? kCntWG : wgs <= 1024 ? 512 : 256;
    hipLaunchKernelGGL(k_count_slots, dim3((unsigned)wgs), dim3(wg), 0, st, topk_idx, seq_off, token_mask, C, k,
                       division(k), E, S, sh, counts, tokens, accumulate);
  } else {
    // small workgroups for short sequences (1000 of 64 choices: 5.7 us, 8.0 with
    // large ones; one of 8192: 7.5 and 5.7)
    hipLaunchKernelGGL(k_count, dim3((unsigned)parts, S), dim3(choices / S <= 1024 ? 256 : kCntWG), 0, st, topk_idx,
                       seq_off, token_mask, C, k, division(k), E, S, counts, tokens, accumulate);
  }
  return launched();
}

size_t moe_balance_workspace_size(int32_t C, int32_t E, int32_t S) {
  if (!batch_ok(C, 1, E) || S < 1 || S > MOE_MAX_SEQUENCES) return 0;
  return bal_ws(C, E, S).total;
}

moe_status moe_balance_fwd(const float* logits, const int32_t* topk_idx, int32_t C, int32_t k,
                           int32_t E, const int32_t* seq_off, int32_t S,
                           const uint8_t* token_mask, int32_t score, float alpha,
                           int32_t* counts, int32_t* tokens, float* probs, float* loss,
                           void* ws, size_t ws_bytes, void* stream) {
  if (!logits || !topk_idx || !counts || !tokens || !probs || !loss) return MOE_ERR_INVALID_ARG;
  if (!aligned4(logits) || !aligned4(topk_idx) || !aligned4(counts) || !aligned4(tokens) ||
      !aligned4(probs) || !aligned4(loss) || !aligned4(seq_off))
    return MOE_ERR_INVALID_ARG;
  if (!batch_ok(C, k, E) || S < 1 || S > MOE_MAX_SEQUENCES) return MOE_ERR_UNSUPPORTED;
  if (!seq_ok(seq_off, S) || (score != MOE_SCORE_SIGMOID && score != MOE_SCORE_SOFTMAX))
    return MOE_ERR_INVALID_ARG;
  if (!ws) return MOE_ERR_WORKSPACE;
  const BalWs W = bal_ws(C, E, S);
  if (ws_bytes < W.total || (uintptr_t)ws % 256) return MOE_ERR_WORKSPACE;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  BalArgs a = {};
  a.logits = logits; a.idx = topk_idx; a.off = seq_off; a.mask = token_mask;
  a.C = C; a.k = k; a.E = E; a.S = S;
  a.vec = E % 4 == 0 && (uintptr_t)logits % 16 == 0;
  a.counts = counts; a.tokens = tokens; a.probs = probs; a.loss = loss; a.alpha = alpha;
  a.ticket = reinterpret_cast<uint32_t*>(w8 + W.ctrl);
  a.psum = reinterpret_cast<float*>(w8 + W.psum);
  a.pcnt = reinterpret_cast<uint16_t*>(w8 + W.pcnt);
  a.ptok = reinterpret_cast<int32_t*>(w8 + W.ptok);
  a.dots = reinterpret_cast<float*>(w8 + W.dots);
  a.shift = slot_shift(C, S);
  a.kmul = division(k);
  a.one = S == 1 && C <= kOneSlot && !seq_off;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int slots = a.one ? 1 : num_slots(C, S);
  RF4_BY_ROW(k_bal_part, E, score == MOE_SCORE_SIGMOID, dim3(slots), kPartWG, st, a);
  if (!a.one) hipLaunchKernelGGL(k_bal_final, dim3(expert_blocks(E), S), dim3(kFinWG), 0, st, a);
  return launched();
}

moe_status moe_balance_bwd(const float* logits, const int32_t* counts, const int32_t* tokens,
                           int32_t C, int32_t k, int32_t E, const int32_t* seq_off, int32_t S,
                           const uint8_t* token_mask, int32_t score, float alpha,
                           const float* grad_loss, float* dlogits, int32_t accumulate,
                           void* stream) {
  if (!logits || !counts || !tokens || !grad_loss || !dlogits) return MOE_ERR_INVALID_ARG;
  if (!aligned4(logits) || !aligned4(dlogits) || !aligned4(counts) || !aligned4(tokens) ||
      !aligned4(grad_loss) || !aligned4(seq_off))
    return MOE_ERR_INVALID_ARG;
  if (!batch_ok(C, k, E) || S < 1 || S > MOE_MAX_SEQUENCES) return MOE_ERR_UNSUPPORTED;
  if (!seq_ok(seq_off, S) || (score != MOE_SCORE_SIGMOID && score != MOE_SCORE_SOFTMAX))
    return MOE_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)C * E * 4;
  if (overlap(logits, bytes, dlogits, bytes)) return MOE_ERR_INVALID_ARG;
  BalArgs a = {};
  a.logits = logits; a.off = seq_off; a.mask = token_mask;
  a.C = C; a.k = k; a.E = E; a.S = S; a.alpha = alpha;
  a.vec = E % 4 == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)dlogits % 16 == 0;
  a.vec_counts = E % 4 == 0 && (uintptr_t)counts % 16 == 0;
  a.counts = const_cast<int32_t*>(counts); a.tokens = const_cast<int32_t*>(tokens);
  a.grad = grad_loss; a.dlogits = dlogits; a.accumulate = accumulate;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  // one token per wave until the chip is half full of waves, then up to 4 (both
  // passes with 1, 2, 4, 8: 2048 tokens x 896 18.7, 18.7, 22.3, 27.7 us; 8192
  // 38.7, 35.9, 36.9, 40.4; 65536 x 448 98.0, 97.8, 93.9, 95.0)
  a.per = C < 8192 ? 1 : C >= 16384 ? 4 : 2;
  const int wg = kBalWaves * a.per;
  RF4_BY_ROW(k_bal_bwd, E, score == MOE_SCORE_SIGMOID, dim3((C + wg - 1) / wg), kBalWG, st, a);
  return launched();
}

moe_status moe_route_bwd(const float* logits, const int32_t* topk_idx, const float* topk_dw,
                         int32_t C, int32_t k, int32_t E, const uint8_t* token_mask,
                         float* dlogits, int32_t accumulate, void* stream) {
  if (!logits || !topk_idx || !topk_dw || !dlogits) return MOE_ERR_INVALID_ARG;
  if (!aligned4(logits) || !aligned4(topk_idx) || !aligned4(topk_dw) || !aligned4(dlogits))
    return MOE_ERR_INVALID_ARG;
  if (!batch_ok(C, k, E)) return MOE_ERR_UNSUPPORTED;
  const int64_t bytes = (int64_t)C * E * 4, chosen = (int64_t)C * k * 4;
  if (overlap(logits, bytes, dlogits, bytes) || overlap(topk_dw, chosen, dlogits, bytes) ||
      overlap(topk_idx, chosen, dlogits, bytes))
    return MOE_ERR_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const bool vec = E % 4 == 0 && (uintptr_t)dlogits % 16 == 0;
  const int per = kBalWaves * (k <= 8 ? 8 : k <= 16 ? 4 : 2);
  const dim3 grid((C + per - 1) / per);
  if (k <= 8) hipLaunchKernelGGL(k_route_bwd<8>, grid, dim3(kBalWG), 0, st, logits, topk_idx, topk_dw, C, k, E, token_mask, dlogits, accumulate, vec);
  else if (k <= 16) hipLaunchKernelGGL(k_route_bwd<16>, grid, dim3(kBalWG), 0, st, logits, topk_idx, topk_dw, C, k, E, token_mask, dlogits, accumulate, vec);
  else hipLaunchKernelGGL(k_route_bwd<32>, grid, dim3(kBalWG), 0, st, logits, topk_idx, topk_dw, C, k, E, token_mask, dlogits, accumulate, vec);
  return launched();
}

}  // extern "C"
