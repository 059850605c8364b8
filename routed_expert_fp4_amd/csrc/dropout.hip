// libroutedfp4, dropout whose mask is a function of a seed, an offset and an
// element's place, so that the backward pass forms it again and nothing stores it:
//
//   y[c][k] = base[c][k] + (kept(c, k) ? x[c][k] / (1 - p) : 0)
//
// Bound by memory: x and base in, y out.  16384 x 7168 in bf16: 119 us for 705 MB, 5.9
// TB/s; all vector instructions together are a twelfth of the waves' time.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include <type_traits>

#include "dense.h"

namespace rf4 {
namespace {

struct DArgs {
  const uint8_t *x, *base;
  uint8_t* y;
  int64_t x_pitch, base_pitch, y_pitch;   // bytes
  int C, K, blocks;                       // blocks of eight columns in a row
  Dropout drop;
};

template <int DT, bool DROP, bool BASE>
__global__ __launch_bounds__(256) void k_dropout(DArgs a) {
  constexpr int B = kBytes<DT>;
  Counter ctr = {};
  if constexpr (DROP) ctr = counter_of(a.drop.rng);
  const int64_t n = (int64_t)a.C * a.blocks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t c = i / a.blocks;
    const int k = 8 * (int)(i - c * a.blocks);
    float v[8];
    const uint8_t *px = a.x + c * a.x_pitch, *pb = a.base + c * a.base_pitch;
    Eight<DT> x, b = {};
    if (a.K % 8 == 0) {                 // one branch for both, which are then on their way together
      x = load8<DT>(px + (int64_t)k * B);
      if constexpr (BASE) b = load8<DT>(pb + (int64_t)k * B);
    } else {
      x = load8_of<DT>(px, k, a.K);
      if constexpr (BASE) b = load8_of<DT>(pb, k, a.K);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = get8<DT>(x, j);
    if constexpr (DROP) drop8f(v, a.drop, ctr, k, (uint32_t)c);
    if constexpr (BASE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += get8<DT>(b, j);
    }
    store8_some<DT>(a.y + c * a.y_pitch + (int64_t)k * B, put8<DT>(v), a.K - k);
  }
}

template <int DT>
void launch_dropout(const DArgs& a, hipStream_t st) {
  const int64_t n = ((int64_t)a.C * a.blocks + 255) / 256;
  const dim3 grid((unsigned)(n < 65536 ? n : 65536));
  if (a.drop.drop) {
    if (a.base) hipLaunchKernelGGL((k_dropout<DT, true, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_dropout<DT, true, false>), grid, dim3(256), 0, st, a);
  } else {
    if (a.base) hipLaunchKernelGGL((k_dropout<DT, false, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_dropout<DT, false, false>), grid, dim3(256), 0, st, a);
  }
}

}  // namespace
}  // namespace rf4

using namespace rf4;

extern "C" moe_status moe_dropout(int32_t dtype, const void* x, int64_t x_pitch, int32_t C, int32_t K, const void* base,
                                  int64_t base_pitch, void* y, int64_t y_pitch, double p, const uint64_t* rng,
                                  void* stream) {
  if (!dense_dtype_ok(dtype) || C < 1 || C > MOE_MAX_BATCH_TOKENS || K < 1 || K > MOE_MAX_QUANT_COLS)
    return MOE_ERR_UNSUPPORTED;
  const int64_t s = dense_size(dtype);
  const Rows rx = {x, x_pitch, K, C, s}, rb = {base, base_pitch, K, C, s}, ry = {y, y_pitch, K, C, s};
  moe_status st;
  if ((st = rows_status(rx)) != MOE_OK || (st = rows_status(ry)) != MOE_OK) return st;
  if (base && (st = rows_status(rb)) != MOE_OK) return st;
  if ((share(rx, ry) && !same(rx, ry)) || (share(rb, ry) && !same(rb, ry))) return MOE_ERR_INVALID_ARG;
  DArgs a = {};
  if ((st = dropout_of(p, rng, a.drop)) != MOE_OK) return st;
  const Rows rr = {rng, 2, 2, 1, 8};
  if (a.drop.drop && share(rr, ry)) return MOE_ERR_INVALID_ARG;
  a.x = static_cast<const uint8_t*>(x); a.x_pitch = x_pitch * s;
  a.base = static_cast<const uint8_t*>(base); a.base_pitch = base_pitch * s;
  a.y = static_cast<uint8_t*>(y); a.y_pitch = y_pitch * s;
  a.C = C; a.K = K; a.blocks = (K + 7) / 8;
  hipStream_t q = reinterpret_cast<hipStream_t>(stream);
  if (dtype == MOE_DT_F32) launch_dropout<MOE_DT_F32>(a, q);
  else if (dtype == MOE_DT_BF16) launch_dropout<MOE_DT_BF16>(a, q);
  else launch_dropout<MOE_DT_F16>(a, q);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
