// libroutedfp4, dense matrices in 4-bit codes with group scales:
//
//   y[c][n] = sum_k x[c][k] W[n][k],   W[n][k] = s[n][g] (q[n][k] - z[n][g]),  g = k / G
//
// One wave per output row: its lanes take 16-byte units of the row's codes
// (32 columns, inside one group), the tokens' products are summed in fp32.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "common.h"

namespace rf4 {
namespace {

struct QArgs {
  const uint8_t* codes;
  int64_t code_pitch;
  const void* scales;
  int64_t scale_pitch;
  const uint8_t* zeros;
  int64_t zero_pitch;
  int N, K, G;
  const void* x;
  int64_t x_pitch;
  int C;
  void* y;
  int64_t y_pitch;
  int accumulate;
};

template <int DT>
__device__ __forceinline__ float ld(const void* p, int64_t i) {
  if (DT == MOE_DT_F32) return static_cast<const float*>(p)[i];
  if (DT == MOE_DT_BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  return __half2float(static_cast<const __half*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void st(void* p, int64_t i, float v) {
  if (DT == MOE_DT_F32) static_cast<float*>(p)[i] = v;
  else if (DT == MOE_DT_BF16) static_cast<__hip_bfloat16*>(p)[i] = __float2bfloat16(v);
  else static_cast<__half*>(p)[i] = __float2half(v);
}

constexpr int kQTok = 8;

template <int DT, int SDT>
__global__ __launch_bounds__(256) void k_quant_row(QArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int n = blockIdx.x * 4 + wave;
  const int c0 = blockIdx.y * kQTok;
  if (n >= a.N) return;
  const uint8_t* row = a.codes + (int64_t)n * a.code_pitch;
  float acc[kQTok];
#pragma unroll
  for (int t = 0; t < kQTok; ++t) acc[t] = 0.0f;
  for (int k0 = 32 * lane; k0 < a.K; k0 += 32 * 64) {
    const uint4 q = *reinterpret_cast<const uint4*>(row + k0 / 2);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const int g = k0 / a.G;
    const float s = ld<SDT>(a.scales, (int64_t)n * a.scale_pitch + g);
    const float z = a.zeros ? (float)a.zeros[(int64_t)n * a.zero_pitch + g] : 8.0f;
    float p[kQTok];
#pragma unroll
    for (int t = 0; t < kQTok; ++t) p[t] = 0.0f;
    for (int i = 0; i < 32 && k0 + i < a.K; ++i) {
      const float v = (float)((w[i >> 3] >> (4 * (i & 7))) & 15u) - z;
#pragma unroll
      for (int t = 0; t < kQTok; ++t)
        if (c0 + t < a.C) p[t] += v * ld<DT>(a.x, (int64_t)(c0 + t) * a.x_pitch + k0 + i);
    }
#pragma unroll
    for (int t = 0; t < kQTok; ++t) acc[t] += s * p[t];
  }
#pragma unroll
  for (int t = 0; t < kQTok; ++t) {
    float v = wave_sum(acc[t]);
    if (lane == 0 && c0 + t < a.C) {
      const int64_t i = (int64_t)(c0 + t) * a.y_pitch + n;
      if (a.accumulate) v += ld<DT>(a.y, i);
      st<DT>(a.y, i, v);
    }
  }
}

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
  return MOE_OK;
}

template <int DT>
void launch_row(const QArgs& a, int sdt, hipStream_t st) {
  const dim3 grid((a.N + 3) / 4, (a.C + kQTok - 1) / kQTok);
  if (sdt == MOE_DT_F32) hipLaunchKernelGGL((k_quant_row<DT, MOE_DT_F32>), grid, dim3(256), 0, st, a);
  else if (sdt == MOE_DT_BF16) hipLaunchKernelGGL((k_quant_row<DT, MOE_DT_BF16>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((k_quant_row<DT, MOE_DT_F16>), grid, dim3(256), 0, st, a);
}

}  // namespace
}  // namespace rf4

using namespace rf4;

extern "C" {

size_t moe_quant_workspace_size(const moe_quant_matrix* m, int32_t dtype, int32_t C) {
  if (matrix_status(m) != MOE_OK || !dtype_ok(dtype) || C < 1 || C > MOE_MAX_TOKENS) return 0;
  return 256;
}

moe_status moe_quant_linear(const moe_quant_matrix* m, int32_t dtype, const void* x,
                            int64_t x_pitch, int32_t C, void* y, int64_t y_pitch,
                            int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  const moe_status ms = matrix_status(m);
  if (ms != MOE_OK) return ms;
  if (!x || !y || x == y) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || C < 1 || C > MOE_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
  if (x_pitch < m->cols || y_pitch < m->rows || (uintptr_t)x % dtype_size(dtype) ||
      (uintptr_t)y % dtype_size(dtype))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (uintptr_t)ws % 256 || ws_bytes < moe_quant_workspace_size(m, dtype, C)) return MOE_ERR_WORKSPACE;
  QArgs a = {};
  a.codes = static_cast<const uint8_t*>(m->codes); a.code_pitch = m->code_pitch;
  a.scales = m->scales; a.scale_pitch = m->scale_pitch;
  a.zeros = m->zeros; a.zero_pitch = m->zero_pitch;
  a.N = m->rows; a.K = m->cols; a.G = m->group;
  a.x = x; a.x_pitch = x_pitch; a.C = C; a.y = y; a.y_pitch = y_pitch; a.accumulate = accumulate;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == MOE_DT_F32) launch_row<MOE_DT_F32>(a, m->scale_dtype, st);
  else if (dtype == MOE_DT_BF16) launch_row<MOE_DT_BF16>(a, m->scale_dtype, st);
  else launch_row<MOE_DT_F16>(a, m->scale_dtype, st);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // extern "C"
