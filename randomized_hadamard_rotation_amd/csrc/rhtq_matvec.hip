// Product of a few rotated rows with 4-bit weights: y[t][r] = sum_k x[t][k] s[r][k / g] c[r][k], fp32 sums.
// Bounded by the code bytes for up to about 64 rows of x.
#include "rhtq_internal.h"
#include "rhtq_serving_device.h"
#include "rhtq_serving_internal.h"

namespace rhtq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float e2m1(uint32_t c) {
  const float m[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
  const float v = m[c & 7];
  return c & 8 ? -v : v;
}

__device__ __forceinline__ float e4m3(uint32_t b) {
  const int e = (b >> 3) & 15, m = b & 7;
  const float v = e == 0 ? ldexpf((float)m, -9) : ldexpf((float)(8 + m), e - 10);
  return b & 128 ? -v : v;
}

__device__ __forceinline__ float group_scale(const MatvecArgs& a, int64_t at) {
  if (a.fmt == RHTQ_FMT_INT4) return load_scale(a.scales, at, a.scale_dtype);
  const uint32_t b = static_cast<const uint8_t*>(a.scales)[at];
  if (a.fmt == RHTQ_FMT_NVFP4) return e4m3(b) * a.tensor_scale[0];
  return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

template <int TX, int TY>
__global__ __launch_bounds__(kThreads) void matvec_kernel(MatvecArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t t = blockIdx.y;
  if (r >= a.rows) return;
  const int group = a.group ? a.group : a.n;
  float acc = 0.0f;
  for (int k = 8 * lane; k < a.n; k += 512) {
    float x[8];
    load_row<TX, 8>(a.x, t * a.n + k, x);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(a.packed + (r * a.n + k) / 2);
    float p = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = (w >> (4 * i)) & 15;
      const float v = a.fmt == RHTQ_FMT_INT4 ? (float)((int)(c << 28) >> 28) : e2m1(c);
      p = __builtin_fmaf(v, x[i], p);
    }
    acc = __builtin_fmaf(p, group_scale(a, r * (a.n / group) + k / group), acc);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) acc += __shfl_xor(acc, d);
  if (lane == 0) {
    if constexpr (TY == RHTQ_IN_F32) static_cast<float*>(a.y)[t * a.rows + r] = acc;
    else static_cast<uint16_t*>(a.y)[t * a.rows + r] = (uint16_t)to16<TY>(acc);
  }
}

template <int TX>
hipError_t launch_x(int out, const MatvecArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.rows + 3) / 4), (unsigned)a.tokens);
  if (out == RHTQ_IN_BF16) hipLaunchKernelGGL((matvec_kernel<TX, RHTQ_IN_BF16>), grid, dim3(kThreads), 0, s, a);
  else if (out == RHTQ_IN_F16) hipLaunchKernelGGL((matvec_kernel<TX, RHTQ_IN_F16>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((matvec_kernel<TX, RHTQ_IN_F32>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_matvec(int x_dtype, int out_dtype, const MatvecArgs& a, hipStream_t s) {
  if (x_dtype == RHTQ_IN_BF16) return launch_x<RHTQ_IN_BF16>(out_dtype, a, s);
  if (x_dtype == RHTQ_IN_F16) return launch_x<RHTQ_IN_F16>(out_dtype, a, s);
  return launch_x<RHTQ_IN_F32>(out_dtype, a, s);
}

}  // namespace rhtq
