// The paged 4-bit cache: new rows are rotated, quantised and stored in their slot; stored rows are read back.
//
// Per row of d = 64, 128 or 256:  y = H diag(s) x / sqrt(d), scale = fl(max|y| / 7), code = rne(y / scale), and back
// x = diag(s) H (code * scale) / sqrt(d).  Reading, the scale leaves the transform (H (c s) = s (H c)), which then runs on
// whole numbers of at most 8 d and is exact.
//
// A row is held by 16 lanes with d / 16 neighbouring elements each, so loads are 16 bytes a lane at d = 128 and the
// transform is three register stages and four between lanes (DPP).  Bounded by memory for prompts (2 d bytes in, d/2 + scale out)
// and by latency for single tokens, so a row's own loads are issued before its place is looked up.
// A workgroup takes 32 neighbouring tokens of one head: their slots lie side by side in a page, so that a page's lines are written whole
// by one XCD's cache.  Head by head within a token instead, 1.75 M rows took 304 us to store and 318 us to read.
#include "rhtq_internal.h"
#include "rhtq_serving_device.h"
#include "rhtq_serving_internal.h"

namespace rhtq {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;
constexpr int kPer = 2;                  // tokens of a group of 16 lanes

// Sequence of row t: the number of sequences that end at or before t, counted by the 16 lanes of the row together.
__device__ __forceinline__ int sequence_of(const int32_t* starts, int seqs, int64_t t) {
  int n = 0;
  for (int i = 1 + (threadIdx.x & 15); i <= seqs; i += 16) n += starts[i] <= t;
  return sum16(n);
}

// Offset of the row's slot counted in rows of the code arrays, or -1 where it has none.
__device__ __forceinline__ int64_t slot_of(const CacheArgs& a, int64_t t, int head) {
  int s = (int)t;
  int64_t pos;
  if (a.starts) {
    s = sequence_of(a.starts, a.seqs, t);
    if (s >= a.seqs || t < a.starts[s]) return -1;
    pos = row_position(t, a.starts[s + 1], a.lengths[s]);
  } else {
    pos = (int64_t)a.lengths[s] - 1;
  }
  if (pos < 0) return -1;
  const int p = page_at(a.table + (int64_t)s * a.width, a.width, a.pages, pos >> a.page_log);
  if (p < 0) return -1;
  return (((int64_t)p * a.kv_heads + head) << a.page_log) + (pos & ((1 << a.page_log) - 1));
}

template <int T, int E>
__global__ __launch_bounds__(kThreads) void append_kernel(CacheArgs a) {
  constexpr int D = 16 * E;
  const int j = threadIdx.x & 15;
  const int head = blockIdx.y, which = blockIdx.z;
  const int64_t t0 = (int64_t)blockIdx.x * (kGroups * kPer) + (threadIdx.x >> 4);
  float v[kPer][E];
  uint32_t signs[E / 4];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t t = t0 + k * kGroups < a.tokens ? t0 + k * kGroups : a.tokens - 1;
    load_row<T, E>(a.x[which], t * a.token_stride[which] + head * a.head_stride[which] + j * E, v[k]);
  }
  load_signs<E>(a.signs[which], j * E, signs);
  int64_t slot[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) slot[k] = t0 + k * kGroups < a.tokens ? slot_of(a, t0 + k * kGroups, head) : -1;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    apply_signs<E>(signs, v[k]);
    fwht16<E>(v[k]);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) amax = fmaxf(amax, __builtin_fabsf(v[k][i]));
    amax = max16(amax);
    const float cnorm = E == 4 ? 0.125f : (E == 8 ? 0.088388347648318447f : 0.0625f);
    const Int4Scale sc = int4_scale(amax, cnorm, a.scale_dtype);
    uint32_t w[(E + 7) / 8] = {};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      // 1.5 * 2^23 + c: the sum's low four bits are the code's
      const float c = fminf(fmaxf(v[k][i] * sc.inv, -8.0f), 7.0f) + 12582912.0f;
      w[i >> 3] |= (__float_as_uint(c) & 15u) << (4 * (i & 7));
    }
    if (slot[k] < 0) continue;
    uint8_t* out = a.codes[which] + slot[k] * (D / 2) + j * (E / 2);
    if constexpr (E == 4) *reinterpret_cast<uint16_t*>(out) = (uint16_t)w[0];
    else if constexpr (E == 8) *reinterpret_cast<uint32_t*>(out) = w[0];
    else *reinterpret_cast<u32x2*>(out) = u32x2{w[0], w[1]};
    if (j == 0) {
      if (a.scale_dtype == RHTQ_SCALE_F32) static_cast<float*>(a.scales[which])[slot[k]] = sc.s;
      else static_cast<__half*>(a.scales[which])[slot[k]] = __float2half_rn(fminf(sc.s, 65504.0f));
    }
  }
}

template <int T, int E>
__global__ __launch_bounds__(kThreads) void read_kernel(CacheArgs a) {
  constexpr int D = 16 * E;
  const int j = threadIdx.x & 15;
  const int head = blockIdx.y, which = blockIdx.z;
  if (!a.y[which]) return;
  const int64_t t0 = (int64_t)blockIdx.x * (kGroups * kPer) + (threadIdx.x >> 4);
  uint32_t signs[E / 4];
  load_signs<E>(a.signs[which], j * E, signs);
  int64_t slot[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) slot[k] = t0 + k * kGroups < a.tokens ? slot_of(a, t0 + k * kGroups, head) : -1;
  uint32_t w[kPer][(E + 7) / 8] = {};
  float s[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    s[k] = 0.0f;
    if (slot[k] < 0) continue;
    const uint8_t* in = a.codes[which] + slot[k] * (D / 2) + j * (E / 2);
    if constexpr (E == 4) w[k][0] = *reinterpret_cast<const uint16_t*>(in);
    else if constexpr (E == 8) w[k][0] = *reinterpret_cast<const uint32_t*>(in);
    else {
      const u32x2 q = *reinterpret_cast<const u32x2*>(in);
      w[k][0] = q.x;
      w[k][1] = q.y;
    }
    s[k] = load_scale(a.scales[which], slot[k], a.scale_dtype);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (t0 + k * kGroups >= a.tokens) continue;
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = (float)((int)(w[k][i >> 3] << (28 - 4 * (i & 7))) >> 28);
    fwht16<E>(v);
    const float cnorm = E == 4 ? 0.125f : (E == 8 ? 0.088388347648318447f : 0.0625f);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= s[k] * cnorm;
    apply_signs<E>(signs, v);
    store_row<T, E>(a.y[which], ((t0 + k * kGroups) * a.kv_heads + head) * D + j * E, v);
  }
}

// Tokens in x, heads in y, keys and values in z.
dim3 grid_of(const CacheArgs& a) {
  constexpr int per = kGroups * kPer;
  return dim3((unsigned)((a.tokens + per - 1) / per), (unsigned)a.kv_heads, 2);
}

template <int T>
hipError_t launch_append_t(const CacheArgs& a, dim3 grid, hipStream_t s) {
  switch (a.head_dim) {
    case 64: hipLaunchKernelGGL((append_kernel<T, 4>), grid, dim3(kThreads), 0, s, a); break;
    case 128: hipLaunchKernelGGL((append_kernel<T, 8>), grid, dim3(kThreads), 0, s, a); break;
    default: hipLaunchKernelGGL((append_kernel<T, 16>), grid, dim3(kThreads), 0, s, a); break;
  }
  return hipGetLastError();
}

template <int T>
hipError_t launch_read_t(const CacheArgs& a, dim3 grid, hipStream_t s) {
  switch (a.head_dim) {
    case 64: hipLaunchKernelGGL((read_kernel<T, 4>), grid, dim3(kThreads), 0, s, a); break;
    case 128: hipLaunchKernelGGL((read_kernel<T, 8>), grid, dim3(kThreads), 0, s, a); break;
    default: hipLaunchKernelGGL((read_kernel<T, 16>), grid, dim3(kThreads), 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(int dtype, const CacheArgs& a, hipStream_t s) {
  const dim3 grid = grid_of(a);
  if (dtype == RHTQ_IN_BF16) return launch_append_t<RHTQ_IN_BF16>(a, grid, s);
  if (dtype == RHTQ_IN_F16) return launch_append_t<RHTQ_IN_F16>(a, grid, s);
  return launch_append_t<RHTQ_IN_F32>(a, grid, s);
}

hipError_t launch_cache_read(int dtype, const CacheArgs& a, hipStream_t s) {
  const dim3 grid = grid_of(a);
  if (dtype == RHTQ_IN_BF16) return launch_read_t<RHTQ_IN_BF16>(a, grid, s);
  if (dtype == RHTQ_IN_F16) return launch_read_t<RHTQ_IN_F16>(a, grid, s);
  return launch_read_t<RHTQ_IN_F32>(a, grid, s);
}

}  // namespace rhtq
