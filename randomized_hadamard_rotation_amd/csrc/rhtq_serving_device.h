// Device helpers of the serving kernels: rows held by 16 lanes, type conversions, signs.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "rhtq.h"
#include "rhtq_device.h"
#include "rhtq_paging.h"

namespace rhtq {

// Value of the lane whose index within its 16 differs in bit B: quad permutes for bits 0 and 1, a half-row mirror (xor 7)
// followed by a quad reverse (xor 3) for bit 2, a rotation by 8 for bit 3.  All are DPP moves, no LDS.
template <int B>
__device__ __forceinline__ int lane_xor16(int v) {
  if constexpr (B == 0) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, false);         // quad_perm [1,0,3,2]
  else if constexpr (B == 1) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, false);    // quad_perm [2,3,0,1]
  else if constexpr (B == 2)
    return __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, false), 0x1B, 0xF, 0xF, false);
  else return __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, false);                         // row_ror:8
}
template <int B>
__device__ __forceinline__ float lane_xor16(float v) {
  return __int_as_float(lane_xor16<B>(__float_as_int(v)));
}

__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, lane_xor16<0>(v));
  v = fmaxf(v, lane_xor16<1>(v));
  v = fmaxf(v, lane_xor16<2>(v));
  return fmaxf(v, lane_xor16<3>(v));
}
__device__ __forceinline__ float sum16(float v) {
  v += lane_xor16<0>(v);
  v += lane_xor16<1>(v);
  v += lane_xor16<2>(v);
  return v + lane_xor16<3>(v);
}
__device__ __forceinline__ int sum16(int v) {
  v += lane_xor16<0>(v);
  v += lane_xor16<1>(v);
  v += lane_xor16<2>(v);
  return v + lane_xor16<3>(v);
}

template <int B, int E>
__device__ __forceinline__ void lane_stage16(float (&v)[E]) {
  // o + v in the lower lane, o - v in the upper: one fma with +-1, rounded as the sum is
  const float sign = (threadIdx.x >> B) & 1 ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = __builtin_fmaf(v[i], sign, lane_xor16<B>(v[i]));
}

// Walsh-Hadamard transform (Sylvester order, no factor) of a row of 16 E elements held by 16 lanes, lane j with elements
// E j .. E j + E - 1: log2 E stages in registers, four between lanes.
template <int E>
__device__ __forceinline__ void fwht16(float (&v)[E]) {
#pragma unroll
  for (int h = 1; h < E; h *= 2)
#pragma unroll
    for (int i = 0; i < E; ++i)
      if ((i & h) == 0) bfly(v[i], v[i | h]);
  lane_stage16<0>(v);
  lane_stage16<1>(v);
  lane_stage16<2>(v);
  lane_stage16<3>(v);
}

// E consecutive values (E = 4, 8 or 16; 16-byte aligned for E >= 8, else 8 E / 4 bytes) as fp32.
template <int T, int E>
__device__ __forceinline__ void load_row(const void* p, int64_t at, float (&v)[E]) {
  if constexpr (T == RHTQ_IN_F32) {
    const float* q = static_cast<const float*>(p) + at;
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const f32x4 t = *reinterpret_cast<const f32x4*>(q + i);
      v[i] = t.x; v[i + 1] = t.y; v[i + 2] = t.z; v[i + 3] = t.w;
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; i += (E >= 8 ? 4 : 2)) {
      if constexpr (E >= 8) {
        const u32x4 t = *reinterpret_cast<const u32x4*>(q + 2 * i);
        w[i] = t.x; w[i + 1] = t.y; w[i + 2] = t.z; w[i + 3] = t.w;
      } else {
        const u32x2 t = *reinterpret_cast<const u32x2*>(q + 2 * i);
        w[i] = t.x; w[i + 1] = t.y;
      }
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      if constexpr (T == RHTQ_IN_BF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        v[2 * i] = __half2float(__ushort_as_half((uint16_t)(w[i] & 0xFFFF)));
        v[2 * i + 1] = __half2float(__ushort_as_half((uint16_t)(w[i] >> 16)));
      }
    }
  }
}

// fp32 to the 16 bits of T, nearest even.
template <int T>
__device__ __forceinline__ uint32_t to16(float v) {
  if constexpr (T == RHTQ_IN_BF16) {
    const __bf16 b = (__bf16)v;
    return __builtin_bit_cast(uint16_t, b);
  } else {
    return __half_as_ushort(__float2half_rn(v));
  }
}

template <int T, int E>
__device__ __forceinline__ void store_row(void* p, int64_t at, const float (&v)[E]) {
  if constexpr (T == RHTQ_IN_F32) {
    float* q = static_cast<float*>(p) + at;
#pragma unroll
    for (int i = 0; i < E; i += 4) *reinterpret_cast<f32x4*>(q + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + at;
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = to16<T>(v[2 * i]) | (to16<T>(v[2 * i + 1]) << 16);
    if constexpr (E >= 8) {
#pragma unroll
      for (int i = 0; i < E / 2; i += 4) *reinterpret_cast<u32x4*>(q + 2 * i) = u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]};
    } else {
      *reinterpret_cast<u32x2*>(q) = u32x2{w[0], w[1]};
    }
  }
}

// Sign bytes of elements at .. at + E - 1 (null: all +1), and x *= +-1 by them.
template <int E>
__device__ __forceinline__ void load_signs(const int8_t* s, int at, uint32_t (&w)[E / 4]) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i) w[i] = 0;
  if (s)
#pragma unroll
    for (int i = 0; i < E / 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(s + at + 4 * i);
}
template <int E>
__device__ __forceinline__ void apply_signs(const uint32_t (&w)[E / 4], float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i)
    v[i] = __uint_as_float(__float_as_uint(v[i]) ^ ((w[i / 4] << (24 - 8 * (i % 4))) & 0x80000000u));
}
template <int E>
__device__ __forceinline__ void apply_signs(const int8_t* s, int at, float (&v)[E]) {
  uint32_t w[E / 4];
  load_signs<E>(s, at, w);
  apply_signs<E>(w, v);
}

// A value that the kernel does not write, at an address that is the same in all lanes, by a scalar load: what waits for vector loads
// does not wait for it, nor the other way round.
__device__ __forceinline__ int32_t load_uniform(const int32_t* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(reinterpret_cast<uintptr_t>(p));
}

}  // namespace rhtq
