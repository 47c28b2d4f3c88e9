// Product of a few rotated rows with 4-bit weights: y[t][r] = sum_k x[t][k] s[r][k / g] c[r][k].
//
// The weights' bytes bound it (rows * n / 2, once), as long as nothing else takes longer than they do; everything here
// serves that.
//  - x is laid out once, by prepare_kernel: every row of x is divided by a power of two 2^e so that it lies in [-1, 1], and each
//    value becomes two halves, hi = fp16(x) and lo = fp16((x - hi) 2^11): 22 bits, more for values near fp16's exponent range's end.
//    The halves stand in the order in which lanes take them as a matrix operand (below), so they are read as they lie.
//  - Codes become fp16 exactly: INT4 by setting them into the low mantissa bits of 1024 (two values per instruction, 1.25 instructions
//    a value in all), E2M1 by the conversion instruction, with the E4M3 scale of a 16-block (product exact: 2 + 4 bits)
//    or the power of two of a 32-block relative to the largest in its 128 values (exact down to 2^-22 of that one; a wave that meets a block
//    further below takes its steps again with each block's power of two on the block's own sum).
//  - v_mfma_f32_16x16x32_f16 multiplies 16 weight rows by 16 rows of halves (8 tokens, hi and lo); sums are fp32.  INT4 scales multiply
//    the sum of their group.  y = 2^e (sum_hi + 2^-11 sum_lo).
//
// Operand rows m = 4 a + b stand for token 2 a + (b & 1) of a tile of 8, half b >> 1, so that one lane gets both halves of its two tokens.
// A step covers 128 values of k in 4 products of 32; product i, lane group q = lane / 16, takes the 8 codes of one dword at
//   4 q + i (groups >= 128, NVFP4, MXFP4: one 16-byte load),  8 (i / 2) + 2 q + i % 2 (groups of 64),  4 i + q (32 and 16)
// of the row's 16 dwords, so that each product lies inside one scale group (groups of 16: two, the operand masked for each in turn).
#include "rhtq_internal.h"
#include "rhtq_serving_device.h"
#include "rhtq_serving_internal.h"

namespace rhtq {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// How the codes are scaled; also what decides the order of k.
enum Mode { M128, M64, M32, M16, MNV, MMX };

constexpr int kStep = 128;         // values of k in a step
constexpr int kFrag = 1024;        // bytes of one operand: 64 lanes x 16

// Dword (of 16) of a row's step that product i takes in lane group q.
template <int MODE>
__host__ __device__ constexpr int dword_of(int i, int q) {
  return MODE == M64 ? 8 * (i / 2) + 2 * q + i % 2 : (MODE == M32 || MODE == M16 ? 4 * i + q : 4 * q + i);
}
// Value (of 8) of a dword in slot j of the operand: INT4 takes nibbles 16 bits apart in pairs, E2M1 neighbours.
template <int MODE>
__host__ __device__ constexpr int value_of(int j) {
  return MODE == MNV || MODE == MMX ? j : (j >> 1) + 4 * (j & 1);
}

// ---- x: halves in operand order -------------------------------------------------------------------------------------------

constexpr int kPrep = 1024;

// x in [-1, 1] as its two halves.
__device__ __forceinline__ void split_halves(float x, _Float16& hi, _Float16& lo) {
  hi = (_Float16)x;
  lo = (_Float16)((x - (float)hi) * 2048.0f);
}

// Largest of a workgroup's values, in every thread.
template <int WAVES>
__device__ __forceinline__ float workgroup_max(float v, float* wave_max) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WAVES; ++i) v = fmaxf(v, wave_max[i]);
  return v;
}

// One workgroup per token of a tile; tokens beyond the last (and k beyond n) become zeros.  Rows of up to 16384 stay in registers between
// the search for the largest value and the split.
template <int MODE, int TX>
__global__ __launch_bounds__(kPrep) void prepare_kernel(MatvecArgs a) {
  __shared__ float wave_max[kPrep / 64];
  constexpr int HELD = 2;
  const int64_t t = blockIdx.x;
  const int64_t tile = t >> 3;
  const int steps = (a.n + kStep - 1) / kStep;
  const bool real = t < a.tokens;
  float v[HELD][8];
  float top = 0.0f;
  // item u: operand i of step s, lane group q -- a dword of 8 values of k; every dword of the row is one item
  auto k_of = [&](int u) { return kStep * (u >> 4) + 8 * dword_of<MODE>((u >> 2) & 3, u & 3); };
#pragma unroll
  for (int h = 0; h < HELD; ++h) {
    const int u = threadIdx.x + h * kPrep, k = k_of(u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[h][j] = 0.0f;
    if (real && k < a.n) load_row<TX, 8>(a.x, t * a.n + k, v[h]);
  }
#pragma unroll
  for (int h = 0; h < HELD; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, __builtin_fabsf(v[h][j]));
  for (int u = threadIdx.x + HELD * kPrep; u < steps * 16; u += kPrep) {
    float w[8] = {};
    if (real && k_of(u) < a.n) load_row<TX, 8>(a.x, t * a.n + k_of(u), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, __builtin_fabsf(w[j]));
  }
  top = workgroup_max<kPrep / 64>(top, wave_max);
  const int e = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;
  if (threadIdx.x == 0) a.exponents[t] = e;
  const int m_hi = 4 * ((int)(t & 7) >> 1) + (int)(t & 1), m_lo = m_hi + 2;
  uint8_t* out = static_cast<uint8_t*>(a.halves) + tile * steps * 4 * kFrag;
  auto put = [&](int u, const float (&w)[8]) {
    f16x8 hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      _Float16 h, l;
      split_halves(__builtin_amdgcn_ldexpf(w[value_of<MODE>(j)], -e), h, l);
      hi[j] = h;
      lo[j] = l;
    }
    uint8_t* o = out + (int64_t)(u >> 2) * kFrag + 256 * (u & 3);
    *reinterpret_cast<f16x8*>(o + 16 * m_hi) = hi;
    *reinterpret_cast<f16x8*>(o + 16 * m_lo) = lo;
  };
#pragma unroll
  for (int h = 0; h < HELD; ++h)
    if ((int)threadIdx.x + h * kPrep < steps * 16) put(threadIdx.x + h * kPrep, v[h]);
  for (int u = threadIdx.x + HELD * kPrep; u < steps * 16; u += kPrep) {
    float w[8] = {};
    if (real && k_of(u) < a.n) load_row<TX, 8>(a.x, t * a.n + k_of(u), w);
    put(u, w);
  }
}

// ---- weights: one step of a row tile ---------------------------------------------------------------------------------------

// Codes of a lane's row, and what scales them.
struct Codes {
  uint32_t w[4];       // product i's dword
  float s[8];          // convert_scales'
  uint32_t e;          // MNV: two E4M3 bytes
  uint32_t b[8];       // the scales as they lie: MMX the step's four E8M0 bytes, INT4 fp32 or fp16
};

// Every load is made, of a place within the row where the row ends inside the step: x is 0 there, and codes and scales are finite.  With a
// branch around a load, a later wait would not know how many are in flight and would wait for all.
template <int MODE, bool F32>
__device__ __forceinline__ void load_codes(const MatvecArgs& a, int64_t row, int step, int q, Codes& c) {
  const int last = a.n / 8 - 16 * step - 1;           // the row's last dword, counted from this step on
  const uint32_t* p = reinterpret_cast<const uint32_t*>(a.packed) + row * (a.n / 8) + 16 * step;
  if constexpr (MODE == M128 || MODE == MNV || MODE == MMX) {
    const int at = 4 * q < last ? 4 * q : last - 3;   // n is a multiple of 32: four dwords at least
    const u32x4 t = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + at));
    c.w[0] = t.x; c.w[1] = t.y; c.w[2] = t.z; c.w[3] = t.w;
  } else if constexpr (MODE == M64) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int at = 8 * g + 2 * q < last ? 8 * g + 2 * q : last - 1;
      const u32x2 t = *reinterpret_cast<const u32x2*>(p + at);
      c.w[2 * g] = t.x;
      c.w[2 * g + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = p[4 * i + q < last ? 4 * i + q : last];
  }
  const int64_t scales = row * a.groups;
  auto scale_at = [&](int64_t at) {
    if constexpr (F32) return static_cast<const uint32_t*>(a.scales)[at];
    else return (uint32_t) static_cast<const uint16_t*>(a.scales)[at];
  };
  if constexpr (MODE == M128) {
    c.b[0] = scale_at(scales + (a.group_log < 0 ? 0 : (kStep * step) >> a.group_log));
  } else if constexpr (MODE == M64 || MODE == M32 || MODE == M16) {
    constexpr int PER = MODE == M64 ? 2 : (MODE == M32 ? 4 : 8);
#pragma unroll
    for (int g = 0; g < PER; ++g) {
      const int at = PER * step + g;
      c.b[g] = scale_at(scales + (at < a.groups ? at : a.groups - 1));
    }
  } else if constexpr (MODE == MNV) {
    const int at = 4 * q < last ? 2 * q : (last - 3) / 2;
    c.e = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(a.scales) + scales + 8 * step + at);
  } else {
    const uint8_t* s = static_cast<const uint8_t*>(a.scales) + scales + 4 * step;
#pragma unroll
    for (int g = 0; g < 4; ++g) c.b[g] = s[4 * g < last ? g : (last - 3) / 4];
  }
}

constexpr int kFar = 22;           // E2M1 codes times 2^-22 are fp16 numbers still (subnormal ones: 0.5 * 2^-22 = 2^-23)

// The scales as fp32, once they are needed.  MXFP4's powers of two: the step's largest 2^(top - 127), and the lane's block relative to it,
// 2^(own - top).  Returns whether the lane's block has codes that do not fit there.
template <int MODE, bool F32>
__device__ __forceinline__ bool convert_scales(Codes& c, int q) {
  if constexpr (MODE == MMX) {
    uint32_t top = 0, own = c.b[0];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      top = c.b[g] > top ? c.b[g] : top;
      own = g == q ? c.b[g] : own;
    }
    c.s[0] = __builtin_amdgcn_ldexpf(1.0f, (int)top - 127);
    c.s[1] = __builtin_amdgcn_ldexpf(1.0f, own + kFar > top ? (int)own - (int)top : -kFar);
    return own + kFar < top && ((c.w[0] | c.w[1] | c.w[2] | c.w[3]) & 0x77777777u) != 0;
  } else if constexpr (MODE != MNV) {
    constexpr int PER = MODE == M128 ? 1 : (MODE == M64 ? 2 : (MODE == M32 ? 4 : 8));
#pragma unroll
    for (int g = 0; g < PER; ++g) c.s[g] = F32 ? __uint_as_float(c.b[g]) : __half2float(__ushort_as_half((uint16_t)c.b[g]));
  }
  return false;
}

__device__ __forceinline__ f16x2 as_f16x2(uint32_t v) { return __builtin_bit_cast(f16x2, v); }

// The 8 codes of product i as fp16, exactly.
template <int MODE>
__device__ __forceinline__ f16x8 unpack(const Codes& c, int i) {
  f16x2 r[4];
  if constexpr (MODE == MNV || MODE == MMX) {
    const float s = MODE == MMX ? c.s[1] : 1.0f;
    r[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c.w[i], s, 0));
    r[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c.w[i], s, 1));
    r[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c.w[i], s, 2));
    r[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c.w[i], s, 3));
    if constexpr (MODE == MNV) {
      // dwords 0, 1 of the lane's 16 bytes are one 16-block, 2, 3 the next
      const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.e, 1.0f, false));
      const f16x2 f = {b[i >> 1], b[i >> 1]};
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] *= f;
    }
  } else {
    const uint32_t w = c.w[i] ^ 0x88888888u, h = w >> 8;           // nibbles are code + 8
    const f16x2 low = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const f16x2 part = {(_Float16)0.0625f, (_Float16)0.0625f}, high = {(_Float16)-72.0f, (_Float16)-72.0f};
    r[0] = as_f16x2((w & 0x000F000Fu) | 0x64006400u) + low;                               // 1024 + u - 1032
    r[1] = __builtin_elementwise_fma(as_f16x2((w & 0x00F000F0u) | 0x64006400u), part, high);   // (1024 + 16 u) / 16 - 72
    r[2] = as_f16x2((h & 0x000F000Fu) | 0x64006400u) + low;
    r[3] = __builtin_elementwise_fma(as_f16x2((h & 0x00F000F0u) | 0x64006400u), part, high);
  }
  f16x8 o;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[2 * k] = r[k][0];
    o[2 * k + 1] = r[k][1];
  }
  return o;
}

__device__ __forceinline__ f32x4 mma(f16x8 x, f16x8 w, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w, c, 0, 0, 0); }

// acc += a step's products of one token tile: x[i] its operands, w[i] the codes.
template <int MODE>
__device__ __forceinline__ void step_into(f32x4& acc, const f16x8 (&x)[4], const f16x8 (&w)[4], const Codes& c) {
  const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (MODE == MNV) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = mma(x[i], w[i], acc);
  } else if constexpr (MODE == M128 || MODE == MMX) {
    f32x4 d = mma(x[0], w[0], z);
#pragma unroll
    for (int i = 1; i < 4; ++i) d = mma(x[i], w[i], d);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(c.s[0], d[k], acc[k]);
  } else if constexpr (MODE == M64) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const f32x4 d = mma(x[2 * g + 1], w[2 * g + 1], mma(x[2 * g], w[2 * g], z));
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(c.s[g], d[k], acc[k]);
    }
  } else if constexpr (MODE == M32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 d = mma(x[i], w[i], z);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(c.s[i], d[k], acc[k]);
    }
  } else {
    // product i holds groups 2 i (lane groups 0, 1) and 2 i + 1 (2, 3): each with the other's codes out
    const bool upper = (threadIdx.x & 63) >= 32;
    const f16x8 none = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 d0 = mma(x[i], upper ? none : w[i], z), d1 = mma(x[i], upper ? w[i] : none, z);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(c.s[2 * i + 1], d1[k], __builtin_fmaf(c.s[2 * i], d0[k], acc[k]));
    }
  }
}

// The same for MXFP4 blocks of any distance: block g's codes are those of lane group g, so that the others' are left out of its products.
__device__ __forceinline__ void far_step_into(f32x4& acc, const f16x8 (&x)[4], Codes& c) {
  const int q = (threadIdx.x & 63) >> 4;
  const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  const f16x8 none = {};
  c.s[1] = 1.0f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    f32x4 d = z;
#pragma unroll
    for (int i = 0; i < 4; ++i) d = mma(x[i], q == g ? unpack<MMX>(c, i) : none, d);
    const float s = __builtin_amdgcn_ldexpf(1.0f, (int)c.b[g] - 127);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(s, d[k], acc[k]);
  }
}

__device__ __forceinline__ void store_y(const MatvecArgs& a, int64_t t, int64_t row, float v) {
  const int64_t at = t * a.rows + row;
  if (a.out_dtype == RHTQ_IN_F32) static_cast<float*>(a.y)[at] = v;
  else if (a.out_dtype == RHTQ_IN_BF16) static_cast<uint16_t*>(a.y)[at] = (uint16_t)to16<RHTQ_IN_BF16>(v);
  else static_cast<uint16_t*>(a.y)[at] = (uint16_t)to16<RHTQ_IN_F16>(v);
}

// Both halves of a token, times the tensor scale and its power of two, in that order: with the power first, x near fp32's largest values
// would overflow before the tensor scale brings the sum back.
__device__ __forceinline__ float whole(const MatvecArgs& a, int exponent, float hi, float lo) {
  const float v = __builtin_fmaf(lo, 1.0f / 2048.0f, hi);
  return __builtin_amdgcn_ldexpf(a.tensor_scale ? v * a.tensor_scale[0] : v, exponent);
}

// ---- few tokens: one tile of 16 rows per workgroup, k split over its waves -----------------------------------------------------
// 4096 x 4096, 1 token 5.7 us; 24576 x 4096 20 us (2.5 TB/s); 12288 x 4096, 4 tokens NVFP4 12.4 us, MXFP4 20.8: the life of a workgroup is
// one wait for its loads, of which x's operands are four for each of the codes'.

constexpr int kWaves = 8;
constexpr int kAhead = 4;          // steps whose codes and operands are in flight
// Rows of x that a workgroup splits into halves itself, and their width, as LDS holds them.  With one token this took 8.5 us instead of 11.4
// for 4096 x 4096 and 24.3 instead of 28.1 for 24576 x 4096 (rotation included); with four, 12.9 instead of 12.1 and 22.1 instead of 19.8.
constexpr int kOwnTokens = 2;
constexpr int kOwnWidth = 4096;
constexpr int64_t kAcross = 1 << 22;   // row tiles in a grid's x, the rest in y: x times its 512 threads stays below 2^32

// OWN: x fp32 is split by every workgroup for itself, in LDS, while its codes are on their way, which saves a launch; otherwise the halves
// lie ready.  MXFP4's steps over far blocks would take 139 registers; four waves a SIMD, with four values spilled there, took 27.2 us for
// the call at 12288 x 4096, 4 tokens, three waves 28.0.
template <int MODE, bool F32, bool OWN>
__global__ __launch_bounds__(64 * kWaves, MODE == MMX ? 4 : 1) void narrow_kernel(MatvecArgs a) {
  __shared__ f32x4 part[kWaves][64];
  __shared__ float wave_max[kOwnTokens][kWaves];
  // operands: rows t + kOwnTokens * half of lane group q of operand i
  __shared__ __attribute__((aligned(16))) f16x8 own[OWN ? kOwnWidth / 8 : 1][2 * kOwnTokens];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, q = lane >> 4;
  const int64_t row0 = (blockIdx.x + blockIdx.y * kAcross) * 16;
  if (row0 >= a.rows) return;
  const int64_t row = row0 + m < a.rows ? row0 + m : a.rows - 1;
  const int steps = (a.n + kStep - 1) / kStep;
  const int s0 = steps * wave / kWaves, s1 = steps * (wave + 1) / kWaves;
  const int token = 2 * (m >> 2) + (m & 1);                       // of this lane's operand row; half m >> 1 & 1
  // rows of no token take another's: nothing reads what comes of them
  const uint8_t* halves = static_cast<const uint8_t*>(a.halves) + 16 * (token < a.tokens ? lane : 16 * q);
  const int own_row = (token < a.tokens ? token : 0) % kOwnTokens + (m & 2 ? kOwnTokens : 0);
  int exponent[kOwnTokens] = {};

  Codes c[kAhead];
  f16x8 v[kAhead][4];
  auto load = [&](int s) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load_codes<MODE, F32>(a, row, s + k < steps ? s + k : steps - 1, q, c[k]);
    if constexpr (!OWN)
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int step = s + k < steps ? s + k : steps - 1;
          v[k][i] = *reinterpret_cast<const f16x8*>(halves + (int64_t)(4 * step + i) * kFrag);
        }
  };
  if constexpr (OWN) {
    // thread u has item u of each token: 8 values of k, at most one item a token (kOwnWidth / 8 threads)
    const int u = threadIdx.x, k = kStep * (u >> 4) + 8 * dword_of<MODE>((u >> 2) & 3, u & 3);
    float x[kOwnTokens][8];
#pragma unroll
    for (int t = 0; t < kOwnTokens; ++t)
      if (t < a.tokens) load_row<RHTQ_IN_F32, 8>(a.x, t * (int64_t)a.n + (k < a.n ? k : 0), x[t]);
    load(s0);
#pragma unroll
    for (int t = 0; t < kOwnTokens; ++t) {
      if (t >= a.tokens) break;
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[t][e] = k < a.n ? x[t][e] : 0.0f;
        top = fmaxf(top, __builtin_fabsf(x[t][e]));
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
      if (lane == 0) wave_max[t][wave] = top;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kOwnTokens; ++t) {
      if (t >= a.tokens) break;
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) top = fmaxf(top, wave_max[t][i]);
      exponent[t] = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;
      f16x8 hi, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        _Float16 h, l;
        split_halves(__builtin_amdgcn_ldexpf(x[t][value_of<MODE>(e)], -exponent[t]), h, l);
        hi[e] = h;
        lo[e] = l;
      }
      if (u < 16 * steps) {
        own[u][t] = hi;
        own[u][t + kOwnTokens] = lo;
      }
    }
    __syncthreads();
  } else {
    load(s0);
  }
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  bool far = false;
  auto step = [&](int s, int k) {
    f16x8 w[4];
    if constexpr (OWN)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k][i] = own[16 * (s + k) + 4 * i + q][own_row];
    far |= convert_scales<MODE, F32>(c[k], q);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = unpack<MODE>(c[k], i);
    step_into<MODE>(acc, v[k], w, c[k]);
  };
  // Whole batches without a branch between their steps: the compiler moves a load behind a branch that may skip its use.
  int s = s0;
  for (; s + kAhead < s1; load(s)) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) step(s, k);
    s += kAhead;
  }
  if (s + kAhead == s1) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) step(s, k);
  } else {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (s + k < s1) step(s, k);
  }
  if constexpr (MODE == MMX)
    if (__any(far)) {
      acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (s = s0; s < s1; ++s) {
        load_codes<MODE, F32>(a, row, s, q, c[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (OWN) v[0][i] = own[16 * s + 4 * i + q][own_row];
          else v[0][i] = *reinterpret_cast<const f16x8*>(halves + (int64_t)(4 * s + i) * kFrag);
        }
        far_step_into(acc, v[0], c[0]);
      }
    }
  part[wave][lane] = acc;
  __syncthreads();
  // 128 results: row m, token 2 q + b of lane (q, m), b = 0, 1
  if (threadIdx.x >= 128) return;
  const int b = threadIdx.x >> 6;
  float hi = 0.0f, lo = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float* p = reinterpret_cast<const float*>(&part[w][lane]);
    hi += p[b];
    lo += p[b + 2];
  }
  const int t = 2 * q + b;
  if (t >= a.tokens || row0 + m >= a.rows) return;
  int e = 0;
  if constexpr (OWN) {
#pragma unroll
    for (int i = 0; i < kOwnTokens; ++i) e = i == t ? exponent[i] : e;
  } else {
    e = a.exponents[t];
  }
  store_y(a, t, row0 + m, whole(a, e, hi, lo));
}

// ---- many tokens: 256 rows x up to 64 tokens per workgroup, k split over the grid -------------------------------------------
// 4096 x 12288, 16 tokens 13.6 us; 4001 x 11008, 61 tokens 28.5 us: bound by a step's LDS reads (32 KB a wave at 64 tokens), matrix
// and vector instructions in turn.  128 rows read x twice as often: 30 us.  Four row tiles a wave halve the LDS reads but leave one wave a
// SIMD: 40 us.

constexpr int kWide = 512;
constexpr int kWideRows = 256;

// TT token tiles.  Eight waves share the operands of x through two buffers in LDS; each has 32 rows of its own.
template <int MODE, bool F32, int TT>
__global__ __launch_bounds__(kWide) void wide_kernel(MatvecArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t buf[2][4 * TT * kFrag];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  const int64_t tile0 = (int64_t)blockIdx.z * TT;
  const int64_t row0 = (int64_t)blockIdx.x * kWideRows + 32 * wave;
  int64_t row[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) row[r] = row0 + 16 * r + m < a.rows ? row0 + 16 * r + m : a.rows - 1;
  const int steps = (a.n + kStep - 1) / kStep;
  const int s0 = (int)((int64_t)steps * blockIdx.y / a.k_splits), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / a.k_splits);
  const uint8_t* halves = static_cast<const uint8_t*>(a.halves);
  // half the workgroup's threads hold a token tile's operands of a step, 16 bytes each
  constexpr int FETCH = (TT + 1) / 2;
  const int tile_half = threadIdx.x >> 8, piece = 16 * (threadIdx.x & 255);
  u32x4 stage[FETCH];
  auto fetch = [&](int s) {
#pragma unroll
    for (int t = 0; t < FETCH; ++t) {
      const int tile = 2 * t + tile_half < TT ? 2 * t + tile_half : 0;
      stage[t] = *reinterpret_cast<const u32x4*>(halves + ((tile0 + tile) * steps + s) * 4 * kFrag + piece);
    }
  };
  auto put = [&](int b) {
#pragma unroll
    for (int t = 0; t < FETCH; ++t)
      if (TT > 1 || tile_half == 0) *reinterpret_cast<u32x4*>(&buf[b][4 * (2 * t + tile_half) * kFrag + piece]) = stage[t];
  };
  f32x4 acc[2][TT] = {};
  bool far = false;
  Codes next[2];
  fetch(s0);
#pragma unroll
  for (int r = 0; r < 2; ++r) load_codes<MODE, F32>(a, row[r], s0, q, next[r]);
  put(0);
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int b = (s - s0) & 1;
    Codes c[2] = {next[0], next[1]};
    if (s + 1 < s1) {
      fetch(s + 1);
#pragma unroll
      for (int r = 0; r < 2; ++r) load_codes<MODE, F32>(a, row[r], s + 1, q, next[r]);
    }
    f16x8 w[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      far |= convert_scales<MODE, F32>(c[r], q);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[r][i] = unpack<MODE>(c[r], i);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      f16x8 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const f16x8*>(&buf[b][(4 * t + i) * kFrag + 16 * lane]);
#pragma unroll
      for (int r = 0; r < 2; ++r) step_into<MODE>(acc[r][t], v, w[r], c[r]);
    }
    if (s + 1 < s1) put(b ^ 1);
    __syncthreads();
  }
  if constexpr (MODE == MMX)
    if (__any(far))                    // no barrier in here: the waves' rows differ
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        acc[0][t] = acc[1][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int s = s0; s < s1; ++s) {
          f16x8 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = *reinterpret_cast<const f16x8*>(halves + (((tile0 + t) * steps + s) * 4 + i) * kFrag + 16 * lane);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            load_codes<MODE, F32>(a, row[r], s, q, next[r]);
            far_step_into(acc[r][t], v, next[r]);
          }
        }
      }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t at = row0 + 16 * r + m;
    if (at >= a.rows) continue;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int64_t tok = 8 * (tile0 + t) + 2 * q + b;
        if (tok >= a.tokens) continue;
        const float v = whole(a, a.exponents[tok], acc[r][t][b], acc[r][t][b + 2]);
        if (a.k_splits == 1) store_y(a, tok, at, v);
        else a.partial[((int64_t)blockIdx.y * a.tokens + tok) * a.rows + at] = v;
      }
  }
}

__global__ __launch_bounds__(256) void join_kernel(MatvecArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, all = a.tokens * a.rows;
  if (i >= all) return;
  float v = 0.0f;
  for (int k = 0; k < a.k_splits; k += 8) {
    float p[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) p[u] = k + u < a.k_splits ? a.partial[(k + u) * all + i] : 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) v += p[u];
  }
  store_y(a, i / a.rows, i % a.rows, v);
}

constexpr int kNarrowTokens = 4;

template <int MODE, bool F32>
hipError_t launch_mode(int x_dtype, const MatvecArgs& a, hipStream_t s) {
  const unsigned padded = (unsigned)matvec_padded(a.tokens);
  const int64_t all16 = (a.rows + 15) / 16;
  const dim3 tiles16((unsigned)(all16 < kAcross ? all16 : kAcross), (unsigned)((all16 + kAcross - 1) / kAcross));
  if (x_dtype == RHTQ_IN_F32 && a.tokens <= kOwnTokens && a.n <= kOwnWidth) {
    hipLaunchKernelGGL((narrow_kernel<MODE, F32, true>), tiles16, dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
  }
  if (x_dtype == RHTQ_IN_BF16) hipLaunchKernelGGL((prepare_kernel<MODE, RHTQ_IN_BF16>), dim3(padded), dim3(kPrep), 0, s, a);
  else if (x_dtype == RHTQ_IN_F16) hipLaunchKernelGGL((prepare_kernel<MODE, RHTQ_IN_F16>), dim3(padded), dim3(kPrep), 0, s, a);
  else hipLaunchKernelGGL((prepare_kernel<MODE, RHTQ_IN_F32>), dim3(padded), dim3(kPrep), 0, s, a);
  if (a.tokens <= kNarrowTokens) {
    hipLaunchKernelGGL((narrow_kernel<MODE, F32, false>), tiles16, dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
  }
  const unsigned tiles = padded / 8, blocks = (unsigned)((a.rows + kWideRows - 1) / kWideRows), ks = (unsigned)a.k_splits;
  if (tiles == 1) hipLaunchKernelGGL((wide_kernel<MODE, F32, 1>), dim3(blocks, ks, 1), dim3(kWide), 0, s, a);
  else if (tiles == 2) hipLaunchKernelGGL((wide_kernel<MODE, F32, 2>), dim3(blocks, ks, 1), dim3(kWide), 0, s, a);
  else if (tiles <= 4) hipLaunchKernelGGL((wide_kernel<MODE, F32, 4>), dim3(blocks, ks, 1), dim3(kWide), 0, s, a);
  else hipLaunchKernelGGL((wide_kernel<MODE, F32, 8>), dim3(blocks, ks, tiles / 8), dim3(kWide), 0, s, a);
  if (a.k_splits > 1)
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)((a.tokens * a.rows + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Tokens padded to whole tiles: 8, 16, 32 or a multiple of 64.
int64_t matvec_padded(int64_t tokens) {
  return tokens <= 8 ? 8 : (tokens <= 16 ? 16 : (tokens <= 32 ? 32 : (tokens + 63) / 64 * 64));
}

// Parts of k: enough workgroups for the chip, two steps each at least; none where one workgroup's waves split k.
int32_t matvec_splits(int64_t tokens, int32_t n, int64_t rows) {
  if (tokens <= kNarrowTokens) return 1;
  const int64_t blocks = (rows + kWideRows - 1) / kWideRows * ((matvec_padded(tokens) + 63) / 64);
  const int64_t steps = (n + kStep - 1) / kStep;
  int64_t k = 256 / blocks;
  if (k > steps / 2) k = steps / 2;
  return k < 1 ? 1 : (int32_t)k;
}

// Bytes: two halves of every value, an exponent a token, and the parts' sums.
int64_t matvec_halves_bytes(int64_t tokens, int32_t n) {
  return matvec_padded(tokens) * ((n + kStep - 1) / kStep * (int64_t)kStep) * 4;
}

hipError_t launch_matvec(int x_dtype, const MatvecArgs& a, hipStream_t s) {
  if (a.fmt == RHTQ_FMT_NVFP4) return launch_mode<MNV, false>(x_dtype, a, s);
  if (a.fmt == RHTQ_FMT_MXFP4) return launch_mode<MMX, false>(x_dtype, a, s);
  const bool f32 = a.scale_dtype == RHTQ_SCALE_F32;
  const int group = a.group_log < 0 || a.group_log > 7 ? 7 : a.group_log;
  if (group == 7) return f32 ? launch_mode<M128, true>(x_dtype, a, s) : launch_mode<M128, false>(x_dtype, a, s);
  if (group == 6) return f32 ? launch_mode<M64, true>(x_dtype, a, s) : launch_mode<M64, false>(x_dtype, a, s);
  if (group == 5) return f32 ? launch_mode<M32, true>(x_dtype, a, s) : launch_mode<M32, false>(x_dtype, a, s);
  return f32 ? launch_mode<M16, true>(x_dtype, a, s) : launch_mode<M16, false>(x_dtype, a, s);
}

}  // namespace rhtq
