// Products of rows that are quantised on both sides: y[t][r] = sum_k a[t][k] w[r][k], dense or with weights by expert.
//
// The codes go to the matrix cores as they are, or as the smallest type that holds them exactly:
//  - INT4 x INT4, INT8 x INT4: v_mfma_i32_16x16x64_i8.  A 4-bit code stands in the upper half of its byte (16 times its value), so that a
//    dword's eight codes are two masks and a shift; the factor 16 or 256 is taken out of the sum.  Sums are whole numbers up to the end of a
//    scale group, then fp32.
//  - MXFP4 x MXFP4, MXFP8 x MXFP4: v_mfma_scale_f32_16x16x128_f8f6f4, which applies both E8M0 scales itself.  E4M3 codes of one product
//    may be 2^17 apart, which its sums do not hold (they were off by up to 2^-13 of the sum of magnitudes); codes of at least 2 and those
//    below go through two instructions, each exact to fp32.
//  - NVFP4 x NVFP4: code times E4M3 block scale has six significant bits and lies in 2^-10 .. 2688, so it is an fp16 number:
//    v_mfma_f32_16x16x32_f16.  The tensor scales multiply the sum.
//
// A step is 128 values of k.  Lane (m, q) of a wave, m = lane & 15, q = lane >> 4, holds values 32 q .. 32 q + 31 of row m of an operand
// (16 bytes of 4-bit codes): one scaled instruction, or two i8 or four f16 ones over parts of the lane's values -- the order of k is the
// same on both sides, and a sum does not care which.  8-bit codes lie as the instruction wants them (E4M3: 16 q .. and 64 + 16 q ..; INT8: 32 q ..,
// even and odd ones apart like the nibbles).  Scale groups below 128 take the lanes of the others out of one operand (groups of 64, 32) or half a
// lane's bytes (16).
#include "rhtq_internal.h"
#include "rhtq_products_internal.h"
#include "rhtq_serving_device.h"

namespace rhtq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

enum Kind { KI4, KI8, KNV, KM4, KM8 };

constexpr int kStep = 128;               // values of k in a step
constexpr int kStepBytes = kStep / 2;    // of a row of 4-bit codes
// INT4 and INT8 with one scale a row on both sides: whole numbers all the way.  127 * 8 * 16 * 2^16 and 64 * 256 * 2^16 are at most 2^30.
constexpr int kMostWholeSum = 1 << 16;

template <int K>
constexpr bool kWhole = K == KI4 || K == KI8;
template <int K>
constexpr int kActBytes = K == KI8 || K == KM8 ? kStep : kStepBytes;   // of a row of activations in a step

// How INT scales apply.  SUB: parts of a step with scales of their own; 0: one scale a row on both sides, applied at the end.
template <int K, int SUB>
constexpr int kScaleWords = kWhole<K> ? (SUB ? SUB : 1) : (K == KNV ? 2 : 1);   // dwords of a row's scales in a step, as LDS holds them

// ---- scales of a row's step -------------------------------------------------------------------------------------------------

// INT: the scale, as it lies, of part j of SUB of a row's step.
template <int SUB>
__device__ __forceinline__ uint32_t part_scale(const RowsArgs& r, int64_t row, int step, int j) {
  const int at = r.group_log < 0 ? 0 : (kStep * step + j * (kStep / SUB)) >> r.group_log;
  const int64_t i = row * r.groups + (at < r.groups ? at : r.groups - 1);
  return r.f32 ? static_cast<const uint32_t*>(r.scales)[i] : static_cast<const uint16_t*>(r.scales)[i];
}

template <int K, int SUB>
__device__ __forceinline__ void load_scales(const RowsArgs& r, int64_t row, int step, uint32_t (&v)[kScaleWords<K, SUB>]) {
  if constexpr (kWhole<K>) {
    if constexpr (SUB > 0) {
#pragma unroll
      for (int j = 0; j < SUB; ++j) v[j] = part_scale<SUB>(r, row, step, j);
    } else {
      v[0] = 0;
    }
  } else {
    constexpr int BLOCKS = K == KNV ? 8 : 4;
    const uint8_t* p = static_cast<const uint8_t*>(r.scales) + row * r.groups + BLOCKS * step;
    if (r.wide) {
      if constexpr (K == KNV) {
        const u32x2 t = *reinterpret_cast<const u32x2*>(p);
        v[0] = t.x;
        v[1] = t.y;
      } else {
        v[0] = *reinterpret_cast<const uint32_t*>(p);
      }
    } else {
      const int last = r.groups - 1 - BLOCKS * step;
#pragma unroll
      for (int i = 0; i < BLOCKS / 4; ++i) {
        v[i] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) v[i] |= (uint32_t)p[4 * i + b < last ? 4 * i + b : last] << (8 * b);
      }
    }
  }
}

// A scale as loaded, in the form that the products use.
template <int K>
__device__ __forceinline__ uint32_t scale_value(const RowsArgs& r, uint32_t v) {
  if constexpr (kWhole<K>) return r.f32 ? v : __float_as_uint(__half2float(__ushort_as_half((uint16_t)v)));
  return v;
}

__device__ __forceinline__ float row_scale(const RowsArgs& r, int64_t row) {
  return r.f32 ? static_cast<const float*>(r.scales)[row * r.groups] : __half2float(static_cast<const __half*>(r.scales)[row * r.groups]);
}

// ---- operands ----------------------------------------------------------------------------------------------------------------

__device__ __forceinline__ i32x4 low_nibbles(u32x4 w) {
  return i32x4{(int)((w.x << 4) & 0xF0F0F0F0u), (int)((w.y << 4) & 0xF0F0F0F0u), (int)((w.z << 4) & 0xF0F0F0F0u), (int)((w.w << 4) & 0xF0F0F0F0u)};
}
__device__ __forceinline__ i32x4 high_nibbles(u32x4 w) {
  return i32x4{(int)(w.x & 0xF0F0F0F0u), (int)(w.y & 0xF0F0F0F0u), (int)(w.z & 0xF0F0F0F0u), (int)(w.w & 0xF0F0F0F0u)};
}
__device__ __forceinline__ i32x8 as_fp4(u32x4 w) { return i32x8{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0}; }

// The 8 codes of a dword times their block's scale (two equal halves), exactly.
__device__ __forceinline__ f16x8 scaled_fp4(uint32_t w, f16x2 s) {
  f16x2 r[4];
  r[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
  r[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
  r[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
  r[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
  f16x8 o;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    r[k] *= s;
    o[2 * k] = r[k][0];
    o[2 * k + 1] = r[k][1];
  }
  return o;
}

// A lane's operand of a step of one row tile, ready for the instructions: of weights (ACT false) or activations.
template <int K, bool ACT>
struct Operand {
  // INT: even and odd values; NV: four parts of 8; MX: the codes (E4M3: the large and the small ones)
  i32x4 part[K == KNV ? 4 : ((K == KM4 || (K == KM8 && !ACT)) ? 1 : (K == KM8 ? 4 : 2))];
  int scale;                             // MX
};

// raw: the lane's codes, 16 bytes, or 32 for 8-bit activations; scale: E8M0 byte, or two E4M3 ones.
template <int K, bool ACT>
__device__ __forceinline__ void make_operand(const u32x4* raw, uint32_t scale, Operand<K, ACT>& o) {
  if constexpr (K == KNV) {
    const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scale, 1.0f, false));
    const f16x2 s0 = {b[0], b[0]}, s1 = {b[1], b[1]};
    o.part[0] = __builtin_bit_cast(i32x4, scaled_fp4(raw[0].x, s0));
    o.part[1] = __builtin_bit_cast(i32x4, scaled_fp4(raw[0].y, s0));
    o.part[2] = __builtin_bit_cast(i32x4, scaled_fp4(raw[0].z, s1));
    o.part[3] = __builtin_bit_cast(i32x4, scaled_fp4(raw[0].w, s1));
  } else if constexpr (K == KI8 && ACT) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      o.part[0][2 * h] = (int)__builtin_amdgcn_perm(raw[h].y, raw[h].x, 0x06040200u);
      o.part[1][2 * h] = (int)__builtin_amdgcn_perm(raw[h].y, raw[h].x, 0x07050301u);
      o.part[0][2 * h + 1] = (int)__builtin_amdgcn_perm(raw[h].w, raw[h].z, 0x06040200u);
      o.part[1][2 * h + 1] = (int)__builtin_amdgcn_perm(raw[h].w, raw[h].z, 0x07050301u);
    }
  } else if constexpr (kWhole<K>) {
    o.part[0] = low_nibbles(raw[0]);
    o.part[1] = high_nibbles(raw[0]);
  } else if constexpr (K == KM8 && ACT) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // bit 6 set: exponent field of 8 or more, a value of at least 2
        const uint32_t v = raw[h][j], t = v & 0x40404040u, large = t | (t - (t >> 6));
        o.part[h][j] = (int)(v & (large | 0x80808080u));
        o.part[2 + h][j] = (int)(v & ~large);
      }
    o.scale = (int)scale;
  } else {
    o.part[0] = __builtin_bit_cast(i32x4, raw[0]);
    o.scale = (int)scale;
  }
}

__device__ __forceinline__ i32x8 join8(i32x4 a, i32x4 b) { return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

// c += a step's products: rows of x to rows of the tile, rows of y to its columns.  Of the formats whose sums run over all of k.
template <int K, bool FIRST_ACT, bool SECOND_ACT>
__device__ __forceinline__ f32x4 step_sum(const Operand<K, FIRST_ACT>& x, const Operand<K, SECOND_ACT>& y, f32x4 c) {
  if constexpr (K == KNV) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x.part[i]), __builtin_bit_cast(f16x8, y.part[i]), c, 0, 0, 0);
    return c;
  } else if constexpr (K == KM4) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join8(x.part[0], i32x4{}), join8(y.part[0], i32x4{}), c, 4, 4, 0, x.scale, 0, y.scale);
  } else if constexpr (FIRST_ACT) {
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join8(x.part[0], x.part[1]), join8(y.part[0], i32x4{}), c, 0, 4, 0, x.scale, 0, y.scale);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join8(x.part[2], x.part[3]), join8(y.part[0], i32x4{}), c, 0, 4, 0, x.scale, 0, y.scale);
  } else {
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join8(x.part[0], i32x4{}), join8(y.part[0], y.part[1]), c, 4, 0, 0, x.scale, 0, y.scale);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join8(x.part[0], i32x4{}), join8(y.part[2], y.part[3]), c, 4, 0, 0, x.scale, 0, y.scale);
  }
}

// Whole sums of part j of SUB of a step.  x is the operand whose other parts are left out.
template <int SUB, class X, class Y>
__device__ __forceinline__ i32x4 whole_sum(const X& x, const Y& y, i32x4 c, int j = 0) {
  const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    i32x4 v = x.part[i];
    if constexpr (SUB > 1) {
      // groups of 16: a lane's first 16 values are two dwords of either part's four
      const int own = SUB == 2 ? q >> 1 : (SUB == 4 ? q : 2 * q);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = own + (SUB == 8 ? k >> 1 : 0) == j ? v[k] : 0;
    }
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, y.part[i], c, 0, 0, 0);
  }
  return c;
}

template <int K>
constexpr float kWholeUnit = K == KI4 ? 1.0f / 256.0f : 1.0f / 16.0f;

// Values of the last step that lie behind the row's end: out of the activations' operand.
template <int K, bool ACT>
__device__ __forceinline__ void cut_tail(u32x4* raw, int left) {
  const int q = (threadIdx.x & 63) >> 4;
  const u32x4 none = {0u, 0u, 0u, 0u};
  if constexpr (K == KM8 && ACT) {
    raw[0] = 16 * q < left ? raw[0] : none;
    raw[1] = 64 + 16 * q < left ? raw[1] : none;
  } else {
    raw[0] = 32 * q < left ? raw[0] : none;
    if constexpr (K == KI8 && ACT) raw[1] = 32 * q < left ? raw[1] : none;
  }
}

// ---- experts -------------------------------------------------------------------------------------------------------------------

struct Span {
  int32_t expert;
  int64_t first;              // rows of y: this tile's first, and the expert's end
  int64_t end;
};

// The slot-th tile of `size` rows, counted through the experts' lists; false where there are fewer.  Every lane of the wave takes part.
__device__ __forceinline__ bool find_span(const ProductArgs& p, int slot, int size, Span& s) {
  if (!p.starts) {
    s = {0, (int64_t)slot * size, p.tokens};
    return s.first < p.tokens;
  }
  const int lane = threadIdx.x & 63;
  const int tokens = (int)p.tokens;
  int before = 0;
  for (int base = 0; base < p.experts; base += 64) {
    const int e = base + lane;
    int from = 0, to = 0;
    if (e < p.experts) {
      from = p.starts[e];
      to = p.starts[e + 1];
    }
    from = from < 0 ? 0 : (from > tokens ? tokens : from);
    to = to < from ? from : (to > tokens ? tokens : to);
    const int tiles = (to - from + size - 1) / size;
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      upto += lane >= d ? v : 0;
    }
    const uint64_t reached = __builtin_amdgcn_ballot_w64(before + upto > slot);
    if (reached) {
      const int l = __builtin_ctzll(reached);
      const int f = __builtin_amdgcn_readlane(from, l), g = __builtin_amdgcn_readlane(to, l);
      const int skipped = before + __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l);
      s.expert = base + l;
      s.first = f + (int64_t)(slot - skipped) * size;
      s.end = g;
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// Row of a for row t of y, -1: none.
__device__ __forceinline__ int64_t row_of(const ProductArgs& p, int64_t t) {
  if (!p.index) return t;
  const int32_t i = p.index[t];
  return i >= 0 && i < p.a_rows ? i : -1;
}

__device__ __forceinline__ void store_one(const ProductArgs& p, int64_t t, int64_t r, float v) {
  const int64_t at = t * p.rows + r;
  if (p.out_dtype == RHTQ_IN_F32) static_cast<float*>(p.y)[at] = v;
  else if (p.out_dtype == RHTQ_IN_BF16) static_cast<uint16_t*>(p.y)[at] = (uint16_t)to16<RHTQ_IN_BF16>(v);
  else static_cast<uint16_t*>(p.y)[at] = (uint16_t)to16<RHTQ_IN_F16>(v);
}

// Four results next to each other; r a multiple of 4.
__device__ __forceinline__ void store_four(const ProductArgs& p, int64_t t, int64_t r, f32x4 v) {
  if ((p.rows & 3) != 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + i < p.rows) store_one(p, t, r + i, v[i]);
    return;
  }
  const int64_t at = t * p.rows + r;
  if (p.out_dtype == RHTQ_IN_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(p.y) + at) = v;
  } else {
    const bool bf = p.out_dtype == RHTQ_IN_BF16;
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = bf ? to16<RHTQ_IN_BF16>(v[i]) : to16<RHTQ_IN_F16>(v[i]);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.y) + at) = u32x2{h[0] | h[1] << 16, h[2] | h[3] << 16};
  }
}

// ---- tiles: codes through LDS ----------------------------------------------------------------------------------------------------

typedef const __attribute__((address_space(1))) uint32_t* GlobalWord;
typedef __attribute__((address_space(3))) uint32_t* LocalWord;

// 16 bytes a lane from global memory to LDS at `to` (the same in all lanes) + 16 * lane.
__device__ __forceinline__ void fetch16(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds((GlobalWord) reinterpret_cast<uintptr_t>(from), (LocalWord) reinterpret_cast<uintptr_t>(to), 16, 0, 0);
}

// Where 16-byte piece c of row r stands in its row: 16 lanes that read the same piece of 16 rows meet 64 different banks.
template <int BYTES>
__device__ __forceinline__ int placed(int r, int c) {
  return BYTES == 64 ? c ^ ((r >> 2) & 3) : c ^ ((r >> 1) & 7);
}

// Block id to tile: blocks of one XCD (every eighth) take neighbouring tiles, in bands of token tiles, so that an XCD's L2 serves each row of
// codes to several of its workgroups.
__device__ __forceinline__ void tile_of(int64_t id, int64_t all, int row_tiles, int token_tiles, int& rt, int& tt) {
  constexpr int XCDS = 8, BAND = 8;
  const int64_t each = all / XCDS, more = all % XCDS, xcd = id % XCDS;
  const int64_t at = xcd * each + (xcd < more ? xcd : more) + id / XCDS;
  const int64_t band_size = (int64_t)BAND * row_tiles;
  const int band = (int)(at / band_size), in = (int)(at % band_size);
  const int first = band * BAND, height = token_tiles - first < BAND ? token_tiles - first : BAND;
  tt = first + in % height;
  rt = in / height;
}

// FR x FT tiles of 16 weight rows x 16 tokens a wave, WR x WT waves.
template <int K, int SUB, int FR, int FT, int WR, int WT>
__global__ __launch_bounds__(64 * WR * WT) void tile_kernel(ProductArgs p, int row_tiles, int token_tiles) {
  constexpr int WAVES = WR * WT, TR = 16 * FR * WR, TT = 16 * FT * WT;
  constexpr int AB = kActBytes<K>, WORDS = kScaleWords<K, SUB>;
  constexpr int CODES = TR * kStepBytes + TT * AB;                 // bytes of a step's codes
  constexpr int PIECES_W = TR * kStepBytes / 1024, PIECES = CODES / 1024;   // of a wave's 64 x 16 bytes
  constexpr int MINE = (PIECES + WAVES - 1) / WAVES;
  constexpr bool SCALES = !(kWhole<K> && SUB == 0);
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][CODES];
  __shared__ __attribute__((aligned(16))) uint32_t scales[2][SCALES ? (TR + TT) * WORDS : 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, q = lane >> 4;
  const int wr = wave % WR, wt = wave / WR;
  int rt, tt;
  tile_of(blockIdx.x, (int64_t)row_tiles * token_tiles, row_tiles, token_tiles, rt, tt);
  Span span;
  if (!find_span(p, tt, TT, span)) return;
  const int64_t row0 = (int64_t)rt * TR, tok0 = span.first;
  const int64_t expert_row = span.expert * p.rows;

  const int steps = (p.n + kStep - 1) / kStep;
  const int s0 = (int)((int64_t)steps * blockIdx.y / p.k_splits), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / p.k_splits);
  const int left = p.n - (steps - 1) * kStep;                      // values in the last step

  // this lane's pieces: where they begin in their rows, and which part of the step's bytes
  const uint8_t* from[MINE];
  int part[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    const int piece = i * WAVES + wave;
    if (piece < PIECES_W) {
      const int r = 16 * piece + (lane >> 2);
      part[i] = 16 * placed<64>(r, lane & 3);
      const int64_t row = row0 + r < p.rows ? row0 + r : p.rows - 1;
      from[i] = p.w.codes + (expert_row + row) * (p.n / 2);
    } else {
      constexpr int PER = AB / 16;
      const int r = (64 * (piece - PIECES_W) + lane) / PER;
      part[i] = 16 * placed<AB>(r, lane % PER);
      const int64_t t = tok0 + r < span.end ? tok0 + r : span.end - 1;
      const int64_t row = row_of(p, t);
      from[i] = p.a.codes + (row < 0 ? 0 : row) * (AB == kStep ? p.n : p.n / 2);
    }
  }
  auto fetch = [&](int s, int b) {
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int piece = i * WAVES + wave;
      if (piece >= PIECES) break;
      const bool weights = piece < PIECES_W;
      const int bytes = weights || AB == kStepBytes ? kStepBytes : kStep;
      int at = part[i];
      if (s == steps - 1) {
        const int end = bytes == kStep ? left : left / 2;          // a multiple of 16: its last piece for those behind it
        at = at < end ? at : end - 16;
      }
      fetch16(from[i] + (int64_t)s * bytes + at, &codes[b][1024 * piece]);
    }
  };
  // a row's scales are one thread's
  constexpr int ROWS_EACH = (TR + TT + 64 * WAVES - 1) / (64 * WAVES);
  uint32_t held[ROWS_EACH][WORDS];
  int64_t scale_row[ROWS_EACH];
#pragma unroll
  for (int i = 0; i < ROWS_EACH; ++i) {
    const int r = threadIdx.x + i * 64 * WAVES;
    if (r < TR) {
      scale_row[i] = expert_row + (row0 + r < p.rows ? row0 + r : p.rows - 1);
    } else {
      const int64_t t = tok0 + r - TR < span.end ? tok0 + r - TR : span.end - 1;
      const int64_t row = row_of(p, t);
      scale_row[i] = row < 0 ? 0 : row;
    }
  }
  auto fetch_scales = [&](int s) {
    if constexpr (SCALES)
#pragma unroll
      for (int i = 0; i < ROWS_EACH; ++i) {
        const int r = threadIdx.x + i * 64 * WAVES;
        if (r < TR) load_scales<K, SUB>(p.w, scale_row[i], s, held[i]);
        else if (r < TR + TT) load_scales<K, SUB>(p.a, scale_row[i], s, held[i]);
      }
  };
  auto put_scales = [&](int b) {
    if constexpr (SCALES)
#pragma unroll
      for (int i = 0; i < ROWS_EACH; ++i) {
        const int r = threadIdx.x + i * 64 * WAVES;
        if (r >= TR + TT) continue;
#pragma unroll
        for (int j = 0; j < WORDS; ++j) {
          const uint32_t v = r < TR ? scale_value<K>(p.w, held[i][j]) : scale_value<K>(p.a, held[i][j]);
          if constexpr (kWhole<K>) scales[b][j * (TR + TT) + r] = v;
          else scales[b][r * WORDS + j] = v;
        }
      }
  };
  // E8M0 byte, or two E4M3 ones, of row r (of TR + TT) and this lane's 32 values
  auto block_scale = [&](int b, int r) -> uint32_t {
    if constexpr (K == KNV) return reinterpret_cast<const uint16_t*>(scales[b])[4 * r + q];
    else if constexpr (!kWhole<K>) return reinterpret_cast<const uint8_t*>(scales[b])[4 * r + q];
    else return 0;
  };

  constexpr bool ENDS = kWhole<K> && SUB == 0;                     // scales at the end
  f32x4 acc[FR][FT] = {};
  i32x4 whole[ENDS ? FR : 1][ENDS ? FT : 1] = {};
  fetch(s0, 0);
  fetch_scales(s0);
  put_scales(0);
  for (int s = s0; s < s1; ++s) {
    const int b = (s - s0) & 1;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");               // this wave's pieces are in LDS; then everybody's
    __syncthreads();
    // everything that this step reads of LDS, before the next one's pieces are on their way
    u32x4 raw_w[FR], raw_a[FT][AB / 64];
    uint32_t sw[FR], sa[FT];
#pragma unroll
    for (int i = 0; i < FR; ++i) {
      const int r = 16 * (FR * wr + i) + m;
      raw_w[i] = *reinterpret_cast<const u32x4*>(&codes[b][r * kStepBytes + 16 * placed<64>(r, q)]);
      sw[i] = block_scale(b, r);
    }
#pragma unroll
    for (int i = 0; i < FT; ++i) {
      const int r = 16 * (FT * wt + i) + m;
      const uint8_t* at = &codes[b][TR * kStepBytes + r * AB];
      if constexpr (AB == 64) {
        raw_a[i][0] = *reinterpret_cast<const u32x4*>(at + 16 * placed<64>(r, q));
      } else {
        raw_a[i][0] = *reinterpret_cast<const u32x4*>(at + 16 * placed<128>(r, K == KM8 ? q : 2 * q));
        raw_a[i][1] = *reinterpret_cast<const u32x4*>(at + 16 * placed<128>(r, K == KM8 ? 4 + q : 2 * q + 1));
      }
      sa[i] = block_scale(b, TR + r);
    }
    if (s + 1 < s1) {
      fetch_scales(s + 1);
      fetch(s + 1, b ^ 1);
    }
    if (s == steps - 1 && left < kStep)
#pragma unroll
      for (int i = 0; i < FT; ++i) cut_tail<K, true>(raw_a[i], left);
    Operand<K, true> a[FT];
#pragma unroll
    for (int i = 0; i < FT; ++i) make_operand<K, true>(raw_a[i], sa[i], a[i]);
#pragma unroll
    for (int i = 0; i < FR; ++i) {
      Operand<K, false> w;
      make_operand<K, false>(&raw_w[i], sw[i], w);
      if constexpr (ENDS) {
#pragma unroll
        for (int j = 0; j < FT; ++j) whole[i][j] = whole_sum<1>(w, a[j], whole[i][j]);
      } else if constexpr (kWhole<K>) {
#pragma unroll 1
        for (int part = 0; part < SUB; ++part) {
          const uint32_t* sc = &scales[b][part * (TR + TT)];
          const f32x4 ws = *reinterpret_cast<const f32x4*>(sc + 16 * (FR * wr + i) + 4 * q);
#pragma unroll
          for (int j = 0; j < FT; ++j) {
            const i32x4 d = whole_sum<SUB>(w, a[j], i32x4{0, 0, 0, 0}, part);
            const float as = __uint_as_float(sc[TR + 16 * (FT * wt + j) + m]);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][j][k] = __builtin_fmaf((float)d[k], ws[k] * as, acc[i][j][k]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = step_sum<K, false, true>(w, a[j], acc[i][j]);
      }
    }
    if (s + 1 < s1) put_scales(b ^ 1);
  }

  float unit = 1.0f;
  if constexpr (kWhole<K>) unit = kWholeUnit<K>;
  if constexpr (K == KNV) unit = p.a.tensor[0] * p.w.tensor[span.expert];
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int64_t t = tok0 + 16 * (FT * wt + j) + m;
    if (t >= span.end) continue;
    const int64_t a_row = row_of(p, t);
    float as = unit;
    if constexpr (ENDS) as *= row_scale(p.a, a_row < 0 ? 0 : a_row);
#pragma unroll
    for (int i = 0; i < FR; ++i) {
      const int64_t r = row0 + 16 * (FR * wr + i) + 4 * q;
      if (r >= p.rows) continue;
      f32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (ENDS) v[k] = (float)whole[i][j][k] * as * row_scale(p.w, expert_row + (r + k < p.rows ? r + k : p.rows - 1));
        else v[k] = acc[i][j][k] * as;
        if (a_row < 0) v[k] = 0.0f;
      }
      if (p.k_splits == 1) {
        store_four(p, t, r, v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r + k < p.rows) p.partial[((int64_t)blockIdx.y * p.tokens + t) * p.rows + r + k] = v[k];
      }
    }
  }
}

// ---- few tokens: codes straight to registers, k split over a workgroup's waves ---------------------------------------------------

constexpr int kWaves = 8;

// 16 weight rows and up to 16 MT tokens a workgroup.
template <int K, int SUB, int MT>
__global__ __launch_bounds__(64 * kWaves) void stream_kernel(ProductArgs p) {
  constexpr int AB = kActBytes<K>, WORDS = kScaleWords<K, SUB>, AHEAD = 2;
  constexpr bool ENDS = kWhole<K> && SUB == 0;
  __shared__ f32x4 part[kWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, q = lane >> 4;
  Span span;
  if (!find_span(p, blockIdx.y, 16 * MT, span)) return;
  const int64_t row0 = (int64_t)blockIdx.x * 16, expert_row = span.expert * p.rows;
  const int64_t row = expert_row + (row0 + m < p.rows ? row0 + m : p.rows - 1);
  const int steps = (p.n + kStep - 1) / kStep;
  const int left = p.n - (steps - 1) * kStep;
  const uint8_t* w_from = p.w.codes + row * (p.n / 2);
  const uint8_t* a_from[MT];
  int64_t a_row[MT];                     // of this lane's operand row
  int64_t sum_row[ENDS || !kWhole<K> ? 1 : MT][4];   // of its four sums
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t t = span.first + 16 * i + m, r = row_of(p, t < span.end ? t : span.end - 1);
    a_row[i] = r < 0 ? 0 : r;
    a_from[i] = p.a.codes + a_row[i] * (AB == kStep ? p.n : p.n / 2);
    if constexpr (kWhole<K> && !ENDS)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum_row[i][k] = __shfl(a_row[i], 4 * q + k);
  }
  struct Step {
    u32x4 w, a[MT][AB / 64];
    uint32_t ws[WORDS], as[MT][kWhole<K> ? 4 : WORDS];   // INT groups of at least 128: of the lane's row, of its four sums
  };
  auto load = [&](int s, Step& c) {
    const bool end = s == steps - 1;
    const int at = end && 16 * q >= left / 2 ? left / 2 - 16 : 16 * q;
    c.w = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w_from + (int64_t)s * kStepBytes + at));
    if constexpr (!kWhole<K> || SUB == 1) load_scales<K, SUB>(p.w, row, s, c.ws);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint8_t* from = a_from[i] + (int64_t)s * AB;
      if constexpr (AB == 64) {
        c.a[i][0] = *reinterpret_cast<const u32x4*>(from + at);
      } else {
        const int x = K == KM8 ? 16 * q : 32 * q, y = K == KM8 ? 64 + 16 * q : 32 * q + 16;
        c.a[i][0] = *reinterpret_cast<const u32x4*>(from + (end && x >= left ? left - 16 : x));
        c.a[i][1] = *reinterpret_cast<const u32x4*>(from + (end && y >= left ? left - 16 : y));
      }
      if constexpr (!kWhole<K>) {
        load_scales<K, SUB>(p.a, a_row[i], s, c.as[i]);
      } else if constexpr (SUB == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) c.as[i][k] = part_scale<1>(p.a, sum_row[i][k], s, 0);
      }
    }
  };
  f32x4 acc[MT] = {};
  i32x4 whole[MT] = {};
  auto take = [&](int s, Step& c) {
    auto own = [&](const uint32_t (&v)[WORDS]) -> uint32_t {
      if constexpr (K == KNV) return (uint32_t)(((uint64_t)v[1] << 32 | v[0]) >> (16 * q)) & 0xFFFFu;
      else return v[0] >> (8 * q) & 0xFFu;
    };
    Operand<K, false> w;
    uint32_t own_scale = 0;
    if constexpr (!kWhole<K>) own_scale = own(c.ws);
    make_operand<K, false>(&c.w, own_scale, w);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (s == steps - 1 && left < kStep) cut_tail<K, true>(c.a[i], left);
      Operand<K, true> a;
      if constexpr (!kWhole<K>) own_scale = own(c.as[i]);
      make_operand<K, true>(c.a[i], own_scale, a);
      if constexpr (ENDS) {
        whole[i] = whole_sum<1>(a, w, whole[i]);
      } else if constexpr (kWhole<K>) {
#pragma unroll 1
        for (int part = 0; part < SUB; ++part) {
          const i32x4 d = whole_sum<SUB>(a, w, i32x4{0, 0, 0, 0}, part);
          const uint32_t ws = SUB == 1 ? c.ws[0] : part_scale<SUB>(p.w, row, s, part);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t as = SUB == 1 ? c.as[i][k] : part_scale<SUB>(p.a, sum_row[i][k], s, part);
            acc[i][k] = __builtin_fmaf((float)d[k], __uint_as_float(scale_value<K>(p.w, ws)) * __uint_as_float(scale_value<K>(p.a, as)), acc[i][k]);
          }
        }
      } else {
        acc[i] = step_sum<K, true, false>(a, w, acc[i]);
      }
    }
  };
  // waves take steps in turn
  Step c[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int s = wave + k * kWaves;
    load(s < steps ? s : steps - 1, c[k]);
  }
  for (int s = wave; s < steps; s += AHEAD * kWaves) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int at = s + k * kWaves, next = at + AHEAD * kWaves;
      if (at < steps) take(at, c[k]);
      load(next < steps ? next : steps - 1, c[k]);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if constexpr (ENDS) part[wave][i][lane] = __builtin_bit_cast(f32x4, whole[i]);
    else part[wave][i][lane] = acc[i];
  }
  __syncthreads();
  // result u: token 4 q + k of tile i, row m
  const float* sums = reinterpret_cast<const float*>(part);
  for (int u = threadIdx.x; u < MT * 256; u += 64 * kWaves) {
    const int i = u >> 8, k = (u >> 6) & 3;
    const int64_t t = span.first + 16 * i + 4 * q + k;
    if (t >= span.end || row0 + m >= p.rows) continue;
    const int64_t r = row_of(p, t);
    float v = 0.0f;
    if constexpr (ENDS) {
      int total = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total += __float_as_int(sums[((w * MT + i) * 64 + lane) * 4 + k]);
      v = (float)total * kWholeUnit<K> * row_scale(p.a, r < 0 ? 0 : r) * row_scale(p.w, row);
    } else {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += sums[((w * MT + i) * 64 + lane) * 4 + k];
      if constexpr (kWhole<K>) v *= kWholeUnit<K>;
      if constexpr (K == KNV) v *= p.a.tensor[0] * p.w.tensor[span.expert];
    }
    store_one(p, t, row0 + m, r < 0 ? 0.0f : v);
  }
}

__global__ __launch_bounds__(256) void join_kernel(ProductArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, all = p.tokens * p.rows;
  if (i >= all) return;
  float v = 0.0f;
  for (int k = 0; k < p.k_splits; ++k) v += p.partial[k * all + i];
  store_one(p, i / p.rows, i % p.rows, v);
}

// ---- which kernel -------------------------------------------------------------------------------------------------------------

enum Form { STREAM16, STREAM32, STREAM64, TILE128, TILE256 };

Form form_of(int64_t tokens, int64_t rows, int32_t experts) {
  const int64_t each = (tokens + experts - 1) / experts;           // of an expert, on average
  if (each <= 16) return STREAM16;
  if (each <= 32) return STREAM32;
  if (each <= 64) return STREAM64;
  const int64_t large = ((rows + 255) / 256) * ((tokens + 255) / 256);
  return each >= 256 && large >= 256 ? TILE256 : TILE128;
}

// Tiles of `size` rows of y: whole ones, and the rest of every expert that has any.
int64_t slots_of(const ProductArgs& p, int size) {
  if (!p.starts) return (p.tokens + size - 1) / size;
  return p.tokens / size + (p.experts < p.tokens ? p.experts : p.tokens);
}

template <int K, int SUB, int MT>
void go_stream(const ProductArgs& p, hipStream_t s) {
  hipLaunchKernelGGL((stream_kernel<K, SUB, MT>), dim3((unsigned)((p.rows + 15) / 16), (unsigned)slots_of(p, 16 * MT)), dim3(64 * kWaves), 0, s, p);
}

template <int K, int SUB, int FR, int FT, int WR, int WT>
void go_tiles(const ProductArgs& p, hipStream_t s) {
  const int row_tiles = (int)((p.rows + 16 * FR * WR - 1) / (16 * FR * WR)), token_tiles = (int)slots_of(p, 16 * FT * WT);
  hipLaunchKernelGGL((tile_kernel<K, SUB, FR, FT, WR, WT>), dim3((unsigned)((int64_t)row_tiles * token_tiles), (unsigned)p.k_splits),
                     dim3(64 * WR * WT), 0, s, p, row_tiles, token_tiles);
  if (p.k_splits > 1)
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)((p.tokens * p.rows + 255) / 256)), dim3(256), 0, s, p);
}

template <int K, int SUB>
hipError_t go(const ProductArgs& p, hipStream_t s) {
  switch (form_of(p.tokens, p.rows, p.experts)) {
    case STREAM16: go_stream<K, SUB, 1>(p, s); break;
    case STREAM32: go_stream<K, SUB, 2>(p, s); break;
    case STREAM64: go_stream<K, SUB, 4>(p, s); break;
    case TILE128: go_tiles<K, SUB, 4, 4, 2, 2>(p, s); break;
    case TILE256:
      if constexpr (SUB < 2) go_tiles<K, SUB, 8, 4, 2, 4>(p, s);
      else go_tiles<K, SUB, 4, 4, 2, 2>(p, s);
      break;
  }
  return hipGetLastError();
}

template <int K>
hipError_t go_whole(const ProductArgs& p, hipStream_t s) {
  const int a = p.a.group_log, w = p.w.group_log;
  if (a < 0 && w < 0 && p.n <= kMostWholeSum) return go<K, 0>(p, s);
  const int least = a < 0 ? w : (w < 0 || a < w ? a : w);
  if (least < 0 || least >= 7) return go<K, 1>(p, s);
  if (least == 6) return go<K, 2>(p, s);
  return least == 5 ? go<K, 4>(p, s) : go<K, 8>(p, s);
}

}  // namespace

int32_t product_splits(int64_t tokens, int32_t n, int64_t rows, int32_t experts, int a_fmt) {
  return 1;
}

hipError_t launch_product(int a_fmt, const ProductArgs& p, hipStream_t s) {
  switch (a_fmt) {
    case RHTQ_FMT_INT4: return go_whole<KI4>(p, s);
    case RHTQ_FMT_INT8: return go_whole<KI8>(p, s);
    case RHTQ_FMT_NVFP4: return go<KNV, 1>(p, s);
    case RHTQ_FMT_MXFP4: return go<KM4, 1>(p, s);
    default: return go<KM8, 1>(p, s);
  }
}

}  // namespace rhtq
