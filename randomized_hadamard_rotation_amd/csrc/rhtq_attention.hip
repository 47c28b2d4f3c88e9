// Attention of one new token per sequence over the paged 4-bit cache, split over the length and joined.
//
//   o = R_v^T sum_j p_j s^v_j c^v_j / sum_j p_j,   p_j = exp(x_j - max x),   x_j = scale * s^k_j (R_k q) . c^k_j
//
// The rotation is orthonormal, so q is rotated once, the codes are used as they lie, and the sum is rotated back once.
// The bytes of the codes and scales bound it, so nothing else may take long:
//  - Both products run on the int8 matrix cores on the codes themselves, 16 c as a byte (a mask, or a shift and a mask, for four
//    codes), exactly.  q and the weights p_j s^v_j go in as two bytes, v = 256 hi + lo, of a 16-bit fixed point relative to the largest of
//    their row: q over its head, the weights over a chunk of 64 positions.
//  - S^T = K Q^T has positions as rows and, as its 16 columns, 8 query heads of one key-value head in hi and in lo bytes: lane (n, g) gets
//    positions 4 g + i of each tile for column n, so after the softmax it holds the 16 weights that it supplies as an operand of
//    O^T = V^T P^T, and nothing moves between lanes but the two halves of a score (a DPP rotation by 8) and two maxima a chunk.
//  - A lane loads one dword (at head_dim 128) of 16 rows of V; 4 x 4 byte transposes in registers make operands of four positions.
//  - One pass: each wave keeps the running maximum m, sum l and the weighted sum o in fp32.  Parts (m, l, o) of waves and of
//    splits join as m = max m_i, l = sum l_i 2^(m_i - m), o likewise, in a fixed order.
// Scores are in units of log2, so a weight is one v_exp_f32.
#include "rhtq_internal.h"
#include "rhtq_serving_device.h"
#include "rhtq_serving_internal.h"

namespace rhtq {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;
constexpr int kWaves = kThreads / 64;
constexpr int kHeads = 8;               // query heads of a tile
constexpr int kChunk = 4;               // tiles that a wave takes at once: 64 positions, the depth of one product
constexpr int kLeastTiles = kWaves * kChunk;   // tiles of a part worth a workgroup
constexpr float kNone = -INFINITY;
constexpr float kLargest = 32639.0f;    // 127 * 256 + 127: the largest two-byte value

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Undo the rotation of one head's sum (E values a lane) and store it.
template <int T, int E>
__device__ __forceinline__ void finish(const AttentionArgs& a, int64_t row, float l, float (&o)[E]) {
  const int j = threadIdx.x & 15;
  const float cnorm = E == 4 ? 0.125f : (E == 8 ? 0.088388347648318447f : 0.0625f);
  const float f = l > 0.0f ? cnorm / l : 0.0f;
  fwht16<E>(o);
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] *= f;
  apply_signs<E>(a.v_signs, j * E, o);
  store_row<T, E>(a.out, row * (16 * E) + j * E, o);
}

// Largest of the four lanes 16 apart.
__device__ __forceinline__ float max_over_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

// What a wave has loaded of a chunk.
template <int D>
struct Loaded {
  u32x4 k[kChunk][D >= 128 ? D / 128 : 1];      // D 64: two dwords used
  uint32_t v[kChunk][4][D >= 128 ? D / 128 : 1];
  uint32_t ks[kChunk][4], vs[kChunk][4];        // raw scales: four fp32, or four fp16 in two words
  int pos[kChunk];                              // first position of the tile, -1: none
};

template <int D, bool F32>
__device__ __forceinline__ void load_chunk(const AttentionArgs& a, const Visible& vis, const int32_t* table, int kv, int first,
                                           int end, Loaded<D>& c) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < kChunk; ++t) {
    const int pos = first + t < end ? tile_at(vis, first + t) * kTile : -1;
    const int page = pos >= 0 ? page_at(table, a.width, a.pages, pos >> a.page_log) : -1;
    c.pos[t] = page >= 0 ? pos : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.vs[t][i] = c.ks[t][i] = 0;
    if (page < 0) {
#pragma unroll
      for (int h = 0; h < (D >= 128 ? D / 128 : 1); ++h) {
        c.k[t][h] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) c.v[t][i][h] = 0;
      }
      continue;
    }
    const int64_t slot = (((int64_t)page * a.kv_heads + kv) << a.page_log) + (pos & ((1 << a.page_log) - 1));
    const uint8_t* k = a.k_codes + slot * (D / 2) + n * (D / 2);
    if constexpr (D == 64) {
      const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(k + 8 * g));
      c.k[t][0] = u32x4{w.x, w.y, 0, 0};
    } else {
#pragma unroll
      for (int h = 0; h < D / 128; ++h)
        c.k[t][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(k + 64 * h + 16 * g));
    }
    const uint8_t* v = a.v_codes + slot * (D / 2) + 4 * g * (D / 2) + n * (D / 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (D == 64) c.v[t][i][0] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(v + i * (D / 2)));
      else if constexpr (D == 128) c.v[t][i][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(v + i * (D / 2)));
      else {
        const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(v + i * (D / 2)));
        c.v[t][i][0] = w.x;
        c.v[t][i][1] = w.y;
      }
    }
    if constexpr (F32) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(static_cast<const float*>(a.k_scales) + slot + 4 * g);
      const u32x4 y = *reinterpret_cast<const u32x4*>(static_cast<const float*>(a.v_scales) + slot + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c.ks[t][i] = x[i];
        c.vs[t][i] = y[i];
      }
    } else {
      const u32x2 x = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.k_scales) + slot + 4 * g);
      const u32x2 y = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.v_scales) + slot + 4 * g);
      c.ks[t][0] = x.x;
      c.ks[t][1] = x.y;
      c.vs[t][0] = y.x;
      c.vs[t][1] = y.y;
    }
  }
}

template <bool F32>
__device__ __forceinline__ float scale_of(const uint32_t (&s)[4], int i) {
  if constexpr (F32) return __uint_as_float(s[i]);
  else return __half2float(__ushort_as_half((uint16_t)(s[i >> 1] >> (16 * (i & 1)))));
}

// Even codes of four bytes as 16 c in each byte, and odd ones.
__device__ __forceinline__ int even_codes(uint32_t w) { return (int)((w << 4) & 0xF0F0F0F0u); }
__device__ __forceinline__ int odd_codes(uint32_t w) { return (int)(w & 0xF0F0F0F0u); }

// Byte of an operand row's element d: the codes of a lane's 16 bytes (8 at D = 64) go in as evens, then odds.
template <int D>
__device__ __forceinline__ int operand_byte(int d) {
  if constexpr (D == 64) return (d >> 4) * 16 + (d & 1) * 8 + ((d & 15) >> 1);
  else return ((2 * (d >> 7) + (d & 1)) * 4 + ((d & 127) >> 5)) * 16 + ((d & 31) >> 1);
}

// One workgroup: a part of one sequence's positions for up to 8 query heads of one key-value head; its waves take the chunks
// in turn.
template <int T, int E, bool F32>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttentionArgs a) {
  constexpr int D = 16 * E;
  constexpr int NK = D / 64;              // products of a score
  constexpr int H = D >= 128 ? D / 128 : 1;
  __shared__ __attribute__((aligned(16))) uint8_t sq[16][D];
  __shared__ float sf[kHeads];
  __shared__ float sm[kWaves][kHeads], sl[kWaves][kHeads];
  __shared__ float so[kWaves][kHeads][D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, g = lane >> 4;
  const int group = threadIdx.x >> 4, j = threadIdx.x & 15;
  int64_t b = blockIdx.x;
  const int split = (int)(b % a.splits);
  b /= a.splits;
  const int head0 = (int)(b % a.head_tiles) * kHeads;
  b /= a.head_tiles;
  const int kv = (int)(b % a.kv_heads), s = (int)(b / a.kv_heads);
  const int heads = a.each - head0 < kHeads ? a.each - head0 : kHeads;
  const Visible vis = visible_of(a.lengths[s], a.width, 1 << a.page_log, a.window, a.sinks);
  const int per = tiles_per_split(vis.tiles, a.splits, kLeastTiles);
  const int t0 = split * per, t1 = t0 + per < vis.tiles ? t0 + per : vis.tiles;
  const int32_t* table = a.table + (int64_t)s * a.width;
  const int64_t row0 = (int64_t)s * a.q_heads + kv * a.each + head0;   // of [seqs][q_heads]

  Loaded<D> c;
  int at = t0 + wave * kChunk;
  if (at < t1) load_chunk<D, F32>(a, vis, table, kv, at, t1, c);

  // q: 16 lanes rotate a head and leave its bytes as operand rows h (hi) and 8 + h (lo)
  if (group < kHeads) {
    float q[E] = {};
    if (group < heads) {
      load_row<T, E>(a.q, s * a.q_seq_stride + (kv * a.each + head0 + group) * a.q_head_stride + j * E, q);
      apply_signs<E>(a.k_signs, j * E, q);
      fwht16<E>(q);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) amax = fmaxf(amax, __builtin_fabsf(q[i]));
    amax = max16(amax);
    const float inv = amax > 0.0f ? kLargest / amax : 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int v = (int)__builtin_rintf(q[i] * inv);
      sq[group][operand_byte<D>(j * E + i)] = (uint8_t)((v + 128) >> 8);
      sq[8 + group][operand_byte<D>(j * E + i)] = (uint8_t)v;
    }
    // what a product of 16 c and the fixed point counts for in a score, log2
    const float cnorm = E == 4 ? 0.125f : (E == 8 ? 0.088388347648318447f : 0.0625f);
    if (j == 0) sf[group] = amax / (16.0f * kLargest) * (cnorm * 1.4426950408889634f) * a.scale;
  }
  __syncthreads();
  i32x4 q[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) q[i] = *reinterpret_cast<const i32x4*>(&sq[n][(4 * i + g) * 16]);
  const float factor = sf[n & 7];
  const int w_own = n < 8 ? 256 : 1, w_other = n < 8 ? 1 : 256;
  // the weights' bytes: 1.5 * 2^23 in front makes the sum's low bits the whole number; hi is its second byte after + 128
  const float magic = 12582912.0f + (n < 8 ? 128.0f : 0.0f);
  const uint32_t pick = n < 8 ? 0x0C0C0501u : 0x0C0C0400u;

  float m = kNone, l = 0.0f;
  float o[E][4] = {};                     // element E (4 g + i) + e of column n
  while (at < t1) {
    float x[kChunk][4], top = kNone;
#pragma unroll
    for (int t = 0; t < kChunk; ++t) {
      i32x4 d = {0, 0, 0, 0};
      if constexpr (D == 64) {
        const i32x4 k = {even_codes(c.k[t][0].x), even_codes(c.k[t][0].y), odd_codes(c.k[t][0].x), odd_codes(c.k[t][0].y)};
        d = __builtin_amdgcn_mfma_i32_16x16x64_i8(k, q[0], d, 0, 0, 0);
      } else {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const u32x4 w = c.k[t][h];
          const i32x4 k0 = {even_codes(w.x), even_codes(w.y), even_codes(w.z), even_codes(w.w)};
          const i32x4 k1 = {odd_codes(w.x), odd_codes(w.y), odd_codes(w.z), odd_codes(w.w)};
          d = __builtin_amdgcn_mfma_i32_16x16x64_i8(k0, q[2 * h], d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_i32_16x16x64_i8(k1, q[2 * h + 1], d, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = __mul24(d[i], w_own) + __mul24(lane_xor16<3>(d[i]), w_other);
        x[t][i] = (float)v * (scale_of<F32>(c.ks[t], i) * factor);
      }
      const int pos = c.pos[t];
      if (pos < 0 || pos + kTile > vis.len || (pos < vis.start && pos + kTile > vis.sinks)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (pos < 0 || !is_visible(vis, pos + 4 * g + i)) x[t][i] = kNone;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, x[t][i]);
    }
    const float mn = fmaxf(m, max_over_groups(top));
    const float base = mn == kNone ? 0.0f : mn;
    const float fade = m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - base);
    m = mn;
    l *= fade;
    top = 0.0f;
    {
      // a score is one rounded number wherever it is used: contracted into x - base it could exceed its own maximum
#pragma clang fp contract(off)
#pragma unroll
      for (int t = 0; t < kChunk; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(x[t][i] - base);
          l += p;
          // what lies behind the last position may hold anything: it has weight 0 whatever its scale
          x[t][i] = x[t][i] == kNone ? 0.0f : p * scale_of<F32>(c.vs[t], i);
          top = fmaxf(top, x[t][i]);
        }
    }
    top = max_over_groups(top);
    const float unit = top > 0.0f ? kLargest / top : 0.0f;
    i32x4 p;
#pragma unroll
    for (int t = 0; t < kChunk; ++t) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(__builtin_fmaf(x[t][i], unit, magic));
      const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], pick), hi = __builtin_amdgcn_perm(w[3], w[2], pick);
      p[t] = (int)__builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
    const float back = top * (1.0f / (16.0f * kLargest)) * (float)w_own;
    // V: byte r of the four rows of a lane's tile, transposed; its low nibbles are element 2 r, its high ones 2 r + 1
    constexpr int R = D / 32;              // bytes of a row that a lane holds
    uint32_t col[R][kChunk];
#pragma unroll
    for (int t = 0; t < kChunk; ++t)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint32_t w0 = c.v[t][0][h], w1 = c.v[t][1][h], w2 = c.v[t][2][h], w3 = c.v[t][3][h];
        const uint32_t x0 = __builtin_amdgcn_perm(w1, w0, 0x05010400u), y0 = __builtin_amdgcn_perm(w3, w2, 0x05010400u);
        col[4 * h][t] = __builtin_amdgcn_perm(y0, x0, 0x05040100u);
        col[4 * h + 1][t] = __builtin_amdgcn_perm(y0, x0, 0x07060302u);
        if constexpr (D >= 128) {
          const uint32_t x1 = __builtin_amdgcn_perm(w1, w0, 0x07030602u), y1 = __builtin_amdgcn_perm(w3, w2, 0x07030602u);
          col[4 * h + 2][t] = __builtin_amdgcn_perm(y1, x1, 0x05040100u);
          col[4 * h + 3][t] = __builtin_amdgcn_perm(y1, x1, 0x07060302u);
        }
      }
    at += kWaves * kChunk;
    if (at < t1) load_chunk<D, F32>(a, vis, table, kv, at, t1, c);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        i32x4 v, d = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < kChunk; ++t) v[t] = odd ? odd_codes(col[r][t]) : even_codes(col[r][t]);
        d = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, p, d, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[2 * r + odd][i] = __builtin_fmaf((float)d[i], back, o[2 * r + odd][i] * fade);
      }
  }
  // both halves of a column's sum; l over the lanes that share it
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = o[e][i] + lane_xor16<3>(o[e][i]);
      if (n < kHeads) so[wave][n][E * (4 * g + i) + e] = v;
    }
  if (lane < kHeads) {
    sm[wave][lane] = m;
    sl[wave][lane] = l;
  }
  __syncthreads();
  if (group >= heads) return;
  m = kNone;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) m = fmaxf(m, sm[k][group]);
  l = 0.0f;
  float r[E] = {};
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    const float f = sm[k][group] == kNone ? 0.0f : __builtin_amdgcn_exp2f(sm[k][group] - m);
    l += sl[k][group] * f;
#pragma unroll
    for (int i = 0; i < E; ++i) r[i] = __builtin_fmaf(f, so[k][group][j * E + i], r[i]);
  }
  const int64_t row = row0 + group;
  if (a.splits == 1) {
    finish<T, E>(a, row, l, r);
    return;
  }
  float* part = a.partial + (row * a.splits + split) * D;
  store_row<RHTQ_IN_F32, E>(part, j * E, r);
  if (j == 0) {
    float* ml = a.partial + (int64_t)a.seqs * a.q_heads * a.splits * D + 2 * (row * a.splits + split);
    ml[0] = m;
    ml[1] = l;
  }
}

template <int T, int E>
__global__ __launch_bounds__(kThreads) void join_kernel(AttentionArgs a) {
  constexpr int D = 16 * E;
  const int j = threadIdx.x & 15;
  const int64_t row = (int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4);
  if (row >= (int64_t)a.seqs * a.q_heads) return;
  const float* ml = a.partial + (int64_t)a.seqs * a.q_heads * a.splits * D + 2 * row * a.splits;
  const float* part = a.partial + row * a.splits * D;
  float m = kNone;
  for (int k = 0; k < a.splits; ++k) m = fmaxf(m, ml[2 * k]);
  float l = 0.0f, o[E] = {};
  for (int k = 0; k < a.splits; ++k) {
    if (ml[2 * k] == kNone) continue;
    const float f = __builtin_amdgcn_exp2f(ml[2 * k] - m);
    l += ml[2 * k + 1] * f;
    float v[E];
    load_row<RHTQ_IN_F32, E>(part, (int64_t)k * D + j * E, v);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = __builtin_fmaf(f, v[i], o[i]);
  }
  finish<T, E>(a, row, l, o);
}

template <int T, int E>
hipError_t launch_te(const AttentionArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.seqs * a.kv_heads * a.head_tiles * a.splits));
  if (a.scale_dtype == RHTQ_SCALE_F32) hipLaunchKernelGGL((attention_kernel<T, E, true>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((attention_kernel<T, E, false>), grid, dim3(kThreads), 0, s, a);
  const int64_t rows = (int64_t)a.seqs * a.q_heads;
  if (a.splits > 1)
    hipLaunchKernelGGL((join_kernel<T, E>), dim3((unsigned)((rows + kGroups - 1) / kGroups)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int T>
hipError_t launch_t(const AttentionArgs& a, hipStream_t s) {
  switch (a.head_dim) {
    case 64: return launch_te<T, 4>(a, s);
    case 128: return launch_te<T, 8>(a, s);
    default: return launch_te<T, 16>(a, s);
  }
}

}  // namespace

int32_t attention_head_tiles(int32_t each) { return (each + kHeads - 1) / kHeads; }

int32_t attention_splits(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t width, int32_t page, int32_t window,
                         int32_t sinks) {
  int64_t tiles = (int64_t)width * page / kTile;
  if (window > 0) {
    const int64_t most = (int64_t)window / kTile + 2 + ((int64_t)sinks + kTile - 1) / kTile;
    if (most < tiles) tiles = most;
  }
  const int64_t rows = (int64_t)seqs * kv_heads * attention_head_tiles(q_heads / kv_heads);
  int64_t want = (2048 + rows - 1) / (rows > 0 ? rows : 1);
  const int64_t most = (tiles + kLeastTiles - 1) / kLeastTiles;
  if (want > most) want = most;
  if (want > 1024) want = 1024;
  return want < 1 ? 1 : (int32_t)want;
}

hipError_t launch_paged_attention(int dtype, const AttentionArgs& a, hipStream_t s) {
  if (dtype == RHTQ_IN_BF16) return launch_t<RHTQ_IN_BF16>(a, s);
  return launch_t<RHTQ_IN_F16>(a, s);
}

}  // namespace rhtq
