// Attention of one new token per sequence over the paged 4-bit cache, split over the length and joined.
//
//   o = R_v^T sum_j p_j s^v_j c^v_j / sum_j p_j,   p_j = exp(x_j - max x),   x_j = scale * s^k_j (R_k q) . c^k_j
//
// The rotation is orthonormal, so q is rotated once, the codes are used as they lie, and the sum is rotated back once.
// The bytes of the codes and scales bound it, so nothing else may take long:
//  - Both products run on the int8 matrix cores on the codes themselves, 16 c as a byte (a mask, or a shift and a mask, for four
//    codes), exactly.  q and the weights p_j s^v_j go in as three signed bytes, v = 65536 a + 256 b + c, whole numbers of up to 2^22 for
//    the power of two above the largest of their row (q over its head, the weights over a chunk of 64 positions): off by at most 2^-22 of it.
//  - S^T = K Q^T has positions as rows and query heads of one key-value head as its 16 columns; lane (n, g) gets positions 4 g + i of each
//    tile for column n.  Up to 4 heads: column 4 h + r is head h's byte r (0: c, 1: b, 2: a, 3: nothing).  The four lanes of a head add up
//    65536 a + 256 b + c as they divide the positions among them, one each, and turn the finished weights' bytes (a 4 x 4 transposition by
//    DPP moves and byte permutes) into the operand of O^T = V^T P^T.  5 to 8 heads: columns h and 8 + h are bytes a and b, and a second
//    product adds c to the upper ones, as 256 b + c.  Lanes n and n + 8 swap halves, finish two positions each and swap the bytes back.
//  - A lane loads one dword (at head_dim 128) of 16 rows of V; 4 x 4 byte transposes in registers make operands of four positions.
//  - One pass: each wave keeps the running maximum m, sum l and the weighted sum o in fp32.  Parts (m, l, o) of waves and of
//    splits join as m = max m_i, l = sum l_i 2^(m_i - m), o likewise, in a fixed order.
// Scores are in units of log2, so a weight is one v_exp_f32.
//
// Two bytes (16 bits) of q and of the weights took the same time with up to 4 heads and 29.7 us where 64 / 8 heads x 4096 positions now take
// 31.7, but one fp16 output in 5 was then another number than the rounded result, for 1 in 200 now.
// Measured: 32 x 32 heads x 4096 positions 98 us (554 MB, 5.6 TB/s; a sum reads 5.7); one sequence of 131072 with 8 key-value heads 27 us
// and 4 us to join (4.3 TB/s); 515 positions of 32 heads 7.8 us, a chain of length, table, codes and the end's exchange.
#include <type_traits>

#include "rhtq_internal.h"
#include "rhtq_serving_device.h"
#include "rhtq_serving_internal.h"

namespace rhtq {
namespace {

constexpr int kWaves = 8;
constexpr int kJoinWaves = 4;           // heads of a join's workgroup
constexpr int kHeads = 8;               // most query heads of a tile
constexpr int kChunk = 4;               // tiles that a wave takes at once: 64 positions, the depth of one product
constexpr int kLeastTiles = kWaves * kChunk;   // tiles of a part worth a workgroup: 512 positions
constexpr int kMostTiles = 320;         // and at most, where the whole is enough for the chip: 5120 positions
constexpr int kEnough = 256;            // workgroups that fill the chip: one of 8 waves on each CU
constexpr float kNone = -INFINITY;
constexpr int kBits = 22;               // of q and the weights as whole numbers

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Undo the rotation of one head's sum (E values a lane) and store it.
template <int T, int E>
__device__ __forceinline__ void finish(const AttentionArgs& a, int64_t row, float l, float (&o)[E]) {
  const int j = threadIdx.x & 15;
  const float cnorm = E == 4 ? 0.125f : (E == 8 ? 0.088388347648318447f : 0.0625f);
  const float f = l == 0.0f ? 0.0f : cnorm * __builtin_amdgcn_rcpf(l);   // NaN where l is
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] *= f;   // before the transform, whose sums could overflow without it
  fwht16<E>(o);
  apply_signs<E>(a.v_signs, j * E, o);
  store_row<T, E>(a.out, row * (16 * E) + j * E, o);
}

// Values of lanes 16 and 32 apart side by side: v_permlane16_swap / v_permlane32_swap of a register with itself leave the even rows' (the
// lower half's) values in one result and the odd rows' (the upper half's) in the other.
__device__ __forceinline__ float max_over_groups(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
}

// Over the lanes of a row of 16 that share a query head: 4 neighbours, or two 8 apart.
template <int HT>
__device__ __forceinline__ float add_over_columns(float v) {
  if constexpr (HT == 4) {
    v += lane_xor16<0>(v);
    return v + lane_xor16<1>(v);
  } else {
    return v + lane_xor16<3>(v);
  }
}

// Largest over all lanes that share a query head: these, and those 16 and 32 apart.
template <int HT>
__device__ __forceinline__ float max_over_head(float v) {
  if constexpr (HT == 4) {
    v = fmaxf(v, lane_xor16<0>(v));
    v = fmaxf(v, lane_xor16<1>(v));
  } else {
    v = fmaxf(v, lane_xor16<3>(v));
  }
  return max_over_groups(v);
}

// Where a chunk's tiles lie: first position (-1: none) and page.  The same in all lanes.
struct Place {
  int pos[kChunk];
  int page[kChunk];
};

// `first` is the same in all lanes, so the table's entries come by scalar loads, which no wait for the codes holds up.
__device__ __forceinline__ void locate(const AttentionArgs& a, const Visible& vis, const int32_t* table, int first, int end, Place& c) {
  int entry[kChunk], at[kChunk];
#pragma unroll
  for (int t = 0; t < kChunk; ++t) {
    at[t] = first + t < end ? tile_at(vis, first + t) * kTile : 0;   // in the table, whose width is at least 1
    entry[t] = load_uniform(table + (at[t] >> a.page_log));
  }
#pragma unroll
  for (int t = 0; t < kChunk; ++t) {
    const bool there = first + t < end && (uint32_t)entry[t] < (uint32_t)a.pages;
    c.page[t] = there ? entry[t] : 0;
    c.pos[t] = there ? at[t] : -1;
  }
}

// What a wave has loaded of a chunk.  PER: positions of a tile that a lane finishes, whose scales it has.
template <int D, bool F32, int PER>
struct Loaded {
  static constexpr int H = D >= 128 ? D / 128 : 1;
  u32x4 k[kChunk][H];                           // D 64: two dwords used
  uint32_t v[kChunk][4][H];
  uint32_t ks[kChunk][F32 ? PER : 1], vs[kChunk][F32 ? PER : 1];   // its scales: fp32, or one or two fp16 in a word
};

// First slot of a tile, counted in rows.  A tile of no page takes page 0, which its weights of 0 make harmless, so that its loads need no
// branch.
__device__ __forceinline__ int64_t slot_of(const AttentionArgs& a, int kv, const Place& at, int t) {
  const int pos = at.pos[t];
  return (((int64_t)at.page[t] * a.kv_heads + kv) << a.page_log) + (pos >= 0 ? pos & ((1 << a.page_log) - 1) : 0);
}

template <bool F32, int PER, int N>
__device__ __forceinline__ void load_scales(const void* p, int64_t slot, uint32_t (&s)[N]) {
  if constexpr (F32) {
    const float* q = static_cast<const float*>(p) + slot;
    if constexpr (PER == 2) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(q);
      s[0] = x.x;
      s[1] = x.y;
    } else {
      s[0] = *reinterpret_cast<const uint32_t*>(q);
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + slot;
    if constexpr (PER == 2) s[0] = *reinterpret_cast<const uint32_t*>(q);
    else s[0] = *q;
  }
}

// First of the PER positions of a tile that lane (n, g) finishes.
template <int PER>
__device__ __forceinline__ int own_position(int n, int g) {
  return PER == 1 ? 4 * g + (n & 3) : 4 * g + 2 * (n >> 3);
}

template <int D, bool F32, int PER>
__device__ __forceinline__ void load_keys(const AttentionArgs& a, int kv, const Place& at, Loaded<D, F32, PER>& c) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < kChunk; ++t) {
    const int64_t slot = slot_of(a, kv, at, t);
    const uint8_t* k = a.k_codes + slot * (D / 2) + n * (D / 2);
    if constexpr (D == 64) {
      const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(k + 8 * g));
      c.k[t][0] = u32x4{w.x, w.y, 0, 0};
    } else {
#pragma unroll
      for (int h = 0; h < D / 128; ++h)
        c.k[t][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(k + 64 * h + 16 * g));
    }
    load_scales<F32, PER>(a.k_scales, slot + own_position<PER>(n, g), c.ks[t]);
  }
}

template <int D, bool F32, int PER>
__device__ __forceinline__ void load_values(const AttentionArgs& a, int kv, const Place& at, Loaded<D, F32, PER>& c) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < kChunk; ++t) {
    const int64_t slot = slot_of(a, kv, at, t);
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
    load_scales<F32, PER>(a.v_scales, slot + own_position<PER>(n, g), c.vs[t]);
  }
}

template <bool F32, int N>
__device__ __forceinline__ float scale_of(const uint32_t (&s)[N], int i) {
  if constexpr (F32) return __uint_as_float(s[i]);
  else return __half2float(__ushort_as_half((uint16_t)(s[0] >> (16 * i))));
}

// a where the lane's mask is all ones, b where it is 0: one v_bfi_b32.
__device__ __forceinline__ int select(int mask, int a, int b) { return (a & mask) | (b & ~mask); }

// Even codes of four bytes as 16 c in each byte, and odd ones.
__device__ __forceinline__ int even_codes(uint32_t w) { return (int)((w << 4) & 0xF0F0F0F0u); }
__device__ __forceinline__ int odd_codes(uint32_t w) { return (int)(w & 0xF0F0F0F0u); }

// Byte of an operand row's element d: the codes of a lane's 16 bytes (8 at D = 64) go in as evens, then odds.
template <int D>
__device__ __forceinline__ int operand_byte(int d) {
  if constexpr (D == 64) return (d >> 4) * 16 + (d & 1) * 8 + ((d & 15) >> 1);
  else return ((2 * (d >> 7) + (d & 1)) * 4 + ((d & 127) >> 5)) * 16 + ((d & 31) >> 1);
}

// Waves a SIMD; a workgroup is two.  Four against three: 32 x 32 heads x 4096 positions 96 us against 106 (fp32 scales 98 against 106);
// 48 x 8 heads, ragged, with a window 22.6 against 20.4 (both types of scales); 64 / 8 heads, where four spill, 36.6 against 31.4.  So 8
// heads take three; of up to 4, fp16 scales take four for the batch, fp32 ones three for the ragged lengths.  head_dim 256 needs the
// registers of two.
constexpr int waves_of(int E, bool F32, int HT) { return E == 16 ? 2 : (F32 || HT == 8 ? 3 : 4); }

// One workgroup: a part of one sequence's positions for up to HT = 4 or 8 query heads of one key-value head; its waves take the chunks
// in turn.
template <int T, int E, bool F32, int HT>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(waves_of(E, F32, HT), waves_of(E, F32, HT))))
void attention_kernel(AttentionArgs a) {
  constexpr int PER = HT == 8 ? 2 : 1;    // positions of a tile that a lane finishes
  constexpr int D = 16 * E;
  constexpr int NK = D / 64;              // products of a score
  constexpr int H = D >= 128 ? D / 128 : 1;
  __shared__ __attribute__((aligned(16))) uint8_t sq[3 * HT + 1][D];   // bytes a, b, c of each head, and zeros
  __shared__ float sf[HT];
  __shared__ float sm[kWaves][HT], sl[kWaves][HT];
  __shared__ __attribute__((aligned(16))) float so[kWaves][HT][D + 4];   // + 4: columns start in other banks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int group = threadIdx.x >> 4, j = threadIdx.x & 15;
  const int split = blockIdx.x, s = blockIdx.z;
  const int kv = blockIdx.y / a.head_tiles, head0 = (blockIdx.y - kv * a.head_tiles) * HT;
  const int heads = a.each - head0 < HT ? a.each - head0 : HT;
  // loads in the order of their use: q's rotation then runs while the first chunk's codes are on their way
  const int length = load_uniform(a.lengths + s);
  uint32_t signs[E / 4];
  float x0[E] = {};
  load_signs<E>(a.k_signs, j * E, signs);
  const int from = group < heads ? group : heads - 1;
  load_row<T, E>(a.q, s * a.q_seq_stride + (kv * a.each + head0 + from) * a.q_head_stride + j * E, x0);
  const Visible vis = visible_of(length, a.width, 1 << a.page_log, a.window, a.sinks);
  const int per = tiles_per_split(vis.tiles, a.splits, kLeastTiles);
  const int t0 = split * per, t1 = t0 + per < vis.tiles ? t0 + per : vis.tiles;
  const int32_t* table = a.table + (int64_t)s * a.width;
  const int64_t row0 = (int64_t)s * a.q_heads + kv * a.each + head0;   // of [seqs][q_heads]

  int at = t0 + wave * kChunk;
  Place next;
  Loaded<D, F32, PER> c;
  // a wave without a chunk loads too (page 0): the number of loads before the first wait is then known
  locate(a, vis, table, at, t1, next);
  load_keys<D, F32, PER>(a, kv, next, c);
  load_values<D, F32, PER>(a, kv, next, c);

  if (threadIdx.x < D / 4) reinterpret_cast<uint32_t*>(sq[3 * HT])[threadIdx.x] = 0;
  // q: 16 lanes rotate a head and leave its bytes as operand rows h (a), HT + h (b) and 2 HT + h (c)
  if (group < HT) {
    apply_signs<E>(signs, x0);
#pragma unroll
    for (int i = 0; i < E; ++i) x0[i] *= 0.0625f;   // about 1 / sqrt(D), exactly: the transform's sums stay as small as the result
    fwht16<E>(x0);
    float amax = 0.0f, none = 0.0f;      // NaN where a value is not finite, which neither a maximum nor a whole number would show
#pragma unroll
    for (int i = 0; i < E; ++i) {
      amax = fmaxf(amax, __builtin_fabsf(x0[i]));
      none = __builtin_fmaf(x0[i], 0.0f, none);
    }
    amax = max16(amax);
    none = sum16(none);
    const int e = __builtin_amdgcn_frexp_expf(amax);   // amax < 2^e; 0 for 0
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float whole = __builtin_rintf(__builtin_amdgcn_ldexpf(x0[i], kBits - e));
      const int v = (int)fminf(fmaxf(whole, -0x1p22f), 0x1p22f);
      const int high = (v + 128) >> 8;   // 256 a + b
      sq[group][operand_byte<D>(j * E + i)] = (uint8_t)((high + 128) >> 8);
      sq[HT + group][operand_byte<D>(j * E + i)] = (uint8_t)high;
      sq[2 * HT + group][operand_byte<D>(j * E + i)] = (uint8_t)v;
    }
    // what a product of 16 c and the fixed point counts for in a score, log2
    const float cnorm = E == 4 ? 0.125f : (E == 8 ? 0.088388347648318447f : 0.0625f);
    if (j == 0) sf[group] = __builtin_amdgcn_ldexpf(cnorm * 1.4426950408889634f, e - kBits) * a.scale + none;   // 16 / 16
  }
  __syncthreads();
  // this lane's head, what its column counts for in a sum, and its operand rows
  const int h = HT == 4 ? n >> 2 : n & 7, r = HT == 4 ? n & 3 : n >> 3;
  const float counts = HT == 4 ? (r == 0 ? 1.0f : (r == 1 ? 256.0f : (r == 2 ? 65536.0f : 0.0f))) : (r ? 1.0f : 256.0f);
  const float partner_counts = HT == 4 ? (r == 0 ? 65536.0f : (r == 1 ? 0.0f : (r == 2 ? 1.0f : 256.0f))) : 0.0f;   // two columns on
  int q_row = (HT == 4 ? (r == 3 ? 3 * HT : (2 - r) * HT + h) : n) * D + 16 * g;
  int c_row = (r ? 2 * HT + h : 3 * HT) * D + 16 * g;   // 8 heads
  const float factor = sf[h];
  // The weights' bytes: 2^23 in front makes the sum's low 23 bits the whole number, + 128 * 257 its third byte a; the others are then
  // b + 128 and c + 128.  Byte selections (12 stands for 0).  4 heads: both stages of the transposition.  8 heads: what the partner gets
  // of the lane's two weights, what the lane keeps, and from the kept and the partner's bytes the operands of both products.
  const float magic = 8388608.0f + 32896.0f;
  const uint32_t near = r & 1 ? 0x03070105u : 0x06020400u, across = r & 2 ? 0x03020706u : 0x05040100u;
  const uint32_t give = r ? 0x0C0C0602u : 0x05040100u, keep = r ? 0x05040100u : 0x0C0C0602u;
  const uint32_t pick = r ? 0x03010705u : 0x05040100u, pick_c = r ? 0x02000604u : 0x0C0C0C0Cu;
  const uint32_t flip = (HT == 4 ? r < 2 : r == 1) ? 0x80808080u : 0u;
  const int odd_column = r & 1 ? -1 : 0, upper = (HT == 4 ? r & 2 : r) ? -1 : 0;

  float m = kNone, l = 0.0f;
  float o[E][4] = {};                     // element E (4 g + i) + e of column n
  // One chunk.  `more`: loads of the next one are issued as soon as registers are free, keys after the scores, values after their
  // transposition.  A constant, so that what is in flight is known where a load is waited for.
  auto chunk = [&](auto more) {
    int positions[kChunk];
#pragma unroll
    for (int t = 0; t < kChunk; ++t) positions[t] = next.pos[t];
    at += kWaves * kChunk;
    if constexpr (more) locate(a, vis, table, at, t1, next);
    // q is read again for every chunk: held, it would take the registers of loads in flight
    i32x4 q[NK], qc[NK];             // qc: 8 heads
    asm("" : "+v"(q_row), "+v"(c_row));
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      q[i] = *reinterpret_cast<const i32x4*>(&sq[0][0] + q_row + 64 * i);
      qc[i] = *reinterpret_cast<const i32x4*>(&sq[0][0] + c_row + 64 * i);
    }
    float x[kChunk][PER], top = kNone;
#pragma unroll
    for (int t = 0; t < kChunk; ++t) {
      i32x4 d = {0, 0, 0, 0}, k[NK];
      if constexpr (D == 64) {
        const u32x4 w = c.k[t][0];
        k[0] = i32x4{even_codes(w.x), even_codes(w.y), odd_codes(w.x), odd_codes(w.y)};
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const u32x4 w = c.k[t][i];
          k[2 * i] = i32x4{even_codes(w.x), even_codes(w.y), even_codes(w.z), even_codes(w.w)};
          k[2 * i + 1] = i32x4{odd_codes(w.x), odd_codes(w.y), odd_codes(w.z), odd_codes(w.w)};
        }
      }
#pragma unroll
      for (int i = 0; i < NK; ++i) d = __builtin_amdgcn_mfma_i32_16x16x64_i8(k[i], q[i], d, 0, 0, 0);
      if constexpr (HT == 8) {
        d = d << 8;
#pragma unroll
        for (int i = 0; i < NK; ++i) d = __builtin_amdgcn_mfma_i32_16x16x64_i8(k[i], qc[i], d, 0, 0, 0);
      }
      float sum[PER];
      if constexpr (HT == 4) {
        // the lower two columns go on with positions 0 and 1, the upper two with 2 and 3; then each with one
        float two[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int own = select(upper, d[2 + i], d[i]), other = lane_xor16<1>(select(upper, d[i], d[2 + i]));
          two[i] = __builtin_fmaf((float)own, counts, (float)other * partner_counts);
        }
        const float own = __int_as_float(select(odd_column, __float_as_int(two[1]), __float_as_int(two[0])));
        sum[0] = own + lane_xor16<0>(__int_as_float(select(odd_column, __float_as_int(two[0]), __float_as_int(two[1]))));
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int own = select(upper, d[2 + i], d[i]), other = lane_xor16<3>(select(upper, d[i], d[2 + i]));
          sum[i] = __builtin_fmaf((float)select(upper, other, own), 256.0f, (float)select(upper, own, other));   // of 256 a, of 256 b + c
        }
      }
      const int pos = positions[t];
      const bool cut = pos < 0 || pos + kTile > vis.len || (pos < vis.start && pos + kTile > vis.sinks);
#pragma unroll
      for (int i = 0; i < PER; ++i) x[t][i] = sum[i] * (scale_of<F32>(c.ks[t], i) * factor);
      if (cut) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int at_pos = pos + own_position<PER>(n, g) + i;
          const bool seen = (at_pos < vis.len) & (pos >= 0) & ((at_pos >= vis.start) | (at_pos < vis.sinks));
          x[t][i] = seen ? x[t][i] : kNone;
        }
      }
      top = fmaxf(top, PER == 2 ? fmaxf(x[t][0], x[t][PER - 1]) : x[t][0]);
    }
    if constexpr (more) load_keys<D, F32, PER>(a, kv, next, c);
    const float mn = fmaxf(m, max_over_head<HT>(top));
    const float base = mn == kNone ? 0.0f : mn;
    const float fade = m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - base);
    if (__any(mn != m)) {
      l *= fade;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[e][i] *= fade;
    }
    m = mn;
    top = 0.0f;
    {
      // a score is one rounded number wherever it is used: contracted into x - base it could exceed its own maximum
#pragma clang fp contract(off)
#pragma unroll
      for (int t = 0; t < kChunk; ++t)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const float p = __builtin_amdgcn_exp2f(x[t][i] - base);
          l += p;
          // what lies behind the last position may hold anything: it has weight 0 whatever its scale
          const float weight = p * scale_of<F32>(c.vs[t], i);
          x[t][i] = x[t][i] == kNone ? 0.0f : weight;
          l = __builtin_fmaf(x[t][i], 0.0f, l);      // NaN for a weight that is not finite
          top = fmaxf(top, x[t][i]);
        }
    }
    top = max_over_head<HT>(top);
    const int e_top = __builtin_amdgcn_frexp_expf(top);
    i32x4 p, pc;
#pragma unroll
    for (int t = 0; t < kChunk; ++t) {
      uint32_t w[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) w[i] = __float_as_uint(__builtin_amdgcn_ldexpf(x[t][i], kBits - e_top) + magic);
      if constexpr (HT == 4) {
        const uint32_t pair = __builtin_amdgcn_perm((uint32_t)lane_xor16<0>((int)w[0]), w[0], near);
        p[t] = (int)(__builtin_amdgcn_perm((uint32_t)lane_xor16<1>((int)pair), pair, across) ^ flip);
      } else {
        const uint32_t own = __builtin_amdgcn_perm(w[1], w[0], keep);
        const uint32_t other = (uint32_t)lane_xor16<3>((int)__builtin_amdgcn_perm(w[1], w[0], give));
        p[t] = (int)(__builtin_amdgcn_perm(other, own, pick) ^ flip);
        pc[t] = (int)(__builtin_amdgcn_perm(other, own, pick_c) ^ flip);
      }
    }
    const float back = __builtin_amdgcn_ldexpf(counts, e_top - kBits - 4);
    // V: byte r of the four rows of a lane's tile, transposed; its low nibbles are element 2 r, its high ones 2 r + 1
    constexpr int R = D / 32;
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
    if constexpr (more) load_values<D, F32, PER>(a, kv, next, c);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        i32x4 v, d = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < kChunk; ++t) v[t] = odd ? odd_codes(col[r][t]) : even_codes(col[r][t]);
        d = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, p, d, 0, 0, 0);
        if constexpr (HT == 8) d = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, pc, d << 8, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[2 * r + odd][i] = __builtin_fmaf((float)d[i], back, o[2 * r + odd][i]);
      }
  };
  if (at < t1) {
    while (at + kWaves * kChunk < t1) chunk(std::true_type{});
    chunk(std::false_type{});
  }
  // l over the lanes that share a head, o over its columns
  l = add_over_columns<HT>(l);
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[e][i] = add_over_columns<HT>(o[e][i]);
  if (r == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<f32x4*>(&so[wave][h][E * (4 * g + i) + e]) = f32x4{o[e][i], o[e + 1][i], o[e + 2][i], o[e + 3][i]};
    if (g == 0) {
      sm[wave][h] = m;
      sl[wave][h] = l;
    }
  }
  __syncthreads();
  if (group >= heads) return;
  m = kNone;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) m = fmaxf(m, sm[k][group]);
  l = 0.0f;
  float res[E] = {};
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    const float f = sm[k][group] == kNone ? 0.0f : __builtin_amdgcn_exp2f(sm[k][group] - m);
    l += sl[k][group] * f;
#pragma unroll
    for (int i = 0; i < E; ++i) res[i] = __builtin_fmaf(f, so[k][group][j * E + i], res[i]);
  }
  const int64_t row = row0 + group;
  if (a.splits == 1) {
    finish<T, E>(a, row, l, res);
    return;
  }
  float* part = a.partial + (row * a.splits + split) * D;
  store_row<RHTQ_IN_F32, E>(part, j * E, res);
  if (j == 0) {
    float* ml = a.partial + (int64_t)a.seqs * a.q_heads * a.splits * D + 2 * (row * a.splits + split);
    ml[0] = m;
    ml[1] = l;
  }
}

// One wave per query head: lane k of a stretch of 64 parts has that part's factor, and the wave's four groups of 16 lanes take the
// parts' sums in turn.
template <int T, int E>
__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(AttentionArgs a) {
  constexpr int D = 16 * E;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int64_t row = (int64_t)blockIdx.x * kJoinWaves + (threadIdx.x >> 6);
  if (row >= (int64_t)a.seqs * a.q_heads) return;
  const float* ml = a.partial + (int64_t)a.seqs * a.q_heads * a.splits * D + 2 * row * a.splits;
  const float* part = a.partial + row * a.splits * D;
  float m = kNone;
  for (int k = lane; k < a.splits; k += 64) m = fmaxf(m, ml[2 * k]);
#pragma unroll
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  float l = 0.0f, o[E] = {};
  for (int first = 0; first < a.splits; first += 64) {
    const int k = first + lane;
    const float f = k < a.splits && ml[2 * k] != kNone ? __builtin_amdgcn_exp2f(ml[2 * k] - m) : 0.0f;
    if (k < a.splits) l += f * ml[2 * k + 1];
    const int some = a.splits - first < 64 ? a.splits - first : 64;
    for (int i = 0; i < some; i += 16) {
      float v[4][E];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int mine = i + 4 * u + g < some ? i + 4 * u + g : some - 1;
        load_row<RHTQ_IN_F32, E>(part, (int64_t)(first + mine) * D + j * E, v[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float w = __shfl(f, i + 4 * u + g);      // 0 beyond the last part
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(w, v[u][e], o[e]);
      }
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    o[e] += __shfl_xor(o[e], 16);
    o[e] += __shfl_xor(o[e], 32);
  }
  if (g == 0) finish<T, E>(a, row, l, o);
}

template <int T, int E>
hipError_t launch_te(const AttentionArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.splits, (unsigned)(a.kv_heads * a.head_tiles), (unsigned)a.seqs), block(64 * kWaves);
  const bool f32 = a.scale_dtype == RHTQ_SCALE_F32;
  if (a.each <= 4) {
    if (f32) hipLaunchKernelGGL((attention_kernel<T, E, true, 4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attention_kernel<T, E, false, 4>), grid, block, 0, s, a);
  } else {
    if (f32) hipLaunchKernelGGL((attention_kernel<T, E, true, 8>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attention_kernel<T, E, false, 8>), grid, block, 0, s, a);
  }
  const int64_t rows = (int64_t)a.seqs * a.q_heads;
  if (a.splits > 1)
    hipLaunchKernelGGL((join_kernel<T, E>), dim3((unsigned)((rows + kJoinWaves - 1) / kJoinWaves)), dim3(64 * kJoinWaves), 0, s, a);
  return hipGetLastError();
}

// No page at all: no position is visible.
constexpr int64_t kZeroBlocks = 1 << 16;
__global__ __launch_bounds__(256) void zero_kernel(uint32_t* out, int64_t words) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)kZeroBlocks * 256) out[i] = 0;
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
  // Enough parts for a workgroup on every CU, and none so long that it would end alone beside shorter sequences.  More cost their
  // start (about 3 us of latency each) and the join: 32 x 8 heads x 4096 positions 29.5 us whole, 32.9 in two parts; one
  // sequence of 131072 32.8 us in 32 parts, 37.0 in 128; 24 x 8 heads of 1 .. 16384 44 us in two, 35 in four, 33 in eight.
  int64_t want = rows > 0 ? (kEnough + rows - 1) / rows : 1;
  if (want < (tiles + kMostTiles - 1) / kMostTiles) want = (tiles + kMostTiles - 1) / kMostTiles;
  const int64_t most = (tiles + kLeastTiles / 2) / kLeastTiles;
  if (want > most) want = most;
  if (want > 1024) want = 1024;
  return want < 1 ? 1 : (int32_t)want;
}

hipError_t launch_paged_attention(int dtype, const AttentionArgs& a, hipStream_t s) {
  if (a.pages == 0 || a.width == 0) {
    const int64_t words = (int64_t)a.seqs * a.q_heads * a.head_dim / 2;
    const int64_t blocks = (words + 255) / 256 < kZeroBlocks ? (words + 255) / 256 : kZeroBlocks;
    hipLaunchKernelGGL(zero_kernel, dim3((unsigned)blocks), dim3(256), 0, s, static_cast<uint32_t*>(a.out), words);
    return hipGetLastError();
  }
  if (dtype == RHTQ_IN_BF16) return launch_t<RHTQ_IN_BF16>(a, s);
  return launch_t<RHTQ_IN_F16>(a, s);
}

}  // namespace rhtq
