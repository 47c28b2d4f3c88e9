// The paged 4-bit cache: new rows are rotated, quantised and stored in their slot; stored rows are read back.
//
// Per row of d = 64, 128 or 256:  y = H diag(s) x / sqrt(d), scale = fl(max|y| / 7), code = rne(y / scale), and back
// x = diag(s) H (code * scale) / sqrt(d).  Reading, the scale leaves the transform (H (c s) = s (H c)), which then runs on
// whole numbers of at most 8 d and is exact.
//
// Bounded by memory for prompts (2 d bytes in, d/2 + scale out, and back) and by latency for single tokens.  The transform has to
// stay out of the way: 7 butterfly stages at d = 128 on the vector units took 209 us to store and 255 us to read 1.71 M rows
// (551 MB each, 108 us at a copy's rate), so five or six of its bits go through the matrix cores, a wave taking 16 tokens of one head:
//
//  Storing (bf16, fp16): element NB k + r, NB = d / 32, k < 32.  For each r the products of H32 over k (v_mfma_f32_16x16x32, exact operands), then
//  log2 NB butterfly stages over r in registers.  A lane loads 16-byte pieces and pairs values of equal r with byte permutes; it
//  ends with d / 16 neighbouring elements of four tokens.  fp32 rows keep the vector form: 16 lanes a row, four stages by DPP.
//  Reading: element 128 h + 2 k + r: the even and the odd codes of a lane's 16 bytes as 16 c in int8, H64 (H32 at d = 64) over k, butterflies over
//  r and h in int32.  The scale leaves the transform, which is exact; it and the signs are applied to the result.
//
// The 16 tokens' slots lie side by side in a page, so that a page's lines are written whole by one XCD's cache.
// Now 190 us to store and 162 us to read those rows: bounded by the vector instructions (about 630 for 16 rows stored) and by the chain of
// lookups, which two tiles a wave share.  32 tokens x 8 heads: 6.3 and 5.8 us, that chain.
#include "rhtq_internal.h"
#include "rhtq_serving_device.h"
#include "rhtq_serving_internal.h"

namespace rhtq {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;
constexpr int kWaves = kThreads / 64;

typedef int i32x4 __attribute__((ext_vector_type(4)));

// token blocks: kColumn in a grid's y, the rest in z
__device__ __forceinline__ int token_block() { return (int)(blockIdx.y + blockIdx.z * kColumn); }

// Places of N tokens of a group of 16 lanes, the same in all of them: offset of the slot in rows of the code arrays, or -1.  A token's
// sequence is the number of sequences that end at or before it, counted by the 16 lanes together.
template <int N>
__device__ __forceinline__ void slots_of(const CacheArgs& a, const int (&t)[N], int head, int64_t (&slot)[N]) {
  if (a.seqs == 0) {                       // nothing of starts (but its 0) and lengths is there to read
#pragma unroll
    for (int k = 0; k < N; ++k) slot[k] = -1;
    return;
  }
  const int tokens = (int)a.tokens;        // below 2^31
  int s[N], pos[N];
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = a.starts ? 0 : t[k];
  if (a.starts) {
    for (int i = 1 + (threadIdx.x & 15); i <= a.seqs; i += 16) {
      const int32_t end = a.starts[i];
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] += end <= t[k];
    }
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = sum16(s[k]);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const bool there = t[k] < tokens && s[k] < a.seqs;
    s[k] = there ? s[k] : 0;
    const int64_t p = a.starts ? row_position(t[k], a.starts[s[k] + 1], a.lengths[s[k]]) : (int64_t)a.lengths[s[k]] - 1;
    const bool fits = there && p >= 0 && p <= INT32_MAX && (!a.starts || t[k] >= a.starts[s[k]]);
    pos[k] = fits ? (int)p : -1;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int p = page_at(a.table + (int64_t)s[k] * a.width, a.width, a.pages, pos[k] >> a.page_log);
    slot[k] = p < 0 ? -1 : (((int64_t)p * a.kv_heads + head) << a.page_log) + (pos[k] & ((1 << a.page_log) - 1));
  }
}

// Rotated row to codes: E neighbouring values in each of 16 lanes; the lane's E / 2 bytes and (lane 0) the scale are stored.
template <int E>
__device__ __forceinline__ void store_codes(const CacheArgs& a, int which, int64_t slot, const float (&v)[E]) {
  constexpr int D = 16 * E;
  const int j = threadIdx.x & 15;
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) amax = fmaxf(amax, __builtin_fabsf(v[i]));
  amax = max16(amax);
  const float cnorm = E == 4 ? 0.125f : (E == 8 ? 0.088388347648318447f : 0.0625f);
  const Int4Scale sc = int4_scale(amax, cnorm, a.scale_dtype);
  // v / s + 8 with 1.5 * 2^23 in front is 0x4B400000 + code + 8, the code rounded to nearest even; shifted sums of eight of them hold the
  // codes + 8 side by side over a constant.  |v / s| <= 7 unless the stored scale is far below amax / 7.
  float c[E];
#pragma unroll
  for (int i = 0; i < E; ++i) c[i] = v[i] * sc.inv;
  if (__any(sc.clamp)) {
#pragma unroll
    for (int i = 0; i < E; ++i) c[i] = fminf(fmaxf(c[i], -8.0f), 7.0f);
  }
  constexpr int PER = E < 8 ? E : 8;
  uint32_t w[E / PER], base = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) base += 0x4B400000u << (4 * i);
#pragma unroll
  for (int k = 0; k < E / PER; ++k) {
    uint32_t sum = 0;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) sum = (sum << 4) + __float_as_uint(c[PER * k + i] + 12582920.0f);
    w[k] = (sum - base) ^ 0x88888888u;
  }
  if (slot < 0) return;
  uint8_t* out = a.codes[which] + slot * (D / 2) + j * (E / 2);
  if constexpr (E == 4) *reinterpret_cast<uint16_t*>(out) = (uint16_t)w[0];
  else if constexpr (E == 8) *reinterpret_cast<uint32_t*>(out) = w[0];
  else *reinterpret_cast<u32x2*>(out) = u32x2{w[0], w[1]};
  if (j == 0) {
    // every element of a rotated row holds each of the row's values, so that the first one is not finite where one of them is not: a NaN scale
    if (a.scale_dtype == RHTQ_SCALE_F32) static_cast<float*>(a.scales[which])[slot] = __builtin_fmaf(v[0], 0.0f, sc.s);
    else static_cast<__half*>(a.scales[which])[slot] = __float2half_rn(__builtin_fmaf(v[0], 0.0f, fminf(sc.s, 65504.0f)));
  }
}

// fp32 rows: 16 lanes a row.
template <int E>
__global__ __launch_bounds__(kThreads) void append_f32_kernel(CacheArgs a) {
  const int j = threadIdx.x & 15;
  const int which = blockIdx.x & 1, head = blockIdx.x >> 1;
  const int t[1] = {token_block() * kGroups + (int)(threadIdx.x >> 4)};
  const int64_t from = t[0] < a.tokens ? t[0] : a.tokens - 1;
  float v[E];
  uint32_t signs[E / 4];
  load_row<RHTQ_IN_F32, E>(a.x[which], from * a.token_stride[which] + head * a.head_stride[which] + j * E, v);
  load_signs<E>(a.signs[which], j * E, signs);
  int64_t slot[1];
  slots_of<1>(a, t, head, slot);
  apply_signs<E>(signs, v);
  fwht16<E>(v);
  store_codes<E>(a, which, slot[0], v);
}

// 8 halves of +-1: the sign of H over k & o for k = 8 values of idx(j).
template <bool H16, typename F>
__device__ __forceinline__ bf16x8 hadamard_operand(int o, F idx) {
  uint32_t w[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t one = H16 ? 0x3C00u : 0x3F80u;
    const uint32_t lo = __builtin_popcount(idx(2 * p) & o) & 1, hi = __builtin_popcount(idx(2 * p + 1) & o) & 1;
    w[p] = (one | (lo << 15)) | ((one | (hi << 15)) << 16);
  }
  bf16x8 r;
  __builtin_memcpy(&r, w, 16);
  return r;
}

template <int T, int D, int TL>
__global__ __launch_bounds__(kThreads) void append_kernel(CacheArgs a) {
  constexpr int NB = D / 32;               // values of r; also the 16-byte pieces of a row that a lane loads
  constexpr int PER = 8 / NB;              // values of one r in a piece
  constexpr int E = D / 16;
  constexpr bool H16 = T == RHTQ_IN_F16;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int which = blockIdx.x & 1, head = blockIdx.x >> 1;
  const int first = (token_block() * kWaves + (int)(threadIdx.x >> 6)) * (16 * TL);
  if (first >= a.tokens) return;
  u32x4 c[TL][NB];
#pragma unroll
  for (int l = 0; l < TL; ++l) {
    const int64_t from = first + 16 * l + n < a.tokens ? first + 16 * l + n : a.tokens - 1;
    const uint16_t* x = static_cast<const uint16_t*>(a.x[which]) + from * a.token_stride[which] + head * a.head_stride[which];
#pragma unroll
    for (int i = 0; i < NB; ++i) c[l][i] = *reinterpret_cast<const u32x4*>(x + 8 * (4 * i + g));
  }
  // sign bits of a piece's values, two to a word
  uint32_t flip[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    uint32_t b[2];
    load_signs<8>(a.signs[which], 8 * (4 * i + g), b);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t two = b[p >> 1] >> (16 * (p & 1));
      flip[i][p] = ((two << 8) & 0x8000u) | ((two << 16) & 0x80000000u);
    }
  }
  bf16x8 h[2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    h[u] = hadamard_operand<H16>(2 * n + u, [&](int j) { return PER * (4 * (j / PER) + g) + j % PER; });
  int t[4 * TL];
  int64_t slot[4 * TL];
#pragma unroll
  for (int k = 0; k < 4 * TL; ++k) t[k] = first + 16 * (k / 4) + 4 * g + k % 4;
  slots_of<4 * TL>(a, t, head, slot);
#pragma unroll
  for (int l = 0; l < TL; ++l) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int p = 0; p < 4; ++p) c[l][i][p] ^= flip[i][p];
    f32x4 d[NB][2];
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      uint32_t w[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int j0 = 2 * p, j1 = 2 * p + 1;
        const uint32_t lo = c[l][j0 / PER][(r + NB * (j0 % PER)) >> 1], hi = c[l][j1 / PER][(r + NB * (j1 % PER)) >> 1];
        w[p] = __builtin_amdgcn_perm(hi, lo, r & 1 ? 0x07060302u : 0x05040100u);
      }
      bf16x8 v;
      __builtin_memcpy(&v, w, 16);
      const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < 2; ++u) d[r][u] = stage1_mma<H16>(v, h[u], z);
    }
#pragma unroll
    for (int b = 1; b < NB; b *= 2)
#pragma unroll
      for (int r = 0; r < NB; ++r)
        if ((r & b) == 0)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const f32x4 s = d[r][u] + d[r | b][u];
            d[r | b][u] = d[r][u] - d[r | b][u];
            d[r][u] = s;
          }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = d[e % NB][e / NB][k];
      store_codes<E>(a, which, slot[4 * l + k], v);
    }
  }
}

// +-1 in int8: the sign of H over k & o for k = k0 + 4 p + e, o = TILES n + u, as bytes e of words p.  Column u = 0 needs no more than a
// parity for each word (and, for H32, for its upper two bytes); u flips bytes by their lowest bits.
template <int D>
__device__ __forceinline__ void hadamard_bytes(int n, int g, uint32_t (&w)[D == 64 ? 2 : 4]) {
  // H64: k = 16 g + 4 p + e, o = 4 n + u; H32: k = 8 g + 4 p + e, o = 2 n + u
  constexpr int P = D == 64 ? 2 : 4;
  const int lane_bits = __builtin_popcount(g & (n >> 2));
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int bits = lane_bits + (D == 64 ? p & (n >> 1) : __builtin_popcount(p & n));
    w[p] = bits & 1 ? 0xFFFFFFFFu : 0x01010101u;
    if (D == 64 && (n & 1)) w[p] ^= 0xFEFE0000u;
  }
}

template <int T, int D, int TL>
__global__ __launch_bounds__(kThreads) void read_kernel(CacheArgs a) {
  constexpr int H = D == 256 ? 2 : 1;
  constexpr int TILES = D == 64 ? 2 : 4;   // of 16 columns
  constexpr int E = 2 * TILES;             // neighbouring elements of a lane's result, in each h
  __shared__ int64_t place[kWaves][16 * TL];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
  const int which = blockIdx.x & 1, head = blockIdx.x >> 1;
  if (!a.y[which]) return;
  const int first = (token_block() * kWaves + wave) * (16 * TL);
  uint32_t signs[H][E / 4];
#pragma unroll
  for (int h = 0; h < H; ++h) load_signs<E>(a.signs[which], 128 * h + E * n, signs[h]);
  uint32_t b[D == 64 ? 2 : 4];
  hadamard_bytes<D>(n, g, b);
  int t[4 * TL];
  int64_t slot[4 * TL];
#pragma unroll
  for (int k = 0; k < 4 * TL; ++k) t[k] = first + 16 * (k / 4) + 4 * g + k % 4;
  slots_of<4 * TL>(a, t, head, slot);
  if (n == 0) {
#pragma unroll
    for (int k = 0; k < 4 * TL; ++k) place[wave][16 * (k / 4) + 4 * g + k % 4] = slot[k];
  }
  __syncthreads();
  if (first >= a.tokens) return;
  // rows without a place take row 0 of the cache, if there is one, and a scale of 0
  uint32_t w[TL][H][4] = {};
  float s[4 * TL] = {};
  if (a.pages > 0) {
#pragma unroll
    for (int l = 0; l < TL; ++l) {
      const int64_t row = place[wave][16 * l + n] < 0 ? 0 : place[wave][16 * l + n];
      const uint8_t* in = a.codes[which] + row * (D / 2);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if constexpr (D == 64) {
          const u32x2 q = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(in + 8 * g));
          w[l][h][0] = q.x;
          w[l][h][1] = q.y;
        } else {
          const u32x4 q = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(in + 64 * h + 16 * g));
#pragma unroll
          for (int p = 0; p < 4; ++p) w[l][h][p] = q[p];
        }
      }
    }
    if (a.scale_dtype == RHTQ_SCALE_F32) {
#pragma unroll
      for (int k = 0; k < 4 * TL; ++k) s[k] = static_cast<const float*>(a.scales[which])[slot[k] < 0 ? 0 : slot[k]];
    } else {
#pragma unroll
      for (int k = 0; k < 4 * TL; ++k) s[k] = __half2float(static_cast<const __half*>(a.scales[which])[slot[k] < 0 ? 0 : slot[k]]);
    }
  }
#pragma unroll
  for (int l = 0; l < TL; ++l) {
    i32x4 d[H][2][TILES];
#pragma unroll
    for (int u = 0; u < TILES; ++u) {
      const i32x4 z = {0, 0, 0, 0};
      if constexpr (D == 64) {
        const uint32_t f = u ? 0xFE00FE00u : 0u;
        const long hb = (long)(((uint64_t)(b[1] ^ f) << 32) | (b[0] ^ f));
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t x = r ? w[l][0][0] & 0xF0F0F0F0u : (w[l][0][0] << 4) & 0xF0F0F0F0u;
          const uint32_t y = r ? w[l][0][1] & 0xF0F0F0F0u : (w[l][0][1] << 4) & 0xF0F0F0F0u;
          d[0][r][u] = __builtin_amdgcn_mfma_i32_16x16x32_i8((long)(((uint64_t)y << 32) | x), hb, z, 0, 0, 0);
        }
      } else {
        const uint32_t f = u == 0 ? 0u : (u == 1 ? 0xFE00FE00u : (u == 2 ? 0xFEFE0000u : 0x00FEFE00u));
        const i32x4 hb = {(int)(b[0] ^ f), (int)(b[1] ^ f), (int)(b[2] ^ f), (int)(b[3] ^ f)};
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            i32x4 v;
#pragma unroll
            for (int p = 0; p < 4; ++p) v[p] = (int)(r ? w[l][h][p] & 0xF0F0F0F0u : (w[l][h][p] << 4) & 0xF0F0F0F0u);
            d[h][r][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, hb, z, 0, 0, 0);
          }
      }
  }
#pragma unroll
    for (int u = 0; u < TILES; ++u) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const i32x4 sum = d[h][0][u] + d[h][1][u];
        d[h][1][u] = d[h][0][u] - d[h][1][u];
        d[h][0][u] = sum;
      }
      if constexpr (H == 2)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const i32x4 sum = d[0][r][u] + d[1][r][u];
          d[1][r][u] = d[0][r][u] - d[1][r][u];
          d[0][r][u] = sum;
        }
    }
    const float cnorm = D == 64 ? 0.125f : (D == 128 ? 0.088388347648318447f : 0.0625f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t[4 * l + k] >= a.tokens) continue;
      const float f = slot[4 * l + k] < 0 ? 0.0f : s[4 * l + k] * (cnorm * 0.0625f);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = slot[4 * l + k] < 0 ? 0.0f : (float)d[h][e & 1][e >> 1][k] * f;
        apply_signs<E>(signs[h], v);
        store_row<T, E>(a.y[which], ((int64_t)t[4 * l + k] * a.kv_heads + head) * D + 128 * h + E * n, v);
      }
    }
  }
}

// Heads of keys and values run fastest, then tokens: workgroups that run together then read and write neighbouring memory.  With tokens first
// they all took the same head of rows 16 KB apart, a few channels' worth: with one tile a wave, 188 us to store and
// 227 us to read where this order took 185 and 220.
static_assert(kMostRows + kColumn * kBlockRows <= INT32_MAX && 32 * kWaves <= kBlockRows && kGroups <= kBlockRows, "row numbers");
dim3 grid_of(const CacheArgs& a, int per) {
  const int64_t blocks = (a.tokens + per - 1) / per, y = blocks < kColumn ? blocks : kColumn;
  return dim3((unsigned)(2 * a.kv_heads), (unsigned)y, (unsigned)((blocks + kColumn - 1) / kColumn));
}

// Two tiles of 16 tokens a wave, looked up together, where that leaves enough waves; one for few tokens, whose latency counts.
template <int T, int TL>
hipError_t launch_append_t(const CacheArgs& a, hipStream_t s) {
  const dim3 grid = grid_of(a, 16 * TL * kWaves);
  switch (a.head_dim) {
    case 64: hipLaunchKernelGGL((append_kernel<T, 64, TL>), grid, dim3(kThreads), 0, s, a); break;
    case 128: hipLaunchKernelGGL((append_kernel<T, 128, TL>), grid, dim3(kThreads), 0, s, a); break;
    default: hipLaunchKernelGGL((append_kernel<T, 256, TL>), grid, dim3(kThreads), 0, s, a); break;
  }
  return hipGetLastError();
}

hipError_t launch_append_f32(const CacheArgs& a, hipStream_t s) {
  const dim3 grid = grid_of(a, kGroups);
  switch (a.head_dim) {
    case 64: hipLaunchKernelGGL((append_f32_kernel<4>), grid, dim3(kThreads), 0, s, a); break;
    case 128: hipLaunchKernelGGL((append_f32_kernel<8>), grid, dim3(kThreads), 0, s, a); break;
    default: hipLaunchKernelGGL((append_f32_kernel<16>), grid, dim3(kThreads), 0, s, a); break;
  }
  return hipGetLastError();
}

template <int T, int TL>
hipError_t launch_read_t(const CacheArgs& a, hipStream_t s) {
  const dim3 grid = grid_of(a, 16 * TL * kWaves);
  switch (a.head_dim) {
    case 64: hipLaunchKernelGGL((read_kernel<T, 64, TL>), grid, dim3(kThreads), 0, s, a); break;
    case 128: hipLaunchKernelGGL((read_kernel<T, 128, TL>), grid, dim3(kThreads), 0, s, a); break;
    default: hipLaunchKernelGGL((read_kernel<T, 256, TL>), grid, dim3(kThreads), 0, s, a); break;
  }
  return hipGetLastError();
}

constexpr int64_t kManyRows = 65536;     // rows of keys: 2 x 4 waves of two tiles on every CU

}  // namespace

hipError_t launch_cache_append(int dtype, const CacheArgs& a, hipStream_t s) {
  const bool many = a.tokens * a.kv_heads >= kManyRows;
  if (dtype == RHTQ_IN_BF16) return many ? launch_append_t<RHTQ_IN_BF16, 2>(a, s) : launch_append_t<RHTQ_IN_BF16, 1>(a, s);
  if (dtype == RHTQ_IN_F16) return many ? launch_append_t<RHTQ_IN_F16, 2>(a, s) : launch_append_t<RHTQ_IN_F16, 1>(a, s);
  return launch_append_f32(a, s);
}

hipError_t launch_cache_read(int dtype, const CacheArgs& a, hipStream_t s) {
  const bool many = a.tokens * a.kv_heads >= kManyRows;
  if (dtype == RHTQ_IN_BF16) return many ? launch_read_t<RHTQ_IN_BF16, 2>(a, s) : launch_read_t<RHTQ_IN_BF16, 1>(a, s);
  if (dtype == RHTQ_IN_F16) return many ? launch_read_t<RHTQ_IN_F16, 2>(a, s) : launch_read_t<RHTQ_IN_F16, 1>(a, s);
  return many ? launch_read_t<RHTQ_IN_F32, 2>(a, s) : launch_read_t<RHTQ_IN_F32, 1>(a, s);
}

}  // namespace rhtq
