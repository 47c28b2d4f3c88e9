// Attention of one new token per sequence over the paged 4-bit cache, split over the length and joined.
//
//   o = H^T diag.. sum_j p_j s^v_j c^v_j / sum_j p_j,   p_j = exp(x_j - max x),   x_j = scale * s^k_j (R q) . c^k_j
//
// The rotation is orthonormal, so q is rotated once, the codes are used as they lie, and the sum is rotated back once.
// Each part of a sequence keeps the running maximum m, the sum l and the weighted sum o (all fp32); parts (m, l, o) join as
// m = max m_i, l = sum l_i exp(m_i - m), o likewise.
#include "rhtq_internal.h"
#include "rhtq_serving_device.h"
#include "rhtq_serving_internal.h"

namespace rhtq {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;
constexpr int kLeastTiles = 16;         // tiles of a part worth a workgroup
constexpr float kNone = -INFINITY;

template <int E>
__device__ __forceinline__ void unpack_row(const uint8_t* in, float (&v)[E]) {
  uint32_t w[(E + 7) / 8];
  if constexpr (E == 4) w[0] = *reinterpret_cast<const uint16_t*>(in);
  else if constexpr (E == 8) w[0] = *reinterpret_cast<const uint32_t*>(in);
  else {
    const u32x2 q = *reinterpret_cast<const u32x2*>(in);
    w[0] = q.x;
    w[1] = q.y;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = (float)((int)(w[i >> 3] << (28 - 4 * (i & 7))) >> 28);
}

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

template <int T, int E>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttentionArgs a) {
  constexpr int D = 16 * E;
  __shared__ float sm[kGroups], sl[kGroups];
  __shared__ float so[kGroups][D];
  const int j = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int split = blockIdx.x % a.splits;
  const int64_t row = blockIdx.x / a.splits;              // [seqs][q_heads]
  const int s = (int)(row / a.q_heads), h = (int)(row % a.q_heads);
  const int kv = h / a.each;
  const Visible vis = visible_of(a.lengths[s], a.width, 1 << a.page_log, a.window, a.sinks);
  const int per = tiles_per_split(vis.tiles, a.splits, kLeastTiles);
  const int t0 = split * per, t1 = t0 + per < vis.tiles ? t0 + per : vis.tiles;

  float q[E];
  load_row<T, E>(a.q, s * a.q_seq_stride + h * a.q_head_stride + j * E, q);
  apply_signs<E>(a.k_signs, j * E, q);
  fwht16<E>(q);
  const float cnorm = E == 4 ? 0.125f : (E == 8 ? 0.088388347648318447f : 0.0625f);
  float m = kNone, l = 0.0f, o[E] = {};
  const int32_t* table = a.table + (int64_t)s * a.width;
  for (int t = t0; t < t1; ++t) {
    const int pos = tile_at(vis, t) * kTile + g;
    const int p = is_visible(vis, pos) ? page_at(table, a.width, a.pages, pos >> a.page_log) : -1;
    if (p < 0) continue;
    const int64_t slot = (((int64_t)p * a.kv_heads + kv) << a.page_log) + (pos & ((1 << a.page_log) - 1));
    float v[E];
    unpack_row<E>(a.k_codes + slot * (D / 2) + j * (E / 2), v);
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) x = __builtin_fmaf(v[i], q[i], x);
    float e, f, mn;
    {
      // the score is one rounded number wherever it is used: contracted into x - mn it could exceed its own maximum
#pragma clang fp contract(off)
      x = sum16(x) * (load_scale(a.k_scales, slot, a.scale_dtype) * cnorm * a.scale);
      mn = fmaxf(m, x);
      f = m == kNone ? 0.0f : __expf(m - mn);
      e = __expf(x - mn);
    }
    m = mn;
    l = l * f + e;
    unpack_row<E>(a.v_codes + slot * (D / 2) + j * (E / 2), v);
    const float ev = e * load_scale(a.v_scales, slot, a.scale_dtype);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = __builtin_fmaf(ev, v[i], o[i] * f);
  }
  if (j == 0) {
    sm[g] = m;
    sl[g] = l;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) so[g][j * E + i] = o[i];
  __syncthreads();
  if (g != 0) return;
  for (int i = 0; i < kGroups; ++i) m = fmaxf(m, sm[i]);
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.0f;
  for (int k = 0; k < kGroups; ++k) {
    const float f = sm[k] == kNone ? 0.0f : __expf(sm[k] - m);
    l += sl[k] * f;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = __builtin_fmaf(f, so[k][j * E + i], o[i]);
  }
  if (a.splits == 1) {
    finish<T, E>(a, row, l, o);
    return;
  }
  float* part = a.partial + (row * a.splits + split) * D;
  store_row<RHTQ_IN_F32, E>(part, j * E, o);
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
    const float f = __expf(ml[2 * k] - m);
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
  const int64_t rows = (int64_t)a.seqs * a.q_heads;
  hipLaunchKernelGGL((attention_kernel<T, E>), dim3((unsigned)(rows * a.splits)), dim3(kThreads), 0, s, a);
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

int32_t attention_splits(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t width, int32_t page, int32_t window,
                         int32_t sinks) {
  int64_t tiles = (int64_t)width * page / kTile;
  if (window > 0) {
    const int64_t most = (int64_t)window / kTile + 2 + ((int64_t)sinks + kTile - 1) / kTile;
    if (most < tiles) tiles = most;
  }
  (void)kv_heads;
  const int64_t rows = (int64_t)seqs * q_heads;
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
