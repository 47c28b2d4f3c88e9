// Handling of the cache's pages: reserving, freeing, trimming, forking, copying and compacting.
//
// The decisions (which page goes where) are prefix sums over the reference counts and the sequences, made by one workgroup
// of 1024 threads: a free page's rank is its place among the free ones in ascending order, so the outcome is the same in
// every run.  They are bounded by the latency of that workgroup's few passes; the bytes are moved by a second kernel over
// (page, layer) pairs at copy speed, which reads the decisions from the workspace.  Reference counts change by integer atomics,
// whose order does not show.
// Measured at 4,400 pages and 64 sequences: fork decisions 13.0 us, reserve 6.6 us, compaction's 5.5 us, each a handful of memory round trips;
// moved pages 306 MB (read and written) in 67 us, 4.6 TB/s.  A thread reads its stretch of the reference counts word by word, twice, so that
// the time grows with the pool.
#include "rhtq_internal.h"
#include "rhtq_paging.h"
#include "rhtq_serving_internal.h"

namespace rhtq {
namespace {

constexpr int kPlan = 1024;
constexpr int kCopy = 256;
constexpr int kCopyBlocks = 4096;      // most workgroups of a copy; they stride over the rest
constexpr int kSeqBlocks = 1 << 20;    // and of a kernel with one workgroup a sequence: a grid holds fewer than 2^32 threads along x
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// N sums over the workgroup at once: v becomes the sum before this thread, total that of all; every thread calls it.
template <int N>
__device__ __forceinline__ void scan(int64_t (&v)[N], int64_t (&total)[N]) {
  __shared__ int64_t wave_sum[N][kPlan / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = v[k];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t o = __shfl_up(x[k], d);
      if (lane >= d) x[k] += o;
    }
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (lane == 63) wave_sum[k][wave] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    int64_t before = 0;
    total[k] = 0;
    for (int i = 0; i < kPlan / 64; ++i) {
      if (i < wave) before += wave_sum[k][i];
      total[k] += wave_sum[k][i];
    }
    v[k] = before + x[k] - v[k];
  }
  __syncthreads();
}

// Stretch of `n` items that this thread looks after: neighbouring ones, so that its rank is the items' own order.
__device__ __forceinline__ void stretch(int n, int& from, int& to) {
  const int per = (n + kPlan - 1) / kPlan;
  from = min((int)threadIdx.x * per, n);
  to = n - from < per ? n : from + per;
}

// Free pages of this thread's stretch.
__device__ __forceinline__ int count_free(const PagesArgs& a) {
  int from, to;
  stretch(a.pages, from, to);
  int mine = 0;
  for (int p = from; p < to; ++p) mine += a.refs[p] <= 0;
  return mine;
}

// Writes the lowest `want` free pages, in order, to list[0 ..]; `at` free ones lie before this thread's stretch.
__device__ __forceinline__ void list_free(const PagesArgs& a, int32_t* list, int64_t at, int64_t want) {
  int from, to;
  stretch(a.pages, from, to);
  for (int p = from; p < to && at < want; ++p)
    if (a.refs[p] <= 0) list[at++] = p;
  __syncthreads();
}

// An entry that names no page, whatever it holds.
__device__ __forceinline__ bool no_page(const PagesArgs& a, int32_t entry) { return (uint32_t)entry >= (uint32_t)a.pages; }

// Page slots that a sequence of this length has positions in.  The next position's slot is length / page: the last of these where that one
// is partly filled.
__device__ __forceinline__ int64_t slots_of(int64_t length, int page) { return (length + page - 1) / page; }

__global__ __launch_bounds__(kPlan) void reserve_kernel(PagesArgs a) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  int from, to;
  stretch(a.seqs, from, to);
  int64_t mine = 0, beyond = 0;
  for (int s = from; s < to; ++s) {
    const int64_t len = a.lengths[s], more = a.add[s];
    if (more < 0 || len < 0) {
      bad = 1;
      continue;
    }
    const int64_t need = slots_of(len + more, a.page);
    if (need > a.width) beyond += need - a.width;
    if (more > 0)
      for (int64_t i = len / a.page; i < need && i < a.width; ++i) {
        const int32_t e = a.table[(int64_t)s * a.width + i];
        if (no_page(a, e)) ++mine;
        else if (a.refs[e] > 1) bad = 1;     // new rows would overwrite another sequence's
      }
  }
  int64_t sums[3] = {mine, beyond, count_free(a)}, all[3];
  scan(sums, all);
  const int64_t wanted = all[0], have = all[2];
  int64_t at = sums[0], short_of = all[1] + (wanted > have ? wanted - have : 0);
  if (short_of > INT32_MAX) short_of = INT32_MAX;
  if (threadIdx.x == 0) a.status[0] = bad ? -1 : (int32_t)short_of;
  if (bad || short_of) return;
  list_free(a, a.work, sums[2], wanted);
  for (int s = from; s < to; ++s) {
    if (a.add[s] == 0) continue;
    const int64_t len = a.lengths[s], need = slots_of(len + a.add[s], a.page);
    for (int64_t i = len / a.page; i < need; ++i) {
      int32_t& e = a.table[(int64_t)s * a.width + i];
      if (no_page(a, e)) {
        e = a.work[at++];
        a.refs[e] = 1;
      }
    }
    a.lengths[s] = (int32_t)(len + a.add[s]);
  }
}

__device__ __forceinline__ void release(const PagesArgs& a, int64_t entry) {
  const int32_t p = atomicExch(a.table + entry, -1);
  if ((uint32_t)p < (uint32_t)a.pages) atomicSub(a.refs + p, 1);
}

__global__ __launch_bounds__(kCopy) void free_kernel(PagesArgs a) {
  for (int64_t k = blockIdx.x; k < a.count; k += kSeqBlocks) {
    const int s = a.src[k];
    if ((uint32_t)s >= (uint32_t)a.seqs) continue;
    for (int i = threadIdx.x; i < a.width; i += kCopy) release(a, (int64_t)s * a.width + i);
    if (threadIdx.x == 0) a.lengths[s] = 0;
  }
}

__global__ __launch_bounds__(kCopy) void trim_kernel(PagesArgs a) {
  for (int64_t s = blockIdx.x; s < a.seqs; s += kSeqBlocks) {
    const int64_t len = clamp_length(a.lengths[s], a.width, a.page);   // where attention's window lies
    for (int i = threadIdx.x; i < a.width; i += kCopy) {
      const int64_t first = (int64_t)i * a.page;
      if (first >= a.sinks && first + a.page <= len - a.window) release(a, s * a.width + i);
    }
  }
}

// Workspace of a fork: [0, pages) the fresh pages, [pages, pages + seqs) marks, then three words for each pair
// (page copied from, page copied to, slots).
__global__ __launch_bounds__(kPlan) void fork_kernel(PagesArgs a) {
  __shared__ int bad;
  int32_t* marks = a.work + a.pages;
  int32_t* pairs = marks + a.seqs;
  if (threadIdx.x == 0) bad = 0;
  for (int s = threadIdx.x; s < a.seqs; s += kPlan) marks[s] = 0;
  for (int i = threadIdx.x; i < a.count; i += kPlan) pairs[3 * i] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < a.count; i += kPlan) {
    const int s = a.src[i], d = a.dst[i];
    if ((uint32_t)s >= (uint32_t)a.seqs || (uint32_t)d >= (uint32_t)a.seqs || a.lengths[s] < 0 || a.lengths[d] != 0 ||
        slots_of(a.lengths[s], a.page) > a.width || atomicAdd(marks + d, 1) != 0)
      bad = 1;
  }
  __syncthreads();
  if (!bad)
    for (int i = threadIdx.x; i < a.count; i += kPlan)
      if (marks[a.src[i]] != 0) bad = 1;
  __syncthreads();
  if (!bad)
    for (int64_t e = threadIdx.x; e < (int64_t)a.count * a.width; e += kPlan)
      if (!no_page(a, a.table[(int64_t)a.dst[e / a.width] * a.width + e % a.width])) bad = 1;
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) a.status[0] = -1;
    return;
  }
  // fresh pages go to the forks in order, one for each partly filled last page
  int from, to;
  stretch(a.count, from, to);
  int mine = 0;
  for (int i = from; i < to; ++i) {
    const int32_t len = a.lengths[a.src[i]];
    mine += len % a.page && page_at(a.table + (int64_t)a.src[i] * a.width, a.width, a.pages, len / a.page) >= 0;
  }
  int64_t sums[2] = {mine, count_free(a)}, all[2];
  scan(sums, all);
  const int64_t wanted = all[0], have = all[1];
  int64_t at = sums[0];
  if (threadIdx.x == 0) a.status[0] = wanted > have ? (int32_t)(wanted - have) : 0;
  if (wanted > have) return;
  list_free(a, a.work, sums[1], wanted);
  for (int i = from; i < to; ++i) {
    const int32_t len = a.lengths[a.src[i]];
    const int last = page_at(a.table + (int64_t)a.src[i] * a.width, a.width, a.pages, len / a.page);
    if (len % a.page && last >= 0) {
      const int32_t fresh = a.work[at++];
      a.refs[fresh] = 1;
      pairs[3 * i] = last;
      pairs[3 * i + 1] = fresh;
      pairs[3 * i + 2] = len % a.page;
    }
    a.lengths[a.dst[i]] = len;
  }
  __syncthreads();
  for (int64_t e = threadIdx.x; e < (int64_t)a.count * a.width; e += kPlan) {
    const int i = (int)(e / a.width), slot = (int)(e % a.width);
    const int64_t s = a.src[i];
    const int32_t len = a.lengths[s];
    int32_t p = -1;
    if (slot < len / a.page) {
      p = page_at(a.table + s * a.width, a.width, a.pages, slot);
      if (p >= 0) atomicAdd(a.refs + p, 1);
    } else if (slot == len / a.page && pairs[3 * i] >= 0) {
      p = pairs[3 * i + 1];
    }
    a.table[(int64_t)a.dst[i] * a.width + slot] = p;
  }
}

// Copies `slots` slots of every head of page `from` to page `to` in one layer: 16 bytes a thread where the bytes allow.
__device__ __forceinline__ void copy_page(const PagesArgs& a, int layer, int from, int to, int slots) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t head = (int64_t)a.page * a.row_bytes[k];
    const int64_t base = ((int64_t)layer * a.pages) * a.kv_heads * head;
    const uint8_t* src = a.data[k] + base + (int64_t)from * a.kv_heads * head;
    uint8_t* dst = a.data[k] + base + (int64_t)to * a.kv_heads * head;
    if (slots == a.page) {             // the whole page is one stretch, a multiple of 32 bytes
      const int64_t words = a.kv_heads * head / 16;
      for (int64_t i = threadIdx.x; i < words; i += kCopy)
        reinterpret_cast<u32x4*>(dst)[i] = reinterpret_cast<const u32x4*>(src)[i];
    } else if (a.row_bytes[k] >= 16) {
      const int words = slots * a.row_bytes[k] / 16, all = words * a.kv_heads;
      for (int i = threadIdx.x; i < all; i += kCopy) {
        const int64_t at = i / words * head / 16 + i % words;
        reinterpret_cast<u32x4*>(dst)[at] = reinterpret_cast<const u32x4*>(src)[at];
      }
    } else {                           // scales: 2 or 4 bytes each
      const int words = slots * a.row_bytes[k] / 2, all = words * a.kv_heads;
      for (int i = threadIdx.x; i < all; i += kCopy) {
        const int64_t at = i / words * head / 2 + i % words;
        reinterpret_cast<uint16_t*>(dst)[at] = reinterpret_cast<const uint16_t*>(src)[at];
      }
    }
  }
}

__global__ __launch_bounds__(kCopy) void fork_copy_kernel(PagesArgs a) {
  if (a.status[0] != 0) return;
  const int32_t* pairs = a.work + a.pages + a.seqs;
  for (int64_t u = blockIdx.x; u < (int64_t)a.count * a.layers; u += gridDim.x) {
    const int i = (int)(u / a.layers), layer = (int)(u % a.layers);
    if (pairs[3 * i] >= 0) copy_page(a, layer, pairs[3 * i], pairs[3 * i + 1], pairs[3 * i + 2]);
  }
}

__global__ __launch_bounds__(kCopy) void copy_kernel(PagesArgs a) {
  for (int64_t u = blockIdx.x; u < (int64_t)a.count * a.layers; u += gridDim.x) {
    const int i = (int)(u / a.layers), layer = (int)(u % a.layers);
    const int from = a.src[i], to = a.dst[i];
    if ((uint32_t)from < (uint32_t)a.pages && (uint32_t)to < (uint32_t)a.pages && from != to)
      copy_page(a, layer, from, to, a.page);
  }
}

// Workspace of a compaction: one word with the number of moves, then (from, to) of each, then each page's new place.
__global__ __launch_bounds__(kPlan) void compact_kernel(PagesArgs a) {
  int from, to;
  stretch(a.pages, from, to);
  int mine = 0;
  for (int p = from; p < to; ++p) mine += a.refs[p] > 0;
  int64_t used_before[1] = {mine}, used_in_all[1];
  scan(used_before, used_in_all);
  const int64_t live = used_in_all[0];
  int holes = 0, movers = 0;
  for (int p = from; p < to; ++p) {
    const bool used = a.refs[p] > 0;
    holes += !used && p < live;
    movers += used && p >= live;
  }
  int64_t sums[2] = {holes, movers}, all[2];
  scan(sums, all);
  int64_t h = sums[0], m = sums[1];
  const int64_t moves = all[1];
  int32_t* pairs = a.work + 1;
  int32_t* place = pairs + 2 * (a.pages / 2 + 1);
  for (int p = from; p < to; ++p) {
    const bool used = a.refs[p] > 0;
    if (!used && p < live) pairs[2 * h++ + 1] = p;
    if (used && p >= live) pairs[2 * m++] = p;
    else place[p] = p;
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < moves; i += kPlan) {
    const int old = pairs[2 * i], now = pairs[2 * i + 1];
    place[old] = now;
    a.refs[now] = a.refs[old];
    a.refs[old] = 0;
  }
  if (threadIdx.x == 0) {
    a.work[0] = (int32_t)moves;
    a.status[0] = (int32_t)live;
  }
}

__global__ __launch_bounds__(kCopy) void compact_move_kernel(PagesArgs a) {
  const int64_t moves = a.work[0];
  const int32_t* pairs = a.work + 1;
  const int32_t* place = pairs + 2 * (a.pages / 2 + 1);
  for (int64_t u = blockIdx.x; u < moves * a.layers; u += gridDim.x) {
    const int i = (int)(u / a.layers), layer = (int)(u % a.layers);
    copy_page(a, layer, pairs[2 * i], pairs[2 * i + 1], a.page);
  }
  if (moves == 0) return;
  const int64_t entries = (int64_t)a.seqs * a.width;
  for (int64_t e = (int64_t)blockIdx.x * kCopy + threadIdx.x; e < entries; e += (int64_t)gridDim.x * kCopy) {
    const int32_t p = a.table[e];
    if ((uint32_t)p < (uint32_t)a.pages && place[p] != p) a.table[e] = place[p];
  }
}

unsigned blocks(int64_t units) { return (unsigned)(units < kCopyBlocks ? (units < 1 ? 1 : units) : kCopyBlocks); }

}  // namespace

hipError_t launch_pages_reserve(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(reserve_kernel, dim3(1), dim3(kPlan), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_pages_free(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(free_kernel, dim3((unsigned)(a.count < kSeqBlocks ? a.count : kSeqBlocks)), dim3(kCopy), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_pages_trim(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(trim_kernel, dim3((unsigned)(a.seqs < kSeqBlocks ? a.seqs : kSeqBlocks)), dim3(kCopy), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_pages_fork(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(fork_kernel, dim3(1), dim3(kPlan), 0, s, a);
  hipLaunchKernelGGL(fork_copy_kernel, dim3(blocks((int64_t)a.count * a.layers)), dim3(kCopy), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_pages_copy(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(copy_kernel, dim3(blocks((int64_t)a.count * a.layers)), dim3(kCopy), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_pages_compact(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(compact_kernel, dim3(1), dim3(kPlan), 0, s, a);
  hipLaunchKernelGGL(compact_move_kernel, dim3(blocks((int64_t)(a.pages / 2 + 1) * a.layers)), dim3(kCopy), 0, s, a);
  return hipGetLastError();
}

}  // namespace rhtq
