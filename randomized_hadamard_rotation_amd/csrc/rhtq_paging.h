// Index arithmetic of the paged cache, shared by the kernels and host checks: plain C++, no HIP header needed.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__) || defined(__HIP__)
#define RHTQ_HD __host__ __device__ __forceinline__
#else
#define RHTQ_HD inline
#endif

namespace rhtq {

constexpr int kTile = 16;   // positions of a tile: divides every page size, so a tile lies in one page

// A cache call's grid has a column of kColumn blocks of up to kBlockRows rows, and as many columns as needed, the last one whole too: up to
// kColumn * kBlockRows row numbers lie behind the last row, and they have to be 32-bit numbers as well.
constexpr int64_t kColumn = 32768;
constexpr int64_t kBlockRows = 128;
constexpr int64_t kMostRows = ((int64_t)1 << 31) - 2 * kColumn * kBlockRows;

// Page of slot group `idx` of a sequence's table row, or -1 where there is none.
RHTQ_HD int page_at(const int32_t* row, int width, int pages, int64_t idx) {
  if (idx < 0 || idx >= width) return -1;
  const int p = row[idx];
  return (uint32_t)p < (uint32_t)pages ? p : -1;
}

// Positions that count: 0 <= len <= width * page.
RHTQ_HD int32_t clamp_length(int32_t len, int width, int page) {
  const int64_t most = (int64_t)width * page;
  if (len < 0) return 0;
  return len > most ? (int32_t)most : len;
}

// Position of row t of sequence s (rows starts[s] .. starts[s+1]-1 end at lengths[s]-1), as int64; may be negative.
RHTQ_HD int64_t row_position(int64_t t, int32_t end, int32_t length) { return (int64_t)length - (int64_t)end + t; }

// The tiles a query looks at: `first` tiles from position 0 (the sinks), then those from tile `from` to the end.
struct Visible {
  int32_t len;      // clamped length
  int32_t sinks;    // positions [0, sinks) and [start, len) are visible
  int32_t start;
  int32_t first;    // tiles of the first stretch
  int32_t from;     // first tile of the second
  int32_t tiles;    // of both
};

RHTQ_HD Visible visible_of(int32_t length, int width, int page, int32_t window, int32_t sinks) {
  Visible v;
  v.len = clamp_length(length, width, page);
  v.sinks = 0;
  v.start = 0;
  if (window > 0 && v.len > window) {
    v.start = v.len - window;
    v.sinks = sinks < v.start ? sinks : v.start;
    if (v.sinks == v.start) v.sinks = v.start = 0;   // nothing between them: all is visible
  }
  v.first = (v.sinks + kTile - 1) / kTile;
  v.from = v.start / kTile;
  if (v.from < v.first) v.first = v.from;            // both stretches meet in one tile: the second has it
  v.tiles = v.first + (v.len + kTile - 1) / kTile - v.from;
  return v;
}

RHTQ_HD int32_t tile_at(const Visible& v, int32_t i) { return i < v.first ? i : v.from + (i - v.first); }

RHTQ_HD bool is_visible(const Visible& v, int32_t pos) { return pos < v.len && (pos >= v.start || pos < v.sinks); }

// Split of `tiles` tiles over at most `splits` parts of at least `least` tiles, a multiple of 4 each: tiles of a part.
RHTQ_HD int32_t tiles_per_split(int32_t tiles, int32_t splits, int32_t least) {
  int32_t per = (tiles + splits - 1) / splits;
  if (per < least) per = least;
  return (per + 3) & ~3;
}

}  // namespace rhtq
