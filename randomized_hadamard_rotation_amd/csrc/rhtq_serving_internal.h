// Interfaces between the serving entry points (rhtq_serving_api.cpp) and their kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serving/rhtq_serving.h"

namespace rhtq {

struct CacheArgs {
  const void* x[2];           // append: keys, values
  void* y[2];                 // read: keys, values (or null)
  int64_t token_stride[2];
  int64_t head_stride[2];
  int64_t tokens;
  uint8_t* codes[2];
  void* scales[2];
  const int8_t* signs[2];
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* starts;
  int32_t seqs;
  int32_t width;
  int32_t pages;
  int32_t kv_heads;
  int32_t page_log;
  int32_t head_dim;
  int32_t scale_dtype;
};

hipError_t launch_cache_append(int dtype, const CacheArgs& a, hipStream_t s);
hipError_t launch_cache_read(int dtype, const CacheArgs& a, hipStream_t s);

struct AttentionArgs {
  const void* q;
  int64_t q_seq_stride;
  int64_t q_head_stride;
  void* out;
  float* partial;             // sums [seqs][q_heads][splits][head_dim], then maximum and sum of weights [seqs][q_heads][splits][2]
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const void* k_scales;
  const void* v_scales;
  const int8_t* k_signs;
  const int8_t* v_signs;
  const int32_t* table;
  const int32_t* lengths;
  int32_t seqs;
  int32_t q_heads;
  int32_t kv_heads;
  int32_t each;               // q_heads / kv_heads
  int32_t head_tiles;         // tiles of 8 query heads that share a key-value head
  int32_t width;
  int32_t pages;
  int32_t page_log;
  int32_t head_dim;
  int32_t scale_dtype;
  int32_t window;
  int32_t sinks;
  int32_t splits;
  float scale;
};

int32_t attention_head_tiles(int32_t each);
// Parts that a sequence's positions are split into, from what the host knows (never from device memory).
int32_t attention_splits(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t width, int32_t page, int32_t window,
                         int32_t sinks);
hipError_t launch_paged_attention(int dtype, const AttentionArgs& a, hipStream_t s);

struct MatvecArgs {
  const void* x;              // [tokens][n], rotated
  void* halves;               // workspace: x in operand order, then the exponents, then the parts' sums
  int32_t* exponents;
  float* partial;
  const uint8_t* packed;
  const void* scales;
  const float* tensor_scale;  // NVFP4, else null
  void* y;
  int64_t tokens;
  int64_t rows;
  int32_t n;
  int32_t groups;             // scales of a row
  int32_t group_log;          // log2 of the group, -1: one group a row
  int32_t fmt;
  int32_t scale_dtype;
  int32_t out_dtype;
  int32_t k_splits;
};

constexpr int64_t kMostWeightRows = ((int64_t)1 << 31) - 1024;   // blocks of 256 rows, 512 threads each: below 2^32 threads
int64_t matvec_padded(int64_t tokens);
int32_t matvec_splits(int64_t tokens, int32_t n, int64_t rows);
int64_t matvec_halves_bytes(int64_t tokens, int32_t n);
hipError_t launch_matvec(int x_dtype, const MatvecArgs& a, hipStream_t s);

struct PagesArgs {
  int32_t* table;
  int32_t* lengths;
  int32_t* refs;
  const int32_t* add;
  const int32_t* src;
  const int32_t* dst;
  int32_t* status;
  int32_t* work;
  uint8_t* data[4];           // k codes, k scales, v codes, v scales
  int32_t row_bytes[4];       // bytes of one slot of one head
  int32_t layers;
  int32_t kv_heads;
  int32_t page;
  int32_t width;
  int32_t seqs;
  int32_t pages;
  int32_t count;
  int32_t window;
  int32_t sinks;
};

hipError_t launch_pages_reserve(const PagesArgs& a, hipStream_t s);
hipError_t launch_pages_free(const PagesArgs& a, hipStream_t s);
hipError_t launch_pages_trim(const PagesArgs& a, hipStream_t s);
hipError_t launch_pages_fork(const PagesArgs& a, hipStream_t s);
hipError_t launch_pages_copy(const PagesArgs& a, hipStream_t s);
hipError_t launch_pages_compact(const PagesArgs& a, hipStream_t s);

}  // namespace rhtq
