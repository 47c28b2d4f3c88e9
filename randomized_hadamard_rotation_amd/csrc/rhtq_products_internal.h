// Interfaces between the entry points of include/serving/rhtq_products.h (rhtq_products_api.cpp) and their kernels.  Not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serving/rhtq_products.h"

namespace rhtq {

// One side of a product: quantised rows.
struct RowsArgs {
  const uint8_t* codes;
  const void* scales;
  const float* tensor;        // NVFP4, else null
  int32_t groups;             // scales of a row
  int32_t group_log;          // log2 of the group, -1: one group a row
  int32_t f32;                // INT4, INT8: fp32 scales (fp16 otherwise)
  int32_t wide;               // E8M0, E4M3: a step's scales of a row can be loaded at once
};

struct ProductArgs {
  RowsArgs a;                 // activations: y's rows
  RowsArgs w;                 // weights: y's columns
  void* y;
  float* partial;             // sums of the parts of k, [k_splits][tokens][rows up to the next multiple of 4]
  const int32_t* starts;      // grouped: [experts + 1], else null
  const int32_t* index;       // grouped: row of a for each row of y, or null
  int64_t tokens;             // rows of y
  int64_t a_rows;
  int64_t rows;               // columns of y
  int32_t n;
  int32_t experts;            // 1 where there are no starts
  int32_t out_dtype;
  int32_t k_splits;
};

// Parts of k that a call's sums are split into (1: no workspace).
int32_t product_splits(int64_t tokens, int32_t n, int64_t rows, int a_fmt);
hipError_t launch_product(int a_fmt, const ProductArgs& p, hipStream_t s);

struct NormArgs {
  const void* x;
  const void* residual;       // or null
  void* residual_out;
  const void* weight;         // or null; x's type
  const int8_t* signs;        // or null
  uint8_t* codes;
  void* scales;
  const float* tensor;
  int64_t tokens;
  int32_t n;
  int32_t block_log;          // -1: no rotation
  int32_t group_log;          // -1: one group a row
  int32_t fmt;
  int32_t f32;                // INT4, INT8: fp32 scales
  float eps;
};

hipError_t launch_norm(int dtype, const NormArgs& a, hipStream_t s);

}  // namespace rhtq
