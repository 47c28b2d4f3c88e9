// Host entry points of include/serving/rhtq_products.h: argument checks, workspace sizes, launches.
// Every check happens before the first HIP call, so a rejected call enqueues nothing.
#include <stdint.h>

#include <climits>
#include <cmath>

#include "rhtq_internal.h"
#include "rhtq_products_internal.h"

namespace {

constexpr int64_t kMostTokens = 1 << 20, kMostRows = 1 << 24;
constexpr int64_t kMostResults = (int64_t)1 << 36;    // grids stay below their limits
constexpr int32_t kMostWidth = 1 << 20, kMostExperts = 32767, kMostNormWidth = 32768;

bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int from_hip(hipError_t e) { return e == hipSuccess ? RHTQ_OK : RHTQ_EHIP; }
int log2_of(int32_t v) { return 31 - __builtin_clz((unsigned)v); }
bool in_type(int t) { return t == RHTQ_IN_BF16 || t == RHTQ_IN_F16 || t == RHTQ_IN_F32; }
bool whole(int fmt) { return fmt == RHTQ_FMT_INT4 || fmt == RHTQ_FMT_INT8; }

// Format, group and scale type of rows of width n: RHTQ_OK or the status.
int check_format(int fmt, int32_t group, int scale_dtype, int32_t n) {
  if (fmt < RHTQ_FMT_INT4 || fmt > RHTQ_FMT_MXFP8) return RHTQ_EINVAL;
  if (whole(fmt)) {
    if (group != 0 && (!is_pow2(group) || group < 16 || n % group)) return RHTQ_EUNSUPPORTED;
    return scale_dtype == RHTQ_SCALE_F32 || scale_dtype == RHTQ_SCALE_F16 ? RHTQ_OK : RHTQ_EUNSUPPORTED;
  }
  if (fmt == RHTQ_FMT_NVFP4) return group == 16 && scale_dtype == RHTQ_SCALE_E4M3 ? RHTQ_OK : RHTQ_EUNSUPPORTED;
  return group == 32 && scale_dtype == RHTQ_SCALE_E8M0 ? RHTQ_OK : RHTQ_EUNSUPPORTED;
}

// Both sides' formats, the sizes and the output's type, without any pointer.
int check_product(const rhtq_rows_t* a, const rhtq_rows_t* w, int64_t a_rows, int64_t tokens, int32_t n, int64_t rows, int out_dtype) {
  if (!a || !w || !in_type(out_dtype) || tokens < 0 || rows < 0 || a_rows < 0) return RHTQ_EINVAL;
  if (n < 32 || n % 32 || n > kMostWidth) return RHTQ_EUNSUPPORTED;
  int st = check_format(a->fmt, a->group, a->scale_dtype, n);
  if (st == RHTQ_OK) st = check_format(w->fmt, w->group, w->scale_dtype, n);
  if (st != RHTQ_OK) return st;
  const int need = whole(a->fmt) ? RHTQ_FMT_INT4 : (a->fmt == RHTQ_FMT_NVFP4 ? RHTQ_FMT_NVFP4 : RHTQ_FMT_MXFP4);
  if (w->fmt != need) return RHTQ_EUNSUPPORTED;
  if (tokens > kMostTokens || a_rows > INT32_MAX || rows > kMostRows || tokens * rows > kMostResults) return RHTQ_EINVAL;
  return RHTQ_OK;
}

bool rows_pointers(const rhtq_rows_t* r) {
  const uintptr_t unit = r->scale_dtype == RHTQ_SCALE_F32 ? 4 : (r->scale_dtype == RHTQ_SCALE_F16 ? 2 : 1);
  return r->codes && r->scales && aligned(r->codes, 16) && aligned(r->scales, unit) &&
         (r->fmt != RHTQ_FMT_NVFP4 || (r->tensor_scale && aligned(r->tensor_scale, 4)));
}

rhtq::RowsArgs rows_args(const rhtq_rows_t* r, int32_t n) {
  rhtq::RowsArgs k{};
  k.codes = static_cast<const uint8_t*>(r->codes);
  k.scales = r->scales;
  k.tensor = r->fmt == RHTQ_FMT_NVFP4 ? r->tensor_scale : nullptr;
  k.groups = r->group ? n / r->group : 1;
  k.group_log = r->group ? log2_of(r->group) : -1;
  k.f32 = r->scale_dtype == RHTQ_SCALE_F32;
  k.wide = n % 128 == 0 && aligned(r->scales, r->fmt == RHTQ_FMT_NVFP4 ? 8 : 4);
  return k;
}

}  // namespace

extern "C" {

int rhtq_products_version(void) { return RHTQ_PRODUCTS_VERSION; }

int64_t rhtq_matmul_workspace(int64_t tokens, int32_t n, int64_t rows, int a_fmt) {
  if (tokens <= 0 || n <= 0 || rows <= 0 || tokens > kMostTokens || rows > kMostRows || n > kMostWidth || tokens * rows > kMostResults) return 0;
  const int64_t parts = rhtq::product_splits(tokens, n, rows, a_fmt);
  return parts > 1 ? 4 * parts * tokens * ((rows + 3) / 4 * 4) : 0;
}

int rhtq_matmul(const rhtq_rows_t* a, int64_t tokens, int32_t n, const rhtq_rows_t* w, int64_t rows, void* y_out, int out_dtype,
                void* workspace, int64_t workspace_bytes, rhtq_stream_t stream) {
  const int st = check_product(a, w, tokens, tokens, n, rows, out_dtype);
  if (st != RHTQ_OK || tokens == 0 || rows == 0) return st;
  if (!rows_pointers(a) || !rows_pointers(w) || !y_out || !aligned(y_out, 16)) return RHTQ_EINVAL;
  const int64_t need = rhtq_matmul_workspace(tokens, n, rows, a->fmt);
  if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return RHTQ_EINVAL;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  rhtq::ProductArgs p{};
  p.a = rows_args(a, n);
  p.w = rows_args(w, n);
  p.y = y_out;
  p.partial = static_cast<float*>(workspace);
  p.tokens = p.a_rows = tokens;
  p.rows = rows;
  p.n = n;
  p.experts = 1;
  p.out_dtype = out_dtype;
  p.k_splits = rhtq::product_splits(tokens, n, rows, a->fmt);
  return from_hip(rhtq::launch_product(a->fmt, p, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_grouped_matmul(const rhtq_rows_t* a, int64_t a_rows, int64_t tokens, int32_t n, const rhtq_rows_t* w, int32_t experts, int64_t rows,
                        const int32_t* starts, const int32_t* index, void* y_out, int out_dtype, rhtq_stream_t stream) {
  const int st = check_product(a, w, a_rows, tokens, n, rows, out_dtype);
  if (st != RHTQ_OK) return st;
  if (experts < 1 || experts > kMostExperts || (!index && a_rows < tokens) || (tokens + 64 * (int64_t)experts) * rows > kMostResults / 2)
    return RHTQ_EINVAL;
  if (tokens == 0 || rows == 0) return RHTQ_OK;
  if (a_rows == 0) return RHTQ_EINVAL;               // an index has to have a row to name
  if (!rows_pointers(a) || !rows_pointers(w) || !starts || !aligned(starts, 4) || !aligned(index, 4) || !y_out || !aligned(y_out, 16))
    return RHTQ_EINVAL;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  rhtq::ProductArgs p{};
  p.a = rows_args(a, n);
  p.w = rows_args(w, n);
  p.y = y_out;
  p.starts = starts;
  p.index = index;
  p.tokens = tokens;
  p.a_rows = a_rows;
  p.rows = rows;
  p.n = n;
  p.experts = experts;
  p.out_dtype = out_dtype;
  p.k_splits = 1;
  return from_hip(rhtq::launch_product(a->fmt, p, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_norm_forward(const void* x, const void* residual, void* residual_out, int in_dtype, int64_t tokens, int32_t n, const void* weight,
                      float eps, const int8_t* signs, int32_t block, int fmt, int32_t group, int scale_dtype, void* codes_out,
                      void* scales_out, const float* tensor_scale, rhtq_stream_t stream) {
  if (!in_type(in_dtype) || tokens < 0 || !(eps >= 0.0f) || std::isinf(eps)) return RHTQ_EINVAL;
  if (n < 32 || n % 32 || n > kMostNormWidth) return RHTQ_EUNSUPPORTED;
  const int st = check_format(fmt, group, scale_dtype, n);
  if (st != RHTQ_OK) return st;
  if (block != 0 && (!is_pow2(block) || block < 16 || n % block || (group != 0 && block % group))) return RHTQ_EUNSUPPORTED;
  if (tokens > ((int64_t)1 << 22) - 1) return RHTQ_EINVAL;   // a grid of 1024 threads each
  if (tokens == 0) return RHTQ_OK;
  if (!x || !codes_out || !scales_out || (residual && !residual_out) || (fmt == RHTQ_FMT_NVFP4 && !tensor_scale)) return RHTQ_EINVAL;
  const uintptr_t unit = scale_dtype == RHTQ_SCALE_F32 ? 4 : (scale_dtype == RHTQ_SCALE_F16 ? 2 : 1);
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(weight, 16) || !aligned(codes_out, 16) ||
      !aligned(scales_out, unit) || !aligned(tensor_scale, 4) || (block != 0 && !aligned(signs, 16)))
    return RHTQ_EINVAL;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  rhtq::NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.residual_out = residual_out;
  a.weight = weight;
  a.signs = block ? signs : nullptr;
  a.codes = static_cast<uint8_t*>(codes_out);
  a.scales = scales_out;
  a.tensor = tensor_scale;
  a.tokens = tokens;
  a.n = n;
  a.block_log = block ? log2_of(block) : -1;
  a.group_log = group ? log2_of(group) : -1;
  a.fmt = fmt;
  a.f32 = scale_dtype == RHTQ_SCALE_F32;
  a.eps = eps;
  return from_hip(rhtq::launch_norm(in_dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
