// C-ABI host functions of the operators between two shares: parameter
// checks and launches. The contract of every entry point is documented in
// include/qrs.h.

#include "qrs_layer.h"

#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstring>

#include "qrs_host.h"

namespace {

using qrs::aligned;
using qrs::fail;
using qrs::ok;
using qrs::overlaps;

constexpr int64_t kSpanLimit = int64_t{1} << 48;  // bytes any tensor may span

// A row-strided tensor: what the checks below need of it.
struct Rows {
  const char* name;
  const void* p;
  int64_t rows, cols, stride, size;  // elements; size in bytes

  uint64_t span() const { return static_cast<uint64_t>(((rows - 1) * stride + cols) * size); }
  bool same(const Rows& o) const { return p == o.p && stride == o.stride && size == o.size; }
  // Every row on an n-byte boundary.
  bool rows_on(int64_t n) const { return aligned(p, static_cast<uintptr_t>(n)) && (rows == 1 || stride * size % n == 0); }
};

qrs_status check_rows(const Rows& t) {
  if (!t.p) return fail(QRS_ERR_INVALID_ARG, "null pointer: %s", t.name);
  if (t.stride < t.cols)
    return fail(QRS_ERR_INVALID_ARG, "%s: row stride %lld is below the row's %lld elements", t.name,
                static_cast<long long>(t.stride), static_cast<long long>(t.cols));
  // Compared before multiplying, so that no product overflows.
  if (t.stride > kSpanLimit / t.size / t.rows)
    return fail(QRS_ERR_INVALID_ARG, "%s: row stride %lld is too large for %lld rows", t.name,
                static_cast<long long>(t.stride), static_cast<long long>(t.rows));
  if (!aligned(t.p, static_cast<uintptr_t>(t.size)))
    return fail(QRS_ERR_INVALID_ARG, "%s is not aligned to its %lld-byte elements", t.name,
                static_cast<long long>(t.size));
  return QRS_OK;
}

// Outputs against inputs and each other. in_place: the inputs that this
// output may be, whole.
qrs_status check_apart(const Rows& out, const Rows* others, int n, bool in_place) {
  for (int i = 0; i < n; ++i) {
    const Rows& o = others[i];
    if (!o.p || (in_place && out.same(o))) continue;
    if (overlaps(out.p, out.span(), o.p, o.span()))
      return fail(QRS_ERR_INVALID_ARG, "%s overlaps %s", out.name, o.name);
  }
  return QRS_OK;
}

qrs_status check_float_type(qrs_out_dtype t, const char* what) {
  if (t != QRS_OUT_F32 && t != QRS_OUT_BF16 && t != QRS_OUT_F16)
    return fail(QRS_ERR_INVALID_ARG, "%s %d is not a qrs_out_dtype", what, static_cast<int>(t));
  return QRS_OK;
}

int64_t type_size(qrs_out_dtype t) { return t == QRS_OUT_F32 ? 4 : 2; }

qrs::OutFormat to_format(qrs_out_dtype t) {
  return t == QRS_OUT_F32 ? qrs::kOutF32 : t == QRS_OUT_BF16 ? qrs::kOutBF16 : qrs::kOutF16;
}

qrs_status check_codes(qrs_x_dtype x, qrs_scale_layout s, bool row_scales) {
  if (x == QRS_X_HIFLOAT8) return fail(QRS_ERR_UNSUPPORTED, "HIFLOAT8 codes are reserved: their encoding is not defined");
  if (x != QRS_X_INT8 && x != QRS_X_FP8_E4M3FN && x != QRS_X_FP8_E5M2)
    return fail(QRS_ERR_INVALID_ARG, "x_dtype %d is not a qrs_x_dtype", static_cast<int>(x));
  if (s != QRS_SCALE_F32_GROUP128 && s != QRS_SCALE_E8M0_BLOCK32 && !(row_scales && s == QRS_SCALE_F32_ROW))
    return fail(QRS_ERR_INVALID_ARG, "scale_layout %d is not a layout of this call", static_cast<int>(s));
  if (s == QRS_SCALE_E8M0_BLOCK32 && x == QRS_X_INT8)
    return fail(QRS_ERR_INVALID_ARG, "INT8 codes are paired with fp32 scales only");
  return QRS_OK;
}

qrs::XFormat to_format(qrs_x_dtype x) {
  return x == QRS_X_INT8 ? qrs::kXInt8 : x == QRS_X_FP8_E4M3FN ? qrs::kXE4M3FN : qrs::kXE5M2;
}

int64_t group_of(qrs_scale_layout s, int64_t h) {
  return s == QRS_SCALE_F32_GROUP128 ? 128 : s == QRS_SCALE_E8M0_BLOCK32 ? 32 : h;
}

qrs_status check_row_shape(int64_t rows, int64_t h) {
  if (rows <= 0) return fail(QRS_ERR_INVALID_ARG, "%lld rows: must be positive", static_cast<long long>(rows));
  if (h < 1 || h > qrs::kMaxRowElems)
    return fail(QRS_ERR_INVALID_ARG, "rows of %lld elements: must be in [1, %lld]", static_cast<long long>(h),
                static_cast<long long>(qrs::kMaxRowElems));
  if (rows > (int64_t{1} << 40) / h)
    return fail(QRS_ERR_INVALID_ARG, "%lld rows: too many", static_cast<long long>(rows));
  return QRS_OK;
}

qrs_status check_eps(float eps) {
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(QRS_ERR_INVALID_ARG, "eps must be finite and not negative");
  return QRS_OK;
}

qrs_status launched(hipError_t e) {
  if (e != hipSuccess) return fail(QRS_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

#define QRS_TRY(call)                        \
  do {                                       \
    const qrs_status st_ = (call);           \
    if (st_ != QRS_OK) return st_;           \
  } while (0)

}  // namespace

extern "C" {

qrs_status qrs_add_rms_norm_quantize(int64_t tokens, int64_t h, qrs_out_dtype io_dtype, qrs_x_dtype x_dtype,
                                     qrs_scale_layout scale_layout, float eps, const void* x, int64_t x_row_stride,
                                     const void* residual, int64_t residual_row_stride, const void* weight,
                                     void* sum_out, int64_t sum_row_stride, void* codes, int64_t codes_row_stride,
                                     void* scales, void* stream) {
  QRS_TRY(check_row_shape(tokens, h));
  QRS_TRY(check_float_type(io_dtype, "io_dtype"));
  QRS_TRY(check_codes(x_dtype, scale_layout, true));
  QRS_TRY(check_eps(eps));
  const int64_t g = group_of(scale_layout, h);
  if (h % g != 0)
    return fail(QRS_ERR_INVALID_ARG, "h %lld is not a multiple of the layout's %lld", static_cast<long long>(h),
                static_cast<long long>(g));
  const int64_t size = type_size(io_dtype);
  const bool e8m0 = scale_layout == QRS_SCALE_E8M0_BLOCK32;
  const Rows in[3] = {{"x", x, tokens, h, x_row_stride, size},
                      {"weight", weight, 1, h, h, size},
                      {"residual", residual, tokens, h, residual_row_stride, size}};
  const Rows out[3] = {{"codes", codes, tokens, h, codes_row_stride, 1},
                       {"scales", scales, tokens, h / g, h / g, e8m0 ? 1 : 4},
                       {"sum_out", residual ? sum_out : nullptr, tokens, h, sum_row_stride, size}};
  const int n = residual ? 3 : 2;
  for (int i = 0; i < n; ++i) QRS_TRY(check_rows(in[i]));
  for (int i = 0; i < n; ++i) QRS_TRY(check_rows(out[i]));
  for (int i = 0; i < n; ++i) {
    QRS_TRY(check_apart(out[i], out + i + 1, n - i - 1, false));
    QRS_TRY(check_apart(out[i], &in[1], 1, false));
    QRS_TRY(check_apart(out[i], &in[0], 1, i == 2));
    if (residual) QRS_TRY(check_apart(out[i], &in[2], 1, i == 2));
  }

  qrs::RowsLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.io_format = to_format(io_dtype);
  l.x_format = to_format(x_dtype);
  l.scale_layout = scale_layout == QRS_SCALE_F32_ROW ? qrs::kScaleF32Row
                   : e8m0                            ? static_cast<int>(qrs::kScaleE8M0Block32)
                                                     : static_cast<int>(qrs::kScaleF32Group128);
  l.norm = true;
  l.vec = h % 8 == 0 && in[0].rows_on(16) && in[1].rows_on(16) && out[0].rows_on(8) &&
          (!residual || (in[2].rows_on(16) && out[2].rows_on(16)));
  l.h = static_cast<uint32_t>(h);
  l.eps = eps;
  l.inv_h = 1.0 / static_cast<double>(h);
  l.rows = static_cast<uint64_t>(tokens);
  l.x = x;
  l.x_stride = static_cast<uint64_t>(x_row_stride);
  l.weight = weight;
  if (residual) {
    l.residual = residual;
    l.residual_stride = static_cast<uint64_t>(residual_row_stride);
    l.sum = sum_out;
    l.sum_stride = static_cast<uint64_t>(sum_row_stride);
  }
  l.codes = codes;
  l.codes_stride = static_cast<uint64_t>(codes_row_stride);
  l.scales = scales;
  return launched(qrs::launch_rows(l, static_cast<hipStream_t>(stream)));
}

qrs_status qrs_quantize_rows(int64_t rows, int64_t cols, qrs_out_dtype in_dtype, qrs_x_dtype x_dtype, const void* x,
                             int64_t x_row_stride, void* codes, int64_t codes_row_stride, float* scales,
                             void* stream) {
  QRS_TRY(check_row_shape(rows, cols));
  QRS_TRY(check_float_type(in_dtype, "in_dtype"));
  QRS_TRY(check_codes(x_dtype, QRS_SCALE_F32_ROW, true));
  const Rows in = {"x", x, rows, cols, x_row_stride, type_size(in_dtype)};
  const Rows out[2] = {{"codes", codes, rows, cols, codes_row_stride, 1}, {"scales", scales, rows, 1, 1, 4}};
  QRS_TRY(check_rows(in));
  for (const Rows& o : out) QRS_TRY(check_rows(o));
  QRS_TRY(check_apart(out[0], &out[1], 1, false));
  for (const Rows& o : out) QRS_TRY(check_apart(o, &in, 1, false));

  qrs::RowsLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.io_format = to_format(in_dtype);
  l.x_format = to_format(x_dtype);
  l.scale_layout = qrs::kScaleF32Row;
  l.norm = false;
  l.vec = cols % 8 == 0 && in.rows_on(16) && out[0].rows_on(8);
  l.h = static_cast<uint32_t>(cols);
  l.rows = static_cast<uint64_t>(rows);
  l.x = x;
  l.x_stride = static_cast<uint64_t>(x_row_stride);
  l.codes = codes;
  l.codes_stride = static_cast<uint64_t>(codes_row_stride);
  l.scales = scales;
  return launched(qrs::launch_rows(l, static_cast<hipStream_t>(stream)));
}

qrs_status qrs_rms_norm_backward_workspace(int64_t tokens, int64_t h, size_t* bytes_out) {
  if (!bytes_out) return fail(QRS_ERR_INVALID_ARG, "null bytes_out");
  *bytes_out = 0;
  QRS_TRY(check_row_shape(tokens, h));
  *bytes_out = static_cast<size_t>(h) * 4 *
               qrs::norm_backward_parts(static_cast<uint64_t>(tokens), static_cast<uint32_t>(h));
  return ok();
}

qrs_status qrs_rms_norm_backward(int64_t tokens, int64_t h, qrs_out_dtype io_dtype, float eps, const void* grad_y,
                                 int64_t grad_y_row_stride, const void* sum, int64_t sum_row_stride,
                                 const void* weight, const void* grad_sum, int64_t grad_sum_row_stride, void* grad_x,
                                 int64_t grad_x_row_stride, float* grad_weight, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  size_t need = 0;
  QRS_TRY(qrs_rms_norm_backward_workspace(tokens, h, &need));
  QRS_TRY(check_float_type(io_dtype, "io_dtype"));
  QRS_TRY(check_eps(eps));
  if (!workspace || workspace_bytes < need)
    return fail(QRS_ERR_INVALID_ARG, "the workspace must hold %zu bytes", need);
  if (!aligned(workspace, 16)) return fail(QRS_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  const int64_t size = type_size(io_dtype);
  const Rows in[4] = {{"sum", sum, tokens, h, sum_row_stride, size},
                      {"weight", weight, 1, h, h, size},
                      {"grad_y", grad_y, tokens, h, grad_y_row_stride, size},
                      {"grad_sum", grad_sum, tokens, h, grad_sum_row_stride, size}};
  const Rows out[3] = {{"grad_x", grad_x, tokens, h, grad_x_row_stride, size},
                       {"grad_weight", grad_weight, 1, h, h, 4},
                       {"workspace", workspace, 1, static_cast<int64_t>(need / 4), static_cast<int64_t>(need / 4), 4}};
  const int n = grad_sum ? 4 : 3;
  for (int i = 0; i < n; ++i) QRS_TRY(check_rows(in[i]));
  for (const Rows& o : out) QRS_TRY(check_rows(o));
  for (int i = 0; i < 3; ++i) {
    QRS_TRY(check_apart(out[i], out + i + 1, 2 - i, false));
    QRS_TRY(check_apart(out[i], in, 2, false));
    QRS_TRY(check_apart(out[i], in + 2, n - 2, i == 0));
  }

  qrs::NormBackwardLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.io_format = to_format(io_dtype);
  l.vec = h % 8 == 0 && out[0].rows_on(16);
  for (int i = 0; i < n; ++i) l.vec = l.vec && in[i].rows_on(16);
  l.h = static_cast<uint32_t>(h);
  l.eps = eps;
  l.inv_h = 1.0 / static_cast<double>(h);
  l.rows = static_cast<uint64_t>(tokens);
  l.grad_y = grad_y;
  l.grad_y_stride = static_cast<uint64_t>(grad_y_row_stride);
  l.sum = sum;
  l.sum_stride = static_cast<uint64_t>(sum_row_stride);
  l.weight = weight;
  l.grad_sum = grad_sum;
  l.grad_sum_stride = static_cast<uint64_t>(grad_sum_row_stride);
  l.grad_x = grad_x;
  l.grad_x_stride = static_cast<uint64_t>(grad_x_row_stride);
  l.grad_weight = grad_weight;
  l.workspace = static_cast<float*>(workspace);
  return launched(qrs::launch_norm_backward(l, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

qrs_status check_matmul_shape(int64_t m, int64_t n, int64_t k, int gated) {
  if (gated != 0 && gated != 1) return fail(QRS_ERR_INVALID_ARG, "gated must be 0 or 1");
  const int64_t limit = int64_t{1} << 31;
  if (m <= 0 || m >= limit || n <= 0 || n >= limit)
    return fail(QRS_ERR_INVALID_ARG, "m %lld, n %lld: must be positive and below 2^31", static_cast<long long>(m),
                static_cast<long long>(n));
  if (k <= 0 || k > qrs::kMaxMatmulK)
    return fail(QRS_ERR_INVALID_ARG, "k %lld: must be in [1, %lld]", static_cast<long long>(k),
                static_cast<long long>(qrs::kMaxMatmulK));
  // 2^24 work-groups of the smallest tile, 64 x 64.
  if (((m + 63) / 64) * ((n + 63) / 64) >= int64_t{1} << 24)
    return fail(QRS_ERR_INVALID_ARG, "m %lld by n %lld: too large", static_cast<long long>(m), static_cast<long long>(n));
  return QRS_OK;
}

qrs_status check_quantized_shape(int64_t n, int gated) {
  if (gated) return fail(QRS_ERR_INVALID_ARG, "the gated product is not written as codes");
  if (n % 128 != 0) return fail(QRS_ERR_INVALID_ARG, "n %lld is not a multiple of 128", static_cast<long long>(n));
  return QRS_OK;
}

// The checks of both products but for the output's type; out and scales as
// the caller describes them (scales.p NULL: no scales).
qrs_status matmul(qrs::MatmulLaunch* l, int64_t m, int64_t n, int64_t k, int gated, const void* a,
                  int64_t a_row_stride, const float* a_scales, const void* b, int64_t b_row_stride,
                  const float* b_scales, const Rows& out, const Rows& scales, void* stream) {
  const int64_t wide = gated ? 2 * n : n;
  const Rows in[4] = {{"a", a, m, k, a_row_stride, 1},
                      {"b", b, wide, k, b_row_stride, 1},
                      {"a_scales", a_scales, 1, m, m, 4},
                      {"b_scales", b_scales, 1, wide, wide, 4}};
  for (const Rows& t : in) QRS_TRY(check_rows(t));
  QRS_TRY(check_rows(out));
  QRS_TRY(check_apart(out, in, 4, false));
  if (l->quantize) {
    QRS_TRY(check_rows(scales));
    QRS_TRY(check_apart(scales, in, 4, false));
    QRS_TRY(check_apart(scales, &out, 1, false));
  }
  l->m = static_cast<uint32_t>(m);
  l->n = static_cast<uint32_t>(n);
  l->k = static_cast<uint32_t>(k);
  l->gated = gated != 0;
  l->vec = k % 16 == 0 && in[0].rows_on(16) && in[1].rows_on(16);
  l->out_vec = out.rows_on(16);
  l->out_near = out.stride * out.size < (int64_t{1} << 22) && scales.stride * scales.size < (int64_t{1} << 22);
  l->a = static_cast<const int8_t*>(a);
  l->a_stride = static_cast<uint64_t>(a_row_stride);
  l->a_scales = a_scales;
  l->b = static_cast<const int8_t*>(b);
  l->b_stride = static_cast<uint64_t>(b_row_stride);
  l->b_scales = b_scales;
  l->out = const_cast<void*>(out.p);
  l->out_stride = static_cast<uint64_t>(out.stride);
  l->scales = const_cast<void*>(scales.p);
  return launched(qrs::launch_matmul(*l, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

qrs_status qrs_matmul_int(int64_t m, int64_t n, int64_t k, int gated, qrs_out_dtype out_dtype, const void* a,
                          int64_t a_row_stride, const float* a_scales, const void* b, int64_t b_row_stride,
                          const float* b_scales, void* out, int64_t out_row_stride, void* stream) {
  QRS_TRY(check_matmul_shape(m, n, k, gated));
  QRS_TRY(check_float_type(out_dtype, "out_dtype"));
  qrs::MatmulLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.quantize = false;
  l.out_format = to_format(out_dtype);
  const Rows o = {"out", out, m, n, out_row_stride, type_size(out_dtype)};
  const Rows none = {"scales", nullptr, 1, 1, 1, 1};
  return matmul(&l, m, n, k, gated, a, a_row_stride, a_scales, b, b_row_stride, b_scales, o, none,
                stream);
}

qrs_status qrs_matmul_int_quantize(int64_t m, int64_t n, int64_t k, qrs_x_dtype x_dtype,
                                   qrs_scale_layout scale_layout, const void* a, int64_t a_row_stride,
                                   const float* a_scales, const void* b, int64_t b_row_stride, const float* b_scales,
                                   void* codes, int64_t codes_row_stride, void* scales, void* stream) {
  QRS_TRY(check_matmul_shape(m, n, k, 0));
  QRS_TRY(check_codes(x_dtype, scale_layout, false));
  QRS_TRY(check_quantized_shape(n, 0));
  const bool e8m0 = scale_layout == QRS_SCALE_E8M0_BLOCK32;
  const int64_t g = e8m0 ? 32 : 128;
  qrs::MatmulLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.quantize = true;
  l.x_format = to_format(x_dtype);
  l.scale_layout = e8m0 ? qrs::kScaleE8M0Block32 : qrs::kScaleF32Group128;
  const Rows o = {"codes", codes, m, n, codes_row_stride, 1};
  if (codes && !o.rows_on(16)) return fail(QRS_ERR_INVALID_ARG, "rows of codes are not on 16-byte boundaries");
  const Rows s = {"scales", scales, m, n / g, n / g, e8m0 ? 1 : 4};
  return matmul(&l, m, n, k, 0, a, a_row_stride, a_scales, b, b_row_stride, b_scales, o, s, stream);
}

qrs_status qrs_matmul_launch_info(int64_t m, int64_t n, int64_t k, int gated, int quantize,
                                  qrs_scale_layout scale_layout, qrs_matmul_info* info_out) {
  if (!info_out) return fail(QRS_ERR_INVALID_ARG, "null info pointer");
  QRS_TRY(check_matmul_shape(m, n, k, gated));
  if (quantize != 0 && quantize != 1) return fail(QRS_ERR_INVALID_ARG, "quantize must be 0 or 1");
  if (quantize) {
    QRS_TRY(check_codes(QRS_X_FP8_E4M3FN, scale_layout, false));
    QRS_TRY(check_quantized_shape(n, gated));
  }
  qrs::MatmulLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.m = static_cast<uint32_t>(m);
  l.n = static_cast<uint32_t>(n);
  l.k = static_cast<uint32_t>(k);
  l.gated = gated != 0;
  l.quantize = quantize != 0;
  l.scale_layout = scale_layout == QRS_SCALE_E8M0_BLOCK32 ? qrs::kScaleE8M0Block32 : qrs::kScaleF32Group128;
  l.vec = k % 16 == 0;
  l.a_stride = l.b_stride = static_cast<uint64_t>(k);
  const qrs::MatmulShape shape = qrs::matmul_shape(l);
  info_out->blocks = shape.blocks;
  info_out->threads_per_block = shape.threads;
  info_out->kernel = static_cast<uint32_t>(shape.kernel.family);
  info_out->tile_m = shape.kernel.tile_m;
  info_out->tile_n = shape.kernel.tile_n;
  return ok();
}

qrs_status qrs_add_layer_norm_quantize(int64_t tokens, int64_t h, qrs_out_dtype io_dtype, qrs_x_dtype x_dtype,
                                       qrs_scale_layout scale_layout, float eps, const void* x, int64_t x_row_stride,
                                       const void* residual, int64_t residual_row_stride, const void* weight,
                                       const void* bias, void* sum_out, int64_t sum_row_stride, void* codes,
                                       int64_t codes_row_stride, void* scales, void* stream) {
  QRS_TRY(check_row_shape(tokens, h));
  QRS_TRY(check_float_type(io_dtype, "io_dtype"));
  QRS_TRY(check_codes(x_dtype, scale_layout, true));
  QRS_TRY(check_eps(eps));
  const int64_t g = group_of(scale_layout, h);
  if (h % g != 0)
    return fail(QRS_ERR_INVALID_ARG, "h %lld is not a multiple of the layout's %lld", static_cast<long long>(h),
                static_cast<long long>(g));
  const int64_t size = type_size(io_dtype);
  const bool e8m0 = scale_layout == QRS_SCALE_E8M0_BLOCK32;
  const Rows x_in = {"x", x, tokens, h, x_row_stride, size}, weight_in = {"weight", weight, 1, h, h, size};
  const Rows bias_in = {"bias", bias, 1, h, h, size};
  const Rows residual_in = {"residual", residual, tokens, h, residual_row_stride, size};
  const Rows out[3] = {{"codes", codes, tokens, h, codes_row_stride, 1},
                       {"scales", scales, tokens, h / g, h / g, e8m0 ? 1 : 4},
                       {"sum_out", residual ? sum_out : nullptr, tokens, h, sum_row_stride, size}};
  const int n = residual ? 3 : 2;
  QRS_TRY(check_rows(x_in));
  QRS_TRY(check_rows(weight_in));
  if (bias) QRS_TRY(check_rows(bias_in));
  if (residual) QRS_TRY(check_rows(residual_in));
  for (int i = 0; i < n; ++i) QRS_TRY(check_rows(out[i]));
  for (int i = 0; i < n; ++i) {
    QRS_TRY(check_apart(out[i], out + i + 1, n - i - 1, false));
    QRS_TRY(check_apart(out[i], &weight_in, 1, false));
    QRS_TRY(check_apart(out[i], &bias_in, 1, false));
    QRS_TRY(check_apart(out[i], &x_in, 1, i == 2));
    QRS_TRY(check_apart(out[i], &residual_in, 1, i == 2));
  }

  qrs::LayerNormLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.io_format = to_format(io_dtype);
  l.x_format = to_format(x_dtype);
  l.scale_layout = scale_layout == QRS_SCALE_F32_ROW ? qrs::kScaleF32Row
                   : e8m0                            ? static_cast<int>(qrs::kScaleE8M0Block32)
                                                     : static_cast<int>(qrs::kScaleF32Group128);
  l.vec = h % 8 == 0 && x_in.rows_on(16) && weight_in.rows_on(16) && out[0].rows_on(8) &&
          (!bias || bias_in.rows_on(16)) && (!residual || (residual_in.rows_on(16) && out[2].rows_on(16)));
  l.h = static_cast<uint32_t>(h);
  l.eps = eps;
  l.inv_h = 1.0 / static_cast<double>(h);
  l.rows = static_cast<uint64_t>(tokens);
  l.x = x;
  l.x_stride = static_cast<uint64_t>(x_row_stride);
  l.weight = weight;
  l.bias = bias;
  if (residual) {
    l.residual = residual;
    l.residual_stride = static_cast<uint64_t>(residual_row_stride);
    l.sum = sum_out;
    l.sum_stride = static_cast<uint64_t>(sum_row_stride);
  }
  l.codes = codes;
  l.codes_stride = static_cast<uint64_t>(codes_row_stride);
  l.scales = scales;
  return launched(qrs::launch_layer_norm(l, static_cast<hipStream_t>(stream)));
}

qrs_status qrs_layer_norm_backward_workspace(int64_t tokens, int64_t h, size_t* bytes_out) {
  if (!bytes_out) return fail(QRS_ERR_INVALID_ARG, "null bytes_out");
  *bytes_out = 0;
  QRS_TRY(check_row_shape(tokens, h));
  *bytes_out = static_cast<size_t>(h) * 8 *
               qrs::layer_norm_backward_parts(static_cast<uint64_t>(tokens), static_cast<uint32_t>(h), false);
  return ok();
}

qrs_status qrs_layer_norm_backward(int64_t tokens, int64_t h, qrs_out_dtype io_dtype, float eps, const void* grad_y,
                                   int64_t grad_y_row_stride, const void* sum, int64_t sum_row_stride,
                                   const void* weight, const void* grad_sum, int64_t grad_sum_row_stride, void* grad_x,
                                   int64_t grad_x_row_stride, float* grad_weight, float* grad_bias, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  size_t need = 0;
  QRS_TRY(qrs_layer_norm_backward_workspace(tokens, h, &need));
  QRS_TRY(check_float_type(io_dtype, "io_dtype"));
  QRS_TRY(check_eps(eps));
  if (!workspace || workspace_bytes < need)
    return fail(QRS_ERR_INVALID_ARG, "the workspace must hold %zu bytes", need);
  if (!aligned(workspace, 16)) return fail(QRS_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  const int64_t size = type_size(io_dtype);
  const Rows in[4] = {{"sum", sum, tokens, h, sum_row_stride, size},
                      {"weight", weight, 1, h, h, size},
                      {"grad_y", grad_y, tokens, h, grad_y_row_stride, size},
                      {"grad_sum", grad_sum, tokens, h, grad_sum_row_stride, size}};
  const Rows out[4] = {{"grad_x", grad_x, tokens, h, grad_x_row_stride, size},
                       {"grad_weight", grad_weight, 1, h, h, 4},
                       {"workspace", workspace, 1, static_cast<int64_t>(need / 4), static_cast<int64_t>(need / 4), 4},
                       {"grad_bias", grad_bias, 1, h, h, 4}};
  const int n = grad_sum ? 4 : 3, n_out = grad_bias ? 4 : 3;
  for (int i = 0; i < n; ++i) QRS_TRY(check_rows(in[i]));
  for (int i = 0; i < n_out; ++i) QRS_TRY(check_rows(out[i]));
  for (int i = 0; i < n_out; ++i) {
    QRS_TRY(check_apart(out[i], out + i + 1, n_out - i - 1, false));
    QRS_TRY(check_apart(out[i], in, 2, false));
    QRS_TRY(check_apart(out[i], in + 2, n - 2, i == 0));
  }

  qrs::LayerNormBackwardLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.io_format = to_format(io_dtype);
  l.vec = h % 8 == 0 && out[0].rows_on(16);
  for (int i = 0; i < n; ++i) l.vec = l.vec && in[i].rows_on(16);
  l.h = static_cast<uint32_t>(h);
  l.eps = eps;
  l.inv_h = 1.0 / static_cast<double>(h);
  l.rows = static_cast<uint64_t>(tokens);
  l.grad_y = grad_y;
  l.grad_y_stride = static_cast<uint64_t>(grad_y_row_stride);
  l.sum = sum;
  l.sum_stride = static_cast<uint64_t>(sum_row_stride);
  l.weight = weight;
  l.grad_sum = grad_sum;
  l.grad_sum_stride = static_cast<uint64_t>(grad_sum_row_stride);
  l.grad_x = grad_x;
  l.grad_x_stride = static_cast<uint64_t>(grad_x_row_stride);
  l.grad_weight = grad_weight;
  l.grad_bias = grad_bias;
  l.workspace = static_cast<float*>(workspace);
  return launched(qrs::launch_layer_norm_backward(l, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

qrs_status check_fp8_type(qrs_x_dtype x, const char* what) {
  if (x != QRS_X_FP8_E4M3FN && x != QRS_X_FP8_E5M2)
    return fail(QRS_ERR_INVALID_ARG, "%s %d is not an 8-bit floating-point type", what, static_cast<int>(x));
  return QRS_OK;
}

constexpr int64_t kSide = 128;  // rows and columns of a block of codes with one scale

int64_t blocks_of(int64_t n) { return (n + kSide - 1) / kSide; }

// Both quantizations of 128 x 128 blocks: codes or codes_t may be NULL, as the
// callers allow.
qrs_status quantize_blocks(bool by_block, int64_t rows, int64_t cols, qrs_out_dtype in_dtype, qrs_x_dtype x_dtype,
                           const void* x, int64_t x_row_stride, void* codes, int64_t codes_row_stride, float* scales,
                           void* codes_t, int64_t rows_t, int64_t codes_t_row_stride, float* scales_t, void* stream) {
  const int64_t limit = int64_t{1} << 31;
  if (rows <= 0 || rows >= limit || cols <= 0 || cols >= limit)
    return fail(QRS_ERR_INVALID_ARG, "rows %lld, cols %lld: must be positive and below 2^31",
                static_cast<long long>(rows), static_cast<long long>(cols));
  if (blocks_of(rows) * blocks_of(cols) >= int64_t{1} << 24)
    return fail(QRS_ERR_INVALID_ARG, "rows %lld by cols %lld: too large", static_cast<long long>(rows),
                static_cast<long long>(cols));
  QRS_TRY(check_float_type(in_dtype, "in_dtype"));
  QRS_TRY(check_fp8_type(x_dtype, "x_dtype"));
  if (codes_t && (rows_t < rows || rows_t > blocks_of(rows) * kSide))
    return fail(QRS_ERR_INVALID_ARG, "rows_t %lld: must be in [%lld, %lld]", static_cast<long long>(rows_t),
                static_cast<long long>(rows), static_cast<long long>(blocks_of(rows) * kSide));
  const Rows in = {"x", x, rows, cols, x_row_stride, type_size(in_dtype)};
  QRS_TRY(check_rows(in));
  const int64_t br = by_block ? blocks_of(rows) : rows, bc = by_block ? blocks_of(cols) : cols;
  const Rows all[4] = {{"codes", codes, rows, cols, codes_row_stride, 1},
                       {"scales", scales, br, blocks_of(cols), blocks_of(cols), 4},
                       {"codes_t", codes_t, cols, rows_t, codes_t_row_stride, 1},
                       {"scales_t", scales_t, bc, blocks_of(rows), blocks_of(rows), 4}};
  Rows out[4];
  int n = 0;
  for (int i = 0; i < 4; ++i)
    if (i < 2 ? codes != nullptr : codes_t != nullptr) out[n++] = all[i];
  for (int i = 0; i < n; ++i) QRS_TRY(check_rows(out[i]));
  for (int i = 0; i < n; ++i) {
    QRS_TRY(check_apart(out[i], out + i + 1, n - i - 1, false));
    QRS_TRY(check_apart(out[i], &in, 1, false));
  }

  qrs::BlocksLaunch l;
  std::memset(&l, 0, sizeof(l));
  l.io_format = to_format(in_dtype);
  l.x_format = to_format(x_dtype);
  l.by_block = by_block;
  l.vec = cols % 8 == 0 && in.rows_on(16) && (!codes || all[0].rows_on(8));
  l.vec_t = codes_t && rows_t % 16 == 0 && all[2].rows_on(16);
  l.rows = static_cast<uint64_t>(rows);
  l.cols = static_cast<uint64_t>(cols);
  l.rows_t = static_cast<uint64_t>(rows_t);
  l.x = x;
  l.x_stride = static_cast<uint64_t>(x_row_stride);
  l.codes = codes;
  l.codes_stride = static_cast<uint64_t>(codes_row_stride);
  l.scales = scales;
  l.codes_t = codes_t;
  l.codes_t_stride = static_cast<uint64_t>(codes_t_row_stride);
  l.scales_t = scales_t;
  return launched(qrs::launch_blocks(l, static_cast<hipStream_t>(stream)));
}

qrs_status check_fp8_shape(int64_t m, int64_t n, int64_t k, int gated) {
  QRS_TRY(check_matmul_shape(m, n, 1, gated));
  if (k <= 0 || k > qrs::kMaxFp8K)
    return fail(QRS_ERR_INVALID_ARG, "k %lld: must be in [1, %lld]", static_cast<long long>(k),
                static_cast<long long>(qrs::kMaxFp8K));
  return QRS_OK;
}

qrs_status check_scale_rows(int b_scale_rows, int gated) {
  if (b_scale_rows != 1 && b_scale_rows != kSide)
    return fail(QRS_ERR_INVALID_ARG, "b_scale_rows %d: must be 1 or 128", b_scale_rows);
  if (gated && b_scale_rows == 1) return fail(QRS_ERR_INVALID_ARG, "the gated product takes scales of 128 rows of b");
  return QRS_OK;
}

void fp8_shape(qrs::MatmulFp8Launch* l, int64_t m, int64_t n, int64_t k, int gated, int b_scale_rows) {
  l->m = static_cast<uint32_t>(m);
  l->n = static_cast<uint32_t>(n);
  l->k = static_cast<uint32_t>(k);
  l->gated = gated != 0;
  l->grouped = b_scale_rows == 1;
  l->groups = static_cast<uint32_t>(blocks_of(k));
  l->up_block = static_cast<uint32_t>(blocks_of(n));
}

// The checks of both products but for the output's type, as matmul() above.
qrs_status matmul_fp8(qrs::MatmulFp8Launch* l, int64_t m, int64_t n, int64_t k, int gated, qrs_x_dtype a_dtype,
                      const void* a, int64_t a_row_stride, const float* a_scales, qrs_x_dtype b_dtype,
                      int b_scale_rows, const void* b, int64_t b_row_stride, const float* b_scales, const Rows& out,
                      const Rows& scales, void* stream) {
  QRS_TRY(check_fp8_type(a_dtype, "a_dtype"));
  QRS_TRY(check_fp8_type(b_dtype, "b_dtype"));
  QRS_TRY(check_scale_rows(b_scale_rows, gated));
  const int64_t wide = gated ? 2 * n : n, groups = blocks_of(k);
  const int64_t scale_rows = b_scale_rows == 1 ? n : gated ? 2 * blocks_of(n) : blocks_of(n);
  const Rows in[4] = {{"a", a, m, k, a_row_stride, 1},
                      {"b", b, wide, k, b_row_stride, 1},
                      {"a_scales", a_scales, m, groups, groups, 4},
                      {"b_scales", b_scales, scale_rows, groups, groups, 4}};
  for (const Rows& t : in) QRS_TRY(check_rows(t));
  QRS_TRY(check_rows(out));
  QRS_TRY(check_apart(out, in, 4, false));
  if (l->quantize) {
    QRS_TRY(check_rows(scales));
    QRS_TRY(check_apart(scales, in, 4, false));
    QRS_TRY(check_apart(scales, &out, 1, false));
    const Rows ws = {"workspace", l->workspace, m, n, n, 4};
    if (ws.p) {
      QRS_TRY(check_rows(ws));
      QRS_TRY(check_apart(ws, in, 4, false));
      QRS_TRY(check_apart(ws, &out, 1, false));
      QRS_TRY(check_apart(ws, &scales, 1, false));
    }
  }
  fp8_shape(l, m, n, k, gated, b_scale_rows);
  l->a_format = to_format(a_dtype);
  l->b_format = to_format(b_dtype);
  l->vec = k % 16 == 0 && in[0].rows_on(16) && in[1].rows_on(16);
  l->out_vec = out.rows_on(16);
  l->a = static_cast<const int8_t*>(a);
  l->a_stride = static_cast<uint64_t>(a_row_stride);
  l->a_scales = a_scales;
  l->b = static_cast<const int8_t*>(b);
  l->b_stride = static_cast<uint64_t>(b_row_stride);
  l->b_scales = b_scales;
  l->out = const_cast<void*>(out.p);
  l->out_stride = static_cast<uint64_t>(out.stride);
  l->scales = const_cast<void*>(scales.p);
  return launched(qrs::launch_matmul_fp8(*l, static_cast<hipStream_t>(stream)));
}

qrs_status matmul_fp8_values(bool binary32, int64_t m, int64_t n, int64_t k, int gated, qrs_out_dtype out_dtype,
                             qrs_x_dtype a_dtype, const void* a, int64_t a_row_stride, const float* a_scales,
                             qrs_x_dtype b_dtype, int b_scale_rows, const void* b, int64_t b_row_stride,
                             const float* b_scales, void* out, int64_t out_row_stride, void* stream) {
  QRS_TRY(check_fp8_shape(m, n, k, gated));
  QRS_TRY(check_float_type(out_dtype, "out_dtype"));
  qrs::MatmulFp8Launch l;
  std::memset(&l, 0, sizeof(l));
  l.quantize = false;
  l.binary32 = binary32;
  l.out_format = to_format(out_dtype);
  const Rows o = {"out", out, m, n, out_row_stride, type_size(out_dtype)};
  const Rows none = {"scales", nullptr, 1, 1, 1, 1};
  return matmul_fp8(&l, m, n, k, gated, a_dtype, a, a_row_stride, a_scales, b_dtype, b_scale_rows, b, b_row_stride,
                    b_scales, o, none, stream);
}

qrs_status check_multiple(int64_t n) {
  if (n % 128 != 0) return fail(QRS_ERR_INVALID_ARG, "n %lld is not a multiple of 128", static_cast<long long>(n));
  return QRS_OK;
}

}  // namespace

extern "C" {

qrs_status qrs_quantize_blocks(int64_t rows, int64_t cols, qrs_out_dtype in_dtype, qrs_x_dtype x_dtype, const void* x,
                               int64_t x_row_stride, void* codes, int64_t codes_row_stride, float* scales,
                               void* codes_t, int64_t rows_t, int64_t codes_t_row_stride, float* scales_t,
                               void* stream) {
  if (!codes && !codes_t) return fail(QRS_ERR_INVALID_ARG, "null pointer: codes, and codes_t");
  return quantize_blocks(true, rows, cols, in_dtype, x_dtype, x, x_row_stride, codes, codes_row_stride, scales,
                         codes_t, rows_t, codes_t_row_stride, scales_t, stream);
}

qrs_status qrs_quantize_transposed(int64_t rows, int64_t cols, qrs_out_dtype in_dtype, qrs_x_dtype x_dtype,
                                   const void* x, int64_t x_row_stride, void* codes_t, int64_t rows_t,
                                   int64_t codes_t_row_stride, float* scales_t, void* codes, int64_t codes_row_stride,
                                   float* scales, void* stream) {
  if (!codes_t) return fail(QRS_ERR_INVALID_ARG, "null pointer: codes_t");
  return quantize_blocks(false, rows, cols, in_dtype, x_dtype, x, x_row_stride, codes, codes_row_stride, scales,
                         codes_t, rows_t, codes_t_row_stride, scales_t, stream);
}

qrs_status qrs_matmul_float(int64_t m, int64_t n, int64_t k, int gated, qrs_out_dtype out_dtype, qrs_x_dtype a_dtype,
                          const void* a, int64_t a_row_stride, const float* a_scales, qrs_x_dtype b_dtype,
                          int b_scale_rows, const void* b, int64_t b_row_stride, const float* b_scales, void* out,
                          int64_t out_row_stride, void* stream) {
  return matmul_fp8_values(false, m, n, k, gated, out_dtype, a_dtype, a, a_row_stride, a_scales, b_dtype, b_scale_rows,
                           b, b_row_stride, b_scales, out, out_row_stride, stream);
}

qrs_status qrs_matmul_float_single(int64_t m, int64_t n, int64_t k, int gated, qrs_out_dtype out_dtype,
                                   qrs_x_dtype a_dtype, const void* a, int64_t a_row_stride, const float* a_scales,
                                   qrs_x_dtype b_dtype, int b_scale_rows, const void* b, int64_t b_row_stride,
                                   const float* b_scales, void* out, int64_t out_row_stride, void* stream) {
  return matmul_fp8_values(true, m, n, k, gated, out_dtype, a_dtype, a, a_row_stride, a_scales, b_dtype, b_scale_rows,
                           b, b_row_stride, b_scales, out, out_row_stride, stream);
}

qrs_status qrs_matmul_float_quantize(int64_t m, int64_t n, int64_t k, int gated, qrs_x_dtype x_dtype,
                                   qrs_scale_layout scale_layout, qrs_x_dtype a_dtype, const void* a,
                                   int64_t a_row_stride, const float* a_scales, qrs_x_dtype b_dtype, const void* b,
                                   int64_t b_row_stride, const float* b_scales, void* codes, int64_t codes_row_stride,
                                   void* scales, void* workspace, size_t workspace_bytes, void* stream) {
  QRS_TRY(check_fp8_shape(m, n, k, gated));
  QRS_TRY(check_codes(x_dtype, scale_layout, false));
  QRS_TRY(check_multiple(n));
  const bool e8m0 = scale_layout == QRS_SCALE_E8M0_BLOCK32;
  const int64_t g = e8m0 ? 32 : 128;
  qrs::MatmulFp8Launch l;
  std::memset(&l, 0, sizeof(l));
  l.quantize = true;
  l.x_format = to_format(x_dtype);
  l.scale_layout = e8m0 ? qrs::kScaleE8M0Block32 : qrs::kScaleF32Group128;
  const Rows o = {"codes", codes, m, n, codes_row_stride, 1};
  if (codes && !o.rows_on(16)) return fail(QRS_ERR_INVALID_ARG, "rows of codes are not on 16-byte boundaries");
  const Rows s = {"scales", scales, m, n / g, n / g, e8m0 ? 1 : 4};
  const uint64_t need = qrs::fp8_workspace(static_cast<uint64_t>(m), static_cast<uint64_t>(n), gated != 0, l.scale_layout);
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(QRS_ERR_INVALID_ARG, "the workspace must hold %llu bytes", static_cast<unsigned long long>(need));
    if (!aligned(workspace, 16)) return fail(QRS_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    l.workspace = static_cast<float*>(workspace);
  }
  return matmul_fp8(&l, m, n, k, gated, a_dtype, a, a_row_stride, a_scales, b_dtype, static_cast<int>(kSide), b,
                    b_row_stride, b_scales, o, s, stream);
}

qrs_status qrs_matmul_float_quantize_workspace(int64_t m, int64_t n, int gated, qrs_scale_layout scale_layout,
                                               size_t* bytes_out) {
  if (!bytes_out) return fail(QRS_ERR_INVALID_ARG, "null bytes_out");
  *bytes_out = 0;
  QRS_TRY(check_matmul_shape(m, n, 1, gated));
  QRS_TRY(check_codes(QRS_X_FP8_E4M3FN, scale_layout, false));
  QRS_TRY(check_multiple(n));
  *bytes_out = qrs::fp8_workspace(static_cast<uint64_t>(m), static_cast<uint64_t>(n), gated != 0,
                                  scale_layout == QRS_SCALE_E8M0_BLOCK32 ? qrs::kScaleE8M0Block32
                                                                         : qrs::kScaleF32Group128);
  return ok();
}

qrs_status qrs_matmul_float_launch_info(int64_t m, int64_t n, int64_t k, int gated, int b_scale_rows, int quantize,
                                        qrs_out_dtype out_dtype, qrs_scale_layout scale_layout,
                                        qrs_matmul_info* info_out) {
  if (!info_out) return fail(QRS_ERR_INVALID_ARG, "null info pointer");
  QRS_TRY(check_fp8_shape(m, n, k, gated));
  QRS_TRY(check_scale_rows(b_scale_rows, gated));
  if (quantize != 0 && quantize != 1) return fail(QRS_ERR_INVALID_ARG, "quantize must be 0 or 1");
  if (quantize) {
    QRS_TRY(check_codes(QRS_X_FP8_E4M3FN, scale_layout, false));
    QRS_TRY(check_multiple(n));
    if (b_scale_rows == 1) return fail(QRS_ERR_INVALID_ARG, "b_scale_rows 1: codes take scales of 128 rows of b");
  } else {
    QRS_TRY(check_float_type(out_dtype, "out_dtype"));
  }
  qrs::MatmulFp8Launch l;
  std::memset(&l, 0, sizeof(l));
  fp8_shape(&l, m, n, k, gated, b_scale_rows);
  l.quantize = quantize != 0;
  l.out_format = quantize ? qrs::kOutF32 : to_format(out_dtype);
  l.scale_layout = scale_layout == QRS_SCALE_E8M0_BLOCK32 ? qrs::kScaleE8M0Block32 : qrs::kScaleF32Group128;
  l.vec = k % 16 == 0;
  l.a_stride = l.b_stride = static_cast<uint64_t>(k);
  const qrs::MatmulShape shape = qrs::matmul_fp8_shape(l);
  info_out->blocks = shape.blocks;
  info_out->threads_per_block = shape.threads;
  info_out->kernel = static_cast<uint32_t>(shape.kernel.family);
  info_out->tile_m = shape.kernel.tile_m;
  info_out->tile_n = shape.kernel.tile_n;
  return ok();
}

}  // extern "C"
