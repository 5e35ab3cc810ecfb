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

}  // extern "C"
