// Internal interface between the host checks of the layer operators
// (qrs_layer.cpp) and their gfx950 kernels (qrs_rows.hip, qrs_matmul.hip).
// Not installed; callers use include/qrs.h.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "qrs_launch.h"

namespace qrs {

// The third scale layout of these operators: one fp32 scale for each row.
constexpr int kScaleF32Row = 2;

// Rows to codes: x quantized (norm = false), or the sum with residual,
// normalized (norm = true). Strides in elements.
struct RowsLaunch {
  OutFormat io_format;
  XFormat x_format;
  int scale_layout;  // ScaleLayout or kScaleF32Row; norm = false: kScaleF32Row
  bool norm;
  bool vec;  // h % 8 == 0, and every row starts on a 16-byte boundary (codes: 8)
  uint32_t h;
  float eps;
  double inv_h;  // 1 / h
  uint64_t rows;
  const void* x;
  uint64_t x_stride;
  const void* residual;  // nullptr: none
  uint64_t residual_stride;
  const void* weight;
  void* sum;  // written where there is a residual
  uint64_t sum_stride;
  void* codes;
  uint64_t codes_stride;
  void* scales;
};

constexpr uint32_t kMaxRowElems = 65536;

// h in [1, kMaxRowElems], a multiple of the layout's group.
hipError_t launch_rows(const RowsLaunch& l, hipStream_t stream);

struct NormBackwardLaunch {
  OutFormat io_format;
  bool vec;  // h % 8 == 0, and every row starts on a 16-byte boundary
  uint32_t h;
  float eps;
  double inv_h;  // 1 / h
  uint64_t rows;
  const void* grad_y;
  uint64_t grad_y_stride;
  const void* sum;
  uint64_t sum_stride;
  const void* weight;
  const void* grad_sum;  // nullptr: zero
  uint64_t grad_sum_stride;
  void* grad_x;
  uint64_t grad_x_stride;
  float* grad_weight;
  float* workspace;  // norm_backward_parts(rows, h) rows of h floats
};

// Work-groups of the backward pass, and rows of its workspace.
uint32_t norm_backward_parts(uint64_t rows, uint32_t h);

hipError_t launch_norm_backward(const NormBackwardLaunch& l, hipStream_t stream);

// P = a b^T of int8 a [m, k] and b [n, k] (gated: [2n, k]), strides in
// bytes, scaled and written as values (quantize = false) or as codes and
// scales (quantize = true).
struct MatmulLaunch {
  uint32_t m, n, k;
  bool gated;
  bool quantize;
  bool vec;      // k % 16 == 0, and every row of a and b starts on a 16-byte boundary
  bool out_vec;   // quantize = false: every row of out starts on a 16-byte boundary
  bool out_near;  // 256 rows of out, and of scales, span less than 2^30 bytes
  OutFormat out_format;      // quantize = false
  XFormat x_format;          // quantize = true
  ScaleLayout scale_layout;  // quantize = true
  const int8_t* a;
  uint64_t a_stride;
  const float* a_scales;
  const int8_t* b;
  uint64_t b_stride;
  const float* b_scales;
  void* out;  // values, or codes
  uint64_t out_stride;
  void* scales;
};

// The largest k whose sums of products (each at most 2^14) fit 32 bits.
constexpr int64_t kMaxMatmulK = 131071;

// Every shape of fewer than 2^24 tiles of 64 x 64 outputs has a kernel whose
// grid a launch holds (fewer than 2^32 work-items); hipErrorInvalidValue,
// launching nothing, beyond that.
hipError_t launch_matmul(const MatmulLaunch& l, hipStream_t stream);

// The kernel that launch_matmul takes: its family, and its tile in tokens and
// rows of b.
enum MatmulFamily : uint32_t { kMatmulTiles = 0, kMatmulFewTokens = 1, kMatmulMid = 2, kMatmulPipe = 3 };
struct MatmulKernel {
  MatmulFamily family;
  uint32_t tile_m, tile_n;
};
struct MatmulShape {
  MatmulKernel kernel;
  uint64_t blocks;
  uint32_t threads;
};
MatmulShape matmul_shape(const MatmulLaunch& l);

}  // namespace qrs
