// gfx950 kernels over rows of activations: residual sum + RMS norm + codes
// and scales, its backward pass, and plain row quantization.
//
//   s = x + residual            (rounded to the activations' type)
//   r = 1 / sqrt(mean(s^2) + eps)
//   y = s * r * weight          (binary32)
//   codes, scales = quantize(y)
//
// A row stays in the registers of one wave or work-group from its load to
// its codes: one pass over memory, with the sum of squares (and, for row
// scales, the maximum of |y|) joined over the lanes in between. The work is
// a stream: x and residual in, s, codes and scales out, and what bounds it
// is HBM.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qrs_device.h"
#include "qrs_layer.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace {

using namespace dev;

// Sum (or maximum) over a work-group of NT lanes, in every lane, in a fixed
// order. `part` holds one value per wave and is used once.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (NT > 64) {
    constexpr int kWaves = NT / 64;
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w];
  }
  return v;
}

template <int NT>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* part) {
  v = wave_max(v);
  if constexpr (NT > 64) {
    constexpr int kWaves = NT / 64;
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v = max(v, part[w]);
  }
  return v;
}

// Codes of one row held as P pieces per lane, piece p at column
// (p * NT + lane) * 8.
template <int XF, int SL, int NT, int P, bool VEC>
__device__ __forceinline__ void quantize_row(float (*v)[kPiece], const RowsLaunch& a, uint64_t row, int lane,
                                             uint32_t* part) {
  uint8_t* codes_row = static_cast<uint8_t*>(a.codes) + row * a.codes_stride;
  if constexpr (SL == kScaleF32Row) {
    uint32_t amax = 0;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < kPiece; ++j) amax = max(amax, abs_bits(v[p][j]));
    amax = block_max<NT>(amax, part);
    float scale;
    const float mul = f32_multiplier(amax, CodeFormat<XF>::kMax, &scale);
#pragma unroll
    for (int p = 0; p < P; ++p)
      store_codes<VEC>(codes_row, (p * NT + lane) * kPiece, a.h, encode_piece<XF>(v[p], mul));
    if (lane == 0) static_cast<float*>(a.scales)[row] = scale;
  } else {
    const uint64_t first = row * (a.h / (SL == kScaleF32Group128 ? 128 : 32));
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * kPiece;
      quantize_group_piece<XF, SL, VEC>(v[p], c < a.h, c, a.h, codes_row, a.scales, first);
    }
  }
}

// NORM: the residual sum and norm in front of the codes; otherwise x itself
// is quantized. NT = 64 takes a row per wave and four rows per work-group;
// larger NT a row per work-group.
template <int IO, int SL, int NT, int P, bool VEC, bool NORM>
__global__ __launch_bounds__(NT == 64 ? 256 : NT) void rows_kernel(const RowsLaunch a) {
  __shared__ float sum_part[NT / 64];
  __shared__ uint32_t max_part[NT / 64];
  const int lane = NT == 64 ? threadIdx.x % 64 : threadIdx.x;
  const uint64_t row = NT == 64 ? static_cast<uint64_t>(blockIdx.x) * 4 + threadIdx.x / 64 : blockIdx.x;
  if (NT == 64 && row >= a.rows) return;  // whole waves; no barrier below for NT = 64
  constexpr int kSize = kOutSize<IO>;
  const char* x_row = static_cast<const char*>(a.x) + row * a.x_stride * kSize;

  float v[P][kPiece];
#pragma unroll
  for (int p = 0; p < P; ++p) load_piece<IO, VEC>(x_row, (p * NT + lane) * kPiece, a.h, v[p]);

  if constexpr (NORM) {
    if (a.residual != nullptr) {
      const char* r_row = static_cast<const char*>(a.residual) + row * a.residual_stride * kSize;
      char* s_row = static_cast<char*>(a.sum) + row * a.sum_stride * kSize;
      float r[P][kPiece];
#pragma unroll
      for (int p = 0; p < P; ++p) load_piece<IO, VEC>(r_row, (p * NT + lane) * kPiece, a.h, r[p]);
#pragma unroll
      for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[p][j] = round_to<IO>(v[p][j] + r[p][j]);
        store_piece<IO, VEC>(s_row, (p * NT + lane) * kPiece, a.h, v[p]);
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < kPiece; ++j) ss += v[p][j] * v[p][j];
    ss = block_sum<NT>(ss, sum_part);
    const float rstd = 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.h) + a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float w[kPiece];
      load_piece<IO, VEC>(a.weight, (p * NT + lane) * kPiece, a.h, w);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) v[p][j] = v[p][j] * rstd * w[j];
    }
  }

  if (a.x_format == kXE4M3FN) {
    quantize_row<kXE4M3FN, SL, NT, P, VEC>(v, a, row, lane, max_part);
  } else if (a.x_format == kXE5M2) {
    quantize_row<kXE5M2, SL, NT, P, VEC>(v, a, row, lane, max_part);
  } else if constexpr (SL != kScaleE8M0Block32) {
    quantize_row<kXInt8, SL, NT, P, VEC>(v, a, row, lane, max_part);
  }
}

// A HIP grid holds fewer than 2^32 work-items: at most 2^20 rows (2^30
// lanes) a launch.
constexpr uint64_t kMaxLaunchRows = uint64_t{1} << 20;

template <int IO, int SL, int NT, int P, bool VEC, bool NORM>
hipError_t launch_rows_as(const RowsLaunch& l, hipStream_t stream) {
  constexpr uint64_t per_block = NT == 64 ? 4 : 1;
  constexpr uint64_t size = kOutSize<IO>;
  const uint64_t scales_per_row = SL == kScaleF32Row ? 1 : l.h / (SL == kScaleF32Group128 ? 128 : 32);
  for (uint64_t r0 = 0; r0 < l.rows; r0 += kMaxLaunchRows) {
    RowsLaunch q = l;
    q.rows = l.rows - r0 < kMaxLaunchRows ? l.rows - r0 : kMaxLaunchRows;
    q.x = static_cast<const char*>(l.x) + r0 * l.x_stride * size;
    if (l.residual) {
      q.residual = static_cast<const char*>(l.residual) + r0 * l.residual_stride * size;
      q.sum = static_cast<char*>(l.sum) + r0 * l.sum_stride * size;
    }
    q.codes = static_cast<char*>(l.codes) + r0 * l.codes_stride;
    q.scales = static_cast<char*>(l.scales) + r0 * scales_per_row * (SL == kScaleE8M0Block32 ? 1 : 4);
    const hipError_t e =
        launch_kernel(rows_kernel<IO, SL, NT, P, VEC, NORM>, dim3(static_cast<uint32_t>((q.rows + per_block - 1) / per_block)),
                      dim3(NT == 64 ? 256 : NT), stream, q);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The smallest shape that holds a row.
template <int IO, int SL, bool VEC, bool NORM>
hipError_t launch_rows_sized(const RowsLaunch& l, hipStream_t stream) {
  if (l.h <= 256 * 4 * kPiece) return launch_rows_as<IO, SL, 256, 4, VEC, NORM>(l, stream);
  if (l.h <= 1024 * 8 * kPiece) return launch_rows_as<IO, SL, 1024, 8, VEC, NORM>(l, stream);
  return hipErrorInvalidValue;
}

template <int IO, int SL, bool NORM>
hipError_t launch_rows_typed(const RowsLaunch& l, hipStream_t stream) {
  return l.vec ? launch_rows_sized<IO, SL, true, NORM>(l, stream) : launch_rows_sized<IO, SL, false, NORM>(l, stream);
}

template <int IO>
hipError_t launch_rows_io(const RowsLaunch& l, hipStream_t stream) {
  if (!l.norm) return launch_rows_typed<IO, kScaleF32Row, false>(l, stream);
  switch (l.scale_layout) {
    case kScaleF32Group128: return launch_rows_typed<IO, kScaleF32Group128, true>(l, stream);
    case kScaleE8M0Block32: return launch_rows_typed<IO, kScaleE8M0Block32, true>(l, stream);
    case kScaleF32Row: return launch_rows_typed<IO, kScaleF32Row, true>(l, stream);
  }
  return hipErrorInvalidValue;
}

// ---- backward ----------------------------------------------------------

// With r = 1 / sqrt(mean(s^2) + eps) and d = weight * grad_y:
//   grad_x      = grad_sum + r * (d - s * (r^2 * mean(d * s)))
//   grad_weight = sum over tokens of grad_y * s * r
// Both row sums (s^2 and d * s) are taken in one reduction. Work-group b
// takes rows b, b + gridDim, ... and keeps its columns' share of grad_weight
// in registers; it leaves one row of partial sums in the workspace, and
// grad_weight_kernel adds those rows in order: a fixed order without atomics.
template <int IO, int NT, int P, bool VEC>
__global__ __launch_bounds__(NT) void norm_backward_kernel(const NormBackwardLaunch a) {
  __shared__ float parts[2][2 * (NT / 64)];
  const int lane = threadIdx.x;
  constexpr int kSize = kOutSize<IO>;
  float dw[P][kPiece];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < kPiece; ++j) dw[p][j] = 0.0f;

  int turn = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const char* dy_row = static_cast<const char*>(a.grad_y) + row * a.grad_y_stride * kSize;
    const char* s_row = static_cast<const char*>(a.sum) + row * a.sum_stride * kSize;
    float dy[P][kPiece], s[P][kPiece];
    float ss = 0.0f, ds = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * kPiece;
      float w[kPiece];
      load_piece<IO, VEC>(dy_row, c, a.h, dy[p]);
      load_piece<IO, VEC>(s_row, c, a.h, s[p]);
      load_piece<IO, VEC>(a.weight, c, a.h, w);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        ss += s[p][j] * s[p][j];
        ds += w[j] * dy[p][j] * s[p][j];
      }
    }
    // Alternating halves of `parts`: a wave that is a row ahead writes the
    // other half, and the next barrier keeps it from going further.
    ss = wave_sum(ss);
    ds = wave_sum(ds);
    constexpr int kWaves = NT / 64;
    if (lane % 64 == 0) {
      parts[turn][lane / 64] = ss;
      parts[turn][kWaves + lane / 64] = ds;
    }
    __syncthreads();
    ss = ds = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      ss += parts[turn][w];
      ds += parts[turn][kWaves + w];
    }
    const float n = static_cast<float>(a.h);
    const float r = 1.0f / __builtin_sqrtf(ss / n + a.eps);
    const float along = r * r * (ds / n);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * kPiece;
      float w[kPiece], g[kPiece];
      load_piece<IO, VEC>(a.weight, c, a.h, w);
      if (a.grad_sum != nullptr) {
        load_piece<IO, VEC>(static_cast<const char*>(a.grad_sum) + row * a.grad_sum_stride * kSize, c, a.h, g);
      } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) g[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        dw[p][j] += dy[p][j] * (s[p][j] * r);
        g[j] += r * (w[j] * dy[p][j] - s[p][j] * along);
      }
      store_piece<IO, VEC>(static_cast<char*>(a.grad_x) + row * a.grad_x_stride * kSize, c, a.h, g);
    }
  }
  float* part_row = a.workspace + static_cast<uint64_t>(blockIdx.x) * a.h;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t c = (p * NT + lane) * kPiece;
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
      if (c + j < a.h) part_row[c + j] = dw[p][j];
  }
}

// grad_weight[c] = sum over the n_parts rows of the workspace: 64 columns a
// work-group, its 16 waves taking every 16th row.
__global__ __launch_bounds__(1024) void grad_weight_kernel(const float* parts, float* grad_weight, uint32_t n_parts,
                                                           uint32_t h) {
  __shared__ float part[16][64];
  const uint32_t c = blockIdx.x * 64 + threadIdx.x % 64;
  const uint32_t w = threadIdx.x / 64;
  float v = 0.0f;
  if (c < h)
    for (uint32_t i = w; i < n_parts; i += 16) v += parts[static_cast<uint64_t>(i) * h + c];
  part[w][threadIdx.x % 64] = v;
  __syncthreads();
  if (w == 0 && c < h) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += part[i][threadIdx.x];
    grad_weight[c] = v;
  }
}

template <int IO, int NT, int P, bool VEC>
hipError_t launch_backward_as(const NormBackwardLaunch& l, hipStream_t stream) {
  const uint32_t parts = norm_backward_parts(l.rows);
  const hipError_t e = launch_kernel(norm_backward_kernel<IO, NT, P, VEC>, dim3(parts), dim3(NT), stream, l);
  if (e != hipSuccess) return e;
  return launch_kernel(grad_weight_kernel, dim3((l.h + 63) / 64), dim3(1024), stream,
                       static_cast<const float*>(l.workspace), l.grad_weight, parts, l.h);
}

template <int IO, bool VEC>
hipError_t launch_backward_sized(const NormBackwardLaunch& l, hipStream_t stream) {
  if (l.h <= 256 * 4 * kPiece) return launch_backward_as<IO, 256, 4, VEC>(l, stream);
  if (l.h <= 1024 * 8 * kPiece) return launch_backward_as<IO, 1024, 8, VEC>(l, stream);
  return hipErrorInvalidValue;
}

template <int IO>
hipError_t launch_backward_io(const NormBackwardLaunch& l, hipStream_t stream) {
  return l.vec ? launch_backward_sized<IO, true>(l, stream) : launch_backward_sized<IO, false>(l, stream);
}

}  // namespace

hipError_t launch_rows(const RowsLaunch& l, hipStream_t stream) {
  switch (l.io_format) {
    case kOutF32: return launch_rows_io<kOutF32>(l, stream);
    case kOutBF16: return launch_rows_io<kOutBF16>(l, stream);
    case kOutF16: return launch_rows_io<kOutF16>(l, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_norm_backward(const NormBackwardLaunch& l, hipStream_t stream) {
  switch (l.io_format) {
    case kOutF32: return launch_backward_io<kOutF32>(l, stream);
    case kOutBF16: return launch_backward_io<kOutBF16>(l, stream);
    case kOutF16: return launch_backward_io<kOutF16>(l, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace qrs
