// gfx950 kernels of the layer norm over rows of activations: residual sum,
// norm, codes and scales, and the norm's backward pass.
//
//   s = x + residual                   (rounded to the activations' type)
//   mean, var of s along the row;  r = 1 / sqrt(var + eps)
//   y = (s - mean) * r * weight + bias (binary32)
//   codes, scales = quantize(y)
//
// A row stays in the registers of one work-group from its load to its codes:
// one pass over memory, bound by HBM.
//
// Mean and variance come from one reduction. A wave adds d = s - s0 and d^2 in
// binary64, s0 being the first of its own elements. Then the mean of d, squared,
// is at most n - 1 times the variance of its n elements (s0, one of them, is that
// far from the mean), so what sum d^2 - (sum d)^2 / n cancels is at most a factor
// of n <= 65536, and it keeps 53 - 16 bits whatever the mean, the size of the
// values or the outliers. The waves' means and sums of squares about them are then
// joined exactly as their definition says.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qrs_device.h"
#include "qrs_layer.h"
#include "qrs_rows_device.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace {

using namespace dev;

// How many of a row's h elements the wave of `lane` holds: piece p of a lane is
// at column (p * NT + lane) * E.
template <int NT, int P, int E>
__device__ __forceinline__ uint32_t wave_count(uint32_t lane, uint32_t h) {
  uint32_t n = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t first = (p * NT + (lane & ~63u)) * E;
    n += min(max(h, first) - first, 64u * E);
  }
  return n;
}

__device__ __forceinline__ float first_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// Sums of d = s - s0 and d^2 over a wave's elements, n of them and inv_n = 1 / n,
// -> their mean and the sum of squares about it (zeros of no elements, with
// inv_n = 0).
struct WaveMoments {
  double mean, squares;
};
__device__ __forceinline__ WaveMoments wave_moments(float s0, double d1, double d2, double inv_n) {
  const double dm = d1 * inv_n;
  return {s0 + dm, d2 - d1 * dm};
}

// A row's mean, as a float and what that leaves, and 1 / sqrt(var + eps).
struct Moments {
  double mean, r, m;  // m = var + eps
  float mean_hi, mean_lo, r32;

  __device__ __forceinline__ void finish(double mean64, double squares, double inv_h, float eps) {
    mean = mean64;
    m = squares * inv_h + static_cast<double>(eps);
    r = inverse_root(m);
    mean_hi = static_cast<float>(mean);
    mean_lo = static_cast<float>(mean - mean_hi);
    r32 = static_cast<float>(r);
  }
  // Whether binary32 does not hold what follows.
  __device__ __forceinline__ bool wide() const {
    return !(m > 0x1p-100 && m < 0x1p100 && __builtin_fabs(mean) < 0x1p100);
  }
  // s - mean: off by two roundings of itself, however large the mean is.
  __device__ __forceinline__ float centred(float s) const { return (s - mean_hi) - mean_lo; }
};

// ---- forward -----------------------------------------------------------

// A format as a type.
template <int XF>
struct Format {
  static constexpr int value = XF;
};

// Codes of a piece of y, whose group of G elements lies in the G / E lanes
// around it (or in the row, with the multiplier given).
template <int SL, int XF, int E>
__device__ __forceinline__ Codes<E> encode_y(const float* y, float mul, uint32_t* scale_bits) {
  if constexpr (SL == kScaleE8M0Block32) {
    mul = mx_multiplier<XF>(group_max<32 / E>(piece_max<E>(y)), scale_bits);
  } else if constexpr (SL == kScaleF32Group128) {
    float scale;
    mul = f32_multiplier(group_max<128 / E>(piece_max<E>(y)), CodeFormat<XF>::kMax, &scale);
    *scale_bits = __builtin_bit_cast(uint32_t, scale);
  }
  return encode_piece<XF, E>(y, mul);
}

// Work-group b takes rows b, b + gridDim, ...; the next row's operands are
// under way while a row is reduced and written.
//
// y takes four roundings of its product (s - mean: two, r, (s - mean) * r) and
// one of the sum with the bias: |error| <= 2^-24 (4.1 |y - bias| + |y|). Rows
// whose variance or mean leaves the range above are taken in binary64.
template <int IO, int SL, int NT, int P8, bool VEC, bool STREAM>
__global__ __launch_bounds__(NT) void layer_norm_kernel(const LayerNormLaunch a) {
  constexpr int E = kPiece16<IO>, P = P8 * 8 / E;  // P8: 8 elements a lane
  constexpr int kWaves = NT / 64;
  __shared__ double part[2][kWaves][2], count[kWaves];
  __shared__ uint32_t max_part[2][kWaves];
  const int lane = threadIdx.x;
  constexpr int kSize = kOutSize<IO>;
  typedef RawPiece<IO, VEC> Raw;
  struct Operands {
    Raw x[P], r[P];
  };
  Operands next;
  Raw w[P], b[P];
  const bool add = a.residual != nullptr;
  auto load_row = [&](uint64_t row) {
    const char* x_row = static_cast<const char*>(a.x) + row * a.x_stride * kSize;
#pragma unroll
    for (int p = 0; p < P; ++p) next.x[p].template load<STREAM>(x_row, (p * NT + lane) * E, a.h);
    if (add) {
      const char* r_row = static_cast<const char*>(a.residual) + row * a.residual_stride * kSize;
#pragma unroll
      for (int p = 0; p < P; ++p) next.r[p].template load<STREAM>(r_row, (p * NT + lane) * E, a.h);
    }
  };
  constexpr bool kAhead = P8 <= 4;  // wider rows leave no registers for a second one
  if (kAhead) load_row(blockIdx.x);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    w[p].template load<false>(a.weight, (p * NT + lane) * E, a.h);
    b[p].template load<false>(a.bias, (p * NT + lane) * E, a.bias != nullptr ? a.h : 0);  // no bias: zeros
  }
  const uint32_t mine = wave_count<NT, P, E>(lane, a.h);
  const double inv_mine = mine == 0 ? 0.0 : 1.0 / mine;
  if (lane % 64 == 0) count[lane / 64] = mine;  // read behind the first row's barrier

  // The parts of the reductions alternate between two halves: a wave that is
  // a row ahead writes the other half, and the next barrier keeps it from
  // going further.
  int turn = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    if (!kAhead) load_row(row);
    const Operands now = next;
    if (kAhead && row + gridDim.x < a.rows) load_row(row + gridDim.x);
    float s[P][E];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      now.x[p].get(s[p]);
      if (add) {
        float r[E];
        now.r[p].get(r);
#pragma unroll
        for (int j = 0; j < E; ++j) s[p][j] = round_to<IO>(s[p][j] + r[j]);
        store_piece<IO, VEC, E>(static_cast<char*>(a.sum) + row * a.sum_stride * kSize, (p * NT + lane) * E, a.h, s[p]);
      }
    }
    const float s0 = first_lane(s[0][0]);
    double d1 = 0.0, d2 = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * E;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const bool in = VEC ? c < a.h : c + j < a.h;
        const double d = in ? static_cast<double>(s[p][j]) - s0 : 0.0;
        d1 += d;
        d2 = __builtin_fma(d, d, d2);
      }
    }
    const WaveMoments wm = wave_moments(s0, wave_sum(d1), wave_sum(d2), inv_mine);
    if (lane % 64 == 0) {
      part[turn][lane / 64][0] = wm.mean;
      part[turn][lane / 64][1] = wm.squares;
    }
    lds_barrier();
    double mean = 0.0, squares = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) mean += count[i] * part[turn][i][0];
    mean *= a.inv_h;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const double d = part[turn][i][0] - mean;
      squares += __builtin_fma(count[i] * d, d, part[turn][i][1]);
    }
    Moments mo;
    mo.finish(mean, squares, a.inv_h, a.eps);
    const bool wide = mo.wide();  // the same in every lane

    // y over s.
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * E;
      float wv[E], bv[E];
      w[p].get(wv);
      b[p].get(bv);
      if (__builtin_expect(wide, false)) {
#pragma unroll
        for (int j = 0; j < E; ++j)
          s[p][j] = static_cast<float>((static_cast<double>(s[p][j]) - mo.mean) * mo.r * wv[j] + bv[j]);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) s[p][j] = __builtin_fmaf(mo.centred(s[p][j]) * mo.r32, wv[j], bv[j]);
      }
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (!(VEC ? c < a.h : c + j < a.h)) s[p][j] = 0.0f;
    }
    uint32_t amax = 0;
    if constexpr (SL == kScaleF32Row) {
#pragma unroll
      for (int p = 0; p < P; ++p) amax = max(amax, piece_max<E>(s[p]));
      amax = wave_max(amax);
      if (lane % 64 == 0) max_part[turn][lane / 64] = amax;
      lds_barrier();
#pragma unroll
      for (int i = 0; i < kWaves; ++i) amax = max(amax, max_part[turn][i]);
    }
    auto write = [&](auto format) {
      constexpr int XF = decltype(format)::value;
      uint8_t* codes_row = static_cast<uint8_t*>(a.codes) + row * a.codes_stride;
      float mul = 0.0f;
      if constexpr (SL == kScaleF32Row) {
        float scale;
        mul = f32_multiplier(amax, CodeFormat<XF>::kMax, &scale);
        if (lane == 0) static_cast<float*>(a.scales)[row] = scale;
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t c = (p * NT + lane) * E;
        uint32_t scale;
        store_codes<VEC, E>(codes_row, c, a.h, encode_y<SL, XF, E>(s[p], mul, &scale));
        if (SL == kScaleE8M0Block32 && c < a.h && c % 32 == 0)
          static_cast<uint8_t*>(a.scales)[row * (a.h / 32) + c / 32] = static_cast<uint8_t>(scale);
        if (SL == kScaleF32Group128 && c < a.h && c % 128 == 0)
          static_cast<uint32_t*>(a.scales)[row * (a.h / 128) + c / 128] = scale;
      }
    };
    if (a.x_format == kXE4M3FN) {
      write(Format<kXE4M3FN>{});
    } else if (a.x_format == kXE5M2) {
      write(Format<kXE5M2>{});
    } else if constexpr (SL != kScaleE8M0Block32) {
      write(Format<kXInt8>{});
    }
  }
}

template <int IO, int SL, int NT, int P, bool VEC, bool STREAM>
hipError_t launch_norm_as(const LayerNormLaunch& l, hipStream_t stream) {
  const uint32_t blocks = NT * P <= 512 ? 4096 : NT < 1024 ? 512 : 256;
  return launch_kernel(layer_norm_kernel<IO, SL, NT, P, VEC, STREAM>,
                       dim3(static_cast<uint32_t>(l.rows < blocks ? l.rows : blocks)), dim3(NT), stream, l);
}

// The smallest shape that holds a row; rows off 16-byte boundaries have two.
template <int IO, int SL, bool VEC, bool STREAM>
hipError_t launch_norm_sized(const LayerNormLaunch& l, hipStream_t stream) {
  if constexpr (VEC) {
    if (l.h <= 256 * 1 * kPiece) return launch_norm_as<IO, SL, 256, 1, VEC, STREAM>(l, stream);
    if (l.h <= 512 * 1 * kPiece) return launch_norm_as<IO, SL, 512, 1, VEC, STREAM>(l, stream);
  }
  if (l.h <= 512 * 2 * kPiece) return launch_norm_as<IO, SL, 512, 2, VEC, STREAM>(l, stream);
  if constexpr (VEC)
    if (l.h <= 1024 * 2 * kPiece) return launch_norm_as<IO, SL, 1024, 2, VEC, STREAM>(l, stream);
  if (l.h <= 1024 * 8 * kPiece) return launch_norm_as<IO, SL, 1024, 8, VEC, STREAM>(l, stream);
  return hipErrorInvalidValue;
}

template <int IO, int SL>
hipError_t launch_norm_typed(const LayerNormLaunch& l, hipStream_t stream) {
  if (!l.vec) return launch_norm_sized<IO, SL, false, false>(l, stream);
  return l.rows * l.h * (kOutSize<IO> * 3 + 1) > kStreamBytes ? launch_norm_sized<IO, SL, true, true>(l, stream)
                                                              : launch_norm_sized<IO, SL, true, false>(l, stream);
}

template <int IO>
hipError_t launch_norm_io(const LayerNormLaunch& l, hipStream_t stream) {
  switch (l.scale_layout) {
    case kScaleF32Group128: return launch_norm_typed<IO, kScaleF32Group128>(l, stream);
    case kScaleE8M0Block32: return launch_norm_typed<IO, kScaleE8M0Block32>(l, stream);
    case kScaleF32Row: return launch_norm_typed<IO, kScaleF32Row>(l, stream);
  }
  return hipErrorInvalidValue;
}

// ---- backward ----------------------------------------------------------

// With u = (s - mean) * r and d = weight * grad_y:
//   grad_x      = grad_sum + r * (d - mean(d) - u * mean(d * u))
//   grad_weight = sum over tokens of grad_y * u
//   grad_bias   = sum over tokens of grad_y
// One reduction a row: beside the moments of s, the sums of d and of d times s's
// distance from the wave's own mean, in binary64; joining the waves moves the
// latter to the row's mean.
//
// Work-group b takes rows b, b + gridDim, ...; the next row's operands are under
// way while a row is reduced and written. It keeps its columns' shares of
// grad_weight and grad_bias in registers and leaves one row of partial sums in
// the workspace, and grad_params_kernel adds those rows in order: a fixed order
// without atomics.
template <int IO, int NT, int P8, bool VEC, bool STREAM>
__global__ __launch_bounds__(NT) void layer_norm_backward_kernel(const LayerNormBackwardLaunch a) {
  constexpr int kWaves = NT / 64;
  __shared__ double part[2][kWaves][4], count[kWaves];
  constexpr int E = kPiece16<IO>, P = P8 * 8 / E;
  const int lane = threadIdx.x;
  constexpr int kSize = kOutSize<IO>;
  typedef RawPiece<IO, VEC> Raw;
  float dw[P][E], db[P][E];
  Raw w[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    w[p].template load<false>(a.weight, (p * NT + lane) * E, a.h);
#pragma unroll
    for (int j = 0; j < E; ++j) dw[p][j] = db[p][j] = 0.0f;
  }
  struct Operands {
    Raw dy[P], s[P], g[P];
  };
  Operands next;
  auto load_row = [&](uint64_t row) {
    const char* dy_row = static_cast<const char*>(a.grad_y) + row * a.grad_y_stride * kSize;
    const char* s_row = static_cast<const char*>(a.sum) + row * a.sum_stride * kSize;
    // Without a grad_sum, s stands in and is taken as zero below.
    const char* g_row = a.grad_sum != nullptr ? static_cast<const char*>(a.grad_sum) + row * a.grad_sum_stride * kSize : s_row;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * E;
      next.dy[p].template load<STREAM>(dy_row, c, a.h);
      next.s[p].template load<STREAM>(s_row, c, a.h);
      next.g[p].template load<STREAM>(g_row, c, a.h);
    }
  };

  constexpr bool kAhead = P8 <= 4;  // wider rows leave no registers for a second one
  if (kAhead) load_row(blockIdx.x);
  const bool keep = a.grad_sum != nullptr;
  const uint32_t mine = wave_count<NT, P, E>(lane, a.h);
  const double inv_mine = mine == 0 ? 0.0 : 1.0 / mine;
  if (lane % 64 == 0) count[lane / 64] = mine;  // read behind the first row's barrier
  int turn = 0;  // halves of `part`, as in the forward pass
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    if (!kAhead) load_row(row);
    const Operands now = next;
    if (kAhead && row + gridDim.x < a.rows) load_row(row + gridDim.x);
    float first[E];
    now.s[0].get(first);
    const float s0 = first_lane(first[0]);
    double d1 = 0.0, d2 = 0.0, g1 = 0.0, gd = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * E;
      float wv[E], dy[E], s[E];
      w[p].get(wv);
      now.dy[p].get(dy);
      now.s[p].get(s);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const bool in = VEC ? c < a.h : c + j < a.h;
        const double d = in ? static_cast<double>(s[j]) - s0 : 0.0;
        const double g = wv[j] * dy[j];  // zero past the row's end
        d1 += d;
        d2 = __builtin_fma(d, d, d2);
        g1 += g;
        gd = __builtin_fma(g, d, gd);
      }
    }
    d1 = wave_sum(d1);
    g1 = wave_sum(g1);
    const WaveMoments wm = wave_moments(s0, d1, wave_sum(d2), inv_mine);
    gd = wave_sum(gd);
    if (lane % 64 == 0) {
      double* to = part[turn][lane / 64];
      to[0] = wm.mean;
      to[1] = wm.squares;
      to[2] = g1;
      to[3] = gd - g1 * (d1 * inv_mine);
    }
    lds_barrier();
    double mean = 0.0, squares = 0.0, sum_d = 0.0, sum_du = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) mean += count[i] * part[turn][i][0];
    mean *= a.inv_h;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const double d = part[turn][i][0] - mean;
      squares += __builtin_fma(count[i] * d, d, part[turn][i][1]);
      sum_d += part[turn][i][2];
      sum_du += __builtin_fma(part[turn][i][2], d, part[turn][i][3]);
    }
    Moments mo;
    mo.finish(mean, squares, a.inv_h, a.eps);
    const double mean_d = sum_d * a.inv_h, mean_du = sum_du * a.inv_h * mo.r;
    const bool wide = mo.wide() || !(__builtin_fabs(mean_d) < 0x1p100 && __builtin_fabs(mean_du) < 0x1p100);
    const float mean_d32 = static_cast<float>(mean_d), mean_du32 = static_cast<float>(mean_du);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * E;
      float wv[E], dy[E], s[E], g[E];
      w[p].get(wv);
      now.dy[p].get(dy);
      now.s[p].get(s);
      now.g[p].get(g);
#pragma unroll
      for (int j = 0; j < E; ++j) g[j] = keep ? g[j] : 0.0f;
      if (__builtin_expect(wide, false)) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const double u = (static_cast<double>(s[j]) - mo.mean) * mo.r;
          dw[p][j] += static_cast<float>(dy[j] * u);
          g[j] = static_cast<float>(g[j] + mo.r * (static_cast<double>(wv[j]) * dy[j] - mean_d - u * mean_du));
        }
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const float u = mo.centred(s[j]) * mo.r32;
          dw[p][j] = __builtin_fmaf(dy[j], u, dw[p][j]);
          g[j] = __builtin_fmaf(mo.r32, __builtin_fmaf(-u, mean_du32, __builtin_fmaf(wv[j], dy[j], -mean_d32)), g[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < E; ++j) db[p][j] += dy[j];
      store_piece<IO, VEC, E>(static_cast<char*>(a.grad_x) + row * a.grad_x_stride * kSize, c, a.h, g);
    }
  }
  float* part_row = a.workspace + static_cast<uint64_t>(blockIdx.x) * 2 * a.h;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t c = (p * NT + lane) * E;
    if (VEC && c < a.h) {
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        *reinterpret_cast<f32x4*>(part_row + c + j) = f32x4{dw[p][j], dw[p][j + 1], dw[p][j + 2], dw[p][j + 3]};
        *reinterpret_cast<f32x4*>(part_row + a.h + c + j) = f32x4{db[p][j], db[p][j + 1], db[p][j + 2], db[p][j + 3]};
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (c + j < a.h) {
          part_row[c + j] = dw[p][j];
          part_row[a.h + c + j] = db[p][j];
        }
    }
  }
}

// Columns of the workspace's n_parts rows [grad_weight | grad_bias] added: 32
// columns (a line of each row) a work-group, its 32 half waves taking every 32nd
// row.
__global__ __launch_bounds__(1024) void grad_params_kernel(const float* parts, float* grad_weight, float* grad_bias,
                                                           uint32_t n_parts, uint32_t h) {
  __shared__ float part[32][33];
  const uint32_t col = threadIdx.x % 32, c = blockIdx.x * 32 + col, w = threadIdx.x / 32;
  float v = 0.0f;
  if (c < 2 * h) {
#pragma unroll 4
    for (uint32_t i = w; i < n_parts; i += 32) v += parts[static_cast<uint64_t>(i) * 2 * h + c];
  }
  part[w][col] = v;
  __syncthreads();
  if (w == 0 && c < 2 * h) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += part[i][col];
    if (c < h)
      grad_weight[c] = v;
    else if (grad_bias != nullptr)
      grad_bias[c - h] = v;
  }
}

template <int IO, int NT, int P, bool VEC, bool STREAM>
hipError_t launch_backward_as(const LayerNormBackwardLaunch& l, hipStream_t stream) {
  const uint32_t parts = layer_norm_backward_parts(l.rows, l.h);
  const hipError_t e =
      launch_kernel(layer_norm_backward_kernel<IO, NT, P, VEC, STREAM>, dim3(parts), dim3(NT), stream, l);
  if (e != hipSuccess) return e;
  return launch_kernel(grad_params_kernel, dim3((2 * l.h + 31) / 32), dim3(1024), stream,
                       static_cast<const float*>(l.workspace), l.grad_weight, l.grad_bias, parts, l.h);
}

// The smallest shape that holds a row, as above.
template <int IO, bool VEC, bool STREAM>
hipError_t launch_backward_sized(const LayerNormBackwardLaunch& l, hipStream_t stream) {
  if constexpr (VEC) {
    if (l.h <= 256 * 1 * kPiece) return launch_backward_as<IO, 256, 1, VEC, STREAM>(l, stream);
    if (l.h <= 256 * 2 * kPiece) return launch_backward_as<IO, 256, 2, VEC, STREAM>(l, stream);
  }
  if (l.h <= 256 * 4 * kPiece) return launch_backward_as<IO, 256, 4, VEC, STREAM>(l, stream);
  if constexpr (VEC)
    if (l.h <= 512 * 4 * kPiece) return launch_backward_as<IO, 512, 4, VEC, STREAM>(l, stream);
  if (l.h <= 1024 * 8 * kPiece) return launch_backward_as<IO, 1024, 8, VEC, STREAM>(l, stream);
  return hipErrorInvalidValue;
}

template <int IO>
hipError_t launch_backward_io(const LayerNormBackwardLaunch& l, hipStream_t stream) {
  if (!l.vec) return launch_backward_sized<IO, false, false>(l, stream);
  return l.rows * l.h * kOutSize<IO> * 4 > kStreamBytes ? launch_backward_sized<IO, true, true>(l, stream)
                                                        : launch_backward_sized<IO, true, false>(l, stream);
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormLaunch& l, hipStream_t stream) {
  switch (l.io_format) {
    case kOutF32: return launch_norm_io<kOutF32>(l, stream);
    case kOutBF16: return launch_norm_io<kOutBF16>(l, stream);
    case kOutF16: return launch_norm_io<kOutF16>(l, stream);
  }
  return hipErrorInvalidValue;
}

uint32_t layer_norm_backward_parts(uint64_t rows, uint32_t h) {
  const uint32_t parts = h <= 256 * kPiece && rows >= 4 * 512 ? 512 : 256;
  return static_cast<uint32_t>(rows < parts ? rows : parts);
}

hipError_t launch_layer_norm_backward(const LayerNormBackwardLaunch& l, hipStream_t stream) {
  switch (l.io_format) {
    case kOutF32: return launch_backward_io<kOutF32>(l, stream);
    case kOutBF16: return launch_backward_io<kOutBF16>(l, stream);
    case kOutF16: return launch_backward_io<kOutF16>(l, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace qrs
