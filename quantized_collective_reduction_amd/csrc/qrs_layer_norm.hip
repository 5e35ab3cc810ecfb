// gfx950 kernels of the layer norm over rows of activations: residual sum,
// norm, codes and scales, and the norm's backward pass.
//
//   s = x + residual                   (rounded to the activations' type)
//   mean, var of s along the row;  r = 1 / sqrt(var + eps)
//   y = (s - mean) * r * weight + bias (rounded to binary32)
//   codes, scales = quantize(y)
//
// A row stays in the registers of one work-group from its load to its codes:
// one pass over memory. The binary64 operations, 42 to 56 vector instructions for
// each element of a lane, take about as long as it: bf16 16384 x 8192 with E4M3FN
// codes 169 us (5.6 TB/s; without them, in a norm by squares alone, 147), 8192 x 5120
// fp32 93 us (5.9); the first one's gradient 188 us (5.7).
//
// Mean and variance come from one reduction. A wave adds d = s - s0 and d^2 in
// binary64, s0 being the first of its own elements. Then the mean of d, squared,
// is at most n - 1 times the variance of its n elements (s0, one of them, is that
// far from the mean), so what sum d^2 - (sum d)^2 / n cancels is at most a factor
// of n <= 65536, and it keeps 53 - 16 bits whatever the mean, the size of the
// values or the outliers. The waves are then joined by their distances from the first
// one's s0, exactly as the definition says: no value as large as the mean is added or
// multiplied by 1 / h, and in a row of equal values every distance is zero.

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
// -> the mean of d and the sum of squares about it (zeros of no elements, with
// inv_n = 0).
struct WaveMoments {
  double dm, squares;
};
__device__ __forceinline__ WaveMoments wave_moments(double d1, double d2, double inv_n) {
  const double dm = d1 * inv_n;
  return {dm, d2 - d1 * dm};
}

// Sum over each row of 16 lanes, in a fixed order, in every lane of it.
__device__ __forceinline__ double sum16(double v) {
  v += lanes(v, [](uint32_t x) { return dpp<kDppSwap1>(x); });
  v += lanes(v, [](uint32_t x) { return dpp<kDppSwap2>(x); });
  v += lanes(v, [](uint32_t x) { return dpp<kDppHalfMirror>(x); });
  return v + lanes(v, [](uint32_t x) { return dpp<kDppMirror>(x); });
}

// A row's mean, as a value s0 of the row and its distance from that, and as a
// float and what that leaves, and 1 / sqrt(var + eps).
struct Moments {
  double distance, r, m;  // m = var + eps
  float s0, mean_hi, mean_lo, r32;

  __device__ __forceinline__ void finish(float first, double from_first, double squares, double inv_h, float eps) {
    s0 = first;
    distance = from_first;
    m = squares * inv_h + static_cast<double>(eps);
    r = inverse_root(m);
    mean_hi = static_cast<float>(s0 + distance);
    mean_lo = static_cast<float>((static_cast<double>(s0) - mean_hi) + distance);
    r32 = static_cast<float>(r);
  }
  // Whether binary32 does not hold what follows. mean_lo is off by 2^-49 of the mean:
  // at most 2^-33 deviations while these are more than 2^-16 of the mean.
  __device__ __forceinline__ bool wide() const {
    const double mean = mean_hi;
    return !(m > 0x1p-100 && m < 0x1p100 && __builtin_fabs(mean) < 0x1p100 && m > mean * mean * 0x1p-32);
  }
  // s - mean: off by two roundings of itself, and 2^-33 deviations.
  __device__ __forceinline__ float centred(float s) const { return (s - mean_hi) - mean_lo; }
  // (s - mean) * r, however large the mean is.
  __device__ __forceinline__ double unit(float s) const {
    return ((static_cast<double>(s) - s0) - distance) * r;
  }
};

// Whether binary32 holds values of about this size, and a few bits less, as normal numbers.
__device__ __forceinline__ bool in_range(double v) {
  return __builtin_fabs(v) >= 0x1p-100 && __builtin_fabs(v) < 0x1p100;
}

// ---- forward -----------------------------------------------------------

// A format as a type.
template <int XF>
struct Format {
  static constexpr int value = XF;
};

// Codes of a piece of y, whose group of elements lies in the lanes around it (or
// in the row, with the multiplier given).
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
// y is computed in binary64 and rounded once to binary32, so that its codes are
// those of the formula but where binary64 itself could not tell: the operations
// fit beside the stream.
template <int IO, int SL, int NT, int P8, bool VEC, bool STREAM>
__global__ __launch_bounds__(NT) void layer_norm_kernel(const LayerNormLaunch a) {
  constexpr int E = kPiece16<IO>, P = P8 * 8 / E;  // P8: 8 elements a lane
  constexpr int kWaves = NT / 64;
  __shared__ double part[2][kWaves][3], count[kWaves];
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
        if (!(VEC ? c < a.h : c + j < a.h)) continue;
        const double d = static_cast<double>(s[p][j]) - s0;
        d1 += d;
        d2 = __builtin_fma(d, d, d2);
      }
    }
    const WaveMoments wm = wave_moments(wave_sum(d1), wave_sum(d2), inv_mine);
    if (lane % 64 == 0) {
      double* to = part[turn][lane / 64];
      to[0] = s0;
      to[1] = wm.dm;
      to[2] = wm.squares;
    }
    lds_barrier();
    // Lane l joins wave l % 16's part, from the first wave's s0 on.
    const int i = lane % 16;
    const double first = part[turn][0][0];
    double n = 0.0, far = 0.0, wave_squares = 0.0;
    if (i < kWaves) {
      n = count[i];
      far = (part[turn][i][0] - first) + part[turn][i][1];
      wave_squares = part[turn][i][2];
    }
    const double distance = sum16(n * far) * a.inv_h, off = far - distance;
    const double squares = sum16(__builtin_fma(n * off, off, wave_squares));
    const double r = inverse_root(squares * a.inv_h + static_cast<double>(a.eps)), shift = -distance * r;

    // y over s.
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * E;
      float wv[E], bv[E];
      if (VEC && c >= a.h) continue;  // zeros, like the weight and the bias
      if (IO != kOutF32) {
        // Unpacked and converted again: kept, they would cost the registers of more
        // waves (bf16 16384 x 8192 179 us, renewed 170; fp32 8192 x 5120 92 and 106).
        as_new(s[p]);
        w[p].renew();
        b[p].renew();
      }
      w[p].get(wv);
      b[p].get(bv);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const double u = __builtin_fma(static_cast<double>(s[p][j]) - first, r, shift);
        const float y = static_cast<float>(__builtin_fma(u, static_cast<double>(wv[j]), static_cast<double>(bv[j])));
        s[p][j] = VEC || c + j < a.h ? y : 0.0f;
      }
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
        uint32_t scale = 0;
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
hipError_t launch_norm_as(const LayerNormLaunch& l, uint32_t blocks, hipStream_t stream) {
  return launch_kernel(layer_norm_kernel<IO, SL, NT, P, VEC, STREAM>,
                       dim3(static_cast<uint32_t>(l.rows < blocks ? l.rows : blocks)), dim3(NT), stream, l);
}

// The smallest shape that holds a row, 16 elements a lane where registers allow:
// few waves a row, which each pay for the reductions. Work-groups that even out by
// themselves, but for binary32 in 768 lanes as many as run at once. us: bf16
// 16384 x 1024 128 x 1 28, 256 x 2 58; 8192 x 4096 256 x 2 45, 512 x 1 50; 16384 x 8192
// 512 x 2 in 256, 512 and 2048 work-groups 202, 178 and 170, 256 x 4 213; 4096 x 7168
// 52, 45 and 44; fp32 8192 x 5120 768 x 1 in 256 and 4096 92 and 110, 512 x 2 96 and 128.
// Rows off 16-byte boundaries have two shapes. Scratch memory takes part of the rows of
// 1024 x 2 lanes of binary32 and of 1024 x 8 (fp32 2048 x 16384 130 us, 3.4 TB/s; bf16
// 1024 x 32768 151, 1.6; off boundaries 4096 x 8191 178, 1.3, 2048 x 16383 1129, 0.2).
template <int IO, int SL, bool VEC, bool STREAM>
hipError_t launch_norm_sized(const LayerNormLaunch& l, hipStream_t stream) {
  if constexpr (VEC) {
    if (l.h <= 128 * 1 * kPiece) return launch_norm_as<IO, SL, 128, 1, VEC, STREAM>(l, 2048, stream);
    if (l.h <= 128 * 2 * kPiece) return launch_norm_as<IO, SL, 128, 2, VEC, STREAM>(l, 2048, stream);
    if (l.h <= 256 * 2 * kPiece) return launch_norm_as<IO, SL, 256, 2, VEC, STREAM>(l, 2048, stream);
    if constexpr (IO == kOutF32)
      if (l.h <= 768 * 1 * kPiece) return launch_norm_as<IO, SL, 768, 1, VEC, STREAM>(l, 256, stream);
  }
  if (l.h <= 512 * 2 * kPiece)
    return launch_norm_as<IO, SL, 512, 2, VEC, STREAM>(l, IO == kOutF32 ? 256 : 2048, stream);
  if constexpr (VEC)
    if (l.h <= 1024 * 2 * kPiece) return launch_norm_as<IO, SL, 1024, 2, VEC, STREAM>(l, 256, stream);
  if (l.h <= 1024 * 8 * kPiece) return launch_norm_as<IO, SL, 1024, 8, VEC, STREAM>(l, 256, stream);
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
//
// Two waves a SIMD where a lane has 16 elements at most: 256 registers, of which binary32
// would take a few more.
template <int IO, int NT, int P8, bool VEC, bool STREAM>
__global__ __launch_bounds__(NT, P8 <= 2 ? 2 : 1) void layer_norm_backward_kernel(const LayerNormBackwardLaunch a) {
  constexpr int kWaves = NT / 64;
  __shared__ double part[2][kWaves][5], count[kWaves];
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
    const char* g_row = s_row;
    if (a.grad_sum != nullptr) g_row = static_cast<const char*>(a.grad_sum) + row * a.grad_sum_stride * kSize;
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
    Operands now = next;
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
        if (!(VEC ? c < a.h : c + j < a.h)) continue;
        const double d = static_cast<double>(s[j]) - s0;
        const double g = wv[j] * dy[j];
        d1 += d;
        d2 = __builtin_fma(d, d, d2);
        g1 += g;
        gd = __builtin_fma(g, d, gd);
      }
    }
    d1 = wave_sum(d1);
    g1 = wave_sum(g1);
    // A wave's products that may have left binary32's range are made again in binary64,
    // unless there is no gradient (half precision's cannot; all of them in binary64 16384
    // x 8192 bf16 195 us, so 190). Loaded once more, the operands cost other rows no
    // registers.
    if (IO != kOutF16 && __builtin_expect(!in_range(g1), false)) {
      uint32_t any = 0;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float dy[E];
        now.dy[p].get(dy);
#pragma unroll
        for (int j = 0; j < E; ++j) any |= abs_bits(dy[j]);
      }
      if (__ballot(any != 0) != 0) {
        g1 = gd = 0.0;
#pragma unroll 1
        for (int p = 0; p < P; ++p) {
          const uint32_t c = (p * NT + lane) * E;
          float wv[E], dy[E], s[E];
          load_piece<IO, VEC, E>(a.weight, c, a.h, wv);
          load_piece<IO, VEC, E>(static_cast<const char*>(a.grad_y) + row * a.grad_y_stride * kSize, c, a.h, dy);
          load_piece<IO, VEC, E>(static_cast<const char*>(a.sum) + row * a.sum_stride * kSize, c, a.h, s);
#pragma unroll
          for (int j = 0; j < E; ++j) {
            if (!(VEC ? c < a.h : c + j < a.h)) continue;
            const double g = static_cast<double>(wv[j]) * dy[j];
            g1 += g;
            gd = __builtin_fma(g, static_cast<double>(s[j]) - s0, gd);
          }
        }
        g1 = wave_sum(g1);
      }
    }
    const WaveMoments wm = wave_moments(d1, wave_sum(d2), inv_mine);
    gd = wave_sum(gd);
    if (lane % 64 == 0) {
      double* to = part[turn][lane / 64];
      to[0] = s0;
      to[1] = wm.dm;
      to[2] = wm.squares;
      to[3] = g1;
      to[4] = gd - g1 * wm.dm;
    }
    lds_barrier();
    const int i = lane % 16;
    const float row_first = static_cast<float>(part[turn][0][0]);
    double n = 0.0, far = 0.0, all[3] = {0.0, 0.0, 0.0};  // of wave i
    if (i < kWaves) {
      n = count[i];
      far = (part[turn][i][0] - row_first) + part[turn][i][1];
#pragma unroll
      for (int e = 0; e < 3; ++e) all[e] = part[turn][i][2 + e];
    }
    const double distance = sum16(n * far) * a.inv_h, off = far - distance;
    const double squares = sum16(__builtin_fma(n * off, off, all[0])), sum_d = sum16(all[1]);
    const double sum_du = sum16(__builtin_fma(all[1], off, all[2]));
    Moments mo;
    mo.finish(row_first, distance, squares, a.inv_h, a.eps);
    const double mean_d = sum_d * a.inv_h, mean_du = sum_du * a.inv_h * mo.r;
    if (IO != kOutF32) {
      // Unpacked again: kept, they would cost the registers of a second work-group
      // (bf16 16384 x 8192 208 us, renewed 190).
#pragma unroll
      for (int p = 0; p < P; ++p) {
        w[p].renew();
        now.dy[p].renew();
        now.s[p].renew();
      }
    }
    // Means of zero, as of rows without a gradient, binary32 holds.
    const double most = __builtin_fmax(__builtin_fabs(mean_d), __builtin_fabs(mean_du));
    const bool wide = mo.wide() || !(most < 0x1p100) || (most < 0x1p-100 && most > 0.0);
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
          const double u = mo.unit(s[j]);
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

// Columns of the workspace's n_parts rows [grad_weight | grad_bias] added, `more`: to
// what is there: 32 columns (a line of each row) a work-group, its 32 half waves taking
// every 32nd row.
__global__ __launch_bounds__(1024) void grad_params_kernel(const float* parts, float* grad_weight, float* grad_bias,
                                                           uint32_t n_parts, uint32_t h, bool more) {
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
    float* to = c < h ? grad_weight + c : grad_bias != nullptr ? grad_bias + (c - h) : nullptr;
    if (to != nullptr) *to = more ? *to + v : v;
  }
}

// Rows that a work-group adds in a chain; batches of more take further launches, whose
// sums are added in order, so that no sum of a column is one of thousands of
// additions to the same value (2^12 additions of 0.7 to a sum are 2^-14.6 off, 64 2^-20;
// one launch and as many as it takes, us: fp32 50021 x 4096 529 and 559, bf16 65536 x
// 4096 458 and 420, 2^20 x 64 1941 and 2136).
constexpr uint32_t kChainRows = 64;

template <int IO, int NT, int P, bool VEC, bool STREAM>
hipError_t launch_backward_as(const LayerNormBackwardLaunch& l, hipStream_t stream) {
  const uint32_t most = layer_norm_backward_parts(l.rows, l.h, IO == kOutF32);
  const uint64_t at_once = static_cast<uint64_t>(kChainRows) * most;
  auto from = [](const void* p, uint64_t elements) {
    return static_cast<const void*>(static_cast<const char*>(p) + elements * kOutSize<IO>);
  };
  for (uint64_t first = 0; first < l.rows; first += at_once) {
    LayerNormBackwardLaunch part = l;
    part.rows = l.rows - first < at_once ? l.rows - first : at_once;
    part.grad_y = from(l.grad_y, first * l.grad_y_stride);
    part.sum = from(l.sum, first * l.sum_stride);
    if (l.grad_sum != nullptr) part.grad_sum = from(l.grad_sum, first * l.grad_sum_stride);
    part.grad_x = const_cast<void*>(from(l.grad_x, first * l.grad_x_stride));
    const uint32_t parts = static_cast<uint32_t>(part.rows < most ? part.rows : most);
    hipError_t e = launch_kernel(layer_norm_backward_kernel<IO, NT, P, VEC, STREAM>, dim3(parts), dim3(NT), stream, part);
    if (e == hipSuccess)
      e = launch_kernel(grad_params_kernel, dim3((2 * l.h + 31) / 32), dim3(1024), stream,
                        static_cast<const float*>(l.workspace), l.grad_weight, l.grad_bias, parts, l.h, first != 0);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The smallest shape that holds a row, as above. us: bf16 16384 x 1024 128 x 1 46,
// 256 x 1 74; 8192 x 2048 128 x 2 37, 256 x 1 42; 8192 x 4096 256 x 2 58, 512 x 1 67;
// 16384 x 8192 256 x 4 190, 512 x 2 216; fp32 8192 x 5120 112 with 512 x 2, 134 with 256 x 4.
template <int IO, bool VEC, bool STREAM>
hipError_t launch_backward_sized(const LayerNormBackwardLaunch& l, hipStream_t stream) {
  if constexpr (VEC) {
    if (l.h <= 128 * 1 * kPiece) return launch_backward_as<IO, 128, 1, VEC, STREAM>(l, stream);
    if (l.h <= 128 * 2 * kPiece) return launch_backward_as<IO, 128, 2, VEC, STREAM>(l, stream);
    if (l.h <= 256 * 2 * kPiece) return launch_backward_as<IO, 256, 2, VEC, STREAM>(l, stream);
  }
  if constexpr (VEC && IO == kOutF32) {
    if (l.h <= 512 * 2 * kPiece) return launch_backward_as<IO, 512, 2, VEC, STREAM>(l, stream);
  } else {
    if (l.h <= 256 * 4 * kPiece) return launch_backward_as<IO, 256, 4, VEC, STREAM>(l, stream);
  }
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

uint32_t layer_norm_backward_parts(uint64_t rows, uint32_t h, bool f32) {
  // One a CU, as each leaves two rows of partial sums; more where rows are narrow, or
  // of 16 bits, which wait for vector instructions, if they have rows to load ahead.
  // us with 256, 512 and 1024: bf16 16384 x 1024 92, 73 and 46; 8192 x 2048 66, 52 and
  // 37; 4096 x 4096 42, 38 and 42; 1021 x 7168 25, 28 and 37; 2560 x 8192 47, 46 and 59;
  // 8192 x 8192 120, 102; 16384 x 8192 226, 190 and 200; 4096 x 16384 112, 126 and 154;
  // fp32 16384 x 1024 93, 69 and 56; 8192 x 2048 70, 54 and 58; 16384 x 4096 177, 192;
  // 8192 x 5120 112, 120.
  uint32_t parts = 256;
  if (h <= 256 * kPiece && rows >= 4 * 1024)
    parts = 1024;
  else if (h <= 256 * kPiece ? rows >= 4 * 512 : !f32 && h <= 1024 * kPiece && rows >= 5 * 512)
    parts = 512;
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
