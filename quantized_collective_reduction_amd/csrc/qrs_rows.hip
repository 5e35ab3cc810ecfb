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
#include "qrs_rows_device.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace {

using namespace dev;

// y * 2^896 rounded to odd: toward zero, the last bit set if that was inexact.
// A second rounding, to fewer bits, then gives what it would give for y. The
// factor puts the exponent of a binary64 where a binary32 has it, subnormal
// numbers included, so that a shift truncates; values that binary32 does not
// hold become NaN.
__device__ __forceinline__ float round_to_odd(double y) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, y);
  const uint32_t low = static_cast<uint32_t>(bits), sign = static_cast<uint32_t>(bits >> 32) & 0x80000000u;
  const uint32_t magnitude = min(static_cast<uint32_t>(bits >> 29), 0x7FC00000u) | min(low & 0x1FFFFFFFu, 1u);
  return __builtin_bit_cast(float, magnitude | sign);
}

// One lane's pieces of a row and what makes values for codes of them.
//
// y = s * r * weight is taken in binary32, with three roundings (r's and those of
// the two products: 3 * 2^-24, where neither s * r nor y is subnormal), and in
// binary64 where that does not do: in rows whose squares leave binary32's range,
// and, with E8M0 scales, where y is so close to a border between two codes that
// the error could decide which one it gets. (In binary64 always, it takes the
// registers of a second work-group: 8192 x 5120 fp32 117 us.)
template <int IO, bool VEC, bool NORM, int P>
struct RowValues {
  static constexpr int E = kPiece16<IO>;
  float v[P][E];  // s, or without a norm the values themselves
  double r;
  bool wide;  // y in binary64
  const RawPiece<IO, VEC>* w;

  // TO_F32: in binary64 where the row is wide.
  template <bool TO_F32>
  __device__ __forceinline__ void piece(int p, float* y) const {
    if constexpr (NORM) {
      float s[E], wv[E];
      operands(p, s, wv);
#pragma unroll
      for (int j = 0; j < E; ++j) y[j] = s[j] * static_cast<float>(r) * wv[j];
      if (TO_F32 && wide) {
        operands(p, s, wv);
#pragma unroll
        for (int j = 0; j < E; ++j) y[j] = static_cast<float>(static_cast<double>(s[j]) * r * static_cast<double>(wv[j]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) y[j] = v[p][j];
    }
  }

  __device__ __forceinline__ void piece_to_odd(int p, float* y) const {
    float s[E], wv[E];
    operands(p, s, wv);
    const double factor = r * 0x1p-896;
#pragma unroll
    for (int j = 0; j < E; ++j) y[j] = round_to_odd(static_cast<double>(s[j]) * factor * static_cast<double>(wv[j]));
  }

 private:
  __device__ __forceinline__ void operands(int p, float (&s)[E], float (&wv)[E]) const {
    w[p].get(wv);
#pragma unroll
    for (int j = 0; j < E; ++j) s[j] = v[p][j];
    as_new(s);
    as_new(wv);
  }
};

// Codes and E8M0 scales of a lane's pieces: those of y in binary32 if both
// ends of the interval y * (1 -+ 2^-22) have them in every lane of the wave,
// else (one wave's row in about 100) those of y rounded to odd.
template <int XF, int P, typename Values>
__device__ __forceinline__ void mx_codes(const Values& row, Codes<Values::E>* codes, uint32_t* scales) {
  constexpr int E = Values::E, G = 32;
  bool sure = !row.wide;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float y[E];
    row.template piece<false>(p, y);
    const uint32_t amax = group_max<G / E>(piece_max<E>(y));
    const float mul = mx_multiplier<XF>(amax, &scales[p]);
    codes[p] = encode_piece<XF, E>(y, mul * (1.0f + 0x1p-22f));
    const Codes<E> low = encode_piece<XF, E>(y, mul * (1.0f - 0x1p-22f));
    sure = sure && (amax + 8) >> 23 == (max(amax, 8u) - 8) >> 23;
#pragma unroll
    for (int k = 0; k < E / 4; ++k) sure = sure && codes[p].w[k] == low.w[k];
  }
  if (__builtin_amdgcn_ballot_w64(!sure) == 0) return;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float y[E];
    row.piece_to_odd(p, y);
    const uint32_t amax = group_max<G / E>(piece_max<E>(y));
    codes[p] = encode_piece<XF, E>(y, mx_multiplier<XF>(amax, &scales[p]));
  }
}

// Codes of one row held as P pieces per lane, piece p at column
// (p * NT + lane) * E.
template <int XF, int SL, int NT, int P, bool VEC, typename Values>
__device__ __forceinline__ void quantize_row(const Values& values, const RowsLaunch& a, uint64_t row, int lane,
                                             uint32_t amax) {
  constexpr int E = Values::E;
  uint8_t* codes_row = static_cast<uint8_t*>(a.codes) + row * a.codes_stride;
  if constexpr (SL == kScaleE8M0Block32) {
    Codes<E> codes[P];
    uint32_t scales[P];
    mx_codes<XF, P>(values, codes, scales);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * E;
      store_codes<VEC, E>(codes_row, c, a.h, codes[p]);
      if (c < a.h && c % 32 == 0)
        static_cast<uint8_t*>(a.scales)[row * (a.h / 32) + c / 32] = static_cast<uint8_t>(scales[p]);
    }
  } else {
    float mul = 0.0f, scale = 0.0f;
    if constexpr (SL == kScaleF32Row) {
      mul = f32_multiplier(amax, CodeFormat<XF>::kMax, &scale);
      if (lane == 0) static_cast<float*>(a.scales)[row] = scale;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t c = (p * NT + lane) * E;
      float y[E];
      values.template piece<true>(p, y);
      if constexpr (SL == kScaleF32Group128)
        mul = f32_multiplier(group_max<128 / E>(piece_max<E>(y)), CodeFormat<XF>::kMax, &scale);
      store_codes<VEC, E>(codes_row, c, a.h, encode_piece<XF, E>(y, mul));
      if (SL == kScaleF32Group128 && c < a.h && c % 128 == 0)
        static_cast<float*>(a.scales)[row * (a.h / 128) + c / 128] = scale;
    }
  }
}

// NORM: the residual sum and norm in front of the codes; otherwise x itself
// is quantized. Work-group b takes rows b, b + gridDim, ...; the next row's
// operands are under way while a row is reduced and written.
//
// The squares are added in binary64 where codes go by more than binary32 (E8M0
// scales); otherwise those of a piece in binary32 and the pieces in binary64. A
// piece of eight 16-bit values has seven roundings (the squares are exact), one
// of four binary32 values four, so r is within 3.5 * 2^-24, and y within 6.5. If
// the sum is not well inside binary32's range, the row is taken in binary64.
template <int IO, int SL, int NT, int P8, bool VEC, bool NORM, bool STREAM>
__global__ __launch_bounds__(NT) void rows_kernel(const RowsLaunch a) {
  constexpr int E = kPiece16<IO>, P = P8 * 8 / E;  // P8: 8 elements a lane
  constexpr int kWaves = NT / 64;
  __shared__ double sum_part[2][kWaves];
  __shared__ uint32_t max_part[2][kWaves];
  const int lane = threadIdx.x;
  constexpr int kSize = kOutSize<IO>;
  typedef RawPiece<IO, VEC> Raw;
  struct Operands {
    Raw x[P], r[NORM ? P : 1];
  };
  Operands next;
  Raw w[NORM ? P : 1];
  const bool add = NORM && a.residual != nullptr;
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
  if constexpr (NORM) {
#pragma unroll
    for (int p = 0; p < P; ++p) w[p].template load<false>(a.weight, (p * NT + lane) * E, a.h);
  }

  // The parts of the reductions alternate between two halves: a wave that is
  // a row ahead writes the other half, and the next barrier keeps it from
  // going further.
  int turn = 0;
  RowValues<IO, VEC, NORM, P> values;
  auto& v = values.v;
  values.w = w;
  values.wide = false;
  auto row_sum = [&](double ss) {
    ss = wave_sum(ss);
    if (lane % 64 == 0) sum_part[turn][lane / 64] = ss;
    lds_barrier();
    ss = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) ss += sum_part[turn][i];
    return ss;
  };
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    if (!kAhead) load_row(row);
    const Operands now = next;
    if (kAhead && row + gridDim.x < a.rows) load_row(row + gridDim.x);
#pragma unroll
    for (int p = 0; p < P; ++p) now.x[p].get(v[p]);
    if constexpr (NORM) {
      if (add) {
        char* s_row = static_cast<char*>(a.sum) + row * a.sum_stride * kSize;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float r[E];
          now.r[p].get(r);
#pragma unroll
          for (int j = 0; j < E; ++j) v[p][j] = round_to<IO>(v[p][j] + r[j]);
          store_piece<IO, VEC, E>(s_row, (p * NT + lane) * E, a.h, v[p]);
        }
      }
      double ss = 0.0;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if constexpr (SL == kScaleE8M0Block32) {
#pragma unroll
          for (int j = 0; j < E; ++j) ss = __builtin_fma(v[p][j], static_cast<double>(v[p][j]), ss);
        } else {
          float q = v[p][0] * v[p][0];
#pragma unroll
          for (int j = 1; j < E; ++j) q = __builtin_fmaf(v[p][j], v[p][j], q);
          ss += q;
        }
      }
      ss = row_sum(ss);
      values.wide = !(ss > 0x1p-70 && ss < 0x1p120);  // the same in every lane
      if (SL != kScaleE8M0Block32 && values.wide) {
        turn ^= 1;
        ss = 0.0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          as_new(v[p]);
#pragma unroll
          for (int j = 0; j < E; ++j) ss = __builtin_fma(v[p][j], static_cast<double>(v[p][j]), ss);
        }
        ss = row_sum(ss);
      }
      values.r = inverse_root(ss * a.inv_h + static_cast<double>(a.eps));
    }

    uint32_t amax = 0;
    if constexpr (SL == kScaleF32Row) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float y[E];
        values.template piece<true>(p, y);
        amax = max(amax, piece_max<E>(y));
      }
      amax = wave_max(amax);
      if (lane % 64 == 0) max_part[turn][lane / 64] = amax;
      lds_barrier();
#pragma unroll
      for (int i = 0; i < kWaves; ++i) amax = max(amax, max_part[turn][i]);
    }
    if (a.x_format == kXE4M3FN) {
      quantize_row<kXE4M3FN, SL, NT, P, VEC>(values, a, row, lane, amax);
    } else if (a.x_format == kXE5M2) {
      quantize_row<kXE5M2, SL, NT, P, VEC>(values, a, row, lane, amax);
    } else if constexpr (SL != kScaleE8M0Block32) {
      quantize_row<kXInt8, SL, NT, P, VEC>(values, a, row, lane, amax);
    }
  }
}

template <int IO, int SL, int NT, int P, bool VEC, bool NORM, bool STREAM>
hipError_t launch_rows_as(const RowsLaunch& l, hipStream_t stream) {
  // Where registers leave two work-groups a CU (one of 1024 lanes), as many as
  // run at once: each loads ahead, and none is left over for a second round.
  // Else many, which even out by themselves. Norm of bf16 rows, us with 512
  // and 4096 work-groups: 2048 x 8192 23.8 and 24.5, 16384 x 8192 148 and 151,
  // 8192 x 4096 42.4 and 40.4, 16384 x 1024 48.2 and 29.8; with 256 and 4096:
  // 2048 x 16384 44.1 and 53.1. 8192 x 5120 fp32 (512 x 2) with 512, 819 and 4096:
  // 94.4, 103 and 94.0. Codes of 16384 x 8192 alone with 512 and 4096: 75.7 and
  // 68.7.
  const uint32_t blocks = !NORM || NT * P <= 512 ? 4096 : NT < 1024 ? 512 : 256;
  return launch_kernel(rows_kernel<IO, SL, NT, P, VEC, NORM, STREAM>,
                       dim3(static_cast<uint32_t>(l.rows < blocks ? l.rows : blocks)), dim3(NT), stream, l);
}

// The smallest shape that holds a row; rows off 16-byte boundaries have two.
// (Norm: scratch memory takes part of rows past 16384 elements, and past 8192 of
// those off 16-byte boundaries.)
template <int IO, int SL, bool VEC, bool NORM, bool STREAM>
hipError_t launch_rows_sized(const RowsLaunch& l, hipStream_t stream) {
  if constexpr (VEC) {
    if (l.h <= 256 * 1 * kPiece) return launch_rows_as<IO, SL, 256, 1, VEC, NORM, STREAM>(l, stream);
    if (l.h <= 512 * 1 * kPiece) return launch_rows_as<IO, SL, 512, 1, VEC, NORM, STREAM>(l, stream);
    // E8M0 codes of 4096 x 4224 and 4096 x 6144 bf16: 31.2 and 34.4 us with
    // 512 x 2, 27.0 and 32.2 with 768 x 1; fp32 scales 32.0 and 31.7, row
    // scales (4096 x 6144) 33.0 and 34.5.
    if constexpr (SL == kScaleE8M0Block32)
      if (l.h <= 768 * 1 * kPiece) return launch_rows_as<IO, SL, 768, 1, VEC, NORM, STREAM>(l, stream);
  }
  if (l.h <= 512 * 2 * kPiece) return launch_rows_as<IO, SL, 512, 2, VEC, NORM, STREAM>(l, stream);
  if constexpr (VEC) {
    if (l.h <= 1024 * 2 * kPiece) return launch_rows_as<IO, SL, 1024, 2, VEC, NORM, STREAM>(l, stream);
    if (l.h <= 1024 * 4 * kPiece) return launch_rows_as<IO, SL, 1024, 4, VEC, NORM, STREAM>(l, stream);
  }
  if (l.h <= 1024 * 8 * kPiece) return launch_rows_as<IO, SL, 1024, 8, VEC, NORM, STREAM>(l, stream);
  return hipErrorInvalidValue;
}

template <int IO, int SL, bool NORM>
hipError_t launch_rows_typed(const RowsLaunch& l, hipStream_t stream) {
  if (!l.vec) return launch_rows_sized<IO, SL, false, NORM, false>(l, stream);
  const uint64_t bytes = l.rows * l.h * (kOutSize<IO> * (NORM ? 3 : 1) + 1);
  return bytes > kStreamBytes ? launch_rows_sized<IO, SL, true, NORM, true>(l, stream)
                              : launch_rows_sized<IO, SL, true, NORM, false>(l, stream);
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

// With r = 1 / sqrt(mean(s^2) + eps), u = s * r and d = weight * grad_y:
//   grad_x      = grad_sum + r * (d - u * mean(d * u))
//   grad_weight = sum over tokens of grad_y * u
// Both row sums (s^2 and d * s) are taken in one reduction: those of a piece
// in binary32, the pieces in binary64. |u| is at most sqrt(h) and |u * mean|
// at most the largest |d * u|, so apart from these sums and d itself nothing
// leaves binary32's range before the result does. Where a sum is not well
// inside it, the row is taken again in binary64. (A sum of d * s of less than
// 2^-100 may have lost products. Of exactly zero, it is that of a row without
// gradients, as in padding, or of products below 2^-150, which cannot show where
// r is at most 2^20.)
//
// Work-group b takes rows b, b + gridDim, ...; the next row's operands are
// under way while a row is reduced and written. It keeps its columns' share of
// grad_weight in registers and leaves one row of partial sums in the workspace,
// and grad_weight_kernel adds those rows in order: a fixed order without
// atomics.
template <int IO, int NT, int P8, bool VEC, bool STREAM>
__global__ __launch_bounds__(NT) void norm_backward_kernel(const NormBackwardLaunch a) {
  constexpr int kWaves = NT / 64;
  __shared__ double parts[2][2 * kWaves];
  constexpr int E = kPiece16<IO>, P = P8 * 8 / E;
  const int lane = threadIdx.x;
  constexpr int kSize = kOutSize<IO>;
  typedef RawPiece<IO, VEC> Raw;
  float dw[P][E];
  Raw w[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    w[p].template load<false>(a.weight, (p * NT + lane) * E, a.h);
#pragma unroll
    for (int j = 0; j < E; ++j) dw[p][j] = 0.0f;
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

  load_row(blockIdx.x);
  const float keep = a.grad_sum != nullptr ? 1.0f : 0.0f;
  // Alternating halves of `parts`: a wave that is a row ahead writes the
  // other half, and the next barrier keeps it from going further.
  int turn = 0;
  auto row_sums = [&](double& ss, double& ds) {
    ss = wave_sum(ss);
    ds = wave_sum(ds);
    if (lane % 64 == 0) {
      parts[turn][lane / 64] = ss;
      parts[turn][kWaves + lane / 64] = ds;
    }
    lds_barrier();
    ss = ds = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      ss += parts[turn][i];
      ds += parts[turn][kWaves + i];
    }
  };
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    Operands now = next;
    if (row + gridDim.x < a.rows) load_row(row + gridDim.x);
    auto operands = [&](int p, float (&wv)[E], float (&dy)[E], float (&s)[E]) {
      w[p].get(wv);
      now.dy[p].get(dy);
      now.s[p].get(s);
    };
    auto renew = [&]() {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        w[p].renew();
        now.dy[p].renew();
        now.s[p].renew();
      }
    };
    // 1024 lanes leave 128 registers each, which unpacked values kept for the
    // second pass overflow (4096 x 16384 bf16 161 us, renewed 101); with fewer
    // lanes unpacking twice costs more (16384 x 8192 bf16 176 us, renewed 186).
    constexpr bool kRenew = NT == 1024;
    double ss = 0.0, ds = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float wv[E], dy[E], s[E];
      operands(p, wv, dy, s);
      float q = s[0] * s[0], t = wv[0] * dy[0] * s[0];
#pragma unroll
      for (int j = 1; j < E; ++j) {
        q = __builtin_fmaf(s[j], s[j], q);
        t = __builtin_fmaf(wv[j] * dy[j], s[j], t);
      }
      ss += q;
      ds += t;
    }
    row_sums(ss, ds);
    if (kRenew) renew();
    const double m = ss * a.inv_h + static_cast<double>(a.eps);
    double r = inverse_root(m), mean = r * (ds * a.inv_h);
    // The same in every lane. Squares lost below 2^-150 do not show in an m of
    // 2^-100, so rows of zeros are ordinary ones.
    const bool wide = !(m > 0x1p-100 && ss < 0x1p120 && __builtin_fabs(mean) < 0x1p110 &&
                        (__builtin_fabs(ds) > 0x1p-100 || (ds == 0.0 && m > 0x1p-40)));
    if (wide) {
      turn ^= 1;
      ss = ds = 0.0;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float wv[E], dy[E], s[E];
        operands(p, wv, dy, s);
        as_new(wv);
        as_new(dy);
        as_new(s);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          ss = __builtin_fma(s[j], static_cast<double>(s[j]), ss);
          ds = __builtin_fma(static_cast<double>(wv[j]) * dy[j], static_cast<double>(s[j]), ds);
        }
      }
      row_sums(ss, ds);
      if (kRenew) renew();
      r = inverse_root(ss * a.inv_h + static_cast<double>(a.eps));
      mean = r * (ds * a.inv_h);
    }
    const float r32 = static_cast<float>(r), mean32 = static_cast<float>(mean);
    auto finish = [&](int p, bool in64) {
      const uint32_t c = (p * NT + lane) * E;
      float wv[E], dy[E], s[E], g[E];
      operands(p, wv, dy, s);
      now.g[p].get(g);
#pragma unroll
      for (int j = 0; j < E; ++j) g[j] = keep != 0.0f ? g[j] : 0.0f;
      if (in64) {
        as_new(wv);
        as_new(dy);
        as_new(s);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const double u = s[j] * r;
          dw[p][j] += static_cast<float>(dy[j] * u);
          g[j] = static_cast<float>(g[j] + r * (static_cast<double>(wv[j]) * dy[j] - u * mean));
        }
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const float u = s[j] * r32;
          dw[p][j] += dy[j] * u;
          g[j] += r32 * (wv[j] * dy[j] - u * mean32);
        }
      }
      store_piece<IO, VEC, E>(static_cast<char*>(a.grad_x) + row * a.grad_x_stride * kSize, c, a.h, g);
    };
    // One loop for each kind of row lets an ordinary row's pieces overlap
    // (1021 x 7168 bf16 16.5 us with a branch in each piece, 15.8), but at
    // 1024 lanes it overflows the registers (4096 x 16384 bf16 101 us, 258).
    if (kRenew) {
#pragma unroll
      for (int p = 0; p < P; ++p) finish(p, wide);
    } else if (__builtin_expect(wide, false)) {
#pragma unroll
      for (int p = 0; p < P; ++p) finish(p, true);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) finish(p, false);
    }
  }
  float* part_row = a.workspace + static_cast<uint64_t>(blockIdx.x) * a.h;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t c = (p * NT + lane) * E;
    if (VEC && c < a.h) {
#pragma unroll
      for (int j = 0; j < E; j += 4)
        *reinterpret_cast<f32x4*>(part_row + c + j) = f32x4{dw[p][j], dw[p][j + 1], dw[p][j + 2], dw[p][j + 3]};
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (c + j < a.h) part_row[c + j] = dw[p][j];
    }
  }
}

// grad_weight[c] = sum over the n_parts rows of the workspace: 32 columns (a
// line of each row) a work-group, its 32 half waves taking every 32nd row.
__global__ __launch_bounds__(1024) void grad_weight_kernel(const float* parts, float* grad_weight, uint32_t n_parts,
                                                           uint32_t h) {
  __shared__ float part[32][33];
  const uint32_t col = threadIdx.x % 32, c = blockIdx.x * 32 + col, w = threadIdx.x / 32;
  float v = 0.0f;
  if (c < h) {
#pragma unroll 4
    for (uint32_t i = w; i < n_parts; i += 32) v += parts[static_cast<uint64_t>(i) * h + c];
  }
  part[w][col] = v;
  __syncthreads();
  if (w == 0 && c < h) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += part[i][col];
    grad_weight[c] = v;
  }
}

template <int IO, int NT, int P, bool VEC, bool STREAM>
hipError_t launch_backward_as(const NormBackwardLaunch& l, hipStream_t stream) {
  const uint32_t parts = norm_backward_parts(l.rows, l.h);
  const hipError_t e = launch_kernel(norm_backward_kernel<IO, NT, P, VEC, STREAM>, dim3(parts), dim3(NT), stream, l);
  if (e != hipSuccess) return e;
  return launch_kernel(grad_weight_kernel, dim3((l.h + 31) / 32), dim3(1024), stream,
                       static_cast<const float*>(l.workspace), l.grad_weight, parts, l.h);
}

template <int IO, bool VEC, bool STREAM>
hipError_t launch_backward_sized(const NormBackwardLaunch& l, hipStream_t stream) {
  // The smallest shape that holds a row, as above. (1024 lanes leave 128
  // registers a lane. Scratch memory takes part of rows past 16384 elements, and
  // past 8192 of binary32 rows and of those off 16-byte boundaries: 4096 x 16384
  // bf16 98 us, 5.5 TB/s; 2048 x 16384 fp32 207 us, 2.6 TB/s.)
  if constexpr (VEC) {
    if (l.h <= 256 * 1 * kPiece) return launch_backward_as<IO, 256, 1, VEC, STREAM>(l, stream);
    if (l.h <= 256 * 2 * kPiece) return launch_backward_as<IO, 256, 2, VEC, STREAM>(l, stream);
  }
  if (l.h <= 256 * 4 * kPiece) return launch_backward_as<IO, 256, 4, VEC, STREAM>(l, stream);
  if constexpr (VEC)
    if (l.h <= 1024 * 2 * kPiece) return launch_backward_as<IO, 1024, 2, VEC, STREAM>(l, stream);
  if (l.h <= 1024 * 8 * kPiece) return launch_backward_as<IO, 1024, 8, VEC, STREAM>(l, stream);
  return hipErrorInvalidValue;
}

template <int IO>
hipError_t launch_backward_io(const NormBackwardLaunch& l, hipStream_t stream) {
  if (!l.vec) return launch_backward_sized<IO, false, false>(l, stream);
  return l.rows * l.h * kOutSize<IO> * 4 > kStreamBytes ? launch_backward_sized<IO, true, true>(l, stream)
                                                        : launch_backward_sized<IO, true, false>(l, stream);
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

uint32_t norm_backward_parts(uint64_t rows, uint32_t h) {
  // One a CU: each leaves a row of partial sums, and holds half of a CU's
  // registers. Two for narrow rows, if they then have rows to load ahead. us
  // with 256, 512 and 1024: 16384 x 8192 bf16 179, 190 and 192; 1021 x 7168
  // bf16 17.5, 19.7 and 26.1; 4096 x 4096 f16 28.3, 29.6 and 33.3; 8192 x 2048
  // bf16 37.0, 29.2 and 31.9; 500 x 2048 bf16 8.0 and 9.7.
  const uint32_t parts = h <= 256 * kPiece && rows >= 4 * 512 ? 512 : 256;
  return static_cast<uint32_t>(rows < parts ? rows : parts);
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
