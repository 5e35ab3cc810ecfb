// Device helpers of the kernels over rows (qrs_rows.hip, qrs_layer_norm.hip):
// pieces of a row as they lie in memory, sums over a wave in binary64, and what
// both norms share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qrs_device.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace dev {

// A piece (16 bytes) as it lies in memory (VEC), so that rows under way cost half the
// registers for 16-bit types; otherwise as floats. STREAM: loads that leave no
// copy in the caches. renew(): from here on the values are to be taken as new
// ones, so that what was unpacked from them is not kept in registers.
template <int IO, bool VEC>
struct RawPiece {
  float v[kPiece16<IO>];
  template <bool STREAM>
  __device__ __forceinline__ void load(const void* row, uint32_t c, uint32_t h) {
    load_piece<IO, VEC, kPiece16<IO>>(row, c, h, v);
  }
  __device__ __forceinline__ void get(float* to) const {
#pragma unroll
    for (int j = 0; j < kPiece16<IO>; ++j) to[j] = v[j];
  }
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int j = 0; j < kPiece16<IO>; ++j) asm volatile("" : "+v"(v[j]));
  }
};
template <int IO>
struct RawPiece16 {
  u32x4 w;
  template <bool STREAM>
  __device__ __forceinline__ void load(const void* row, uint32_t c, uint32_t h) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(row) + c);
    w = u32x4{0u, 0u, 0u, 0u};
    if (c < h) w = STREAM ? __builtin_nontemporal_load(p) : *p;
  }
  __device__ __forceinline__ void get(float* to) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2<IO>(w[j], to + 2 * j);
  }
  __device__ __forceinline__ void renew() { asm volatile("" : "+v"(w)); }
};
template <>
struct RawPiece<kOutF32, true> {
  f32x4 w;
  template <bool STREAM>
  __device__ __forceinline__ void load(const void* row, uint32_t c, uint32_t h) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(row) + c);
    w = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (c < h) w = STREAM ? __builtin_nontemporal_load(p) : *p;
  }
  __device__ __forceinline__ void get(float* to) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) to[j] = w[j];
  }
  __device__ __forceinline__ void renew() { asm volatile("" : "+v"(w)); }
};
template <>
struct RawPiece<kOutBF16, true> : RawPiece16<kOutBF16> {};
template <>
struct RawPiece<kOutF16, true> : RawPiece16<kOutF16> {};

// Operands beyond this many bytes pass through the Infinity Cache (256 MB)
// without being found there again: they are loaded as a stream (backward
// pass, 1074 MB: 195 us, as a stream 174; 59 MB, found there: 20.2 and 21.6).
constexpr uint64_t kStreamBytes = uint64_t{256} << 20;

// v from the lanes that f takes its 32-bit halves from.
template <typename F>
__device__ __forceinline__ double lanes(double v, F f) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = f(static_cast<uint32_t>(b)), hi = f(static_cast<uint32_t>(b >> 32));
  return __builtin_bit_cast(double, lo | hi << 32);
}

__device__ __forceinline__ double wave_sum(double v) {
  v += lanes(v, [](uint32_t x) { return dpp<kDppSwap1>(x); });
  v += lanes(v, [](uint32_t x) { return dpp<kDppSwap2>(x); });
  v += lanes(v, [](uint32_t x) { return dpp<kDppHalfMirror>(x); });
  v += lanes(v, [](uint32_t x) { return dpp<kDppMirror>(x); });
  double row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = lanes(v, [i](uint32_t x) { return lane_value(x, 16 * i); });
  return (row[0] + row[1]) + (row[2] + row[3]);
}

// 1 / sqrt(m): the hardware's estimate (about 2^-24) and one Newton step.
__device__ __forceinline__ double inverse_root(double m) {
  const double q = __builtin_amdgcn_rsq(m);
  return __builtin_isinf(m) ? 0.0 : q * __builtin_fma(-0.5 * m * q, q, 1.5);
}

// Values that are to be taken as new ones: what is made of them is not kept
// over rows, or made ahead of the branch that needs it, at the cost of the
// registers that let more waves run.
template <int E>
__device__ __forceinline__ void as_new(float (&v)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) asm volatile("" : "+v"(v[j]));
}

template <int E>
__device__ __forceinline__ uint32_t piece_max(const float* y) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < E; ++j) amax = max(amax, abs_bits(y[j]));
  return amax;
}

}  // namespace dev
}  // namespace qrs
