// Device helpers of the product kernels (qrs_matmul.hip, qrs_matmul_fp8.h):
// what a finished piece of outputs goes through, and how operands reach LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qrs_device.h"
#include "qrs_layer.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace dev {

constexpr uint32_t kCus = 256;

// g / (1 + exp(-g)) as g * n / (1 + e) with e = exp(-|g|) and n = 1, or e for
// negative g: nothing overflows, and where e would be subnormal (g < -64) it is
// held times 2^64 and g times 2^-64. exp as a power of two whose exponent's
// rounding error is put back as a factor, 1 / d as the hardware's estimate and
// one Newton step: each within a few units of the last place, for a third of
// the instructions of the library's exp and divide (512 tokens by 5120 ups,
// k = 1024: 17.5 us -> 16.5). Beyond 200, e is 0 whatever its scale.
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;
  const float x = __builtin_fminf(__builtin_fabsf(g), 200.0f);
  const bool far = g < -64.0f;
  const float p = -x * kLog2e;
  const float low = __builtin_fmaf(-x, kLog2eLow, __builtin_fmaf(-x, kLog2e, -p));
  const float e0 = __builtin_amdgcn_exp2f(far ? p + 64.0f : p);  // this sum is exact: |p| is at least 92
  const float e = __builtin_fmaf(e0, low * kLn2, e0);
  const float d = 1.0f + e;  // far: e, 2^-28 at most even so, has no part in it
  const float r = __builtin_amdgcn_rcpf(d);
  const float inverse = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  return (far ? g * 0x1p-64f : g) * (g < 0.0f ? e * inverse : inverse);
}

// The codes of a piece and its group's scale (E8M0 code or binary32 bits),
// the mode chosen at run time: a kernel's epilogue repeats this for every
// fragment, and a copy for each mode would be five times the code.
// `no_nan`: the scales that v was multiplied by leave no NaN in it, and the
// maximum may be one of numbers; else it is one of bits, where NaN stands
// above infinity.
__device__ __forceinline__ Codes<kPiece> encode_group(const MatmulLaunch& a, const float* v, bool no_nan,
                                                       uint32_t* scale_bits) {
  float m = __builtin_fmaxf(__builtin_fabsf(v[0]), __builtin_fabsf(v[1]));
#pragma unroll
  for (int j = 2; j < kPiece; ++j) m = __builtin_fmaxf(m, __builtin_fabsf(v[j]));
  uint32_t bits = __builtin_bit_cast(uint32_t, m);
  if (!no_nan) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) bits = max(bits, abs_bits(v[j]));
  }
  uint32_t amax = group_max<4>(bits);
  float mul;
  if (a.scale_layout == kScaleE8M0Block32) {
    mul = a.x_format == kXE4M3FN ? mx_multiplier<kXE4M3FN>(amax, scale_bits) : mx_multiplier<kXE5M2>(amax, scale_bits);
  } else {
    amax = max(amax, dpp<kDppHalfMirror>(amax));
    amax = max(amax, dpp<kDppMirror>(amax));
    const float top = a.x_format == kXE4M3FN ? CodeFormat<kXE4M3FN>::kMax
                      : a.x_format == kXE5M2 ? CodeFormat<kXE5M2>::kMax
                                             : CodeFormat<kXInt8>::kMax;
    float scale;
    mul = f32_multiplier(amax, top, &scale);
    *scale_bits = __builtin_bit_cast(uint32_t, scale);
  }
  if (a.x_format == kXE4M3FN) return encode_piece<kXE4M3FN>(v, mul);
  if (a.x_format == kXE5M2) return encode_piece<kXE5M2>(v, mul);
  return encode_piece<kXInt8>(v, mul);
}

__device__ __forceinline__ void finish_codes(const MatmulLaunch& a, uint32_t i, uint32_t j0, bool active, bool no_nan,
                                             const float* v) {
  uint32_t scale;
  const Codes<kPiece> codes = encode_group(a, v, no_nan, &scale);
  if (!active) return;
  store_codes<true, kPiece>(static_cast<uint8_t*>(a.out) + static_cast<uint64_t>(i) * a.out_stride, j0, a.n, codes);
  if (a.scale_layout == kScaleE8M0Block32) {
    if (j0 % 32 == 0)
      static_cast<uint8_t*>(a.scales)[static_cast<uint64_t>(i) * (a.n / 32) + j0 / 32] = static_cast<uint8_t>(scale);
  } else {
    if (j0 % 128 == 0) static_cast<uint32_t*>(a.scales)[static_cast<uint64_t>(i) * (a.n / 128) + j0 / 128] = scale;
  }
}

// Eight outputs of a row off 16-byte boundaries: the hardware stores 16 bytes at any
// address of an element (333 x 5003, k = 7168, of 8-bit floats from memory: floats 37 us, with a
// store for each element 40; bf16 27.3 and 29.1).
template <int OF>
__device__ __forceinline__ void store_piece_anywhere(void* row, uint32_t c, const float* v) {
  if constexpr (OF == kOutF32) {
    typedef float floats __attribute__((ext_vector_type(4), aligned(4)));
    floats* p = reinterpret_cast<floats*>(static_cast<float*>(row) + c);
    p[0] = floats{v[0], v[1], v[2], v[3]};
    p[1] = floats{v[4], v[5], v[6], v[7]};
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
    *reinterpret_cast<words*>(static_cast<uint16_t*>(row) + c) =
        words{pack2<OF>(v[0], v[1]), pack2<OF>(v[2], v[3]), pack2<OF>(v[4], v[5]), pack2<OF>(v[6], v[7])};
  }
}

template <int OF>
__device__ __forceinline__ void finish_values(const MatmulLaunch& a, uint32_t i, uint32_t j0, const float* v) {
  char* row = static_cast<char*>(a.out) + static_cast<uint64_t>(i) * a.out_stride * kOutSize<OF>;
  if (j0 + kPiece > a.n) {
    store_piece<OF, false, kPiece>(row, j0, a.n, v);
  } else if (a.out_vec) {
    store_piece<OF, true, kPiece>(row, j0, a.n, v);
  } else {
    store_piece_anywhere<OF>(row, j0, v);
  }
}

// 16 bytes [k, k + 16) of a row, zeros from `end` on. VEC: the row starts on
// a 16-byte boundary and `end` is a multiple of 16.
template <bool VEC>
__device__ __forceinline__ u32x4 load16(const int8_t* row, uint32_t k, uint32_t end) {
  u32x4 w = {0u, 0u, 0u, 0u};
  if constexpr (VEC) {
    if (k < end) w = *reinterpret_cast<const u32x4*>(row + k);
  } else {
#pragma unroll
    for (int t = 0; t < 16; ++t)
      if (k + t < end) w[t / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + t])) << (8 * (t % 4));
  }
  return w;
}

typedef __attribute__((address_space(3))) void* lds_ptr;

template <int N>
__device__ __forceinline__ void wait_loads_and_sync() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Offsets of rows within a tile stay below kFar; a lane that has nothing to
// load adds kFar, which is past the buffer's range, so that the hardware's
// range check gives zero.
constexpr uint32_t kFar = 1u << 30;

// Tiles in the order in which an XCD should run them: patches of kGroup
// token tiles by whole columns share their operands in its L2.
struct TileOrder {
  uint32_t tiles_m, tiles_n;
  __device__ void at(uint32_t tile, uint32_t* tm, uint32_t* tn) const {
    constexpr uint32_t kGroup = 8;
    const uint32_t group = tile / (kGroup * tiles_n), in_group = tile % (kGroup * tiles_n);
    const uint32_t group_m = min(kGroup, tiles_m - group * kGroup);
    *tm = group * kGroup + in_group % group_m;
    *tn = in_group / group_m;
  }
};

}  // namespace dev
}  // namespace qrs
