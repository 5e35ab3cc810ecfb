// Device helpers of the layer kernels (qrs_rows.hip, qrs_matmul.hip): typed
// loads and stores of 8-element pieces, lane reductions, and the codes and
// scales of a piece. qrs_quantize.hip states the same code rules for its own
// stream; oracle/quantize.py is the definition of both.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qrs_launch.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace dev {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kPiece = 8;  // consecutive elements a lane owns

template <int OF>
constexpr int kOutSize = OF == kOutF32 ? 4 : 2;

// The piece that is one 16-byte load or store.
template <int OF>
constexpr int kPiece16 = 16 / kOutSize<OF>;

// Two floats -> one word of the 16-bit type, nearest-even.
template <int OF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f32x2 pr = {a, b};
  if constexpr (OF == kOutBF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, f16x2));
}

template <int OF>
__device__ __forceinline__ void unpack2(uint32_t w, float* v) {
  if constexpr (OF == kOutBF16) {
    v[0] = __builtin_bit_cast(float, w << 16);
    v[1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
  } else {
    const f16x2 h = __builtin_bit_cast(f16x2, w);
    v[0] = static_cast<float>(h[0]);
    v[1] = static_cast<float>(h[1]);
  }
}

// Nearest value of the activations' type, as a float.
template <int OF>
__device__ __forceinline__ float round_to(float v) {
  if constexpr (OF == kOutF32) return v;
  float r[2];
  unpack2<OF>(pack2<OF>(v, v), r);
  return r[0];
}

template <int OF>
__device__ __forceinline__ float load1(const void* row, uint32_t c) {
  if constexpr (OF == kOutF32) return static_cast<const float*>(row)[c];
  const uint32_t h = static_cast<const uint16_t*>(row)[c];
  float r[2];
  unpack2<OF>(h, r);
  return r[0];
}

template <int OF>
__device__ __forceinline__ void store1(void* row, uint32_t c, float v) {
  if constexpr (OF == kOutF32)
    static_cast<float*>(row)[c] = v;
  else
    static_cast<uint16_t*>(row)[c] = static_cast<uint16_t>(pack2<OF>(v, 0.0f));
}

// Elements [c, c + E) of a row, zeros from column h on. VEC: the row starts
// on a 16-byte boundary and h is a multiple of 8, so a piece is whole.
template <int OF, bool VEC, int E>
__device__ __forceinline__ void load_piece(const void* row, uint32_t c, uint32_t h, float* v) {
  if constexpr (VEC) {
    if (c < h) {
      if constexpr (OF == kOutF32) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(row) + c + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i + j] = a[j];
        }
      } else {
        static_assert(E == 8, "one 16-byte load");
        const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(row) + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack2<OF>(w[j], v + 2 * j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = c + j < h ? load1<OF>(row, c + j) : 0.0f;
  }
}

// One 16-byte store is made past the caches (norm of 2048 x 8192 bf16: 27.0 us
// through them, 26.3 past them); two of a lane (8 binary32 elements) cover
// half lines each, which the caches have to join (8192 x 5120 f32: 101 us, past
// them 112).
template <int OF, bool VEC, int E>
__device__ __forceinline__ void store_piece(void* row, uint32_t c, uint32_t h, const float* v) {
  if constexpr (VEC) {
    if (c < h) {
      if constexpr (OF == kOutF32) {
        f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(row) + c);
        if constexpr (E == 4) {
          __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, p);
        } else {
          p[0] = f32x4{v[0], v[1], v[2], v[3]};
          p[1] = f32x4{v[4], v[5], v[6], v[7]};
        }
      } else {
        static_assert(E == 8, "one 16-byte store");
        const u32x4 w = {pack2<OF>(v[0], v[1]), pack2<OF>(v[2], v[3]), pack2<OF>(v[4], v[5]), pack2<OF>(v[6], v[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(row) + c));
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (c + j < h) store1<OF>(row, c + j, v[j]);
  }
}

// E codes, four a word.
template <int E>
struct Codes {
  uint32_t w[E / 4];
};

template <bool VEC, int E>
__device__ __forceinline__ void store_codes(uint8_t* row, uint32_t c, uint32_t h, const Codes<E>& codes) {
  if constexpr (VEC) {
    if (c < h) {
      if constexpr (E == 8)
        *reinterpret_cast<u32x2*>(row + c) = u32x2{codes.w[0], codes.w[1]};
      else
        *reinterpret_cast<uint32_t*>(row + c) = codes.w[0];
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (c + j < h) row[c + j] = static_cast<uint8_t>(codes.w[j / 4] >> (8 * (j % 4)));
  }
}

// Lane l's value of v from the lane that the DPP control names.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
}

// quad_perm [1,0,3,2] and [2,3,0,1] combine the lanes of each quad; then
// row_half_mirror (lane i <-> 7-i) and row_mirror (i <-> 15-i) pair quads
// across the half row and the row of 16.
constexpr int kDppSwap1 = 0xB1, kDppSwap2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// Largest v of each aligned group of L consecutive lanes (4, 8, 16 or 32), in
// every lane of it. v holds the bits of a non-negative float, which order as
// integers do; NaN is above infinity, so it wins.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = max(v, dpp<kDppSwap1>(v));
  v = max(v, dpp<kDppSwap2>(v));
  if constexpr (L >= 8) v = max(v, dpp<kDppHalfMirror>(v));
  if constexpr (L >= 16) v = max(v, dpp<kDppMirror>(v));
  if constexpr (L >= 32) {
    constexpr int kXor16 = 0x401F;  // lane i <-> i ^ 16 of each half wave
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(v), kXor16)));
  }
  return v;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = group_max<16>(v);
  return max(max(lane_value(v, 0), lane_value(v, 16)), max(lane_value(v, 32), lane_value(v, 48)));
}

// Sum over the wave in a fixed order, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kDppSwap1>(v);
  v += dpp<kDppSwap2>(v);
  v += dpp<kDppHalfMirror>(v);
  v += dpp<kDppMirror>(v);
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return (__builtin_bit_cast(float, lane_value(b, 0)) + __builtin_bit_cast(float, lane_value(b, 16))) +
         (__builtin_bit_cast(float, lane_value(b, 32)) + __builtin_bit_cast(float, lane_value(b, 48)));
}

// A work-group barrier that orders LDS accesses alone: __syncthreads would also
// wait for the loads of the next row.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Between writes to LDS and reads of them by other lanes of the same wave, and
// between such reads and the next writes. LDS serves a wave's accesses in
// order, so this costs no instruction; it keeps the compiler from moving one
// across the other where a single lane's addresses differ.
__device__ __forceinline__ void lds_wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

template <int XF>
struct CodeFormat;
template <>
struct CodeFormat<kXInt8> {
  static constexpr float kMax = 127.0f;
};
template <>
struct CodeFormat<kXE4M3FN> {
  static constexpr float kMax = 448.0f;
  static constexpr int kEmax = 8;  // 448 = 1.75 * 2^8
};
template <>
struct CodeFormat<kXE5M2> {
  static constexpr float kMax = 57344.0f;
  static constexpr int kEmax = 15;  // 57344 = 1.75 * 2^15
};

// 2^k for k in [-127, 127] as an exact binary32 (2^-127 is subnormal).
__device__ __forceinline__ float exp2_int(int k) {
  return __builtin_bit_cast(float, k >= -126 ? static_cast<uint32_t>(k + 127) << 23 : 0x00400000u);
}

// What a group with this absolute maximum is multiplied by, and its scale.
// f32 scales: scale = amax / qmax, at least 2^-126 (zero groups included).
__device__ __forceinline__ float f32_multiplier(uint32_t amax_bits, float top, float* scale) {
  const float amax = __builtin_bit_cast(float, amax_bits);
  const float s = amax / top;
  const bool small = s < 0x1p-126f;
  *scale = small ? 0x1p-126f : s;
  return small ? 0x1p126f : top / amax;
}

// E8M0: the scale 2^(floor(log2 amax) - emax) limited to [2^-127, 2^127];
// zero groups take the smallest, NaN and infinity the NaN code.
template <int XF>
__device__ __forceinline__ float mx_multiplier(uint32_t amax_bits, uint32_t* code) {
  constexpr int kEmax = CodeFormat<XF>::kEmax;
  // floor(log2 amax) + 127 is the exponent field; subnormal maxima (below
  // 2^-126) fall under the lower limit like 2^-126 itself.
  const int field = static_cast<int>(amax_bits >> 23);
  const int shared = max(field - 127 - kEmax, -127);
  *code = field == 255 ? 255u : static_cast<uint32_t>(shared + 127);
  return exp2_int(-shared);
}

// E values times mul, clamped and rounded nearest-even to codes.
template <int XF, int E = kPiece>
__device__ __forceinline__ Codes<E> encode_piece(const float* v, float mul) {
  constexpr float kMax = CodeFormat<XF>::kMax;
  float q[E];
#pragma unroll
  for (int j = 0; j < E; ++j) q[j] = fminf(fmaxf(v[j] * mul, -kMax), kMax);
  Codes<E> codes;
#pragma unroll
  for (int k = 0; k < E / 4; ++k) {
    const float* p = q + 4 * k;
    if constexpr (XF == kXInt8) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = static_cast<uint32_t>(static_cast<int32_t>(__builtin_rintf(p[j]))) & 0xFFu;
      codes.w[k] = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
    } else if constexpr (XF == kXE4M3FN) {
      int t = __builtin_amdgcn_cvt_pk_fp8_f32(p[0], p[1], 0, false);
      codes.w[k] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(p[2], p[3], t, true));
    } else {
      int t = __builtin_amdgcn_cvt_pk_bf8_f32(p[0], p[1], 0, false);
      codes.w[k] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_bf8_f32(p[2], p[3], t, true));
    }
  }
  return codes;
}

}  // namespace dev
}  // namespace qrs
