// gfx950 kernels of the product of 8-bit floating-point codes with scales for
// groups of 128 of k,
//
//   out[i][j] = sum_g (sum_{k in g} a[i][k] * b[j][k]) * fp32(a_scales[i][g] * b_scales[j or j / 128][g])
//
// of its gated form silu(gate) * up (two products over the same tokens), and of
// both as codes and scales.
//
// The matrix instructions for 8-bit floats add the products of eight consecutive
// codes with 2^-14 of the largest one as the last place (measured: 448 * 448 + 4
// is 448 * 448, where the 4 stands in the same eight): 1.5e-5 of the result's norm for
// normal values, 100 times what binary32 sums leave. So codes are widened to
// bfloat16, which holds every one of them (two codes an instruction), and the
// bfloat16 instructions, whose sums keep binary32 (1e-8 of the norm), multiply them at half the
// rate. Kernels that wait for memory lose nothing by it.
//
// A group's sums of a 16 x 16 fragment are four instructions of 32 k; they are
// then multiplied by the scales' product and added in binary32 by one fused
// operation, and rounded once at the end.
//
// b is the first operand of the matrix instructions and a the second: a lane
// then holds four consecutive output channels of one token. Of a group's 128
// codes of a row a lane multiplies 32, the chunks lane / 16 and 4 + lane / 16 of 16
// bytes: which ones does not matter as long as both operands agree.
//
// This file is compiled once for each pair of formats (qrs_matmul_fp8_*.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qrs_device.h"
#include "qrs_layer.h"
#include "qrs_matmul_device.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace {

using namespace dev;

// What a kernel instance multiplies.
enum Form : int { kPlain = 0, kGatedForm = 1, kGrouped = 2 };

constexpr uint32_t kGroup = 128;  // of k: a scale of a, and of b

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes as bfloat16.
template <XFormat F>
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
  bf16x2 p[4];
  if constexpr (F == kXE4M3FN) {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  } else {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
  }
  const u32x4 w = {__builtin_bit_cast(uint32_t, p[0]), __builtin_bit_cast(uint32_t, p[1]),
                   __builtin_bit_cast(uint32_t, p[2]), __builtin_bit_cast(uint32_t, p[3])};
  return __builtin_bit_cast(bf16x8, w);
}

// A lane's 16 N codes of a fragment.
template <int N>
struct Wide {
  bf16x8 part[2 * N];

  template <XFormat F>
  __device__ __forceinline__ void set(int n, const i32x4& codes) {
    part[2 * n] = widen<F>(codes[0], codes[1]);
    part[2 * n + 1] = widen<F>(codes[2], codes[3]);
  }
};

// The sums of a 16 x 16 fragment over its 64 N codes of each row.
template <int N>
__device__ __forceinline__ f32x4 group_sums(const Wide<N>& b, const Wide<N>& a) {
  f32x4 sums = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = 0; t < 2 * N; ++t) sums = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.part[t], a.part[t], sums, 0, 0, 0);
  return sums;
}

__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& sums, float scale) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(sums[e], scale, acc[e]);
}
__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& sums, float a_scale, const f32x4& b_scales) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(sums[e], a_scale * b_scales[e], acc[e]);
}

// Eight outputs [j0, j0 + 8) of token i: v, or silu(v) * up. Where codes are
// written, all lanes of a group (16 or 4 consecutive ones) call this together.
template <int FORM>
__device__ __forceinline__ void finish_outputs(const MatmulFp8Launch& a, uint32_t i, uint32_t j0, bool active, float* v,
                                               const float* up) {
  if constexpr (FORM == kGatedForm) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) v[j] = silu(v[j]) * up[j];
  }
  if (FORM != kGrouped && a.quantize) {
    finish_codes(a, i, j0, active, false, v);
  } else if (active) {
    if (a.out_format == kOutF32)
      finish_values<kOutF32>(a, i, j0, v);
    else if (a.out_format == kOutBF16)
      finish_values<kOutBF16>(a, i, j0, v);
    else
      finish_values<kOutF16>(a, i, j0, v);
  }
}

// ---- general tile kernel -----------------------------------------------

// 64 tokens by 128 outputs (gated: 128 gate and 128 up rows of b), a group of k
// at a time through LDS, four waves of 64 tokens each. For operands off 16-byte
// boundaries and offsets past 30 bits.
constexpr int kTileM = 64, kTileN = 128;

template <int FORM>
struct Tile {
  static constexpr int kRows = FORM == kGatedForm ? 2 * kTileN : kTileN;  // of b
  static constexpr int kPitch = kGroup + 16;                              // bytes of a staged row
  static constexpr int kCPitch = kRows + 4;                               // words of the staged sums
  static constexpr int kOperands = (kTileM + kRows) * kPitch, kSums = kTileM * kCPitch * 4;
  static constexpr int kLds = kOperands > kSums ? kOperands : kSums;
  static constexpr int FM = kTileM / 16, FN = kRows / 4 / 16;
};

template <XFormat AF, XFormat BF, bool VEC, int FORM>
__global__ __launch_bounds__(256) void tile_kernel(const MatmulFp8Launch a) {
  using T = Tile<FORM>;
  constexpr int FM = T::FM, FN = T::FN;
  __shared__ __attribute__((aligned(16))) char lds[T::kLds];
  char* la = lds;
  char* lb = lds + kTileM * T::kPitch;
  const uint32_t tiles_n = (a.n + kTileN - 1) / kTileN;
  const uint32_t i0 = blockIdx.x / tiles_n * kTileM;
  const uint32_t j0 = blockIdx.x % tiles_n * kTileN;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  // Row r of the tile's part of b.
  auto row_of = [&](uint32_t r) { return min(j0 + r % kTileN, a.n - 1) + (r >= kTileN ? a.n : 0); };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const float* sa[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i)
    sa[i] = a.a_scales + static_cast<uint64_t>(min(i0 + 16 * i + lane % 16, a.m - 1)) * a.groups;
  // The wave's 16 FN rows of b lie in one block.
  const float* sb = a.b_scales + static_cast<uint64_t>(j0 / kTileN + (wave >= 2 && FORM == kGatedForm ? a.up_block : 0)) * a.groups;

  for (uint32_t g = 0; g < a.groups; ++g) {
    const uint32_t r = threadIdx.x / 8, chunk = threadIdx.x % 8 * 16;
    constexpr int kA = kTileM / 32, kB = T::kRows / 32;
    u32x4 w[kA + kB];
#pragma unroll
    for (int t = 0; t < kA + kB; ++t) {
      // Rows past the end: the last one, not stored.
      const int8_t* row = t < kA ? a.a + min(i0 + r + 32 * t, a.m - 1) * a.a_stride
                                 : a.b + static_cast<uint64_t>(row_of(r + 32 * (t - kA))) * a.b_stride;
      w[t] = load16<VEC>(row, g * kGroup + chunk, a.k);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kA + kB; ++t)
      *reinterpret_cast<u32x4*>((t < kA ? la + (r + 32 * t) * T::kPitch : lb + (r + 32 * (t - kA)) * T::kPitch) + chunk) = w[t];
    __syncthreads();
    auto fragment = [&](const char* rows, int n) {
      return *reinterpret_cast<const i32x4*>(rows + lane % 16 * T::kPitch + lane / 16 * 16 + n * 64);
    };
    Wide<2> fb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int n = 0; n < 2; ++n) fb[j].template set<BF>(n, fragment(lb + (FN * wave + j) * 16 * T::kPitch, n));
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      Wide<2> fa;
#pragma unroll
      for (int n = 0; n < 2; ++n) fa.template set<AF>(n, fragment(la + i * 16 * T::kPitch, n));
      const float token = sa[i][g];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const f32x4 sums = group_sums(fb[j], fa);
        if constexpr (FORM == kGrouped) {
          f32x4 s;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[e] = a.b_scales[static_cast<uint64_t>(row_of((FN * wave + j) * 16 + lane / 16 * 4 + e)) * a.groups + g];
          add_scaled(acc[i][j], sums, token, s);
        } else {
          add_scaled(acc[i][j], sums, token * sb[g]);
        }
      }
    }
  }
  __syncthreads();
  // Lane l holds channels 4 (l / 16) .. + 3 of token l % 16 of each fragment.
  float* lc = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      *reinterpret_cast<f32x4*>(lc + (16 * i + lane % 16) * T::kCPitch + (FN * wave + j) * 16 + lane / 16 * 4) = acc[i][j];
  __syncthreads();
  constexpr uint32_t pieces = kTileN / kPiece;
  for (uint32_t t = threadIdx.x; t < kTileM * pieces; t += 256) {
    const uint32_t i = t / pieces, j = t % pieces * kPiece;
    const float* p = lc + i * T::kCPitch + j;
    float v[kPiece], up[kPiece];
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      v[e] = p[e];
      if constexpr (FORM == kGatedForm) up[e] = p[kTileN + e];
    }
    finish_outputs<FORM>(a, i0 + i, j0 + j, i0 + i < a.m && j0 + j < a.n, v, up);
  }
}

// A kernel and its grid for a call.
struct Choice {
  MatmulKernel id;
  void (*kernel)(MatmulFp8Launch);
  uint64_t blocks;
  uint32_t threads;

  // A HIP grid holds fewer than 2^32 work-items.
  bool fits() const { return blocks * threads < uint64_t{1} << 32; }
};

uint64_t tiles_of(const MatmulFp8Launch& l, uint32_t tile_m, uint32_t outputs) {
  return static_cast<uint64_t>((l.m + tile_m - 1) / tile_m) * ((l.n + outputs - 1) / outputs);
}

template <XFormat AF, XFormat BF, bool VEC, int FORM>
Choice general_tiles(const MatmulFp8Launch& l) {
  return {{kMatmulTiles, kTileM, static_cast<uint32_t>(Tile<FORM>::kRows)}, tile_kernel<AF, BF, VEC, FORM>,
          tiles_of(l, kTileM, kTileN), 256};
}

template <XFormat AF, XFormat BF, int FORM>
Choice choose_form(const MatmulFp8Launch& l) {
  return l.vec ? general_tiles<AF, BF, true, FORM>(l) : general_tiles<AF, BF, false, FORM>(l);
}

template <XFormat AF, XFormat BF>
Choice choose(const MatmulFp8Launch& l) {
  if (l.grouped) return choose_form<AF, BF, kGrouped>(l);
  return l.gated ? choose_form<AF, BF, kGatedForm>(l) : choose_form<AF, BF, kPlain>(l);
}

template <XFormat AF, XFormat BF>
hipError_t launch_formats(const MatmulFp8Launch& l, hipStream_t stream) {
  const Choice c = choose<AF, BF>(l);
  if (!c.fits()) return hipErrorInvalidValue;
  return launch_kernel(c.kernel, dim3(static_cast<uint32_t>(c.blocks)), dim3(c.threads), stream, l);
}

}  // namespace

hipError_t launch_fp8_e4m3_e4m3(const MatmulFp8Launch& l, hipStream_t stream);
hipError_t launch_fp8_e4m3_e5m2(const MatmulFp8Launch& l, hipStream_t stream);
hipError_t launch_fp8_e5m2_e4m3(const MatmulFp8Launch& l, hipStream_t stream);
hipError_t launch_fp8_e5m2_e5m2(const MatmulFp8Launch& l, hipStream_t stream);

}  // namespace qrs
