// gfx950 kernels of the 8-bit integer product
//
//   out[i][j] = fp32(fp32(sum_k a[i][k] * b[j][k]) * a_scales[i]) * b_scales[j]
//
// and of its gated form silu(g) * u (two products over the same tokens) and
// quantized form (codes and scales of one rank's partial sums). The sums are
// exact in 32-bit integers, so any split of k or of the tiles gives the same
// bits, and only the epilogue rounds: once to binary32, once for each scale,
// once to the output.
//
// b is the first operand of the matrix instructions and a the second: a lane
// then holds consecutive output channels of one token, which is how the
// epilogue stages the sums through LDS into 8-channel pieces.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qrs_device.h"
#include "qrs_layer.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace {

using namespace dev;

// ---- epilogue ----------------------------------------------------------

__device__ __forceinline__ void channel_scales(const float* s, uint32_t n, uint32_t j0, float* v) {
#pragma unroll
  for (int j = 0; j < kPiece; ++j) v[j] = j0 + j < n ? s[j0 + j] : 0.0f;
}

// Eight outputs [j0, j0 + 8) of token i from their integer sums. `active`
// says whether i and j0 are inside the output; in the quantized form all
// lanes of a group (16 or 4 consecutive ones) call this together.
__device__ __forceinline__ void finish_piece(const MatmulLaunch& a, uint32_t i, uint32_t j0, bool active,
                                             const int32_t* acc, const int32_t* up) {
  float v[kPiece], sb[kPiece];
  const float sa = active ? a.a_scales[i] : 0.0f;
  channel_scales(a.b_scales, active ? a.n : 0, j0, sb);
#pragma unroll
  for (int j = 0; j < kPiece; ++j) v[j] = static_cast<float>(acc[j]) * sa * sb[j];
  if (a.quantize) {
    uint8_t* codes_row = static_cast<uint8_t*>(a.out) + static_cast<uint64_t>(i) * a.out_stride;
    if (a.scale_layout == kScaleF32Group128) {
      const uint64_t first = static_cast<uint64_t>(i) * (a.n / 128);
      if (a.x_format == kXE4M3FN)
        quantize_group_piece<kXE4M3FN, kScaleF32Group128, true>(v, active, j0, a.n, codes_row, a.scales, first);
      else if (a.x_format == kXE5M2)
        quantize_group_piece<kXE5M2, kScaleF32Group128, true>(v, active, j0, a.n, codes_row, a.scales, first);
      else
        quantize_group_piece<kXInt8, kScaleF32Group128, true>(v, active, j0, a.n, codes_row, a.scales, first);
    } else {
      const uint64_t first = static_cast<uint64_t>(i) * (a.n / 32);
      if (a.x_format == kXE4M3FN)
        quantize_group_piece<kXE4M3FN, kScaleE8M0Block32, true>(v, active, j0, a.n, codes_row, a.scales, first);
      else
        quantize_group_piece<kXE5M2, kScaleE8M0Block32, true>(v, active, j0, a.n, codes_row, a.scales, first);
    }
    return;
  }
  if (!active) return;
  if (a.gated) {
    channel_scales(a.b_scales + a.n, a.n, j0, sb);
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const float u = static_cast<float>(up[j]) * sa * sb[j];
      v[j] = v[j] / (1.0f + expf(-v[j])) * u;
    }
  }
  const uint64_t row = static_cast<uint64_t>(i) * a.out_stride;
  const bool whole = a.out_vec && j0 + kPiece <= a.n;
  if (a.out_format == kOutF32) {
    float* p = static_cast<float*>(a.out) + row;
    whole ? store_piece<kOutF32, true>(p, j0, a.n, v) : store_piece<kOutF32, false>(p, j0, a.n, v);
  } else if (a.out_format == kOutBF16) {
    uint16_t* p = static_cast<uint16_t*>(a.out) + row;
    whole ? store_piece<kOutBF16, true>(p, j0, a.n, v) : store_piece<kOutBF16, false>(p, j0, a.n, v);
  } else {
    uint16_t* p = static_cast<uint16_t*>(a.out) + row;
    whole ? store_piece<kOutF16, true>(p, j0, a.n, v) : store_piece<kOutF16, false>(p, j0, a.n, v);
  }
}

// ---- general tile kernel -----------------------------------------------

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

// 64 tokens by 128 rows of b (gated: 64 gate and 64 up channels), 64 bytes
// of k at a time through LDS. Four waves, each 64 tokens by 32 rows of b in
// 16x16x64 products.
constexpr int kTileM = 64, kTileN = 128, kTileK = 64;
constexpr int kPitch = kTileK + 16;   // bytes; rows 5 quarter-lines apart
constexpr int kCPitch = kTileN + 4;   // words of the staged sums

template <bool VEC>
__global__ __launch_bounds__(256) void tile_kernel(const MatmulLaunch a) {
  __shared__ __attribute__((aligned(16))) char lds[kTileM * kCPitch * 4];
  static_assert((kTileM + kTileN) * kPitch <= kTileM * kCPitch * 4, "operands share the staging buffer");
  char* la = lds;
  char* lb = lds + kTileM * kPitch;
  const uint32_t tile_n = a.gated ? kTileN / 2 : kTileN;
  const uint32_t tiles_n = (a.n + tile_n - 1) / tile_n;
  const uint32_t i0 = blockIdx.x / tiles_n * kTileM;
  const uint32_t j0 = blockIdx.x % tiles_n * tile_n;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;

  i32x4 acc[4][2];  // [token frag][b frag]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  // Thread t loads chunk t % 4 (16 bytes) of rows t / 4 and, for b, 64 more.
  const uint32_t r = threadIdx.x / 4, chunk = threadIdx.x % 4 * 16;
  const uint32_t ra = min(i0 + r, a.m - 1);  // rows past the end: any row, not stored
  const int8_t* pa = a.a + ra * a.a_stride;
  const int8_t* pb[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t rb = a.gated ? min(j0 + r, a.n - 1) + (h ? a.n : 0) : min(j0 + r + 64 * h, a.n - 1);
    pb[h] = a.b + rb * a.b_stride;
  }
  for (uint32_t k0 = 0; k0 < a.k; k0 += kTileK) {
    const u32x4 wa = load16<VEC>(pa, k0 + chunk, a.k);
    const u32x4 wb0 = load16<VEC>(pb[0], k0 + chunk, a.k);
    const u32x4 wb1 = load16<VEC>(pb[1], k0 + chunk, a.k);
    __syncthreads();
    *reinterpret_cast<u32x4*>(la + r * kPitch + chunk) = wa;
    *reinterpret_cast<u32x4*>(lb + r * kPitch + chunk) = wb0;
    *reinterpret_cast<u32x4*>(lb + (r + 64) * kPitch + chunk) = wb1;
    __syncthreads();
    i32x4 fa[4], fb[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      fa[i] = *reinterpret_cast<const i32x4*>(la + (16 * i + lane % 16) * kPitch + lane / 16 * 16);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      fb[j] = *reinterpret_cast<const i32x4*>(lb + (32 * wave + 16 * j + lane % 16) * kPitch + lane / 16 * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
  }
  __syncthreads();
  // Lane l holds channels 4 * (l / 16) .. + 3 of token l % 16 of each frag.
  int32_t* lc = reinterpret_cast<int32_t*>(lds);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<i32x4*>(lc + (16 * i + lane % 16) * kCPitch + 32 * wave + 16 * j + lane / 16 * 4) = acc[i][j];
  __syncthreads();
  const uint32_t pieces = tile_n / kPiece;
  for (uint32_t t = threadIdx.x; t < kTileM * pieces; t += 256) {
    const uint32_t i = t / pieces, j = t % pieces * kPiece;
    const int32_t* p = lc + i * kCPitch + j;
    finish_piece(a, i0 + i, j0 + j, i0 + i < a.m && j0 + j < a.n, p, p + kTileN / 2);
  }
}

template <bool VEC>
hipError_t launch_tiles(const MatmulLaunch& l, hipStream_t stream) {
  const uint32_t tile_n = l.gated ? kTileN / 2 : kTileN;
  const uint64_t tiles = static_cast<uint64_t>((l.m + kTileM - 1) / kTileM) * ((l.n + tile_n - 1) / tile_n);
  if (tiles >= uint64_t{1} << 24) return hipErrorInvalidValue;  // 2^32 work-items
  return launch_kernel(tile_kernel<VEC>, dim3(static_cast<uint32_t>(tiles)), dim3(256), stream, l);
}

}  // namespace

uint64_t matmul_workspace_bytes(uint32_t, uint32_t, uint32_t, bool) { return 0; }

hipError_t launch_matmul(const MatmulLaunch& l, hipStream_t stream) {
  return l.vec ? launch_tiles<true>(l, stream) : launch_tiles<false>(l, stream);
}

}  // namespace qrs
