// gfx950 kernel that quantizes 128 x 128 blocks of a matrix to 8-bit
// floating-point codes, and writes them as they lie, transposed, or both: the
// operands of the product in qrs_matmul_fp8.h and of its gradients.
//
//   scale = amax / qmax, codes = RNE(clamp(v * (qmax / amax), +-qmax))
//
// with amax over the block (weights), or over 128 columns of a row for the
// codes and 128 rows of a column for the transposed ones (activations and
// gradients, whose transposes are multiplied along the tokens).
//
// A work-group of 256 lanes holds a block in registers, 8 x 8 values a lane, so
// one read of the matrix serves both outputs. A lane's eight rows of a column are
// the eight bytes of a piece of the transpose, which goes through LDS and leaves in whole
// lines. The kernel is a stream, bound by HBM: bf16 7168 x 8192 with blocks 31 us
// (5.7 TB/s), with the transpose beside them 40 (5.8).

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

constexpr int kSide = 128;

// v: a piece's values -> their largest magnitude as bits (NaN above infinity).
__device__ __forceinline__ uint32_t max_bits(const float (&v)[kPiece]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kPiece; ++j) m = max(m, abs_bits(v[j]));
  return m;
}

// f32_multiplier, with zero for NaN: what lies beside a matrix's rows in a block is
// zero and has to stay so, whatever the rows hold.
__device__ __forceinline__ float block_multiplier(uint32_t amax, float top, float* scale) {
  const float mul = f32_multiplier(amax, top, scale);
  return mul == mul ? mul : 0.0f;
}

// A piece of x; 16-bit types as a stream that leaves no copy in the caches, of any size.
// us through the caches and as a stream, bf16 both ways from memory: 1021 x 5120 12.5 and
// 9.6, 4096 x 4096 17.9 and 15.1, 7168 x 8192 58.4 and 48.7; transposed alone 16384 x 8192
// 93 and 74; a linear layer's gradients, whose operands an operation just wrote, 1021 x
// 3584 x 4096 90.9 and 88.0, 4096 x 8192 x 7168 873 and 851. (Only a matrix of 130 to 240
// MB that is read again and again gains by a copy: 4096 x 8192 27.7 and 31.8; and 8192 x
// 8192 fp32 85 and 92.)
template <int IO, bool VEC>
__device__ __forceinline__ void load_values(const void* row, uint32_t c, uint32_t h, float* v) {
  if constexpr (VEC && IO != kOutF32) {
    RawPiece<IO, true> raw;
    raw.template load<true>(row, c, h);
    raw.get(v);
  } else {
    load_piece<IO, VEC, kPiece>(row, c, h, v);
  }
}

// STREAM: the transposed codes leave past the caches, for matrices whose input and
// outputs are more than half of the Infinity Cache's 256 MB and that write the rows' own
// codes beside them. us of blocks through the caches and so, bf16 1021 x 5120 8.9 and 8.9,
// 4096 x 4096 13.3 and 14.2, 4096 x 8192 28.6 and 27.6, 7168 x 8192 44.9 and 40.5, 16384 x
// 8192 116 and 95 (alone, 16384 x 8192 75 and 89). Products that read the codes next find
// them in the cache: with both products of 1021 tokens a weight of 3584 x 4096 66.7 and
// 72.3, a linear layer's gradients 4096 x 3584 x 4096 234 and 238; so do larger ones (of
// 4096 tokens, a weight of 8192 x 7168 497 and 511), but their own time gains more where
// nothing reads them at once.
constexpr uint64_t kStreamCodes = uint64_t{128} << 20;

template <int IO, int XF, bool BY_BLOCK, bool VEC, bool STREAM>
__global__ __launch_bounds__(256) void blocks_kernel(const BlocksLaunch a) {
  // The transposed codes: piece b (8 rows) of column c in slot b ^ (c / 8) of the
  // column's 128 bytes, which spreads the columns of a write over the banks.
  __shared__ __attribute__((aligned(16))) uint8_t turned[kSide * kSide];
  __shared__ uint32_t maxima[4][kSide];
  __shared__ float row_mul[kSide], col_mul[kSide];
  const uint32_t tiles_c = static_cast<uint32_t>((a.cols + kSide - 1) / kSide);
  const uint32_t tr = blockIdx.x / tiles_c, tc = blockIdx.x % tiles_c;
  const uint64_t r0 = static_cast<uint64_t>(tr) * kSide, c0 = static_cast<uint64_t>(tc) * kSide;
  const uint32_t rows = static_cast<uint32_t>(min<uint64_t>(kSide, a.rows - r0));
  const uint32_t cols = static_cast<uint32_t>(min<uint64_t>(kSide, a.cols - c0));
  const uint32_t wave = threadIdx.x / 64, pc = threadIdx.x % 16, pr = threadIdx.x / 16;

  // Rows 8 pr .. + 7, columns 8 pc .. + 7; zeros outside.
  float v[kPiece][kPiece];
  const char* x = static_cast<const char*>(a.x) + (r0 * a.x_stride + c0) * kOutSize<IO>;
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    const uint32_t r = pr * kPiece + i;
    load_values<IO, VEC>(x + static_cast<uint64_t>(min(r, rows - 1)) * a.x_stride * kOutSize<IO>, pc * kPiece,
                         r < rows ? cols : 0, v[i]);
  }

  constexpr float kMax = CodeFormat<XF>::kMax;
  float block_mul = 0.0f, block_scale = 0.0f;
  if constexpr (BY_BLOCK) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) amax = max(amax, max_bits(v[i]));
    amax = wave_max(amax);
    if (threadIdx.x % 64 == 0) maxima[wave][0] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) amax = max(amax, maxima[i][0]);
    block_mul = block_multiplier(amax, kMax, &block_scale);
    if (threadIdx.x == 0) {
      const uint32_t tiles_r = static_cast<uint32_t>((a.rows + kSide - 1) / kSide);
      if (a.codes) a.scales[static_cast<uint64_t>(tr) * tiles_c + tc] = block_scale;
      if (a.codes_t) a.scales_t[static_cast<uint64_t>(tc) * tiles_r + tr] = block_scale;
    }
  }
  if constexpr (!BY_BLOCK) {
    // A group's two divisions are made once: a row's by one of the 16 lanes that hold
    // it, a column's by one of the work-group (4096 x 8192 bf16 both ways 32 us, by
    // every lane 36).
    if (a.codes) {
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const uint32_t amax = group_max<16>(max_bits(v[i]));
        mine = pc == static_cast<uint32_t>(i) ? amax : mine;
      }
      const uint32_t r = pr * kPiece + pc;
      if (pc < kPiece) {
        float scale;
        row_mul[r] = block_multiplier(mine, kMax, &scale);
        if (r < rows) a.scales[(r0 + r) * tiles_c + tc] = scale;
      }
    }
    if (a.codes_t) {
      // Lanes 16 apart hold the same columns.
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) m = max(m, abs_bits(v[i][j]));
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
        if (threadIdx.x % 64 < 16) maxima[wave][pc * kPiece + j] = m;
      }
      __syncthreads();
      const uint32_t c = threadIdx.x;
      if (c < kSide) {
        const uint32_t tiles_r = static_cast<uint32_t>((a.rows + kSide - 1) / kSide);
        float scale;
        col_mul[c] = block_multiplier(max(max(maxima[0][c], maxima[1][c]), max(maxima[2][c], maxima[3][c])), kMax, &scale);
        if (c < cols) a.scales_t[(c0 + c) * tiles_r + tr] = scale;
      }
    }
    __syncthreads();
  }
  if (a.codes) {
    uint8_t* out = static_cast<uint8_t*>(a.codes) + r0 * a.codes_stride + c0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const uint32_t r = pr * kPiece + i;
      const float mul = BY_BLOCK ? block_mul : row_mul[r];
      if (r < rows) store_codes<VEC, kPiece>(out + r * a.codes_stride, pc * kPiece, cols, encode_piece<XF>(v[i], mul));
    }
  }
  if (!a.codes_t) return;

#pragma unroll
  for (int j = 0; j < kPiece; ++j) {
    float column[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) column[i] = v[i][j];
    const Codes<kPiece> codes = encode_piece<XF>(column, BY_BLOCK ? block_mul : col_mul[pc * kPiece + j]);
    *reinterpret_cast<u32x2*>(turned + (pc * kPiece + j) * kSide + (pr ^ pc) * kPiece) = u32x2{codes.w[0], codes.w[1]};
  }
  __syncthreads();
  // 16 rows of a column a lane.
  const uint32_t rows_t = static_cast<uint32_t>(min<uint64_t>(kSide, a.rows_t - r0));
  uint8_t* out = static_cast<uint8_t*>(a.codes_t) + c0 * a.codes_t_stride + r0;
  const uint32_t r = threadIdx.x % 8 * 16;
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    const uint32_t c = i * 32 + threadIdx.x / 8, key = c / kPiece;
    u32x4 w = *reinterpret_cast<const u32x4*>(turned + c * kSide + ((r / kPiece) ^ (key & ~1u)) * kPiece);
    if (key % 2) w = u32x4{w[2], w[3], w[0], w[1]};
    if (c >= cols) continue;
    uint8_t* to = out + c * a.codes_t_stride + r;
    if (a.vec_t) {
      u32x4* p = reinterpret_cast<u32x4*>(to);
      if (r >= rows_t) continue;
      if constexpr (STREAM)
        __builtin_nontemporal_store(w, p);
      else
        *p = w;
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (r + j < rows_t) to[j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
    }
  }
}

template <int IO, int XF, bool BY_BLOCK>
hipError_t launch_typed(const BlocksLaunch& l, hipStream_t stream) {
  const uint64_t tiles = (l.rows + kSide - 1) / kSide * ((l.cols + kSide - 1) / kSide);
  if (tiles == 0 || tiles >= uint64_t{1} << 24) return hipErrorInvalidValue;  // a grid holds fewer than 2^32 work-items
  const bool stream_t = l.codes && l.codes_t && l.rows * l.cols * (kOutSize<IO> + 2) > kStreamCodes;
  return launch_kernel(!l.vec     ? blocks_kernel<IO, XF, BY_BLOCK, false, false>
                       : stream_t ? blocks_kernel<IO, XF, BY_BLOCK, true, true>
                                  : blocks_kernel<IO, XF, BY_BLOCK, true, false>,
                       dim3(static_cast<uint32_t>(tiles)), dim3(256), stream, l);
}

template <int IO>
hipError_t launch_io(const BlocksLaunch& l, hipStream_t stream) {
  if (l.x_format == kXE4M3FN)
    return l.by_block ? launch_typed<IO, kXE4M3FN, true>(l, stream) : launch_typed<IO, kXE4M3FN, false>(l, stream);
  if (l.x_format == kXE5M2)
    return l.by_block ? launch_typed<IO, kXE5M2, true>(l, stream) : launch_typed<IO, kXE5M2, false>(l, stream);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_blocks(const BlocksLaunch& l, hipStream_t stream) {
  switch (l.io_format) {
    case kOutF32: return launch_io<kOutF32>(l, stream);
    case kOutBF16: return launch_io<kOutBF16>(l, stream);
    case kOutF16: return launch_io<kOutF16>(l, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace qrs
