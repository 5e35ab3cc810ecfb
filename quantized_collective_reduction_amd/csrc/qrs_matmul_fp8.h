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

// ---- pipelined tile kernel ---------------------------------------------

// 256 tokens by 256 rows of b, a group of k a block, two blocks in LDS. Eight
// waves of 64 tokens by 128 rows of b. Work-groups stay on the card and walk over
// tiles; operands and scales go from memory straight into LDS, a block ahead and
// across the end of a tile, so that a tile's epilogue runs while the next one's
// first block arrives.
//
// A load covers 8 rows of 128 bytes. Chunk c (16 bytes) of row r lies in slot
// c ^ (r / 2 % 8), which keeps a wave's reads of 16 rows off each other's banks;
// the loads fill LDS in lane order, so each lane asks for the chunk that belongs in
// its slot. One more load a wave brings the scales of 64 of the 512 rows.
//
// In the gated form a wave's rows of b are 32 gates, their ups, 32 gates and
// their ups.
struct Pipe {
  static constexpr int kSide = 256, kThreads = 512, kWaveM = 64, kWaveN = 128;
  static constexpr int FM = kWaveM / 16, FN = kWaveN / 16;
  static constexpr int kLoads = 4;  // of a, and of b, for each wave
  static constexpr int kOperands = 2 * kSide * static_cast<int>(kGroup), kBlock = kOperands + 2 * kSide * 4;
  static constexpr int kMaxima = 2 * kBlock, kLds = kMaxima + 2 * kSide * 4;
};

// Rows of 16 lanes: first's odd ones exchanged with second's even ones.
__device__ __forceinline__ void swap_rows(float& first, float& second) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, first),
                                                  __builtin_bit_cast(uint32_t, second), false, false);
  const uint32_t one = r[0], other = r[1];  // a bit_cast of a vector's element takes the first one
  first = __builtin_bit_cast(float, one);
  second = __builtin_bit_cast(float, other);
}

// The largest of lanes l % 16 + 16 {0, 1, 2, 3}, in each of them.
__device__ __forceinline__ uint32_t rows_max(uint32_t v) {
  auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(r[0], r[1]);
}

// What a group with this maximum is multiplied by, and its scale (E8M0 code or
// binary32 bits); codes of a piece.
__device__ __forceinline__ float code_multiplier(const MatmulLaunch& a, uint32_t amax, uint32_t* scale_bits) {
  if (a.scale_layout == kScaleE8M0Block32)
    return a.x_format == kXE4M3FN ? mx_multiplier<kXE4M3FN>(amax, scale_bits) : mx_multiplier<kXE5M2>(amax, scale_bits);
  const float top = a.x_format == kXE4M3FN ? CodeFormat<kXE4M3FN>::kMax
                    : a.x_format == kXE5M2 ? CodeFormat<kXE5M2>::kMax
                                           : CodeFormat<kXInt8>::kMax;
  float scale;
  const float mul = f32_multiplier(amax, top, &scale);
  *scale_bits = __builtin_bit_cast(uint32_t, scale);
  return mul;
}
__device__ __forceinline__ Codes<kPiece> encode_as(const MatmulLaunch& a, const float* v, float mul) {
  if (a.x_format == kXE4M3FN) return encode_piece<kXE4M3FN>(v, mul);
  if (a.x_format == kXE5M2) return encode_piece<kXE5M2>(v, mul);
  return encode_piece<kXInt8>(v, mul);
}
__device__ __forceinline__ uint32_t max_bits(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kPiece; ++j) m = max(m, abs_bits(v[j]));
  return m;
}

template <XFormat AF, XFormat BF, int FORM>
__global__ __launch_bounds__(Pipe::kThreads, 2) void pipe_kernel(const MatmulFp8Launch a) {
#ifdef __HIP_DEVICE_COMPILE__  // the buffer builtins' types exist in the device pass alone
  using P = Pipe;
  constexpr int FM = P::FM, FN = P::FN;
  __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave % 4, wn = wave / 4;

  // Work-groups go round the eight XCDs: XCD x runs one eighth of the tiles,
  // consecutive ones, its work-groups taking every (gridDim / 8)th.
  constexpr uint32_t kOut = FORM == kGatedForm ? P::kSide / 2 : P::kSide, kWaveOut = kOut / 2;
  const TileOrder order = {(a.m + P::kSide - 1) / P::kSide, (a.n + kOut - 1) / kOut};
  const uint32_t tiles = order.tiles_m * order.tiles_n;
  const uint32_t xcd = blockIdx.x % 8, stride = gridDim.x / 8;
  const uint32_t end = (tiles / 8) * (xcd + 1) + min(xcd + 1, tiles % 8);
  uint32_t tile = (tiles / 8) * xcd + min(xcd, tiles % 8) + blockIdx.x / 8;
  if (tile >= end) return;

  // The loads' cursor: a tile, a block in it, and the lanes' offsets.
  __amdgpu_buffer_rsrc_t ra, rb, rs;
  uint32_t off_a[P::kLoads], off_b[P::kLoads], off_s = 0;
  uint32_t load_tile = tile, load_block = 0, load_slot = 0;
  // The chunk of an even or odd load: rows 8 t + l / 8, so r / 2 % 8 = 4 (t % 2) + l / 16.
  const uint32_t chunk[2] = {(lane % 8 ^ lane / 16) * 16u, (lane % 8 ^ (4 + lane / 16)) * 16u};
  auto aim_tile = [&]() {
    uint32_t tm, tn;
    order.at(load_tile, &tm, &tn);
    const uint32_t i0 = tm * P::kSide, j0 = tn * kOut;
    ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.a + static_cast<uint64_t>(i0) * a.a_stride), 0, kFar,
                                           0x00020000);
    rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.b + static_cast<uint64_t>(j0) * a.b_stride), 0, kFar,
                                           0x00020000);
    // Rows past the end load the last row; what they give is not stored. Row r of
    // the tile's part of b is channel channel(r), an up if up(r).
    auto channel = [&](uint32_t r) {
      if constexpr (FORM == kGatedForm) return min(j0 + r / 64 * 32 + r % 32, a.n - 1);
      return min(j0 + r, a.n - 1);
    };
    auto up = [](uint32_t r) { return FORM == kGatedForm && r / 32 % 2 == 1; };
#pragma unroll
    for (int t = 0; t < P::kLoads; ++t) {
      const uint32_t r = (wave * P::kLoads + t) * 8 + lane / 8;
      off_a[t] = (min(i0 + r, a.m - 1) - i0) * static_cast<uint32_t>(a.a_stride) + chunk[t % 2];
      off_b[t] = (channel(r) - j0 + (up(r) ? a.n : 0)) * static_cast<uint32_t>(a.b_stride) + chunk[t % 2];
    }
    const uint32_t r = wave % 4 * 64 + lane;
    uint32_t first, row;  // of the scales: the tile's, and this lane's
    if (wave < 4) {
      first = i0;
      row = min(i0 + r, a.m - 1);
    } else {
      first = FORM == kGrouped ? j0 : j0 / kGroup;
      row = FORM == kGrouped ? channel(r) : channel(r) / kGroup + (up(r) ? a.up_block : 0);
    }
    const float* scales = (wave < 4 ? a.a_scales : a.b_scales) + static_cast<uint64_t>(first) * a.groups;
    rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(scales), 0, kFar, 0x00020000);
    off_s = (row - first) * a.groups * 4;
  };
  auto load = [&]() {
    const uint32_t k = __builtin_amdgcn_readfirstlane(load_block * kGroup);
    char* base = lds + load_slot * P::kBlock;
#pragma unroll
    for (int t = 0; t < P::kLoads; ++t) {
      const uint32_t far = k + chunk[t % 2] < a.k ? 0 : kFar;  // past the end of k: zeros
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(base + (wave * P::kLoads + t) * 1024), 16, off_a[t] + far, k,
                                               0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (lds_ptr)(base + P::kSide * kGroup + (wave * P::kLoads + t) * 1024), 16, off_b[t] + far, k, 0, 0);
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(base + P::kOperands + wave * 256), 4, off_s,
                                             __builtin_amdgcn_readfirstlane(load_block * 4), 0, 0);
  };
  auto advance = [&]() {  // whether there is a block
    load_slot ^= 1;
    if (++load_block == a.groups) {
      load_block = 0;
      load_tile += stride;
      if (load_tile >= end) return false;
      aim_tile();
    }
    return true;
  };

  // Lane l reads row l % 16 of a fragment, chunks l / 16 and 4 + l / 16.
  const uint32_t lane_off[2] = {lane % 16 * kGroup + ((lane / 16) ^ (lane % 16 / 2)) * 16u,
                                lane % 16 * kGroup + ((4 + lane / 16) ^ (lane % 16 / 2)) * 16u};
  f32x4 acc[FM][FN];
  auto compute = [&](uint32_t slot) {
    const char* base = lds + slot * P::kBlock;
    const char* la = base + wm * P::kWaveM * kGroup;
    const char* lb = base + P::kSide * kGroup + wn * P::kWaveN * kGroup;
    const float* sa = reinterpret_cast<const float*>(base + P::kOperands) + wm * P::kWaveM + lane % 16;
    const float* sb = reinterpret_cast<const float*>(base + P::kOperands) + P::kSide + wn * P::kWaveN;
    float token[FM], scale[FORM == kGatedForm ? 2 : 1][FM];
    Wide<2> fa[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      token[i] = sa[16 * i];
#pragma unroll
      for (int n = 0; n < 2; ++n)
        fa[i].template set<AF>(n, *reinterpret_cast<const i32x4*>(la + lane_off[n] + i * 16 * kGroup));
    }
    if constexpr (FORM != kGrouped) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        scale[0][i] = token[i] * sb[0];
        if constexpr (FORM == kGatedForm) scale[1][i] = token[i] * sb[32];
      }
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      Wide<2> fb;
#pragma unroll
      for (int n = 0; n < 2; ++n)
        fb.template set<BF>(n, *reinterpret_cast<const i32x4*>(lb + lane_off[n] + j * 16 * kGroup));
      f32x4 sums[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) sums[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < FM; ++i)
          sums[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb.part[t], fa[i].part[t], sums[i], 0, 0, 0);
      if constexpr (FORM == kGrouped) {
        const f32x4 channels = *reinterpret_cast<const f32x4*>(sb + 16 * j + lane / 16 * 4);
#pragma unroll
        for (int i = 0; i < FM; ++i) add_scaled(acc[i][j], sums[i], token[i], channels);
      } else {
#pragma unroll
        for (int i = 0; i < FM; ++i) add_scaled(acc[i][j], sums[i], scale[FORM == kGatedForm ? j / 2 % 2 : 0][i]);
      }
    }
  };

  aim_tile();
  load();
  uint32_t slot = 0;
  bool whole_before = false;
  for (; tile < end; tile += stride) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t g = 0; g < a.groups; ++g) {
      // The block has landed, and every wave is done with the one before it,
      // whose place the next one takes. Loads and stores are counted in order: at
      // a tile's first block the stores of a whole tile's epilogue, 8 at least
      // and all behind the loads, may be under way.
      if (g == 0 && whole_before)
        wait_loads_and_sync<8>();
      else
        wait_loads_and_sync<0>();
      if (advance()) load();
      compute(slot);
      slot ^= 1;
    }

    uint32_t tm, tn;
    order.at(tile, &tm, &tn);
    const uint32_t i0 = tm * P::kSide + wm * P::kWaveM + lane % 16;
    // Two fragments of 16 channels: with their rows of lanes exchanged, a lane
    // holds eight consecutive channels.
    const uint32_t j0 = tn * kOut + wn * kWaveOut + lane / 16 % 2 * 16 + lane / 32 * 8;
    const bool whole = tm * P::kSide + P::kSide <= a.m && tn * kOut + kOut <= a.n && (a.quantize || a.out_vec);
    constexpr int kPieces = kWaveOut / 32;  // of a token, for each lane
    // Outputs p of token fragment i.
    auto piece = [&](int i, int p, float* v) {
      auto pair = [&](int j, float* to) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          to[e] = acc[i][j][e];
          to[4 + e] = acc[i][j + 1][e];
          swap_rows(to[e], to[4 + e]);
        }
      };
      if constexpr (FORM == kGatedForm) {
        float up[kPiece];
        pair(4 * p, v);
        pair(4 * p + 2, up);
#pragma unroll
        for (int e = 0; e < kPiece; ++e) v[e] = silu(v[e]) * up[e];
      } else {
        pair(2 * p, v);
      }
    };
    if (FORM != kGrouped && a.quantize) {
      const bool mx = a.scale_layout == kScaleE8M0Block32;
      float v[FM][kPieces][kPiece];
      uint32_t amax[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        amax[i] = 0;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          piece(i, p, v[i][p]);
          amax[i] = max(amax[i], max_bits(v[i][p]));
        }
        if (!mx) amax[i] = rows_max(amax[i]);
      }
      if (FORM == kGatedForm && !mx) {
        // 64 outputs a wave: the other half of a group is in the wave beside it.
        uint32_t* maxima = reinterpret_cast<uint32_t*>(lds + P::kMaxima);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          if (lane < 16) maxima[wn * P::kSide + wm * P::kWaveM + 16 * i + lane] = amax[i];
        lds_barrier();
#pragma unroll
        for (int i = 0; i < FM; ++i)
          amax[i] = max(amax[i], maxima[(1 - wn) * P::kSide + wm * P::kWaveM + 16 * i + lane % 16]);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const uint32_t token = i0 + 16 * i;
        uint32_t scale = 0;
        float mul = 0.0f;
        if (!mx) mul = code_multiplier(a, amax[i], &scale);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const uint32_t j = j0 + 32 * p;
          if (mx) mul = code_multiplier(a, rows_max(max_bits(v[i][p])), &scale);
          const Codes<kPiece> codes = encode_as(a, v[i][p], mul);
          if (token >= a.m || j >= a.n) continue;
          store_codes<true, kPiece>(static_cast<uint8_t*>(a.out) + static_cast<uint64_t>(token) * a.out_stride, j, a.n,
                                    codes);
          if (mx && j % 32 == 0)
            static_cast<uint8_t*>(a.scales)[static_cast<uint64_t>(token) * (a.n / 32) + j / 32] =
                static_cast<uint8_t>(scale);
          if (!mx && j % 128 == 0)
            static_cast<uint32_t*>(a.scales)[static_cast<uint64_t>(token) * (a.n / 128) + j / 128] = scale;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          float v[kPiece];
          piece(i, p, v);
          const uint32_t token = i0 + 16 * i, j = j0 + 32 * p;
          if (token >= a.m || j >= a.n) continue;
          if (a.out_format == kOutF32)
            finish_values<kOutF32>(a, token, j, v);
          else if (a.out_format == kOutBF16)
            finish_values<kOutBF16>(a, token, j, v);
          else
            finish_values<kOutF16>(a, token, j, v);
        }
    }
    whole_before = whole;
  }
  // Nothing is in flight to this work-group's LDS when it ends.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#endif
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
Choice pipe(const MatmulFp8Launch&) {
  return {{kMatmulPipe, Pipe::kSide, Pipe::kSide}, pipe_kernel<AF, BF, FORM>, kCus, Pipe::kThreads};
}

template <XFormat AF, XFormat BF, int FORM>
Choice choose_form(const MatmulFp8Launch& l) {
  if (!l.vec) return general_tiles<AF, BF, false, FORM>(l);
  // All but the general kernel hold offsets within a tile in 30 bits.
  const uint64_t up_rows = FORM == kGatedForm ? l.n : 0, up_blocks = FORM == kGatedForm ? l.up_block : 0;
  const bool near = (256 + up_rows) * l.b_stride + l.k < kFar && 256 * l.a_stride + l.k < kFar &&
                    (257 + up_blocks) * l.groups * 4 < kFar;
  if (!near) return general_tiles<AF, BF, true, FORM>(l);
  if (l.m > 256) return pipe<AF, BF, FORM>(l);
  return general_tiles<AF, BF, true, FORM>(l);
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
