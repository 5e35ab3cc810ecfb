// gfx950 kernels of the product of 8-bit floating-point codes with scales for
// groups of 128 of k,
//
//   out[i][j] = sum_g (sum_{k in g} a[i][k] * b[j][k]) * fp32(a_scales[i][g] * b_scales[j or j / 128][g])
//
// of its gated form silu(gate) * up (two products over the same tokens), and of
// both as codes and scales.
//
// The matrix instructions for 8-bit floats cut the products of eight consecutive codes
// toward zero to multiples of 2^-13 of the largest one, taken by the codes' powers of two
// (measured: beside 256 * 256 and beside 448 * 448, 7 is gone and 12 is 8, where they stand
// in the same eight), and add them: 1.5e-5 of the result's norm for normal values, whose
// other products mostly lie whole above that, 100 times what binary32 sums leave, a
// hundredth of what rounding to 16 bits does. So outputs of 16 bits may use them (unless
// the caller asks for binary32 sums, as where large products cancel), and for the others
// codes are widened to bfloat16, which holds every one of them (two codes an instruction),
// and the bfloat16 instructions, whose sums keep binary32 (1e-8 of the norm), multiply them
// at half the rate. Kernels that wait for memory lose nothing by it and always widen.
//
// A group's sums of a 16 x 16 fragment are one instruction of 128 k, or four of 32;
// they are then multiplied by the scales' product and added in binary32 by one fused
// operation, and rounded once at the end. That is a vector operation for every four
// (fragments' elements by lanes) products of the matrix unit's rate, and the two run
// side by side only where the code keeps both fed.
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

typedef const __attribute__((address_space(1))) void* global_ptr;

// A wave's own loads to LDS but the last N have landed; its reads of LDS have.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_reads() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

template <XFormat AF, XFormat BF>
__device__ __forceinline__ f32x4 sums8(const i32x8& b, const i32x8& a) {
  // Operand formats: 0 E4M3, 1 E5M2. Both scale codes zero: the plain instruction.
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, BF == kXE5M2 ? 1 : 0,
                                                          AF == kXE5M2 ? 1 : 0, 0, 0, 0, 0);
}

// Two of four codes, the high or the low ones, as bfloat16.
template <XFormat F, bool HIGH>
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
  if constexpr (F == kXE4M3FN)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, HIGH));
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, 1.0f, HIGH));
}

// Eight codes as bfloat16.
template <XFormat F>
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
  const u32x4 w = {widen2<F, false>(lo), widen2<F, true>(lo), widen2<F, false>(hi), widen2<F, true>(hi)};
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

// The products of a 16 x 16 fragment over its 64 N codes of each row.
template <int N>
__device__ __forceinline__ void add_products(f32x4& sums, const Wide<N>& b, const Wide<N>& a) {
#pragma unroll
  for (int t = 0; t < 2 * N; ++t) sums = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.part[t], a.part[t], sums, 0, 0, 0);
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
  const uint32_t b_block = j0 / kTileN + (wave >= 2 && FORM == kGatedForm ? a.up_block : 0);
  const float* sb = a.b_scales + static_cast<uint64_t>(b_block) * a.groups;

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
      *reinterpret_cast<u32x4*>((t < kA ? la + (r + 32 * t) * T::kPitch : lb + (r + 32 * (t - kA)) * T::kPitch) + chunk) =
          w[t];
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
        f32x4 sums = {0.0f, 0.0f, 0.0f, 0.0f};
        add_products(sums, fb[j], fa);
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
      *reinterpret_cast<f32x4*>(lc + (16 * i + lane % 16) * T::kCPitch + (FN * wave + j) * 16 + lane / 16 * 4) =
          acc[i][j];
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
//
// 4096 x 8192, k = 7168 to bf16 219 to 238 us (2.0 to 2.2 PFLOP/s, of 2.55 that a
// product without scales reaches here), 8192 cubed 501 to 540: the scaled additions
// beside the matrix instructions, and the power limit (without the checks of k's end
// for every load, a tenth of the other instructions, the same time). Widened, 4096 x
// 8192, k = 4096 to binary32 233 to 247 us (1.1 to 1.2 PFLOP/s, of 1.3 for bfloat16).
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

template <XFormat AF, XFormat BF, int FORM, bool WIDE>
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
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ra, (lds_ptr)(base + (wave * P::kLoads + t) * 1024), 16, off_a[t] + far, k, 0, 0);
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
  // A block's scales: of this lane's tokens times those of b's rows (grouped: kept apart).
  struct Scales {
    float token[FM], product[FORM == kGatedForm ? 2 : 1][FM];
  };
  auto read_scales = [&](const char* base, Scales& s) {
    const float* sa = reinterpret_cast<const float*>(base + P::kOperands) + wm * P::kWaveM + lane % 16;
    const float* sb = reinterpret_cast<const float*>(base + P::kOperands) + P::kSide + wn * P::kWaveN;
#pragma unroll
    for (int i = 0; i < FM; ++i) s.token[i] = sa[16 * i];
    if constexpr (FORM != kGrouped) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        s.product[0][i] = s.token[i] * sb[0];
        if constexpr (FORM == kGatedForm) s.product[1][i] = s.token[i] * sb[32];
      }
    }
  };
  // Adds a fragment's sums; x = FM j + i.
  auto add = [&](const Scales& s, const f32x4& channels, const f32x4& sums, int x) {
    const int i = x % FM, j = x / FM;
    if constexpr (FORM == kGrouped)
      add_scaled(acc[i][j], sums, s.token[i], channels);
    else
      add_scaled(acc[i][j], sums, s.product[FORM == kGatedForm ? j / 2 % 2 : 0][i]);
  };
  auto read_channels = [&](const char* base, int j) {
    if constexpr (FORM != kGrouped) return f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const float* sb = reinterpret_cast<const float*>(base + P::kOperands) + P::kSide + wn * P::kWaveN;
    return *reinterpret_cast<const f32x4*>(sb + 16 * j + lane / 16 * 4);
  };

  auto compute = [&](uint32_t slot) {
    const char* base = lds + slot * P::kBlock;
    const char* la = base + wm * P::kWaveM * kGroup;
    const char* lb = base + P::kSide * kGroup + wn * P::kWaveN * kGroup;
    Scales scales;
    read_scales(base, scales);
    auto read = [&](const char* rows, int f, int n) {
      return *reinterpret_cast<const i32x4*>(rows + lane_off[n] + f * 16 * kGroup);
    };
    if constexpr (WIDE) {
      Wide<2> fa[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n) fa[i].template set<AF>(n, read(la, i, n));
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        Wide<2> fb;
#pragma unroll
        for (int n = 0; n < 2; ++n) fb.template set<BF>(n, read(lb, j, n));
        f32x4 sums[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) sums[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < FM; ++i)
            sums[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb.part[t], fa[i].part[t], sums[i], 0, 0, 0);
        const f32x4 channels = read_channels(base, j);
#pragma unroll
        for (int i = 0; i < FM; ++i) add(scales, channels, sums[i], FM * j + i);
      }
    } else {
      constexpr int kBehind = 4, kRing = kBehind + 1;
      f32x4 sums[kRing], channels[3];  // of the next, this and the last fragment of b
      auto fragment = [&](const char* rows, int f) {
        return __builtin_shufflevector(read(rows, f, 0), read(rows, f, 1), 0, 1, 2, 3, 4, 5, 6, 7);
      };
      i32x8 fa[FM], fb[2];
      fb[0] = fragment(lb, 0);
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = fragment(la, i);
      channels[0] = read_channels(base, 0);
#pragma unroll
      for (int x = 0; x < FM * FN + kBehind; ++x) {
        const int i = x % FM, j = x / FM;
        if (x < FM * FN) {
          sums[x % kRing] = sums8<AF, BF>(fb[j % 2], fa[i]);
          if (i == 0 && j + 1 < FN) {
            fb[(j + 1) % 2] = fragment(lb, j + 1);
            channels[(j + 1) % 3] = read_channels(base, j + 1);
          }
        }
        static_assert(kBehind <= FM, "the last fragment's scales are kept");
        if (x >= kBehind) add(scales, channels[(x - kBehind) / FM % 3], sums[(x - kBehind) % kRing], x - kBehind);
        __builtin_amdgcn_sched_barrier(0);
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

// ---- few tokens --------------------------------------------------------

// Up to 8 * M8 tokens: the weights are read once and bound the time. A
// work-group takes 32 or 16 (RB) rows of b times GW (gated: in runs of RB / 2 gates
// and their ups); its GW parts of KW waves take RB rows each and share k: wave w
// of a part takes every KW'th group of k, a line of 128 bytes of each row.
//
// Lines go from memory straight into a ring of the wave's own in LDS, S - 1 of them
// ahead, so no wave waits for another before its last line, and no register for
// a line under way. (With lines in registers, 16 waves of them, those that the
// widened codes leave too few: 8192 x 8192 19.1 us.) A load covers 8 rows; chunk c
// of row r lies in slot c ^ (r / 2 % 8), as in the pipelined tiles. One more load
// brings the scales of the rows of b and of the tokens, one a lane.
//
// The waves' sums meet in LDS and are added in the order of the waves.
//
// One token by 8192 x 8192 12.5 to 13.3 us, 5.4 to 5.0 TB/s (three sets of weights in turn,
// and more than the Infinity Cache holds).
template <int M8, int GW, int KW, int RB, int FORM>
struct Few {
  static constexpr int kWaves = GW * KW, MT = (M8 + 1) / 2, FB = RB / 16;
  static constexpr int kLoadsB = RB / 8, kLoads = kLoadsB + M8 + 1;  // of a line
  static constexpr int kScales = (RB + 8 * M8) * 128, kLine = kScales + 64 * 4;
  // Two work-groups a CU where that leaves each a line ahead.
  static constexpr int kPair = 81920 / (kWaves * kLine), kAlone = 163840 / (kWaves * kLine);
  static constexpr int kFit = kPair >= 2 ? kPair : kAlone;
  static constexpr int S = kFit < 3 ? kFit : 3;
  static constexpr int kRing = kWaves * S * kLine + (M8 == 1 ? 1024 : 0);  // a fragment of 8 tokens is read as 16 rows
  static constexpr int kPitch = RB + 4;                    // words of a token's sums
  static constexpr int kSums = kWaves * 16 * MT * kPitch * 4;
  static constexpr int kLds = kRing > kSums ? kRing : kSums;
  static constexpr uint32_t kRows = RB * GW, kOut = FORM == kGatedForm ? kRows / 2 : kRows;
  static_assert(S >= 2 && RB + 8 * M8 <= 64 && kLoads * (S - 1) < 64, "a line under way, a scale a lane, the counter");
};

template <XFormat AF, XFormat BF, int M8, int GW, int KW, int RB, int FORM>
__global__ __launch_bounds__(64 * GW * KW) void few_tokens_kernel(const MatmulFp8Launch a) {
#ifdef __HIP_DEVICE_COMPILE__
  using P = Few<M8, GW, KW, RB, FORM>;
  constexpr int MT = P::MT, FB = P::FB, S = P::S;
  constexpr bool kGated = FORM == kGatedForm;
  __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t part = wave / KW, kw = wave % KW;
  const uint32_t j0 = blockIdx.x * P::kOut;

  // Row r of the work-group's part of b.
  auto channel = [&](uint32_t r) { return min(j0 + (kGated ? r / RB * (RB / 2) + r % (RB / 2) : r), a.n - 1); };
  auto up = [](uint32_t r) { return kGated && r % RB >= RB / 2; };
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.a), 0, kFar, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.b + static_cast<uint64_t>(j0) * a.b_stride), 0, kFar, 0x00020000);
  // Load t of a line covers rows 8 t .. 8 t + 7, of b and then tokens.
  const uint32_t chunk[2] = {(lane % 8 ^ lane / 16) * 16u, (lane % 8 ^ (4 + lane / 16)) * 16u};
  uint32_t off_b[P::kLoadsB], off_a[M8];
#pragma unroll
  for (int t = 0; t < P::kLoadsB; ++t) {
    const uint32_t r = part * RB + 8 * t + lane / 8;
    off_b[t] = (channel(r) - j0 + (up(r) ? a.n : 0)) * static_cast<uint32_t>(a.b_stride) + chunk[t % 2];
  }
#pragma unroll
  for (int t = 0; t < M8; ++t)  // tokens past the last: the last one, not stored
    off_a[t] = min(8u * t + lane / 8, a.m - 1) * static_cast<uint32_t>(a.a_stride) + chunk[t % 2];
  const float* scale;
  if (lane < RB) {
    const uint32_t r = part * RB + lane;
    const uint32_t row = FORM == kGrouped ? channel(r) : channel(r) / kGroup + (up(r) ? a.up_block : 0);
    scale = a.b_scales + static_cast<uint64_t>(row) * a.groups;
  } else {
    scale = a.a_scales + static_cast<uint64_t>(min(static_cast<uint32_t>(lane - RB), a.m - 1)) * a.groups;
  }
  char* mine = lds + wave * S * P::kLine;
  auto load = [&](uint32_t g, uint32_t slot) {
    const uint32_t at = min(g, a.groups - 1), k = g * kGroup;  // past the last group: zeros
    char* to = mine + slot * P::kLine;
#pragma unroll
    for (int t = 0; t < P::kLoadsB; ++t) {
      const uint32_t far = k + chunk[t % 2] < a.k ? 0 : kFar;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(to + t * 1024), 16, off_b[t] + far, k, 0, 2);  // streamed
    }
#pragma unroll
    for (int t = 0; t < M8; ++t) {
      const uint32_t far = k + chunk[t % 2] < a.k ? 0 : kFar;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(to + RB * 128 + t * 1024), 16, off_a[t] + far, k, 0, 0);
    }
    __builtin_amdgcn_global_load_lds((global_ptr)(scale + at), (lds_ptr)(to + P::kScales), 4, 0, 0);
  };

  f32x4 acc[MT][FB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < FB; ++h) acc[i][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (uint32_t s = 0; s < S; ++s) load(kw + s * KW, s);
  const uint32_t lane_off[2] = {lane % 16 * 128 + ((lane / 16) ^ (lane % 16 / 2)) * 16u,
                                lane % 16 * 128 + ((4 + lane / 16) ^ (lane % 16 / 2)) * 16u};
  uint32_t slot = 0;
  for (uint32_t g = kw; g < a.groups; g += KW) {
    wait_loads<P::kLoads*(S - 1)>();
    const char* line = mine + slot * P::kLine;
    const float* scales = reinterpret_cast<const float*>(line + P::kScales);
    i32x4 fb[FB][2], fa[MT][2];
    float token[MT];
    f32x4 channels[FB];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int h = 0; h < FB; ++h) fb[h][n] = *reinterpret_cast<const i32x4*>(line + h * 2048 + lane_off[n]);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[i][n] = *reinterpret_cast<const i32x4*>(line + (FB + i) * 2048 + lane_off[n]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) token[i] = scales[RB + 16 * i + lane % 16];
#pragma unroll
    for (int h = 0; h < FB; ++h) channels[h] = *reinterpret_cast<const f32x4*>(scales + 16 * h + lane / 16 * 4);
    wait_reads();
    load(g + S * KW, slot);
    slot = slot + 1 == S ? 0 : slot + 1;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      Wide<2> wa;
#pragma unroll
      for (int n = 0; n < 2; ++n) wa.template set<AF>(n, fa[i][n]);
#pragma unroll
      for (int h = 0; h < FB; ++h) {
        Wide<2> wb;
#pragma unroll
        for (int n = 0; n < 2; ++n) wb.template set<BF>(n, fb[h][n]);
        f32x4 sums = {0.0f, 0.0f, 0.0f, 0.0f};
        add_products(sums, wb, wa);
        if constexpr (FORM == kGrouped)
          add_scaled(acc[i][h], sums, token[i], channels[h]);
        else
          add_scaled(acc[i][h], sums, token[i] * channels[h][0]);
      }
    }
  }

  wait_loads_and_sync<0>();
  // Lane l holds channels 4 (l / 16) .. + 3 of token l % 16.
  float* sums = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < FB; ++h)
      *reinterpret_cast<f32x4*>(sums + ((wave * MT + i) * 16 + lane % 16) * P::kPitch + h * 16 + lane / 16 * 4) =
          acc[i][h];
  __syncthreads();
  constexpr uint32_t pieces = P::kOut / kPiece, part_pieces = pieces / GW;
  // Of M8 = 1 a fragment's first 8 tokens.
  for (uint32_t t = threadIdx.x; t < 8 * M8 * pieces; t += 64 * P::kWaves) {
    const uint32_t i = t / pieces, piece = t % pieces;
    const float* row = sums + (piece / part_pieces * KW * 16 * MT + i) * P::kPitch + piece % part_pieces * kPiece;
    float v[kPiece], ups[kPiece];
#pragma unroll
    for (int e = 0; e < kPiece; ++e) v[e] = ups[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const float* p = row + w * 16 * MT * P::kPitch;
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        v[e] += p[e];
        if constexpr (kGated) ups[e] += p[RB / 2 + e];
      }
    }
    const uint32_t j = j0 + piece * kPiece;
    finish_outputs<FORM>(a, i, j, i < a.m && j < a.n, v, ups);
  }
#endif
}

// ---- tens to hundreds of tokens ----------------------------------------

// Too few tiles of the pipelined kernel for 256 CUs: TM tokens by TN rows of
// b a work-group. Its eight waves are KG ways of sharing k, WM of the tokens and
// the rest of the rows of b; wave (g, w) takes group g of each stage's KG groups.
//
// A stage is KG groups of k of all rows, loaded straight into LDS, 8 rows a
// load, S - 1 stages ahead, with their scales, so that most of LDS holds operands in
// flight, in whole lines. What bounds these tiles is how fast operands come
// into a CU, and next the widening of their codes. Slots as in the pipelined tiles.
// Two waves a SIMD hide each other's reads; one barrier a stage. 333 by 5120, k =
// 7168 to bf16 30 us, to binary32 37; with stages of half the length and twice as
// many, a quarter more bytes under way, 33 and 42.
template <int TM, int TN, int KG, int WM, int S>
struct Mid {
  static constexpr int kThreads = 512, kWavesN = 8 / KG / WM, WTM = TM / WM, WTN = TN / kWavesN;
  static constexpr int FM = WTM / 16, FN = WTN / 16;
  static constexpr int kRows = TM + TN;
  static constexpr int kOperands = kRows * KG * 128, kStage = kOperands + 8 * 64 * 4;
  static constexpr int kLoads = kOperands / 1024 / 8 + 1;  // of a wave
  static constexpr int kPitch = TN + 4;                    // words of a token's sums
  static constexpr int kSums = KG * TM * kPitch * 4;
  static constexpr int kLds = S * kStage > kSums ? S * kStage : kSums;
  static_assert(kOperands % 8192 == 0 && WTN % 16 == 0 && WTM % 16 == 0, "whole loads and fragments");
  static_assert(kRows * KG <= 512 && kLds <= 163840, "one scale a lane");
};

template <XFormat AF, XFormat BF, int TM, int TN, int KG, int WM, int S, int FORM, bool WIDE>
__global__ __launch_bounds__(512, 2) void mid_kernel(const MatmulFp8Launch a) {
#ifdef __HIP_DEVICE_COMPILE__
  using P = Mid<TM, TN, KG, WM, S>;
  constexpr int FM = P::FM, FN = P::FN;
  constexpr bool kGated = FORM == kGatedForm;
  // One array: with several, the compiler tells their accesses apart and
  // waits for every load to LDS before it reads any.
  __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int kg = wave % KG, wm = wave / KG % WM, wn = wave / KG / WM;

  constexpr uint32_t kOut = kGated ? TN / 2 : TN;
  const TileOrder order = {(a.m + TM - 1) / TM, (a.n + kOut - 1) / kOut};
  const uint32_t tiles = order.tiles_m * order.tiles_n, xcd = blockIdx.x % 8;
  uint32_t tm, tn;
  order.at((tiles / 8) * xcd + min(xcd, tiles % 8) + blockIdx.x / 8, &tm, &tn);
  const uint32_t i0 = tm * TM, j0 = tn * kOut;
  // Row r of the tile's part of b: in the gated form every fragment of 16
  // gates is followed by their ups.
  auto channel = [&](uint32_t r) { return min(j0 + (kGated ? r / 32 * 16 + r % 16 : r), a.n - 1); };
  auto up = [](uint32_t r) { return kGated && r % 32 >= 16; };
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.a + static_cast<uint64_t>(i0) * a.a_stride), 0, kFar, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.b + static_cast<uint64_t>(j0) * a.b_stride), 0, kFar, 0x00020000);

  // Load t covers rows 8 (t % (kRows / 8)) .. + 7 of group t / (kRows / 8);
  // lane l the chunk of row l / 8 whose slot is l % 8.
  constexpr int kCodeLoads = P::kLoads - 1;
  uint32_t offset[kCodeLoads], in_k[kCodeLoads];
#pragma unroll
  for (int t = 0; t < kCodeLoads; ++t) {
    const uint32_t at = wave * kCodeLoads + t, r = at % (P::kRows / 8) * 8 + lane / 8;
    in_k[t] = at / (P::kRows / 8) * 128 + (lane % 8 ^ (r / 2 % 8)) * 16;
    const uint32_t q = r - TM;
    offset[t] = (r < TM ? (min(i0 + r, a.m - 1) - i0) * static_cast<uint32_t>(a.a_stride)
                        : (channel(q) - j0 + (up(q) ? a.n : 0)) * static_cast<uint32_t>(a.b_stride)) + in_k[t];
  }
  // Lane l of wave w loads the scale of row (64 w + l) % kRows in group (64 w + l) / kRows.
  const uint32_t scale_at = threadIdx.x, scale_row = scale_at % P::kRows;
  const uint32_t scale_group = min(scale_at / P::kRows, KG - 1u);
  const float* scale;
  if (scale_row < TM) {
    scale = a.a_scales + static_cast<uint64_t>(min(i0 + scale_row, a.m - 1)) * a.groups;
  } else {
    const uint32_t q = scale_row - TM;
    const uint32_t row = FORM == kGrouped ? channel(q) : channel(q) / kGroup + (up(q) ? a.up_block : 0);
    scale = a.b_scales + static_cast<uint64_t>(row) * a.groups;
  }
  // Load t of stage st, to `slot`; `full`: the stage ends inside k.
  auto load = [&](uint32_t st, uint32_t slot, int t, bool full) {
    char* to = lds + slot * P::kStage;
    if (t == kCodeLoads) {  // past the last group: its scales, which nothing is multiplied by
      __builtin_amdgcn_global_load_lds((global_ptr)(scale + min(st * KG + scale_group, a.groups - 1)),
                                       (lds_ptr)(to + P::kOperands + wave * 256), 4, 0, 0);
      return;
    }
    const uint32_t k = __builtin_amdgcn_readfirstlane(st * KG * 128);
    const uint32_t at = wave * kCodeLoads + t;
    const uint32_t far = full || k + in_k[t] < a.k ? 0 : kFar;  // past the end of k: zeros
    __builtin_amdgcn_raw_ptr_buffer_load_lds(at % (P::kRows / 8) * 8 < TM ? ra : rb, (lds_ptr)(to + at * 1024), 16,
                                             offset[t] + far, k, 0, 0);
  };

  const uint32_t stages = (a.groups + KG - 1) / KG, full_stages = a.k / (KG * 128);
#pragma unroll
  for (uint32_t st = 0; st < S; ++st)  // past the last stage: zeros
#pragma unroll
    for (int t = 0; t < P::kLoads; ++t) load(st, st, t, false);

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // Lane l reads row l % 16 of a fragment, chunks l / 16 and 4 + l / 16.
  const uint32_t lane_off[2] = {lane % 16 * 128 + ((lane / 16) ^ (lane % 16 / 2)) * 16u,
                                lane % 16 * 128 + ((4 + lane / 16) ^ (lane % 16 / 2)) * 16u};
  const char* frag_a = lds + (kg * P::kRows + wm * P::WTM) * 128;
  const char* frag_b = lds + (kg * P::kRows + TM + wn * P::WTN) * 128;
  const char* scales_a = lds + P::kOperands + (kg * P::kRows + wm * P::WTM + lane % 16) * 4;
  const char* scales_b = lds + P::kOperands + (kg * P::kRows + TM + wn * P::WTN + lane / 16 * 4) * 4;
  constexpr int kScalesB = FORM == kGrouped ? 4 : 1;  // of a lane, in each fragment
  struct Fragments {  // of a stage
    i32x4 a[FM][2], b[FN][2];
    float token[FM], channel[FN][kScalesB];
  } now, next;
  auto read_a = [&](Fragments& f, uint32_t slot, int i) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
      f.a[i][n] = *reinterpret_cast<const i32x4*>(frag_a + slot * P::kStage + i * 2048 + lane_off[n]);
    f.token[i] = *reinterpret_cast<const float*>(scales_a + slot * P::kStage + 64 * i);
  };
  auto read_b = [&](Fragments& f, uint32_t slot, int j) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
      f.b[j][n] = *reinterpret_cast<const i32x4*>(frag_b + slot * P::kStage + j * 2048 + lane_off[n]);
#pragma unroll
    for (int e = 0; e < kScalesB; ++e)
      f.channel[j][e] = *reinterpret_cast<const float*>(scales_b + slot * P::kStage + 64 * j + 4 * e);
  };
  // Fragment x = KF u + q joins the q-th kept and the u-th streamed fragment: of
  // the operand with fewer of them all are kept widened, of the other one at a time.
  constexpr bool kKeepA = FM < FN;
  constexpr int KF = kKeepA ? FM : FN, SF = kKeepA ? FN : FM;
  auto add = [&](const Fragments& f, const f32x4& sums, int x) {
    const int i = kKeepA ? x % KF : x / KF, j = kKeepA ? x / KF : x % KF;
    const float* c = f.channel[j];
    if constexpr (FORM == kGrouped)
      add_scaled(acc[i][j], sums, f.token[i], f32x4{c[0], c[1], c[2], c[3]});
    else
      add_scaled(acc[i][j], sums, f.token[i] * c[0]);
  };
  // Two codes' widening of a streamed or kept fragment: `word` of its 16.
  auto widen_word = [&](Wide<2>& to, const Fragments& f, bool kept, int index, int word) {
    const bool of_a = kept == kKeepA;
    const i32x4& chunk = of_a ? f.a[index][word / 8] : f.b[index][word / 8];
    const uint32_t codes = static_cast<uint32_t>(chunk[word / 2 % 4]);
    u32x4 w = __builtin_bit_cast(u32x4, to.part[word / 4]);
    if (of_a)
      w[word % 4] = word % 2 ? widen2<AF, true>(codes) : widen2<AF, false>(codes);
    else
      w[word % 4] = word % 2 ? widen2<BF, true>(codes) : widen2<BF, false>(codes);
    to.part[word / 4] = __builtin_bit_cast(bf16x8, w);
  };
  Wide<2> kept[KF], streamed[2];
  auto widen_kept = [&](const Fragments& f, int q) {
#pragma unroll
    for (int w = 0; w < 16; ++w) widen_word(kept[q], f, true, q, w);
  };
  auto widen_first = [&](const Fragments& f) {
#pragma unroll
    for (int w = 0; w < 16; ++w) widen_word(streamed[0], f, false, 0, w);
  };
  // Multiplies stage st (in registers, its LDS `slot`) while stage st + 1 is
  // read and stage st + S loaded into st's place in LDS. Every matrix
  // instruction has others behind it: the widening of the next streamed fragment,
  // the scaled addition of the sums before, reads and loads.
  auto stage = [&](uint32_t st, uint32_t slot, bool full) {
    wait_loads_and_sync<P::kLoads*(S - 2)>();
    const uint32_t after = slot + 1 == S ? 0 : slot + 1;
    const bool live = full || st * KG + kg < a.groups;  // scales past the last group may be anything
    constexpr int kSteps = WIDE ? 4 * FM * FN : FM * FN, kReads = FM + FN;
    constexpr int kBehind = WIDE ? 1 : 2, kRing = kBehind + 1;
    f32x4 sums[kRing];
#pragma unroll
    for (int y = 0; y < kSteps; ++y) {
      if constexpr (WIDE) {
        const int x = y / 4, t = y % 4, q = x % KF, u = x / KF;
        f32x4& to = sums[x % kRing];
        if (t == 0) to = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const bf16x8 k = kept[q].part[t], v = streamed[u % 2].part[t];
        to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kKeepA ? v : k, kKeepA ? k : v, to, 0, 0, 0);
        constexpr int kWords = 4 / KF;  // for each step
        if (u + 1 < SF) {
#pragma unroll
          for (int w = 0; w < kWords; ++w)
            widen_word(streamed[(u + 1) % 2], now, false, u + 1, (y % (4 * KF)) * kWords + w);
        }
        if (x > 0 && live) {  // a quarter of the fragment before
          const f32x4& from = sums[(x - 1) % kRing];
          const int i = kKeepA ? (x - 1) % KF : (x - 1) / KF, j = kKeepA ? (x - 1) / KF : (x - 1) % KF;
          const float scale = now.token[i] * now.channel[j][t % kScalesB];
          acc[i][j][t] = __builtin_fmaf(from[t], scale, acc[i][j][t]);
        }
      } else {
        auto whole = [](const i32x4 (&f)[2]) { return __builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7); };
        const int i = kKeepA ? y % KF : y / KF, j = kKeepA ? y / KF : y % KF;
        sums[y % kRing] = sums8<AF, BF>(whole(now.b[j]), whole(now.a[i]));
        if (y >= kBehind && live) add(now, sums[(y - kBehind) % kRing], y - kBehind);
      }
#pragma unroll
      for (int r = y * kReads / kSteps; r < (y + 1) * kReads / kSteps; ++r) {
        if (r < FN)
          read_b(next, after, r);
        else
          read_a(next, after, r - FN);
      }
#pragma unroll
      for (int t = y * P::kLoads / kSteps; t < (y + 1) * P::kLoads / kSteps; ++t) load(st + S, slot, t, full);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int x = FM * FN - kBehind; x < FM * FN; ++x)
      if (live) add(now, sums[x % kRing], x);
    now = next;
    if constexpr (WIDE) {
      widen_first(now);
#pragma unroll
      for (int q = 0; q < KF; ++q) widen_kept(now, q);
    }
  };
  wait_loads_and_sync<P::kLoads*(S - 1)>();
#pragma unroll
  for (int j = 0; j < FN; ++j) read_b(now, 0, j);
#pragma unroll
  for (int i = 0; i < FM; ++i) read_a(now, 0, i);
  if constexpr (WIDE) {
    widen_first(now);
#pragma unroll
    for (int q = 0; q < KF; ++q) widen_kept(now, q);
  }
  uint32_t st = 0;
  // Rounds with fixed slots and nothing to check, while all that they load is
  // inside k; then a stage at a time.
  for (; st + 2 * S <= full_stages; st += S) {
#pragma unroll
    for (uint32_t r = 0; r < S; ++r) stage(st + r, r, true);
  }
  for (; st < stages; ++st) stage(st, st % S, false);

  // The KG partial sums meet in LDS, and are added in order.
  float* sums = reinterpret_cast<float*>(lds);
  wait_loads_and_sync<0>();
  // Lane l holds channels 4 (l / 16) .. + 3 of token l % 16 of a fragment.
  float* at = sums + (kg * TM + wm * P::WTM + lane % 16) * P::kPitch + wn * P::WTN + lane / 16 * 4;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) *reinterpret_cast<f32x4*>(at + i * 16 * P::kPitch + j * 16) = acc[i][j];
  __syncthreads();
  constexpr uint32_t pieces = kOut / kPiece;
  static_assert(TM * pieces % 64 == 0, "whole waves");
  for (uint32_t t = threadIdx.x; t < TM * pieces; t += P::kThreads) {
    const uint32_t i = t / pieces, jj = t % pieces * kPiece;
    const float* row = sums + i * P::kPitch + (kGated ? jj / 16 * 32 + jj % 16 : jj);
    float v[kPiece], ups[kPiece];
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      v[e] = row[e];
      if constexpr (kGated) ups[e] = row[16 + e];
#pragma unroll
      for (int g = 1; g < KG; ++g) {
        v[e] += row[g * TM * P::kPitch + e];
        if constexpr (kGated) ups[e] += row[g * TM * P::kPitch + 16 + e];
      }
    }
    finish_outputs<FORM>(a, i0 + i, j0 + jj, i0 + i < a.m && j0 + jj < a.n, v, ups);
  }
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

template <XFormat AF, XFormat BF, int M8, int GW, int KW, int RB, int FORM>
Choice few(const MatmulFp8Launch& l) {
  using P = Few<M8, GW, KW, RB, FORM>;
  return {{kMatmulFewTokens, 8 * M8, P::kRows}, few_tokens_kernel<AF, BF, M8, GW, KW, RB, FORM>,
          tiles_of(l, 8 * M8, P::kOut), 64 * P::kWaves};
}

// Groups of 128 outputs (256 rows of b, gated; 64 rows for E8M0 scales) are more than
// a work-group should read for few tokens: a CU takes 40 GB/s. Their values go
// through the workspace, and a second kernel makes the codes (16 tokens, gated,
// 2 x 3584 x 8192: 44 us in one kernel, 15 in two; with E8M0 scales 23).
bool by_workspace(const MatmulFp8Launch& l) {
  return l.quantize && fp8_workspace(l.m, l.n, l.gated, l.scale_layout) != 0;
}

// Sixteen rows of b a wave: more work-groups, two of them a CU, keep more lines under
// way than 32 rows do (one token, us with 16 and 32: 8192 x 8192 13.3 and 17.3,
// 28672 x 8192 38.4 and 53.6; 16 tokens, 8192 x 8192 15.8 and 19.7), but for more
// than 16 tokens, whose own lines would be two of three (32 tokens 22.9 and 19.9).
template <XFormat AF, XFormat BF, int M8, int FORM>
Choice few_sized(const MatmulFp8Launch& l) {
  constexpr int RB = M8 == 4 ? 32 : 16;
  if constexpr (FORM == kPlain) {
    // E8M0 scales need 32 outputs in a work-group.
    if (l.quantize && !by_workspace(l)) return few<AF, BF, M8, 32 / RB, RB / 4, RB, FORM>(l);
  }
  return few<AF, BF, M8, 1, M8 == 2 ? 4 : 8, RB, FORM>(l);
}

// Whether codes are widened: for outputs of binary32, and codes, whose scales are, and
// where the caller asks for it.
bool wide(const MatmulFp8Launch& l) { return l.quantize || l.out_format == kOutF32 || l.binary32; }

// The ways of adding that calls take a tile in.
enum Ways : int { kNarrow = 1, kWide = 2, kBoth = 3 };

template <XFormat AF, XFormat BF, int TM, int TN, int KG, int WM, int S, int FORM, int WAYS = kBoth>
Choice mid(const MatmulFp8Launch& l) {
  Choice c = {{kMatmulMid, TM, TN}, mid_kernel<AF, BF, TM, TN, KG, WM, S, FORM, WAYS == kWide>,
              tiles_of(l, TM, FORM == kGatedForm ? TN / 2 : TN), 512};
  if constexpr (WAYS == kBoth)
    if (wide(l)) c.kernel = mid_kernel<AF, BF, TM, TN, KG, WM, S, FORM, true>;
  return c;
}

// Rows of operands that the busiest CU loads with tiles of TM tokens by TN
// rows of b: what a call's time goes by.
template <int TM, int TN, int FORM>
uint64_t rows_a_cu(const MatmulFp8Launch& l) {
  return (tiles_of(l, TM, FORM == kGatedForm ? TN / 2 : TN) + kCus - 1) / kCus * (TM + TN);
}

template <XFormat AF, XFormat BF, int FORM>
Choice pipe(const MatmulFp8Launch& l) {
  return {{kMatmulPipe, Pipe::kSide, Pipe::kSide},
          wide(l) ? pipe_kernel<AF, BF, FORM, true> : pipe_kernel<AF, BF, FORM, false>, kCus, Pipe::kThreads};
}

template <XFormat AF, XFormat BF, int FORM>
Choice choose_form(const MatmulFp8Launch& l) {
  if (!l.vec) return general_tiles<AF, BF, false, FORM>(l);
  // All but the general kernel hold offsets within a tile in 30 bits.
  const uint64_t up_rows = FORM == kGatedForm ? l.n : 0, up_blocks = FORM == kGatedForm ? l.up_block : 0;
  const bool near = (256 + up_rows) * l.b_stride + l.k < kFar && 256 * l.a_stride + l.k < kFar &&
                    (257 + up_blocks) * l.groups * 4 < kFar;
  if (!near) return general_tiles<AF, BF, true, FORM>(l);
  if (l.m <= kMaxFewTokens) {
    const Choice c = l.m <= 8    ? few_sized<AF, BF, 1, FORM>(l)
                     : l.m <= 16 ? few_sized<AF, BF, 2, FORM>(l)
                                 : few_sized<AF, BF, 4, FORM>(l);
    return c.fits() ? c : general_tiles<AF, BF, true, FORM>(l);
  }
  // The tile whose busiest CU loads least. The pipelined kernel's rows count a
  // quarter more: its matrix units and the power limit bound it. us of bf16 outputs with
  // <64, 32>, <64, 64>, <64, 128>, <128, 128>, <128, 256> and <256, 256>: 48 by 8192, k = 4096
  // 12, 15, 21, 21, 33 and 51; 128 by 8192, k = 8192 43, 29, 40, 69, 89 and 108; 512 by 4096,
  // k = 8192 77, 51, 37, 60, 82 and 120; 1024 by 4096, k = 4096 69, 45, 34, 30, 37 and 58;
  // 1024 by 8192, k = 2048 93, 56, 41, 34, 25 and 33; 2048 by 8192, k = 2048 184, 109, 80, 64,
  // 48 and 40. (Binary32 outputs the same but for <128, 256>, whose widened codes overflow the registers.)
  uint64_t least = ~uint64_t{0};
  Choice best = general_tiles<AF, BF, true, FORM>(l);
  auto offer = [&](uint64_t rows, const Choice& c) {
    if (rows < least && c.fits()) {
      least = rows;
      best = c;
    }
  };
  offer(rows_a_cu<256, 256, FORM>(l) * 5 / 4, pipe<AF, BF, FORM>(l));
  const bool group = l.quantize && l.scale_layout == kScaleF32Group128;  // 128 outputs a tile
  if constexpr (FORM == kGatedForm) {
    if (group) {
      offer(rows_a_cu<64, 256, FORM>(l), mid<AF, BF, 64, 256, 1, 2, 3, FORM, kWide>(l));
      return best;
    }
  }
  if constexpr (FORM != kGrouped)  // whose scales overflow the registers, too
    if (!wide(l)) offer(rows_a_cu<128, 256, FORM>(l), mid<AF, BF, 128, 256, 1, 2, 3, FORM, kNarrow>(l));
  offer(rows_a_cu<128, 128, FORM>(l), mid<AF, BF, 128, 128, 1, 2, 4, FORM>(l));
  offer(rows_a_cu<64, 128, FORM>(l), mid<AF, BF, 64, 128, 2, 1, 3, FORM>(l));
  if (group) return best;
  offer(rows_a_cu<64, 64, FORM>(l), mid<AF, BF, 64, 64, 2, 2, 4, FORM>(l));
  if (!l.quantize || FORM == kPlain) offer(rows_a_cu<64, 32, FORM>(l), mid<AF, BF, 64, 32, 4, 2, 3, FORM>(l));
  return best;
}

template <XFormat AF, XFormat BF>
Choice choose(const MatmulFp8Launch& l) {
  if (l.grouped) return choose_form<AF, BF, kGrouped>(l);
  return l.gated ? choose_form<AF, BF, kGatedForm>(l) : choose_form<AF, BF, kPlain>(l);
}

// Codes of values in binary32 [m, n].
__global__ __launch_bounds__(256) void codes_kernel(const MatmulFp8Launch a) {
  const uint32_t pieces = a.n / kPiece;  // a multiple of a group's 16
  const uint32_t t = blockIdx.x * 256 + threadIdx.x, i = t / pieces, j = t % pieces * kPiece;
  float v[kPiece];
  load_piece<kOutF32, true, kPiece>(a.workspace + static_cast<uint64_t>(min(i, a.m - 1)) * a.n, j, a.n, v);
  finish_codes(a, i, j, i < a.m, false, v);
}

template <XFormat AF, XFormat BF>
hipError_t launch_formats(const MatmulFp8Launch& l, hipStream_t stream) {
  const Choice c = choose<AF, BF>(l);
  if (!c.fits()) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(c.blocks)), block(c.threads);
  if (!(c.id.family == kMatmulFewTokens && by_workspace(l))) return launch_kernel(c.kernel, grid, block, stream, l);
  MatmulFp8Launch values = l;
  values.quantize = false;
  values.out_format = kOutF32;
  values.out_vec = true;
  values.out = l.workspace;
  values.out_stride = l.n;
  const hipError_t e = launch_kernel(c.kernel, grid, block, stream, values);
  if (e != hipSuccess) return e;
  return launch_kernel(codes_kernel, dim3((l.m * (l.n / kPiece) + 255) / 256), dim3(256), stream, l);
}

}  // namespace

hipError_t launch_fp8_e4m3_e4m3(const MatmulFp8Launch& l, hipStream_t stream);
hipError_t launch_fp8_e4m3_e5m2(const MatmulFp8Launch& l, hipStream_t stream);
hipError_t launch_fp8_e5m2_e4m3(const MatmulFp8Launch& l, hipStream_t stream);
hipError_t launch_fp8_e5m2_e5m2(const MatmulFp8Launch& l, hipStream_t stream);

}  // namespace qrs
