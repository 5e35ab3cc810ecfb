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

// The scales of channels [j0, j0 + 8) of a token's piece.
struct PieceScales {
  float b[kPiece], up[kPiece];
};

__device__ __forceinline__ PieceScales piece_scales(const MatmulLaunch& a, uint32_t j0) {
  PieceScales s;
#pragma unroll
  for (int j = 0; j < kPiece; ++j) {
    s.b[j] = j0 + j < a.n ? a.b_scales[j0 + j] : 0.0f;
    s.up[j] = a.gated && j0 + j < a.n ? a.b_scales[a.n + j0 + j] : 0.0f;
  }
  return s;
}

// Eight outputs [j0, j0 + 8) of token i from their integer sums. `active`
// says whether i and j0 are inside the output; in the quantized form all
// lanes of a group (16 or 4 consecutive ones) call this together.
__device__ __forceinline__ void finish_piece(const MatmulLaunch& a, uint32_t i, uint32_t j0, bool active, float sa,
                                             const PieceScales& s, const int32_t* acc, const int32_t* up) {
  float v[kPiece];
#pragma unroll
  for (int j = 0; j < kPiece; ++j) v[j] = static_cast<float>(acc[j]) * sa * s.b[j];
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
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const float u = static_cast<float>(up[j]) * sa * s.up[j];
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
    finish_piece(a, i0 + i, j0 + j, i0 + i < a.m && j0 + j < a.n, a.a_scales[min(i0 + i, a.m - 1)],
                 piece_scales(a, j0 + j), p, p + kTileN / 2);
  }
}

template <bool VEC>
hipError_t launch_tiles(const MatmulLaunch& l, hipStream_t stream) {
  const uint32_t tile_n = l.gated ? kTileN / 2 : kTileN;
  const uint64_t tiles = static_cast<uint64_t>((l.m + kTileM - 1) / kTileM) * ((l.n + tile_n - 1) / tile_n);
  if (tiles >= uint64_t{1} << 24) return hipErrorInvalidValue;  // 2^32 work-items
  return launch_kernel(tile_kernel<VEC>, dim3(static_cast<uint32_t>(tiles)), dim3(256), stream, l);
}

// ---- pipelined tile kernel ---------------------------------------------

// TM tokens by TN rows of b, kStep bytes of k a stage, S stages in LDS.
// Waves of WTM tokens by WTN rows of b in 32x32x32 products.
//
// Operands go from memory straight into LDS, S - 1 stages ahead. A stage's
// row is 64 bytes, four chunks of 16; chunk c of row r lies in slot
// c ^ (r / 4 % 4), so that the sixteen lanes that LDS serves at once (rows
// r .. r + 15, one chunk) touch each of its 64 banks once. The load fills LDS
// in lane order, so each lane asks for the chunk that belongs in its slot.
//
// One barrier a stage, between the products of its first and second half:
// by then every wave holds the stage's second half in registers (its LDS is
// free for the stage S ahead), and the next stage has landed, so its first
// half is read while the second half is multiplied.
constexpr int kStep = 64;
constexpr int kChunks = kStep / 16;

typedef __attribute__((address_space(3))) void* lds_ptr;

template <int N>
__device__ __forceinline__ void wait_loads_and_sync() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Orders what was issued since the last barrier: R reads from LDS
// each behind one of the first products, then L loads to LDS each behind one
// of the next, so that the matrix unit never waits for a row of other
// instructions to issue.
template <int R, int L>
__device__ __forceinline__ void spread() {
  constexpr int kMfma = 0x8, kVmemRead = 0x20, kDsRead = 0x100;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kVmemRead, 1, 0);
  }
}

template <int TM, int TN, int WTM, int WTN, int S>
struct Pipe {
  static constexpr int kWavesM = TM / WTM, kWavesN = TN / WTN, kWaves = kWavesM * kWavesN, kThreads = 64 * kWaves;
  static constexpr int FM = WTM / 32, FN = WTN / 32;
  static constexpr int kLoadsA = TM / 16 / kWaves, kLoadsB = TN / 16 / kWaves, kLoads = kLoadsA + kLoadsB;
  static constexpr int kStageBytes = (TM + TN) * kStep;
  static constexpr int kSumPitch = WTN + 4;  // words of a staged token
  static constexpr int kLds = S * kStageBytes > kWaves * 32 * kSumPitch * 4 ? S * kStageBytes : kWaves * 32 * kSumPitch * 4;
  static_assert(TM % (16 * kWaves) == 0 && TN % (16 * kWaves) == 0, "whole loads a wave");
};

template <int TM, int TN, int WTM, int WTN, int S>
__global__ __launch_bounds__((Pipe<TM, TN, WTM, WTN, S>::kThreads), 1) void pipe_kernel(const MatmulLaunch a) {
#ifdef __HIP_DEVICE_COMPILE__  // the buffer builtins' types exist in the device pass alone
  using P = Pipe<TM, TN, WTM, WTN, S>;
  constexpr int FM = P::FM, FN = P::FN;
  __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
  __shared__ float token_scale[TM];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave % P::kWavesM, wn = wave / P::kWavesM;

  // Work-groups go round the eight XCDs, so XCD x takes every eighth one:
  // give it a run of consecutive tiles, and order tiles so that a run is a
  // patch of kGroup tokens-tiles by whole columns, which shares its operands
  // in the XCD's L2.
  constexpr uint32_t kGroup = 8;
  const uint32_t tile_n = a.gated ? TN / 2 : TN;
  const uint32_t tiles_m = (a.m + TM - 1) / TM, tiles_n = (a.n + tile_n - 1) / tile_n, tiles = tiles_m * tiles_n;
  const uint32_t xcd = blockIdx.x % 8, turn = blockIdx.x / 8;
  const uint32_t tile = xcd * (tiles / 8) + min(xcd, tiles % 8) + turn;
  const uint32_t group = tile / (kGroup * tiles_n), in_group = tile % (kGroup * tiles_n);
  const uint32_t group_m = min(kGroup, tiles_m - group * kGroup);
  const uint32_t i0 = (group * kGroup + in_group % group_m) * TM;
  const uint32_t j0 = in_group / group_m * tile_n;

  // Addresses: a uniform base, a lane's offset of 32 bits, and k in a scalar.
  __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.a + static_cast<uint64_t>(i0) * a.a_stride), 0, 0x7FFFFFFF, 0x00020000);
  __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.b + static_cast<uint64_t>(j0) * a.b_stride), 0, 0x7FFFFFFF, 0x00020000);
  uint32_t off_a[P::kLoadsA], off_b[P::kLoadsB];
  const uint32_t row16 = lane / kChunks;
  const uint32_t chunk = (lane % kChunks ^ row16 / 4 % kChunks) * 16;
#pragma unroll
  for (int t = 0; t < P::kLoadsA; ++t) {
    // Rows past the end load the last row; what they give is not stored.
    const uint32_t r = (wave * P::kLoadsA + t) * 16 + row16;
    off_a[t] = (min(i0 + r, a.m - 1) - i0) * static_cast<uint32_t>(a.a_stride);
  }
  const uint32_t up_rows = a.n;  // gated: where the up channels start
#pragma unroll
  for (int t = 0; t < P::kLoadsB; ++t) {
    const uint32_t r = (wave * P::kLoadsB + t) * 16 + row16;
    uint32_t j = r;
    if (a.gated) j = r / WTN * (WTN / 2) + r % (WTN / 2);  // a wave's rows: WTN / 2 gates, then their ups
    j = min(j0 + j, a.n - 1) - j0;
    if (a.gated && r % WTN >= WTN / 2) j += up_rows;
    off_b[t] = j * static_cast<uint32_t>(a.b_stride);
  }

  auto load_stage = [&](uint32_t slot, uint32_t k, uint32_t in_row) {
    const uint32_t k0 = __builtin_amdgcn_readfirstlane(k);
    char* base = lds + slot * P::kStageBytes;
#pragma unroll
    for (int t = 0; t < P::kLoadsA; ++t)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(base + (wave * P::kLoadsA + t) * 1024), 16,
                                               off_a[t] + in_row, k0, 0, 0);
#pragma unroll
    for (int t = 0; t < P::kLoadsB; ++t)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(base + TM * kStep + (wave * P::kLoadsB + t) * 1024), 16,
                                               off_b[t] + in_row, k0, 0, 0);
  };

  // A ragged end of k is the first stage: its chunks past the end load the
  // row's first chunk instead, and a's are then cleared in LDS, which is
  // enough for the products to be zero.
  const uint32_t tail = a.k % kStep;
  const uint32_t first_full = tail != 0 ? 1 : 0;
  const uint32_t stages = a.k / kStep + first_full;
  auto load = [&](uint32_t st) { load_stage(st % S, (st - first_full) * kStep, chunk); };

  i32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  for (uint32_t t = threadIdx.x; t < TM; t += P::kThreads) token_scale[t] = a.a_scales[min(i0 + t, a.m - 1)];
  if (tail != 0) load_stage(0, a.k - tail, chunk < tail ? chunk : 0);
#pragma unroll
  for (uint32_t st = 0; st < S; ++st)
    if (st >= first_full && st < stages) load(st);

  if (tail != 0) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (chunk >= tail) {
#pragma unroll
      for (int t = 0; t < P::kLoadsA; ++t)
        *reinterpret_cast<u32x4*>(lds + (wave * P::kLoadsA + t) * 1024 + lane * 16) = u32x4{0u, 0u, 0u, 0u};
    }
    wait_loads_and_sync<0>();
  } else if (stages >= S) {
    wait_loads_and_sync<P::kLoads * (S - 1)>();
  } else {
    wait_loads_and_sync<0>();
  }

  // Lane l reads row l % 32 of a fragment, chunk l / 32 of the half's two.
  const uint32_t swz = lane / 4 % kChunks;
  const uint32_t lane_off[2] = {lane % 32 * kStep + ((lane / 32) ^ swz) * 16, lane % 32 * kStep + ((2 + lane / 32) ^ swz) * 16};
  const char* base_a = lds + wm * WTM * kStep;
  const char* base_b = lds + TM * kStep + wn * WTN * kStep;
  i32x4 fa[2][FM], fb[2][FN];
  auto read_half = [&](uint32_t slot, int half) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
      fa[half][i] = *reinterpret_cast<const i32x4*>(base_a + slot * P::kStageBytes + i * 32 * kStep + lane_off[half]);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      fb[half][j] = *reinterpret_cast<const i32x4*>(base_b + slot * P::kStageBytes + j * 32 * kStep + lane_off[half]);
  };
  auto multiply = [&](int half) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[half][j], fa[half][i], acc[i][j], 0, 0, 0);
  };

  read_half(0, 0);
  uint32_t st = 0;
  for (; st + S < stages; ++st) {
    read_half(st % S, 1);
    multiply(0);
    spread<FM + FN, 0>();
    wait_loads_and_sync<P::kLoads * (S - 2)>();
    read_half((st + 1) % S, 0);
    load(st + S);
    multiply(1);
    spread<FM + FN, P::kLoads>();
  }
  for (; st + 1 < stages; ++st) {
    read_half(st % S, 1);
    multiply(0);
    wait_loads_and_sync<0>();
    read_half((st + 1) % S, 0);
    multiply(1);
  }
  read_half(st % S, 1);
  multiply(0);
  multiply(1);

  // Epilogue: a wave's 32 tokens at a time through its own part of LDS.
  __syncthreads();
  int32_t* sums = reinterpret_cast<int32_t*>(lds) + wave * 32 * P::kSumPitch;
  const uint32_t out_n = a.gated ? WTN / 2 : WTN;  // output channels of a wave
  const uint32_t pieces = out_n / kPiece;
  const uint32_t jj = lane % pieces * kPiece, j = j0 + wn * out_n + jj;
  const PieceScales scales = piece_scales(a, j);
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    // Lane l holds token l % 32, channels 8 q + 4 (l / 32) .. + 3.
#pragma unroll
    for (int g = 0; g < FN; ++g)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<i32x4*>(sums + lane % 32 * P::kSumPitch + 32 * g + 8 * q + lane / 32 * 4) =
            i32x4{acc[f][g][4 * q], acc[f][g][4 * q + 1], acc[f][g][4 * q + 2], acc[f][g][4 * q + 3]};
    for (uint32_t t = lane / pieces; t < 32; t += 64 / pieces) {
      const uint32_t i = i0 + wm * WTM + 32 * f + t;
      const int32_t* p = sums + t * P::kSumPitch + jj;
      int32_t v[kPiece], u[kPiece];
#pragma unroll
      for (int e = 0; e < kPiece; ++e) v[e] = p[e];
      if (a.gated) {
#pragma unroll
        for (int e = 0; e < kPiece; ++e) u[e] = p[WTN / 2 + e];
      }
      finish_piece(a, i, j, i < a.m && j < a.n, token_scale[wm * WTM + 32 * f + t], scales, v, u);
    }
  }
#endif
}

template <int TM, int TN, int WTM, int WTN, int S>
hipError_t launch_pipe(const MatmulLaunch& l, hipStream_t stream) {
  const uint32_t tile_n = l.gated ? TN / 2 : TN;
  const uint32_t tiles = ((l.m + TM - 1) / TM) * ((l.n + tile_n - 1) / tile_n);
  return launch_kernel(pipe_kernel<TM, TN, WTM, WTN, S>, dim3(tiles), dim3(Pipe<TM, TN, WTM, WTN, S>::kThreads), stream, l);
}

}  // namespace

uint64_t matmul_workspace_bytes(uint32_t, uint32_t, uint32_t, bool) { return 0; }

hipError_t launch_matmul(const MatmulLaunch& l, hipStream_t stream) {
  if (!l.vec) return launch_tiles<false>(l, stream);
  // The pipelined kernel's offsets within a tile are 31 bits.
  const bool near = l.a_stride < (1u << 22) && (l.b_stride * (static_cast<uint64_t>(l.gated ? l.n : 0) + 512)) < (1u << 31);
  if (!near || l.m <= 64) return launch_tiles<true>(l, stream);
  return launch_pipe<256, 256, 128, 128, 4>(l, stream);
}

}  // namespace qrs
