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
#include "qrs_matmul_device.h"

// One rounding per operation: never fuse.
#pragma clang fp contract(off)

namespace qrs {
namespace {

using namespace dev;

// ---- epilogue ----------------------------------------------------------

// What a kernel instance writes.
enum Finish : int { kValues = 0, kGated = 1, kCodes = 2 };

// The scales of channels [j0, j0 + 8): of the product, or of its gate, and
// of its up channels.
struct PieceScales {
  float b[kPiece], up[kPiece];

  __device__ bool finite() const {
    bool all = true;
#pragma unroll
    for (int j = 0; j < kPiece; ++j) all = all && abs_bits(b[j]) < 0x7F800000u;
    return all;
  }
};

template <int F>
__device__ __forceinline__ PieceScales piece_scales(const MatmulLaunch& a, uint32_t j0) {
  PieceScales s;
#pragma unroll
  for (int j = 0; j < kPiece; ++j) {
    s.b[j] = j0 + j < a.n ? a.b_scales[j0 + j] : 0.0f;
    if constexpr (F == kGated) s.up[j] = j0 + j < a.n ? a.b_scales[a.n + j0 + j] : 0.0f;
  }
  return s;
}

// Whether an integer sum times a token's scale is finite for certain: the
// scale is below 2^95.
__device__ __forceinline__ bool keeps_finite(float token_scale) { return abs_bits(token_scale) < 0x6F000000u; }

// v: a piece's integer sums as binary32 times the token's scale sa (gated: of
// the gates; up: of the ups) -> the outputs as binary32.
template <int F>
__device__ __forceinline__ void scale_piece(const PieceScales& s, float* v, const float* up) {
#pragma unroll
  for (int j = 0; j < kPiece; ++j) v[j] *= s.b[j];
  if constexpr (F == kGated) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) v[j] = silu(v[j]) * (up[j] * s.up[j]);
  }
}

// Eight outputs [j0, j0 + 8) of token i; v and up as for scale_piece. `active`
// says whether i and j0 are inside the output; where codes are written, all
// lanes of a group (16 or 4 consecutive ones) call this together.
template <int F>
__device__ __forceinline__ void finish_piece(const MatmulLaunch& a, uint32_t i, uint32_t j0, bool active, float sa,
                                             const PieceScales& s, float* v, const float* up) {
  scale_piece<F>(s, v, up);
  if constexpr (F == kCodes) {
    finish_codes(a, i, j0, active, keeps_finite(sa) && s.finite(), v);
  } else {
    if (!active) return;
    if (a.out_format == kOutF32)
      finish_values<kOutF32>(a, i, j0, v);
    else if (a.out_format == kOutBF16)
      finish_values<kOutBF16>(a, i, j0, v);
    else
      finish_values<kOutF16>(a, i, j0, v);
  }
}

// ---- general tile kernel -----------------------------------------------

// 64 tokens by 128 rows of b (gated: 64 gate and 64 up channels), 64 bytes
// of k at a time through LDS. Four waves, each 64 tokens by 32 rows of b in
// 16x16x64 products.
constexpr int kTileM = 64, kTileN = 128, kTileK = 64;
constexpr int kPitch = kTileK + 16;   // bytes; rows 5 quarter-lines apart
constexpr int kCPitch = kTileN + 4;   // words of the staged sums

template <bool VEC, int F>
__global__ __launch_bounds__(256) void tile_kernel(const MatmulLaunch a) {
  __shared__ __attribute__((aligned(16))) char lds[kTileM * kCPitch * 4];
  static_assert((kTileM + kTileN) * kPitch <= kTileM * kCPitch * 4, "operands share the staging buffer");
  char* la = lds;
  char* lb = lds + kTileM * kPitch;
  constexpr uint32_t tile_n = F == kGated ? kTileN / 2 : kTileN;
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
    const uint32_t rb = F == kGated ? min(j0 + r, a.n - 1) + (h ? a.n : 0) : min(j0 + r + 64 * h, a.n - 1);
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
  constexpr uint32_t pieces = tile_n / kPiece;
  for (uint32_t t = threadIdx.x; t < kTileM * pieces; t += 256) {
    const uint32_t i = t / pieces, j = t % pieces * kPiece;
    const int32_t* p = lc + i * kCPitch + j;
    const float sa = a.a_scales[min(i0 + i, a.m - 1)];
    float v[kPiece], up[kPiece];
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      v[e] = static_cast<float>(p[e]) * sa;
      if constexpr (F == kGated) up[e] = static_cast<float>(p[kTileN / 2 + e]) * sa;
    }
    finish_piece<F>(a, i0 + i, j0 + j, i0 + i < a.m && j0 + j < a.n, sa, piece_scales<F>(a, j0 + j), v, up);
  }
}

// A kernel and its grid for a call.
struct Choice {
  MatmulKernel id;
  void (*kernel)(MatmulLaunch);
  uint64_t blocks;
  uint32_t threads;

  // A HIP grid holds fewer than 2^32 work-items.
  bool fits() const { return blocks * threads < uint64_t{1} << 32; }
};

uint64_t tiles_of(const MatmulLaunch& l, uint32_t tile_m, uint32_t tile_n) {
  return static_cast<uint64_t>((l.m + tile_m - 1) / tile_m) * ((l.n + tile_n - 1) / tile_n);
}

template <bool VEC, int F>
Choice general_tiles(const MatmulLaunch& l) {
  constexpr uint32_t tile_n = F == kGated ? kTileN / 2 : kTileN;
  return {{kMatmulTiles, kTileM, kTileN}, tile_kernel<VEC, F>, tiles_of(l, kTileM, tile_n), 256};
}

// ---- pipelined tile kernel ---------------------------------------------

// TM tokens by TN rows of b, 128 bytes of k a block, two blocks in LDS.
// Waves of WTM tokens by 128 rows of b in 16x16x64 products: with operands
// of random bits the card's power limit holds a loop of these from registers
// to 4.1 POP/s, and of 32x32x32 ones (more accumulator traffic) to 3.5.
//
// Work-groups stay on the card and walk over tiles. Operands go from memory
// straight into LDS, a block ahead and across the end of a tile, so that a
// tile's epilogue runs while the next one's first blocks arrive. A load
// covers 8 rows of 128 bytes: of whole lines the L2 caches deliver 32 TB/s,
// of 16 half lines a load 17 TB/s.
//
// Chunk c (16 bytes) of row r lies in slot c ^ (r / 2 % 8). LDS serves a
// 16-byte read of a wave in four groups of 16 lanes, {0-3, 12-15, 20-23,
// 24-27} and {4-11, 16-19, 28-31} of each half; with this order of slots none
// of them has two lanes on a bank. The loads fill LDS in lane order, so each
// lane asks for the chunk that belongs in its slot.
//
// A block is two stages of 64 bytes of k. A wave's products of a stage are
// four quarters, of half its a and half its b fragments each, in an order in
// which consecutive quarters share one half: then the other is free to be
// read for the quarter after, and one set of fragment registers is enough (a
// second one costs 32 moves a stage):
//   first stage   (a0 b0) (a0 b1)   (a1 b1) (a1 b0)
//   second stage  (a0 b1) (a0 b0) | (a1 b0) (a1 b1)
// At the bar, the block's one barrier, every wave holds all of the block that
// it still needs in registers (its LDS is free for the block after next) and
// the next block has landed.
constexpr int kStep = 64;
constexpr int kBlockK = 2 * kStep;
constexpr int kWaveN = 128;
[[maybe_unused]] constexpr int kLoadQuarters = 4;  // quarters that a block's loads are spread over

// acc += b a^T of one 16x16x64 product, in place. (Used in the device pass
// alone, like the rest of the pipeline.) Written out because the
// compiler takes a result for a value of its own and, over several stages,
// moves accumulators between registers inside the pipeline. It sees no
// matrix instruction here, so the waits that such results need before other
// instructions touch them stand in settle().
[[maybe_unused]] __device__ __forceinline__ void mfma(i32x4& acc, const i32x4& b, const i32x4& a) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}

// acc = b a^T.
[[maybe_unused]] __device__ __forceinline__ void mfma_first(i32x4& acc, const i32x4& b, const i32x4& a) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, 0" : "=a"(acc) : "v"(b), "v"(a));
}

// A row of accumulators, readable by other instructions (after at most 18
// cycles).
template <int N>
__device__ __forceinline__ void settle(i32x4 (&acc)[N]) {
  static_assert(N == 8, "one operand for each");
  asm volatile("s_nop 15\n\ts_nop 3"
               : "+a"(acc[0]), "+a"(acc[1]), "+a"(acc[2]), "+a"(acc[3]), "+a"(acc[4]), "+a"(acc[5]), "+a"(acc[6]),
                 "+a"(acc[7]));
}

template <int TM, int TN, int WTM>
struct Pipe {
  static constexpr int kWavesM = TM / WTM, kWavesN = TN / kWaveN, kWaves = kWavesM * kWavesN, kThreads = 64 * kWaves;
  static constexpr int FM = WTM / 16, FN = kWaveN / 16;
  static constexpr int kLoadsA = TM / 8 / kWaves, kLoadsB = TN / 8 / kWaves, kLoads = kLoadsA + kLoadsB;
  static constexpr int kBlockBytes = (TM + TN) * kBlockK;
  static constexpr int kSumsBytes = 16 * kWaveN * 4;  // 16 tokens of a wave
  static constexpr int kLds = 2 * kBlockBytes + kWaves * kSumsBytes;
  static constexpr int kPerCu = 163840 / kLds;  // work-groups a CU holds
  static_assert(TM % (8 * kWaves) == 0 && TN % (8 * kWaves) == 0, "whole loads a wave");
  static_assert(kLoads % 4 == 0 && FM % 2 == 0, "quarters");
};

#ifdef __HIP_DEVICE_COMPILE__
// Stores of a wave's part of a tile that lies whole inside the output, from
// token i0 and channel j0 on; this lane's are of token i0 + row + t and
// channels j0 + col .. + 7. A uniform base, a lane's offset and the token in a
// scalar, so that no address is computed for a store. They go past the caches
// (16384 x 8192 bf16 values: 404 -> 379 us; they fill L2 otherwise), but for
// binary32, two stores of half lines a piece.
template <int F>
struct WholeTile {
  static constexpr int kStream = 2;
  __amdgpu_buffer_rsrc_t out, scales;
  uint32_t out_lane, out_row, scale_lane, scale_row;
  bool has_scale;

  __device__ __forceinline__ WholeTile(const MatmulLaunch& a, uint32_t i0, uint32_t j0, uint32_t row, uint32_t col) {
    const uint32_t size = F == kCodes ? 1 : a.out_format == kOutF32 ? 4 : 2;
    out_row = static_cast<uint32_t>(a.out_stride) * size;
    out_lane = row * out_row + col * size;
    out = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<char*>(a.out) + static_cast<uint64_t>(i0) * out_row + static_cast<uint64_t>(j0) * size, 0, kFar,
        0x00020000);
    if constexpr (F == kCodes) {
      const bool mx = a.scale_layout == kScaleE8M0Block32;
      const uint32_t g = mx ? 32 : 128, scale_size = mx ? 1 : 4;
      scale_row = a.n / g * scale_size;
      scale_lane = row * scale_row + col / g * scale_size;
      has_scale = col % g == 0;
      scales = __builtin_amdgcn_make_buffer_rsrc(
          static_cast<char*>(a.scales) + static_cast<uint64_t>(i0) * scale_row + j0 / g * scale_size, 0, kFar,
          0x00020000);
    }
  }

  __device__ __forceinline__ void store(const MatmulLaunch& a, uint32_t t, const float* v, bool no_nan) const {
    if constexpr (F == kCodes) {
      uint32_t scale;
      const Codes<kPiece> codes = encode_group(a, v, no_nan, &scale);
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{codes.w[0], codes.w[1]}, out, out_lane, t * out_row, kStream);
      if (has_scale) {
        if (a.scale_layout == kScaleE8M0Block32)
          __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(scale), scales, scale_lane, t * scale_row, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b32(scale, scales, scale_lane, t * scale_row, 0);
      }
    } else if (a.out_format == kOutF32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 w = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), out, out_lane + 16 * h, t * out_row, 0);
      }
    } else {
      const bool bf = a.out_format == kOutBF16;
      u32x4 w;
#pragma unroll
      for (int h = 0; h < 4; ++h)
        w[h] = bf ? pack2<kOutBF16>(v[2 * h], v[2 * h + 1]) : pack2<kOutF16>(v[2 * h], v[2 * h + 1]);
      __builtin_amdgcn_raw_buffer_store_b128(w, out, out_lane, t * out_row, kStream);
    }
  }
};
#endif

template <int TM, int TN, int WTM, int F>
__global__ __launch_bounds__((Pipe<TM, TN, WTM>::kThreads), 1) void pipe_kernel(const MatmulLaunch a) {
#ifdef __HIP_DEVICE_COMPILE__  // the buffer builtins' types exist in the device pass alone
  using P = Pipe<TM, TN, WTM>;
  constexpr int FM = P::FM, FN = P::FN, HM = FM / 2, HN = FN / 2;
  __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave % P::kWavesM, wn = wave / P::kWavesM;

  // Work-groups go round the eight XCDs: XCD x runs one eighth of the tiles,
  // consecutive ones, its work-groups taking every (gridDim / 8)th.
  constexpr uint32_t tile_n = F == kGated ? TN / 2 : TN;
  const TileOrder order = {(a.m + TM - 1) / TM, (a.n + tile_n - 1) / tile_n};
  const uint32_t tiles = order.tiles_m * order.tiles_n;
  const uint32_t xcd = blockIdx.x % 8, stride = gridDim.x / 8;
  const uint32_t end = (tiles / 8) * (xcd + 1) + min(xcd + 1, tiles % 8);
  uint32_t tile = (tiles / 8) * xcd + min(xcd, tiles % 8) + blockIdx.x / 8;
  if (tile >= end) return;

  // The loads' cursor: a tile, a block in it, and the lanes' offsets. Load t
  // of a wave covers 8 rows; lane l the chunk of row l / 8 whose slot is l % 8.
  const uint32_t blocks = (a.k + kBlockK - 1) / kBlockK;
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t off_a[P::kLoadsA], off_b[P::kLoadsB];
  uint32_t load_tile = tile, load_block = 0, load_slot = 0, load_k = 0, far[2] = {0, 0};
  // The chunk of an even or odd load: rows 8 t + l / 8, so r / 2 % 8 = 4 (t % 2) + l / 16.
  const uint32_t chunk[2] = {(lane % 8 ^ lane / 16) * 16u, (lane % 8 ^ (4 + lane / 16)) * 16u};
  auto aim_tile = [&]() {
    uint32_t tm, tn;
    order.at(load_tile, &tm, &tn);
    const uint32_t i0 = tm * TM, j0 = tn * tile_n;
    ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.a + static_cast<uint64_t>(i0) * a.a_stride), 0, kFar,
                                           0x00020000);
    rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.b + static_cast<uint64_t>(j0) * a.b_stride), 0, kFar,
                                           0x00020000);
    // Rows past the end load the last row; what they give is not stored.
#pragma unroll
    for (int t = 0; t < P::kLoadsA; ++t) {
      const uint32_t r = (wave * P::kLoadsA + t) * 8 + lane / 8;
      off_a[t] = (min(i0 + r, a.m - 1) - i0) * static_cast<uint32_t>(a.a_stride);
    }
#pragma unroll
    for (int t = 0; t < P::kLoadsB; ++t) {
      const uint32_t r = (wave * P::kLoadsB + t) * 8 + lane / 8;
      uint32_t j = r;
      if constexpr (F == kGated) j = r / kWaveN * (kWaveN / 2) + r % (kWaveN / 2);  // a wave's gates, then its ups
      j = min(j0 + j, a.n - 1) - j0;
      if (F == kGated && r % kWaveN >= kWaveN / 2) j += a.n;
      off_b[t] = j * static_cast<uint32_t>(a.b_stride);
    }
  };
  auto aim_block = [&]() {  // no branch: this runs inside the pipeline
    load_k = __builtin_amdgcn_readfirstlane(load_block * kBlockK);
    const uint32_t k_end = load_tile < end ? a.k : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) far[h] = load_k + chunk[h] < k_end ? chunk[h] : kFar;
  };
  auto advance = [&]() {
    load_slot ^= 1;
    ++load_block;
    aim_block();
  };
  auto next_tile = [&]() {
    load_slot ^= 1;
    load_block = 0;
    load_tile += stride;
    if (load_tile < end) aim_tile();
    aim_block();
  };
  // Load t of the cursor's block: a's, then b's.
  static_assert(P::kLoadsA % 2 == 0 && P::kLoadsB % 2 == 0, "loads alternate between even and odd rows of 8");
  auto load = [&](int t) {
    char* base = lds + load_slot * P::kBlockBytes;
    if (t < P::kLoadsA) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(base + (wave * P::kLoadsA + t) * 1024), 16,
                                               off_a[t] + far[t % 2], load_k, 0, 0);
    } else {
      const int u = t - P::kLoadsA;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(base + TM * kBlockK + (wave * P::kLoadsB + u) * 1024), 16,
                                               off_b[u] + far[u % 2], load_k, 0, 0);
    }
  };

  // A quarter issues kQuarter loads; kEarly quarters' worth of a block's go
  // out in the block before the one that precedes it ends.
  constexpr int kQuarter = P::kLoads / kLoadQuarters, kEarly = kLoadQuarters < 2 ? kLoadQuarters : 2;
  aim_tile();
  aim_block();
#pragma unroll
  for (int t = 0; t < P::kLoads; ++t) load(t);
  advance();
#pragma unroll
  for (int t = 0; t < kEarly * kQuarter; ++t) load(t);

  // Lane l reads row l % 16 of a fragment, chunk l / 16 of a stage's four.
  const uint32_t lane_off[2] = {lane % 16 * kBlockK + ((lane / 16) ^ (lane % 16 / 2)) * 16u,
                                lane % 16 * kBlockK + ((4 + lane / 16) ^ (lane % 16 / 2)) * 16u};
  const char* base_a = lds + wm * WTM * kBlockK;
  const char* base_b = lds + TM * kBlockK + wn * kWaveN * kBlockK;
  i32x4 acc[FM][FN], fa[FM], fb[FN];
  uint32_t slot = 0;
  // A tile's first bar waits for loads that were issued before the last
  // epilogue's stores. Loads and stores are counted in order: where all of
  // that epilogue's stores were made (a whole tile: one a piece at least), it
  // lets that many be under way.
  constexpr int kWholeStores = FM * 16 * (F == kGated ? kWaveN / 2 : kWaveN) / kPiece / 64;
  bool whole_before = false;
  auto read_a = [&](uint32_t from, int st, int i) {
    fa[i] = *reinterpret_cast<const i32x4*>(base_a + from * P::kBlockBytes + lane_off[st] + i * 16 * kBlockK);
  };
  auto read_b = [&](uint32_t from, int st, int j) {
    fb[j] = *reinterpret_cast<const i32x4*>(base_b + from * P::kBlockBytes + lane_off[st] + j * 16 * kBlockK);
  };
  // Products of a's half ha and b's half hb, each with at most one other
  // instruction behind it: first the reads of the quarter after, of stage st
  // of block `from`, then the loads of `part`, spread over the rest. In this
  // order, so that the matrix unit never waits for a row of others.
  auto quarter = [&](int ha, int hb, bool reads_a, uint32_t from, int st, int half, int part, bool first = false) {
    const int reads = reads_a ? HM : HN;
    const int loads = part < kLoadQuarters ? kQuarter : 0;
    constexpr int kProducts = HM * HN, kOthers = (HM > HN ? HM : HN) + kQuarter;
    const int each = kProducts > reads + kQuarter ? (kProducts - reads) / kQuarter : 1;
#pragma unroll
    for (int x = 0; x < (kProducts > kOthers ? kProducts : kOthers); ++x) {
      if (x < kProducts) {
        const int i = ha * HM + x / HN, j = hb * HN + x % HN;
        if (first)
          mfma_first(acc[i][j], fb[j], fa[i]);
        else
          mfma(acc[i][j], fb[j], fa[i]);
      }
      if (x < reads) {
        if (reads_a)
          read_a(from, st, half * HM + x);
        else
          read_b(from, st, half * HN + x);
      } else if ((x - reads) % each == 0 && (x - reads) / each < loads) {
        load(part * kQuarter + (x - reads) / each);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  constexpr int kNone = kLoadQuarters;
  // `first`: the tile's first block, whose next block is all on its way.
  // `last_load`: the cursor's block is its tile's last.
  auto block = [&](bool first, bool last_load) {
    const uint32_t next = slot ^ 1;
    quarter(0, 0, false, slot, 0, 1, first ? kNone : 2, first);
    quarter(0, 1, true, slot, 0, 1, first ? kNone : 3, first);
    quarter(1, 1, true, slot, 1, 0, kNone, first);
    quarter(1, 0, false, slot, 1, 1, kNone, first);
    quarter(0, 1, false, slot, 1, 0, kNone);
    quarter(0, 0, true, slot, 1, 1, kNone);
    if (last_load)
      next_tile();
    else
      advance();
    if (first && whole_before)
      wait_loads_and_sync<kWholeStores>();
    else
      wait_loads_and_sync<0>();
    quarter(1, 0, true, next, 0, 0, 0);
    quarter(1, 1, false, next, 0, 0, 1);
    slot = next;
  };

  wait_loads_and_sync<kEarly * kQuarter>();
#pragma unroll
  for (int i = 0; i < HM; ++i) read_a(0, 0, i);
#pragma unroll
  for (int j = 0; j < HN; ++j) read_b(0, 0, j);
#pragma unroll
  for (int t = kEarly * kQuarter; t < P::kLoads; ++t) load(t);
  constexpr uint32_t out_n = F == kGated ? kWaveN / 2 : kWaveN;  // output channels of a wave
  constexpr uint32_t pieces = out_n / kPiece;
  int32_t* sums = reinterpret_cast<int32_t*>(lds + 2 * P::kBlockBytes + wave * P::kSumsBytes);
  for (; tile < end; tile += stride) {
    uint32_t tm, tn;
    order.at(tile, &tm, &tn);
    const uint32_t i0 = tm * TM + wm * WTM;
    const uint32_t j = tn * tile_n + wn * out_n + lane % pieces * kPiece;
    // At a block's bar the loads move on to the block after next: to the next
    // tile's first two in this tile's last two.
    if (blocks == 2) {
      block(true, true);
    } else {
      block(true, false);
      for (uint32_t b = 3; b < blocks; ++b) block(false, false);
      block(false, true);
    }
    // Scales, asked for a block ahead of their use.
    constexpr uint32_t kPass = 64 / pieces;  // tokens at a time
    float sa[FM][16 / kPass];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (uint32_t t = 0; t < 16 / kPass; ++t)
        sa[i][t] = a.a_scales[min(i0 + 16 * i + t * kPass + lane / pieces, a.m - 1)];
    const PieceScales sb = piece_scales<F>(a, j);
    block(false, false);
#pragma unroll
    for (int t = kEarly * kQuarter; t < P::kLoads; ++t) load(t);

    // 16 tokens at a time through the wave's own part of LDS; 16-byte units
    // of a token's row are xored with the token, which keeps writes of one
    // column off one bank.
    auto stage_sums = [&](int i) {
      __builtin_amdgcn_sched_barrier(0);  // one fragment's values in registers at a time
      lds_wave_order();
      settle(acc[i]);
#pragma unroll
      for (int g = 0; g < FN; ++g)  // lane l holds channels 4 (l / 16) .. + 3 of token l % 16
        *reinterpret_cast<i32x4*>(sums + lane % 16 * kWaveN + ((4 * g + lane / 16) ^ (lane % 16)) * 4) = acc[i][g];
      lds_wave_order();
    };
    auto values = [&](uint32_t t, uint32_t unit, float scale, float* v) {
      const i32x4* row = reinterpret_cast<const i32x4*>(sums + t * kWaveN);
      const i32x4 lo = row[unit ^ t], hi = row[(unit + 1) ^ t];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = static_cast<float>(lo[e]) * scale;
        v[4 + e] = static_cast<float>(hi[e]) * scale;
      }
    };
    const uint32_t unit = lane % pieces * 2;
    whole_before = tm * TM + TM <= a.m && (tn + 1) * tile_n <= a.n && (F == kCodes || a.out_vec) && a.out_near;
    if (whole_before) {
      const WholeTile<F> whole(a, i0, tn * tile_n + wn * out_n, lane / pieces, lane % pieces * kPiece);
      const bool sb_finite = F != kCodes || sb.finite();
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        stage_sums(i);
#pragma unroll
        for (uint32_t p = 0; p < 16 / kPass; ++p) {
          const uint32_t t = p * kPass + lane / pieces;
          float v[kPiece], up[kPiece];
          values(t, unit, sa[i][p], v);
          if constexpr (F == kGated) values(t, unit + 2 * pieces, sa[i][p], up);
          scale_piece<F>(sb, v, up);
          whole.store(a, 16 * i + p * kPass, v, sb_finite && keeps_finite(sa[i][p]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        stage_sums(i);
#pragma unroll 1
        for (uint32_t p = 0; p < 16 / kPass; ++p) {
          const uint32_t t = p * kPass + lane / pieces;
          const uint32_t token = i0 + 16 * i + t;
          const float scale = a.a_scales[min(token, a.m - 1)];
          float v[kPiece], up[kPiece];
          values(t, unit, scale, v);
          if constexpr (F == kGated) values(t, unit + 2 * pieces, scale, up);
          finish_piece<F>(a, token, j, token < a.m && j < a.n, scale, sb, v, up);
        }
      }
    }
  }
  // Nothing is in flight to this work-group's LDS when it ends.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#endif
}

// ---- few tokens --------------------------------------------------------

// Up to 16 * MT tokens: the weights are read once and bound the time, so
// many loads are in flight at once, straight into registers. A work-group of
// 16 waves takes RB * GW rows of b (gated: in runs of RB / 2 gates and their
// ups); its GW groups of KW waves take RB rows each and share k: wave w of a
// group takes every KW'th 128 bytes of its rows (a line of each), kPairs of
// them in flight.
//
// Eight neighbouring lanes load the line of a row. Fragments want one row a
// lane, but loads of that shape cost an access to the first cache for every
// lane (16 bytes a cycle: 12.5 us for one token by 1024 x 8192), so a wave
// turns its lines round in its own part of LDS; chunk c of row r lies in slot
// c ^ (r / 2 % 8), which keeps the reads off each other's banks.
//
// The waves' integer sums meet in LDS, where the order of the additions
// cannot matter.
template <int MT, int GW, int RB, int F>
__global__ __launch_bounds__(1024) void few_tokens_kernel(const MatmulLaunch a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int KW = 16 / GW;
  constexpr int kPairs = MT == 1 ? 4 : 2, FB = RB / 16, kLinesB = RB / 8;
  constexpr uint32_t kRows = RB * GW, kOut = F == kGated ? kRows / 2 : kRows;
  constexpr uint32_t kPitch = kRows + 4;
  __shared__ __attribute__((aligned(16))) int32_t sums[16 * MT * kPitch];
  __shared__ float row_scale[kRows], token_scale[16 * MT];
  constexpr int kWaveRows = RB + 16 * MT;  // of b, then the tokens
  __shared__ __attribute__((aligned(128))) char turn[16 * kWaveRows * 128];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t group = wave / KW, kw = wave % KW;
  const uint32_t j0 = blockIdx.x * kOut;

  auto row_of = [&](uint32_t r) {  // of the work-group's part of b
    if constexpr (F == kGated) return min(j0 + r / RB * (RB / 2) + r % (RB / 2), a.n - 1) + (r % RB >= RB / 2 ? a.n : 0);
    return min(j0 + r, a.n - 1);
  };
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.a), 0, kFar, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.b + static_cast<uint64_t>(j0) * a.b_stride), 0, kFar, 0x00020000);
  // Load t of a line covers rows 8 t .. 8 t + 7; tokens past the last are zeros.
  const uint32_t chunk = lane % 8 * 16;
  uint32_t off_b[kLinesB], off_a[2 * MT];
#pragma unroll
  for (int t = 0; t < kLinesB; ++t)
    off_b[t] = (row_of(group * RB + 8 * t + lane / 8) - j0) * static_cast<uint32_t>(a.b_stride) + chunk;
#pragma unroll
  for (int t = 0; t < 2 * MT; ++t) {
    const uint32_t i = 8 * t + lane / 8;
    off_a[t] = i < a.m ? i * static_cast<uint32_t>(a.a_stride) + chunk : kFar;
  }
  char* mine = turn + wave * kWaveRows * 128;

  i32x4 acc[MT][FB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < FB; ++h) acc[i][h] = i32x4{0, 0, 0, 0};
  // One of the work-group's scales a thread: of its rows of b, then of the tokens.
  const bool has_scale = threadIdx.x < kRows + 16 * MT;
  const float* scale_at = threadIdx.x < kRows ? a.b_scales + row_of(threadIdx.x)
                                              : a.a_scales + min(threadIdx.x - kRows, a.m - 1);
  float scale = 0.0f;
  const uint32_t pairs = (a.k + 127) / 128;
  for (uint32_t p0 = kw; p0 < pairs; p0 += KW * kPairs) {
    i32x4 lb[kPairs][kLinesB], la[kPairs][2 * MT];
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      const uint32_t k = (p0 + q * KW) * 128;
      const uint32_t far = k + chunk < a.k ? 0 : kFar;  // past the end of k: zeros
#pragma unroll
      for (int t = 0; t < kLinesB; ++t)
        lb[q][t] = __builtin_amdgcn_raw_buffer_load_b128(rb, off_b[t] + far, k, 2);  // 2: streamed, not kept
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) la[q][t] = __builtin_amdgcn_raw_buffer_load_b128(ra, off_a[t] | far, k, 0);
    }
    if (p0 == kw && has_scale) scale = *scale_at;  // behind the first operands, which do not wait for it
    __builtin_amdgcn_sched_barrier(0);  // all loads, then the products
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      auto put = [&](int t, const i32x4& v) {  // rows 8 t .. 8 t + 7 of the wave's
        const uint32_t slot = lane % 8 ^ (t % 2 * 4 + lane / 16);
        *reinterpret_cast<i32x4*>(mine + (8 * t + lane / 8) * 128 + slot * 16) = v;
      };
      auto fragment = [&](int f, int unit) {  // rows 16 f .. 16 f + 15, chunks 4 unit ..
        const uint32_t slot = (4 * unit + lane / 16) ^ (lane % 16 / 2);
        return *reinterpret_cast<const i32x4*>(mine + (16 * f + lane % 16) * 128 + slot * 16);
      };
#pragma unroll
      for (int t = 0; t < kLinesB; ++t) put(t, lb[q][t]);
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) put(kLinesB + t, la[q][t]);
      lds_wave_order();
#pragma unroll
      for (int unit = 0; unit < 2; ++unit) {
        i32x4 fb[FB];
#pragma unroll
        for (int h = 0; h < FB; ++h) fb[h] = fragment(h, unit);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const i32x4 fa = fragment(FB + i, unit);
#pragma unroll
          for (int h = 0; h < FB; ++h) acc[i][h] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[h], fa, acc[i][h], 0, 0, 0);
        }
      }
      lds_wave_order();
    }
  }

  for (uint32_t t = threadIdx.x; t < 16 * MT * kPitch; t += 1024) sums[t] = 0;
  if (kw >= pairs && has_scale) scale = *scale_at;  // a wave without a step
  if (threadIdx.x < kRows)
    row_scale[threadIdx.x] = scale;
  else if (threadIdx.x < kRows + 16 * MT)
    token_scale[threadIdx.x - kRows] = scale;
  __syncthreads();
  // Lane l holds channels 4 (l / 16) .. + 3 of token l % 16.
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < FB; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        atomicAdd(&sums[(16 * i + lane % 16) * kPitch + group * RB + h * 16 + lane / 16 * 4 + e], acc[i][h][e]);
  __syncthreads();
  constexpr uint32_t pieces = kOut / kPiece;
  static_assert(16 * MT * pieces <= 1024, "one piece a thread");
  if (threadIdx.x >= 16 * MT * pieces) return;
  const uint32_t i = threadIdx.x / pieces, jj = threadIdx.x % pieces * kPiece;
  const uint32_t r = F == kGated ? jj / (RB / 2) * RB + jj % (RB / 2) : jj;
  const int32_t* row = sums + i * kPitch + r;
  float v[kPiece], up[kPiece];
  PieceScales sb;
#pragma unroll
  for (int e = 0; e < kPiece; ++e) {
    v[e] = static_cast<float>(row[e]) * token_scale[i];
    sb.b[e] = row_scale[r + e];
    if constexpr (F == kGated) {
      up[e] = static_cast<float>(row[RB / 2 + e]) * token_scale[i];
      sb.up[e] = row_scale[r + RB / 2 + e];
    }
  }
  finish_piece<F>(a, i, j0 + jj, i < a.m && j0 + jj < a.n, token_scale[i], sb, v, up);
#endif
}

template <int MT, int GW, int RB, int F>
Choice few(const MatmulLaunch& l) {
  constexpr uint32_t out = (F == kGated ? RB / 2 : RB) * GW;
  return {{kMatmulFewTokens, 16 * MT, RB * GW}, few_tokens_kernel<MT, GW, RB, F>, tiles_of(l, 16 * MT, out), 1024};
}

template <int MT, int F>
Choice few_sized(const MatmulLaunch& l) {
  if constexpr (F == kCodes) {
    // Codes need a whole group of 128 or 32 channels in one work-group.
    if (l.scale_layout == kScaleF32Group128) return few<MT, 4, 32, F>(l);
    return few<MT, 1, 32, F>(l);
  } else {
    // Narrow work-groups where wide ones would leave half of the CUs idle.
    const uint32_t rows = F == kGated ? 2 * l.n : l.n;
    return rows <= 16 * kCus ? few<MT, 1, 16, F>(l) : few<MT, 1, 32, F>(l);
  }
}

// ---- tens to hundreds of tokens ----------------------------------------

// Too few tiles of the pipelined kernel for 256 CUs: TM tokens by TN rows of
// b a work-group, whose eight waves also share k, so that its sums need no
// second pass through memory. Wave (g, w) takes 64-byte step g of each
// stage's KG steps and TN / (8 / KG) rows of b.
//
// A stage is KG / 2 blocks of rows of 128 bytes, loaded straight into LDS, 8
// rows a load, S - 1 stages ahead, so that most of LDS holds operands in
// flight, in whole lines. What bounds these tiles is how fast operands come
// into a CU: 333 tokens by 5120, k = 7168 (f16, 240 tiles of 64 x 128) ask L2
// for 325 MB, 82 % of it found there, at 50 GB/s a CU with weights from HBM
// (27 us) and 68 with weights in the Infinity Cache (20 us): 25 and 34 bytes a
// cycle of the 64 that a CU can take, the matrix units busy for a quarter of
// the time. More in flight is what is missing, and LDS is full. Slots as
// in few_tokens_kernel. Two waves a SIMD hide each other's reads; one barrier a
// stage.
template <int TM, int TN, int KG, int S>
struct Mid {
  static constexpr int kThreads = 512, kWavesN = 8 / KG, WTN = TN / kWavesN;
  static constexpr int FM = TM / 16, FN = WTN / 16;
  static constexpr int kRows = TM + TN, kStageK = 64 * KG;
  static constexpr int kStageBytes = kRows * kStageK;
  static constexpr int kLoads = kStageBytes / 1024 / 8;  // a wave
  static constexpr int kPitch = TN + 4;  // words of a token's sums
  static constexpr int kScales = S * kStageBytes > TM * kPitch * 4 ? S * kStageBytes : TM * kPitch * 4;
  static constexpr int kLds = kScales + kRows * 4;
  static_assert(KG % 2 == 0 && kStageBytes % 8192 == 0 && WTN % 16 == 0 && TM % 16 == 0, "whole loads and fragments");
  static_assert(kRows <= kThreads, "one scale a thread");
};

template <int TM, int TN, int KG, int S, int F>
__global__ __launch_bounds__(512, 1) void mid_kernel(const MatmulLaunch a) {
#ifdef __HIP_DEVICE_COMPILE__
  using P = Mid<TM, TN, KG, S>;
  constexpr int FM = P::FM, FN = P::FN;
  // One array: with several, the compiler tells their accesses apart and
  // waits for every load to LDS before it reads any.
  __shared__ __attribute__((aligned(1024))) char lds[P::kLds];
  float* scales = reinterpret_cast<float*>(lds + P::kScales);
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int g = wave % KG, wn = wave / KG;

  constexpr uint32_t kOut = F == kGated ? TN / 2 : TN;
  const TileOrder order = {(a.m + TM - 1) / TM, (a.n + kOut - 1) / kOut};
  const uint32_t tiles = order.tiles_m * order.tiles_n, xcd = blockIdx.x % 8;
  uint32_t tm, tn;
  order.at((tiles / 8) * xcd + min(xcd, tiles % 8) + blockIdx.x / 8, &tm, &tn);
  const uint32_t i0 = tm * TM, j0 = tn * kOut;
  // Row r of the tile's part of b: in the gated form every fragment of 16
  // gates is followed by their ups.
  auto row_of = [&](uint32_t r) {
    if constexpr (F == kGated) return min(j0 + r / 32 * 16 + r % 16, a.n - 1) + (r % 32 >= 16 ? a.n : 0);
    return min(j0 + r, a.n - 1);
  };
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.a + static_cast<uint64_t>(i0) * a.a_stride), 0, kFar, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.b + static_cast<uint64_t>(j0) * a.b_stride), 0, kFar, 0x00020000);

  // Load t covers rows 8 (t % (kRows / 8)) .. + 7 of block t / (kRows / 8);
  // lane l the chunk of row l / 8 whose slot is l % 8.
  uint32_t offset[P::kLoads], in_k[P::kLoads];
#pragma unroll
  for (int t = 0; t < P::kLoads; ++t) {
    const uint32_t at = wave * P::kLoads + t, r = at % (P::kRows / 8) * 8 + lane / 8;
    in_k[t] = at / (P::kRows / 8) * 128 + (lane % 8 ^ (r / 2 % 8)) * 16;
    offset[t] = (r < TM ? (min(i0 + r, a.m - 1) - i0) * static_cast<uint32_t>(a.a_stride)
                        : (row_of(r - TM) - j0) * static_cast<uint32_t>(a.b_stride)) + in_k[t];
  }
  // Load t of stage st, to `slot`; `full`: the stage ends inside k.
  auto load = [&](uint32_t st, uint32_t slot, int t, bool full) {
    const uint32_t k = __builtin_amdgcn_readfirstlane(st * P::kStageK);
    const uint32_t at = wave * P::kLoads + t;
    char* to = lds + slot * P::kStageBytes + at * 1024;
    const uint32_t far = full || k + in_k[t] < a.k ? 0 : kFar;  // past the end of k: zeros
    __builtin_amdgcn_raw_ptr_buffer_load_lds(at % (P::kRows / 8) * 8 < TM ? ra : rb, (lds_ptr)to, 16, offset[t] + far, k,
                                             0, 0);
  };

  float scale = 0.0f;
  if (threadIdx.x < P::kRows)
    scale = threadIdx.x < TM ? a.a_scales[min(i0 + threadIdx.x, a.m - 1)] : a.b_scales[row_of(threadIdx.x - TM)];
  const uint32_t stages = (a.k + P::kStageK - 1) / P::kStageK, full_stages = a.k / P::kStageK;
#pragma unroll
  for (uint32_t st = 0; st < S; ++st)  // past the last stage: zeros
#pragma unroll
    for (int t = 0; t < P::kLoads; ++t) load(st, st, t, false);

  i32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const uint32_t chunk_slot = ((4 * (g % 2) + lane / 16) ^ (lane % 16 / 2)) * 16;
  const char* frag = lds + g / 2 * P::kRows * 128 + lane % 16 * 128 + chunk_slot;
  const char* frag_b = frag + (TM + wn * P::WTN) * 128;
  i32x4 fa[2][FM], fb[2][FN];  // of even and odd stages
  auto read = [&](int set, uint32_t slot, int x) {
    const uint32_t base = slot * P::kStageBytes;
    if (x < FN)
      fb[set][x] = *reinterpret_cast<const i32x4*>(frag_b + base + x * 16 * 128);
    else
      fa[set][x - FN] = *reinterpret_cast<const i32x4*>(frag + base + (x - FN) * 16 * 128);
  };
  // Multiplies stage st (in registers, its LDS `slot`) while stage st + 1 is
  // read and stage st + S loaded into st's place in LDS.
  auto stage = [&](uint32_t st, uint32_t slot, int set, bool full) {
    wait_loads_and_sync<P::kLoads * (S - 2)>();
    constexpr int kProducts = FM * FN, kReads = FM + FN, kOthers = kReads + P::kLoads;
    const uint32_t next = slot + 1 == S ? 0 : slot + 1;
#pragma unroll
    for (int x = 0; x < (kProducts > kOthers ? kProducts : kOthers); ++x) {
      if (x < kProducts) {
        const int i = x / FN, j = x % FN;
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
      }
      if (x < kReads)
        read(1 - set, next, x);
      else if (x < kOthers)
        load(st + S, slot, x - kReads, full);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  wait_loads_and_sync<P::kLoads * (S - 1)>();
#pragma unroll
  for (int x = 0; x < FM + FN; ++x) read(0, 0, x);
  // Rounds with fixed slots and nothing to check, while all that they load is
  // inside k; then two stages a round (an odd last one is followed by zeros).
  constexpr uint32_t kRound = S % 2 == 0 ? S : 2 * S;
  uint32_t st = 0;
  for (; st + S + kRound <= full_stages; st += kRound) {
#pragma unroll
    for (uint32_t r = 0; r < kRound; ++r) stage(st + r, r % S, r % 2, true);
  }
  for (; st < stages; st += 2) {
    stage(st, st % S, 0, false);
    stage(st + 1, (st + 1) % S, 1, false);
  }

  // The KG partial sums meet in LDS: one wave of each column writes, the
  // others add.
  wait_loads_and_sync<0>();
  int32_t* sums = reinterpret_cast<int32_t*>(lds);
  // Lane l holds channels 4 (l / 16) .. + 3 of token l % 16 of a fragment.
  int32_t* at = sums + lane % 16 * P::kPitch + wn * P::WTN + lane / 16 * 4;
  if (g == 0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) *reinterpret_cast<i32x4*>(at + i * 16 * P::kPitch + j * 16) = acc[i][j];
  }
  if (threadIdx.x < P::kRows) scales[threadIdx.x] = scale;
  __syncthreads();
  if (g != 0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) atomicAdd(at + i * 16 * P::kPitch + j * 16 + e, acc[i][j][e]);
  }
  __syncthreads();
  constexpr uint32_t pieces = kOut / kPiece;
  static_assert(TM * pieces % 64 == 0, "whole waves");
  for (uint32_t t = threadIdx.x; t < TM * pieces; t += P::kThreads) {
    const uint32_t i = t / pieces, jj = t % pieces * kPiece;
    const uint32_t r = F == kGated ? jj / 16 * 32 + jj % 16 : jj;
    const int32_t* row = sums + i * P::kPitch + r;
    float v[kPiece], up[kPiece];
    PieceScales sb;
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      v[e] = static_cast<float>(row[e]) * scales[i];
      sb.b[e] = scales[TM + r + e];
      if constexpr (F == kGated) {
        up[e] = static_cast<float>(row[16 + e]) * scales[i];
        sb.up[e] = scales[TM + r + 16 + e];
      }
    }
    finish_piece<F>(a, i0 + i, j0 + jj, i0 + i < a.m && j0 + jj < a.n, scales[i], sb, v, up);
  }
#endif
}

template <int TM, int TN, int KG, int S, int F>
Choice mid(const MatmulLaunch& l) {
  return {{kMatmulMid, TM, TN}, mid_kernel<TM, TN, KG, S, F>, tiles_of(l, TM, F == kGated ? TN / 2 : TN), 512};
}

template <int TM, int TN, int WTM, int F>
Choice pipe(const MatmulLaunch&) {
  using P = Pipe<TM, TN, WTM>;
  return {{kMatmulPipe, TM, TN}, pipe_kernel<TM, TN, WTM, F>, kCus * P::kPerCu, P::kThreads};
}

// Rows of operands that the busiest CU loads with tiles of TM tokens by TN
// rows of b: what a call's time goes by.
template <int TM, int TN, int F>
uint64_t rows_a_cu(const MatmulLaunch& l) {
  return (tiles_of(l, TM, F == kGated ? TN / 2 : TN) + kCus - 1) / kCus * (TM + TN);
}

template <int F>
Choice choose(const MatmulLaunch& l) {
  if (!l.vec) return general_tiles<false, F>(l);
  // All but the general kernel hold offsets within a tile in 30 bits.
  const bool near = (256 + (F == kGated ? static_cast<uint64_t>(l.n) : 0)) * l.b_stride + l.k < kFar &&
                    256 * l.a_stride + l.k < kFar;
  if (!near) return general_tiles<true, F>(l);
  if (l.m <= 32) {
    const Choice c = l.m <= 16 ? few_sized<1, F>(l) : few_sized<2, F>(l);
    return c.fits() ? c : general_tiles<true, F>(l);
  }
  // The tile whose busiest CU loads least. The pipelined kernel's rows count
  // a quarter more: its CU takes 33 to 39 GB/s (the matrix units and the
  // power limit bound it), the others' 39 to 47 once most CUs have a tile.
  // k = 5120, rows of a CU and time of <256, 256> and of the best other:
  // 1536 tokens by 8192, 512 rows 75 us and 768 rows 87; 1024 by 5120, 512
  // rows 74 us and 384 rows 48; 4096 by 9472, 1536 rows 204 us and 1920 rows
  // 221.
  const bool narrow = F != kCodes || l.scale_layout == kScaleE8M0Block32;  // less than 128 channels a tile
  uint64_t least = ~uint64_t{0};
  Choice best = general_tiles<true, F>(l);
  auto offer = [&](uint64_t rows, const Choice& c) {
    if (rows < least && c.fits()) {
      least = rows;
      best = c;
    }
  };
  if (l.k > kBlockK) offer(rows_a_cu<256, 256, F>(l) * 5 / 4, pipe<256, 256, 128, F>(l));
  offer(rows_a_cu<128, 256, F>(l), mid<128, 256, 2, 3, F>(l));
  offer(rows_a_cu<128, 128, F>(l), mid<128, 128, 2, 4, F>(l));
  offer(rows_a_cu<64, 128, F>(l), mid<64, 128, 2, 6, F>(l));
  if (narrow) {
    offer(rows_a_cu<64, 64, F>(l), mid<64, 64, 4, 4, F>(l));
    offer(rows_a_cu<64, 32, F>(l), mid<64, 32, 8, 3, F>(l));
  }
  return best;
}

Choice choose(const MatmulLaunch& l) {
  if (l.quantize) return choose<kCodes>(l);
  return l.gated ? choose<kGated>(l) : choose<kValues>(l);
}

}  // namespace

MatmulShape matmul_shape(const MatmulLaunch& l) {
  const Choice c = choose(l);
  return {c.id, c.blocks, c.threads};
}

hipError_t launch_matmul(const MatmulLaunch& l, hipStream_t stream) {
  const Choice c = choose(l);
  if (!c.fits()) return hipErrorInvalidValue;
  return launch_kernel(c.kernel, dim3(static_cast<uint32_t>(c.blocks)), dim3(c.threads), stream, l);
}

}  // namespace qrs
