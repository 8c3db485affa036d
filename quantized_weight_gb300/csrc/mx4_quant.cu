// mx4_quant.cu -- rows to microscaled 4-bit codes and back (format in mx4.cuh).
//
// A block's scale is the power of two 2 ** (floor(log2(max |x|)) - 2), so its largest value lies between 4 and 8 of it and
// the codes reach 6: the exponent field of max |x| less 2, no arithmetic.  x times the inverse power is exact in float32
// (or far below the first border), so the codes are the nearest ones to the exact quotient, halves to the even code.
//
// A value is read once (2 or 4 bytes) and leaves as 17/32 of a byte.  Measured: 17408 x 5120 float32 56 us, all of measured HBM;
// 8192 x 5120 bfloat16 18.4 us, 85 % (with 8 elements a lane 22.4: instructions); 4093 x 2048 bfloat16 to 8 places each 12.5 us,
// 62 %, and 24576 sorted rows of 1408 20.9 us, 62 % (no unit is above 60 % there: places are loaded first, then rows); back,
// 17408 x 5120, 61 us, 98 % (with a lane's two stores 32 bytes apart 84).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_attend.h"
#include "kv_launch.h"
#include "mx4.cuh"
#include "mx4_launch.h"
#include "qmm_device.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Elements of a row that a lane takes: 32 bytes.  bfloat16 is bound by instructions as much as by memory, and what a block
// costs once (its scale, the maximum over its lanes) is then shared by two lanes rather than four.
template <bool BF16>
constexpr int per_lane() { return BF16 ? 16 : 8; }
template <bool BF16>
constexpr int chunk_of() { return 32 * per_lane<BF16>(); }     // of a warp
constexpr int kLoads = 2;                                      // of 16 bytes, a lane

struct Raw {
  uint4 a[kLoads];
};

template <bool BF16>
__device__ __forceinline__ Raw load(const void *x, int64_t at) {
  const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(x) + at * (BF16 ? 2 : 4));
  Raw r;
#pragma unroll
  for (int i = 0; i < kLoads; i++) r.a[i] = __ldcs(p + i);
  return r;
}

// A lane's words of codes, and the scale of its block (the same in all of the block's lanes).  The whole warp calls it.
template <bool BF16>
struct Codes {
  uint32_t w[per_lane<BF16>() / 8];
};
template <bool BF16>
__device__ __forceinline__ Codes<BF16> encode(const Raw &raw, uint32_t &scale) {
  constexpr int N = per_lane<BF16>();
  float v[N];
#pragma unroll
  for (int i = 0; i < kLoads; i++) {
    const uint32_t w[4] = {raw.a[i].x, raw.a[i].y, raw.a[i].z, raw.a[i].w};
#pragma unroll
    for (int j = 0; j < 4; j++)
      if constexpr (BF16) {
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        v[4 * i + j] = __uint_as_float(w[j]);
      }
  }
  float most = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i + 1 < N; i += 2) most = max3_nan(most, fabsf(v[i]), fabsf(v[i + 1]));
  uint32_t m = __float_as_uint(max3_nan(most, fabsf(v[N - 1]), 0.0f));
#pragma unroll
  for (int o = 1; o < kMxBlock / N; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));   // (not negative: bits order as values)
  const uint32_t top = (m >> 23) & 255;               // exponent field; 255: an infinity or a NaN is there
  scale = top == 255 ? 255 : top < 2 ? 0 : top - 2;
  const float inv = __uint_as_float((254 - scale) << 23);     // 2 ** (127 - scale)
  Codes<BF16> c;
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; j++) u[j] = v[i + j] * inv;
    c.w[i / 8] = mx4_encode(u);
  }
  return c;
}

// The four scales of a scale tile's row, in all lanes of its 128 elements.
template <bool BF16>
__device__ __forceinline__ uint32_t scale_word(uint32_t scale, int lane) {
  constexpr int LANES = kMxBlock / per_lane<BF16>();  // of a block
  uint32_t w = scale << (8 * ((lane / LANES) & 3));
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, LANES);
  return w | __shfl_xor_sync(0xFFFFFFFFu, w, 2 * LANES);
}
// Lanes of a scale tile's row.
template <bool BF16>
constexpr int tile_lanes() { return kMxTileK / per_lane<BF16>(); }

template <bool BF16>
__device__ __forceinline__ void put_codes(uint32_t *codes, int64_t at, const Codes<BF16> &c) {
  if constexpr (BF16)
    *reinterpret_cast<uint2 *>(codes + (at >> 3)) = make_uint2(c.w[0], c.w[1]);
  else
    codes[at >> 3] = c.w[0];
}

struct QuantParams {
  const void *x;
  int64_t x_matrix, x_row;
  const int32_t *places;
  uint32_t *codes;
  uint8_t *scales;
  int64_t rows, K, k_tiles;
  int64_t scale_bytes;                       // of a matrix
  int64_t k, out_rows;
  int sorted;                                // x has the places' rows, and an entry of them is a token
  uint32_t units;                            // warps' pieces of work: of
  Divisor chunks, lanes, row_tiles;          // chunks of a row, rows r % 32 of a tile that exist in some tile, tiles of a matrix
};

// A warp takes a chunk of the four rows r, r + 32, r + 64 and r + 96 of a tile: their scales are 16 bytes in a row of the
// scale tile, and 4 KB of loads are in flight a warp.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  uint32_t chunk = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (chunk >= p.units) return;
  uint32_t r32 = p.chunks.split(chunk), tile = p.lanes.split(r32);
  const int64_t matrix = p.row_tiles.split(tile);
  const int64_t row0 = (int64_t)tile * kMxRows + r32, col = (int64_t)chunk * chunk_of<BF16>() + per_lane<BF16>() * lane;
  if (row0 >= p.rows) return;
  const bool in = col < p.K;
  Raw raw[4];
#pragma unroll
  for (int g = 0; g < 4; g++) {
    raw[g] = Raw{};
    if (in && row0 + 32 * g < p.rows) raw[g] = load<BF16>(p.x, matrix * p.x_matrix + (row0 + 32 * g) * p.x_row + col);
  }
  uint32_t words[4];
#pragma unroll
  for (int g = 0; g < 4; g++) {
    uint32_t scale;
    const Codes<BF16> codes = encode<BF16>(raw[g], scale);
    words[g] = scale_word<BF16>(scale, lane);
    if (in && row0 + 32 * g < p.rows) put_codes<BF16>(p.codes, (matrix * p.rows + row0 + 32 * g) * p.K + col, codes);
  }
  constexpr int TL = tile_lanes<BF16>();
  const int64_t kt = (int64_t)chunk * (32 / TL) + lane / TL;
  if (lane % TL == 0 && kt < p.k_tiles)
    *reinterpret_cast<uint4 *>(p.scales + matrix * p.scale_bytes + mx4_scale_word(row0, kt, p.k_tiles)) =
        make_uint4(words[0], words[1], words[2], words[3]);
}

// A warp takes CHUNKS chunks of a token's row, and stores them to each of its places (sorted: the place's own row).
template <bool BF16, int CHUNKS>
__global__ void __launch_bounds__(kThreads) quantize_routed_kernel(const QuantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int CHUNK = chunk_of<BF16>(), TL = tile_lanes<BF16>();
  const int lane = threadIdx.x & 31;
  uint32_t chunk = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (chunk >= p.units) return;
  const int64_t t = p.chunks.split(chunk), col0 = (int64_t)chunk * (CHUNKS * CHUNK) + per_lane<BF16>() * lane;
  const int mine = lane < p.k ? p.places[t * p.k + lane] : -1;
  int64_t from = t;
  if (p.sorted) {
    from = __shfl_sync(0xFFFFFFFFu, mine, 0);
    if (from < 0 || from >= p.out_rows) return;
  }
  Raw raw[CHUNKS];
#pragma unroll
  for (int g = 0; g < CHUNKS; g++) {
    raw[g] = Raw{};
    if (col0 + g * CHUNK < p.K) raw[g] = load<BF16>(p.x, from * p.x_row + col0 + g * CHUNK);
  }
  Codes<BF16> codes[CHUNKS];
  uint32_t words[CHUNKS];
#pragma unroll
  for (int g = 0; g < CHUNKS; g++) {
    uint32_t scale;
    codes[g] = encode<BF16>(raw[g], scale);
    words[g] = scale_word<BF16>(scale, lane);
  }
  const int64_t kt0 = (int64_t)chunk * (CHUNKS * 32 / TL) + lane / TL;
  for (int j = 0; j < (int)p.k; j++) {
    const int64_t row = __shfl_sync(0xFFFFFFFFu, mine, j);
    if (row < 0 || row >= p.out_rows) continue;
    uint8_t *scales = p.scales + mx4_scale_word(row, kt0, p.k_tiles);
#pragma unroll
    for (int g = 0; g < CHUNKS; g++) {
      if (col0 + g * CHUNK < p.K) put_codes<BF16>(p.codes, row * p.K + col0 + g * CHUNK, codes[g]);
      if (lane % TL == 0 && kt0 + g * (32 / TL) < p.k_tiles)
        *reinterpret_cast<uint32_t *>(scales + g * (32 / TL) * kMxTileBytes) = words[g];
    }
  }
}

struct DequantParams {
  const uint32_t *codes;
  const uint8_t *scales;
  float *w;
  int64_t rows, k_tiles, scale_bytes;
  int64_t words, first;            // words of codes of all matrices; a launch's first row
  Divisor k8, per_matrix;          // words of a row; rows of a matrix
};

constexpr int kWordsAThread = 4;

// A thread takes words 256 apart; `first` rows come before the launch's.
__global__ void __launch_bounds__(kThreads) dequant_kernel(const DequantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t t0 = blockIdx.x * (kThreads * kWordsAThread) + threadIdx.x;
  uint32_t code[kWordsAThread], scale[kWordsAThread];
  const int64_t base = p.first * p.k8.d;
#pragma unroll
  for (int i = 0; i < kWordsAThread; i++) {
    uint32_t at = t0 + i * kThreads;
    code[i] = scale[i] = 0;
    if (base + at >= p.words) continue;
    code[i] = __ldcs(p.codes + base + at);
    uint32_t r = (uint32_t)p.first + p.k8.split(at);     // (at is then the word of its row)
    const int64_t matrix = p.per_matrix.split(r);
    const uint32_t block = at >> 2;
    scale[i] = p.scales[matrix * p.scale_bytes + mx4_scale_word(r, block >> 2, p.k_tiles) + (block & 3)];
  }
  // a store of the warp is 32 lanes' four values in a row: lane l's come from the word of lane 16 h + l / 2, its half l % 2
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kWordsAThread; i++) {
    const int64_t first = base + t0 - lane + i * kThreads;          // the warp's first word
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int from = 16 * h + (lane >> 1);
      const uint32_t word = __shfl_sync(0xFFFFFFFFu, code[i], from) >> (16 * (lane & 1));
      const float s = mx4_scale(__shfl_sync(0xFFFFFFFFu, scale[i], from));
      if (first + from >= p.words) continue;
      const float2 lo = mx4_pair(word & 255), hi = mx4_pair((word >> 8) & 255);
      __stcs(reinterpret_cast<float4 *>(p.w) + 2 * first + 32 * h + lane, make_float4(lo.x * s, lo.y * s, hi.x * s, hi.y * s));
    }
  }
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantArgs &a, cudaStream_t s) {
  QuantParams p{};
  p.x = a.x, p.x_matrix = a.x_matrix, p.x_row = a.x_row, p.places = a.places;
  p.codes = static_cast<uint32_t *>(a.codes), p.scales = static_cast<uint8_t *>(a.scales);
  p.rows = a.rows, p.K = a.K, p.k_tiles = mx4_k_tiles(a.K), p.scale_bytes = mx4_scales_bytes(a.rows, a.K);
  p.k = a.sorted ? 1 : a.k, p.out_rows = a.out_rows, p.sorted = a.sorted;
  int64_t units;
  const int chunk = a.bf16 ? chunk_of<true>() : chunk_of<false>();
  int chunks = a.bf16 ? 2 : 4;       // of a warp, of routed rows
  if (a.places) {
    // (fewer where a row has not so many, or where there are too few rows to occupy the SMs)
    const int64_t rows = a.sorted ? a.rows * a.k : a.rows;
    auto pieces = [&](int c) { return (a.K + c * chunk - 1) / (c * chunk); };
    while (chunks > 1 && (rows * pieces(chunks) < 16 * kv_sms() || pieces(chunks / 2) == 1)) chunks /= 2;
    p.chunks = Divisor((uint32_t)pieces(chunks));
    units = rows * p.chunks.d;
  } else {
    p.chunks = Divisor((uint32_t)((a.K + chunk - 1) / chunk));
    p.lanes = Divisor(a.rows < 32 ? (uint32_t)a.rows : 32);
    p.row_tiles = Divisor((uint32_t)((a.rows + kMxRows - 1) / kMxRows));
    units = a.matrices * p.row_tiles.d * p.lanes.d * p.chunks.d;
  }
  if (units > 0x7FFFFFFF) return cudaErrorInvalidValue;      // (more than a TB of codes)
  p.units = (uint32_t)units;
  const int64_t grid = (units + kWarps - 1) / kWarps;
  auto kern = a.bf16 ? quantize_kernel<true> : quantize_kernel<false>;
  if (a.places && a.bf16) kern = chunks == 2 ? quantize_routed_kernel<true, 2> : quantize_routed_kernel<true, 1>;
  if (a.places && !a.bf16)
    kern = chunks == 4 ? quantize_routed_kernel<false, 4> : chunks == 2 ? quantize_routed_kernel<false, 2> : quantize_routed_kernel<false, 1>;
  return launch_after(kern, grid, kThreads, 0, s, p);
}

cudaError_t launch_mx4_dequant(const void *codes, const void *scales, float *w, int64_t matrices, int64_t rows, int64_t K,
                               cudaStream_t s) {
  DequantParams p{};
  p.codes = static_cast<const uint32_t *>(codes), p.scales = static_cast<const uint8_t *>(scales), p.w = w;
  p.rows = rows, p.words = matrices * rows * (K / 8);
  p.k8 = Divisor((uint32_t)(K / 8)), p.per_matrix = Divisor((uint32_t)rows);
  p.k_tiles = mx4_k_tiles(K), p.scale_bytes = mx4_scales_bytes(rows, K);
  // rows whose words are counted in 31 bits, a launch
  constexpr int64_t BLOCK = kThreads * kWordsAThread;
  const int64_t most = (0x7FFFFFFF - BLOCK) / (K / 8);
  for (; p.first < matrices * rows; p.first += most) {
    const int64_t left = matrices * rows - p.first, words = (left < most ? left : most) * (K / 8);
    DequantParams q = p;
    q.words = p.first * (K / 8) + words;
    const cudaError_t e = launch_after(dequant_kernel, (words + BLOCK - 1) / BLOCK, kThreads, 0, s, q);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qmm
