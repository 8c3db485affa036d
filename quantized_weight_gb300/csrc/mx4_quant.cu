// mx4_quant.cu -- rows to microscaled 4-bit codes and back (format in mx4.cuh).
//
// A block's scale is the power of two 2 ** (floor(log2(max |x|)) - 2), so its largest value lies between 4 and 8 of it and
// the codes reach 6: the exponent field of max |x| less 2, no arithmetic.  x times the inverse power is exact in float32
// (or far below the first border), so the codes are the nearest ones to the exact quotient, halves to the even code.
//
// All three kernels are bound by memory: a value is read once (2 or 4 bytes) and leaves as 17/32 of a byte.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_launch.h"
#include "mx4.cuh"
#include "mx4_launch.h"
#include "qmm_device.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 256;         // elements that a warp takes at once: 8 a lane, 4 lanes a block, 2 scale tiles

// A lane's 8 elements.
struct Eight {
  float v[8];
};

template <bool BF16>
struct Raw {
  uint4 a, b;                       // b: float32 only
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load8(const void *x, int64_t at) {
  Raw<BF16> r{};
  if constexpr (BF16) {
    r.a = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + at));
  } else {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(x) + at);
    r.a = __ldcs(p);
    r.b = __ldcs(p + 1);
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ Eight widen(const Raw<BF16> &r) {
  Eight e;
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; i++)
    e.v[i] = BF16 ? __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16) : __uint_as_float(w[i]);
  return e;
}

// A lane's word of codes, and the scale of its block (the same in its 4 lanes).  The whole warp calls it.
__device__ __forceinline__ uint32_t encode8(const Eight &e, uint32_t &scale) {
  const float a = max3_nan(max3_nan(fabsf(e.v[0]), fabsf(e.v[1]), fabsf(e.v[2])), fabsf(e.v[3]), fabsf(e.v[4]));
  uint32_t m = __float_as_uint(max3_nan(max3_nan(a, fabsf(e.v[5]), fabsf(e.v[6])), fabsf(e.v[7]), 0.0f));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));     // (of values that are not negative, the bits order as they do)
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  const uint32_t top = (m >> 23) & 255;               // exponent field; 255: an infinity or a NaN is there
  scale = top == 255 ? 255 : top < 2 ? 0 : top - 2;
  const float inv = __uint_as_float((254 - min(scale, 253u)) << 23);      // 2 ** (127 - scale)
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = e.v[i] * inv;
  return mx4_encode(v);
}

// The four scales of a scale tile's row, in lanes 0..15 those of the first tile of a chunk, in 16..31 the second's.
__device__ __forceinline__ uint32_t scale_word(uint32_t scale, int lane) {
  uint32_t w = scale << (8 * ((lane >> 2) & 3));
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
  return w | __shfl_xor_sync(0xFFFFFFFFu, w, 8);
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

// A warp takes a chunk (of bfloat16, two) of the four rows r, r + 32, r + 64 and r + 96 of a tile: their scales are 16 bytes
// in a row of the scale tile, and 4 KB of loads are in flight a warp.
template <bool BF16>
constexpr int chunks_a_warp() { return BF16 ? 2 : 1; }

template <bool BF16>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  uint32_t chunk = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (chunk >= p.units) return;
  uint32_t r32 = p.chunks.split(chunk), tile = p.lanes.split(r32);
  const int64_t matrix = p.row_tiles.split(tile);
  constexpr int CHUNKS = chunks_a_warp<BF16>();
  const int64_t row0 = (int64_t)tile * kMxRows + r32, col0 = (int64_t)chunk * (CHUNKS * kChunk) + 8 * lane;
  if (row0 >= p.rows) return;
  Raw<BF16> raw[CHUNKS][4];
#pragma unroll
  for (int c = 0; c < CHUNKS; c++)
#pragma unroll
    for (int g = 0; g < 4; g++) {
      raw[c][g] = Raw<BF16>{};
      if (col0 + c * kChunk < p.K && row0 + 32 * g < p.rows)
        raw[c][g] = load8<BF16>(p.x, matrix * p.x_matrix + (row0 + 32 * g) * p.x_row + col0 + c * kChunk);
    }
#pragma unroll
  for (int c = 0; c < CHUNKS; c++) {
    uint32_t words[4];
    const int64_t col = col0 + c * kChunk;
#pragma unroll
    for (int g = 0; g < 4; g++) {
      uint32_t scale;
      const uint32_t code = encode8(widen(raw[c][g]), scale);
      words[g] = scale_word(scale, lane);
      if (col < p.K && row0 + 32 * g < p.rows) p.codes[((matrix * p.rows + row0 + 32 * g) * p.K + col) >> 3] = code;
    }
    const int64_t kt = ((int64_t)chunk * CHUNKS + c) * 2 + (lane >> 4);
    if ((lane & 15) == 0 && kt < p.k_tiles)
      *reinterpret_cast<uint4 *>(p.scales + matrix * p.scale_bytes + mx4_scale_word(row0, kt, p.k_tiles)) =
          make_uint4(words[0], words[1], words[2], words[3]);
  }
}

// A warp takes up to 4 chunks of a token's row, and stores them to each of its places (sorted: the place's own row).
template <bool BF16>
__global__ void __launch_bounds__(kThreads) quantize_routed_kernel(const QuantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  uint32_t chunk = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (chunk >= p.units) return;
  const int64_t t = p.chunks.split(chunk), col0 = (int64_t)chunk * (4 * kChunk) + 8 * lane;
  const int mine = lane < p.k ? p.places[t * p.k + lane] : -1;
  int64_t from = t;
  if (p.sorted) {
    from = __shfl_sync(0xFFFFFFFFu, mine, 0);
    if (from < 0 || from >= p.out_rows) return;
  }
  Raw<BF16> raw[4];
#pragma unroll
  for (int g = 0; g < 4; g++) {
    raw[g] = Raw<BF16>{};
    if (col0 + g * kChunk < p.K) raw[g] = load8<BF16>(p.x, from * p.x_row + col0 + g * kChunk);
  }
  uint32_t codes[4], words[4];
#pragma unroll
  for (int g = 0; g < 4; g++) {
    uint32_t scale;
    codes[g] = encode8(widen(raw[g]), scale);
    words[g] = scale_word(scale, lane);
  }
  for (int j = 0; j < (int)p.k; j++) {
    const int64_t row = __shfl_sync(0xFFFFFFFFu, mine, j);
    if (row < 0 || row >= p.out_rows) continue;
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int64_t col = col0 + g * kChunk, kt = (col - 8 * lane) / kMxTileK + (lane >> 4);
      if (col < p.K) p.codes[(row * p.K + col) >> 3] = codes[g];
      if ((lane & 15) == 0 && kt < p.k_tiles)
        *reinterpret_cast<uint32_t *>(p.scales + mx4_scale_word(row, kt, p.k_tiles)) = words[g];
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
  if (a.places) {
    p.chunks = Divisor((uint32_t)((a.K + 4 * kChunk - 1) / (4 * kChunk)));
    units = (a.sorted ? a.rows * a.k : a.rows) * p.chunks.d;
  } else {
    const int each = kChunk * (a.bf16 ? chunks_a_warp<true>() : chunks_a_warp<false>());
    p.chunks = Divisor((uint32_t)((a.K + each - 1) / each));
    p.lanes = Divisor(a.rows < 32 ? (uint32_t)a.rows : 32);
    p.row_tiles = Divisor((uint32_t)((a.rows + kMxRows - 1) / kMxRows));
    units = a.matrices * p.row_tiles.d * p.lanes.d * p.chunks.d;
  }
  if (units > 0x7FFFFFFF) return cudaErrorInvalidValue;      // (more than a TB of codes)
  p.units = (uint32_t)units;
  const int64_t grid = (units + kWarps - 1) / kWarps;
  auto kern = a.places ? (a.bf16 ? quantize_routed_kernel<true> : quantize_routed_kernel<false>)
                       : (a.bf16 ? quantize_kernel<true> : quantize_kernel<false>);
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
