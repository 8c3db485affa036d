// mx4_layout.h -- sizes of the microscaled format's scale tiles, quotients by sizes, and what a CTA of its product holds in
// shared memory.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace qmm {

constexpr int kMxBlock = 32;        // elements that share a scale
constexpr int kMxRows = 128;        // rows of a scale tile
constexpr int kMxTileK = 128;       // elements of a row in a scale tile
constexpr int kMxTileBytes = 512;

__host__ __device__ inline int64_t mx4_k_tiles(int64_t K) { return (K + kMxTileK - 1) / kMxTileK; }
__host__ __device__ inline int64_t mx4_scales_bytes(int64_t rows, int64_t K) {
  return (rows + kMxRows - 1) / kMxRows * mx4_k_tiles(K) * kMxTileBytes;
}

// Quotients of whole numbers below 2^31 by a divisor known to the host, as a product's upper half (a 64-bit division is some
// hundred instructions, more than all else that these kernels do for a word).  Granlund and Montgomery, "Division by invariant
// integers using multiplication" (1994): m = floor(2^32 (2^s - d) / d) + 1 with s the least of 2^s >= d.
struct Divisor {
  uint32_t d = 1, m = 1, s = 0;
  Divisor() = default;
  explicit Divisor(uint32_t by) : d(by) {
    while (((uint64_t)1 << s) < by) s++;
    m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - by)) / by + 1);
  }
  __host__ __device__ __forceinline__ uint32_t quotient(uint32_t n) const {
    return (uint32_t)(((((uint64_t)m * n) >> 32) + n) >> s);
  }
  // n becomes the remainder
  __host__ __device__ __forceinline__ uint32_t split(uint32_t &n) const {
    const uint32_t q = quotient(n);
    n -= q * d;
    return q;
  }
};

namespace mx4 {                            // of the product (mx4_gemm.cu)

constexpr int BM = 128;                    // weight rows of a tile
constexpr int BK = 256;                    // elements of a stage: 128 bytes of a row, one swizzle atom wide
constexpr int MAX_STAGES = 8;
constexpr int MAX_SPLIT = 8;
// Shared memory: what one CTA may have, and what each of two on an SM may, which has 228 KB and keeps 1 KB of it a CTA.
constexpr int SMEM_LIMIT = 227 * 1024, SMEM_OF_TWO = 228 * 1024 / 2 - 1024;

// One piece of work: a weight tile and a token tile.
struct alignas(16) Item {
  int n0;                                  // first row of the weight tile (a pair's: of its first CTA's)
  int row;                                 // first row of the token tile in x and y
  int rows;                                // tokens of it
  int expert;
};
constexpr int LISTED = 32;                 // items of a CTA that are found before it begins

struct Layout {                            // of a CTA's shared memory
  int a, b, sfa, sfb, stage;               // bytes: weights, tokens, scales, all
  int ring, red, list, bars, total;
};
__host__ __device__ inline Layout layout(bool gated, int ts, int ctas, int stages, int split, int experts) {
  Layout l;
  const int two = gated ? 2 : 1;
  l.a = two * BM * (BK / 2);
  l.b = ts / ctas * (BK / 2);
  l.sfa = two * 2 * kMxTileBytes;
  l.sfb = (ts > kMxRows ? 2 : 1) * 2 * kMxTileBytes;
  l.stage = l.a + l.b + l.sfa + l.sfb;     // (multiples of 1024 bytes)
  l.ring = stages * l.stage;
  l.red = split > 1 ? two * ts * BM * 4 : 0;
  l.list = LISTED * (int)sizeof(Item) + (3 * experts + 1) * 4;     // items; starts, counts, and token tiles before
  l.list = (l.list + 15) & ~15;
  l.bars = 8 * (2 * MAX_STAGES + 4 + 2) + 16 + 4 * MAX_SPLIT;
  l.total = l.ring + l.red + l.list + l.bars + 1024;   // (1024: the ring begins at a multiple of it)
  return l;
}

// Depth of the ring in what such a CTA may have.
inline int ring_stages(bool gated, int ts, int ctas, int split, int experts, bool two_an_sm) {
  const Layout l = layout(gated, ts, ctas, 0, split, experts);
  const int n = ((two_an_sm ? SMEM_OF_TWO : SMEM_LIMIT) - l.total) / l.stage;
  return n < MAX_STAGES ? n : MAX_STAGES;
}

}  // namespace mx4
}  // namespace qmm
