// kv_layout.cuh -- the byte layout of the 4-bit key/value cache, shared by the
// kernels that write it (append), read it back (read) and attend over it.
//
// The cache of one layer is [pages][kv_heads][page / 16] tiles of 16 tokens.
// Keeping a head's tiles of a page together makes a page one contiguous run
// per head, and a tile is a multiple of 16 bytes, so that it is copied in
// 16-byte pieces.  A tile is
//
//   K codes   8 * D bytes   32-bit words [max(1, D/128)][row 16][t 4][WC], WC = min(4, D/32):
//                           nibble i of word w' of chunk c is element 32 (WC c + w') + 8t + i of the row's token
//   V codes   8 * D bytes   32-bit words [D/64][g 8][t 4][w' 4]: byte r is token 4t + r; its low nibble
//                           is element d = 16 (4c + w') + g, its high nibble element d + 8
//   K coefs  64 * G bytes   [row 16][group][scale, bias] binary16, G = D / group
//   V coefs  64 * G bytes   the same
//
// with token j of the tile in row 8 (j % 2) + 2 (j / 4) + (j / 2) % 2.
//
// Both code areas are in the order in which lane 4g + t of a warp feeds
// mma.sync.m16n8k16 A fragments.  Four ANDs and a shift turn a word into the four
// operand registers of exact binary16 integers (nibbles at bits 0..3 and 4..7
// of each half).  For keys (A = token rows x elements) lane (g, t) takes rows
// g and g + 8; a word's 32 elements over t lie inside one group of any size
// >= 32.  For values (A = elements x tokens) the two halves of a masked word
// are tokens (4t, 4t + 2), and of the shifted word tokens (4t + 1, 4t + 3),
// so a byte never holds codes of two tokens: appending a token writes whole
// bytes and never reads one.  The row order above puts token 4t + {0, 2} in rows 2t
// and 2t + 1, and 4t + {1, 3} in rows 8 + 2t and 9 + 2t: the score tile of the
// key product, transposed, is then the B operand of the value product as it stands.
#pragma once
#include <cstdint>

namespace qmm {

constexpr int kKvTile = 16;   // tokens per tile

struct KvGeom {
  int D, group, G;            // head dimension, group, groups per head
  int lg_group8;              // log2 of a group's eights
  int page, lg_page;          // tokens per page (a power of two, >= 16)
  int tile_bytes, head_bytes; // one tile; one head's tiles of a page
  int kv_heads;
  int64_t pages;
};

__host__ __device__ __forceinline__ int kv_tile_bytes(int D, int group) { return 16 * D + 128 * (D / group); }

inline KvGeom kv_geom(int64_t pages, int64_t kv_heads, int64_t D, int page, int group) {
  KvGeom g{};
  g.D = (int)D;
  g.group = group;
  g.G = (int)D / group;
  g.lg_group8 = __builtin_ctz((unsigned)group) - 3;
  g.page = page;
  g.lg_page = __builtin_ctz((unsigned)page);
  g.tile_bytes = kv_tile_bytes(g.D, group);
  g.head_bytes = page / kKvTile * g.tile_bytes;
  g.kv_heads = (int)kv_heads;
  g.pages = pages;
  return g;
}

__device__ __forceinline__ int kv_row(int j) { return 8 * (j & 1) + 2 * (j >> 2) + ((j >> 1) & 1); }

// Byte offset of the tile that holds slot `slot` of head `h` (64 bits: a cache may exceed 4 GB).
__device__ __forceinline__ int64_t kv_tile_at(const KvGeom &g, int slot, int h) {
  const int pg = slot >> g.lg_page, off = slot & (g.page - 1);
  return ((int64_t)pg * g.kv_heads + h) * g.head_bytes + (off >> 4) * g.tile_bytes;
}

// Byte offset inside a tile of the K word with elements 8m .. 8m + 7 of row `row`.
__device__ __forceinline__ int kv_k_word(int D, int row, int m) {
  const int wc = D >= 128 ? 4 : D >> 5, w = m >> 2;
  return (((w / wc * 16 + row) * 4 + (m & 3)) * wc + w % wc) * 4;
}
// Byte offset inside a tile of the V word with elements (d, d + 8), d % 16 < 8, of tokens 4t .. 4t + 3.
__device__ __forceinline__ int kv_v_word(int D, int d, int t) {
  return 8 * D + (((d >> 6) * 8 + (d & 7)) * 4 + t) * 16 + ((d >> 4) & 3) * 4;
}
__device__ __forceinline__ int kv_k_coef(const KvGeom &g, int row, int grp) { return 16 * g.D + (row * g.G + grp) * 4; }
__device__ __forceinline__ int kv_v_coef(const KvGeom &g, int row, int grp) { return kv_k_coef(g, row, grp) + 64 * g.G; }

}  // namespace qmm
