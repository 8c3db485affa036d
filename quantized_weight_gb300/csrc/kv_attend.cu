// kv_attend.cu -- attention over the 4-bit cache: which kernel takes a call.
#include "kv_attend.h"

namespace qmm {

size_t kv_attend_workspace(int64_t, int64_t, int64_t, int64_t head_dim, int64_t) {
  // Counters, then two partial results for each of two teams an SM: 16 rows (heads of 256: 8) with maxima and sums.  One size
  // for all calls of a head dimension, since a few MB matter less than a buffer that the next call finds too small.
  return 4 * kKvMaxCtas + (size_t)kv_max_ctas(2) * 2 * (head_dim == 256 ? 8 : 16) * (size_t)(head_dim + 2) * sizeof(float);
}

// The prompt kernel takes 2.6 us for a block of 128 keys and two tiles of 128 rows, 2.0 us with one tile (heads of 256:
// 1.3 us, 64 keys, one tile), with an item on one SM; the warp kernel spreads any work over all SMs, at 0.39 ns a row and
// 128 keys (0.43 ns, 64 keys).  So the prompt kernel pays from so many rows on for each round of its items over
// the SMs.  Measured, prompt / warp kernel in us, 8 kv heads of 128: 2048 rows, 8000 keys 146 / 60; 8192 rows, 4000
// keys 82 / 112; 16384 rows, 4000 keys 82 / 201; 128 items of 32 rows, 4000 keys 63 / 65; 512 items of 20 rows, 2000 keys
// 134 / 117, of 64 rows 137 / 225.  Heads of 64: 32 items of 256 rows, 4000 keys 71 / 78.  Heads of 256: 64 items of 128
// rows, 4000 keys 85 / 223; 512 items of 20 rows, 2000 keys 198 / 185.
// (Requests of equal length and equal queries; the rule sees no more of a ragged or mixed step than max_fresh.)
bool kv_attend_tiles(bool bf16, int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_fresh) {
  const int64_t rows = max_fresh * (heads / kv_heads);         // of q, a request and kv head
  if (!bf16 || rows <= 16) return false;
  const int64_t per = head_dim == 256 ? 128 : 256, items = B * kv_heads * ((rows + per - 1) / per);
  const int64_t rounds = (items + kv_max_ctas(1) - 1) / kv_max_ctas(1);
  const int64_t border = head_dim == 256 ? 3200 : head_dim == 128 ? (rows > 128 ? 6200 : 3900) : rows > 128 ? 8000 : 4500;
  return B * kv_heads * rows > border * rounds;
}

cudaError_t launch_kv_attend(const KvAttendArgs &a, cudaStream_t s) {
  if (kv_attend_tiles(a.bf16 != 0, a.B, a.heads, a.kv_heads, a.head_dim, a.max_fresh)) return launch_kv_prefill(a, s);
  const int64_t rows = a.max_fresh * (a.heads / a.kv_heads);
  const int nt = rows <= 8 ? 1 : 2;
  if (a.head_dim == 64) return launch_kv_warp_d64(a, nt, s);
  if (a.head_dim == 128) return launch_kv_warp_d128(a, nt, s);
  if (a.head_dim == 256) return launch_kv_warp_d256(a, s);
  return cudaErrorNotSupported;
}

}  // namespace qmm
