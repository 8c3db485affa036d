// kv_attend.cu -- attention over the 4-bit cache: which kernel takes a call.
#include "kv_attend.h"

namespace qmm {

size_t kv_attend_workspace(int64_t, int64_t, int64_t, int64_t head_dim, int64_t) {
  // counters, then two partial results a team: 8 rows for each of 3 teams an SM, or 16 of 2, with maxima and sums
  return 4 * 1024 + (size_t)kv_max_ctas(2) * 2 * 16 * (size_t)(head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attend(const KvAttendArgs &a, cudaStream_t s) {
  const int64_t rows = a.max_fresh * (a.heads / a.kv_heads);   // of q, a request and kv head
  if (a.bf16) {
    // A block of 128 keys takes the prompt kernel 2.7 us for up to 256 rows of an item, which stays on one SM; the
    // warp kernel takes 1.7 us for 16 rows, but spreads any work over all SMs.  So the prompt kernel pays from about
    // 4000 rows on for each round of items over the SMs (4096 tokens, 32 / 8 heads of 128: 180 against 1448 us; one
    // request of 160 rows would be 16 times slower on it).  Heads of 256 have the same border within 10 %.
    const int64_t per = a.head_dim == 256 ? 128 : 256, items = a.B * a.kv_heads * ((rows + per - 1) / per);
    const int64_t rounds = (items + kv_max_ctas(1) - 1) / kv_max_ctas(1);
    if (a.B * a.kv_heads * rows > 4000 * rounds && rows > 16) return launch_kv_prefill(a, s);
  }
  const int nt = rows <= 8 ? 1 : 2;
  if (a.head_dim == 64) return launch_kv_warp_d64(a, nt, s);
  if (a.head_dim == 128) return launch_kv_warp_d128(a, nt, s);
  if (a.head_dim == 256) return launch_kv_warp_d256(a, s);
  return cudaErrorNotSupported;
}

}  // namespace qmm
