// kv_attend.cu -- attention over the 4-bit cache: which kernel takes a call.
#include "kv_attend.h"

namespace qmm {

size_t kv_attend_workspace(int64_t, int64_t, int64_t, int64_t head_dim, int64_t) {
  // counters, then two partial results a team: 8 rows for each of 3 teams an SM, or 16 of 2, with maxima and sums
  return 4 * 1024 + (size_t)kv_max_ctas(2) * 2 * 16 * (size_t)(head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attend(const KvAttendArgs &a, cudaStream_t s) {
  const int64_t rows = a.max_fresh * (a.heads / a.kv_heads);
  if (a.bf16 && rows > 64) return launch_kv_prefill(a, s);
  const int nt = rows <= 8 ? 1 : 2;
  if (a.head_dim == 64) return launch_kv_warp_d64(a, nt, s);
  if (a.head_dim == 128) return launch_kv_warp_d128(a, nt, s);
  if (a.head_dim == 256) return launch_kv_warp_d256(a, s);
  return cudaErrorNotSupported;
}

}  // namespace qmm
