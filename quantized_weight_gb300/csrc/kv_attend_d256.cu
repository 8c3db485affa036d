// kv_attend_d256.cu -- the warp-level attention kernels for heads of 256 elements.
#include "kv_attend_warp.cuh"

namespace qmm {

cudaError_t launch_kv_warp_d256(const KvAttendArgs &a, cudaStream_t s) {
  const int G = 256 / a.group;
  if (G == 8) return a.bf16 ? kvw::launch<256, 8, 1, false>(a, s) : kvw::launch<256, 8, 1, true>(a, s);
  if (G == 4) return a.bf16 ? kvw::launch<256, 4, 1, false>(a, s) : kvw::launch<256, 4, 1, true>(a, s);
  if (G == 2) return a.bf16 ? kvw::launch<256, 2, 1, false>(a, s) : kvw::launch<256, 2, 1, true>(a, s);
  return cudaErrorNotSupported;
}

}  // namespace qmm
