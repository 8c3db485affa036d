// kv_attend_d64.cu -- the warp-level attention kernels for heads of 64 elements.
#include "kv_attend_warp.cuh"

namespace qmm {

cudaError_t launch_kv_warp_d64(const KvAttendArgs &a, int nt, cudaStream_t s) {
  const int G = 64 / a.group;
  if (G == 2)
    return a.bf16 ? (nt == 1 ? kvw::launch<64, 2, 1, false>(a, s) : kvw::launch<64, 2, 2, false>(a, s))
                  : (nt == 1 ? kvw::launch<64, 2, 1, true>(a, s) : kvw::launch<64, 2, 2, true>(a, s));
  if (G == 1)
    return a.bf16 ? (nt == 1 ? kvw::launch<64, 1, 1, false>(a, s) : kvw::launch<64, 1, 2, false>(a, s))
                  : (nt == 1 ? kvw::launch<64, 1, 1, true>(a, s) : kvw::launch<64, 1, 2, true>(a, s));
  return cudaErrorNotSupported;
}

}  // namespace qmm
