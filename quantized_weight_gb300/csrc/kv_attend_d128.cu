// kv_attend_d128.cu -- the warp-level attention kernels for heads of 128 elements.
#include "kv_attend_warp.cuh"

namespace qmm {

cudaError_t launch_kv_warp_d128(const KvAttendArgs &a, int nt, cudaStream_t s) {
  const int G = 128 / a.group;
  if (G == 4)
    return a.bf16 ? (nt == 1 ? kvw::launch<128, 4, 1, false>(a, s) : kvw::launch<128, 4, 2, false>(a, s))
                  : (nt == 1 ? kvw::launch<128, 4, 1, true>(a, s) : kvw::launch<128, 4, 2, true>(a, s));
  if (G == 2)
    return a.bf16 ? (nt == 1 ? kvw::launch<128, 2, 1, false>(a, s) : kvw::launch<128, 2, 2, false>(a, s))
                  : (nt == 1 ? kvw::launch<128, 2, 1, true>(a, s) : kvw::launch<128, 2, 2, true>(a, s));
  if (G == 1)
    return a.bf16 ? (nt == 1 ? kvw::launch<128, 1, 1, false>(a, s) : kvw::launch<128, 1, 2, false>(a, s))
                  : (nt == 1 ? kvw::launch<128, 1, 1, true>(a, s) : kvw::launch<128, 1, 2, true>(a, s));
  return cudaErrorNotSupported;
}

}  // namespace qmm
