// kv_attend.h -- arguments of the attention over the 4-bit cache, between the
// C ABI (api.cu, which has validated them) and the kernels.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace qmm {

struct KvAttendArgs {
  const void *q;                        // [tokens, heads, head_dim], strided
  void *out;                            // [tokens, heads, head_dim], contiguous, q's type
  const void *cache;
  const int32_t *table;                 // [B, max_blocks]
  const int32_t *lens;                  // [B]
  const int32_t *cu;                    // [B + 1], or null: query b is request b's only one
  void *workspace;
  int64_t q_token, q_head;              // strides in elements
  int64_t tokens, B, max_blocks, max_fresh;
  int64_t pages, kv_heads, head_dim, heads;
  int page, group;
  int bf16;                             // q and out: bfloat16, else float32
  float scale;
  int64_t window;                       // 0: none
};

// SMs of the current device, asked once a device.  Without one (sizes can be asked for anywhere): a GB300's, not kept.
constexpr int kKvMaxDevices = 64;
inline int kv_sms() {
  static std::atomic<int> known[kKvMaxDevices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    const bool keep = dev >= 0 && dev < kKvMaxDevices;
    if (keep && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0) {
      if (keep) known[dev].store(n, std::memory_order_relaxed);
      return n;
    }
  }
  (void)cudaGetLastError();
  return 152;
}

// CTAs of a launch with `per_sm` CTAs an SM: at most 1024 (their counters are the workspace's first 4096 bytes).
constexpr int kKvMaxCtas = 1024;
inline int kv_max_ctas(int per_sm) {
  const int n = kv_sms() * per_sm;
  return n > kKvMaxCtas ? kKvMaxCtas : n;
}

size_t kv_attend_workspace(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_fresh);
// Whether a call takes the prompt kernel, tiles of 128 rows of q.
bool kv_attend_tiles(bool bf16, int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_fresh);
cudaError_t launch_kv_attend(const KvAttendArgs &a, cudaStream_t s);

// Many queries a request, bfloat16 (kv_prefill.cu); its waits are bounded and report here.
cudaError_t launch_kv_prefill(const KvAttendArgs &a, cudaStream_t s);
cudaError_t read_clear_kv_status(int *status, cudaStream_t s);
void set_kv_test_wait(unsigned long long limit_ns);

// Per head dimension (one translation unit each); nt: tiles of 8 rows of q an item
// (heads of 256: one, since registers and shared memory hold no more).
cudaError_t launch_kv_warp_d64(const KvAttendArgs &a, int nt, cudaStream_t s);
cudaError_t launch_kv_warp_d128(const KvAttendArgs &a, int nt, cudaStream_t s);
cudaError_t launch_kv_warp_d256(const KvAttendArgs &a, cudaStream_t s);

}  // namespace qmm
