// kv_attend.cu -- softmax attention of a step's queries over the 4-bit cache:
//
//   out[i] = sum_j p_j v_j,   p = softmax_j(scale * q_i . k_j)
//
// over the cached tokens j that query i may see (causal, optional window).
// One CTA per (query token, head): scores of 128 tokens at a time, one token a
// thread, with a running maximum and sum; then one thread per output element.
#include <cuda_bf16.h>

#include "kv_attend.h"
#include "kv_layout.cuh"
#include "qmm_device.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 128;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) attend_kernel(const KvAttendArgs p, const KvGeom g) {
  __shared__ float qs[256], sc[kThreads], red[kThreads / 32];
  __shared__ int slot_s[kThreads];
  const int t = blockIdx.x, h = blockIdx.y, kvh = h / (p.heads / g.kv_heads);
  int b = t, i = 0, n = 1;
  if (p.cu) {
    int lo = 0, hi = (int)p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    b = lo;
    if (t < p.cu[b] || t >= p.cu[b + 1]) return;
    i = t - p.cu[b];
    n = p.cu[b + 1] - p.cu[b];
  }
  const int len = max(0, p.lens[b]);
  const int64_t pos = (int64_t)len - n + i;
  const int64_t most = min((int64_t)len, p.max_blocks << g.lg_page);
  const int hi = (int)max((int64_t)0, min(most, pos + 1));
  const int lo = p.window > 0 ? (int)max((int64_t)0, pos + 1 - p.window) : 0;
  const int tid = threadIdx.x;
  for (int d = tid; d < g.D; d += kThreads) {
    const int64_t at = t * p.q_token + h * p.q_head + d;
    qs[d] = (BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[at]) : static_cast<const float *>(p.q)[at]) *
            (p.scale * 1.44269504088896340736f);
  }
  float m = __int_as_float(0xFF800000), l = 0.0f, acc[2] = {0.0f, 0.0f};
  const uint8_t *cache = static_cast<const uint8_t *>(p.cache);
  for (int j0 = lo; j0 < hi; j0 += kThreads) {
    __syncthreads();
    const int j = j0 + tid;
    float s = __int_as_float(0xFF800000);
    int slot = -1;
    if (j < hi) {
      const int page = p.table[b * p.max_blocks + (j >> g.lg_page)];
      if (page >= 0 && page < g.pages) slot = (page << g.lg_page) + (j & (g.page - 1));
    }
    if (slot >= 0) {
      const uint8_t *tile = cache + kv_tile_at(g, slot, kvh);
      const int row = kv_row(slot & 15);
      s = 0.0f;
      for (int mm = 0; mm < g.D / 8; mm++) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(tile + kv_k_word(g.D, row, mm));
        const uint32_t c = *reinterpret_cast<const uint32_t *>(tile + kv_k_coef(g, row, 8 * mm / g.group));
        const float sk = h2f((uint16_t)c), bk = h2f((uint16_t)(c >> 16));
        for (int e = 0; e < 8; e++) s += qs[8 * mm + e] * (sk * (float)((w >> (4 * e)) & 15u) + bk);
      }
    }
    float mx = s;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float mu = mn == __int_as_float(0xFF800000) ? 0.0f : mn;
    const float alpha = exp2f(m - mu);
    m = mn;
    sc[tid] = exp2f(s - mu);
    slot_s[tid] = slot;
    __syncthreads();
    l *= alpha;
    acc[0] *= alpha, acc[1] *= alpha;
    for (int u = 0; u < kThreads && j0 + u < hi; u++) {
      const int sl = slot_s[u];
      if (sl < 0) continue;
      const float pr = sc[u];
      l += pr;
      const uint8_t *tile = cache + kv_tile_at(g, sl, kvh);
      for (int e = 0; e < 2; e++) {
        const int d = tid + e * kThreads;
        if (d >= g.D) break;
        const int jj = sl & 15;
        const uint32_t by = tile[kv_v_word(g.D, d & ~8, jj >> 2) + (jj & 3)];
        const uint32_t c = *reinterpret_cast<const uint32_t *>(tile + kv_v_coef(g, kv_row(jj), d / g.group));
        acc[e] += pr * (h2f((uint16_t)c) * (float)((by >> ((d & 8) >> 1)) & 15u) + h2f((uint16_t)(c >> 16)));
      }
    }
  }
  for (int e = 0; e < 2; e++) {
    const int d = tid + e * kThreads;
    if (d >= g.D) break;
    const float o = l == 0.0f ? 0.0f : acc[e] / l;
    const int64_t at = ((int64_t)t * p.heads + h) * g.D + d;
    if (BF16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16(o);
    else static_cast<float *>(p.out)[at] = o;
  }
}

}  // namespace

size_t kv_attend_workspace(int64_t, int64_t, int64_t, int64_t, int64_t) { return 16; }

cudaError_t launch_kv_attend(const KvAttendArgs &a, cudaStream_t s) {
  const KvGeom g = kv_geom(a.pages, a.kv_heads, a.head_dim, a.page, a.group);
  const dim3 grid((unsigned)a.tokens, (unsigned)a.heads);
  if (a.bf16) attend_kernel<true><<<grid, kThreads, 0, s>>>(a, g);
  else attend_kernel<false><<<grid, kThreads, 0, s>>>(a, g);
  return cudaGetLastError();
}

}  // namespace qmm
