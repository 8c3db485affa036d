// mx4_gemm.cu -- y = x * w^T of two microscaled 4-bit matrices, for one matrix w or for the rows of each expert.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_launch.h"
#include "mx4.cuh"
#include "mx4_launch.h"
#include "qmm_device.cuh"

namespace qmm {

__device__ int g_mx4_status = 0;

namespace {

struct Params {
  const uint32_t *x, *w;
  const uint8_t *xs, *ws;
  const int32_t *starts, *counts;
  void *y;
  int64_t M, N, K, k_tiles, w_scale_bytes;
  int64_t m_tiles, n_tiles;
};

constexpr int kTile = 32;

template <bool GATED, bool BF16>
__global__ void __launch_bounds__(256) simple_kernel(const Params p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float xs[kTile][kTile + 1], ws[GATED ? 2 : 1][kTile][kTile + 1];
  const int64_t nt = blockIdx.x % p.n_tiles, mt = blockIdx.x / p.n_tiles % p.m_tiles, e = blockIdx.x / p.n_tiles / p.m_tiles;
  int64_t start = 0, count = p.M;
  if (p.starts) {
    start = p.starts[e], count = p.counts[e];
    if (start < 0 || start % kMxRows != 0 || start >= p.M) count = 0;
    count = min(count, p.M - start);
  }
  const int64_t m0 = mt * kTile, n0 = nt * kTile;
  if (m0 >= count) return;
  float acc[GATED ? 2 : 1][4] = {};
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  for (int64_t k0 = 0; k0 < p.K; k0 += kTile) {
    {
      for (int i = threadIdx.x; i < 128 * (GATED ? 3 : 2); i += 256) {
        const int which = i / 128, r = (i % 128) / 4, c = i % 4;
        const int64_t row = which == 0 ? start + m0 + r : n0 + r;
        const bool in = which == 0 ? m0 + r < count : n0 + r < p.N;
        uint32_t code = 0, scale = 0;
        if (in) {
          const int64_t matrix = which == 0 ? 0 : e * (GATED ? 2 : 1) + which - 1;
          code = (which == 0 ? p.x : p.w)[((which == 0 ? row : matrix * p.N + row) * p.K + k0) / 8 + c];
          scale = (which == 0 ? p.xs : p.ws + matrix * p.w_scale_bytes)[mx4_scale_word(row, k0 / 128, p.k_tiles) + (k0 / 32) % 4];
        }
        const float s = mx4_scale(scale);
        float *to = which == 0 ? &xs[r][8 * c] : &ws[which - 1][r][8 * c];
        for (int j = 0; j < 4; j++) {
          const float2 f = mx4_pair((code >> (8 * j)) & 255);
          to[2 * j] = f.x * s, to[2 * j + 1] = f.y * s;
        }
      }
    }
    __syncthreads();
    for (int k = 0; k < kTile; k++)
      for (int g = 0; g < (GATED ? 2 : 1); g++)
        for (int i = 0; i < 4; i++) acc[g][i] += xs[ty + 8 * i][k] * ws[g][tx][k];
    __syncthreads();
  }
  for (int i = 0; i < 4; i++) {
    const int64_t m = m0 + ty + 8 * i, n = n0 + tx;
    if (m >= count || n >= p.N) continue;
    float v = acc[0][i];
    if constexpr (GATED) v = v / (1.0f + expf(-v)) * acc[1][i];
    if constexpr (BF16)
      static_cast<__nv_bfloat16 *>(p.y)[(start + m) * p.N + n] = __float2bfloat16_rn(v);
    else
      static_cast<float *>(p.y)[(start + m) * p.N + n] = v;
  }
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4GemmArgs &a, cudaStream_t s) {
  Params p{};
  p.x = (const uint32_t *)a.x_codes, p.w = (const uint32_t *)a.codes;
  p.xs = (const uint8_t *)a.x_scales, p.ws = (const uint8_t *)a.scales;
  p.starts = a.starts, p.counts = a.counts, p.y = a.y;
  p.M = a.M, p.N = a.N, p.K = a.K, p.k_tiles = mx4_k_tiles(a.K), p.w_scale_bytes = mx4_scales_bytes(a.N, a.K);
  p.m_tiles = (a.M + kTile - 1) / kTile, p.n_tiles = (a.N + kTile - 1) / kTile;
  const int64_t grid = p.m_tiles * p.n_tiles * (a.starts ? a.experts : 1);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto kern = a.gated ? (a.bf16 ? simple_kernel<true, true> : simple_kernel<true, false>)
                      : (a.bf16 ? simple_kernel<false, true> : simple_kernel<false, false>);
  return launch_after(kern, grid, 256, 0, s, p);
}

cudaError_t read_clear_mx4_status(int *status, cudaStream_t) {
  *status = 0;
  return cudaSuccess;
}

}  // namespace qmm
