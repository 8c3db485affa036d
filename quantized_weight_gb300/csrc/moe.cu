// moe.cu -- tokens to experts and back: the plan (each token's best experts, and the tokens sorted by expert) and the
// weighted sum of a token's rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_attend.h"
#include "kv_launch.h"
#include "mx4_launch.h"
#include "qmm_device.cuh"
#include "sm100_ptx.cuh"

namespace qmm {
namespace {

using namespace sm100;

// ---------------------------------------------------------------- the best experts of a token

// Keys that order as logits do: NaN first, then from +infinity down; -0 and 0 are one value.  A key up to kMasked is
// -infinity's: such an expert is never taken.
constexpr uint32_t kMasked = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return v != v ? 0xFFFFFFFFu : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);     // (0xFFFFFFFF gives a NaN)
}

struct PlanParams {
  const void *logits;
  int64_t stride, T;
  int E, k, bf16, normalize;
  int64_t per_warp;        // tokens a warp of the sorting kernel takes
  int32_t *experts;
  float *weights;
  int32_t *places, *starts, *counts;
};

// One token by one warp: lane holds the experts p * 32 + lane.
template <int PER>
__device__ __forceinline__ void best_experts(const PlanParams &p, int64_t t, int lane) {
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int e = i * 32 + lane;
    key[i] = 0;
    if (e < p.E) {
      const int64_t at = t * p.stride + e;
      key[i] = key_of(p.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.logits)[at] << 16)
                             : static_cast<const float *>(p.logits)[at]);
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < PER; i++) top = max(top, key[i]);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  const float most = value_of(top);
  float all = 0.0f;        // of the softmax over every expert
  if (!p.normalize) {
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (key[i] > kMasked) all += expf(value_of(key[i]) - most);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  }
  int mine = -1;           // lane j: the j-th expert, and its logit's key
  uint32_t mine_key = 0;
  for (int j = 0; j < p.k; j++) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (key[i] > best) best = key[i], at = i * 32 + lane;
    const uint32_t win = __reduce_max_sync(0xFFFFFFFFu, best);
    if (win <= kMasked) break;
    const int e = (int)__reduce_min_sync(0xFFFFFFFFu, best == win ? (unsigned)at : 0xFFFFFFFFu);
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (i * 32 + lane == e) key[i] = 0;
    if (lane == j) mine = e, mine_key = win;
  }
  float w = mine >= 0 ? expf(value_of(mine_key) - most) : 0.0f;
  if (p.normalize) {
    all = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  }
  if (lane < p.k) {
    p.experts[t * p.k + lane] = mine;
    p.weights[t * p.k + lane] = mine >= 0 ? w / all : 0.0f;
  }
}

constexpr int kBestThreads = 256;
template <int PER>
__global__ void __launch_bounds__(kBestThreads) best_kernel(const PlanParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = (int64_t)blockIdx.x * (kBestThreads / 32) + (threadIdx.x >> 5);
  if (t < p.T) best_experts<PER>(p, t, threadIdx.x & 31);
}

// ---------------------------------------------------------------- the sort

// A stable counting sort of the tokens' entries by one cluster: each warp counts its tokens' experts, the counts of the
// warps before it (in its CTA by a thread an expert, in the other CTAs through shared memory) and the padded totals of
// the experts before say where its entries begin, and it hands out places in order.  With PER > 0 the warps also choose
// their tokens' experts, one launch in all.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortCluster = 8;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int PER, bool CLUSTER>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const PlanParams p) {
  extern __shared__ uint32_t count[];          // [warp][E], then totals [E] of this CTA
  __shared__ uint32_t sums[kSortWarps];
  uint32_t *total = count + kSortWarps * p.E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = threadIdx.x, E = p.E;
  const int rank = CLUSTER ? (int)cluster_ctarank() : 0;
  uint32_t *own = count + warp * E;
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) count[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t0 = min(p.T, (rank * kSortWarps + warp) * p.per_warp), t1 = min(p.T, t0 + p.per_warp);
  if constexpr (PER > 0) {
    for (int64_t t = t0; t < t1; t++) best_experts<PER>(p, t, lane);
    __syncwarp();
  }
  const int64_t i0 = t0 * p.k, i1 = t1 * p.k;
  for (int64_t i = i0 + lane; i < i1; i += 32) {
    const int x = p.experts[i];
    if (x >= 0) atomicAdd(own + x, 1u);
  }
  __syncthreads();
  uint32_t mine = 0;                           // entries of expert e in this CTA
  if (e < E) {
    for (int w = 0; w < kSortWarps; w++) {
      const uint32_t c = count[w * E + e];
      count[w * E + e] = mine;
      mine += c;
    }
    total[e] = mine;
  }
  uint32_t before = 0, whole = mine;           // entries of expert e in the CTAs before, and in all
  if constexpr (CLUSTER) {
    cluster_sync();
    if (e < E) {
      whole = 0;
      for (int r = 0; r < kSortCluster; r++) {
        const uint32_t c = ld_cluster_u32(mapa_shared(smem_addr(total + e), r));
        if (r < rank) before += c;
        whole += c;
      }
    }
    cluster_sync();                            // (nobody leaves while its totals are read)
  }
  // where expert e's rows begin
  const uint32_t padded = (whole + 127u) & ~127u;
  uint32_t at = padded;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, at, o);
    if (lane >= o) at += v;
  }
  if (lane == 31) sums[warp] = at;
  __syncthreads();
  if (warp == 0) {
    uint32_t v = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    sums[lane] = v;
  }
  __syncthreads();
  at += (warp > 0 ? sums[warp - 1] : 0) - padded;
  if (e < E) {
    if (rank == 0) p.starts[e] = (int)at, p.counts[e] = (int)whole;
    for (int w = 0; w < kSortWarps; w++) count[w * E + e] += at + before;
  }
  __syncthreads();
  for (int64_t i = i0; i < i1; i += 32) {
    const int x = i + lane < i1 ? p.experts[i + lane] : -1;
    const unsigned like = __match_any_sync(0xFFFFFFFFu, x);
    const int ahead = __popc(like & ((1u << lane) - 1));
    const uint32_t base = x >= 0 ? own[x] : 0;
    __syncwarp();
    if (x >= 0 && ahead == 0) own[x] = base + __popc(like);
    __syncwarp();
    if (i + lane < i1) p.places[i + lane] = x >= 0 ? (int)(base + ahead) : -1;
  }
}

// ---------------------------------------------------------------- back

struct CombineParams {
  const void *y;
  const float *weights;
  const int32_t *places;
  void *out;
  int64_t T, R, N, pieces;
  int k;
};

constexpr int kCombineThreads = 128;

template <bool BF16>
__device__ __forceinline__ float one(const void *y, int64_t at) {
  return BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(y)[at] << 16) : static_cast<const float *>(y)[at];
}
template <bool BF16>
__device__ __forceinline__ void put(void *y, int64_t at, float v) {
  if constexpr (BF16)
    static_cast<__nv_bfloat16 *>(y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float *>(y)[at] = v;
}

// A block takes a piece of one token's row: V elements a thread (1 where rows are not made of whole 16-byte words).
template <bool Y16, bool O16, int V>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x / p.pieces, n = ((blockIdx.x % p.pieces) * kCombineThreads + threadIdx.x) * V;
  if (n >= p.N) return;
  float sum[V];
#pragma unroll
  for (int v = 0; v < V; v++) sum[v] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < p.k; j++) {
    const int64_t row = p.places[t * p.k + j];
    if (row < 0 || row >= p.R) continue;
    const float w = p.weights ? p.weights[t * p.k + j] : 1.0f;
    const int64_t at = row * p.N + n;
    if constexpr (V == 1) {
      sum[0] += w * one<Y16>(p.y, at);
    } else if constexpr (Y16) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.y) + at));
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int v = 0; v < 4; v++) {
        sum[2 * v] += w * __uint_as_float(x[v] << 16);
        sum[2 * v + 1] += w * __uint_as_float(x[v] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p.y) + at + v));
        sum[v] += w * u.x, sum[v + 1] += w * u.y, sum[v + 2] += w * u.z, sum[v + 3] += w * u.w;
      }
    }
  }
  const int64_t at = t * p.N + n;
  if constexpr (V == 1) {
    put<O16>(p.out, at, sum[0]);
  } else if constexpr (O16) {
    uint32_t x[V / 2];
#pragma unroll
    for (int v = 0; v < V / 2; v++) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(sum[2 * v], sum[2 * v + 1]);
      x[v] = *reinterpret_cast<const uint32_t *>(&b);
    }
    __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at), make_uint4(x[0], x[1], x[2], x[3]));
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 4)
      __stcs(reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at + v),
             make_float4(sum[v], sum[v + 1], sum[v + 2], sum[v + 3]));
  }
}

template <int V>
void (*combine_for(bool y16, bool o16))(CombineParams) {
  if (y16) return o16 ? combine_kernel<true, true, V> : combine_kernel<true, false, V>;
  return o16 ? combine_kernel<false, true, V> : combine_kernel<false, false, V>;
}

template <int PER>
cudaError_t launch_best(const PlanParams &p, cudaStream_t s) {
  return launch_after(best_kernel<PER>, (p.T + kBestThreads / 32 - 1) / (kBestThreads / 32), kBestThreads, 0, s, p);
}

template <int PER, bool CLUSTER>
cudaError_t launch_sort(const PlanParams &p, cudaStream_t s) {
  const size_t smem = (size_t)(kSortWarps + 1) * p.E * sizeof(uint32_t);
  auto kern = sort_kernel<PER, CLUSTER>;
  if (smem > 48 * 1024 - 512) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(CLUSTER ? kSortCluster : 1);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {kSortCluster, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int PER>
cudaError_t launch_plan(PlanParams p, cudaStream_t s) {
  if (p.T <= 2 * kSortWarps) {
    p.per_warp = (p.T + kSortWarps - 1) / kSortWarps;
    return launch_sort<PER, false>(p, s);
  }
  const cudaError_t e = launch_best<PER>(p, s);
  if (e != cudaSuccess) return e;
  p.per_warp = (p.T + kSortWarps * kSortCluster - 1) / (kSortWarps * kSortCluster);
  return launch_sort<0, true>(p, s);
}

}  // namespace

cudaError_t launch_moe_plan(const MoePlanArgs &a, cudaStream_t s) {
  PlanParams p{};
  p.logits = a.logits, p.stride = a.stride, p.T = a.T, p.E = (int)a.E, p.k = (int)a.k;
  p.bf16 = a.bf16, p.normalize = a.normalize;
  p.experts = a.experts, p.weights = a.weights, p.places = a.places, p.starts = a.starts, p.counts = a.counts;
  const int per = (p.E + 31) / 32;
  if (per <= 1) return launch_plan<1>(p, s);
  if (per <= 2) return launch_plan<2>(p, s);
  if (per <= 4) return launch_plan<4>(p, s);
  if (per <= 8) return launch_plan<8>(p, s);
  if (per <= 16) return launch_plan<16>(p, s);
  return launch_plan<32>(p, s);
}

cudaError_t launch_moe_combine(const MoeCombineArgs &a, cudaStream_t s) {
  CombineParams p{};
  p.y = a.y, p.weights = a.weights, p.places = a.places, p.out = a.out;
  p.T = a.T, p.R = a.R, p.N = a.N, p.k = (int)a.k;
  // whole 16-byte words on both sides (8 elements a thread where one of them is bfloat16)
  const int v = a.y_bf16 || a.out_bf16 ? 8 : 4;
  const bool wide = a.N % v == 0;
  p.pieces = (a.N + kCombineThreads * (wide ? v : 1) - 1) / (kCombineThreads * (wide ? v : 1));
  if (p.T * p.pieces > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto kern = !wide ? combine_for<1>(a.y_bf16, a.out_bf16)
              : v == 8 ? combine_for<8>(a.y_bf16, a.out_bf16) : combine_kernel<false, false, 4>;
  return launch_after(kern, p.T * p.pieces, kCombineThreads, 0, s, p);
}

}  // namespace qmm
