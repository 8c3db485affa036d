// moe.cu -- tokens to experts and back: the plan (each token's best experts, and the tokens sorted by expert) and the
// weighted sum of a token's rows.
//
// Measured: 8 tokens, 6 of 64 experts 5.2 to 5.7 us, one block: a launch, six rounds of maxima, the barriers of the sort.  16381
// tokens, 8 of 128 19 us (12.8 and 11.4 us of cold caches): the choice is bound by its 360 instructions a token, which keep the ALU
// 72 % busy, the sort by what its 16 SMs wait for (loads, barriers and shared memory; 8 SMs took 3.7 us longer, and three kernels
// with the counts kept in `places` 11).  The sum is bound by memory: 8191 tokens of 6 rows of 2048 bfloat16 39.7 us, 87 % of
// measured HBM (rows of an odd length 83 %).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_attend.h"
#include "kv_launch.h"
#include "mx4.cuh"
#include "mx4_launch.h"
#include "qmm_device.cuh"
#include "sm100_ptx.cuh"

namespace qmm {
namespace {

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
  int whole;               // rows of logits can be read in vectors
  int wide;                // four places of a token lie at a multiple of 16 bytes (the array itself needs only 4)
  int64_t tokens;          // of a CTA of the sorting kernel
  int blocks;              // of 32 tokens, that its shared memory holds at once
  int32_t *experts;
  float *weights;
  int32_t *places, *starts, *counts;
};

// One token by LANES lanes, each with PER experts in a row, so that of equal keys the lowest lane's is the lowest expert's.
// A lane keeps its best; a round is one maximum over the lanes, and only the lane that had it looks for its next.  Few lanes
// a token let a round's instructions serve several tokens.  `live`: the lanes' token exists.  The whole warp calls it.
template <int LANES, int PER>
__device__ __forceinline__ void best_experts(const PlanParams &p, int64_t t, bool live, int lane) {
  constexpr int OWN = kMoeMaxK / LANES;        // of the token's choices, each lane keeps every LANES-th
  const int sub = lane & (LANES - 1), e0 = PER * sub;
  uint32_t key[PER];
  const int64_t row = t * p.stride + e0;
  if (PER % 4 == 0 && p.whole) {      // E is a multiple of PER, rows begin at 16 bytes: eight bytes or more at a time
    const bool in = live && e0 < p.E;
#pragma unroll
    for (int i = 0; i + 3 < PER; i += 4) {
      float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (in && p.bf16) {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.logits) + row + i);
        v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
        v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
      } else if (in) {
        const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.logits) + row + i);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
      }
#pragma unroll
      for (int j = 0; j < 4; j++) key[i + j] = key_of(v[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; i++) {
      key[i] = 0;
      if (live && e0 + i < p.E)
        key[i] = key_of(p.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.logits)[row + i] << 16)
                               : static_cast<const float *>(p.logits)[row + i]);
    }
  }
  uint32_t best = 0;
  int at = 0;
  auto look = [&]() {      // (no chain of comparisons: maxima by pairs, then which have it)
    uint32_t m[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) m[i] = key[i];
#pragma unroll
    for (int o = PER / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; i++) m[i] = max(m[i], m[i + o]);
    best = m[0];
    uint32_t had = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) had |= (key[i] == best ? 1u : 0u) << i;
    at = __ffs(had) - 1;
  };
  auto over_lanes = [&](uint32_t v) {
    if constexpr (LANES == 32) {
      return __reduce_max_sync(0xFFFFFFFFu, v);
    } else {
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
      return v;
    }
  };
  auto sum_lanes = [&](float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  };
  look();
  uint32_t win = over_lanes(best);
  const float most = value_of(win);
  float all = 0.0f;        // of the softmax
  if (!p.normalize) {
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (key[i] > kMasked) all += expf(value_of(key[i]) - most);
  }
  int mine[OWN];
  float w[OWN];
  bool more = true;
#pragma unroll
  for (int q = 0; q < OWN; q++) {
    mine[q] = -1, w[q] = 0.0f;
    for (int j = 0; j < LANES && more; j++) {
      more = q * LANES + j < p.k && __any_sync(0xFFFFFFFFu, win > kMasked);
      if (!more) break;
      const unsigned had = __ballot_sync(0xFFFFFFFFu, best == win) >> (lane & ~(LANES - 1));
      const int from = __ffs(had) - 1;         // (of those with the lanes of this token; some lane has its maximum)
      const int e = __shfl_sync(0xFFFFFFFFu, e0 + at, from, LANES);
      if (win > kMasked) {
        if (j == sub) mine[q] = e, w[q] = value_of(win);
        if (sub == from) {
#pragma unroll
          for (int i = 0; i < PER; i++)
            if (i == at) key[i] = 0;
          look();
        }
      }
      win = over_lanes(best);
    }
  }
#pragma unroll
  for (int q = 0; q < OWN; q++) {
    if (q * LANES >= p.k) break;
    w[q] = mine[q] >= 0 ? expf(w[q] - most) : 0.0f;
    if (p.normalize) all += w[q];
  }
  all = sum_lanes(all);
#pragma unroll
  for (int q = 0; q < OWN; q++) {
    const int j = q * LANES + sub;
    if (q * LANES >= p.k) break;
    if (live && j < p.k) {
      p.experts[t * p.k + j] = mine[q];
      p.weights[t * p.k + j] = mine[q] >= 0 ? w[q] / all : 0.0f;
    }
  }
}

// The tokens t0 .. t1 - 1 by `warps` warps, of which this one is `warp`.
template <int LANES, int PER>
__device__ __forceinline__ void best_of(const PlanParams &p, int64_t t0, int64_t t1, int warp, int warps, int lane) {
  constexpr int AT_ONCE = 32 / LANES;
  for (int64_t t = t0 + warp * AT_ONCE; t < t1; t += warps * AT_ONCE) {
    const int64_t own = t + lane / LANES;
    best_experts<LANES, PER>(p, own, own < t1, lane);
  }
}

constexpr int kBestThreads = 128;
template <int LANES, int PER>
__global__ void __launch_bounds__(kBestThreads) best_kernel(const PlanParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int TOKENS = kBestThreads / LANES;
  const int64_t t0 = (int64_t)blockIdx.x * TOKENS;
  best_of<LANES, PER>(p, t0, min(p.T, t0 + TOKENS), threadIdx.x >> 5, kBestThreads / 32, threadIdx.x & 31);
}

// ---------------------------------------------------------------- the sort
//
// A stable counting sort.  Of 32 tokens and an expert, a word says which of the tokens have it (by atomic or, whose order
// changes nothing); so an entry's place is where its expert's rows begin, plus that expert's entries in the words before
// (sums of their bits), plus the bits below its own.  One CTA does few tokens, its warps choosing their experts first; a
// cluster does many, the experts' totals of its CTAs going through shared memory.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortCluster = 16, kSortBlocks = 64;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Where the rows of expert threadIdx.x begin, given its entries (0 past the last expert): a block's exclusive sum of counts
// rounded up to 128.
__device__ __forceinline__ uint32_t begin_of(uint32_t entries, uint32_t *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t padded = (entries + 127u) & ~127u;
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
  return at + (warp > 0 ? sums[warp - 1] : 0) - padded;
}

// LANES 0: the experts are chosen already, and a cluster sorts.
template <int LANES, int PER>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const PlanParams p) {
  constexpr bool CLUSTER = LANES == 0;
  extern __shared__ uint32_t mask[];           // [block][E] words, then [block][E] sums of 16 bits
  __shared__ uint32_t total[kMoeMaxExperts], next[kMoeMaxExperts], part[kSortThreads], sums[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E, k = p.k;
  uint16_t *before = reinterpret_cast<uint16_t *>(mask + p.blocks * E);
  const int rank = CLUSTER ? (int)sm100::cluster_ctarank() : 0;
  // a thread an expert and group of blocks
  int EP = 32;
  while (EP < E) EP *= 2;
  const int groups = kSortThreads / EP, e = threadIdx.x & (EP - 1), g = threadIdx.x / EP;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c0 = min(p.T, rank * p.tokens), c1 = min(p.T, c0 + p.tokens);
  if constexpr (!CLUSTER) {
    best_of<LANES, PER>(p, c0, c1, warp, kSortWarps, lane);
    __syncthreads();
  }

  // eight of a token's experts from the j-th on, -1 past its last (loads that wait for nothing between them)
  auto load8 = [&](int64_t t, int j, int (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = t < c1 && j + i < k ? p.experts[t * k + j + i] : -1;
  };
  // the words of the blocks from token t0 on, their sums, and the totals
  auto count = [&](int64_t t0) {
    const int n = (int)min((int64_t)p.blocks, (c1 - t0 + 31) / 32);
    for (int i = threadIdx.x; i < n * E; i += kSortThreads) mask[i] = 0;
    __syncthreads();
    for (int b = warp; b < n; b += kSortWarps) {
      const int64_t t = t0 + 32 * b + lane;
      for (int j = 0; j < k; j += 8) {
        int x[8];
        load8(t, j, x);
#pragma unroll
        for (int i = 0; i < 8; i++)
          if (x[i] >= 0) atomicOr(mask + b * E + x[i], 1u << lane);
      }
    }
    __syncthreads();
    const int b0 = n * g / groups, b1 = n * (g + 1) / groups;
    uint32_t sum = 0;
    if (e < E)
      for (int b = b0; b < b1; b++) sum += __popc(mask[b * E + e]);
    part[threadIdx.x] = sum;
    __syncthreads();
    if (e < E) {
      uint32_t at = 0;
      for (int i = 0; i < g; i++) at += part[i * EP + e];
      for (int b = b0; b < b1; b++) {
        before[b * E + e] = (uint16_t)at;
        at += __popc(mask[b * E + e]);
      }
      if (g == groups - 1) total[e] = at;
    }
    __syncthreads();
  };
  auto hand_out = [&](int64_t t0) {
    const int n = (int)min((int64_t)p.blocks, (c1 - t0 + 31) / 32);
    for (int b = warp; b < n; b += kSortWarps) {
      const int64_t t = t0 + 32 * b + lane;
      for (int j = 0; j < k; j += 8) {
        int x[8];
        load8(t, j, x);
#pragma unroll
        for (int i = 0; i < 8; i++)
          if (x[i] >= 0) x[i] = (int)(next[x[i]] + before[b * E + x[i]] + __popc(mask[b * E + x[i]] & ((1u << lane) - 1)));
        if (t < c1) {
          if (p.wide) {
#pragma unroll
            for (int i = 0; i < 8; i += 4)
              if (j + i < k) *reinterpret_cast<int4 *>(p.places + t * k + j + i) = make_int4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
              if (j + i < k) p.places[t * k + j + i] = x[i];
          }
        }
      }
    }
  };

  const bool once = c1 - c0 <= 32 * p.blocks;
  if (once) {
    count(c0);
  } else {
    for (int i = threadIdx.x; i < E; i += kSortThreads) total[i] = 0;
    __syncthreads();
    for (int64_t i = c0 * k + threadIdx.x; i < c1 * k; i += 8 * kSortThreads) {
      int x[8];
#pragma unroll
      for (int a = 0; a < 8; a++) x[a] = i + a * kSortThreads < c1 * k ? p.experts[i + a * kSortThreads] : -1;
#pragma unroll
      for (int a = 0; a < 8; a++)
        if (x[a] >= 0) atomicAdd(total + x[a], 1u);
    }
    __syncthreads();
  }
  uint32_t earlier = 0, whole = 0;             // entries of expert threadIdx.x in the CTAs before, and in all
  if constexpr (CLUSTER) {
    sm100::cluster_sync();
    if (threadIdx.x < E)
      for (int r = 0; r < kSortCluster; r++) {
        const uint32_t c = ld_cluster_u32(sm100::mapa_shared(sm100::smem_addr(total + threadIdx.x), r));
        if (r < rank) earlier += c;
        whole += c;
      }
    sm100::cluster_sync();                     // (nobody leaves or counts on while its totals are read)
  } else if (threadIdx.x < E) {
    whole = total[threadIdx.x];
  }
  const uint32_t begin = begin_of(whole, sums);
  if (threadIdx.x < E) {
    next[threadIdx.x] = begin + earlier;
    if (rank == 0) p.starts[threadIdx.x] = (int)begin, p.counts[threadIdx.x] = (int)whole;
  }
  __syncthreads();
  if (once) {
    hand_out(c0);
    return;
  }
  for (int64_t t0 = c0; t0 < c1; t0 += 32 * p.blocks) {
    count(t0);
    hand_out(t0);
    __syncthreads();
    if (threadIdx.x < E) next[threadIdx.x] += total[threadIdx.x];
  }
}

// ---------------------------------------------------------------- back

struct CombineParams {
  const void *y;
  const float *weights;
  const int32_t *places;
  void *out;
  int64_t T, R, N;
  Divisor pieces;          // blocks of a token
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

// A block takes a piece of one token's row: V elements in a row a thread or, where rows are not made of whole 16-byte words
// (V = 1), four that are a block's threads apart.
template <bool Y16, bool O16, int V>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int U = V == 1 ? 4 : 1, S = V == 1 ? kCombineThreads : 1, ALL = V * U;
  uint32_t piece = blockIdx.x;
  const int64_t t = p.pieces.split(piece), n = (int64_t)piece * (kCombineThreads * ALL) + threadIdx.x * V;
  if (n >= p.N) return;
  float sum[ALL];
#pragma unroll
  for (int v = 0; v < ALL; v++) sum[v] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < p.k; j++) {
    const int64_t row = p.places[t * p.k + j];
    if (row < 0 || row >= p.R) continue;
    const float w = p.weights ? p.weights[t * p.k + j] : 1.0f;
    const int64_t at = row * p.N + n;
    if constexpr (V == 1) {
#pragma unroll
      for (int u = 0; u < U; u++)
        if (n + u * S < p.N) sum[u] += w * one<Y16>(p.y, at + u * S);
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
#pragma unroll
    for (int u = 0; u < U; u++)
      if (n + u * S < p.N) put<O16>(p.out, at + u * S, sum[u]);
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

constexpr int64_t kFewTokens = 32;      // what one CTA plans

template <int LANES, int PER>
cudaError_t launch_sort(PlanParams p, int ctas, cudaStream_t s) {
  p.tokens = (p.T + ctas - 1) / ctas;
  // words of 32 bits and sums of 16, as far as 160 KB of shared memory go
  const int64_t fit = 160 * 1024 / (6 * p.E), blocks = (p.tokens + 31) / 32;
  p.blocks = (int)(blocks < fit ? blocks : fit);
  if (p.blocks > kSortBlocks) p.blocks = kSortBlocks;
  const size_t smem = (size_t)6 * p.blocks * p.E;
  auto kern = sort_kernel<LANES, PER>;
  cudaError_t e = cudaSuccess;
  if (smem > 32 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// PER: experts of a lane where 32 lanes have a token.
template <int PER>
cudaError_t launch_plan(PlanParams p, cudaStream_t s) {
  // lanes of a token, and experts of a lane, where many are planned (4 lanes for up to 128 experts: 12.2 us instead of 11.5 for
  // 16381 tokens, their chains of dependent instructions being longer; 32 lanes: 11.2 us)
  constexpr int LANES = PER <= 8 ? 8 : 32, MANY = 32 / LANES * PER;
  const int size = p.bf16 ? 2 : 4, per = p.T <= kFewTokens ? PER : MANY;
  p.whole = per % 4 == 0 && p.E % per == 0 && reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.stride * size % 16 == 0;
  if (p.T <= kFewTokens) return launch_sort<32, PER>(p, 1, s);
  constexpr int64_t TOKENS = kBestThreads / LANES;     // of a block
  const cudaError_t e = launch_after(best_kernel<LANES, MANY>, (p.T + TOKENS - 1) / TOKENS, kBestThreads, 0, s, p);
  return e != cudaSuccess ? e : launch_sort<0, 0>(p, kSortCluster, s);
}

}  // namespace

cudaError_t launch_moe_plan(const MoePlanArgs &a, cudaStream_t s) {
  PlanParams p{};
  p.logits = a.logits, p.stride = a.stride, p.T = a.T, p.E = (int)a.E, p.k = (int)a.k;
  p.bf16 = a.bf16, p.normalize = a.normalize;
  p.experts = a.experts, p.weights = a.weights, p.places = a.places, p.starts = a.starts, p.counts = a.counts;
  p.wide = p.k % 4 == 0 && reinterpret_cast<uintptr_t>(p.places) % 16 == 0;
  if (p.E <= 32) return launch_plan<1>(p, s);
  if (p.E <= 64) return launch_plan<2>(p, s);
  if (p.E <= 128) return launch_plan<4>(p, s);
  if (p.E <= 256) return launch_plan<8>(p, s);
  if (p.E <= 512) return launch_plan<16>(p, s);
  return launch_plan<32>(p, s);
}

cudaError_t launch_moe_combine(const MoeCombineArgs &a, cudaStream_t s) {
  CombineParams p{};
  p.y = a.y, p.weights = a.weights, p.places = a.places, p.out = a.out;
  p.T = a.T, p.R = a.R, p.N = a.N, p.k = (int)a.k;
  // whole 16-byte words on both sides (8 elements a thread where one of them is bfloat16)
  const int v = a.y_bf16 || a.out_bf16 ? 8 : 4;
  const bool wide = a.N % v == 0;
  const int64_t each = kCombineThreads * (wide ? v : 4), pieces = (a.N + each - 1) / each;
  if (p.T * pieces > 0x7FFFFFFF) return cudaErrorInvalidValue;       // (more of out than there is memory)
  p.pieces = Divisor((uint32_t)pieces);
  auto kern = !wide ? combine_for<1>(a.y_bf16, a.out_bf16)
              : v == 8 ? combine_for<8>(a.y_bf16, a.out_bf16) : combine_kernel<false, false, 4>;
  return launch_after(kern, p.T * pieces, kCombineThreads, 0, s, p);
}

}  // namespace qmm
