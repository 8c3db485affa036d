// mx4_gemm.cu -- y = x * w^T of two microscaled 4-bit matrices on the block-scaled tensor cores, for one matrix w or for the
// rows of each expert.
//
// The tensor core takes e2m1 codes and their scales as they are stored, so nothing is converted on the way: TMA brings tiles
// of 256 elements (128 bytes of a row) of both operands into shared memory, bulk copies the scale tiles, tcgen05.cp puts
// the scales into TMEM, and tcgen05.mma (kind::mxf4) sums 64 elements at a time in float32.
//
// The MMA computes D[128 weight rows, tokens] = w * x^T: the weights are its M side, so that one kernel serves decode
// steps (16 tokens are an N of 16, and the weights stream through once) and prompts alike, and a warp's stores are 32
// consecutive n of a token.  gated: two weight tiles and two accumulators, whose values meet in the same thread.
//
// Roles of a CTA (one an SM, walking over items = weight tile x token tile):
//   warp 0     copies, a ring of stages (mbarriers: full by transaction bytes, empty by the MMAs' commit)
//   warp 1     TMEM allocation and the MMA issuer
//   warps 2-9  epilogue: tcgen05.ld, silu, rounding, stores; two accumulators where TMEM holds them, so that an item's
//              epilogue goes beside the next one's products
// A call with few items splits K over the CTAs of a cluster: each writes its partial tile into the shared memory of the CTA
// that owns the token, and the owner adds them up in the order of the ranks, so that the sum is the same every time.
//
// Every wait is bounded (bounded_wait.cuh).  One that runs out ends the CTA's work: it writes nothing more, waits for its
// copies and MMAs in flight, frees its TMEM, and qmm_check() reports it.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <atomic>

#include "bounded_wait.cuh"
#include "kv_attend.h"
#include "mx4.cuh"
#include "mx4_launch.h"
#include "mx4_ptx.cuh"
#include "qmm_device.cuh"

namespace qmm {

__device__ int g_mx4_status = 0;   // QMM_OK or QMM_ERR_DEVICE_TIMEOUT (-6)

namespace {

using namespace sm100;

constexpr int BM = 128;                    // weight rows of a tile
constexpr int BK = 256;                    // elements of a stage: 128 bytes of a row, one swizzle atom wide
constexpr int MMA_K = 64;
constexpr int EPI_WARP0 = 2, EPI_WARPS = 8;
constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int EPI_THREADS = 32 * EPI_WARPS;
constexpr int MAX_STAGES = 8;
constexpr int MAX_SPLIT = 8;
constexpr int SMEM_LIMIT = 227 * 1024;
constexpr int TMEM_COLS = 512;

struct Params {
  const uint8_t *xs, *ws;
  const int32_t *starts, *counts;          // null: one matrix, M rows
  void *y;
  int64_t M, N;                            // rows of x, rows of a matrix
  int64_t m_tiles, n_tiles;                // (m_tiles: one matrix only)
  int64_t w_scale_bytes;                   // of a matrix
  int k_tiles, k_stages, k_steps;          // scale tiles of a row, stages and MMAs along K
  int experts, bf16;
  int ts;                                  // tokens of a tile: 64, 128, 192 or 256
  int box;                                 // rows of x in a copy
  int stages, bufs;                        // ring depth, accumulators
  int split;                               // CTAs of a cluster, each with a part of K
};

struct Layout {                            // of a CTA's shared memory
  int a, b, sfa, sfb, stage;               // bytes: weights, tokens, scales, all
  int ring, red, list, bars, total;
};
__host__ __device__ inline Layout layout(bool gated, int ts, int stages, int split, int experts) {
  Layout l;
  const int two = gated ? 2 : 1;
  l.a = two * BM * (BK / 2);
  l.b = ts * (BK / 2);
  l.sfa = two * 2 * kMxTileBytes;
  l.sfb = (ts > kMxRows ? 2 : 1) * 2 * kMxTileBytes;
  l.stage = l.a + l.b + l.sfa + l.sfb;     // (multiples of 1024 bytes)
  l.ring = stages * l.stage;
  l.red = split > 1 ? two * ts * BM * 4 : 0;
  l.list = (3 * experts + 1) * 4;          // starts, counts, and token tiles before
  l.list = (l.list + 15) & ~15;
  l.bars = 8 * (2 * MAX_STAGES + 4 + 1) + 16 + 4 * MAX_SPLIT;
  l.total = l.ring + l.red + l.list + l.bars + 1024;   // (1024: the ring begins at a multiple of it)
  return l;
}

// One piece of work: a weight tile and a token tile.
struct Item {
  int64_t n0;                              // first row of the weight tile
  int64_t row;                             // first row of the token tile in x and y
  int rows;                                // tokens of it
  int expert;
};

struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) s = 0, ph ^= 1u;
  }
};

template <bool GATED>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w, const Params p) {
  constexpr int TWO = GATED ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const Layout l = layout(GATED, p.ts, p.stages, p.split, p.experts);
  float *red = reinterpret_cast<float *>(smem + l.ring);
  int32_t *starts = reinterpret_cast<int32_t *>(smem + l.ring + l.red), *counts = starts + p.experts, *before = counts + p.experts;
  const uint32_t bars = sbase + l.ring + l.red + l.list;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (MAX_STAGES + s); };
  auto acc_full = [&](int b) { return bars + 8 * (2 * MAX_STAGES + b); };
  auto acc_empty = [&](int b) { return bars + 8 * (2 * MAX_STAGES + 2 + b); };
  const uint32_t drain_bar = bars + 8 * (2 * MAX_STAGES + 4);
  uint8_t *tail = smem + l.ring + l.red + l.list + 8 * (2 * MAX_STAGES + 5);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tail);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
  uint32_t *fine = reinterpret_cast<uint32_t *>(tail + 8);       // [split]: that CTA's part is whole
  const WaitCtl ctl{abort_flag, &g_mx4_status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; s++) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), EPI_THREADS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_x);
    tma_prefetch_desc(&tmap_w);
  }
  if (warp == 1) tmem_alloc(smem_addr(tmem_slot), TMEM_COLS);
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    // the experts' rows, made to fit x, and the token tiles before each
    int sum = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + lane;
      int64_t start = 0, count = p.M;
      if (p.starts) {
        start = e < p.experts ? p.starts[e] : 0, count = e < p.experts ? p.counts[e] : 0;
        if (start < 0 || start >= p.M || start % kMxRows != 0 || count < 0) start = 0, count = 0;
        if (count > p.M - start) count = p.M - start;
      }
      const int tiles = e < p.experts ? (int)((count + p.ts - 1) / p.ts) : 0;
      int at = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, at, o);
        if (lane >= o) at += v;
      }
      if (e < p.experts) starts[e] = (int)start, counts[e] = (int)count, before[e + 1] = sum + at;
      sum += __shfl_sync(0xFFFFFFFFu, at, 31);
    }
    if (lane == 0) before[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (p.split > 1) cluster_sync();             // (no CTA writes into one that has not begun)

  const int64_t items = (int64_t)before[p.experts] * p.n_tiles;
  const int64_t first = p.split > 1 ? blockIdx.x / p.split : blockIdx.x, step = p.split > 1 ? gridDim.x / p.split : gridDim.x;
  // this CTA's stages of K
  const int ks0 = (int)((int64_t)p.k_stages * rank / p.split), ks1 = (int)((int64_t)p.k_stages * (rank + 1) / p.split);

  auto item_at = [&](int64_t i) {
    Item it;
    int lo = 0, hi = p.experts;                // the last expert whose items begin at or before i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)before[mid] * p.n_tiles <= i) lo = mid; else hi = mid;
    }
    const int64_t tiles = before[lo + 1] - before[lo], j = i - (int64_t)before[lo] * p.n_tiles;
    const int64_t nt = j / tiles;
    const int m0 = (int)(j - nt * tiles) * p.ts;
    it.expert = lo;
    it.n0 = nt * BM;
    it.row = (int64_t)starts[lo] + m0;
    it.rows = min(counts[lo] - m0, p.ts);
    return it;
  };

  Ring ring;                                   // (of the copying and the issuing thread)
  int issued = 0;                              // stages so far
  int local = 0;                               // items so far
  bool ok = true;
  for (int64_t i = first; i < items; i += step, local++) {
    const Item it = item_at(i);
    const int buf = local % p.bufs;
    const uint32_t use = (local / p.bufs) & 1;
    // tokens of the tile before its first: its scale tile may begin 64 rows earlier
    const int shift = (int)(it.row & (kMxRows - 1));
    const int sf_tiles = (shift + it.rows + kMxRows - 1) / kMxRows;
    if (warp == 0) {
      // -------------------------------------------------------- copies
      if (lane == 0 && ok) {
        const int boxes = (it.rows + p.box - 1) / p.box;
        const int64_t w_row = (int64_t)it.expert * TWO * p.N + it.n0;
        const uint8_t *ws = p.ws + (int64_t)it.expert * TWO * p.w_scale_bytes + (it.n0 >> 7) * p.k_tiles * kMxTileBytes;
        const uint8_t *xs = p.xs + (it.row >> 7) * p.k_tiles * kMxTileBytes;
        for (int ks = ks0; ks < ks1; ks++, issued++, ring.next(p.stages)) {
          const uint32_t base = sbase + ring.s * l.stage, bar = full(ring.s);
          if (!wait_bounded(empty(ring.s), ring.ph ^ 1, ctl)) { ok = false; break; }
          const uint32_t sf = (uint32_t)min(2, p.k_tiles - 2 * ks) * kMxTileBytes;
          mbar_arrive_expect_tx(bar, l.a + boxes * p.box * (BK / 2) + (TWO + sf_tiles) * sf);
#pragma unroll
          for (int g = 0; g < TWO; g++) {
            tma_load_2d(base + g * BM * (BK / 2), &tmap_w, ks * (BK / 2), (int)(w_row + g * p.N), bar);
            bulk_copy(base + l.a + l.b + g * 2 * kMxTileBytes, ws + g * p.w_scale_bytes + (int64_t)ks * 2 * kMxTileBytes, sf, bar);
          }
          for (int b = 0; b < boxes; b++)
            tma_load_2d(base + l.a + b * p.box * (BK / 2), &tmap_x, ks * (BK / 2), (int)it.row + b * p.box, bar);
          for (int t = 0; t < sf_tiles; t++)
            bulk_copy(base + l.a + l.b + l.sfa + t * 2 * kMxTileBytes,
                      xs + ((int64_t)t * p.k_tiles + 2 * ks) * kMxTileBytes, sf, bar);
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- products
      if (lane == 0 && ok) {
        ok = wait_bounded(acc_empty(buf), use ^ 1, ctl);
        tc_fence_after();
        const int n = (it.rows + 15) & ~15;
        const uint32_t id0 = idesc_mxf4(BM, n, 0), id1 = idesc_mxf4(BM, n, 1);
        const uint32_t d = tmem + buf * TWO * p.ts;
        for (int ks = ks0; ks < ks1 && ok; ks++, issued++, ring.next(p.stages)) {
          if (!wait_bounded(full(ring.s), ring.ph, ctl)) { ok = false; break; }
          tc_fence_after();
          const uint32_t base = sbase + ring.s * l.stage;
          // scales: by turns in two places, 8 columns a weight tile (4 a scale tile) and 16 for the tokens
          const uint32_t sfa = tmem + p.bufs * TWO * p.ts + (issued & 1) * (8 * TWO + 16), sfb = sfa + 8 * TWO;
          const int sts = min(2, p.k_tiles - 2 * ks);
          for (int a = 0; a < sts; a++) {
#pragma unroll
            for (int g = 0; g < TWO; g++)
              tmem_cp_32x16b(sfa + g * 8 + a * 4, smem_desc_scales(base + l.a + l.b + (g * 2 + a) * kMxTileBytes));
            for (int t = 0; t < sf_tiles; t++)
              tmem_cp_32x16b(sfb + a * 8 + t * 4, smem_desc_scales(base + l.a + l.b + l.sfa + (t * 2 + a) * kMxTileBytes));
          }
          const uint64_t ad = smem_desc_sw128(base), bd = smem_desc_sw128(base + l.a);
          const int steps = min(BK / MMA_K, p.k_steps - ks * (BK / MMA_K));
          for (int j = 0; j < steps; j++) {
#pragma unroll
            for (int g = 0; g < TWO; g++)
              umma_mxf4(d + g * p.ts, ad + g * (BM * (BK / 2) / 16) + 2 * j, bd + 2 * j, j & 1 ? id1 : id0,
                        sfa + g * 8 + (j >> 1) * 4, sfb + (j >> 1) * 8 + (shift >> 5), ks > ks0 || j > 0);
          }
          umma_commit(empty(ring.s));
        }
        if (ok) umma_commit(acc_full(buf));
      }
    } else {
      // -------------------------------------------------------- epilogue
      const int q = warp & 3, half = (warp - EPI_WARP0) >> 2;      // TMEM lane quarter; which chunks of 16 tokens
      const int r = q * 32 + lane;
      const int64_t n = it.n0 + r;
      if (ok) ok = __all_sync(0xFFFFFFFFu, wait_bounded(acc_full(buf), use, ctl));
      if (ok) {
        tc_fence_after();
        const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + buf * TWO * p.ts;
#pragma unroll 1
        for (int c = 16 * half; c < it.rows; c += 32) {
          uint32_t v[TWO][16];
          __syncwarp();
#pragma unroll
          for (int g = 0; g < TWO; g++) tmem_ld_32x32b_x16(d + g * p.ts + c, v[g]);
          tmem_ld_wait();
          if (p.split > 1) {
            // token c + j of the tile belongs to rank (c + j) % split, as its row (c + j) / split
#pragma unroll
            for (int j = 0; j < 16; j++) {
              const int t = c + j;
              if (t < it.rows)
#pragma unroll
                for (int g = 0; g < TWO; g++)
                  st_cluster_f32(mapa_shared(smem_addr(red + ((rank * (p.ts / p.split) + t / p.split) * TWO + g) * BM + r), t % p.split),
                                 __uint_as_float(v[g][j]));
            }
          } else if (n < p.N) {
#pragma unroll
            for (int j = 0; j < 16; j++) {
              if (c + j >= it.rows) break;
              float o = __uint_as_float(v[0][j]);
              if constexpr (GATED) o = o / (1.0f + expf(-o)) * __uint_as_float(v[TWO - 1][j]);
              const int64_t at = (it.row + c + j) * p.N + n;
              if (p.bf16)
                __stcs(static_cast<unsigned short *>(p.y) + at, __bfloat16_as_ushort(__float2bfloat16_rn(o)));
              else
                __stcs(static_cast<float *>(p.y) + at, o);
            }
          }
        }
        tc_fence_before();
        mbar_arrive(acc_empty(buf));
      }
    }
    if (p.split > 1) {
      __syncthreads();                         // (every epilogue warp has sent its part, or none will)
      if (threadIdx.x < p.split) st_cluster_u32(mapa_shared(smem_addr(fine + rank), threadIdx.x), *abort_flag ? 0u : 1u);
      __syncwarp();
      cluster_sync();
      bool whole = true;
      for (int s = 0; s < p.split; s++) whole = whole && fine[s] != 0;
      if (whole) {
        const int own = (it.rows - rank + p.split - 1) / p.split;     // tokens of this CTA
        for (int x = threadIdx.x; x < own * BM; x += NUM_THREADS) {
          const int t = x / BM, r = x % BM;
          float sum[TWO];
#pragma unroll
          for (int g = 0; g < TWO; g++) {
            sum[g] = 0.0f;
            for (int s = 0; s < p.split; s++) sum[g] += red[((s * (p.ts / p.split) + t) * TWO + g) * BM + r];
          }
          float o = sum[0];
          if constexpr (GATED) o = o / (1.0f + expf(-o)) * sum[TWO - 1];
          if (it.n0 + r < p.N) {
            const int64_t at = (it.row + t * p.split + rank) * p.N + it.n0 + r;
            if (p.bf16)
              __stcs(static_cast<unsigned short *>(p.y) + at, __bfloat16_as_ushort(__float2bfloat16_rn(o)));
            else
              __stcs(static_cast<float *>(p.y) + at, o);
          }
        }
      }
      __syncwarp();
      if (i + step < items) cluster_sync();    // (its neighbours read what the next item overwrites)
    }
  }
  if (warp == 0 && lane == 0) {
    // every copy lands before this CTA's memory goes to another
    for (int j = issued > p.stages ? issued - p.stages : 0; j < issued; j++) wait_drain(full(j % p.stages), (j / p.stages) & 1);
  }
  if (warp == 1 && lane == 0 && !ok) {
    umma_commit(drain_bar);
    wait_drain(drain_bar, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    known.store(fn, std::memory_order_relaxed);
  }
  return fn;
}

// Rows of K / 2 bytes, in boxes of 128 bytes by `box` rows.
bool encode_rows(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m, const void *base, int64_t rows, int64_t K, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  const cuuint32_t boxes[2] = {BK / 2, (cuuint32_t)box}, one[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, boxes, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4GemmArgs &a, cudaStream_t s) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode();
  if (!encode) return cudaErrorNotSupported;
  const int two = a.gated ? 2 : 1, sms = kv_max_ctas(1);
  Params p{};
  p.xs = static_cast<const uint8_t *>(a.x_scales), p.ws = static_cast<const uint8_t *>(a.scales);
  p.starts = a.starts, p.counts = a.counts, p.y = a.y, p.M = a.M, p.N = a.N;
  p.n_tiles = (a.N + BM - 1) / BM;
  p.w_scale_bytes = mx4_scales_bytes(a.N, a.K);
  p.k_tiles = (int)mx4_k_tiles(a.K), p.k_stages = (int)((a.K + BK - 1) / BK), p.k_steps = (int)((a.K + MMA_K - 1) / MMA_K);
  p.experts = (int)a.experts, p.bf16 = a.bf16;
  // rows that an expert has, about
  const int64_t met = a.starts ? (a.routed < a.experts ? (a.routed > 1 ? a.routed : 1) : a.experts) : 1;
  const int64_t rows = a.starts ? (a.routed + met - 1) / met : a.M;
  p.ts = rows <= 64 ? 64 : a.gated || rows <= 128 ? 128 : 192;
  p.box = rows <= 16 ? 16 : 64;
  p.bufs = 2 * two * p.ts + 2 * (8 * two + 16) <= TMEM_COLS ? 2 : 1;
  // items, about, and parts of K that give every SM one
  const int64_t items = met * ((rows + p.ts - 1) / p.ts) * p.n_tiles;
  p.split = 1;
  if (p.ts == 64)
    while (p.split < MAX_SPLIT && items * p.split * 2 <= sms && p.k_stages >= 2 * p.split) p.split *= 2;
  const int tail = layout(a.gated, p.ts, 0, p.split, p.experts).total;
  p.stages = (SMEM_LIMIT - tail) / layout(a.gated, p.ts, 1, p.split, p.experts).stage;
  if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
  const Layout l = layout(a.gated, p.ts, p.stages, p.split, p.experts);
  CUtensorMap tx, tw;
  if (!encode_rows(encode, &tx, a.x_codes, a.M, a.K, p.box) ||
      !encode_rows(encode, &tw, a.codes, a.experts * two * a.N, a.K, BM))
    return cudaErrorInvalidValue;
  auto kern = a.gated ? mx4_gemm_kernel<true> : mx4_gemm_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT);
  if (e != cudaSuccess) return e;
  int64_t most = a.starts ? (a.M / p.ts + a.experts + 1) * p.n_tiles : items;   // items at most
  int64_t grid = sms / p.split;
  if (most < grid) grid = most;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(grid * p.split));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = l.total;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)p.split, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tx, tw, p);
}

cudaError_t read_clear_mx4_status(int *status, cudaStream_t s) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_mx4_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_mx4_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
  }
  *status = v;
  return cudaSuccess;
}

}  // namespace qmm
