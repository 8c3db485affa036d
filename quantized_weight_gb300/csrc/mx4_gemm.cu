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
// Roles of a CTA (one an SM, or two for the narrowest tiles, walking over items = weight tile x token tile):
//   warp 0     copies, a ring of stages (mbarriers: full by transaction bytes, empty by the MMAs' commit)
//   warp 1     TMEM allocation and the MMA issuer
//   warps 2-9  epilogue: an accumulator goes to registers at once, so that the next item's products can begin where TMEM
//              holds only one; then silu, rounding and stores
// Tiles have 64 to 256 tokens (cut_for says which).  Many tokens go to pairs of CTAs (cta_group::2): 256 weight rows by 256
// tokens, of which each CTA holds half.  One CTA's tile of 128 x 256 makes the tensor core read 12 KB of shared memory for
// 64 elements along K, while 12 KB come in, in the 128 cycles that the products take: 192 bytes a cycle of 128, which held
// it at 67 % of the tensor core's 10.3 PFLOP/s.  A pair reads and fills 8 KB each.
// A call with few items splits K over the CTAs of a cluster: each writes its partial tile into the shared memory of the CTA
// that owns the token, and the owner adds them up in the order of the ranks, so that the sum is the same every time.
//
// Measured: 8192 x 17408 x 5120 (bfloat16 out) 212 us, 6.9 PFLOP/s; what remains is the end of an item (its accumulator's
// way to registers, the next one's first scales) and, of 8 %, the stores.  1 x 151936 x 2048 29.5 us, 83 % of measured HBM.  Few
// and small items are bound by latency: 8 x 4096 x 4096 takes 7.2 us of a floor of 1.3.
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

using namespace mx4;
using namespace sm100;

constexpr int MMA_K = 64;
constexpr int EPI_WARP0 = 2, EPI_WARPS = 8;
constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);

struct Params {
  const uint8_t *xs, *ws;
  const int32_t *starts, *counts;          // null: one matrix, M rows
  void *y;
  int64_t M, N;                            // rows of x, rows of a matrix
  int n_tiles, most_tiles;                 // weight tiles of 128 rows (a pair: 256) of a matrix, token tiles at most
  int64_t w_scale_bytes;                   // of a matrix
  int k_tiles, k_stages, k_steps;          // scale tiles of a row, stages and MMAs along K
  int experts;
  int box;                                 // rows of x in a copy
  int stages;                              // ring depth
  int split;                               // CTAs of a cluster, each with a part of K
  unsigned long long test_wait_ns;         // test hook: the epilogues' first wait is for nothing, and runs out after so long
};

struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) s = 0, ph ^= 1u;
  }
};

template <bool BF16>
__device__ __forceinline__ void store(void *y, int64_t at, float v) {
  if constexpr (BF16)
    __stcs(static_cast<unsigned short *>(y) + at, __bfloat16_as_ushort(__float2bfloat16_rn(v)));
  else
    __stcs(static_cast<float *>(y) + at, v);
}

// silu(z) * u of z from kFar up, in six instructions for a bfloat16 result: the quick exponential does there, whose relative
// error is below 2^-22 of its own and |z| * 2^-23 of its argument's, 2^-16.9 in all.  A gated item's epilogue is as long as
// its products.
constexpr float kFar = -64.0f;
template <bool BF16>
__device__ __forceinline__ float gate(float z, float u) {
  float e, r;
  if constexpr (BF16)
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));     // 2^(-z log2(e))
  else
    e = expf(-z);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return z * r * u;
}

// Below, 1 + exp(z) is 1 and silu(z) * u = z * exp(z) * u, which a large u makes a whole result where exp(-z) is past float32
// already.  So exp(z) is taken by halves, the second one last: no step of z * h * u * h loses what the result has (h is not
// normal below -175, which costs the result 2^-140 at most).
__device__ __forceinline__ float gate_far(float z, float u) {
  const float h = expf(0.5f * z);
  return z * h * u * h;
}

// wait_bounded for an accumulator, which of a pair the other CTA's epilogue frees, too.  The tensor core stands still
// meanwhile, so the one warp that waits here tests for a while without sleeping (2 % of a gated prompt; the epilogue's eight
// warps doing so cost more than they gain).
template <bool CLUSTER>
__device__ __forceinline__ bool wait_soon(uint32_t bar, uint32_t parity, const WaitCtl &ctl) {
  for (int i = 0; i < 4000; i++) {
    if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_test(bar, parity)) return true;
    if (*ctl.abort) return false;
  }
  return wait_bounded(bar, parity, ctl) && (!CLUSTER || mbar_try_wait_cluster(bar, parity));
}

// TS: tokens of a tile.  CTAS 2: a pair of CTAs has a tile of 256 weight rows, 128 each, and each half of the tokens in its
// shared memory.
template <bool GATED, bool BF16, int TS, int CTAS>
__global__ void __launch_bounds__(NUM_THREADS, TS == 64 && !GATED ? 2 : 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                    const __grid_constant__ CUtensorMap tmap_xs, const __grid_constant__ CUtensorMap tmap_ws, const Params p) {
  constexpr int TWO = GATED ? 2 : 1;
  constexpr bool PAIR = CTAS == 2, SPLITS = TS == 64 && !PAIR;
  constexpr int SF_COLS = 2 * (8 * TWO + 16);                             // of scales: two places by turns
  constexpr int BUFS = 2 * TWO * TS + SF_COLS <= 512 ? 2 : 1;             // accumulators that TMEM holds
  constexpr int TMEM_COLS = BUFS * TWO * TS + SF_COLS <= 256 ? 256 : 512; // (256: room for the next call's)
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const Layout l = layout(GATED, TS, CTAS, p.stages, p.split, p.experts);
  float *red = reinterpret_cast<float *>(smem + l.ring);
  Item *listed = reinterpret_cast<Item *>(smem + l.ring + l.red);
  int32_t *starts = reinterpret_cast<int32_t *>(listed + LISTED), *counts = starts + p.experts, *before = counts + p.experts;
  const uint32_t bars = sbase + l.ring + l.red + l.list;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (MAX_STAGES + s); };
  auto acc_full = [&](int b) { return bars + 8 * (2 * MAX_STAGES + b); };
  auto acc_empty = [&](int b) { return bars + 8 * (2 * MAX_STAGES + 2 + b); };
  const uint32_t drain_bar = bars + 8 * (2 * MAX_STAGES + 4), never_bar = drain_bar + 8;
  uint8_t *tail = smem + l.ring + l.red + l.list + 8 * (2 * MAX_STAGES + 6);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tail);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
  uint32_t *fine = reinterpret_cast<uint32_t *>(tail + 8);       // [split]: that CTA's part is whole; of a pair: how it ended
  const WaitCtl ctl{abort_flag, &g_mx4_status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the CTA of its cluster (one that splits K, or a pair)
  const int rank = PAIR || (SPLITS && p.split > 1) ? (int)cluster_ctarank() : 0, cluster_log = PAIR ? 1 : SPLITS ? __ffs(p.split) - 1 : 0;
  const int part = PAIR ? 0 : rank, split_log = PAIR ? 0 : cluster_log, in_pair = PAIR ? rank : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; s++) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), CTAS * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    mbar_init(never_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmap_x);
    tma_prefetch_desc(&tmap_w);
  }
  if (warp == 1) tmem_alloc_for<CTAS>(smem_addr(tmem_slot), TMEM_COLS);
  if (SPLITS && warp == 0 && !p.starts && p.M <= TS) {
    // the weights of the first item begin to move into L2 (where later writes reach them, too) before the kernel before has ended
    const int nt = blockIdx.x >> cluster_log;
    const int k0 = (int)((int64_t)p.k_stages * part >> split_log), k1 = (int)((int64_t)p.k_stages * (part + 1) >> split_log);
    if (lane < TWO * p.stages && k0 + lane / TWO < k1)
      tma_prefetch_2d(&tmap_w, (k0 + lane / TWO) * (BK / 2), (int)((lane % TWO) * p.N + (int64_t)nt * BM));
  }
  pdl_wait();
  // (by the warp that has allocated: the next launch's CTAs may begin once one thread of each CTA says so, and one that took
  // this SM's tensor memory first would wait for this launch, and this launch for the memory)
  if (warp == 1) pdl_launch_dependents();
  if (warp == 0) {
    // the experts' rows, made to fit x, and the token tiles before each
    uint32_t sum = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32 * 4) {
      int s4[4], c4[4];                                // (loads that wait for nothing between them)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int e = e0 + 32 * q + lane;
        s4[q] = p.starts && e < p.experts ? p.starts[e] : 0;
        c4[q] = p.starts ? (e < p.experts ? p.counts[e] : 0) : (int)p.M;
      }
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int e = e0 + 32 * q + lane;
        if (e - lane >= p.experts) break;
        int start = s4[q];
        int64_t count = c4[q];
        if (start < 0 || start >= p.M || start % kMxRows != 0 || count < 0) start = 0, count = 0;
        if (count > p.M - start) count = p.M - start;
        uint32_t at = e < p.experts ? (uint32_t)((count + TS - 1) / TS) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, at, o);
          if (lane >= o) at += v;
        }
        at = min(sum + at, (uint32_t)p.most_tiles);    // (more only where experts share rows)
        if (e < p.experts) starts[e] = start, counts[e] = (int)count, before[e + 1] = (int)at;
        sum = __shfl_sync(0xFFFFFFFFu, at, 31);
      }
    }
    if (lane == 0) before[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (PAIR)
    cluster_sync();                            // (its barriers are waited for and arrived at by both)
  else if (SPLITS && p.split > 1)
    cluster_arrive();

  const int items = before[p.experts] * p.n_tiles;
  const int first = blockIdx.x >> cluster_log, step = gridDim.x >> cluster_log;
  // this CTA's stages of K
  const int ks0 = (int)((int64_t)p.k_stages * part >> split_log), ks1 = (int)((int64_t)p.k_stages * (part + 1) >> split_log);

  // the tokens that a tile's MMAs take
  auto tokens_of = [](int rows) { return PAIR ? (rows + 31) & ~31 : (rows + 15) & ~15; };
  auto item_at = [&](int i) {
    Item it;
    // the last expert whose items begin at or before i, by the whole warp
    int lo = -1;
    for (int e = lane; e - lane < p.experts; e += 32)
      lo += __popc(__ballot_sync(0xFFFFFFFFu, e < p.experts && before[e] * p.n_tiles <= i));
    const int tiles = before[lo + 1] - before[lo], j = i - before[lo] * p.n_tiles;
    const int nt = tiles == 1 ? j : j / tiles, m0 = (j - nt * tiles) * TS;
    it.expert = lo;
    it.n0 = nt * (CTAS * BM);
    it.row = starts[lo] + m0;
    it.rows = min(counts[lo] - m0, TS);
    return it;
  };

  // (finding one takes some 600 cycles, which each role would else spend between two items)
  for (int t = warp; t < LISTED && first + t * step < items; t += NUM_THREADS / 32) {
    const Item it = item_at(first + t * step);
    if (lane == 0) listed[t] = it;
  }
  __syncthreads();

  // (a reduction over equal values leaves its result in a uniform register, where the operands of copies and MMAs have to
  // be: from ordinary registers a stage's instructions took 1600 cycles to issue)
  auto uniform = [](uint32_t v) { return __reduce_max_sync(0xFFFFFFFFu, v); };
  auto uniform64 = [&](uint64_t v) { return (uint64_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v); };
  // (a pair's copies complete on the first CTA's barriers)
  const uint32_t base0 = uniform(sbase), stage_bytes = uniform(l.stage), tmem0 = uniform(tmem), empty0 = uniform(empty(0));
  const uint32_t full0 = uniform(PAIR ? mapa_shared(full(0), 0) : full(0)), box_bytes = uniform(p.box * (BK / 2));
  Ring ring;                                   // (of the copying and the issuing warp)
  int issued = 0;                              // stages so far
  int ready = 0;                               // stages known to have landed
  int local = 0;                               // items so far
  // (test hook: the copying warp of one CTA of each pair, the first or the second by turns, is one that gave up)
  bool ok = !(PAIR && p.test_wait_ns != 0 && warp == 0 && in_pair == (first & 1));
  for (int i = first; i < items; i += step, local++) {
    const Item it = local < LISTED ? listed[local] : item_at(i);
    const int64_t n0 = it.n0 + in_pair * BM;   // of this CTA
    const int buf = local & (BUFS - 1);
    const uint32_t use = (uint32_t)(BUFS == 2 ? local >> 1 : local) & 1;
    // tokens of the tile before its first: its scale tile may begin 64 rows earlier
    const int shift = (int)(it.row & (kMxRows - 1));
    const int sf_tiles = (shift + it.rows + kMxRows - 1) / kMxRows;
    if (warp == 0) {
      // -------------------------------------------------------- copies
      if (ok) {
        // (a pair's second CTA has the second half of the tokens, and its weight rows may lie past the last)
        const uint32_t boxes = PAIR ? 1 : uniform((it.rows + p.box - 1) / p.box);
        const uint32_t row = uniform((uint32_t)it.row + in_pair * (tokens_of(it.rows) / 2));
        const int64_t w_tile = PAIR ? min(n0 >> 7, (p.N - 1) >> 7) : n0 >> 7;
        const uint32_t w_row = uniform((uint32_t)((int64_t)it.expert * TWO * p.N + n0)), w_next = (uint32_t)p.N;
        const uint64_t ws = uniform64(reinterpret_cast<uint64_t>(p.ws) + (int64_t)it.expert * TWO * p.w_scale_bytes +
                                      w_tile * p.k_tiles * kMxTileBytes);
        const uint64_t xs = uniform64(reinterpret_cast<uint64_t>(p.xs) + ((int64_t)it.row >> 7) * p.k_tiles * kMxTileBytes);
        const uint32_t two_tiles = uniform(sf_tiles == 2);
        const uint32_t ws_tile = uniform((uint32_t)(((int64_t)it.expert * TWO * ((p.N + 127) >> 7) + w_tile) * p.k_tiles));
        const uint32_t ws_next = uniform((uint32_t)(((p.N + 127) >> 7) * p.k_tiles)), xs_tile = uniform((uint32_t)(((int64_t)it.row >> 7) * p.k_tiles));
        const uint32_t each = l.a + boxes * box_bytes, sfs = TWO + 1 + two_tiles;
        for (int ks = ks0; ks < ks1; ks++, issued++, ring.next(p.stages)) {
          if (!__all_sync(0xFFFFFFFFu, wait_bounded(empty(ring.s), ring.ph ^ 1, ctl))) { ok = false; break; }
          const uint32_t now = uniform(ring.s | (uint32_t)min(2, p.k_tiles - 2 * ks) << 4 | (uint32_t)ks << 8);
          const uint32_t slot = now & 15, k = now >> 8, sf = (now >> 4 & 15) * kMxTileBytes;
          const uint32_t base = base0 + slot * stage_bytes, bar = full0 + 8 * slot;
          if (PAIR) {
            if (elect_one()) {
              if (in_pair == 0) mbar_arrive_expect_tx(full(0) + 8 * slot, 2 * (uint32_t)l.stage);
#pragma unroll
              for (int g = 0; g < TWO; g++) {
                tma_load_2d_pair(base + g * BM * (BK / 2), &tmap_w, k * (BK / 2), w_row + g * w_next, bar);
                tma_load_2d_pair(base + l.a + l.b + g * 2 * kMxTileBytes, &tmap_ws, 0, ws_tile + g * ws_next + 2 * k, bar);
              }
              tma_load_2d_pair(base + l.a, &tmap_x, k * (BK / 2), row, bar);
#pragma unroll
              for (int t = 0; t < (TS > kMxRows ? 2 : 1); t++)
                tma_load_2d_pair(base + l.a + l.b + l.sfa + t * 2 * kMxTileBytes, &tmap_xs, 0, xs_tile + t * p.k_tiles + 2 * k, bar);
            }
          } else if (elect_one()) {
            mbar_arrive_expect_tx(bar, each + sfs * sf);
#pragma unroll
            for (int g = 0; g < TWO; g++) {
              tma_load_2d(base + g * BM * (BK / 2), &tmap_w, k * (BK / 2), w_row + g * w_next, bar);
              bulk_copy(base + l.a + l.b + g * 2 * kMxTileBytes, ws + g * p.w_scale_bytes + (uint64_t)k * 2 * kMxTileBytes, sf, bar);
            }
            tma_load_2d(base + l.a, &tmap_x, k * (BK / 2), row, bar);
            bulk_copy(base + l.a + l.b + l.sfa, xs + (uint64_t)k * 2 * kMxTileBytes, sf, bar);
            if (two_tiles)
              bulk_copy(base + l.a + l.b + l.sfa + 2 * kMxTileBytes, xs + ((uint64_t)p.k_tiles + 2 * k) * kMxTileBytes, sf, bar);
            for (uint32_t b = 1; b < boxes; b++)
              tma_load_2d(base + l.a + b * box_bytes, &tmap_x, k * (BK / 2), row + b * p.box, bar);
          }
          __syncwarp();
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- products
      if (ok && in_pair == 0)
        ok = __all_sync(0xFFFFFFFFu, wait_soon<PAIR>(acc_empty(buf), use ^ 1, ctl));
      if (ok && in_pair == 0) {
        tc_fence_after();
        const uint32_t what = uniform((uint32_t)(tokens_of(it.rows) >> 3) | (uint32_t)(shift >> 5) << 8 | (uint32_t)buf << 10);
        const uint32_t id = idesc_mxf4(CTAS * BM, 0) | (what & 255) << 17;
        const uint32_t off = TS % kMxRows == 0 ? 0 : what >> 8 & 3;
        const uint32_t d = tmem0 + (what >> 10) * (TWO * TS), sf0 = tmem0 + BUFS * TWO * TS;
        const uint64_t ops = smem_desc_sw128(0), scales = smem_desc_scales(0);
        const uint32_t at0 = base0 >> 4, stage16 = stage_bytes >> 4;
        for (int ks = ks0; ks < ks1; ks++, issued++, ring.next(p.stages)) {
          // (one reduction a stage: its slot, whether sums are there already, its MMAs; before the wait, which takes as long)
          const uint32_t now = uniform(ring.s | (uint32_t)(ks > ks0) << 8 | (uint32_t)min(BK / MMA_K, p.k_steps - ks * (BK / MMA_K)) << 16);
          if constexpr (!SPLITS) {
            if (!__all_sync(0xFFFFFFFFu, wait_bounded(full(ring.s), ring.ph, ctl))) { ok = false; break; }
            tc_fence_after();
          } else if (ready == 0) {
            // a lane a stage from this one on: one test (of some 150 cycles) says how many have landed
            const int slot = ring.s + lane, wrap = slot >= p.stages;
            const bool landed = lane < p.stages && mbar_test(full(slot - wrap * p.stages), ring.ph ^ wrap);
            ready = __ffs(~__ballot_sync(0xFFFFFFFFu, landed)) - 1;
            if (ready == 0) {
              if (!__all_sync(0xFFFFFFFFu, wait_bounded(full(ring.s), ring.ph, ctl))) { ok = false; break; }
              ready = 1;
            }
            tc_fence_after();
          }
          if constexpr (SPLITS) ready--;
          const uint32_t slot = now & 255, more = now >> 8 & 1, steps = now >> 16;
          // scales: by turns in two places, 8 columns a weight tile (4 a scale tile) and 16 for the tokens
          const uint32_t sfa = sf0 + (slot & 1) * (SF_COLS / 2), sfb = sfa + 8 * TWO;
          const uint32_t at = at0 + slot * stage16, bar = empty0 + 8 * slot;
          const uint64_t ad = ops | at, bd = ops | (at + (l.a >> 4));
          const uint64_t sd = scales | (at + ((l.a + l.b) >> 4)), td = scales | (at + ((l.a + l.b + l.sfa) >> 4));
          // (where the tokens' second scale tile was not loaded, no MMA looks at what is copied from its place)
          auto scales_of = [&](int a) {
#pragma unroll
            for (int g = 0; g < TWO; g++) tmem_cp_32x16b<CTAS>(sfa + g * 8 + a * 4, sd + (g * 2 + a) * (kMxTileBytes / 16));
#pragma unroll
            for (int t = 0; t < (TS > kMxRows ? 2 : 1); t++) tmem_cp_32x16b<CTAS>(sfb + a * 8 + 4 * t, td + (2 * t + a) * (kMxTileBytes / 16));
          };
          auto products_of = [&](int j) {
#pragma unroll
            for (int g = 0; g < TWO; g++)
              umma_mxf4<CTAS>(d + g * TS, ad + g * (BM * (BK / 2) / 16) + 2 * j, bd + 2 * j, j & 1 ? id | kSecondScales : id,
                              sfa + g * 8 + (j >> 1) * 4, sfb + (j >> 1) * 8 + off, j > 0 ? 1u : more);
          };
          if (elect_one()) {
            // two MMAs a scale tile; the last stage may have fewer
            scales_of(0);
            products_of(0);
            if (steps > 1) products_of(1);
            if (steps > 2) {
              scales_of(1);
              products_of(2);
              if (steps > 3) products_of(3);
            }
            commit_mxf4<CTAS>(bar);
          }
          __syncwarp();
        }
        if (ok && elect_one()) commit_mxf4<CTAS>(acc_full(buf));
        __syncwarp();
      }
    } else {
      // -------------------------------------------------------- epilogue
      const int q = warp & 3, half = (warp - EPI_WARP0) >> 2;      // TMEM lane quarter; which half of the tile's tokens
      const int r = q * 32 + lane;
      const int64_t n = n0 + r;
      if (p.test_wait_ns != 0 && local == 0) ok = __all_sync(0xFFFFFFFFu, wait_bounded(never_bar, 0, ctl, p.test_wait_ns));
      if (ok) ok = __all_sync(0xFFFFFFFFu, wait_bounded(acc_full(buf), use, ctl));
      if (ok) {
        tc_fence_after();
        // everything to registers, so that the next item's products can begin
        constexpr int CHUNKS = TS / 32;                            // of 16 tokens, a warp
        uint32_t v[CHUNKS][TWO][16];
        const int c0 = half * (TS / 2), left = it.rows - c0;       // tokens of this half
        const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + buf * TWO * TS + c0;
#pragma unroll
        for (int c = 0; c < CHUNKS; c++)
          if (16 * c < left) {
#pragma unroll
            for (int g = 0; g < TWO; g++) tmem_ld_32x32b_x16(d + g * TS + 16 * c, v[c][g]);
          }
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {                       // (an arrival a thread, and of a pair from the other CTA, took 1 us)
          if (in_pair == 0)
            mbar_arrive(acc_empty(buf));
          else
            mbar_arrive_cluster(mapa_shared(acc_empty(buf), 0));
        }
        if (SPLITS && p.split > 1) {
          if (local == 0) cluster_wait();      // (no CTA writes into one that has not begun)
          // token t of the tile belongs to rank t % split, as its row t / split
          const int sh = __ffs(p.split) - 1;
          const uint32_t mine = smem_addr(red + (part * (TS >> sh) * TWO) * BM + r);
#pragma unroll
          for (int c = 0; c < CHUNKS; c++)
#pragma unroll
            for (int j = 0; j < 16; j++) {
              const int t = 16 * c + j;
              if (t >= left) break;
#pragma unroll
              for (int g = 0; g < TWO; g++)
                st_cluster_f32(mapa_shared(mine + (((c0 + t) >> sh) * TWO + g) * BM * 4, t & (p.split - 1)), __uint_as_float(v[c][g][j]));
            }
        } else if (n < p.N) {
          if constexpr (GATED) {
            // a z below kFar (one test for 16) becomes 32, whose silu is 32, and its u what is then right
#pragma unroll
            for (int c = 0; c < CHUNKS; c++) {
              bool far = false;
#pragma unroll
              for (int j = 0; j < 16; j++) far = far || __uint_as_float(v[c][0][j]) < kFar;
              if (!far) continue;
#pragma unroll
              for (int j = 0; j < 16; j++) {
                const float z = __uint_as_float(v[c][0][j]);
                if (!(z < kFar)) continue;
                v[c][TWO - 1][j] = __float_as_uint(gate_far(z, __uint_as_float(v[c][TWO - 1][j])) * 0.03125f);
                v[c][0][j] = __float_as_uint(32.0f);
              }
            }
          }
          auto out = [&](int c, int j) {
            return GATED ? gate<BF16>(__uint_as_float(v[c][0][j]), __uint_as_float(v[c][TWO - 1][j])) : __uint_as_float(v[c][0][j]);
          };
          const int64_t step = p.N * (BF16 ? 2 : 4);
          char *at = static_cast<char *>(p.y) + ((int64_t)it.row + c0) * step + n * (BF16 ? 2 : 4);
#pragma unroll
          for (int c = 0; c < CHUNKS; c++) {
            if (16 * c + 16 <= left) {
#pragma unroll
              for (int j = 0; j < 16; j++, at += step) store<BF16>(at, 0, out(c, j));
            } else {
#pragma unroll
              for (int j = 0; j < 16; j++, at += step) {
                if (16 * c + j >= left) break;
                store<BF16>(at, 0, out(c, j));
              }
            }
          }
        }
      }
    }
    if (SPLITS && p.split > 1) {
      if (local == 0 && (warp < EPI_WARP0 || !ok)) cluster_wait();
      __syncthreads();                         // (every epilogue warp has sent its part, or none will)
      if (threadIdx.x < p.split) st_cluster_u32(mapa_shared(smem_addr(fine + part), threadIdx.x), *abort_flag ? 0u : 1u);
      __syncwarp();
      cluster_sync();
      bool whole = true;
      for (int s = 0; s < p.split; s++) whole = whole && fine[s] != 0;
      if (whole) {
        const int sh = __ffs(p.split) - 1, own = (it.rows - part + p.split - 1) >> sh;     // tokens of this CTA
        for (int x = threadIdx.x; x < own * BM; x += NUM_THREADS) {
          const int t = x / BM, r = x % BM;
          float sum[TWO];
#pragma unroll
          for (int g = 0; g < TWO; g++) {
            sum[g] = 0.0f;
            for (int s = 0; s < p.split; s++) sum[g] += red[((s * (TS >> sh) + t) * TWO + g) * BM + r];
          }
          if (GATED) sum[0] = sum[0] < kFar ? gate_far(sum[0], sum[TWO - 1]) : gate<BF16>(sum[0], sum[TWO - 1]);
          if (n0 + r < p.N) store<BF16>(p.y, ((int64_t)it.row + t * p.split + part) * p.N + n0 + r, sum[0]);
        }
      }
      __syncwarp();
      if (i + step < items) cluster_sync();    // (its neighbours read what the next item overwrites)
    }
  }
  if (SPLITS && p.split > 1 && local == 0) cluster_wait();
  bool gave_up = false;                        // some wait of the CTA, or of the pair
  if constexpr (PAIR) {
    // A stage that the MMAs have read has landed in both CTAs.
    if (warp == 0 && ok)
      for (int j = issued > p.stages ? issued - p.stages : 0; j < issued && ok; j++)
        ok = __all_sync(0xFFFFFFFFu, wait_bounded(empty(j % p.stages), (j / p.stages) & 1, ctl));
    tc_fence_before();
    __syncthreads();                           // (no role issues anything more, or gives up)
    // Each tells both how many stages it has copied, and whether a wait gave up.
    if (threadIdx.x < 2) st_cluster_u32(mapa_shared(smem_addr(fine + in_pair), threadIdx.x), (uint32_t)issued << 1 | (*abort_flag ? 1u : 0u));
    __syncwarp();
    cluster_sync();                            // (and of what follows, only where a wait gave up does any touch the other's memory)
    gave_up = (fine[0] | fine[1]) & 1;
    if (gave_up && warp == 0 && in_pair == 0) {
      // Every copy lands before any memory goes to others.  The first CTA's barriers have the bytes of both; of a stage that
      // only the second has copied they expect them now, and of one that it has not they do without.
      const int n0 = (int)(fine[0] >> 1), n1 = (int)(fine[1] >> 1), n = max(n0, n1);
      for (int j = max(0, n - p.stages); j < n; j++) {
        const uint32_t bar = full(j % p.stages);
        if (lane == 0 && j >= n0) mbar_arrive_expect_tx(bar, (uint32_t)l.stage);
        if (lane == 0 && j >= n1) mbar_complete_tx(bar, (uint32_t)l.stage);
        __syncwarp();
        wait_drain(bar, (j / p.stages) & 1);
      }
    }
  } else {
    // every copy lands before this CTA's memory goes to another
    if (warp == 0)
      for (int j = issued > p.stages ? issued - p.stages : 0; j < issued; j++) wait_drain(full(j % p.stages), (j / p.stages) & 1);
    tc_fence_before();
    __syncthreads();
    gave_up = *abort_flag != 0;
  }
  if (gave_up && warp == 1) {                  // (whichever wait gave up, MMAs may be in flight)
    if (in_pair == 0 && elect_one()) commit_mxf4<CTAS>(drain_bar);
    __syncwarp();
    wait_drain(drain_bar, 0);
  }
  if (PAIR && gave_up) {
    __syncwarp();
    cluster_sync();                            // (each one's memory is the other's, too, until both have ended)
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_for<CTAS>(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side

std::atomic<unsigned long long> g_test_wait_ns{0};

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

// Scale tiles, two at a time.
bool encode_scales(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m, const void *base, int64_t bytes) {
  const cuuint64_t dims[2] = {kMxTileBytes / 4, (cuuint64_t)(bytes / kMxTileBytes)};
  const cuuint64_t strides[1] = {kMxTileBytes};
  const cuuint32_t boxes[2] = {kMxTileBytes / 4, 2}, one[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), dims, strides, boxes, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

template <bool GATED, bool BF16, int TS, int CTAS>
cudaError_t launch_tile(const Mx4GemmArgs &a, Params p, int box, int64_t items, int64_t most, int sms, cudaStream_t s) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap tx, tw, txs{}, tws{};
  if (!encode_rows(encode, &tx, a.x_codes, a.M, a.K, box) ||
      !encode_rows(encode, &tw, a.codes, a.experts * (GATED ? 2 : 1) * a.N, a.K, BM))
    return cudaErrorInvalidValue;
  if (CTAS == 2 && (!encode_scales(encode, &txs, a.x_scales, mx4_scales_bytes(a.M, a.K)) ||
                    !encode_scales(encode, &tws, a.scales, a.experts * (GATED ? 2 : 1) * p.w_scale_bytes)))
    return cudaErrorInvalidValue;
  p.box = box;
  p.n_tiles = (p.n_tiles + CTAS - 1) / CTAS;
  p.most_tiles = (int)(a.M / TS + a.experts);
  // Parts of K where items leave SMs without work: two CTAs an SM with rings of half its shared memory (gated: one; and eight
  // to a cluster do not all find room).  A stage takes 320 ns (gated: 400), joining the parts 3 us: 8 x 4096 x 4096 8.7, 9.6,
  // 7.6, 7.2 us with 1, 2, 4, 8 parts, 8 x 5120 x 17408 23.4, 17.5, 14.2 us with 1, 2, 4, 8 x 12288 x 4096 9.3, 10.6 us with 1, 2.
  constexpr bool TWO_AN_SM = TS == 64 && CTAS == 1 && !GATED;
  const int64_t room = TWO_AN_SM ? 2 * sms : sms;
  p.split = 1;
  if (TS == 64 && CTAS == 1) {
    int64_t least = (int64_t)p.k_stages * (GATED ? 400 : 320);
    for (int split = 2; split <= (GATED ? 4 : MAX_SPLIT) && items * split <= room && p.k_stages >= split; split *= 2) {
      const int64_t cost = (int64_t)((p.k_stages + split - 1) / split) * (GATED ? 400 : 320) + 2900 + 50 * split;
      if (cost < least) least = cost, p.split = split;
    }
  }
  const bool two_an_sm = TWO_AN_SM && items * p.split > sms;
  p.stages = ring_stages(GATED, TS, CTAS, p.split, p.experts, two_an_sm);
  // (a part of K that is shorter than the ring leaves the next call's CTAs room to begin)
  const int part = (p.k_stages + p.split - 1) / p.split;
  if (items * p.split <= room && p.stages > part) p.stages = part;
  const int smem = layout(GATED, TS, CTAS, p.stages, p.split, p.experts).total;
  auto kern = mx4_gemm_kernel<GATED, BF16, TS, CTAS>;
  const int cluster = CTAS == 2 ? 2 : p.split;
  int64_t grid = (two_an_sm ? room : sms) / cluster;
  if (most < grid) grid = most;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(grid * cluster));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  // (the limit of shared memory is raised once a device, and once more where a launch says that it was lost with the context)
  static std::atomic<int> set_for{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool set = set_for.load(std::memory_order_relaxed) == dev + 1;
  for (int pass = 0;; pass++) {
    if (!set || pass > 0) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT);
      if (e != cudaSuccess) return e;
      set_for.store(dev + 1, std::memory_order_relaxed);
    }
    e = cudaLaunchKernelEx(&cfg, kern, tx, tw, txs, tws, p);
    if (!(e == cudaErrorInvalidValue && set && pass == 0)) return e;
    (void)cudaGetLastError();
  }
}

// How a call is cut: tokens of a tile, by one CTA (128 weight rows) or a pair (256), and about how many items that makes.
struct Cut {
  int ts, ctas;
  int64_t items;
};

// A stage of 256 elements takes so many ns, an item's beginning and end so many more, and the SMs take items in rounds: wide
// tiles and pairs where there are many tokens, narrow ones where those fill the SMs better.  Measured, us, for tiles of 64,
// 128, 192, 256 tokens and pairs with 256: 8192 x 8192 x 8192: 313, 270, 211, 176, 153; 1024 x 6144 x 2048 (float32): 15.8,
// 13.1, 11.8, 14.7, 14.6; 256 x 4096 x 4096: 9.2, 9.1, 9.9, 10.9, 11.3; 4096 x 4096 x 1024: 18.8, 15.8, 13.9, 13.9, 17.2.  8191
// tokens by 6 of 64 experts of 2048 x 1408: 129, 103, 90, 86, 91; by 2 of 8 of 4096 x 4096: 175, 149, 114, 104, 96.  Gated, 64
// and 128 tokens and pairs with 128: 1024 x 4096 x 4096: 31, 20.5, 19.0; 8192 x 8192 x 8192: 691, 384, 303; 8191 tokens by 6 of 64
// experts of 1408 x 2048: 220, 131, 145, of 1536 x 4096: 434, 251, 228; by 8 of 128 of 768 x 2048: 164, 100, 110
// (where the rule takes pairs: its gated figures are of an earlier state, these times come to 417 and 900 ns for 128 tokens, 287
// and 2100 for pairs).
Cut cut_for(bool gated, const Mx4GemmArgs &a, int sms) {
  // experts that are met and rows of each, about
  const int64_t met = a.starts ? (a.routed < a.experts ? (a.routed > 1 ? a.routed : 1) : a.experts) : 1;
  const int64_t rows = a.starts ? (a.routed + met - 1) / met : a.M;
  const double stages = (double)((a.K + BK - 1) / BK);
  struct { int ts, ctas; double stage, item; } const ways[2][5] = {
      {{64, 1, 310, 500}, {128, 1, 320, 700}, {192, 1, 335, 1050}, {256, 1, 355, 1400}, {256, 2, 280, 2100}},
      {{64, 1, 400, 400}, {128, 1, 450, 500}, {128, 2, 325, 1300}}};
  Cut best{0, 1, 0};
  double least = 0;
  for (const auto &w : ways[gated]) {
    if (w.ts == 0) break;
    if (w.ts > 64 && 2 * rows <= w.ts) continue;       // (mostly empty)
    // (an expert's last tile is half empty on average)
    const double each = (double)rows / w.ts + 0.5, tiles = a.starts ? met * (each > 1 ? each : 1) : (double)((rows + w.ts - 1) / w.ts);
    const double items = tiles * (double)((a.N + BM * w.ctas - 1) / (BM * w.ctas));
    double rounds = items * w.ctas / sms;
    rounds = rounds < 1 ? 1 : rounds < 1e9 ? (double)(int64_t)(rounds + 0.999) : rounds;
    const double cost = rounds * (stages * w.stage + w.item);
    if (best.ts == 0 || cost < least) best = {w.ts, w.ctas, (int64_t)items}, least = cost;
  }
  if (best.items < 1) best.items = 1;
  return best;
}

template <bool GATED, bool BF16>
cudaError_t launch_type(const Mx4GemmArgs &a, const Params &p, cudaStream_t s) {
  const int sms = kv_max_ctas(1);
  const Cut c = cut_for(GATED, a, sms);
  const int64_t n_tiles = (p.n_tiles + c.ctas - 1) / c.ctas;
  const int64_t most = (a.starts ? a.M / c.ts + a.experts : (a.M + c.ts - 1) / c.ts) * n_tiles;      // items at most
  const bool few = a.starts ? a.routed <= 16 * a.experts : a.M <= 16;
  if (c.ts == 64) return launch_tile<GATED, BF16, 64, 1>(a, p, few ? 16 : 64, c.items, most, sms, s);
  if (c.ctas == 2) {
    if constexpr (GATED) return launch_tile<true, BF16, 128, 2>(a, p, 64, c.items, most, sms, s);
    return launch_tile<false, BF16, 256, 2>(a, p, 128, c.items, most, sms, s);
  }
  if (GATED || c.ts == 128) return launch_tile<GATED, BF16, 128, 1>(a, p, 128, c.items, most, sms, s);
  if (c.ts == 192) return launch_tile<false, BF16, 192, 1>(a, p, 192, c.items, most, sms, s);
  return launch_tile<false, BF16, 256, 1>(a, p, 256, c.items, most, sms, s);
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4GemmArgs &a, cudaStream_t s) {
  Params p{};
  p.xs = static_cast<const uint8_t *>(a.x_scales), p.ws = static_cast<const uint8_t *>(a.scales);
  p.starts = a.starts, p.counts = a.counts, p.y = a.y, p.M = a.M, p.N = a.N;
  p.n_tiles = (int)((a.N + BM - 1) / BM);
  p.w_scale_bytes = mx4_scales_bytes(a.N, a.K);
  p.k_tiles = (int)mx4_k_tiles(a.K), p.k_stages = (int)((a.K + BK - 1) / BK), p.k_steps = (int)((a.K + MMA_K - 1) / MMA_K);
  p.experts = (int)a.experts;
  p.test_wait_ns = g_test_wait_ns.exchange(0, std::memory_order_relaxed);
  if (a.gated) return a.bf16 ? launch_type<true, true>(a, p, s) : launch_type<true, false>(a, p, s);
  return a.bf16 ? launch_type<false, true>(a, p, s) : launch_type<false, false>(a, p, s);
}

void set_mx4_test_wait(unsigned long long limit_ns) { g_test_wait_ns.store(limit_ns, std::memory_order_relaxed); }

int mx4_gemm_tile(const Mx4GemmArgs &a) {
  const Cut c = cut_for(a.gated, a, kv_max_ctas(1));
  return c.ts | (c.ctas == 2 ? 1024 : 0);
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
