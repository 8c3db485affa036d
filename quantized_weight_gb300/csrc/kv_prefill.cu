// kv_prefill.cu -- attention over the 4-bit cache for many queries a request
// (prompts and their chunks), bfloat16, on tcgen05.
//
// An item is (request, kv head, up to NQ tiles of 128 rows of q), a row being a
// (query token, query head of the group) pair; it walks the keys that its rows see in
// blocks of KB tokens with a running maximum and sum:
//
//   S = Q K^T (TMEM) -> P = exp2(c S - m), binary16, over S (TMEM) -> O += P V (TMEM)
//
// Roles of the persistent CTA, one an SM (16 warps):
//   warp 0           TMEM and the MMA issue (one thread's)
//   warp 1           items, from a ticket counter (longest first within a request)
//   warps 2, 3       the cache's tiles of a block, keys and values, to shared
//                    memory as they are (cp.async; a tile without a page: zeros)
//   warps 4-7, 8-11  softmax of row tile 0 and 1, a row a thread: maximum,
//                    exponentials, P, O's rescaling, and the tile's q and output
//   warps 12-15      codes to binary16: keys, and values transposed (heads of
//                    256 have one row tile: warps 8-11 then take the keys)
// The two row tiles alternate: while one tile's softmax runs, the tensor core
// has the other's products.  With one row tile (heads of 256, or the rest of a request) the
// blocks alternate instead, between the same two score buffers.  Step i of an item uses score
// buffer i % 2, and S(i + 2) is issued right after PV(i): it overwrites P(i),
// which that product has read by then, since MMAs execute in order.
// The converting warps finish keys of block n and values of block n - 1 as one
// phase, so that the MMA warp waits once a block for both (a look at a barrier
// takes it some 250 cycles, however long it has been complete).
//
// Shared memory holds the operands K-major with the 128-byte swizzle.  The cache's
// row order (kv_layout.cuh) is the order of a tile's tokens in both key rows and
// value columns, so nothing is shuffled: a key word is eight elements of a row, and the words of four
// token quads at one element are two 16-byte runs of tokens.  The order inside a
// tile shows only in the mask.
//
// Precision: q is exact in binary16 after a power of two per row; keys and values are s * q + b
// rounded once to binary16, keys as a 16th of themselves, which is in range for all finite s and b.  Values
// stand as they are, for their low end; an item that meets coefficients with which one could pass
// 65504 is done a second time with a 16th of its values (a look at every coefficient of a block: 158.7 against 156.4 us
// for the prompt below; a masked value may not become infinite, since 0 times it is not 0).  P is
// rounded to binary16 at 2^7 to 2^15 of the largest weight, which keeps 11 bits of weights down to 2^-21 of it (a
// long context has many such beside a large one) and multiples of 2^-31 below; the reference
// maximum follows the true one only when that has grown by 2^8, so O is seldom
// rescaled; sums and accumulators are float32.
//
// Bound: 4 * D flops a row and key on the tensor cores (1024 cycles a step of 128 rows and 128 keys at D = 128).  Measured: a
// prompt of 4096 tokens, 32 query and 8 kv heads of 128, 158 us: 44 % of the measured matrix rate; chunks over 700 to 9000
// tokens, 16 and 4 heads of 256, 305 us: 39 %.  By its own clock a step takes some 2100 cycles: issue of its 16 MMAs 1300 (80
// each; unrolled and rolled alike), waits 700; the softmax of a tile (2200 to 2600 cycles of columns, 850 of the mask's test and
// the tail, 1050 of waits) and the conversion (3000 of the 4200 a block of two steps) are as long, so that no role has slack.
// Slower, and gone: conversion from global memory (keys 1700 and values 1250 cycles, but 950 and 1050 for their loads:
// 176 us), a wait by one lane of a warp (241 us), rolled MMA loops (188 against 179 us), TMEM loads of scores ahead (153 against
// 155 us here, slower for heads of 256).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "bounded_wait.cuh"
#include "kv_attend.h"
#include "kv_launch.h"
#include "kv_layout.cuh"
#include "qmm_device.cuh"
#include "sm100_ptx.cuh"

namespace qmm {

__device__ int g_kv_status = 0;   // QMM_OK or QMM_ERR_DEVICE_TIMEOUT (-6)

namespace {

using namespace sm100;

constexpr int QROWS = 128;                       // rows of a q tile (MMA M)
constexpr int MMA_WARP = 0, ITEM_WARP = 1, COPY_WARP0 = 2, SOFT_WARP0 = 4, DQ_WARP0 = 12;
constexpr int ITEM_READERS = 15;                 // warps that take every item: all but the one that hands them out
// Four warpgroups: 128 registers a thread, which every role fits in.
// Shared memory leaves the L1 cache a few KB, so that spilled registers would come back from L2.
constexpr int THREADS = 32 * 16;
constexpr int ITEM_SLOTS = 3;
constexpr float GROW = 8.0f;                     // log2 by which scores may exceed the reference maximum
constexpr float P_EXP = 7.0f;                    // P is 2^7 at the reference maximum (2^15 at most); l and O carry the factor, too

struct Params {
  KvAttendArgs a;
  KvGeom g;
  int ratio;
  unsigned long long test_wait_ns;  // test hook: a wait of every CTA runs out after so long
};
std::atomic<unsigned long long> g_test_wait_ns{0};

struct Item {
  int b, kvh, r0, rows;             // rows r0 .. r0 + rows - 1 of the request
  int tiles;                        // row tiles (1 or 2); 0: no more items
  int blk0, blocks;                 // blocks of keys
  int vlo, vhi;                     // tokens that any row sees
  int flo, fhi;                     // tokens that all rows see
  int base, hi, cu0;                // position of the first query; tokens that can be read; its token
  int vexp;                         // values stand in shared memory divided by 2^vexp
};

template <int D_, int G_>
struct Cfg {
  static constexpr int D = D_, G = G_;
  static constexpr int NQ = D == 256 ? 1 : 2;              // row tiles
  static constexpr int KB = D == 256 ? 64 : 128;           // keys a block
  static constexpr int TILE = 16 * D + 128 * G;
  static constexpr int Q_BYTES = QROWS * D * 2, KV_BYTES = KB * D * 2;
  static constexpr int OFF_K = NQ * Q_BYTES, OFF_V = OFF_K + 2 * KV_BYTES, OFF_RAW = OFF_V + 2 * KV_BYTES;
  static constexpr int HALF = 8 * D + 64 * G;              // a tile's keys or values in the cache: codes, coefficients
  static constexpr int RAW = KB / 16 * HALF, OFF_END = OFF_RAW + 2 * RAW;
  static constexpr int EDGES = 8;                          // blocks of an item that only some rows see: at most 3 at either end
  static constexpr int NOTES = EDGES * G * (KB / 32);      // a bit a (block, group, position)
  static constexpr int SMALL = 576 + 4 * NOTES * 4;
  static constexpr int SMEM = OFF_END + SMALL + 1024;      // the last for alignment
};

// barriers (8 bytes each).  FULL has eight, taken in turn: the warps that arrive on one may be five phases ahead of the last one
// complete (two blocks ahead, and an item of one block is two phases).
enum { S_FULL = 0, P_FULL = 2, PV_DONE = 4, Q_FULL = 6, FULL = 8, K_EMPTY = 16, V_EMPTY = 18, IT_FULL = 20,
       IT_EMPTY = IT_FULL + ITEM_SLOTS, DRAIN = IT_EMPTY + ITEM_SLOTS, IT_NEXT, RAW_FULL, RAW_EMPTY = RAW_FULL + 2,
       S_LAST = RAW_EMPTY + 2, DQ_SYNC = S_LAST + ITEM_SLOTS, NEVER, BARS };

__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from TMEM: lane = row, a 32-bit column = two consecutive k.
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// D f32, A and B binary16, both K-major
constexpr uint32_t idesc_f16(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two codes, exact: the low nibbles of a word's halves, and those above them.
// A code below exponent 25's leading one is 1024 + code (or 1024 + 16 code).
__device__ __forceinline__ uint32_t codes_lo(uint32_t x) { return hsub2(and_or(x, 0x000F000Fu, 0x64006400u), 0x64006400u); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t x) {
  return hfma2(and_or(x, 0x00F000F0u, 0x64006400u), 0x2C002C00u /* 1/16 */, 0xD400D400u /* -64 */);
}
// Keys stand in shared memory divided by 2^4: a nibble shifted to the top of the mantissa is the code times 2^-18 (a
// binary16 subnormal), so that one multiply-add with scale * 2^14 makes the value, where 2^14 scale is in range.  (Nibbles
// where they lie, divided by 2^10, take two instructions a word less, 2 % of the kernel, but keys below 2^-4 then lose
// bits to binary16's subnormals instead of keys below 2^-10.)
constexpr float KEY_UNIT = 16.0f;
// Values stand there as they are.  Scale and bias (magnitudes) from which on s * code + b may pass 65504: 15 * 2^11 + 2^15 does
// not.  A 16th of a value is in range whatever they are.
__device__ __forceinline__ bool large_value(uint32_t m) { return (m & 0xFFFFu) >= 0x6800u || m >= 0x78000000u; }
__device__ __forceinline__ void sts128(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ int token_of(int pos) { return 4 * ((pos & 7) >> 1) + 2 * (pos & 1) + (pos >> 3); }   // inverse of kv_row

// 16 bytes, or zeros for `bytes` 0 (nothing is read then)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

struct Phase {
  uint32_t v = 0;
  __device__ __forceinline__ uint32_t next() {
    const uint32_t p = v;
    v ^= 1u;
    return p;
  }
};

// A warp's wait.  What waits longer than a first look does it in one place for all: the roles' code has to stay in the
// instruction caches.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, WaitCtl{abort, &g_kv_status}));
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl &ctl) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_on(bar, parity, ctl.abort);
}

// The test hook's wait (out of line: it runs only when the hook is set).
__device__ __noinline__ void test_wait(uint32_t never_bar, WaitCtl ctl, unsigned long long limit_ns) {
  wait_bounded(never_bar, 0, ctl, limit_ns);
}

// One warp, the seldom path of the softmax: this lane's row of O (unless o_tm is all ones) and of the first `cols`
// columns of P (two binary16 values each) times f.  Not inlined, so that it takes no registers from the path that is run.
template <int D>
__device__ __noinline__ void rescale(uint32_t o_tm, uint32_t p_tm, int cols, float f) {
  tc_fence_after();
  if (o_tm != 0xFFFFFFFFu)
    for (int ch = 0; ch < D; ch += 16) {
      uint32_t w[16];
      tmem_ld_32x32b_x16(o_tm + ch, w);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; i++) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
      tmem_st_x16(o_tm + ch, w);
    }
  tmem_st_wait();
  const __half2 f16 = __float2half2_rn(f);
  for (int ch = 0; ch < cols; ch += 16) {
    uint32_t w[16];
    tmem_ld_32x32b_x16(p_tm + ch, w);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&w[i]), f16);
      w[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
    tmem_st_x16(p_tm + ch, w);
  }
}

template <int D, int G>
__global__ void __launch_bounds__(THREADS, 1) prefill_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D, G>;
  constexpr int KB = C::KB, NQ = C::NQ, TILE = C::TILE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_addr(smem);
  const uint32_t bars = sb + C::OFF_END;
  uint8_t *small = smem + C::OFF_END;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(small + 304);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(small + 308);
  int *noted = reinterpret_cast<int *>(small + 312);                         // [4] items: has notes
  volatile int *over = reinterpret_cast<int *>(small + 328);                 // [4] items: values may pass binary16's range
  uint32_t *kvalid = reinterpret_cast<uint32_t *>(small + 352);              // [8] blocks: tiles with a page
  Item *items = reinterpret_cast<Item *>(small + 384);                       // [ITEM_SLOTS]
  static_assert(8 * BARS <= 304 && 384 + ITEM_SLOTS * sizeof(Item) <= 576, "small arrays");
  uint32_t *notes = reinterpret_cast<uint32_t *>(small + 576);               // [4] items x NOTES: values taken out
  auto bar = [&](int i) { return bars + 8 * i; };
  const WaitCtl ctl{abort_flag, &g_kv_status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const KvAttendArgs &a = p.a;
  const int hkv = p.g.kv_heads;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ITEM_SLOTS; i++) {
      mbar_init(bar(IT_FULL + i), 1);
      mbar_init(bar(IT_EMPTY + i), ITEM_READERS);        // a warp an arrival
      mbar_init(bar(S_LAST + i), 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(bar(S_FULL + i), 1);
      mbar_init(bar(P_FULL + i), 128);
      mbar_init(bar(PV_DONE + i), 1);
      mbar_init(bar(Q_FULL + i), 128);
      mbar_init(bar(K_EMPTY + i), 1);
      mbar_init(bar(V_EMPTY + i), 1);
      mbar_init(bar(RAW_FULL + i), 32);
      mbar_init(bar(RAW_EMPTY + i), 128);
    }
    for (int i = 0; i < 8; i++) mbar_init(bar(FULL + i), NQ == 2 ? 128 : 256);
    mbar_init(bar(DRAIN), 1);
    mbar_init(bar(DQ_SYNC), 4);
    mbar_init(bar(NEVER), 1);                            // nothing arrives here (the test hook's wait)
    mbar_init(bar(IT_NEXT), NQ == 2 ? 4 : 8);            // a warp that converts an arrival
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_addr(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  // The next item, for every warp but the one that hands them out; it stays in shared memory until the warp lets go of it.
  int it_slot = 0;
  uint32_t it_ph = 0;
  auto next_item = [&]() -> const Item * {
    if (!warp_wait(bar(IT_FULL + it_slot), it_ph, ctl)) return nullptr;
    return items[it_slot].tiles > 0 ? items + it_slot : nullptr;
  };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(IT_EMPTY + it_slot));
    if (++it_slot == ITEM_SLOTS) it_slot = 0, it_ph ^= 1u;
  };

  if (warp == COPY_WARP0 || warp == COPY_WARP0 + 1) {
    // ------------------------------------------------------------ copies: a block's keys, or its values, as the cache has them
    const bool vals = warp != COPY_WARP0;
    const uint32_t raw = sb + C::OFF_RAW + (vals ? C::RAW : 0);
    const uint8_t *cache = static_cast<const uint8_t *>(a.cache) + 16 * lane;
    uint32_t ph = 1;
    int kb = 0;
    bool ok = true;
    while (const Item *ip = next_item()) {
      const Item &it = *ip;
      const int32_t *tab = a.table + it.b * a.max_blocks;
      auto page_of = [&](int blk) {                          // a tile a lane
        const int64_t tok = (int64_t)blk * KB + lane * 16;
        return lane < KB / 16 && tok < it.vhi ? tab[tok >> p.g.lg_page] : -1;
      };
      int pg = it.blocks > 0 ? page_of(it.blk0) : -1;
      for (int n = 0; n < it.blocks; n++, kb++, ph ^= 1u) {
        const int blk = it.blk0 + n, next = n + 1 < it.blocks ? page_of(blk + 1) : -1;
        const bool there = pg >= 0 && pg < p.g.pages;
        const uint32_t valid = __ballot_sync(0xffffffffu, there);
        const int64_t at = !there ? 0 : ((int64_t)pg * hkv + it.kvh) * p.g.head_bytes +
                                            ((((int64_t)blk * KB + lane * 16) & (p.g.page - 1)) >> 4) * TILE;
        if (!warp_wait(bar(RAW_EMPTY + vals), ph, ctl)) { ok = false; break; }
#pragma unroll 1
        for (int tl = 0; tl < KB / 16; tl++) {
          const uint8_t *src = cache + __shfl_sync(0xffffffffu, at, tl);
          const uint32_t bytes = (valid >> tl) & 1u ? 16u : 0u, dst = raw + tl * C::HALF;   // zeros without a page
#pragma unroll
          for (int c = 0; c < D / 64; c++) {
            const int q = c * 32 + lane;                     // values: eight lanes later read one quad of tokens each, from
                                                             // 8 different groups of banks
            cp_async16(dst + (vals ? q ^ ((q >> 3) & 3) : q) * 16, src + (vals ? 8 * D : 0) + c * 512, bytes);
          }
          if (lane < 4 * G) cp_async16(dst + 8 * D + lane * 16, src + 16 * D + (vals ? 64 * G : 0), bytes);
        }
        cp_async_wait_all();
        if (!vals && lane == 0) kvalid[kb & 7] = valid;
        mbar_arrive(bar(RAW_FULL + vals));
        pg = next;
      }
      if (!ok) break;
      release();
    }
  } else if (warp == ITEM_WARP) {
    // ------------------------------------------------------------ items
    unsigned *ticket = static_cast<unsigned *>(a.workspace) + (kKvMaxCtas - 1), *done = ticket - 1;
    int cb = 0;                               // requests before cb are behind this CTA's tickets
    int64_t cfirst = 0;                       // items before request cb
    uint32_t ph = 1, next = 1;
    int before = 0;                           // slot of the item before
    bool again = false;
    for (int slot = 0, n_item = 0;; n_item++) {
      // A ticket is drawn when the conversion for the item before it is done: earlier, CTAs would sit on items that others
      // could begin.
      if (!warp_wait(bar(IT_NEXT), next, ctl)) break;
      next ^= 1u;
      // The item before had values beyond binary16's range, and wrote nothing: once more, with a 16th of them.
      again = !again && n_item > 0 && over[(n_item - 1) & 3] != 0;
      unsigned t = 0;
      if (lane == 0 && !again) t = atomicAdd(ticket, 1u);
      t = __shfl_sync(0xffffffffu, t, 0);
      Item it{};
      for (; cb < a.B && !again; cb += 32) {
        const int b = cb + lane;
        int n = 0, len = 0, c0 = 0, tiles = 0;
        if (b < a.B) {
          len = max(0, a.lens[b]);
          c0 = a.cu ? max(0, min(a.cu[b], (int)a.tokens)) : b;
          n = a.cu ? max(c0, min(a.cu[b + 1], (int)a.tokens)) - c0 : 1;
          tiles = (n * p.ratio + NQ * QROWS - 1) / (NQ * QROWS);
        }
        int end = tiles * hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, end, o);
          if (lane >= o) end += u;
        }
        const int all = __shfl_sync(0xffffffffu, end, 31);
        if ((int64_t)t < cfirst + all) {
          const int k = (int)((int64_t)t - cfirst);
          const int src = __ffs(__ballot_sync(0xffffffffu, end > k)) - 1;
          const int idx = k - (__shfl_sync(0xffffffffu, end - tiles * hkv, src));
          n = __shfl_sync(0xffffffffu, n, src);
          len = __shfl_sync(0xffffffffu, len, src);
          c0 = __shfl_sync(0xffffffffu, c0, src);
          tiles = __shfl_sync(0xffffffffu, tiles, src);
          it.b = cb + src;
          it.kvh = idx % hkv;
          it.r0 = (tiles - 1 - idx / hkv) * NQ * QROWS;
          it.rows = min(NQ * QROWS, n * p.ratio - it.r0);
          it.tiles = it.rows > QROWS ? 2 : 1;
          it.base = len - n;
          it.cu0 = c0;
          it.hi = (int)min((int64_t)len, a.max_blocks << p.g.lg_page);
          const int64_t f = (int64_t)it.base + it.r0 / p.ratio, l = (int64_t)it.base + (it.r0 + it.rows - 1) / p.ratio;
          const int64_t lo = a.window > 0 ? f + 1 - a.window : 0;
          it.vlo = (int)max((int64_t)0, min(lo, (int64_t)it.hi));
          it.vhi = (int)max((int64_t)0, min(l + 1, (int64_t)it.hi));
          it.flo = a.window > 0 ? (int)max((int64_t)0, min(l + 1 - a.window, (int64_t)it.hi)) : 0;
          it.fhi = (int)max((int64_t)0, min(f + 1, (int64_t)it.hi));
          it.blk0 = it.vlo / KB;
          it.blocks = it.vhi > it.vlo ? (it.vhi + KB - 1) / KB - it.blk0 : 0;
          break;
        }
        cfirst += all;
      }
      if (!warp_wait(bar(IT_EMPTY + slot), ph, ctl)) break;
      if (lane == 0) {
        items[slot] = again ? items[before] : it;
        if (again) items[slot].vexp = 4;
        mbar_arrive(bar(IT_FULL + slot));
      }
      if (!again && it.tiles == 0) break;
      before = slot;
      if (++slot == ITEM_SLOTS) slot = 0, ph ^= 1u;
    }
    // the last CTA through leaves the counters zero for the next call
    if (lane == 0) {
      __threadfence();
      if (atomicAdd(done, 1u) == gridDim.x - 1) {
        *ticket = 0u;
        *done = 0u;
      }
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t id_s = idesc_f16(QROWS, KB), id_o = idesc_f16(QROWS, D);
    Phase pf[2], qf[2];
    int kb = 0, full = 0;                     // blocks and phases of FULL before this item
    // Descriptors differ in the start address alone (the low word, in 16-byte units).
    const uint64_t first = smem_desc_sw128(sb);
    const uint32_t desc0 = (uint32_t)first, desc_hi = (uint32_t)(first >> 32);
    // (a reduction over equal values leaves its result in a uniform register, where an MMA's operands have to be)
    auto uniform = [](uint32_t v) { return __reduce_max_sync(0xffffffffu, v); };
    auto desc = [&](uint32_t lo) { return (uint64_t)desc_hi << 32 | lo; };
    bool ok = true;
    const uint32_t tm0 = __shfl_sync(0xffffffffu, tmem, 0);
    while (const Item *ip = next_item()) {
      const Item &it = *ip;
      const int nt = __shfl_sync(0xffffffffu, it.tiles, 0), N = __shfl_sync(0xffffffffu, nt * it.blocks, 0);
      {
        int have = 0;                         // phases of FULL waited for: keys of blocks below it, values of those before them
        auto up_to = [&](int n) -> bool {
          for (; have < n; have++, full++)
            if (!warp_wait(bar(FULL + (full & 7)), (full >> 3) & 1, ctl)) return false;
          return true;
        };
        auto scores = [&](int i) {
          const int x = nt == 2 ? i & 1 : 0, kbuf = (kb + (nt == 2 ? i >> 1 : i)) & 1, buf = i & 1;
          const uint32_t kd = uniform(desc0 + ((C::OFF_K + kbuf * C::KV_BYTES) >> 4)), qd = uniform(desc0 + (x * C::Q_BYTES >> 4));
          const uint32_t dt = uniform(tm0 + buf * 128);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++)        // 64 elements a column of 128-byte rows, 16 a product
              umma_f16_ss(dt, desc(qd + (kk / 4) * (QROWS * 128 / 16) + 2 * (kk % 4)),
                          desc(kd + (kk / 4) * (KB * 128 / 16) + 2 * (kk % 4)), id_s, kk != 0);
            umma_commit(bar(S_FULL + buf));
            if (x == nt - 1) umma_commit(bar(K_EMPTY + kbuf));
            if (NQ == 2 && nt == 1 && i > 0 && i == N - 1) umma_commit(bar(S_LAST + it_slot));
          }
          __syncwarp();
        };
        for (int i = 0; i < 2 && i < N && ok; i++) {
          ok = up_to(nt == 2 ? 1 : i + 1) && (i >= nt || warp_wait(bar(Q_FULL + i), qf[i].next(), ctl));
          tc_fence_after();
          if (ok) scores(i);
        }
        for (int i = 0; i < N && ok; i++) {
          const int x = nt == 2 ? i & 1 : 0, j = nt == 2 ? i >> 1 : i, buf = i & 1, vbuf = (kb + j) & 1;
          // values of this block (and, with two row tiles, keys of the next), then P
          if (!up_to(j + 2) || !warp_wait(bar(P_FULL + buf), pf[buf].next(), ctl)) { ok = false; break; }
          tc_fence_after();
          const uint32_t vd = uniform(desc0 + ((C::OFF_V + vbuf * C::KV_BYTES) >> 4));
          const uint32_t ot = uniform(tm0 + 256 + x * D), pt = uniform(tm0 + buf * 128);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < KB / 16; kk++)
              umma_f16_ts(ot, pt + 8 * kk, desc(vd + (kk / 4) * (D * 128 / 16) + 2 * (kk % 4)), id_o,
                          (j | kk) != 0);
            umma_commit(bar(PV_DONE + x));
            if (x == nt - 1) umma_commit(bar(V_EMPTY + vbuf));
          }
          __syncwarp();
          if (i + 2 < N) {
            if (nt == 1) {
              if (!up_to(i + 3)) { ok = false; break; }
              tc_fence_after();
            }
            scores(i + 2);
          }
        }
      }
      if (!ok) break;
      kb += it.blocks;
      release();
    }
  } else if (warp >= (NQ == 2 ? DQ_WARP0 : SOFT_WARP0 + 4)) {
    // ------------------------------------------------------------ codes: keys
    // One warpgroup has both, or, where there is no second row tile, its softmax warps take the keys.
    auto codes = [&](auto with_keys, auto with_values) {
      constexpr bool KEYS = decltype(with_keys)::value, VALUES = decltype(with_values)::value;
      constexpr int NC = D >= 128 ? D / 128 : 1, WC = D >= 128 ? 4 : D / 32;   // pieces of WC words
      constexpr int GK = G / NC;                               // groups in a piece's 32 WC elements
      constexpr int PW = KB / 16 * NC * 2 / 4;                 // pieces a thread: a warp has 8 rows x 4 of them at a time,
      constexpr int TW = KB / 64;                              // and whole tiles in all
      const int w4 = warp & 3, t = lane & 3;
      // values
      constexpr int CB = D / 64;                               // blocks of 64 elements
      constexpr int GV = G > CB ? 2 : 1;                       // groups in one (group of 32: two)
      constexpr int UNITS = KB / 16 * CB * 8;                  // (tile, block, element % 8): the threads with work
      const int u = threadIdx.x & 127, g8 = u & 7, vc = (u >> 3) % CB, vt = (u >> 3) / CB;
      const bool act = u < UNITS;
      Phase ke[2], ve[2], kr, vr, together;
      // The four warps with the values, at one place.  Not a named barrier, whose wait has no end: one of them may have given
      // up a wait that the others passed.
      auto sync_values = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(DQ_SYNC));
        return warp_wait(bar(DQ_SYNC), together.next(), ctl);
      };
      ke[0].v = ke[1].v = ve[0].v = ve[1].v = 1;
      int kb = 0, full = 0, n_item = 0;                        // blocks, phases of FULL and items before
      bool ok = true;
      for (; const Item *ip = next_item(); n_item++) {
        const Item &it = *ip;
        // this item's notes, last used four items ago
        uint32_t *my_notes = notes + (n_item & 3) * C::NOTES;
        if constexpr (VALUES) {
          for (int i = u; i < C::NOTES; i += 128) my_notes[i] = 0u;
          if (u == 0) noted[n_item & 3] = 0, over[n_item & 3] = 0;
          if (!sync_values()) break;
        }
        const bool sixteenth = it.vexp != 0;
        uint32_t w[PW][WC], cf[PW][GK];
        auto take_keys = [&]() {
#pragma unroll
          for (int i = 0; i < PW; i++) {
            const int c = i / 2 % NC, row = (i & 1) * 8 + ((lane >> 2) & 1) * 4 + (lane >> 3);
            const uint8_t *s = smem + C::OFF_RAW + (w4 * TW + i / (2 * NC)) * C::HALF;
            if constexpr (WC == 4) {
              const uint4 v = *reinterpret_cast<const uint4 *>(s + ((c * 16 + row) * 4 + t) * 16);
              w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2 *>(s + (row * 4 + t) * 8);
              w[i][0] = v.x, w[i][1] = v.y;
            }
            const uint8_t *cp = s + 8 * D + (row * G + c * GK) * 4;
            if constexpr (GK == 1) {
              cf[i][0] = *reinterpret_cast<const uint32_t *>(cp);
            } else if constexpr (GK == 2) {
              const uint2 v = *reinterpret_cast<const uint2 *>(cp);
              cf[i][0] = v.x, cf[i][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4 *>(cp);
              cf[i][0] = v.x, cf[i][1] = v.y, cf[i][2] = v.z, cf[i][3] = v.w;
            }
          }
        };
        uint4 vw[4];
        uint32_t vf[16][GV];
        const uint8_t *raw_v = smem + C::OFF_RAW + C::RAW + (act ? vt : 0) * C::HALF;
        const uint8_t *coefs = raw_v + 8 * D + (G > CB ? 2 * vc : vc * G / CB) * 4;
        auto take_values = [&]() {
#pragma unroll
          for (int i = 0; i < 4; i++) vw[i] = *reinterpret_cast<const uint4 *>(raw_v + ((vc * 8 + g8) * 4 + (i ^ (g8 >> 1))) * 16);
#pragma unroll
          for (int r = 0; r < 16; r++) {
            if constexpr (GV == 1) {
              vf[r][0] = *reinterpret_cast<const uint32_t *>(coefs + r * G * 4);
            } else {
              const uint2 v = *reinterpret_cast<const uint2 *>(coefs + r * G * 4);
              vf[r][0] = v.x, vf[r][GV - 1] = v.y;
            }
          }
        };
        // a phase: keys of block n, values of the block before
        for (int n = 0; it.blocks > 0 && n <= it.blocks; n++, full++) {
          if (KEYS && n < it.blocks) {
            const int buf = (kb + n) & 1;
            if (!warp_wait(bar(RAW_FULL), kr.next(), ctl)) { ok = false; break; }
            take_keys();
            mbar_arrive(bar(RAW_EMPTY));
            if (!warp_wait(bar(K_EMPTY + buf), ke[buf].next(), ctl)) { ok = false; break; }
            {
              const uint32_t dst = sb + C::OFF_K + buf * C::KV_BYTES;
              uint32_t most = 0;
#pragma unroll
              for (int i = 0; i < PW; i++)
#pragma unroll
                for (int k = 0; k < GK; k++) {
                  // x + 0 x: infinities become NaN.  (An infinite key's score may be -inf, which the softmax would take for a
                  // key that is not there.)
                  cf[i][k] = hfma2(cf[i][k], 0u, cf[i][k]);
                  most = max(most, cf[i][k] & 0x7FFFu);
                }
              const bool large = __any_sync(0xffffffffu, most >= 0x4400u);   // a scale of 4 or more
#pragma unroll                                               // (rolled: chunks of heads of 256 in 320 instead of 295 us)
              for (int i = 0; i < PW; i++) {
                const int c = i / 2 % NC, row = (i & 1) * 8 + ((lane >> 2) & 1) * 4 + (lane >> 3);
                const int pos = (w4 * TW + i / (2 * NC)) * 16 + row;
#pragma unroll
                for (int k = 0; k < WC; k++) {
                  const uint32_t cc = cf[i][k / (WC / GK)], x = w[i][k];
                  const uint32_t b2 = hmul2(prmt(cc, cc, 0x3232), 0x2C002C00u /* 1/16 */);
                  // nibbles (0, 4), (1, 5), (2, 6), (3, 7) -> elements 0 .. 7 in order
                  uint32_t e04, e15, e26, e37;
                  if (!large) {
                    const uint32_t s2 = hmul2(prmt(cc, cc, 0x1010), 0x74007400u /* 2^14 */);
                    e04 = hfma2(x << 6 & 0x03C003C0u, s2, b2), e15 = hfma2(x << 2 & 0x03C003C0u, s2, b2);
                    e26 = hfma2(x >> 2 & 0x03C003C0u, s2, b2), e37 = hfma2(x >> 6 & 0x03C003C0u, s2, b2);
                  } else {
                    const uint32_t s2 = hmul2(prmt(cc, cc, 0x1010), 0x2C002C00u), y = x >> 8;
                    e04 = hfma2(codes_lo(x), s2, b2), e15 = hfma2(codes_hi(x), s2, b2);
                    e26 = hfma2(codes_lo(y), s2, b2), e37 = hfma2(codes_hi(y), s2, b2);
                  }
                  const int d = 32 * (WC * c + k) + 8 * t, ch = (d & 63) >> 3;
                  sts128(dst + (d >> 6) * (KB * 128) + pos * 128 + ((ch ^ (row & 7)) << 4), prmt(e04, e15, 0x5410),
                         prmt(e26, e37, 0x5410), prmt(e04, e15, 0x7632), prmt(e26, e37, 0x7632));
                }
              }
            }
          }
          if (VALUES && n > 0) {
            const int j = n - 1, blk = it.blk0 + j, buf = (kb + j) & 1;
            if (!warp_wait(bar(RAW_FULL + 1), vr.next(), ctl)) { ok = false; break; }
            if (sixteenth) {
#pragma unroll 1
              for (int i = u; i < KB * G; i += 128) {
                uint32_t *c = reinterpret_cast<uint32_t *>(smem + C::OFF_RAW + C::RAW + i / (16 * G) * C::HALF + 8 * D) + i % (16 * G);
                *c = hmul2(*c, 0x2C002C00u /* 1/16 */);
              }
              if (!sync_values()) { ok = false; break; }
            }
            take_values();
            // Tokens that no row sees become zeros, whatever the cache holds there.  Where only some rows see the block, a
            // non-finite coefficient must not meet the zero probability of a row that does not: it is taken out, too, and
            // noted for the rows that do.
            const bool edge = blk * KB < it.flo || (int64_t)(blk + 1) * KB > it.fhi;
            if (edge && act) {
              uint32_t out[GV] = {};                             // rows to zero, by group
              const int e = blk * KB < it.flo ? j : 4 + blk - it.fhi / KB;
#pragma unroll 1
              for (int r = 0; r < 16; r++) {
                const int64_t tok = (int64_t)blk * KB + vt * 16 + token_of(r);
#pragma unroll
                for (int g = 0; g < GV; g++) {
                  if (tok < it.vlo || tok >= it.vhi) {
                    out[g] |= 1u << r;
                  } else {
                    const uint32_t m = *(reinterpret_cast<const uint32_t *>(coefs + r * G * 4) + g) & 0x7FFF7FFFu;
                    if ((m & 0xFFFFu) >= 0x7C00u || (m >> 16) >= 0x7C00u) {
                      const int pos = vt * 16 + r, grp = (G > CB ? 2 * vc : vc * G / CB) + g;
                      atomicOr(&my_notes[(e * G + grp) * (KB / 32) + (pos >> 5)], 1u << (pos & 31));
                      noted[n_item & 3] = 1;
                      out[g] |= 1u << r;
                    } else if (large_value(m)) {
                      over[n_item & 3] = 1;
                    }
                  }
                }
              }
#pragma unroll
              for (int r = 0; r < 16; r++)
#pragma unroll
                for (int g = 0; g < GV; g++)
                  if ((out[g] >> r) & 1u) vf[r][g] = 0u;
            } else if (act) {                                    // the eight threads with the same coefficients look at two rows each
              uint32_t most = 0;
#pragma unroll
              for (int r = 0; r < 2; r++)
#pragma unroll
                for (int g = 0; g < GV; g++)
                  most = __vmaxu2(most, *(reinterpret_cast<const uint32_t *>(coefs + (2 * g8 + r) * G * 4) + g) & 0x7FFF7FFFu);
              if (large_value(most)) over[n_item & 3] = 1;
            }
            mbar_arrive(bar(RAW_EMPTY + 1));
            if (!warp_wait(bar(V_EMPTY + buf), ve[buf].next(), ctl)) { ok = false; break; }
            if (act) {
              uint32_t s2[16 * GV / 2], b2[16 * GV / 2];           // per pair of tokens (rows 2t, 2t + 1)
#pragma unroll
              for (int r = 0; r < 8; r++)
#pragma unroll
                for (int g = 0; g < GV; g++) {
                  s2[g * 8 + r] = prmt(vf[2 * r][g], vf[2 * r + 1][g], 0x5410);
                  b2[g * 8 + r] = prmt(vf[2 * r][g], vf[2 * r + 1][g], 0x7632);
                }
              uint32_t dst = sb + C::OFF_V + buf * C::KV_BYTES + (vt >> 2) * (D * 128) + (64 * vc + g8) * 128;
              const uint32_t ch0 = (uint32_t)((((vt & 3) * 2) ^ g8) << 4), ch1 = (uint32_t)((((vt & 3) * 2 + 1) ^ g8) << 4);
              // a word of each token quad at a time; the words move up in their registers, so that the loop stays rolled
              // (unrolled, the five roles' code does not stay in the instruction caches)
#pragma unroll 1
              for (int w4 = 0; w4 < 4; w4++, dst += 16 * 128) {
#pragma unroll
                for (int odd = 0; odd < 2; odd++) {
                  uint32_t lo[4], hi[4];
#pragma unroll
                  for (int t = 0; t < 4; t++) {
                    const uint32_t y = vw[t].x >> (8 * odd);
                    lo[t] = hfma2(codes_lo(y), s2[4 * odd + t], b2[4 * odd + t]);
                    hi[t] = hfma2(codes_hi(y), s2[4 * odd + t], b2[4 * odd + t]);
                  }
                  sts128(dst + (odd ? ch1 : ch0), lo[0], lo[1], lo[2], lo[3]);
                  sts128(dst + 8 * 128 + (odd ? ch1 : ch0), hi[0], hi[1], hi[2], hi[3]);
                }
#pragma unroll
                for (int t = 0; t < 4; t++) vw[t].x = vw[t].y, vw[t].y = vw[t].z, vw[t].z = vw[t].w;
                if constexpr (GV == 2) {
                  if (w4 == 1)                                     // the second group's coefficients
#pragma unroll
                    for (int r = 0; r < 8; r++) s2[r] = s2[8 * (GV - 1) + r], b2[r] = b2[8 * (GV - 1) + r];
                }
              }
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(FULL + (full & 7)));
        }
        if (!ok) break;
        kb += it.blocks;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(IT_NEXT));
        release();
      }
    };
    if constexpr (NQ == 2) codes(std::true_type(), std::true_type());
    else if (warp < DQ_WARP0) codes(std::true_type(), std::false_type());
    else codes(std::false_type(), std::true_type());
  } else {
    // ------------------------------------------------------------ softmax
    const int x = (warp - SOFT_WARP0) >> 2, row = threadIdx.x & 127;
    const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16), o_tm = tm + 256 + x * D;
    const float NINF = __int_as_float(0xFF800000);
    uint32_t s_base[2] = {0, 0};                   // score tiles finished in either buffer before this item
    int pv_base = 0, blk_base = 0, n_item = 0;     // this tile's PV products, the blocks and the items before this item
    uint32_t last_ph = 0;                          // S_LAST's parities, a bit an item slot
    bool ok = true;
    for (; const Item *ip = next_item(); n_item++) {
      const Item &it = *ip;
      auto leave = [&]() {
        s_base[0] += it.tiles == 2 ? it.blocks : (it.blocks + 1) >> 1;
        s_base[1] += it.tiles == 2 ? it.blocks : it.blocks >> 1;
        blk_base += it.blocks;
        release();
      };
      // The first tile alone: its scores take turns in both buffers, the second of which is this tile's in the next item.  A
      // parity tells apart only a phase and the next, so the item is left when its last scores are there.
      if (x >= it.tiles) {
        if (it.blocks > 1) {
          if (!warp_wait(bar(S_LAST + it_slot), (last_ph >> it_slot) & 1u, ctl)) break;
          last_ph ^= 1u << it_slot;
        }
        leave();
        continue;
      }
      const int r = it.r0 + x * QROWS + row, qi = r / p.ratio, hq = r - qi * p.ratio;
      const bool real = x * QROWS + row < it.rows;
      // ---------------------------------------------------------- q: binary16, the row's largest element in [2^14, 2^15)
      float c = 0.0f;
      const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + (int64_t)(it.cu0 + qi) * a.q_token +
                                                         (int64_t)(it.kvh * p.ratio + hq) * a.q_head);
      if (it.blocks > 0) {
        constexpr int HOLD = D <= 128 ? D / 8 : 16;            // pieces of 8 elements in registers at a time
        uint4 v[HOLD];
        uint32_t mx = 0;
#pragma unroll 1
        for (int h = 0; h < D / 8; h += HOLD) {
#pragma unroll
          for (int i = 0; i < HOLD; i++) v[i] = real ? src[h + i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int i = 0; i < HOLD; i++)
            mx = __vmaxu2(__vmaxu2(mx, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu)),
                          __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
        }
        mx = max(mx & 0xFFFFu, mx >> 16);                      // bfloat16 bits of the largest |element|
        const int ex = mx == 0u || mx >= 0x7F80u ? 0 : min(126, 14 - ((int)(mx >> 7) - 127));
        const float f = __int_as_float((ex + 127) << 23);
        // never 0, which a masked score of -inf would make NaN
        c = fmaxf(ldexpf(a.scale * (KEY_UNIT * 1.44269504088896340736f), -ex), 1.17549435e-38f);
        const uint32_t dst = sb + x * C::Q_BYTES + row * 128;
#pragma unroll 1
        for (int h0 = D / 8 - HOLD; h0 >= 0; h0 -= HOLD) {     // the last pieces read are still there
          if (h0 != D / 8 - HOLD)
#pragma unroll
            for (int i = 0; i < HOLD; i++) v[i] = real ? src[h0 + i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int i = 0; i < HOLD; i++) {
            const int h = h0 + i;
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; k++) o[k] = pack_f16(__uint_as_float(u[k] << 16) * f, __uint_as_float(u[k] & 0xFFFF0000u) * f);
            sts128(dst + (h >> 3) * (QROWS * 128) + (((h & 7) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(Q_FULL + x));
      }
      if (p.test_wait_ns != 0 && warp == SOFT_WARP0 && it.blocks > 0) {    // score products are in flight
        test_wait(bar(NEVER), ctl, p.test_wait_ns);
        break;
      }
      const int64_t pos = (int64_t)it.base + qi;
      const int khi = real ? (int)max((int64_t)0, min(pos + 1, (int64_t)it.hi)) : 0;
      const int klo = a.window > 0 ? (int)max((int64_t)0, min(pos + 1 - a.window, (int64_t)it.hi)) : 0;
      float m = NINF, l = 0.0f;                              // reference maximum (log2 units), sum
      for (int k = 0; k < it.blocks; k++) {
        const int buf = it.tiles == 2 ? x : k & 1, t0 = (it.blk0 + k) * KB;
        const bool seen = __all_sync(0xffffffffu, !real || (klo <= t0 && khi >= t0 + KB));
        if (!warp_wait(bar(S_FULL + buf), (s_base[buf] + (it.tiles == 2 ? k : k >> 1)) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        const uint32_t pages = kvalid[(blk_base + k) & 7];
        const uint32_t s_tm = tm + buf * 128;
        // Scores of tokens that the row does not see become -inf, in a pass of their own: few blocks have any.
        if (!seen || pages != (1u << (KB / 16)) - 1) {
#pragma unroll 1
          for (int ch = 0; ch < KB / 16; ch++) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(s_tm + 16 * ch, v);
            tmem_ld_wait();
            const int t1 = t0 + 16 * ch, k1 = (pages >> ch) & 1u ? khi : 0;   // nothing of a tile without a page
#pragma unroll
            for (int i = 0; i < 16; i++)
              if (t1 + token_of(i) < klo || t1 + token_of(i) >= k1) v[i] = 0xFF800000u;
            tmem_st_x16(s_tm + 16 * ch, v);
          }
          tmem_st_wait();
        }
        // 32 columns at a time, read once: their maximum, then, with the reference, their exponentials.  Only where the
        // maximum has outgrown the reference is what was summed before rescaled: l, O and the block's P so far.
        const f2 c2 = f2_make(c, c);
        auto columns = [&](const uint32_t (&v)[32], int h) {
          float m4[4] = {NINF, NINF, NINF, NINF};
#pragma unroll
          for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int j = 0; j < 4; j++)
              m4[j] = fmaxf(fmaxf(m4[j], __uint_as_float(v[i + 2 * j])), __uint_as_float(v[i + 2 * j + 1]));
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
          const bool grow = mx > m + GROW || (m == NINF && mx > NINF);
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? mx : m, f = mn == m ? 1.0f : ex2(m - mn);
            m = mn;
            l *= f;
            if (k > 0 && !warp_wait(bar(PV_DONE + x), (pv_base + k - 1) & 1, ctl)) ok = false;
            rescale<D>(k > 0 ? o_tm : 0xFFFFFFFFu, s_tm, h / 2, f);
          }
          const float mu = m == NINF ? 0.0f : m;
          const f2 mu2 = f2_make(P_EXP - mu, P_EXP - mu);
          f2 l2[2] = {f2_zero(), f2_zero()};
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 16; i++) {
            float e0, e1;
            f2_split(f2_fma(f2_bits(v[2 * i], v[2 * i + 1]), c2, mu2), e0, e1);
            e0 = ex2(e0), e1 = ex2(e1);
            l2[i & 1] = f2_add(l2[i & 1], f2_make(e0, e1));
            o[i] = pack_f16(e0, e1);
          }
          tmem_st_x16(s_tm + h / 2, o);                // over score columns that have been read
          float la, lb;
          f2_split(f2_add(l2[0], l2[1]), la, lb);
          l += la + lb;
        };
        {
          uint32_t v[32];
#pragma unroll 1
          for (int h = 0; h < KB; h += 32) {
            tmem_ld_32x32b_x32(s_tm + h, v);
            tmem_ld_wait();
            columns(v, h);
          }
        }
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        // A parity tells apart only a phase and the next, so no PV may finish before the one ahead of it has been seen: with
        // two row tiles, S of this step came after that PV; with one, it is waited for here, before the next is let go.
        if (it.tiles == 1 && k > 0 &&
            !warp_wait(bar(PV_DONE + x), (pv_base + k - 1) & 1, ctl)) { ok = false; break; }
        mbar_arrive(bar(P_FULL + buf));
      }
      if (!ok) break;
      // ---------------------------------------------------------- output
      if (it.blocks > 0) {
        if (!warp_wait(bar(PV_DONE + x), (pv_base + it.blocks - 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        pv_base += it.blocks;
      }
      // groups that a noted (non-finite) value makes NaN
      uint32_t nan_groups = 0;
      if (it.blocks > 0 && noted[n_item & 3]) {
        const uint32_t *my_notes = notes + (n_item & 3) * C::NOTES;
        for (int e = 0; e < C::EDGES; e++) {
          const int blk = e < 4 ? it.blk0 + e : it.fhi / KB + e - 4;
          for (int ps = 0; ps < KB; ps++) {
            const int tok = blk * KB + (ps & ~15) + token_of(ps & 15);
            if (tok >= klo && tok < khi)
              for (int g = 0; g < G; g++)
                if ((my_notes[(e * G + g) * (KB / 32) + (ps >> 5)] >> (ps & 31)) & 1u) nan_groups |= 1u << g;
          }
        }
      }
      // an item that is done again leaves its rows to the second time (q may be where they go)
      const bool again = it.vexp == 0 && over[n_item & 3] != 0;
      const float inv = l == 0.0f ? 0.0f : (it.vexp == 0 ? 1.0f : 16.0f) / l;
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)(it.cu0 + qi) * a.heads + it.kvh * p.ratio + hq) * D;
#pragma unroll 1
      for (int ch = 0; ch < D / 16; ch++) {
        uint32_t v[16];
        if (it.blocks > 0) {
          __syncwarp();
          tmem_ld_32x32b_x16(o_tm + 16 * ch, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 16; i++) v[i] = 0u;
        }
        if (real && !again) {
          const bool bad = (nan_groups >> (16 * ch / (D / G))) & 1u;
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; i++) {
            float y0 = __uint_as_float(v[2 * i]) * inv, y1 = __uint_as_float(v[2 * i + 1]) * inv;
            if (bad) y0 = y1 = __int_as_float(0x7FC00000);
            const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
            o[i] = *reinterpret_cast<const uint32_t *>(&h);
          }
          *reinterpret_cast<uint4 *>(out + 16 * ch) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(out + 16 * ch + 8) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      tc_fence_before();
      leave();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    // No wait is left that could give up, so the flag is final: if one did, MMAs may be in flight, which are waited for (bounded)
    // before TMEM goes.
    if (*abort_flag && elect_one()) {
      umma_commit(bar(DRAIN));
      wait_drain(bar(DRAIN), 0);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int G>
cudaError_t launch(const KvAttendArgs &a, cudaStream_t s) {
  using C = Cfg<D, G>;
  Params p{};
  p.a = a;
  p.g = kv_geom(a.pages, a.kv_heads, a.head_dim, a.page, a.group);
  p.ratio = (int)(a.heads / a.kv_heads);
  p.test_wait_ns = g_test_wait_ns.exchange(0, std::memory_order_relaxed);
  // never more CTAs than items
  const int64_t items = (a.tokens * p.ratio / (C::NQ * QROWS) + (a.tokens < a.B ? a.tokens : a.B)) * a.kv_heads;
  static std::atomic<int> set_for{0};
  return launch_large(prefill_kernel<D, G>, items < kv_max_ctas(1) ? items : kv_max_ctas(1), THREADS, C::SMEM, s, p, set_for);
}

}  // namespace

cudaError_t launch_kv_prefill(const KvAttendArgs &a, cudaStream_t s) {
  const int D = (int)a.head_dim, G = D / a.group;
  if (D == 64) return G == 1 ? launch<64, 1>(a, s) : launch<64, 2>(a, s);
  if (D == 128) return G == 1 ? launch<128, 1>(a, s) : G == 2 ? launch<128, 2>(a, s) : launch<128, 4>(a, s);
  if (D == 256) return G == 2 ? launch<256, 2>(a, s) : G == 4 ? launch<256, 4>(a, s) : launch<256, 8>(a, s);
  return cudaErrorNotSupported;
}

void set_kv_test_wait(unsigned long long limit_ns) { g_test_wait_ns.store(limit_ns, std::memory_order_relaxed); }

cudaError_t read_clear_kv_status(int *status, cudaStream_t s) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_kv_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_kv_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
  }
  *status = v;
  return cudaSuccess;
}

}  // namespace qmm
