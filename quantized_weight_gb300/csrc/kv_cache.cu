// kv_cache.cu -- the 4-bit key/value cache around the attention: plan (block
// tables and slots from request lengths), append (quantize into slots), read
// (slots back to values).  The layout is in kv_layout.cuh.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_layout.cuh"
#include "qmm_device.cuh"
#include "qmm_launch.h"

namespace qmm {
namespace {

// ---------------------------------------------------------------- plan

constexpr int kPlanThreads = 512;

struct PlanParams {
  const int32_t *cached, *fresh, *free_pages;
  int32_t *table, *slots, *positions, *cu, *lens, *need;
  int64_t n_free, max_blocks, tokens;
  int B, lg_page;
};

__device__ __forceinline__ int sat32(int64_t v) { return v > 0x7FFFFFFF ? 0x7FFFFFFF : (int)v; }

// Exclusive scan over the block of one value pair per thread; returns the totals too.
__device__ __forceinline__ void scan_pair(int64_t &a, int64_t &b, int64_t &ta, int64_t &tb, int64_t (*sh)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += u, y += v;
  }
  if (lane == 31) sh[warp][0] = x, sh[warp][1] = y;
  __syncthreads();
  int64_t pa = 0, pb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; w++) {
    if (w == warp) pa = ta, pb = tb;
    ta += sh[w][0], tb += sh[w][1];
  }
  a = pa + x - a;
  b = pb + y - b;
}

// Every CTA scans all requests (a few thousand lengths at most, so one scan
// costs less than handing its result over), then writes its share of the
// tokens and of the table rows.  Table entries that this call writes are never
// read by it: a token's page comes from the free list or from an older entry.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_sm[];
  int32_t *cu = plan_sm, *first = plan_sm + p.B;        // per request: first token, first of its free pages
  __shared__ int64_t sh[kPlanThreads / 32][2];
  const int P1 = (1 << p.lg_page) - 1;
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  int64_t at = 0, nd = 0;
  for (int b = b0; b < b1; b++) {
    const int64_t c = max(0, p.cached[b]), f = max(0, p.fresh[b]);
    at += f;
    nd += ((c + f + P1) >> p.lg_page) - ((c + P1) >> p.lg_page);
  }
  int64_t tokens, need;
  scan_pair(at, nd, tokens, need, sh);
  for (int b = b0; b < b1; b++) {
    const int64_t c = max(0, p.cached[b]), f = max(0, p.fresh[b]);
    cu[b] = sat32(at);
    first[b] = sat32(nd);
    if (blockIdx.x == 0) p.cu[b] = sat32(at), p.lens[b] = sat32(c + f);
    at += f;
    nd += ((c + f + P1) >> p.lg_page) - ((c + P1) >> p.lg_page);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.cu[p.B] = sat32(tokens), *p.need = sat32(need);
  __syncthreads();

  const int64_t gid = blockIdx.x * (int64_t)kPlanThreads + threadIdx.x, gsz = (int64_t)gridDim.x * kPlanThreads;
  for (int64_t t = gid; t < p.tokens; t += gsz) {
    int slot = -1, pos = 0;
    if (t < tokens) {
      int lo = 0, hi = p.B - 1;                           // the last request that begins at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int64_t c = max(0, p.cached[lo]), ps = c + (t - cu[lo]);
      const int64_t have = (c + P1) >> p.lg_page, col = ps >> p.lg_page;
      int page = -1;
      if (col < p.max_blocks) {
        if (col < have) page = p.table[lo * p.max_blocks + col];
        else if (first[lo] + col - have < p.n_free) page = p.free_pages[first[lo] + col - have];
      }
      const int64_t s = ((int64_t)page << p.lg_page) + (ps & P1);
      if (page >= 0 && s <= 0x7FFFFFFF) slot = (int)s;
      pos = sat32(ps);
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  const int lane = threadIdx.x & 31;
  for (int64_t b = gid >> 5; b < p.B; b += gsz >> 5) {
    const int64_t c = max(0, p.cached[b]), f = max(0, p.fresh[b]);
    const int64_t have = (c + P1) >> p.lg_page, tot = min(p.max_blocks, (c + f + P1) >> p.lg_page);
    for (int64_t col = have + lane; col < tot; col += 32) {
      const int64_t i = first[b] + col - have;
      p.table[b * p.max_blocks + col] = i < p.n_free ? p.free_pages[i] : -1;
    }
  }
}

// ---------------------------------------------------------------- append

constexpr int kRowThreads = 128;

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

__device__ __forceinline__ int order_key(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ uint16_t half_bits_rn(float f) {
  return isnan(f) ? (uint16_t)0x7E00u : __half_as_ushort(__float2half_rn(f));
}

struct AppendParams {
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;     // strides in elements
  const int32_t *slots;
  uint8_t *cache;
  int64_t tokens;
  KvGeom g;
};

// One thread per eight elements of one (token, head) row of K or V.
template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const AppendParams p) {
  const KvGeom &g = p.g;
  const int tpr = g.D >> 3;                              // threads per row: 8, 16 or 32
  const int64_t row = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) / tpr;
  const int m = threadIdx.x % tpr;
  const int64_t rows = p.tokens * g.kv_heads * 2;
  const bool in = row < rows;
  const bool isv = in && row >= rows / 2;
  const int64_t r = isv ? row - rows / 2 : row;
  const int64_t t = r / g.kv_heads;
  const int h = (int)(r % g.kv_heads);
  const int slot = in ? p.slots[t] : -1;
  const bool ok = slot >= 0 && (slot >> g.lg_page) < g.pages;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = 0.0f;
  if (ok) {
    const int64_t off = isv ? t * p.v_token + h * p.v_head : t * p.k_token + h * p.k_head;
    load8<BF16>(static_cast<const uint8_t *>(isv ? p.v : p.k) + (off + 8 * m) * (BF16 ? 2 : 4), v);
  }
  int kmin = 0x7FFFFFFF, kmax = (int)0x80000000;
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (!isnan(v[i])) {
      const int k = order_key(v[i]);
      kmin = min(kmin, k), kmax = max(kmax, k);
    }
  for (int o = 1; o < g.group >> 3; o <<= 1) {
    kmin = min(kmin, __shfl_xor_sync(0xffffffffu, kmin, o));
    kmax = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
  }
  const float nan = __int_as_float(0x7FC00000);
  const float lo = kmin == 0x7FFFFFFF ? nan : __int_as_float(order_key(__int_as_float(kmin)));
  const float hi = kmax == (int)0x80000000 ? nan : __int_as_float(order_key(__int_as_float(kmax)));
  const uint16_t sh = half_bits_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)), bh = half_bits_rn(lo);
  const float s = h2f(sh), b = h2f(bh);
  uint32_t word = 0;
  if (s > 0.0f && isfinite(s))
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float q = fminf(fmaxf(roundf(__fdiv_rn(__fsub_rn(v[i], b), s)), 0.0f), 15.0f);
      word |= (uint32_t)(int)q << (4 * i);
    }
  const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 1);
  if (!ok) return;
  const int j = slot & 15, tr = kv_row(j);
  uint8_t *tile = p.cache + kv_tile_at(g, slot, h);
  if (!isv) {
    *reinterpret_cast<uint32_t *>(tile + kv_k_word(g.D, tr, m)) = word;
  } else {
    const uint32_t lw = m & 1 ? other : word, hw = m & 1 ? word : other;   // elements d and d + 8
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int e = 4 * (m & 1) + i, d = 16 * (m >> 1) + e;
      tile[kv_v_word(g.D, d, j >> 2) + (j & 3)] = (uint8_t)(((lw >> (4 * e)) & 15u) | (((hw >> (4 * e)) & 15u) << 4));
    }
  }
  if (m % (g.group >> 3) == 0) {
    const int grp = m / (g.group >> 3);
    *reinterpret_cast<uint32_t *>(tile + (isv ? kv_v_coef(g, tr, grp) : kv_k_coef(g, tr, grp))) = sh | ((uint32_t)bh << 16);
  }
}

// ---------------------------------------------------------------- read

struct ReadParams {
  const int32_t *slots;
  const uint8_t *cache;
  void *k, *v;
  int64_t tokens;
  KvGeom g;
};

template <bool BF16>
__device__ __forceinline__ void store8(void *p, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *(reinterpret_cast<float4 *>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// One thread per eight elements of one (token, head) row of K or V.
template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const ReadParams p) {
  const KvGeom &g = p.g;
  const int tpr = g.D >> 3;
  const int64_t row = (blockIdx.x * (int64_t)kRowThreads + threadIdx.x) / tpr;
  const int m = threadIdx.x % tpr;
  const int64_t rows = p.tokens * g.kv_heads * 2;
  if (row >= rows) return;
  const bool isv = row >= rows / 2;
  const int64_t r = isv ? row - rows / 2 : row;
  const int64_t t = r / g.kv_heads;
  const int h = (int)(r % g.kv_heads), slot = p.slots[t];
  float v[8];
  if (slot >= 0 && (slot >> g.lg_page) < g.pages) {
    const int j = slot & 15, tr = kv_row(j), grp = 8 * m / g.group;
    const uint8_t *tile = p.cache + kv_tile_at(g, slot, h);
    const uint32_t c = *reinterpret_cast<const uint32_t *>(tile + (isv ? kv_v_coef(g, tr, grp) : kv_k_coef(g, tr, grp)));
    const float s = h2f((uint16_t)c), b = h2f((uint16_t)(c >> 16));
    uint32_t word = 0;
    if (!isv) {
      word = *reinterpret_cast<const uint32_t *>(tile + kv_k_word(g.D, tr, m));
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const uint32_t by = tile[kv_v_word(g.D, 16 * (m >> 1) + i, j >> 2) + (j & 3)];
        word |= ((by >> (4 * (m & 1))) & 15u) << (4 * i);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __fadd_rn(__fmul_rn(s, (float)((word >> (4 * i)) & 15u)), b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __int_as_float(0x7FC00000);
  }
  store8<BF16>(static_cast<uint8_t *>(isv ? p.v : p.k) + (r * g.D + 8 * m) * (BF16 ? 2 : 4), v);
}

}  // namespace

cudaError_t launch_kv_plan(const int32_t *cached, const int32_t *fresh, const int32_t *free_pages, int64_t n_free,
                           int32_t *table, int64_t B, int64_t max_blocks, int page, int64_t tokens, int32_t *slots,
                           int32_t *positions, int32_t *cu, int32_t *lens, int32_t *need, cudaStream_t s) {
  PlanParams p{cached, fresh, free_pages, table, slots, positions, cu, lens, need, n_free, max_blocks, tokens,
               (int)B, __builtin_ctz((unsigned)page)};
  const size_t smem = 2 * sizeof(int32_t) * (size_t)B;
  cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * kKvPlanMaxB);
  if (e != cudaSuccess) return e;
  int64_t work = tokens > B * 32 ? tokens : B * 32;
  int64_t grid = (work + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
  grid = grid < 1 ? 1 : grid > 152 ? 152 : grid;
  plan_kernel<<<(int)grid, kPlanThreads, smem, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const void *k, const void *v, bool bf16, int64_t k_token, int64_t k_head, int64_t v_token,
                             int64_t v_head, const int32_t *slots, void *cache, int64_t tokens, int64_t pages,
                             int64_t kv_heads, int64_t D, int page, int group, cudaStream_t s) {
  AppendParams p{k, v, k_token, k_head, v_token, v_head, slots, static_cast<uint8_t *>(cache), tokens,
                 kv_geom(pages, kv_heads, D, page, group)};
  const int64_t threads = tokens * kv_heads * 2 * (D / 8), grid = (threads + kRowThreads - 1) / kRowThreads;
  if (bf16) append_kernel<true><<<(unsigned)grid, kRowThreads, 0, s>>>(p);
  else append_kernel<false><<<(unsigned)grid, kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const int32_t *slots, const void *cache, void *k, void *v, bool bf16, int64_t tokens,
                           int64_t pages, int64_t kv_heads, int64_t D, int page, int group, cudaStream_t s) {
  ReadParams p{slots, static_cast<const uint8_t *>(cache), k, v, tokens, kv_geom(pages, kv_heads, D, page, group)};
  const int64_t threads = tokens * kv_heads * 2 * (D / 8), grid = (threads + kRowThreads - 1) / kRowThreads;
  if (bf16) read_kernel<true><<<(unsigned)grid, kRowThreads, 0, s>>>(p);
  else read_kernel<false><<<(unsigned)grid, kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qmm
