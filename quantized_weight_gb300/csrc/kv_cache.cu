// kv_cache.cu -- the 4-bit key/value cache around the attention: plan (block
// tables and slots from request lengths), append (quantize into slots), read
// (slots back to values).  The layout is in kv_layout.cuh.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "kv_attend.h"
#include "kv_launch.h"
#include "kv_layout.cuh"
#include "qmm_device.cuh"
#include "qmm_launch.h"

namespace qmm {
namespace {

// ---------------------------------------------------------------- plan

constexpr int kPlanThreads = 512;
constexpr size_t kPlanStatic = kPlanThreads / 32 * 2 * sizeof(int64_t);   // the scan's shared memory, beside two prefix sums a request

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

// Bound: latency; the bytes are a few a request and a token (0.04 us for 256 prompts of 90 000 tokens).
// Every CTA scans all requests (a few thousand lengths at most, so one scan
// costs less than handing its result over), then writes its share of the
// tokens and of the table rows.  Table entries that this call writes are never
// read by it: a token's page comes from the free list or from an older entry.
// Measured: 48 requests of one token 3.2 us, 256 prompts 4.8 us (launch, two dependent loads, scan, a search a token).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_sm[];
  int32_t *cu = plan_sm, *first = plan_sm + p.B;        // per request: first token, first of its free pages
  __shared__ int64_t sh[kPlanThreads / 32][2];
  const int P1 = (1 << p.lg_page) - 1;
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  pdl_wait();
  pdl_launch_dependents();
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

// ---------------------------------------------------------------- tokens a warp takes
//
// append and read work by the warp: one token or four, and some of the keys and
// values of its heads.  Four tokens whose slots are an aligned, consecutive quad share the
// value words of their tile, so that the warp moves 16-byte pieces of it; a token
// outside such a quad (a decode step's, a prompt's ends) moves its own bytes.
// Finding the quads and placing the tokens costs as much as the rows of a head or
// two, so that a warp has one of them only where there would be too few warps otherwise.

constexpr int kRowWarps = 4, kRowThreads = 32 * kRowWarps;

struct Rows {
  const int32_t *slots;
  int64_t tokens;
  int per_warp;                // token indexes a warp looks at: 4, or 1 where that leaves too few warps
  int parts, part;             // warps that share them; keys and values of a head (each one row) a warp takes
  KvGeom g;
};

// The slot of token i if it lies in the cache, else -1.
__device__ __forceinline__ int slot_of(const Rows &p, int64_t i) {
  const int s = i >= 0 && i < p.tokens ? p.slots[i] : -1;
  return s >= 0 && (s >> p.g.lg_page) < p.g.pages ? s : -1;
}

// Calls quad(first token, its slot) and single(token, slot) for what falls to this warp's tokens: a quad to the warp that
// has its first token.  Every lane takes part.
template <class Quad, class Single>
__device__ __forceinline__ void each_run(const Rows &p, int64_t unit, Quad quad, Single single) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = unit * p.per_warp;
  // lane k: token t0 - 3 + k (k < 10), the slots around this warp's tokens
  const int s = lane < 10 ? slot_of(p, t0 - 3 + lane) : -1;
  // a quad begins at lane k: slots s, s + 1, s + 2, s + 3 with s a multiple of 4
  const int s1 = __shfl_down_sync(0xffffffffu, s, 1), s2 = __shfl_down_sync(0xffffffffu, s, 2), s3 = __shfl_down_sync(0xffffffffu, s, 3);
  const unsigned heads = __ballot_sync(0xffffffffu, lane < 7 && s >= 0 && (s & 3) == 0 && s1 == s + 1 && s2 == s + 2 && s3 == s + 3);
  const unsigned inside = heads | heads << 1 | heads << 2 | heads << 3;
  for (int k = 0; k < p.per_warp && t0 + k < p.tokens; k++) {
    const int sk = __shfl_sync(0xffffffffu, s, 3 + k);
    if ((heads >> (3 + k)) & 1u) quad(t0 + k, sk);
    else if (!((inside >> (3 + k)) & 1u)) single(t0 + k, sk);
  }
}

inline int64_t row_grid(Rows &p) {
  // one token and row a warp while that gives no more than 16 warps an SM; beyond, the work of a token counts, not its
  // latency, and a warp takes as much as leaves 64 an SM
  const int64_t rows = 2 * p.g.kv_heads;
  p.per_warp = p.tokens * rows <= kv_sms() * 16 ? 1 : 4;
  const int64_t units = (p.tokens + p.per_warp - 1) / p.per_warp;
  int64_t part = units * rows / (kv_sms() * 64);
  part = part < 1 ? 1 : part > rows ? rows : part;
  p.parts = (int)((rows + part - 1) / part);
  p.part = (int)((rows + p.parts - 1) / p.parts);
  return (units * p.parts + kRowWarps - 1) / kRowWarps;
}

// 16 bytes read once, past L1.  (Not a read-only load: the kernel before this one may still have been writing them when this
// one was launched.)
__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Eight elements as they lie in memory.
template <bool BF16>
struct Raw {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const uint8_t *p) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); i++) w[i] = ld_once(p + 16 * i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); i++) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[BF16 ? 0 : 1].x, w[BF16 ? 0 : 1].y, w[BF16 ? 0 : 1].z, w[BF16 ? 0 : 1].w};
#pragma unroll
    for (int i = 0; i < 8; i++)
      v[i] = __uint_as_float(!BF16 ? u[i] : i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
  }
};

// ---------------------------------------------------------------- append

__device__ __forceinline__ uint16_t half_bits_rn(float f) {
  return isnan(f) ? (uint16_t)0x7E00u : __half_as_ushort(__float2half_rn(f));
}

struct AppendParams {
  Rows r;
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;     // strides in elements
  uint8_t *cache;
};

// The least and the greatest of a group, `lanes` lanes with eight elements each.  NaN are skipped (NaN is left where a
// group has nothing else) and -0 lies below +0: the order of fminf and fmaxf here, and of the two-element bfloat16 forms.
template <bool BF16>
__device__ __forceinline__ void range8(const Raw<BF16> &x, const float (&v)[8], int lanes, float &lo, float &hi) {
  if constexpr (BF16) {
    auto b2 = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
    const __nv_bfloat162 mn = __hmin2(__hmin2(b2(x.w[0].x), b2(x.w[0].y)), __hmin2(b2(x.w[0].z), b2(x.w[0].w)));
    const __nv_bfloat162 mx = __hmax2(__hmax2(b2(x.w[0].x), b2(x.w[0].y)), __hmax2(b2(x.w[0].z), b2(x.w[0].w)));
    // least and negated greatest side by side: one exchange a step
    const uint32_t a = *reinterpret_cast<const uint32_t *>(&mn), b = *reinterpret_cast<const uint32_t *>(&mx) ^ 0x80008000u;
    __nv_bfloat162 r = __hmin2(b2(prmt(a, b, 0x5410u)), b2(prmt(a, b, 0x7632u)));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
      if (o < lanes) r = __hmin2(r, b2(__shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&r), o)));
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&r);
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float((u & 0xFFFF0000u) ^ 0x80000000u);
  } else {
    lo = fminf(fminf(fminf(v[0], v[1]), fminf(v[2], v[3])), fminf(fminf(v[4], v[5]), fminf(v[6], v[7])));
    hi = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
      if (o < lanes) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
  }
}

// Eight elements of a row a lane: the codes, element i in nibble i, and scale | bias << 16.
// The quotient (x - bias) / scale, correctly rounded, decides a code only through its rounding, that is only next to a
// half-integer.  A product with the approximate reciprocal is, between 0 and 15, within 1e-5 of it; where no element of
// the lane comes so near to a half, or rounds to something else than 0 .. 15 (NaN too), the product's roundings are
// the codes, elsewhere the division is taken.
template <bool BF16>
__device__ __forceinline__ uint32_t quantize8(const Raw<BF16> &x, int lanes, uint32_t &coef) {
  float v[8], lo, hi;
  x.values(v);
  range8<BF16>(x, v, lanes, lo, hi);
  const uint16_t sh = half_bits_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)), bh = half_bits_rn(lo);
  coef = sh | ((uint32_t)bh << 16);
  const float s = h2f(sh), b = h2f(bh);
  if (!(s > 0.0f && isfinite(s))) return 0u;
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
  constexpr float MAGIC = 12582912.0f;                     // 1.5 * 2^23: the integer lands in the low mantissa bits
  const f2 b2 = f2_make(b, b), inv2 = f2_make(inv, inv), magic2 = f2_make(MAGIC, MAGIC);
  uint32_t word = 0, all = 0;
  float worst = 0.0f;
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    const f2 t = f2_mul(f2_sub(f2_make(v[i], v[i + 1]), b2), inv2), r = f2_add(t, magic2);
    float d0, d1, r0, r1;
    f2_split(f2_sub(t, f2_sub(r, magic2)), d0, d1);
    f2_split(r, r0, r1);
    worst = fmaxf(worst, fmaxf(fabsf(d0), fabsf(d1)));
    const uint32_t n0 = __float_as_uint(r0) - __float_as_uint(MAGIC), n1 = __float_as_uint(r1) - __float_as_uint(MAGIC);
    all |= n0 | n1;
    word = (word * 16u + n1) * 16u + n0;
  }
  if (worst > 0.49998f || all > 15u) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float q = fminf(fmaxf(roundf(__fdiv_rn(__fsub_rn(v[i], b), s)), 0.0f), 15.0f);
      word |= (uint32_t)(int)q << (4 * i);
    }
  }
  return word;
}

// A warp quantizes a row of a head at a time (a group's least and greatest by shuffles, eight elements a lane); keys go out as
// words, the values of a quad through 4 * D / 2 bytes of shared memory as 16-byte pieces.
// Bound: 16381 tokens of 8 heads of 128 in bfloat16 are 67 MB read and 19 MB written, 12.7 us; measured 38 us, at 70 % of
// the schedulers' issue slots (31 M instructions, 30 an element, half of them the quantization, most of the rest the
// values' transposition and addresses).  A step of 64 tokens: 3.4 us, launch and two dependent loads.
template <bool BF16, int D>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const AppendParams p) {
  constexpr int TPR = D / 8, RP = 32 / TPR;                // lanes a row, rows at a time
  __shared__ __align__(16) uint8_t bytes_s[kRowWarps][4 * (D / 2)];
  const KvGeom &g = p.r.g;
  const int lane = threadIdx.x & 31, m = lane % TPR, sub = lane / TPR;
  uint8_t *bytes = bytes_s[threadIdx.x >> 5];              // [token 4][w][e]: codes of elements 16 w + e and 16 w + 8 + e
  const int64_t wid = blockIdx.x * (int64_t)kRowWarps + (threadIdx.x >> 5);
  const int64_t unit = wid / p.r.parts;
  const int hv0 = (int)(wid - unit * p.r.parts) * p.r.part, hv1 = min(hv0 + p.r.part, 2 * g.kv_heads);
  pdl_wait();
  pdl_launch_dependents();
  if (unit * p.r.per_warp >= p.r.tokens) return;           // whole warps
  const int lanes = g.group >> 3, grp = m >> g.lg_group8;

  // `n` tokens from t on, their slots from `slot` on (n = 4: an aligned quad)
  auto rows = [&](auto count, int64_t t, int slot) {
    constexpr int n = decltype(count)::value, PASSES = n > RP ? n / RP : 1;
    Raw<BF16> ahead[PASSES];
    auto fetch = [&](int hv) {
      const uint8_t *src = static_cast<const uint8_t *>(hv & 1 ? p.v : p.k);
      const int64_t token = hv & 1 ? p.v_token : p.k_token, head = (int64_t)(hv >> 1) * (hv & 1 ? p.v_head : p.k_head);
#pragma unroll
      for (int ps = 0; ps < PASSES; ps++) {
        const int r = ps * RP + sub;
        if (r < n) ahead[ps].load(src + ((t + r) * token + head + 8 * m) * (BF16 ? 2 : 4));
        else ahead[ps].zero();
      }
    };
    fetch(hv0);
#pragma unroll 1
    for (int hv = hv0; hv < hv1; hv++) {
      const int h = hv >> 1;
      const bool isv = hv & 1;
      Raw<BF16> x[PASSES];
#pragma unroll
      for (int ps = 0; ps < PASSES; ps++) x[ps] = ahead[ps];
      if (hv + 1 < hv1) fetch(hv + 1);
      uint8_t *tile = p.cache + kv_tile_at(g, slot, h);
#pragma unroll
      for (int ps = 0; ps < PASSES; ps++) {
        const int r = ps * RP + sub, j = (slot & 15) + r, row = kv_row(j & 15);
        uint32_t coef;
        const uint32_t word = quantize8<BF16>(x[ps], lanes, coef), other = __shfl_xor_sync(0xffffffffu, word, 1);
        if (r < n && (m & (lanes - 1)) == 0)
          *reinterpret_cast<uint32_t *>(tile + (isv ? kv_v_coef(g, row, grp) : kv_k_coef(g, row, grp))) = coef;
        if (!isv) {
          if (r < n) *reinterpret_cast<uint32_t *>(tile + kv_k_word(D, row, m)) = word;
        } else {
          // this lane's four bytes: elements e, e + 8 of its 16, e from 0 (even m) or 4 (odd m)
          const uint32_t lw = (m & 1 ? other : word) >> (16 * (m & 1)), hw = (m & 1 ? word : other) >> (16 * (m & 1));
          const uint32_t lx = (lw & 0xFu) | (lw & 0xF0u) << 4 | (lw & 0xF00u) << 8 | (lw & 0xF000u) << 12;
          const uint32_t hx = (hw & 0xFu) | (hw & 0xF0u) << 4 | (hw & 0xF00u) << 8 | (hw & 0xF000u) << 12;
          const uint32_t by = lx | hx << 4;
          if constexpr (n == 4) {
            *reinterpret_cast<uint32_t *>(bytes + r * (D / 2) + 4 * m) = by;
          } else if (r < n) {
#pragma unroll
            for (int i = 0; i < 4; i++)
              tile[kv_v_word(D, 16 * (m >> 1) + 4 * (m & 1) + i, j >> 2) + (j & 3)] = (uint8_t)(by >> (8 * i));
          }
        }
      }
      if constexpr (n == 4) {
        if (isv) {
          __syncwarp();
          if (lane < D / 8) {                                // (c, e): a word of each 16 elements of 64, four tokens a word
            const int c = lane >> 3, e = lane & 7;
            uint32_t o[4];
#pragma unroll
            for (int w = 0; w < 4; w++) {
              const uint8_t *b = bytes + (4 * c + w) * 8 + e;
              o[w] = b[0] | (uint32_t)b[D / 2] << 8 | (uint32_t)b[2 * (D / 2)] << 16 | (uint32_t)b[3 * (D / 2)] << 24;
            }
            *reinterpret_cast<uint4 *>(tile + kv_v_word(D, 64 * c + e, (slot & 15) >> 2)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          __syncwarp();
        }
      }
    }
  };
  each_run(p.r, unit, [&](int64_t t, int slot) { rows(std::integral_constant<int, 4>(), t, slot); },
           [&](int64_t t, int slot) {
             if (slot >= 0) rows(std::integral_constant<int, 1>(), t, slot);
           });
}

// ---------------------------------------------------------------- read

struct ReadParams {
  Rows r;
  const uint8_t *cache;
  void *k, *v;
};

// Eight values, written past the caches' keeping: bfloat16 in one piece; float32 in two, 8 elements apart (see read_kernel).
template <bool BF16>
__device__ __forceinline__ void store8(void *p, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(u[0], u[1], u[2], u[3]));
  } else {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 2, make_float4(v[4], v[5], v[6], v[7]));
  }
}

// Four codes, a byte each, to s * q + b (the product is exact, so this is one rounding).
__device__ __forceinline__ void values4(uint32_t q, float s, float b, float *v) {
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t h = prmt(q, 0x64646464u, i ? 0x7372u : 0x5150u);         // two binary16 values 1024 + q
    const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&h), __float2half2_rn(1024.0f));
    const float2 f = __half22float2(c);
    v[2 * i] = fmaf(s, f.x, b);
    v[2 * i + 1] = fmaf(s, f.y, b);
  }
}

// Bound: bytes for float32 (16381 tokens of 8 heads of 128: 19 MB read and 134 MB written, 22.6 us; measured 24.0 us).  For
// bfloat16 and heads of 64 the start of a warp: slots, then tiles (30011 tokens of 4 heads: 8.6 MB read and 31 MB written,
// 5.8 us; measured 14.4 us with 40 of 64 warps an SM; 48 and 64, in fewer registers, 15.4 and 16.1 us).  100 tokens: 2.5 us.
template <bool BF16, int D>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const ReadParams p) {
  constexpr int TPR = D / 8, RP = 32 / TPR;
  __shared__ __align__(16) uint8_t bytes_s[kRowWarps][4 * (D / 2)];
  const KvGeom &g = p.r.g;
  const int lane = threadIdx.x & 31, m = lane % TPR, sub = lane / TPR;
  uint8_t *bytes = bytes_s[threadIdx.x >> 5];
  const int64_t wid = blockIdx.x * (int64_t)kRowWarps + (threadIdx.x >> 5);
  const int64_t unit = wid / p.r.parts;
  const int hv0 = (int)(wid - unit * p.r.parts) * p.r.part, hv1 = min(hv0 + p.r.part, 2 * g.kv_heads);
  pdl_wait();
  pdl_launch_dependents();
  if (unit * p.r.per_warp >= p.r.tokens) return;

  auto rows = [&](auto count, int64_t t, int slot) {
    constexpr int n = decltype(count)::value, PASSES = n > RP ? n / RP : 1;
    // what the next row has in the cache: coefficients; a key's words, a single value's bytes or a lane's words of a quad's
    uint32_t coef_ahead[PASSES], ahead[4];
    auto fetch = [&](int hv) {
      const bool isv = hv & 1;
      const uint8_t *tile = p.cache + (slot >= 0 ? kv_tile_at(g, slot, hv >> 1) : 0);
#pragma unroll
      for (int i = 0; i < 4; i++) ahead[i] = 0u;
#pragma unroll
      for (int ps = 0; ps < PASSES; ps++) {
        const int r = ps * RP + sub, j = (slot & 15) + r, row = kv_row(j & 15), grp = m >> g.lg_group8;
        coef_ahead[ps] = 0u;
        if (r < n && slot >= 0) {
          coef_ahead[ps] = *reinterpret_cast<const uint32_t *>(tile + (isv ? kv_v_coef(g, row, grp) : kv_k_coef(g, row, grp)));
          if (!isv) {
            ahead[ps] = *reinterpret_cast<const uint32_t *>(tile + kv_k_word(D, row, m));
          } else if (n == 1) {
#pragma unroll
            for (int i = 0; i < 8; i++)
              ahead[i >> 2] |= (uint32_t)tile[kv_v_word(D, 16 * (m >> 1) + i, j >> 2) + (j & 3)] << (8 * (i & 3));
          }
        }
      }
      if (n == 4 && isv && lane < D / 8) {
        const uint4 o = *reinterpret_cast<const uint4 *>(tile + kv_v_word(D, 64 * (lane >> 3) + (lane & 7), (slot & 15) >> 2));
        ahead[0] = o.x, ahead[1] = o.y, ahead[2] = o.z, ahead[3] = o.w;
      }
    };
    fetch(hv0);
#pragma unroll 1
    for (int hv = hv0; hv < hv1; hv++) {
      const int h = hv >> 1;
      const bool isv = hv & 1;
      uint8_t *dst = static_cast<uint8_t *>(isv ? p.v : p.k);
      uint32_t coef[PASSES], raw[4], q[PASSES][2];           // q: codes, bytes of elements 0..3 and 4..7
#pragma unroll
      for (int i = 0; i < 4; i++) raw[i] = ahead[i];
#pragma unroll
      for (int ps = 0; ps < PASSES; ps++) coef[ps] = coef_ahead[ps];
      if (hv + 1 < hv1) fetch(hv + 1);
      if (!isv) {
#pragma unroll
        for (int ps = 0; ps < PASSES; ps++) {
          const uint32_t a = raw[ps] & 0x0F0F0F0Fu, b = (raw[ps] >> 4) & 0x0F0F0F0Fu;   // even and odd elements
          q[ps][0] = prmt(a, b, 0x5140u);
          q[ps][1] = prmt(a, b, 0x7362u);
        }
      } else if constexpr (n == 1) {
        q[0][0] = (raw[0] >> (4 * (m & 1))) & 0x0F0F0F0Fu;
        q[0][1] = (raw[1] >> (4 * (m & 1))) & 0x0F0F0F0Fu;
      } else {
        if (lane < D / 8) {
          const int c = lane >> 3, e = lane & 7;
#pragma unroll
          for (int i = 0; i < 4; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) bytes[r * (D / 2) + (4 * c + i) * 8 + e] = (uint8_t)(raw[i] >> (8 * r));
        }
        __syncwarp();
#pragma unroll
        for (int ps = 0; ps < PASSES; ps++) {
          const uint2 x = *reinterpret_cast<const uint2 *>(bytes + (ps * RP + sub) * (D / 2) + 8 * (m >> 1));
          q[ps][0] = (x.x >> (4 * (m & 1))) & 0x0F0F0F0Fu;
          q[ps][1] = (x.y >> (4 * (m & 1))) & 0x0F0F0F0Fu;
        }
        __syncwarp();
      }
      // float32: two lanes write their 16 elements eight at a time, so that a store fills 32-byte sectors (halves of them cost
      // the path to L2 as much as whole ones: 16381 tokens of 8 heads of 128 in 29.6 us)
      if constexpr (!BF16) {
#pragma unroll
        for (int ps = 0; ps < PASSES; ps++) {
          const uint32_t x = __shfl_xor_sync(0xffffffffu, m & 1 ? q[ps][0] : q[ps][1], 1);
          if (m & 1) q[ps][0] = x;
          else q[ps][1] = x;
        }
      }
      const int d = BF16 ? 8 * m : 8 * (m & ~1) + 4 * (m & 1);
#pragma unroll
      for (int ps = 0; ps < PASSES; ps++) {
        const int r = ps * RP + sub;
        if (r < n) {
          float v[8];
          const float s = h2f((uint16_t)coef[ps]), b = h2f((uint16_t)(coef[ps] >> 16));
          values4(q[ps][0], s, b, v);
          values4(q[ps][1], s, b, v + 4);
          if (slot < 0)
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = __int_as_float(0x7FC00000);
          store8<BF16>(dst + (((t + r) * g.kv_heads + h) * D + d) * (BF16 ? 2 : 4), v);
        }
      }
    }
  };
  each_run(p.r, unit, [&](int64_t t, int slot) { rows(std::integral_constant<int, 4>(), t, slot); },
           [&](int64_t t, int slot) { rows(std::integral_constant<int, 1>(), t, slot); });
}

}  // namespace

cudaError_t launch_kv_plan(const int32_t *cached, const int32_t *fresh, const int32_t *free_pages, int64_t n_free,
                           int32_t *table, int64_t B, int64_t max_blocks, int page, int64_t tokens, int32_t *slots,
                           int32_t *positions, int32_t *cu, int32_t *lens, int32_t *need, cudaStream_t s) {
  PlanParams p{cached, fresh, free_pages, table, slots, positions, cu, lens, need, n_free, max_blocks, tokens,
               (int)B, __builtin_ctz((unsigned)page)};
  const size_t smem = 2 * sizeof(int32_t) * (size_t)B;
  if (smem + kPlanStatic > 48 * 1024) {                    // beyond what a launch has without asking
    const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * kKvPlanMaxB);
    if (e != cudaSuccess) return e;
  }
  int64_t work = tokens > B * 32 ? tokens : B * 32;
  int64_t grid = (work + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
  grid = grid < 1 ? 1 : grid > kv_sms() ? kv_sms() : grid;
  return launch_after(plan_kernel, grid, kPlanThreads, smem, s, p);
}

cudaError_t launch_kv_append(const void *k, const void *v, bool bf16, int64_t k_token, int64_t k_head, int64_t v_token,
                             int64_t v_head, const int32_t *slots, void *cache, int64_t tokens, int64_t pages,
                             int64_t kv_heads, int64_t D, int page, int group, cudaStream_t s) {
  AppendParams p{{slots, tokens, 4, 1, 1, kv_geom(pages, kv_heads, D, page, group)}, k, v, k_token, k_head, v_token, v_head,
                 static_cast<uint8_t *>(cache)};
  const int64_t grid = row_grid(p.r);
  auto kern = D == 64 ? (bf16 ? append_kernel<true, 64> : append_kernel<false, 64>)
              : D == 128 ? (bf16 ? append_kernel<true, 128> : append_kernel<false, 128>)
                         : (bf16 ? append_kernel<true, 256> : append_kernel<false, 256>);
  return launch_after(kern, grid, kRowThreads, 0, s, p);
}

cudaError_t launch_kv_read(const int32_t *slots, const void *cache, void *k, void *v, bool bf16, int64_t tokens,
                           int64_t pages, int64_t kv_heads, int64_t D, int page, int group, cudaStream_t s) {
  ReadParams p{{slots, tokens, 4, 1, 1, kv_geom(pages, kv_heads, D, page, group)}, static_cast<const uint8_t *>(cache), k, v};
  const int64_t grid = row_grid(p.r);
  auto kern = D == 64 ? (bf16 ? read_kernel<true, 64> : read_kernel<false, 64>)
              : D == 128 ? (bf16 ? read_kernel<true, 128> : read_kernel<false, 128>)
                         : (bf16 ? read_kernel<true, 256> : read_kernel<false, 256>);
  return launch_after(kern, grid, kRowThreads, 0, s, p);
}

}  // namespace qmm
