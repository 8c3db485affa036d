// kv_attend_warp.cuh -- attention over the 4-bit cache on the warp-level tensor
// cores (mma.sync m16n8k16): single tokens, drafts of a few tokens, and float32
// queries of any number.
//
// For one kv head and R = queries * (heads / kv_heads) rows of q,
//   s[t, r] = scale * sum_g ( sk[t,g] * sum_{d in g} code_k[t,d] q[r,d] + bk[t,g] * sum_{d in g} q[r,d] )
//   o[r, d] = sum_t p[t,r] sv[t,g(d)] code_v[t,d] + sum_t p[t,r] bv[t,g(d)],   p = exp(s - max)
// so the codes enter the tensor cores as they are, as exact binary16 integers
// (a masked nibble is the integer times 2^-24, and 16 times it for the upper nibble of
// a byte), and scales and biases act on 16 x 8 score tiles in float32.
//
// Orientation.  Tokens (keys) and elements (values) are the 16-wide M side, up
// to 8 rows of q the N side: S^T = K q^T, O^T = V^T P^T.  A group of up to 8
// query heads then fills an MMA's N (16 rows of q on the M side would leave half of it
// empty), and the transposed score tile becomes the B operand of the value
// product by one movmatrix per 8 x 8 block.  q is scaled per row by the power
// of two that puts its largest element in [2^14, 2^15).
//
// Precision.  HL (float32 queries): q and p * sv enter as two binary16 terms
// each, which keeps 22 bits of them.  Otherwise (bfloat16) as one: q is exact
// in it, p * sv is rounded to 11 bits.  p * sv is scaled by a power of two that follows the
// largest sv met, so small scales do not fall into binary16's
// subnormals.  MMA chains run over a unit of tokens and are then added to
// float32 registers (chains over the whole context would pick up the tensor core's truncation at every step).
//
// Work split.  Items are (request, kv head, tile of 8 NT rows); the units of
// 32 or 64 tokens of all items form one line, which is cut into equal runs, one
// a team of 4 or 8 warps, wherever the cuts fall: ragged batches and single long
// requests load all SMs alike, decided on the device from the lengths.  An item's
// start counts as units, too, and a cut near an item's border moves there, so that
// no item is begun for little.  Inside a team the warps take units in turn, each
// with a ring of its own in shared memory (cp.async, up to 4 units deep, filled across the
// ends of items: no barrier between the warps), and join at the end of an item.  An item cut
// between teams leaves partial results in the workspace; the team that finishes
// last (a counter) adds them up in the line's order, so the result does not depend on which it is.
//
// Measured (GB300; the bytes are each visible token's codes and coefficients once, at 6.78 TB/s):
//   4 requests of 60000 to 130000 tokens, 40 query and 8 kv heads of 128, float32: 115 us, 66 us of bytes (3.9 TB/s).
//     Bound: two warps a scheduler (255 registers) issue in 49 % of the cycles, between fixed latencies; the tensor pipe is 38 %
//     busy (two MMAs a product for float32).
//   64 requests of 64 to 8192 tokens, 32 and 8 heads of 128, bfloat16: 41 us, 20 us of bytes.  The start (lengths, list of items,
//     q: 4 us) and the last items' joins are a fifth of it.
//   1 request of 777 tokens, 16 and 8 heads of 128, float32: 12 us; 24 requests of drafts, heads of 64: 18 us.  Bound: latency of
//     the chain launch, lengths, pages, first tiles, join, parts.
// Slower, and gone: bulk copies with barriers (a warp waits 250 cycles for a barrier long complete and 500 to issue a copy:
// 126 against 118 us for the first case), four small CTAs an SM instead of teams in one (17.3 against 14.5 us for the third).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "kv_attend.h"
#include "kv_launch.h"
#include "kv_layout.cuh"
#include "qmm_device.cuh"
#include "sm100_ptx.cuh"

namespace qmm {
namespace kvw {

using namespace sm100;

constexpr int kMaxSegs = 32;           // items a team lists at a time
constexpr int kSmemMax = 227 * 1024;

struct Params {
  KvAttendArgs a;
  KvGeom g;
  int ratio;             // query heads per kv head
  int team;              // warps that share an item: 4 or all
  int min_units;         // units worth a team of its own
  int head;              // units that an item's start counts as
  int shift;             // the line counts units in steps of 2^shift, so that it fits 32 bits
};

// One item (or the part of it) that a team works on.
struct Seg {
  int b, kvh, r0, rows;           // rows r0 .. r0 + rows - 1 of the request's R
  int a, e;                       // units [a, e), clipped to what the rows see
  int vlo, vhi;                   // tokens that any of the rows sees
  int flo, fhi;                   // tokens that all rows see
  int base;                       // position of the request's first query
  int hi;                         // tokens that can be read
  int cu0;
  int c0, nseg;                   // first team and number of teams that share the item
};

// A team's place on the line of units (shared memory).  Once the team has begun, its first warp alone reads the place; `segs`
// and `more` are written between the two barriers around the listing and read after the second.
struct Line {
  int at, off, end;               // next step to list; the same from request b's first one on; end of the team's run
  int b, segs, last;              // request; items listed; this team adds the parts up
  int more;                       // steps are left behind those listed
};

template <int D, int G, int NT, bool HL>
struct Cfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int W = 8;                                    // warps
  static constexpr int TW = 4;                                   // warps of a small team
  static constexpr int TEAMS = W / TW;
  static constexpr int THREADS = 32 * W;
  static constexpr int UT = NT == 1 && D <= 128 ? 4 : 2;         // tiles a warp takes at a time (registers)
  static constexpr int UNIT = 16 * UT;                           // their tokens
  static constexpr int TILE = 16 * D + 128 * G;                  // bytes
  static constexpr int KS = D / 16;                              // MMA k-steps of a score
  static constexpr int QW = HL ? 4 : 2;                          // 32-bit words of q per lane and k-step
  static constexpr bool QREG = KS * NT * QW <= 32;               // q fragments stay in registers
  static constexpr int OS = D + 4;                               // row stride of the join area (floats)
  // Shared memory: the warps' rings, then an area a small team (a team of all
  // warps has them all): q fragments or, later, its warps' results | small arrays.
  static constexpr int QF = KS * NT * 32 * QW * 4;
  static constexpr int RES = ROWS * OS * 4;                      // a warp's results
  static constexpr int small = (ROWS * G * 4 /* qsum */ + ROWS * 4 /* fq */ + ROWS * 8 /* limits */ +
                                2 * ROWS * 4 /* M, L */ + 15) / 16 * 16 + kMaxSegs * (int)sizeof(Seg);
  static constexpr int rest = TEAMS * small + 2 * W * ROWS * 4 /* m, l per warp */ + W * 8 /* scan */ +
                              TEAMS * (int)sizeof(Line);
  // all warps leave results at once where two units a warp still fit beside them, else half of them after the other half
  static constexpr int RW = W * RES + rest + W * 2 * UT * TILE <= kSmemMax ? TW : TW / 2;
  static constexpr int JOIN = RW * RES > QF ? RW * RES : QF;
  static constexpr int fixed = TEAMS * JOIN + rest;
  static constexpr int fit = (kSmemMax - fixed) / (W * UT * TILE);
  static constexpr int S = fit > 4 ? 4 : fit;                    // units in flight a warp
  static_assert(S >= 2, "the ring needs two units a warp");
  static constexpr int SMEM = W * S * UT * TILE + fixed;
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  const __half2 h = *reinterpret_cast<const __half2 *>(&v);
  return __half22float2(h);
}
__device__ __forceinline__ uint32_t sub_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// x + 0 x in both halves: infinities become NaN, all else stays.  A key's infinite bias or scale may make its score -inf, which
// the softmax would take for a key that is not there.
__device__ __forceinline__ uint32_t nan_for_inf(uint32_t x) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %1;" : "=r"(d) : "r"(x), "r"(0u));
  return d;
}
// Nibble I of both halves of a word as an MMA operand: the masked code as it lies is a binary16 subnormal, which the MMA
// multiplies exactly.  Plain: nibbles 0 and 2 are code * 2^-24, 1 and 3 code * 2^-20.  But the MMA adds a product up to the
// precision that its operands' exponents give, and a subnormal's leading zeros are lost from it: with codes of 2^-24 the
// errors of float32 outputs were 5 to 10 times float32's own.  HL therefore shifts every nibble to 2^-20 (the same errors as
// with normal numbers, at 115 against 131 us for the 117 MB of 131072 tokens).
template <bool HL, int I>
__device__ __forceinline__ uint32_t operand(uint32_t x) {
  if constexpr (HL) return (I == 0 ? x << 4 : x >> (4 * I - 4)) & 0x00F000F0u;
  return (x >> (8 * (I / 2))) & (I % 2 ? 0x00F000F0u : 0x000F000Fu);
}
// The same for values: HL centres them, code - 8, which is exact, and adds 8 scale to the bias.  Weights are positive,
// so without it the sum of the products is large and the bias takes most of it back (errors 10 times as large).
template <bool HL, int I>
__device__ __forceinline__ uint32_t value_operand(uint32_t x) {
  return HL ? sub_f16(operand<HL, I>(x), 0x00800080u) : operand<HL, I>(x);
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// Exponent S with max * 2^S in [2^14, 2^15) from the largest |x|'s bits; 0 for zero and non-finite.
__device__ __forceinline__ int row_exp(uint32_t mbits) {
  if (mbits == 0u || mbits >= 0x7F800000u) return 0;
  const int S = 14 - ((int)(mbits >> 23) - 127);
  return S > 126 ? 126 : S;
}

// 16 bytes, or zeros for `bytes` 0 (nothing is read then)
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// The warps of a team; `all` is a constant of the launch.
__device__ __forceinline__ void team_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
}

// A request as the split sees it.
struct Req {
  int n, len, hi, lo, base, cu0;      // queries; tokens; readable end; first unit; position and token of the first query
  int steps, tiles;                   // steps of an item on the line, its start counted as `head` units; row tiles
  int units;
};

template <int ROWS, int UNIT>
__device__ __forceinline__ Req request(const Params &p, int b, int head) {
  Req r;
  const KvAttendArgs &a = p.a;
  r.len = max(0, a.lens[b]);
  if (a.cu) {
    const int c0 = max(0, min(a.cu[b], (int)a.tokens)), c1 = max(c0, min(a.cu[b + 1], (int)a.tokens));
    r.cu0 = c0;
    r.n = c1 - c0;
  } else {
    r.cu0 = b;
    r.n = 1;
  }
  r.base = r.len - r.n;                                     // may be negative: such queries see nothing
  r.hi = (int)min((int64_t)r.len, a.max_blocks << p.g.lg_page);
  const int64_t first = a.window > 0 ? (int64_t)r.base + 1 - a.window : 0;
  r.lo = first > 0 ? (int)min(first, (int64_t)r.hi) / UNIT : 0;
  r.tiles = r.n * p.ratio <= ROWS ? (r.n > 0) : (r.n * p.ratio + ROWS - 1) / ROWS;
  // an item without tokens still has its zeros written
  r.units = r.n == 0 ? 0 : max(1, (r.hi + UNIT - 1) / UNIT - r.lo);
  r.steps = r.n == 0 ? 0 : ((head + r.units - 1) >> p.shift) + 1;
  return r;
}

__device__ __forceinline__ int div_small(int a, int b) { return a < b ? 0 : a / b; }   // most often 0

template <int G>
__device__ __forceinline__ void load_coefs(const uint8_t *p, uint32_t (&c)[G]) {
  if constexpr (G == 1) {
    c[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (G == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    c[0] = v.x, c[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < G; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
      c[i] = v.x, c[i + 1] = v.y, c[i + 2] = v.z, c[i + 3] = v.w;
    }
  }
}

template <int D, int G, int NT, bool HL>
__global__ void __launch_bounds__(Cfg<D, G, NT, HL>::THREADS, 1) attend_warp_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D, G, NT, HL>;
  constexpr int W = C::W, ROWS = C::ROWS, KS = C::KS, QW = C::QW, OS = C::OS, UT = C::UT, UNIT = C::UNIT, S = C::S;
  constexpr int TILE = C::TILE, STAGE = UT * TILE;
  constexpr int WPL = D / 32;                    // key words per lane and row
  constexpr int WPG = WPL / G;                   // of them in a group
  constexpr int VW = D / 16;                     // value words per lane
  constexpr int CODE = HL ? 20 : 24;             // an operand is its code times 2^-CODE;
  constexpr float ODD = HL ? 1.0f : 0.0625f;     // 1 / ODD times that from an odd nibble
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lg = lane >> 2, lt = lane & 3;
  const int tw = p.team, tthreads = tw * 32;     // this team's warps and threads
  const int team = tw == W ? 0 : warp / C::TW, twarp = tw == W ? warp : warp % C::TW, tid = twarp * 32 + lane;
  uint8_t *at = smem + W * S * STAGE + team * C::JOIN;
  uint32_t *qf = reinterpret_cast<uint32_t *>(at);
  float *join = reinterpret_cast<float *>(at);
  at = smem + W * S * STAGE + C::TEAMS * C::JOIN + team * C::small;
  float *qsum = reinterpret_cast<float *>(at);   // [G][ROWS]
  float *fq = qsum + ROWS * G;                   // [ROWS]
  int *lim = reinterpret_cast<int *>(fq + ROWS); // [ROWS][2]: tokens [lo, hi) a row sees
  float *cm = reinterpret_cast<float *>(lim + 2 * ROWS), *cl = cm + ROWS;    // [ROWS]
  Seg *segs = reinterpret_cast<Seg *>(at + (ROWS * G * 4 + ROWS * 20 + 15) / 16 * 16);
  at = smem + W * S * STAGE + C::TEAMS * (C::JOIN + C::small);
  float *wm = reinterpret_cast<float *>(at) + team * tw * ROWS, *wl = wm + W * ROWS;    // [warp][ROWS]
  int *scan = reinterpret_cast<int *>(at + 2 * W * ROWS * 4);                // [2][W]
  Line *lines = reinterpret_cast<Line *>(scan + 2 * W);                      // [teams]

  const uint32_t my_ring = smem_addr(smem) + warp * S * STAGE;
  const uint8_t *ring_ptr = smem + warp * S * STAGE;
  pdl_wait();
  pdl_launch_dependents();

  // ---------------------------------------------------------------- the team's run of units
  // An item's start counts as `head` units: q, the join and the partial result
  // take a team about as long.
  const KvAttendArgs &a = p.a;
  const int B = (int)a.B, hkv = p.g.kv_heads, head = p.head;
  const int per = (B + C::THREADS - 1) / C::THREADS;
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  int64_t mine64 = 0;
  int parts_b = 0;
  Req r{};                                                           // where a thread has one request: that one
  for (int b = b0; b < b1; b++) {
    r = request<ROWS, UNIT>(p, b, head);
    mine64 += (int64_t)r.steps * r.tiles * hkv;
    parts_b = (int)min((int64_t)parts_b + (int64_t)((r.units + p.min_units - 1) / p.min_units) * r.tiles * hkv, (int64_t)1024);
  }
  const int mine = (int)min(mine64, (int64_t)0x7FFFFFFF);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  // teams asked for, and the line's length again in 2^20 steps, which does not wrap where the one in steps does
  const unsigned sums = __reduce_add_sync(0xffffffffu, (unsigned)parts_b | (unsigned)min(mine >> 20, 2047) << 16);
  if (lane == 31) scan[warp] = inc, scan[W + warp] = (int)sums;
  __syncthreads();
  int total = 0, before = inc - mine, want = 0, long_line = 0;       // want: teams, an item having one per min_units begun
#pragma unroll
  for (int w = 0; w < W; w++) {
    if (w < warp) before += scan[w];
    total += scan[w];
    want += scan[W + w] & 0xFFFF;
    long_line += (unsigned)scan[W + w] >> 16;
  }
  if (long_line >= 1536) return;                                     // offsets that overlap: not a step's
  const int A = min(min(want, total), (int)gridDim.x * (W / tw));
  if (A == 0) return;
  // Team c begins at cut c, which leaves c / A of the line before it, moved to
  // the border of its item where that is near, so that no item is begun for a few units.
  const int each = total / A, more = total - each * A;               // the first `more` teams have a step more
  const int near = min(head >> p.shift, each * 3 / 4);
#pragma unroll 1
  for (int k = 0; k < 2 * (W / tw); k++) {
    const int c = (k >> 1) * gridDim.x + blockIdx.x + (k & 1);       // few teams: on SMs of their own
    if (c > A) continue;
    const int x = c * each + min(c, more);
    Line &l = lines[k >> 1];
    if (x == total) {
      if (threadIdx.x == 0) {
        if (k & 1) l.end = x;
        else l.at = x;
      }
    } else if (before <= x && x < before + mine) {
      int b = b0, off = x - before;
      if (per > 1)
        for (;; b++) {
          r = request<ROWS, UNIT>(p, b, head);
          const int n = r.steps * r.tiles * hkv;
          if (off < n) break;
          off -= n;
        }
      const int in = off % r.steps;
      const int move = in < near ? -in : r.steps - in < near ? r.steps - in : 0;
      if (k & 1) l.end = x + move;
      else l.at = x + move, l.off = off + move, l.b = b;
    }
  }
  __syncthreads();
  const int me = team * gridDim.x + blockIdx.x;
  if (me >= A) return;
  Line *line = lines + team;
  if (line->at >= line->end) return;                                 // cuts moved onto one another: nothing to list

  int islot = 0, tslot = 0;                                          // this warp's ring: next slot to fill, to take
  uint32_t notes = 0;                                                // UT bits a slot: tiles without a page
  do {
    // -------------------------------------------------------------- list the next items: 32 requests, up to kMaxSegs items
    team_sync(team, tthreads);
    if (twarp == 0) {
      const int cb = line->b, b = cb + lane;
      const int lo = line->off, hi = lo + (line->end - line->at);    // the team's run, from request cb's first step on
      const int g = line->at - lo;                                   // that step on the line
      Req q{};
      if (b < B) q = request<ROWS, UNIT>(p, b, head);
      const int n = q.steps * q.tiles * hkv;
      int end = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += u;
      }
      const int first = end - n, s0 = max(first, lo), s1 = min(end, hi);
      const int i0 = s1 > s0 ? div_small(s0 - first, q.steps) : 0;
      const int cnt = s1 > s0 ? div_small(s1 - 1 - first, q.steps) - i0 + 1 : 0;
      int to = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += u;
      }
      const int listed = min(kMaxSegs, __shfl_sync(0xffffffffu, to, 31));
      // a lane an item: the request it is of is the first one whose items reach past it
      int src = 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (__shfl_sync(0xffffffffu, to, src + o - 1) <= lane) src += o;
      src = min(src, 31);
      Req t;
      t.steps = __shfl_sync(0xffffffffu, q.steps, src);
      t.tiles = __shfl_sync(0xffffffffu, q.tiles, src);
      t.n = __shfl_sync(0xffffffffu, q.n, src);
      t.base = __shfl_sync(0xffffffffu, q.base, src);
      t.hi = __shfl_sync(0xffffffffu, q.hi, src);
      t.lo = __shfl_sync(0xffffffffu, q.lo, src);
      t.cu0 = __shfl_sync(0xffffffffu, q.cu0, src);
      const int idx = __shfl_sync(0xffffffffu, i0, src) + lane - (__shfl_sync(0xffffffffu, to - cnt, src));
      const int i_s = __shfl_sync(0xffffffffu, first, src) + idx * t.steps, i_e = i_s + t.steps;   // the item's steps
      if (lane < listed) {
        const int x0 = max(i_s, lo) - i_s, x1 = min(i_e, hi) - i_s;
        Seg s;
        s.b = cb + src;
        s.kvh = t.tiles == 1 ? idx : idx / t.tiles;
        s.r0 = (idx - s.kvh * t.tiles) * ROWS;
        s.rows = min(ROWS, t.n * p.ratio - s.r0);
        const int f = div_small(s.r0, p.ratio), l = div_small(s.r0 + s.rows - 1, p.ratio);   // first and last query of the tile
        const int64_t w = a.window > 0 ? a.window : (int64_t)1 << 40;
        auto clip = [&](int64_t v) { return (int)(v < 0 ? 0 : v > t.hi ? t.hi : v); };
        s.vlo = clip((int64_t)t.base + f + 1 - w);
        s.vhi = clip((int64_t)t.base + l + 1);
        s.flo = clip((int64_t)t.base + l + 1 - w);
        s.fhi = clip((int64_t)t.base + f + 1);
        auto unit = [&](int x) { return t.lo + (int)max((int64_t)0, ((int64_t)x << p.shift) - head); };
        s.a = max(unit(x0), s.vlo / UNIT);
        s.e = min(unit(x1), (s.vhi + UNIT - 1) / UNIT);
        if (s.vhi <= s.vlo) s.e = s.a;
        s.base = t.base;
        s.hi = t.hi;
        s.cu0 = t.cu0;
        // The teams of the item: a cut is, once moved, at or before the item's first step if it falls before
        // step `near` (or the item's end), and before the item's end if it is not moved there.  The last cut
        // at or before a step is that of the team which has the step before cuts are moved.
        auto owner = [&](int x) {
          const int longer = more * (each + 1);
          return x < longer ? x / (each + 1) : more + (x - longer) / each;
        };
        const int to_first = max(1, min(near, t.steps)), to_last = near > 0 ? max(t.steps - near + 1, to_first) : t.steps;
        s.c0 = owner(g + i_s + to_first - 1);
        s.nseg = owner(g + i_s + to_last - 1) - s.c0 + 1;
        segs[lane] = s;
      }
      // where the list ends, the request that holds that step, and the place in it
      const int stop = listed > 0 ? __shfl_sync(0xffffffffu, min(i_e, hi), listed - 1) : __shfl_sync(0xffffffffu, end, 31);
      const unsigned m = __ballot_sync(0xffffffffu, end > stop);
      const int nx = m ? __ffs(m) - 1 : 31;
      const int nx_first = __shfl_sync(0xffffffffu, first, nx), nx_end = __shfl_sync(0xffffffffu, end, nx);
      if (lane == 0) {
        line->segs = listed;
        line->b = m ? cb + nx : cb + 32;
        line->off = m ? stop - nx_first : stop - nx_end;
        line->at = g + stop;
        line->more = stop < hi && line->b < B;
      }
    }
    team_sync(team, tthreads);
    const int nsegs = line->segs;
    if (nsegs == 0) continue;                                        // 32 requests without an item

    // -------------------------------------------------------------- producer: this warp's units, in order
    // Each lane holds the page of a part of one of the warp's next units (a unit
    // has 1, 2 or 4 parts, after the page size).
    const int lg_parts = UNIT > p.g.page ? (UNIT == 4 * p.g.page ? 2 : 1) : 0;
    const uint8_t *cache_lane = static_cast<const uint8_t *>(a.cache) + lane * 16;
    const int64_t page_bytes = (int64_t)hkv * p.g.head_bytes;
    int ps = -1, pu = 0, pe = 0, pk = 0, pid = -1;                   // segment, next unit, end, place among the lanes
    auto fetch_pages = [&]() {
      const Seg &s = segs[ps];
      const int64_t tok = (int64_t)(pu + (lane >> lg_parts) * tw) * UNIT + (lane & ((1 << lg_parts) - 1)) * p.g.page;
      pid = tok < s.vhi && tok < (int64_t)pe * UNIT ? a.table[s.b * a.max_blocks + (tok >> p.g.lg_page)] : -1;
      pk = 0;
    };
    auto open_seg = [&]() {                                          // the next segment that has a unit for this warp
      while (++ps < nsegs) {
        pu = segs[ps].a + twarp;
        pe = segs[ps].e;
        if (pu < pe) return fetch_pages();
      }
    };
    // One unit into the ring, as one group of copies (an empty one past the end,
    // so that the count of groups stays that of units).  A tile without a page is zeros.
    auto issue = [&]() {
      if (ps < nsegs) {
        const int tile0 = (pu * UNIT & (p.g.page - 1)) >> 4, kvh = segs[ps].kvh;
        uint32_t dst = my_ring + islot * STAGE + lane * 16, note = 0;
#pragma unroll
        for (int i = 0; i < UT; i++) {
          const int pg = __shfl_sync(0xffffffffu, pid, (pk << lg_parts) + (i << lg_parts) / UT);
          const bool v = pg >= 0 && pg < p.g.pages;
          const uint8_t *src = cache_lane + (v ? pg * page_bytes : 0) + kvh * p.g.head_bytes +
                               ((tile0 + i) & ((p.g.page >> 4) - 1)) * TILE;
          if (!v) note |= 1u << i;
#pragma unroll
          for (int o = 0; o < TILE; o += 512)
            if (o + 512 <= TILE || o + lane * 16 < TILE) cp_async16z(dst + i * TILE + o, src + o, v ? 16u : 0u);
        }
        notes = (notes & ~(((1u << UT) - 1) << (UT * islot))) | note << (UT * islot);
        islot = islot + 1 == S ? 0 : islot + 1;
        pu += tw;
        if (pu >= pe) open_seg();
        else if (++pk == (32 >> lg_parts)) fetch_pages();
      }
      cp_async_commit();
    };

    // A segment's q: eight elements of a row a thread, fetched while the warps of the segment before it join.
    constexpr int PIECES = ROWS * (D / 8), QI = (PIECES + C::TW * 32 - 1) / (C::TW * 32), QV = HL ? 2 : 1;
    uint4 qraw[QI][QV];
    auto fetch_q = [&](const Seg &s) {
#pragma unroll
      for (int it = 0; it < QI; it++) {
        const int i = tid + it * tthreads, row = i / (D / 8), m = i % (D / 8);
        if (i < PIECES && row < s.rows) {
          const int r = s.r0 + row, qi = div_small(r, p.ratio), hq = r - qi * p.ratio;
          const int64_t off = (int64_t)(s.cu0 + qi) * a.q_token + (int64_t)(s.kvh * p.ratio + hq) * a.q_head + 8 * m;
          const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.q) + off * (HL ? 4 : 2));
#pragma unroll
          for (int j = 0; j < QV; j++) qraw[it][j] = src[j];
        } else {
#pragma unroll
          for (int j = 0; j < QV; j++) qraw[it][j] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    fetch_q(segs[0]);
    open_seg();
    for (int s = 0; s < S; s++) issue();

    for (int si = 0; si < nsegs; si++) {
      const Seg &sg = segs[si];
      const int rows = sg.rows;
      if (si > 0) team_sync(team, tthreads);                         // the results of the segment before are read
      // ------------------------------------------------------------ q -> fragments, sums, limits
#pragma unroll
      for (int it = 0; it < QI; it++) {
        const int i = tid + it * tthreads, row = i / (D / 8), m = i % (D / 8);
        if (i >= PIECES) break;                                      // whole warps: D / 8 lanes a row
        float v[8];
        if constexpr (HL) {
          const uint32_t u[8] = {qraw[it][0].x, qraw[it][0].y, qraw[it][0].z, qraw[it][0].w,
                                 qraw[it][QV - 1].x, qraw[it][QV - 1].y, qraw[it][QV - 1].z, qraw[it][QV - 1].w};
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] = __uint_as_float(u[j]);
        } else {
          const uint32_t u[4] = {qraw[it][0].x, qraw[it][0].y, qraw[it][0].z, qraw[it][0].w};
#pragma unroll
          for (int j = 0; j < 4; j++) v[2 * j] = __uint_as_float(u[j] << 16), v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) mx = max(mx, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 1; o < D / 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int ex = row_exp(mx);
        const float f = pow2i(ex);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] *= f, sum += v[j];
#pragma unroll
        for (int o = 1; o < D / G / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (m % (D / G / 8) == 0) qsum[m / (D / G / 8) * ROWS + row] = sum * pow2i(-CODE);
        if (m == 0) {
          // log2(e); never 0, which a masked score of -inf would make NaN
          fq[row] = fmaxf(ldexpf(a.scale * 1.44269504088896340736f, CODE - ex), 1.17549435e-38f);
          const int qi = div_small(sg.r0 + row, p.ratio);
          const int64_t pos = (int64_t)sg.base + qi;
          const int64_t lo = a.window > 0 ? pos + 1 - a.window : 0;
          lim[2 * row] = (int)max((int64_t)0, min(lo, (int64_t)sg.hi));
          lim[2 * row + 1] = row < rows ? (int)max((int64_t)0, min(pos + 1, (int64_t)sg.hi)) : 0;
        }
        // word w = m / 4 of lane (row % 8, t = m % 4): k-steps 2w (nibbles 0 4 | 1 5) and 2w + 1 (2 6 | 3 7)
        const int w = m >> 2, t = m & 3, n = row >> 3, ln = (row & 7) * 4 + t;
#pragma unroll
        for (int st = 0; st < 2; st++) {
          const float x0 = v[2 * st], x1 = v[2 * st + 4], z0 = v[2 * st + 1] * ODD, z1 = v[2 * st + 5] * ODD;
          uint32_t *dst = qf + (((2 * w + st) * NT + n) * 32 + ln) * QW;
          const uint32_t h0 = pack_f16(x0, x1), h1 = pack_f16(z0, z1);
          dst[0] = h0, dst[1] = h1;
          if constexpr (HL) {
            const float2 e0 = unpack_f16(h0), e1 = unpack_f16(h1);
            dst[2] = pack_f16(x0 - e0.x, x1 - e0.y), dst[3] = pack_f16(z0 - e1.x, z1 - e1.y);
          }
        }
      }
      team_sync(team, tthreads);

      uint32_t qr[C::QREG ? KS : 1][NT][QW];
      auto load_q = [&](int ks, int n, uint32_t (&d)[QW]) {
        const uint32_t *src = qf + ((ks * NT + n) * 32 + lane) * QW;
        if constexpr (HL) {
          const uint4 v = *reinterpret_cast<const uint4 *>(src);
          d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(src);
          d[0] = v.x, d[1] = v.y;
        }
      };
      if constexpr (C::QREG) {
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int n = 0; n < NT; n++) load_q(ks, n, qr[ks][n]);
      }
      float f[NT][2];
#pragma unroll
      for (int n = 0; n < NT; n++) f[n][0] = fq[8 * n + 2 * lt], f[n][1] = fq[8 * n + 2 * lt + 1];

      const float NINF = __int_as_float(0xFF800000);
      float o[NT][VW][4], ob[NT][2][G], mr[NT][2], lr[NT][2];
      float mu[NT][2];                                               // the running maximum, 0 where nothing was seen
#pragma unroll
      for (int n = 0; n < NT; n++) {
#pragma unroll
        for (int w = 0; w < VW; w++) o[n][w][0] = o[n][w][1] = o[n][w][2] = o[n][w][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; c++) {
          mr[n][c] = NINF, mu[n][c] = 0.0f, lr[n][c] = 0.0f;
#pragma unroll
          for (int g = 0; g < G; g++) ob[n][c][g] = 0.0f;
        }
      }
      int ve = 1;                                                    // largest exponent field among the value scales so far
      float vf = pow2i(28);                                          // 2^(29 - ve)
      const int tk = 4 * (lg >> 1) + 2 * (lg & 1);                   // token of row lg in its tile; row lg + 8 is the next one

      for (int u = sg.a + twarp; u < sg.e; u += tw) {
        cp_async_wait<S - 1>();
        __syncwarp();
        const uint8_t *st = ring_ptr + tslot * STAGE;
        const uint32_t note = (notes >> (UT * tslot)) & ((1u << UT) - 1);
        tslot = tslot + 1 == S ? 0 : tslot + 1;
        const bool full = note == 0 && u * UNIT >= sg.flo && u * UNIT + UNIT <= sg.fhi;

        // ---------------------------------------------------------- scores of the unit
        float y[UT][NT][4];
#pragma unroll
        for (int i0 = 0; i0 < UT; i0 += 2) {                         // two tiles share the q operands
          uint32_t kw[2][2][WPL], kc[2][2][G];                       // tile, row half
#pragma unroll
          for (int i = 0; i < 2; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const uint8_t *tile = st + (i0 + i) * TILE;
              const int row = lg + 8 * h;
              if constexpr (WPL == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(tile + (row * 4 + lt) * 8);
                kw[i][h][0] = v.x, kw[i][h][1] = v.y;
              } else {
#pragma unroll
                for (int c = 0; c < WPL / 4; c++) {
                  const uint4 v = *reinterpret_cast<const uint4 *>(tile + ((c * 16 + row) * 4 + lt) * 16);
                  kw[i][h][4 * c] = v.x, kw[i][h][4 * c + 1] = v.y, kw[i][h][4 * c + 2] = v.z, kw[i][h][4 * c + 3] = v.w;
                }
              }
              load_coefs<G>(tile + 16 * D + row * G * 4, kc[i][h]);
            }
#pragma unroll
          for (int g = 0; g < G; g++) {
            float c[2][NT][4];
#pragma unroll
            for (int w = g * WPG; w < (g + 1) * WPG; w++) {
#pragma unroll
              for (int s2 = 0; s2 < 2; s2++) {
                uint32_t qv[NT][QW];
#pragma unroll
                for (int n = 0; n < NT; n++) {
                  if constexpr (C::QREG) {
#pragma unroll
                    for (int j = 0; j < QW; j++) qv[n][j] = qr[2 * w + s2][n][j];
                  } else {
                    load_q(2 * w + s2, n, qv[n]);
                  }
                }
#pragma unroll
                for (int i = 0; i < 2; i++) {
                  const uint32_t x0 = kw[i][0][w], x1 = kw[i][1][w];
                  const uint32_t a0 = s2 ? operand<HL, 2>(x0) : operand<HL, 0>(x0), a1 = s2 ? operand<HL, 2>(x1) : operand<HL, 0>(x1);
                  const uint32_t a2 = s2 ? operand<HL, 3>(x0) : operand<HL, 1>(x0), a3 = s2 ? operand<HL, 3>(x1) : operand<HL, 1>(x1);
#pragma unroll
                  for (int n = 0; n < NT; n++) {
                    if (w == g * WPG && s2 == 0) mma_z(c[i][n], a0, a1, a2, a3, qv[n][0], qv[n][1]);
                    else mma(c[i][n], a0, a1, a2, a3, qv[n][0], qv[n][1]);
                    if constexpr (HL) mma(c[i][n], a0, a1, a2, a3, qv[n][2], qv[n][3]);
                  }
                }
              }
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
              const float2 qs = *reinterpret_cast<const float2 *>(qsum + g * ROWS + 8 * n + 2 * lt);
#pragma unroll
              for (int i = 0; i < 2; i++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                  const float2 k = unpack_f16(nan_for_inf(kc[i][h][g]));     // scale, bias
                  const float t0 = g == 0 ? k.y * qs.x : fmaf(k.y, qs.x, y[i0 + i][n][2 * h]);
                  const float t1 = g == 0 ? k.y * qs.y : fmaf(k.y, qs.y, y[i0 + i][n][2 * h + 1]);
                  y[i0 + i][n][2 * h] = fmaf(k.x, c[i][n][2 * h], t0);
                  y[i0 + i][n][2 * h + 1] = fmaf(k.x, c[i][n][2 * h + 1], t1);
                }
            }
          }
        }
        uint32_t vc[UT][2][G];                                        // value scale and bias: tile, row half, group
#pragma unroll
        for (int i = 0; i < UT; i++)
#pragma unroll
          for (int h = 0; h < 2; h++) load_coefs<G>(st + i * TILE + 16 * D + 64 * G + (lg + 8 * h) * G * 4, vc[i][h]);
        // A token that some rows do not see may hold infinite or NaN value coefficients, which reach those that do see it whatever
        // its weight there (0, where its exponential underflows).
        bool guard = false;
        if (!full) {
          uint32_t worst = 0;
#pragma unroll
          for (int i = 0; i < UT; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const int tok = u * UNIT + 16 * i + tk + h;
              const bool there = ((note >> i) & 1) == 0 && tok >= sg.vlo && tok < sg.vhi;
#pragma unroll
              for (int n = 0; n < NT; n++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                  const int2 l = *reinterpret_cast<const int2 *>(lim + 2 * (8 * n + 2 * lt + c));
                  if (!there || tok < l.x || tok >= l.y) y[i][n][2 * h + c] = NINF;
                }
#pragma unroll
              for (int g = 0; g < G; g++) {
                if (!there) vc[i][h][g] = 0u;
                worst = __vmaxu2(worst, vc[i][h][g] & 0x7FFF7FFFu);
              }
            }
          guard = __any_sync(0xffffffffu, (worst & 0xFFFFu) >= 0x7C00u || worst >= 0x7C000000u);
        }

        // ---------------------------------------------------------- running maximum and largest value scale
        // Both move in the first units of an item and seldom after: one vote
        // asks whether any lane met a larger one, and only then is what is summed so far rescaled.
        uint32_t smax = vc[0][0][0];
#pragma unroll
        for (int i = 0; i < UT; i++)
#pragma unroll
          for (int h = 0; h < 2; h++)
#pragma unroll
            for (int g = 0; g < G; g++) smax = __vmaxu2(smax, vc[i][h][g]);
        bool grow = (int)((smax & 0xFFFFu) >> 10) > ve;              // a negative scale is above all others here
        float mx[NT][2];
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int c = 0; c < 2; c++) {
            float v = fmaxf(y[0][n][c], y[0][n][2 + c]);
#pragma unroll
            for (int i = 1; i < UT; i++) v = fmaxf(v, fmaxf(y[i][n][c], y[i][n][2 + c]));
            mx[n][c] = v * f[n][c];
            grow |= mx[n][c] > mr[n][c];
          }
        if (__any_sync(0xffffffffu, grow)) {
          smax = 0;                                                  // now of magnitudes
#pragma unroll
          for (int i = 0; i < UT; i++)
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
              for (int g = 0; g < G; g++) smax = max(smax, vc[i][h][g] & 0x7FFFu);
          const int ve2 = max(ve, (int)(__reduce_max_sync(0xffffffffu, smax) >> 10));
          const float vr = pow2i(ve - ve2);                          // what is summed so far, in the new units
          ve = ve2;
          vf = pow2i(29 - ve2);                                      // largest scale -> [2^14, 2^15)
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int c = 0; c < 2; c++) {
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) mx[n][c] = fmaxf(mx[n][c], __shfl_xor_sync(0xffffffffu, mx[n][c], off));
              const float mn = fmaxf(mr[n][c], mx[n][c]);
              const float alpha = mn == mr[n][c] ? 1.0f : ex2(mr[n][c] - mn);
              mr[n][c] = mn;
              mu[n][c] = mn == NINF ? 0.0f : mn;
              lr[n][c] *= alpha;
#pragma unroll
              for (int g = 0; g < G; g++) ob[n][c][g] *= alpha;
#pragma unroll
              for (int w = 0; w < VW; w++) o[n][w][c] *= alpha * vr, o[n][w][2 + c] *= alpha * vr;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int c = 0; c < 2; c++)
#pragma unroll
            for (int i = 0; i < UT; i++)
#pragma unroll
              for (int h = 0; h < 2; h++) {
                const float e = ex2(fmaf(y[i][n][2 * h + c], f[n][c], -mu[n][c]));
                y[i][n][2 * h + c] = e;
                lr[n][c] += e;
              }
        // ---------------------------------------------------------- p * sv as B operands, bias sums
        uint32_t pf[UT][G][NT][HL ? 4 : 2];
        auto weigh = [&](auto guarded) {
          uint32_t hidden = 0;                                       // a bit a (tile, row half, row of q) that does not see the token
          if constexpr (decltype(guarded)::value) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
              for (int c = 0; c < 2; c++) {
                const int2 l = *reinterpret_cast<const int2 *>(lim + 2 * (8 * n + 2 * lt + c));
#pragma unroll
                for (int i = 0; i < UT; i++)
#pragma unroll
                  for (int h = 0; h < 2; h++) {
                    const int tok = u * UNIT + 16 * i + tk + h;
                    if (tok < l.x || tok >= l.y) hidden |= 1u << (((2 * i + h) * NT + n) * 2 + c);
                  }
              }
          }
#pragma unroll
          for (int g = 0; g < G; g++)
#pragma unroll
            for (int i = 0; i < UT; i++)
#pragma unroll
              for (int h = 0; h < 2; h++) {
                const float2 sv = unpack_f16(vc[i][h][g]);
                const float bias = HL ? fmaf(8.0f, sv.x, sv.y) : sv.y, ss = sv.x * vf;
#pragma unroll
                for (int n = 0; n < NT; n++) {
                  const float p0 = y[i][n][2 * h], p1 = y[i][n][2 * h + 1];
                  float e0 = p0 * ss, e1 = p1 * ss;
                  if constexpr (decltype(guarded)::value) {
                    const int bit = ((2 * i + h) * NT + n) * 2;
                    if ((hidden >> bit) & 1u) e0 = 0.0f;
                    else ob[n][0][g] = fmaf(p0, bias, ob[n][0][g]);
                    if ((hidden >> (bit + 1)) & 1u) e1 = 0.0f;
                    else ob[n][1][g] = fmaf(p1, bias, ob[n][1][g]);
                  } else {
                    ob[n][0][g] = fmaf(p0, bias, ob[n][0][g]);
                    ob[n][1][g] = fmaf(p1, bias, ob[n][1][g]);
                  }
                  const uint32_t hi = pack_f16(e0, e1);
                  pf[i][g][n][h] = movmatrix(hi);
                  if constexpr (HL) {
                    const float2 r = unpack_f16(hi);
                    pf[i][g][n][2 + h] = movmatrix(pack_f16(e0 - r.x, e1 - r.y));
                  }
                }
              }
        };
        if (!guard) weigh(std::false_type());
        else weigh(std::true_type());
        // ---------------------------------------------------------- values
#pragma unroll
        for (int c = 0; c < VW / 4; c++) {
          uint32_t vw[UT][4];
#pragma unroll
          for (int i = 0; i < UT; i++) {
            const uint4 v = *reinterpret_cast<const uint4 *>(st + i * TILE + 8 * D + (c * 32 + lane) * 16);
            vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
          }
#pragma unroll
          for (int x = 0; x < 4; x++) {
            const int w = 4 * c + x, g = w / (VW / G);
            float d[NT][4];
#pragma unroll
            for (int i = 0; i < UT; i++) {
              const uint32_t a0 = value_operand<HL, 0>(vw[i][x]), a1 = value_operand<HL, 1>(vw[i][x]);
              const uint32_t a2 = value_operand<HL, 2>(vw[i][x]), a3 = value_operand<HL, 3>(vw[i][x]);
#pragma unroll
              for (int n = 0; n < NT; n++) {
                if (i == 0) mma_z(d[n], a0, a1, a2, a3, pf[i][g][n][0], pf[i][g][n][1]);
                else mma(d[n], a0, a1, a2, a3, pf[i][g][n][0], pf[i][g][n][1]);
                if constexpr (HL) mma(d[n], a0, a1, a2, a3, pf[i][g][n][2], pf[i][g][n][3]);
              }
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
#pragma unroll
              for (int r = 0; r < 4; r++) o[n][w][r] += d[n][r];
            }
          }
        }
        __syncwarp();                                                // every lane has read the unit
        issue();
      }

      if (si + 1 < nsegs) fetch_q(segs[si + 1]);
      // ------------------------------------------------------------ join the warps
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            lr[n][c] += __shfl_xor_sync(0xffffffffu, lr[n][c], off);
#pragma unroll
            for (int g = 0; g < G; g++) ob[n][c][g] += __shfl_xor_sync(0xffffffffu, ob[n][c][g], off);
          }
          if (lg == 0) wm[twarp * ROWS + 8 * n + 2 * lt + c] = mr[n][c], wl[twarp * ROWS + 8 * n + 2 * lt + c] = lr[n][c];
        }
      team_sync(team, tthreads);
      // every warp's share in units of the common maximum
      const float unit = pow2i(CODE - 29 + ve);                      // 2^CODE / 2^(29 - ve)
      float sc[NT][2];
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const int row = 8 * n + 2 * lt + c;
          float M = NINF;
          for (int w = 0; w < tw; w++) M = fmaxf(M, wm[w * ROWS + row]);
          const float m0 = M == NINF ? 0.0f : M;
          sc[n][c] = ex2(mr[n][c] - m0);
          if (twarp == 0 && lg == 0) {
            float L = 0.0f;
            for (int w = 0; w < tw; w++) L = fmaf(wl[w * ROWS + row], ex2(wm[w * ROWS + row] - m0), L);
            cm[row] = M, cl[row] = L;
          }
        }
      auto each_out = [&](auto fn) {                                     // fn(row, element, value) over this lane's outputs
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int w = 0; w < VW; w++) {
            const int g = w / (VW / G);
#pragma unroll
            for (int r = 0; r < 4; r++) {
              const int c = r & 1;
              const float v = fmaf(o[n][w][r], r < 2 ? unit : unit * ODD, ob[n][c][g]) * sc[n][c];
              fn(8 * n + 2 * lt + c, 16 * w + lg + (r < 2 ? 0 : 8), v);
            }
          }
      };
      constexpr bool AT_ONCE = C::RW == C::TW;
      const int half = AT_ONCE ? tw : tw / 2;                        // results side by side
      if (AT_ONCE || twarp >= half) {
        float *j = join + (AT_ONCE ? twarp : twarp - half) * ROWS * OS;
        each_out([&](int row, int d, float v) { j[row * OS + d] = v; });
      }
      team_sync(team, tthreads);
      if constexpr (!AT_ONCE) {
        if (twarp < half) {
          float *j = join + twarp * ROWS * OS;
          each_out([&](int row, int d, float v) { j[row * OS + d] += v; });
        }
        team_sync(team, tthreads);
      }
      // ------------------------------------------------------------ the item's rows, whole or as a partial result
      auto put_row = [&](int row, int d, float4 v) {
        const int r = sg.r0 + row, qi = div_small(r, p.ratio), hq = r - qi * p.ratio;
        const int64_t off = ((int64_t)(sg.cu0 + qi) * a.heads + sg.kvh * p.ratio + hq) * D + d;
        if constexpr (HL) {
          *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + off) = v;
        } else {
          const __nv_bfloat162 h0 = __floats2bfloat162_rn(v.x, v.y), h1 = __floats2bfloat162_rn(v.z, v.w);
          *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + off) =
              make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
        }
      };
      constexpr int PART = ROWS * (D + 2);                           // floats of a partial result: maxima, sums, rows
      float *parts = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + 4 * kKvMaxCtas);
      const bool whole = sg.nseg == 1;
      float *mine_p = parts + (int64_t)(2 * me + (me == sg.c0 ? 1 : 0)) * PART;
      for (int i = tid; i < rows * (D / 4); i += tthreads) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = 0; w < half; w++) {
          const float4 x = *reinterpret_cast<const float4 *>(join + (w * ROWS + row) * OS + d);
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        if (whole) {
          const float L = cl[row], inv = L == 0.0f ? 0.0f : 1.0f / L;
          v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
          put_row(row, d, v);
        } else {
          __stcg(reinterpret_cast<float4 *>(mine_p + 2 * ROWS + row * D + d), v);
        }
      }
      if (!whole) {
        if (tid < rows) __stcg(mine_p + tid, cm[tid]), __stcg(mine_p + ROWS + tid, cl[tid]);
        __threadfence();
        team_sync(team, tthreads);
        unsigned *count = static_cast<unsigned *>(a.workspace) + sg.c0;
        if (tid == 0) {
          const unsigned old = atomicAdd(count, 1u);
          line->last = old == (unsigned)sg.nseg - 1;
        }
        team_sync(team, tthreads);
        if (line->last) {                                              // every other part is in: add them in CTA order
          __threadfence();
          auto part = [&](int k) { return parts + (int64_t)(2 * (sg.c0 + k) + (k == 0 ? 1 : 0)) * PART; };
          // weights of the parts a row: 2^(m_k - M) / L, kept where the warps' results were
          float *wt = join;                                          // [nseg][ROWS], as many parts at a time as fit
          constexpr int FIT = C::JOIN / 4 / ROWS;
          for (int row = twarp; row < rows; row += tw) {
            float M = NINF, L = 0.0f;                                // online over the lane's parts, then over lanes
            for (int k = lane; k < sg.nseg; k += 32) {
              const float m = __ldcg(part(k) + row), l = __ldcg(part(k) + ROWS + row);
              const float mn = fmaxf(M, m), m0 = mn == NINF ? 0.0f : mn;
              L = L * ex2(M - m0) + l * ex2(m - m0);
              M = mn;
              if (k < FIT) wt[k * ROWS + row] = m;
            }
            float mx = M;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float m0 = mx == NINF ? 0.0f : mx;
            L *= ex2(M - m0);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            for (int k = lane; k < min(sg.nseg, FIT); k += 32) wt[k * ROWS + row] = ex2(wt[k * ROWS + row] - m0) * inv;
            if (lane == 0) cm[row] = m0, cl[row] = inv;
          }
          team_sync(team, tthreads);
          for (int i = tid; i < rows * (D / 4); i += tthreads) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            constexpr int AT = 8;                                    // loads in flight
            for (int k0 = 0; k0 < sg.nseg; k0 += AT) {
              float4 x[AT];
#pragma unroll
              for (int j = 0; j < AT; j++)
                if (k0 + j < sg.nseg) x[j] = __ldcg(reinterpret_cast<const float4 *>(part(k0 + j) + 2 * ROWS + row * D + d));
#pragma unroll
              for (int j = 0; j < AT; j++)
                if (k0 + j < sg.nseg) {
                  const int k = k0 + j;
                  const float w = k < FIT ? wt[k * ROWS + row] : ex2(__ldcg(part(k) + row) - cm[row]) * cl[row];
                  v.x = fmaf(w, x[j].x, v.x), v.y = fmaf(w, x[j].y, v.y);
                  v.z = fmaf(w, x[j].z, v.z), v.w = fmaf(w, x[j].w, v.w);
                }
            }
            put_row(row, d, v);
          }
          if (tid == 0) *count = 0u;
        }
      }
    }
  } while (line->more);
}

// ---------------------------------------------------------------- host side

template <int D, int G, int NT, bool HL>
cudaError_t launch(const KvAttendArgs &a, cudaStream_t s) {
  using C = Cfg<D, G, NT, HL>;
  Params p{};
  p.a = a;
  p.g = kv_geom(a.pages, a.kv_heads, a.head_dim, a.page, a.group);
  if (a.pages == 0) p.g.head_bytes = 0;                // addresses stay in the workspace, which stands for an empty cache
  p.ratio = (int)(a.heads / a.kv_heads);
  // Items that far outnumber the SMs go to small teams, whose joins overlap; fewer
  // items to whole CTAs, which leave fewer parts to add up.  Small teams / whole CTAs in us, caches cold, bfloat16 of 64 to 8192
  // tokens, heads of 128: 64 items 24.7 / 23.6, 192: 31.8 / 33.8, 288: 35.0 / 37.0, 312: 36.0 / 38.0, 400: 40.1 / 43.1, 768: 58.5 / 65.7.
  // float32 of 600 tokens, heads of 64: 64 items 19.6 / 14.5, 192: 21.6 / 21.6, 288: 27.8 / 22.7, 312: 25.7 / 27.7, 400: 28.5 / 27.8,
  // 768: 33.9 / 44.2.  bfloat16 of 4000 tokens, heads of 256: 64 items 37.0 / 36.0, 288: 83.1 / 84.1, 312: 87.2 / 89.2, 768: 173 / 179.
  // So the border is not sharp: between 130 and 400 items either is ahead by a few us, after the tokens.  Captured in a
  // graph: 8 items of 777 tokens 14.5 / 11.6, 32 of 60000 and more 119 / 117.
  const int64_t items = a.B * a.kv_heads * ((a.max_fresh * p.ratio + C::ROWS - 1) / C::ROWS);
  p.team = items > 2 * kv_max_ctas(1) ? C::TW : C::W;
  // (units a warp of 1 / 1.5 / 2 / 3 for an item's start: 46.0 / 42.4 / 41.0 / 42.8 us for the 512 items; one unit a warp as
  // the least that is worth a team: 14.1 us for the 8 items)
  p.min_units = 2 * p.team;
  p.head = 2 * p.team;
  // the most steps that the line can have, in 32 bits
  const double most = ((double)a.tokens * a.heads / C::ROWS + (double)a.tokens * a.kv_heads) *
                      ((double)a.max_blocks * a.page / C::UNIT + 2 + p.head);
  while (most / (1 << p.shift) > 1e9) p.shift++;
  static std::atomic<int> set_for{0};
  return launch_large(attend_warp_kernel<D, G, NT, HL>, kv_max_ctas(1), C::THREADS, C::SMEM, s, p, set_for);
}

}  // namespace kvw
}  // namespace qmm
