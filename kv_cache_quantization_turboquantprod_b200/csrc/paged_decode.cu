// tq_paged_decode_attention: one query token per sequence over 4-bit pages.
//
// Bound: the pages' bytes (1.25 d per token and KV head).  At the measured
// copy rate an SM receives one cell (16 tokens of a KV head, 20 d bytes) every
// ~110 cycles at d = 128, so a warp scheduler has ~440 issue slots a cell.
//
// Split.  All cells of the batch, in the order (sequence, KV head, position),
// are cut into equal contiguous ranges, one per block (two blocks an SM, one
// at d = 256), so ragged lengths leave no tail; a range's warps take its cells
// in turn.  The part of a unit (sequence, KV head) that a range holds is
// merged across the warps; a unit inside one range goes straight to the
// output, the parts of the others (at most two a range: its first and its
// last) to the workspace, where paged_combine_kernel joins them in order.
//
// A warp is its own pipeline: one lane keeps the next cells' bulk copies in
// flight into the warp's ring, with the page number loaded one cell earlier
// still, so no warp waits for another inside a range.
//
// Products.  The codes enter the tensor cores as they are stored: a 4-bit
// field in the low bits of a half is the subnormal n 2^-24 (or n 2^-20 one
// field up), an exact fp16 operand, so eight codes cost five integer
// operations and no conversion.
//  * scores: A = codes of 16 tokens x 16 channels, B = the query of up to 8
//    heads, scaled by a power of two to fp16's top (exact for bf16 and fp16
//    queries), one f32 accumulator per group of 32 channels; then
//    x = sum_j scale_j acc_j + sum_j zero_j qsum_j, the second sum as one
//    more product with the group sums of q in two fp16 parts.
//  * values: A = codes of 16 channels x 16 tokens, B = p scale_j, f32
//    accumulators; sum p zero_j in f32 beside it.  fp16 outputs take p scale_j
//    in two fp16 parts (22 bits), bf16 outputs in one (2^-12 against the
//    output's own 2^-9).
// mma.sync carries them: 17 products of 16 x 8 x 16 a cell keep its tensor
// pipe busy a third of the time that the bytes take, and the operands come
// from registers without a trip through tensor memory.
//
// Softmax.  Weights are 2^(x - M) with a running reference M per head that
// only has to keep p scale_j below 2^14; it moves (and the accumulators with
// it) when a token exceeds it by 2^4, which one vote per cell finds out.
#include "paged.cuh"
#include "sm100.cuh"
#include "tq_common.cuh"
#include "tq_kernels.h"

namespace tq {
namespace {

using namespace sm100;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr float kTop = 10.f, kSlack = 4.f;  // p scale <= 2^10 when M moves, < 2^14 always

__host__ __device__ constexpr int blocks_per_sm(int d) { return d == 256 ? 1 : 2; }

template <int D>
struct Smem {
  static constexpr int kRing = kWarps * kStages * Cell<D>::kBytes;
  static constexpr int kBars = kRing;                            // [kWarps][kStages] u64
  static constexpr int kScan = kBars + kWarps * kStages * 8;     // 16 long long
  static constexpr int kState = kScan + 128;                     // [kWarps][8][2] floats: M, l
  static constexpr int kMerge = kState + kWarps * 8 * 2 * 4;     // [kWarps][G][D] floats
  static constexpr size_t bytes(int G) { return kMerge + (size_t)kWarps * G * D * 4; }
};

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) { return pack2<__half>(a, b); }
__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }

// Cells of a sequence; lengths beyond the table's row count as that row.
__device__ __forceinline__ int cells_of(const PagedView &c, int b) {
  const int cap = c.max_pages << c.page_shift;
  return (min(max(c.len[b], 0), cap) + kCell - 1) / kCell;
}

__device__ __forceinline__ long long warp_sum_ll(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Cells before sequence `upto` and of the whole batch, times h_kv.  All
// threads of the block (at most 256) call; scratch: 16 long long.
__device__ __forceinline__ void sum_cells(const PagedView &c, int upto, long long *scratch, long long *before,
                                          long long *total) {
  long long s = 0, t = 0;
  for (int b = threadIdx.x; b < c.batch; b += blockDim.x) {
    const int n = cells_of(c, b);
    t += n;
    if (b < upto) s += n;
  }
  s = warp_sum_ll(s);
  t = warp_sum_ll(t);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    scratch[threadIdx.x >> 5] = s;
    scratch[8 + (threadIdx.x >> 5)] = t;
  }
  __syncthreads();
  s = t = 0;
  for (int w = 0; w < warps; ++w) {
    s += scratch[w];
    t += scratch[8 + w];
  }
  __syncthreads();
  *before = s * c.h_kv;
  *total = t * c.h_kv;
}

// Cells of a block's range: an equal share, at least one per warp.
__host__ __device__ __forceinline__ long long range_cells(long long total, int blocks) {
  const long long per = (total + blocks - 1) / blocks;
  return per < kWarps ? kWarps : per;
}

// A place in the order (sequence, KV head, cell).
struct Cursor {
  int b, h, cell, cells;
  __device__ __forceinline__ void settle(const PagedView &c) {
    while (cell >= cells) {
      cell -= cells;
      if (++h == c.h_kv) {
        h = 0;
        do {
          if (++b >= c.batch) {  // past the end: never used
            cells = 0x7fffffff;
            return;
          }
          cells = cells_of(c, b);
        } while (cells == 0);
      }
    }
  }
};

template <int D, class T>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D)) paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a,
                                                                                  unsigned long long wait_ns) {
  using C = Cell<D>;
  using S = Smem<D>;
  constexpr int NG = C::kGroups, P = C::kP;
  constexpr bool kTwoParts = __is_same(T, __half);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int G = a.h_q / a.c.h_kv;
  uint8_t *const ring = smem + warp * kStages * C::kBytes;
  uint64_t *const bars = reinterpret_cast<uint64_t *>(smem + S::kBars) + warp * kStages;
  long long *const scan = reinterpret_cast<long long *>(smem + S::kScan);
  float *const state = reinterpret_cast<float *>(smem + S::kState);
  float *const merge = reinterpret_cast<float *>(smem + S::kMerge);

  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  // ---- this block's range, and the sequence it starts in
  long long total, unused;
  sum_cells(a.c, 0, scan, &unused, &total);
  pdl_trigger();
  const long long per = range_cells(total, gridDim.x);
  const long long c0 = per * blockIdx.x;
  if (c0 >= total) return;
  const int count = (int)(min(c0 + per, total) - c0);
  {
    long long base = 0;
    for (int b0 = 0; b0 < a.c.batch; b0 += kThreads) {
      const int b = b0 + tid;
      const long long n = b < a.c.batch ? (long long)cells_of(a.c, b) * a.c.h_kv : 0;
      long long inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      long long ahead = base, all = base;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) ahead += scan[w];
        all += scan[w];
      }
      __syncthreads();
      if (ahead + inc > c0 && ahead + inc - n <= c0) {
        scan[8] = b;
        scan[9] = ahead + inc - n;
      }
      base = all;
      if (base > c0) break;
    }
    __syncthreads();
  }
  Cursor here;  // the range's first cell
  here.b = (int)scan[8];
  here.cells = cells_of(a.c, here.b);
  here.h = (int)((c0 - scan[9]) / here.cells);
  here.cell = (int)((c0 - scan[9]) % here.cells);

  // ---- the warp's copies: cells warp, warp + kWarps, .. of the range
  Cursor next = here;
  next.cell += warp;
  next.settle(a.c);
  const int mine = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;
  int asked = 0;            // cells whose copy was issued
  int page = mine > 0 ? page_of(a.c, next.b, next.cell * kCell) : -1;
  uint32_t bad_stage = 0;   // stages whose cell has no page
  auto issue = [&]() {      // copy of cell `asked`; then look up the next cell's page
    if (asked >= mine) return;
    const int s = asked % kStages;
    if (page >= 0) {
      bad_stage &= ~(1u << s);
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[s], C::kBytes);
        bulk_g2s(ring + s * C::kBytes, cell_ptr<D>(a.c, page, next.cell * kCell, next.h), C::kBytes, &bars[s]);
      }
    } else {
      bad_stage |= 1u << s;
      if (lane == 0) mbar_arrive(&bars[s]);
    }
    ++asked;
    if (asked < mine) {
      next.cell += kWarps;
      next.settle(a.c);
      page = page_of(a.c, next.b, next.cell * kCell);
    }
  };
  __syncwarp();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue();

  int used = 0;             // cells taken
  int at = 0;               // first cell of the current part, counted from the range's start
  bool dead = false;        // a wait ran out
  const float kInf = INFINITY;

  while (at < count) {
    // ---- one part: cells [at, end) of the range, all of unit (here.b, here.h)
    const int end = min(count, at + here.cells - here.cell);
    const int len = a.c.len[here.b];
    bool bad = len > (a.c.max_pages << a.c.page_shift);

    // queries: head g of the unit, lane t's channels 32 j + 8 t .. + 7
    uint32_t qb[NG][4];     // (0, 4), (2, 6) at weight 1; (1, 5), (3, 7) at 1/16
    uint32_t qz[2];         // group sums of q, two fp16 parts, 2^-6
    float c1[2], c2[2];     // heads 2 t, 2 t + 1: factors of the two score sums
    {
      float x[NG][8], big = 0.f;
      const T *q = reinterpret_cast<const T *>(a.q) + (size_t)here.b * a.q_stride + (size_t)(here.h * G + g) * D + 8 * t;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if (g < G)
          load8(q + 32 * j, x[j]);
        else
#pragma unroll
          for (int e = 0; e < 8; ++e) x[j][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[j][e]));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // 2^eq big lies in [2^14, 2^15); infinities stay what they are
      const int field = (__float_as_int(big) >> 23) & 255;
      const int eq = field == 0 || field == 255 ? 0 : min(141 - field, 120);
      const float up = ldexpf(1.f, eq);
      float sum[NG];
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        sum[j] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[j][e] *= up;
          sum[j] += x[j][e];
        }
        qb[j][0] = pack_half2(x[j][0], x[j][4]);
        qb[j][1] = pack_half2(x[j][2], x[j][6]);
        qb[j][2] = pack_half2(x[j][1] * 0.0625f, x[j][5] * 0.0625f);
        qb[j][3] = pack_half2(x[j][3] * 0.0625f, x[j][7] * 0.0625f);
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
        sum[j] *= 0.015625f;
      }
      // operand slots k = 2 t + i (and + 8): group and part
      float hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j)
          if (j == (2 * t + i) % NG) v = sum[j];
        hi[i] = __half2float(__float2half_rn(v));
        lo[i] = v - hi[i];
      }
      const int part = (2 * t) / NG;
      const uint32_t ph = pack_half2(hi[0], hi[1]), pl = pack_half2(lo[0], lo[1]);
      qz[0] = NG == 8 ? ph : part == 0 ? ph : part == 1 ? pl : 0u;
      qz[1] = NG == 8 ? pl : 0u;
      const int e0 = __shfl_sync(0xffffffffu, eq, 8 * t), e1 = __shfl_sync(0xffffffffu, eq, 8 * t + 4);
      c1[0] = ldexpf(a.scale_log2, 24 - e0);
      c1[1] = ldexpf(a.scale_log2, 24 - e1);
      c2[0] = ldexpf(a.scale_log2, 6 - e0);
      c2[1] = ldexpf(a.scale_log2, 6 - e1);
    }

    float acc[2 * NG][4], zs[NG][2], M[2] = {-kInf, -kInf}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
    for (int j = 0; j < NG; ++j) zs[j][0] = zs[j][1] = 0.f;

    for (int idx = used * kWarps + warp; idx < end && !dead; idx += kWarps, ++used) {
      __syncwarp();
      issue();
      const int s = used % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars[s], (used / kStages) & 1, wait_ns))) {
        dead = true;
        if (lane == 0) atomicOr(a.c.errors, TQ_ERRF_DECODE_WAIT);
        break;
      }
      if (bad_stage >> s & 1u) {
        bad = true;
        continue;
      }
      uint8_t *const cell = ring + s * C::kBytes;
      const int valid = len - (here.cell + idx - at) * kCell;
      if (valid < kCell) {
        // slots behind the sequence may hold anything: give them scale and zero 0
        for (int i = lane; i < kCell * NG; i += 32) {
          const int n = i / NG, j = i % NG;
          if (n >= valid) {
            *reinterpret_cast<uint16_t *>(cell + C::kKeyScale + C::scale_at(n, j)) = 0;
            *reinterpret_cast<uint16_t *>(cell + C::kKeyZero + C::key_zero_at(n, j)) = 0;
            *reinterpret_cast<uint16_t *>(cell + C::kValScale + C::scale_at(n, j)) = 0;
            *reinterpret_cast<uint16_t *>(cell + C::kValZero + C::scale_at(n, j)) = 0;
          }
        }
        fence_proxy_async_smem();  // before a later copy into this stage
        __syncwarp();
      }

      // ---- scores of tokens g and g + 8 for heads 2 t and 2 t + 1
      float x[4] = {0.f, 0.f, 0.f, 0.f};  // (g, 2t), (g, 2t+1), (g+8, 2t), (g+8, 2t+1)
      const uint32_t pick = (g & 1) ? 0x7632 : 0x5410;  // halves e = g & 1 of a pair of words
#pragma unroll
      for (int jp = 0; jp < NG / P; ++jp) {
        uint32_t w0[P], w1[P];
        const uint8_t *k0 = cell + C::key_word(g, jp * P, t), *k1 = cell + C::key_word(g + 8, jp * P, t);
        if constexpr (P == 4) {
          const uint4 u = *reinterpret_cast<const uint4 *>(k0), v = *reinterpret_cast<const uint4 *>(k1);
          w0[0] = u.x; w0[1] = u.y; w0[2] = u.z; w0[3] = u.w;
          w1[0] = v.x; w1[1] = v.y; w1[2] = v.z; w1[3] = v.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(k0), v = *reinterpret_cast<const uint2 *>(k1);
          w0[0] = u.x; w0[1] = u.y;
          w1[0] = v.x; w1[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < P; i += 2) {
          // scales of groups j, j + 1: words (s, e) -> tokens g, g + 8
          const uint4 sw = *reinterpret_cast<const uint4 *>(cell + C::kKeyScale + C::scale_at(g & 7, jp * P + i) - 2 * (g & 1));
          const uint32_t pair[2] = {__byte_perm(sw.x, sw.y, pick), __byte_perm(sw.z, sw.w, pick)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = jp * P + i + k;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t u = w0[i + k], v = w1[i + k], us = u >> 8, vs = v >> 8;
            mma16(d, u & 0x000f000fu, v & 0x000f000fu, us & 0x000f000fu, vs & 0x000f000fu, qb[j][0], qb[j][1]);
            mma16(d, u & 0x00f000f0u, v & 0x00f000f0u, us & 0x00f000f0u, vs & 0x00f000f0u, qb[j][2], qb[j][3]);
            const float2 sc = unpack_half2(pair[k]);
            x[0] = fmaf(sc.x, d[0], x[0]);
            x[1] = fmaf(sc.x, d[1], x[1]);
            x[2] = fmaf(sc.y, d[2], x[2]);
            x[3] = fmaf(sc.y, d[3], x[3]);
          }
        }
      }
      {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const int zg = (2 * t) % NG;
        const uint32_t z0 = *reinterpret_cast<const uint32_t *>(cell + C::kKeyZero + C::key_zero_at(g, zg));
        const uint32_t z1 = *reinterpret_cast<const uint32_t *>(cell + C::kKeyZero + C::key_zero_at(g + 8, zg));
        mma16(d, z0, z1, z0, z1, qz[0], qz[1]);
        x[0] = fmaf(c1[0], x[0], c2[0] * d[0]);
        x[1] = fmaf(c1[1], x[1], c2[1] * d[1]);
        x[2] = fmaf(c1[0], x[2], c2[0] * d[2]);
        x[3] = fmaf(c1[1], x[3], c2[1] * d[3]);
      }
      if (valid < kCell) {
        if (g >= valid) x[0] = x[1] = -kInf;
        if (g + 8 >= valid) x[2] = x[3] = -kInf;
      }

      // ---- value scales and zeros of tokens g and g + 8
      uint32_t vs[NG], vz[NG];
#pragma unroll
      for (int j = 0; j < NG; j += 2) {
        const uint4 sw = *reinterpret_cast<const uint4 *>(cell + C::kValScale + C::scale_at(g & 7, j) - 2 * (g & 1));
        vs[j] = __byte_perm(sw.x, sw.y, pick);
        vs[j + 1] = __byte_perm(sw.z, sw.w, pick);
        const uint4 zw = *reinterpret_cast<const uint4 *>(cell + C::kValZero + C::scale_at(g & 7, j) - 2 * (g & 1));
        vz[j] = __byte_perm(zw.x, zw.y, pick);
        vz[j + 1] = __byte_perm(zw.z, zw.w, pick);
      }
      // exponent e with every scale of the two tokens below 2^e
      uint32_t top = vs[0];
#pragma unroll
      for (int j = 1; j < NG; ++j) top = __vmaxu2(top, vs[j]);
      top = max(top & 0xffffu, top >> 16);
      const float e = (float)((int)(top >> 10) - 14);
      float need[2] = {fmaxf(x[0], x[2]) + e - kTop, fmaxf(x[1], x[3]) + e - kTop};
      if (__any_sync(0xffffffffu, need[0] > M[0] + kSlack || need[1] > M[1] + kSlack)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) need[i] = fmaxf(need[i], __shfl_xor_sync(0xffffffffu, need[i], o));
          need[i] = fmaxf(need[i], M[i]);
          const float f = M[i] == -kInf ? 0.f : exp2f(M[i] - need[i]);
          M[i] = need[i];
          l[i] *= f;
#pragma unroll
          for (int k = 0; k < 2 * NG; ++k) {
            acc[k][i] *= f;
            acc[k][i + 2] *= f;
          }
#pragma unroll
          for (int j = 0; j < NG; ++j) zs[j][i] *= f;
        }
      }
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2_approx(x[i] - M[i & 1]);
      l[0] += p[0] + p[2];
      l[1] += p[1] + p[3];

      // ---- values
#pragma unroll
      for (int jp = 0; jp < NG / P; ++jp) {
        uint32_t w0[P], w1[P];
        const uint8_t *v0 = cell + C::val_half(2 * t, jp * P, g), *v1 = cell + C::val_half(2 * t + 8, jp * P, g);
        if constexpr (P == 4) {
          const uint4 u = *reinterpret_cast<const uint4 *>(v0), v = *reinterpret_cast<const uint4 *>(v1);
          w0[0] = u.x; w0[1] = u.y; w0[2] = u.z; w0[3] = u.w;
          w1[0] = v.x; w1[1] = v.y; w1[2] = v.z; w1[3] = v.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(v0), v = *reinterpret_cast<const uint2 *>(v1);
          w0[0] = u.x; w0[1] = u.y;
          w1[0] = v.x; w1[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int j = jp * P + i;
          const float2 sc = unpack_half2(vs[j]), ze = unpack_half2(vz[j]);
          zs[j][0] = fmaf(p[0], ze.x, fmaf(p[2], ze.y, zs[j][0]));
          zs[j][1] = fmaf(p[1], ze.x, fmaf(p[3], ze.y, zs[j][1]));
          const float y[4] = {p[0] * sc.x, p[1] * sc.x, p[2] * sc.y, p[3] * sc.y};
          const uint32_t h0 = pack_half2(y[0], y[1]), h1 = pack_half2(y[2], y[3]);
          const uint32_t b0 = transpose8(h0), b1 = transpose8(h1);
          const uint32_t u = w0[i], v = w1[i], us = u >> 8, vv = v >> 8;
          mma16(acc[2 * j], u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u, b0, b1);
          mma16(acc[2 * j + 1], us & 0x000f000fu, us & 0x00f000f0u, vv & 0x000f000fu, vv & 0x00f000f0u, b0, b1);
          if constexpr (kTwoParts) {
            const float2 r0 = unpack_half2(h0), r1 = unpack_half2(h1);
            const uint32_t q0 = transpose8(pack_half2(y[0] - r0.x, y[1] - r0.y));
            const uint32_t q1 = transpose8(pack_half2(y[2] - r1.x, y[3] - r1.y));
            mma16(acc[2 * j], u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u, q0, q1);
            mma16(acc[2 * j + 1], us & 0x000f000fu, us & 0x00f000f0u, vv & 0x000f000fu, vv & 0x00f000f0u, q0, q1);
          }
        }
      }
    }

    // ---- merge the part across the warps
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
#pragma unroll
        for (int j = 0; j < NG; ++j) zs[j][i] += __shfl_xor_sync(0xffffffffu, zs[j][i], o);
      }
    }
    if (bad || dead) l[0] = l[1] = __int_as_float(0x7fffffff);
    if (bad && lane == 0) atomicOr(a.c.errors, TQ_ERRF_PAGE);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = 2 * t + i;
      if (h < G) {
        if (g == 0) {
          state[(warp * 8 + h) * 2] = M[i];
          state[(warp * 8 + h) * 2 + 1] = l[i];
        }
        float *o = merge + (size_t)(warp * G + h) * D + 4 * g;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const float w = 16777216.f, z = zs[j][i];
          *reinterpret_cast<float4 *>(o + 32 * j) =
              make_float4(fmaf(acc[2 * j][i], w, z), fmaf(acc[2 * j][i + 2], w * 0.0625f, z), fmaf(acc[2 * j + 1][i], w, z),
                          fmaf(acc[2 * j + 1][i + 2], w * 0.0625f, z));
        }
      }
    }
    __syncthreads();
    const bool whole = here.cell == 0 && end - at == here.cells;
    float *const part = a.partials + ((size_t)blockIdx.x * 2 + (at == 0 ? 0 : 1)) * G * (D + 4);
    for (int i = tid; i < G * D / 4; i += kThreads) {
      const int h = i / (D / 4), c = 4 * (i % (D / 4));
      float top = -kInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, state[(w * 8 + h) * 2]);
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(state[(w * 8 + h) * 2] - top);
        const float4 v = *reinterpret_cast<const float4 *>(merge + (size_t)(w * G + h) * D + c);
        sum = fmaf(f, state[(w * 8 + h) * 2 + 1], sum);
        o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
      }
      if (whole) {
        const float r = 1.f / sum;
        T *out = reinterpret_cast<T *>(a.out) + (size_t)here.b * a.out_stride + (size_t)(here.h * G + h) * D + c;
        *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(o.x * r, o.y * r), pack2<T>(o.z * r, o.w * r));
      } else {
        *reinterpret_cast<float4 *>(part + h * D + c) = o;
        if (c == 0) {
          part[G * D + 2 * h] = top;
          part[G * D + 2 * h + 1] = sum;
        }
      }
    }
    __syncthreads();
    here.cell += end - at;
    at = end;
    if (at < count) here.settle(a.c);
  }
  // a warp that gave up still waits for its own copies
  if (dead)
    for (int i = used; i < asked; ++i) mbar_wait(&bars[i % kStages], (i / kStages) & 1);
}

// Joins the parts of each unit that more than one range holds; zeros for
// empty sequences.  One block a unit.
template <int D, class T>
__global__ void __launch_bounds__(128) paged_combine_kernel(const __grid_constant__ PagedDecodeArgs a, int blocks) {
  __shared__ long long scan[16];
  __shared__ float wt[8][512];
  const int b = blockIdx.x / a.c.h_kv, h = blockIdx.x % a.c.h_kv, tid = threadIdx.x;
  const int G = a.h_q / a.c.h_kv;
  long long before, total;
  sum_cells(a.c, b, scan, &before, &total);
  const int cells = cells_of(a.c, b);
  T *const out = reinterpret_cast<T *>(a.out) + (size_t)b * a.out_stride + (size_t)h * G * D;
  if (cells == 0) {
    pdl_wait();
    for (int i = tid; i < G * D / 8; i += 128) reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const long long per = range_cells(total, blocks);
  const long long u0 = before + (long long)h * cells, u1 = u0 + cells;
  const int first = (int)(u0 / per), last = (int)((u1 - 1) / per), n = last - first + 1;
  pdl_wait();
  if (n == 1) return;
  // the unit is the last part of its first range unless that range starts with it
  auto part = [&](int i) {
    const int slot = i == 0 && u0 % per != 0 ? 1 : 0;
    return a.partials + ((size_t)(first + i) * 2 + slot) * G * (D + 4);
  };
  __shared__ float tops[8], sums[8];
  const int warp = tid >> 5, lane = tid & 31;
  for (int hq = warp; hq < G; hq += 4) {
    float top = -INFINITY, sum = 0.f;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, part(i)[G * D + 2 * hq]);
    top = warp_max(top);
    for (int i = lane; i < n; i += 32) {
      const float f = exp2f(part(i)[G * D + 2 * hq] - top);
      if (i < 512) wt[hq][i] = f;
      sum = fmaf(f, part(i)[G * D + 2 * hq + 1], sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      tops[hq] = top;
      sums[hq] = sum;
    }
  }
  __syncthreads();
  for (int i = tid; i < G * D / 4; i += 128) {
    const int hq = i / (D / 4), c = 4 * (i % (D / 4));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float *p = part(k);
      const float f = k < 512 ? wt[hq][k] : exp2f(p[G * D + 2 * hq] - tops[hq]);
      const float4 v = *reinterpret_cast<const float4 *>(p + hq * D + c);
      o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
    }
    const float r = 1.f / sums[hq];
    *reinterpret_cast<uint2 *>(out + hq * D + c) = make_uint2(pack2<T>(o.x * r, o.y * r), pack2<T>(o.z * r, o.w * r));
  }
}

template <int D, class T>
cudaError_t launch(const PagedDecodeArgs &a, cudaStream_t stream) {
  const int G = a.h_q / a.c.h_kv, blocks = a.num_sms * blocks_per_sm(D);
  const size_t smem = Smem<D>::bytes(G);
  auto *kernel = paged_decode_kernel<D, T>;
  // (always for the widest group, so that no order of calls lowers it)
  static std::atomic<int> allowed[kAttributeDevices];
  cudaError_t e = allow_smem(kernel, Smem<D>::bytes(TQ_PAGED_MAX_GQA), allowed);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, kThreads, smem, stream>>>(a, wait_limit_ns());
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_combine_kernel<D, T>, dim3(a.c.batch * a.c.h_kv), dim3(128), 0, stream, a, blocks);
}

}  // namespace

size_t paged_decode_workspace(int d, int h_kv, int h_q, int batch, int num_sms) {
  (void)batch;
  return (size_t)num_sms * blocks_per_sm(d) * 2 * (h_q / h_kv) * (d + 4) * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedDecodeArgs &a, int d, tq_dtype dt, cudaStream_t stream) {
  const bool bf = dt == TQ_BF16;
  if (d == 64) return bf ? launch<64, __nv_bfloat16>(a, stream) : launch<64, __half>(a, stream);
  if (d == 128) return bf ? launch<128, __nv_bfloat16>(a, stream) : launch<128, __half>(a, stream);
  return bf ? launch<256, __nv_bfloat16>(a, stream) : launch<256, __half>(a, stream);
}

}  // namespace tq
