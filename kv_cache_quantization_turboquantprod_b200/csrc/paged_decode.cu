// tq_paged_decode_attention: one query token per sequence over 4-bit pages.
//
// Bound: the pages' bytes (1.25 d per token and KV head).  At the measured
// copy rate an SM receives one cell (16 tokens of a KV head, 20 d bytes) every
// ~110 cycles at d = 128, so a warp scheduler has ~440 issue slots a cell; a
// warp takes ~310 instructions for one.  In a capture issue is active in 58% of
// the cycles, the ALU pipe in 53%, the tensor pipe in 33%, at 3.6 warps a
// scheduler: what remains beside the bytes is the dependent latency of a warp's
// own chain, with no registers or shared memory for more warps.
// Measured, 32/8 heads, 16 sequences of 16-32K tokens: d = 128, bf16 102 us, 5.25
// TB/s (80% of the copy rate), fp16 (two parts of p) 143; d = 64 73 (56%: a step
// has half the bytes and 0.7 of the instructions) and 99; d = 256, 16/4 heads, 94
// (87%) and 139.  32 such sequences at d = 128 180 us, 4 x 131072 tokens 123 (212
// and 142 under the power cap).  Short work is latency: 1 x 4096 tokens 11.3 us, 61 sequences of up to
// 1500 tokens at d = 256 23 us in bf16, 26 in fp16.
//
// Split.  All steps (pairs of cells) of the batch, in the order (sequence, KV
// head, position), are cut into equal contiguous ranges, one per block (two
// blocks an SM, one at d = 256), and a range into equal parts for its warps,
// so ragged lengths leave no tail.  A warp works through its part alone: units
// (sequence, KV head) that lie inside it go straight to the output; of the
// others it leaves at most two (its first and its last) in shared memory,
// which the block joins once at its end.  A unit that spans blocks goes to the
// workspace in at most two records a block, which paged_combine_kernel joins
// in order.  (Joined by the last block to write one, with a counter a unit, it
// spilled and took 112 us for the 102, 14.2 for the 11.6, and the workspace
// had to start as zeros.)
//
// A warp is its own pipeline: one lane keeps the next step's bulk copy in
// flight into the warp's ring, with the page number loaded one step earlier
// still, so no warp waits for another.
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
//  * values: A = codes of 16 channels x 16 tokens, B = p scale_j of 16 tokens
//    x 8 heads (p's fragment transposed by movmatrix); then, once a step, A =
//    ones in the codes' weights, B = sums of p zero_j over four of the step's
//    tokens, into the same accumulators: what they hold stays of the values' size.  (With sum p zero
//    kept apart, both sums grow with the context and cancel at the end, and the
//    tensor cores' truncating additions show: 1.7e-3 of the output at 131072
//    tokens.)  sum p is one more product (A = ones).  bf16 outputs take p, p
//    scale_j and p zero_j in fp16 (2^-11 each against the output's own 2^-8);
//    fp16 outputs take them in two fp16 parts (22 bits), and the codes moved up
//    to multiples of 2^-18: the tensor cores align a subnormal operand's product
//    as if the operand were 2^-14, so a code at 2^-24 loses ten bits of the 24
//    (2.4e-4 off in an output of 1.0 where values reach 4; at 2^-18 the output's
//    rounding is all that shows; 16 x 32768 tokens at d = 256 88 -> 91 us, d = 128
//    142 -> 143).  bf16 outputs and the scores do not see those bits.
// mma.sync carries them: 18 products of 16 x 8 x 16 and 4 of half the depth a
// cell keep its tensor pipe busy for less than half of the time that the bytes
// take, and the operands come from registers without a trip through tensor memory.  (Queries as A with
// idle rows 8..15 need no transposition, but their zero registers cost 60
// moves a cell.)
//
// Softmax.  Weights are 2^(x - M) with a running reference M per head that
// only has to keep p, p scale_j and p zero_j in fp16's range, and a bound E of
// the scales' and zeros' exponents; both move (and the accumulators with them) when a token
// exceeds them, which one vote a step (two cells) finds out.  One bound serves
// groups within 2^8 of each other.  Where a step shows groups further apart, p
// scale_j of the small ones would fall below fp16's normal range (2048 tokens,
// values of 4000 beside 0.001: 5% rms in bf16 outputs, 6% in fp16, where it is 0.3
// and 0.04 now, the outputs' own rounding); from there on every
// group has its own bound E_j, its scales and zeros are brought to 2^6 in
// shared memory before they are used, each step anew, and its accumulators
// hold units of 2^(E_j - 6).  An output is then off, beside its roundings, by
// some 2^-22 of the largest value of its own group.  (2^-E_j on p for each group
// and cell instead, always or in a second copy of the products, took 4% more time
// of every call.)
#include "paged.cuh"
#include "sm100.cuh"
#include "tq_common.cuh"
#include "tq_kernels.h"

namespace tq {
namespace {

using namespace sm100;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStep = 2;    // cells of a step
constexpr int kStages = 2;  // steps in a warp's ring
constexpr float kTop = 9.f, kSlack = 4.f;  // p 2^E <= 2^9 when M moves, < 2^13 always (four p zero_j stay below 2^16)
// The least bound E (p stays in fp16's range); groups whose bounds lie further than kSpan apart are brought to
// 2^kCommon each, and the lanes' E holds E_j - kApart (below every e, so that each step finds its way there).
constexpr int kLeast = -2, kSpan = 8, kCommon = 6, kApart = 1000;

__host__ __device__ constexpr int blocks_per_sm(int d) { return d == 256 ? 1 : 2; }

// What a warp leaves of a unit: its place, and which of the unit's ends it has.
struct Record {
  int b, h;
  int ends;   // 1: the unit's first step, 2: its last
  int place;  // -1: none; else the first step, counted from the block's range
};

template <int D>
struct Smem {
  static constexpr int kStage = kStep * Cell<D>::kBytes;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kBars = kRing;                            // [kWarps][kStages] u64
  static constexpr int kScan = kBars + kWarps * kStages * 8;     // 16 long long
  static constexpr int kInfo = kScan + 128;                      // [kWarps][2] Record
  // The last records' M and l lie beside the first ones' where the join reads
  // them faster (61 sequences at d = 256 22.3 us for 22.8), and behind their
  // sums at d = 128, where the room would cost an SM its second block (8 query
  // heads a KV head: 132 us for 104).
  static constexpr bool kApart = D != 128;
  static constexpr int kState = kInfo + kWarps * 2 * 16;                  // [kWarps][1 or 2][8][2] floats: M, l
  static constexpr int kMerge = kState + kWarps * (kApart ? 2 : 1) * 64;  // [kWarps][G][D] floats: first records' sums
  static constexpr size_t bytes(int G) { return kMerge + (size_t)kWarps * G * D * 4; }
  // (a kilobyte a block is the system's)
  static_assert(blocks_per_sm(D) * (kMerge + kWarps * TQ_PAGED_MAX_GQA * D * 4 + 1024) <= 228 * 1024, "blocks an SM");
};

// c += a b, and d = a b, for m16n8k16 fp16 operands.
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// c += a b for m16n8k8.
__device__ __forceinline__ void mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) { return pack2<__half>(a, b); }
__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b), *reinterpret_cast<__half2 *>(&c));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// The P words of a lane.
template <int P>
__device__ __forceinline__ void load_words(uint32_t (&w)[P], const uint8_t *p) {
  if constexpr (P == 4) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    w[0] = u.x; w[1] = u.y;
  }
}

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

// Steps of a sequence: two cells each, the last one perhaps one.
__device__ __forceinline__ int steps_of(const PagedView &c, int b) { return (cells_of(c, b) + kStep - 1) / kStep; }

// Steps before sequence `upto` and of the whole batch, times h_kv.  All
// threads of the block (at most 256) call; scratch: 16 long long.
__device__ __forceinline__ void sum_steps(const PagedView &c, int upto, long long *scratch, long long *before,
                                          long long *total) {
  long long s = 0, t = 0;
  for (int b = threadIdx.x; b < c.batch; b += blockDim.x) {
    const int n = steps_of(c, b);
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

// Steps of a block's range: an equal share, at least one per warp.
__host__ __device__ __forceinline__ long long range_steps(long long total, int blocks) {
  const long long per = (total + blocks - 1) / blocks;
  return per < kWarps ? kWarps : per;
}

// A place in the order (sequence, KV head, step).
struct Cursor {
  int b, h, step, steps;
  __device__ __forceinline__ void settle(const PagedView &c) {
    while (step >= steps) {
      step -= steps;
      if (++h == c.h_kv) {
        h = 0;
        do {
          if (++b >= c.batch) {  // past the end: never used
            steps = 0x7fffffff;
            return;
          }
          steps = steps_of(c, b);
        } while (steps == 0);
      }
    }
  }
};

// A warp that gives up still waits for its own copies: records will take their place.
__device__ __noinline__ void give_up(uint64_t *bars, int used, int asked, unsigned int *errors) {
  if ((threadIdx.x & 31) == 0) atomicOr(errors, TQ_ERRF_DECODE_WAIT);
  for (int i = used; i < asked; ++i) mbar_wait(&bars[i % kStages], (i / kStages) & 1);
}

template <int D, class T>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D)) paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a) {
  using C = Cell<D>;
  using S = Smem<D>;
  constexpr int NG = C::kGroups, P = C::kP;
  constexpr bool kTwoParts = __is_same(T, __half);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = lane >> 2, t = lane & 3;
  const int G = a.h_q / a.c.h_kv;
  uint8_t *const ring = smem + warp * kStages * S::kStage;
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
  long long total, c0, per;
  {
    // inclusive sum over the block's threads: sequences base + tid
    auto prefix = [&](int base, long long n, long long *all) {
      long long inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      long long sum = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) inc += scan[w];
        sum += scan[w];
      }
      *all = sum;
      return inc;
    };
    long long n = tid < a.c.batch ? (long long)steps_of(a.c, tid) * a.c.h_kv : 0, all;
    long long inc = prefix(0, n, &all);
    total = all;
    if (a.c.batch > kThreads) {
      long long unused;
      __syncthreads();
      sum_steps(a.c, 0, scan, &unused, &total);
    }
    pdl_trigger();
    per = range_steps(total, gridDim.x);
    c0 = per * blockIdx.x;
    if (c0 >= total) return;
    long long before = 0;
    for (int b0 = 0;;) {
      if (before + inc > c0 && before + inc - n <= c0) {
        scan[8] = b0 + tid;
        scan[9] = before + inc - n;
      }
      before += all;
      b0 += kThreads;
      if (before > c0 || b0 >= a.c.batch) break;
      __syncthreads();
      n = b0 + tid < a.c.batch ? (long long)steps_of(a.c, b0 + tid) * a.c.h_kv : 0;
      inc = prefix(b0, n, &all);
    }
    __syncthreads();
  }
  const int count = (int)(min(c0 + per, total) - c0);
  // the warp's part: steps [at, stop) of the range
  int at = (int)((long long)count * warp / kWarps);
  const int stop = (int)((long long)count * (warp + 1) / kWarps), mine = stop - at;
  Cursor here;  // step `at`
  // (broadcast from one lane: what the whole warp shares can stay in uniform registers)
  here.b = __shfl_sync(0xffffffffu, (int)scan[8], 0);
  here.steps = __shfl_sync(0xffffffffu, steps_of(a.c, here.b), 0);
  const int into = __shfl_sync(0xffffffffu, (int)(c0 - scan[9]), 0);
  here.h = into / here.steps;
  here.step = into % here.steps + at;
  if (mine > 0) here.settle(a.c);

  // ---- the warp's copies.  The page of a step's cells (one page where pages
  // hold two cells or more) is looked up a step before their copy.
  Cursor next = here;
  const int per_page = a.c.page_shift - 4;  // log2 of the cells of a page
  const uint32_t head_bytes = (uint32_t)C::kBytes << per_page;
  const size_t page_bytes = (size_t)head_bytes * a.c.h_kv;
  const bool joined = per_page > 0;
  int cells = 0, page0 = 0, page1 = 0;
  const int32_t *row = a.c.table;
  auto enter = [&] {  // next.b changed
    cells = cells_of(a.c, next.b);
    row = a.c.table + (size_t)next.b * a.c.table_stride;
  };
  auto look = [&] {
    page0 = row[(kStep * next.step) >> per_page];
    if (!joined) page1 = kStep * next.step + 1 < cells ? row[kStep * next.step + 1] : 0;
  };
  int asked = 0;  // steps whose copies were issued
  if (mine > 0) {
    enter();
    look();
  }
  uint32_t bad_stage = 0;  // stages with a cell that has no page
  auto issue = [&] {       // copies of step `asked`; then look the next one up
    if (asked >= mine) return;
    const int s = asked % kStages, first = kStep * next.step, have = min(cells - first, kStep);
    const bool bad = (uint32_t)page0 >= (uint32_t)a.c.num_pages || (!joined && (uint32_t)page1 >= (uint32_t)a.c.num_pages);
    bad_stage = (bad_stage & ~(1u << s)) | ((uint32_t)bad << s);
    if (lane == 0 && !a.c.withhold) {
      uint8_t *const to = ring + s * S::kStage;
      const uint8_t *const from = a.c.data + (size_t)page0 * page_bytes + (size_t)next.h * head_bytes;
      if (bad) {
        mbar_arrive(&bars[s]);
      } else if (joined) {
        mbar_arrive_expect_tx(&bars[s], have * C::kBytes);
        bulk_g2s(to, from + (first & ((1 << per_page) - 1)) * C::kBytes, have * C::kBytes, &bars[s]);
      } else {
        mbar_arrive_expect_tx(&bars[s], have * C::kBytes);
        bulk_g2s(to, from, C::kBytes, &bars[s]);
        if (have > 1)
          bulk_g2s(to + C::kBytes, a.c.data + (size_t)page1 * page_bytes + (size_t)next.h * head_bytes, C::kBytes, &bars[s]);
      }
    }
    if (++asked < mine) {
      if (++next.step >= next.steps) {
        const int was = next.b;
        next.settle(a.c);
        if (next.b != was) enter();
      }
      look();
    }
  };
  __syncwarp();
  issue();

  int used = 0;       // steps taken
  Record *const info = reinterpret_cast<Record *>(smem + S::kInfo);
  if (lane < 2) info[2 * warp + lane].place = -1;
  const int begin = at;
  bool dead = false;  // a wait ran out
  const float kInf = INFINITY;

  while (at < stop) {
    // ---- steps [at, end) of the range, all of unit (here.b, here.h)
    const int end = min(stop, at + here.steps - here.step);
    const int len = a.c.len[here.b];
    bool bad = len > (a.c.max_pages << a.c.page_shift);

    // queries: head g of the unit, lane t's channels 32 j + 8 t .. + 7
    uint32_t qb[NG][4];  // (0, 4), (2, 6) at weight 1; (1, 5), (3, 7) at 1/16
    uint32_t qz[2];      // group sums of q, two fp16 parts, 2^-6
    float c1[2];         // heads 2 t, 2 t + 1: from the products' scale to base-2 logits
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
      c1[0] = ldexpf(a.scale_log2, 24 - __shfl_sync(0xffffffffu, eq, 8 * t));
      c1[1] = ldexpf(a.scale_log2, 24 - __shfl_sync(0xffffffffu, eq, 8 * t + 4));
    }

    // acc[2 j + i]: channels 32 j + 4 g + 2 i (rows g) and + 1 (rows g + 8), heads 2 t and 2 t + 1;
    // ps: sum p of heads 2 t and 2 t + 1 (every row the same); M: heads 2 t and 2 t + 1
    float acc[2 * NG][4], ps[4] = {0.f, 0.f, 0.f, 0.f}, M[2] = {-kInf, -kInf};
    int E = kLeast;  // of all groups; groups apart: E_j - kApart of group g % NG
    auto unit_of = [](int e) { return e < kLeast ? e + kApart - kCommon : 0; };  // exponent of the unit of acc[2 j], acc[2 j + 1]
    constexpr uint32_t kOnes = 0x3c003c00u, kOnesEven = 0x00010001u, kOnesOdd = 0x00100010u, kOnesTwo = 0x04000400u;
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;

    for (int idx = at; idx < end && !dead; ++idx, ++used) {
      __syncwarp();
      issue();
      const int s = used % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars[s], (used / kStages) & 1, a.c.wait_ns))) {
        dead = true;
        give_up(bars, a.c.withhold ? asked : used, asked, a.c.errors);
        break;
      }
      if (bad_stage >> s & 1u) {
        bad = true;
        continue;
      }
      uint8_t *const stage = ring + s * S::kStage;
      const int valid = len - (here.step + idx - at) * (kStep * kCell);
      if (valid < kStep * kCell) {
        // slots behind the sequence may hold anything: give them scale and zero 0
        for (int i = lane; i < kStep * kCell * NG; i += 32) {
          const int n = i / NG, j = i % NG;
          if (n >= valid) {
            uint8_t *const cell = stage + (n / kCell) * C::kBytes;
            *reinterpret_cast<uint16_t *>(cell + C::kKeyScale + C::scale_at(n % kCell, j)) = 0;
            *reinterpret_cast<uint16_t *>(cell + C::kKeyZero + C::key_zero_at(n % kCell, j)) = 0;
            *reinterpret_cast<uint16_t *>(cell + C::kValScale + C::scale_at(n % kCell, j)) = 0;
            *reinterpret_cast<uint16_t *>(cell + C::kValZero + C::scale_at(n % kCell, j)) = 0;
          }
        }
        fence_proxy_async_smem();  // before a later copy into this stage
        __syncwarp();
      }

      // ---- scores (to be scaled by c1): x[.][0, 1] token g of a cell, heads 2 t and 2 t + 1; x[.][2, 3] token g + 8
      float x[kStep][4];
      const uint32_t pick = (g & 1) ? 0x7632 : 0x5410;  // halves e = g & 1 of two words
#pragma unroll
      for (int ce = 0; ce < kStep; ++ce) {
        const uint8_t *const cell = stage + ce * C::kBytes;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int jp = 0; jp < NG / P; ++jp) {
          uint32_t w0[P], w1[P];
          load_words(w0, cell + C::key_word(g, jp * P, t));
          load_words(w1, cell + C::key_word(g + 8, jp * P, t));
#pragma unroll
          for (int i = 0; i < P; i += 2) {
            const uint4 sw = *reinterpret_cast<const uint4 *>(cell + C::kKeyScale + C::scale_at(g & 6, jp * P + i));
            const uint32_t pair[2] = {__byte_perm(sw.x, sw.y, pick), __byte_perm(sw.z, sw.w, pick)};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int j = jp * P + i + k;
              const uint32_t u = w0[i + k], v = w1[i + k], us = u >> 8, vs = v >> 8;
              float d[4];
              mma16_zero(d, u & 0x000f000fu, v & 0x000f000fu, us & 0x000f000fu, vs & 0x000f000fu, qb[j][0], qb[j][1]);
              mma16(d, u & 0x00f000f0u, v & 0x00f000f0u, us & 0x00f000f0u, vs & 0x00f000f0u, qb[j][2], qb[j][3]);
              const float2 sc = unpack_half2(pair[k]);
              y[0] = fmaf(sc.x, d[0], y[0]);
              y[1] = fmaf(sc.x, d[1], y[1]);
              y[2] = fmaf(sc.y, d[2], y[2]);
              y[3] = fmaf(sc.y, d[3], y[3]);
            }
          }
        }
        const uint32_t z0 = *reinterpret_cast<const uint32_t *>(cell + C::kKeyZero + C::key_zero_at(g, (2 * t) % NG));
        const uint32_t z1 = *reinterpret_cast<const uint32_t *>(cell + C::kKeyZero + C::key_zero_at(g + 8, (2 * t) % NG));
        float d[4];
        mma16_zero(d, z0, z1, z0, z1, qz[0], qz[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[ce][i] = fmaf(0x1p-18f, d[i], y[i]);
      }
      // masked slots
      bool none[kStep][2];
#pragma unroll
      for (int ce = 0; ce < kStep; ++ce) {
        none[ce][0] = ce * kCell + g >= valid;
        none[ce][1] = ce * kCell + g + 8 >= valid;
      }

      // ---- the reference: every scale and zero below 2^E, every x at most M + kTop + kSlack - E
      uint32_t top = 0;  // (a lane looks at one group of its tokens, the lanes of a t at all of them)
#pragma unroll
      for (int ce = 0; ce < kStep; ++ce) {
        const uint8_t *const at = stage + ce * C::kBytes + C::scale_at(2 * t, g % NG);
        const uint2 sw = *reinterpret_cast<const uint2 *>(at + C::kValScale), zw = *reinterpret_cast<const uint2 *>(at + C::kValZero);
        top = __vmaxu2(__vmaxu2(__vmaxu2(sw.x, sw.y), __vmaxu2(zw.x & 0x7fff7fffu, zw.y & 0x7fff7fffu)), top);
      }
      top = max(top & 0xffffu, top >> 16);
      int e = (int)(top >> 10) - 14;
      float p[kStep][4], far = -kInf;  // x - M
#pragma unroll
      for (int ce = 0; ce < kStep; ++ce)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          p[ce][i] = fmaf(c1[0], x[ce][i], -M[0]);
          p[ce][i + 1] = fmaf(c1[1], x[ce][i + 1], -M[1]);
          if (none[ce][i / 2]) p[ce][i] = p[ce][i + 1] = -kInf;
          far = max3f(far, p[ce][i], p[ce][i + 1]);
        }
      if (__any_sync(0xffffffffu, far > kTop + kSlack - (float)E || e > E)) {
        const bool were_apart = E < kLeast;
        e = max(max(e, __shfl_xor_sync(0xffffffffu, e, 1)), kLeast);
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
        const int all = max(__reduce_max_sync(0xffffffffu, e), E);
        const bool apart = __any_sync(0xffffffffu, were_apart || all - e > kSpan);
        const int to_e = apart ? max(e - kApart, E < kLeast ? E : -kApart + kLeast) : all;
        const float shift = (float)(apart ? kCommon : all), up = shift - (float)(were_apart ? kCommon : E);
        if (apart) {
          const int unit = unit_of(to_e);
          const float ratio = __int_as_float((127 + unit_of(E) - unit) << 23);
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            const float f = __shfl_sync(0xffffffffu, ratio, 4 * j);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[2 * j + k / 4][k % 4] *= f;
          }
          // the step's value scales and zeros, each lane those of a group
          const int j = lane % NG;
          const __half f = __float2half_rn(__int_as_float((127 - __shfl_sync(0xffffffffu, unit, 4 * j)) << 23));
          for (int n = lane / NG; n < kStep * kCell; n += 32 / NG) {
            uint8_t *const at = stage + (n / kCell) * C::kBytes + C::scale_at(n % kCell, j);
            __half *const s = reinterpret_cast<__half *>(at + C::kValScale), *const z = reinterpret_cast<__half *>(at + C::kValZero);
            *s = __hmul(*s, f);
            *z = __hmul(*z, f);
          }
          fence_proxy_async_smem();  // before a later copy into this stage
          __syncwarp();
        }
        E = to_e;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float big = -kInf;
#pragma unroll
          for (int ce = 0; ce < kStep; ++ce)
#pragma unroll
            for (int o = 0; o < 2; ++o) big = none[ce][o] ? big : fmaxf(big, c1[i] * x[ce][2 * o + i]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
          const float to = fmaxf(big - kTop + shift, M[i] + up);
          const float f = M[i] == -kInf ? 0.f : exp2f(M[i] - to);
          M[i] = to;
          ps[i] *= f;
          ps[i + 2] *= f;
#pragma unroll
          for (int k = 0; k < 2 * NG; ++k) {
            acc[k][i] *= f;
            acc[k][i + 2] *= f;
          }
#pragma unroll
          for (int ce = 0; ce < kStep; ++ce)
#pragma unroll
            for (int o = 0; o < 2; ++o) p[ce][2 * o + i] = none[ce][o] ? -kInf : fmaf(c1[i], x[ce][2 * o + i], -to);
        }
      }

      // ---- values; zf: sums of p zero_j over the lane's tokens 2 t and 2 t + 8, and 2 t + 1 and 2 t + 9, of both cells
      float2 zf[kTwoParts ? NG : 1];
      uint32_t zh[kTwoParts ? 1 : NG];
#pragma unroll
      for (int ce = 0; ce < kStep; ++ce) {
        const uint8_t *const cell = stage + ce * C::kBytes;
        // tokens 2 t, 2 t + 1 (and + 8) of head g
        uint32_t ph[2], pl[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const float p0 = ex2_approx(p[ce][2 * o]), p1 = ex2_approx(p[ce][2 * o + 1]);
          const uint32_t w = pack_half2(p0, p1);
          ph[o] = transpose8(w);
          if constexpr (kTwoParts) {
            const float2 r = unpack_half2(w);
            pl[o] = transpose8(pack_half2(p0 - r.x, p1 - r.y));
          }
        }
        mma16(ps, kOnes, kOnes, kOnes, kOnes, ph[0], ph[1]);
        if constexpr (kTwoParts) mma16(ps, kOnes, kOnes, kOnes, kOnes, pl[0], pl[1]);
#pragma unroll
        for (int jp = 0; jp < NG / P; ++jp) {
          uint32_t w0[P], w1[P];
          load_words(w0, cell + C::val_half(2 * t, jp * P, g));
          load_words(w1, cell + C::val_half(2 * t + 8, jp * P, g));
#pragma unroll
          for (int i = 0; i < P; i += 2) {
            const uint4 sw = *reinterpret_cast<const uint4 *>(cell + C::kValScale + C::scale_at(2 * t, jp * P + i));
            const uint4 zw = *reinterpret_cast<const uint4 *>(cell + C::kValZero + C::scale_at(2 * t, jp * P + i));
            const uint32_t sc[2][2] = {{sw.x, sw.y}, {sw.z, sw.w}}, ze[2][2] = {{zw.x, zw.y}, {zw.z, zw.w}};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int j = jp * P + i + k;
              const uint32_t u = w0[i + k], v = w1[i + k];
              uint32_t b0, b1;
              if constexpr (kTwoParts) {
                const float2 s0 = unpack_half2(sc[k][0]), s1 = unpack_half2(sc[k][1]);
                const float2 h0 = unpack_half2(ph[0]), h1 = unpack_half2(ph[1]), l0 = unpack_half2(pl[0]), l1 = unpack_half2(pl[1]);
                // the codes as multiples of 2^-18
                const uint32_t e0 = u << 6 & 0x03c003c0u, o0 = u << 2 & 0x03c003c0u, e2 = u >> 2 & 0x03c003c0u, o2 = u >> 6 & 0x03c003c0u;
                const uint32_t e1 = v << 6 & 0x03c003c0u, o1 = v << 2 & 0x03c003c0u, e3 = v >> 2 & 0x03c003c0u, o3 = v >> 6 & 0x03c003c0u;
                const float pt[4] = {h0.x + l0.x, h0.y + l0.y, h1.x + l1.x, h1.y + l1.y};
                const float y[4] = {pt[0] * s0.x, pt[1] * s0.y, pt[2] * s1.x, pt[3] * s1.y};
                const float2 z0 = unpack_half2(ze[k][0]), z1 = unpack_half2(ze[k][1]);
                zf[j].x = fmaf(pt[0], z0.x, fmaf(pt[2], z1.x, ce ? zf[j].x : 0.f));
                zf[j].y = fmaf(pt[1], z0.y, fmaf(pt[3], z1.y, ce ? zf[j].y : 0.f));
                b0 = pack_half2(y[0], y[1]);
                b1 = pack_half2(y[2], y[3]);
                const float2 r0 = unpack_half2(b0), r1 = unpack_half2(b1);
                const uint32_t q0 = pack_half2(y[0] - r0.x, y[1] - r0.y), q1 = pack_half2(y[2] - r1.x, y[3] - r1.y);
                mma16(acc[2 * j], e0, o0, e1, o1, q0, q1);
                mma16(acc[2 * j + 1], e2, o2, e3, o3, q0, q1);
                mma16(acc[2 * j], e0, o0, e1, o1, b0, b1);
                mma16(acc[2 * j + 1], e2, o2, e3, o3, b0, b1);
              } else {
                b0 = mul_half2(ph[0], sc[k][0]);
                b1 = mul_half2(ph[1], sc[k][1]);
                zh[j] = fma_half2(ph[1], ze[k][1], ce ? fma_half2(ph[0], ze[k][0], zh[j]) : mul_half2(ph[0], ze[k][0]));
                const uint32_t us = u >> 8, vs = v >> 8;
                mma16(acc[2 * j], u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u, b0, b1);
                mma16(acc[2 * j + 1], us & 0x000f000fu, us & 0x00f000f0u, vs & 0x000f000fu, vs & 0x00f000f0u, b0, b1);
              }
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if constexpr (kTwoParts) {
          // high and low part in the two halves of k; 2^-18 = 2^-14 2^-4
          const float zx = zf[j].x * 0.0625f, zy = zf[j].y * 0.0625f;
          const uint32_t h = pack_half2(zx, zy);
          const float2 r = unpack_half2(h);
          const uint32_t lo = pack_half2(zx - r.x, zy - r.y);
          mma16(acc[2 * j], kOnesTwo, kOnesTwo, kOnesTwo, kOnesTwo, h, lo);
          mma16(acc[2 * j + 1], kOnesTwo, kOnesTwo, kOnesTwo, kOnesTwo, h, lo);
        } else {
          mma8(acc[2 * j], kOnesEven, kOnesOdd, zh[j]);
          mma8(acc[2 * j + 1], kOnesEven, kOnesOdd, zh[j]);
        }
      }
    }

    // ---- a unit that is all here goes to the output, the rest to a record
    if (bad && lane == 0) atomicOr(a.c.errors, TQ_ERRF_PAGE);
    if (bad || dead) ps[0] = ps[1] = __int_as_float(0x7fffffff);
    const int ends = (here.step == 0 ? 1 : 0) | (here.step + end - at == here.steps ? 2 : 0);
    const int slot = 2 * warp + (at == begin ? 0 : 1);
    // the last record lies in the warp's own ring, whose copies have all landed and been used
    float *const rec = at == begin ? merge + (size_t)warp * G * D : reinterpret_cast<float *>(ring);
    float *const rec_state = S::kApart ? state + slot * 16 : at == begin ? state + warp * 16 : rec + G * D;
    if (ends != 3) {
      __syncwarp();
      if (g == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (2 * t + i < G) {
            rec_state[2 * (2 * t + i)] = M[i];
            rec_state[2 * (2 * t + i) + 1] = ps[i];
          }
      if (lane == 0) info[slot] = Record{here.b, here.h, ends, at};
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const float w = __int_as_float((127 + (kTwoParts ? 18 : 24) + unit_of(__shfl_sync(0xffffffffu, E, 4 * j))) << 23);
      const float w_odd = kTwoParts ? w : w * 0.0625f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (2 * t + i < G) {
          const float4 o = make_float4(acc[2 * j][i] * w, acc[2 * j][i + 2] * w_odd, acc[2 * j + 1][i] * w,
                                       acc[2 * j + 1][i + 2] * w_odd);
          if (ends != 3) {
            *reinterpret_cast<float4 *>(rec + (2 * t + i) * D + 32 * j + 4 * g) = o;
          } else {
            const float r = 1.f / ps[i];
            T *out = reinterpret_cast<T *>(a.out) + (size_t)here.b * a.out_stride + (size_t)(here.h * G + 2 * t + i) * D;
            *reinterpret_cast<uint2 *>(out + 32 * j + 4 * g) = make_uint2(pack2<T>(o.x * r, o.y * r), pack2<T>(o.z * r, o.w * r));
          }
        }
      }
    }
    here.step += end - at;
    at = end;
    if (at < stop) here.settle(a.c);
  }

  // ---- the block joins its warps' records: runs of one unit, in order
  __syncthreads();
  for (int r = 0; r < 2 * kWarps;) {
    const Record first = info[r];
    if (first.place < 0) {
      ++r;
      continue;
    }
    int last = r, ends = first.ends;
    for (int k = r + 1; k < 2 * kWarps; ++k) {
      const Record next = info[k];
      if (next.place < 0) continue;
      if (next.b != first.b || next.h != first.h) break;
      last = k;
      ends |= next.ends;
    }
    float *const part = a.partials + ((size_t)blockIdx.x * 2 + (first.place == 0 ? 0 : 1)) * G * (D + 4);
    for (int i = tid; i < G * D / 4; i += kThreads) {
      const int h = i / (D / 4), c = 4 * (i % (D / 4));
      float top = -kInf, sum = 0.f;
      auto sums = [&](int k) {
        return k & 1 ? reinterpret_cast<const float *>(smem + (k / 2) * kStages * S::kStage) : merge + (size_t)(k / 2) * G * D;
      };
      auto states = [&](int k) {
        return (S::kApart ? state + k * 16 : k & 1 ? sums(k) + G * D : state + (k / 2) * 16) + 2 * h;
      };
      for (int k = r; k <= last; ++k)
        if (info[k].place >= 0) top = fmaxf(top, states(k)[0]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = r; k <= last; ++k) {
        if (info[k].place < 0) continue;
        const float f = exp2f(states(k)[0] - top);
        const float4 v = *reinterpret_cast<const float4 *>(sums(k) + h * D + c);
        sum = fmaf(f, states(k)[1], sum);
        o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
      }
      if (ends == 3) {
        const float q = 1.f / sum;
        T *out = reinterpret_cast<T *>(a.out) + (size_t)first.b * a.out_stride + (size_t)(first.h * G + h) * D + c;
        *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(o.x * q, o.y * q), pack2<T>(o.z * q, o.w * q));
      } else {
        *reinterpret_cast<float4 *>(part + h * D + c) = o;
        if (c == 0) {
          part[G * D + 2 * h] = top;
          part[G * D + 2 * h + 1] = sum;
        }
      }
    }
    r = last + 1;
  }
}

// Joins the records of each unit that more than one range holds; zeros for
// empty sequences.  Four warps share a query head's records, a lane holds D / 32
// channels.  What a block is to join it finds while the decode kernel still runs.
// kRanges false: a block a unit and query head.  True, for more units than
// ranges, most of which would have nothing to join: a block a range (x), for the
// unit that starts in it and goes on, and query head of the group (y).
template <int D, class T, bool kRanges>
__global__ void __launch_bounds__(128) paged_combine_kernel(const __grid_constant__ PagedDecodeArgs a, int blocks) {
  constexpr int E = D / 32;
  __shared__ long long scan[16];
  __shared__ float parts[4][D];
  const int G = a.h_q / a.c.h_kv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int head, first = 0, n = 0, second = 0;  // of the group; the unit's first range, how many, which record there
  T *out;
  if constexpr (kRanges) {
    head = blockIdx.y;
    long long before = 0, total;
    sum_steps(a.c, 0, scan, &before, &total);
    const long long per = range_steps(total, blocks), start = per * blockIdx.x, end = start + per;
    int b = 0, h = 0;
    if (end < total) {  // the unit of step `end`
      before = 0;
      for (int b0 = 0; before <= end; b0 += 128) {
        const long long mine = b0 + tid < a.c.batch ? (long long)steps_of(a.c, b0 + tid) * a.c.h_kv : 0;
        long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        for (int w = 0; w < warp; ++w) inc += scan[w];
        inc += before;
        if (inc > end && inc - mine <= end) {
          scan[8] = b0 + tid;
          scan[9] = inc - mine;
        }
        before += scan[0] + scan[1] + scan[2] + scan[3];
        __syncthreads();
      }
      b = (int)scan[8];
      const int steps = steps_of(a.c, b);
      h = (int)((end - scan[9]) / steps);
      const long long u0 = scan[9] + (long long)h * steps;
      if (u0 >= start && u0 < end) {
        first = blockIdx.x;
        n = (int)((u0 + steps - 1) / per) - first + 1;
        second = u0 != start;
      }
    }
    pdl_wait();
    auto row_of = [&](int b, int h) { return reinterpret_cast<T *>(a.out) + (size_t)b * a.out_stride + (size_t)(h * G + head) * D; };
    for (int i = blockIdx.x; i < a.c.batch; i += blocks)
      if (cells_of(a.c, i) == 0)
        for (int k = tid; k < a.c.h_kv * (D / 8); k += 128)
          reinterpret_cast<uint4 *>(row_of(i, k / (D / 8)))[k % (D / 8)] = make_uint4(0, 0, 0, 0);
    out = row_of(b, h);
  } else {
    const int hq = blockIdx.x % a.h_q, b = blockIdx.x / a.h_q;
    long long before, total;
    sum_steps(a.c, b, scan, &before, &total);
    const int steps = steps_of(a.c, b);
    head = hq % G;
    out = reinterpret_cast<T *>(a.out) + (size_t)b * a.out_stride + (size_t)hq * D;
    if (steps == 0) {
      pdl_wait();
      for (int i = tid; i < D / 8; i += 128) reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
      return;
    }
    const long long per = range_steps(total, blocks), u0 = before + (long long)(hq / G) * steps, u1 = u0 + steps;
    first = (int)(u0 / per);
    n = (int)((u1 - 1) / per) - first + 1;
    second = u0 % per != 0;  // the second record of its first range unless that range starts with it
    pdl_wait();
  }
  if (n <= 1) return;
  const size_t size = (size_t)G * (D + 4);
  const float *const base = a.partials + (size_t)first * 2 * size;
  auto record = [&](int i) { return base + (size_t)(2 * i + (i == 0 ? second : 0)) * size; };
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, record(i)[G * D + 2 * head]);
  top = warp_max(top);
  float o[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  // four records' loads in flight
  for (int i = warp; i < n; i += 16) {
    float2 state[4], v[4][E / 2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float *p = record(min(i + 4 * k, n - 1));
      state[k] = *reinterpret_cast<const float2 *>(p + G * D + 2 * head);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) v[k][e] = *reinterpret_cast<const float2 *>(p + head * D + 64 * e + 2 * lane);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + 4 * k < n) {
        const float f = exp2f(state[k].x - top);
        sum = fmaf(f, state[k].y, sum);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          o[2 * e] = fmaf(f, v[k][e].x, o[2 * e]);
          o[2 * e + 1] = fmaf(f, v[k][e].y, o[2 * e + 1]);
        }
      }
  }
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<float2 *>(&parts[warp][32 * e + 2 * lane]) = make_float2(o[e], o[e + 1]);
  __shared__ float sums[4];
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  const float r = 1.f / (sums[0] + sums[1] + sums[2] + sums[3]);
  for (int c = 2 * tid; c < D; c += 256) {
    float y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) y[i] = (parts[0][c + i] + parts[1][c + i] + parts[2][c + i] + parts[3][c + i]) * r;
    *reinterpret_cast<uint32_t *>(out + c) = pack2<T>(y[0], y[1]);
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
  kernel<<<blocks, kThreads, smem, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // us with a block a range (a unit): 256 sequences of 512 tokens, 8 KV heads, d
  // = 128 46 (56), 40 of up to 3000, d = 64 26.5 (26.9), 16 of 512 13.3 (11.9),
  // 1 of 16384, 2 KV heads, d = 256 16.6 (14.5).
  if ((long long)a.c.batch * a.c.h_kv > blocks)
    return launch_pdl(paged_combine_kernel<D, T, true>, dim3(blocks, G), dim3(128), 0, stream, a, blocks);
  return launch_pdl(paged_combine_kernel<D, T, false>, dim3(a.c.batch * a.h_q), dim3(128), 0, stream, a, blocks);
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
