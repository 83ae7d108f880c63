// tq_prompt_attention: causal attention of packed sequences with grouped
// heads on the fifth-generation tensor cores.
//
// Bound: the tensor pipe (4 d flops a visible pair and query head; a 128 x 128
// score tile is 1024 cycles of products at d = 128), beside it the SM's 16
// exponentials a cycle (1024 cycles a tile) and shared memory's 128 bytes a
// cycle (a product of 128 rows x 128 keys reads its operands in the 64 cycles
// that it takes, one of 64 keys in 48 for 32).  Measured, bf16: d = 128, 32/8
// heads, 8192 tokens 433 us, 1270 TFLOP/s (78% of the rate of one large bf16
// product; 510 us, the same share, under the power cap); d = 256, 16/8 heads,
// where products of 64 keys bind, 467 us, 1177 TFLOP/s; d = 64, 32/8 heads, 327
// us, 840 TFLOP/s.  In captures (d = 128, 256, 64) the tensor pipe is busy 63, 57
// and 39% of the cycles, the exponential unit 56, 25 and 69%, issue 49, 29 and 58%:
// at d = 64 exponentials come first, and waits for tensor memory and hand-offs
// keep their unit from filling.  Short: 512 tokens, 12/2 heads, 9.9 us, most of
// it the launch, the first copies and the end.
//
// Rows.  A tile's 128 rows are (token, query head of the group) pairs of one
// KV head: 128 / G tokens with their G heads, so K and V are read once for
// the group and short prompts fill the tile.  A block walks the keys that its
// one or two tiles see (struct Prompt: three shapes).
//
// Roles.  Warp 0 has the TMA engine copy Q once and the K and V tiles through
// a ring (128-byte swizzle, one box per 64 channels); warp 1 issues the
// products: S = Q K^T into tensor memory, and O += P V with P read from
// tensor memory and V as it lies (MN-major).  Eight softmax warps a tile, two
// threads a row (one per half of the step's keys), read S, keep the running
// maximum and sum in float32, write P over S in the operand type and divide at
// the end.  Scores and weights of (step, tile) in turn go through two or three
// S buffers, so that one tile's softmax runs under the other's products, or one
// step's under the next one's.  Where a tile of 128-key steps has no buffer to
// come ahead in, P is handed over in halves, so that products start under the
// second half's exponentials (at d = 64 a third buffer and whole hand-overs
// take 348 us, halves 355, halves without the third buffer 374).  An eighth of
// the exponentials are polynomials (8192 tokens at d = 64: none 345 us, a
// sixteenth 333, an eighth 327, a quarter 342).
//
// The running maximum only moves when a row's grows by more than 2^8 (P stays
// in range of both types, and the sum in float32), so a row's two threads
// mostly need one barrier with a vote to agree, and O is seldom rescaled; the
// threads do it themselves, between the products that write and read it.
//
// A scale of either sign: a negative one negates Q in the product's
// descriptor.
//
// Masked scores are replaced, not added to, so what K holds there does not
// matter.  0 x NaN is NaN, so V is looked at before it is used wherever a row
// of the block does not see a key of the step (the last steps): warps 2 and 3
// clear the rows that nothing sees (another sequence's, or padding), and
// replace infinities and NaN by 0, noting for each channel the first key that
// had one; at the end the rows that see that key get NaN there.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "paged.cuh"
#include "sm100.cuh"
#include "tq_common.cuh"
#include "tq_kernels.h"

namespace tq {
namespace {

using namespace sm100;

// A block's shape.  NQ = 2, KT = 128: two tiles share the keys, 128 a step, one S
// buffer each (three for both at d = 64), one block an SM.  NQ = 1: one tile, two
// S buffers; KT = 64 keys a step and two blocks an SM (one at d = 256), or KT =
// 128 and one block.
template <int D, int NQ, int KT>
struct Prompt {
  static_assert(D < 256 || (NQ == 1 && KT == 64), "O does not fit beside S");
  static_assert(NQ == 1 || KT == 128, "two tiles take 128 keys");
  static constexpr int kBufs = NQ == 2 && D == 64 ? 3 : 2;  // S buffers
  static constexpr bool kAhead = kBufs > NQ;        // a tile's scores may come before its last weights are used
  static constexpr int kBlocks = KT == 128 || D == 256 ? 1 : 2;  // blocks of an SM
  static constexpr int kKeys = KT;
  static constexpr bool kHalves = kKeys == 128 && !kAhead;  // P is handed over in two halves
  static constexpr int kSlabs = D / 64;             // 64-channel boxes
  static constexpr int kQSlab = 128 * 128, kSlab = kKeys * 128;
  static constexpr int kQTile = kQSlab * kSlabs, kStage = kSlab * kSlabs;
  static constexpr int kStages = D == 64 ? 8 : kBlocks == 2 ? 4 : 5;
  static constexpr int kThreads = 128 + 256 * NQ;
  static constexpr int kExchange = NQ * kQTile + kStages * kStage;  // [NQ][2][128] floats, [NQ][2][4] ints
  static constexpr int kBad = kExchange + NQ * (1024 + 32);  // [D] ints: the first key with a special value
  static constexpr int kBars = kBad + D * 4;
  static constexpr size_t kSmem = kBars + 384;
  // tensor memory columns: S (and P over it) of buffer or tile x, O of tile x
  static constexpr uint32_t kColumns = kBlocks == 2 ? 256 : 512;
  __host__ __device__ static constexpr uint32_t s_col(int x) { return (uint32_t)kKeys * x; }
  __host__ __device__ static constexpr uint32_t o_col(int x) { return (uint32_t)(kBufs * kKeys) + (uint32_t)D * x; }
  // P of keys 16 k .. + 15, from the S buffer's first column: each half over the first half of its own S
  __host__ __device__ static constexpr uint32_t p_col(int k) {
    return k < kKeys / 32 ? 8u * k : (uint32_t)kKeys / 2 + 8u * (k - kKeys / 32);
  }
  // registers of a thread: copies and products, softmax; together at most what
  // the launch has (96, 80 or 168 a thread)
  static constexpr int kFew = 40, kMany = NQ == 2 ? 104 : kBlocks == 1 ? 216 : 96;
};

// 2^y for two y in [-inf, 9] (or NaN) without the exponential unit: y is cut
// into an integer and a rest in [-1/2, 1/2], whose power is the polynomial of
// degree 5 with the least largest relative error there (by Remez' exchange;
// 2^-22 in float32).  Below 2^-127 the result is 0.
__device__ __forceinline__ float2 exp2_poly(float2 y) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(y.x) : "f"(-127.f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(y.y) : "f"(-127.f));
  auto both = [](float v) { return make_float2(v, v); };
  const float2 t = add2(y, both(12582912.f));  // 1.5 2^23: the integer in the low bits
  const float2 n = add2(t, both(-12582912.f));
  const float2 f = fma2(n, both(-1.f), y);
  float2 p = fma2(both(0x1.5c08e4p-10f), f, both(0x1.3d0c52p-7f));
  p = fma2(p, f, both(0x1.c6b6e4p-5f));
  p = fma2(p, f, both(0x1.ebf918p-3f));
  p = fma2(p, f, both(0x1.62e428p-1f));
  p = fma2(p, f, both(0x1.000002p+0f));
  p.x *= __int_as_float((__float_as_int(t.x) << 23) + 0x3f800000);
  p.y *= __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000);
  return p;
}

// Sequence of block u: sequence b owns blocks [cu[b] / tb + b, cu[b + 1] / tb
// + b + 1), at least as many as its rows need (32-way search, warp-wide).
__device__ __forceinline__ int block_sequence(const int32_t *cu, int batch, int rows, int tb, int u) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lane * step;
    const bool below = at < n && clamp_cu(cu, lo + at, rows) / tb + lo + at <= u;
    const int k = max(__popc(__ballot_sync(0xffffffffu, below)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

template <int D, class T, int NQ, int KT>
__global__ void __launch_bounds__(Prompt<D, NQ, KT>::kThreads, Prompt<D, NQ, KT>::kBlocks)
    prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int units) {
  using C = Prompt<D, NQ, KT>;
  constexpr int ST = C::kStages;
  constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
  constexpr int NB = C::kBufs;
  extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzle's atoms)
  uint8_t *const stages = smem + NQ * C::kQTile;
  float *const exchange = reinterpret_cast<float *>(smem + C::kExchange);
  int *const exchange_ok = reinterpret_cast<int *>(exchange + NQ * 256), *const bad = reinterpret_cast<int *>(smem + C::kBad);
  uint64_t *const bars = reinterpret_cast<uint64_t *>(smem + C::kBars);
  // s_full, p_ready and p_half: by S buffer; o_done: by tile
  uint64_t *const q_full = bars, *const kv_full = bars + 1, *const kv_empty = kv_full + ST, *const s_full = kv_empty + ST,
                  *const p_ready = s_full + NB, *const p_half = p_ready + NB, *const o_done = p_half + NB,
                  *const v_here = o_done + 2, *const v_clear = v_here + ST, *const drained = v_clear + ST;
  uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  // the block's first row, its tokens and first head, for the end (out of the registers until then); [3]: V had
  // special values
  volatile int *const place = abort_flag + 1;

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int G = a.h_q / a.h_kv, tpt = 128 / G, tb = tpt * NQ;

  // ---- the block's rows and keys; later blocks of a sequence see more keys
  // and start first
  const int h = blockIdx.x % a.h_kv, u = units - 1 - (int)(blockIdx.x / a.h_kv);
  const int b = block_sequence(a.cu_q, a.batch, a.T_q, tb, u);
  const int q0 = clamp_cu(a.cu_q, b, a.T_q), nq = max(clamp_cu(a.cu_q, b + 1, a.T_q) - q0, 0);
  const int i0 = (u - (q0 / tb + b)) * tb;
  if (i0 < 0 || i0 >= nq) return;
  const int k0 = clamp_cu(a.cu_k, b, a.T_k), nk = max(clamp_cu(a.cu_k, b + 1, a.T_k) - k0, 0);
  const int shift = nk - nq;  // query i sees keys j <= i + shift
  // steps of a tile; keys that the block sees, and its steps (the last tile with rows has most)
  auto keys_of = [&](int x) { return i0 + x * tpt < nq ? max(min(nk, min(nq, i0 + (x + 1) * tpt) + shift), 0) : 0; };
  auto steps_of = [&](int x) { return (keys_of(x) + KT - 1) / KT; };
  const int seen = max(keys_of(0), NQ == 2 ? keys_of(1) : 0), most = (seen + KT - 1) / KT;
  // the first step with a key that some row does not see: V is looked at from there on
  const int looked = max(min(min(nk, i0 + 1 + shift), seen), 0) / KT;

  if (warp == 0 && lane == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&v_here[s], 1);
      mbar_init(&v_clear[s], 2);
    }
    for (int x = 0; x < NB; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_ready[x], 8);
      mbar_init(&p_half[x], 8);
    }
    for (int x = 0; x < NQ; ++x) mbar_init(&o_done[x], 1);
    mbar_init(drained, 1);
    *abort_flag = 0;
    place[0] = q0 + i0;
    place[1] = min(nq - i0, tb);
    place[2] = h * G;
    place[3] = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < D; i += C::kThreads) bad[i] = 0x7fffffff;
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const unsigned int hint = (unsigned int)(a.wait_ns < 1000000ull ? a.wait_ns : 1000000ull);
  bool timed_out = false;
  // for a whole warp: its lanes go on, or give up, together
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, pipe_wait(bar, parity, abort_flag, a.wait_ns, hint, &timed_out));
  };

  // Scores and weights of (step, tile) in turn go through the S buffers: the
  // place of tile x's step j in that order.  (Where the second tile has steps, the first has no more.)
  const int steps0 = steps_of(0), steps1 = NQ == 2 ? steps_of(1) : 0;
  auto turn_of = [&](int x, int j) {
    return NQ == 1 || steps1 == 0 ? j : x == 0 ? 2 * j : j < steps0 ? 2 * j + 1 : steps0 + j;
  };

  // which use of its stage among the steps that are looked at V of step j is: V's place comes round every so many steps
  auto use_of = [&](int j) { return (uint32_t)((j - looked) / (ST % 2 ? ST : ST / 2)) & 1u; };

  if (warp < 4) {
    reg_dealloc<C::kFew>();
    if (warp == 0) {
      // ---- copies
      if (lane == 0 && most > 0) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(NQ * C::kSlabs * tpt * G * 128));
        for (int x = 0; x < NQ; ++x)
          for (int s = 0; s < C::kSlabs; ++s)
            tma_load_4d(smem + x * C::kQTile + s * C::kQSlab, &qmap, 64 * s, 0, h, q0 + i0 + x * tpt, q_full);
        int item = 0;  // K and V tiles in turn
        for (; item < (a.withhold == 1 ? 0 : 2 * most); ++item) {
          const int st = item % ST;
          if (item >= ST && !pipe_wait(&kv_empty[st], (item / ST - 1) & 1, abort_flag, a.wait_ns, hint, &timed_out)) break;
          mbar_arrive_expect_tx(&kv_full[st], C::kStage);
          for (int s = 0; s < C::kSlabs; ++s)
            tma_load_3d(stages + st * C::kStage + s * C::kSlab, item & 1 ? &vmap : &kmap, 64 * s, h, k0 + (item >> 1) * KT,
                        &kv_full[st]);
          if ((item & 1) && item >> 1 >= looked) mbar_arrive(&v_here[st]);
        }
        // shared memory is the block's until its own copies have landed
        mbar_wait(q_full, 0);
        for (int i = max(0, item - ST); i < item; ++i) mbar_wait(&kv_full[i % ST], (i / ST) & 1);
      }
    } else if (warp == 1) {
      // ---- products.  The whole warp runs the loop, so that descriptors stay in
      // uniform registers; one lane issues.
      const uint32_t leader = elect_one();
      const uint32_t is = idesc_16bit(128, KT, kBf16, false, a.negate), io = idesc_16bit(128, D, kBf16, true, false);
      const uint32_t sa = smem_u32(stages);
      const uint64_t qd = smem_desc_sw128(smem_u32(smem), 16, 1024), kd = smem_desc_sw128(sa, 16, 1024),
                     vd = smem_desc_sw128(sa, C::kSlab, 1024);
      // where the next K and V tile lie in the ring: items 0, 2, .. and 1, 3, ..
      struct Place {
        int st;
        uint32_t phase;
        __device__ __forceinline__ void advance() {
          st += 2;
          if (st >= ST) {
            st -= ST;
            phase ^= 1;
          }
        }
      } kp{0, 0}, vp{1, 0};
      auto scores = [&](int x, int buf) {  // S[buf] = Q[x] K^T
        const uint64_t kt = kd + (uint32_t)(kp.st * (C::kStage >> 4));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_f16_ss_if(leader, tmem + C::s_col(buf), qd + (uint32_t)((x * C::kQTile + (k / 4) * C::kQSlab + (k % 4) * 32) >> 4),
                        kt + (uint32_t)(((k / 4) * C::kSlab + (k % 4) * 32) >> 4), is, k > 0);
        mma_commit_if(leader, &s_full[buf]);
      };
      // O[x] += P V over the first 32 keys of each half, over the others, or over all
      auto values = [&](int x, int buf, int j, int which) {
        const uint64_t vt = vd + (uint32_t)(vp.st * (C::kStage >> 4));
#pragma unroll
        for (int k = 0; k < KT / 16; ++k)
          if (which == 2 || (k >> 1 & 1) == which)
            mma_f16_ts_if(leader, tmem + C::o_col(x), tmem + C::s_col(buf) + C::p_col(k), vt + (uint32_t)(k * 128), io,
                          j > 0 || k > 0);
        if (C::kAhead && which != 0) mma_commit_if(leader, &o_done[x]);
      };
      auto release = [&](Place &p) {
        mma_commit_if(leader, &kv_empty[p.st]);
        p.advance();
      };
      auto landed = [&](const Place &p) { return wait(&kv_full[p.st], p.phase); };
      // V of step j is here, and looked at
      auto value_tile = [&](int j) {
        if (!landed(vp)) return false;
        return j < looked || wait(&v_clear[vp.st], use_of(j));
      };
      // the (step, tile) whose scores, and whose products with V, come next
      struct Turn {
        int x, j, buf;
        uint32_t phase;
      } sc{steps0 > 0 ? 0 : NQ - 1, 0, 0, 0}, pv = sc;
      auto starts = [&](const Turn &t) { return t.x == 0 || t.j >= steps0; };      // its step's first tile, last tile
      auto ends = [&](const Turn &t) { return t.x == NQ - 1 || t.j >= steps1; };
      auto advance = [&](Turn &t) {
        if (ends(t)) {
          ++t.j;
          t.x = t.j < steps0 ? 0 : NQ - 1;
        } else {
          t.x = 1;
        }
        if (++t.buf == NB) {
          t.buf = 0;
          t.phase ^= 1;
        }
      };
      // (each K and V tile is asked for just before its first use and given back
      // just after its last, or the copies do not come in time)
      auto next_scores = [&] {
        if (sc.j >= most) return true;
        // Where a tile goes on alone the buffers would let its scores come further ahead.  Not before the tile's
        // products of a step earlier (two, with buffers to come ahead): whoever has these scores knows those done
        // (and can tell the step between by o_done's parity), and may change O.
        constexpr int kBack = C::kAhead ? 2 : 1;
        if (NQ == 2 && (pv.j < sc.j - kBack || (pv.j == sc.j - kBack && pv.x <= sc.x))) return true;
        if (starts(sc) && !landed(kp)) return false;
        tc_fence_after();
        scores(sc.x, sc.buf);
        if (ends(sc)) release(kp);
        advance(sc);
        return true;
      };
      bool ok = most == 0 || wait(q_full, 0);
      for (int i = 0; ok && i < NB; ++i) ok = next_scores();
      while (ok && pv.j < most) {
        if (NQ == 2 && pv.x == 0 && pv.j + 2 < min(steps0, steps1) && sc.x == NB - 2 && sc.j == pv.j + 1) {
          // a whole step in the middle, the same turns without their case distinctions: after the products of a
          // buffer's weights, that buffer's next scores
#pragma unroll
          for (int x = 0; x < NQ; ++x) {
            if (x == 0) ok = value_tile(pv.j);
            if (ok && C::kHalves) {
              ok = wait(&p_half[pv.buf], pv.phase);
              tc_fence_after();
              if (ok) values(x, pv.buf, pv.j, 0);
            }
            ok = ok && wait(&p_ready[pv.buf], pv.phase);
            tc_fence_after();
            if (!ok) break;
            values(x, pv.buf, pv.j, C::kHalves ? 1 : 2);
            if (x == 1) release(vp);
            const int y = NB == 3 ? 1 - x : x;  // the scores' tile
            if (y == 0) ok = landed(kp);
            tc_fence_after();
            if (!ok) break;
            scores(y, pv.buf);
            if (y == 1) release(kp);
            const bool wraps = pv.buf == NB - 1;
            pv.buf = wraps ? 0 : pv.buf + 1;
            pv.phase ^= wraps;
          }
          sc.buf = pv.buf;
          ++pv.j;
          ++sc.j;
          continue;
        }
        if (starts(pv)) ok = value_tile(pv.j);
        if (ok && C::kHalves) {
          ok = wait(&p_half[pv.buf], pv.phase);
          tc_fence_after();
          if (ok) values(pv.x, pv.buf, pv.j, 0);
        }
        ok = ok && wait(&p_ready[pv.buf], pv.phase);
        tc_fence_after();
        if (!ok) break;
        values(pv.x, pv.buf, pv.j, C::kHalves ? 1 : 2);
        if (ends(pv)) release(vp);
        advance(pv);
        ok = next_scores();
      }
      // tensor and shared memory stay until every product has finished
      mma_commit_if(leader, drained);
      __syncwarp();
      mbar_wait(drained, 0);
    } else {
      // ---- the look at V.  (The loader tells of a copy when it issues it: until
      // then the stage's barrier may stand a phase behind, which a parity does
      // not tell from the phase after.)
      constexpr uint32_t field = kBf16 ? 0x7f807f80u : 0x7c007c00u, one = kBf16 ? 0x00800080u : 0x04000400u;
      constexpr int kUnits = C::kStage / 16 / 64, kBatch = 8;  // 16-byte pieces of a lane
      static_assert(kUnits % kBatch == 0, "whole batches");
      for (int j = looked; j < most; ++j) {
        const int st = (2 * j + 1) % ST;
        if (!wait(&v_here[st], use_of(j)) || !wait(&kv_full[st], (2 * j + 1) / ST & 1)) break;
        uint4 *const v = reinterpret_cast<uint4 *>(stages + st * C::kStage);
        const int rows = seen - j * KT, first = (warp - 2) * 32 + lane;  // rows that something sees
        if (rows < KT)
          for (int i = first; i < 64 * kUnits; i += 64)
            if (i / 8 % KT >= rows) v[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int i0 = 0; i0 < kUnits; i0 += kBatch) {
          uint32_t any = 0;
          uint4 u[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) u[k] = v[first + 64 * (i0 + k)];
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            any |= ((u[k].x & field) + one) | ((u[k].y & field) + one) | ((u[k].z & field) + one) | ((u[k].w & field) + one);
          if (any & 0x80008000u) {
#pragma unroll 1
            for (int k = 0; k < kBatch; ++k) {
              const int i = first + 64 * (i0 + k), row = i / 8 % KT, channel = i / (8 * KT) * 64 + (i % 8 ^ (row & 7)) * 8;
              uint16_t *const at = reinterpret_cast<uint16_t *>(v + i);
#pragma unroll 1
              for (int e = 0; e < 8; ++e)
                if ((at[e] & field & 0xffffu) == (field & 0xffffu)) {
                  at[e] = 0;
                  atomicMin(&bad[channel + e], j * KT + row);
                  place[3] = 1;
                }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_clear[st]);
      }
    }
  } else {
    // ---- softmax: tile x, row r, half `part` of the step's keys (and of the output's channels)
    reg_alloc<C::kMany>();
    constexpr int KH = KT / 2, DH = D / 2;
    const int x = (warp - 4) >> 3, quarter = warp & 3, part = ((warp - 4) >> 2) & 1, r = quarter * 32 + lane;
    const int pair_bar = 1 + 4 * x + quarter, mine_at = (2 * x + part) * 128 + r, other_at = (2 * x + (part ^ 1)) * 128 + r;
    const uint32_t lanes = (uint32_t)quarter * 32u << 16;
    // keys that this row sees, and that every row of the tile sees (rows that
    // belong to no token go on as if they did; nothing reads them)
    const int lim = min(nk, i0 + x * tpt + r / G + 1 + shift), easy = min(nk, i0 + x * tpt + 1 + shift), steps = x ? steps1 : steps0;
    const float c = a.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < steps; ++j) {
      const int turn = turn_of(x, j), buf = turn % NB;
      ok = wait(&s_full[buf], turn / NB & 1);
      tc_fence_after();
      const uint32_t st = tmem + C::s_col(buf) + lanes + part * KH;
      const int vis = (j + 1) * KT > easy ? lim - j * KT - part * KH : KH;  // keys of the half that the row sees
      // 32 scores, masked ones -inf.  (The first 32 stay in registers between the
      // maximum and the weights; the others are read twice: tensor memory is
      // nearer than the registers that all of them would take.)
      auto load = [&](int i, uint32_t (&s)[32]) {
        tmem_ld32(st + 32 * i, s);
        tmem_wait_ld();
        if (__any_sync(0xffffffffu, vis < 32 * (i + 1))) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * i + e >= vis) s[e] = 0xff800000u;
        }
      };
      float top = -INFINITY;
      uint32_t s[32];
      if (ok) {
#pragma unroll
        for (int i = KH / 32 - 1; i >= 0; --i) {
          load(i, s);
          float top2 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            top = max3f(top, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
            top2 = max3f(top2, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
          }
          top = fmaxf(top, top2);
        }
      }
      // The maximum moves only where it grew by more than 2^8 (from -inf to
      // anything; not from -inf to -inf).
      if (named_bar_or(pair_bar, 64, (top - m) * c > 8.f || !ok)) {
        exchange[mine_at] = top;
        if (lane == 0) exchange_ok[(2 * x + part) * 4 + quarter] = ok;
        named_bar_sync(pair_bar, 64);
        top = fmaxf(top, exchange[other_at]);
        ok = ok && exchange_ok[(2 * x + (part ^ 1)) * 4 + quarter];
        if (!ok) break;
        const float was = m;
        if ((top - m) * c > 8.f) m = top;
        const float f = was == m ? 1.f : ex2_approx((was - m) * c);  // was = -inf: 0
        l *= f;
        if (j > 0) {
          // O's last product first (or the scores were issued behind it).  Should this run out, the warp leaves O and goes
          // on, so that its partner finds it at the barriers: the abort flag is up, and no row of the block comes from O.
          bool there = true;
          if constexpr (C::kAhead) {
            there = wait(&o_done[x], (j - 1) & 1);
            if (a.withhold == 2 && part) there = wait(&o_done[x], j & 1);  // a test of that: not before P is handed over
            tc_fence_after();
          }
          const uint32_t ot = tmem + C::o_col(x) + lanes + part * DH;
#pragma unroll 1
          for (int i = 0; i < DH && there; i += 32) {
            uint32_t o[32];
            tmem_ld32(ot + i, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(ot + i, o);
          }
        }
      }
      const float mc = m == -INFINITY ? 0.f : m * c;
      const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < KH / 32; ++i) {
        uint32_t p[16];
        if (i > 0) load(i, s);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 y = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, mc2);
          if (e % 8 == 7) {  // an eighth of them: the exponential unit's queue is the shorter for it
            y = exp2_poly(y);
          } else {
            y.x = ex2_approx(y.x);
            y.y = ex2_approx(y.y);
          }
          sum = add2(sum, y);
          p[e] = pack2<T>(y.x, y.y);
        }
        tmem_st16(st + 16 * i, p);
        if (C::kHalves && i == 0) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_half[buf]);
        }
      }
      l += sum.x + sum.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[buf]);
    }
    // ---- the output: the halves' sums, then rows through shared memory (Q's
    // place; no product reads it any more), 16 bytes a lane
    if (ok) {
      named_bar_sync(pair_bar, 64);  // (the last exchange has been read)
      exchange[mine_at] = l;
      named_bar_sync(pair_bar, 64);
      l += exchange[other_at];
      // (not o_done: by now it may stand one or two products behind the last,
      // and a parity cannot tell the last but one from the one after the last)
      // Where a role has given up, products may be missing before it, or O have changed under one.
      if (most > 0) ok = wait(drained, 0) && __all_sync(0xffffffffu, *abort_flag == 0);
    }
    tc_fence_after();
    // a row that sees nothing is zero whatever its product holds
    const bool none = ok && lim <= 0;
    const float w = !ok ? __int_as_float(0x7fffffff) : 1.f / l;
    const bool special = place[3] != 0;
    constexpr int NC = DH / 8;  // 16-byte pieces of a row's half
    uint8_t *const rows = smem + (warp - 4) * 32 * NC * 16;
#pragma unroll
    for (int i = 0; i < DH; i += 32) {
      uint32_t o[32];
      if (steps > 0 && ok) {
        tmem_ld32(tmem + C::o_col(x) + lanes + part * DH + i, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0;
      }
      if (special) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (bad[part * DH + i + e] < lim) o[e] = 0x7fffffffu;
      }
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = none ? 0u : pack2<T>(__uint_as_float(o[e + 2 * k]) * w, __uint_as_float(o[e + 2 * k + 1]) * w);
        const int piece = (i + e) / 8;
        *reinterpret_cast<uint4 *>(rows + (lane * NC + (piece ^ (lane & (NC < 8 ? NC - 1 : 7)))) * 16) =
            make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
    __syncwarp();
    const int group = a.h_q / a.h_kv, rows_of_tile = 128 / group * group, tok = x * (128 / group) + r / group;
    const long long mine = r < rows_of_tile && tok < place[1] ? (long long)(place[0] + tok) * a.out_stride +
                                                                    (long long)(place[2] + r % group) * D + part * DH
                                                              : -1;
#pragma unroll 4
    for (int i = lane; i < 32 * NC; i += 32) {
      const int row = i / NC, piece = i % NC;
      const long long at = __shfl_sync(0xffffffffu, mine, row);
      if (at >= 0)
        *reinterpret_cast<uint4 *>(reinterpret_cast<T *>(a.out) + at + piece * 8) =
            *reinterpret_cast<const uint4 *>(rows + (row * NC + (piece ^ (row & (NC < 8 ? NC - 1 : 7)))) * 16);
    }
  }
  if (timed_out) atomicOr(a.errors, TQ_ERRF_PROMPT_WAIT);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kColumns);
  }
}

// The driver's tensor-map encoder, looked up once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// [tokens][heads][D] rows as (channel, head of a group, group, token) with
// boxes of 64 channels x per heads x 1 group x `box` tokens; rank 3 (no
// groups) where per is 0.
template <int D, class T>
bool encode(CUtensorMap *map, const void *p, long long stride, int heads, int per, int tokens, int box) {
  const auto type = __is_same(T, __nv_bfloat16) ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const cuuint64_t row = (cuuint64_t)stride * 2;
  auto *enc = encoder();
  if (!enc) return false;
  if (per) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)per, (cuuint64_t)(heads / per), (cuuint64_t)tokens};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)per * D * 2, row};
    const cuuint32_t b[4] = {64, (cuuint32_t)per, 1, (cuuint32_t)box};
    return enc(map, type, 4, const_cast<void *>(p), dims, strides, b, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, row};
  const cuuint32_t b[3] = {64, 1, (cuuint32_t)box};
  return enc(map, type, 3, const_cast<void *>(p), dims, strides, b, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, class T, int NQ, int KT>
cudaError_t launch(const PromptArgs &a, cudaStream_t stream) {
  using C = Prompt<D, NQ, KT>;
  const int G = a.h_q / a.h_kv, tpt = 128 / G;
  const long long units = a.T_q / (tpt * NQ) + (long long)a.batch;
  if (units * a.h_kv > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  CUtensorMap q, k, v;
  // with no keys at all the K and V maps are never read: any rows will do
  const bool none = a.T_k == 0;
  if (!encode<D, T>(&q, a.q, a.q_stride, a.h_q, G, a.T_q, tpt) ||
      !encode<D, T>(&k, none ? a.q : a.k, none ? a.q_stride : a.k_stride, none ? a.h_q : a.h_kv, 0, none ? a.T_q : a.T_k, C::kKeys) ||
      !encode<D, T>(&v, none ? a.q : a.v, none ? a.q_stride : a.v_stride, none ? a.h_q : a.h_kv, 0, none ? a.T_q : a.T_k, C::kKeys))
    return cudaErrorInvalidValue;
  auto *kernel = prompt_kernel<D, T, NQ, KT>;
  static std::atomic<int> allowed[kAttributeDevices];
  const cudaError_t e = allow_smem(kernel, C::kSmem, allowed);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)(units * a.h_kv), C::kThreads, C::kSmem, stream>>>(a, q, k, v, (int)units);
  return cudaGetLastError();
}

template <int D, class T>
cudaError_t launch_d(const PromptArgs &a, cudaStream_t stream) {
  // Long sequences: two tiles share the keys' copies and operand reads, and
  // products of 128 keys read shared memory at the rate the tensor pipe takes.
  // Short ones: two blocks an SM hide each other's start and end.  32/8 heads,
  // us with two tiles a block (one tile): d = 128, bf16: 2 x 4096 tokens 246
  // (262), 1 x 2048 41 (43), 4 x 2048 154 (153), 8 x 1536 196 (187), 32 x 512
  // 167 (145); d = 64, fp16, where two tiles have a third score buffer: 2 x
  // 4096 194 (222), 8 x 1536 159 (164), 16 x 1024 172 (169), 32 x 512 139 (124).
  // The host knows the sums and not the lengths, so one long prompt among short
  // ones gets the shape of the average (8192 tokens and fifteen of 16, d = 128: 490
  // us, the 8192 alone, with two tiles a block, 451).
  // Few tiles: one tile a block and 128 keys a step, half as many steps one after
  // the other.  Up to a tile an SM from 384 keys on (12/2 heads, bf16: 512 tokens
  // 10.4 us for 11.4 with 64 keys a step, 300 tokens 9.4 both ways; 32/8 heads,
  // 700 tokens, 184 tiles: 15.2 for 14.0), up to two from 1280 on (12/2 heads,
  // 2400 tokens 27 for 39 with two tiles a block, 8/8 heads, 5000 tokens, 312
  // tiles: 61 for 73; 7000 tokens, 440 tiles: 105 for 97; 32/8 heads, 1500
  // tokens, 376 tiles: 35 for 27).
  if constexpr (D < 256) {
    int sms;
    const cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const long long tiles = (a.T_q / (128 / (a.h_q / a.h_kv)) + (long long)a.batch) * a.h_kv;
    const long long few = a.T_k >= 1280ll * a.batch ? 2ll * sms : sms;
    if (tiles <= few && a.T_k >= 384ll * a.batch) return launch<D, T, 1, 128>(a, stream);
    if (a.T_k >= (D == 64 ? 1280ll : 2048ll) * a.batch) return launch<D, T, 2, 128>(a, stream);
  }
  return launch<D, T, 1, 64>(a, stream);
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, int d, tq_dtype dt, cudaStream_t stream) {
  const bool bf = dt == TQ_BF16;
  if (d == 64) return bf ? launch_d<64, __nv_bfloat16>(a, stream) : launch_d<64, __half>(a, stream);
  if (d == 128) return bf ? launch_d<128, __nv_bfloat16>(a, stream) : launch_d<128, __half>(a, stream);
  return bf ? launch_d<256, __nv_bfloat16>(a, stream) : launch_d<256, __half>(a, stream);
}

}  // namespace tq
