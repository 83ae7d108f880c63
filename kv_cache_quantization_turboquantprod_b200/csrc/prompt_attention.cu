// tq_prompt_attention: causal attention of packed sequences with grouped
// heads on the fifth-generation tensor cores.
//
// Bound: the tensor pipe (4 d flops a visible pair and query head) and, next
// to it, the exponentials: a 128 x 128 score tile is 1024 cycles of products
// at d = 128 and 1024 cycles of the SM's 16 exponentials a cycle.
//
// Rows.  A tile's 128 rows are (token, query head of the group) pairs of one
// KV head: 128 / G tokens with their G heads, so K and V are read once for
// the group and short prompts fill the tile.  A block takes two such tiles
// (one at d = 256) of one sequence and KV head and walks the keys that they
// see, 128 at a time (64 at d = 256).
//
// Roles.  Warp 0 has the TMA engine copy Q once and the K and V tiles through
// a ring (128-byte swizzle, one box per 64 channels); warp 1 issues the
// products: S = Q K^T into tensor memory, and O += P V with P read from
// tensor memory and V as it lies (MN-major).  Each tile's four softmax warps,
// a thread a row, read S, keep the running maximum and sum in float32, write
// P over S in the operand type and divide at the end.  The two tiles alternate:
// one's softmax runs under the other's products.  At d = 256 one tile
// alternates between two S buffers instead (two tiles' O do not fit).
//
// The running maximum only moves when a row's grows by more than 2^8 (P stays
// in range of both types, and the sum in float32), so O is seldom rescaled;
// the row's own thread does it, between the products that write and read it.
// A scale of either sign: a negative one negates Q in the product's
// descriptor.
//
// Masked scores are replaced, not added to, so what K holds there does not
// matter; V rows that no row of the block sees (another sequence's, or
// padding) are cleared in shared memory by warp 2 before they are used, since
// 0 x NaN is NaN.
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

template <int D>
struct Prompt {
  static constexpr int kTiles = D == 256 ? 1 : 2;   // query tiles of a block
  static constexpr int kKeys = D == 256 ? 64 : 128; // keys of a step
  static constexpr int kSlabs = D / 64;             // 64-channel boxes
  static constexpr int kQSlab = 128 * 128, kSlab = kKeys * 128;
  static constexpr int kQTile = kQSlab * kSlabs, kStage = kSlab * kSlabs;
  static constexpr int kStages = D == 64 ? 8 : 5;
  static constexpr int kThreads = 128 + 128 * kTiles;
  static constexpr int kBars = kTiles * kQTile + kStages * kStage;
  static constexpr size_t kSmem = kBars + 512 + 1024;  // 1024: alignment of the base
  // tensor memory columns: S (and P over it) of buffer x, O of tile x
  __host__ __device__ static constexpr uint32_t s_col(int x) { return 128u * x; }
  __host__ __device__ static constexpr uint32_t o_col(int x) { return 256u + (uint32_t)D * x; }
};

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

template <int D, class T>
__global__ void __launch_bounds__(Prompt<D>::kThreads, 1)
    prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int units) {
  using C = Prompt<D>;
  constexpr int KT = C::kKeys, NQ = C::kTiles, ST = C::kStages;
  constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *const stages = smem + NQ * C::kQTile;
  uint64_t *const bars = reinterpret_cast<uint64_t *>(smem + C::kBars);
  uint64_t *const q_full = bars, *const kv_full = bars + 1, *const kv_empty = kv_full + ST, *const s_full = kv_empty + ST,
                  *const p_ready = s_full + 2, *const o_done = p_ready + 2, *const v_last = o_done + 2,
                  *const v_clear = v_last + 1, *const drained = v_clear + 1;
  uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  int steps[2], seen = 0, most = 0;  // key steps of each tile; keys and steps of the block
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int last = min(nq, i0 + (x + 1) * tpt) - 1;
    const int keys = x < NQ && i0 + x * tpt < nq ? max(min(nk, last + 1 + shift), 0) : 0;
    steps[x] = (keys + KT - 1) / KT;
    seen = max(seen, keys);
    most = max(most, steps[x]);
  }
  const bool clears = seen < most * KT;  // the last V tile has rows that nothing sees

  if (warp == 0 && lane == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_ready[x], 4);
      mbar_init(&o_done[x], 1);
    }
    mbar_init(v_last, 1);
    mbar_init(v_clear, 1);
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const unsigned int hint = (unsigned int)(a.wait_ns < 1000000ull ? a.wait_ns : 1000000ull);
  bool timed_out = false;
  // for a whole warp: its lanes go on, or give up, together
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, pipe_wait(bar, parity, abort_flag, a.wait_ns, hint, &timed_out));
  };

  if (warp < 4) {
    if constexpr (NQ == 2) reg_dealloc<64>();
    if (warp == 0) {
      // ---- copies
      if (lane == 0 && most > 0) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(NQ * C::kSlabs * tpt * G * 128));
        for (int x = 0; x < NQ; ++x)
          for (int s = 0; s < C::kSlabs; ++s)
            tma_load_4d(smem + x * C::kQTile + s * C::kQSlab, &qmap, 64 * s, 0, h, q0 + i0 + x * tpt, q_full);
        int item = 0;
        for (; item < 2 * most; ++item) {
          const int st = item % ST;
          if (item >= ST && !pipe_wait(&kv_empty[st], (item / ST - 1) & 1, abort_flag, a.wait_ns, hint, &timed_out)) break;
          mbar_arrive_expect_tx(&kv_full[st], C::kStage);
          for (int s = 0; s < C::kSlabs; ++s)
            tma_load_3d(stages + st * C::kStage + s * C::kSlab, item & 1 ? &vmap : &kmap, 64 * s, h, k0 + (item >> 1) * KT,
                        &kv_full[st]);
        }
        // shared memory is the block's until its own copies have landed
        mbar_wait(q_full, 0);
        for (int i = max(0, item - ST); i < item; ++i) mbar_wait(&kv_full[i % ST], (i / ST) & 1);
      }
    } else if (warp == 1) {
      // ---- products
      const uint32_t is = idesc_16bit(128, KT, kBf16, false, a.negate), io = idesc_16bit(128, D, kBf16, true, false);
      const uint32_t qa = smem_u32(smem), sa = smem_u32(stages);
      auto scores = [&](int x, int buf, int j) {  // S[buf] = Q[x] K(j)^T
        const uint32_t ka = sa + ((2 * j) % ST) * C::kStage;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_f16_ss(tmem + C::s_col(buf), smem_desc_sw128(qa + x * C::kQTile + (k / 4) * C::kQSlab + (k % 4) * 32, 16, 1024),
                       smem_desc_sw128(ka + (k / 4) * C::kSlab + (k % 4) * 32, 16, 1024), is, k > 0);
          mma_commit(&s_full[buf]);
        }
        __syncwarp();
      };
      auto values = [&](int x, int buf, int j) {  // O[x] += P[buf] V(j)
        const uint32_t va = sa + ((2 * j + 1) % ST) * C::kStage;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            mma_f16_ts(tmem + C::o_col(x), tmem + C::s_col(buf) + 8 * k, smem_desc_sw128(va + k * 2048, C::kSlab, 1024), io,
                       j > 0 || k > 0);
          mma_commit(&o_done[x]);
        }
        __syncwarp();
      };
      auto release = [&](int item) {
        if (elect_one()) mma_commit(&kv_empty[item % ST]);
        __syncwarp();
      };
      auto landed = [&](int item) { return wait(&kv_full[item % ST], (item / ST) & 1); };
      // the last V tile goes to warp 2 first
      auto cleared = [&] {
        if (lane == 0) mbar_arrive(v_last);
        return wait(v_clear, 0);
      };
      bool ok = most == 0 || (wait(q_full, 0) && landed(0));
      tc_fence_after();
      if constexpr (NQ == 2) {
        if (ok && most > 0) {
          if (steps[0] > 0) scores(0, 0, 0);
          if (steps[1] > 0) scores(1, 1, 0);
          release(0);
        }
        for (int j = 0; ok && j < most; ++j) {
          ok = landed(2 * j + 1) && (j + 1 == most || landed(2 * j + 2));
          if (ok && clears && j + 1 == most) ok = cleared();
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (ok && j < steps[x]) {
              ok = wait(&p_ready[x], j & 1);
              tc_fence_after();
              if (ok) {
                values(x, x, j);
                if (j + 1 < steps[x]) scores(x, x, j + 1);
              }
            }
          }
          if (ok) {
            release(2 * j + 1);
            if (j + 1 < most) release(2 * j + 2);
          }
        }
      } else {
        if (ok && most > 0) {
          scores(0, 0, 0);
          release(0);
        }
        for (int j = 0; ok && j < most; ++j) {
          if (j + 1 < most) {
            ok = landed(2 * j + 2);
            tc_fence_after();
            if (!ok) break;
            scores(0, (j + 1) & 1, j + 1);
            release(2 * j + 2);
          }
          ok = landed(2 * j + 1) && (!clears || j + 1 < most || cleared()) && wait(&p_ready[j & 1], (j >> 1) & 1);
          tc_fence_after();
          if (ok) {
            values(0, j & 1, j);
            release(2 * j + 1);
          }
        }
      }
      // tensor and shared memory stay until every product has finished
      if (elect_one()) mma_commit(drained);
      __syncwarp();
      mbar_wait(drained, 0);
    } else if (warp == 2 && clears && most > 0) {
      // ---- V rows that nothing sees
      const int item = 2 * most - 1, rows = most * KT - seen;
      if (wait(v_last, 0)) {
        uint8_t *v = stages + (item % ST) * C::kStage + (KT - rows) * 128;
        for (int i = lane; i < rows * 8; i += 32)
#pragma unroll
          for (int s = 0; s < C::kSlabs; ++s) *reinterpret_cast<uint4 *>(v + s * C::kSlab + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_clear);
      }
    }
  } else {
    // ---- softmax: tile x, row r
    if constexpr (NQ == 2) reg_alloc<216>();
    const int x = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
    const int tok = i0 + x * tpt + r / G;
    const bool live = r < tpt * G && tok < nq;
    const int lim = live ? min(nk, tok + 1 + shift) : 0;      // keys this row sees
    const int easy = min(nk, i0 + x * tpt + 1 + shift);       // keys that every row of the tile sees
    const float c = a.scale_log2;
    float m = -INFINITY, l = 0.f;
    const int n = steps[x];
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int buf = NQ == 2 ? x : j & 1, phase = NQ == 2 ? j & 1 : (j >> 1) & 1;
      ok = wait(&s_full[buf], phase);
      if (!ok) break;
      tc_fence_after();
      const uint32_t st = tmem + C::s_col(buf) + lanes;
      uint32_t s[KT / 32][32];
#pragma unroll
      for (int i = 0; i < KT / 32; ++i) tmem_ld32(st + 32 * i, s[i]);
      tmem_wait_ld();
      if ((j + 1) * KT > easy || r >= tpt * G) {
        const int vis = lim - j * KT;
#pragma unroll
        for (int i = 0; i < KT; ++i)
          if (i >= vis) s[i / 32][i % 32] = 0xff800000u;
      }
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < KT; i += 2)
        top = max3f(top, __uint_as_float(s[i / 32][i % 32]), __uint_as_float(s[i / 32][i % 32 + 1]));
      // move the maximum only where it grew by more than 2^8
      const bool grow = (top - m) * c > 8.f;  // from -inf to anything; not from -inf to -inf
      if (__any_sync(0xffffffffu, grow)) {
        const float was = m;
        if (grow) m = fmaxf(m, top);
        const float f = was == m ? 1.f : ex2_approx((was - m) * c);  // was = -inf: 0
        l *= f;
        if (j > 0) {
          if constexpr (NQ == 1) {
            ok = wait(&o_done[x], (j - 1) & 1);  // (at NQ = 2 the scores were issued behind it)
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t ot = tmem + C::o_col(x) + lanes;
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
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
#pragma unroll
      for (int i = 0; i < KT / 32; ++i) {
        uint32_t p[16];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p0 = ex2_approx(fmaf(__uint_as_float(s[i][2 * e]), c, -mc));
          const float p1 = ex2_approx(fmaf(__uint_as_float(s[i][2 * e + 1]), c, -mc));
          sum += p0 + p1;
          p[e] = pack2<T>(p0, p1);
        }
        l += sum;
        tmem_st16(st + 16 * i, p);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[buf]);
    }
    // (at NQ = 1 the last scores do not stand behind the last product but one)
    if (NQ == 1 && n > 1 && ok) ok = wait(&o_done[x], n & 1);
    if (n > 0 && ok) ok = wait(&o_done[x], (n - 1) & 1);
    tc_fence_after();
    const float w = !ok ? __int_as_float(0x7fffffff) : l == 0.f ? 0.f : 1.f / l;
    T *out = reinterpret_cast<T *>(a.out) + (size_t)(q0 + tok) * a.out_stride + (size_t)(h * G + r % G) * D;
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      uint32_t o[32];
      if (n > 0 && ok) {
        tmem_ld32(tmem + C::o_col(x) + lanes + i, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0;
      }
      if (live) {
        // a row that sees nothing is zero whatever its product holds
        const bool none = lim <= 0 && ok;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = none ? 0.f : __uint_as_float(o[e + k]) * w;
          store8(out + i + e, y);
        }
      }
    }
  }
  if (timed_out) atomicOr(a.errors, TQ_ERRF_PROMPT_WAIT);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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

template <int D, class T>
cudaError_t launch(const PromptArgs &a, cudaStream_t stream) {
  using C = Prompt<D>;
  const int G = a.h_q / a.h_kv, tpt = 128 / G, tb = tpt * C::kTiles;
  const long long units = a.T_q / tb + (long long)a.batch;
  if (units * a.h_kv > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  CUtensorMap q, k, v;
  // with no keys at all the K and V maps are never read: any rows will do
  const bool none = a.T_k == 0;
  if (!encode<D, T>(&q, a.q, a.q_stride, a.h_q, G, a.T_q, tpt) ||
      !encode<D, T>(&k, none ? a.q : a.k, none ? a.q_stride : a.k_stride, none ? a.h_q : a.h_kv, 0, none ? a.T_q : a.T_k, C::kKeys) ||
      !encode<D, T>(&v, none ? a.q : a.v, none ? a.q_stride : a.v_stride, none ? a.h_q : a.h_kv, 0, none ? a.T_q : a.T_k, C::kKeys))
    return cudaErrorInvalidValue;
  auto *kernel = prompt_kernel<D, T>;
  static std::atomic<int> allowed[kAttributeDevices];
  const cudaError_t e = allow_smem(kernel, C::kSmem, allowed);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)(units * a.h_kv), C::kThreads, C::kSmem, stream>>>(a, q, k, v, (int)units);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, int d, tq_dtype dt, cudaStream_t stream) {
  const bool bf = dt == TQ_BF16;
  if (d == 64) return bf ? launch<64, __nv_bfloat16>(a, stream) : launch<64, __half>(a, stream);
  if (d == 128) return bf ? launch<128, __nv_bfloat16>(a, stream) : launch<128, __half>(a, stream);
  return bf ? launch<256, __nv_bfloat16>(a, stream) : launch<256, __half>(a, stream);
}

}  // namespace tq
