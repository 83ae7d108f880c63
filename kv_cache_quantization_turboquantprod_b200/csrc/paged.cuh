// The paged 4-bit cache (layout in include/tq.h) and launch interface of the
// paged and prompt kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tq.h"

namespace tq {

constexpr int kCell = 16;  // tokens of a cell

// A pool and the sequences of a call, as the kernels take them.
struct PagedView {
  uint8_t *data;
  const int32_t *len, *table;
  int batch, max_pages, table_stride;
  int page_shift;  // log2 of the tokens of a page
  int num_pages, h_kv;
  unsigned int *errors;
  unsigned long long wait_ns;  // limit of the bounded waits
  int withhold;                // tests of the timeout path (tq_test_withhold_handoffs); 1: no copies
};

// Sections and strides of a cell of head dim D (bytes).
template <int D>
struct Cell {
  static constexpr int kGroups = D / 32;
  static constexpr int kP = kGroups < 4 ? kGroups : 4;  // code words a lane takes together
  static constexpr int kKeys = 0, kVals = 8 * D;
  static constexpr int kKeyScale = 16 * D, kKeyZero = kKeyScale + 32 * kGroups;
  static constexpr int kValScale = kKeyZero + 32 * kGroups, kValZero = kValScale + 32 * kGroups;
  static constexpr int kBytes = 20 * D;

  // Word of token n's channels 32 j + 8 u .. + 7.
  __host__ __device__ static constexpr int key_word(int n, int j, int u) {
    return (j / kP) * 256 * kP + n * 16 * kP + u * 4 * kP + (j % kP) * 4;
  }
  // Half word of token n's channels 32 j + 4 g .. + 3.
  __host__ __device__ static constexpr int val_half(int n, int j, int g) {
    return kVals + (j / kP) * 256 * kP + (n >> 3) * 128 * kP + (g * 4 + ((n >> 1) & 3)) * 4 * kP + (j % kP) * 4 +
           2 * (n & 1);
  }
  // Byte offset of (token n, group j) in a scale section.
  __host__ __device__ static constexpr int scale_at(int n, int j) {
    return ((n >> 1) & 3) * 8 * kGroups + j * 8 + (n >> 3) * 4 + (n & 1) * 2;
  }
  __host__ __device__ static constexpr int key_zero_at(int n, int j) { return (n * kGroups + j) * 2; }
};

// Lengths and first positions beyond any table's row, without overflow.
__device__ __forceinline__ int clamp_position(int x) { return min(max(x, -(1 << 30)), 1 << 30); }

// The page of position pos of sequence b; -1 where the table has none.
__device__ __forceinline__ int page_of(const PagedView &c, int b, int pos) {
  const int i = pos >> c.page_shift;
  if (pos < 0 || i >= c.max_pages) return -1;
  const int p = c.table[(size_t)b * c.table_stride + i];
  return p >= 0 && p < c.num_pages ? p : -1;
}

// Cell of position pos (page p) and KV head h.  64-bit: a pool may be
// larger than 4 GB.
template <int D>
__device__ __forceinline__ uint8_t *cell_ptr(const PagedView &c, int p, int pos, int h) {
  const int cells = 1 << (c.page_shift - 4);
  const size_t at = ((size_t)p * c.h_kv + h) * cells + ((pos >> 4) & (cells - 1));
  return c.data + at * Cell<D>::kBytes;
}

// Packed rows grouped by spans of 2^S positions: sequence b, whose rows are
// cu[b] .. cu[b + 1] - 1 at positions first .. , owns the units [(cu[b] >> S) +
// 2 b, (cu[b + 1] >> S) + 2 (b + 1)), one per span that its rows touch; n rows
// touch at most (n + 2^S - 2) / 2^S + 1 <= n / 2^S + 2 spans, and the range has
// at least n / 2^S + 2 units, so no prefix sum is needed.  cu is clamped to
// [0, rows].
__device__ __forceinline__ int clamp_cu(const int32_t *cu, int b, int rows) { return min(max(cu[b], 0), rows); }
template <int S>
__host__ __device__ __forceinline__ long long span_units(int rows, int batch) {
  return (rows >> S) + 2ll * batch;
}

// Sequence that owns unit u.  Warp-cooperative 32-way search: every lane
// probes one of 32 equal steps (one round per factor of 32 in the batch).
template <int S>
__device__ __forceinline__ int unit_sequence(const int32_t *cu, int batch, int rows, int u) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const bool below = at < n && (clamp_cu(cu, lo + at, rows) >> S) + 2 * (lo + at) <= u;
    const int k = max(__popc(__ballot_sync(0xffffffffu, below)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// A unit's sequence, its rows and two of its entries (x, y: [batch], y may be
// null).  Up to 32 sequences: every lane loads one's, so that one memory
// latency passes instead of three.
struct Unit {
  int b, r0, r1, x, y;
};
template <int S>
__device__ __forceinline__ Unit find_unit(const int32_t *cu, const int32_t *x, const int32_t *y, int batch, int rows, int u) {
  Unit t;
  if (batch <= 32) {
    const int lane = threadIdx.x & 31, i = min(lane, batch - 1);
    const int c0 = clamp_cu(cu, i, rows), c1 = clamp_cu(cu, i + 1, rows), xi = x[i], yi = y ? y[i] : 0;
    const bool below = lane < batch && (c0 >> S) + 2 * lane <= u;
    t.b = max(__popc(__ballot_sync(0xffffffffu, below)) - 1, 0);
    t.r0 = __shfl_sync(0xffffffffu, c0, t.b);
    t.r1 = __shfl_sync(0xffffffffu, c1, t.b);
    t.x = __shfl_sync(0xffffffffu, xi, t.b);
    t.y = __shfl_sync(0xffffffffu, yi, t.b);
  } else {
    t.b = unit_sequence<S>(cu, batch, rows, u);
    t.r0 = clamp_cu(cu, t.b, rows);
    t.r1 = clamp_cu(cu, t.b + 1, rows);
    t.x = x[t.b];
    t.y = y ? y[t.b] : 0;
  }
  t.r1 = max(t.r1, t.r0);
  return t;
}

// Rows as 32-bit values: eight consecutive elements of T.
template <class T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2 && __is_same(T, __half)) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x; x[2 * i + 1] = f.y;
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (__is_same(T, __half)) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}
template <class T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
struct PagedAppendArgs {
  PagedView c;
  const float *rope;  // null: no rotation
  int rotary_dim, max_positions, interleaved;
  const int32_t *cu;
  const void *q, *k, *v;
  void *q_out, *k_out;
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int h_q, T;
};
cudaError_t launch_paged_append(const PagedAppendArgs &a, int d, tq_dtype dt, cudaStream_t stream);

struct PagedGatherArgs {
  PagedView c;
  const int32_t *cu, *first;
  void *k_out, *v_out;
  long long k_stride, v_stride;
  int rows;
};
cudaError_t launch_paged_gather(const PagedGatherArgs &a, int d, tq_dtype dt, cudaStream_t stream);

struct PagedDecodeArgs {
  PagedView c;
  const void *q;
  void *out;
  long long q_stride, out_stride;
  int h_q;
  float scale_log2;  // softmax scale times log2(e)
  float *partials;   // workspace
  int num_sms;
};
size_t paged_decode_workspace(int d, int h_kv, int h_q, int batch, int num_sms);
cudaError_t launch_paged_decode(const PagedDecodeArgs &a, int d, tq_dtype dt, cudaStream_t stream);

struct PromptArgs {
  const void *q, *k, *v;
  void *out;
  long long q_stride, k_stride, v_stride, out_stride;
  const int32_t *cu_q, *cu_k;
  int T_q, T_k, h_q, h_kv, batch;
  float scale_log2;  // |softmax scale| times log2(e), at least 1e-30
  int negate;        // the scale is negative
  unsigned long long wait_ns;
  int withhold;
  unsigned int *errors;
};
cudaError_t launch_prompt(const PromptArgs &a, int d, tq_dtype dt, cudaStream_t stream);

}  // namespace tq
