// tq_paged_append: rotation by position, 4-bit min/max quantization and the
// scatter into pages, one launch.
//
// Mathematics.  A pair (a, b) of a head row turns by its position's angle; the
// products of two values of at most 24 bits are exact in float64, so each
// output is one float64 rounding and one to float32, whatever the order.  A
// group's codes follow include/tq.h: scale and codes are taken in float32 (the
// quotients' relative errors stay below 2^-21, at most 7e-6 of a code) and
// again in float64 where they lie that near a rounding boundary, so every
// stored bit is the exact one.
//
// A block takes one cell (16 positions of a sequence) and one KV head, with
// the query heads that read it: their rows share the positions, so cosines
// and sines are loaded and widened once per thread.  A warp takes 256 channels
// of rows (two rows at d = 128): it has each row's piece (the group's query
// heads, the key, the value) copied into shared memory by one bulk copy, so
// that what is in flight does not depend on registers, and turns and encodes
// them without waiting for the block's other warps.  A cell that the call
// fills is put together in shared memory and stored in 16-byte pieces; one
// that it fills in part (a decode step's single token) is stored in place, as
// words and half words that no other token shares.
//
// Bound: the rows' and pages' bytes on paper; measured, instruction issue (the
// float64 products of the rotation, their conversions, the codes; in a capture
// issue 69% of the cycles, the conversion unit and the ALU 48% each; at 32/8
// heads 32 of 40 turned rows are queries).  4 x 8192
// tokens, 32/8 heads, d = 128, bf16: 797 MB in 193 us, 4.1 TB/s (fp32: 1535 MB in
// 229 us, the copy rate; bf16 with a thread per
// 16 channels with its rows in registers: 266; a warp per cell with the rare
// exact codes inlined: 738, out of the instruction cache).  23 ragged fp16
// sequences, 12/2 heads, d = 64: 12.4 us.  One token of 32 sequences: 6.0 us,
// latency.  1024 threads an SM: room for 1280 gave 192 us too, with spills.
#include "paged.cuh"
#include "sm100.cuh"
#include "tq_common.cuh"
#include "tq_kernels.h"

namespace tq {
namespace {

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// fp16 of (hi - lo) / 15, rounded once.  The float32 quotient decides unless
// it lies next to a rounding boundary or below fp16's normal range.
__device__ __forceinline__ __half group_scale(float lo, float hi) {
  const float q = (hi - lo) * (1.f / 15.f);
  const int low = __float_as_int(q) & 0x1fff;
  if (abs(low - 0x1000) <= 16 || q < 0x1p-13f) {
    // the float64 quotient, by its reciprocal and one correction
    const double d = (double)hi - (double)lo, e = d * (1.0 / 15.0);
    return __double2half(fma(fma(-15.0, e, d), 1.0 / 15.0, e));
  }
  return __float2half_rn(q);
}

// Codes of eight channels, a quarter of a group; the group's other quarters
// lie in the other three lanes of an aligned quad.  Nibble i of the word is
// channel i.  Minimum and maximum carry a NaN on, so its group stores NaN.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], __half *scale, __half *zero) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const __half z = __float2half_rn(lo);
  const __half s = group_scale(lo, hi);
  const float zf = __half2float(z), sf = __half2float(s);
  const float inv = sf > 0.f ? __fdividef(1.f, sf) : 0.f;
  constexpr float kInt = 8388608.f;  // 2^23: the sum's low bits are the rounded code
  uint32_t w = 0;
  bool near = false;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float t = fminf(fmaxf((x[i] - zf) * inv, 0.f), 15.f);  // NaN: fmaxf gives 0
    const float m = t + kInt;
    near |= fabsf(t - (m - kInt)) > 0.5f - 1e-5f;
    w = (w << 4) + __float_as_uint(m);
  }
  w -= 0x4b000000u + 0xb0000000u;  // 2^23's bits, which the shifts have moved out but for channels 0 and 1
  if (near) {
    w = 0;
#pragma unroll 1
    for (int i = 7; i >= 0; --i) {
      const double t = ((double)x[i] - (double)zf) / (double)sf;
      w = w << 4 | (uint32_t)fmin(fmax(rint(t), 0.0), 15.0);
    }
  }
  *scale = s;
  *zero = z;
  return w;
}

// Four elements as they lie in memory.
template <class T>
struct Raw {
  uint32_t w[sizeof(T)];
};
template <class T>
__device__ __forceinline__ void fetch(Raw<T> &r, const T *p) {
  if constexpr (sizeof(T) == 4) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    r.w[0] = u.x; r.w[1] = u.y;
  }
}
template <class T>
__device__ __forceinline__ void widen(const Raw<T> &r, float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (__is_same(T, __half)) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
        x[2 * i] = f.x; x[2 * i + 1] = f.y;
      } else {
        x[2 * i] = __uint_as_float(r.w[i] << 16);
        x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
      }
    }
  }
}
template <class T>
__device__ __forceinline__ void store4(T *p, const float (&x)[4]) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
}
// Shared memory of a block: the warps' barriers, the assembled cell, the turned
// keys in float32 (rows padded by 16 bytes) and the rows as they came.
template <int D, class T>
struct AppendSmem {
  static constexpr int kImage = 128, kPad = D + 4;
  static constexpr int kKeys = kImage + Cell<D>::kBytes;
  static constexpr int kRows = kKeys + kCell * kPad * 4;
  static constexpr size_t bytes(int G) { return kRows + (size_t)kCell * (G + 2) * D * sizeof(T); }
};

// 2 D threads: thread (n, p) of row n = tid / (D / 8) turns two chunks of four
// channels, a and b, which hold whole pairs, and encodes eight channels.
template <int D, class T>
__global__ void __launch_bounds__(2 * D, 1024 / (2 * D)) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  using C = Cell<D>;
  using S = AppendSmem<D, T>;
  constexpr int kChunks = D / 8, kOwn = 32 / kChunks;  // rows of a warp
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t *const bar = reinterpret_cast<uint64_t *>(smem) + warp;
  uint8_t *const image = smem + S::kImage;
  float *const keys = reinterpret_cast<float *>(smem + S::kKeys);
  T *const rows = reinterpret_cast<T *>(smem + S::kRows);
  if (lane == 0) {
    sm100::mbar_init(bar, 1);
    sm100::fence_mbar_init();
  }
  const int h = blockIdx.x % a.c.h_kv, u = blockIdx.x / a.c.h_kv;
  const Unit unit = find_unit<4>(a.cu, a.c.len, nullptr, a.c.batch, a.T, u);
  const int b = unit.b, r0 = unit.r0, r1 = unit.r1;
  const int first = clamp_position(unit.x) - (r1 - r0);  // position of row r0
  const int cell = (first >> 4) + u - ((r0 >> 4) + 2 * b);
  // rows of this cell: positions 16 cell .. 16 cell + 15
  const int lo = max(16 * cell, first), hi = min(16 * cell + 16, first + (r1 - r0));
  if (lo >= hi) return;

  // ---- the warp's rows: [row][query heads of the group, key, value][D]
  const int G = a.q ? a.h_q / a.c.h_kv : 0, row_elems = (G + 2) * D;
  const int own = 16 * cell + warp * kOwn;  // the warp's first position
  const int from = max(own, lo), count = max(min(own + kOwn, hi) - from, 0);
  __syncwarp();
  if (lane == 0 && count > 0) sm100::mbar_arrive_expect_tx(bar, (uint32_t)(count * row_elems * sizeof(T)));
  if (lane < 3 * count && a.c.withhold != 1) {
    const int pos = from + lane / 3, kind = lane % 3;
    T *const to = rows + (pos - 16 * cell) * row_elems;
    const size_t row = (size_t)(r0 + (pos - first));
    if (kind == 0) {
      if (G) sm100::bulk_g2s(to, reinterpret_cast<const T *>(a.q) + row * a.q_stride + (size_t)h * G * D, G * D * sizeof(T), bar);
    } else if (kind == 1) {
      sm100::bulk_g2s(to + G * D, reinterpret_cast<const T *>(a.k) + row * a.k_stride + (size_t)h * D, D * sizeof(T), bar);
    } else {
      sm100::bulk_g2s(to + (G + 1) * D, reinterpret_cast<const T *>(a.v) + row * a.v_stride + (size_t)h * D, D * sizeof(T), bar);
    }
  }

  // ---- meanwhile the page and the angles
  const int n = tid / kChunks, p = tid % kChunks, pos = 16 * cell + n;
  const bool live = pos >= lo && pos < hi, rotates = a.rope != nullptr;
  const bool in_table = !rotates || (pos >= 0 && pos < a.max_positions);
  // tokens outside the rotation's table are not stored
  const int last = rotates ? min(hi, a.max_positions) : hi;
  const bool stored = live && pos < last, whole = last - lo == kCell;
  const int half = a.rotary_dim / 2;
  const bool turn = rotates && live && in_table && 8 * p < a.rotary_dim;
  const bool split = turn && !a.interleaved;  // pairs (i, i + half): chunk a and chunk b
  const int ca = split ? 4 * p : 8 * p, cb = split ? half + 4 * p : 8 * p + 4;
  double cs[4], sn[4];
  if (turn) {
    const float *table = a.rope + (size_t)pos * a.rotary_dim + 4 * p;
    const float4 c = *reinterpret_cast<const float4 *>(table), s = *reinterpret_cast<const float4 *>(table + half);
    cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
    sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
  }
  const int page = page_of(a.c, b, lo);
  if (page < 0 && tid == 0) atomicOr(a.c.errors, TQ_ERRF_PAGE);
  if (live && !in_table && p == 0 && h == 0) atomicOr(a.c.errors, TQ_ERRF_POSITION);
  // Should the wait run out, the warp's rows stay unwritten, and it waits for its copies before it leaves: the shared
  // memory is the next block's then.  (withhold 1: no copies; 2: they count as late.)
  const bool ok =
      count > 0 && __all_sync(0xffffffffu, a.c.withhold != 2 && sm100::mbar_wait(bar, 0, a.c.wait_ns));
  if (count > 0 && !ok) {
    if (lane == 0) atomicOr(a.c.errors, TQ_ERRF_QUANTIZE_WAIT);
    if (a.c.withhold != 1) sm100::mbar_wait(bar, 0);
  }

  if (ok) {
    // ---- rotation: turns the chunks a and b of a head row
    const T *const mine = rows + n * row_elems;
    auto rotate = [&](const T *from, float (&x)[4], float (&y)[4]) {
      Raw<T> ra, rb;
      fetch(ra, from + ca);
      fetch(rb, from + cb);
      widen(ra, x);
      widen(rb, y);
      auto pair = [](float &u, float &v, double c, double w) {
        const double s = u, t = v;
        u = (float)fma(s, c, -(t * w));
        v = (float)fma(t, c, s * w);
      };
      if (split) {
#pragma unroll
        for (int i = 0; i < 4; ++i) pair(x[i], y[i], cs[i], sn[i]);
      } else if (turn) {
        pair(x[0], x[1], cs[0], sn[0]);
        pair(x[2], x[3], cs[1], sn[1]);
        pair(y[0], y[1], cs[2], sn[2]);
        pair(y[2], y[3], cs[3], sn[3]);
      } else if (!in_table) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = y[i] = __int_as_float(0x7fffffff);
      }
    };
    if (live) {
      const size_t row = (size_t)(r0 + (pos - first));
      float x[4], y[4];
      rotate(mine + G * D, x, y);
      *reinterpret_cast<float4 *>(&keys[n * S::kPad + ca]) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4 *>(&keys[n * S::kPad + cb]) = make_float4(y[0], y[1], y[2], y[3]);
      if (a.k_out) {
        T *o = reinterpret_cast<T *>(a.k_out) + row * a.k_out_stride + (size_t)h * D;
        store4(o + ca, x);
        store4(o + cb, y);
      }
      T *o = reinterpret_cast<T *>(a.q_out) + row * a.q_out_stride + (size_t)h * G * D;
      const T *from = mine;
#pragma unroll 2
      for (int g = 0; g < G; ++g, o += D, from += D) {
        rotate(from, x, y);
        store4(o + ca, x);
        store4(o + cb, y);
      }
    }
    __syncwarp();

    // ---- codes of channels 8 p .. + 7 of row n, keys and then values; the four
    // lanes of a group belong to one row, every lane takes part in the shuffles
    // and stored rows write
    if (page >= 0) {
      uint8_t *const to = whole ? image : cell_ptr<D>(a.c, page, lo, h);
      const int j = p >> 2, w4 = p & 3;
      float z[8];
      __half scale, zero;
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = 0.f;
      if (stored) load8(&keys[n * S::kPad + 8 * p], z);
      uint32_t w = encode8(z, &scale, &zero);
      if (stored) {
        *reinterpret_cast<uint32_t *>(to + C::key_word(n, j, w4)) = w;
        if (w4 == 0) *reinterpret_cast<__half *>(to + C::kKeyScale + C::scale_at(n, j)) = scale;
        if (w4 == 1) *reinterpret_cast<__half *>(to + C::kKeyZero + C::key_zero_at(n, j)) = zero;
        load8(mine + (G + 1) * D + 8 * p, z);
      }
      w = encode8(z, &scale, &zero);
      if (stored) {
        *reinterpret_cast<uint16_t *>(to + C::val_half(n, j, 2 * w4)) = (uint16_t)w;
        *reinterpret_cast<uint16_t *>(to + C::val_half(n, j, 2 * w4 + 1)) = (uint16_t)(w >> 16);
        if (w4 == 2) *reinterpret_cast<__half *>(to + C::kValScale + C::scale_at(n, j)) = scale;
        if (w4 == 3) *reinterpret_cast<__half *>(to + C::kValZero + C::scale_at(n, j)) = zero;
      }
    }
  }
  if (whole && page >= 0) {
    if (!__syncthreads_and(ok)) return;
    uint4 *const to = reinterpret_cast<uint4 *>(cell_ptr<D>(a.c, page, lo, h));
    for (int i = tid; i < C::kBytes / 16; i += 2 * D) to[i] = reinterpret_cast<const uint4 *>(image)[i];
  }
}

template <int D, class T>
cudaError_t launch(const PagedAppendArgs &a, cudaStream_t stream) {
  using S = AppendSmem<D, T>;
  const long long blocks = span_units<4>(a.T, a.c.batch) * a.c.h_kv;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  static std::atomic<int> allowed[kAttributeDevices];
  const cudaError_t e = allow_smem(paged_append_kernel<D, T>, S::bytes(TQ_PAGED_MAX_GQA), allowed);
  if (e != cudaSuccess) return e;
  paged_append_kernel<D, T><<<(unsigned)blocks, 2 * D, S::bytes(a.q ? a.h_q / a.c.h_kv : 0), stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PagedAppendArgs &a, tq_dtype dt, cudaStream_t stream) {
  switch (dt) {
    case TQ_F32: return launch<D, float>(a, stream);
    case TQ_BF16: return launch<D, __nv_bfloat16>(a, stream);
    default: return launch<D, __half>(a, stream);
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs &a, int d, tq_dtype dt, cudaStream_t stream) {
  return d == 64 ? launch_d<64>(a, dt, stream) : d == 128 ? launch_d<128>(a, dt, stream) : launch_d<256>(a, dt, stream);
}

}  // namespace tq
