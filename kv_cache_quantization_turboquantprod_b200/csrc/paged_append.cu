// tq_paged_append: rotation by position, 4-bit min/max quantization and the
// scatter into pages, one launch.
//
// Mathematics.  A pair (a, b) of a head row turns by its position's angle; the
// products of two values of at most 24 bits are exact in float64, so each
// output is one float64 rounding and one to float32, whatever the order.  A
// group's codes follow include/tq.h; the quotient is taken in float32 by the
// scale's reciprocal (relative error below 2^-22, so at most 4e-6 at the
// largest code) and again in float64 where it lies within 1e-5 of a rounding
// boundary, so every code is the exact one.
//
// A block takes one cell (16 positions of a sequence) and one KV head, with
// the query heads that read it: their rows share the positions, so cosines
// and sines are loaded and widened once per thread.  A cell that the call
// fills is put together in shared memory and stored in 16-byte pieces; one
// that it fills in part (a decode step's single token) is stored in place,
// as words and half words that no other token shares.
#include "paged.cuh"
#include "tq_common.cuh"

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
  const __half s = __double2half(((double)hi - (double)lo) / 15.0);
  const float zf = __half2float(z), sf = __half2float(s);
  const float inv = sf > 0.f ? 1.f / sf : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = (x[i] - zf) * inv;
    float r = rintf(t);
    if (fabsf(t - r) > 0.5f - 1e-5f && sf > 0.f) r = (float)rint(((double)x[i] - (double)zf) / (double)sf);
    w |= (uint32_t)fminf(fmaxf(r, 0.f), 15.f) << (4 * i);  // NaN: fmaxf gives 0
  }
  *scale = s;
  *zero = z;
  return w;
}

// D threads: thread (n, p) of row n = tid / (D / 16) rotates two chunks of
// eight channels, a and b, which hold whole pairs.
template <int D, class T>
__global__ void __launch_bounds__(D) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  using C = Cell<D>;
  constexpr int kChunks = D / 8, kRowThreads = D / 16, kPad = D + 4;
  __shared__ __align__(16) float keys[kCell * kPad];
  __shared__ __align__(16) uint8_t image[C::kBytes];
  const int tid = threadIdx.x;
  const int h = blockIdx.x % a.c.h_kv;
  const int u = blockIdx.x / a.c.h_kv;
  const int b = unit_sequence(a.cu, a.c.batch, a.T, u);
  const int r0 = clamp_cu(a.cu, b, a.T), r1 = max(clamp_cu(a.cu, b + 1, a.T), r0);
  const int first = a.c.len[b] - (r1 - r0);  // position of row r0
  const int cell = (first >> 4) + u - ((r0 >> 4) + 2 * b);
  // rows of this cell: positions 16 cell .. 16 cell + 15
  const int lo = max(16 * cell, first), hi = min(16 * cell + 16, first + (r1 - r0));
  if (lo >= hi) return;
  const int page = page_of(a.c, b, lo);
  // tokens outside the rotation's table are not stored
  const int last = a.rope ? min(hi, a.max_positions) : hi;
  const bool whole = last - lo == kCell;
  if (page < 0 && tid == 0) atomicOr(a.c.errors, TQ_ERRF_PAGE);
  uint8_t *const cellp = page < 0 ? image : cell_ptr<D>(a.c, page, lo, h);
  uint8_t *const to = whole ? image : cellp;

  // ---- rotation
  const int n = tid / kRowThreads, p = tid % kRowThreads;
  const int pos = 16 * cell + n;
  const bool live = pos >= lo && pos < hi;
  const bool rotates = a.rope != nullptr;
  const bool in_table = !rotates || (pos >= 0 && pos < a.max_positions);
  if (live && !in_table && p == 0 && h == 0) atomicOr(a.c.errors, TQ_ERRF_POSITION);
  const int half = a.rotary_dim / 2;
  const bool turn = rotates && live && in_table && 16 * p < a.rotary_dim;
  const bool split = turn && !a.interleaved;  // pairs (i, i + half): chunk a and chunk b
  const int ca = split ? 8 * p : 16 * p, cb = split ? half + 8 * p : 16 * p + 8;
  double cs[8], sn[8];
  if (turn) {
    float f[8];
    const float *row = a.rope + (size_t)pos * a.rotary_dim + 8 * p;
    load8(row, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = f[i];
    load8(row + half, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) sn[i] = f[i];
  }
  auto rotate = [&](float (&x)[8], float (&y)[8]) {
    if (!turn) {
      if (live && !in_table)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = y[i] = __int_as_float(0x7fffffff);
      return;
    }
    auto one = [](float &s, float &t, double c, double w) {
      const double ds = s, dt = t;
      s = (float)fma(ds, c, -(dt * w));
      t = (float)fma(dt, c, ds * w);
    };
    if (split) {
#pragma unroll
      for (int i = 0; i < 8; ++i) one(x[i], y[i], cs[i], sn[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        one(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
        one(y[2 * i], y[2 * i + 1], cs[4 + i], sn[4 + i]);
      }
    }
  };
  const size_t row = (size_t)(r0 + (pos - first));
  float x[8], y[8];
  if (live) {
    const T *k = reinterpret_cast<const T *>(a.k) + row * a.k_stride + (size_t)h * D;
    load8(k + ca, x);
    load8(k + cb, y);
    rotate(x, y);
    if (a.k_out) {
      T *o = reinterpret_cast<T *>(a.k_out) + row * a.k_out_stride + (size_t)h * D;
      store8(o + ca, x);
      store8(o + cb, y);
    }
    *reinterpret_cast<float4 *>(&keys[n * kPad + ca]) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(&keys[n * kPad + ca + 4]) = make_float4(x[4], x[5], x[6], x[7]);
    *reinterpret_cast<float4 *>(&keys[n * kPad + cb]) = make_float4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<float4 *>(&keys[n * kPad + cb + 4]) = make_float4(y[4], y[5], y[6], y[7]);
    if (a.q) {
      const int G = a.h_q / a.c.h_kv;
      const T *q = reinterpret_cast<const T *>(a.q) + row * a.q_stride + (size_t)h * G * D;
      T *o = reinterpret_cast<T *>(a.q_out) + row * a.q_out_stride + (size_t)h * G * D;
      for (int g = 0; g < G; ++g) {
        load8(q + g * D + ca, x);
        load8(q + g * D + cb, y);
        rotate(x, y);
        store8(o + g * D + ca, x);
        store8(o + g * D + cb, y);
      }
    }
  }
  __syncthreads();
  if (page < 0) return;

  // ---- codes: units of eight channels; the four lanes of a group belong to
  // one row, every lane takes part in the shuffles and stored rows write
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int i = it * D + tid, m = i / kChunks, chunk = i % kChunks;
    const int at = 16 * cell + m, j = chunk >> 2, w4 = chunk & 3;
    const bool stored = at >= lo && at < last;
    float kx[8], vx[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) kx[e] = vx[e] = 0.f;
    if (stored) {
      load8(&keys[m * kPad + 8 * chunk], kx);
      load8(reinterpret_cast<const T *>(a.v) + (size_t)(r0 + (at - first)) * a.v_stride + (size_t)h * D + 8 * chunk, vx);
    }
    __half ks, kz, vs, vz;
    const uint32_t kw = encode8(kx, &ks, &kz), vw = encode8(vx, &vs, &vz);
    if (stored) {
      *reinterpret_cast<uint32_t *>(to + C::key_word(m, j, w4)) = kw;
      *reinterpret_cast<uint16_t *>(to + C::val_half(m, j, 2 * w4)) = (uint16_t)vw;
      *reinterpret_cast<uint16_t *>(to + C::val_half(m, j, 2 * w4 + 1)) = (uint16_t)(vw >> 16);
      const int section[4] = {C::kKeyScale + C::scale_at(m, j), C::kKeyZero + C::key_zero_at(m, j),
                              C::kValScale + C::scale_at(m, j), C::kValZero + C::scale_at(m, j)};
      const __half number[4] = {ks, kz, vs, vz};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (w4 == e) *reinterpret_cast<__half *>(to + section[e]) = number[e];
    }
  }
  if (whole) {
    __syncthreads();
    for (int i = tid; i < C::kBytes / 16; i += D)
      reinterpret_cast<uint4 *>(cellp)[i] = reinterpret_cast<const uint4 *>(image)[i];
  }
}

template <int D, class T>
cudaError_t launch(const PagedAppendArgs &a, cudaStream_t stream) {
  const long long blocks = cell_units(a.T, a.c.batch) * a.c.h_kv;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  paged_append_kernel<D, T><<<(unsigned)blocks, D, 0, stream>>>(a);
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
