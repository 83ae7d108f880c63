// tq_paged_gather: the values that 4-bit pages stand for, as contiguous rows.
//
// A warp takes one cell (16 positions) of one KV head: it fetches the cell's
// 20 d bytes in 16-byte pieces into shared memory and writes each row's keys
// and values eight channels a lane, so that a warp stores whole rows.
//
// Bound: bytes, 4/5 of them written.  16 sequences of up to 9000 tokens, 8
// heads, d = 64, fp16: 215 MB in 37.4 us, 5.75 TB/s (88% of the copy rate); 4 x
// 8192 tokens, 8 heads, d = 128, bf16: 176 MB in 31 us; 16384 tokens of 2
// heads: 5.4 us, half of it the launch.  Short-lived blocks of four warps carry
// the latency: a cell's fetch, then its rows, many blocks an SM.
#include "paged.cuh"
#include "tq_common.cuh"

namespace tq {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void expand8(uint32_t w, float s, float z, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((w >> (4 * i)) & 15u), s, z);
}

template <int D, class T>
__global__ void __launch_bounds__(32 * kWarps) paged_gather_kernel(const __grid_constant__ PagedGatherArgs a) {
  using C = Cell<D>;
  constexpr int kChunks = D / 8;
  __shared__ __align__(16) uint8_t cells[kWarps][C::kBytes];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long id = (long long)blockIdx.x * kWarps + warp;
  const int h = (int)(id % a.c.h_kv);
  const long long u = id / a.c.h_kv;
  if (u >= span_units<4>(a.rows, a.c.batch)) return;
  const Unit unit = find_unit<4>(a.cu, a.c.len, a.first, a.c.batch, a.rows, (int)u);
  const int b = unit.b, r0 = unit.r0, r1 = unit.r1, first = clamp_position(unit.y), len = unit.x;
  const int cell = (first >> 4) + (int)u - ((r0 >> 4) + 2 * b);
  const int lo = max(16 * cell, first), hi = min(16 * cell + 16, first + (r1 - r0));
  if (lo >= hi) return;
  const int page = page_of(a.c, b, lo);
  if (lane == 0 && (page < 0 || hi > len)) atomicOr(a.c.errors, TQ_ERRF_PAGE);
  uint8_t *const img = cells[warp];
  if (page >= 0) {
    const uint4 *src = reinterpret_cast<const uint4 *>(cell_ptr<D>(a.c, page, lo, h));
#pragma unroll
    for (int i = 0; i < C::kBytes / 16; i += 32)
      if (i + lane < C::kBytes / 16) reinterpret_cast<uint4 *>(img)[i + lane] = src[i + lane];
  }
  __syncwarp();
#pragma unroll 4
  for (int i = lane; i < kCell * kChunks; i += 32) {
    const int n = i / kChunks, chunk = i % kChunks, j = chunk >> 2, w4 = chunk & 3;
    const int pos = 16 * cell + n;
    if (pos < lo || pos >= hi) continue;
    const size_t row = (size_t)(r0 + (pos - first));
    T *ko = reinterpret_cast<T *>(a.k_out) + row * a.k_stride + (size_t)h * D + 8 * chunk;
    T *vo = reinterpret_cast<T *>(a.v_out) + row * a.v_stride + (size_t)h * D + 8 * chunk;
    auto half_at = [&](int at) { return __half2float(*reinterpret_cast<const __half *>(img + at)); };
    float x[8], y[8];
    if (page >= 0 && pos < len) {
      expand8(*reinterpret_cast<const uint32_t *>(img + C::key_word(n, j, w4)), half_at(C::kKeyScale + C::scale_at(n, j)),
              half_at(C::kKeyZero + C::key_zero_at(n, j)), x);
      const uint32_t w = *reinterpret_cast<const uint16_t *>(img + C::val_half(n, j, 2 * w4)) |
                         (uint32_t)*reinterpret_cast<const uint16_t *>(img + C::val_half(n, j, 2 * w4 + 1)) << 16;
      expand8(w, half_at(C::kValScale + C::scale_at(n, j)), half_at(C::kValZero + C::scale_at(n, j)), y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = y[e] = __int_as_float(0x7fffffff);
    }
    store8(ko, x);
    store8(vo, y);
  }
}

template <int D, class T>
cudaError_t launch(const PagedGatherArgs &a, cudaStream_t stream) {
  const long long warps = span_units<4>(a.rows, a.c.batch) * a.c.h_kv;
  const long long blocks = (warps + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  paged_gather_kernel<D, T><<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PagedGatherArgs &a, tq_dtype dt, cudaStream_t stream) {
  switch (dt) {
    case TQ_F32: return launch<D, float>(a, stream);
    case TQ_BF16: return launch<D, __nv_bfloat16>(a, stream);
    default: return launch<D, __half>(a, stream);
  }
}

}  // namespace

cudaError_t launch_paged_gather(const PagedGatherArgs &a, int d, tq_dtype dt, cudaStream_t stream) {
  return d == 64 ? launch_d<64>(a, dt, stream) : d == 128 ? launch_d<128>(a, dt, stream) : launch_d<256>(a, dt, stream);
}

}  // namespace tq
