// tq_paged_decode_attention, simplest form: a warp per (sequence, query head)
// walks the cached tokens, a lane holding d / 32 channels, with the running
// maximum and sum of the softmax in float32.
#include "paged.cuh"
#include "tq_common.cuh"

namespace tq {
namespace {

template <int D, class T>
__global__ void __launch_bounds__(32) paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a) {
  using C = Cell<D>;
  constexpr int E = D / 32;  // channels of a lane
  const int lane = threadIdx.x;
  const int b = blockIdx.x / a.h_q, hq = blockIdx.x % a.h_q, h = hq / (a.h_q / a.c.h_kv);
  const int len = a.c.len[b];
  const T *q = reinterpret_cast<const T *>(a.q) + (size_t)b * a.q_stride + (size_t)hq * D;
  float qx[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qx[e] = (float)q[E * lane + e] * a.scale_log2;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  for (int pos = 0; pos < len; ++pos) {
    const int page = page_of(a.c, b, pos);
    if (page < 0) {
      bad = true;
      break;
    }
    const uint8_t *cell = cell_ptr<D>(a.c, page, pos, h);
    const int n = pos & 15;
    float kx[E], vx[E], s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = E * lane + e, j = c >> 5, r = c & 31;
      auto half_at = [&](int at) { return __half2float(*reinterpret_cast<const __half *>(cell + at)); };
      const int kc = (cell[C::key_word(n, j, r >> 3) + ((r & 7) >> 1)] >> (4 * (r & 1))) & 15;
      const int vc = (cell[C::val_half(n, j, r >> 2) + ((r & 3) >> 1)] >> (4 * (r & 1))) & 15;
      kx[e] = fmaf((float)kc, half_at(C::kKeyScale + C::scale_at(n, j)), half_at(C::kKeyZero + C::key_zero_at(n, j)));
      vx[e] = fmaf((float)vc, half_at(C::kValScale + C::scale_at(n, j)), half_at(C::kValZero + C::scale_at(n, j)));
      s = fmaf(qx[e], kx[e], s);
    }
    s = warp_sum(s);
    const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = fmaf(l, f, p);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f, p * vx[e]);
  }
  if (bad && lane == 0) atomicOr(a.c.errors, TQ_ERRF_PAGE);
  T *out = reinterpret_cast<T *>(a.out) + (size_t)b * a.out_stride + (size_t)hq * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[E * lane + e] = (T)(bad ? __int_as_float(0x7fffffff) : len > 0 ? o[e] / l : 0.f);
}

template <int D>
cudaError_t launch_d(const PagedDecodeArgs &a, tq_dtype dt, cudaStream_t stream) {
  const unsigned blocks = (unsigned)(a.c.batch * a.h_q);
  if (dt == TQ_BF16)
    paged_decode_kernel<D, __nv_bfloat16><<<blocks, 32, 0, stream>>>(a);
  else
    paged_decode_kernel<D, __half><<<blocks, 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t paged_decode_workspace(int d, int h_kv, int h_q, int batch, int num_sms) {
  (void)d; (void)h_kv; (void)h_q; (void)batch; (void)num_sms;
  return 256;
}

cudaError_t launch_paged_decode(const PagedDecodeArgs &a, int d, tq_dtype dt, cudaStream_t stream) {
  return d == 64 ? launch_d<64>(a, dt, stream) : d == 128 ? launch_d<128>(a, dt, stream) : launch_d<256>(a, dt, stream);
}

}  // namespace tq
