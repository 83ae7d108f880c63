// tq_prompt_attention, simplest form: a warp per (query row, head) walks the
// keys it sees, a lane holding d / 32 channels, with the running maximum and
// sum of the softmax in float32.
#include "paged.cuh"
#include "tq_common.cuh"

namespace tq {
namespace {

template <int D, class T>
__global__ void __launch_bounds__(128) prompt_simt_kernel(const __grid_constant__ PromptArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int hq = (int)(id % a.h_q);
  const long long r = id / a.h_q;
  if (r >= a.T_q) return;
  const int row = (int)r;
  // the sequence of this row
  int b = 0;
  while (b < a.batch && min(max(a.cu_q[b + 1], 0), a.T_q) <= row) ++b;
  if (b == a.batch) return;
  const int q0 = min(max(a.cu_q[b], 0), a.T_q), q1 = min(max(a.cu_q[b + 1], 0), a.T_q);
  if (row < q0) return;
  const int k0 = min(max(a.cu_k[b], 0), a.T_k), k1 = max(min(max(a.cu_k[b + 1], 0), a.T_k), k0);
  const int seen = min(k1 - k0, row - q0 + 1 + (k1 - k0) - (q1 - q0));
  const int h = hq / (a.h_q / a.h_kv);
  const T *q = reinterpret_cast<const T *>(a.q) + (size_t)row * a.q_stride + (size_t)hq * D;
  float qx[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qx[e] = (float)q[E * lane + e] * a.scale_log2;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < seen; ++j) {
    const T *k = reinterpret_cast<const T *>(a.k) + (size_t)(k0 + j) * a.k_stride + (size_t)h * D;
    const T *v = reinterpret_cast<const T *>(a.v) + (size_t)(k0 + j) * a.v_stride + (size_t)h * D;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qx[e], (float)k[E * lane + e], s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = fmaf(l, f, p);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f, p * (float)v[E * lane + e]);
  }
  T *out = reinterpret_cast<T *>(a.out) + (size_t)row * a.out_stride + (size_t)hq * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[E * lane + e] = (T)(seen > 0 ? o[e] / l : 0.f);
}

template <int D>
cudaError_t launch_d(const PromptArgs &a, tq_dtype dt, cudaStream_t stream) {
  const long long blocks = ((long long)a.T_q * a.h_q + 3) / 4;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (dt == TQ_BF16)
    prompt_simt_kernel<D, __nv_bfloat16><<<(unsigned)blocks, 128, 0, stream>>>(a);
  else
    prompt_simt_kernel<D, __half><<<(unsigned)blocks, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, int d, tq_dtype dt, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  return d == 64 ? launch_d<64>(a, dt, stream) : d == 128 ? launch_d<128>(a, dt, stream) : launch_d<256>(a, dt, stream);
}

}  // namespace tq
