// C-ABI entry points of the paged 4-bit cache and of the prompt attention
// (include/tq.h): host-side validation and launches.  Nothing here allocates
// or synchronises.
#include <cmath>

#include "paged.cuh"
#include "tq_kernels.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t dtype_size(tq_dtype t) { return t == TQ_F32 ? 4 : 2; }

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// Rows of `row` elements, `stride` apart, read and written 16 bytes at a time.
bool rows_ok(const void *p, long long stride, long long row, tq_dtype t) {
  return p && aligned(p, 16) && stride >= row && (size_t)stride * dtype_size(t) % 16 == 0;
}

// Bytes of a pool of valid arguments; false where they are more than an address holds.
bool pool_bytes(int d, int h_kv, int page_tokens, int num_pages, size_t *out) {
  const size_t cells = (size_t)num_pages * h_kv, cell = (size_t)(page_tokens / 16) * 20 * d;
  return !__builtin_mul_overflow(cells, cell, out);
}

tq_status check_cache(const tq_paged_cache *c) {
  if (!c || !c->data || !aligned(c->data, 256)) return TQ_ERR_INVALID_ARGUMENT;
  if (!head_dim_ok(c->d)) return TQ_ERR_UNSUPPORTED;
  if (c->page_tokens < 16 || c->page_tokens > 1024 || (c->page_tokens & (c->page_tokens - 1))) return TQ_ERR_UNSUPPORTED;
  if (c->h_kv < 1 || c->num_pages < 1) return TQ_ERR_INVALID_ARGUMENT;
  size_t bytes;
  return pool_bytes(c->d, c->h_kv, c->page_tokens, c->num_pages, &bytes) ? TQ_OK : TQ_ERR_CAPACITY;
}

tq_status check_batch(const tq_paged_cache *c, const tq_paged_batch *s) {
  if (!s || s->batch < 1 || s->max_pages < 1 || s->table_stride < s->max_pages) return TQ_ERR_INVALID_ARGUMENT;
  if (!s->len || !s->block_table || !aligned(s->len, 4) || !aligned(s->block_table, 4)) return TQ_ERR_INVALID_ARGUMENT;
  // positions and cell units are 32-bit
  if ((long long)s->max_pages * c->page_tokens > (1ll << 30) || s->batch > (1 << 20)) return TQ_ERR_CAPACITY;
  return TQ_OK;
}

tq_status view(const tq_paged_cache *c, const tq_paged_batch *s, tq::PagedView *v) {
  v->data = static_cast<uint8_t *>(c->data);
  v->len = s->len;
  v->table = s->block_table;
  v->batch = s->batch;
  v->max_pages = s->max_pages;
  v->table_stride = s->table_stride;
  v->page_shift = 0;
  while ((1 << v->page_shift) < c->page_tokens) ++v->page_shift;
  v->num_pages = c->num_pages;
  v->h_kv = c->h_kv;
  v->wait_ns = tq::wait_limit_ns();
  v->withhold = tq::handoffs_withheld();
  return tq::device_error_word(&v->errors) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

tq_status check_heads(int h_q, int h_kv) {
  if (h_kv < 1 || h_q < h_kv || h_q % h_kv) return TQ_ERR_INVALID_ARGUMENT;
  return h_q / h_kv > TQ_PAGED_MAX_GQA ? TQ_ERR_UNSUPPORTED : TQ_OK;
}

tq_status done(cudaError_t e) { return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA; }

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace

extern "C" {

tq_status tq_make_rope_table(int max_positions, int rotary_dim, double theta, float *table) {
  if (!table || max_positions < 1 || !(theta > 0.0) || !std::isfinite(theta)) return TQ_ERR_INVALID_ARGUMENT;
  if (rotary_dim < 16 || rotary_dim > 256 || rotary_dim % 16) return TQ_ERR_UNSUPPORTED;
  const int half = rotary_dim / 2;
  double inv[128];
  for (int j = 0; j < half; ++j) inv[j] = std::pow(theta, -2.0 * j / rotary_dim);
  for (int p = 0; p < max_positions; ++p) {
    float *row = table + (size_t)p * rotary_dim;
    for (int j = 0; j < half; ++j) {
      row[j] = (float)std::cos(p * inv[j]);
      row[half + j] = (float)std::sin(p * inv[j]);
    }
  }
  return TQ_OK;
}

size_t tq_paged_bytes(int d, int h_kv, int page_tokens, int num_pages) {
  if (!head_dim_ok(d) || h_kv < 1 || num_pages < 1) return 0;
  if (page_tokens < 16 || page_tokens > 1024 || (page_tokens & (page_tokens - 1))) return 0;
  size_t bytes;
  return pool_bytes(d, h_kv, page_tokens, num_pages, &bytes) ? bytes : 0;
}

tq_status tq_paged_append(const tq_paged_cache *c, const tq_paged_batch *s, const tq_rope *rope, const int32_t *cu_new,
                          const void *q, const void *k, const void *v, tq_dtype dtype, int h_q, int T, long long q_stride,
                          long long k_stride, long long v_stride, void *q_out, void *k_out, long long q_out_stride,
                          long long k_out_stride, tq_stream_t stream) {
  tq_status st = check_cache(c);
  if (st != TQ_OK) return st;
  if ((st = check_batch(c, s)) != TQ_OK) return st;
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_UNSUPPORTED;
  if (rope) {
    if (rope->rotary_dim < 16 || rope->rotary_dim > c->d || rope->rotary_dim % 16) return TQ_ERR_UNSUPPORTED;
    if (!rope->table || !aligned(rope->table, 16) || rope->max_positions < 1) return TQ_ERR_INVALID_ARGUMENT;
  }
  if (T < 0 || !cu_new || !aligned(cu_new, 4)) return TQ_ERR_INVALID_ARGUMENT;
  if (T == 0) return TQ_OK;
  const long long row = (long long)c->h_kv * c->d;
  if (!rows_ok(k, k_stride, row, dtype) || !rows_ok(v, v_stride, row, dtype)) return TQ_ERR_INVALID_ARGUMENT;
  if (k_out && !rows_ok(k_out, k_out_stride, row, dtype)) return TQ_ERR_INVALID_ARGUMENT;
  if (k_out == k && k_out_stride != k_stride) return TQ_ERR_INVALID_ARGUMENT;
  if (q) {
    if ((st = check_heads(h_q, c->h_kv)) != TQ_OK) return st;
    const long long qrow = (long long)h_q * c->d;
    if (!rows_ok(q, q_stride, qrow, dtype) || !rows_ok(q_out, q_out_stride, qrow, dtype)) return TQ_ERR_INVALID_ARGUMENT;
    if (q_out == q && q_out_stride != q_stride) return TQ_ERR_INVALID_ARGUMENT;
  }
  if (T > (1 << 30) || tq::span_units<4>(T, s->batch) * c->h_kv > 0x7fffffffll) return TQ_ERR_CAPACITY;
  tq::PagedAppendArgs a;
  if ((st = view(c, s, &a.c)) != TQ_OK) return st;
  a.rope = rope ? rope->table : nullptr;
  a.rotary_dim = rope ? rope->rotary_dim : 0;
  a.max_positions = rope ? rope->max_positions : 0;
  a.interleaved = rope ? rope->interleaved : 0;
  a.cu = cu_new;
  a.q = q; a.k = k; a.v = v; a.q_out = q_out; a.k_out = k_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.q_out_stride = q_out_stride; a.k_out_stride = k_out_stride;
  a.h_q = q ? h_q : 0; a.T = T;
  return done(tq::launch_paged_append(a, c->d, dtype, (cudaStream_t)stream));
}

tq_status tq_paged_gather(const tq_paged_cache *c, const tq_paged_batch *s, const int32_t *cu_rows, const int32_t *first,
                          int rows, void *k_out, void *v_out, tq_dtype dtype, long long k_stride, long long v_stride,
                          tq_stream_t stream) {
  tq_status st = check_cache(c);
  if (st != TQ_OK) return st;
  if ((st = check_batch(c, s)) != TQ_OK) return st;
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_UNSUPPORTED;
  if (rows < 0 || !cu_rows || !aligned(cu_rows, 4) || !aligned(first, 4)) return TQ_ERR_INVALID_ARGUMENT;
  if (rows == 0) return TQ_OK;
  const long long row = (long long)c->h_kv * c->d;
  if (!rows_ok(k_out, k_stride, row, dtype) || !rows_ok(v_out, v_stride, row, dtype)) return TQ_ERR_INVALID_ARGUMENT;
  if (rows > (1 << 30) || tq::span_units<4>(rows, s->batch) * c->h_kv > 0x7fffffffll) return TQ_ERR_CAPACITY;
  tq::PagedGatherArgs a;
  if ((st = view(c, s, &a.c)) != TQ_OK) return st;
  a.cu = cu_rows; a.first = first;
  a.k_out = k_out; a.v_out = v_out; a.k_stride = k_stride; a.v_stride = v_stride;
  a.rows = rows;
  return done(tq::launch_paged_gather(a, c->d, dtype, (cudaStream_t)stream));
}

size_t tq_paged_decode_workspace_size(const tq_paged_cache *c, int batch, int h_q) {
  if (check_cache(c) != TQ_OK || batch < 1 || check_heads(h_q, c->h_kv) != TQ_OK) return 0;
  int sms = 0;
  if (tq::device_sm_count(&sms) != cudaSuccess) return 0;
  return tq::paged_decode_workspace(c->d, c->h_kv, h_q, batch, sms);
}

tq_status tq_paged_decode_attention(const tq_paged_cache *c, const tq_paged_batch *s, const void *q, tq_dtype dtype, int h_q,
                                    long long q_stride, float softmax_scale, void *out, long long out_stride,
                                    void *workspace, size_t workspace_bytes, tq_stream_t stream) {
  tq_status st = check_cache(c);
  if (st != TQ_OK) return st;
  if ((st = check_batch(c, s)) != TQ_OK) return st;
  if (dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_UNSUPPORTED;
  if ((st = check_heads(h_q, c->h_kv)) != TQ_OK) return st;
  if (!std::isfinite(softmax_scale * kLog2e)) return TQ_ERR_INVALID_ARGUMENT;
  const long long row = (long long)h_q * c->d;
  if (!rows_ok(q, q_stride, row, dtype) || !rows_ok(out, out_stride, row, dtype)) return TQ_ERR_INVALID_ARGUMENT;
  if ((long long)s->batch * h_q > 0x7fffffffll) return TQ_ERR_CAPACITY;
  if (!workspace || !aligned(workspace, 256)) return TQ_ERR_WORKSPACE;
  tq::PagedDecodeArgs a;
  if (tq::device_sm_count(&a.num_sms) != cudaSuccess) return TQ_ERR_CUDA;
  if (workspace_bytes < tq::paged_decode_workspace(c->d, c->h_kv, h_q, s->batch, a.num_sms)) return TQ_ERR_WORKSPACE;
  if ((st = view(c, s, &a.c)) != TQ_OK) return st;
  a.c.withhold = a.c.withhold == 1;  // (decided here: the test of it in the kernel's loop cost 2%)
  a.q = q; a.out = out; a.q_stride = q_stride; a.out_stride = out_stride;
  a.h_q = h_q; a.scale_log2 = softmax_scale * kLog2e;
  a.partials = static_cast<float *>(workspace);
  return done(tq::launch_paged_decode(a, c->d, dtype, (cudaStream_t)stream));
}

tq_status tq_prompt_attention(const void *q, const void *k, const void *v, tq_dtype dtype, int T_q, int T_k, int h_q,
                              int h_kv, int d, long long q_stride, long long k_stride, long long v_stride,
                              const int32_t *cu_q, const int32_t *cu_k, int batch, float softmax_scale, void *out,
                              long long out_stride, tq_stream_t stream) {
  if (!head_dim_ok(d)) return TQ_ERR_UNSUPPORTED;
  if (dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_UNSUPPORTED;
  tq_status st = check_heads(h_q, h_kv);
  if (st != TQ_OK) return st;
  if (T_q < 0 || T_k < 0 || batch < 1 || !cu_q || !cu_k || !aligned(cu_q, 4) || !aligned(cu_k, 4))
    return TQ_ERR_INVALID_ARGUMENT;
  if (batch > (1 << 20) || T_q > (1 << 30) || T_k > (1 << 30)) return TQ_ERR_CAPACITY;
  if (!std::isfinite(softmax_scale * kLog2e)) return TQ_ERR_INVALID_ARGUMENT;
  if (T_q == 0) return TQ_OK;
  const long long qrow = (long long)h_q * d, row = (long long)h_kv * d;
  if (!rows_ok(q, q_stride, qrow, dtype) || !rows_ok(out, out_stride, qrow, dtype)) return TQ_ERR_INVALID_ARGUMENT;
  if (T_k > 0 && (!rows_ok(k, k_stride, row, dtype) || !rows_ok(v, v_stride, row, dtype))) return TQ_ERR_INVALID_ARGUMENT;
  tq::PromptArgs a;
  a.q = q; a.k = k; a.v = v; a.out = out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.out_stride = out_stride;
  a.cu_q = cu_q; a.cu_k = cu_k;
  a.T_q = T_q; a.T_k = T_k; a.h_q = h_q; a.h_kv = h_kv; a.batch = batch;
  // a scale of 0 becomes one that leaves every weight at 1 (masked scores
  // are infinite, and 0 times infinity is NaN)
  a.scale_log2 = std::fmax(std::fabs(softmax_scale) * kLog2e, 1e-30f);
  a.negate = softmax_scale < 0.f;
  a.wait_ns = tq::wait_limit_ns();
  a.withhold = tq::handoffs_withheld();
  if (tq::device_error_word(&a.errors) != cudaSuccess) return TQ_ERR_CUDA;
  return done(tq::launch_prompt(a, d, dtype, (cudaStream_t)stream));
}

}  // extern "C"
