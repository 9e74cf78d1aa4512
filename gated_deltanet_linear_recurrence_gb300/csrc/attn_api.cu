// attn_api.cu — the C ABI of the attention layers' operators (norms and rotation, the
// paged cache, attention of prompts and over the cache): argument validation and launches.  Declarations and contracts: include/gdn.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_params.h"
#include "gdn.h"

namespace {

constexpr int32_t kMaxGroup = 8;  // query heads per KV head

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool head_dim_ok(int32_t d) { return d == 128 || d == 256; }

gdn_status check_heads(int32_t h_q, int32_t h_kv, int32_t head_dim) {
  if (h_q <= 0 || h_kv <= 0 || head_dim <= 0) return GDN_ERR_INVALID_ARG;
  if (!head_dim_ok(head_dim) || h_q % h_kv != 0 || h_q / h_kv > kMaxGroup || h_kv > 65535)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}

// Distance between tokens, in elements: whole 16-byte steps, at least one token.
gdn_status check_stride(int64_t stride, int64_t row) {
  if (stride < row) return GDN_ERR_INVALID_ARG;
  return stride % 8 != 0 ? GDN_ERR_MISALIGNED : GDN_OK;
}

gdn_status check_cache(int32_t num_seqs, int32_t h_kv, int32_t head_dim, int32_t page_size,
                       int32_t num_pages, int32_t max_pages, int dtype) {
  if (num_seqs < 0 || num_pages < 0 || max_pages < 0 || page_size <= 0) return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_CACHE_BF16 && dtype != GDN_CACHE_E4M3) return GDN_ERR_UNSUPPORTED_DTYPE;
  const gdn_status st = check_heads(h_kv, h_kv, head_dim);
  if (st != GDN_OK) return st;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)max_pages * page_size > INT32_MAX - 2047 ||
      (int64_t)num_pages * h_kv * page_size >= (int64_t)UINT32_MAX)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}

gdn::PagedCache make_cache(const void* k_pages, const void* v_pages, const uint8_t* k_exp,
                           const uint8_t* v_exp, const int32_t* table, int32_t h_kv,
                           int32_t head_dim, int32_t page_size, int32_t num_pages,
                           int32_t max_pages, int dtype) {
  gdn::PagedCache c{};
  c.k_pages = const_cast<void*>(k_pages);
  c.v_pages = const_cast<void*>(v_pages);
  c.k_exp = const_cast<uint8_t*>(k_exp);
  c.v_exp = const_cast<uint8_t*>(v_exp);
  c.table = table;
  c.h_kv = h_kv;
  c.head_dim = head_dim;
  while ((1 << c.page_shift) < page_size) ++c.page_shift;
  c.num_pages = num_pages;
  c.max_pages = max_pages;
  c.dtype = dtype;
  return c;
}

// The pointers: the table wherever it has entries (a position's page is looked up before
// it is compared with the pool's size), the pages where the pool has some too.
gdn_status check_pages(const gdn::PagedCache& c) {
  const bool any = c.num_pages > 0 && c.max_pages > 0;
  if (c.max_pages > 0 && !c.table) return GDN_ERR_NULL_POINTER;
  if (any && (!c.k_pages || !c.v_pages)) return GDN_ERR_NULL_POINTER;
  if (any && c.dtype == GDN_CACHE_E4M3 && (!c.k_exp || !c.v_exp)) return GDN_ERR_NULL_POINTER;
  if (!aligned(c.k_pages, 16) || !aligned(c.v_pages, 16) || !aligned(c.table, 4))
    return GDN_ERR_MISALIGNED;
  if (c.dtype == GDN_CACHE_E4M3 && (!aligned(c.k_exp, 8) || !aligned(c.v_exp, 8)))
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

gdn_status rows_call(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                     const gdn::PagedCache& cache, const int32_t* cu_seqlens,
                     const int32_t* start_pos, int32_t num_seqs, int64_t total_tokens,
                     bool append, gdn_stream_t stream) {
  const int64_t row = (int64_t)cache.h_kv * cache.head_dim;
  gdn_status st = check_stride(k_stride, row);
  if (st == GDN_OK) st = check_stride(v_stride, row);
  if (st != GDN_OK) return st;
  if (num_seqs == 0) return total_tokens == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens || !start_pos) return GDN_ERR_NULL_POINTER;
  if (total_tokens == 0) return GDN_OK;
  if (!k || !v) return GDN_ERR_NULL_POINTER;
  st = check_pages(cache);
  if (st != GDN_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_seqlens, 4) || !aligned(start_pos, 4))
    return GDN_ERR_MISALIGNED;
  gdn::KvRowsArgs a{};
  a.k = const_cast<void*>(k);
  a.v = const_cast<void*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cache = cache;
  a.cu_seqlens = cu_seqlens;
  a.start = start_pos;
  a.num_seqs = num_seqs;
  a.total_tokens = total_tokens;
  if (!gdn::device_error_word(&a.err)) return GDN_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = append ? gdn::launch_kv_append(a, s) : gdn::launch_kv_gather(a, s);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// Heads, rotation and norm of gdn_qk_norm_rope and gdn_kv_append_rope; what they share goes into a.
gdn_status check_rope(gdn::RopeArgs& a, int32_t h_q, int32_t h_kv, int32_t head_dim, int32_t rotary_dim,
                      const int32_t* positions, int32_t num_axes, const uint8_t* axis_of, const float* inv_freq,
                      const float* q_weight, const float* k_weight, float norm_eps, uint32_t options) {
  if (head_dim <= 0 || rotary_dim <= 0 || num_axes < 1) return GDN_ERR_INVALID_ARG;
  if (options & ~(uint32_t)(GDN_ROPE_RMSNORM | GDN_ROPE_INTERLEAVED)) return GDN_ERR_INVALID_ARG;
  if (!head_dim_ok(head_dim) || h_q > 65535 || h_kv > 65535 || num_axes > 4) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (rotary_dim > head_dim || rotary_dim % 8 != 0) return GDN_ERR_UNSUPPORTED_SHAPE;
  a.norm = (options & GDN_ROPE_RMSNORM) != 0;
  if (a.norm ? !(norm_eps >= 0.f) : q_weight != nullptr || k_weight != nullptr) return GDN_ERR_INVALID_ARG;
  if (num_axes > 1 && (!axis_of || !positions)) return GDN_ERR_NULL_POINTER;
  for (int i = 0; num_axes > 1 && i < rotary_dim / 2; ++i) {
    if (axis_of[i] >= num_axes) return GDN_ERR_INVALID_ARG;
    a.axis_of[i] = axis_of[i];
  }
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.head_dim = head_dim;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.rotary = rotary_dim;
  a.axes = num_axes;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = norm_eps;
  a.pairs = (options & GDN_ROPE_INTERLEAVED) != 0;
  return GDN_OK;
}

gdn_status check_rope_pointers(const gdn::RopeArgs& a) {
  if (!a.inv_freq) return GDN_ERR_NULL_POINTER;
  if (!aligned(a.q, 16) || !aligned(a.q_out, 16) || !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16) ||
      !aligned(a.positions, 4) || !aligned(a.inv_freq, 4))
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_qk_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, void* q_out,
                            void* k_out, int64_t q_out_stride, int64_t k_out_stride, const int32_t* positions,
                            int32_t num_axes, const uint8_t* axis_of, const float* inv_freq, int32_t rotary_dim,
                            const float* q_weight, const float* k_weight, float norm_eps, int64_t total_tokens,
                            int32_t h_q, int32_t h_kv, int32_t head_dim, gdn_dtype dtype, uint32_t options,
                            gdn_stream_t stream) {
  if (total_tokens < 0 || h_q <= 0 || h_kv <= 0) return GDN_ERR_INVALID_ARG;
  gdn::RopeArgs a{};
  gdn_status st = check_rope(a, h_q, h_kv, head_dim, rotary_dim, positions, num_axes, axis_of, inv_freq, q_weight,
                             k_weight, norm_eps, options);
  if (st == GDN_OK) st = check_stride(q_stride, (int64_t)h_q * head_dim);
  if (st == GDN_OK) st = check_stride(k_stride, (int64_t)h_kv * head_dim);
  if (st == GDN_OK) st = check_stride(q_out_stride, (int64_t)h_q * head_dim);
  if (st == GDN_OK) st = check_stride(k_out_stride, (int64_t)h_kv * head_dim);
  if (st != GDN_OK) return st;
  if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED_DTYPE;
  if (total_tokens > INT32_MAX) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (total_tokens == 0) return GDN_OK;
  if (!q || !k || !q_out || !k_out || !positions) return GDN_ERR_NULL_POINTER;
  a.q = q;
  a.q_stride = q_stride;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.k_out = k_out;
  a.k_out_stride = k_out_stride;
  a.rows.k = const_cast<void*>(k);
  a.rows.k_stride = k_stride;
  a.rows.total_tokens = total_tokens;
  st = check_rope_pointers(a);
  if (st != GDN_OK) return st;
  if (!aligned(k, 16) || !aligned(k_out, 16)) return GDN_ERR_MISALIGNED;
  return gdn::launch_qk_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv_append_rope(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                              int64_t v_stride, void* q_out, int64_t q_out_stride, void* k_pages, void* v_pages,
                              uint8_t* k_exp, uint8_t* v_exp, const int32_t* page_table, const int32_t* cu_seqlens,
                              const int32_t* start_pos, const int32_t* positions, int32_t num_axes,
                              const uint8_t* axis_of, const float* inv_freq, int32_t rotary_dim,
                              const float* q_weight, const float* k_weight, float norm_eps, int32_t num_seqs,
                              int64_t total_tokens, int32_t h_q, int32_t h_kv, int32_t head_dim, int32_t page_size,
                              int32_t num_pages, int32_t max_pages, gdn_cache_dtype cache_dtype, uint32_t options,
                              gdn_stream_t stream) {
  if (total_tokens < 0 || h_q < 0) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_cache(num_seqs, h_kv, head_dim, page_size, num_pages, max_pages, cache_dtype);
  if (st != GDN_OK) return st;
  gdn::RopeArgs a{};
  st = check_rope(a, h_q, h_kv, head_dim, rotary_dim, positions, num_axes, axis_of, inv_freq, q_weight, k_weight,
                  norm_eps, options);
  if (st == GDN_OK && h_q > 0) st = check_stride(q_stride, (int64_t)h_q * head_dim);
  if (st == GDN_OK && h_q > 0) st = check_stride(q_out_stride, (int64_t)h_q * head_dim);
  if (st == GDN_OK) st = check_stride(k_stride, (int64_t)h_kv * head_dim);
  if (st == GDN_OK) st = check_stride(v_stride, (int64_t)h_kv * head_dim);
  if (st != GDN_OK) return st;
  if (total_tokens > INT32_MAX) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (num_seqs == 0) return total_tokens == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens || !start_pos) return GDN_ERR_NULL_POINTER;
  if (total_tokens == 0) return GDN_OK;
  if (!k || !v || (h_q > 0 && (!q || !q_out))) return GDN_ERR_NULL_POINTER;
  a.q = h_q > 0 ? q : nullptr;
  a.q_stride = q_stride;
  a.q_out = h_q > 0 ? q_out : nullptr;
  a.q_out_stride = q_out_stride;
  a.rows.k = const_cast<void*>(k);
  a.rows.v = const_cast<void*>(v);
  a.rows.k_stride = k_stride;
  a.rows.v_stride = v_stride;
  a.rows.cache = make_cache(k_pages, v_pages, k_exp, v_exp, page_table, h_kv, head_dim, page_size, num_pages,
                            max_pages, cache_dtype);
  a.rows.cu_seqlens = cu_seqlens;
  a.rows.start = start_pos;
  a.rows.num_seqs = num_seqs;
  a.rows.total_tokens = total_tokens;
  st = check_pages(a.rows.cache);
  if (st == GDN_OK) st = check_rope_pointers(a);
  if (st != GDN_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_seqlens, 4) || !aligned(start_pos, 4))
    return GDN_ERR_MISALIGNED;
  if (!gdn::device_error_word(&a.rows.err)) return GDN_ERR_CUDA;
  return gdn::launch_kv_append_rope(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK
                                                                                             : GDN_ERR_CUDA;
}

gdn_status gdn_kv_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                         void* k_pages, void* v_pages, uint8_t* k_exp, uint8_t* v_exp,
                         const int32_t* page_table, const int32_t* cu_seqlens,
                         const int32_t* start_pos, int32_t num_seqs, int64_t total_tokens,
                         int32_t h_kv, int32_t head_dim, int32_t page_size, int32_t num_pages,
                         int32_t max_pages, gdn_cache_dtype cache_dtype, gdn_stream_t stream) {
  if (total_tokens < 0) return GDN_ERR_INVALID_ARG;
  const gdn_status st =
      check_cache(num_seqs, h_kv, head_dim, page_size, num_pages, max_pages, cache_dtype);
  if (st != GDN_OK) return st;
  if (total_tokens > INT32_MAX) return GDN_ERR_UNSUPPORTED_SHAPE;
  return rows_call(k, v, k_stride, v_stride,
                   make_cache(k_pages, v_pages, k_exp, v_exp, page_table, h_kv, head_dim,
                              page_size, num_pages, max_pages, cache_dtype),
                   cu_seqlens, start_pos, num_seqs, total_tokens, true, stream);
}

gdn_status gdn_kv_gather(void* k, void* v, int64_t k_stride, int64_t v_stride,
                         const void* k_pages, const void* v_pages, const uint8_t* k_exp,
                         const uint8_t* v_exp, const int32_t* page_table,
                         const int32_t* cu_seqlens, const int32_t* start_pos, int32_t num_seqs,
                         int64_t total_tokens, int32_t h_kv, int32_t head_dim, int32_t page_size,
                         int32_t num_pages, int32_t max_pages, gdn_cache_dtype cache_dtype,
                         gdn_stream_t stream) {
  if (total_tokens < 0) return GDN_ERR_INVALID_ARG;
  const gdn_status st =
      check_cache(num_seqs, h_kv, head_dim, page_size, num_pages, max_pages, cache_dtype);
  if (st != GDN_OK) return st;
  if (total_tokens > INT32_MAX) return GDN_ERR_UNSUPPORTED_SHAPE;
  return rows_call(k, v, k_stride, v_stride,
                   make_cache(k_pages, v_pages, k_exp, v_exp, page_table, h_kv, head_dim,
                              page_size, num_pages, max_pages, cache_dtype),
                   cu_seqlens, start_pos, num_seqs, total_tokens, false, stream);
}

size_t gdn_attn_decode_paged_workspace_size(int32_t h_q, int32_t h_kv, int32_t head_dim) {
  if (check_heads(h_q, h_kv, head_dim) != GDN_OK) return 0;
  return gdn::paged_attn_workspace_bytes(h_q, h_kv, head_dim);
}

gdn_status gdn_attn_decode_paged(const void* q, int64_t q_stride, const void* k_pages,
                                 const void* v_pages, const uint8_t* k_exp, const uint8_t* v_exp,
                                 const int32_t* page_table, const int32_t* cache_len, void* o,
                                 int32_t batch, int32_t h_q, int32_t h_kv, int32_t head_dim,
                                 int32_t page_size, int32_t num_pages, int32_t max_pages,
                                 gdn_cache_dtype cache_dtype, float scale, void* workspace,
                                 size_t workspace_bytes, gdn_stream_t stream) {
  gdn_status st = check_heads(h_q, h_kv, head_dim);
  if (st == GDN_OK)
    st = check_cache(batch, h_kv, head_dim, page_size, num_pages, max_pages, cache_dtype);
  if (st == GDN_OK) st = check_stride(q_stride, (int64_t)h_q * head_dim);
  if (st != GDN_OK) return st;
  if ((int64_t)batch * h_q > INT32_MAX) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (batch == 0) return GDN_OK;
  if (!q || !o || !cache_len || !workspace) return GDN_ERR_NULL_POINTER;
  const gdn::PagedCache cache = make_cache(k_pages, v_pages, k_exp, v_exp, page_table, h_kv,
                                           head_dim, page_size, num_pages, max_pages, cache_dtype);
  st = check_pages(cache);
  if (st != GDN_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(cache_len, 4))
    return GDN_ERR_MISALIGNED;
  if (workspace_bytes < gdn::paged_attn_workspace_bytes(h_q, h_kv, head_dim))
    return GDN_ERR_WORKSPACE_TOO_SMALL;
  gdn::PagedAttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.cache = cache;
  a.cache_len = cache_len;
  a.o = o;
  a.partial = static_cast<float*>(workspace);
  a.batch = batch;
  a.h_q = h_q;
  a.scale = scale;
  if (!gdn::device_error_word(&a.err)) return GDN_ERR_CUDA;
  return gdn::launch_attn_decode_paged(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

size_t gdn_attn_prefill_paged_workspace_size(int32_t h_q, int32_t h_kv, int32_t head_dim, gdn_cache_dtype cache_dtype,
                                             int64_t total_q) {
  if (check_heads(h_q, h_kv, head_dim) != GDN_OK || total_q < 0) return 0;
  if (cache_dtype != GDN_CACHE_BF16 && cache_dtype != GDN_CACHE_E4M3) return 0;
  return gdn::paged_prefill_workspace_bytes(head_dim) +
         (gdn::paged_prefill_widens(total_q, h_q / h_kv, cache_dtype) ? gdn::kPagedPrefillWideBytes : 0);
}

gdn_status gdn_attn_prefill_paged(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages,
                                  const uint8_t* k_exp, const uint8_t* v_exp, const int32_t* page_table,
                                  const int32_t* cu_seqlens_q, const int32_t* cache_len, void* o, int32_t num_seqs,
                                  int64_t total_q, int32_t h_q, int32_t h_kv, int32_t head_dim, int32_t page_size,
                                  int32_t num_pages, int32_t max_pages, gdn_cache_dtype cache_dtype, float scale,
                                  int32_t window, int32_t sinks, void* workspace, size_t workspace_bytes,
                                  gdn_stream_t stream) {
  if (total_q < 0 || window < 0 || sinks < 0) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_heads(h_q, h_kv, head_dim);
  if (st == GDN_OK)
    st = check_cache(num_seqs, h_kv, head_dim, page_size, num_pages, max_pages, cache_dtype);
  if (st == GDN_OK) st = check_stride(q_stride, (int64_t)h_q * head_dim);
  if (st != GDN_OK) return st;
  if (total_q > INT32_MAX) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (num_seqs == 0) return total_q == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens_q || !cache_len) return GDN_ERR_NULL_POINTER;
  if (total_q == 0) return GDN_OK;
  if (!q || !o || !workspace) return GDN_ERR_NULL_POINTER;
  const gdn::PagedCache cache = make_cache(k_pages, v_pages, k_exp, v_exp, page_table, h_kv, head_dim, page_size,
                                           num_pages, max_pages, cache_dtype);
  st = check_pages(cache);
  if (st != GDN_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(cu_seqlens_q, 4) ||
      !aligned(cache_len, 4))
    return GDN_ERR_MISALIGNED;
  const size_t least = gdn::paged_prefill_workspace_bytes(head_dim);
  if (workspace_bytes < least) return GDN_ERR_WORKSPACE_TOO_SMALL;
  gdn::PagedPrefillArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.cache = cache;
  a.cu_q = cu_seqlens_q;
  a.cache_len = cache_len;
  a.o = o;
  a.partial = static_cast<float*>(workspace);
  a.num_seqs = num_seqs;
  a.total_q = total_q;
  a.h_q = h_q;
  // a window that no position reaches past is none
  a.window = window < (int64_t)max_pages * page_size ? window : 0;
  a.sinks = a.window ? sinks : 0;
  a.scale = scale;
  if (gdn::paged_prefill_widens(total_q, h_q / h_kv, cache_dtype)) {  // whole rows of K and V that the rest holds
    const int64_t row = (int64_t)h_kv * head_dim * 2, rows = (int64_t)((workspace_bytes - least) / (2 * (size_t)row));
    a.wide_rows = rows < INT32_MAX - 2047 ? rows : INT32_MAX - 2047;
    a.wide_k = static_cast<uint8_t*>(workspace) + least;
    a.wide_v = static_cast<uint8_t*>(a.wide_k) + a.wide_rows * row;
  }
  if (!gdn::device_error_word(&a.err)) return GDN_ERR_CUDA;
  return gdn::launch_attn_prefill_paged(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK
                                                                                                 : GDN_ERR_CUDA;
}

gdn_status gdn_attn_prefill(const void* q, const void* k, const void* v, void* o,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                            int32_t num_seqs, int64_t total_q, int64_t total_k, int32_t h_q,
                            int32_t h_kv, int32_t head_dim, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, gdn_dtype dtype, float scale, gdn_stream_t stream) {
  if (num_seqs < 0 || total_q < 0 || total_k < 0) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_heads(h_q, h_kv, head_dim);
  if (st == GDN_OK) st = check_stride(q_stride, (int64_t)h_q * head_dim);
  if (st == GDN_OK) st = check_stride(k_stride, (int64_t)h_kv * head_dim);
  if (st == GDN_OK) st = check_stride(v_stride, (int64_t)h_kv * head_dim);
  if (st != GDN_OK) return st;
  if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED_DTYPE;
  if (total_q > INT32_MAX || total_k > INT32_MAX) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (num_seqs == 0) return total_q == 0 && total_k == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens_q || !cu_seqlens_k) return GDN_ERR_NULL_POINTER;
  if (total_q == 0) return GDN_OK;
  if (!q || !o || (total_k > 0 && (!k || !v))) return GDN_ERR_NULL_POINTER;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4))
    return GDN_ERR_MISALIGNED;
  gdn::AttnPrefillArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.num_seqs = num_seqs;
  a.total_q = total_q;
  a.total_k = total_k;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.head_dim = head_dim;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.scale = scale;
  if (!gdn::device_error_word(&a.err)) return GDN_ERR_CUDA;
  return gdn::launch_attn_prefill(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

}  // extern "C"
