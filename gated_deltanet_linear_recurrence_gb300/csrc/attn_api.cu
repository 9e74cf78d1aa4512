// attn_api.cu — the C ABI of the paged cache and of prompt attention: argument
// validation and launches.  Declarations and contracts: include/gdn.h.
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

}  // namespace

extern "C" {

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
