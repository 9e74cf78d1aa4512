// attn_params.h — launch arguments of the attention layers' operators (the
// paged key-value cache, decode attention over it, prompt attention), passed
// from the C ABI layer to the kernels.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

// Device error code added by the paged cache (value of gdn_status).
enum PagedDeviceError : int { kErrBadPage = 11 };

enum CacheDtype : int { kCacheBF16 = 1, kCacheE4M3 = 2 };

// The paged cache.  Pages [num_pages][h_kv][page_size][D] of bf16 or e4m3 rows;
// with e4m3 an exponent byte (bias 127) per row, [num_pages][h_kv][page_size].
// Position p of sequence n is slot p % page_size of page table[n][p / page_size].
struct PagedCache {
  void* k_pages;
  void* v_pages;
  uint8_t* k_exp;
  uint8_t* v_exp;
  const int32_t* table;  // [num_seqs][max_pages]
  int32_t h_kv, head_dim;
  int32_t page_shift;  // page_size = 1 << page_shift
  int32_t num_pages, max_pages;
  int dtype;  // CacheDtype
};

// Rows of packed tokens [T][h_kv][D] bf16 (token strides in elements) written
// into the cache at positions start[n] .., or read back from there.
struct KvRowsArgs {
  void* k;
  void* v;
  int64_t k_stride, v_stride;
  PagedCache cache;
  const int32_t* cu_seqlens;  // [num_seqs + 1]
  const int32_t* start;       // [num_seqs]
  int32_t num_seqs;
  int64_t total_tokens;
  int* err;
};

// Norms and rotation of the heads of q and k: dense outputs, or k with v into the cache
// (rows.k, rows.v and their strides are the inputs there).
constexpr int kMaxRotated = 256;  // rotary_dim
struct RopeArgs {
  const void* q;  // [T][h_q][D] bf16; strides in elements between tokens
  int64_t q_stride;
  void* q_out;
  int64_t q_out_stride;
  void* k_out;  // dense outputs only
  int64_t k_out_stride;
  int32_t h_q, h_kv, head_dim;
  const int32_t* positions;  // [axes][T]; nullptr: the positions in the cache
  const float* inv_freq;     // [rotary / 2]
  int32_t rotary, axes;
  const float* q_weight;  // [D] or nullptr (ones)
  const float* k_weight;
  float eps;
  bool norm, pairs;
  int32_t groups;  // of a token's rows, taken by a warp: chosen at the launch
  KvRowsArgs rows;
  uint8_t axis_of[kMaxRotated / 2];  // axis of each frequency's positions
};

// One query of each sequence over its cache_len[b] cached rows.
struct PagedAttnArgs {
  const void* q;  // [B][h_q][D] bf16, q_stride elements between sequences
  int64_t q_stride;
  PagedCache cache;
  const int32_t* cache_len;  // [B]
  void* o;                   // [B][h_q][D] bf16, dense
  float* partial;            // [ctas][2][G][D + 2]
  int32_t batch, h_q;
  int32_t ctas;  // CTAs that share the batch's key tiles
  float scale;
  int* err;
};

// Packed causal prompt attention: the a queries of a sequence are the last a of
// its b positions.
struct AttnPrefillArgs {
  const void* q;  // [Tq][h_q][D] bf16
  const void* k;  // [Tk][h_kv][D]
  const void* v;
  void* o;  // [Tq][h_q][D], dense
  const int32_t* cu_q;
  const int32_t* cu_k;
  int32_t num_seqs;
  int64_t total_q, total_k;
  int32_t h_q, h_kv, head_dim;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  int32_t by_sequence;  // order of the tiles, chosen at the launch
  int* err;
};

// Attention of packed new tokens over the paged cache: the a queries of a sequence are the
// last a of its cache_len[n] cached positions.
struct PagedPrefillArgs {
  const void* q;  // [Tq][h_q][D] bf16
  int64_t q_stride;
  PagedCache cache;
  const int32_t* cu_q;
  const int32_t* cache_len;
  void* o;         // [Tq][h_q][D], dense
  float* partial;  // [pairs][2][256][D + 2], and what the joining pass has to know
  int32_t num_seqs;
  int64_t total_q;
  int32_t h_q;
  int32_t window, sinks;  // keys a query sees of the last (0: all), and of the first
  int32_t pairs;          // of CTAs that share the work
  int32_t group, tile;    // query heads a KV head, tokens of a pair (the launch fills these in)
  uint32_t tile_inv;      // floor((2^32 - 1) / tile) + 1
  float scale;
  // e4m3: room for rows that are widened once, [wide_rows][h_kv][D] bf16 of K and of V
  void* wide_k;
  void* wide_v;
  int64_t wide_rows;
  int* err;
};
constexpr int32_t kPagedPrefillMaxPairs = 80;  // bounds the workspace

constexpr int32_t kPagedMaxCtas = 640;  // bounds the workspace of the paged decode

size_t paged_attn_workspace_bytes(int32_t h_q, int32_t h_kv, int32_t head_dim);
cudaError_t launch_kv_append(const KvRowsArgs& a, cudaStream_t stream);
cudaError_t launch_kv_gather(const KvRowsArgs& a, cudaStream_t stream);
cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_kv_append_rope(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_attn_decode_paged(const PagedAttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_prefill(const AttnPrefillArgs& a, cudaStream_t stream);
size_t paged_prefill_workspace_bytes(int32_t head_dim);  // without room for widened rows
bool paged_prefill_widens(int64_t total_q, int32_t group, int dtype);
constexpr size_t kPagedPrefillWideBytes = (size_t)128 << 20;  // that room, as asked for
cudaError_t launch_attn_prefill_paged(const PagedPrefillArgs& a, cudaStream_t stream);

// The current device's error word (gdn_api.cu); false when it cannot be located.
bool device_error_word(int** out);

}  // namespace gdn
