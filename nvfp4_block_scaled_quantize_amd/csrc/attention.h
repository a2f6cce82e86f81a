// attention.h -- launcher interfaces of the serving attention operators.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

// ---------------------------------------------------------------- division by a run-time number
// floor(j / d) = (j * magic) >> (32 + shift) for 0 <= j < 2^31, 2 <= d < 2^31: magic =
// ceil(2^(32+shift) / d), shift = ceil(log2 d) - 1 (division_magic); d = 1 has magic 0.
__device__ __forceinline__ int divide(int j, uint32_t magic, int shift) {
  return magic ? (int)(__umulhi((uint32_t)j, magic) >> shift) : j;
}
inline void division_magic(int d, uint32_t& magic, int& shift) {
  magic = 0;
  shift = 0;
  if (d <= 1) return;
  int up = 0;
  while ((1ll << up) < d) ++up;
  shift = up - 1;
  magic = (uint32_t)(((1ull << (32 + shift)) + d - 1) / d);
}

// floor(a / b) for 0 <= a < 2^52, 0 < b < 2^52: the binary64 quotient is within one of it.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  const int64_t q = (int64_t)((double)a / (double)b), r = a - q * b;
  return r < 0 ? q - 1 : r >= b ? q + 1 : q;
}

// Bytes from a page's first row to the row at `place`: a page has up to 2^30 places of up to 256 bytes.
__host__ __device__ __forceinline__ int64_t place_bytes(int place, int row_bytes) { return (int64_t)place * row_bytes; }

struct PageMapsArgs {
  const int32_t* ctx_lens;
  const int32_t* new_lens;
  int32_t* block_table;        // [seqs, max_pages], extended in place
  const int32_t* free_pages;   // [num_free]
  int seqs, max_pages, num_free, page_size;
  int64_t tokens;              // entries of slot_map and positions
  int32_t* cu_new;             // [seqs + 1]
  int32_t* kv_lens;            // [seqs], may be ctx_lens
  int64_t* slot_map;
  int32_t* positions;
  int32_t* taken;              // [1]
  uint32_t magic;              // division by page_size, set by the launcher
  int shift;
};
hipError_t launch_page_maps(const PageMapsArgs& a, hipStream_t s);

struct KvWriteArgs {
  const void* k;
  const void* v;
  int64_t tokens;
  int kv_heads, head_dim;
  int64_t k_stride, k_head_stride, v_stride, v_head_stride;   // elements
  const int64_t* slot_map;
  void* k_cache;
  void* v_cache;
  int page_size;
  int64_t num_pages;
};
hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t s);

struct AttnArgs {
  const void* q;               // [tokens, q_heads, head_dim] by strides
  const void* k;               // prompt: [tokens, kv_heads, head_dim] by strides; paged: the cache
  const void* v;
  int dtype;
  const int32_t* cu;           // [seqs + 1] first token of each request
  const int32_t* kv_lens;      // paged: [seqs]
  const int32_t* block_table;  // paged: [seqs, max_pages]
  int seqs, tokens, q_heads, kv_heads, head_dim;
  int page_size, max_pages;
  int64_t num_pages;
  int64_t q_stride, q_head_stride, k_stride, k_head_stride, v_stride, v_head_stride;   // elements
  float scale;
  int window;                  // 0: no window
  void* out;                   // [tokens, q_heads, head_dim]
  float* lse;                  // [tokens, q_heads] or null
  void* workspace;             // paged
  // set by the launchers: q_heads / kv_heads, and its division (see divide)
  int group, group_shift;
  uint32_t group_magic;
};
bool prompt_attn_fits(const AttnArgs& a);   // the grid
hipError_t launch_prompt_attn(const AttnArgs& a, hipStream_t s);
size_t paged_attn_workspace_bytes(int64_t seqs, int64_t tokens, int q_heads, int kv_heads, int head_dim);
hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s);

}  // namespace nvfp4
