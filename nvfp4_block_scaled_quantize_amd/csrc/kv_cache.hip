// kv_cache.hip -- the paged key/value cache's bookkeeping and its writer, for
// gfx950.
//
// A cache is two arrays [num_pages, kv_heads, page_size, head_dim] (keys,
// values); a request's position p lies in page block_table[request][p /
// page_size] at place p % page_size, and slot = page * page_size + place
// numbers the places of all pages.
#include "attention.h"
#include "internal.h"
#include "device_common.h"

namespace nvfp4 {

namespace {

// ---------------------------------------------------------------- maps
// One launch.  Request i holds held_i = ceil(ctx_i / P) pages and needs
// need_i = ceil((ctx_i + new_i) / P) - held_i more (both capped at the table's
// width); its pages are free_pages[first_i ..] with first_i = sum_{j<i} need_j,
// its tokens cu_i = sum_{j<i} new_j onwards.  A new page's first place always
// belongs to a new token, so the token at that place writes the table entry
// and every output is written by exactly one thread.
//
// Both sums are needed by every workgroup, and a launch (or a grid-wide wait)
// costs more than forming them again: each workgroup sums all the requests
// (contiguous shares per thread, one scan over the threads), keeps the starts
// that fall into its own range of tokens in LDS, and finds each token's
// request by a running maximum over those starts.
constexpr int kMapThreads = 256;
constexpr int kMapTokens = 2048;                       // tokens per workgroup
constexpr int kMapPer = kMapTokens / kMapThreads;

constexpr int kMost = 0x7FFFFFFF;

__device__ __forceinline__ int len_of(const int32_t* p, int i) { return p[i] > 0 ? p[i] : 0; }
__device__ __forceinline__ int clamp64(int64_t v) { return v < kMost ? (int)v : kMost; }

// Pages of n tokens: ceil(n / page_size), at most the table's width.
__device__ __forceinline__ int pages_of(const PageMapsArgs& a, int n) {
  const int p = n > 0 ? divide(n - 1, a.magic, a.shift) + 1 : 0;
  return p < a.max_pages ? p : a.max_pages;
}

// Exclusive prefix of v over the threads of the workgroup; total in `all`.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s, int64_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 63) s[wave] = x;
  __syncthreads();
  int64_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kMapThreads / 64; ++w) {
    if (w < wave) before += s[w];
    all += s[w];
  }
  return before + x - v;
}

__global__ void __launch_bounds__(kMapThreads) page_maps_kernel(PageMapsArgs a) {
  __shared__ int64_t scan[kMapThreads / 64];
  __shared__ int start_req[kMapTokens];        // request that starts at this token of the range, or -1
  __shared__ int start_cu[kMapTokens];         // its first token
  __shared__ int64_t start_page[kMapTokens];   // its first page in the free list
  __shared__ int wave_last[kMapThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kMapTokens;
  const int width = a.max_pages;
  for (int k = tid; k < kMapTokens; k += kMapThreads) start_req[k] = -1;

  const int per = (a.seqs + kMapThreads - 1) / kMapThreads;
  const int i0 = tid * per, i1 = (i0 + per < a.seqs) ? i0 + per : a.seqs;
  int64_t tok = 0, pag = 0;
  for (int i = i0; i < i1; ++i) {
    const int c = len_of(a.ctx_lens, i), m = len_of(a.new_lens, i);
    tok += m;
    pag += pages_of(a, clamp64((int64_t)c + m)) - pages_of(a, c);
  }
  int64_t all_tok, all_pag;
  int64_t at = block_scan(tok, scan, all_tok);
  int64_t page = block_scan(pag, scan, all_pag);   // its first barrier orders the fill of start_req
  const bool mine = (tid % gridDim.x) == blockIdx.x;   // writes this share's cu_new and kv_lens
  for (int i = i0; i < i1; ++i) {
    const int c = len_of(a.ctx_lens, i), m = len_of(a.new_lens, i), all = clamp64((int64_t)c + m);
    if (m > 0 && at < t0 + kMapTokens && at + m > t0) {
      const int k = (int)(at > t0 ? at - t0 : 0);
      start_req[k] = i;
      start_cu[k] = (int)at;
      start_page[k] = page;
    }
    if (mine) {
      a.cu_new[i] = clamp64(at);
      a.kv_lens[i] = all;
    }
    at += m;
    page += pages_of(a, all) - pages_of(a, c);
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_new[a.seqs] = clamp64(all_tok);
    a.taken[0] = clamp64(all_pag);
  }
  __syncthreads();

  // last start at or before each token: thread tid looks at kMapPer tokens,
  // then a scan of maxima over the threads
  int last[kMapPer];
  int run = -1;
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) {
    const int idx = tid * kMapPer + k;
    if (start_req[idx] >= 0) run = idx;
    last[k] = run;
  }
  int inc = run;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(inc, off, 64);
    if (lane >= off && y > inc) inc = y;
  }
  if (lane == 63) wave_last[wave] = inc;
  __syncthreads();
  int before = __shfl_up(inc, 1, 64);
  if (lane == 0) before = -1;
  for (int w = 0; w < wave; ++w) before = wave_last[w] > before ? wave_last[w] : before;
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) {
    const int64_t t = t0 + tid * kMapPer + k;
    if (t >= a.tokens) break;
    const int st = last[k] > before ? last[k] : before;
    int64_t slot = -1;
    int32_t position = -1;
    if (st >= 0 && t < all_tok) {
      const int i = start_req[st];
      const int c = len_of(a.ctx_lens, i);
      position = clamp64(c + (t - start_cu[st]));
      const int col = divide(position, a.magic, a.shift), place = position - col * a.page_size;
      const int held = pages_of(a, c);
      int pg = -1;
      if (col < held) {
        pg = a.block_table[(int64_t)i * width + col];
      } else if (col < width) {
        const int64_t f = start_page[st] + (col - held);
        if (f < a.num_free) pg = a.free_pages[f];
        if (place == 0) a.block_table[(int64_t)i * width + col] = pg;
      }
      if (pg >= 0) slot = (int64_t)pg * a.page_size + place;
    }
    a.slot_map[t] = slot;
    a.positions[t] = position;
  }
}

// ---------------------------------------------------------------- writer
// A copy: token t's row of each head goes to its slot.  One thread moves U
// bytes; a token's rows are consecutive units, so the reads of a wave are
// whole cache lines and every (page, head) place is one contiguous row.
template <typename U>
__global__ void __launch_bounds__(256) kv_write_kernel(KvWriteArgs a, int units_row, int64_t total) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += step) {
    const int64_t row = quotient(u, units_row);           // (token, head)
    const int64_t t = quotient(row, a.kv_heads);
    const int h = (int)(row - t * a.kv_heads), c = (int)(u - row * units_row);
    const int64_t slot = a.slot_map[t];
    if (slot < 0 || slot >= a.num_pages * a.page_size) continue;
    const int64_t page = quotient(slot, a.page_size), place = slot - page * a.page_size;
    const int64_t to = ((page * a.kv_heads + h) * a.page_size + place) * units_row + c;
    const char* k = (const char*)a.k + (t * a.k_stride + (int64_t)h * a.k_head_stride) * 2;
    const char* v = (const char*)a.v + (t * a.v_stride + (int64_t)h * a.v_head_stride) * 2;
    const U x = ((const U*)k)[c], y = ((const U*)v)[c];
    ((U*)a.k_cache)[to] = x;
    ((U*)a.v_cache)[to] = y;
  }
}

}  // namespace

hipError_t launch_page_maps(const PageMapsArgs& a, hipStream_t s) {
  const int64_t blocks = (a.tokens + kMapTokens - 1) / kMapTokens;
  PageMapsArgs c = a;
  division_magic(c.page_size, c.magic, c.shift);
  page_maps_kernel<<<dim3((unsigned)(blocks > 0 ? blocks : 1)), dim3(kMapThreads), 0, s>>>(c);
  return hipGetLastError();
}

hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t s) {
  const bool wide = a.head_dim % 8 == 0 && a.k_stride % 8 == 0 && a.v_stride % 8 == 0 &&
                    a.k_head_stride % 8 == 0 && a.v_head_stride % 8 == 0 &&
                    (((uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache) % 16) == 0;
  const int units_row = wide ? a.head_dim / 8 : a.head_dim;
  const int64_t total = a.tokens * a.kv_heads * units_row;
  int64_t blocks = (total + 255) / 256;
  if (blocks > 65536) blocks = 65536;
  if (wide) kv_write_kernel<u32x4><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(a, units_row, total);
  else kv_write_kernel<uint16_t><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(a, units_row, total);
  return hipGetLastError();
}

}  // namespace nvfp4
