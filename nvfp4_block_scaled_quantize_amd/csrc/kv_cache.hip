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
// request by a running maximum over those starts.  Sums are 32 bits and stop at
// 2^31 - 1 (min(a + b, 2^31 - 1) is associative), so lengths that break the
// contract cannot index anything.
//
// Bound by the chain of dependent steps (lengths, scan, starts, table, store),
// not by bytes: 256 requests of one token 3.2 us, 333 requests of 266k tokens
// 6.5 us (3.4 MB).  With 64-bit sums and a scan each for tokens and pages 7.1
// and 11.4 us.
constexpr int kMapThreads = 256;
constexpr int kMapPer = 4;
constexpr int kMapTokens = kMapThreads * kMapPer;      // tokens per workgroup
constexpr uint32_t kMost = 0x7FFFFFFFu;

__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return a + b < kMost ? a + b : kMost; }
__device__ __forceinline__ uint32_t len_of(const int32_t* p, int i) { return p[i] > 0 ? (uint32_t)p[i] : 0u; }

// Pages of n tokens: ceil(n / page_size), at most the table's width.
__device__ __forceinline__ uint32_t pages_of(const PageMapsArgs& a, uint32_t n) {
  const int p = n > 0 ? divide((int)(n - 1), a.magic, a.shift) + 1 : 0;
  return (uint32_t)(p < a.max_pages ? p : a.max_pages);
}

__global__ void __launch_bounds__(kMapThreads) page_maps_kernel(PageMapsArgs a) {
  constexpr int kWaves = kMapThreads / 64;
  __shared__ uint32_t sums[2][kWaves];
  __shared__ int owner[kMapTokens];            // a request starts at this token (its place in the range), or -1
  __shared__ int4 starts[kMapTokens];          // request, its cached length, first token, first free page
  __shared__ int wave_last[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kMapTokens;
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) owner[k * kMapThreads + tid] = -1;

  const int per = (a.seqs + kMapThreads - 1) / kMapThreads;
  const int i0 = tid * per, i1 = (i0 + per < a.seqs) ? i0 + per : a.seqs;
  uint32_t tok = 0, pag = 0, c0 = 0, m0 = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t c = len_of(a.ctx_lens, i), m = len_of(a.new_lens, i);
    if (i == i0) { c0 = c; m0 = m; }
    tok = add(tok, m);
    pag = add(pag, pages_of(a, add(c, m)) - pages_of(a, c));
  }
  uint32_t x = tok, y = pag;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t u = __shfl_up(x, off, 64), v = __shfl_up(y, off, 64);
    if (lane >= off) {
      x = add(x, u);
      y = add(y, v);
    }
  }
  if (lane == 63) {
    sums[0][wave] = x;
    sums[1][wave] = y;
  }
  // exclusive: the inclusive value of the lane before
  uint32_t at = __shfl_up(x, 1, 64), page = __shfl_up(y, 1, 64);
  if (lane == 0) at = page = 0;
  __syncthreads();   // also orders the fill of owner
  uint32_t all_tok = 0, all_pag = 0, tb = 0, pb = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w == wave) { tb = all_tok; pb = all_pag; }
    all_tok = add(all_tok, sums[0][w]);
    all_pag = add(all_pag, sums[1][w]);
  }
  at = add(at, tb);
  page = add(page, pb);
  const bool mine = (tid % gridDim.x) == blockIdx.x;   // writes this share's cu_new and kv_lens
  for (int i = i0; i < i1; ++i) {
    const uint32_t c = i == i0 ? c0 : len_of(a.ctx_lens, i), m = i == i0 ? m0 : len_of(a.new_lens, i);
    const uint32_t all = add(c, m);
    if (m > 0 && at < t0 + kMapTokens && (int64_t)at + m > t0) {
      const int k = at > t0 ? (int)(at - t0) : 0;
      owner[k] = k;
      starts[k] = make_int4(i, (int)c, (int)at, (int)page);
    }
    if (mine) {
      a.cu_new[i] = (int32_t)at;
      if (a.kv_lens) a.kv_lens[i] = (int32_t)all;
    }
    at = add(at, m);
    page = add(page, pages_of(a, all) - pages_of(a, c));
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_new[a.seqs] = (int32_t)all_tok;
    a.taken[0] = (int32_t)all_pag;
  }
  __syncthreads();

  // last start at or before each token: kMapPer consecutive tokens per thread,
  // then a scan of maxima over the threads
  int last[kMapPer], run = -1;
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) {
    const int o = owner[tid * kMapPer + k];
    run = o >= 0 ? o : run;
    last[k] = run;
  }
  int inc = run;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int u = __shfl_up(inc, off, 64);
    if (lane >= off && u > inc) inc = u;
  }
  if (lane == 63) wave_last[wave] = inc;
  int before = __shfl_up(inc, 1, 64);
  if (lane == 0) before = -1;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w)
    if (w < wave && wave_last[w] > before) before = wave_last[w];
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) owner[tid * kMapPer + k] = last[k] > before ? last[k] : before;
  __syncthreads();
  // from here on neighbouring threads have neighbouring tokens
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) {
    const int idx = k * kMapThreads + tid;
    const int64_t t = t0 + idx;
    const int st = owner[idx];
    int64_t slot = -1;
    int32_t position = -1;
    if (st >= 0 && t < (int64_t)all_tok && t < a.tokens) {
      const int4 s = starts[st];
      position = (int32_t)add((uint32_t)s.y, (uint32_t)(t - s.z));
      const int col = divide(position, a.magic, a.shift), place = position - col * a.page_size;
      const int held = (int)pages_of(a, (uint32_t)s.y);
      int pg = -1;
      if (col < held) {
        pg = a.block_table[(int64_t)s.x * a.max_pages + col];
      } else if (col < a.max_pages) {
        const int64_t f = (int64_t)s.w + (col - held);
        if (f < a.num_free) pg = a.free_pages[f];
        if (place == 0) a.block_table[(int64_t)s.x * a.max_pages + col] = pg;
      }
      if (pg >= 0) slot = (int64_t)pg * a.page_size + place;
    }
    if (t < a.tokens) {
      a.slot_map[t] = slot;
      a.positions[t] = position;
    }
  }
}

// kv_lens alone, where they replace ctx_lens.
__global__ void __launch_bounds__(kMapThreads) grow_kernel(int32_t* lens, const int32_t* new_lens, int seqs) {
  const int i = blockIdx.x * kMapThreads + threadIdx.x;
  if (i < seqs) lens[i] = (int32_t)add(len_of(lens, i), len_of(new_lens, i));
}

// ---------------------------------------------------------------- writer
// A copy: token t's row of each head goes to its slot.  One thread moves U
// bytes; a token's rows are consecutive units, so the reads of a wave are
// whole cache lines and every (page, head) place is one contiguous row.  Bound
// by memory: 16384 tokens of 8 heads of 128 (133.5 MB read and written) take
// 21.4 us, 6.2 TB/s, where the rows partly come from the last cache (28 us from
// memory); 256 tokens 3.0 us, a launch.  Units of 16 bytes where everything is
// aligned to them, else of 2.
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
  // Lengths updated in place: one workgroup reads and writes each of them in the same thread, but of
  // several each reads all of them, so they are written after the last has read.
  const bool later = a.kv_lens == a.ctx_lens && blocks > 1;
  if (later) c.kv_lens = nullptr;
  page_maps_kernel<<<dim3((unsigned)(blocks > 0 ? blocks : 1)), dim3(kMapThreads), 0, s>>>(c);
  if (later && a.seqs > 0)
    grow_kernel<<<dim3((unsigned)((a.seqs + kMapThreads - 1) / kMapThreads)), dim3(kMapThreads), 0, s>>>(
        a.kv_lens, a.new_lens, a.seqs);
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
