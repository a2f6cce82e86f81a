// rope_kv.hip -- rotation of queries and keys by their positions, with the keys and values appended
// to the paged cache on the way, for gfx950.
//
// Pair i of a head's row turns by the angle p f_i:  (a, b) -> (a c - b s, a s + b c), c = m cos(p f_i),
// s = m sin(p f_i).  The angle is formed in binary64: p f_i is off by at most 2^-53 of itself, so in
// turns (p f_i / 2 pi) by less than 2^-23 for f_i <= 1 and every 31-bit position; the whole turns drop out exactly,
// and the rest, at most half a turn, goes through the binary32 sine and cosine.  In binary32 a position
// of 10^5 would already be off by 2^-8 radians.
//
// Bound by memory (each row is read once and written once or twice); a pair's sine and cosine cost some
// hundred operations, so they are formed once per token for all heads and kept in LDS.  Measured, 32/8 heads of
// 128: 16384 tokens 90 us (436 MB, 4.8 TB/s; a large copy 5.1 TB/s), 64 tokens 4.4 us, a launch and a chain of two loads.
// Where the rows or the turning runs are not aligned to 16 bytes, everything goes element by element: 16384 tokens
// of odd strides 179 us, of dimension 80 with 40 turned 140 us (all 80 turned, aligned: 64 us).
#include "attention.h"
#include "device_common.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kPairs = 256;        // pairs of a workgroup's tokens (a rotary dimension has at most 512)
constexpr int kMaxTokens = 8;      // tokens of a workgroup
constexpr int kDeep = 4;           // items of a thread in flight

// A thread's unit of E pairs: E = 8 (16-byte accesses) or 1.  `first` and `second` are the raw
// elements of the unit in memory order: split pairs (2 E elements in two runs), neighbours (one run).
template <int E>
struct Raw {
  uint16_t v[2 * E];
};

template <int E>
__device__ __forceinline__ void get(const uint16_t* p, uint16_t* v) {
  if constexpr (E == 8) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
    __builtin_memcpy(v, &w, 16);
  } else {
    v[0] = p[0];
  }
}
template <int E>
__device__ __forceinline__ void put(uint16_t* p, const uint16_t* v) {
  if constexpr (E == 8) {
    u32x4 w;
    __builtin_memcpy(&w, v, 16);
    *reinterpret_cast<u32x4*>(p) = w;
  } else {
    p[0] = v[0];
  }
}

// An item is one unit of one row: of a query or key row a unit of 2 E elements that turn together
// (R / 2E of them) or that stay ((D - R) / 2E, the last one may be half), of a value row 2 E elements.
struct Item {
  const uint16_t* from;   // null: nothing to do
  uint16_t* to;           // null: not wanted
  uint16_t* cache;        // null: no slot, or a query
  int lo, hi;             // the unit's two runs of E elements; hi < 0: one run only
  int pair;               // its first pair's place in LDS, or -1: copied
};

template <int DT, int E, bool PAIRED>
__global__ void __launch_bounds__(kThreads) rope_kv_kernel(RopeKvArgs a) {
  __shared__ float2 turn[kPairs];
  __shared__ int64_t place_row[kMaxTokens];   // row of the token's slot for head 0, or -1
  __shared__ int position[kMaxTokens];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_each;
  const int here = (int)(a.tokens - t0 < a.tokens_each ? a.tokens - t0 : a.tokens_each);
  const int half = a.rotary_dim / 2;
  // this workgroup's share of the rows of its tokens
  const int items = here * a.items_token;
  const int i0 = (int)((int64_t)items * blockIdx.y / gridDim.y), i1 = (int)((int64_t)items * (blockIdx.y + 1) / gridDim.y);

  if (tid < here) {
    const int64_t t = t0 + tid, slot = a.slot_map[t];
    position[tid] = a.positions[t];
    int64_t row = -1;
    if (slot >= 0 && slot < a.num_pages * a.page_size) {
      const int64_t page = quotient(slot, a.page_size);
      row = page * a.kv_heads * a.page_size + (slot - page * a.page_size);
    }
    place_row[tid] = row;
  }
  for (int i = tid; i < here * half; i += kThreads) {
    const int t = divide(i, a.half_magic, a.half_shift), p = i - t * half;
    const int at = a.positions[t0 + t];
    const double turns = (double)at * (double)a.inv_freq[p] * 0.15915494309189535;   // 1 / 2 pi
    const float rest = (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.0f * rest, &s, &c);
    turn[i] = make_float2(c * a.mscale, s * a.mscale);
  }
  __syncthreads();

  constexpr int kUnit = 2 * E;
  auto item_of = [&](int i) __attribute__((always_inline)) {
    Item m;
    m.from = nullptr;
    m.to = m.cache = nullptr;
    m.lo = m.hi = 0;
    m.pair = -1;
    if (i >= i1) return m;
    const int t = divide(i, a.token_magic, a.token_shift);
    int r = i - t * a.items_token;
    if (position[t] < 0) return m;
    const int head = divide(r, a.row_magic, a.row_shift), u = r - head * a.items_row;   // rows: q heads, k heads, v heads
    const int64_t token = t0 + t;
    const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.kv_heads;
    const int h = is_q ? head : is_v ? head - a.q_heads - a.kv_heads : head - a.q_heads;
    const int64_t row = place_row[t];
    if (is_q) {
      m.from = (const uint16_t*)a.q + token * a.q_stride + h * a.q_head_stride;
      m.to = (uint16_t*)a.q_out + token * a.qo_stride + h * a.qo_head_stride;
    } else if (!is_v) {
      m.from = (const uint16_t*)a.k + token * a.k_stride + h * a.k_head_stride;
      if (a.k_out) m.to = (uint16_t*)a.k_out + token * a.ko_stride + h * a.ko_head_stride;
    } else {
      m.from = (const uint16_t*)a.v + token * a.v_stride + h * a.v_head_stride;
    }
    if (!is_q && row >= 0)
      m.cache = (uint16_t*)(is_v ? a.v_cache : a.k_cache) + (row + (int64_t)h * a.page_size) * a.head_dim;
    if (!m.to && !m.cache) {
      m.from = nullptr;
      return m;
    }
    // the unit's place: turning units first, then what stays
    const int turning = is_v ? 0 : half / E;
    if (u < turning) {
      m.lo = PAIRED ? kUnit * u : E * u;
      m.hi = PAIRED ? m.lo + E : m.lo + half;
      m.pair = t * half + E * u;
    } else {
      m.lo = (is_v ? 0 : a.rotary_dim) + kUnit * (u - turning);
      m.hi = m.lo + E < a.head_dim ? m.lo + E : -1;
    }
    return m;
  };

  for (int i = i0 + tid; i < i1; i += kThreads * kDeep) {
    Item m[kDeep];
    Raw<E> x[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      m[d] = item_of(i + d * kThreads);
      if (m[d].from) {
        get<E>(m[d].from + m[d].lo, x[d].v);
        if (m[d].hi >= 0) get<E>(m[d].from + m[d].hi, x[d].v + E);
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (!m[d].from) continue;
      if (m[d].pair >= 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int ia = PAIRED ? 2 * e : e, ib = PAIRED ? 2 * e + 1 : e + E;
          const float2 cs = turn[m[d].pair + e];
          const float p = unpack1<DT>(x[d].v[ia]), q = unpack1<DT>(x[d].v[ib]);
          x[d].v[ia] = round16<DT>(__builtin_fmaf(p, cs.x, -(q * cs.y)));
          x[d].v[ib] = round16<DT>(__builtin_fmaf(p, cs.y, q * cs.x));
        }
      }
      if (m[d].to) {
        put<E>(m[d].to + m[d].lo, x[d].v);
        if (m[d].hi >= 0) put<E>(m[d].to + m[d].hi, x[d].v + E);
      }
      if (m[d].cache) {
        put<E>(m[d].cache + m[d].lo, x[d].v);
        if (m[d].hi >= 0) put<E>(m[d].cache + m[d].hi, x[d].v + E);
      }
    }
  }
}

template <int DT, int E>
void launch(const RopeKvArgs& a, dim3 grid, hipStream_t s) {
  if (a.interleaved) rope_kv_kernel<DT, E, true><<<grid, dim3(kThreads), 0, s>>>(a);
  else rope_kv_kernel<DT, E, false><<<grid, dim3(kThreads), 0, s>>>(a);
}

}  // namespace

hipError_t launch_rope_kv(const RopeKvArgs& args, hipStream_t s) {
  RopeKvArgs a = args;
  const int half = a.rotary_dim / 2;
  // 16-byte accesses where the runs of a unit and all rows allow them
  const uintptr_t ptrs = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q_out | (uintptr_t)a.k_out |
                         (uintptr_t)a.k_cache | (uintptr_t)a.v_cache;
  const int64_t steps = a.q_stride | a.q_head_stride | a.k_stride | a.k_head_stride | a.v_stride | a.v_head_stride |
                        a.qo_stride | a.qo_head_stride | a.ko_stride | a.ko_head_stride;
  const bool wide = ptrs % 16 == 0 && steps % 8 == 0 && a.head_dim % 8 == 0 && half % 8 == 0;
  const int E = wide ? 8 : 1;
  // rows have the same number of items: a value row has no more than a query row
  a.items_row = half / E + (a.head_dim - a.rotary_dim + 2 * E - 1) / (2 * E);
  a.items_token = a.items_row * (a.q_heads + 2 * a.kv_heads);
  // several tokens to a workgroup where there are many, so that a workgroup's angles fill its threads
  int each = kPairs / half;
  if (each > kMaxTokens) each = kMaxTokens;
  while (each > 1 && (a.tokens + each - 1) / each < 1024) each /= 2;
  if (each < 1) each = 1;
  a.tokens_each = each;
  const int64_t blocks = (a.tokens + each - 1) / each;
  // few tokens: their rows go to several workgroups, each with the angles
  int split = 1;
  while (blocks * split < 256 && a.items_token * each / split > kThreads) split *= 2;
  division_magic(half, a.half_magic, a.half_shift);
  division_magic(a.items_token, a.token_magic, a.token_shift);
  division_magic(a.items_row, a.row_magic, a.row_shift);
  const dim3 grid((unsigned)blocks, (unsigned)split);
  if (a.dtype == kBf16) {
    if (wide) launch<kBf16, 8>(a, grid, s);
    else launch<kBf16, 1>(a, grid, s);
  } else {
    if (wide) launch<kFp16, 8>(a, grid, s);
    else launch<kFp16, 1>(a, grid, s);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
