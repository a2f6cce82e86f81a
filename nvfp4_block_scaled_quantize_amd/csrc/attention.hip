// attention.hip -- attention over whole packed prompts and attention of new
// tokens over a paged key/value cache, for gfx950.
//
// Row i of a request's m new tokens over L keys sits at position p = L - m + i
// and sees the keys j <= p, j > p - window (window > 0), j < L:
//   s_j = scale * q . k_j,   out = sum_j e^{s_j} v_j / sum_j e^{s_j},
//   lse = log sum_j e^{s_j};   a row that sees nothing: out = 0, lse = -inf.
//
// The query heads that share a key/value head are rows of one problem: row r
// of a request is (token r / G, query head h G + r % G), G = q_heads /
// kv_heads, so keys and values are read once for the group.
//
// One pass over the keys with a running maximum: with t_j = s_j log2 e,
//   m' = max(m, t), l = l 2^{m - m'} + sum 2^{t_j - m'}, O = O 2^{m - m'} + ...
// in binary32 throughout; only the weights 2^{t - m} are rounded to the
// inputs' type, because the matrix cores multiply them with the values (l sums
// the unrounded ones).  The maximum is kept while the new one exceeds it by less
// than 2^8, and the rescaling of O is skipped for most tiles.  m stands kShift
// above the maximum that it was set to, so that the weights end where their
// type has room (see kShift).
//
// t_j - m is one fma(s_j, scale log2 e, -m): what m's own rounding leaves is the
// same factor for all keys of a row and cancels in O / l, but it must not leave
// the exponent's range, and from |m| = 2^28 on half a unit in m's last place
// does.  A wave that met such a row (|m| >= kBig, scores of millions)
// computes its rows again, from a reference r, the largest raw score so far:
// scores become s_j - r as they come, m stays at kShift and the maximum never lags
// (see again).
//
// Matrix operands (v_mfma_f32_32x32x16, lane = 32 h + c): the score tile is
// formed transposed, S^T = K Q^T, so that a lane holds 16 of the 32 keys of
// ONE row c.  Row maxima and sums are then in-lane (plus one exchange between
// the half-waves), and the lane's weights, rounded and packed, are already
// the B operand of O^T += V^T P^T: the key order inside a product may be any
// as long as both operands share it, and V^T is read from the row-major tile
// by the transposing LDS read in just that order.  m, l and the rescaling are
// one value per lane.
#include "attention.h"
#include "internal.h"
#include "device_common.h"
#include "lds_dma.h"

#include <atomic>

namespace nvfp4 {

namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kKeep = 8.0f;   // the maximum may lag by this much (log2)
// bf16: no weight exceeds 1, so that values near the type's largest do not leave binary32 where the
// weighted mean does not.  fp16: weights reach 2^14 (of 65504), so that those of many keys far below the
// largest are not lost: the type rounds to 0 what is below 2^-25, here 2^-31 of the largest.
template <int DT>
constexpr float kShift = DT == kBf16 ? kKeep : -6.0f;
constexpr float kBig = 4194304.0f;   // 2^22: the steps of a maximum are still half a unit of log2

__device__ const uint4 kZeros[64] = {};   // rows that do not exist are copied from here

template <int DT>
__device__ __forceinline__ v16f mfma(v8s a, v8s b, v16f c) {
  if constexpr (DT == kBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Rounds to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (DT == kBf16) {
    typedef __bf16 v2b __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){x, y}, v2b));
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){x, y}, v2h));
  }
}

// Maximum and sum of a lane's value and that of the same lane of the other half-wave.
__device__ __forceinline__ float both_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Wave-uniform values, kept in scalar registers.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uni64(int64_t v) {
  return (int64_t)(((uint64_t)(uint32_t)uni((int)(v >> 32)) << 32) | (uint32_t)uni((int)v));
}

__device__ __forceinline__ int token_of(const AttnArgs& a, int row) { return divide(row, a.group_magic, a.group_shift); }

// ---------------------------------------------------------------- LDS tiles
// A tile is rows of DP elements; 16-byte chunk p of row r holds chunk p ^
// swz(r) of the row.  LDS serves 256 bytes (all 64 banks) a cycle: 16 lanes of
// a b128 read, here 16 consecutive rows at one chunk, or 32 lanes of a
// transposing read, 64 bytes of each of four consecutive rows.  Rows of 256
// bytes start at the same bank, so swz puts the low row bits above the bits
// that tell the chunks of 64 bytes apart and is different for 16 rows; rows of
// 128 bytes differ in half the banks by themselves.
template <int DP>
__device__ __forceinline__ int swz(int r) {
  return DP == 64 ? ((r & 2) << 1) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
}

template <int DP>
__device__ __forceinline__ int chunk_at(int row, int chunk) {
  return row * (DP * 2) + ((chunk ^ swz<DP>(row)) * 16);
}

// Row `row` of V^T: four keys row..row+3 for the 16 values of d in
// 16 dblk .. 16 dblk + 15, one d per lane of a 16-lane group.
template <int DP>
__device__ __forceinline__ uint32_t tr_at(int row, int dblk, int i) {
  const int r = row + (i >> 2), chunk = dblk * 2 + ((i & 3) >> 1);
  return (uint32_t)(chunk_at<DP>(r, chunk) + (i & 1) * 8);
}

typedef __attribute__((address_space(3))) v4s* lds_v4s;
__device__ __forceinline__ v4s read_tr(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(uintptr_t)at);
}
__device__ __forceinline__ v8s read_b128(uint32_t at) {
  return *(__attribute__((address_space(3))) v8s*)(uintptr_t)at;
}

__device__ __forceinline__ void zero_lds(uint32_t at) {
  *(__attribute__((address_space(3))) u32x4*)(uintptr_t)at = (u32x4){0, 0, 0, 0};
}

// ---------------------------------------------------------------- sources
// Where the keys and values of one (request, key/value head) are.
struct Source {
  const char* k;         // prompt: first row; paged: the cache at this head
  const char* v;
  int64_t k_step, v_step;   // prompt: bytes from key to key; paged: bytes from page to page (k_step)
  const int32_t* table;  // paged: the request's row of the block table
  int page_size;
  uint32_t magic;        // paged: key / page_size as a multiply-high (see divide)
  int shift;
  int64_t num_pages;
  int keys;              // keys that exist
  int d_bytes;           // bytes of a row
};

__device__ __forceinline__ int page_of(const Source& s, int j) { return divide(j, s.magic, s.shift); }

template <bool PAGED>
__device__ __forceinline__ void row_at(const Source& s, int j, int page, int chunk_bytes, const char*& k, const char*& v) {
  const char* zero = reinterpret_cast<const char*>(kZeros);
  bool there = j < s.keys && chunk_bytes < s.d_bytes;
  if constexpr (PAGED) {
    there = there && (uint32_t)page < (uint64_t)s.num_pages;
    const int64_t off = (int64_t)page * s.k_step + place_bytes(j - page_of(s, j) * s.page_size, s.d_bytes) + chunk_bytes;
    k = there ? s.k + off : zero;
    v = there ? s.v + off : zero;
  } else {
    k = there ? s.k + (int64_t)j * s.k_step + chunk_bytes : zero;
    v = there ? s.v + (int64_t)j * s.v_step + chunk_bytes : zero;
  }
}

// ---------------------------------------------------------------- one tile
// State of the 32 rows of a wave.
template <int DP>
struct Rows {
  v8s q[DP / 16];      // B operand: lane's row, d = 16 st + 8 h ..
  v16f o[DP / 32];     // O^T: d = 32 t + 8 (i / 4) + 4 h + i % 4
  float m, l;          // log2 units; l: this half-wave's keys only
  float far;           // the score (before scaling) that m is raised at; of a big row its reference
  int lo, hi;          // the row sees the keys lo <= j < hi
  uint64_t late;       // lanes whose row needs a reference
  uint64_t big;        // lanes whose row counts from one
};

// A row starts at the lowest number instead of -inf: differences of maxima are
// then never inf - inf, and every weight of a row that has seen nothing is
// 2^(-inf) = 0.
constexpr float kLowest = -3.40282346638528859812e+38f;

struct Scaling {
  float c, inv;   // scale log2 e and its inverse, in scalar registers
  __device__ __forceinline__ explicit Scaling(float scale)
      : c(__uint_as_float(uni(__float_as_uint(scale * kLog2e)))), inv(__uint_as_float(uni(__float_as_uint(1.0f / c)))) {}
};

template <int DT>
__device__ __forceinline__ uint32_t not_finite_bits() { return DT == kBf16 ? 0x7F80u : 0x7C00u; }

// A lane's operand addresses relative to a tile (which starts at a multiple of
// 256): chunk 2 st + h of K row `col` is at k ^ 32 st, and V^T's keys 4 h ..
// for d = 32 t .. are at v ^ 64 t -- the swizzle and the chunk number are
// joined by exclusive or.
template <int DP>
struct Lanes {
  uint32_t k, v;
  __device__ __forceinline__ explicit Lanes(int lane) {
    k = (uint32_t)chunk_at<DP>(lane & 31, lane >> 5);
    v = tr_at<DP>(4 * (lane >> 5), (lane >> 4) & 1, lane & 15);
  }
  static constexpr uint32_t kDown = 32;   // what 8 rows further down change in the swizzle
};

// K operand of score product n: 16 d of 32 keys; products of KT key groups alternate.
template <int DP, int KT>
__device__ __forceinline__ v8s key_operand(const Lanes<DP>& ln, uint32_t k_lds, int n) {
  return read_b128(((k_lds + ln.k) ^ (n / KT * 32)) + n % KT * 32 * DP * 2);
}

// V^T operand of value product n: d tile n % (DP / 32), 16 keys n / (DP / 32).
// Element e: key 4 h + e (e < 4), 8 + 4 h + e - 4 -- the order of the weights.
template <int DP>
__device__ __forceinline__ v8s value_operand(const Lanes<DP>& ln, uint32_t v_lds, int n) {
  constexpr uint32_t kRow = DP * 2;
  const uint32_t at = (v_lds + ln.v) ^ (n % (DP / 32) * 64), down = n / (DP / 32) * 16 * kRow;
  const v4s x = read_tr(at + down), y = read_tr((at ^ Lanes<DP>::kDown) + down + 8 * kRow);
  return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ v16f zero16() {
  v16f z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}

// S^T = K Q^T for KT x 32 keys.
template <int DT, int DP, int KT>
__device__ __forceinline__ void scores(v16f (&s)[KT], const Rows<DP>& w, const Lanes<DP>& ln, uint32_t k_lds) {
#pragma unroll
  for (int n = 0; n < KT * DP / 16; ++n)
    s[n % KT] = mfma<DT>(key_operand<DP, KT>(ln, k_lds, n), w.q[n / KT], n < KT ? zero16() : s[n % KT]);
}

__device__ __forceinline__ float largest(const v16f& s) {
  float top = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, s[i]);
  return top;
}

// A rare step on the accumulators is written as a loop of at most one turn, with a count that the
// compiler does not know: they are then updated where they are, while a branch gets a second set of
// registers for them and copies between the two in the common path.
__device__ __forceinline__ int turns_if(int positive) {
  int n = uni(positive < 1 ? positive : 1);
  asm volatile("" : "+s"(n));
  return n;
}

// A row's reference.
template <int DP>
__device__ __forceinline__ float reference(const Rows<DP>& w) {
  return __builtin_amdgcn_inverse_ballot_w64(w.big) ? w.far : 0.0f;
}

// log2 of how far the maximum (m, ref) lies above (m2, ref2): the references are scores, and their
// difference is exact where it matters.
__device__ __forceinline__ float above(float m, float ref, float m2, float ref2, float c) {
  return __builtin_fmaf(ref - ref2, c, m) - m2;
}

template <int DP>
__device__ __forceinline__ void rescale(Rows<DP>& w, float a) {
  w.l *= a;
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) w.o[t][i] *= a;
}

__device__ __forceinline__ int turns_any(uint64_t lanes) {   // see turns_if
  int turns;
  asm volatile("s_cmp_lg_u64 %1, 0\n\ts_cselect_b32 %0, 1, 0" : "=s"(turns) : "s"(lanes) : "scc");
  return turns;
}

// Raises the maximum to `top` (a score, of both half-waves) where it lags by more than kKeep, and notes
// the rows that this is not enough for.
template <int DT, int DP>
__device__ __forceinline__ void raise(Rows<DP>& w, float top, const Scaling& sc) {
#pragma unroll 1
  for (int turns = turns_any(__ballot(top > w.far)); turns > 0; --turns) {
    const float t = __builtin_fmaf(top, sc.c, kShift<DT>), m = __builtin_fmaxf(w.m, t), a = __builtin_amdgcn_exp2f(w.m - m);
    w.late |= __ballot(t > w.m && __builtin_fabsf(t) >= kBig);
    w.m = m;
    w.far = (m + (kKeep - kShift<DT>)) * sc.inv;
    rescale(w, a);
  }
}

// The same with references, which are taken off the scores `s`.
template <int DT, int DP>
__device__ __forceinline__ void raise(Rows<DP>& w, float top, const Scaling& sc, v16f& s) {
#pragma unroll 1
  for (int turns = turns_any(__ballot(top > w.far) | w.big); turns > 0; --turns) {
    const float old = reference(w), t = __builtin_fmaf(top, sc.c, kShift<DT>);
    const bool was = __builtin_amdgcn_inverse_ballot_w64(w.big), is = was || (t > w.m && __builtin_fabsf(t) >= kBig);
    const float ref = was ? __builtin_fmaxf(old, top) : is ? top : 0.0f;
    const float m = is ? kShift<DT> : __builtin_fmaxf(w.m, t);
    const float a = __builtin_amdgcn_exp2f(above(w.m, old, m, ref, sc.c));
    w.m = m;
    w.far = is ? ref : (m + (kKeep - kShift<DT>)) * sc.inv;
    w.big = __ballot(is);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] -= ref;
    rescale(w, a);
  }
}

// Whether the values of 32 rows are all finite.
template <int DT, int DP>
__device__ __forceinline__ bool all_finite(uint32_t v_lds, int lane) {
  asm volatile("" : "+v"(lane));
  typedef unsigned short v2u __attribute__((ext_vector_type(2)));
  v2u most = {0, 0};
#pragma unroll 4
  for (int n = 0; n < 32 * DP * 2 / 1024; ++n) {
    const u32x4 x = __builtin_bit_cast(u32x4, read_b128(v_lds + n * 1024 + lane * 16));
#pragma unroll
    for (int e = 0; e < 4; ++e) most = __builtin_elementwise_max(most, __builtin_bit_cast(v2u, x[e] & 0x7FFF7FFFu));
  }
  const uint32_t big = most[0] > most[1] ? most[0] : most[1];
  return !__any(big >= not_finite_bits<DT>());
}

// Where some row does not see some key of a tile and a value there is not finite, 0 * inf in the
// matrix cores would carry it to rows that do not see it.  The products of such a tile are formed with
// 0 in place of those values, and they are added one by one to the rows that see them.  Rare: short
// rather than fast.
template <int DT>
__device__ __forceinline__ v8s finite_only(v8s v) {
  u32x4 x = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((x[e] & 0x7FFFu) >= not_finite_bits<DT>()) x[e] &= 0xFFFF0000u;
    if (((x[e] >> 16) & 0x7FFFu) >= not_finite_bits<DT>()) x[e] &= 0xFFFFu;
  }
  return __builtin_bit_cast(v8s, x);
}

template <int DT, int DP>
__device__ __forceinline__ void add_not_finite(Rows<DP>& w, const v16f& s, float c, int kb, uint32_t v_lds, int lane) {
  asm volatile("" : "+v"(lane));
  const int h = lane >> 5;
  typedef __attribute__((address_space(3))) u32x2* lds_2;
#pragma unroll 1
  for (int key = 0; key < 32; ++key) {
    // the row's score of this key: register 4 (key / 8) + key % 4 of half-wave key / 4 % 2
    float x = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) x = i == key / 8 * 4 + key % 4 ? s[i] : x;
    const float mine = __builtin_amdgcn_exp2f(__builtin_fmaf(x, c, -w.m));
    const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(mine), __float_as_uint(mine), false, false);
    const float p = __uint_as_float((key & 4) ? both[1] : both[0]);
    const bool sees = kb + key >= w.lo && kb + key < w.hi;
#pragma unroll
    for (int t = 0; t < DP / 32; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x2 y2 = *(lds_2)(uintptr_t)(v_lds + chunk_at<DP>(key, t * 4 + i) + 8 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t y = (y2[e / 2] >> (16 * (e % 2))) & 0xFFFFu;
          const bool add = sees && (y & 0x7FFFu) >= not_finite_bits<DT>();
          w.o[t][4 * i + e] += add ? p * unpack1<DT>((uint16_t)y) : 0.0f;
        }
      }
  }
}

// Adds 32 keys from key kb, whose scores are `s` and whose values are at v_lds.  `hidden` > 0: some
// row does not see some of them.  REF: rows may have references.
template <int DT, int DP, bool REF = false>
__device__ __forceinline__ void add_keys(Rows<DP>& w, const Lanes<DP>& ln, v16f& s, uint32_t v_lds, int kb,
                                         const Scaling& sc, int hidden, int lane) {
  constexpr int kTiles = DP / 32;
  int odd = 0;   // some value is not finite
#pragma unroll 1
  for (int turns = turns_if(hidden); turns > 0; --turns) {
    const int lo = w.lo - kb - 4 * (lane >> 5);
    const uint32_t count = w.hi > w.lo ? w.hi - w.lo : 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = (uint32_t)(8 * (i / 4) + i % 4 - lo) < count ? s[i] : -__builtin_inff();
    odd = uni(all_finite<DT, DP>(v_lds, lane) ? 0 : 1);
  }
  if constexpr (REF) raise<DT>(w, both_max(largest(s)), sc, s);
  else raise<DT>(w, both_max(largest(s)), sc);
  v8s p[2];
  float sum[2] = {w.l, 0.0f};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = half * 8 + e * 2;
      const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], sc.c, -w.m));
      const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + 1], sc.c, -w.m));
      sum[0] += x;
      sum[1] += y;
      d[e] = pack2<DT>(x, y);
    }
    p[half] = __builtin_bit_cast(v8s, (u32x4){d[0], d[1], d[2], d[3]});
  }
  w.l = sum[0] + sum[1];
#pragma unroll 1
  for (int turns = turns_if(1 - odd); turns > 0; --turns) {
    asm volatile("" : "+s"(v_lds));   // the reads belong into the loop
#pragma unroll
    for (int n = 0; n < 2 * kTiles; ++n)
      w.o[n % kTiles] = mfma<DT>(value_operand(ln, v_lds, n), p[n / kTiles], w.o[n % kTiles]);
  }
#pragma unroll 1
  for (int turns = turns_if(odd); turns > 0; --turns) {
    asm volatile("" : "+s"(v_lds));
#pragma unroll
    for (int n = 0; n < 2 * kTiles; ++n)
      w.o[n % kTiles] = mfma<DT>(finite_only<DT>(value_operand(ln, v_lds, n)), p[n / kTiles], w.o[n % kTiles]);
    add_not_finite<DT, DP>(w, s, sc.c, kb, v_lds, lane);
  }
}

// Adds 64 keys that every row sees, whose scores are `cur` with the largest `top`, and forms the next
// 64 keys' scores `nxt` and `top`, in an order that keeps the matrix cores fed: the weights of the
// current keys beside the score products of the next, then the value products.  Operands are read
// from LDS kAhead products ahead (`f`: on entry the first K operands, on return those of the step
// after, whose rows are at k_after), and each matrix instruction is followed by the share of the
// vector work that fits beside it; the scheduling barriers keep that order.
//
// Two waves share a SIMD, and each issues an instruction every 4 cycles at best: a step has to stay
// well under its matrix time of 1024 cycles (DP = 128) in instructions.  With 32 keys a step the
// votes, the branches and the addresses cost as much as the weights do.
constexpr int kAhead = 4, kGroups = 2;

template <int DT, int DP>
__device__ __forceinline__ void add_tile(Rows<DP>& w, const Lanes<DP>& ln, const v16f (&cur)[kGroups],
                                         v16f (&nxt)[kGroups], float& top, v8s (&f)[kAhead], uint32_t k_next,
                                         uint32_t k_after, uint32_t v_lds, const Scaling& sc) {
  constexpr int kTiles = DP / 32, kScores = kGroups * DP / 16, kValues = kGroups * 2 * kTiles;
  constexpr int kPer = 16 * kGroups / kScores;              // weights per score product
  constexpr int kShare = 16 * kGroups / (kValues - 2) + 1;  // maxima per value product
  static_assert(kScores % kAhead == 0 && kValues % kAhead == 0 && kPer % 2 == 0, "operand ring");
  raise<DT>(w, top, sc);
  uint32_t d[kGroups * 8];
  float sum[2] = {w.l, 0.0f};
  __builtin_amdgcn_sched_barrier(0);
  // the wave at its score products, which have vector work beside them, goes before one at its value
  // products (1 % of a long prompt; the other way round is slower)
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int n = 0; n < kScores; ++n) {
    nxt[n % kGroups] = mfma<DT>(f[n % kAhead], w.q[n / kGroups], n < kGroups ? zero16() : nxt[n % kGroups]);
    f[n % kAhead] = n + kAhead < kScores ? key_operand<DP, kGroups>(ln, k_next, n + kAhead)
                                         : value_operand(ln, v_lds, n + kAhead - kScores);
#pragma unroll
    for (int i = n * kPer; i < (n + 1) * kPer; i += 2) {
      const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(cur[i / 16][i % 16], sc.c, -w.m));
      const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(cur[i / 16][i % 16 + 1], sc.c, -w.m));
      sum[0] += x;
      sum[1] += y;
      d[i / 2] = pack2<DT>(x, y);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  w.l = sum[0] + sum[1];
  __builtin_amdgcn_s_setprio(0);
  float best = 0.0f;
#pragma unroll
  for (int n = 0; n < kValues; ++n) {
    const int k = n / kTiles * 4;
    const v8s p = __builtin_bit_cast(v8s, (u32x4){d[k], d[k + 1], d[k + 2], d[k + 3]});
    w.o[n % kTiles] = mfma<DT>(f[n % kAhead], p, w.o[n % kTiles]);
    f[n % kAhead] = n + kAhead < kValues ? value_operand(ln, v_lds, n + kAhead)
                                         : key_operand<DP, kGroups>(ln, k_after, n + kAhead - kValues);
    // the next scores are ready by the second product
    if (n == 1) best = nxt[0][0];
    if (n >= 1)
#pragma unroll
      for (int i = (n - 1) * kShare; i < n * kShare && i < 16 * kGroups; ++i) best = __builtin_fmaxf(best, nxt[i / 16][i % 16]);
    __builtin_amdgcn_sched_barrier(0);
  }
  top = both_max(best);
}

// ---------------------------------------------------------------- items
// One (request, block of rows, key/value head).
struct Item {
  int start;      // request's first token
  int news;       // its new tokens
  int keys;       // its keys
  int head;       // key/value head
  int row0;       // first row of the block
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Loads the rows row0 .. of a wave; rows past the request's last take the last
// one's limits and zero queries.
template <int DP>
__device__ __forceinline__ void load_rows(Rows<DP>& w, const AttnArgs& a, const Item& it, int row0, int lane) {
  const int rows = it.news * a.group, h = lane >> 5;
  const int r = row0 + (lane & 31), at = r < rows ? r : rows - 1;
  const int tok = token_of(a, at), hd = it.head * a.group + at - tok * a.group;
  const char* q = (const char*)a.q + ((int64_t)(it.start + tok) * a.q_stride + (int64_t)hd * a.q_head_stride) * 2;
#pragma unroll
  for (int st = 0; st < DP / 16; ++st) {
    const int ch = 2 * st + h;
    v8s x = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r < rows && ch * 8 < a.head_dim) x = *(const v8s*)(q + ch * 16);
    w.q[st] = x;
  }
  const int p = it.keys - it.news + tok;
  w.hi = p + 1;
  w.lo = (a.window > 0 && p + 1 > a.window) ? p + 1 - a.window : 0;
  w.m = kLowest;
  w.far = -__builtin_inff();
  w.late = w.big = 0;
  w.l = 0.0f;
#pragma unroll
  for (int t = 0; t < DP / 32; ++t) w.o[t] = zero16();
}

// The rows of a wave again, with references: 32 keys at a time, from first_key on every `step`-th such
// group before end_key.  `lds`: 32 rows of DP elements of the wave's own, for the keys and then the values
// of a group.  Rare: short rather than fast (every wave of an 8192-token prompt: 590 -> 2250 us; of 8 decodes
// over 8192 keys 48 -> 170 us, of 800 new tokens over them 173 -> 918 us).
template <int DT, int DP, bool PAGED>
__device__ __forceinline__ void again(Rows<DP>& w, const AttnArgs& a, const Source& s, const Item& it, int row0,
                                      int first_key, int end_key, int step, const Scaling& sc, uint32_t lds) {
  constexpr int kChunks = DP / 8, kRowsPer = 64 / kChunks;
  uint32_t ones = ~0u;
  asm volatile("" : "+s"(ones));   // nothing here is shared with the common path and kept in registers for it
  const int lane = __builtin_amdgcn_mbcnt_hi(ones, __builtin_amdgcn_mbcnt_lo(ones, 0));
  load_rows<DP>(w, a, it, row0, lane);
  const Lanes<DP> ln(lane);
#pragma unroll 1
  for (int kb = uni(first_key); kb < end_key; kb += step) {
    v16f x[1];
#pragma unroll 1
    for (int values = 0; values < 2; ++values) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // what is there has been read
#pragma unroll 1
      for (int n = 0; n < 32 / kRowsPer; ++n) {
        const int r = n * kRowsPer + lane / kChunks, j = kb + r;
        int page = 0;
        if constexpr (PAGED) page = j < s.keys ? s.table[page_of(s, j)] : -1;
        const char *k, *v;
        row_at<PAGED>(s, j, page, ((lane % kChunks) ^ swz<DP>(r)) * 16, k, v);
        dma16_at(values ? v : k, (uint32_t)uni(lds + n * 1024));
      }
      wait_vmcnt_le<0>();
      asm volatile("" ::: "memory");
      if (!values) scores<DT, DP, 1>(x, w, ln, lds);
    }
    add_keys<DT, DP, true>(w, ln, x[0], lds, kb, sc, 1, lane);
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

__device__ __forceinline__ float lse_of(float m, float ref, float l, float c) {
  return l == 0.0f ? -__builtin_inff() : (__builtin_fmaf(ref, c, m) + __builtin_log2f(l)) * kLn2;
}

// Writes a wave's finished rows, through its part `lds` of the tiles (32 rows of DP elements): a lane
// holds every second 8 bytes of one row, and memory is written 16 bytes a lane, whole rows at a time
// (8192 ragged tokens 89.5 -> 85.0 us, 32 prompts of 256 tokens 84 -> 65 us).  16-byte chunk p of
// row r is at chunk p ^ (r mod the chunks of a row).
template <int DT, int DP>
__device__ __forceinline__ void store_rows(const Rows<DP>& w, const AttnArgs& a, const Item& it, int row0, int lane,
                                           uint32_t lds) {
  typedef __attribute__((address_space(3))) u32x2* lds_2;
  constexpr int kChunks = DP / 8, kRowsPer = 64 / kChunks;
  const int rows = it.news * a.group, h = lane >> 5, c = lane & 31;
  const float l = both_sum(w.l), inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(lds_2)(uintptr_t)(lds + c * DP * 2 + ((t * 4 + i) ^ (c & (kChunks - 1))) * 16 + h * 8) =
          (u32x2){pack2<DT>(w.o[t][4 * i] * inv, w.o[t][4 * i + 1] * inv),
                  pack2<DT>(w.o[t][4 * i + 2] * inv, w.o[t][4 * i + 3] * inv)};
  auto place = [&](int r) {   // (token, head) of row r
    const int tok = token_of(a, r);
    return (int64_t)(it.start + tok) * a.q_heads + it.head * a.group + r - tok * a.group;
  };
  const int chunk = lane % kChunks;
#pragma unroll
  for (int n = 0; n < 32 / kRowsPer; ++n) {
    const int r = n * kRowsPer + lane / kChunks;
    const v8s x = read_b128(lds + r * DP * 2 + (chunk ^ (r & (kChunks - 1))) * 16);
    if (row0 + r < rows && chunk * 8 < a.head_dim)
      *(v8s*)((uint16_t*)a.out + place(row0 + r) * a.head_dim + chunk * 8) = x;
  }
  if (a.lse && h == 0 && row0 + c < rows) a.lse[place(row0 + c)] = lse_of(w.m, reference(w), l, a.scale * kLog2e);
}

// Part of rows whose keys are split over workgroups: O (unnormalized) [rows][DP], (m, l, reference, 0) [rows].
template <int DP>
__device__ __forceinline__ void store_part(const Rows<DP>& w, float* o, float* ml, int r, int lane) {
  const int h = lane >> 5;
  const float l = both_sum(w.l);
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(v4f*)(o + (int64_t)r * DP + t * 32 + 8 * i + 4 * h) =
          (v4f){w.o[t][4 * i], w.o[t][4 * i + 1], w.o[t][4 * i + 2], w.o[t][4 * i + 3]};
  const float ref = reference(w);
  if (h == 0) *(v4f*)(ml + 4 * r) = (v4f){w.m, l, ref, 0.0f};
}

// ---------------------------------------------------------------- many rows
// A workgroup of NW = 4 or 8 waves, 32 rows each; all waves share the tiles of
// 64 keys, copied global -> LDS.  A wave takes up to half the registers of two
// waves' SIMD, so a CU holds two workgroups of four waves or one of eight.  Two
// meet no common barrier, the start and end of one (10 us of loads, stores and
// dispatch) lie beside the work of the other, and blocks of 128 rows waste less
// above the diagonal; but every tile is copied twice as often.  So prompts have
// four waves and paged work, whose workgroups start and end once, has eight.
// Measured, 4 / 8 waves: 8192 ragged tokens 89.3 / 95.4 us, 9001 tokens of head
// dimension 64, window 1024 58.8 / 81.7, 210 tokens 12.1 / 14.3, one prompt of
// 8192 541 / 536; 1700 new tokens over 16k keys 1006 / 557 (head dimension 64:
// 360 / 328), where the copies from pages are what costs.
constexpr int kShares = 256;   // of paged work: the workgroups of eight waves that 256 CUs hold
constexpr int kMostRows = 32 * 8;
constexpr int kPromptWaves = 4;
constexpr int kCopyWaves = 4;
constexpr int kTile = 64;

template <int DP>
constexpr int tile_bytes() { return kTile * DP * 2; }

// Copies of one wave: kIters instructions for a tile of K or V, each of kRowsPer whole rows.  The
// copy path of a CU takes 64 bytes a cycle, 512 cycles for a tile of K and V (DP = 128), and a wave
// waits while it is busy.  Of eight waves only the first four copy: the others, which share the SIMDs
// with them, compute meanwhile, and the two are out of step from then on (530 us with all eight
// copying, 523 us).
template <int DP, bool PAGED, bool FULL>
struct TileCopy {
  static constexpr int kChunks = DP / 8;                    // 16-byte chunks of a row
  static constexpr int kRowsPer = 64 / kChunks;             // rows of one copy instruction
  static constexpr int kIters = kTile / (kRowsPer * kCopyWaves);
  static_assert(kIters >= 1 && (kCopyWaves * kRowsPer) % 16 == 0, "a lane's swizzle is the same in all its copies");
  const Source& s;
  int wave, lane;
  // The lane's place in an instruction, as a byte offset (paged) or as the byte of its row and, in the
  // upper half, the row: with an offset each for K and V the 128-wide prompt kernel spills them, and
  // reloading one waits for the copies in flight.
  uint32_t at;
  bool mine;                // the lane's bytes exist (not FULL: rows shorter than DP, whose rest is zeroed once)
  bool whole;               // the rows of an instruction lie in one page

  __device__ __forceinline__ TileCopy(const Source& src, int wv, int ln) : s(src), wave(wv), lane(ln) {
    const int row = lane / kChunks;
    at = (uint32_t)(((lane % kChunks) ^ swz<DP>(wave * kRowsPer + row)) * 16);
    mine = at < (uint32_t)s.d_bytes;
    at += PAGED ? (uint32_t)(row * s.d_bytes) : (uint32_t)row << 16;
    if constexpr (PAGED) whole = s.page_size % kRowsPer == 0;
    else whole = s.k_step < (1 << 27) && s.v_step < (1 << 27);
  }
  // Page of each instruction's first row, in scalar registers.
  struct Pages { int id[PAGED ? kIters : 1]; };
  __device__ __forceinline__ Pages pages(int kb) const {
    Pages p{};
    if constexpr (PAGED) {
      if (whole && wave < kCopyWaves) {
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
          const int j = kb + (it * kCopyWaves + wave) * kRowsPer;
          const auto at = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)(s.table + page_of(s, j < s.keys ? j : 0));
          p.id[it] = *at;
        }
      }
    }
    return p;
  }
  template <bool V>
  __device__ __forceinline__ void issue(int kb, const Pages& p, uint32_t lds) const {
    if (wave >= kCopyWaves) return;
    if (whole && kb + kTile <= s.keys) {
      if (!FULL && !mine) return;
      uint32_t ofs = at;
      if constexpr (!PAGED) {
        asm volatile("" : "+v"(ofs));   // formed here each time
        ofs = (ofs >> 16) * (uint32_t)(V ? s.v_step : s.k_step) + (ofs & 0xFFFFu);
      }
      const int j0 = kb + wave * kRowsPer;
      const char* base = V ? s.v : s.k;
      if constexpr (PAGED) {
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
          const int j = j0 + it * kCopyWaves * kRowsPer;
          const int64_t off = (int64_t)p.id[it] * s.k_step + place_bytes(j - page_of(s, j) * s.page_size, FULL ? DP * 2 : s.d_bytes);
          const bool there = (uint32_t)p.id[it] < (uint64_t)s.num_pages;
          dma16(there ? base + off : reinterpret_cast<const char*>(kZeros), ofs, lds + (it * kCopyWaves + wave) * 1024);
        }
      } else {
        const int64_t step = V ? s.v_step : s.k_step;
        base += j0 * step;
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
          dma16(base, ofs, lds + (it * kCopyWaves + wave) * 1024);
          base += step * (kCopyWaves * kRowsPer);
        }
      }
    } else {
      int l = lane;
      asm volatile("" : "+v"(l));   // nothing of this path is kept in registers beside the common one
#pragma unroll 1
      for (int it = 0; it < kIters; ++it) {
        const int r = (it * kCopyWaves + wave) * kRowsPer + l / kChunks, j = kb + r;
        int page = 0;
        if constexpr (PAGED) page = j < s.keys ? s.table[page_of(s, j)] : -1;
        const char *k, *v;
        row_at<PAGED>(s, j, page, ((l % kChunks) ^ swz<DP>(r)) * 16, k, v);
        dma16_at(V ? v : k, (uint32_t)uni(lds + (it * kCopyWaves + wave) * 1024));
      }
    }
  }
};

// Runs the keys of tiles [t0, t1) (tiles of 64 from key 0) through the block.
// The scores of the next tile are formed while the weights of the current one
// are, and the first operands of the tile after that are read ahead: iteration
// t uses K(t + 1), K(t + 2) and V(t) while K(t + 3) and V(t + 1) are on their
// way (three buffers of K, two of V, one barrier a tile).
template <int DT, int DP, int NW, bool PAGED, bool FULL>
__device__ __forceinline__ void run_block(const AttnArgs& a, const Source& s, const Item& it, int t0, int t1,
                                          Rows<DP>& w, uint32_t lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int rows = it.news * a.group;
  const int first = it.row0 + wave * 32;
  constexpr int kBytes = tile_bytes<DP>(), kHalf = kBytes / 2;
  using Copy = TileCopy<DP, PAGED, FULL>;
  const Copy cp(s, wave, lane);
  typename Copy::Pages p1{}, p2{}, p3{};   // of the tiles t + 1 .. t + 3
  uint32_t k_now = lds, k_next = lds + kBytes, k_after = lds + 2 * kBytes;
  uint32_t v_now = lds + 3 * kBytes, v_next = lds + 4 * kBytes;
  if constexpr (!FULL) {
    for (int n = tid; n < 5 * kBytes / 16; n += 64 * NW) zero_lds(lds + n * 16);
    lds_barrier();
  }
  if (t0 < t1) {
    const auto p0 = cp.pages(t0 * kTile);
    p1 = cp.pages((t0 + 1) * kTile);
    p2 = cp.pages((t0 + 2) * kTile);
    p3 = cp.pages((t0 + 3) * kTile);
    cp.template issue<false>(t0 * kTile, p0, k_now);
    cp.template issue<true>(t0 * kTile, p0, v_now);
    if (t0 + 1 < t1) cp.template issue<false>((t0 + 1) * kTile, p1, k_next);
    if (t0 + 2 < t1) cp.template issue<false>((t0 + 2) * kTile, p2, k_after);
  }
  load_rows<DP>(w, a, it, first, lane);
  // limits of the wave's rows: positions of its first and last row
  const bool active = first < rows;
  const int end = first + 32 < rows ? first + 32 : rows;
  const int pos0 = it.keys - it.news + token_of(a, first), pos1 = it.keys - it.news + (end > 0 ? token_of(a, end - 1) : 0);
  const int hi_min = uni(pos0 + 1), hi_max = uni(active ? pos1 + 1 : 0);
  const int lo_min = uni((a.window > 0 && hi_min > a.window) ? hi_min - a.window : 0);
  const int lo_max = uni((a.window > 0 && pos1 + 1 > a.window) ? pos1 + 1 - a.window : 0);
  const Scaling sc(a.scale);
  const Lanes<DP> ln(lane);
  // tiles that some row of the wave sees; those that every row sees
  const int w0 = clampi(lo_min / kTile, t0, t1), w1 = clampi((hi_max + kTile - 1) / kTile, w0, t1);
  const int full0 = (lo_max + kTile - 1) / kTile, full1 = hi_min < 0 ? 0 : hi_min / kTile < w1 ? hi_min / kTile : w1;
  int t = t0;
  auto begin = [&]() {
    wait_vmcnt_le<0>();
    lds_barrier();   // the copies have arrived, and K(t) and V(t - 1) have been read by all waves
    if (t + 3 < t1) cp.template issue<false>((t + 3) * kTile, p3, k_now);
    if (t + 1 < t1) cp.template issue<true>((t + 1) * kTile, p1, v_next);
  };
  auto end_tile = [&]() {
    const uint32_t k_old = k_now, v_old = v_now;
    k_now = k_next;
    k_next = k_after;
    k_after = k_old;
    v_now = v_next;
    v_next = v_old;
    ++t;
    p1 = p2;
    p2 = p3;
    p3 = cp.pages((t + 3) * kTile);
  };
  auto skip_to = [&](int stop) {
#pragma unroll 1
    while (t < stop) {
      begin();
      end_tile();
    }
  };
  wait_vmcnt_le<0>();
  lds_barrier();
  skip_to(w0);
  v16f sa[kGroups];
  if (t < w1) scores<DT, DP, kGroups>(sa, w, ln, k_now);
#pragma unroll 1
  while (t < w1) {
    // A single tile that every row sees goes this way in prompts only (210 tokens 11.2 -> 10.0 us; in the
    // paged kernel of padded rows it costs registers: 161 -> 179 us for a chunk of head dimension 80).
    if (t >= full0 && t + (PAGED ? 1 : 0) < full1) {
      v16f sb[kGroups];
      v8s f[kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) f[n] = key_operand<DP, kGroups>(ln, k_next, n);
      float top = both_max(__builtin_fmaxf(largest(sa[0]), largest(sa[1])));
      // two tiles a turn, so that the scores change places; past the last tile the next scores are
      // formed from whatever the buffer holds, and not used
#pragma unroll 1
      while (t + 1 < full1) {
        begin();
        add_tile<DT, DP>(w, ln, sa, sb, top, f, k_next, k_after, v_now, sc);
        end_tile();
        begin();
        add_tile<DT, DP>(w, ln, sb, sa, top, f, k_next, k_after, v_now, sc);
        end_tile();
      }
      if (t < full1) {
        begin();
        add_tile<DT, DP>(w, ln, sa, sb, top, f, k_next, k_after, v_now, sc);
        end_tile();
#pragma unroll
        for (int g = 0; g < kGroups; ++g) sa[g] = sb[g];
      }
    } else {
      begin();
      v16f x = sa[0];
#pragma unroll 1
      for (int g = 0; g < kGroups; ++g) {
        const int kb = t * kTile + g * 32;
        const int hidden = kb + 32 - hi_min > lo_max - kb ? kb + 32 - hi_min : lo_max - kb;
        if (kb < hi_max && kb + 32 > lo_min) add_keys<DT, DP>(w, ln, x, v_now + g * kHalf, kb, sc, hidden, lane);
        x = sa[1];
      }
      if (t + 1 < w1) scores<DT, DP, kGroups>(sa, w, ln, k_next);
      end_tile();
    }
  }
  skip_to(t1);
  lds_barrier();   // the buffers may be filled again
#pragma unroll 1
  for (int turns = turns_any(w.late); turns > 0; --turns)
    again<DT, DP, PAGED>(w, a, s, it, first, t0 * kTile, t1 * kTile, 32, sc, lds + wave * 32 * DP * 2);
}

// Tiles of `unit` keys that the rows row0 .. row0 + block - 1 see.
__device__ __forceinline__ void tiles_of(const AttnArgs& a, const Item& it, int row0, int block, int unit, int& t0, int& t1) {
  const int rows = it.news * a.group;
  const int end = row0 + block < rows ? row0 + block : rows;
  const int p0 = it.keys - it.news + token_of(a, row0), p1 = it.keys - it.news + token_of(a, end - 1);
  const int lo = (a.window > 0 && p0 + 1 > a.window) ? p0 + 1 - a.window : 0;
  t0 = lo / unit;
  t1 = p1 + 1 > 0 ? (p1 + unit) / unit : 0;
  if (t1 < t0) t1 = t0;
}

extern __shared__ __align__(1024) unsigned char dyn_lds[];

// Sum and maximum of a wave's non-negative values.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp0(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false); }
__device__ __forceinline__ int wave_sum(int v) {
  v += dpp0<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  v += dpp0<0x112, 0xF>(v);
  v += dpp0<0x114, 0xF>(v);
  v += dpp0<0x118, 0xF>(v);
  v += dpp0<0x142, 0xA>(v);   // row_bcast 15, 31
  v += dpp0<0x143, 0xC>(v);
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ int wave_or(int v) {
  v |= dpp0<0x111, 0xF>(v);
  v |= dpp0<0x112, 0xF>(v);
  v |= dpp0<0x114, 0xF>(v);
  v |= dpp0<0x118, 0xF>(v);
  v |= dpp0<0x142, 0xA>(v);
  v |= dpp0<0x143, 0xC>(v);
  return __builtin_amdgcn_readlane(v, 63);
}

// Whole prompts.  Workgroup (b, h): b counts blocks of rows over all requests,
// of which the host only knows a bound; the surplus, at the end, has nothing to
// do.  Request `seqs` is what follows the last prompt, rows without keys, which
// are set to 0.
//
// Workgroups go to the shader engines in turn, whatever these have left to do,
// so neighbours should have the same length: the blocks come by their number
// in the request, longest first (level L: block L of every request that has
// one).  Up to 4 x 64 requests are held by each wave, 4 per lane; of more, the
// blocks come in the requests' order.  Measured against the requests' order with
// the surplus between the requests: 128 prompts of 64 tokens 106 -> 73 us, 8192
// ragged tokens 97.6 -> 89.3 us.
//
// Key/value heads are the fastest index, so that workgroups on one XCD
// (dispatched round robin) share a head.
//
// Bound by the matrix cores and the instructions beside them for long prompts
// (8192 tokens, 550 GFLOP: 525 .. 555 us, 1.0 PFLOP/s, 0.68 of the rate of a
// large matrix product; the matrix cores are busy 64 % of the cycles), for short
// ones by a workgroup's start and end (ragged 8192 tokens, 365 keys a row on
// average: 94 us from memory, 83 where the caches hold part of the inputs, with
// 33 us of products).  At 128 dimensions 11 to 12 registers are spilled, none of
// them inside the blocks of 32 products; with rows shorter than 128 one is
// reloaded in every second tile.
template <int DT, int DP, bool FULL>
__global__ void __launch_bounds__(64 * kPromptWaves, 2) prompt_attn_kernel(AttnArgs a) {
  constexpr int NW = kPromptWaves, kRows = 32 * NW, kThreads = 64 * NW, kHold = 4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int head = blockIdx.x % a.kv_heads, b = blockIdx.x / a.kv_heads;
  auto limits = [&](int i, int& start, int& stop) {   // returns the blocks of request i
    start = clampi(a.cu[i], 0, a.tokens);
    stop = i < a.seqs ? clampi(a.cu[i + 1], start, a.tokens) : a.tokens;
    return (int)((uint32_t)((stop - start) * a.group + kRows - 1) / kRows);   // tokens * group <= 2^30
  };
  int req = -1, start = 0, stop = 0, block = 0;
  if (a.seqs <= 64 * kHold) {
    int n[kHold], first[kHold], end[kHold], all = 0, bits = 0;
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int i = k * 64 + lane;
      n[k] = first[k] = end[k] = 0;
      if (i < a.seqs) n[k] = limits(i, first[k], end[k]);
      all += n[k];
      bits |= n[k];
    }
    all = wave_sum(all);
    if (b >= all) {
      req = a.seqs;
      block = b - all;
      if (block >= uni(limits(req, start, stop))) return;   // surplus
    } else {
      // the largest L with more than b blocks at the levels from L on
      bits = wave_or(bits);
      int level = 0, above = 0;
      for (int bit = 31 - __builtin_clz(bits); bit >= 0; --bit) {
        const int l = level | (1 << bit);
        int x = 0;
#pragma unroll
        for (int k = 0; k < kHold; ++k) x += n[k] > l ? n[k] - l : 0;
        x = wave_sum(x);
        if (x > b) level = l;
        else above = x;   // ends as the blocks above the level
      }
      block = level;
      int left = b - above;   // which of the requests that have this block
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const uint64_t has = __ballot(n[k] > level);
        const int here = __popcll(has);
        if (req < 0 && left < here) {
          const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(has >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)has, 0));
          const int l = __builtin_ctzll(__ballot(n[k] > level && before == left));
          req = k * 64 + l;
          start = __builtin_amdgcn_readlane(first[k], l);
          stop = __builtin_amdgcn_readlane(end[k], l);
        }
        left -= here;
      }
    }
  } else {
    int* lds = reinterpret_cast<int*>(dyn_lds);   // before the tiles
    const int n = a.seqs + 1, per = (n + kThreads - 1) / kThreads;
    const int i0 = tid * per, i1 = i0 + per < n ? i0 + per : n;
    int v = 0;
    for (int i = i0; i < i1; ++i) v += limits(i, start, stop);
    int x = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(x, off, 64);
      if (lane >= off) x += y;
    }
    if (lane == 63) lds[tid >> 6] = x;
    if (tid == 0) lds[NW] = -1;
    __syncthreads();
    int before = x - v;
#pragma unroll
    for (int k = 0; k < NW; ++k)
      if (k < tid >> 6) before += lds[k];
    if (b >= before && b < before + v) {
      for (int i = i0; i < i1; ++i) {
        const int m = limits(i, start, stop);
        if (b < before + m) {
          lds[NW] = i;
          lds[NW + 1] = m - 1 - (b - before);   // a request's longest rows first
          break;
        }
        before += m;
      }
    }
    __syncthreads();
    req = uni(lds[NW]);
    block = uni(lds[NW + 1]);
    __syncthreads();   // the tiles take their place
    // starts that do not rise can make a block that does not exist
    if (req < 0 || block < 0 || block >= uni(limits(req, start, stop))) return;
  }
  start = uni(start);
  stop = uni(stop);
  req = uni(req);
  block = uni(block);
  const int news = stop - start;
  Item it{start, news, news, head, block * kRows};
  Source s{};
  s.k = (const char*)a.k + ((int64_t)start * a.k_stride + (int64_t)head * a.k_head_stride) * 2;
  s.v = (const char*)a.v + ((int64_t)start * a.v_stride + (int64_t)head * a.v_head_stride) * 2;
  s.k_step = a.k_stride * 2;
  s.v_step = a.v_stride * 2;
  s.keys = news;
  s.d_bytes = a.head_dim * 2;
  int t0 = 0, t1 = 0;
  if (req < a.seqs) tiles_of(a, it, it.row0, kRows, kTile, t0, t1);
  Rows<DP> w;
  run_block<DT, DP, NW, false, FULL>(a, s, it, t0, t1, w, lds_addr(dyn_lds));
  const int wave = uni(tid >> 6);
  store_rows<DT, DP>(w, a, it, it.row0 + wave * 32, lane, lds_addr(dyn_lds) + wave * 32 * DP * 2);
}

// ---------------------------------------------------------------- paged: work split
// The work of a call is the sequence of units (request, head, block of rows,
// tile of keys), tiles innermost, and every workgroup takes an equal share of
// consecutive units: long and short requests balance whatever their lengths,
// which only the device knows.  What an item costs besides its tiles (finding
// it, its queries, the first copies, its results) counts as kExtra units ahead
// of its tiles; a share that ends among those has none of the item's work.  A share that starts or ends inside an item
// leaves a part (O, m, l) in the workspace, and combine_kernel joins the parts.
// Each workgroup sums the units of all requests itself (up to 63 requests: one
// load and one scan in every wave; more: consecutive requests per thread, of
// which the kernels have 128, 512 and 256), which is cheaper than another launch.
struct Split {
  int min_rows;   // requests with min_rows <= rows <= max_rows take part
  int max_rows;
};

// Measured with 64-key units (64 requests of 100 .. 8192 keys): 158 us without, 122 / 111 / 104 /
// 102 / 101 / 103 / 106 us with 1 / 2 / 3 / 4 / 5 / 6 / 8.
constexpr int kExtra = 4;

struct Req {
  int start, news, keys;
  int t0, tiles;    // tiles that some row sees
  int blocks;
  int64_t units;    // of all heads
};

// BLOCK rows, UNIT keys of a tile (powers of two).
template <int BLOCK, int UNIT>
__device__ __forceinline__ Req request(const AttnArgs& a, const Split& sp, int i) {
  Req r;
  r.start = clampi(a.cu[i], 0, a.tokens);
  const int stop = i < a.seqs ? clampi(a.cu[i + 1], r.start, a.tokens) : a.tokens;
  r.news = stop - r.start;
  r.keys = i < a.seqs ? clampi(a.kv_lens[i], 0, a.max_pages * a.page_size) : 0;
  const int rows = r.news * a.group;
  r.units = 0;
  r.t0 = r.tiles = r.blocks = 0;
  if (rows >= sp.min_rows && rows <= sp.max_rows && rows > 0) {
    const int p = r.keys - r.news;   // position of the first row
    const int lo = (a.window > 0 && p + 1 > a.window) ? p + 1 - a.window : 0;
    r.t0 = lo / UNIT;
    const int t1 = (int)((uint32_t)(r.keys + UNIT - 1) / UNIT);
    r.tiles = t1 > r.t0 ? t1 - r.t0 : 1;   // a request without keys still has its rows written
    r.blocks = (int)((uint32_t)(rows + BLOCK - 1) / BLOCK);
    r.units = (int64_t)r.blocks * (r.tiles + kExtra) * a.kv_heads;
  }
  return r;
}

// The place of a share's first unit, and access to the requests from there on.  Up to 63 requests
// (and the rows past the last) are held one per lane, by every wave for itself: one load, a scan over
// the lanes and no barrier.  More are summed by the workgroup and loaded again when they are reached;
// so are they, without KEEP, where the registers to hold them are missing.
template <int BLOCK, int UNIT, int SHARES, int NT, bool KEEP = true>
struct Plan {
  const AttnArgs& a;
  const Split& sp;
  Req mine;         // of request `lane`
  int req;          // request of the first unit, > seqs if past the end
  int64_t before;   // units before this request
  int64_t total, share;

  __device__ __forceinline__ Plan(const AttnArgs& args, const Split& split, int w, int64_t* lds) : a(args), sp(split) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (a.seqs < 64) {
      mine = Req{};
      if (lane <= a.seqs) mine = request<BLOCK, UNIT>(a, sp, lane);
      int64_t x = mine.units;
#pragma unroll 1
      for (int off = 1; off <= a.seqs; off <<= 1) {
        const int64_t y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
      }
      set_total(lane64(x, a.seqs));
      const int64_t u = share * w;
      // the requests whose units end at or before u come first
      req = __popcll(__ballot(lane <= a.seqs && x <= u));
      before = req > 0 ? lane64(x, req - 1) : 0;
      return;
    }
    const int n = a.seqs + 1, per = (n + NT - 1) / NT;
    const int i0 = tid * per, i1 = i0 + per < n ? i0 + per : n;
    int64_t v = 0;
    for (int i = i0; i < i1; ++i) v += request<BLOCK, UNIT>(a, sp, i).units;
    int64_t x = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t y = __shfl_up(x, off, 64);
      if (lane >= off) x += y;
    }
    if (lane == 63) lds[wave] = x;
    if (tid == 0) lds[NT / 64] = n;
    __syncthreads();
    int64_t start = x - v, all = 0;
#pragma unroll
    for (int k = 0; k < NT / 64; ++k) {
      if (k < wave) start += lds[k];
      all += lds[k];
    }
    set_total(uni64(all));
    const int64_t u = share * w;
    if (u >= start && u < start + v) {
      for (int i = i0; i < i1; ++i) {
        const int64_t r = request<BLOCK, UNIT>(a, sp, i).units;
        if (u < start + r) {
          lds[NT / 64] = i;
          lds[NT / 64 + 1] = start;
          break;
        }
        start += r;
      }
    }
    __syncthreads();
    req = uni((int)lds[NT / 64]);
    before = req < n ? uni64(lds[NT / 64 + 1]) : 0;
    __syncthreads();   // the LDS may be used for something else
  }
  __device__ __forceinline__ static int64_t lane64(int64_t v, int l) {
    return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32) |
                     (uint32_t)__builtin_amdgcn_readlane((int)v, l));
  }
  __device__ __forceinline__ void set_total(int64_t all) {
    total = all;
    share = (all + SHARES - 1) / SHARES;
    if (share < 1) share = 1;
  }
  __device__ __forceinline__ Req get(int i) const {
    if (KEEP && a.seqs < 64) {
      Req r;
      r.start = __builtin_amdgcn_readlane(mine.start, i);
      r.news = __builtin_amdgcn_readlane(mine.news, i);
      r.keys = __builtin_amdgcn_readlane(mine.keys, i);
      r.t0 = __builtin_amdgcn_readlane(mine.t0, i);
      r.tiles = __builtin_amdgcn_readlane(mine.tiles, i);
      r.blocks = __builtin_amdgcn_readlane(mine.blocks, i);
      r.units = lane64(mine.units, i);
      return r;
    }
    return request<BLOCK, UNIT>(a, sp, i);
  }
};

// Segment of a share: the tiles [t0, t1) of one item.
struct Segment {
  Item it;
  int req, t0, t1;
};

template <int DP, int ROWS, int SHARES>
__device__ __forceinline__ void part_of(float* ws, int slot, float*& o, float*& ml) {
  ml = ws + (int64_t)slot * ROWS * 4;
  o = ws + (int64_t)SHARES * 2 * ROWS * 4 + (int64_t)slot * ROWS * DP;
}

__device__ __forceinline__ void paged_source(const AttnArgs& a, const Item& it, int req, Source& s, uint32_t magic, int shift) {
  const int64_t head = (int64_t)a.page_size * a.head_dim * 2;
  s.k = (const char*)a.k + it.head * head;
  s.v = (const char*)a.v + it.head * head;
  s.k_step = s.v_step = head * a.kv_heads;
  s.table = a.block_table + (int64_t)(req < a.seqs ? req : 0) * a.max_pages;
  s.page_size = a.page_size;
  s.magic = magic;
  s.shift = shift;
  s.num_pages = a.num_pages;
  s.keys = it.keys;
  s.d_bytes = a.head_dim * 2;
}

// Walks the segments of share w; f(segment, slot or -1).
template <int BLOCK, int UNIT, int SHARES, int NT, bool KEEP, typename F>
__device__ __forceinline__ void for_segments(const AttnArgs& a, const Split& sp, int w, int64_t* lds, F f) {
  const Plan<BLOCK, UNIT, SHARES, NT, KEEP> pl(a, sp, w, lds);
  int64_t u = pl.share * w;
  const int64_t begin = u, end = u + pl.share < pl.total ? u + pl.share : pl.total;
  int64_t before = pl.before;
#pragma unroll 1
  for (int req = pl.req; req <= a.seqs && u < end; ++req) {
    const Req r = pl.get(req);
#pragma unroll 1
    while (u < end && u < before + r.units) {
      const int cost = r.tiles + kExtra;
      const int64_t item = quotient(u - before, cost);   // (head, block)
      const int at = (int)(u - before - item * cost);
      const int head = (int)quotient(item, r.blocks), rb = (int)(item - (int64_t)head * r.blocks);
      const int64_t left = end - u;
      const int count = left < cost - at ? (int)left : cost - at;
      const int first = at > kExtra ? at - kExtra : 0, last = at + count - kExtra;
      if (last > first) {
        Segment g;
        g.it = Item{uni(r.start), uni(r.news), uni(r.keys), uni(head), uni(rb * BLOCK)};
        g.req = req;
        g.t0 = uni(r.t0 + first);
        // no key at all: the unit only writes the rows
        g.t1 = uni(r.t0 + (r.keys == 0 ? first : last));
        f(g, uni(first == 0 && last == r.tiles ? -1 : 2 * w + (u > begin ? 1 : 0)));
      }
      u += count;
    }
    before += r.units;
  }
}

// ---------------------------------------------------------------- paged: many rows
// 1700 new tokens over 9k and 16k keys, 515 GFLOP, take 520 .. 550 us, 0.6 of a
// large matrix product's rate; the joining of the parts 26 us (67 MB written and
// read).  The matrix cores are busy 48 % of the cycles (a long prompt: 64 %): one
// workgroup a CU, whose eight waves meet at a barrier every tile, finds a page
// and forms a 64-bit address for each copy, and the XCDs' L2s fetch the keys and
// values about three times over.  At 128 dimensions 50 to 55 registers are
// spilled, none of them inside the blocks of 32 products.
template <int DT, int DP, bool FULL>
__global__ void __launch_bounds__(512, 2)
paged_rows_kernel(AttnArgs a, Split sp, uint32_t magic, int shift) {
  int64_t* lds = reinterpret_cast<int64_t*>(dyn_lds);   // before the tiles
  constexpr int NW = 8, kRows = kMostRows;
  // an XCD takes consecutive shares, so that workgroups that read the same keys share its L2
  const int w = (blockIdx.x & 7) * (kShares / 8) + (blockIdx.x >> 3);
  for_segments<kRows, kTile, kShares, 64 * NW, false>(a, sp, w, lds, [&](const Segment& g, int slot) {
    Source s;
    paged_source(a, g.it, g.req, s, magic, shift);
    int b0, b1;
    tiles_of(a, g.it, g.it.row0, kRows, kTile, b0, b1);
    const int t0 = uni(g.t0 > b0 ? g.t0 : b0), t1 = uni(g.t1 < b1 ? g.t1 : b1);
    Rows<DP> rows;
    run_block<DT, DP, NW, true, FULL>(a, s, g.it, t0, t1, rows, lds_addr(dyn_lds));
    const int row = uni(threadIdx.x >> 6) * 32, lane = threadIdx.x & 63;
    if (slot < 0) {
      store_rows<DT, DP>(rows, a, g.it, g.it.row0 + row, lane, lds_addr(dyn_lds) + row * DP * 2);
    } else {
      float *o, *ml;
      part_of<DP, kRows, kShares>((float*)a.workspace, slot, o, ml);
      store_part<DP>(rows, o, ml, row + (lane & 31), lane);
    }
    lds_barrier();   // the tiles may be filled again
  });
}

// ---------------------------------------------------------------- paged: few rows
// Up to 32 rows of an item (decode steps: the heads of a group, a few tokens).
// Nothing is shared between waves but the queries: wave w takes the 32-key
// tiles w, w + NW, ... and copies them itself, two tiles ahead, without a
// barrier; the waves' states are joined at the end.  Page ids come from a
// window of the block table in LDS: a load of them from memory would be waited
// for together with the copies in flight (vector loads) or with the operands
// from LDS (scalar loads).
//
// Bound by memory where the keys are many: 64 requests of 100 .. 8192 keys (468
// MB) take 102 us, 4.6 TB/s, with the joining of parts (7 us); 4 requests of 100k
// keys (1.95 GB) 342 us, 5.7 TB/s, above the 5.1 TB/s of a copy that also writes.
// One request of 1000 keys takes 10.1 us and 5.0 us to join: latency (lengths,
// split, page ids, one or two tiles, exchange).
constexpr int kWindow = 256;   // page ids a wave keeps
constexpr int kFewRows = 32, kFewWaves = 2;
constexpr int kFewShares = 512;    // two workgroups on each CU

template <int DT, int DP, int NW, bool FULL>
__global__ void __launch_bounds__(64 * NW, 1)
paged_few_kernel(AttnArgs a, Split sp, uint32_t magic, int shift) {
  __shared__ int64_t lds[NW + 2];
  __shared__ int win[NW][kWindow];
  __shared__ float join_ml[NW][32][3];   // maximum, sum, reference
  constexpr int kChunks = DP / 8, kRowsPer = 64 / kChunks, kIters = 32 / kRowsPer;
  constexpr int kHalf = 32 * DP * 2, kStage = 2 * kHalf;   // bytes of a tile of K, of K and V
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const uint32_t mem = lds_addr(dyn_lds) + wave * 2 * kStage;
  float* join_o = (float*)dyn_lds;          // [NW][32][DP] after the copies
  const Lanes<DP> ln(lane);
  // the lane's row and chunk in copy 0; in copy it the row is kRowsPer it further down and the
  // swizzle differs in its two lowest bits
  const uint32_t row_ofs = (lane / kChunks) * (FULL ? DP : a.head_dim) * 2;
  const int chunk0 = (lane % kChunks) ^ swz<DP>(lane / kChunks);
  const int w = (blockIdx.x & 7) * (kFewShares / 8) + (blockIdx.x >> 3);
  for_segments<kFewRows, 32 * NW, kFewShares, 64 * NW, true>(a, sp, w, lds, [&](const Segment& g, int slot) {
    Source s;
    paged_source(a, g.it, g.req, s, magic, shift);
    const int group = a.group, rows = g.it.news * group;
    const int last = (g.it.row0 + 32 < rows ? g.it.row0 + 32 : rows) - 1;
    const int p0 = g.it.keys - g.it.news + token_of(a, g.it.row0), p1 = g.it.keys - g.it.news + token_of(a, last);
    const int hi_min = p0 + 1, hi_max = p1 + 1;
    const int lo_min = (a.window > 0 && hi_min > a.window) ? hi_min - a.window : 0;
    const int lo_max = (a.window > 0 && hi_max > a.window) ? hi_max - a.window : 0;
    const Scaling sc(a.scale);
    const int n = g.t1 - g.t0;
    const bool whole = s.page_size % 8 == 0;   // eight keys lie in one page
    if constexpr (!FULL) {   // what the copies leave out of the rows
      for (int m = lane; m < 2 * kStage / 16; m += 64) zero_lds(mem + m * 16);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    const int64_t k_to_v = s.v - s.k;
    int win0 = 0, win1 = 0;   // pages held
    auto hold = [&](int kb) {   // the pages of keys kb .. kb + 31
      const int first = page_of(s, kb), end = page_of(s, kb + 31 < s.keys ? kb + 31 : s.keys - 1) + 1;
      if (first >= win0 && end <= win1) return;
      win0 = first;
      win1 = first + kWindow;
#pragma unroll
      for (int k = 0; k < kWindow; k += 64)
        win[wave][k + lane] = first + k + lane < a.max_pages ? s.table[first + k + lane] : -1;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
    auto issue = [&](int t) {
      const int kb = ((g.t0 + t) * NW + wave) * 32;
      const uint32_t to = mem + (t & 1) * kStage;
      if (kb < s.keys) hold(kb);
      if (whole && kb + 32 <= s.keys) {
        const int ids = win[wave][page_of(s, kb + (lane & 3) * 8) - win0];
#pragma unroll
        for (int n8 = 0; n8 < 4; ++n8) {
          const int id = __builtin_amdgcn_readlane(ids, n8), j = kb + n8 * 8;
          const bool there = (uint32_t)id < (uint64_t)s.num_pages;
          const int64_t off = (int64_t)id * s.k_step + place_bytes(j - page_of(s, j) * s.page_size, FULL ? DP * 2 : s.d_bytes);
          const char* k = there ? s.k + off : reinterpret_cast<const char*>(kZeros);
          const char* v = there ? k + k_to_v : k;
#pragma unroll
          for (int m = 0; m < 8 / kRowsPer; ++m) {
            const int it = n8 * (8 / kRowsPer) + m, skip = there ? m * kRowsPer * (FULL ? DP * 2 : s.d_bytes) : 0;
            const uint32_t chunk = (uint32_t)(chunk0 ^ (it * kRowsPer / 4 % 4)) * 16;
            if (FULL || chunk < (uint32_t)s.d_bytes) {
              dma16(k + skip, row_ofs + chunk, to + it * 1024);
              dma16(v + skip, row_ofs + chunk, to + kHalf + it * 1024);
            }
          }
        }
      } else {
#pragma unroll 1
        for (int it = 0; it < kIters; ++it) {
          const int r = it * kRowsPer + lane / kChunks, j = kb + r;
          const int page = j < s.keys ? win[wave][page_of(s, j) - win0] : -1;
          const char *kr, *vr;
          row_at<true>(s, j, page, ((lane % kChunks) ^ swz<DP>(r)) * 16, kr, vr);
          dma16_at(kr, (uint32_t)uni(to + it * 1024));
          dma16_at(vr, (uint32_t)uni(to + kHalf + it * 1024));
        }
      }
    };
    Rows<DP> st;
    load_rows<DP>(st, a, g.it, g.it.row0, lane);
    if (n > 0 && (g.t0 * NW + wave) * 32 < s.keys) hold((g.t0 * NW + wave) * 32);
    wait_vmcnt_le<0>();   // the queries: from here on only copies are waited for
#pragma unroll 1
    for (int t = -2; t < n; ++t) {
      if (t >= 0) {
        const int kb = ((g.t0 + t) * NW + wave) * 32;
        const uint32_t at = mem + (t & 1) * kStage;
        const bool more = t + 1 < n, seen = kb < hi_max && kb + 32 > lo_min;
        if (more) wait_vmcnt_le<2 * kIters>();
        else wait_vmcnt_le<0>();
        asm volatile("" ::: "memory");
        if (seen) {
          v16f x[1];
          scores<DT, DP, 1>(x, st, ln, at);
          add_keys<DT, DP>(st, ln, x[0], at + kHalf, kb, sc,
                           kb + 32 - hi_min > lo_max - kb ? kb + 32 - hi_min : lo_max - kb, lane);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      if (t + 2 < n) issue(t + 2);
    }
#pragma unroll 1
    for (int turns = turns_any(st.late); turns > 0; --turns)
      again<DT, DP, true>(st, a, s, g.it, g.it.row0, (g.t0 * NW + wave) * 32, g.t1 * NW * 32, NW * 32, sc, mem);
    // join the waves: weights 2^(m_w - m)
    const int h = lane >> 5, col = lane & 31;
    const float l = both_sum(st.l), own = reference(st);
    if (h == 0) {
      join_ml[wave][col][0] = st.m;
      join_ml[wave][col][1] = l;
      join_ml[wave][col][2] = own;
    }
    __syncthreads();
    // the largest maximum of row r, and its reference
    auto largest_of = [&](int r, float& m, float& ref) {
      m = join_ml[0][r][0];
      ref = join_ml[0][r][2];
#pragma unroll
      for (int k = 1; k < NW; ++k)
        if (above(join_ml[k][r][0], join_ml[k][r][2], m, ref, sc.c) > 0.0f) {
          m = join_ml[k][r][0];
          ref = join_ml[k][r][2];
        }
    };
    float m, ref;
    largest_of(col, m, ref);
    const float mine = __builtin_amdgcn_exp2f(above(st.m, own, m, ref, sc.c));
    // a row stored from bank 4 col on: the 32 rows of a store take all banks in turn
    if (g.it.row0 + col < rows)
#pragma unroll
    for (int t = 0; t < DP / 32; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v4f x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = st.o[t][4 * i + e] * mine;
        const int q = t * 8 + 2 * i + h;
        *(v4f*)(join_o + (wave * 32 + col) * DP + ((q ^ (col & (DP / 4 - 1))) * 4)) = x;
      }
    __syncthreads();
    // thread: one row's four values of d at a time
    float *po = nullptr, *pml = nullptr;
    if (slot >= 0) part_of<DP, kFewRows, kFewShares>((float*)a.workspace, slot, po, pml);
    for (int k = tid; k < 32 * (DP / 4); k += 64 * NW) {
      const int r = k / (DP / 4), q = k % (DP / 4), row = g.it.row0 + r;
      if (row >= rows) continue;
      float mm, rr;
      largest_of(r, mm, rr);
      float ll = 0.0f;
      v4f o = {0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        ll += join_ml[x][r][1] * __builtin_amdgcn_exp2f(above(join_ml[x][r][0], join_ml[x][r][2], mm, rr, sc.c));
        const v4f y = *(const v4f*)(join_o + (x * 32 + r) * DP + ((q ^ (r & (DP / 4 - 1))) * 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += y[e];
      }
      if (slot < 0) {
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        const int tok = token_of(a, row);
        const int64_t at = (int64_t)(g.it.start + tok) * a.q_heads + g.it.head * group + row - tok * group;
        if (q * 4 < a.head_dim)
          *(u32x2*)((uint32_t*)a.out + at * (a.head_dim / 2) + q * 2) =
              (u32x2){pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
        if (a.lse && q == 0) a.lse[at] = lse_of(mm, rr, ll, sc.c);
      } else {
        *(v4f*)(po + (int64_t)r * DP + q * 4) = o;
        if (q == 0) *(v4f*)(pml + 4 * r) = (v4f){mm, ll, rr, 0.0f};
      }
    }
    __syncthreads();   // join_o is the next segment's tile memory
  });
}

// ---------------------------------------------------------------- paged: join the parts
// Workgroup w: the item that share w's first unit lies inside of, if no
// earlier share starts inside it too.  Its parts are the last segment of share
// w - 1 and the first segments of the shares from w on.  The parts come from
// other XCDs' L2s, so a load takes most of a microsecond and what counts is
// that few wait for one another: 8 teams of threads (DP = 128; a team holds a
// row) either take 8 rows, each reading kBatch parts at a time (ROWS = 256: two
// or three parts where the items are many; a single item has up to SHARES, which
// are then read in sequence), or every 8th part of one row after another (ROWS =
// 32: a long request alone has dozens of parts).
constexpr int kBatch = 4;

// Block (bx, by) of the items of one kind, whose parts are at ws.
template <int DT, int DP, int ROWS, int UNIT, int SHARES>
__device__ __forceinline__ void combine(const AttnArgs& a, const Split& sp, float* ws, int bx, int by) {
  constexpr int kQ = DP / 4, kTeams = 256 / kQ;
  constexpr bool kByPart = ROWS <= 32;
  __shared__ int64_t lds[6];
  __shared__ v4f part_ml[kByPart ? kBatch : 1][kTeams];
  __shared__ v4f part_o[kByPart ? kBatch : 1][kTeams][kQ];
  const int w = bx + 1, tid = threadIdx.x;
  const Plan<ROWS, UNIT, SHARES, 256> pl(a, sp, w, lds);
  if (pl.req > a.seqs || pl.share * w >= pl.total) return;
  const Req r = pl.get(pl.req);
  const int cost = r.tiles + kExtra;
  const int64_t item = quotient(pl.share * w - pl.before, cost);   // (head, block) in this request
  const int64_t s0 = pl.before + item * cost, s1 = s0 + cost;
  // the share starts inside the item's tiles, and it is the first that does
  if (pl.share * w - s0 <= kExtra || pl.share * (w - 1) - s0 > kExtra) return;
  const int last = (int)quotient(s1 + pl.share - 1, pl.share) - 1;
  const int head = (int)quotient(item, r.blocks), rb = (int)(item - (int64_t)head * r.blocks);
  const int group = a.group, rows = r.news * group - rb * ROWS < ROWS ? r.news * group - rb * ROWS : ROWS;
  const int first_slot = 2 * (w - 1) + (s0 > pl.share * (w - 1) ? 1 : 0);
  const int q = tid % kQ, g = tid / kQ;
  const float c = a.scale * kLog2e;
  auto load = [&](int j, int row, v4f& ml, v4f& x) {   // part j
    float *po, *pml;
    part_of<DP, ROWS, SHARES>(ws, j == w - 1 ? first_slot : 2 * j, po, pml);
    ml = *(const v4f*)(pml + 4 * row);
    x = *(const v4f*)(po + (int64_t)row * DP + q * 4);
  };
  const v4f none = {kLowest, 0.0f, 0.0f, 0.0f};   // maximum, sum, reference
  auto join = [&](v4f& ml, v4f& o, v4f pml, v4f x) {
    const float d = above(pml[0], pml[2], ml[0], ml[2], c);
    const float u = __builtin_amdgcn_exp2f(__builtin_fminf(-d, 0.0f)), v = __builtin_amdgcn_exp2f(__builtin_fminf(d, 0.0f));
    ml[1] = ml[1] * u + pml[1] * v;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * u + x[e] * v;
    ml[0] = d > 0.0f ? pml[0] : ml[0];
    ml[2] = d > 0.0f ? pml[2] : ml[2];
  };
  auto write = [&](int row, v4f ml, v4f o) {
    const float l = ml[1], inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int gr = rb * ROWS + row, tok = token_of(a, gr);
    const int64_t at = (int64_t)(r.start + tok) * a.q_heads + head * group + gr - tok * group;
    if (q * 4 < a.head_dim)
      *(u32x2*)((uint32_t*)a.out + at * (a.head_dim / 2) + q * 2) =
          (u32x2){pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
    if (a.lse && q == 0) a.lse[at] = lse_of(ml[0], ml[2], l, c);
  };
  if constexpr (!kByPart) {
    const int row = by * kTeams + g;
    if (row >= rows) return;
    v4f ml = none, o = {0, 0, 0, 0};
    for (int j = w - 1; j <= last; j += kBatch) {
      v4f p[kBatch], x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) load(j + k < last ? j + k : last, row, p[k], x[k]);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (j + k <= last) join(ml, o, p[k], x[k]);
    }
    write(row, ml, o);
  } else {
    for (int row0 = 0; row0 < rows; row0 += kBatch) {
      v4f ml[kBatch], o[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ml[k] = none;
        o[k] = (v4f){0, 0, 0, 0};
      }
      for (int j = w - 1 + g; j <= last; j += kTeams) {
        v4f p[kBatch], x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) load(j, row0 + k < rows ? row0 + k : rows - 1, p[k], x[k]);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) join(ml[k], o[k], p[k], x[k]);
      }
      if (row0 > 0) __syncthreads();
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (q == 0) part_ml[k][g] = ml[k];
        part_o[k][g][q] = o[k];
      }
      __syncthreads();
      if (g < kBatch && row0 + g < rows) {
        v4f jml = none, jo = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kTeams; ++k) join(jml, jo, part_ml[g][k], part_o[g][k][q]);
        write(row0 + g, jml, jo);
      }
    }
  }
}

// Joins the parts of both kinds in one launch: one for each takes 3 to 5 us even if nothing was split
// (100 new tokens for each of 4 requests over 3000 keys 68.9 -> 63.4 us).  The few-row items'
// workgroups come first; a kind that the call does not run has no rows.
template <int DT, int DP>
__global__ void __launch_bounds__(256) combine_kernel(AttnArgs a, Split few, Split many, float* many_ws) {
  const int few_blocks = few.max_rows > 0 ? kFewShares - 1 : 0, b = (int)blockIdx.x - few_blocks;
  if (b < 0)
    combine<DT, DP, kFewRows, 32 * kFewWaves, kFewShares>(a, few, (float*)a.workspace, blockIdx.x, 0);
  else
    combine<DT, DP, kMostRows, kTile, kShares>(a, many, many_ws, b % (kShares - 1), b / (kShares - 1));
}

// ---------------------------------------------------------------- host
// three tiles of K and two of V
template <int DP>
constexpr size_t many_lds_bytes() { return 5 * tile_bytes<DP>(); }
template <int DP>
constexpr size_t few_lds_bytes() { return kFewWaves * 2 * 2 * 32 * DP * 2; }

int padded_dim(int d) { return d <= 64 ? 64 : 128; }

// Which of the two kernels a call can need: a request of more than kFewRows
// rows needs more than one token per request on average or a group of heads
// above kFewRows; where one request makes the call, its size is known.
bool needs_many(int64_t seqs, int64_t tokens, int group) {
  if (tokens <= seqs) return false;
  return tokens * group > kFewRows;
}
bool needs_few(int64_t seqs, int64_t tokens, int group) {
  if (!needs_many(seqs, tokens, group)) return true;
  return seqs > 1;
}

AttnArgs with_group(const AttnArgs& a) {
  AttnArgs c = a;
  c.group = a.q_heads / a.kv_heads;
  division_magic(c.group, c.group_magic, c.group_shift);
  return c;
}

// Launch of kernel F with more dynamic LDS than the 64 KiB a kernel gets unasked; asked for once on
// each device.
template <auto F, typename... A>
hipError_t launch_lds(unsigned grid, unsigned block, size_t lds, hipStream_t s, A... args) {
  static std::atomic<uint64_t> asked{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(asked.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(F), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  F<<<dim3(grid), dim3(block), lds, s>>>(args...);
  return hipGetLastError();
}

// At least the blocks of rows of all requests.
int64_t prompt_blocks(const AttnArgs& a) {
  return (int64_t)a.tokens * (a.q_heads / a.kv_heads) / (32 * kPromptWaves) + a.seqs + 1;
}

template <int DT, int DP, bool FULL>
hipError_t prompt_full(const AttnArgs& a, hipStream_t s) {
  return launch_lds<prompt_attn_kernel<DT, DP, FULL>>((unsigned)(prompt_blocks(a) * a.kv_heads), 64 * kPromptWaves,
                                                      many_lds_bytes<DP>(), s, with_group(a));
}

// Bytes of the parts of few-row and of many-row items.
size_t few_bytes(int padded) { return (size_t)kFewShares * 2 * kFewRows * (padded + 4) * sizeof(float); }
size_t many_bytes(int padded) { return (size_t)kShares * 2 * kMostRows * (padded + 4) * sizeof(float); }

template <int DT, int DP>
hipError_t prompt_dp(const AttnArgs& a, hipStream_t s) {
  return a.head_dim == DP ? prompt_full<DT, DP, true>(a, s) : prompt_full<DT, DP, false>(a, s);
}

template <int DT, int DP, bool FULL>
hipError_t paged_dp(const AttnArgs& a, hipStream_t s) {
  const AttnArgs c = with_group(a);
  const bool many = needs_many(a.seqs, a.tokens, c.group), few = needs_few(a.seqs, a.tokens, c.group);
  uint32_t magic;
  int shift;
  division_magic(a.page_size, magic, shift);
  hipError_t e = hipSuccess;
  constexpr int kTeams = 256 / (DP / 4);   // rows of a combining workgroup
  const Split none{1, 0}, sf = few ? Split{1, many ? kFewRows : 0x7FFFFFFF} : none;
  const Split sm = many ? Split{few ? kFewRows + 1 : 1, 0x7FFFFFFF} : none;
  AttnArgs cm = c;
  if (few) cm.workspace = (char*)c.workspace + few_bytes(DP);
  if (few) {
    e = launch_lds<paged_few_kernel<DT, DP, kFewWaves, FULL>>(kFewShares, 64 * kFewWaves, few_lds_bytes<DP>(), s, c, sf, magic, shift);
    if (e != hipSuccess) return e;
  }
  if (many) {
    e = launch_lds<paged_rows_kernel<DT, DP, FULL>>(kShares, 512, many_lds_bytes<DP>(), s, cm, sm, magic, shift);
    if (e != hipSuccess) return e;
  }
  const int blocks = (few ? kFewShares - 1 : 0) + (many ? (kShares - 1) * (kMostRows / kTeams) : 0);
  combine_kernel<DT, DP><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(c, sf, sm, (float*)cm.workspace);
  return hipGetLastError();
}

}  // namespace

size_t paged_attn_workspace_bytes(int64_t seqs, int64_t tokens, int q_heads, int kv_heads, int head_dim) {
  const int group = q_heads / kv_heads;
  const int dim = padded_dim(head_dim);
  return (needs_few(seqs, tokens, group) ? few_bytes(dim) : 0) + (needs_many(seqs, tokens, group) ? many_bytes(dim) : 0);
}

// HIP takes fewer than 2^32 threads in a dimension of the grid.
bool prompt_attn_fits(const AttnArgs& a) { return prompt_blocks(a) * a.kv_heads * (64 * kPromptWaves) < (1LL << 32); }

hipError_t launch_prompt_attn(const AttnArgs& a, hipStream_t s) {
  const bool wide = padded_dim(a.head_dim) == 128;
  if (a.dtype == kBf16) return wide ? prompt_dp<kBf16, 128>(a, s) : prompt_dp<kBf16, 64>(a, s);
  return wide ? prompt_dp<kFp16, 128>(a, s) : prompt_dp<kFp16, 64>(a, s);
}

template <int DT>
static hipError_t paged_type(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim == 128) return paged_dp<DT, 128, true>(a, s);
  if (a.head_dim > 64) return paged_dp<DT, 128, false>(a, s);
  return a.head_dim == 64 ? paged_dp<DT, 64, true>(a, s) : paged_dp<DT, 64, false>(a, s);
}

hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s) {
  return a.dtype == kBf16 ? paged_type<kBf16>(a, s) : paged_type<kFp16>(a, s);
}

}  // namespace nvfp4
