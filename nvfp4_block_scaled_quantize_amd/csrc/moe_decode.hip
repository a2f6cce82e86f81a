// moe_decode.hip -- a whole routed MoE layer for up to 32 tokens on NVFP4 expert weights, for gfx950:
// router product, sigmoid group top-k (the selection of moe.hip), fc1, activation (ReLU^2 or SwiGLU),
// fc2 and the weighted sum, in five launches (three for one token).
//
//  1. router  : logits[t, e] = x_t . Wr_e in binary32, one workgroup per expert and four tokens; clears the
//               maxima that fc1 takes; BF16 x also as scaled FP16 (below).
//  2. plan    : one workgroup: one wave per token selects its experts; then the entries (an expert and up to 16 of
//               its tokens) and a row of h and o for every pair of token and expert.
//  3. fc1     : h = act(W1_e x) for the rows of every entry, binary32, and each row's largest |h|.
//  4. fc2     : o = W2_e h for the rows of every entry, binary32.
//  5. combine : the weighted sum over each token's o, in rank order.
// One token: fc1 selects by itself (2 us less than a launch for it), and fc2 has all its experts in one
// workgroup, so their sum needs no launch either.
//
// The weights' bytes bound it: each chosen expert's rows are read once (twice with more than 16 tokens), straight
// from memory into registers, the waves of a workgroup splitting K in blocks of 256, and the waves' sums are
// joined through LDS.  A lane's 16 bytes = 32 codes of its row feed four v_mfma_f32_16x16x32_f16: instruction m takes
// codes 8 m .. 8 m + 7 of every lane, and the activation operand the same k.  E2M1 * E4M3 is exact in FP16.
//
// The activations must be FP16 for that.  FP16 x is used as it is.  BF16 x is multiplied by the power
// of two that brings the token's largest value to [2^14, 2^15): exact down to 2^-31 of the largest, what is
// below is off by at most 2^-39 of it.  h (binary32) is brought to the same range by the pair's
// largest h and split into two FP16 numbers, the value and what its rounding left: off by less than 2^-20 of itself or,
// where FP16's smallest step of 2^-24 is more, 2^-38 of the largest (for one token: of the largest h times its factor).
//
// Measured: the kernels' medians in a trace (which adds some 0.4 us to each), the whole layer without one (among other
// calls; with weights that the last cache may hold, and with ones that it cannot), and the weights at the rate of a large
// copy (5.1 TB/s):
// 1 token, 8 of 64 experts, 2048 / 1024, ReLU^2    router 2.6, fc1 9.5, fc2 6.7; 17.9 us;                     3.7 us
// 16 tokens of the same layer                      3.9, plan 5.2, 17.1, 18.4, combine 4.6; 44 to 46 us;       26 us
// 4 tokens, 8 of 128, 4096 / 1536, SwiGLU          4.8, 5.1, 50.0, 27.2, 4.8; 82 to 88 us;                    61 us
// What is above it is the launches' own time, the dependent loads at their starts (4 to 5 us of a large one) and the
// last round of units, which not all workgroups have.
#include "device_common.h"
#include "internal.h"
#include "moe_decode.h"

namespace nvfp4 {

namespace {

constexpr int kMaxT = kMoeDecodeMaxTokens;
constexpr int kMaxK = 16;                    // top_k
constexpr int kMaxPairs = kMaxT * kMaxK;
constexpr int kPerLane = 4;                  // experts <= 256

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// A pair (token, rank) has the number p = token * top_k + rank; its row q of h and o is its place when the
// pairs are sorted by expert.
struct Ws {
  float* logits;      // [T, E]
  uint32_t* xmax;     // [T] largest |x| (binary32 bits)
  uint32_t* hmax;     // [P] largest |h| of row q (binary32 bits)
  float* wts;         // [P] weight of pair p
  int32_t* row_of;    // [P] its row q
  int4* chosen;       // [min(P, 2 E)] {expert, first row, mask of its tokens, entries}, one for up to 16 tokens
  _Float16* xs;       // [T, hidden] scaled x (BF16 only)
  float* h;           // [P, inter]
  float* o;           // [P, hidden]
};

size_t carve(void* base, int T, int E, int P, int hidden, int inter, Ws* w) {
  unsigned char* p = reinterpret_cast<unsigned char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return p + here;
  };
  Ws s;
  s.logits = reinterpret_cast<float*>(take((size_t)T * E * 4));
  s.xmax = reinterpret_cast<uint32_t*>(take((size_t)T * 4));
  s.hmax = reinterpret_cast<uint32_t*>(take((size_t)P * 4));
  s.wts = reinterpret_cast<float*>(take((size_t)P * 4));
  s.row_of = reinterpret_cast<int32_t*>(take((size_t)P * 4));
  s.chosen = reinterpret_cast<int4*>(take((size_t)(P < 2 * E ? P : 2 * E) * 16));
  s.xs = reinterpret_cast<_Float16*>(take((size_t)T * hidden * 2));
  s.h = reinterpret_cast<float*>(take((size_t)P * inter * 4));
  s.o = reinterpret_cast<float*>(take((size_t)P * hidden * 4));
  if (w) *w = s;
  return at;
}

// The power of two that brings a largest value to [2^14, 2^15).
__device__ __forceinline__ int up_exponent(uint32_t bits) {
  const int e = (int)(bits >> 23) - 127;   // -127 for zeros and subnormal numbers
  return 14 - e < 127 ? 14 - e : 127;
}
__device__ __forceinline__ float up_scale(uint32_t bits) { return __builtin_ldexpf(1.0f, up_exponent(bits)); }

// A factor as its fraction (0.5 <= |f| < 1, or 0, inf, NaN) and the power of two beside it: of a global scale and the power
// of two that a sum was scaled by, or of a weight and a global, the quotient or product may leave binary32 where the result
// does not.
struct Factor {
  float f;
  int e;
};
__device__ __forceinline__ Factor split(float x) {
  return Factor{__builtin_amdgcn_frexp_mantf(x), __builtin_amdgcn_frexp_expf(x)};
}
__device__ __forceinline__ float times(float v, const Factor& x) { return __builtin_ldexpf(v * x.f, x.e); }

// ---------------------------------------------------------------- router
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x141>(v);
  v += dpp_f32<0x140>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

template <int DT, int TB>
__global__ void __launch_bounds__(256)
moe_router(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, int T, int E, int hidden, Ws ws, int P) {
  __shared__ float part[4][TB];
  __shared__ float top[4][TB];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int unit0 = (int)((int64_t)(hidden / 8) * e / E), unit1 = (int)((int64_t)(hidden / 8) * (e + 1) / E);
  const int t0 = (int)blockIdx.y * TB;
  if (e == 0 && t0 == 0)
    for (int i = tid; i < P; i += 256) ws.hmax[i] = 0u;
  float sum[TB], big[TB];
#pragma unroll
  for (int j = 0; j < TB; ++j) sum[j] = big[j] = 0.0f;
  for (int u = tid; u < hidden / 8; u += 256) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(wr + (int64_t)e * hidden + 8 * u);
    u32x4 v[TB];
#pragma unroll
    for (int j = 0; j < TB; ++j)
      v[j] = *reinterpret_cast<const u32x4*>(x + (int64_t)(t0 + j < T ? t0 + j : T - 1) * hidden + 8 * u);
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b, c, d;
        unpack2<DT>(w[i], a, b);
        unpack2<DT>(v[j][i], c, d);
        sum[j] = __builtin_fmaf(a, c, sum[j]);
        sum[j] = __builtin_fmaf(b, d, sum[j]);
        big[j] = __builtin_fmaxf(big[j], __builtin_fmaxf(__builtin_fabsf(c), __builtin_fabsf(d)));
      }
  }
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const float s = wave_sum(sum[j]), m = wave_max_dpp(big[j]);
    if (lane == 0) {
      part[wave][j] = s;
      top[wave][j] = m;
    }
  }
  __syncthreads();
  if (tid < TB && t0 + tid < T) {
    ws.logits[(int64_t)(t0 + tid) * E + e] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
    if (e == 0)
      ws.xmax[t0 + tid] = __float_as_uint(__builtin_fmaxf(__builtin_fmaxf(top[0][tid], top[1][tid]),
                                                          __builtin_fmaxf(top[2][tid], top[3][tid])));
  }
  if constexpr (DT == kBf16) {
    // this workgroup's columns of the tokens in FP16
    const int units = unit1 - unit0;
    for (int i = tid; i < units * TB; i += 256) {
      const int j = i / units, u = unit0 + i - j * units;
      if (t0 + j >= T) continue;
      const float scale = up_scale(__float_as_uint(__builtin_fmaxf(__builtin_fmaxf(top[0][j], top[1][j]),
                                                                   __builtin_fmaxf(top[2][j], top[3][j]))));
      const int64_t at = (int64_t)(t0 + j) * hidden + 8 * u;
      const u32x4 v = *reinterpret_cast<const u32x4*>(x + at);
      v8h o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o[2 * q] = (_Float16)(bf16_lo(v[q]) * scale);
        o[2 * q + 1] = (_Float16)(bf16_hi(v[q]) * scale);
      }
      *reinterpret_cast<v8h*>(ws.xs + at) = o;
    }
  }
}

// ---------------------------------------------------------------- selection
// Binary32 numbers as integers in the same order; 0 is below all of them.  NaN ranks with -inf.
__device__ __forceinline__ uint32_t rank_key(float v) {
  if (v != v) v = -__builtin_inff();
  const uint32_t b = __float_as_uint(v);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  const uint32_t u = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  return u > v ? u : v;
}
// Largest over the wave (rows of 16 lanes by lane exchange, then the four rows).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max_dpp<0xB1>(v);
  v = max_dpp<0x4E>(v);
  v = max_dpp<0x141>(v);
  v = max_dpp<0x140>(v);
  uint32_t m = 0u;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t u = (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * r);
    m = u > m ? u : m;
  }
  return m;
}

struct RouteArgs {
  const float* bias;
  int T, E, top_k, n_group, topk_group, norm;
  float scaling;
};

// The two largest of a group, joined with a neighbour's.
__device__ __forceinline__ void join_two(float& v1, float& v2, float u1, float u2) {
  v2 = __builtin_fmaxf(__builtin_fminf(v1, u1), __builtin_fmaxf(v2, u2));
  v1 = __builtin_fmaxf(v1, u1);
}

// One wave scores one token's experts: lane l holds experts l + 64 i, i < N, their scores s and the keys of their biased
// scores.  A group's score is the sum of its two best biased scores, and the experts outside the best groups have
// the key 0.  Groups of 2, 4, .. 64 experts are lanes next to one another; others go through LDS (sb, sg: E and
// n_group entries).
template <int N>
__device__ __forceinline__ void score_token(const RouteArgs& a, const float* __restrict__ logits, int t, float* sb,
                                            float* sg, float (&s)[N], uint32_t (&key)[N]) {
  const int lane = threadIdx.x & 63;
  const int gsize = a.E / a.n_group;
  const float ninf = -__builtin_inff();
  float b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 64 * i;
    s[i] = 0.0f;
    b[i] = ninf;
    key[i] = 0u;
    if (e < a.E) {
      s[i] = sigmoid_f32(logits[(int64_t)t * a.E + e]);
      b[i] = s[i] + a.bias[e];
      if (b[i] != b[i]) b[i] = ninf;
      key[i] = rank_key(b[i]);
    }
  }
  if (a.n_group > 1) {
    float mine[N];   // the score of each expert's group
    int before[N];
#pragma unroll
    for (int i = 0; i < N; ++i) before[i] = 0;
    if ((gsize & (gsize - 1)) == 0 && gsize <= 64) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v1 = b[i], v2 = ninf;
        if (gsize >= 2) join_two(v1, v2, dpp_f32<0xB1>(v1), dpp_f32<0xB1>(v2));
        if (gsize >= 4) join_two(v1, v2, dpp_f32<0x4E>(v1), dpp_f32<0x4E>(v2));
        if (gsize >= 8) join_two(v1, v2, dpp_f32<0x141>(v1), dpp_f32<0x141>(v2));
        if (gsize >= 16) join_two(v1, v2, dpp_f32<0x140>(v1), dpp_f32<0x140>(v2));
        if (gsize >= 32) join_two(v1, v2, __shfl_xor(v1, 16, 64), __shfl_xor(v2, 16, 64));
        if (gsize >= 64) join_two(v1, v2, __shfl_xor(v1, 32, 64), __shfl_xor(v2, 32, 64));
        mine[i] = gsize > 1 ? v1 + v2 : v1;
        if (mine[i] != mine[i]) mine[i] = ninf;
      }
      int j = 0;   // group number, and its score
#pragma unroll
      for (int k = 0; k < N; ++k)
        for (int l = 0; l < 64 && j < a.n_group; l += gsize, ++j) {
          const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine[k]), l));
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const bool earlier = 64 * k + l + gsize <= lane + 64 * i;   // an earlier group than the lane's
            before[i] += (v > mine[i] || (v == mine[i] && earlier)) ? 1 : 0;
          }
        }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane + 64 * i < a.E) sb[lane + 64 * i] = b[i];
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // only this wave reads what it wrote
      for (int g = lane; g < a.n_group; g += 64) {
        float v1 = ninf, v2 = ninf;
        for (int j = 0; j < gsize; ++j) join_two(v1, v2, sb[g * gsize + j], ninf);
        float sum = gsize > 1 ? v1 + v2 : v1;
        if (sum != sum) sum = ninf;
        sg[g] = sum;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (lane + 64 * i >= a.E) continue;
        const int g = (lane + 64 * i) / gsize;
        for (int j = 0; j < a.n_group; ++j) before[i] += (sg[j] > sg[g] || (sg[j] == sg[g] && j < g)) ? 1 : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (before[i] >= a.topk_group) key[i] = 0u;
  }
}

// One wave takes a token's top_k experts one after the other, ties to the lower index: lane k receives the one of
// rank k and its weight.
template <int N>
__device__ __forceinline__ void select_token(const RouteArgs& a, const float* __restrict__ logits, int t, float* sb,
                                             float* sg, int& id, float& weight) {
  const int lane = threadIdx.x & 63;
  float s[N];
  uint32_t key[N];
  score_token<N>(a, logits, t, sb, sg, s, key);
  float sum = 0.0f, mine = 0.0f;
  int chosen = 0;
  for (int k = 0; k < a.top_k; ++k) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = key[i] > m ? key[i] : m;
    m = wave_max_u32(m);
    int e = -1;
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t hit = __ballot(key[i] == m);
      if (e < 0 && hit != 0) {
        const int l = __builtin_ctzll(hit);
        e = l + 64 * i;
        w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s[i]), l));
        if (lane == l) key[i] = 0u;
      }
    }
    sum = sum + w;
    if (lane == k) {
      mine = w;
      chosen = e;
    }
  }
  id = chosen;
  weight = (a.norm ? mine / sum : mine) * a.scaling;
}

// ---------------------------------------------------------------- plan
constexpr int kPlanWaves = 16;

template <int N>
__global__ void __launch_bounds__(64 * kPlanWaves) moe_plan(RouteArgs a, Ws ws, int32_t* ids_out, float* w_out) {
  __shared__ float scratch[kPlanWaves][2][64 * N];
  __shared__ int32_t ids[kMaxPairs];
  __shared__ uint32_t takers[256];   // tokens that chose the expert
  __shared__ int first[256];         // its first row
  __shared__ int sums[2][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid < 256) takers[tid] = 0u;
  __syncthreads();
  for (int t = wave; t < a.T; t += kPlanWaves) {
    int id;
    float w;
    select_token<N>(a, ws.logits, t, scratch[wave][0], scratch[wave][1], id, w);
    if (lane < a.top_k) {
      const int p = t * a.top_k + lane;
      ids[p] = id;
      ws.wts[p] = w;
      if (ids_out) ids_out[p] = id;
      if (w_out) w_out[p] = w;
      atomicOr(&takers[id], 1u << t);
    }
  }
  __syncthreads();
  // sums over the experts before each: rows and entries
  uint32_t m = 0u;
  int rows = 0, some = 0, r = 0, u = 0;   // some: entries of the expert, up to 16 tokens each
  if (tid < 256) {
    m = takers[tid];
    r = rows = __popc(m);
    u = some = (rows + 15) / 16;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(r, off, 64), y = __shfl_up(u, off, 64);
      if (lane >= off) {
        r += x;
        u += y;
      }
    }
    if (lane == 63) {
      sums[0][wave] = r;
      sums[1][wave] = u;
    }
  }
  __syncthreads();
  int n = 0;
  if (tid < 256) {
    int br = 0, bu = 0;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (v == wave) {
        br = r - rows;
        bu = u - some;
      }
      n += sums[1][v];
    }
    for (int v = 0; v < wave; ++v) {
      br += sums[0][v];
      bu += sums[1][v];
    }
    first[tid] = br;
    uint32_t rest = m;   // the tokens after the 16th
    for (int i = 0; i < 16; ++i) rest &= rest - 1u;
    if (some > 0) ws.chosen[bu] = make_int4(tid, br, (int)(m ^ rest), n);
    if (some > 1) ws.chosen[bu + 1] = make_int4(tid, br + 16, (int)rest, n);
  }
  __syncthreads();
  for (int p = tid; p < a.T * a.top_k; p += 64 * kPlanWaves) {
    const int e = ids[p], t = p / a.top_k;
    ws.row_of[p] = first[e] + __popc(takers[e] & ((1u << t) - 1u));
  }
}

// ---------------------------------------------------------------- expert rows
__device__ __forceinline__ v8h dequant8(uint32_t codes, _Float16 s16) {
  const v2h s2 = {s16, s16};
  const v2h p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s2;
  const v2h p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s2;
  const v2h p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s2;
  const v2h p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s2;
  v8h r;
  r[0] = p0[0]; r[1] = p0[1]; r[2] = p1[0]; r[3] = p1[1];
  r[4] = p2[0]; r[5] = p2[1]; r[6] = p3[0]; r[7] = p3[1];
  return r;
}

// A lane's part of a 256-k block of 16 rows: 64 codes in two halves and their four E4M3 bytes, as loaded.
struct Piece {
  u32x4 codes[2];
  uint32_t sf[2];   // plain: sf[0] holds all four; TW: two each
};

// k of half d of lane group g in block c.  Plain rows: a lane's 64 k follow one another, so the four lanes
// of a row read its whole 128-byte line and one dword of scales each.  TW (below): two chunks of 128.
template <bool TW>
__device__ __forceinline__ int first_k(int c, int d, int g) {
  return TW ? 256 * c + 128 * d + 32 * g : 256 * c + 64 * g + 32 * d;
}

// Expert weights [E, rows, K]: plain (codes [rows, K / 2], E4M3 [rows, K / 16]) or TW, the layout of
// nvfp4_pretile_weight of the stacked [E rows, K] matrix, in which a 128-k chunk of 16 rows is 1 KiB of codes
// and 128 B of E4M3 pairs in lane order.  K % 64 = 0 (TW: 128), so in the last block a lane's half is whole or
// past the row; there it reads the block's start again, and scales() is 0.  Not live: one address for all lanes.  (Nothing is done with what is
// loaded before it is used: the loads after these must not wait.)
template <bool TW>
__device__ __forceinline__ void load_piece(const uint8_t* __restrict__ w, const uint8_t* __restrict__ sf, int64_t row16,
                                           int c, int K, int lane, bool live, Piece& p) {
  if constexpr (TW) {
    const int64_t tile = (row16 / 16) * (K / 128) + 2 * c;
    const int64_t next = 256 * c + 128 < K ? tile + 1 : tile;
    const int l = live ? lane : 0;
    p.codes[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + tile * 1024 + 16 * l));
    p.codes[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + next * 1024 + 16 * l));
    p.sf[0] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(sf + tile * 128 + 2 * l));
    p.sf[1] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(sf + next * 128 + 2 * l));
  } else {
    const int g = lane >> 4;
    const bool in = live && 256 * c + 64 * g < K;
    const int64_t row = row16 + (live ? lane & 15 : 0);
    const uint8_t* at = w + row * (K / 2) + 128 * c + (in ? 32 * g : 0);
    p.codes[0] = *reinterpret_cast<const u32x4*>(at);
    p.codes[1] = *reinterpret_cast<const u32x4*>(at + 16);
    p.sf[0] = *reinterpret_cast<const uint32_t*>(sf + row * (K / 16) + 16 * c + (in ? 4 * g : 0));
  }
}
// The pieces loaded ahead, once they are there.  (A plain copy ends up after the next loads, at the loop's end, and
// waits for them.)
__device__ __forceinline__ uint32_t take(uint32_t from) {
  uint32_t to;
  asm volatile("v_mov_b32 %0, %1" : "=v"(to) : "v"(from) : "memory");
  return to;
}
template <bool TW>
__device__ __forceinline__ void take(Piece& to, const Piece& from) {
#pragma unroll
  for (int d = 0; d < 2; ++d) {
#pragma unroll
    for (int q = 0; q < 4; ++q) to.codes[d][q] = take(from.codes[d][q]);
    if (TW || d == 0) to.sf[d] = take(from.sf[d]);
  }
}

// The two scales of half d.
template <bool TW>
__device__ __forceinline__ void scales(const Piece& p, int d, int c, int K, int g, _Float16 (&s)[2]) {
  const uint32_t b = first_k<TW>(c, d, g) < K ? (TW ? p.sf[d] : p.sf[0] >> (16 * d)) : 0u;
  s[0] = (_Float16)__builtin_amdgcn_cvt_f32_fp8((int)b, 0);
  s[1] = (_Float16)__builtin_amdgcn_cvt_f32_fp8((int)b, 1);
}

struct FcArgs {
  const void* src;       // FC 1: x or its scaled form [T, hidden]; FC 2: h
  const uint8_t* w;
  const uint8_t* sf;
  const float* g;
  int rows, K;           // rows of one expert, and their length
  int inter, hidden;
  int scaled;            // FC 1: src is scaled by up_scale(xmax)
  RouteArgs route;
  int32_t* ids_out;      // FC 1, one token
  float* w_out;
  void* out;             // FC 2: [T, hidden]
  int out_type;
  Ws ws;
};

// The activations of one half of a block for 16 token slots as they are stored: lane (slot, g) holds 32 k,
// as FP16 or binary32; zeros for slots without a token and past K.
template <int FC>
struct RawAct {
  u32x4 v[FC == 1 ? 4 : 8];
};
template <int FC>
__device__ __forceinline__ void load_act(const void* src, int64_t row, bool there, int K, int k0, RawAct<FC>& r) {
  constexpr int kN = FC == 1 ? 4 : 8, kBytes = FC == 1 ? 2 : 4;
#pragma unroll
  for (int m = 0; m < kN; ++m) r.v[m] = u32x4{0u, 0u, 0u, 0u};
  if (there && k0 < K) {
    const u32x4* p = reinterpret_cast<const u32x4*>((const char*)src + (row * K + k0) * kBytes);
#pragma unroll
    for (int m = 0; m < kN; ++m) r.v[m] = p[m];
  }
}

// What the FP16 numbers p leave of a and b.  Nothing of an infinity: inf - inf is NaN, of which and a number the maximum is
// the number, and beside the infinity that changes no sum.  (A remainder is below 2^-10 of 2^15.)
__device__ __forceinline__ v2h rest2(float a, float b, const v2h& p) {
  const v2h q = __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_pkrtz(a - (float)p[0], b - (float)p[1]));
  const v2h least = {(_Float16)-64.0f, (_Float16)-64.0f};
  return __builtin_elementwise_max(q, least);
}

// Operands of instruction m.  FC 1: as stored.  FC 2: scaled and split; both roundings are toward zero, the first
// leaves less than 2^-10 of the value (of normal numbers), the second less than 2^-10 of that or 2^-24.
template <int FC>
__device__ __forceinline__ void act_operand(const RawAct<FC>& r, int m, float scale, v8h& hi, v8h& lo) {
  if constexpr (FC == 1) {
    hi = __builtin_bit_cast(v8h, r.v[m]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = __uint_as_float(r.v[2 * m + i / 2][2 * (i & 1)]) * scale;
      const float b = __uint_as_float(r.v[2 * m + i / 2][2 * (i & 1) + 1]) * scale;
      const v2h p = __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_pkrtz(a, b));
      const v2h q = rest2(a, b, p);
      hi[2 * i] = p[0];
      hi[2 * i + 1] = p[1];
      lo[2 * i] = q[0];
      lo[2 * i + 1] = q[1];
    }
  }
}

// 16 RT weight rows of an entry (an expert and up to 16 of its tokens) are a unit; the units of all entries, in
// order, are divided evenly among the workgroups (one unit to a workgroup instead: fc1 of 16 tokens 31 us, not
// 18), so one has a few units of one entry or two.  Its waves take the
// 256-k blocks of a unit in turn, each loads the weights of its next block (of this unit or the next) before it
// works on the one at hand, and their sums are joined through LDS, in two buffers: one barrier for a unit.
// KEEP: a wave has one block of every unit, and holds its activations for all units of the entry.
template <int FC, bool GATED, bool TW, int RT, int NW, bool KEEP>
__global__ void __launch_bounds__(64 * NW, 2) moe_expert_rows(FcArgs a, int units) {
  __shared__ v4f part[2][NW][RT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, grp = lane >> 4;

  const int n = __builtin_amdgcn_readfirstlane(a.ws.chosen[0].w);
  auto entry = [&](int y) __attribute__((always_inline)) {
    int4 v = a.ws.chosen[y];
    v.x = __builtin_amdgcn_readfirstlane(v.x);
    v.y = __builtin_amdgcn_readfirstlane(v.y);
    v.z = __builtin_amdgcn_readfirstlane(v.z);
    return v;
  };
  const uint32_t total = (uint32_t)n * (uint32_t)units, each = total / gridDim.x, more_by_one = total - each * gridDim.x;
  const int lo = (int)(blockIdx.x * each + (blockIdx.x < more_by_one ? blockIdx.x : more_by_one));
  const int hi = lo + (int)each + (blockIdx.x < more_by_one ? 1 : 0);
  if (lo >= hi) return;   // the whole workgroup
  int y = (int)((uint32_t)lo / (uint32_t)units), x = lo - y * units;
  int4 mine = entry(y), after = entry(y + 1 < n ? y + 1 : y);

  // weight rows of a unit's RT groups of 16: consecutive rows, or for SwiGLU in fc1 gate rows, then the up rows
  constexpr int kCols = (GATED ? RT / 2 : RT) * 16;   // results per token
  auto row16 = [&](int e, int x, int i) __attribute__((always_inline)) {
    const int r = !GATED || i < RT / 2 ? x * kCols + 16 * i : a.inter + x * kCols + 16 * (i - RT / 2);
    return (int64_t)e * a.rows + r;
  };
  const int blocks = (a.K + 255) / 256;

  // what belongs to an entry: lane (slot r16, grp) has the slot's token (slot s: the s-th of the mask) or row of h, the
  // bits of the largest value that it was, or will be, scaled by, what turns its sums into results, and with KEEP its operands
  int ns = 0;
  bool there = false;
  int64_t arow = 0;
  uint32_t top = 0u;
  float big = 0.0f, ge = 0.0f, rest = 1.0f;   // fc2: times ge, times rest
  RawAct<FC> raw[2];
  v8h kept[2][4], kept_lo[2][4];
  auto load_acts = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < 2; ++d) load_act<FC>(a.src, arow, there, a.K, first_k<TW>(c, d, grp), raw[d]);
  };
  auto enter = [&]() __attribute__((always_inline)) {
    const uint32_t tokens = (uint32_t)mine.z;
    ns = __popc(tokens);
    there = r16 < ns;
    if constexpr (FC == 1) {
      uint32_t m = tokens;
#pragma unroll
      for (int i = 0; i < 15; ++i) m = i < r16 ? m & (m - 1) : m;
      arow = there ? __builtin_ctz(m) : 0;
      top = a.scaled ? a.ws.xmax[arow] : 0u;
    } else {
      arow = mine.y + (there ? r16 : 0);
      top = a.ws.hmax[arow];
    }
    ge = a.g[mine.x];
    if constexpr (FC == 2) {
      const Factor f = split(ge);
      const int e = f.e - up_exponent(top);   // half of it each: neither leaves binary32 before the result does
      ge = __builtin_ldexpf(f.f, e / 2);
      rest = __builtin_ldexpf(1.0f, e - e / 2);
    }
    asm volatile("" : "+v"(top), "+v"(ge), "+v"(rest));   // waited for here, and not in a unit with loads on their way
    big = 0.0f;
    if constexpr (KEEP) {
      if (wave < blocks) {
        load_acts(wave);
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
          for (int m = 0; m < 4; ++m)
            act_operand<FC>(raw[d], m, FC == 2 ? up_scale(top) : 1.0f, kept[d][m], kept_lo[d][m]);
      }
    }
  };
  // fc1: the entry's largest |h| of each token
  auto leave = [&]() __attribute__((always_inline)) {
    if constexpr (FC == 1) {
      big = __builtin_fmaxf(big, __shfl_xor(big, 16, 64));
      big = __builtin_fmaxf(big, __shfl_xor(big, 32, 64));
      if (wave < kCols / 16 && grp == 0 && there) atomicMax(a.ws.hmax + mine.y + r16, __float_as_uint(big));
    }
  };

  Piece ahead[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    load_piece<TW>(a.w, a.sf, row16(mine.x, x, i), wave < blocks ? wave : 0, a.K, lane, true, ahead[i]);
  enter();
  for (int u = lo; u < hi; ++u) {
    v4f acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const bool crosses = x + 1 == units;
    for (int c = wave; c < blocks; c += NW) {
      Piece w[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) take<TW>(w[i], ahead[i]);
      if constexpr (!KEEP) load_acts(c);
      // the next block; after the last one the lanes read one piece, and nothing uses it (a branch here would make
      // the waits for the activations wait for these loads as well)
      const bool more = !KEEP && c + NW < blocks, live = more || u + 1 < hi;
      const int ne = more || !crosses ? mine.x : after.x, nx = more ? x : crosses ? 0 : x + 1;
#pragma unroll
      for (int i = 0; i < RT; ++i)
        load_piece<TW>(a.w, a.sf, row16(ne, nx, i), more ? c + NW : wave, a.K, lane, live, ahead[i]);
      __builtin_amdgcn_sched_barrier(0);   // issued before the work, not after it
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        _Float16 sc[RT][2];
#pragma unroll
        for (int i = 0; i < RT; ++i) scales<TW>(w[i], d, c, a.K, grp, sc[i]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          v8h hi8, lo8;
          if constexpr (KEEP) {
            hi8 = kept[d][m];
            lo8 = kept_lo[d][m];
          } else {
            act_operand<FC>(raw[d], m, FC == 2 ? up_scale(top) : 1.0f, hi8, lo8);
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const v8h wv = dequant8(w[i].codes[d][m], sc[i][m / 2]);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, hi8, acc[i], 0, 0, 0);
            if constexpr (FC == 2) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, lo8, acc[i], 0, 0, 0);
          }
        }
      }
    }
    v4f(*sums)[RT][64] = part[(u - lo) & 1];
#pragma unroll
    for (int i = 0; i < RT; ++i) sums[wave][i][lane] = acc[i];
    // LDS only: the loads ahead stay in flight
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    auto joined = [&](int tile) __attribute__((always_inline)) {
      v4f s = sums[0][tile][lane];
#pragma unroll
      for (int v = 1; v < NW; ++v) {
        const v4f q = sums[v][tile][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += q[i];
      }
      return s;
    };
    // results: lane (slot r16, columns 4 grp .. + 3) of a tile, one tile a wave
    static_assert(kCols / 16 <= NW, "one tile a wave");
    if (wave < kCols / 16) {
      v4f v = joined(wave);
      v4f up;
      if constexpr (GATED) up = joined(wave + RT / 2);
      const int col = x * kCols + 16 * wave + 4 * grp;
      if constexpr (FC == 1) {
        // sums are below 2^43, and h above 2^-126 comes of a result above 2^-63: f stays above 2^-106 where it matters
        const float f = a.scaled ? ge / up_scale(top) : ge;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] = GATED ? swiglu_f32(v[q] * f, up[q] * f) : relu2_or_nan_f32(v[q] * f);
          big = __builtin_fmaxf(big, __builtin_fabsf(v[q]));
        }
        if (there) *reinterpret_cast<v4f*>(a.ws.h + (int64_t)(mine.y + r16) * a.inter + col) = v;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = v[q] * ge * rest;
        if (there) *reinterpret_cast<v4f*>(a.ws.o + (int64_t)(mine.y + r16) * a.hidden + col) = v;
      }
    }
    ++x;
    if (crosses && u + 1 < hi) {
      leave();
      x = 0;
      ++y;
      mine = after;
      after = entry(y + 1 < n ? y + 1 : y);
      enter();
    }
  }
  leave();
}

// out[t] = sum over the token's experts, in rank order, of weight times o, binary32: a thread has four columns.
__global__ void __launch_bounds__(128) moe_combine(FcArgs a) {
  const int t = blockIdx.y, top_k = a.route.top_k;
  const int col = ((int)blockIdx.x * 128 + (int)threadIdx.x) * 4;
  if (col >= a.hidden) return;
  v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int k = 0; k < top_k; ++k) {
    const v4f v = *reinterpret_cast<const v4f*>(a.ws.o + (int64_t)a.ws.row_of[t * top_k + k] * a.hidden + col);
    const float wk = a.ws.wts[t * top_k + k];
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = __builtin_fmaf(wk, v[q], s[q]);
  }
  uint16_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = round16(s[q], a.out_type);
  const u32x2 v = {o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16};
  *reinterpret_cast<u32x2*>((uint16_t*)a.out + (int64_t)t * a.hidden + col) = v;
}

// fc1 for one token: 32 weight rows of one of its experts a workgroup.  Every workgroup selects by itself: all waves
// score the experts, each ranks them against its share of the keys, and the sums of the ranks are the places;
// experts of the same key have the same rank, and take the places from there on in order.  The last wave of the first
// workgroup lists the selection for fc2.  All 16 columns of the matrix instruction are the token.
constexpr int kOneRowsWaves = 8;
template <bool GATED, bool TW, int N>
__global__ void __launch_bounds__(64 * kOneRowsWaves) moe_one_rows(FcArgs a) {
  constexpr int NW = kOneRowsWaves;
  __shared__ float scratch[NW][2][64 * N];
  __shared__ int ranks[NW][64 * N];
  __shared__ float part[NW][32];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = lane >> 4, y = blockIdx.y, top_k = a.route.top_k;
  const int blocks = (a.K + 255) / 256;
  float s[N];
  uint32_t key[N];
  score_token<N>(a.route, a.ws.logits, 0, scratch[wave][0], scratch[wave][1], s, key);
  {
    int rank[N];
#pragma unroll
    for (int i = 0; i < N; ++i) rank[i] = 0;
    // wave w: the experts 64 k + 8 w .. + 7 of every k
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int j = 0; j < 64 / NW; ++j) {
        const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)key[k], wave * (64 / NW) + j);
#pragma unroll
        for (int i = 0; i < N; ++i) rank[i] += other > key[i] ? 1 : 0;
      }
#pragma unroll
    for (int i = 0; i < N; ++i) ranks[wave][64 * i + lane] = rank[i];
  }
  __syncthreads();
  int rank[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int r = 0;
#pragma unroll
    for (int v = 0; v < NW; ++v) r += ranks[v][64 * i + lane];
    rank[i] = key[i] != 0u ? r : 64 * N;
  }
  // place k: the first of those of the largest rank that is not above k, after as many as it has places before k
  auto at_place = [&](int k) __attribute__((always_inline)) {
    for (int r = k; r >= 0; --r) {
      int skip = k - r, e = -1;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        uint64_t hit = __ballot(rank[i] == r);
        if (e >= 0 || hit == 0) continue;
        for (; skip > 0 && hit != 0; --skip) hit &= hit - 1;
        if (hit != 0) e = 64 * i + __builtin_ctzll(hit);
      }
      if (e >= 0) return e;
    }
    return 0;
  };
  const int e = at_place(y);

  v4f acc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t row = (int64_t)e * a.rows + (int64_t)blockIdx.x * (GATED ? 16 : 32);
  for (int c = wave; c < blocks; c += NW) {
    Piece w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      load_piece<TW>(a.w, a.sf, row + (GATED ? a.inter : 16) * i, c, a.K, lane, true, w[i]);
    RawAct<1> x[2];
#pragma unroll
    for (int d = 0; d < 2; ++d) load_act<1>(a.src, 0, true, a.K, first_k<TW>(c, d, grp), x[d]);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      _Float16 sc[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) scales<TW>(w[i], d, c, a.K, grp, sc[i]);
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(dequant8(w[i].codes[d][m], sc[i][m / 2]),
                                                          __builtin_bit_cast(v8h, x[d].v[m]), acc[i], 0, 0, 0);
    }
  }
  if ((lane & 15) == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<v4f*>(&part[wave][16 * i + 4 * grp]) = acc[i];
  }
  __syncthreads();
  if (wave == 0) {
    constexpr int kCols = GATED ? 16 : 32;
    float v = part[0][lane & 31];
#pragma unroll
    for (int q = 1; q < NW; ++q) v += part[q][lane & 31];
    Factor f = split(a.g[e]);
    if (a.scaled) f.e -= up_exponent(a.ws.xmax[0]);
    float h;
    if constexpr (GATED) h = swiglu_f32(times(v, f), times(__shfl_xor(v, 16, 64), f));
    else h = relu2_or_nan_f32(times(v, f));
    if (lane < kCols) a.ws.h[(int64_t)y * a.inter + (int64_t)blockIdx.x * kCols + lane] = h;
    const uint32_t big = wave_max_u32(lane < kCols ? __float_as_uint(__builtin_fmaxf(__builtin_fabsf(h), 0.0f)) : 0u);
    if (lane == 0) atomicMax(a.ws.hmax + y, big);
  }
  if (blockIdx.x == 0 && y == 0 && wave == NW - 1) {
    float sum = 0.0f, mine = 0.0f;
    int id = 0;
    for (int k = 0; k < top_k; ++k) {
      const int ek = at_place(k);
      float w = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (ek / 64 == i) w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s[i]), ek % 64));
      sum = sum + w;
      if (lane == k) {
        mine = w;
        id = ek;
      }
    }
    if (lane < top_k) {
      const float w = (a.route.norm ? mine / sum : mine) * a.route.scaling;
      a.ws.chosen[lane] = make_int4(id, lane, 1, top_k);
      a.ws.wts[lane] = w;
      if (a.ids_out) a.ids_out[lane] = id;
      if (a.w_out) a.w_out[lane] = w;
    }
  }
}

// fc2 and the sum for one token: a workgroup has 16 output columns of all its experts, as one product over the
// experts' h one after the other, each h already times weight and scale of its expert.  The 16 waves take the (expert,
// 256-k block) steps in turn, two at a time.  A wave converts the 256 h of a step once (4 a lane) and hands them to its
// lanes through LDS; all 16 columns of the matrix instruction are the same token.
constexpr int kOneWaves = 16;
template <bool TW>
__global__ void __launch_bounds__(64 * kOneWaves) moe_one_out(FcArgs a) {
  __shared__ __attribute__((aligned(16))) _Float16 acts[kOneWaves][2][2][256];   // wave, step of two, high and low part
  __shared__ float part[kOneWaves][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = lane >> 4, top_k = a.route.top_k;
  const int blocks = (a.K + 255) / 256, steps = top_k * blocks;
  const int k = lane < top_k ? lane : 0;
  const int e = a.ws.chosen[k].x;
  const Factor fw = split(a.ws.wts[k]), fg = split(a.g[e]);
  const Factor f{fw.f * fg.f, fw.e + fg.e};
  // the largest h times its factor goes to [2^14, 2^15): the exponents of the products, and the largest of them (|e| < 512)
  const uint32_t big = __float_as_uint(__uint_as_float(a.ws.hmax[k]) * f.f) & 0x7FFFFFFFu;
  const int up = 14 + 512 - (int)wave_max_u32(big != 0u ? (uint32_t)((int)(big >> 23) - 127 + f.e + 512) : 0u);
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = wave; s0 < steps; s0 += 2 * kOneWaves) {
    Piece w[2];
    v4f h[2];
    Factor fk[2];
    int c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = s0 + i * kOneWaves < steps ? s0 + i * kOneWaves : s0, rank = s / blocks;
      c[i] = s - rank * blocks;
      const int ek = __builtin_amdgcn_readlane(e, rank);
      fk[i].f = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f.f), rank));
      fk[i].e = __builtin_amdgcn_readlane(f.e, rank) + up;
      load_piece<TW>(a.w, a.sf, (int64_t)ek * a.rows + 16 * (int)blockIdx.x, c[i], a.K, lane, true, w[i]);
      const int at = 256 * c[i] + 4 * lane;
      h[i] = *reinterpret_cast<const v4f*>(a.ws.h + (int64_t)rank * a.inter + (at < a.K ? at : 0));
      if (at >= a.K) h[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const float v0 = times(h[i][q], fk[i]), v1 = times(h[i][q + 1], fk[i]);
        const v2h p = __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_pkrtz(v0, v1));
        const v2h r = rest2(v0, v1, p);
        *reinterpret_cast<v2h*>(&acts[wave][i][0][4 * lane + q]) = p;
        *reinterpret_cast<v2h*>(&acts[wave][i][1][4 * lane + q]) = r;
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // only this wave reads what it wrote
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i > 0 && s0 + kOneWaves >= steps) break;   // the whole wave
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        _Float16 sc[2];
        scales<TW>(w[i], d, c[i], a.K, grp, sc);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const v8h wv = dequant8(w[i].codes[d][m], sc[m / 2]);
          const int at = first_k<TW>(0, d, grp) + 8 * m;
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, *reinterpret_cast<const v8h*>(&acts[wave][i][0][at]), acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, *reinterpret_cast<const v8h*>(&acts[wave][i][1][at]), acc, 0, 0, 0);
        }
      }
    }
    asm volatile("" ::: "memory");
  }
  if ((lane & 15) == 0) *reinterpret_cast<v4f*>(&part[wave][4 * grp]) = acc;
  __syncthreads();
  if (tid >= 16) return;
  float s = part[0][tid];
#pragma unroll
  for (int v = 1; v < kOneWaves; ++v) s += part[v][tid];
  s = __builtin_ldexpf(s, -up);
  ((uint16_t*)a.out)[16 * (int)blockIdx.x + tid] = round16(s, a.out_type);
}

template <int DT>
void launch_router(const MoeDecodeArgs& m, const Ws& ws, int P, hipStream_t s) {
  const uint16_t* x = reinterpret_cast<const uint16_t*>(m.x);
  const uint16_t* wr = reinterpret_cast<const uint16_t*>(m.router);
  if (m.tokens == 1) moe_router<DT, 1><<<dim3(m.experts), dim3(256), 0, s>>>(x, wr, m.tokens, m.experts, m.hidden, ws, P);
  else moe_router<DT, 4><<<dim3(m.experts, (m.tokens + 3) / 4), dim3(256), 0, s>>>(x, wr, m.tokens, m.experts, m.hidden, ws, P);
}

// Eight waves where a row is long enough for them (K = 2048: fc1 of 16 tokens 18 us, with four 24 us), else four: one or
// two workgroups to a compute unit (`slots`); more of them at a time divide the units worse (4 tokens of 64 experts: 33 us,
// twice as many 39 us).
//
// 32 weight rows to a unit, 64 for long rows (more than a block for every wave, so that activations are read again with
// every unit) where that leaves three units to a workgroup.  Whole layers, hidden = inter, one token for each expert, us,
// with 32 / 64 rows:
//   K = 2304: 16 experts (2.2 units each) 52 / 56, 24 (3.4) 68 / 65, 32 (4.5) 84 / 80, 64 (9) 150 / 126;
//   K = 2112: 16 (2.1) 51 / 55, 24 (3.1) 62 / 61, 64 (8.2) 139 / 122;  K = 4096: 16 (4) 107 / 100, 48 (12) 274 / 226.
// Shorter rows, where a wave holds its activations: 64 rows are never better.  K = 2048: 16 experts (2) 36 / 44, 48 (6)
// 62 / 68, 128 (16) 125 / 139;  K = 1280: 48 (3.8) 40 / 42, 152 (12) 91 / 91;  K = 1024: 64 (2) 35 / 42, 256 (8) 89 / 91.
template <int FC, bool GATED, bool TW>
void launch_rows(const FcArgs& a, int experts, hipStream_t s) {
  const int blocks = (a.K + 255) / 256, slots = blocks <= 4 ? 512 : 256;
  const bool wide = blocks > 8 && (int64_t)(a.rows / 64) * experts >= 3 * slots;
  const int units = a.rows / (wide ? 64 : 32);
  const int64_t most = (int64_t)units * experts;
  const dim3 grid((unsigned)(most < slots ? most : slots));
  if (blocks <= 4) moe_expert_rows<FC, GATED, TW, 2, 4, true><<<grid, dim3(256), 0, s>>>(a, units);
  else if (blocks <= 8) moe_expert_rows<FC, GATED, TW, 2, 8, true><<<grid, dim3(512), 0, s>>>(a, units);
  else if (!wide) moe_expert_rows<FC, GATED, TW, 2, 8, false><<<grid, dim3(512), 0, s>>>(a, units);
  else moe_expert_rows<FC, GATED, TW, 4, 8, false><<<grid, dim3(512), 0, s>>>(a, units);
}

template <bool GATED, bool TW>
void launch_one_rows(const FcArgs& a, hipStream_t s) {
  const dim3 grid(a.rows / 32, a.route.top_k), block(64 * kOneRowsWaves);
  if (a.route.E <= 64) moe_one_rows<GATED, TW, 1><<<grid, block, 0, s>>>(a);
  else moe_one_rows<GATED, TW, kPerLane><<<grid, block, 0, s>>>(a);
}

template <bool TW>
void launch_layer(const MoeDecodeArgs& m, const Ws& ws, hipStream_t s) {
  const int P = m.tokens * m.top_k;
  const int experts = P < m.experts ? P : m.experts;   // at most so many are chosen
  const bool gated = m.act == kActSwiglu;
  FcArgs a{};
  a.route = RouteArgs{m.bias, m.tokens, m.experts, m.top_k, m.n_group, m.topk_group, m.norm, m.scaling};
  a.ids_out = m.ids_out;
  a.w_out = m.w_out;
  a.inter = m.inter;
  a.hidden = m.hidden;
  a.ws = ws;
  a.out = m.out;
  a.out_type = m.dtype;
  if (m.tokens > 1) {
    const dim3 block(64 * kPlanWaves);
    if (m.experts <= 64) moe_plan<1><<<dim3(1), block, 0, s>>>(a.route, ws, m.ids_out, m.w_out);
    else if (m.experts <= 128) moe_plan<2><<<dim3(1), block, 0, s>>>(a.route, ws, m.ids_out, m.w_out);
    else moe_plan<kPerLane><<<dim3(1), block, 0, s>>>(a.route, ws, m.ids_out, m.w_out);
  }
  a.scaled = m.dtype == kBf16;
  a.src = a.scaled ? (const void*)ws.xs : m.x;
  a.w = m.w1;
  a.sf = m.w1_sf;
  a.g = m.w1_g;
  a.rows = gated ? 2 * m.inter : m.inter;
  a.K = m.hidden;
  if (m.tokens == 1) {
    if (gated) launch_one_rows<true, TW>(a, s);
    else launch_one_rows<false, TW>(a, s);
  } else {
    if (gated) launch_rows<1, true, TW>(a, experts, s);
    else launch_rows<1, false, TW>(a, experts, s);
  }
  a.src = ws.h;
  a.w = m.w2;
  a.sf = m.w2_sf;
  a.g = m.w2_g;
  a.rows = m.hidden;
  a.K = m.inter;
  if (m.tokens == 1) {
    moe_one_out<TW><<<dim3(m.hidden / 16), dim3(64 * kOneWaves), 0, s>>>(a);
  } else {
    launch_rows<2, false, TW>(a, experts, s);
    moe_combine<<<dim3((m.hidden + 511) / 512, m.tokens), dim3(128), 0, s>>>(a);
  }
}

template <int DT>
void launch_type(const MoeDecodeArgs& m, const Ws& ws, hipStream_t s) {
  launch_router<DT>(m, ws, m.tokens * m.top_k, s);
  if (m.tiled) launch_layer<true>(m, ws, s);
  else launch_layer<false>(m, ws, s);
}

}  // namespace

size_t moe_decode_workspace_bytes(int tokens, int experts, int top_k, int hidden, int inter) {
  return carve(nullptr, tokens, experts, tokens * top_k, hidden, inter, nullptr);
}

hipError_t launch_moe_decode(const MoeDecodeArgs& m, hipStream_t s) {
  Ws ws;
  carve(m.workspace, m.tokens, m.experts, m.tokens * m.top_k, m.hidden, m.inter, &ws);
  if (m.dtype == kBf16) launch_type<kBf16>(m, ws, s);
  else launch_type<kFp16>(m, ws, s);
  return hipGetLastError();
}

}  // namespace nvfp4
