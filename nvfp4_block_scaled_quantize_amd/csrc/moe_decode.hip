// moe_decode.hip -- a whole routed MoE layer for up to 32 tokens on NVFP4 expert weights, for gfx950:
// router product, sigmoid group top-k (the selection of moe.hip), fc1, activation (ReLU^2 or SwiGLU),
// fc2 and the weighted sum, in four launches (three for one token).
//
//  1. router : logits[t, e] = x_t . Wr_e in binary32, one workgroup per expert; clears what the other
//              launches count in; BF16 x also as scaled FP16 (below).
//  2. plan   : one workgroup: one wave per token selects its experts; then the chosen experts, the tokens of
//              each, and a row for every pair of them.  For one token every wave of fc1 selects by itself:
//              that takes 2 us of fc1's time, a launch 4 us.
//  3. fc1    : one workgroup per (chosen expert, 16 RT weight rows): h = act(W1_e x) for the tokens that
//              chose it, binary32.
//  4. fc2    : one workgroup per (chosen expert, 16 RT rows of W2) computes o = W2_e h for the expert's tokens,
//              binary32; the last workgroup of each row range to arrive (an atomic counter) adds the
//              chosen experts' o with their weights in rank order, whatever the order of arrival.
//
// The weights' bytes bound it: each chosen expert's rows are read once, straight from memory into
// registers (no LDS), the waves of a workgroup splitting K in chunks of 128, and the waves' sums are joined
// through LDS.  A lane loads 16 bytes = 32 codes of its row (lane r + 16 g: row r, k = 32 g ..), which feed
// four v_mfma_f32_16x16x32_f16: instruction m takes codes 8 m .. 8 m + 7 of every lane, and the activation
// operand the same k.  E2M1 * E4M3 is exact in FP16.
//
// The activations must be FP16 for that.  FP16 x is used as it is.  BF16 x is multiplied by the power
// of two that brings the token's largest value to [2^14, 2^15): exact down to 2^-31 of the largest, what is
// below is off by at most 2^-39 of it.  h (binary32) is brought to the same range by the pair's
// largest h and split into two FP16 numbers, the value and what its rounding left: off by less than 2^-20 of itself.
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
  int4* chosen;       // [min(P, E)] {expert or -1, first row, mask of its tokens, experts chosen}
  uint32_t* count;    // [row ranges of fc2] workgroups that are done
  _Float16* xs;       // [T, hidden] scaled x (BF16 only)
  float* h;           // [P, inter]
  float* o;           // [P, hidden]
};

constexpr int ranges_of(int hidden) { return (hidden + 31) / 32; }

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
  s.chosen = reinterpret_cast<int4*>(take((size_t)(P < E ? P : E) * 16));
  s.count = reinterpret_cast<uint32_t*>(take((size_t)ranges_of(hidden) * 4));
  s.xs = reinterpret_cast<_Float16*>(take((size_t)T * hidden * 2));
  s.h = reinterpret_cast<float*>(take((size_t)P * inter * 4));
  s.o = reinterpret_cast<float*>(take((size_t)P * hidden * 4));
  if (w) *w = s;
  return at;
}

// The power of two that brings a largest value to [2^14, 2^15).
__device__ __forceinline__ float up_scale(uint32_t bits) {
  const int e = (int)(bits >> 23) - 127;   // -127 for zeros and subnormal numbers
  return __builtin_ldexpf(1.0f, 14 - e < 127 ? 14 - e : 127);
}

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
moe_router(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, int T, int E, int hidden, Ws ws, int P,
           int ranges) {
  __shared__ float part[4][TB];
  __shared__ float top[4][TB];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int unit0 = (int)((int64_t)(hidden / 8) * e / E), unit1 = (int)((int64_t)(hidden / 8) * (e + 1) / E);
  if (e == 0) {
    for (int i = tid; i < P; i += 256) ws.hmax[i] = 0u;
    for (int i = tid; i < ranges; i += 256) ws.count[i] = 0u;
  }
  for (int t0 = 0; t0 < T; t0 += TB) {
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
    __syncthreads();
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

// One wave selects one token's experts: lane l holds experts l + 64 i, i < N.  A group's score is the sum of
// its two best biased scores, the best groups are kept, and the top_k experts of those are taken one
// after the other, ties to the lower index: lane k receives the one of rank k and its weight.  Groups of 2, 4,
// .. 64 experts are lanes next to one another; others go through LDS (sb, sg: E and n_group entries).
template <int N>
__device__ __forceinline__ void select_token(const RouteArgs& a, const float* __restrict__ logits, int t, float* sb,
                                             float* sg, int& id, float& weight) {
  const int lane = threadIdx.x & 63;
  const int gsize = a.E / a.n_group;
  const float ninf = -__builtin_inff();
  float s[N], b[N];
  uint32_t key[N];
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
  // sums over the experts before each: rows, and experts that have any
  uint32_t m = 0u;
  int rows = 0, some = 0, r = 0, u = 0;
  if (tid < 256) {
    m = takers[tid];
    r = rows = __popc(m);
    u = some = m != 0u ? 1 : 0;
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
    if (m != 0u) ws.chosen[bu] = make_int4(tid, br, (int)m, n);
    const int most = a.T * a.top_k < a.E ? a.T * a.top_k : a.E;
    if (tid >= n && tid < most) ws.chosen[tid] = make_int4(-1, 0, 0, n);
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
// past the row; there it reads the block's start again, and scales() is 0.  (Nothing is done with what is
// loaded before it is used: the loads after these must not wait.)
template <bool TW>
__device__ __forceinline__ void load_piece(const uint8_t* __restrict__ w, const uint8_t* __restrict__ sf, int64_t row16,
                                           int c, int K, int lane, Piece& p) {
  if constexpr (TW) {
    const int64_t tile = (row16 / 16) * (K / 128) + 2 * c;
    const int64_t next = 256 * c + 128 < K ? tile + 1 : tile;
    p.codes[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + tile * 1024 + 16 * lane));
    p.codes[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + next * 1024 + 16 * lane));
    p.sf[0] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(sf + tile * 128 + 2 * lane));
    p.sf[1] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(sf + next * 128 + 2 * lane));
  } else {
    const int g = lane >> 4;
    const bool in = 256 * c + 64 * g < K;
    const int64_t row = row16 + (lane & 15);
    const uint8_t* at = w + row * (K / 2) + 128 * c + (in ? 32 * g : 0);
    p.codes[0] = *reinterpret_cast<const u32x4*>(at);
    p.codes[1] = *reinterpret_cast<const u32x4*>(at + 16);
    p.sf[0] = *reinterpret_cast<const uint32_t*>(sf + row * (K / 16) + 16 * c + (in ? 4 * g : 0));
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

// Operands of instruction m.  FC 1: as stored.  FC 2: scaled and split; both roundings are toward zero,
// the first leaves less than 2^-10 of the value, the second less than 2^-10 of that.
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
      const v2h q = __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_pkrtz(a - (float)p[0], b - (float)p[1]));
      hi[2 * i] = p[0];
      hi[2 * i + 1] = p[1];
      lo[2 * i] = q[0];
      lo[2 * i + 1] = q[1];
    }
  }
}

// Four numbers to and from memory that workgroups on other dies read: the accesses go past the caches
// of this die one by one.  (A fence would write back a whole die's cache: with one in each workgroup fc2 of 16
// tokens took 120 us instead of 27.)
__device__ __forceinline__ void store_shared(float* p, const v4f& v) {
  const uint64_t a = __float_as_uint(v[0]) | (uint64_t)__float_as_uint(v[1]) << 32;
  const uint64_t b = __float_as_uint(v[2]) | (uint64_t)__float_as_uint(v[3]) << 32;
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p) + 1, b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ v4f load_shared(const float* p) {
  const uint64_t a = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t b = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p) + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return v4f{__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)), __uint_as_float((uint32_t)b),
             __uint_as_float((uint32_t)(b >> 32))};
}

// SEL > 0: fc1 of one token, whose experts (SEL 64 of them at most) every wave selects by itself.
template <int FC, bool GATED, bool TW, int RT, int TT, int NW, int SEL>
__global__ void __launch_bounds__(64 * NW, TT == 1 ? 4 : 2) moe_expert_rows(FcArgs a) {
  constexpr int kThreads = 64 * NW;
  constexpr int kPairsEach = (kMaxPairs + kThreads - 1) / kThreads;
  __shared__ v4f part[NW][RT * TT][64];
  __shared__ float scratch[SEL ? NW : 1][2][64 * (SEL ? SEL : 1)];
  __shared__ float wts[FC == 2 ? kMaxPairs : 1];
  __shared__ int rows[FC == 2 ? kMaxPairs : 1];   // row of each pair
  __shared__ uint32_t slot_max[16 * TT];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int T = a.route.T, top_k = a.route.top_k, P = T * top_k;

  // for the last workgroup of the row range: on its way before anything else
  float pw[kPairsEach];
  int pr[kPairsEach];
  if constexpr (FC == 2) {
#pragma unroll
    for (int i = 0; i < kPairsEach; ++i) {
      const int p = tid + i * kThreads;
      pw[i] = a.ws.wts[p < P ? p : 0];
      pr[i] = a.ws.row_of[p < P ? p : 0];
    }
  } else {
    if (tid < 16 * TT) slot_max[tid] = 0u;
  }
  // this workgroup's expert, its first row, its tokens, how many experts there are
  int4 mine;
  if constexpr (SEL > 0) {
    int id;
    float w;
    select_token<SEL>(a.route, a.ws.logits, 0, scratch[wave][0], scratch[wave][1], id, w);
    mine = make_int4(__builtin_amdgcn_readlane(id, (int)blockIdx.y), (int)blockIdx.y, 1, top_k);
    if (blockIdx.x == 0 && wave == 0) {
      if (lane == 0) a.ws.chosen[blockIdx.y] = mine;
      if (blockIdx.y == 0 && lane < top_k) {
        a.ws.wts[lane] = w;
        a.ws.row_of[lane] = lane;
        if (a.ids_out) a.ids_out[lane] = id;
        if (a.w_out) a.w_out[lane] = w;
      }
    }
  } else {
    mine = a.ws.chosen[blockIdx.y];
    if (mine.x < 0) return;   // fewer experts than workgroups: the whole workgroup
  }
  const int e = mine.x, q0 = mine.y;
  const uint32_t tokens = (uint32_t)mine.z;
  const int ns = __popc(tokens);

  // token slots of this lane: slot s is the s-th token of the mask
  int64_t arow[TT];
  uint32_t top[TT];   // bits of the largest value that the operand was, or will be, scaled by
  bool there[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int s = 16 * j + r16;
    there[j] = s < ns;
    if constexpr (FC == 1) {
      uint32_t m = tokens;
      for (int i = 0; i < 16 * TT - 1; ++i) m = i < s ? m & (m - 1) : m;
      arow[j] = there[j] ? __builtin_ctz(m) : 0;
      top[j] = a.scaled ? a.ws.xmax[arow[j]] : 0u;
    } else {
      arow[j] = q0 + (there[j] ? s : 0);
      top[j] = a.ws.hmax[arow[j]];
    }
  }

  // weight rows of the tile's RT groups of 16: consecutive rows, or for SwiGLU in fc1 gate rows, then the up rows
  constexpr int kCols = (GATED ? RT / 2 : RT) * 16;   // results per token
  const int col0 = (int)blockIdx.x * kCols;
  int64_t row16[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = !GATED ? col0 + 16 * i : i < RT / 2 ? col0 + 16 * i : a.inter + col0 + 16 * (i - RT / 2);
    row16[i] = (int64_t)e * a.rows + r;
  }
  v4f acc[RT][TT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const float ge = a.g[e];

  const int blocks = (a.K + 255) / 256;
  for (int c = wave; c < blocks; c += NW) {
    Piece w[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) load_piece<TW>(a.w, a.sf, row16[i], c, a.K, lane, w[i]);
    RawAct<FC> raw[2][TT];
    auto load_half = [&](int d) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < TT; ++j)
        if (j == 0 || ns > 16 * j) load_act<FC>(a.src, arow[j], there[j], a.K, first_k<TW>(c, d, grp), raw[d][j]);
    };
    load_half(0);
    if constexpr (FC == 1) load_half(1);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      if constexpr (FC == 2) {
        if (d == 1) load_half(1);
      }
      _Float16 sc[RT][2];
#pragma unroll
      for (int i = 0; i < RT; ++i) scales<TW>(w[i], d, c, a.K, grp, sc[i]);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        v8h wv[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) wv[i] = dequant8(w[i].codes[d][m], sc[i][m / 2]);
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          if (j > 0 && ns <= 16 * j) break;   // the whole workgroup
          v8h hi, lo;
          act_operand<FC>(raw[d][j], m, FC == 2 ? up_scale(top[j]) : 1.0f, hi, lo);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv[i], hi, acc[i][j], 0, 0, 0);
            if constexpr (FC == 2) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv[i], lo, acc[i][j], 0, 0, 0);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) part[wave][i * TT + j][lane] = acc[i][j];
  if constexpr (FC == 2) {
#pragma unroll
    for (int i = 0; i < kPairsEach; ++i) {
      const int p = tid + i * kThreads;
      if (p < P) {
        rows[p] = pr[i];
        wts[p] = pw[i];
      }
    }
  }
  __syncthreads();
  auto joined = [&](int tile) __attribute__((always_inline)) {
    v4f s = part[0][tile][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) {
      const v4f q = part[v][tile][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += q[i];
    }
    return s;
  };
  // results: lane (slot r16, columns 4 grp .. + 3) of a tile
  constexpr int kOutTiles = kCols / 16 * TT;
  for (int tile = wave; tile < kOutTiles; tile += NW) {
    const int i = tile / TT, j = tile % TT, slot = 16 * j + r16;
    if (16 * j >= ns) continue;
    v4f y = joined(tile);
    v4f up;
    if constexpr (GATED) up = joined(tile + RT / 2 * TT);
    if (slot >= ns) continue;
    const int col = col0 + 16 * i + 4 * grp;
    const uint32_t bits = TT == 1 || j == 0 ? top[0] : top[TT - 1];
    const float f = FC == 2 || a.scaled ? ge / up_scale(bits) : ge;
    if constexpr (FC == 1) {
      v4f hv;
      float m = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        hv[q] = GATED ? swiglu_f32(y[q] * f, up[q] * f) : relu2_f32(y[q] * f);
        m = __builtin_fmaxf(m, __builtin_fabsf(hv[q]));
      }
      *reinterpret_cast<v4f*>(a.ws.h + (int64_t)(q0 + slot) * a.inter + col) = hv;
      atomicMax(&slot_max[slot], __float_as_uint(m));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] *= f;
      store_shared(a.ws.o + (int64_t)(q0 + slot) * a.hidden + col, y);
    }
  }
  if constexpr (FC == 1) {
    __syncthreads();
    if (tid < ns) atomicMax(a.ws.hmax + q0 + tid, slot_max[tid]);
  } else {
    // this workgroup's results are in memory before it counts itself; the one that counts last sees all of them
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
      const uint32_t n = __hip_atomic_fetch_add(a.ws.count + blockIdx.x, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = n == (uint32_t)(mine.w - 1) ? 1 : 0;
    }
    __syncthreads();
    if (!last) return;
    constexpr int kQuads = kCols / 4;
    for (int i = tid; i < T * kQuads; i += kThreads) {
      const int t = i / kQuads, col = col0 + 4 * (i - t * kQuads);
      v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
      for (int k = 0; k < top_k; ++k) {
        const v4f v = load_shared(a.ws.o + (int64_t)rows[t * top_k + k] * a.hidden + col);
        const float wk = wts[t * top_k + k];
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] = __builtin_fmaf(wk, v[q], s[q]);
      }
      uint16_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = a.out_type == kBf16 ? __builtin_bit_cast(uint16_t, (__bf16)s[q]) : __builtin_bit_cast(uint16_t, (_Float16)s[q]);
      u32x2 v = {o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16};
      *reinterpret_cast<u32x2*>((uint16_t*)a.out + (int64_t)t * a.hidden + col) = v;
    }
  }
}

template <int DT>
void launch_router(const MoeDecodeArgs& m, const Ws& ws, int P, hipStream_t s) {
  const uint16_t* x = reinterpret_cast<const uint16_t*>(m.x);
  const uint16_t* wr = reinterpret_cast<const uint16_t*>(m.router);
  const dim3 grid(m.experts), block(256);
  if (m.tokens == 1) moe_router<DT, 1><<<grid, block, 0, s>>>(x, wr, m.tokens, m.experts, m.hidden, ws, P, ranges_of(m.hidden));
  else if (m.tokens <= 4) moe_router<DT, 4><<<grid, block, 0, s>>>(x, wr, m.tokens, m.experts, m.hidden, ws, P, ranges_of(m.hidden));
  else moe_router<DT, 8><<<grid, block, 0, s>>>(x, wr, m.tokens, m.experts, m.hidden, ws, P, ranges_of(m.hidden));
}

// 64 weight rows to a workgroup where there are enough of them to fill the chip, else 32; then eight waves where
// a row is long enough for them.
template <int FC, bool GATED, bool TW>
void launch_rows(const FcArgs& a, int experts, hipStream_t s) {
  const bool many = (int64_t)(a.rows / 64) * experts >= 512;
  const dim3 grid(many ? a.rows / 64 : a.rows / 32, experts), block(256);
  if constexpr (FC == 1) {
    if (a.route.T == 1) {
      const bool eight = a.K > 1024;
      const dim3 one(a.rows / 32, experts), waves(eight ? 512 : 256);
      if (a.route.E <= 64) {
        if (eight) moe_expert_rows<FC, GATED, TW, 2, 1, 8, 1><<<one, waves, 0, s>>>(a);
        else moe_expert_rows<FC, GATED, TW, 2, 1, 4, 1><<<one, waves, 0, s>>>(a);
      } else {
        if (eight) moe_expert_rows<FC, GATED, TW, 2, 1, 8, kPerLane><<<one, waves, 0, s>>>(a);
        else moe_expert_rows<FC, GATED, TW, 2, 1, 4, kPerLane><<<one, waves, 0, s>>>(a);
      }
      return;
    }
  }
  if (a.route.T <= 16) {
    if (many) moe_expert_rows<FC, GATED, TW, 4, 1, 4, 0><<<grid, block, 0, s>>>(a);
    else if (a.K > 1024) moe_expert_rows<FC, GATED, TW, 2, 1, 8, 0><<<grid, dim3(512), 0, s>>>(a);
    else moe_expert_rows<FC, GATED, TW, 2, 1, 4, 0><<<grid, block, 0, s>>>(a);
  } else {
    if (many) moe_expert_rows<FC, GATED, TW, 4, 2, 4, 0><<<grid, block, 0, s>>>(a);
    else moe_expert_rows<FC, GATED, TW, 2, 2, 4, 0><<<grid, block, 0, s>>>(a);
  }
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
  if (gated) launch_rows<1, true, TW>(a, experts, s);
  else launch_rows<1, false, TW>(a, experts, s);
  a.src = ws.h;
  a.w = m.w2;
  a.sf = m.w2_sf;
  a.g = m.w2_g;
  a.rows = m.hidden;
  a.K = m.inter;
  launch_rows<2, false, TW>(a, experts, s);
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
