// moe_decode.hip -- a whole routed MoE layer for up to 32 tokens on NVFP4 expert weights, for gfx950:
// router product, sigmoid group top-k (the selection of moe.hip), fc1, activation (ReLU^2 or SwiGLU),
// fc2 and the weighted sum, in three launches (four for more than 8 tokens).
//
//  1. router : logits[t, e] = x_t . Wr_e in binary32, one workgroup per expert; clears what the other
//              launches count in; BF16 x also as scaled FP16 (below).
//  (2. select: more than 8 tokens: one wave per token.)
//  3. fc1    : one workgroup per (chosen expert, 16 RT weight rows).  For up to 8 tokens every workgroup
//              selects all tokens' experts again from the logits, which takes less than a launch.  It
//              finds its expert and the tokens that chose it, and computes h = act(W1_e x) for them,
//              binary32.
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
constexpr int kSelectAgain = 8;              // tokens up to which fc1 selects by itself

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// A pair (token, rank) has the number p = token * top_k + rank; its row q of h and o is its place when the
// pairs are sorted by expert.
struct Ws {
  float* logits;      // [T, E]
  uint32_t* xmax;     // [T] largest |x| (binary32 bits)
  uint32_t* hmax;     // [P] largest |h| of row q (binary32 bits)
  int32_t* ids;       // [P] expert of pair p
  float* wts;         // [P] its weight
  int32_t* row_of;    // [P] its row q
  int4* chosen;       // [min(P, E)] {expert or -1, first row, rows, experts chosen}
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
  s.ids = reinterpret_cast<int32_t*>(take((size_t)P * 4));
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

// One wave selects one token's experts: lane l holds experts l + 64 i.  A group's score is the sum of its
// two best biased scores, the best groups are kept, and the top_k experts of those are taken one
// after the other, ties to the lower index.
__device__ __forceinline__ void select_token(const RouteArgs& a, const float* __restrict__ logits, int t, float* sb,
                                             float* sg, int32_t* ids, float* wts) {
  const int lane = threadIdx.x & 63;
  const int gsize = a.E / a.n_group;
  float s[kPerLane];
  uint32_t key[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 64 * i;
    s[i] = 0.0f;
    key[i] = 0u;
    if (e < a.E) {
      s[i] = sigmoid_f32(logits[(int64_t)t * a.E + e]);
      float b = s[i] + a.bias[e];
      if (b != b) b = -__builtin_inff();
      key[i] = rank_key(b);
      if (a.n_group > 1) sb[e] = b;
    }
  }
  if (a.n_group > 1) {
    const float ninf = -__builtin_inff();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // only this wave reads what it wrote
    for (int g = lane; g < a.n_group; g += 64) {
      float v1 = ninf, v2 = ninf;
      for (int j = 0; j < gsize; ++j) {
        const float v = sb[g * gsize + j];
        v2 = __builtin_fmaxf(v2, __builtin_fminf(v1, v));
        v1 = __builtin_fmaxf(v1, v);
      }
      float sum = gsize > 1 ? v1 + v2 : v1;
      if (sum != sum) sum = ninf;
      sg[g] = sum;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 64 * i;
      if (e < a.E) {
        const int g = e / gsize;
        const float mine = sg[g];
        int before = 0;
        for (int j = 0; j < a.n_group; ++j) {
          const float v = sg[j];
          before += (v > mine || (v == mine && j < g)) ? 1 : 0;
        }
        if (before >= a.topk_group) key[i] = 0u;
      }
    }
  }
  float sum = 0.0f, mine = 0.0f;
  int chosen = 0;
  for (int k = 0; k < a.top_k; ++k) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) m = key[i] > m ? key[i] : m;
    m = wave_max_u32(m);
    int e = -1;
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
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
  if (lane < a.top_k) {
    ids[lane] = chosen;
    wts[lane] = (a.norm ? mine / sum : mine) * a.scaling;
  }
}

__global__ void __launch_bounds__(64) moe_select(RouteArgs a, Ws ws) {
  __shared__ float sb[64 * kPerLane], sg[64 * kPerLane];
  const int t = blockIdx.x;
  select_token(a, ws.logits, t, sb, sg, ws.ids + t * a.top_k, ws.wts + t * a.top_k);
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

// A lane's part of one 128-k chunk of 16 rows: 32 codes and their two E4M3 bytes.
struct Piece {
  u32x4 codes;
  uint32_t sf;
};

// Expert weights [E, rows, K]: plain (codes [rows, K / 2], E4M3 [rows, K / 16]) or TW, the layout of
// nvfp4_pretile_weight of the stacked [E rows, K] matrix, in which a chunk of 16 rows is 1 KiB of codes
// and 128 B of E4M3 pairs in lane order.  In the last chunk of a plain row with K % 128 = 64 lanes of
// groups 2 and 3 have no k: they read the first half again, as zeros.
template <bool TW>
__device__ __forceinline__ Piece load_piece(const uint8_t* __restrict__ w, const uint8_t* __restrict__ sf, int64_t row16,
                                            int c, int K, int lane) {
  Piece p;
  if constexpr (TW) {
    const int64_t tile = (row16 / 16) * (K / 128) + c;
    p.codes = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + tile * 1024 + 16 * lane));
    p.sf = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(sf + tile * 128 + 2 * lane));
  } else {
    const int64_t row = row16 + (lane & 15);
    int g = lane >> 4;
    const bool in = 128 * c + 32 * g < K;
    if (!in) g -= 2;
    p.codes = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + row * (K / 2) + 64 * c + 16 * g));
    p.sf = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(sf + row * (K / 16) + 8 * c + 2 * g));
    if (!in) p.sf = 0u;   // scale 0
  }
  return p;
}

struct FcArgs {
  const void* src;       // FC 1: x or its scaled form [T, hidden]; FC 2: h
  const uint8_t* w;
  const uint8_t* sf;
  const float* g;
  int rows, K;           // rows of one expert, and their length
  int inter, hidden;
  int scaled;            // FC 1: src is scaled by up_scale(xmax)
  int select;            // FC 1: the experts are selected here
  RouteArgs route;
  int32_t* ids_out;
  float* w_out;
  void* out;             // FC 2: [T, hidden]
  int out_type;
  Ws ws;
};

// The activations of one chunk for 16 token slots as they are stored: lane (slot, g) holds
// k = 128 c + 32 g .. + 31, as 32 FP16 or 32 binary32 numbers; zeros for slots without a token and past K.
template <int FC>
struct RawAct {
  u32x4 v[FC == 1 ? 4 : 8];
};
template <int FC>
__device__ __forceinline__ void load_act(const void* src, int64_t row, bool there, int K, int c, int g, RawAct<FC>& r) {
  constexpr int kN = FC == 1 ? 4 : 8, kBytes = FC == 1 ? 2 : 4;
#pragma unroll
  for (int m = 0; m < kN; ++m) r.v[m] = u32x4{0u, 0u, 0u, 0u};
  if (there && 128 * c + 32 * g < K) {
    const u32x4* p = reinterpret_cast<const u32x4*>((const char*)src + (row * K + 128 * c + 32 * g) * kBytes);
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

template <int FC, bool GATED, bool TW, int RT, int TT, int NW>
__global__ void __launch_bounds__(64 * NW, TT == 1 ? 4 : 2) moe_expert_rows(FcArgs a) {
  constexpr int kThreads = 64 * NW;
  constexpr int kAhead = FC == 1 ? 2 : 1;   // chunks of a wave in flight
  __shared__ v4f part[NW][RT * TT][64];
  __shared__ float scratch[FC == 1 ? NW : 1][2][64 * kPerLane];
  __shared__ int32_t ids[FC == 1 ? kMaxPairs : 1];
  __shared__ float wts[kMaxPairs];
  __shared__ int rows[kMaxPairs];         // FC 1: pair of each token slot; FC 2: row of each pair
  __shared__ uint32_t used[8];            // experts that some token chose
  __shared__ uint32_t slot_max[16 * TT];
  __shared__ int found[2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int T = a.route.T, top_k = a.route.top_k, P = T * top_k;

  int4 mine;   // this workgroup's expert, its first row, its rows, chosen experts
  if constexpr (FC == 1) {
    if (tid < 8) used[tid] = 0u;
    if (tid < 16 * TT) slot_max[tid] = 0u;
    if (a.select) {
      for (int t = wave; t < T; t += NW)
        select_token(a.route, a.ws.logits, t, scratch[wave][0], scratch[wave][1], ids + t * top_k, wts + t * top_k);
    } else {
      for (int p = tid; p < P; p += kThreads) {
        ids[p] = a.ws.ids[p];
        wts[p] = a.ws.wts[p];
      }
    }
    __syncthreads();
    for (int p = tid; p < P; p += kThreads) atomicOr(&used[ids[p] >> 5], 1u << (ids[p] & 31));
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      for (int p = tid; p < P; p += kThreads) {
        if (a.select) a.ws.wts[p] = wts[p];
        if (a.ids_out) a.ids_out[p] = ids[p];
        if (a.w_out) a.w_out[p] = wts[p];
      }
    }
    __syncthreads();
    // the blockIdx.y-th chosen expert
    int e = -1, n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = used[i];
      const int c = __popc(m);
      if (e < 0 && (int)blockIdx.y < n + c) {
        for (int j = (int)blockIdx.y - n; j > 0; --j) m &= m - 1;
        e = 32 * i + __builtin_ctz(m);
      }
      n += c;
    }
    mine = make_int4(__builtin_amdgcn_readfirstlane(e), 0, 0, n);
  } else {
    mine = a.ws.chosen[blockIdx.y];
    mine.x = __builtin_amdgcn_readfirstlane(mine.x);
  }
  const int e = mine.x;
  if (e < 0) {   // fewer experts than workgroups: the whole workgroup
    if (FC == 1 && blockIdx.x == 0 && tid == 0) a.ws.chosen[blockIdx.y] = mine;
    return;
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
  // the first chunks' weights are on their way while the tokens are looked up
  const int chunks = (a.K + 127) / 128;
  Piece w[kAhead][RT];
  auto load_weights = [&](int c0) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int c = c0 + d * NW < chunks ? c0 + d * NW : c0;   // past the end: again the first, not used
        w[d][i] = load_piece<TW>(a.w, a.sf, row16[i], c, a.K, lane);
      }
  };
  if (wave < chunks) load_weights(wave);

  if constexpr (FC == 1) {
    // its pairs in order (an expert appears at most once per token), and how many pairs come before them
    if (wave == 0) {
      int at = 0, before = 0;
      for (int p0 = 0; p0 < P; p0 += 64) {
        const int p = p0 + lane, id = p < P ? ids[p] : 256;
        const uint64_t m = __ballot(id == e);
        before += __popcll(__ballot(id < e));
        if ((m >> lane) & 1ull) rows[at + __popcll(m & ((1ull << lane) - 1ull))] = p;
        at += __popcll(m);
      }
      if (lane == 0) {
        found[0] = before;
        found[1] = at;
      }
      if (blockIdx.x == 0) {
        if (lane == 0) a.ws.chosen[blockIdx.y] = make_int4(e, before, at, mine.w);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (lane < at) a.ws.row_of[rows[lane]] = before + lane;
      }
    }
    lds_barrier();   // does not wait for the weights
    mine.y = found[0];
    mine.z = found[1];
  }
  const int q0 = mine.y, ns = mine.z;

  // token slots of this lane
  int64_t arow[TT];
  float ascale[TT];
  bool there[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int s = 16 * j + r16;
    there[j] = s < ns;
    arow[j] = FC == 1 ? (there[j] ? rows[s] / top_k : 0) : q0 + s;
    ascale[j] = 1.0f;
    if (FC == 2 && there[j]) ascale[j] = up_scale(a.ws.hmax[q0 + s]);
  }
  v4f acc[RT][TT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  for (int c0 = wave; c0 < chunks; c0 += NW * kAhead) {
    if (c0 != wave) load_weights(c0);
    RawAct<FC> raw[kAhead][TT];
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
#pragma unroll
      for (int j = 0; j < TT; ++j)
        if (j == 0 || ns > 16 * j) load_act<FC>(a.src, arow[j], there[j], a.K, c0 + d * NW, grp, raw[d][j]);
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      if (c0 + d * NW >= chunks) break;   // the whole wave
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const _Float16 s0 = (_Float16)__builtin_amdgcn_cvt_f32_fp8((int)w[d][i].sf, 0);
        const _Float16 s1 = (_Float16)__builtin_amdgcn_cvt_f32_fp8((int)w[d][i].sf, 1);
        w[d][i].sf = (uint32_t)__builtin_bit_cast(uint16_t, s0) | (uint32_t)__builtin_bit_cast(uint16_t, s1) << 16;
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        v8h wv[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
          wv[i] = dequant8(w[d][i].codes[m], __builtin_bit_cast(_Float16, (uint16_t)(m < 2 ? w[d][i].sf : w[d][i].sf >> 16)));
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          if (j > 0 && ns <= 16 * j) break;   // the whole workgroup
          v8h hi, lo;
          act_operand<FC>(raw[d][j], m, ascale[j], hi, lo);
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
    // for the last workgroup of the row range
    for (int p = tid; p < P; p += kThreads) {
      rows[p] = a.ws.row_of[p];
      wts[p] = a.ws.wts[p];
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
  const float ge = a.g[e];
  constexpr int kOutTiles = kCols / 16 * TT;
  for (int tile = wave; tile < kOutTiles; tile += NW) {
    const int i = tile / TT, j = tile % TT, slot = 16 * j + r16;
    if (16 * j >= ns) continue;
    v4f y = joined(tile);
    v4f up;
    if constexpr (GATED) up = joined(tile + RT / 2 * TT);
    if (slot >= ns) continue;
    const int col = col0 + 16 * i + 4 * grp;
    if constexpr (FC == 1) {
      const float f = a.scaled ? ge / up_scale(a.ws.xmax[rows[slot] / top_k]) : ge;
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
      const float f = ge / up_scale(a.ws.hmax[q0 + slot]);
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
      found[0] = n == (uint32_t)(mine.w - 1) ? 1 : 0;
    }
    __syncthreads();
    if (!found[0]) return;
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

template <int FC, bool GATED, bool TW, int RT>
void launch_rows(const FcArgs& a, int tiles, int experts, hipStream_t s) {
  const dim3 grid(tiles, experts);
  // eight waves where a workgroup has a compute unit for itself, four where several share one
  if ((int64_t)tiles * experts <= 512) {
    if (a.route.T <= 16) moe_expert_rows<FC, GATED, TW, RT, 1, 8><<<grid, dim3(512), 0, s>>>(a);
    else moe_expert_rows<FC, GATED, TW, RT, 2, 8><<<grid, dim3(512), 0, s>>>(a);
  } else {
    if (a.route.T <= 16) moe_expert_rows<FC, GATED, TW, RT, 1, 4><<<grid, dim3(256), 0, s>>>(a);
    else moe_expert_rows<FC, GATED, TW, RT, 2, 4><<<grid, dim3(256), 0, s>>>(a);
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
  a.select = m.tokens <= kSelectAgain;
  if (!a.select) moe_select<<<dim3(m.tokens), dim3(64), 0, s>>>(a.route, ws);
  a.scaled = m.dtype == kBf16;
  a.src = a.scaled ? (const void*)ws.xs : m.x;
  a.w = m.w1;
  a.sf = m.w1_sf;
  a.g = m.w1_g;
  a.rows = gated ? 2 * m.inter : m.inter;
  a.K = m.hidden;
  if (gated) launch_rows<1, true, TW, 2>(a, a.rows / 32, experts, s);
  else launch_rows<1, false, TW, 2>(a, a.rows / 32, experts, s);
  a.src = ws.h;
  a.w = m.w2;
  a.sf = m.w2_sf;
  a.g = m.w2_g;
  a.rows = m.hidden;
  a.K = m.inter;
  launch_rows<2, false, TW, 4>(a, a.rows / 64, experts, s);
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
