// fp8_quantize.hip -- E4M3 quantization with one binary32 scale per 128 values of a row
// (activations) or per 128 x 128 values (weights), for gfx950.
//
//   y = the input after the activation in front (none, SwiGLU, ReLU^2), binary32
//   s = max(amax / 448, 2^-126) over the block, code = E4M3_RNE(y * (1 / s))
//
// Division and reciprocal are correctly rounded, so |y| (1 / s) <= 448 (1 + 2^-22), which rounds to
// 448: no code saturates.  The lower limit keeps 1 / s finite; a block of zeros has zero codes.
// NaN stays NaN and does not enter amax; a block with an infinity has s = inf, its finite values
// become 0 and the infinity NaN.
#include "attention.h"
#include "device_common.h"
#include "fp8.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr float kTiny = 0x1p-126f;

// Eight inputs from raw words (16 bytes), one type.
template <int DT, int ACT>
__device__ __forceinline__ void values8(const u32x4& g, const u32x4& u, float* y) {
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2<DT>(gw[i], a, b);
    if constexpr (ACT == kActSwiglu) {
      float c, d;
      unpack2<DT>(uw[i], c, d);
      a = swiglu_f32(a, c);
      b = swiglu_f32(b, d);
    } else if constexpr (ACT == kActRelu2) {
      a = relu2_or_nan_f32(a);
      b = relu2_or_nan_f32(b);
    }
    y[2 * i] = a;
    y[2 * i + 1] = b;
  }
}

template <bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  if constexpr (VEC) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  } else {
    u32x4 r;
    r.x = p[0] | (uint32_t)p[1] << 16;
    r.y = p[2] | (uint32_t)p[3] << 16;
    r.z = p[4] | (uint32_t)p[5] << 16;
    r.w = p[6] | (uint32_t)p[7] << 16;
    return r;
  }
}

__device__ __forceinline__ float amax8(const float* y) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = __builtin_fmaxf(m, __builtin_fabsf(y[e]));
  return m;
}

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* p, const float* y, float inv) {
  u32x2 c;
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * inv, y[1] * inv, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * inv, y[3] * inv, w, true);
  c.x = (uint32_t)w;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * inv, y[5] * inv, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * inv, y[7] * inv, w, true);
  c.y = (uint32_t)w;
  if constexpr (VEC) {
    *reinterpret_cast<u32x2*>(p) = c;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] = (uint8_t)(c.x >> (8 * e));
      p[4 + e] = (uint8_t)(c.y >> (8 * e));
    }
  }
}

// ---------------------------------------------------------------- 1 x 128
// Sixteen lanes hold a block, eight values each: its maximum needs four lane exchanges and no LDS, and
// every load and store of a wave is contiguous.  A thread takes kPer blocks, all of its loads in
// flight before the first exchange.  Bound by memory: 8192 x 14336 of SwiGLU (591 MB) 119 us, 5.0 TB/s.
constexpr int kPer = 4;

template <int DT, int ACT, bool VEC>
__global__ void __launch_bounds__(256)
fp8_quant_rows(const uint16_t* __restrict__ x, int k, int nkb, uint32_t magic, int shift, int blocks,
               uint8_t* __restrict__ codes, float* __restrict__ scale) {
  const int c = threadIdx.x & 15;
  const int first = (int)blockIdx.x * (16 * kPer) + (threadIdx.x >> 4);   // < 2^30
  u32x4 g[kPer], u[kPer];
  int64_t at[kPer];   // first value of the lane's eight in the output, or -1
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = first + 16 * i;
    const int row = divide(b < blocks ? b : blocks - 1, magic, shift);
    const int col = ((b < blocks ? b : blocks - 1) - row * nkb) * 128 + 8 * c;
    const bool in = col < k;
    at[i] = b < blocks && in ? (int64_t)row * k + col : -1;
    const int64_t from = (int64_t)row * (ACT == kActSwiglu ? 2 * (int64_t)k : k) + (in ? col : 0);
    g[i] = load8<VEC>(x + from);
    if constexpr (ACT == kActSwiglu) u[i] = load8<VEC>(x + from + k);
    if (!in) {
      g[i] = u32x4{0u, 0u, 0u, 0u};   // past the row's end: zeros, which no maximum notices
      u[i] = g[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float y[8];
    values8<DT, ACT>(g[i], u[i], y);
    const float amax = row16_max(amax8(y));
    const float s = __builtin_fmaxf(amax / 448.0f, kTiny);
    const float inv = 1.0f / s;
    if (at[i] >= 0) store8<VEC>(codes + at[i], y, inv);
    if (c == 0 && first + 16 * i < blocks) scale[first + 16 * i] = s;
  }
}

// ---------------------------------------------------------------- 128 x 128
// One workgroup per block: 16 lanes a row, 16 rows at a time, everything in registers between the
// maximum and the encoding.  Bound by memory: 7300 x 8272 (181 MB) 41 us, 4.4 TB/s.
template <int DT, int ACT, bool VEC>
__global__ void __launch_bounds__(256)
fp8_quant_tiles(const uint16_t* __restrict__ x, int64_t rows, int k, int nkb, uint32_t magic, int shift,
                uint8_t* __restrict__ codes, float* __restrict__ scale) {
  __shared__ float red[4];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int rb = divide((int)blockIdx.x, magic, shift);
  const int64_t row0 = (int64_t)rb * 128;
  const int col = ((int)blockIdx.x - rb * nkb) * 128 + 8 * c;
  u32x4 g[8], u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 16 * i + r;
    const bool in = row < rows && col < k;
    const int64_t from = in ? row * (ACT == kActSwiglu ? 2 * (int64_t)k : k) + col : 0;
    g[i] = load8<VEC>(x + from);
    if constexpr (ACT == kActSwiglu) u[i] = load8<VEC>(x + from + k);
    if (!in) {
      g[i] = u32x4{0u, 0u, 0u, 0u};
      u[i] = g[i];
    }
  }
  float y[8][8], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    values8<DT, ACT>(g[i], u[i], y[i]);
    m = __builtin_fmaxf(m, amax8(y[i]));
  }
  m = wave_max_dpp(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  const float amax = __builtin_fmaxf(__builtin_fmaxf(red[0], red[1]), __builtin_fmaxf(red[2], red[3]));
  const float s = __builtin_fmaxf(amax / 448.0f, kTiny);
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 16 * i + r;
    if (row < rows && col < k) store8<VEC>(codes + row * k + col, y[i], inv);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

template <int DT, int ACT, bool VEC>
void launch(const Fp8QuantArgs& a, hipStream_t s) {
  const int nkb = (a.k + 127) / 128;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x);
  uint32_t magic;
  int shift;
  division_magic(nkb, magic, shift);
  if (a.block_rows == 1) {
    const int64_t blocks = a.rows * nkb;   // below 2^30 - 2^16 (checked by the entry point)
    fp8_quant_rows<DT, ACT, VEC><<<dim3((unsigned)((blocks + 16 * kPer - 1) / (16 * kPer))), dim3(256), 0, s>>>(
        x, a.k, nkb, magic, shift, (int)blocks, a.codes, a.scale);
  } else {
    fp8_quant_tiles<DT, ACT, VEC><<<dim3((unsigned)((a.rows + 127) / 128 * nkb)), dim3(256), 0, s>>>(
        x, a.rows, a.k, nkb, magic, shift, a.codes, a.scale);
  }
}

template <int DT, int ACT>
void launch_aligned(const Fp8QuantArgs& a, hipStream_t s) {
  // k % 16 == 0: the rows are aligned as the first one is
  if (((uintptr_t)a.x % 16) == 0 && ((uintptr_t)a.codes % 8) == 0) launch<DT, ACT, true>(a, s);
  else launch<DT, ACT, false>(a, s);
}

template <int DT>
void launch_act(const Fp8QuantArgs& a, hipStream_t s) {
  if (a.act == kActSwiglu) launch_aligned<DT, kActSwiglu>(a, s);
  else if (a.act == kActRelu2) launch_aligned<DT, kActRelu2>(a, s);
  else launch_aligned<DT, kActNone>(a, s);
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, hipStream_t s) {
  if (a.dtype == kBf16) launch_act<kBf16>(a, s);
  else launch_act<kFp16>(a, s);
  return hipGetLastError();
}

}  // namespace nvfp4
