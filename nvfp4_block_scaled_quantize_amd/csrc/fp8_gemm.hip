// fp8_gemm.hip -- y[B, N] = sum_k a[b, k] sa[b, k / 128] w[n, k] sw[n / 128, k / 128] for E4M3 operands
// with binary32 scales per 128 (activations 1 x 128, weights 128 x 128), for gfx950.
//
// The matrix instruction that takes 128 k at once (v_mfma_f32_16x16x128_f8f6f4) forms the sum of one
// K-block in binary32 from zero; the scale of the block, sa sw, is then applied by one fma per output
// into the running binary32 sum.  The weight is the instruction's first operand: a lane's four results
// are four consecutive columns of one row of y, so one product sa sw serves a whole 16 x 16 tile.  An
// instruction takes 32 clocks, its four fmas 16 clocks of the vector pipe beside it.
//
// The k order inside a block is free as long as both operands share it: lane group g = lane / 16 takes the
// 16-byte pieces g and g + 4 of its row's 128 bytes.
#include <type_traits>

#include "device_common.h"
#include "fp8.h"
#include "internal.h"
#include "lds_dma.h"

namespace nvfp4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

// Sum of one K-block for a 16 x 16 tile: rows from w, columns from a.
__device__ __forceinline__ v4f mfma_block(const v8i& w, const v8i& a) {
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ v8i join(u32x4 p, u32x4 q) {
  v8i r = {(int)p.x, (int)p.y, (int)p.z, (int)p.w, (int)q.x, (int)q.y, (int)q.z, (int)q.w};
  return r;
}

template <int DT>
__device__ __forceinline__ uint16_t round16(float x) {
  if constexpr (DT == kBf16) return __builtin_bit_cast(uint16_t, (__bf16)x);
  else return __builtin_bit_cast(uint16_t, (_Float16)x);
}

// Four consecutive columns n .. n + 3 of a row; `wide`: all of them exist and are 8-byte aligned.
template <int DT>
__device__ __forceinline__ void store4(uint16_t* row, int n, int N, bool wide, const v4f& v) {
  if (wide) {
    u32x2 o;
    o.x = round16<DT>(v[0]) | (uint32_t)round16<DT>(v[1]) << 16;
    o.y = round16<DT>(v[2]) | (uint32_t)round16<DT>(v[3]) << 16;
    *reinterpret_cast<u32x2*>(row + n) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) row[n + i] = round16<DT>(v[i]);
  }
}

// ---------------------------------------------------------------- tiles (many rows)
// BT rows of a by BF rows of w per workgroup, one 128-k block per stage, two stage buffers: the copies of
// the next stage (global -> LDS, 16 bytes a lane) are in flight while a stage is computed.  LDS holds
// the rows' 128 bytes with piece p of row r at p ^ ((r / 2) mod 8): the 16 lanes of an operand read
// touch 16 different places of 16 bytes.
template <int TT, int FT, int WT, int WF>
struct Tile {
  static constexpr int kWaves = WT * WF;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRowsA = 16 * TT * WT, kRowsW = 16 * FT * WF;
  static constexpr int kCopies = (kRowsA + kRowsW) / 8 / kWaves;   // 16-byte copies of a wave and stage
  static constexpr int kWOff = 0, kAOff = kRowsW * 128;
  static constexpr int kSAOff = (kRowsW + kRowsA) * 128;           // scales of the rows of a
  static constexpr int kSWOff = kSAOff + kRowsA * 4;               // scales of the blocks of w, 64 entries
  static constexpr int kStage = kSWOff + 256;
  static constexpr int kScaleWaves = kRowsA / 64;                  // waves that copy scales of a
  static_assert(kRowsW % (8 * kWaves) == 0 && kRowsA % (8 * kWaves) == 0, "a copy stays in one operand");
  static_assert(kScaleWaves < kWaves && kRowsA % 64 == 0, "one wave at least copies the scales of w");
  static_assert(128 % (16 * FT) == 0, "a wave's columns share the scales of w");
};

template <int DT, int TT, int FT, int WT, int WF>
__global__ void __launch_bounds__(64 * WT * WF)
fp8_gemm_tiles(Fp8GemmArgs g, int tiles_m, int tiles_n) {
  using C = Tile<TT, FT, WT, WF>;
  __shared__ __attribute__((aligned(256))) unsigned char lds[2 * C::kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave % WT, wf = wave / WT;
  int tm, tn;
  {
    // consecutive ids go to different XCDs: each XCD walks its own run of tiles, eight rows of tiles deep,
    // so its resident workgroups share row stripes of both operands in its L2
    const int total = tiles_m * tiles_n;
    int t = blockIdx.x;
    if (total % 8 == 0) t = (t & 7) * (total / 8) + (t >> 3);
    constexpr int kDeep = 8;
    const int band = t / (kDeep * tiles_n), rest = t - band * kDeep * tiles_n;
    const int deep = tiles_m - band * kDeep < kDeep ? tiles_m - band * kDeep : kDeep;
    tm = band * kDeep + rest % deep;
    tn = rest / deep;
  }
  const int K = g.K, nkb = (K + 127) / 128;
  const int m0 = tm * C::kRowsA, n0 = tn * C::kRowsW;
  const uint32_t l0 = lds_addr(lds);

  // copies: wave w, copy i moves rows 8 (w kCopies + i) .. + 7 of the stage (rows of w first), lane l the
  // piece (l mod 8) of row l / 8.  Rows past an operand's end repeat its last row (never stored).
  uint32_t from[C::kCopies];
  const int sub = lane >> 3;
#pragma unroll
  for (int i = 0; i < C::kCopies; ++i) {
    const int c = wave * C::kCopies + i;
    const bool is_w = c < C::kRowsW / 8;
    const int r = is_w ? 8 * c + sub : 8 * c - C::kRowsW + sub;
    const int last = is_w ? g.N - 1 - n0 : g.B - 1 - m0;
    from[i] = (uint32_t)(r < last ? r : last) * (uint32_t)K;
  }
  // the piece a lane copies: (l mod 8) ^ ((row / 2) mod 8), row = 8 c + l / 8
  const int piece0 = (lane & 7) ^ (lane >> 4);   // even c; odd c: ^ 4
  const int tail = (K & 127) / 16;               // pieces of the last block, 0: whole
  const uint8_t* wbase = g.w + (int64_t)n0 * K;
  const uint8_t* abase = g.a + (int64_t)m0 * K;
  // scales: a wave copies those of 64 rows of a, or the blocks of w
  const bool scales_a = wave < C::kScaleWaves;
  const float* sbase;
  uint32_t sfrom;
  if (scales_a) {
    const int r = 64 * wave + lane, last = g.B - 1 - m0;
    sbase = g.as + (int64_t)m0 * nkb;
    sfrom = (uint32_t)(r < last ? r : last) * (uint32_t)nkb * 4u;
  } else {
    const int last = (g.N - 1) / 128 - n0 / 128;
    const int b = (C::kRowsW + 127) / 128 - 1 < last ? (C::kRowsW + 127) / 128 - 1 : last;
    sbase = g.ws + (int64_t)(n0 / 128) * nkb;
    sfrom = (uint32_t)(lane < b ? lane : b) * (uint32_t)nkb * 4u;
  }
  const uint32_t sto = scales_a ? C::kSAOff + 256 * wave : C::kSWOff;

  auto issue = [&](int kb) __attribute__((always_inline)) {
    const uint32_t st = l0 + (kb & 1) * C::kStage;
    const bool cut = tail != 0 && kb == nkb - 1;
#pragma unroll
    for (int i = 0; i < C::kCopies; ++i) {
      const int c = wave * C::kCopies + i;   // kCopies is even: the parity of c is that of i
      int p = piece0 ^ (4 * (i & 1));
      if (cut && p >= tail) p = 0;           // past the row's end: any place of the row, cleared later
      const bool is_w = c < C::kRowsW / 8;
      dma16((is_w ? wbase : abase) + (int64_t)kb * 128, from[i] + 16u * p, st + c * 1024);
    }
    dma4(sbase + kb, sfrom, st + sto);
  };

  v4f acc[TT][FT];
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int i = 0; i < FT; ++i) acc[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const int r16 = lane & 15, grp = lane >> 4;
  const uint32_t operand = r16 * 128 + 16 * (grp ^ (r16 >> 1 & 7));   // piece grp; piece grp + 4: ^ 64
  typedef const __attribute__((address_space(3))) unsigned char* lptr;
  auto read = [&](uint32_t at) __attribute__((always_inline)) {
    typedef const __attribute__((address_space(3))) u32x4* vptr;
    return *(vptr)(uintptr_t)at;
  };

  issue(0);
  for (int kb = 0; kb < nkb; ++kb) {
    // this wave's copies have landed and its reads of the other buffer are done; then everyone's
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const uint32_t st = l0 + (kb & 1) * C::kStage;
    if (kb + 1 < nkb) {
      issue(kb + 1);
    } else if (tail) {
      // the pieces past the rows' end: zeros
      for (int i = tid; i < (C::kRowsA + C::kRowsW) * 8; i += C::kThreads) {
        const int r = i >> 3;
        if (((i & 7) ^ (r >> 1 & 7)) >= tail) *reinterpret_cast<u32x4*>(lds + (kb & 1) * C::kStage + 16 * i) = u32x4{0, 0, 0, 0};
      }
      __syncthreads();
    }
    const uint32_t wl = st + C::kWOff + wf * (16 * FT) * 128 + operand;
    const uint32_t al = st + C::kAOff + wt * (16 * TT) * 128 + operand;
    v8i wv[FT];
#pragma unroll
    for (int i = 0; i < FT; ++i) wv[i] = join(read(wl + 2048 * i), read((wl ^ 64) + 2048 * i));
    typedef const __attribute__((address_space(3))) float* fptr;
    const float sw = *(fptr)(uintptr_t)(st + C::kSWOff + 4 * ((n0 % 128 + wf * 16 * FT) / 128));
    const uint32_t sa = st + C::kSAOff + 4 * (wt * 16 * TT + r16);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const v8i av = join(read(al + 2048 * j), read((al ^ 64) + 2048 * j));
      const float s = *(fptr)(uintptr_t)(sa + 64 * j) * sw;
#pragma unroll
      for (int i = 0; i < FT; ++i) {
        const v4f p = mfma_block(wv[i], av);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][i][q] = __builtin_fmaf(p[q], s, acc[j][i][q]);
      }
    }
  }

  const bool vec = g.N % 4 == 0 && ((uintptr_t)g.y % 8) == 0;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int m = m0 + (wt * TT + j) * 16 + r16;
    if (m >= g.B) continue;
    uint16_t* row = (uint16_t*)g.y + (int64_t)m * g.N;
#pragma unroll
    for (int i = 0; i < FT; ++i) {
      const int n = n0 + (wf * FT + i) * 16 + 4 * grp;
      if (n < g.N) store4<DT>(row, n, g.N, vec, acc[j][i]);
    }
  }
}

// ---------------------------------------------------------------- streams (few rows)
// A workgroup holds all rows of a (up to 16 TT) against 16 FT rows of w; its eight waves take the
// K-blocks in turn, straight from memory into registers (every byte of w is read once, by one wave),
// and their sums are joined through LDS.  Bound by the bytes of w.
constexpr int kSsWaves = 8;

template <int DT, int TT, int FT, int U>
__global__ void __launch_bounds__(64 * kSsWaves)
fp8_gemm_stream(Fp8GemmArgs g) {
  __shared__ v4f part[kSsWaves][TT * FT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int K = g.K, nkb = (K + 127) / 128;
  const int n0 = blockIdx.x * 16 * FT;
  const uint8_t* wrow[FT];
  const uint8_t* arow[TT];
  const float* srow[TT];
#pragma unroll
  for (int i = 0; i < FT; ++i) {
    const int n = n0 + 16 * i + r16;
    wrow[i] = g.w + (int64_t)(n < g.N ? n : g.N - 1) * K + 16 * grp;
  }
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int m = 16 * j + r16 < g.B ? 16 * j + r16 : g.B - 1;
    arow[j] = g.a + (int64_t)m * K + 16 * grp;
    srow[j] = g.as + (int64_t)m * nkb;
  }
  const float* swrow = g.ws + (int64_t)(n0 / 128) * nkb;   // 16 FT divides 128
  v4f acc[TT][FT];
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int i = 0; i < FT; ++i) acc[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // K-blocks that are whole; a last one that is not goes through the masked turn below
  const int whole = K / 128;
  int kb = wave;
  for (; kb < whole; kb += kSsWaves * U) {
    u32x4 wq[U][FT][2], aq[U][TT][2];
    float sa[U][TT], sw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = kb + kSsWaves * u < whole ? kb + kSsWaves * u : kb;   // past the end: again the first, with scale 0
      const int64_t o = (int64_t)b * 128;
#pragma unroll
      for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wq[u][i][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow[i] + o + 64 * h));
#pragma unroll
      for (int j = 0; j < TT; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) aq[u][j][h] = *reinterpret_cast<const u32x4*>(arow[j] + o + 64 * h);
        sa[u][j] = srow[j][b];
      }
      sw[u] = swrow[b];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u > 0 && kb + kSsWaves * u >= whole) break;   // the same for the whole wave
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const float s = sa[u][j] * sw[u];
#pragma unroll
        for (int i = 0; i < FT; ++i) {
          const v4f p = mfma_block(join(wq[u][i][0], wq[u][i][1]), join(aq[u][j][0], aq[u][j][1]));
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[j][i][q] = __builtin_fmaf(p[q], s, acc[j][i][q]);
        }
      }
    }
  }
  if (whole < nkb && wave == whole % kSsWaves) {
    const int valid = (K & 127) / 16;
    const u32x4 zero = {0, 0, 0, 0};
    const bool in0 = grp < valid, in1 = grp + 4 < valid;
    const int64_t o0 = in0 ? (int64_t)whole * 128 : 0, o1 = in1 ? (int64_t)whole * 128 + 64 : 0;
    v8i wv[FT];
#pragma unroll
    for (int i = 0; i < FT; ++i) {
      // K >= 128 is not given: the pieces read in place of missing ones are the row's first (16 grp < K
      // does not hold for a short row, so those lanes read the row's start)
      const uint8_t* base = wrow[i] - 16 * grp;
      const u32x4 p = *reinterpret_cast<const u32x4*>(in0 ? wrow[i] + o0 : base);
      const u32x4 q = *reinterpret_cast<const u32x4*>(in1 ? wrow[i] + o1 : base);
      wv[i] = join(in0 ? p : zero, in1 ? q : zero);
    }
    const float sw = swrow[whole];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const uint8_t* base = arow[j] - 16 * grp;
      const u32x4 p = *reinterpret_cast<const u32x4*>(in0 ? arow[j] + o0 : base);
      const u32x4 q = *reinterpret_cast<const u32x4*>(in1 ? arow[j] + o1 : base);
      const v8i av = join(in0 ? p : zero, in1 ? q : zero);
      const float s = srow[j][whole] * sw;
#pragma unroll
      for (int i = 0; i < FT; ++i) {
        const v4f r = mfma_block(wv[i], av);
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[j][i][t] = __builtin_fmaf(r[t], s, acc[j][i][t]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int i = 0; i < FT; ++i) part[wave][j * FT + i][lane] = acc[j][i];
  __syncthreads();
  const bool vec = g.N % 4 == 0 && ((uintptr_t)g.y % 8) == 0;
  for (int t = wave; t < TT * FT; t += kSsWaves) {
    v4f sum = part[0][t][lane];
#pragma unroll
    for (int v = 1; v < kSsWaves; ++v) {
      const v4f p = part[v][t][lane];
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[q] += p[q];
    }
    const int m = (t / FT) * 16 + r16, n = n0 + (t % FT) * 16 + 4 * grp;
    if (m < g.B && n < g.N) store4<DT>((uint16_t*)g.y + (int64_t)m * g.N, n, g.N, vec, sum);
  }
}

template <int DT, int TT, int FT, int WT, int WF>
void tiles(const Fp8GemmArgs& g, hipStream_t s) {
  using C = Tile<TT, FT, WT, WF>;
  const int tm = (g.B + C::kRowsA - 1) / C::kRowsA, tn = (g.N + C::kRowsW - 1) / C::kRowsW;
  fp8_gemm_tiles<DT, TT, FT, WT, WF><<<dim3((unsigned)(tm * tn)), dim3(C::kThreads), 0, s>>>(g, tm, tn);
}

template <int DT, int TT, int FT, int U>
void stream(const Fp8GemmArgs& g, hipStream_t s) {
  fp8_gemm_stream<DT, TT, FT, U><<<dim3((unsigned)((g.N + 16 * FT - 1) / (16 * FT))), dim3(64 * kSsWaves), 0, s>>>(g);
}

template <int DT>
void launch(const Fp8GemmArgs& g, hipStream_t s) {
  if (g.B <= 16) return stream<DT, 1, 1, 4>(g, s);
  if (g.B <= 32) return stream<DT, 2, 2, 2>(g, s);
  if (g.B <= 64) return stream<DT, 4, 2, 2>(g, s);
  const int64_t big = (int64_t)((g.B + 255) / 256) * ((g.N + 255) / 256);
  if (big >= 192) return tiles<DT, 8, 4, 2, 4>(g, s);
  return tiles<DT, 4, 4, 2, 2>(g, s);
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t s) {
  if (g.out_dtype == kBf16) launch<kBf16>(g, s);
  else launch<kFp16>(g, s);
  return hipGetLastError();
}

}  // namespace nvfp4
