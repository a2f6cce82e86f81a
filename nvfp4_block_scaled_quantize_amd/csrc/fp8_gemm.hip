// fp8_gemm.hip -- y[B, N] = sum_k a[b, k] sa[b, k / 128] w[n, k] sw[n / 128, k / 128] for E4M3 operands
// with binary32 scales per 128 (activations 1 x 128, weights 128 x 128), for gfx950.
//
// The matrix instructions form the sum of one K-block in binary32 from zero (v_mfma_f32_32x32x64_f8f6f4 twice, or
// v_mfma_f32_16x16x128_f8f6f4 once); the scale of the block, sa sw, is then applied by one fma per output
// into the running binary32 sum.  The weight is the instruction's first operand: a lane's results lie in one
// row of y, in runs of four consecutive columns, so one product sa sw serves a whole tile.  The instructions of
// a tile and block take four times as long as its fmas, which run beside them.
//
// What the instruction adds is not quite binary32: it joins eight neighbouring products at a time, each cut to a
// multiple of 2^(ea + eb - 13), 2^(ea + eb) the power of two in the largest of them (measured: beside 256 * 256 a
// product of 8 stays, of 12 becomes 8, of 4 vanishes; the older v_mfma_f32_16x16x32_fp8_fp8 does the same).  For
// normal operands a block's sums are off by 2^-16 of their size, an eighth of FP16's rounding.  Products in FP16
// would avoid it at half the rate.
//
// The k order inside a block is free as long as both operands share it.
#include <type_traits>

#include "device_common.h"
#include "fp8.h"
#include "internal.h"
#include "lds_dma.h"

namespace nvfp4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

// Sum of one K-block for a 16 x 16 tile: rows from w, columns from a.
__device__ __forceinline__ v4f mfma_block(const v8i& w, const v8i& a) {
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, 0, 0, 0);
}

// The same for a 32 x 32 tile in two instructions of 64 k: pieces (w0, a0) and (w1, a1) of the block.
__device__ __forceinline__ v16f mfma_block32(const v8i (&w)[2], const v8i (&a)[2]) {
  const v16f zero = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  const v16f p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[0], a[0], zero, 0, 0, 0, 0, 0, 0);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[1], a[1], p, 0, 0, 0, 0, 0, 0);
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
//
// The copies' lines bound it: every 64 x 16 bytes of a copy are eight lines of the L2, but one binary32 scale for
// each of 64 rows is 64 lines.  So the scales of a row are copied four blocks at a time (SB = 4) where their rows
// are aligned to that, and each line that the workgroups of a die share is asked for ahead by one of them.
// CUT: K ends inside a block.
template <int TT, int FT, int WT, int WF, int SB>
struct Tile {
  static constexpr int kWaves = WT * WF;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRowsA = 32 * TT * WT, kRowsW = 32 * FT * WF;
  static constexpr int kCopies = (kRowsA + kRowsW) / 8 / kWaves;   // 16-byte copies of a wave and stage
  static constexpr int kWOff = 0, kAOff = kRowsW * 128;
  // scales of the rows of a, and of (up to 64) blocks of w: SB = 1: one block's with every stage; SB = 4: four
  // blocks' in two buffers of their own
  static constexpr int kScales = (kRowsA + 64) * 4 * SB;
  static constexpr int kStage = (kRowsW + kRowsA) * 128 + (SB == 1 ? kScales : 0);
  static constexpr int kSAOff = SB == 1 ? (kRowsW + kRowsA) * 128 : 2 * kStage;
  static constexpr int kSWOff = kSAOff + kRowsA * 4 * SB;
  static constexpr int kNowhere = 2 * kStage + (SB == 4 ? 2 * kScales : 0);   // 256 SB bytes per wave that nothing reads
  static constexpr int kBytes = kNowhere + 256 * SB * kWaves;
  static constexpr int kScaleWaves = kRowsA / 64;                  // waves that copy scales of a
  static_assert(kRowsW % (8 * kCopies) == 0 && kRowsA % (8 * kCopies) == 0 && kCopies % 2 == 0,
                "a wave copies rows of one operand");
  static_assert(kScaleWaves < kWaves && kRowsA % 64 == 0, "one wave at least copies the scales of w");
  static_assert(128 % (32 * FT) == 0, "a wave's columns share the scales of w");
};

template <int DT, int TT, int FT, int WT, int WF, int SB, bool CUT>
__global__ void __launch_bounds__(64 * WT * WF)
fp8_gemm_tiles(Fp8GemmArgs g, int tiles_m, int tiles_n) {
  using C = Tile<TT, FT, WT, WF, SB>;
  __shared__ __attribute__((aligned(256))) unsigned char lds[C::kBytes];
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
  const bool copies_w = wave < C::kRowsW / 8 / C::kCopies;
  const int row0 = copies_w ? 8 * wave * C::kCopies : 8 * wave * C::kCopies - C::kRowsW;   // first row of this wave's copies
  const int last_row = copies_w ? g.N - 1 - n0 : g.B - 1 - m0;
  // the piece: (l mod 8) ^ ((row / 2) mod 8), row = 8 i + l / 8 (row0 is a multiple of 16)
  const int piece = (lane & 7) ^ (lane >> 4);   // even i; odd i: ^ 4
  uint32_t from[C::kCopies];
#pragma unroll
  for (int i = 0; i < C::kCopies; ++i) {
    const int r = row0 + 8 * i + (lane >> 3);
    from[i] = (uint32_t)(r < last_row ? r : last_row) * (uint32_t)K + 16u * (piece ^ (4 * (i & 1)));
    asm volatile("" : "+v"(from[i]));   // one register each (the product's upper half is not kept)
  }
  const uint8_t* base = copies_w ? g.w + (int64_t)n0 * K : g.a + (int64_t)m0 * K;
  // in a last block that is cut short, pieces past the row's end are copied from zeros
  const int tail = (K & 127) / 16;              // pieces of the last block, 0: whole
  const bool gone[2] = {tail != 0 && piece >= tail, tail != 0 && (piece ^ 4) >= tail};
  // lines of a later stage, brought into the L2 by a copy to a place nothing reads: the workgroups of a row (column)
  // of tiles take every eighth (fourth) row each
  const int r_ahead = copies_w ? row0 + 8 * (lane & 7) + (tm & 7) : row0 + 4 * (lane & 15) + (tn & 3);
  uint32_t from_ahead = (uint32_t)(r_ahead < last_row ? r_ahead : last_row) * (uint32_t)K;
  asm volatile("" : "+v"(from_ahead));
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

  // copies [lo, hi) of stage kb, and with the first the scales.  There is no branch around them (the additions
  // between the instructions would move behind it): a stage past the last copies the last block again.
  auto issue = [&](int kb, int lo, int hi) __attribute__((always_inline)) {
    const uint32_t st = l0 + (kb & 1) * C::kStage;
    const bool end = kb >= nkb - 1;
    kb = kb < nkb ? kb : nkb - 1;
    const uint8_t* at = base + (int64_t)kb * 128;
    if (lo == 0) {
      const uint32_t to = scales_a ? C::kSAOff + 256 * SB * wave : C::kSWOff;
      if constexpr (SB == 1) {
        dma4(sbase + kb, sfrom, st + to);
      } else {
        // with the first of four blocks; with the others one line goes nowhere
        const bool first = (kb & 3) == 0;
        const uint32_t four = l0 + (kb >> 2 & 1) * C::kScales + to;
        dma16(sbase + (kb & ~3), first ? sfrom : 0u, first ? four : l0 + C::kNowhere + 256 * SB * wave);
      }
    }
#pragma unroll
    for (int i = lo; i < hi; ++i) {
      const uint32_t to = st + (wave * C::kCopies + i) * 1024;
      if constexpr (CUT)
        dma16_at(gone[i & 1] && end ? reinterpret_cast<const uint8_t*>(kZeros) : at + from[i], to);
      else
        dma16(at, from[i], to);
    }
  };
  auto issue_ahead = [&](int kb) __attribute__((always_inline)) {
    dma4(base + (int64_t)(kb < nkb ? kb : nkb - 1) * 128, from_ahead, l0 + C::kNowhere + 256 * SB * wave);
  };

  v16f acc[TT][FT];
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[j][i][q] = 0.0f;

  // lane (row r32, half h): pieces h and h + 2 of its row for the first instruction, h + 4 and h + 6 for the second
  const int r32 = lane & 31, h = lane >> 5;
  const uint32_t operand = r32 * 128 + 16 * (h ^ (r32 >> 1 & 7));   // piece h; others: ^ 32, ^ 64, ^ 96
  auto read = [&](uint32_t at) __attribute__((always_inline)) {
    typedef const __attribute__((address_space(3))) u32x4* vptr;
    return *(vptr)(uintptr_t)at;
  };
  auto read1 = [&](uint32_t at) __attribute__((always_inline)) {
    typedef const __attribute__((address_space(3))) float* fptr;
    return *(fptr)(uintptr_t)at;
  };

  // Tile t = (j, i): its block sum is added to the running sum while the next tile's is formed.
  v8i av[2][2], wv[FT][2];
  v16f sum[2];
  float scale[2], sw;
  auto add = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 16; ++q)
      acc[t / FT][t % FT][q] = __builtin_fmaf(sum[t & 1][q], scale[t / FT & 1], acc[t / FT][t % FT][q]);
  };
  const uint32_t wl = l0 + wf * (32 * FT) * 128 + operand, al = l0 + C::kAOff + wt * (32 * TT) * 128 + operand;
  const uint32_t sal = l0 + C::kSAOff + 4 * SB * (wt * 32 * TT + r32);
  const uint32_t swl = l0 + C::kSWOff + 4 * SB * ((n0 % 128 + wf * 32 * FT) / 128);
  auto scales_of = [&](int kb) __attribute__((always_inline)) {
    return SB == 1 ? (kb & 1) * C::kStage : (kb >> 2 & 1) * C::kScales + 4 * (kb & 3);
  };
  auto read_a = [&](int kb, int j) __attribute__((always_inline)) {
    const uint32_t at = al + (kb & 1) * C::kStage;
    av[j & 1][0] = join(read(at + 4096 * j), read((at ^ 32) + 4096 * j));
    av[j & 1][1] = join(read((at ^ 64) + 4096 * j), read((at ^ 96) + 4096 * j));
    scale[j & 1] = read1(sal + scales_of(kb) + 128 * SB * j);
  };
  auto read_w = [&](int kb, int i) __attribute__((always_inline)) {
    const uint32_t at = wl + (kb & 1) * C::kStage;
    wv[i][0] = join(read(at + 4096 * i), read((at ^ 32) + 4096 * i));
    wv[i][1] = join(read((at ^ 64) + 4096 * i), read((at ^ 96) + 4096 * i));
  };

  // Stage kb is computed while stage kb + 1 lands.  Before its last row of tiles everyone's copies of the next
  // stage have landed and everyone's reads of this one are done: the next stage's first operands are read
  // during that row, and the copies of stage kb + 2 follow into this stage's buffer, spread over it and the
  // next stage's first rows.
  constexpr int kParts = TT - 1;
  constexpr int kEach = (C::kCopies + kParts - 1) / kParts;
  constexpr int kRowsOf = (C::kCopies + kEach - 1) / kEach;   // rows of tiles that copies follow
  static_assert(TT % 2 == 0 && kRowsOf < TT, "copies, then the line ahead, then the wait");
  issue(0, 0, C::kCopies);
  issue_ahead(2);
  issue(1, 0, kEach);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kEach + 2) : "memory");
  read_a(0, 0);
#pragma unroll
  for (int i = 0; i < FT; ++i) read_w(0, i);
  sw = read1(swl + scales_of(0));
  for (int kb = 0; kb < nkb; ++kb) {
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      // all but the line ahead have landed
      if (j + 1 == TT) asm volatile("s_waitcnt vmcnt(1) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      scale[j & 1] *= sw;
#pragma unroll
      for (int i = 0; i < FT; ++i) {
        const int t = j * FT + i;
        sum[t & 1] = mfma_block32(wv[i], av[j & 1]);
        if (t >= 1) add(t - 1);
        if (i == 0) {
          if (j + 1 < TT) read_a(kb, j + 1);
          else read_a(kb + 1, 0);
        }
        if (j + 1 == TT) read_w(kb + 1, i);
      }
      if (j + 1 == TT) {
        add(TT * FT - 1);
        sw = read1(swl + scales_of(kb + 1));
      }
      if (j + 1 == TT) {
        issue(kb + 2, 0, kEach);
      } else if (j + 1 < kRowsOf) {
        issue(kb + 1, (j + 1) * kEach, (j + 2) * kEach < C::kCopies ? (j + 2) * kEach : C::kCopies);
      }
      if (j + 1 == kRowsOf || (kRowsOf == 1 && j == 0)) issue_ahead(kb + 3);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy into LDS outlives the workgroup

  const bool vec = g.N % 4 == 0 && ((uintptr_t)g.y % 8) == 0;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int m = m0 + (wt * TT + j) * 32 + r32;
    if (m >= g.B) continue;
    uint16_t* row = (uint16_t*)g.y + (int64_t)m * g.N;
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + (wf * FT + i) * 32 + 8 * q + 4 * h;
        const v4f v = {acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
        if (n < g.N) store4<DT>(row, n, g.N, vec, v);
      }
  }
}

// ---------------------------------------------------------------- small tiles (a few hundred rows)
// Where tiles of the sizes above would leave compute units idle: 64 rows of a by 128 rows of w, eight waves in two
// groups that take the K-blocks in turn, three stage buffers each (two stages in flight while one is computed).
// Bound by the lines between the L2 and the compute units.
constexpr int kSmRowsA = 64, kSmRowsW = 128, kSmStages = 3, kSmGroups = 2, kSmWaves = 4;   // waves of a group
constexpr int kSmCopies = (kSmRowsA + kSmRowsW) / 8 / kSmWaves;                            // of a wave and stage
constexpr int kSmAOff = kSmRowsW * 128, kSmSAOff = (kSmRowsW + kSmRowsA) * 128, kSmSWOff = kSmSAOff + kSmRowsA * 4;
constexpr int kSmStage = kSmSWOff + 256;
static_assert(kSmRowsW % (8 * kSmWaves) == 0 && kSmRowsA == 64, "a copy stays in one operand; one wave copies the scales of a");

template <int DT, bool CUT>
__global__ void __launch_bounds__(64 * kSmWaves * kSmGroups)
fp8_gemm_small(Fp8GemmArgs g, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(256))) unsigned char lds[kSmGroups * kSmStages * kSmStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), group = wave / kSmWaves, gw = wave % kSmWaves;
  // the tiles of one column of tiles (the same rows of w) follow one another on one XCD
  int t = blockIdx.x;
  const int total = tiles_m * tiles_n;
  if (total % 8 == 0) t = (t & 7) * (total / 8) + (t >> 3);
  const int tn = t / tiles_m, tm = t - tn * tiles_m;
  const int K = g.K, nkb = (K + 127) / 128;
  const int m0 = tm * kSmRowsA, n0 = tn * kSmRowsW;
  const uint32_t l0 = lds_addr(lds) + group * (kSmStages * kSmStage);

  // copies: wave w, copy i moves rows 8 (4 i + w) .. + 7 of the stage (rows of w first), lane l the piece (l mod 8)
  // of row l / 8
  uint32_t from[kSmCopies];
  const int tail = (K & 127) / 16;
  const int piece = (lane & 7) ^ (((gw & 1) * 4 + (lane >> 4)) & 7);   // ^ ((row / 2) mod 8), row = 32 i + 8 w + l / 8
  const bool gone = tail != 0 && piece >= tail;
#pragma unroll
  for (int i = 0; i < kSmCopies; ++i) {
    const bool is_w = 32 * i < kSmRowsW;
    const int r = 32 * i + 8 * gw + (lane >> 3) - (is_w ? 0 : kSmRowsW), last = is_w ? g.N - 1 - n0 : g.B - 1 - m0;
    from[i] = (uint32_t)(r < last ? r : last) * (uint32_t)K + 16u * piece;
    asm volatile("" : "+v"(from[i]));   // one register each
  }
  const uint8_t* wbase = g.w + (int64_t)n0 * K;
  const uint8_t* abase = g.a + (int64_t)m0 * K;
  const float* sbase = gw == 0 ? g.as + (int64_t)m0 * nkb : g.ws + (int64_t)(n0 / 128) * nkb;
  const uint32_t sfrom = gw == 0 ? (uint32_t)(lane < g.B - 1 - m0 ? lane : g.B - 1 - m0) * (uint32_t)nkb * 4u : 0u;
  // stage s of this group: block s kSmGroups + group, or again the last block (not used)
  auto issue = [&](int s, uint32_t buf) __attribute__((always_inline)) {
    const int b = s * kSmGroups + group, kb = b < nkb ? b : nkb - 1;
    const bool end = kb == nkb - 1;
#pragma unroll
    for (int i = 0; i < kSmCopies; ++i) {
      const uint8_t* at = (32 * i < kSmRowsW ? wbase : abase) + (int64_t)kb * 128;
      const uint32_t to = l0 + buf + (4 * i + gw) * 1024;
      if constexpr (CUT) dma16_at(gone && end ? reinterpret_cast<const uint8_t*>(kZeros) : at + from[i], to);
      else dma16(at, from[i], to);
    }
    dma4(sbase + kb, sfrom, l0 + buf + (gw == 0 ? kSmSAOff : kSmSWOff));
  };

  const int wt = gw & 1, wf = gw >> 1;   // this wave's 32 rows of a and 64 of w
  const int r32 = lane & 31, h = lane >> 5;
  const uint32_t operand = r32 * 128 + 16 * (h ^ (r32 >> 1 & 7));
  auto read = [&](uint32_t at) __attribute__((always_inline)) {
    typedef const __attribute__((address_space(3))) u32x4* vptr;
    return *(vptr)(uintptr_t)at;
  };
  auto read1 = [&](uint32_t at) __attribute__((always_inline)) {
    typedef const __attribute__((address_space(3))) float* fptr;
    return *(fptr)(uintptr_t)at;
  };
  v16f acc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[i][q] = 0.0f;
  auto compute = [&](uint32_t buf) __attribute__((always_inline)) {
    const uint32_t al = l0 + buf + kSmAOff + wt * 4096 + operand, wl = l0 + buf + wf * 8192 + operand;
    const v8i a[2] = {join(read(al), read(al ^ 32)), join(read(al ^ 64), read(al ^ 96))};
    const float s = read1(l0 + buf + kSmSAOff + 4 * (wt * 32 + r32)) * read1(l0 + buf + kSmSWOff);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const v8i w[2] = {join(read(wl + 4096 * i), read((wl ^ 32) + 4096 * i)),
                        join(read((wl ^ 64) + 4096 * i), read((wl ^ 96) + 4096 * i))};
      const v16f p = mfma_block32(w, a);
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][q] = __builtin_fmaf(p[q], s, acc[i][q]);
    }
  };

  const int steps = (nkb + kSmGroups - 1) / kSmGroups;
  uint32_t buf = 0, fill = 0;
#pragma unroll
  for (int s = 0; s < kSmStages - 1; ++s) {
    issue(s, fill);
    fill += kSmStage;
  }
  for (int s = 0; s < steps; ++s) {
    // this wave's copies of stage s have landed and its reads of the stage before are done; then everyone's
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kSmStages - 2) * (kSmCopies + 1)) : "memory");
    issue(s + kSmStages - 1, fill);
    fill = fill + kSmStage < kSmStages * kSmStage ? fill + kSmStage : 0;
    if (s * kSmGroups + group < nkb) compute(buf);
    buf = buf + kSmStage < kSmStages * kSmStage ? buf + kSmStage : 0;
  }
  // the second group's sums go to the first through LDS
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  v4f* part = reinterpret_cast<v4f*>(lds);
  if (group == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        part[((gw * 2 + i) * 4 + q) * 64 + lane] = v4f{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
  }
  __syncthreads();
  const int m = m0 + wt * 32 + r32;
  if (group == 1 || m >= g.B) return;
  const bool vec = g.N % 4 == 0 && ((uintptr_t)g.y % 8) == 0;
  uint16_t* row = (uint16_t*)g.y + (int64_t)m * g.N;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = n0 + wf * 64 + 32 * i + 8 * q + 4 * h;
      v4f v = part[((gw * 2 + i) * 4 + q) * 64 + lane];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += acc[i][4 * q + r];
      if (n < g.N) store4<DT>(row, n, g.N, vec, v);
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
  using C = Tile<TT, FT, WT, WF, 4>;
  const int tm = (g.B + C::kRowsA - 1) / C::kRowsA, tn = (g.N + C::kRowsW - 1) / C::kRowsW;
  const dim3 grid((unsigned)(tm * tn)), block(C::kThreads);
  const bool cut = g.K % 128 != 0, four = (g.K + 127) / 128 % 4 == 0 && (((uintptr_t)g.as | (uintptr_t)g.ws) % 16) == 0;
  if (four) {
    if (cut) fp8_gemm_tiles<DT, TT, FT, WT, WF, 4, true><<<grid, block, 0, s>>>(g, tm, tn);
    else fp8_gemm_tiles<DT, TT, FT, WT, WF, 4, false><<<grid, block, 0, s>>>(g, tm, tn);
  } else {
    if (cut) fp8_gemm_tiles<DT, TT, FT, WT, WF, 1, true><<<grid, block, 0, s>>>(g, tm, tn);
    else fp8_gemm_tiles<DT, TT, FT, WT, WF, 1, false><<<grid, block, 0, s>>>(g, tm, tn);
  }
}

template <int DT>
void small_tiles(const Fp8GemmArgs& g, hipStream_t s) {
  const int tm = (g.B + kSmRowsA - 1) / kSmRowsA, tn = (g.N + kSmRowsW - 1) / kSmRowsW;
  const dim3 grid((unsigned)(tm * tn)), block(64 * kSmWaves * kSmGroups);
  if (g.K % 128 != 0) fp8_gemm_small<DT, true><<<grid, block, 0, s>>>(g, tm, tn);
  else fp8_gemm_small<DT, false><<<grid, block, 0, s>>>(g, tm, tn);
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
  // The sizes of tiles: microseconds per K-block for a round of tiles over the chip, as measured (K = 4096 to 8192),
  // times the rounds.  64 x 128: 256 at a time (512 x 4096 x 4096: 16 us, with 128 x 128 tiles 27 us); 128 x 128: 512 at
  // a time, faster while there is one per compute unit (2048 x 2048 x 4096: 28 us, with 64 x 128 33 us); 256 x 256: 256
  // at a time (4096 x 8192 x 8192: 254 us; 1000 x 8192 x 8192: 127 us, with 128 x 128 tiles 89 us).
  auto count = [&](int64_t rows, int64_t cols) { return (g.B + rows - 1) / rows * ((g.N + cols - 1) / cols); };
  auto rounds = [](int64_t n, int64_t slots) { return (double)((n + slots - 1) / slots); };
  const int64_t mid = count(128, 128);
  const double small_cost = 0.6 * rounds(count(64, 128), 256);
  const double mid_cost = mid <= 256 ? 0.9 : 1.4 * rounds(mid, 512);
  const double big_cost = 2.0 * rounds(count(256, 256), 256);
  if (big_cost <= small_cost && big_cost <= mid_cost) return tiles<DT, 4, 2, 2, 4>(g, s);
  if (mid_cost < small_cost) return tiles<DT, 2, 2, 2, 2>(g, s);
  return small_tiles<DT>(g, s);
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t s) {
  if (g.out_dtype == kBf16) launch<kBf16>(g, s);
  else launch<kFp16>(g, s);
  return hipGetLastError();
}

}  // namespace nvfp4
