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
#include "fp8_tiles.h"
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

// Four consecutive columns n .. n + 3 of a row, of which those below N exist.  One store of eight bytes at any
// alignment of two (global memory takes those): 3000 x 4098 x 1024 23 us, with four stores 42 us
// (4097 columns, rows at odd places: 32 and 41 us).
template <int DT>
__device__ __forceinline__ void store4(uint16_t* row, int n, int N, const v4f& v) {
  if (n + 4 <= N) {
    u32x2 o;
    o.x = round16<DT>(v[0]) | (uint32_t)round16<DT>(v[1]) << 16;
    o.y = round16<DT>(v[2]) | (uint32_t)round16<DT>(v[3]) << 16;
    __builtin_memcpy(row + n, &o, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (n + i < N) row[n + i] = round16<DT>(v[i]);
  }
}

// Workgroup b of `total` runs on XCD b mod 8: its place when each XCD has one run of consecutive places.
__device__ __forceinline__ int run_of_die(int b, int total) {
  const int die = b & 7, more = total & 7;
  return die * (total >> 3) + (die < more ? die : more) + (b >> 3);
}

// ---------------------------------------------------------------- tiles (many rows)
// BT rows of a by BF rows of w per workgroup, one 128-k block per stage, two stage buffers: the copies of
// the next stage (global -> LDS, 16 bytes a lane) are in flight while a stage is computed.  LDS holds
// the rows' 128 bytes with piece p of row r at p ^ ((r / 2) mod 8): the 16 lanes of an operand read
// touch 16 different places of 16 bytes.
//
// The matrix cores are busy for 57 % of the time: operand reads from LDS, the issue of the copies and the scales' fma do
// not hide behind them fully.  What the copies cost is lines: every 64 x 16 bytes of one are eight lines of the L2, but one
// binary32 scale for each of 64 rows is 64 lines.  So the scales of a row are copied four blocks at a time (SB = 4) where
// their rows are aligned to that (us, against one block at a time: 4096 x 8192 x 8192 239 / 243, x 8176 260 / 267, 1000 x
// 8192 x 8192 82.4 / 83.6, but 2048 x 2048 x 4096 30.2 / 28.8), and each line that the workgroups of a die share is asked
// for ahead by one of them.  4096 x 8192 x 8192: 239 to 255 us by the clocks of the moment, 2.2 PFLOP/s; a library product
// with one scale takes 202 us.
// CUT: K ends inside a block.
template <int TT, int FT, int WT, int WF, int SB>
struct Tile {
  static constexpr int kWaves = WT * WF;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRowsA = 16 * TT * WT, kRowsW = 16 * FT * WF;
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
  static_assert(128 % (16 * FT) == 0, "a wave's columns share the scales of w");
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
    const int t = run_of_die(blockIdx.x, total);
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

  v4f acc[TT][FT];
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int i = 0; i < FT; ++i) acc[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const int r16 = lane & 15, grp = lane >> 4;
  const uint32_t operand = r16 * 128 + 16 * (grp ^ (r16 >> 1 & 7));   // piece grp; piece grp + 4: ^ 64
  auto read = [&](uint32_t at) __attribute__((always_inline)) {
    typedef const __attribute__((address_space(3))) u32x4* vptr;
    return *(vptr)(uintptr_t)at;
  };
  auto read1 = [&](uint32_t at) __attribute__((always_inline)) {
    typedef const __attribute__((address_space(3))) float* fptr;
    return *(fptr)(uintptr_t)at;
  };

  // Tile t = (j, i): its block sum is added to the running sum two instructions later, when it is there.
  v8i av[4], wv[FT];
  v4f sum[3];
  float scale[4], sw;
  auto add = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      acc[t / FT][t % FT][q] = __builtin_fmaf(sum[t % 3][q], scale[t / FT & 3], acc[t / FT][t % FT][q]);
  };
  const uint32_t wl = l0 + C::kWOff + wf * (16 * FT) * 128 + operand, al = l0 + C::kAOff + wt * (16 * TT) * 128 + operand;
  const uint32_t sal = l0 + C::kSAOff + 4 * SB * (wt * 16 * TT + r16);
  const uint32_t swl = l0 + C::kSWOff + 4 * SB * ((n0 % 128 + wf * 16 * FT) / 128);
  auto scales_of = [&](int kb) __attribute__((always_inline)) {
    return SB == 1 ? (kb & 1) * C::kStage : (kb >> 2 & 1) * C::kScales + 4 * (kb & 3);
  };
  auto read_a = [&](int kb, int j) __attribute__((always_inline)) {
    const uint32_t buf = (kb & 1) * C::kStage;
    av[j & 3] = join(read(al + buf + 2048 * j), read((al ^ 64) + buf + 2048 * j));
    scale[j & 3] = read1(sal + scales_of(kb) + 64 * SB * j);
  };
  auto read_w = [&](uint32_t buf, int i) __attribute__((always_inline)) {
    wv[i] = join(read(wl + buf + 2048 * i), read((wl ^ 64) + buf + 2048 * i));
  };

  // Stage kb is computed while stage kb + 1 lands.  Before its last row of tiles everyone's copies of the next
  // stage have landed and everyone's reads of this one are done: the next stage's first operands are read
  // during that row, and the copies of stage kb + 2 follow into this stage's buffer, spread over it and the
  // next stage's first rows.
  constexpr int kEach = TT >= 8 ? 2 : 4;
  constexpr int kAheadRow = C::kCopies / kEach - 1;   // the row after the last copies
  static_assert(TT % 4 == 0 && C::kCopies % kEach == 0 && kAheadRow < TT - 1, "copies, then the line ahead, then the wait");
  issue(0, 0, C::kCopies);
  issue_ahead(2);
  issue(1, 0, kEach);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kEach + 2) : "memory");
  read_a(0, 0);
#pragma unroll
  for (int i = 0; i < FT; ++i) read_w(0, i);
  read_a(0, 1);
  sw = read1(swl + scales_of(0));
  for (int kb = 0; kb < nkb; ++kb) {
    const uint32_t other = (~kb & 1) * C::kStage;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      // all but the line ahead have landed
      if (j + 1 == TT) asm volatile("s_waitcnt vmcnt(1) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (j + 2 < TT) read_a(kb, j + 2);
      if (j + 1 == TT) read_a(kb + 1, 0);
      scale[j & 3] *= sw;
#pragma unroll
      for (int i = 0; i < FT; ++i) {
        const int t = j * FT + i;
        sum[t % 3] = mfma_block(wv[i], av[j & 3]);
        if (t >= 2) add(t - 2);
        if (j + 1 == TT) read_w(other, i);
      }
      if (j + 1 == TT) {
        add(TT * FT - 2);
        add(TT * FT - 1);
        sw = read1(swl + scales_of(kb + 1));
        read_a(kb + 1, 1);
      }
      if (j + 1 == TT) {
        issue(kb + 2, 0, kEach);
      } else if (j < kAheadRow) {
        issue(kb + 1, (j + 1) * kEach, (j + 2) * kEach);
      } else if (j == kAheadRow) {
        issue_ahead(kb + 3);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy into LDS outlives the workgroup

#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int m = m0 + (wt * TT + j) * 16 + r16;
    if (m >= g.B) continue;
    uint16_t* row = (uint16_t*)g.y + (int64_t)m * g.N;
#pragma unroll
    for (int i = 0; i < FT; ++i) {
      const int n = n0 + (wf * FT + i) * 16 + 4 * grp;
      if (n < g.N) store4<DT>(row, n, g.N, acc[j][i]);
    }
  }
}

// ---------------------------------------------------------------- small tiles (a few hundred rows)
// Where tiles of the sizes above would leave compute units idle: 64 rows of a by 32, 64 or 128 rows of w, eight waves in
// groups of W that take the K-blocks in turn, S stage buffers each: S - 1 stages are in flight while the block of one
// more is in registers and worked on.  A compute unit takes in about 33 bytes a clock of what is not in its L2 yet (of
// lines that are, 64), however early it asks: issuing the copies is what the waves wait for, so as many compute units
// as possible are kept busy, and the scales, a line for each row, are copied four blocks at a time.  777 x 2120 x 7184
// 29.5 us, 64 x 8192 x 8192 14.0 us (4.9 TB/s).
constexpr int kSmRowsA = 64, kSmAll = 8;   // waves
template <int FT, int W, int S>
struct Small {
  static constexpr int kGroups = kSmAll / W;
  static constexpr int kRowsW = 16 * FT * W;
  static constexpr int kCopies = (kSmRowsA + kRowsW) / 8 / W;   // of a wave and stage
  static constexpr int kAOff = kRowsW * 128, kStage = (kRowsW + kSmRowsA) * 128;
  // scales of four blocks at a time, in four buffers: 64 rows of a, then w
  static constexpr int kScales = kGroups * S * kStage, kScalesW = 64 * 16, kFour = kScalesW + 256;
  static constexpr int kNowhere = kScales + 4 * kFour, kBytes = kNowhere + 256;
  static_assert(kSmRowsA == 64 && kRowsW % (8 * W) == 0, "a copy stays in one operand");
  static_assert(kGroups == 2 || kGroups == 4, "a stage has two or four blocks");
};

template <int DT, int FT, int W, int S, bool CUT>
__global__ void __launch_bounds__(64 * kSmAll)
fp8_gemm_small(Fp8GemmArgs g, int tiles_m, int tiles_n) {
  using C = Small<FT, W, S>;
  __shared__ __attribute__((aligned(256))) unsigned char lds[C::kBytes];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), group = wave / W, gw = wave % W;
  // the tiles of one column of tiles (the same rows of w) follow one another on one XCD
  const int t = run_of_die(blockIdx.x, tiles_m * tiles_n);
  const int tn = t / tiles_m, tm = t - tn * tiles_m;
  const int K = g.K, nkb = (K + 127) / 128;
  const int m0 = tm * kSmRowsA, n0 = tn * C::kRowsW;
  const uint32_t lds0 = lds_addr(lds), l0 = lds0 + group * (S * C::kStage);

  // copies: wave w, copy i moves rows 8 (W i + w) .. + 7 of the stage (rows of w first), lane l the piece (l mod 8)
  // of row l / 8
  uint32_t from[C::kCopies];
  const int tail = (K & 127) / 16;
  const int piece = (lane & 7) ^ (((gw & 1) * 4 + (lane >> 4)) & 7);   // ^ ((row / 2) mod 8), row = 8 W i + 8 w + l / 8
  const bool gone = tail != 0 && piece >= tail;
#pragma unroll
  for (int i = 0; i < C::kCopies; ++i) {
    const bool is_w = 8 * W * i < C::kRowsW;
    const int r = 8 * W * i + 8 * gw + (lane >> 3) - (is_w ? 0 : C::kRowsW), last = is_w ? g.N - 1 - n0 : g.B - 1 - m0;
    from[i] = (uint32_t)(r < last ? r : last) * (uint32_t)K + 16u * piece;
    asm volatile("" : "+v"(from[i]));   // one register each
  }
  const uint8_t* wbase = g.w + (int64_t)n0 * K;
  const uint8_t* abase = g.a + (int64_t)m0 * K;
  // the scales: waves 0 to 3 copy four blocks of 16 rows of a each, the others those of w (all lanes' rows the same)
  const bool of_a = wave < 4;
  const int srow = 16 * wave + (lane >> 2);
  const uint32_t sfrom = of_a ? (uint32_t)(srow < g.B - 1 - m0 ? srow : g.B - 1 - m0) * (uint32_t)nkb * 4u : 0u;
  const float* wscale = g.ws + (int64_t)(n0 / 128) * nkb;
  const float* sbase = of_a ? g.as + (int64_t)m0 * nkb : wscale;
  // stage s of this group: block s kGroups + group, or again the last block (not used)
  auto issue = [&](int s, uint32_t buf, int first, int past) __attribute__((always_inline)) {
    const int b = s * C::kGroups + group, kb = b < nkb ? b : nkb - 1;
    const bool end = kb == nkb - 1;
#pragma unroll
    for (int i = 0; i < C::kCopies; ++i) {
      if (i < first || i >= past) continue;
      const uint8_t* at = (8 * W * i < C::kRowsW ? wbase : abase) + (int64_t)kb * 128;
      const uint32_t to = l0 + buf + (W * i + gw) * 1024;
      if constexpr (CUT) dma16_at(gone && end ? reinterpret_cast<const uint8_t*>(kZeros) : at + from[i], to);
      else dma16(at, from[i], to);
    }
    if (past < C::kCopies) return;
    const int first4 = s * C::kGroups & ~3, sb = first4 + (lane & 3);
    const uint32_t at = 4u * (uint32_t)(sb < nkb ? sb : nkb - 1);
    const uint32_t four = lds0 + C::kScales + (first4 / 4 & 3) * C::kFour;
    if (C::kGroups == 4 || s % 2 == 0) dma4(sbase, sfrom + at, four + (of_a ? 256 * wave : C::kScalesW));
    else dma4(wscale, 0u, lds0 + C::kNowhere);   // every stage is the same number of copies
  };

  const int wt = gw & 1, wf = gw >> 1;   // this wave's 32 rows of a and 32 FT of w
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
  v16f acc[FT];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[i][q] = 0.0f;
  // operands and scale of a block in registers: read while the block before is worked on
  v8i a[2][2], w[2][FT][2];
  float scale[2];
  auto fetch = [&](int s, uint32_t buf, int set) __attribute__((always_inline)) {
    const uint32_t al = l0 + buf + C::kAOff + wt * 4096 + operand, wl = l0 + buf + wf * (4096 * FT) + operand;
    a[set][0] = join(read(al), read(al ^ 32));
    a[set][1] = join(read(al ^ 64), read(al ^ 96));
#pragma unroll
    for (int i = 0; i < FT; ++i) {
      w[set][i][0] = join(read(wl + 4096 * i), read((wl ^ 32) + 4096 * i));
      w[set][i][1] = join(read((wl ^ 64) + 4096 * i), read((wl ^ 96) + 4096 * i));
    }
    const int kb = s * C::kGroups + group;
    const uint32_t four = lds0 + C::kScales + (kb / 4 & 3) * C::kFour + 4 * (kb & 3);
    scale[set] = read1(four + 16 * (wt * 32 + r32)) * read1(four + C::kScalesW);
  };
  const int steps = (nkb + C::kGroups - 1) / C::kGroups;
#pragma unroll
  for (int s = 0; s < S; ++s) issue(s, s * C::kStage, 0, C::kCopies);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S - 1) * (C::kCopies + 1)) : "memory");
  fetch(0, 0, 0);
  uint32_t buf = 0;   // of the stage at hand
  auto step = [&](int s, int set) __attribute__((always_inline)) {
    const uint32_t next = buf + C::kStage < S * C::kStage ? buf + C::kStage : 0;
    // this wave's copies of the next stage have landed and its reads of this one are done; then everyone's
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * (C::kCopies + 1)) : "memory");
    // the copies (a compute unit takes 16 clocks for each) go between the products: before them all, a wave would
    // stand and wait to issue them for as long as the products take
    v16f p[FT];
#pragma unroll
    for (int i = 0; i < FT; ++i) {
      p[i] = mfma_block32(w[set][i], a[set]);
      __builtin_amdgcn_sched_barrier(0);
      issue(s + S, buf, C::kCopies * i / FT, C::kCopies * (i + 1) / FT);
      __builtin_amdgcn_sched_barrier(0);
    }
    fetch(s + 1, next, set ^ 1);
    buf = next;
    if (s * C::kGroups + group < nkb) {
#pragma unroll
      for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][q] = __builtin_fmaf(p[i][q], scale[set], acc[i][q]);
    }
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, 0);
    if (s + 1 < steps) step(s + 1, 1);
  }
  // the other groups' sums go to the first through LDS
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  v4f* part = reinterpret_cast<v4f*>(lds);
  if (group > 0) {
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        part[(((wave - W) * FT + i) * 4 + q) * 64 + lane] =
            v4f{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
  }
  __syncthreads();
  const int m = m0 + wt * 32 + r32;
  if (group > 0 || m >= g.B) return;
  uint16_t* row = (uint16_t*)g.y + (int64_t)m * g.N;
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = n0 + wf * (32 * FT) + 32 * i + 8 * q + 4 * h;
      v4f v = {acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
#pragma unroll
      for (int h = 1; h < C::kGroups; ++h) {
        const v4f o = part[((((h - 1) * W + gw) * FT + i) * 4 + q) * 64 + lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += o[r];
      }
      if (n < g.N) store4<DT>(row, n, g.N, v);
    }
}

// ---------------------------------------------------------------- streams (few rows)
// A workgroup holds all rows of a (up to 8; the instruction has room for 16) against 16 rows of w; its waves take the K-blocks in turn, kAhead of
// them in flight a wave, straight from memory into registers (every byte of w is read once, by one wave), and their
// sums are joined through LDS.  Bound by the latency of a chain of K / 128 / (8 kAhead) loads: 1 x 4096 x 4096 6.6 us.
constexpr int kAhead = 4, kStreamWaves = 8;
template <int DT>
__global__ void __launch_bounds__(64 * kStreamWaves)
fp8_gemm_stream(Fp8GemmArgs g) {
  constexpr int NW = kStreamWaves;
  __shared__ v4f part[NW][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, grp = lane >> 4;
  const int K = g.K, nkb = (K + 127) / 128;
  const int n0 = blockIdx.x * 16;
  const int wr = n0 + r16 < g.N ? n0 + r16 : g.N - 1, ar = r16 < g.B ? r16 : g.B - 1;
  const uint8_t* wrow = g.w + (int64_t)wr * K;
  const uint8_t* arow = g.a + (int64_t)ar * K;
  const float* srow = g.as + (int64_t)ar * nkb;
  const float* swrow = g.ws + (int64_t)(n0 / 128) * nkb;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](const v8i& w, const v8i& a, float scale) __attribute__((always_inline)) {
    const v4f p = mfma_block(w, a);
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = __builtin_fmaf(p[q], scale, acc[q]);
  };

  // K-blocks that are whole; a last one that is not goes through the masked turn below
  const int whole = K / 128;
  for (int kb = wave; kb < whole; kb += NW * kAhead) {
    u32x4 wq[kAhead][2], aq[kAhead][2];
    float sa[kAhead], sw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int b = kb + NW * u < whole ? kb + NW * u : kb;   // past the end: again the first, not used
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wq[u][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow + 16 * grp + (int64_t)b * 128 + 64 * h));
        aq[u][h] = *reinterpret_cast<const u32x4*>(arow + 16 * grp + (int64_t)b * 128 + 64 * h);
      }
      sa[u] = srow[b];
      sw[u] = swrow[b];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (u > 0 && kb + NW * u >= whole) break;   // the same for the whole wave
      add(join(wq[u][0], wq[u][1]), join(aq[u][0], aq[u][1]), sa[u] * sw[u]);
    }
  }
  if (whole < nkb && wave == whole % NW) {
    // pieces of 16 bytes past the row's end count as zeros; what is read in their place is the row's first piece
    const int valid = (K & 127) / 16;
    const bool in[2] = {grp < valid, grp + 4 < valid};
    u32x4 wv[2], av[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t o = in[h] ? (int64_t)whole * 128 + 64 * h + 16 * grp : 0;
      const u32x4 zero = {0, 0, 0, 0};
      wv[h] = *reinterpret_cast<const u32x4*>(wrow + o);
      av[h] = *reinterpret_cast<const u32x4*>(arow + o);
      if (!in[h]) wv[h] = av[h] = zero;
    }
    add(join(wv[0], wv[1]), join(av[0], av[1]), srow[whole] * swrow[whole]);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int v = 1; v < NW; ++v) {
    const v4f p = part[v][lane];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] += p[q];
  }
  const int n = n0 + 4 * grp;
  if (r16 < g.B && n < g.N) store4<DT>((uint16_t*)g.y + (int64_t)r16 * g.N, n, g.N, acc);
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

template <int DT, int FT, int W, int S>
void small_tiles(const Fp8GemmArgs& g, hipStream_t s) {
  constexpr int kRowsW = Small<FT, W, S>::kRowsW;
  const int tm = (g.B + kSmRowsA - 1) / kSmRowsA, tn = (g.N + kRowsW - 1) / kRowsW;
  const dim3 grid((unsigned)(tm * tn)), block(64 * kSmAll);
  if (g.K % 128 != 0) fp8_gemm_small<DT, FT, W, S, true><<<grid, block, 0, s>>>(g, tm, tn);
  else fp8_gemm_small<DT, FT, W, S, false><<<grid, block, 0, s>>>(g, tm, tn);
}

template <int DT>
void stream(const Fp8GemmArgs& g, hipStream_t s) {
  fp8_gemm_stream<DT><<<dim3((unsigned)((g.N + 15) / 16)), dim3(64 * kStreamWaves), 0, s>>>(g);
}

constexpr bool is(Fp8Tiles t, int rows, int cols, int threads) {
  return kFp8TileSizes[t].rows == rows && kFp8TileSizes[t].cols == cols && kFp8TileSizes[t].threads == threads;
}
static_assert(is(kFp8Tiles64x32, kSmRowsA, Small<1, 2, 3>::kRowsW, 64 * kSmAll) &&
              is(kFp8Tiles64x64, kSmRowsA, Small<1, 4, 4>::kRowsW, 64 * kSmAll) &&
              is(kFp8Tiles64x128, kSmRowsA, Small<2, 4, 3>::kRowsW, 64 * kSmAll) &&
              is(kFp8Tiles128x128, Tile<4, 4, 2, 2, 4>::kRowsA, Tile<4, 4, 2, 2, 4>::kRowsW, Tile<4, 4, 2, 2, 4>::kThreads) &&
              is(kFp8Tiles256x256, Tile<8, 4, 2, 4, 4>::kRowsA, Tile<8, 4, 2, 4, 4>::kRowsW, Tile<8, 4, 2, 4, 4>::kThreads),
              "the kernels have the sizes that they are chosen by");

template <int DT>
void launch(const Fp8GemmArgs& g, hipStream_t s) {
  switch (fp8_tiles(g.B, g.N)) {
    case kFp8Stream: return stream<DT>(g, s);
    case kFp8Tiles64x32: return small_tiles<DT, 1, 2, 3>(g, s);
    case kFp8Tiles64x64: return small_tiles<DT, 1, 4, 4>(g, s);
    case kFp8Tiles64x128: return small_tiles<DT, 2, 4, 3>(g, s);
    case kFp8Tiles128x128: return tiles<DT, 4, 4, 2, 2>(g, s);
    case kFp8Tiles256x256: return tiles<DT, 8, 4, 2, 4>(g, s);
  }
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t s) {
  if (g.out_dtype == kBf16) launch<kBf16>(g, s);
  else launch<kFp16>(g, s);
  return hipGetLastError();
}

}  // namespace nvfp4
