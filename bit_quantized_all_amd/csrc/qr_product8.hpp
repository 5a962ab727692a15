// qr_product8.hpp -- gfx950 kernels of the products of 8-bit rows
// (include/qr_rows.h): y = x W^T for one weight or one per group of rows.
//
// y[m][c] = (sum over k of x[m][k] w[c][k]) xs[m] ws[c], codes of signed bytes.
// The sum is a whole number below 2^31 (k <= QR_MAX_ROW_K), which the matrix
// unit's 32-bit sums hold without rounding, in whatever order they are taken; so
// k may be shared out at will.  It is rounded once, to fp32, when it is scaled.
#pragma once

#include "qr_product.hpp"
#include "qr_rows.h"

namespace qr {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kRowRun = 128;  // bytes that a row of codes is padded to a multiple of

// Dense products have offsets == nullptr and one expert; `blocks` counts the
// runs of a row.
struct Product8Args : ProductArgs {
  const float* xs;
  const float* ws;
};

// A sum times the scales of its two rows, in the range of fp32 at every step where
// the result is: |sum| is at least 1, below 2^31, a scale at most 2^121 (the
// largest |x| over 127).  A small first scale is multiplied as it is, a large one by
// 2^-32, after which the second may be as small as there are.
__device__ __forceinline__ float scaled(int sum, float xs, float ws) {
  const bool large = xs > 0x1p64f;
  return (float)sum * (large ? xs * 0x1p-32f : xs) * ws * (large ? 0x1p32f : 1.0f);
}

// ---------------------------------------------------------------------------
// fragments from memory
// ---------------------------------------------------------------------------

// One workgroup of KW waves multiplies 16 MF rows of x by 16 NF rows of the
// weight (gated: NF / 2 fragments of the gate rows and as many of the up rows).
// The waves share the runs of k, wave w has runs w, w + KW, ...; their sums, whole
// numbers, are added up in LDS in whatever order.  The matrix unit's product is 16
// x 16 x 64: lane (r = lane & 15, g = lane >> 4) holds 16 bytes of row r of either
// side, and which bytes of k they are does not matter as long as both sides have
// the same.  The weight is the unit's A, so that a lane gets four neighbouring
// columns of one row of y.
//
// Bound by memory where the weight is all there is to read (16 rows, gated, n = k =
// 8192: 27 us, 5 TB/s; 64 tokens of 8 of 64 experts with 1024 x 2048, gated: 53 us, as
// much), by what a CU takes from L2, 50 bytes a ns, where rows of x are read beside it (137
// x 5003 x 4129: 462 KB a workgroup, 9 of 18 us), and by latency below (1 x 4096 x 4096: 5.2).
//
// Fragments come straight from memory, 64 bytes of 16 rows at a time, the next
// run's while one is multiplied.  The workgroups begin at different runs: rows lie a
// power of two apart, and if all of them read the same columns of their rows at the
// same time, they meet in a few of the memory's channels (16 rows, gated, n = k = 8192:
// 28.2 us and 33.0 on the device; n = k = 8192: 14.1 and 20.9).
template <int DT, bool GATED, int MF, int NF, int KW>
__global__ __launch_bounds__(kWave* KW) void fragments8_kernel(Product8Args a) {
  constexpr int HALVES = GATED ? 2 : 1, OUT = NF / HALVES;
  static_assert(OUT * HALVES == NF, "as many gate as up fragments");
  __shared__ int sums[MF][NF][4][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, g = lane >> 4;
  RowTile rt = find_rows<16 * MF>(a, a.tile0 + blockIdx.x / a.ntiles);
  if (rt.m0 >= rt.m1) return;
  rt.zero |= a.xrows == 0;  // every row number is out of range then
  const int n0 = (int)(blockIdx.x % a.ntiles) * 16 * OUT;
  const long long row_bytes = (long long)a.blocks * kRowRun;
  for (int t = threadIdx.x; t < MF * NF * 4 * kWave; t += kWave * KW) (&sums[0][0][0][0])[t] = 0;

  if (!rt.zero && wave < a.blocks) {
    struct Set {
      i32x4 w[2][NF], x[2][MF];
    };
    // columns past the last repeat it, rows past the end the last, rows of no source the first of x
    const uint8_t *x[MF], *w[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int c = n0 + 16 * (f % OUT) + r;
      w[f] = a.w + (((long long)rt.expert * HALVES + f / OUT) * a.n + (c < a.n ? c : a.n - 1)) * row_bytes + 16 * g;
    }
    const int runs = (a.blocks - wave + KW - 1) / KW;
    const int turn = (int)((blockIdx.x / kXCDs * 0x9E3779B1u >> 16) % (unsigned)runs);
    auto at = [&](int run) {
      run += turn;
      return (size_t)(wave + KW * (run < runs ? run : run - runs)) * kRowRun;
    };
    auto load_w = [&](Set& to, int run) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) to.w[h][f] = *reinterpret_cast<const i32x4*>(w[f] + at(run) + 64 * h);
    };
    auto load_x = [&](Set& to, int run) {
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) to.x[h][i] = *reinterpret_cast<const i32x4*>(x[i] + at(run) + 64 * h);
    };
    i32x4 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[i][f] = i32x4{0, 0, 0, 0};
    auto multiply = [&](const Set& s) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int f = 0; f < NF; ++f) acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(s.w[h][f], s.x[h][i], acc[i][f], 0, 0, 0);
    };
    Set p, q;
    // the first weights need not wait for the numbers of the rows of x, which are a trip to memory of their own
    load_w(p, 0);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = rt.m0 + 16 * i + r;
      const long long s = source_row(a, m < rt.m1 ? m : rt.m1 - 1);
      x[i] = a.x + (s < 0 ? 0 : s) * row_bytes + 16 * g;
    }
    load_x(p, 0);
    // no branch around a load, which would make the products before it wait for it
    int b = 0;
    for (; b + 2 < runs; b += 2) {
      load_w(q, b + 1);
      load_x(q, b + 1);
      multiply(p);
      load_w(p, b + 2);
      load_x(p, b + 2);
      multiply(q);
    }
    if (b + 1 < runs) {
      load_w(q, b + 1);
      load_x(q, b + 1);
      multiply(p);
      multiply(q);
    } else {
      multiply(p);
    }
    __syncthreads();  // sums are zero
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          __hip_atomic_fetch_add(&sums[i][f][j][lane], acc[i][f][j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  } else {
    __syncthreads();
  }
  __syncthreads();
  // fragment (i, f) of y is stored by wave (i OUT + f) % KW
  for (int frag = wave; frag < MF * OUT; frag += KW) {
    const int i = frag / OUT, f = frag % OUT;
    const int m = rt.m0 + 16 * i + r, c = n0 + 16 * f + 4 * g;
    if (m >= rt.m1 || c >= a.n) continue;
    const long long src = rt.zero ? -1 : source_row(a, m);
    const float xs = src >= 0 ? a.xs[src] : 0.0f;
    const float* ws = a.ws + (long long)(rt.zero ? 0 : rt.expert) * HALVES * a.n + c;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int cj = c + j < a.n ? j : a.n - 1 - c;
      const float p = scaled(sums[i][f][j][lane], xs, ws[cj]);
      v[j] = GATED ? gate(p, scaled(sums[i][NF - OUT + f][j][lane], xs, ws[(GATED ? a.n : 0) + cj])) : p;
      if (src < 0) v[j] = 0.0f;
    }
    uint8_t* to = a.y + 2 * (m * a.ldy + c);
    const u32x2 o = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
    if (c + 4 <= a.n) {
      *reinterpret_cast<u32x2_any*>(to) = o;
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (c + j < a.n) reinterpret_cast<uint16_t*>(to)[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

// Number of row tiles that find_rows() hands out, of groups whose offsets are in order or not: every wave
// counts them on its own, a lane an expert.
template <int BM>
__device__ __forceinline__ int count_tiles(const ProductArgs& a) {
  const int lane = threadIdx.x & (kWave - 1);
  int count = 0, top = 0;
  for (int e0 = 0; e0 <= a.experts; e0 += kWave) {
    const int e = e0 + lane;  // e == experts: the rows of no expert
    int lo = a.slots, hi = a.slots;
    if (e <= a.experts) {
      lo = clampi(a.offsets[e], 0, a.slots);
      hi = e < a.experts ? clampi(a.offsets[e + 1], 0, a.slots) : a.slots;
    }
    // an offset below an earlier one counts as that one
    lo = lo > top ? lo : top;
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) {
      const int o = __shfl_up(lo, s);
      if (lane >= s && o > lo) lo = o;
    }
    hi = hi > lo ? hi : lo;
    top = __builtin_amdgcn_readlane(hi, kWave - 1);
    int mine = hi > lo ? (hi - lo + BM - 1) / BM : 0;
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) mine += __shfl_xor(mine, s);
    count += mine;
  }
  return __builtin_amdgcn_readfirstlane(count);
}

// The workgroup's tile.  Of groups the launch is an upper bound on the tiles: those that there are are dealt to the XCDs.
// An XCD's run of them goes through a group in bands of up to kGroupBand row tiles by all columns, which end with the
// group, so that its weight is read no more often than it has bands (8192 tokens, 2 of 16 experts, gated, 4096 x 4096, in
// turn on one card: 585 us, and 603 with bands of 4 that go on from one group into the next; cards differ by more, 570 to 602).
constexpr int kGroupBand = 8;
template <int BM>
__device__ __forceinline__ RowTile find_tile(const ProductArgs& a, int& col) {
  if (!a.offsets) {
    const TileIndex t = tile_index(blockIdx.x, gridDim.x, a.ntiles);
    col = t.col;
    return find_rows<BM>(a, a.tile0 + t.row);
  }
  const int here = min(count_tiles<BM>(a) - a.tile0, (int)(gridDim.x / a.ntiles)), total = here * a.ntiles;
  RowTile rt = {};
  col = 0;
  if ((int)blockIdx.x >= total) return rt;
  const int xcd = blockIdx.x % kXCDs, rest = total % kXCDs;
  const int t = xcd * (total / kXCDs) + (xcd < rest ? xcd : rest) + blockIdx.x / kXCDs;
  int begin = 0, tiles = 0;
  rt = find_rows<BM>(a, a.tile0 + t / a.ntiles, &begin, &tiles);                                 // of the same group
  const int first = max(begin - a.tile0, 0), rows = min(begin + tiles - a.tile0, here) - first;  // in this launch
  const int in = t - first * a.ntiles, band = in / (kGroupBand * a.ntiles), at = in - band * kGroupBand * a.ntiles;
  const int high = min(rows - band * kGroupBand, kGroupBand);
  col = at / high;
  return find_rows<BM>(a, a.tile0 + first + band * kGroupBand + at % high);
}

// A workgroup of WM x WN waves computes a tile of 16 WM MI rows of x by 16 WN NI
// rows of the weight, each wave MI x NI fragments.  A stage is one run of 128
// bytes of every row; it goes to LDS without a stop in registers while the one
// before is multiplied, in two buffers.
//
// LDS: a row is 8 units of 16 bytes, unit u of row R at place u ^ (R / 2 % 8), so
// that 16 lanes that read one unit of 16 rows hit all 64 banks; the lanes that
// load it take their units in that order.
//
// What bounds it is the clock, which the products pull down to 1.9 GHz or so, and
// what a CU takes from L2, 12 to 14 TB/s in all: 8192 x 8192 x 8192 in 418 to 447 us
// (2460 to 2630 TOP/s; the unit alone, on such codes, runs at 4280) with the unit
// busy 67 % of the time; 340 without the loads, 413 without the reads of LDS, 410
// without the scales and stores, 288 of products alone.  So a tile is as large as
// registers allow, and the product is 16 x 16 x 64: at 32 x 32 x 32 the unit draws
// more (3600 TOP/s alone, 484 to 490 us here).  Two buffers of 64 KB, of runs of 128
// bytes, did better than four or five of 64 bytes (518 to 523, at 32 x 32 x 32), and as
// well as a ring of five half stages (440); the smaller tiles have three and four, for
// which there is room.
//
// The column fragments of a wave interleave: row 4 q + j of fragment f is column 4
// OUT q + 4 f + j, so that a lane has 4 OUT neighbours of a row of y and four
// lanes a run of it.  Gated: the first half of a wave's fragments are gate rows,
// the second the same columns' up rows.
template <int DT, bool GATED, int WM, int WN, int MI, int NI, int NB>
__global__ __launch_bounds__(kWave* WM* WN, 2) void tiles8_kernel(Product8Args a) {
  constexpr int WAVES = WM * WN, HALVES = GATED ? 2 : 1, OUT = NI / HALVES;
  static_assert(OUT * HALVES == NI, "as many gate as up fragments");
  constexpr int BM = 16 * WM * MI, BN = 16 * WN * NI, COLS = 16 * OUT;  // COLS: of y of one wave
  constexpr int XI = BM / 8 / WAVES, WI = BN / 8 / WAVES, LOADS = XI + WI;  // of one wave in a stage: 8 rows each
  static_assert(XI * 8 * WAVES == BM && WI * 8 * WAVES == BN, "the waves share the loads evenly");
  // A stage is 2 steps of 64 bytes, each MI slots of NI products with one fragment of x.  Fragments of x
  // are read from LDS kAhead slots before they are multiplied, into a ring; those of the weight a step before.
  constexpr int SLOTS = 2 * MI, kAhead = 3, kRing = 4;
  static_assert(SLOTS % kRing == 0 && MI >= NI && MI > kAhead, "rings begin anew with each stage");
  __shared__ i32x4 lds[NB][BM + BN][8];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int r = lane & 15, g = lane >> 4;
  int col;
  RowTile rt = find_tile<BM>(a, col);
  if (rt.m0 >= rt.m1) return;
  rt.zero |= a.xrows == 0;  // every row number is out of range then
  const int n0 = col * (BN / HALVES);
  const long long row_bytes = (long long)a.blocks * kRowRun;

  i32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int f = 0; f < NI; ++f) acc[i][f] = i32x4{0, 0, 0, 0};
  const int c0 = n0 + COLS * wn + 4 * OUT * g;  // the lane's columns of y
  const float* ws = a.ws + (long long)(rt.zero ? 0 : rt.expert) * HALVES * a.n;
  float wscale[HALVES][4 * OUT], xscale[MI];
  int src[MI];  // rows of x of the lane's rows of y
#pragma unroll
  for (int q = 0; q < HALVES; ++q)
#pragma unroll
    for (int j = 0; j < 4 * OUT; ++j) wscale[q][j] = 0.0f;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    xscale[i] = 0.0f;
    src[i] = -1;
  }

  if (!rt.zero) {
    auto place = [](int row) { return (row >> 1) & 7; };
    // load l of this wave brings rows 8 (WI wave + l) + lane / 8 of the tile's weight rows; columns past the last
    // repeat it
    const uint8_t* wbase[WI];
    uint32_t woff[WI];
#pragma unroll
    for (int l = 0; l < WI; ++l) {
      const int R = 8 * (WI * wave + l), f = R / 16 % NI, q = R % 16 + (lane >> 3);
      const int c = COLS * (R / 16 / NI) + 4 * OUT * (q >> 2) + 4 * (f % OUT) + (q & 3);
      wbase[l] = a.w + (((long long)rt.expert * HALVES + f / OUT) * a.n + n0) * row_bytes;
      woff[l] = (uint32_t)(n0 + c < a.n ? c : a.n - 1 - n0) * (uint32_t)row_bytes + 16 * ((lane & 7) ^ place(q));
    }
    // rows past the end repeat the last, rows of no source the first of x
    const uint8_t* xp[XI];
#pragma unroll
    for (int l = 0; l < XI; ++l) {
      const int R = 8 * (XI * wave + l) + (lane >> 3), m = rt.m0 + R;
      const long long s = source_row(a, m < rt.m1 ? m : rt.m1 - 1);
      xp[l] = a.x + (s < 0 ? 0 : s) * row_bytes + 16 * ((lane & 7) ^ place(R));
    }
    // the scales of the end: asked for here, without branches around their loads, so that nobody waits for them there
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int m = rt.m0 + 16 * (MI * wm + i) + r;
      src[i] = (int)source_row(a, m < rt.m1 ? m : rt.m1 - 1);  // below 2^30
    }
    const uint32_t base = lds_address(&lds[0][0][0]);
    auto fetch = [&](int st, int buf, int l) {
      const uint32_t to = base + (uint32_t)(buf * (BM + BN) * kRowRun);
      if (l < WI)
        load_to_lds(wbase[l < WI ? l : 0] + (size_t)st * kRowRun, woff[l < WI ? l : 0],
                    to + (uint32_t)kRowRun * BM + 1024u * (WI * wave + l));
      else
        load_to_lds(xp[l < WI ? 0 : l - WI] + (size_t)st * kRowRun, to + 1024u * (XI * wave + l - WI));
    };
    i32x4 x[kRing], w[2][NI];
    auto read_x = [&](int buf, int t) {
      const int R = 16 * (MI * wm + t % MI) + r;
      x[t % kRing] = lds[buf][R][(4 * (t / MI) + g) ^ place(r)];
    };
    auto read_w = [&](int buf, int s, int f) { w[s][f] = lds[buf][BM + 16 * (NI * wn + f) + r][(4 * s + g) ^ place(r)]; };
    const int stages = a.blocks;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b < stages) {
#pragma unroll
        for (int l = 0; l < LOADS; ++l) fetch(b, b, l);
      }
    }
    // (a wait for as many loads as were asked for after the first stage's also covers those of the scales)
#pragma unroll
    for (int q = 0; q < HALVES; ++q)
#pragma unroll
      for (int j = 0; j < 4 * OUT; ++j) wscale[q][j] = ws[q * a.n + (c0 + j < a.n ? c0 + j : a.n - 1)];
#pragma unroll
    for (int i = 0; i < MI; ++i) xscale[i] = a.xs[src[i] < 0 ? 0 : src[i]];
    if (NB <= stages) loads_done<(NB - 1) * LOADS>(); else loads_done<0>();
    stage_barrier();
#pragma unroll
    for (int f = 0; f < NI; ++f) read_w(0, 0, f);
#pragma unroll
    for (int t = 0; t < kAhead; ++t) read_x(0, t);
    for (int st = 0, buf = 0; st < stages; ++st) {
      const int next = buf + 1 < NB ? buf + 1 : 0;
#pragma unroll
      for (int t = 0; t < SLOTS; ++t) {
        const int s = t / MI, i = t % MI, left = SLOTS - t;
        if (left == kAhead) {
          // The next stage is there for every wave, and every wave has read the last of this one.
          if (st + NB <= stages) loads_done<(NB - 2) * LOADS>(); else loads_done<0>();
          __builtin_amdgcn_s_waitcnt(0xc07f);  // LDS; a builtin, so that the compiler does not wait once more
          asm volatile("s_barrier" ::: "memory");
        }
        // (after the last stage what lies there is read for nobody)
        if (left > kAhead) read_x(buf, t + kAhead); else read_x(next, t + kAhead - SLOTS);
        if (s == 0 && i < NI) read_w(buf, 1, i);
        if (left <= kAhead) {
#pragma unroll
          for (int f = NI * (kAhead - left) / kAhead; f < NI * (kAhead - left + 1) / kAhead; ++f) read_w(next, 0, f);
          if (st + NB < stages) {
#pragma unroll
            for (int l = LOADS * (kAhead - left) / kAhead; l < LOADS * (kAhead - left + 1) / kAhead; ++l) fetch(st + NB, buf, l);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < NI; ++f) acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s][f], x[t % kRing], acc[i][f], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      buf = next;
    }
  }

#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = rt.m0 + 16 * (MI * wm + i) + r;
    if (m >= rt.m1 || c0 >= a.n) continue;
    uint8_t* to = a.y + 2 * (m * a.ldy + c0);
    uint16_t o[4 * OUT];
#pragma unroll
    for (int p = 0; p < OUT; ++p) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float q = scaled(acc[i][p][j], xscale[i], wscale[0][4 * p + j]);
        v[j] = GATED ? gate(q, scaled(acc[i][NI - OUT + p][j], xscale[i], wscale[HALVES - 1][4 * p + j])) : q;
        if (src[i] < 0) v[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t two = pack2<DT>(v[2 * j], v[2 * j + 1]);
        o[4 * p + 2 * j] = (uint16_t)two;
        o[4 * p + 2 * j + 1] = (uint16_t)(two >> 16);
      }
    }
    if (c0 + 4 * OUT <= a.n) {
      if constexpr (OUT == 1) {
        u32x2 v;
        __builtin_memcpy(&v, o, 8);
        *reinterpret_cast<u32x2_any*>(to) = v;
      } else {
#pragma unroll
        for (int p = 0; p < OUT; p += 2) {
          u32x4 v;
          __builtin_memcpy(&v, o + 4 * p, 16);
          *reinterpret_cast<u32x4_any*>(to + 8 * p) = v;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4 * OUT - 1; ++j)
        if (c0 + j < a.n) reinterpret_cast<uint16_t*>(to)[j] = o[j];
    }
  }
}

qr_status launch_product8(int dt, bool gated, const Product8Args& a, hipStream_t st);

}  // namespace qr
