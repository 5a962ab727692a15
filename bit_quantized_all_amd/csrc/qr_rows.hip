// qr_rows.hip -- the C ABI of include/qr_rows.h: host-side argument checks (no
// HIP call before they pass), and the kernels of the norm, of the 8-bit rows and
// of the router's choice.  The products' kernels are in qr_product8.hpp.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qr.h"
#include "qr_host.hpp"
#include "qr_product8.hpp"
#include "qr_rows.h"

namespace qr {

// ---------------------------------------------------------------------------
// norm, and values to 8-bit rows
// ---------------------------------------------------------------------------

struct RowArgs {
  const uint8_t* x;
  const uint8_t* residual;  // may be nullptr, as may total, y and codes
  const uint8_t* weight;
  uint8_t* total;
  uint8_t* y;
  uint8_t* codes;
  float* scales;
  long long ldx, ldr, ldt, ldy;  // row strides in values
  long long row_bytes;           // of a row of codes
  int rows, k;
  float eps;
};

constexpr int kRowThreads = 256;

// Sum (or largest) of one value a thread over the workgroup, for every thread.
template <typename T, typename OP>
__device__ __forceinline__ T over_group(T v, OP op, T* lds) {
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) v = op(v, __shfl_xor(v, s));
  __syncthreads();  // everyone has read what lay there
  if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kRowThreads / kWave; ++w) v = op(v, lds[w]);
  return v;
}

// Values 8 c .. 8 c + 7 of a row of k in fp32; those from k on are zero.
template <int DT>
__device__ __forceinline__ void load_values(const uint8_t* row, int c, int k, float (&v)[8]) {
  const u32x4 w = 8 * c + 8 <= k ? *reinterpret_cast<const u32x4_any*>(row + 16 * (size_t)c) : load_x8_tail(row, 8 * c, k);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = lo_to_f32<DT>(w[i]);
    v[2 * i + 1] = hi_to_f32<DT>(w[i]);
  }
}

template <int DT>
__device__ __forceinline__ void store_values(uint8_t* row, int c, int k, const float (&v)[8]) {
  const u32x4 o = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
  if (8 * c + 8 <= k) {
    *reinterpret_cast<u32x4_any*>(row + 16 * (size_t)c) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * c + i < k) reinterpret_cast<uint16_t*>(row)[8 * c + i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
  }
}

// The factors of a norm's row: y = (h * up) * down * weight.
struct NormFactors {
  float up, down;
};

// What scales a row to codes: q = round(y * up * inverse).
struct CodeFactors {
  float up, inverse, scale;
};
__device__ __forceinline__ CodeFactors code_factors(uint32_t largest_bits) {
  const float largest = __builtin_bit_cast(float, largest_bits);
  if (largest_bits >= 0x7f800000u) return {0.0f, 0.0f, __builtin_nanf("")};
  if (largest_bits == 0) return {0.0f, 0.0f, 0.0f};
  // 127 / max|x| leaves the range where max|x| is below 2^-121
  const float up = largest < 0x1p-60f ? 0x1p80f : 1.0f;
  return {up, 127.0f / (largest * up), largest / 127.0f};
}
__device__ __forceinline__ uint32_t code(float v, const CodeFactors& f) {
  return f.inverse == 0.0f ? 0u : (uint32_t)(int)fminf(fmaxf(rintf(v * f.up * f.inverse), -127.0f), 127.0f) & 0xffu;
}

// Values 8 c .. 8 c + 7 of a row of k, without a branch that lanes part at: chunks past the last are zero.
template <int DT>
__device__ __forceinline__ u32x4 load_chunk(const uint8_t* row, int c, int chunks, int k) {
  if (k % 8) return load_x8_tail(row, 8 * c, k);
  const u32x4 v = *reinterpret_cast<const u32x4_any*>(row + 16 * (size_t)(c < chunks ? c : chunks - 1));
  return c < chunks ? v : u32x4{0u, 0u, 0u, 0u};
}

// W waves hold a row in registers, C chunks of 8 values a lane: one read and one write of everything, which is what
// bounds it (32768 x 4096 bf16, residual, total and codes: 939 MB in 168 us, 5.6 TB/s; to codes alone 403 MB in 70).
// Sums go over a wave by shuffles, over several through LDS.
template <int DT, bool NORM, int W, int C>
__global__ __launch_bounds__(W > 4 ? kWave * W : kRowThreads) void rows_kernel(RowArgs a) {
  constexpr int ROWS = W < 4 ? 4 / W : 1, LANES = kWave * W;
  __shared__ float lds[ROWS][W];
  __shared__ uint32_t lds_bits[ROWS][W];
  const int group = W < 4 ? threadIdx.x / LANES : 0, lane = threadIdx.x % LANES;
  const long long row = (long long)blockIdx.x * ROWS + group;
  const bool here = ROWS == 1 || row < a.rows;  // (a workgroup's waves meet at no barrier where it has several rows)
  if (!here) return;
  const int chunks = (a.k + 7) / 8;
  u32x4 xv[C], rv[C];
#pragma unroll
  for (int i = 0; i < C; ++i) xv[i] = load_chunk<DT>(a.x + 2 * row * a.ldx, LANES * i + lane, chunks, a.k);
  if (NORM && a.residual) {
#pragma unroll
    for (int i = 0; i < C; ++i) rv[i] = load_chunk<DT>(a.residual + 2 * row * a.ldr, LANES * i + lane, chunks, a.k);
  }
  float h[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[i][2 * j] = lo_to_f32<DT>(xv[i][j]);
      h[i][2 * j + 1] = hi_to_f32<DT>(xv[i][j]);
    }
  auto over_row = [&](auto v, auto op, auto& shared) {
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) v = op(v, __shfl_xor(v, s));
    if constexpr (W > 1) {
      if (lane % kWave == 0) shared[group][lane / kWave] = v;
      __syncthreads();
      v = shared[group][0];
#pragma unroll
      for (int w = 1; w < W; ++w) v = op(v, shared[group][w]);
    }
    return v;
  };
  if constexpr (NORM) {
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i][2 * j] += lo_to_f32<DT>(rv[i][j]);
          h[i][2 * j + 1] += hi_to_f32<DT>(rv[i][j]);
        }
      if (a.total) {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (LANES * i + lane < chunks) store_values<DT>(a.total + 2 * row * a.ldt, LANES * i + lane, a.k, h[i]);
      }
    }
    u32x4 wv[C];
#pragma unroll
    for (int i = 0; i < C; ++i) wv[i] = load_chunk<DT>(a.weight, LANES * i + lane, chunks, a.k);
    auto squares = [&](float up) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[i][j] * up, h[i][j] * up, sum);
      return over_row(sum, [](float p, float q) { return p + q; }, lds);
    };
    float up = 1.0f, mean = squares(1.0f) / (float)a.k;
    // squares that leave the range of fp32 above or below: once more, scaled
    if (mean == __builtin_inff())
      up = 0x1p-80f;
    else if (mean + a.eps < 0x1p-80f)
      up = 0x1p90f;
    if (up != 1.0f) {
      if constexpr (W > 1) __syncthreads();  // everyone has read the first sum
      mean = squares(up) / (float)a.k;
    }
    const float down = 1.0f / sqrtf(mean + a.eps * up * up);
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[i][2 * j] = h[i][2 * j] * up * down * lo_to_f32<DT>(wv[i][j]);
        h[i][2 * j + 1] = h[i][2 * j + 1] * up * down * hi_to_f32<DT>(wv[i][j]);
      }
    if (a.y) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (LANES * i + lane < chunks) store_values<DT>(a.y + 2 * row * a.ldy, LANES * i + lane, a.k, h[i]);
    }
    if (!a.codes) return;
  }
  uint32_t largest = 0;
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // of two magnitudes the larger bits are the larger value, and those of infinity and NaN are larger still
      const uint32_t bits = __builtin_bit_cast(uint32_t, h[i][j]) & 0x7fffffffu;
      largest = bits > largest ? bits : largest;
    }
  const CodeFactors cf = code_factors(over_row(largest, [](uint32_t p, uint32_t q) { return p > q ? p : q; }, lds_bits));
  if (lane == 0) a.scales[row] = cf.scale;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = LANES * i + lane;
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j >> 2] |= code(h[i][j], cf) << (8 * (j & 3));
    if (8 * c < a.row_bytes) *reinterpret_cast<u32x2*>(a.codes + row * a.row_bytes + 8 * c) = u32x2{q[0], q[1]};
  }
}

// Rows that are longer than registers hold: read once for each of the squares, the largest value and the result.  A
// workgroup a row, a load at a time a thread, so bound by latency: 1 x 130944 bf16 to 8-bit rows 50 us, with the norm
// and a residual 112; 300 x 40000 25 and 48, where the bytes would take 7 and 14.
template <int DT, bool NORM>
__global__ __launch_bounds__(kRowThreads) void long_rows_kernel(RowArgs a) {
  __shared__ float lds[kRowThreads / kWave];
  __shared__ uint32_t lds_bits[kRowThreads / kWave];
  const long long row = blockIdx.x;
  const uint8_t* x = a.x + 2 * row * a.ldx;
  const uint8_t* residual = a.residual ? a.residual + 2 * row * a.ldr : nullptr;
  const int chunks = (a.k + 7) / 8;
  auto load = [&](int c, float (&h)[8]) {
    load_values<DT>(x, c, a.k, h);
    if (NORM && residual) {
      float r[8];
      load_values<DT>(residual, c, a.k, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] += r[i];
    }
  };
  NormFactors nf = {1.0f, 1.0f};
  if constexpr (NORM) {
    auto squares = [&](float up) {
      float sum = 0.0f;
      for (int c = threadIdx.x; c < chunks; c += kRowThreads) {
        float h[8];
        load(c, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(h[i] * up, h[i] * up, sum);
      }
      return over_group(sum, [](float p, float q) { return p + q; }, lds);
    };
    float mean = squares(1.0f) / (float)a.k;
    // squares that leave the range of fp32 above or below: once more, scaled
    if (mean == __builtin_inff())
      nf.up = 0x1p-80f;
    else if (mean + a.eps < 0x1p-80f)
      nf.up = 0x1p90f;
    if (nf.up != 1.0f) mean = squares(nf.up) / (float)a.k;
    nf.down = 1.0f / sqrtf(mean + a.eps * nf.up * nf.up);
  }
  auto norm = [&](int c, float (&h)[8]) {
    if constexpr (NORM) {
      float w[8];
      load_values<DT>(a.weight, c, a.k, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = h[i] * nf.up * nf.down * w[i];
    }
  };
  CodeFactors cf = {0.0f, 0.0f, 0.0f};
  if (a.codes) {
    uint32_t largest = 0;
    for (int c = threadIdx.x; c < chunks; c += kRowThreads) {
      float h[8];
      load(c, h);
      norm(c, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // of two magnitudes the larger bits are the larger value, and those of infinity and NaN are larger still
        const uint32_t bits = 8 * c + i < a.k ? __builtin_bit_cast(uint32_t, h[i]) & 0x7fffffffu : 0u;
        largest = bits > largest ? bits : largest;
      }
    }
    cf = code_factors(over_group(largest, [](uint32_t p, uint32_t q) { return p > q ? p : q; }, lds_bits));
    if (threadIdx.x == 0) a.scales[row] = cf.scale;
  }
  const int padded = a.codes ? (int)(a.row_bytes / 8) : chunks;
  for (int c = threadIdx.x; c < padded; c += kRowThreads) {
    float h[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (c < chunks) {
      load(c, h);
      if (NORM && a.total) store_values<DT>(a.total + 2 * row * a.ldt, c, a.k, h);
      norm(c, h);
      if (NORM && a.y) store_values<DT>(a.y + 2 * row * a.ldy, c, a.k, h);
    }
    if (a.codes) {
      uint32_t q[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i >> 2] |= (8 * c + i < a.k ? code(h[i], cf) : 0u) << (8 * (i & 3));
      *reinterpret_cast<u32x2*>(a.codes + row * a.row_bytes + 8 * c) = u32x2{q[0], q[1]};
    }
  }
}

// ---------------------------------------------------------------------------
// 8-bit rows to values
// ---------------------------------------------------------------------------

struct DecodeArgs {
  const uint8_t* codes;
  const float* scales;
  uint8_t* y;
  long long ldy, row_bytes;
  int rows, k;
};

// A workgroup a row.  Memory: 32768 x 4096 in 59 us, 403 MB of which the codes are still in the last-level cache.
// Narrow rows, which leave threads without work, are bound by the number of workgroups (65536 x 128 bf16: 17 us for 25 MB, x 512:
// 18 for 101 MB), few long ones by latency (1 x 130944: 16).
template <int DT>
__global__ __launch_bounds__(kRowThreads) void decode_rows_kernel(DecodeArgs a) {
  const long long row = blockIdx.x;
  const float s = a.scales[row];
  const int chunks = (a.k + 7) / 8;
  for (int c = threadIdx.x; c < chunks; c += kRowThreads) {
    const u32x2 q = *reinterpret_cast<const u32x2*>(a.codes + row * a.row_bytes + 8 * c);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sbyte(q[i >> 2], i & 3) * s;
    store_values<DT>(a.y + 2 * row * a.ldy, c, a.k, v);
  }
}

// ---------------------------------------------------------------------------
// router's choice
// ---------------------------------------------------------------------------

constexpr int kMaxExpertGroups = 64;  // a lane each

struct ChooseArgs {
  const uint8_t* logits;
  const float* bias;
  float* gates;
  int32_t* ids;
  long long ldl;
  int tokens, experts, top, groups, top_groups, best;
  int each;       // experts of a group
  int span_bits;  // choose_rows_kernel: log2 of the lanes that hold a group,
  int per;        // and experts of a lane
  bool sigmoid, renormalise;
  float factor;
};

template <int DT>
__device__ __forceinline__ float logit(const ChooseArgs& a, long long t, int e) {
  float l;
  if constexpr (DT == 2)
    l = reinterpret_cast<const float*>(a.logits)[t * a.ldl + e];
  else
    l = lo_to_f32<DT>(reinterpret_cast<const uint16_t*>(a.logits)[t * a.ldl + e]);
  // NaN: out of the choice; +inf: the largest finite value
  return l > -__builtin_inff() ? fminf(l, 3.402823466e38f) : -__builtin_inff();
}

// The largest value over the lanes and its number, the lower one of equals.
__device__ __forceinline__ void first_largest(double& v, int& at) {
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) {
    const double o = __shfl_xor(v, s);
    const int i = __shfl_xor(at, s);
    if (o > v || (o == v && i < at)) {
      v = o;
      at = i;
    }
  }
}

// The gate of a chosen expert with logit l (-inf: none), `base` the row's largest logit where p is not
// renormalised.  LARGEST and SUM go over the lanes that hold the token's chosen.
//
// sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)).  Renormalised, every score may take the same factor, so that
// those of the chosen do not vanish together: the largest of them has exp(0).
//
// In fp32, in units of 2^-24 of the gate: the difference of logits d, exp 2, sigmoid's other factor 5 (1 + exp(-|l|) 2,
// reciprocal 2, product 1), quotient and factor 2; the sum of the chosen, each off by as much, d no more than 4 on
// average, and 6 additions: 17; the softmax's sum below 7 twice, 4 and V + 4 (see choose_in_row): with V = 32, 54.
// In all below d + 60.
template <typename LARGEST, typename SUM>
__device__ __forceinline__ float gate_of(const ChooseArgs& a, float l, float base, float sum, LARGEST largest_of,
                                         SUM sum_of) {
  const float none = -__builtin_inff();
  const float low = a.sigmoid ? fminf(l, 0.0f) : l;
  if (a.renormalise)
    base = largest_of(low);
  else if (a.sigmoid)
    base = 0.0f;
  float p = l > none ? expf(low - base) : 0.0f;
  if (a.sigmoid) p *= __builtin_amdgcn_rcpf(1.0f + expf(-fabsf(l)));
  if (a.renormalise)
    p /= sum_of(p);
  else if (!a.sigmoid)
    p /= sum;
  return l > none ? p * a.factor : 0.0f;
}

// A wave chooses for one token, with ranks in 64 bits in LDS: what rows of 16 lanes do not hold.
template <int DT>
__device__ __forceinline__ void choose_token(const ChooseArgs& a, long long t, double* ranks) {
  const int lane = threadIdx.x & (kWave - 1);
  const float none = -__builtin_inff();
  float largest = none;
  for (int e = lane; e < a.experts; e += kWave) largest = fmaxf(largest, logit<DT>(a, t, e));
  for (int s = 1; s < kWave; s <<= 1) largest = fmaxf(largest, __shfl_xor(largest, s));
  double sum = 0.0;
  if (!a.sigmoid && largest > none) {
    for (int e = lane; e < a.experts; e += kWave) sum += exp((double)logit<DT>(a, t, e) - (double)largest);
    for (int s = 1; s < kWave; s <<= 1) sum += __shfl_xor(sum, s);
  }
  const bool by_score = a.bias || (a.best == 2 && a.groups > 1);
  for (int e = lane; e < a.experts; e += kWave) {
    const float l = logit<DT>(a, t, e);
    double rank = none;
    if (l > none) {
      rank = (double)l;
      if (by_score) {
        const double p = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)largest) / sum;
        const double r = a.bias ? p + (double)a.bias[e] : p;
        rank = r > none ? r : (double)none;  // a bias of NaN
      }
    }
    ranks[e] = rank;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (a.groups > 1) {
    const int each = a.each;
    double value = none;
    if (lane < a.groups) {
      double first = none, second = none;
      for (int i = 0; i < each; ++i) {
        const double r = ranks[lane * each + i];
        if (r > first) {
          second = first;
          first = r;
        } else if (r > second) {
          second = r;
        }
      }
      value = a.best == 2 && second > none ? first + second : first;
    }
    unsigned long long kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      double v = value;
      int g = lane;
      first_largest(v, g);
      if (!(v > none)) break;
      kept |= 1ull << g;
      if (g == lane) value = none;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int e = lane; e < a.experts; e += kWave) {
      if (!(kept >> (e / each) & 1))
        ranks[e] = none;
      else if (!a.bias && ranks[e] > none)
        ranks[e] = (double)logit<DT>(a, t, e);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  int mine = -1;  // lane j has the j-th expert
  for (int j = 0; j < a.top; ++j) {
    double v = none;
    int at = a.experts;
    for (int e = lane; e < a.experts; e += kWave) {
      if (ranks[e] > v) {
        v = ranks[e];
        at = e;
      }
    }
    first_largest(v, at);
    if (!(v > none)) break;
    if (lane == j) mine = at;
    if (lane == at % kWave) ranks[at] = none;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  const float gate = gate_of(
      a, mine >= 0 ? logit<DT>(a, t, mine) : none, largest, (float)sum,
      [](float v) {
        for (int s = 1; s < kWave; s <<= 1) v = fmaxf(v, __shfl_xor(v, s));
        return v;
      },
      [](float v) {
        for (int s = 1; s < kWave; s <<= 1) v += __shfl_xor(v, s);
        return v;
      });
  if (lane < a.top) {
    a.ids[t * a.top + lane] = mine;
    a.gates[t * a.top + lane] = gate;
  }
}

template <int DT>
__global__ __launch_bounds__(kWave) void choose_kernel(ChooseArgs a) {
  __shared__ double ranks[QR_MAX_EXPERTS];
  choose_token<DT>(a, blockIdx.x, ranks);
}

// A row of 16 lanes chooses for one token, a lane holding the ranks of V neighbouring experts in registers, in
// fp32.  Ranks, and groups' values, that are nearer to each other than fp32 may be off leave the choice open; the
// wave then takes the same steps in 64 bits.  (Without a bias the logits are compared, which is exact.)
//
// A lane's ranks are sorted once, without their numbers.  A round takes the largest of the row's 16 first ones, and
// its lane moves up; the number is looked up by the value at the end.  Bound by vector instructions, which fill 86 %
// of the time: 32768 tokens, 256 experts, 8 of them from 4 of 8 groups by sigmoid and bias: 22.5 us, 1240 a wave of 4
// tokens, half of them in the 9 rounds; biases of -5, with more tokens that are open, 24.  (A round that searched all
// ranks: 28.8, where this took 24.7; groups compared by branches and the
// chosen one found by scalar masks: 32.3; a wave a token, with ranks in LDS in 64 bits: 141.)
constexpr int kChooseLanes = 16, kChooseThreads = 256;

template <int N>
__device__ __forceinline__ float row_ror(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x120 + N, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ double row_ror(double v) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  i32x2 w = __builtin_bit_cast(i32x2, v);
  w.x = __builtin_amdgcn_mov_dpp(w.x, 0x120 + N, 0xF, 0xF, true);
  w.y = __builtin_amdgcn_mov_dpp(w.y, 0x120 + N, 0xF, 0xF, true);
  return __builtin_bit_cast(double, w);
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }
template <typename K>
__device__ __forceinline__ K row_max(K v) {
  v = larger(v, row_ror<8>(v));
  v = larger(v, row_ror<4>(v));
  v = larger(v, row_ror<2>(v));
  return larger(v, row_ror<1>(v));
}
// (The same bits in every lane: each step adds two values in one or the other order.)
template <typename K>
__device__ __forceinline__ K row_sum(K v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  return v + row_ror<1>(v);
}

// Batcher's odd-even merge sort, the largest first.  V is a power of two.
template <typename K, int V>
__device__ __forceinline__ void sort_down(K (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // i is the upper of a pair: pairs of blocks of d that begin at d % p, both in the same run of 2 p
        if (i >= d % p && (i - d % p) / d % 2 == 0 && i + d < V && i / (2 * p) == (i + d) / (2 * p)) {
          const K most = larger(k[i], k[i + d]);
          k[i + d] = smaller(k[i], k[i + d]);
          k[i] = most;
        }
      }
}

// A lane of a row holds at most `per` neighbours of a group, from this expert on.
__device__ __forceinline__ int first_of(const ChooseArgs& a, int lane) {
  return (lane >> a.span_bits) * a.each + (lane & ((1 << a.span_bits) - 1)) * a.per;
}
__device__ __forceinline__ int count_of(const ChooseArgs& a, int lane) {
  const int left = a.each - (lane & ((1 << a.span_bits) - 1)) * a.per;  // in the group
  return lane >> a.span_bits < a.groups ? min(max(left, 0), a.per) : 0;
}

// The lane's values of a row of one for each expert, `fill` past the last.
template <int DT, int V>
__device__ __forceinline__ void load_run(const ChooseArgs& a, const uint8_t* row, int lane, float fill, float (&k)[V]) {
  constexpr int BYTES = DT == 2 ? 4 : 2, PER = V * BYTES >= 16 ? 16 / BYTES : V;  // values of one load
  typedef uint32_t words __attribute__((ext_vector_type(PER * BYTES >= 4 ? PER * BYTES / 4 : 1), aligned(BYTES)));
  const int first = first_of(a, lane), count = count_of(a, lane);
  if (PER * BYTES >= 4 && a.per == V && a.each % V == 0) {  // V or none
    if (count > 0) {
#pragma unroll
      for (int q = 0; q < V / PER; ++q) {
        const words w = *reinterpret_cast<const words*>(row + (first + PER * q) * BYTES);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if constexpr (DT == 2)
            k[PER * q + i] = __builtin_bit_cast(float, (uint32_t)w[i]);
          else
            k[PER * q + i] = i & 1 ? hi_to_f32<DT == 2 ? 0 : DT>(w[i / 2]) : lo_to_f32<DT == 2 ? 0 : DT>(w[i / 2]);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) k[v] = fill;
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v < count ? first + v : 0;
    float x;
    if constexpr (DT == 2)
      x = reinterpret_cast<const float*>(row)[e];
    else
      x = lo_to_f32<DT == 2 ? 0 : DT>(reinterpret_cast<const uint16_t*>(row)[e]);
    k[v] = v < count ? x : fill;
  }
}

// The row's choice from its logits l (clamped, -inf: out), into chosen[0 .. top - 1] in LDS, -1 for none; `sum` of
// the softmax where it is needed.  Returns whether it is open (K = float only).
template <typename K, int V, typename LOGIT>
__device__ __forceinline__ bool choose_in_row(const ChooseArgs& a, const float (&l)[V], float largest, float& sum,
                                              int* chosen, LOGIT logit_at) {
  constexpr bool kExact = sizeof(K) == 8;
  const int lane = threadIdx.x & (kChooseLanes - 1), row = (threadIdx.x & (kWave - 1)) / kChooseLanes;
  const K none = -__builtin_inff();
  const bool by_score = a.bias || (a.best == 2 && a.groups > 1);
  K k[V], total = 0;
  if (by_score || (!a.sigmoid && !a.renormalise && !kExact)) {
    // (-inf times 0 is NaN, which larger() takes for none)
    if (a.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (kExact)
          k[v] = 1.0 / (1.0 + exp(-(double)l[v]));
        else
          k[v] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[v]));
        k[v] = larger(k[v] + (K)(l[v] * 0.0f), none);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (kExact)
          k[v] = l[v] > -__builtin_inff() ? exp((double)l[v] - (double)largest) : 0.0;
        else
          k[v] = l[v] > -__builtin_inff() ? __expf(l[v] - largest) : 0.0f;
        total += k[v];
      }
      total = row_sum(total);
      sum = (float)total;
#pragma unroll
      for (int v = 0; v < V; ++v) k[v] = larger(k[v] / total + (K)(l[v] * 0.0f), none);
    }
  }
  bool open = false;
  // What two ranks may be off together, and as much again.  sigmoid: the exponential's argument and value are off
  // by (|l| + 2) 2^-23, of which p (1 - p) <= 1 / 4, and p (1 - p) |l| < 1 / 4, come through; the sum and the
  // reciprocal by 2^-23 and 2^-24 of p: in all below 2^-22.  softmax: the exponential by (d + 2) 2^-23 of it, d the
  // distance to the largest logit, p d < 1 / 2 of the largest p; the sum by that on average, where d < 7, and V + 4
  // steps; the quotient by two: (V + 32) 2^-24 of the largest p.  The sum with the bias by half a step.
  const float slack = a.sigmoid ? 0x1p-20f : (V + 32) * 0x1p-22f / sum;
  if (a.bias) {
    float b[V];
    load_run<2, V>(a, reinterpret_cast<const uint8_t*>(a.bias), lane, 0.0f, b);
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = larger(k[v] + (K)b[v], none);  // a bias of NaN: none
  }
  if (a.groups > 1) {
    K one = none, two = none;  // the largest ranks of the lane, of the group
    if (by_score) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        two = larger(two, smaller(one, k[v]));
        one = larger(one, k[v]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) one = larger(one, (K)l[v]);
    }
    for (int s = 0; s < a.span_bits; ++s) {
      const K o = __shfl_xor(one, 1 << s), w = __shfl_xor(two, 1 << s);
      two = larger(larger(two, w), smaller(one, o));
      one = larger(one, o);
    }
    // Of two ranks their mean in fp32, which holds it where their sum is past its range; a second that there is not is 0.
    const K share = a.best == 2 && !kExact ? (K)0.5 : (K)1;
    const bool both = a.best == 2 && two > none;
    const K value = both ? share * one + share * two : share * one;
    int before = 0;
    auto look = [&](auto N) {  // at the group of the lane that many below, around the row
      constexpr int n = decltype(N)::value;
      if (n & ((1 << a.span_bits) - 1)) return;  // the same for the whole launch
      const K o = row_ror<n>(value);
      before += (int)(o > value) | ((int)(o == value) & (int)(lane >= n));
    };
    auto all = [&](auto... n) { (look(n), ...); };
    all(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{}, std::integral_constant<int, 3>{},
        std::integral_constant<int, 4>{}, std::integral_constant<int, 5>{}, std::integral_constant<int, 6>{},
        std::integral_constant<int, 7>{}, std::integral_constant<int, 8>{}, std::integral_constant<int, 9>{},
        std::integral_constant<int, 10>{}, std::integral_constant<int, 11>{}, std::integral_constant<int, 12>{},
        std::integral_constant<int, 13>{}, std::integral_constant<int, 14>{}, std::integral_constant<int, 15>{});
    // A group is kept if fewer than top_groups come before it.
    const bool kept = before < a.top_groups && value > none;
    if constexpr (!kExact) {
      // What the value may be off, and as much again: two ranks by 2^-24 of either's magnitude besides slack / 2, and
      // their sum by as much of its own.  It is open which groups are kept if not all of them are above all others by
      // what both are off.
      const float off = share * slack + share * 0x1p-22f * fabsf(one) + (both ? share * 0x1p-22f * fabsf(two) : 0.0f);
      const float least = -row_max(kept ? off - value : none), most = row_max(!kept && value > none ? value + off : none);
      open = by_score && !(most < least);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = kept ? a.bias ? k[v] : (K)l[v] : none;
  } else if (!a.bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = l[v];
  }
  K sorted[V], last = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) sorted[v] = k[v];
  sort_down(sorted);
  // With a bias, in fp32, it goes on until a rank is clearly below the one before it, and the top-th at least.
  const bool ahead = a.bias && !kExact;
  bool done = false, sort = false;
  int count = 0, before_from = -1, again = 0;
  int from = -1, nth = 0;  // lane j: the j-th chosen is the nth of its value in lane `from`
  K value = none;
  for (int j = 0; j < (ahead ? kChooseLanes : a.top); ++j) {
    const K most = row_max(sorted[0]);
    done |= !(most > none);
    const bool equal = last == most;
    if (ahead) {
      // (NaN, of two ranks of +inf, is not clear)
      const bool clear = (float)(last - most) > slack + 0x1p-21f * fabsf((float)most);
      done |= j >= a.top && clear;
      sort |= !done && j && !clear;
    }
    last = most;
    if (__all(done)) break;
    // the first of the row's lanes that has it
    const uint32_t has = (uint32_t)(__ballot(sorted[0] == most) >> (16 * row)) & 0xffffu;
    const int winner = __builtin_ctz(has | 0x10000u);
    again = equal && winner == before_from ? again + 1 : 0;
    before_from = winner;
    if (lane == j && !done) {
      from = winner;
      nth = again;
      value = most;
    }
    const bool mine = winner == lane;
#pragma unroll
    for (int v = 0; v < V && v < kChooseLanes; ++v) {
      const K here = sorted[v], next = v + 1 < V ? sorted[v + 1] : none;  // values: a choice of elements would be an index
      sorted[v] = mine ? next : here;
    }
    count += !done;
  }
  // Where it lies in that lane: the first of its value, the nth where there are several.
  uint32_t places = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    places |= __shfl(k[v], (threadIdx.x & 48) + (from & 15)) == value ? 1u << v : 0u;
  for (; __any(nth > 0); --nth) places &= nth > 0 ? places - 1 : ~0u;
  chosen[lane] = from < 0 ? -1 : first_of(a, from) + __builtin_ctz(places | 0x80000000u);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if constexpr (!kExact) {
    if (ahead && count == kChooseLanes && a.experts > kChooseLanes && !done) open = true;  // nothing clearly below was seen
    if (__any(sort && !open)) {
      // Lane j takes the j-th of those seen to 64 bits, and its place among them is the number that come before it.
      double all = 0.0;
      if (!a.sigmoid) {
#pragma unroll 1
        for (int v = 0; v < count_of(a, lane); ++v) {
          const float x = logit_at(first_of(a, lane) + v);
          all += x > -__builtin_inff() ? exp((double)x - (double)largest) : 0.0;
        }
        all = row_sum(all);
      }
      const int id = chosen[lane];
      double rank = -__builtin_inf();
      if (id >= 0) {
        const double x = logit_at(id);
        rank = (a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)largest) / all) + (double)a.bias[id];
      }
      int before = 0;
      for (int q = 0; q < kChooseLanes; ++q) {
        const double o = __shfl(rank, (threadIdx.x & 48) + q);
        const int e = __shfl(id, (threadIdx.x & 48) + q);
        before += e >= 0 && (o > rank || (o == rank && e < id));
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (id >= 0 && sort) chosen[before] = id;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
  return open;
}

template <int DT, int V>
__global__ __launch_bounds__(kChooseThreads) void choose_rows_kernel(ChooseArgs a) {
  constexpr int WAVES = kChooseThreads / kWave, ROWS = kWave / kChooseLanes;
  __shared__ int lds[WAVES][ROWS][kChooseLanes];
  const float none = -__builtin_inff();
  const int wave = threadIdx.x / kWave, row = (threadIdx.x & (kWave - 1)) / kChooseLanes;
  const int lane = threadIdx.x & (kChooseLanes - 1);  // of the row
  const long long first = ((long long)blockIdx.x * WAVES + wave) * ROWS, t = first + row;
  if (first >= a.tokens) return;
  const bool here = t < a.tokens;

  float l[V], largest = none, sum = 1.0f;
  load_run<DT, V>(a, a.logits + (DT == 2 ? 4 : 2) * (here ? t : (long long)a.tokens - 1) * a.ldl, lane, none, l);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    l[v] = fminf(larger(l[v], none), 3.402823466e38f);  // NaN: -inf
    largest = larger(largest, l[v]);
  }
  largest = row_max(largest);
  int* chosen = lds[wave][row];
  auto logit_at = [&](int e) { return logit<DT>(a, here ? t : (long long)a.tokens - 1, e); };
  if (__any(choose_in_row<float, V>(a, l, largest, sum, chosen, logit_at) && here)) {
    // (All four tokens, for one that is open; the gates keep the sum in fp32, so that they do not depend on the others.)
    float again = sum;
    choose_in_row<double, V>(a, l, largest, again, chosen, logit_at);
  }
  if (!here) return;
  const int mine = lane < a.top ? chosen[lane] : -1;
  const float gate = gate_of(a, mine >= 0 ? logit<DT>(a, t, mine) : none, largest, sum, row_max<float>, row_sum<float>);
  if (lane < a.top) {
    a.ids[t * a.top + lane] = mine;
    a.gates[t * a.top + lane] = gate;
  }
}

template <int DT>
static auto choose_kernel_of(int run) -> void (*)(ChooseArgs) {
  switch (run) {
    case 1: return choose_rows_kernel<DT, 1>;
    case 2: return choose_rows_kernel<DT, 2>;
    case 4: return choose_rows_kernel<DT, 4>;
    case 8: return choose_rows_kernel<DT, 8>;
    case 16: return choose_rows_kernel<DT, 16>;
    case 32: return choose_rows_kernel<DT, 32>;
    default: return choose_kernel<DT>;
  }
}

// ---------------------------------------------------------------------------
// host-side argument checks (no HIP call)
// ---------------------------------------------------------------------------

static long long row_bytes(size_t k) { return (long long)((k + kRowRun - 1) / kRowRun * kRowRun); }
static bool bad_k(size_t k) { return k < 1 || k > QR_MAX_ROW_K; }

// Calls `launch(first, count)` for as many rows at a time as a launch holds, `per` rows a workgroup of `threads`.
template <typename LAUNCH>
static qr_status in_launches(long long rows, int per, int threads, LAUNCH launch) {
  const long long fit = kMaxLaunchThreads / threads * per;
  for (long long r = 0; r < rows; r += fit) {
    const qr_status s = launch(r, rows - r < fit ? rows - r : fit);
    if (s != QR_OK) return s;
  }
  return QR_OK;
}

// How a row is shared out: by W waves of C chunks a lane, a workgroup of fewer than four waves holding several.
// Few waves of some chunks where there are many rows, one chunk a lane where there are few (us, bf16, W x C; the
// last three: to 8-bit rows and back):
//   norm, residual   1 x 4096       1x8 6.8    4x2 3.4    16x1 3.0
//                    16 x 8192                 4x4 4.8    16x1 3.5
//                    1000 x 2048    1x4 7.0    4x1 4.6    16x1 7.9
//                    32768 x 4096   1x8 235    4x2 189    16x1 245
//                    20000 x 8192              4x4 237    16x1 225
//   norm             65536 x 1024   1x2 52     4x1 83     16x1 270
//   rows             777 x 5003                4x3 9.2    16x1 10.7
//                    20000 x 5120              4x3 120    16x1 152
//                    20000 x 7168              4x4 162    16x1 166
// Rows of over 32768 values are read again for each of a norm's steps.
struct RowShape {
  int waves, chunks, rows, threads;  // rows: of a workgroup; waves == 0: long rows
};
static RowShape row_shape(long long rows, int k) {
  const int w = rows <= 512 ? (k <= 512 ? 1 : k <= 2048 ? 4 : 16) : (k <= 1024 ? 1 : k <= 7168 ? 4 : 16);
  const int c = (k + 512 * w - 1) / (512 * w);
  if (c > 4) return {0, 0, 1, kRowThreads};
  return {w, c, w < 4 ? 4 / w : 1, w > 4 ? kWave * w : kRowThreads};
}

template <int DT, bool NORM, int W>
static auto row_kernel_of(int chunks) -> void (*)(RowArgs) {
  if constexpr (W > 1) {
    if (chunks == 3) return rows_kernel<DT, NORM, W, 3>;
    if (chunks == 4) return rows_kernel<DT, NORM, W, 4>;
  }
  return chunks == 1 ? rows_kernel<DT, NORM, W, 1> : rows_kernel<DT, NORM, W, 2>;
}
template <int DT, bool NORM>
static auto row_kernel_of(const RowShape& s) -> void (*)(RowArgs) {
  switch (s.waves) {
    case 0: return long_rows_kernel<DT, NORM>;
    case 1: return row_kernel_of<DT, NORM, 1>(s.chunks);
    case 4: return row_kernel_of<DT, NORM, 4>(s.chunks);
    default: return row_kernel_of<DT, NORM, 16>(s.chunks);
  }
}
static auto row_kernel_of(qr_dtype dtype, bool norm, const RowShape& s) -> void (*)(RowArgs) {
  if (dtype == QR_FP16) return norm ? row_kernel_of<kFp16, true>(s) : row_kernel_of<kFp16, false>(s);
  return norm ? row_kernel_of<kBf16, true>(s) : row_kernel_of<kBf16, false>(s);
}

static qr_status launch_rows(qr_dtype dtype, bool norm, const RowArgs& args, hipStream_t st) {
  const RowShape shape = row_shape(args.rows, args.k);
  return in_launches(args.rows, shape.rows, shape.threads, [&](long long first, long long count) {
    RowArgs a = args;
    a.x += 2 * first * a.ldx;
    if (a.residual) a.residual += 2 * first * a.ldr;
    if (a.total) a.total += 2 * first * a.ldt;
    if (a.y) a.y += 2 * first * a.ldy;
    if (a.codes) {
      a.codes += first * a.row_bytes;
      a.scales += first;
    }
    a.rows = (int)count;
    return launch_1d(row_kernel_of(dtype, norm, shape), (count + shape.rows - 1) / shape.rows, shape.threads, st, a);
  });
}

static qr_status product8(qr_dtype dtype, int gated, const int8_t* x, const float* xs, size_t xrows, const int8_t* w,
                          const float* ws, const int32_t* offsets, const int32_t* rows, bool grouped, void* y,
                          size_t ldy, size_t slots, size_t experts, size_t n, size_t k, void* stream) {
  if (bad_dtype(dtype)) return QR_ERR_UNSUPPORTED;
  if (n < 1 || n > QR_MAX_N || bad_k(k) || slots > QR_MAX_SLOTS || xrows > QR_MAX_SLOTS || experts < 1 ||
      experts > QR_MAX_EXPERTS || ldy < n || ldy > kMaxStride)
    return QR_ERR_SIZE;
  if (grouped && !rows && xrows < slots) return QR_ERR_SIZE;
  if (slots == 0) return QR_OK;
  if (((!x || !xs) && xrows) || !w || !ws || !y || (grouped && !offsets)) return QR_ERR_ARG;
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(xs, 4) || misaligned(ws, 4) || misaligned(y, 2) ||
      misaligned(offsets, 4) || misaligned(rows, 4))
    return QR_ERR_ALIGN;
  const size_t wrows = experts * n * (gated ? 2 : 1), rb = (size_t)row_bytes(k), ys = span(slots, ldy, n);
  if (overlap(y, ys, x, xrows * rb) || overlap(y, ys, xs, 4 * xrows) || overlap(y, ys, w, wrows * rb) ||
      overlap(y, ys, ws, 4 * wrows) || (offsets && overlap(y, ys, offsets, 4 * (experts + 1))) ||
      (rows && overlap(y, ys, rows, 4 * slots)))
    return QR_ERR_ALIAS;
  Product8Args a = {};
  a.x = (const uint8_t*)x;
  a.xs = xs;
  a.w = (const uint8_t*)w;
  a.ws = ws;
  a.y = (uint8_t*)y;
  a.offsets = offsets;
  a.rows = rows;
  a.ldy = (long long)ldy;
  a.xrows = (long long)xrows;
  a.slots = (int)slots;
  a.experts = (int)experts;
  a.n = (int)n;
  a.k = (int)k;
  a.blocks = (int)(rb / kRowRun);
  return launch_product8(dtype, gated != 0, a, (hipStream_t)stream);
}

}  // namespace qr

using namespace qr;

extern "C" {

size_t qr_row_bytes(size_t rows, size_t k) {
  return bad_k(k) || rows < 1 || rows > (size_t)1 << 40 ? 0 : rows * (size_t)row_bytes(k);
}

qr_status qr_encode_rows(qr_dtype dtype, const void* x, size_t ldx, int8_t* codes, float* scales, size_t rows,
                         size_t k, void* stream) {
  if (bad_dtype(dtype)) return QR_ERR_UNSUPPORTED;
  if (bad_k(k) || rows > QR_MAX_SLOTS || ldx < k || ldx > kMaxStride) return QR_ERR_SIZE;
  if (rows == 0) return QR_OK;
  if (!x || !codes || !scales) return QR_ERR_ARG;
  if (misaligned(x, 2) || misaligned(codes, 16) || misaligned(scales, 4)) return QR_ERR_ALIGN;
  const size_t cb = rows * (size_t)row_bytes(k), xb = span(rows, ldx, k);
  if (overlap(codes, cb, x, xb) || overlap(scales, 4 * rows, x, xb) || overlap(codes, cb, scales, 4 * rows))
    return QR_ERR_ALIAS;
  RowArgs a = {};
  a.x = (const uint8_t*)x;
  a.codes = (uint8_t*)codes;
  a.scales = scales;
  a.ldx = (long long)ldx;
  a.row_bytes = row_bytes(k);
  a.rows = (int)rows;
  a.k = (int)k;
  return launch_rows(dtype, false, a, (hipStream_t)stream);
}

qr_status qr_decode_rows(qr_dtype dtype, const int8_t* codes, const float* scales, void* y, size_t ldy, size_t rows,
                         size_t k, void* stream) {
  if (bad_dtype(dtype)) return QR_ERR_UNSUPPORTED;
  if (bad_k(k) || rows > QR_MAX_SLOTS || ldy < k || ldy > kMaxStride) return QR_ERR_SIZE;
  if (rows == 0) return QR_OK;
  if (!codes || !scales || !y) return QR_ERR_ARG;
  if (misaligned(y, 2) || misaligned(codes, 16) || misaligned(scales, 4)) return QR_ERR_ALIGN;
  const size_t ys = span(rows, ldy, k);
  if (overlap(y, ys, codes, rows * (size_t)row_bytes(k)) || overlap(y, ys, scales, 4 * rows)) return QR_ERR_ALIAS;
  DecodeArgs args = {};
  args.codes = (const uint8_t*)codes;
  args.scales = scales;
  args.y = (uint8_t*)y;
  args.ldy = (long long)ldy;
  args.row_bytes = row_bytes(k);
  args.k = (int)k;
  return in_launches((long long)rows, 1, kRowThreads, [&](long long first, long long count) {
    DecodeArgs a = args;
    a.codes += first * a.row_bytes;
    a.scales += first;
    a.y += 2 * first * a.ldy;
    a.rows = (int)count;
    return launch_1d(dtype == QR_FP16 ? decode_rows_kernel<kFp16> : decode_rows_kernel<kBf16>, count, kRowThreads,
                     (hipStream_t)stream, a);
  });
}

qr_status qr_norm(qr_dtype dtype, const void* x, size_t ldx, const void* residual, size_t ldr, const void* weight,
                  float eps, void* total, size_t ldt, void* y, size_t ldy, int8_t* codes, float* scales, size_t rows,
                  size_t k, void* stream) {
  if (bad_dtype(dtype)) return QR_ERR_UNSUPPORTED;
  auto bad_ld = [&](const void* p, size_t ld) { return p && (ld < k || ld > kMaxStride); };
  if (bad_k(k) || rows > QR_MAX_SLOTS || ldx < k || ldx > kMaxStride || bad_ld(residual, ldr) || bad_ld(total, ldt) ||
      bad_ld(y, ldy))
    return QR_ERR_SIZE;
  if (!(eps >= 0.0f) || (total && !residual) || !codes != !scales) return QR_ERR_ARG;
  if (rows == 0) return QR_OK;
  if (!x || !weight || (!y && !codes)) return QR_ERR_ARG;
  if (misaligned(x, 2) || misaligned(residual, 2) || misaligned(weight, 2) || misaligned(total, 2) || misaligned(y, 2) ||
      misaligned(codes, 16) || misaligned(scales, 4))
    return QR_ERR_ALIGN;
  const size_t cb = rows * (size_t)row_bytes(k), sb = 4 * rows;
  // of an output matrix and an input one: apart, or the very same rows
  auto shares = [&](const void* out, size_t ldo, const void* in, size_t ldi) {
    return out && in && !(out == in && (ldo == ldi || rows == 1)) && overlap_rows(out, rows, ldo, k, in, rows, ldi, k);
  };
  auto in_bytes = [&](const void* p, size_t n, const void* m, size_t ld, size_t r) {
    return p && m && overlap(p, n, m, span(r, ld, k));
  };
  if (shares(total, ldt, x, ldx) || shares(total, ldt, residual, ldr) || shares(y, ldy, x, ldx) ||
      shares(y, ldy, residual, ldr) || (total && y && overlap_rows(total, rows, ldt, k, y, rows, ldy, k)) ||
      in_bytes(weight, 2 * k, total, ldt, rows) || in_bytes(weight, 2 * k, y, ldy, rows))
    return QR_ERR_ALIAS;
  if (codes && (overlap(codes, cb, scales, sb) || overlap(codes, cb, weight, 2 * k) || overlap(scales, sb, weight, 2 * k)))
    return QR_ERR_ALIAS;
  const struct {
    const void* p;
    size_t ld;
  } matrices[] = {{x, ldx}, {residual, ldr}, {total, ldt}, {y, ldy}};
  for (const auto& m : matrices)
    if (codes && (in_bytes(codes, cb, m.p, m.ld, rows) || in_bytes(scales, sb, m.p, m.ld, rows))) return QR_ERR_ALIAS;
  RowArgs a = {};
  a.x = (const uint8_t*)x;
  a.residual = (const uint8_t*)residual;
  a.weight = (const uint8_t*)weight;
  a.total = (uint8_t*)total;
  a.y = (uint8_t*)y;
  a.codes = (uint8_t*)codes;
  a.scales = scales;
  a.ldx = (long long)ldx;
  a.ldr = (long long)ldr;
  a.ldt = (long long)ldt;
  a.ldy = (long long)ldy;
  a.row_bytes = row_bytes(k);
  a.rows = (int)rows;
  a.k = (int)k;
  a.eps = eps;
  return launch_rows(dtype, true, a, (hipStream_t)stream);
}

qr_status qr_linear8(qr_dtype dtype, int gated, const int8_t* x, const float* xs, const int8_t* w, const float* ws,
                     void* y, size_t ldy, size_t m, size_t n, size_t k, void* stream) {
  return product8(dtype, gated, x, xs, m, w, ws, nullptr, nullptr, false, y, ldy, m, 1, n, k, stream);
}

qr_status qr_experts8(qr_dtype dtype, int gated, const int8_t* x, const float* xs, size_t tokens, const int8_t* w,
                      const float* ws, const int32_t* offsets, const int32_t* rows, void* y, size_t ldy, size_t slots,
                      size_t experts, size_t n, size_t k, void* stream) {
  return product8(dtype, gated, x, xs, tokens, w, ws, offsets, rows, true, y, ldy, slots, experts, n, k, stream);
}

qr_status qr_choose(qr_dtype dtype, qr_score score, const void* logits, size_t ldl, const float* bias, size_t groups,
                    size_t top_groups, int group_best, int renormalise, float factor, float* gates, int32_t* ids,
                    size_t tokens, size_t experts, size_t top, void* stream) {
  if ((bad_dtype(dtype) && dtype != QR_FP32) || (score != QR_SOFTMAX && score != QR_SIGMOID)) return QR_ERR_UNSUPPORTED;
  if (experts < 1 || experts > QR_MAX_EXPERTS || top < 1 || top > QR_MAX_TOP || top > experts ||
      tokens > QR_MAX_SLOTS / top || ldl < experts || ldl > kMaxStride || groups < 1 || groups > kMaxExpertGroups ||
      experts % groups || top_groups < 1 || top_groups > groups || group_best < 1 || group_best > 2 ||
      (size_t)group_best > experts / groups)
    return QR_ERR_SIZE;
  if (!(factor - factor == 0.0f)) return QR_ERR_ARG;
  if (tokens == 0) return QR_OK;
  if (!logits || !gates || !ids) return QR_ERR_ARG;
  const unsigned width = dtype == QR_FP32 ? 4 : 2;
  if (misaligned(logits, width) || misaligned(bias, 4) || misaligned(gates, 4) || misaligned(ids, 4)) return QR_ERR_ALIGN;
  const size_t out = 4 * tokens * top, in = width * ((tokens - 1) * ldl + experts);
  if (overlap(gates, out, ids, out) || overlap(gates, out, logits, in) || overlap(ids, out, logits, in) ||
      (bias && (overlap(gates, out, bias, 4 * experts) || overlap(ids, out, bias, 4 * experts))))
    return QR_ERR_ALIAS;
  ChooseArgs args = {};
  args.logits = (const uint8_t*)logits;
  args.bias = bias;
  args.gates = gates;
  args.ids = ids;
  args.ldl = (long long)ldl;
  args.experts = (int)experts;
  args.top = (int)top;
  args.groups = (int)groups;
  args.top_groups = (int)top_groups;
  args.best = group_best;
  args.sigmoid = score == QR_SIGMOID;
  args.renormalise = renormalise != 0;
  args.factor = factor;
  args.each = args.experts / args.groups;
  // A row of 16 lanes where they hold the experts, up to 32 each, a group in 1, 2, 4 ... of them: 32768 tokens of 160
  // experts in 8 groups 24 us, by a wave a token 107; 8 of 512 in one 27, with a bias 49, of 1024 by a wave a token 216.
  int span_bits = 4, run = 1;
  while (args.groups << span_bits > kChooseLanes && span_bits > 0) --span_bits;
  const int held = (args.each + (1 << span_bits) - 1) >> span_bits;
  while (run < held) run <<= 1;
  // (one group, or groups that lanes hold evenly: whole runs, which are loaded as such)
  args.per = groups == 1 ? run : held;
  args.span_bits = span_bits;
  const bool in_rows = top <= kChooseLanes && run <= 32 && args.groups << span_bits <= kChooseLanes;
  const int per_group = in_rows ? kChooseThreads / kChooseLanes : 1, threads = in_rows ? kChooseThreads : kWave;
  return in_launches((long long)tokens, per_group, threads, [&](long long first, long long count) {
    ChooseArgs a = args;
    a.logits += width * first * a.ldl;
    a.gates += first * a.top;
    a.ids += first * a.top;
    a.tokens = (int)count;
    auto kernel = dtype == QR_FP16 ? choose_kernel_of<kFp16> : dtype == QR_BF16 ? choose_kernel_of<kBf16> : choose_kernel_of<2>;
    return launch_1d(kernel(in_rows ? run : 0), (count + per_group - 1) / per_group, threads, (hipStream_t)stream, a);
  });
}

}  // extern "C"
