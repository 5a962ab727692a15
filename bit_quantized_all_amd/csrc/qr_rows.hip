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

template <int DT, bool NORM>
__global__ __launch_bounds__(kRowThreads) void rows_kernel(RowArgs a) {
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
      nf.up = 0x1p-70f;
    else if (mean + a.eps < 0x1p-80f)
      nf.up = 0x1p60f;
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

// A wave chooses for one token.
template <int DT>
__global__ __launch_bounds__(kWave) void choose_kernel(ChooseArgs a) {
  __shared__ double ranks[QR_MAX_EXPERTS];
  const long long t = blockIdx.x;
  const int lane = threadIdx.x;
  const float none = -__builtin_inff();
  float largest = none;
  for (int e = lane; e < a.experts; e += kWave) largest = fmaxf(largest, logit<DT>(a, t, e));
  for (int s = 1; s < kWave; s <<= 1) largest = fmaxf(largest, __shfl_xor(largest, s));
  double sum = 0.0;
  if (!a.sigmoid && largest > none) {
    for (int e = lane; e < a.experts; e += kWave) sum += exp((double)logit<DT>(a, t, e) - (double)largest);
    for (int s = 1; s < kWave; s <<= 1) sum += __shfl_xor(sum, s);
  }
  for (int e = lane; e < a.experts; e += kWave) {
    const float l = logit<DT>(a, t, e);
    double p = 0.0, rank = none;
    if (l > none) {
      p = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)largest) / sum;
      // without a bias in the order of the logits
      const double r = a.bias ? p + (double)a.bias[e] : a.best == 2 && a.groups > 1 ? p : (double)l;
      rank = r > none ? r : (double)none;  // a bias of NaN
    }
    ranks[e] = rank;
  }
  __syncthreads();
  unsigned long long kept = ~0ull;
  const int each = a.experts / a.groups;
  if (a.groups > 1) {
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
    kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      double v = value;
      int g = lane;
      first_largest(v, g);
      if (!(v > none)) break;
      kept |= 1ull << g;
      if (g == lane) value = none;
    }
  }
  __syncthreads();
  for (int e = lane; e < a.experts; e += kWave) {
    if (!(kept >> (a.groups > 1 ? e / each : 0) & 1)) ranks[e] = none;
    else if (!a.bias && ranks[e] > none) ranks[e] = (double)logit<DT>(a, t, e);
  }
  __syncthreads();
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
    __syncthreads();
  }
  // sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)).  Renormalised, every score may take the same
  // factor, so that those of the chosen do not vanish together: the largest of them has exp(0).
  const float l = mine >= 0 ? logit<DT>(a, t, mine) : none;
  const float low = a.sigmoid ? fminf(l, 0.0f) : l;
  float base = a.sigmoid ? 0.0f : largest;
  if (a.renormalise) {
    base = low;
    for (int s = 1; s < kWave; s <<= 1) base = fmaxf(base, __shfl_xor(base, s));
  }
  float p = mine >= 0 ? expf(low - base) : 0.0f;
  if (a.sigmoid) p /= 1.0f + expf(-fabsf(l));
  if (a.renormalise) {
    float total = p;
    for (int s = 1; s < kWave; s <<= 1) total += __shfl_xor(total, s);
    p /= total;
  } else if (!a.sigmoid) {
    p /= (float)sum;
  }
  if (lane < a.top) {
    a.ids[t * a.top + lane] = mine;
    a.gates[t * a.top + lane] = mine >= 0 ? p * a.factor : 0.0f;
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

static qr_status launch_rows(qr_dtype dtype, bool norm, const RowArgs& args, hipStream_t st) {
  return in_launches(args.rows, 1, kRowThreads, [&](long long first, long long count) {
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
    auto kernel = dtype == QR_FP16 ? (norm ? rows_kernel<kFp16, true> : rows_kernel<kFp16, false>)
                                   : (norm ? rows_kernel<kBf16, true> : rows_kernel<kBf16, false>);
    return launch_1d(kernel, count, kRowThreads, st, a);
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
  return in_launches((long long)tokens, 1, kWave, [&](long long first, long long count) {
    ChooseArgs a = args;
    a.logits += width * first * a.ldl;
    a.gates += first * a.top;
    a.ids += first * a.top;
    a.tokens = (int)count;
    return launch_1d(dtype == QR_FP16   ? choose_kernel<kFp16>
                     : dtype == QR_BF16 ? choose_kernel<kBf16>
                                        : choose_kernel<2>,
                     count, kWave, (hipStream_t)stream, a);
  });
}

}  // extern "C"
