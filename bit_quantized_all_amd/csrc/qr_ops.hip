// qr_ops.hip -- the C ABI of include/qr_ops.h: host-side argument checks (no
// HIP call before they pass), and the kernels of the routing plan and of the
// combination.  The products' kernels are in qr_product.hpp.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qr.h"
#include "qr_ops.h"
#include "qr_product.hpp"

namespace qr {

// (The caller sees to it that a launch holds fewer than 2^32 threads.)
template <typename... P>
static qr_status launch_1d(void (*kernel)(P...), long long groups, int threads, hipStream_t st, P... args) {
  void* argv[] = {static_cast<void*>(&args)...};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)groups), dim3(threads), argv, 0, st) ==
                 hipSuccess
             ? QR_OK
             : QR_ERR_HIP;
}

// ---------------------------------------------------------------------------
// routing plan: a stable counting sort of the expert slots by expert
// ---------------------------------------------------------------------------

// Bound by latency: a few trips to memory and barriers one after another.  512
// slots of 64 experts, one workgroup: 3.7 us on the device; 262144 slots of 256
// experts (2 MB of numbers and places), 128 workgroups: 2.6 us to count, 9.8 to
// place.  A place depends on the slots before it alone, so no order of
// execution shows in the plan.

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / kWave;
// A large plan: 2048 slots a workgroup, up to 512 workgroups (two a CU, as many as
// run at a time), and in larger plans equal parts.  Each of them adds up the
// counts of all, so that their number has to be bounded for the work to grow
// as the slots do: 8.4 million slots of 256 experts 111 us, 134 million 1.40 ms.
constexpr int kRouteChunk = 2048;
constexpr int kRouteChunks = 512;
constexpr int kRouteSmall = 4096;      // slots up to which one workgroup does it all
static_assert(QR_MAX_EXPERTS <= kRouteThreads, "one thread per expert");

struct RouteArgs {
  const void* ids;
  int32_t* offsets;
  int32_t* rows;
  int32_t* pos;
  int32_t* counts;  // [chunks][experts]
  int slots, top, experts, chunks, per_chunk;
};

// Expert of slot i, -1 if it is dropped.
template <typename ID>
__device__ __forceinline__ int expert_of(const RouteArgs& a, int i) {
  const ID e = static_cast<const ID*>(a.ids)[i];
  return e >= 0 && e < (ID)a.experts ? (int)e : -1;
}

// Adds the slots [begin, end) to count[], by expert.
template <typename ID>
__device__ __forceinline__ void count_slots(const RouteArgs& a, int begin, int end, int* count) {
  for (int i = begin + (int)threadIdx.x; i < end; i += kRouteThreads) {
    const int e = expert_of<ID>(a, i);
    if (e >= 0) atomicAdd(&count[e], 1);  // integers: any order gives the same counts
  }
}

// Slots of each chunk by expert.
template <typename ID>
__global__ __launch_bounds__(kRouteThreads) void route_count_kernel(RouteArgs a) {
  __shared__ int count[QR_MAX_EXPERTS];
  const int tid = threadIdx.x;
  if (tid < a.experts) count[tid] = 0;
  __syncthreads();
  const long long begin = (long long)blockIdx.x * a.per_chunk;
  const long long end = begin + a.per_chunk < a.slots ? begin + a.per_chunk : a.slots;
  count_slots<ID>(a, (int)begin, (int)end, count);
  __syncthreads();
  if (tid < a.experts) a.counts[(size_t)blockIdx.x * a.experts + tid] = count[tid];
}

// Places each slot of a chunk: the row of a slot is where its expert begins,
// plus that expert's slots in earlier chunks, in earlier steps of this
// workgroup, in earlier waves of this step, and in earlier lanes.
template <typename ID>
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs a) {
  __shared__ int count[QR_MAX_EXPERTS];                      // all slots by expert
  __shared__ int next[QR_MAX_EXPERTS];                       // row of the expert's next slot
  __shared__ uint16_t in_wave[kRouteWaves][QR_MAX_EXPERTS];  // of this step
  __shared__ int wave_sum[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  if (tid < a.experts) {
    count[tid] = next[tid] = 0;
    for (int w = 0; w < kRouteWaves; ++w) in_wave[w][tid] = 0;
  }
  __syncthreads();
  if (a.chunks == 1) {
    count_slots<ID>(a, 0, a.slots, count);
    __syncthreads();
  } else {
    // An expert's counts are added up by as many threads as there are, 16
    // loads of each in flight: the loads' latency is what this costs (262144
    // slots of 256 experts: 23 us with one thread and one load at a time).
    int width = 1;
    while (width < a.experts) width <<= 1;
    const int e = tid & (width - 1), parts = kRouteThreads / width;
    int before = 0, all = 0;
    if (e < a.experts) {
      for (int c0 = tid / width * 16; c0 < a.chunks; c0 += parts * 16) {
        int v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = c0 + i < a.chunks ? a.counts[(size_t)(c0 + i) * a.experts + e] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          all += v[i];
          before += c0 + i < (int)blockIdx.x ? v[i] : 0;
        }
      }
      atomicAdd(&count[e], all);
      atomicAdd(&next[e], before);
    }
    __syncthreads();
  }
  // exclusive scan over the experts
  const int mine = tid < a.experts ? count[tid] : 0;
  int upto = mine;
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) {
    const int o = __shfl_up(upto, s);
    if (lane >= s) upto += o;
  }
  if (lane == kWave - 1) wave_sum[wave] = upto;
  __syncthreads();
  int begin = upto - mine, kept = 0;
#pragma unroll
  for (int w = 0; w < kRouteWaves; ++w) {
    if (w < wave) begin += wave_sum[w];
    kept += wave_sum[w];
  }
  if (tid < a.experts) next[tid] += begin;
  if (blockIdx.x == 0) {
    if (tid < a.experts) a.offsets[tid] = begin;
    if (tid == 0) a.offsets[a.experts] = kept;
  }
  __syncthreads();

  const long long first = (long long)blockIdx.x * a.per_chunk;
  const long long last = first + a.per_chunk < a.slots ? first + a.per_chunk : a.slots;
  for (long long i0 = first; i0 < last; i0 += kRouteThreads) {
    const int i = (int)(i0 + tid);
    const bool here = i0 + tid < last;
    const int e = here ? expert_of<ID>(a, i) : -1;
    // lanes of this wave with the same expert
    unsigned long long same = __ballot(e >= 0);
    for (int bit = 1; bit < a.experts; bit <<= 1) {
      const unsigned long long set = __ballot((e & bit) != 0);
      same &= (e & bit) ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (e >= 0 && rank == 0) in_wave[wave][e] = (uint16_t)__popcll(same);
    __syncthreads();
    if (e >= 0) {
      int row = next[e] + rank;
      for (int w = 0; w < wave; ++w) row += in_wave[w][e];
      a.rows[row] = i / a.top;
      a.pos[i] = row;
    } else if (here) {
      a.pos[i] = -1;
    }
    // rows past the last kept slot have no token
    if (here && i >= kept) a.rows[i] = -1;
    __syncthreads();
    if (tid < a.experts) {
      int sum = 0;
      for (int w = 0; w < kRouteWaves; ++w) {
        sum += in_wave[w][tid];
        in_wave[w][tid] = 0;
      }
      next[tid] += sum;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// combination
// ---------------------------------------------------------------------------

constexpr int kCombineThreads = 256;

struct CombineArgs {
  const uint8_t* y;
  const int32_t* pos;
  const float* gates;
  uint8_t* out;
  long long ldy, ldo;
  long long slots;
  int tokens, top, n;
  int lane_bits;  // a workgroup is 2^lane_bits column groups of 8 by tokens
  int col_groups;
};

// A thread sums 8 neighbouring columns of one token, in the order of the
// slots, in fp32.  Bound by reading the expert rows and writing the sums: 32768
// tokens with 2 rows each, a twentieth dropped, n 4096 fp16 (780 MB): 139 us, 5.6
// TB/s (144 with every load by the way of a row's end).  64 tokens with 8 rows, n
// 2048: 4.3 us on the device, where an empty kernel takes 2.5.
template <int DT>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(CombineArgs a) {
  const int cols = 1 << a.lane_bits;
  const long long t = (long long)(blockIdx.x / a.col_groups) * (kCombineThreads >> a.lane_bits) +
                      (threadIdx.x >> a.lane_bits);
  const int c = 8 * ((int)(blockIdx.x % a.col_groups) * cols + (int)(threadIdx.x & (cols - 1)));
  if (t >= a.tokens || c >= a.n) return;
  float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  const int32_t* pos = a.pos + t * a.top;
  const float* gates = a.gates + t * a.top;
  for (int j = 0; j < a.top; ++j) {
    const int p = pos[j];
    if (p < 0 || p >= a.slots) continue;
    const float w = gates[j];
    const uint8_t* row = a.y + 2 * p * a.ldy;
    const u32x4 v = c + 8 <= a.n ? *reinterpret_cast<const u32x4_any*>(row + 2 * (size_t)c) : load_x8_tail(row, c, a.n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[2 * i] = __builtin_fmaf(w, lo_to_f32<DT>(v[i]), s[2 * i]);
      s[2 * i + 1] = __builtin_fmaf(w, hi_to_f32<DT>(v[i]), s[2 * i + 1]);
    }
  }
  uint8_t* o = a.out + 2 * t * a.ldo;
  const u32x4 v = {pack2<DT>(s[0], s[1]), pack2<DT>(s[2], s[3]), pack2<DT>(s[4], s[5]), pack2<DT>(s[6], s[7])};
  if (c + 8 <= a.n) {
    *reinterpret_cast<u32x4_any*>(o + 2 * (size_t)c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.n) *reinterpret_cast<uint16_t*>(o + 2 * (size_t)(c + i)) = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
}

// ---------------------------------------------------------------------------
// host-side argument checks (no HIP call)
// ---------------------------------------------------------------------------

static int weight_tile_bytes(int fmt) {
  switch (fmt) {
    case QR_INT4: return Format<4>::kTileBytes;
    case QR_ASYM4: return Format<20>::kTileBytes;
    case QR_FP4: return Format<36>::kTileBytes;
    default: return 0;
  }
}

// 32-value blocks of one padded weight row.
static size_t row_blocks(int fmt, size_t k) { return fmt == QR_ASYM4 ? (k + 127) / 128 * 4 : (k + 31) / 32; }

static bool bad_dtype(int dt) { return dt != QR_FP16 && dt != QR_BF16; }
static bool misaligned(const void* p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return na && nb && a0 < b0 + nb && b0 < a0 + na;
}

// Bytes from the first to the last value of `rows` rows of `cols` 2-byte values.
static size_t span(size_t rows, size_t ld, size_t cols) { return rows ? 2 * ((rows - 1) * ld + cols) : 0; }

// Whether two matrices share a value.  Rows of one stride may lie beside each
// other in a larger matrix (columns of it): there the distance of the first rows,
// within a stride, tells.  A matrix of one row has the other's stride.
static bool overlap_rows(const void* a, size_t ra, size_t lda, size_t ca, const void* b, size_t rb, size_t ldb, size_t cb) {
  if (!overlap(a, span(ra, lda, ca), b, span(rb, ldb, cb))) return false;
  const size_t ld = 2 * (ra > 1 ? lda : ldb);
  if (ra > 1 && rb > 1 && lda != ldb) return true;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  const size_t from = b0 >= a0 ? (b0 - a0) % ld : (ld - (a0 - b0) % ld) % ld;  // of b's row, from a's
  return from < 2 * ca || from + 2 * cb > ld;
}

// Row strides up to 2^32 values keep every byte offset of 2^30 rows within 63 bits.
constexpr size_t kMaxStride = (size_t)1 << 32;

static qr_status product(qr_format fmt, qr_dtype dtype, int gated, const void* x, size_t ldx, size_t xrows,
                         const void* w, const int32_t* offsets, const int32_t* rows, bool grouped, void* y, size_t ldy,
                         size_t slots, size_t experts, size_t n, size_t k, void* stream) {
  if (!weight_tile_bytes(fmt) || bad_dtype(dtype)) return QR_ERR_UNSUPPORTED;
  if (n < 1 || n > QR_MAX_N || k < 1 || k > QR_MAX_K || slots > QR_MAX_SLOTS || xrows > QR_MAX_SLOTS ||
      experts < 1 || experts > QR_MAX_EXPERTS || ldx < k || ldy < n || ldx > kMaxStride || ldy > kMaxStride)
    return QR_ERR_SIZE;
  const size_t wrows = experts * n * (gated ? 2 : 1);
  const size_t wbytes = qr_weight_bytes(fmt, wrows, k);
  if (!wbytes) return QR_ERR_SIZE;
  if (grouped && !rows && xrows < slots) return QR_ERR_SIZE;
  if (slots == 0) return QR_OK;
  if ((!x && xrows) || !w || !y || (grouped && !offsets)) return QR_ERR_ARG;
  if (misaligned(x, 2) || misaligned(y, 2) || misaligned(w, 16) || misaligned(offsets, 4) || misaligned(rows, 4))
    return QR_ERR_ALIGN;
  const size_t ys = span(slots, ldy, n);
  if (overlap_rows(y, slots, ldy, n, x, xrows, ldx, k) || overlap(y, ys, w, wbytes) ||
      (offsets && overlap(y, ys, offsets, 4 * (experts + 1))) || (rows && overlap(y, ys, rows, 4 * slots)))
    return QR_ERR_ALIAS;
  ProductArgs a = {};
  a.x = (const uint8_t*)x;
  a.w = (const uint8_t*)w;
  a.y = (uint8_t*)y;
  a.offsets = offsets;
  a.rows = rows;
  a.ldx = (long long)ldx;
  a.ldy = (long long)ldy;
  a.xrows = (long long)xrows;
  a.slots = (int)slots;
  a.experts = (int)experts;
  a.n = (int)n;
  a.k = (int)k;
  a.blocks = (int)row_blocks(fmt, k);
  hipStream_t st = (hipStream_t)stream;
  switch (fmt) {
    case QR_INT4: return launch_product_int4(dtype, gated != 0, a, st);
    case QR_ASYM4: return launch_product_asym4(dtype, gated != 0, a, st);
    default: return launch_product_fp4(dtype, gated != 0, a, st);
  }
}

// Slots of one workgroup: whole steps of its threads.
static size_t route_per_chunk(size_t slots) {
  if (slots <= (size_t)kRouteSmall) return slots;
  if (slots <= (size_t)kRouteChunk * kRouteChunks) return kRouteChunk;
  const size_t part = (slots + kRouteChunks - 1) / kRouteChunks;
  return (part + kRouteThreads - 1) / kRouteThreads * kRouteThreads;
}

static int route_chunks(size_t slots) {
  const size_t per = route_per_chunk(slots);
  return slots <= per ? 1 : (int)((slots + per - 1) / per);
}

static bool bad_plan(size_t tokens, size_t top, size_t experts) {
  return top < 1 || top > QR_MAX_TOP || experts < 1 || experts > QR_MAX_EXPERTS || tokens > QR_MAX_SLOTS / top;
}

}  // namespace qr

using namespace qr;

extern "C" {

size_t qr_weight_bytes(qr_format fmt, size_t rows, size_t k) {
  const int tb = weight_tile_bytes(fmt);
  if (!tb || k < 1 || k > QR_MAX_K || rows < 1 || rows > (size_t)QR_MAX_TILES * kTileValues) return 0;
  const size_t tiles = (rows * (row_blocks(fmt, k) * kBlockValues) + kTileValues - 1) / kTileValues;
  return tiles > (size_t)QR_MAX_TILES ? 0 : tiles * (size_t)tb;
}

qr_status qr_linear(qr_format fmt, qr_dtype dtype, int gated, const void* x, size_t ldx, const void* w, void* y,
                    size_t ldy, size_t m, size_t n, size_t k, void* stream) {
  return product(fmt, dtype, gated, x, ldx, m, w, nullptr, nullptr, false, y, ldy, m, 1, n, k, stream);
}

qr_status qr_experts(qr_format fmt, qr_dtype dtype, int gated, const void* x, size_t ldx, size_t tokens,
                     const void* w, const int32_t* offsets, const int32_t* rows, void* y, size_t ldy, size_t slots,
                     size_t experts, size_t n, size_t k, void* stream) {
  return product(fmt, dtype, gated, x, ldx, tokens, w, offsets, rows, true, y, ldy, slots, experts, n, k, stream);
}

size_t qr_route_workspace(size_t tokens, size_t top, size_t experts) {
  if (bad_plan(tokens, top, experts)) return 0;
  const int chunks = route_chunks(tokens * top);
  return chunks == 1 ? 0 : (size_t)chunks * experts * 4;
}

qr_status qr_route(const void* ids, int id_bytes, int32_t* offsets, int32_t* rows, int32_t* pos, size_t tokens,
                   size_t top, size_t experts, void* workspace, void* stream) {
  if (id_bytes != 4 && id_bytes != 8) return QR_ERR_UNSUPPORTED;
  if (bad_plan(tokens, top, experts)) return QR_ERR_SIZE;
  const size_t slots = tokens * top, ws = qr_route_workspace(tokens, top, experts);
  if (!offsets || (slots && (!ids || !rows || !pos)) || (ws && !workspace)) return QR_ERR_ARG;
  if (misaligned(ids, id_bytes) || misaligned(offsets, 4) || misaligned(rows, 4) || misaligned(pos, 4) ||
      misaligned(workspace, 4))
    return QR_ERR_ALIGN;
  const void* buf[] = {offsets, rows, pos, workspace, ids};
  const size_t len[] = {4 * (experts + 1), 4 * slots, 4 * slots, ws, (size_t)id_bytes * slots};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (overlap(buf[i], len[i], buf[j], len[j])) return QR_ERR_ALIAS;
  RouteArgs a = {};
  a.ids = ids;
  a.offsets = offsets;
  a.rows = rows;
  a.pos = pos;
  a.counts = (int32_t*)workspace;
  a.slots = (int)slots;
  a.top = (int)top;
  a.experts = (int)experts;
  a.chunks = route_chunks(slots);
  a.per_chunk = (int)route_per_chunk(slots);
  hipStream_t st = (hipStream_t)stream;
  if (a.chunks > 1) {
    const qr_status s = launch_1d(id_bytes == 4 ? route_count_kernel<int32_t> : route_count_kernel<int64_t>, a.chunks,
                                  kRouteThreads, st, a);
    if (s != QR_OK) return s;
  }
  return launch_1d(id_bytes == 4 ? route_place_kernel<int32_t> : route_place_kernel<int64_t>, a.chunks, kRouteThreads,
                   st, a);
}

qr_status qr_combine(qr_dtype dtype, const void* y, size_t ldy, size_t slots, const int32_t* pos, const float* gates,
                     void* out, size_t ldo, size_t tokens, size_t top, size_t n, void* stream) {
  if (bad_dtype(dtype)) return QR_ERR_UNSUPPORTED;
  if (n < 1 || n > QR_MAX_N || top < 1 || top > QR_MAX_TOP || tokens > QR_MAX_SLOTS / top || slots > QR_MAX_SLOTS ||
      ldy < n || ldo < n || ldy > kMaxStride || ldo > kMaxStride)
    return QR_ERR_SIZE;
  if (tokens == 0) return QR_OK;
  if ((!y && slots) || !pos || !gates || !out) return QR_ERR_ARG;
  if (misaligned(y, 2) || misaligned(out, 2) || misaligned(pos, 4) || misaligned(gates, 4)) return QR_ERR_ALIGN;
  const size_t os = span(tokens, ldo, n);
  if (overlap_rows(out, tokens, ldo, n, y, slots, ldy, n) || overlap(out, os, pos, 4 * tokens * top) ||
      overlap(out, os, gates, 4 * tokens * top))
    return QR_ERR_ALIAS;
  CombineArgs a = {};
  a.y = (const uint8_t*)y;
  a.pos = pos;
  a.gates = gates;
  a.out = (uint8_t*)out;
  a.ldy = (long long)ldy;
  a.ldo = (long long)ldo;
  a.slots = (long long)slots;
  a.tokens = (int)tokens;
  a.top = (int)top;
  a.n = (int)n;
  const int cols = (a.n + 7) / 8;  // column groups of 8
  while ((1 << a.lane_bits) < cols && (1 << a.lane_bits) < kCombineThreads) ++a.lane_bits;
  a.col_groups = (cols + (1 << a.lane_bits) - 1) >> a.lane_bits;
  const int per_group = kCombineThreads >> a.lane_bits;
  // as many tokens at a time as a launch holds (the columns of one group of them always fit)
  static_assert((QR_MAX_N / 8 + kCombineThreads) * 1LL < 0xffffffffLL, "a group of tokens fits a launch");
  const long long fit = kMaxLaunchThreads / ((long long)a.col_groups * kCombineThreads);
  const long long most = (fit > 1 ? fit : 1) * per_group;
  for (long long t = 0; t < (long long)tokens; t += most) {
    const long long now = (long long)tokens - t < most ? (long long)tokens - t : most;
    a.tokens = (int)now;
    a.pos = pos + t * a.top;
    a.gates = gates + t * a.top;
    a.out = (uint8_t*)out + 2 * t * a.ldo;
    const qr_status s = launch_1d(dtype == QR_FP16 ? combine_kernel<kFp16> : combine_kernel<kBf16>,
                                  (now + per_group - 1) / per_group * a.col_groups, kCombineThreads, (hipStream_t)stream, a);
    if (s != QR_OK) return s;
  }
  return QR_OK;
}

}  // extern "C"
