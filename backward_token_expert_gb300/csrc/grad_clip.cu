// Global gradient norm over a list of tensors, and clipping by it:
//   norm = sqrt(sum over all elements g^2),  dst = min(1, max_norm / norm) src.
//
// The list's device table holds chunks: runs of one tensor, so that tensors of
// any size give the warps equal shares and a warp finds its work with one
// 32-byte load.
//
//   gc_small   up to 512 KB: one cluster, a chunk a warp, held in registers
//              between the norm and the scaling (2 KB 2.4 us, 160 KB 3.8 against
//              5.6 by gc_hold, 500 KB 4.9 against 5.6).
//   gc_hold    up to 24 MB: one launch, the chunks held in shared memory over a
//              barrier of the grid.
//   gc_norm    one warp per chunk; each block leaves its sum of squares (fp64).
//   gc_stats   adds the blocks' sums (the norm alone).
//   gc_clip    launched dependently; every block adds the same sums in the
//              same order, so all take the same coefficient, and scales its
//              chunks, last ones first: those are still in L2.
//   gc_ring    the same for lists beyond the L2, through shared memory.
//
// Bound by memory: the norm has to be known before the first value is scaled, so
// what neither the SMs nor the L2 hold is read twice.  2.4 GB of fp32: 1040 us,
// the norm at 6.8 TB/s and the scaling at 7.0 (4.8 GB moved, some of it from L2);
// 59 MB of bf16 in 400 tensors 31 us; 160 KB in six tensors 4 us, most of it launch
// and latency.
//
// Squares: a lane's batch of values (32 fp32 or 64 bf16) is squared and summed
// in fp32 while its largest magnitude lies in [2^-56, 2^52]: no sum of squares
// overflows, and a square that fp32 holds as a subnormal is off by at most
// 2^-150, 2^-38 of the largest square.  Other batches are squared in fp64
// (exact); batches of zeros add nothing.  A lane of gc_norm adds its many batches
// in fp64.  The other sums (of a lane's one to three batches in gc_small and gc_hold,
// over lanes, warps and blocks) are added in fp32 where fp32 holds every term and the
// sum with room to spare, in fp64 where not.  On the way to the norm a square passes at most
// 18 roundings in its batch, 22 in those sums and one in the root: 21 of 2^-24 on
// the norm at the worst, 1.3e-6.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "lrm_internal.cuh"
#include "vec.cuh"

struct lrm_grad_list {
  int device;
  int by;  // which kernels (Plan)
  long long chunks;
  int in_place, has_dst;  // every dst is its src; every non-empty tensor has a dst
  int grid_norm, grid_clip;  // of gc_norm; of gc_hold, gc_clip or gc_ring
  void* table;
};

namespace lrm {
namespace {

constexpr int GC_THREADS = 512;
constexpr int GC_WARPS = GC_THREADS / 32;
constexpr int GC_BATCH = 8;                                    // 16-byte loads a lane has in flight
constexpr int GC_BATCH_BYTES = 32 * 16 * GC_BATCH;             // a warp's batch
constexpr int GC_MAX_GRID = 152 * 4;                           // of gc_norm: sizes the partial sums
constexpr int64_t GC_LARGE_BYTES = int64_t{128} << 20;         // about the L2's size
constexpr int GC_RING_WARPS = 4, GC_RING_THREADS = 32 * GC_RING_WARPS, GC_STAGES = 3;
constexpr int GC_RING_BYTES = 4 * GC_BATCH_BYTES;               // a stage, and the chunks of such lists
constexpr int GC_RING_SMEM = GC_RING_WARPS * GC_STAGES * GC_RING_BYTES;
constexpr int GC_HELD = 3;                                     // chunks a warp of gc_hold keeps in shared memory
constexpr int GC_HOLD_SMEM = GC_WARPS * GC_HELD * GC_BATCH_BYTES;
constexpr int GC_SMS = 152;                                    // the shares of the warps are cut for this many SMs
constexpr int64_t GC_HOLD_BYTES = int64_t{24} << 20;           // of 29 MB that GC_SMS blocks hold: chunks are not all full
constexpr unsigned long long GC_DRAIN_NS = 1000000000ull;      // for copies under way after a wait ran out
constexpr int GC_SMALL_THREADS = 512;
constexpr int GC_SMALL_WARPS = GC_SMALL_THREADS / 32;
constexpr int GC_SMALL_CLUSTER = 8;
constexpr int GC_SMALL_CHUNKS = GC_SMALL_WARPS * GC_SMALL_CLUSTER;
constexpr int64_t GC_SMALL_BYTES = 512 << 10;                  // a cluster's latency against a grid's launch and barrier

// A chunk's kind: its type and what of it lies on 16-byte boundaries.
enum : int32_t { GC_BF16 = 1, GC_DST_ANY = 2, GC_SRC_ANY = 4 };

struct __align__(32) Chunk {
  const void* src;
  void* dst;
  int32_t n;     // elements
  int32_t kind;  // without GC_SRC_ANY: src 16-byte aligned, n a multiple of 16 bytes; without GC_DST_ANY: dst too
  int64_t pad;
};

// The table's head: the blocks' sums, then the arrivals at gc_hold's barrier and the list's status word (zero
// when the list is made).
constexpr size_t GC_ARRIVALS_OFF = GC_MAX_GRID * sizeof(double);
constexpr size_t GC_STATUS_OFF = GC_ARRIVALS_OFF + 128;
constexpr size_t GC_SCRATCH_BYTES = GC_ARRIVALS_OFF + 256;

// The chunks of a list, in order: sink(chunk) for each.  Tensors whose src
// starts off a 16-byte boundary get a short first chunk up to it.
template <typename Sink>
void for_chunks(const lrm_tensor* tensors, int32_t count, int64_t chunk_bytes, Sink sink) {
  for (int32_t i = 0; i < count; ++i) {
    const lrm_tensor& t = tensors[i];
    const int64_t es = t.dtype == LRM_F32 ? 4 : 2, per = 16 / es;
    const char* src = static_cast<const char*>(t.src);
    char* dst = static_cast<char*>(t.dst);
    int64_t at = 0;
    while (at < t.n) {
      const char* s = src + at * es;
      char* d = dst == nullptr ? nullptr : dst + at * es;
      const int64_t left = t.n - at, off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(s) % 16) / es;
      int64_t n;
      int32_t any = GC_SRC_ANY | GC_DST_ANY;
      if (off != 0) {
        n = per - off < left ? per - off : left;
      } else if (left < per) {
        n = left;
      } else {
        const int64_t whole = left / per * per, most = chunk_bytes / es;
        n = whole < most ? whole : most;
        any = d == nullptr || aligned(d, 16) ? 0 : GC_DST_ANY;
      }
      Chunk c;
      c.src = s;
      c.dst = d;
      c.n = static_cast<int32_t>(n);
      c.kind = (t.dtype == LRM_F32 ? 0 : GC_BF16) | any;
      c.pad = 0;
      sink(c);
      at += n;
    }
  }
}

// Number of chunks of for_chunks without walking them.
int64_t count_chunks(const lrm_tensor* tensors, int32_t count, int64_t chunk_bytes) {
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    const lrm_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const int64_t es = t.dtype == LRM_F32 ? 4 : 2, per = 16 / es, most = chunk_bytes / es;
    const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.src) % 16) / es;
    int64_t left = t.n;
    if (off != 0) {
      ++total;
      left -= per - off < left ? per - off : left;
    }
    const int64_t whole = left / per * per;
    total += (whole + most - 1) / most + (left > whole ? 1 : 0);
  }
  return total;
}

// How a list is worked on, and how it is cut.
enum : int { GC_BY_SMALL, GC_BY_HOLD, GC_BY_CLIP, GC_BY_RING };
struct Plan {
  int by;
  int64_t chunk_bytes, chunks;
};

Plan plan_of(const lrm_tensor* tensors, int32_t count) {
  int64_t bytes = 0, skew = 0;  // skew: of tensors whose dst lies on another place of the 16-byte grid than src
  for (int32_t i = 0; i < count; ++i) {
    const int64_t b = tensors[i].n * (tensors[i].dtype == LRM_F32 ? 4 : 2);
    const uintptr_t src = reinterpret_cast<uintptr_t>(tensors[i].src), dst = reinterpret_cast<uintptr_t>(tensors[i].dst);
    bytes += b;
    if (dst != 0 && (src ^ dst) % 16 != 0) skew += b;
  }
  const auto plan = [&](int by, int64_t b) { return Plan{by, b, count_chunks(tensors, count, b)}; };
  // bulk copies need both ends on the grid; what is not wants the warps of gc_clip (200 MB off it: 1460 us by
  // gc_ring's four warps an SM)
  if (bytes > GC_LARGE_BYTES && skew <= bytes / 16) return plan(GC_BY_RING, GC_RING_BYTES);
  // chunks for up to 32 warps of gc_small, or as many as it has
  if (bytes <= GC_SMALL_BYTES)
    for (int64_t b = 512; b <= GC_BATCH_BYTES; b *= 2) {
      const Plan p = plan(GC_BY_SMALL, b);
      if (p.chunks <= (b < GC_BATCH_BYTES ? 32 : GC_SMALL_CHUNKS)) return p;
    }
  // up to a batch of a warp, cut so that the warps get equal numbers: of one block an SM, or of two
  const auto even = [&](int64_t warps) {
    const int64_t rounds = (bytes + warps * GC_BATCH_BYTES - 1) / (warps * GC_BATCH_BYTES);
    const int64_t b = (bytes + warps * rounds - 1) / (warps * rounds);
    return b > 512 ? (b + 127) / 128 * 128 : int64_t{512};
  };
  if (bytes <= GC_HOLD_BYTES) {
    const Plan p = plan(GC_BY_HOLD, even(GC_SMS * GC_WARPS));
    if (p.chunks <= static_cast<int64_t>(GC_HELD) * GC_SMS * GC_WARPS) return p;
  }
  return plan(GC_BY_CLIP, even(2 * GC_SMS * GC_WARPS));
}

lrm_status check_tensors(const lrm_tensor* tensors, int32_t count) {
  if (count < 0 || (count > 0 && tensors == nullptr)) return LRM_ERR_INVALID_ARG;
  int64_t elements = 0;
  for (int32_t i = 0; i < count; ++i) {
    const lrm_tensor& t = tensors[i];
    if (t.n < 0 || (t.dtype != LRM_F32 && t.dtype != LRM_BF16)) return LRM_ERR_INVALID_ARG;
    if (t.n > (static_cast<int64_t>(1) << 42)) return LRM_ERR_SHAPE;
    elements += t.n;
    if (elements > (static_cast<int64_t>(1) << 43)) return LRM_ERR_SHAPE;
    if (t.n > 0 && t.src == nullptr) return LRM_ERR_INVALID_ARG;
    const size_t es = t.dtype == LRM_F32 ? 4 : 2;
    if (!aligned(t.src, es) || !aligned(t.dst, es)) return LRM_ERR_ALIGN;
  }
  return LRM_OK;
}

__device__ __forceinline__ bool in_fp32_range(float mx) { return mx >= 0x1p-56f && mx <= 0x1p52f; }

template <bool F32>
__device__ __forceinline__ void unpack(const uint4& x, float (&v)[8]) {
  if constexpr (F32) {
    v[0] = __uint_as_float(x.x);
    v[1] = __uint_as_float(x.y);
    v[2] = __uint_as_float(x.z);
    v[3] = __uint_as_float(x.w);
  } else {
    v[0] = bf16_lo(x.x);
    v[1] = bf16_hi(x.x);
    v[2] = bf16_lo(x.y);
    v[3] = bf16_hi(x.y);
    v[4] = bf16_lo(x.z);
    v[5] = bf16_hi(x.z);
    v[6] = bf16_lo(x.w);
    v[7] = bf16_hi(x.w);
  }
}

template <bool F32>
__device__ __noinline__ double exact_squares(uint4 x) {
  float v[8];
  unpack<F32>(x, v);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 8); ++i) sum += static_cast<double>(v[i]) * v[i];
  return sum;
}

// A lane's sum of squares: of batches that fp32 holds, and of the others.
struct Squares {
  float f;
  double d;
};

__device__ __forceinline__ bool is_wide(const Squares& q) { return (__double2hiint(q.d) | __double2loint(q.d)) != 0; }
__device__ __forceinline__ void add_to(double& sum, const Squares& q) {
  sum += q.f;
  if (is_wide(q)) sum += q.d;
}

// Adds the squares of a lane's batch; places beyond the chunk hold 0.
template <bool F32>
__device__ __forceinline__ void batch_squares(const uint4 (&x)[GC_BATCH], Squares& sum) {
  float mx = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < GC_BATCH; ++j) {
    float v[8];
    unpack<F32>(x[j], v);
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 8); ++i) {
      mx = fmaxf(mx, fabsf(v[i]));
      a[i % 4] = fmaf(v[i], v[i], a[i % 4]);
    }
  }
  const float s = (a[0] + a[1]) + (a[2] + a[3]);
  if (in_fp32_range(mx)) {
    sum.f += s;  // a NaN among the values is in s
  } else if (mx != 0.f || s != 0.f) {
#pragma unroll 1
    for (int j = 0; j < GC_BATCH; ++j) {
      uint4 y = x[0];
#pragma unroll
      for (int i = 1; i < GC_BATCH; ++i)
        if (i == j) y = x[i];
      sum.d += exact_squares<F32>(y);
    }
  }
}

__device__ __forceinline__ void batch_squares(const uint4 (&x)[GC_BATCH], bool f32, Squares& sum) {
  if (f32)
    batch_squares<true>(x, sum);
  else
    batch_squares<false>(x, sum);
}

__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ void load_batch(const uint4* p, int v0, int nv, int lane, uint4 (&x)[GC_BATCH]) {
  if (v0 + 32 * GC_BATCH <= nv) {
#pragma unroll
    for (int j = 0; j < GC_BATCH; ++j) x[j] = ld_once(p + v0 + lane + 32 * j);
  } else {
#pragma unroll
    for (int j = 0; j < GC_BATCH; ++j) {
      const int v = v0 + lane + 32 * j;
      x[j] = v < nv ? ld_once(p + v) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

__device__ __forceinline__ uint4 scale_f32x4(const uint4& x, float c) {
  return make_uint4(__float_as_uint(__uint_as_float(x.x) * c), __float_as_uint(__uint_as_float(x.y) * c),
                    __float_as_uint(__uint_as_float(x.z) * c), __float_as_uint(__uint_as_float(x.w) * c));
}

__device__ __forceinline__ void store_batch(uint4* q, int v0, int nv, int lane, const uint4 (&x)[GC_BATCH], bool f32,
                                            float coef) {
#pragma unroll
  for (int j = 0; j < GC_BATCH; ++j) {
    const int v = v0 + lane + 32 * j;
    if (v < nv) __stcs(q + v, f32 ? scale_f32x4(x[j], coef) : scale_bf16x8(x[j], coef));
  }
}

__device__ __forceinline__ bool is_f32(const Chunk& c) { return (c.kind & GC_BF16) == 0; }
__device__ __forceinline__ bool src_vec(const Chunk& c) { return (c.kind & GC_SRC_ANY) == 0; }
__device__ __forceinline__ bool both_vec(const Chunk& c) { return (c.kind & (GC_SRC_ANY | GC_DST_ANY)) == 0; }
__device__ __forceinline__ int vectors(const Chunk& c) { return c.n / (is_f32(c) ? 4 : 8); }

// Chunks off the 16-byte grid, element by element, GC_BATCH of them a lane at a
// time.
__device__ __forceinline__ float any_load(const Chunk& c, int i) {
  return is_f32(c) ? static_cast<const float*>(c.src)[i]
                   : __bfloat162float(static_cast<const __nv_bfloat16*>(c.src)[i]);
}
// (a chunk whose src is off the grid is shorter than a vector: a lane an element)
__device__ __forceinline__ void any_squares(const Chunk& c, int lane, Squares& sum) {
  const float v = lane < c.n ? any_load(c, lane) : 0.f;
  if (v == 0.f) return;
  if (in_fp32_range(fabsf(v)))
    sum.f = fmaf(v, v, sum.f);
  else
    sum.d += static_cast<double>(v) * v;
}
__device__ __noinline__ void any_scale(const Chunk& c, float coef, int lane) {
  for (int i0 = lane; i0 < c.n; i0 += 32 * GC_BATCH) {
    float v[GC_BATCH];
#pragma unroll
    for (int j = 0; j < GC_BATCH; ++j)
      if (i0 + 32 * j < c.n) v[j] = any_load(c, i0 + 32 * j);
#pragma unroll
    for (int j = 0; j < GC_BATCH; ++j) {
      const int i = i0 + 32 * j;
      if (i >= c.n) continue;
      if (is_f32(c))
        static_cast<float*>(c.dst)[i] = v[j] * coef;
      else
        static_cast<__nv_bfloat16*>(c.dst)[i] = __float2bfloat16_rn(v[j] * coef);
    }
  }
}

// Sums of squares (v >= 0, infinite or NaN) over a warp, for every lane.  The
// SM's fp64 unit takes a warp's addition in 16 clocks, so sums that fp32 holds
// with room to spare are added in fp32 (six roundings more).
__device__ __forceinline__ bool fits_f32(double v) {
  const int ex = __double2hiint(v) >> 20;  // biased exponent; negative values do not occur
  return v == 0.0 || (ex >= 1023 - 112 && ex <= 1023 + 121);
}
__device__ __forceinline__ double warp_sum(double v) {
  if (__all_sync(0xffffffffu, fits_f32(v))) {
    float f = static_cast<float>(v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
    return f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A block's sum, for warp 0.  The common case leaves the fp64 unit alone.
__device__ __forceinline__ double block_squares(const Squares& mine) {
  __shared__ float s_f[32];
  __shared__ double s_d[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float f = mine.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
  if (lane == 0) s_f[warp] = f;
  const int any_wide = __syncthreads_or(is_wide(mine));
  if (warp == 0) {
    f = lane < static_cast<int>(blockDim.x >> 5) ? s_f[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
  }
  double sum = f;
  if (any_wide) {
    const double d = warp_sum(mine.d);
    if (lane == 0) s_d[warp] = d;
    __syncthreads();
    if (warp == 0) sum += warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? s_d[lane] : 0.0);
  }
  return sum;
}

__device__ __forceinline__ lrm_grad_stats make_stats(double squares, float max_norm) {
  lrm_grad_stats r;
  if (fits_f32(squares)) {
    r.norm = sqrtf(static_cast<float>(squares));
    r.nonfinite = 0;
    r.coef = r.norm > max_norm ? max_norm / r.norm : 1.f;
    return r;
  }
  const double norm = sqrt(squares);
  r.norm = static_cast<float>(norm);
  r.nonfinite = isfinite(norm) ? 0 : 1;
  r.coef = !r.nonfinite && norm > max_norm ? static_cast<float>(max_norm / norm) : 1.f;
  return r;
}

// cleared: the stats that gc_ring's blocks write together, or null.
__global__ void __launch_bounds__(GC_THREADS, 2) gc_norm(const Chunk* __restrict__ chunks, long long count,
                                                      double* __restrict__ partial,
                                                      lrm_grad_stats* __restrict__ cleared) {
  __shared__ double s_sum[GC_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_launch();
  if (cleared != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *cleared = lrm_grad_stats{0.f, 1.f, 0};
  const long long step = static_cast<long long>(gridDim.x) * GC_WARPS;
  long long i = static_cast<long long>(blockIdx.x) * GC_WARPS + warp;
  double sum = 0.0;
  Chunk next = {};
  if (i < count) next = chunks[i];
  for (; i < count; i += step) {
    const Chunk c = next;
    if (i + step < count) next = chunks[i + step];
    if (src_vec(c)) {
      const int nv = vectors(c);
      for (int v0 = 0; v0 < nv; v0 += 32 * GC_BATCH) {
        uint4 x[GC_BATCH];
        load_batch(static_cast<const uint4*>(c.src), v0, nv, lane, x);
        Squares q{0.f, 0.0};
        batch_squares(x, is_f32(c), q);
        add_to(sum, q);
      }
    } else {
      Squares q{0.f, 0.0};
      any_squares(c, lane, q);
      add_to(sum, q);
    }
  }
  sum = warp_sum(sum);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    sum = warp_sum(lane < GC_WARPS ? s_sum[lane] : 0.0);
    if (lane == 0) partial[blockIdx.x] = sum;
  }
}

// The blocks' sums added in a fixed order; the whole block gets the result.
// One thread takes the root and the quotient: the SM's fp64 unit finishes two
// lanes a clock, and every warp doing so cost 7 us.
__device__ lrm_grad_stats block_stats(const double* __restrict__ partial, int nblk, float max_norm) {
  __shared__ double s_part[GC_WARPS];
  __shared__ lrm_grad_stats s_stats;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double a = 0.0;
  for (int i = threadIdx.x; i < nblk; i += blockDim.x) a += __ldcg(partial + i);  // written by the kernel before: not through L1
  if (warp * 32 < nblk) a = warp_sum(a);
  if (lane == 0) s_part[warp] = a;
  __syncthreads();
  if (warp == 0) {
    a = warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? s_part[lane] : 0.0);
    if (lane == 0) s_stats = make_stats(a, max_norm);
  }
  __syncthreads();
  return s_stats;
}

__global__ void __launch_bounds__(GC_THREADS) gc_stats(const double* __restrict__ partial, int nblk,
                                                       lrm_grad_stats* __restrict__ stats) {
  grid_dependency_wait();
  const lrm_grad_stats r = block_stats(partial, nblk, INFINITY);
  if (threadIdx.x == 0) *stats = r;
}

// In the context's word and in the list's own: lists may share a context.
__device__ __forceinline__ void raise_timeout(unsigned int* status, unsigned int* own_status) {
  raise_flag(status, LRM_ERR_TIMEOUT);
  raise_flag(own_status, LRM_ERR_TIMEOUT);
}

// Every block of the launch arrives once and waits for the others (all are
// resident: the launch is cooperative).  The arrivals are never reset, so that a
// call needs nothing cleared before it: they are a multiple of the grid between
// calls.
//
// All blocks return the same: true once all have arrived, or false if one gave
// up before that.  A block gives up by setting the call's bit in the word that
// counts the arrivals, and only while the count is short, so whoever sees all
// arrivals sees the bit as well.  `late` blocks give up before they arrive, and
// so do those that are given no time while there are others to wait for.  The
// calls of a list take the two bits in turn; the first to arrive clears the
// other one, which only the call before used.
constexpr unsigned long long GC_COUNT = (1ull << 62) - 1;
__device__ __forceinline__ unsigned long long ld_acquire(const unsigned long long* p) {
  unsigned long long v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long given_up_bit(unsigned long long call) { return 1ull << (62 + (call & 1)); }
__device__ bool grid_barrier(unsigned long long* arrivals, bool late, unsigned long long wait_ns) {
  __shared__ int s_ok;
  __syncthreads();
  if (threadIdx.x == 0) {
    // this block's arrival is missing, so the count is still that of this call
    if (late || (wait_ns == 0 && gridDim.x > 1))
      atomicOr(arrivals, given_up_bit((ld_acquire(arrivals) & GC_COUNT) / gridDim.x));
    __threadfence();
    const unsigned long long mine = atomicAdd(arrivals, 1ull), call = (mine & GC_COUNT) / gridDim.x;
    const unsigned long long want = (call + 1) * gridDim.x, bit = given_up_bit(call), old_bit = given_up_bit(call + 1);
    if ((mine & old_bit) != 0 && (mine & GC_COUNT) == call * gridDim.x) atomicAnd(arrivals, ~old_bit);
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
      const unsigned long long now = ld_acquire(arrivals);
      if ((now & bit) != 0) {
        s_ok = 0;
        break;
      }
      if ((now & GC_COUNT) >= want) {
        s_ok = 1;
        break;
      }
      // fails where another block came in between, at most a grid's number of times; looked at again in both cases
      if ((it & 15u) == 0 && globaltimer_ns() - t0 > wait_ns) atomicCAS(arrivals, now, now | bit);
    }
  }
  __syncthreads();
  return s_ok != 0;
}

// Norm and scaling in one launch, for lists of up to GC_HELD chunks a warp: they
// come to shared memory by bulk copies and stay there over the grid's barrier, so
// that they are read once (4 MB of fp32 6.8 us against 8.8 with two launches, 8 MB
// 7.3 against 9.3, 16 MB 10.2 against 11.9; holding part of a longer list and
// reading the rest twice gains nothing: 60 MB 33.6 us against 32.0).
__global__ void __launch_bounds__(GC_THREADS, 1) gc_hold(const Chunk* __restrict__ chunks, long long count,
                                                        double* __restrict__ partial, unsigned long long* arrivals,
                                                        int scale, float max_norm, int in_place,
                                                        lrm_grad_stats* __restrict__ stats,
                                                        unsigned long long wait_ns, unsigned int* status,
                                                        unsigned int* own_status) {
  extern __shared__ __align__(128) unsigned char gc_smem[];
  __shared__ uint64_t s_full[GC_WARPS][GC_HELD];
  __shared__ int s_late;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint4* held = reinterpret_cast<uint4*>(gc_smem + warp * (GC_HELD * GC_BATCH_BYTES));
  constexpr int HELD_VECS = GC_BATCH_BYTES / 16;
  uint64_t* full = s_full[warp];
  const long long step = static_cast<long long>(gridDim.x) * GC_WARPS;
  const long long first = static_cast<long long>(blockIdx.x) * GC_WARPS + warp;
  if (threadIdx.x == 0) s_late = 0;
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < GC_HELD; ++j) mbar_init(&full[j], 1);
    fence_mbar_init();
  }
  __syncthreads();
  Chunk kept[GC_HELD];
#pragma unroll
  for (int j = 0; j < GC_HELD; ++j) {
    kept[j].n = 0;
    if (first + j * step < count) kept[j] = chunks[first + j * step];
  }
#pragma unroll
  for (int j = 0; j < GC_HELD; ++j) {
    if (kept[j].n > 0 && src_vec(kept[j]) && lane == 0) {
      const uint32_t bytes = static_cast<uint32_t>(vectors(kept[j])) * 16u;
      mbar_arrive_expect_tx(&full[j], bytes);
      bulk_load(held + j * HELD_VECS, kept[j].src, bytes, &full[j]);
    }
  }
  Squares sum{0.f, 0.0};
#pragma unroll
  for (int j = 0; j < GC_HELD; ++j) {
    const Chunk& c = kept[j];
    if (c.n == 0) continue;
    if (src_vec(c)) {
      if (!mbar_wait(&full[j], 0, wait_ns, nullptr)) s_late = 1;
      const int nv = vectors(c);
      uint4 x[GC_BATCH];
#pragma unroll
      for (int b = 0; b < GC_BATCH; ++b) {
        const int v = lane + 32 * b;
        x[b] = v < nv ? held[j * HELD_VECS + v] : make_uint4(0u, 0u, 0u, 0u);
      }
      batch_squares(x, is_f32(c), sum);
    } else {
      any_squares(c, lane, sum);
    }
  }
  const double total = block_squares(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = total;
  if (!grid_barrier(arrivals, s_late != 0, wait_ns)) {  // in every block: none of them scales
    if (threadIdx.x == 0) {
      raise_timeout(status, own_status);
      if (blockIdx.x == 0) *stats = lrm_grad_stats{nanf(""), 1.f, 1};
    }
    if (s_late) {  // a late copy gets a last chance to land before the block ends
#pragma unroll
      for (int j = 0; j < GC_HELD; ++j)
        if (kept[j].n > 0 && src_vec(kept[j])) mbar_wait(&full[j], 0, GC_DRAIN_NS, nullptr);
    }
    return;
  }
  if (!scale && blockIdx.x != 0) return;
  const lrm_grad_stats r = block_stats(partial, gridDim.x, scale ? max_norm : INFINITY);
  if (blockIdx.x == 0 && threadIdx.x == 0) *stats = r;
  if (!scale || (in_place && r.coef == 1.f)) return;
#pragma unroll
  for (int j = 0; j < GC_HELD; ++j) {
    const Chunk& c = kept[j];
    if (c.n == 0) continue;
    if (both_vec(c)) {
      const int nv = vectors(c);
      uint4* q = static_cast<uint4*>(c.dst);
      const bool f32 = is_f32(c);
#pragma unroll
      for (int b = 0; b < GC_BATCH; ++b) {
        const int v = lane + 32 * b;
        if (v < nv) {
          const uint4 x = held[j * HELD_VECS + v];
          __stcs(q + v, f32 ? scale_f32x4(x, r.coef) : scale_bf16x8(x, r.coef));
        }
      }
    } else {
      any_scale(c, r.coef, lane);
    }
  }
}

__global__ void __launch_bounds__(GC_THREADS) gc_clip(const Chunk* __restrict__ chunks, long long count,
                                                      const double* __restrict__ partial, int nblk, float max_norm,
                                                      int in_place, lrm_grad_stats* __restrict__ stats) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * GC_WARPS;
  long long i = count - 1 - (static_cast<long long>(blockIdx.x) * GC_WARPS + warp);
  Chunk next = {};
  if (i >= 0) next = chunks[i];  // the table was there before gc_norm began
  grid_dependency_wait();
  const lrm_grad_stats r = block_stats(partial, nblk, max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *stats = r;
  if (in_place && r.coef == 1.f) return;
  for (; i >= 0; i -= step) {
    const Chunk c = next;
    if (i >= step) next = chunks[i - step];
    if (both_vec(c)) {
      const int nv = vectors(c);
      for (int v0 = 0; v0 < nv; v0 += 32 * GC_BATCH) {
        uint4 x[GC_BATCH];
        load_batch(static_cast<const uint4*>(c.src), v0, nv, lane, x);
        store_batch(static_cast<uint4*>(c.dst), v0, nv, lane, x, is_f32(c), r.coef);
      }
    } else {
      any_scale(c, r.coef, lane);
    }
  }
}

// The stats that gc_norm cleared are written by block 0 of gc_ring and, where a
// copy does not come, by that copy's warp, in any order: a norm's bits grow with it
// and NaN's are above them all, so the maximum stands for both.
__device__ __forceinline__ void merge_stats(lrm_grad_stats* stats, float norm, int nonfinite) {
  atomicMax(reinterpret_cast<unsigned int*>(&stats->norm), __float_as_uint(norm));
  atomicOr(&stats->nonfinite, nonfinite);
}

// The scaling of lists beyond the L2.  A warp's ring: its chunks come by bulk
// copies GC_STAGES ahead, are scaled in shared memory and leave by bulk copies,
// so that DRAM sees runs of 16 KB each way (2.4 GB of fp32, norm and scaling:
// 1038 us; through registers 1099; 8 KB runs 1108, four stages of 12 KB 1083, two
// of 16 KB for six warps 1058).  The first copies are under way before the norm is
// known: gc_norm does not write what they read.
__global__ void __launch_bounds__(GC_RING_THREADS, 1) gc_ring(const Chunk* __restrict__ chunks, long long count,
                                                             const double* __restrict__ partial, int nblk,
                                                             float max_norm, int in_place,
                                                             lrm_grad_stats* __restrict__ stats,
                                                             unsigned long long wait_ns, unsigned int* status,
                                                             unsigned int* own_status) {
  extern __shared__ __align__(128) unsigned char gc_smem[];
  __shared__ uint64_t s_full[GC_RING_WARPS][GC_STAGES];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* ring = gc_smem + warp * (GC_STAGES * GC_RING_BYTES);
  uint64_t* full = s_full[warp];
  const long long step = static_cast<long long>(gridDim.x) * GC_RING_WARPS;
  const long long first = count - 1 - (static_cast<long long>(blockIdx.x) * GC_RING_WARPS + warp);
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < GC_STAGES; ++j) mbar_init(&full[j], 1);
    fence_mbar_init();
  }
  __syncwarp();
  Chunk held[GC_STAGES];
  const auto fetch = [&](int j, long long i) {  // stage j takes chunk i
    held[j].n = 0;
    if (i < 0) return;
    held[j] = chunks[i];
    if (both_vec(held[j]) && lane == 0) {
      const uint32_t bytes = static_cast<uint32_t>(vectors(held[j])) * 16u;
      mbar_arrive_expect_tx(&full[j], bytes);
      bulk_load(ring + j * GC_RING_BYTES, held[j].src, bytes, &full[j]);
    }
  };
#pragma unroll
  for (int j = 0; j < GC_STAGES; ++j) fetch(j, first - j * step);
  grid_dependency_wait();
  const lrm_grad_stats r = block_stats(partial, nblk, max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    stats->coef = r.coef;
    merge_stats(stats, r.norm, r.nonfinite);
  }
  const bool scale = !(in_place && r.coef == 1.f);
  uint32_t phases = 0;  // bit j: the parity that stage j's next copy completes
  bool ok = true;
  for (long long i = first; i >= 0 && ok; i -= GC_STAGES * step) {
#pragma unroll
    for (int j = 0; j < GC_STAGES; ++j) {
      const Chunk c = held[j];
      const long long at = i - j * step;
      uint4* buf = reinterpret_cast<uint4*>(ring + j * GC_RING_BYTES);
      if (ok && c.n > 0) {
        if (both_vec(c)) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[j], (phases >> j) & 1u, wait_ns, nullptr));
          if (ok) {
            phases ^= 1u << j;
            held[j].n = 0;  // nothing under way in this stage
            if (scale) {
              const int nv = vectors(c);
              const bool f32 = is_f32(c);
#pragma unroll 4
              for (int v = lane; v < nv; v += 32) buf[v] = f32 ? scale_f32x4(buf[v], r.coef) : scale_bf16x8(buf[v], r.coef);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) bulk_store(c.dst, buf, static_cast<uint32_t>(nv) * 16u);
            }
          }
        } else {
          held[j].n = 0;
          if (scale) any_scale(c, r.coef, lane);
        }
      }
      if (lane == 0) bulk_commit();
      // the stage of the chunk before this one is free once its store has read it
      if (at != first && ok && scale) {
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
        fetch((j + GC_STAGES - 1) % GC_STAGES, at + step - GC_STAGES * step);
      }
    }
    if (!scale) break;
  }
  if (!ok && lane == 0) {
    raise_timeout(status, own_status);
    merge_stats(stats, nanf(""), 1);
  }
  // copies still under way (after a wait that ran out) get a last chance to land
#pragma unroll
  for (int j = 0; j < GC_STAGES; ++j)
    if (held[j].n > 0 && both_vec(held[j])) mbar_wait(&full[j], (phases >> j) & 1u, GC_DRAIN_NS, nullptr);
  if (lane == 0) bulk_wait<0>();
}

// One cluster, a chunk a warp, the values in registers between the norm and the
// scaling; every block gets the other blocks' sums.  scale = 0: the norm alone.
__global__ void __launch_bounds__(GC_SMALL_THREADS) gc_small(const Chunk* __restrict__ chunks, int count, int scale,
                                                             float max_norm, int in_place,
                                                             lrm_grad_stats* __restrict__ stats) {
  __shared__ double s_rank[GC_SMALL_CLUSTER];
  __shared__ lrm_grad_stats s_stats;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), ranks = static_cast<int>(gridDim.x);
  const int i = rank * static_cast<int>(blockDim.x >> 5) + warp;
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this block has started
  Chunk c = {};
  if (i < count) c = chunks[i];
  const bool vec = i < count && src_vec(c);
  uint4 x[GC_BATCH];
  Squares sum{0.f, 0.0};
  if (vec) {
    load_batch(static_cast<const uint4*>(c.src), 0, vectors(c), lane, x);
    batch_squares(x, is_f32(c), sum);
  } else if (i < count) {
    any_squares(c, lane, sum);
  }
  double total = block_squares(sum);
  if (ranks > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 0 && lane < ranks)
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(mapa_shared(&s_rank[rank], lane)), "d"(total) : "memory");
    cluster_sync_all();
  }
  if (threadIdx.x == 0) {
    if (ranks > 1) {
      total = 0.0;
      for (int r = 0; r < ranks; ++r) total += s_rank[r];
    }
    s_stats = make_stats(total, scale ? max_norm : INFINITY);
    if (rank == 0) *stats = s_stats;
  }
  __syncthreads();
  const lrm_grad_stats r = s_stats;
  if (!scale || (in_place && r.coef == 1.f)) return;
  if (vec && both_vec(c))
    store_batch(static_cast<uint4*>(c.dst), 0, vectors(c), lane, x, is_f32(c), r.coef);
  else if (i < count)
    any_scale(c, r.coef, lane);
}

const Chunk* chunks_of(const lrm_grad_list* list) {
  return reinterpret_cast<const Chunk*>(static_cast<char*>(list->table) + GC_SCRATCH_BYTES);
}

unsigned int* status_of(const lrm_grad_list* list) {
  return reinterpret_cast<unsigned int*>(static_cast<char*>(list->table) + GC_STATUS_OFF);
}

lrm_status launch_small(const lrm_grad_list* list, int scale, float max_norm, lrm_grad_stats* stats, cudaStream_t s) {
  const int count = static_cast<int>(list->chunks);
  int ranks = (count + 7) / 8;  // eight warps a block, more once there are eight blocks
  ranks = ranks < 1 ? 1 : ranks < GC_SMALL_CLUSTER ? ranks : GC_SMALL_CLUSTER;
  const int warps = count > 0 ? (count + ranks - 1) / ranks : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(32 * warps);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, gc_small, chunks_of(list), count, scale, max_norm, list->in_place, stats) !=
      cudaSuccess) {
    cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  return LRM_OK;
}

// scale = 0: the norm alone.
lrm_status launch_hold(lrm_ctx* ctx, const lrm_grad_list* list, int scale, float max_norm, lrm_grad_stats* stats,
                       cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(list->grid_clip);
  cfg.blockDim = dim3(GC_THREADS);
  cfg.dynamicSmemBytes = GC_HOLD_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  unsigned long long* arrivals =
      reinterpret_cast<unsigned long long*>(static_cast<char*>(list->table) + GC_ARRIVALS_OFF);
  if (cudaLaunchKernelEx(&cfg, gc_hold, chunks_of(list), list->chunks, static_cast<double*>(list->table), arrivals,
                         scale, max_norm, list->in_place, stats, ctx->wait_budget_ns, ctx->d_status,
                         status_of(list)) != cudaSuccess) {
    cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  return LRM_OK;
}

lrm_status launch_norm(const lrm_grad_list* list, lrm_grad_stats* cleared, cudaStream_t s) {
  if (list->chunks == 0) return LRM_OK;
  gc_norm<<<list->grid_norm, GC_THREADS, 0, s>>>(chunks_of(list), list->chunks, static_cast<double*>(list->table),
                                                 cleared);
  return launch_status();
}

}  // namespace
}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_grad_table_size(const lrm_tensor* tensors, int32_t count, size_t* bytes) {
  if (bytes == nullptr) return LRM_ERR_INVALID_ARG;
  const lrm_status st = check_tensors(tensors, count);
  if (st != LRM_OK) return st;
  *bytes = GC_SCRATCH_BYTES + static_cast<size_t>(plan_of(tensors, count).chunks) * sizeof(Chunk);
  return LRM_OK;
}

extern "C" lrm_status lrm_grad_list_create(lrm_ctx* ctx, const lrm_tensor* tensors, int32_t count, void* table,
                                           size_t table_bytes, void* stream, lrm_grad_list** out) {
  if (out == nullptr) return LRM_ERR_INVALID_ARG;
  *out = nullptr;
  if (ctx == nullptr) return LRM_ERR_INVALID_ARG;
  size_t need = 0;
  lrm_status st = lrm_grad_table_size(tensors, count, &need);
  if (st != LRM_OK) return st;
  if (table == nullptr || table_bytes < need) return LRM_ERR_WORKSPACE;
  if (!aligned(table, 256)) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) {
    cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  if (cap != cudaStreamCaptureStatusNone) return LRM_ERR_INVALID_ARG;
  lrm_grad_list* list = static_cast<lrm_grad_list*>(calloc(1, sizeof(lrm_grad_list)));
  if (list == nullptr) return LRM_ERR_CUDA;
  list->device = ctx->device;
  list->table = table;
  list->in_place = 1;
  list->has_dst = 1;
  for (int32_t i = 0; i < count; ++i) {
    if (tensors[i].n == 0) continue;
    if (tensors[i].dst == nullptr) list->has_dst = 0;
    if (tensors[i].dst != tensors[i].src) list->in_place = 0;
  }
  const Plan plan = plan_of(tensors, count);
  list->by = plan.by;
  list->chunks = plan.chunks;
  list->grid_clip = 1;
  if (list->chunks > 0) {
    // the arrivals (zero) and, after them, the chunks
    constexpr size_t head = GC_SCRATCH_BYTES - GC_ARRIVALS_OFF;
    const size_t size = head + static_cast<size_t>(list->chunks) * sizeof(Chunk);
    char* host = static_cast<char*>(aligned_alloc(256, (size + 255) / 256 * 256));
    if (host == nullptr) {
      free(list);
      return LRM_ERR_CUDA;
    }
    memset(host, 0, head);
    Chunk* at = reinterpret_cast<Chunk*>(host + head);
    for_chunks(tensors, count, plan.chunk_bytes, [&](const Chunk& c) { *at++ = c; });
    cudaError_t e = cudaMemcpyAsync(static_cast<char*>(table) + GC_ARRIVALS_OFF, host, size, cudaMemcpyHostToDevice, s);
    // where the GPU reads pageable memory itself the copy may still be reading `host` when the call returns
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    free(host);
    if (e != cudaSuccess) {
      cudaGetLastError();
      free(list);
      return LRM_ERR_CUDA;
    }
    const long long blocks = (list->chunks + GC_WARPS - 1) / GC_WARPS;
    static thread_local int dev = -1, resident_norm = 0, resident_clip = 0;
    if (dev != ctx->device) {
      if (cudaFuncSetAttribute(gc_hold, cudaFuncAttributeMaxDynamicSharedMemorySize, GC_HOLD_SMEM) != cudaSuccess ||
          cudaFuncSetAttribute(gc_ring, cudaFuncAttributeMaxDynamicSharedMemorySize, GC_RING_SMEM) != cudaSuccess) {
        cudaGetLastError();
        free(list);
        return LRM_ERR_CUDA;
      }
      resident_norm = resident_grid(ctx, gc_norm, GC_THREADS, 0);
      resident_clip = resident_grid(ctx, gc_clip, GC_THREADS, 0);
      dev = ctx->device;
    }
    const int gn = resident_norm < GC_MAX_GRID ? resident_norm : GC_MAX_GRID;
    // a part with fewer SMs than the plan counts on
    if (plan.by == GC_BY_HOLD && plan.chunks > static_cast<int64_t>(GC_HELD) * ctx->sm_count * GC_WARPS)
      list->by = GC_BY_CLIP;
    const int gc = list->by == GC_BY_CLIP ? resident_clip : ctx->sm_count;
    list->grid_norm = static_cast<int>(blocks < gn ? blocks : gn);
    list->grid_clip = static_cast<int>(blocks < gc ? blocks : gc);
  }
  *out = list;
  return LRM_OK;
}

extern "C" lrm_status lrm_grad_list_destroy(lrm_grad_list* list) {
  free(list);
  return LRM_OK;
}

extern "C" lrm_status lrm_grad_list_status(lrm_ctx* ctx, const lrm_grad_list* list, void* stream, uint32_t* flags) {
  if (ctx == nullptr || list == nullptr || flags == nullptr || list->device != ctx->device) return LRM_ERR_INVALID_ARG;
  *flags = 0;
  if (list->chunks == 0) return LRM_OK;  // its table was not written, and nothing of it can fail
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int host = 0;
  LRM_CHECK_CUDA(cudaMemcpyAsync(&host, status_of(list), sizeof(host), cudaMemcpyDeviceToHost, s));
  LRM_CHECK_CUDA(cudaStreamSynchronize(s));
  if (host != 0) {
    LRM_CHECK_CUDA(cudaMemsetAsync(status_of(list), 0, sizeof(host), s));
    LRM_CHECK_CUDA(cudaStreamSynchronize(s));
  }
  *flags = host;
  return LRM_OK;
}

extern "C" lrm_status lrm_grad_norm(lrm_ctx* ctx, const lrm_grad_list* list, lrm_grad_stats* stats, void* stream) {
  if (ctx == nullptr || list == nullptr || stats == nullptr || list->device != ctx->device) return LRM_ERR_INVALID_ARG;
  if (!aligned(stats, 4)) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (list->by == GC_BY_SMALL) return launch_small(list, 0, 0.f, stats, s);
  if (list->by == GC_BY_HOLD) return launch_hold(ctx, list, 0, 0.f, stats, s);
  const lrm_status st = launch_norm(list, nullptr, s);
  if (st != LRM_OK) return st;
  return launch_dependent(gc_stats, 1, GC_THREADS, 0, 1, s, static_cast<const double*>(list->table), list->grid_norm,
                          stats);
}

extern "C" lrm_status lrm_grad_clip(lrm_ctx* ctx, const lrm_grad_list* list, float max_norm, lrm_grad_stats* stats,
                                    void* stream) {
  if (ctx == nullptr || list == nullptr || stats == nullptr || list->device != ctx->device || !list->has_dst ||
      !(max_norm >= 0.f))
    return LRM_ERR_INVALID_ARG;
  if (!aligned(stats, 4)) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (list->by == GC_BY_SMALL) return launch_small(list, 1, max_norm, stats, s);
  if (list->by == GC_BY_HOLD) return launch_hold(ctx, list, 1, max_norm, stats, s);
  const lrm_status st = launch_norm(list, list->by == GC_BY_RING ? stats : nullptr, s);
  if (st != LRM_OK) return st;
  const Chunk* chunks = chunks_of(list);
  const double* partial = static_cast<const double*>(list->table);
  if (list->by == GC_BY_RING)
    return launch_dependent(gc_ring, list->grid_clip, GC_RING_THREADS, GC_RING_SMEM, 1, s, chunks, list->chunks, partial,
                            list->grid_norm, max_norm, list->in_place, stats, ctx->wait_budget_ns, ctx->d_status,
                            status_of(list));
  return launch_dependent(gc_clip, list->grid_clip, GC_THREADS, 0, 1, s, chunks, list->chunks, partial,
                          list->grid_norm, max_norm, list->in_place, stats);
}
