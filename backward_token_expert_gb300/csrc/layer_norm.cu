// Layer norm of the rows of a [rows, width] tensor, forward and backward
// (Ba, Kiros and Hinton, 2016): with mean and variance of a row,
//   y  = (x - mean) rstd gamma + beta,   rstd = 1 / sqrt(var + eps)
//   d  = dy gamma,  xhat = (x - mean) rstd
//   dx = rstd (d - mean(d) - xhat mean(d xhat)) [+ dres]
//   dgamma = sum over rows of dy xhat,   dbeta = sum over rows of dy
// Both read every value once and write every result once, so memory bounds
// them.  All sums are fp32, the variance is that of the centred values, and each
// output is rounded once.
//
// A thread has the same columns in every row it takes part in, so gamma, beta
// and, in the backward, the sums of the weights' gradients stay in its registers
// while the rows stream through, with the next row's loads in flight while one is
// reduced.  Narrow rows share a warp.  Arithmetic is on pairs (packed fp32
// instructions).  Rows that do not start at a
// 16-byte boundary (a width that is no multiple of the vector, or a tensor that
// starts between two) are read and written in the aligned vectors that cover
// them, and a block takes only rows that start at the same place of a vector
// (every N-th row at most).  A vector that is shared with the neighbouring row is
// masked where it is used and stored element by element.
#include <type_traits>

#include "f32x2.cuh"
#include "lrm_internal.cuh"
#include "swiglu.cuh"
#include "vec.cuh"

namespace lrm {
namespace {

constexpr int MAX_WIDTH = 16384;
// Columns of a thread that holds its columns' weights, and the registers that needs: 64 bytes of a row forward, 32
// backward, where the sums take their place.
template <typename T>
constexpr int FWD_COLS = sizeof(T) == 2 ? 32 : 16;
template <typename T>
constexpr int FWD_REGS = sizeof(T) == 2 ? 128 : 96;
template <typename T>
constexpr int BWD_COLS = sizeof(T) == 2 ? 16 : 8;
template <typename T>
constexpr int BWD_REGS = sizeof(T) == 2 ? 128 : 112;
// threads that fit an SM beside one another
constexpr int threads_per_sm(int regs) { return 65536 / regs / 128 * 128; }

// a 16-byte vector of a type as pairs of fp32 values
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static __forceinline__ void unpack(const uint4& w, F2 (&f)[2]) {
    f[0] = F2(__uint_as_float(w.x), __uint_as_float(w.y));
    f[1] = F2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  __device__ static __forceinline__ uint4 pack(const F2 (&f)[2]) {
    const float2 a = f[0].get(), b = f[1].get();
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
  __device__ static __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
};
template <>
struct Vec<uint16_t> {  // bf16 bits
  static constexpr int N = 8;
  __device__ static __forceinline__ void unpack(const uint4& w, F2 (&f)[4]) {
    f[0] = F2(bf16_lo(w.x), bf16_hi(w.x));
    f[1] = F2(bf16_lo(w.y), bf16_hi(w.y));
    f[2] = F2(bf16_lo(w.z), bf16_hi(w.z));
    f[3] = F2(bf16_lo(w.w), bf16_hi(w.w));
  }
  __device__ static __forceinline__ uint4 pack(const F2 (&f)[4]) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = f[i].get();
      r[i] = pack_bf16x2(a.x, a.y);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};

constexpr int MAX_WARPS = 16;

// Sums over a row's threads: `lanes` of a warp by shuffles, then, where a row has several warps, the warps' sums
// through shared memory in a fixed order.  `slot` alternates between calls, so that one barrier a call is enough.
template <int K>
__device__ __forceinline__ void row_sum(float (&s)[K], int lanes, float (*buf)[K][MAX_WARPS], int& slot) {
  for (int o = min(lanes, 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (lanes <= 32) return;
  const int warp = threadIdx.x >> 5, warps = lanes >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < K; ++i) buf[slot][i][warp] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < K; ++i) {
    s[i] = 0.0f;
    for (int w = 0; w < warps; w += 4) {  // zeros beyond the row's warps
      const float4 f = *reinterpret_cast<const float4*>(&buf[slot][i][w]);
      s[i] += (f.x + f.y) + (f.z + f.w);
    }
  }
  slot ^= 1;
}

// place of column c among the skewed weights in shared memory: a warp's lanes read columns 8 (or 4) apart, which
// the skew spreads over all banks
__device__ __forceinline__ int skew(int c, int n) { return c + c / n; }

// The rows of a block and a thread's columns, which are the same in all of them: rows of class blockIdx.x % classes
// (rows `classes` apart start at one place of a vector).  `lanes` threads have a row: a power of two up to a warp (the
// block then has several rows at a time) or the whole block.
template <typename T, int NV, bool ALIGNED>
struct Block {
  static constexpr int N = Vec<T>::N;
  int lanes, lane, groups, group, cls, classes, lead, count, width;
  long long step, rows;

  __device__ __forceinline__ Block(int rows_, int width_, int shift, int classes_, int lanes_)
      : lanes(lanes_), lane(threadIdx.x % lanes_), groups(blockDim.x / lanes_), group(threadIdx.x / lanes_),
        cls(blockIdx.x % classes_), classes(classes_), width(width_),
        step(static_cast<long long>(gridDim.x / classes_) * groups * classes_), rows(rows_) {
    // elements before the row in its first vector; vectors that cover a row
    lead = ALIGNED ? 0 : static_cast<int>((static_cast<long long>(cls) * width + shift) % N);
    count = (lead + width + N - 1) / N;
  }
  // a vector with elements that are not the row's own: its first or last at most
  __device__ __forceinline__ bool edge(int i) const {
    return !ALIGNED && ((vector(i) == 0 && lead > 0) || (vector(i) == count - 1 && lead + width < count * N));
  }
  __device__ __forceinline__ long long first() const {
    return (static_cast<long long>(blockIdx.x / classes) * groups + group) * classes + cls;
  }
  // the block goes on while its first row is there: all its threads take part in the sums of every pass
  __device__ __forceinline__ long long first_of_block() const {
    return static_cast<long long>(blockIdx.x / classes) * groups * classes + cls;
  }
  __device__ __forceinline__ int vector(int i) const { return lane + i * lanes; }
  __device__ __forceinline__ int column(int i) const { return vector(i) * N - lead; }
  // Vector i of a row as it lies in memory: its elements outside the row are a neighbour's, which clean() removes where
  // the values are used (masking here would wait for them).
  __device__ __forceinline__ uint4 load(const T* base, long long row, int i) const {
    if (vector(i) >= count) return make_uint4(0u, 0u, 0u, 0u);
    const long long e0 = row * width + column(i);
    if (ALIGNED || (e0 >= 0 && e0 + N <= rows * width)) return ld_stream(reinterpret_cast<const uint4*>(base + e0));
    uint32_t w[4] = {0u, 0u, 0u, 0u};  // reaches beyond the tensor
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (column(i) + j >= 0 && column(i) + j < width) {
        if constexpr (N == 4)
          w[j] = __float_as_uint(base[e0 + j]);
        else
          w[j / 2] |= static_cast<uint32_t>(base[e0 + j]) << (16 * (j % 2));
      }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 clean(const uint4& r, int i) const {
    if (!edge(i)) return r;
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      constexpr int PER = N / 4;  // elements of a 32-bit word
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int c = column(i) + k * PER + j;
        if (c < 0 || c >= width) w[k] &= PER == 1 ? 0u : (j == 0 ? 0xFFFF0000u : 0x0000FFFFu);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(T* base, long long row, int i, const F2 (&f)[N / 2]) const {
    if (vector(i) >= count) return;
    T* at = base + row * width + column(i);
    const uint4 r = Vec<T>::pack(f);
    if (!edge(i)) {
      *reinterpret_cast<uint4*>(at) = r;
      return;
    }
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (column(i) + j >= 0 && column(i) + j < width) {
        if constexpr (N == 4)
          at[j] = __uint_as_float(w[j]);
        else
          at[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
      }
  }
  // the pair's weights, 0 outside the row
  __device__ __forceinline__ F2 weights(const float* p, int i, int pair) const {
    const int c = column(i) + 2 * pair;
    return F2(c >= 0 && c < width ? __ldg(p + c) : 0.0f, c + 1 >= 0 && c + 1 < width ? __ldg(p + c + 1) : 0.0f);
  }
  __device__ __forceinline__ F2 skewed(const float* p, int i, int pair) const {
    const int c = column(i) + 2 * pair;
    return F2(p[skew(min(max(c, 0), width - 1), N)], p[skew(min(max(c + 1, 0), width - 1), N)]);
  }
};

constexpr uint64_t DRAIN_NS = 2000000000ull;

// The rows of a block of more than one warp, copied ahead into shared memory: slot n % depth holds row
// first + n step, A arrays one after the other, as the aligned vectors that cover the row.
template <typename T, int A>
struct Ring {
  uint8_t* slots;
  uint64_t* bars;
  int depth, stride;  // rows; bytes of an array's row
  const T* src[A];
  const uint8_t* valid;
  unsigned int* status;
  unsigned long long budget_ns;

  __device__ __forceinline__ const uint4* slot(int n, int array) const {
    return reinterpret_cast<const uint4*>(slots + ((n % depth) * A + array) * stride);
  }
  // One thread: copies row `row` into slot n % depth, unless it is padding.  Vectors that reach beyond the tensor are
  // left to their readers.
  template <int NV, bool ALIGNED>
  __device__ __forceinline__ void issue(const Block<T, NV, ALIGNED>& b, int n, long long row, bool wanted) const {
    uint64_t* bar = bars + n % depth;
    const long long e0 = row * b.width - b.lead;
    const int v0 = !ALIGNED && e0 < 0 ? 1 : 0;
    const int v1 = b.count - (!ALIGNED && e0 + static_cast<long long>(b.count) * b.N > b.rows * b.width ? 1 : 0);
    const uint32_t bytes = v1 > v0 ? (v1 - v0) * 16 : 0;
    if (!wanted || bytes == 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, A * bytes);
#pragma unroll
    for (int a = 0; a < A; ++a)
      bulk_load(slots + ((n % depth) * A + a) * stride + v0 * 16, src[a] + e0 + v0 * b.N, bytes, bar);
  }
  // Row n has arrived.  A wait that runs out is flagged and goes on up to a limit of its own, so that no copy is left
  // on its way into the memory of a block that is gone.
  __device__ __forceinline__ void wait(int n) const {
    if (mbar_wait(bars + n % depth, (n / depth) & 1, budget_ns, nullptr)) return;
    raise_flag(status, LRM_ERR_TIMEOUT);
    mbar_wait(bars + n % depth, (n / depth) & 1, DRAIN_NS, nullptr);
  }
  template <int NV, bool ALIGNED>
  __device__ __forceinline__ uint4 read(const Block<T, NV, ALIGNED>& b, int n, int array, long long row, int i) const {
    if (b.vector(i) >= b.count) return make_uint4(0u, 0u, 0u, 0u);
    if (!ALIGNED && b.edge(i)) {
      const long long e0 = row * b.width + b.column(i);
      if (e0 < 0 || e0 + b.N > b.rows * b.width) return b.load(src[array], row, i);
    }
    return slot(n, array)[b.vector(i)];
  }
};
constexpr int MAX_DEPTH = 8;

__device__ __forceinline__ void clear_sums(float* buf, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) buf[i] = 0.0f;
}

// HOLD (64 bytes of a row's columns a thread): gamma and beta in registers, the next row's values loaded ahead; else
// (wider rows than that gives) gamma and beta in shared memory, skewed.  (32768 bf16 rows of 2048 values: 51 us, and 62
// with 32 bytes a thread, 92 with 16; one warp a row with gamma and beta in shared memory takes 58, rows through a ring
// of bulk copies 61.)
template <typename T, int NV, bool HOLD, bool ALIGNED>
__global__ void __maxnreg__(HOLD ? FWD_REGS<T> : 128)
    layer_norm_kernel(const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
                      const uint8_t* __restrict__ valid, int rows, int width, int shift, int classes, float eps,
                      int lanes, T* __restrict__ y, float* __restrict__ stats) {
  constexpr int N = Vec<T>::N, P = N / 2;
  extern __shared__ float s_dyn[];  // !HOLD: gamma and beta, skewed
  __shared__ __align__(16) float s_buf[2][1][MAX_WARPS];
  clear_sums(&s_buf[0][0][0], 2 * MAX_WARPS);
  grid_dependency_wait();
  const Block<T, NV, ALIGNED> b(rows, width, shift, classes, lanes);
  const int per = skew(width, N) + 1;
  if (!HOLD)
    for (int c = threadIdx.x; c < width; c += blockDim.x) {
      s_dyn[skew(c, N)] = __ldg(gamma + c);
      s_dyn[per + skew(c, N)] = __ldg(beta + c);
    }
  __syncthreads();
  F2 ga[HOLD ? NV : 1][P], be[HOLD ? NV : 1][P];
  if constexpr (HOLD)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < P; ++j) ga[i][j] = b.weights(gamma, i, j), be[i][j] = b.weights(beta, i, j);
  const float inv = 1.0f / static_cast<float>(width);
  int slot = 0;
  uint4 raw[NV];
  bool on = false;  // the row whose values are in raw is there and no padding
  auto fetch = [&](long long row) {
    on = row < rows && (valid == nullptr || valid[row] != 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = on ? b.load(x, row, i) : make_uint4(0u, 0u, 0u, 0u);
  };
  long long row = b.first();
  fetch(row);
  for (long long q = b.first_of_block(); q < rows; q += b.step, row += b.step) {
    F2 f[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<T>::unpack(b.clean(raw[i], i), f[i]);
    const bool counted = on;
    if (HOLD) fetch(row + b.step);
    F2 acc(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < P; ++j) acc = add2(acc, f[i][j]);  // zeros outside the row
    float s[1] = {acc.get().x + acc.get().y};
    row_sum(s, lanes, s_buf, slot);
    const float mean = s[0] * inv;
    const F2 minus(-mean, -mean);
    acc = F2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < P; ++j) f[i][j] = add2(f[i][j], minus);
      if (b.vector(i) >= b.count || b.edge(i)) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const int c = b.column(i) + 2 * j;
          const float2 v = f[i][j].get();
          f[i][j] = F2(c >= 0 && c < width ? v.x : 0.0f, c + 1 >= 0 && c + 1 < width ? v.y : 0.0f);
        }
      }
#pragma unroll
      for (int j = 0; j < P; ++j) acc = fma2(f[i][j], f[i][j], acc);
    }
    s[0] = acc.get().x + acc.get().y;
    row_sum(s, lanes, s_buf, slot);
    const float rstd = 1.0f / sqrtf(s[0] * inv + eps);
    if (row < rows) {
      const F2 scale(rstd, rstd);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if constexpr (HOLD)
            f[i][j] = fma2(mul2(f[i][j], scale), ga[i][j], be[i][j]);
          else
            f[i][j] = fma2(mul2(f[i][j], scale), b.skewed(s_dyn, i, j), b.skewed(s_dyn + per, i, j));
          if (!counted) f[i][j] = F2(0.0f, 0.0f);
        }
        b.store(y, row, i, f[i]);
      }
      if (b.lane == 0) *reinterpret_cast<float2*>(stats + row * 2) = counted ? make_float2(mean, rstd) : make_float2(0.0f, 0.0f);
    }
    if (!HOLD) fetch(row + b.step);
  }
}

// How a row's values reach a thread of the backward, which holds 32 bytes of a row's columns: HOLD, loaded a row ahead
// into registers; RING (fp32, where that takes too many), through shared memory; WIDE, more columns than registers
// have room for the sums beside gamma, which lies in shared memory then, skewed.
enum Mode { HELD, RING, WIDE };

struct RingArgs {
  int depth;
  unsigned int* status;
  unsigned long long budget_ns;
};

// Backward.  Blocks leave their sums of the weights' gradients in partial [blocks, 2, width], which weight_sum_kernel
// adds in a fixed order; where a block has several rows at a time, they are added through shared memory first.
// Modes as above; WIDE: gamma lies in shared memory and the second pass over a row reads it again, out of the L2.
template <typename T, int NV, Mode MODE, bool ALIGNED, bool RES>
__global__ void __maxnreg__(MODE != WIDE ? BWD_REGS<T> : 128)
    layer_norm_bwd_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ gamma,
                          const float* __restrict__ stats, const uint8_t* __restrict__ valid,
                          const T* __restrict__ dres, int rows, int width, int shift, int classes, int lanes,
                          const RingArgs args, T* __restrict__ dx, float* __restrict__ partial) {
  constexpr int N = Vec<T>::N, P = N / 2;
  constexpr bool HOLD = MODE != WIDE;
  // HELD, several rows at a time: [groups][2][width]; RING: the rows; WIDE: gamma, skewed
  extern __shared__ __align__(16) float s_dyn[];
  __shared__ __align__(16) float s_buf[2][2][MAX_WARPS];
  __shared__ __align__(8) uint64_t s_bars[MAX_DEPTH];
  clear_sums(&s_buf[0][0][0], 4 * MAX_WARPS);
  grid_dependency_wait();
  const Block<T, NV, ALIGNED> b(rows, width, shift, classes, lanes);
  const float inv = 1.0f / static_cast<float>(width);
  F2 dg[NV][P], db[NV][P], ga[HOLD ? NV : 1][P];
  if (!HOLD)
    for (int c = threadIdx.x; c < width; c += blockDim.x) s_dyn[skew(c, N)] = __ldg(gamma + c);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if constexpr (HOLD) ga[i][j] = b.weights(gamma, i, j);
      dg[i][j] = db[i][j] = F2(0.0f, 0.0f);
    }
  auto weight = [&](int i, int j) {
    if constexpr (HOLD)
      return ga[i][j];
    else
      return b.skewed(s_dyn, i, j);
  };
  int slot = 0;
  constexpr int HV = HOLD ? NV : 1;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 nx[HV], ny[HV], nr[HV];  // HELD: the next row's
  float mean = 0.0f, rstd = 0.0f;
  bool on = false;
  auto counts = [&](long long r) { return r < rows && (valid == nullptr || valid[r] != 0); };
  auto fetch = [&](long long r) {
    on = counts(r);
    mean = rstd = 0.0f;
    if (on) {
      mean = __ldg(stats + r * 2);
      rstd = __ldg(stats + r * 2 + 1);
    }
    if constexpr (MODE == HELD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        nx[i] = on ? b.load(x, r, i) : none;
        ny[i] = on ? b.load(dy, r, i) : none;
        if (RES) nr[i] = on ? b.load(dres, r, i) : none;
      }
    }
  };
  Ring<T, RES ? 3 : 2> ring{reinterpret_cast<uint8_t*>(s_dyn), s_bars, args.depth, b.count * 16, {x, dy}, valid,
                            args.status, args.budget_ns};
  if constexpr (RES) ring.src[2] = dres;
  long long row = b.first();
  bool ahead = false;  // RING, the first thread: whether the row after those on their way counts
  if constexpr (MODE == RING) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < args.depth; ++i) mbar_init(s_bars + i, 1);
      fence_mbar_init();
      for (int i = 0; i < args.depth; ++i)
        if (row + i * b.step < rows) ring.issue(b, i, row + i * b.step, counts(row + i * b.step));
      ahead = counts(row + args.depth * b.step);
    }
    __syncthreads();
  }
  fetch(row);
  int n = 0;
  for (long long q = b.first_of_block(); q < rows; q += b.step, row += b.step, ++n) {
    const bool counted = on;
    const F2 minus(-mean, -mean), scale(rstd, rstd);
    uint4 xr[HV], yr[HV], rr[HV];
    if constexpr (MODE == RING) {
      ring.wait(n);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xr[i] = counted ? ring.read(b, n, 0, row, i) : none;
        yr[i] = counted ? ring.read(b, n, 1, row, i) : none;
        rr[i] = RES && counted ? ring.read(b, n, RES ? 2 : 0, row, i) : none;
      }
    } else if constexpr (HOLD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) xr[i] = nx[i], yr[i] = ny[i], rr[i] = RES ? nr[i] : none;
    }
    if constexpr (HOLD) fetch(row + b.step);
    // xhat and dy of vector i, twice out of the same 16 bytes: fp32 copies would take twice the registers in bf16
    auto values = [&](int i, F2 (&vx)[P], F2 (&vy)[P]) {
      const int k = HOLD ? i : 0;
      if constexpr (!HOLD) {
        xr[0] = counted ? b.load(x, row, i) : none;
        yr[0] = counted ? b.load(dy, row, i) : none;
      }
      Vec<T>::unpack(b.clean(xr[k], i), vx);
      Vec<T>::unpack(b.clean(yr[k], i), vy);
#pragma unroll
      for (int j = 0; j < P; ++j) vx[j] = mul2(add2(vx[j], minus), scale);
    };
    F2 s0(0.0f, 0.0f), s1(0.0f, 0.0f);
    // the elements of a vector that are not the row's own have dy = 0 and add nothing
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      F2 vx[P], vy[P];
      values(i, vx, vy);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const F2 d = mul2(vy[j], weight(i, j));
        s0 = add2(s0, d);
        s1 = fma2(d, vx[j], s1);
        dg[i][j] = fma2(vy[j], vx[j], dg[i][j]);
        db[i][j] = add2(db[i][j], vy[j]);
      }
    }
    float s[2] = {s0.get().x + s0.get().y, s1.get().x + s1.get().y};
    row_sum(s, lanes, s_buf, slot);
    if constexpr (MODE == RING) {  // all threads have read the row: its slot takes the next one
      if (threadIdx.x == 0 && row + args.depth * b.step < rows) {
        ring.issue(b, n + args.depth, row + args.depth * b.step, ahead);
        ahead = counts(row + (args.depth + 1) * b.step);
      }
    }
    if constexpr (HOLD && sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {  // unpacked anew below
        asm volatile("" : "+r"(xr[i].x), "+r"(xr[i].y), "+r"(xr[i].z), "+r"(xr[i].w));
        asm volatile("" : "+r"(yr[i].x), "+r"(yr[i].y), "+r"(yr[i].z), "+r"(yr[i].w));
      }
    }
    if (row < rows) {
      const F2 m0(-s[0] * inv, -s[0] * inv), m1(-s[1] * inv, -s[1] * inv);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        F2 vx[P], vy[P], vr[P];
        values(i, vx, vy);
        if constexpr (RES) {
          if constexpr (!HOLD) rr[0] = counted ? b.load(dres, row, i) : none;
          Vec<T>::unpack(rr[HOLD ? i : 0], vr);  // a neighbour's values go no further than the store
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const F2 g = fma2(vx[j], m1, fma2(vy[j], weight(i, j), m0));
          if constexpr (RES)
            vx[j] = fma2(g, scale, vr[j]);
          else
            vx[j] = mul2(g, scale);
          if (!counted) vx[j] = F2(0.0f, 0.0f);
        }
        b.store(dx, row, i, vx);
      }
    }
    if (!HOLD) fetch(row + b.step);
  }
  float* out = b.groups > 1 ? s_dyn + b.group * 2 * width : partial + static_cast<size_t>(blockIdx.x) * 2 * width;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int c = b.column(i) + 2 * j;
      const float2 g = dg[i][j].get(), e = db[i][j].get();
      if (c >= 0 && c < width) {
        out[c] = g.x;
        out[width + c] = e.x;
      }
      if (c + 1 >= 0 && c + 1 < width) {
        out[c + 1] = g.y;
        out[width + c + 1] = e.y;
      }
    }
  if (b.groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) {
      float sum = 0.0f;
      for (int g = 0; g < b.groups; ++g) sum += s_dyn[g * 2 * width + c];
      partial[static_cast<size_t>(blockIdx.x) * 2 * width + c] = sum;
    }
  }
}

constexpr int WS_ROWS = 32;  // threads that share a column's blocks

// column c of [dgamma | dbeta] = the sum of the blocks' partial sums
__global__ void __launch_bounds__(32 * WS_ROWS)
    weight_sum_kernel(const float* __restrict__ partial, int blocks, int width, float* __restrict__ dgamma,
                      float* __restrict__ dbeta) {
  __shared__ float s[WS_ROWS][33];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (c < 2 * width)
    for (int b = part; b < blocks; b += WS_ROWS) sum += __ldg(partial + static_cast<size_t>(b) * 2 * width + c);
  s[part][lane] = sum;
  __syncthreads();
  sum = s[lane][part];  // thread (part, lane): partial sum `lane` of column `part` of the block
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int col = blockIdx.x * 32 + part;
  if (lane == 0 && col < 2 * width) (col < width ? dgamma[col] : dbeta[col - width]) = sum;
}

int ceil_div(long long a, int b) { return static_cast<int>((a + b - 1) / b); }

// Vectors of a row at most.
template <typename T>
int row_vectors(int width, bool aligned_rows) {
  constexpr int N = Vec<T>::N;
  return aligned_rows ? width / N : (width + 2 * (N - 1)) / N;
}

template <typename T>
bool aligned_rows(const void* a, const void* b, const void* c, const void* d, int width) {
  return width % Vec<T>::N == 0 && aligned(a, 16) && aligned(b, 16) && aligned(c, 16) && aligned(d, 16);
}

// elements between the 16-byte boundary before p and p
template <typename T>
int shift_of(const void* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) % 16) / sizeof(T));
}

// How a call cuts its work; the same for the backward's launch and its workspace's size.
struct Plan {
  int lanes, nv, threads, classes, blocks, per_sm;
};

// `most`: vectors a thread at most, `resident`: threads an SM has room for
template <typename T>
Plan plan(int sm_count, int rows, int width, bool al, int most, int resident) {
  Plan p;
  const int nvec = row_vectors<T>(width, al);
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes * most < nvec) p.lanes *= 2;
  while (p.lanes >= 32 && p.lanes < 32 * MAX_WARPS && p.lanes * most < nvec) p.lanes += 32;
  p.nv = ceil_div(nvec, p.lanes);
  p.threads = p.lanes > 32 ? p.lanes : 128;
  p.classes = 1;
  if (!al) {
    p.classes = Vec<T>::N;
    for (int w = width; p.classes > 1 && w % 2 == 0; w /= 2) p.classes /= 2;
  }
  const int groups = p.threads / p.lanes;
  const int per_class = ceil_div(ceil_div(rows, p.classes), groups);
  p.per_sm = resident / p.threads;
  if (p.per_sm < 1) p.per_sm = 1;
  int blocks = sm_count * p.per_sm / p.classes;
  if (blocks < 1) blocks = 1;
  p.blocks = p.classes * (per_class < blocks ? (per_class > 0 ? per_class : 1) : blocks);
  return p;
}
template <typename T>
Plan bwd_plan(int sm_count, int rows, int width, bool al) {
  return plan<T>(sm_count, rows, width, al, BWD_COLS<T> / Vec<T>::N, threads_per_sm(BWD_REGS<T>));
}

// Rows of a ring: as many as the blocks of an SM have room for beside one another.
int ring_depth(const Plan& p, int arrays, int width, int type_size) {
  const int row = arrays * (width * type_size + 32);  // with the vectors it shares
  const int depth = 200 * 1024 / p.per_sm / row;
  return depth < 2 ? 2 : depth > MAX_DEPTH ? MAX_DEPTH : depth;
}

// Calls go(vectors a thread, mode): WIDE up to 5 vectors in bf16 and 9 in fp32 at the largest width, one more than it
// fills where rows are cut.
template <typename T, typename Go>
lrm_status with_vectors(const Plan& p, Go go) {
  constexpr int HOLDS = BWD_COLS<T> / Vec<T>::N;
  using Wide = std::integral_constant<Mode, WIDE>;
  if (p.nv <= HOLDS) {
    if constexpr (sizeof(T) == 4)
      if (p.lanes > 32) return go(std::integral_constant<int, HOLDS>(), std::integral_constant<Mode, RING>());
    return go(std::integral_constant<int, HOLDS>(), std::integral_constant<Mode, HELD>());
  }
  if (p.nv <= 3) return go(std::integral_constant<int, 3>(), Wide());
  if constexpr (Vec<T>::N == 4)
    if (p.nv > 5) return go(std::integral_constant<int, 9>(), Wide());
  return go(std::integral_constant<int, 5>(), Wide());
}

template <typename Kern>
lrm_status allow_smem(Kern kern, size_t smem) {
  if (smem > 40 * 1024)
    LRM_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
  return LRM_OK;
}

template <typename T, bool ALIGNED>
lrm_status forward(lrm_ctx* ctx, const void* x, const float* gamma, const float* beta, const uint8_t* valid, int rows,
                   int width, float eps, void* y, float* stats, cudaStream_t s) {
  constexpr int HOLDS = FWD_COLS<T> / Vec<T>::N;
  const Plan p = plan<T>(ctx->sm_count, rows, width, ALIGNED, HOLDS, threads_per_sm(FWD_REGS<T>));
  auto go = [&](auto n, auto hold) {
    auto kern = layer_norm_kernel<T, decltype(n)::value, decltype(hold)::value, ALIGNED>;
    const size_t smem = decltype(hold)::value ? 0 : 2 * (width + width / Vec<T>::N + 1) * sizeof(float);
    const lrm_status st = allow_smem(kern, smem);
    if (st != LRM_OK) return st;
    return launch_dependent(kern, p.blocks, p.threads, smem, 0, s, static_cast<const T*>(x), gamma, beta, valid, rows,
                            width, shift_of<T>(x), p.classes, eps, p.lanes, static_cast<T*>(y), stats);
  };
  if (p.nv <= HOLDS) return go(std::integral_constant<int, HOLDS>(), std::true_type());
  // fp32 above 8192 columns, bf16 where the widest rows are cut
  if constexpr (Vec<T>::N == 4)
    if (p.nv > 5) return go(std::integral_constant<int, 9>(), std::false_type());
  return go(std::integral_constant<int, 5>(), std::false_type());
}

template <typename T, bool ALIGNED, bool RES>
lrm_status backward(lrm_ctx* ctx, const void* x, const void* dy, const float* gamma, const float* stats,
                    const uint8_t* valid, const void* dres, int rows, int width, void* dx, float* dgamma,
                    float* dbeta, float* partial, cudaStream_t s) {
  const Plan p = bwd_plan<T>(ctx->sm_count, rows, width, ALIGNED);
  const int groups = p.threads / p.lanes;
  const lrm_status st = with_vectors<T>(p, [&](auto n, auto mode) {
    constexpr Mode MODE = decltype(mode)::value;
    auto kern = layer_norm_bwd_kernel<T, decltype(n)::value, MODE, ALIGNED, RES>;
    constexpr int ARRAYS = RES ? 3 : 2;
    const RingArgs ring{ring_depth(p, ARRAYS, width, sizeof(T)), ctx->d_status, ctx->wait_budget_ns};
    const size_t smem = MODE == WIDE   ? (width + width / Vec<T>::N + 1) * sizeof(float)
                        : MODE == RING ? static_cast<size_t>(ring.depth) * ARRAYS * row_vectors<T>(width, ALIGNED) * 16
                        : groups > 1   ? static_cast<size_t>(groups) * 2 * width * sizeof(float)
                                       : 0;
    const lrm_status a = allow_smem(kern, smem);
    if (a != LRM_OK) return a;
    return launch_dependent(kern, p.blocks, p.threads, smem, 0, s, static_cast<const T*>(x),
                            static_cast<const T*>(dy), gamma, stats, valid, static_cast<const T*>(dres), rows, width,
                            shift_of<T>(x), p.classes, p.lanes, ring, static_cast<T*>(dx), partial);
  });
  if (st != LRM_OK) return st;
  return launch_dependent(weight_sum_kernel, ceil_div(2ll * width, 32), 32 * WS_ROWS, 0, 0, s, partial, p.blocks,
                          width, dgamma, dbeta);
}

size_t bwd_bytes(int sm_count, int rows, int width) {
  // whatever the type and the alignment of the tensors
  int blocks = 0;
  for (int al = 0; al < 2; ++al) {
    const int a = bwd_plan<float>(sm_count, rows, width, al != 0 && width % 4 == 0).blocks;
    const int b = bwd_plan<uint16_t>(sm_count, rows, width, al != 0 && width % 8 == 0).blocks;
    blocks = a > blocks ? a : blocks;
    blocks = b > blocks ? b : blocks;
  }
  return static_cast<size_t>(blocks) * 2 * width * sizeof(float);
}

lrm_status check_norm(const lrm_ctx* ctx, int dtype, int rows, int width) {
  if (ctx == nullptr || rows < 0 || width < 1) return LRM_ERR_INVALID_ARG;
  if (dtype != LRM_F32 && dtype != LRM_BF16) return LRM_ERR_INVALID_ARG;
  return width > MAX_WIDTH ? LRM_ERR_SHAPE : LRM_OK;
}

}  // namespace
}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_layer_norm(lrm_ctx* ctx, const void* x, int32_t dtype, const float* gamma,
                                     const float* beta, const uint8_t* valid, int32_t rows, int32_t width, float eps,
                                     void* y, float* stats, void* stream) {
  const lrm_status st = check_norm(ctx, dtype, rows, width);
  if (st != LRM_OK) return st;
  if (!(eps >= 0.0f)) return LRM_ERR_INVALID_ARG;
  if (rows == 0) return LRM_OK;
  if (x == nullptr || gamma == nullptr || beta == nullptr || y == nullptr || stats == nullptr)
    return LRM_ERR_INVALID_ARG;
  const size_t es = dtype == LRM_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(stats, 8))
    return LRM_ERR_ALIGN;
  // the vectors of a row cut x and y alike
  if (reinterpret_cast<uintptr_t>(x) % 16 != reinterpret_cast<uintptr_t>(y) % 16) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == LRM_F32)
    return aligned_rows<float>(x, y, nullptr, nullptr, width)
               ? forward<float, true>(ctx, x, gamma, beta, valid, rows, width, eps, y, stats, s)
               : forward<float, false>(ctx, x, gamma, beta, valid, rows, width, eps, y, stats, s);
  return aligned_rows<uint16_t>(x, y, nullptr, nullptr, width)
             ? forward<uint16_t, true>(ctx, x, gamma, beta, valid, rows, width, eps, y, stats, s)
             : forward<uint16_t, false>(ctx, x, gamma, beta, valid, rows, width, eps, y, stats, s);
}

extern "C" lrm_status lrm_layer_norm_workspace(const lrm_ctx* ctx, int32_t rows, int32_t width, size_t* bytes) {
  const lrm_status st = check_norm(ctx, LRM_F32, rows, width);
  if (st != LRM_OK) return st;
  if (bytes == nullptr) return LRM_ERR_INVALID_ARG;
  *bytes = bwd_bytes(ctx->sm_count, rows, width);
  return LRM_OK;
}

extern "C" lrm_status lrm_layer_norm_backward(lrm_ctx* ctx, const void* x, int32_t dtype, const void* dy,
                                              const float* gamma, const float* stats, const uint8_t* valid,
                                              const void* dres, int32_t rows, int32_t width, void* dx, float* dgamma,
                                              float* dbeta, void* ws, size_t ws_bytes, void* stream) {
  const lrm_status st = check_norm(ctx, dtype, rows, width);
  if (st != LRM_OK) return st;
  if (dgamma == nullptr || dbeta == nullptr) return LRM_ERR_INVALID_ARG;
  if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return LRM_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows > 0) {
    if (x == nullptr || dy == nullptr || gamma == nullptr || stats == nullptr || dx == nullptr)
      return LRM_ERR_INVALID_ARG;
    if (ws == nullptr || ws_bytes < bwd_bytes(ctx->sm_count, rows, width)) return LRM_ERR_WORKSPACE;
    const size_t es = dtype == LRM_F32 ? 4 : 2;
    if (!aligned(x, es) || !aligned(gamma, 4) || !aligned(stats, 8) || !aligned(ws, 4)) return LRM_ERR_ALIGN;
    const uintptr_t at = reinterpret_cast<uintptr_t>(x) % 16;
    if (reinterpret_cast<uintptr_t>(dy) % 16 != at || reinterpret_cast<uintptr_t>(dx) % 16 != at ||
        (dres != nullptr && reinterpret_cast<uintptr_t>(dres) % 16 != at))
      return LRM_ERR_ALIGN;
  }
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  if (rows == 0) {
    LRM_CHECK_CUDA(cudaMemsetAsync(dgamma, 0, width * sizeof(float), s));
    LRM_CHECK_CUDA(cudaMemsetAsync(dbeta, 0, width * sizeof(float), s));
    return LRM_OK;
  }
  float* part = static_cast<float*>(ws);
  auto go = [&](auto type, auto al) {
    using T = decltype(type);
    constexpr bool ALIGNED = decltype(al)::value;
    return dres != nullptr ? backward<T, ALIGNED, true>(ctx, x, dy, gamma, stats, valid, dres, rows, width, dx,
                                                        dgamma, dbeta, part, s)
                           : backward<T, ALIGNED, false>(ctx, x, dy, gamma, stats, valid, dres, rows, width, dx,
                                                         dgamma, dbeta, part, s);
  };
  if (dtype == LRM_F32)
    return aligned_rows<float>(x, dy, dx, dres, width) ? go(float(), std::true_type()) : go(float(), std::false_type());
  return aligned_rows<uint16_t>(x, dy, dx, dres, width) ? go(uint16_t(), std::true_type())
                                                         : go(uint16_t(), std::false_type());
}
