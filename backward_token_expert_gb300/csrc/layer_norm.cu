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
// Columns of a thread that holds its columns' weights, and the registers that needs: 64 bytes of a row forward (48 of
// unaligned ones, whose edges take registers: 20011 bf16 rows of 1497 values took 38 us so, 56 with 64, 42 with 32), 32
// backward, where the sums take their place.
template <typename T, bool ALIGNED>
constexpr int FWD_COLS = (ALIGNED ? 64 : 48) / sizeof(T);
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
constexpr int MAX_GROUPS = 8;  // rows of more than one warp that a block has at a time

// Sums over a row's threads: `lanes` of a warp by shuffles, then, where a row has several warps, the warps' sums
// through shared memory in a fixed order.  `slot` alternates between calls, so that one barrier a call is enough, which
// is that of the row's threads alone.
template <int K>
__device__ __forceinline__ void row_sum(float (&s)[K], int lanes, int group, float (*buf)[K][MAX_WARPS], int& slot) {
  for (int o = min(lanes, 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (lanes <= 32) return;
  const int warp = (threadIdx.x >> 5) - group * (lanes >> 5), warps = lanes >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < K; ++i) buf[slot][i][warp] = s[i];
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
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
  uint32_t step, rows;  // rows and a few steps beyond them fit 32 bits
  uint4* edges;  // shared: the bits of the row's own elements in its first and its last vector
  using Bits = std::conditional_t<(NV * N > 32), uint64_t, uint32_t>;
  Bits own_bits = 0;  // !ALIGNED

  // The block's threads meet before the first clean().
  __device__ __forceinline__ Block(int rows_, int width_, int shift, int classes_, int lanes_, uint4* edges_)
      : lanes(lanes_), lane(threadIdx.x % lanes_), groups(blockDim.x / lanes_), group(threadIdx.x / lanes_),
        cls(blockIdx.x % classes_), classes(classes_), width(width_),
        step(gridDim.x / classes_ * groups * classes_), rows(rows_), edges(edges_) {
    // elements before the row in its first vector; vectors that cover a row
    lead = ALIGNED ? 0 : static_cast<int>((static_cast<long long>(cls) * width + shift) % N);
    count = (lead + width + N - 1) / N;
    if (ALIGNED) return;
    const uint32_t first = ~0u << lead, last = (1u << (lead + width - (count - 1) * N)) - 1u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t w = (1u << N) - 1u;
      if (vector(i) == 0) w &= first;
      if (vector(i) == count - 1) w &= last;
      if (vector(i) < count) own_bits |= static_cast<Bits>(w) << (i * N);
    }
    if (threadIdx.x < 2) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = 0u;
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
          if ((threadIdx.x == 0 ? first : last) >> (k * (N / 4) + j) & 1u) w[k] |= N == 4 ? ~0u : 0xFFFFu << (16 * j);
      }
      edges[threadIdx.x] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // bit j: element j of vector i is the row's own
  __device__ __forceinline__ uint32_t own(int i) const {
    return static_cast<uint32_t>(own_bits >> (i * N)) & ((1u << N) - 1u);
  }
  // a vector with elements that are not the row's own
  __device__ __forceinline__ bool edge(int i) const { return !ALIGNED && own(i) != (1u << N) - 1u; }
  __device__ __forceinline__ uint32_t first() const {
    return (blockIdx.x / classes * groups + group) * classes + cls;
  }
  // the block goes on while its first row is there: all its threads take part in the sums of every pass
  __device__ __forceinline__ uint32_t first_of_block() const {
    return blockIdx.x / classes * groups * classes + cls;
  }
  // element offset of a row's column, and of what lies behind the last row
  __device__ __forceinline__ long long at(uint32_t row, int c) const {
    return static_cast<long long>(static_cast<uint64_t>(row) * static_cast<uint32_t>(width)) + c;
  }
  __device__ __forceinline__ long long end() const { return at(rows, 0); }
  __device__ __forceinline__ int vector(int i) const { return lane + i * lanes; }
  __device__ __forceinline__ int column(int i) const { return vector(i) * N - lead; }
  // Vector i of a row as it lies in memory: its elements outside the row are a neighbour's, which clean() removes where
  // the values are used (masking here would wait for them).
  __device__ __forceinline__ uint4 load(const T* base, uint32_t row, int i) const {
    if (vector(i) >= count) return make_uint4(0u, 0u, 0u, 0u);
    const long long e0 = at(row, column(i));
    // of rows that fill a vector only the first and the last can reach beyond the tensor
    if (ALIGNED || (width >= N && row > 0 && row < rows - 1) || (e0 >= 0 && e0 + N <= end()))
      return ld_stream(reinterpret_cast<const uint4*>(base + e0));
    uint32_t w[4] = {0u, 0u, 0u, 0u};  // reaches beyond the tensor
#pragma unroll 1
    for (int j = 0; j < N; ++j) {  // element by element from the top, in few instructions: two vectors of a tensor come here
      const T* from = base + e0 + j;
      const bool mine = own(i) >> j & 1u;
      if constexpr (N == 4) {
        w[0] = w[1], w[1] = w[2], w[2] = w[3];
        w[3] = mine ? __float_as_uint(*from) : 0u;
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
        w[3] = w[3] >> 16 | (mine ? static_cast<uint32_t>(*from) : 0u) << 16;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 clean(uint4 r, int i) const {
    if (!edge(i)) return r;
    if (vector(i) == 0) r = both(r, edges[0]);
    if (vector(i) == count - 1) r = both(r, edges[1]);
    return r;
  }
  __device__ static __forceinline__ uint4 both(const uint4& a, const uint4& b) {
    return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
  }
  // zeros for the elements of vector i that are not the row's own
  __device__ __forceinline__ void zero_outside(F2 (&f)[N / 2], int i) const {
    if (ALIGNED && vector(i) >= count) {
#pragma unroll
      for (int j = 0; j < N / 2; ++j) f[j] = F2(0.0f, 0.0f);
    }
    if (edge(i)) {
      const uint32_t mine = own(i);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float2 v = f[j].get();
        f[j] = F2(mine >> (2 * j) & 1u ? v.x : 0.0f, mine >> (2 * j + 1) & 1u ? v.y : 0.0f);
      }
    }
  }
  // zeros for a row that does not count
  __device__ __forceinline__ void store(T* base, uint32_t row, int i, const F2 (&f)[N / 2], bool counted) const {
    if (vector(i) >= count) return;
    T* to = base + at(row, column(i));
    const uint32_t keep = counted ? ~0u : 0u;
    uint4 r = Vec<T>::pack(f);
    r = make_uint4(r.x & keep, r.y & keep, r.z & keep, r.w & keep);
    if (!edge(i)) {
      *reinterpret_cast<uint4*>(to) = r;
      return;
    }
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (own(i) >> j & 1u) {
        if constexpr (N == 4)
          to[j] = __uint_as_float(w[j]);
        else
          to[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
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
  unsigned int* status;
  unsigned long long budget_ns;

  __device__ __forceinline__ const uint4* slot(int n, int array) const {
    return reinterpret_cast<const uint4*>(slots + ((n % depth) * A + array) * stride);
  }
  // One thread: copies row `row` into slot n % depth, unless it is padding.  Vectors that reach beyond the tensor are
  // left to their readers.
  template <int NV, bool ALIGNED>
  __device__ __forceinline__ void issue(const Block<T, NV, ALIGNED>& b, int n, uint32_t row, bool wanted) const {
    uint64_t* bar = bars + n % depth;
    const long long e0 = b.at(row, -b.lead);
    const int v0 = !ALIGNED && e0 < 0 ? 1 : 0;
    const int v1 = b.count - (!ALIGNED && e0 + static_cast<long long>(b.count) * b.N > b.end() ? 1 : 0);
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
  __device__ __forceinline__ uint4 read(const Block<T, NV, ALIGNED>& b, int n, int array, uint32_t row, int i) const {
    if (b.vector(i) >= b.count) return make_uint4(0u, 0u, 0u, 0u);
    if (!ALIGNED && b.edge(i)) {
      const long long e0 = b.at(row, b.column(i));
      if (e0 < 0 || e0 + b.N > b.end()) return b.load(src[array], row, i);
    }
    return slot(n, array)[b.vector(i)];
  }
};
constexpr int MAX_DEPTH = 8;

__device__ __forceinline__ void clear_sums(float* buf, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) buf[i] = 0.0f;
}

// HOLD (64 bytes of a row's columns a thread): gamma and beta in registers, the next row's values loaded ahead; else
// (wider rows than that gives) gamma and beta in shared memory, skewed.  (32768 bf16 rows of 2048 values: 50 us, and 62
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
  __shared__ uint4 s_edges[2];
  const Block<T, NV, ALIGNED> b(rows, width, shift, classes, lanes, s_edges);
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
  auto fetch = [&](uint32_t row) {
    on = row < b.rows && (valid == nullptr || valid[row] != 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = on ? b.load(x, row, i) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint32_t row = b.first();
  fetch(row);
  for (uint32_t q = b.first_of_block(); q < b.rows; q += b.step, row += b.step) {
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
    row_sum(s, lanes, 0, s_buf, slot);
    const float mean = s[0] * inv;
    const F2 minus(-mean, -mean);
    acc = F2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < P; ++j) f[i][j] = add2(f[i][j], minus);
      b.zero_outside(f[i], i);
#pragma unroll
      for (int j = 0; j < P; ++j) acc = fma2(f[i][j], f[i][j], acc);
    }
    s[0] = acc.get().x + acc.get().y;
    row_sum(s, lanes, 0, s_buf, slot);
    const float rstd = 1.0f / sqrtf(s[0] * inv + eps);
    if (row < b.rows) {
      const F2 scale(rstd, rstd);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if constexpr (HOLD)
            f[i][j] = fma2(mul2(f[i][j], scale), ga[i][j], be[i][j]);
          else
            f[i][j] = fma2(mul2(f[i][j], scale), b.skewed(s_dyn, i, j), b.skewed(s_dyn + per, i, j));
        }
        b.store(y, row, i, f[i], counted);
      }
      if (b.lane == 0) reinterpret_cast<float2*>(stats)[row] = counted ? make_float2(mean, rstd) : make_float2(0.0f, 0.0f);
    }
    if (!HOLD) fetch(row + b.step);
  }
}

// How a row's values reach a thread of the backward, which holds 32 bytes of a row's columns: HELD, loaded a row ahead
// into registers; RING (fp32, where that takes too many), through shared memory; WIDE, more columns than registers
// have room for the sums beside gamma, which lies in shared memory then, skewed.
enum Mode { HELD, RING, WIDE };

struct RingArgs {
  int depth;
  unsigned int* status;
  unsigned long long budget_ns;
};

// Backward.  Instructions bound it in bf16 (32768 rows of 2048 values: 76 us, and 99 when the second pass unpacked the
// values anew instead of keeping xhat and d) and memory in fp32 (with a residual's gradient 160 us).  Blocks leave
// their sums of the weights' gradients in partial [blocks, 2, width], which weight_sum_kernel adds in a fixed order;
// where a block has several rows at a time, they are added through shared memory first.  Modes as above; WIDE: gamma
// lies in shared memory and the second pass over a row reads it again, out of the L2.
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
  __shared__ __align__(16) float s_buf[MAX_GROUPS][2][2][MAX_WARPS];
  __shared__ __align__(8) uint64_t s_bars[MAX_DEPTH];
  clear_sums(&s_buf[0][0][0][0], MAX_GROUPS * 4 * MAX_WARPS);
  grid_dependency_wait();
  __shared__ uint4 s_edges[2];
  const Block<T, NV, ALIGNED> b(rows, width, shift, classes, lanes, s_edges);
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
  auto counts = [&](uint32_t r) { return r < b.rows && (valid == nullptr || valid[r] != 0); };
  auto fetch = [&](uint32_t r, bool counted) {
    on = counted;
    mean = rstd = 0.0f;
    if (on) {
      const float2 st = __ldg(reinterpret_cast<const float2*>(stats) + r);
      mean = st.x;
      rstd = st.y;
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
  Ring<T, RES ? 3 : 2> ring{reinterpret_cast<uint8_t*>(s_dyn), s_bars, args.depth, b.count * 16, {x, dy}, args.status,
                            args.budget_ns};
  if constexpr (RES) ring.src[2] = dres;
  uint32_t row = b.first();
  bool ahead = false;  // RING, the first thread: whether the row after those on their way counts
  if constexpr (MODE == RING) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < args.depth; ++i) mbar_init(s_bars + i, 1);
      fence_mbar_init();
      for (int i = 0; i < args.depth; ++i)
        if (row + i * b.step < b.rows) ring.issue(b, i, row + i * b.step, counts(row + i * b.step));
      ahead = counts(row + args.depth * b.step);
    }
    __syncthreads();
  }
  fetch(row, counts(row));
  bool next_on = counts(row + b.step);
  int n = 0;
  for (uint32_t q = b.first_of_block(); q < b.rows; q += b.step, row += b.step, ++n) {
    const bool counted = on;
    const float mu = mean, rs = rstd;
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
    // xhat and dy of vector i, zeros where they are not the row's own: -mean rstd, what xhat would be there, may be
    // infinite where the row's own values are not
    const F2 minus(-mu, -mu), scale(rs, rs);
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
      b.zero_outside(vx, i);
    };
    F2 vx[HV][P], vd[HV][P];  // HOLD: xhat and d, kept for the second pass
    F2 s0(0.0f, 0.0f), s1(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = HOLD ? i : 0;
      F2 vy[P];
      values(i, vx[k], vy);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        vd[k][j] = mul2(vy[j], weight(i, j));
        s0 = add2(s0, vd[k][j]);
        s1 = fma2(vd[k][j], vx[k][j], s1);
        dg[i][j] = fma2(vy[j], vx[k][j], dg[i][j]);
        db[i][j] = add2(db[i][j], vy[j]);
      }
    }
    if constexpr (HOLD) {
      fetch(row + b.step, next_on);
      next_on = counts(row + 2 * b.step);
    }
    float s[2] = {s0.get().x + s0.get().y, s1.get().x + s1.get().y};
    row_sum(s, lanes, b.group, s_buf[lanes > 32 ? b.group : 0], slot);
    if constexpr (MODE == RING) {  // all threads have read the row: its slot takes the next one
      if (threadIdx.x == 0 && row + args.depth * b.step < b.rows) {
        ring.issue(b, n + args.depth, row + args.depth * b.step, ahead);
        ahead = counts(row + (args.depth + 1) * b.step);
      }
    }
    if (row < b.rows) {
      const float c0 = -s[0] * inv * rs, c1 = -s[1] * inv * rs;
      const F2 m0(c0, c0), m1(c1, c1);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int k = HOLD ? i : 0;
        F2 vr[P], vo[P];
        if constexpr (!HOLD) {
          values(i, vx[0], vd[0]);
#pragma unroll
          for (int j = 0; j < P; ++j) vd[0][j] = mul2(vd[0][j], weight(i, j));
        }
        if constexpr (RES) {
          if constexpr (!HOLD) rr[0] = counted ? b.load(dres, row, i) : none;
          Vec<T>::unpack(rr[k], vr);  // a neighbour's values go no further than the store
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const F2 t = fma2(vx[k][j], m1, RES ? add2(vr[j], m0) : m0);
          vo[j] = fma2(vd[k][j], scale, t);
        }
        b.store(dx, row, i, vo, counted);
      }
    }
    if (!HOLD) {
      fetch(row + b.step, next_on);
      next_on = counts(row + 2 * b.step);
    }
  }
  grid_dependency_launch();
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

constexpr int WS_COLS = 16, WS_PARTS = 64;  // of a block: columns, threads that share a column's sums

// Column c of [dgamma | dbeta] = the sum of the blocks' partial sums.  Latency bounds it: the loads of a thread are all
// in flight at once (READS, for the one wave of blocks that leave sums).
__global__ void __launch_bounds__(WS_COLS* WS_PARTS)
    weight_sum_kernel(const float* __restrict__ partial, int blocks, int width, float* __restrict__ dgamma,
                      float* __restrict__ dbeta) {
  constexpr int READS = 12;
  __shared__ float s[WS_PARTS][WS_COLS + 1];
  grid_dependency_wait();
  const int col = threadIdx.x % WS_COLS, part = threadIdx.x / WS_COLS;
  const int c = blockIdx.x * WS_COLS + col;
  float sum = 0.0f;
  if (c < 2 * width)
    for (int b = part; b < blocks; b += READS * WS_PARTS) {
      float v[READS];
#pragma unroll
      for (int i = 0; i < READS; ++i)
        v[i] = b + i * WS_PARTS < blocks ? __ldg(partial + static_cast<size_t>(b + i * WS_PARTS) * 2 * width + c) : 0.0f;
#pragma unroll
      for (int i = 0; i < READS; ++i) sum += v[i];
    }
  s[part][col] = sum;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= WS_COLS) return;
  sum = s[lane][warp] + s[lane + 32][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int to = blockIdx.x * WS_COLS + warp;
  if (lane == 0 && to < 2 * width) (to < width ? dgamma[to] : dbeta[to - width]) = sum;
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

// `most`: vectors a thread at most, `resident`: threads an SM has room for, `together`: in as few blocks as that takes
template <typename T>
Plan plan(int sm_count, int rows, int width, bool al, int most, int resident, bool together) {
  Plan p;
  const int nvec = row_vectors<T>(width, al);
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes * most < nvec) p.lanes *= 2;
  while (p.lanes >= 32 && p.lanes < 32 * MAX_WARPS && p.lanes * most < nvec) p.lanes += 32;
  p.nv = ceil_div(nvec, p.lanes);
  p.threads = p.lanes > 32 ? p.lanes : 128;
  if (together && p.nv <= most) {
    // no more rows at a time than give every SM a block
    int groups = ceil_div(rows, sm_count);
    if (groups > resident / p.lanes) groups = resident / p.lanes;
    if (groups * p.lanes > p.threads) p.threads = ceil_div(groups * p.lanes, 32) * 32;
  }
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
  // A block leaves one sum of the weights' gradients: one block an SM with several rows at a time takes 58 us for 20011
  // bf16 rows of 1497 values, a block a row 62 (10 and 16 for 760 rows).  A ring's block has one row.
  const Plan p = plan<T>(sm_count, rows, width, al, BWD_COLS<T> / Vec<T>::N, threads_per_sm(BWD_REGS<T>), false);
  if (sizeof(T) == 4 && p.lanes > 32) return p;
  return plan<T>(sm_count, rows, width, al, BWD_COLS<T> / Vec<T>::N, threads_per_sm(BWD_REGS<T>), true);
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
  constexpr int HOLDS = FWD_COLS<T, ALIGNED> / Vec<T>::N;
  const Plan p = plan<T>(ctx->sm_count, rows, width, ALIGNED, HOLDS, threads_per_sm(FWD_REGS<T>), false);
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
  return launch_dependent(weight_sum_kernel, ceil_div(2ll * width, WS_COLS), WS_COLS * WS_PARTS, 0, 0, s, partial, p.blocks,
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
