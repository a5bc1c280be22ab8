// Layer norm of the rows of a [rows, width] tensor, forward and backward
// (Ba, Kiros and Hinton, 2016): with mean and variance of a row,
//   y  = (x - mean) rstd gamma + beta,   rstd = 1 / sqrt(var + eps)
//   d  = dy gamma,  xhat = (x - mean) rstd
//   dx = rstd (d - mean(d) - xhat mean(d xhat)) [+ dres]
//   dgamma = sum over rows of dy xhat,   dbeta = sum over rows of dy
// Both read every value once and write every result once, so memory bounds
// them.  A row's values stay in registers between its statistics and its
// output: the variance is that of the centred values, all sums are fp32, and
// each output is rounded once.
//
// Rows that do not start at a 16-byte boundary (a width that is no multiple of
// the vector, or a tensor that starts between two) are read and written in the
// aligned vectors that cover them; a vector that is shared with the
// neighbouring row is stored element by element, and one that reaches beyond
// the tensor is read so too.
#include <type_traits>

#include "lrm_internal.cuh"
#include "swiglu.cuh"
#include "vec.cuh"

namespace lrm {
namespace {

constexpr int MAX_WIDTH = 16384;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  __device__ static __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ static __forceinline__ float get(const float* p) { return *p; }
  __device__ static __forceinline__ void put(float* p, float v) { *p = v; }
};
template <>
struct Vec<uint16_t> {  // bf16 bits
  static constexpr int N = 8;
  __device__ static __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
  }
  __device__ static __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  __device__ static __forceinline__ float get(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
  }
  __device__ static __forceinline__ void put(uint16_t* p, float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t*>(&b);
  }
};

// The vectors that cover a row: `lead` elements of the first one belong to what lies before the row.
template <typename T, bool ALIGNED>
struct RowSpan {
  static constexpr int N = Vec<T>::N;
  long long start;  // first element of the row
  int lead, count;  // elements before the row in its first vector; vectors

  // `shift`: elements of the tensor's start beyond a 16-byte boundary
  __device__ __forceinline__ RowSpan(long long row, int width, int shift) {
    start = row * width;
    lead = ALIGNED ? 0 : static_cast<int>((start + shift) % N);
    count = (lead + width + N - 1) / N;
  }
  // Vector v of the row as fp32; elements outside the row are 0.
  __device__ __forceinline__ uint4 load_raw(const T* base, int v, int width, long long total) const {
    const long long e0 = start - lead + static_cast<long long>(v) * N;
    if constexpr (ALIGNED) {
      return ld_stream(reinterpret_cast<const uint4*>(base + e0));
    } else {
      if (e0 >= 0 && e0 + N <= total) return ld_stream(reinterpret_cast<const uint4*>(base + e0));
      float f[N];
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = e0 + j >= 0 && e0 + j < total ? Vec<T>::get(base + e0 + j) : 0.0f;
      return Vec<T>::pack(f);
    }
  }
  // first column of vector v (negative in a row's first vector where `lead` > 0)
  __device__ __forceinline__ int column(int v) const { return v * N - lead; }
  __device__ __forceinline__ void store(T* base, int v, int width, const float (&f)[N]) const {
    const int c0 = column(v);
    T* at = base + start + c0;
    if constexpr (ALIGNED) {
      *reinterpret_cast<uint4*>(at) = Vec<T>::pack(f);
    } else {
      if (c0 >= 0 && c0 + N <= width) {
        *reinterpret_cast<uint4*>(at) = Vec<T>::pack(f);
        return;
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c0 + j >= 0 && c0 + j < width) Vec<T>::put(at + j, f[j]);
    }
  }
};

// Sum over a row's threads: its warps' lanes by shuffles, then, with more than one warp, over the block through
// shared memory.  `slot` alternates between calls, so that one barrier a call is enough.
template <int K>
__device__ __forceinline__ void row_sum(float (&s)[K], int warps, float (*buf)[32][K], int& slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < K; ++i) buf[slot][warp][i] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < K; ++i) s[i] = lane < warps ? buf[slot][lane][i] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  slot ^= 1;
}

// place of column c among the skewed weights in shared memory: a warp's lanes read columns 8 (or 4) apart, which
// the skew spreads over all banks
__device__ __forceinline__ int skew(int c, int n) { return c + c / n; }

// `warps` warps a row: the whole block, or 1 (the block's warps then have rows of their own).
template <typename T, int NV, bool ALIGNED>
__global__ void __launch_bounds__(512)
    layer_norm_kernel(const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
                      const uint8_t* __restrict__ valid, int rows, int width, int shift, float eps, int warps, T* y,
                      float* __restrict__ stats) {
  constexpr int N = Vec<T>::N;
  extern __shared__ float s_weights[];  // ALIGNED: none; else gamma and beta, skewed
  __shared__ float s_buf[2][32][1];
  grid_dependency_wait();
  const int per = skew(width, N) + 1;
  if (!ALIGNED) {
    for (int c = threadIdx.x; c < width; c += blockDim.x) {
      s_weights[skew(c, N)] = gamma[c];
      s_weights[per + skew(c, N)] = beta[c];
    }
    __syncthreads();
  }
  const int lanes = warps * 32;
  const int groups = blockDim.x / lanes;  // rows the block has at a time
  const int lane = threadIdx.x % lanes;
  const long long total = static_cast<long long>(rows) * width;
  const float inv = 1.0f / static_cast<float>(width);
  int slot = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * groups + threadIdx.x / lanes; row < rows;
       row += static_cast<long long>(gridDim.x) * groups) {
    const RowSpan<T, ALIGNED> span(row, width, shift);
    if (valid != nullptr && valid[row] == 0) {  // the same for all threads of the row
      const float zero[N] = {};
      for (int v = lane; v < span.count; v += lanes) span.store(y, v, width, zero);
      if (lane < 2) stats[row * 2 + lane] = 0.0f;
      continue;
    }
    uint4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * lanes;
      raw[i] = v < span.count ? span.load_raw(x, v, width, total) : make_uint4(0u, 0u, 0u, 0u);
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[N];
      Vec<T>::unpack(raw[i], f);
      const int c0 = span.column(lane + i * lanes);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (ALIGNED ? c0 < width : (c0 + j >= 0 && c0 + j < width)) s[0] += f[j];
    }
    row_sum(s, warps, s_buf, slot);
    const float mean = s[0] * inv;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[N];
      Vec<T>::unpack(raw[i], f);
      const int c0 = span.column(lane + i * lanes);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (ALIGNED ? c0 < width : (c0 + j >= 0 && c0 + j < width)) s[0] = fmaf(f[j] - mean, f[j] - mean, s[0]);
    }
    row_sum(s, warps, s_buf, slot);
    const float rstd = 1.0f / sqrtf(s[0] * inv + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * lanes;
      if (v >= span.count) continue;
      float f[N];
      Vec<T>::unpack(raw[i], f);
      const int c0 = span.column(v);
      if (ALIGNED) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
          const float4 g = __ldg(reinterpret_cast<const float4*>(gamma + c0 + j));
          const float4 b = __ldg(reinterpret_cast<const float4*>(beta + c0 + j));
          f[j] = fmaf((f[j] - mean) * rstd, g.x, b.x);
          f[j + 1] = fmaf((f[j + 1] - mean) * rstd, g.y, b.y);
          f[j + 2] = fmaf((f[j + 2] - mean) * rstd, g.z, b.z);
          f[j + 3] = fmaf((f[j + 3] - mean) * rstd, g.w, b.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int c = min(max(c0 + j, 0), width - 1);
          f[j] = fmaf((f[j] - mean) * rstd, s_weights[skew(c, N)], s_weights[per + skew(c, N)]);
        }
      }
      span.store(y, v, width, f);
    }
    if (lane == 0) {
      stats[row * 2] = mean;
      stats[row * 2 + 1] = rstd;
    }
  }
}

// Backward.  A thread has the same columns in every row of its block, so the weights' gradients are sums in its
// registers: where rows start at different places of a vector, a block takes only rows of one place (rows `classes`
// apart).  Blocks leave their sums in partial [blocks, 2, width], which weight_sum_kernel adds in a fixed order.
// `warps` as above; with one warp a row, the block's warps add their sums through shared memory first.
// With one vector a thread, a row's values and gamma stay in registers; with more, where they would not fit beside
// the sums, gamma lies in shared memory (skewed) and the second pass over a row reads it again, out of the L2.
template <typename T, int NV, bool ALIGNED>
__global__ void __launch_bounds__(512)
    layer_norm_bwd_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ gamma,
                          const float* __restrict__ stats, const uint8_t* __restrict__ valid,
                          const T* __restrict__ dres, int rows, int width, int shift, int classes, int warps,
                          T* __restrict__ dx, float* __restrict__ partial) {
  constexpr int N = Vec<T>::N;
  constexpr bool HOLD = NV == 1;
  extern __shared__ float s_dyn[];  // HOLD and one warp a row: [warps of the block][2][width]; !HOLD: gamma, skewed
  __shared__ float s_buf[2][32][2];
  grid_dependency_wait();
  const int lanes = warps * 32;
  const int groups = blockDim.x / lanes;
  const int lane = threadIdx.x % lanes, group = threadIdx.x / lanes;
  const int cls = blockIdx.x % classes;
  const long long step = static_cast<long long>(gridDim.x / classes) * groups;
  const long long total = static_cast<long long>(rows) * width;
  const float inv = 1.0f / static_cast<float>(width);
  const int lead = RowSpan<T, ALIGNED>(cls, width, shift).lead;  // that of all the block's rows
  float dg[NV][N], db[NV][N], ga[N];
  if (!HOLD) {
    for (int c = threadIdx.x; c < width; c += blockDim.x) s_dyn[skew(c, N)] = __ldg(gamma + c);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = (lane + i * lanes) * N - lead + j;
      if (HOLD) ga[j] = c >= 0 && c < width ? __ldg(gamma + c) : 0.0f;
      dg[i][j] = db[i][j] = 0.0f;
    }
  auto weight = [&](int c0, int j) { return HOLD ? ga[j] : s_dyn[skew(min(max(c0 + j, 0), width - 1), N)]; };
  int slot = 0;
  for (long long q = static_cast<long long>(blockIdx.x / classes) * groups + group; q * classes + cls < rows;
       q += step) {
    const long long row = q * classes + cls;
    const RowSpan<T, ALIGNED> span(row, width, shift);
    if (valid != nullptr && valid[row] == 0) {
      const float zero[N] = {};
      for (int v = lane; v < span.count; v += lanes) span.store(dx, v, width, zero);
      continue;
    }
    const float mean = __ldg(stats + row * 2), rstd = __ldg(stats + row * 2 + 1);
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint4 xr, yr, rr = none;
    if (HOLD && dres != nullptr && lane < span.count) rr = span.load_raw(dres, lane, width, total);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * lanes;
      xr = v < span.count ? span.load_raw(x, v, width, total) : none;
      yr = v < span.count ? span.load_raw(dy, v, width, total) : none;
      float fx[N], fy[N];
      Vec<T>::unpack(xr, fx);
      Vec<T>::unpack(yr, fy);
      const int c0 = span.column(v);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (ALIGNED ? c0 < width : (c0 + j >= 0 && c0 + j < width)) {
          const float xhat = (fx[j] - mean) * rstd, d = fy[j] * weight(c0, j);
          s[0] += d;
          s[1] = fmaf(d, xhat, s[1]);
          dg[i][j] = fmaf(fy[j], xhat, dg[i][j]);
          db[i][j] += fy[j];
        }
    }
    row_sum(s, warps, s_buf, slot);
    const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * lanes;
      if (v >= span.count) continue;
      if (!HOLD) {
        xr = span.load_raw(x, v, width, total);
        yr = span.load_raw(dy, v, width, total);
        if (dres != nullptr) rr = span.load_raw(dres, v, width, total);
      }
      float fx[N], fy[N], fr[N];
      Vec<T>::unpack(xr, fx);
      Vec<T>::unpack(yr, fy);
      Vec<T>::unpack(rr, fr);
      const int c0 = span.column(v);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float xhat = (fx[j] - mean) * rstd;
        const float g = rstd * (fmaf(fy[j], weight(c0, j), -m0) - xhat * m1);
        fx[j] = dres != nullptr ? g + fr[j] : g;
      }
      span.store(dx, v, width, fx);
    }
  }
  float* out = groups > 1 ? s_dyn + group * 2 * width : partial + static_cast<size_t>(blockIdx.x) * 2 * width;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = (lane + i * lanes) * N - lead + j;
      if (c >= 0 && c < width) {
        out[c] = dg[i][j];
        out[width + c] = db[i][j];
      }
    }
  if (groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) {
      float sum = 0.0f;
      for (int g = 0; g < groups; ++g) sum += s_dyn[g * 2 * width + c];
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

template <typename T, int NV, bool ALIGNED>
lrm_status launch_fwd(lrm_ctx* ctx, const T* x, const float* gamma, const float* beta, const uint8_t* valid, int rows,
                      int width, float eps, int warps, T* y, float* stats, cudaStream_t s) {
  auto kern = layer_norm_kernel<T, NV, ALIGNED>;
  const int threads = warps == 1 ? 128 : warps * 32;
  const size_t smem = ALIGNED ? 0 : 2 * (width + width / Vec<T>::N + 1) * sizeof(float);
  static thread_local int dev = -1, of_threads = 0, cap = 0;  // the last launch's: occupancy queries cost microseconds
  static thread_local size_t of_smem = 0;
  if (dev != ctx->device || of_threads != threads || of_smem != smem) {
    LRM_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
    cap = resident_grid(ctx, kern, threads, smem);
    dev = ctx->device, of_threads = threads, of_smem = smem;
  }
  const int need = ceil_div(rows, threads / (32 * warps));
  return launch_dependent(kern, need < cap ? need : cap, threads, smem, 0, s, x, gamma, beta, valid, rows, width,
                          shift_of<T>(x), eps, warps, y, stats);
}

template <typename T, bool ALIGNED>
lrm_status forward(lrm_ctx* ctx, const void* x, const float* gamma, const float* beta, const uint8_t* valid, int rows,
                   int width, float eps, void* y, float* stats, cudaStream_t s) {
  const int nvec = row_vectors<T>(width, ALIGNED);
  constexpr int MOST = 64 / Vec<T>::N;  // vectors a lane: 64 values
  int warps = 1;
  while (warps * 32 * MOST < nvec) warps *= 2;
  // few rows: more warps a row, for their latency
  while (warps < 16 && warps * 32 < nvec && static_cast<long long>(rows) * warps < ctx->sm_count * 4) warps *= 2;
  const int nv = ceil_div(nvec, warps * 32);
  auto go = [&](auto n) {
    return launch_fwd<T, decltype(n)::value, ALIGNED>(ctx, static_cast<const T*>(x), gamma, beta, valid, rows, width,
                                                      eps, warps, static_cast<T*>(y), stats, s);
  };
  if (nv <= 1) return go(std::integral_constant<int, 1>());
  if (nv <= 2) return go(std::integral_constant<int, 2>());
  if (nv <= 4) return go(std::integral_constant<int, 4>());
  if (MOST == 8 || nv <= 8) return go(std::integral_constant<int, 8>());
  return go(std::integral_constant<int, MOST>());
}

// How the backward cuts its work, the same for the launch and for the workspace's size.
struct BwdPlan {
  int warps, nv, threads, classes, blocks;
};

template <typename T>
BwdPlan bwd_plan(int sm_count, int rows, int width, bool al) {
  BwdPlan p;
  const int nvec = row_vectors<T>(width, al);
  p.warps = 1;
  while (p.warps < 16 && p.warps * 32 < nvec) ++p.warps;
  p.nv = ceil_div(nvec, p.warps * 32);
  p.threads = p.warps == 1 ? 256 : p.warps * 32;
  p.classes = 1;
  if (!al) {
    p.classes = Vec<T>::N;
    for (int w = width; p.classes > 1 && w % 2 == 0; w /= 2) p.classes /= 2;
  }
  const int groups = p.threads / (32 * p.warps);
  const int per_class = ceil_div(ceil_div(rows, p.classes), groups);
  int per_sm = 1024 / p.threads;
  if (per_sm < 1) per_sm = 1;
  int most = sm_count * per_sm / p.classes;
  if (most < 1) most = 1;
  p.blocks = p.classes * (per_class < most ? (per_class > 0 ? per_class : 1) : most);
  return p;
}

template <typename T, int NV, bool ALIGNED>
lrm_status launch_bwd(const BwdPlan& p, const T* x, const T* dy, const float* gamma, const float* stats,
                      const uint8_t* valid, const T* dres, int rows, int width, T* dx, float* partial,
                      cudaStream_t s) {
  auto kern = layer_norm_bwd_kernel<T, NV, ALIGNED>;
  const int groups = p.threads / (32 * p.warps);
  const size_t smem = groups > 1 ? static_cast<size_t>(groups) * 2 * width * sizeof(float)
                      : NV > 1   ? static_cast<size_t>(width + width / Vec<T>::N + 1) * sizeof(float)
                                 : 0;
  if (smem > 40 * 1024)
    LRM_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
  return launch_dependent(kern, p.blocks, p.threads, smem, 0, s, x, dy, gamma, stats, valid, dres, rows, width,
                          shift_of<T>(x), p.classes, p.warps, dx, partial);
}

template <typename T, bool ALIGNED>
lrm_status backward(lrm_ctx* ctx, const void* x, const void* dy, const float* gamma, const float* stats,
                    const uint8_t* valid, const void* dres, int rows, int width, void* dx, float* dgamma,
                    float* dbeta, float* partial, cudaStream_t s) {
  const BwdPlan p = bwd_plan<T>(ctx->sm_count, rows, width, ALIGNED);
  auto go = [&](auto n) {
    return launch_bwd<T, decltype(n)::value, ALIGNED>(p, static_cast<const T*>(x), static_cast<const T*>(dy), gamma,
                                                      stats, valid, static_cast<const T*>(dres), rows, width,
                                                      static_cast<T*>(dx), partial, s);
  };
  // vectors a thread: up to 5 in bf16 and 9 in fp32 at the largest width, one more than it fills where rows are cut
  lrm_status st;
  if (p.nv <= 1)
    st = go(std::integral_constant<int, 1>());
  else if (p.nv <= 2)
    st = go(std::integral_constant<int, 2>());
  else if (p.nv <= 3)
    st = go(std::integral_constant<int, 3>());
  else if (p.nv <= 5)
    st = go(std::integral_constant<int, 5>());
  else
    st = go(std::integral_constant<int, Vec<T>::N == 4 ? 9 : 5>());
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
  if (!aligned(x, es) || !aligned(y, es) || !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(stats, 4))
    return LRM_ERR_ALIGN;
  // the vectors of a row cut x and y alike
  if (reinterpret_cast<uintptr_t>(x) % 16 != reinterpret_cast<uintptr_t>(y) % 16) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == LRM_F32)
    return aligned_rows<float>(x, y, gamma, beta, width)
               ? forward<float, true>(ctx, x, gamma, beta, valid, rows, width, eps, y, stats, s)
               : forward<float, false>(ctx, x, gamma, beta, valid, rows, width, eps, y, stats, s);
  return aligned_rows<uint16_t>(x, y, gamma, beta, width)
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
    if (!aligned(x, es) || !aligned(gamma, 4) || !aligned(stats, 4) || !aligned(ws, 4)) return LRM_ERR_ALIGN;
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
  if (dtype == LRM_F32)
    return aligned_rows<float>(x, dy, dx, dres, width)
               ? backward<float, true>(ctx, x, dy, gamma, stats, valid, dres, rows, width, dx, dgamma, dbeta, part, s)
               : backward<float, false>(ctx, x, dy, gamma, stats, valid, dres, rows, width, dx, dgamma, dbeta, part,
                                        s);
  return aligned_rows<uint16_t>(x, dy, dx, dres, width)
             ? backward<uint16_t, true>(ctx, x, dy, gamma, stats, valid, dres, rows, width, dx, dgamma, dbeta, part, s)
             : backward<uint16_t, false>(ctx, x, dy, gamma, stats, valid, dres, rows, width, dx, dgamma, dbeta, part,
                                         s);
}
