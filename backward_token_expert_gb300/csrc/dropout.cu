// Dropout with a residual, out_i = residual_i + (kept_i ? x_i / (1 - p) : 0),
// whose mask is never stored: element i is kept unless word i mod 4 of
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, SC 2011) at counter
// (i div 4, offset) with the seed as key is below floor(p 2^32).  The backward
// draws the same mask again: it is the same call on the gradient.
//
// One read of x and residual, one write: memory bounds it as long as the ten
// rounds (two 32 x 32 -> 64 bit products and two three-way exclusive ors for four
// elements each) hide behind it, which takes all the threads an SM can have (32
// registers).  The round keys come with the launch; what the block's counters have
// in common in rounds 1 and 2 is computed once.  67108864 elements: fp32 82 us
// (0.96 of the HBM's rate), bf16 with a residual 64 us (0.93), bf16 alone, where
// eight elements move only 32 bytes, 56 us (0.70).  There no unit is full: the pipe
// of the wide products is busy for 65 % of the cycles, the ALU 58, issue 57, DRAM
// 47; a thread's loads, draws and stores follow one another.
#include "lrm_internal.cuh"
#include "vec.cuh"

namespace lrm {
namespace {

constexpr int DR_THREADS = 256;
template <typename T>
constexpr int VECTORS = sizeof(T) == 2 ? 2 : 1;  // a thread has in flight

struct RoundKeys {
  uint32_t a[10], b[10];
};

// Philox4x32-10 of the counters (word 0 = a thread's, the other three the same for the whole block): rounds 1 and 2
// then have one product of the thread's own each, the other is the block's.
struct Philox {
  uint32_t r1_c0, r1_c1, r1_c3;  // round 1: c0 and c1; what is exclusive-ored into c2
  uint32_t r2_c0, r2_c2, r2_c3;  // round 2: what goes into c0 and c2; c3
  __device__ __forceinline__ Philox(uint32_t block_hi, uint64_t offset, const RoundKeys& k) {
    const uint64_t p1 = static_cast<uint64_t>(static_cast<uint32_t>(offset)) * 0xCD9E8D57u;
    r1_c0 = static_cast<uint32_t>(p1 >> 32) ^ block_hi ^ k.a[0];
    r1_c1 = static_cast<uint32_t>(p1);
    r1_c3 = static_cast<uint32_t>(offset >> 32) ^ k.b[0];
    const uint64_t p0 = static_cast<uint64_t>(r1_c0) * 0xD2511F53u;
    r2_c0 = r1_c1 ^ k.a[1];
    r2_c2 = static_cast<uint32_t>(p0 >> 32) ^ k.b[1];
    r2_c3 = static_cast<uint32_t>(p0);
  }
  __device__ __forceinline__ void operator()(uint32_t word, const RoundKeys& k, uint32_t (&c)[4]) const {
    const uint64_t p0 = static_cast<uint64_t>(word) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(static_cast<uint32_t>(p0 >> 32) ^ r1_c3) * 0xCD9E8D57u;
    c[0] = static_cast<uint32_t>(p1 >> 32) ^ r2_c0;
    c[1] = static_cast<uint32_t>(p1);
    c[2] = static_cast<uint32_t>(p0) ^ r2_c2;
    c[3] = r2_c3;
#pragma unroll
    for (int r = 2; r < 10; ++r) {
      const uint64_t q0 = static_cast<uint64_t>(c[0]) * 0xD2511F53u, q1 = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
      c[0] = static_cast<uint32_t>(q1 >> 32) ^ c[1] ^ k.a[r];
      c[1] = static_cast<uint32_t>(q1);
      c[2] = static_cast<uint32_t>(q0 >> 32) ^ c[3] ^ k.b[r];
      c[3] = static_cast<uint32_t>(q0);
    }
  }
};

struct DropoutArgs {
  RoundKeys keys;
  uint64_t offset;
  const uint64_t* step;  // device value added to offset, or NULL
  uint32_t last;         // the largest word that drops its element
  float scale;           // 1 / (1 - p)
};

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_float<uint16_t>(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ uint16_t from_float<uint16_t>(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

// DROP = false: p = 0, nothing is drawn.  VECTOR: 16-byte accesses.
template <typename T, bool DROP, bool VECTOR, bool RES>
__global__ void __launch_bounds__(DR_THREADS, 8)
    dropout_kernel(const T* x, const T* residual, long long n, const __grid_constant__ DropoutArgs a, T* out) {
  constexpr int N = 16 / sizeof(T);
  grid_dependency_wait();
  const uint64_t offset = a.offset + (a.step != nullptr ? __ldg(a.step) : 0);
  const long long items = (n + N - 1) / N;
  constexpr int U = VECTORS<T>;
  for (long long i0 = static_cast<long long>(blockIdx.x) * (U * DR_THREADS); i0 < items;
       i0 += static_cast<long long>(gridDim.x) * (U * DR_THREADS)) {
    T xv[U][N], rv[U][N];
    bool whole[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long e0 = (i0 + u * DR_THREADS + threadIdx.x) * N;
      whole[u] = VECTOR && e0 + N <= n;
      if (whole[u]) {
        // plain loads: out may be x or residual
        *reinterpret_cast<uint4*>(xv[u]) = *reinterpret_cast<const uint4*>(x + e0);
        if (RES) *reinterpret_cast<uint4*>(rv[u]) = *reinterpret_cast<const uint4*>(residual + e0);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          xv[u][j] = e0 + j < n ? x[e0 + j] : T(0);
          rv[u][j] = RES && e0 + j < n ? residual[e0 + j] : T(0);
        }
      }
    }
    // a block's counters start at a multiple of U DR_THREADS N / 4, so they share their upper word
    const uint64_t q0 = static_cast<uint64_t>(i0) * (N / 4);
    const Philox draw(static_cast<uint32_t>(q0 >> 32), offset, a.keys);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long e0 = (i0 + u * DR_THREADS + threadIdx.x) * N;
#pragma unroll
      for (int b = 0; b < N / 4; ++b) {
        uint32_t w[4];
        if (DROP) draw(static_cast<uint32_t>(q0) + (u * DR_THREADS + threadIdx.x) * (N / 4) + b, a.keys, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = b * 4 + j;
          const float r = RES ? to_float(rv[u][m]) : 0.0f;
          const float v = RES ? fmaf(to_float(xv[u][m]), a.scale, r) : to_float(xv[u][m]) * a.scale;
          xv[u][m] = from_float<T>(!DROP || w[j] > a.last ? v : r);
        }
      }
      if (whole[u]) {
        *reinterpret_cast<uint4*>(out + e0) = *reinterpret_cast<const uint4*>(xv[u]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (e0 + j < n) out[e0 + j] = xv[u][j];
      }
    }
  }
}

template <typename T, bool DROP, bool VECTOR, bool RES>
lrm_status launch(lrm_ctx* ctx, const void* x, const void* residual, long long n, const DropoutArgs& a, void* out,
                  cudaStream_t s) {
  auto kern = dropout_kernel<T, DROP, VECTOR, RES>;
  static thread_local int dev = -1, cap = 0;
  if (dev != ctx->device) {
    cap = resident_grid(ctx, kern, DR_THREADS, 0);
    dev = ctx->device;
  }
  constexpr long long per = static_cast<long long>(VECTORS<T> * DR_THREADS) * (16 / sizeof(T));
  const long long need = (n + per - 1) / per;
  return launch_dependent(kern, static_cast<int>(need < cap ? need : cap), DR_THREADS, 0, 0, s,
                          static_cast<const T*>(x), static_cast<const T*>(residual), n, a, static_cast<T*>(out));
}

template <typename T, bool DROP, bool VECTOR>
lrm_status dispatch2(lrm_ctx* ctx, const void* x, const void* residual, long long n, const DropoutArgs& a, void* out,
                     cudaStream_t s) {
  return residual != nullptr ? launch<T, DROP, VECTOR, true>(ctx, x, residual, n, a, out, s)
                             : launch<T, DROP, VECTOR, false>(ctx, x, residual, n, a, out, s);
}

template <typename T>
lrm_status dispatch(lrm_ctx* ctx, const void* x, const void* residual, long long n, bool drop, const DropoutArgs& a,
                    void* out, cudaStream_t s) {
  const bool vec = aligned(x, 16) && aligned(out, 16) && aligned(residual, 16);
  if (drop)
    return vec ? dispatch2<T, true, true>(ctx, x, residual, n, a, out, s)
               : dispatch2<T, true, false>(ctx, x, residual, n, a, out, s);
  return vec ? dispatch2<T, false, true>(ctx, x, residual, n, a, out, s)
             : dispatch2<T, false, false>(ctx, x, residual, n, a, out, s);
}

}  // namespace
}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_dropout_add(lrm_ctx* ctx, const void* x, const void* residual, int32_t dtype, int64_t n,
                                      double p, uint64_t seed, uint64_t offset, const uint64_t* step, void* out,
                                      void* stream) {
  if (ctx == nullptr || n < 0 || !(p >= 0.0 && p <= 1.0)) return LRM_ERR_INVALID_ARG;
  if (dtype != LRM_F32 && dtype != LRM_BF16) return LRM_ERR_INVALID_ARG;
  if (n == 0) return LRM_OK;
  if (x == nullptr || out == nullptr) return LRM_ERR_INVALID_ARG;
  const size_t es = dtype == LRM_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(out, es) || !aligned(residual, es) || !aligned(step, 8)) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  const uint64_t below = static_cast<uint64_t>(p * 4294967296.0);  // words that drop: 0 .. below - 1
  DropoutArgs a;
  for (int r = 0; r < 10; ++r) {
    a.keys.a[r] = static_cast<uint32_t>(seed) + r * 0x9E3779B9u;
    a.keys.b[r] = static_cast<uint32_t>(seed >> 32) + r * 0xBB67AE85u;
  }
  a.offset = offset;
  a.step = step;
  a.last = static_cast<uint32_t>(below - 1);
  a.scale = p < 1.0 ? static_cast<float>(1.0 / (1.0 - p)) : 0.0f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == LRM_F32 ? dispatch<float>(ctx, x, residual, n, below > 0, a, out, s)
                          : dispatch<uint16_t>(ctx, x, residual, n, below > 0, a, out, s);
}
