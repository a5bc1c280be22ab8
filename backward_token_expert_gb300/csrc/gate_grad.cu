// The gate weights' gradient on the retained pairs: with y_t = sum_u alpha_u
// W_e phi_u and the input-gradient rows dphi_c[r] = (alpha_u g_t) W_e,
//   alpha_u dL/dalpha_u = <alpha_u g_t, W_e phi_u> = <dphi_c[r], phi_c[r]>,
// the form in which the router's softmax takes it (no division by alpha).
//
// HBM-bound: 4 I bytes a row are read once.  One warp per row, 16-byte
// streaming loads (two of each operand at a time a lane; four took 31.6 us, not 27.8, for 30011 rows of 1496), products and sums in
// fp32, one 4-byte store at the pair's place.  The pairs that were not retained
// are zeroed by gate_zero; gate_grad_kernel is launched dependently and waits
// for it only before its first store, so that the zeroing costs no time of its
// own.  87204 rows of 768 take 41.4 us (6.5 TB/s).
#include "lrm_internal.cuh"
#include "vec.cuh"

namespace lrm {
namespace {

constexpr int GG_THREADS = 256;
constexpr int GG_WARPS = GG_THREADS / 32;
constexpr int GG_BATCH = 2;

// Adds the products of the 8 bf16 values of x and y into 8 fp32 chains (each
// product is exact in fp32).
__device__ __forceinline__ void acc_dot8(const uint4& x, const uint4& y, float (&a)[8]) {
  a[0] = fmaf(bf16_lo(x.x), bf16_lo(y.x), a[0]);
  a[1] = fmaf(bf16_hi(x.x), bf16_hi(y.x), a[1]);
  a[2] = fmaf(bf16_lo(x.y), bf16_lo(y.y), a[2]);
  a[3] = fmaf(bf16_hi(x.y), bf16_hi(y.y), a[3]);
  a[4] = fmaf(bf16_lo(x.z), bf16_lo(y.z), a[4]);
  a[5] = fmaf(bf16_hi(x.z), bf16_hi(y.z), a[5]);
  a[6] = fmaf(bf16_lo(x.w), bf16_lo(y.w), a[6]);
  a[7] = fmaf(bf16_hi(x.w), bf16_hi(y.w), a[7]);
}

__global__ void __launch_bounds__(GG_THREADS) gate_zero(float* __restrict__ dgate, int N) {
  grid_dependency_launch();
  const long long step = static_cast<long long>(gridDim.x) * GG_THREADS;
  for (long long i = static_cast<long long>(blockIdx.x) * GG_THREADS + threadIdx.x; i < N; i += step) dgate[i] = 0.f;
}

__global__ void __launch_bounds__(GG_THREADS) gate_grad_kernel(const uint4* __restrict__ dphi,
                                                               const uint4* __restrict__ phi,
                                                               const int32_t* __restrict__ sel_offsets, int E,
                                                               const int32_t* __restrict__ sel_ids, int max_rows,
                                                               int N, int iv, float* __restrict__ dgate,
                                                               unsigned int* status) {
  const int lane = threadIdx.x & 31;
  const int rows = min(max(__ldg(sel_offsets + E), 0), max_rows);
  const int warps_total = gridDim.x * GG_WARPS;
  bool zeroed = false;
  for (long long r = blockIdx.x * GG_WARPS + (threadIdx.x >> 5); r < rows; r += warps_total) {
    const uint4* x = dphi + static_cast<size_t>(r) * iv;
    const uint4* y = phi + static_cast<size_t>(r) * iv;
    const int u = __ldg(sel_ids + r);
    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int v0 = lane; v0 < iv; v0 += 32 * GG_BATCH) {
      uint4 xs[GG_BATCH], ys[GG_BATCH];
#pragma unroll
      for (int j = 0; j < GG_BATCH; ++j) {
        const int v = v0 + 32 * j;
        xs[j] = v < iv ? ld_stream(x + v) : make_uint4(0u, 0u, 0u, 0u);
        ys[j] = v < iv ? ld_stream(y + v) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < GG_BATCH; ++j) acc_dot8(xs[j], ys[j], a);
    }
    float s = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (!zeroed) {
      grid_dependency_wait();
      zeroed = true;
    }
    if (lane == 0) {
      if (u >= 0 && u < N)
        dgate[u] = s;
      else
        raise_flag(status, LRM_ERR_INDEX);
    }
  }
  if (!zeroed) grid_dependency_wait();
}

}  // namespace
}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_gate_grad(lrm_ctx* ctx, const uint16_t* dphi_c, const uint16_t* phi_c,
                                    const int32_t* sel_offsets, const int32_t* sel_ids, lrm_dims dims,
                                    int32_t max_rows, float* dgate, void* stream) {
  if (ctx == nullptr) return LRM_ERR_INVALID_ARG;
  lrm_status st = check_dims(dims);
  if (st != LRM_OK) return st;
  if (max_rows < 0 || sel_offsets == nullptr) return LRM_ERR_INVALID_ARG;
  const int N = dims.T * dims.k;
  if (N == 0) return LRM_OK;
  if (dgate == nullptr || (max_rows > 0 && (dphi_c == nullptr || phi_c == nullptr || sel_ids == nullptr)))
    return LRM_ERR_INVALID_ARG;
  if (!aligned(dphi_c, 16) || !aligned(phi_c, 16) || !aligned(sel_offsets, 4) || !aligned(sel_ids, 4) ||
      !aligned(dgate, 4))
    return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int zero_need = static_cast<int>((static_cast<long long>(N) + 4 * GG_THREADS - 1) / (4 * GG_THREADS));
  gate_zero<<<zero_need < ctx->sm_count ? zero_need : ctx->sm_count, GG_THREADS, 0, s>>>(dgate, N);
  if ((st = launch_status()) != LRM_OK || max_rows == 0) return st;
  static thread_local int dev = -1, grid = 0;
  if (dev != ctx->device) {
    grid = resident_grid(ctx, gate_grad_kernel, GG_THREADS, 0);
    dev = ctx->device;
  }
  const long long need = (static_cast<long long>(max_rows) + GG_WARPS - 1) / GG_WARPS;
  return launch_dependent(gate_grad_kernel, static_cast<int>(need < grid ? need : grid), GG_THREADS, 0, 1, s,
                          reinterpret_cast<const uint4*>(dphi_c), reinterpret_cast<const uint4*>(phi_c), sel_offsets,
                          dims.E, sel_ids, max_rows, N, dims.I / 8, dgate, ctx->d_status);
}
