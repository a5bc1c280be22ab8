// The gate weights' gradient on the retained pairs: with y_t = sum_u alpha_u
// W_e phi_u and the input-gradient rows dphi_c[r] = (alpha_u g_t) W_e,
//   alpha_u dL/dalpha_u = <alpha_u g_t, W_e phi_u> = <dphi_c[r], phi_c[r]>,
// the form in which the router's softmax takes it (no division by alpha).
//
// HBM-bound: 4 I bytes a row are read once.  A warp takes one row, or up to
// eight short ones (200000 rows of 64: 10.7 us, one a warp 38.9), by 16-byte
// streaming loads, two of each operand at a time a lane (30011 rows of 1496:
// 27.8 us, four at a time 31.6); products and sums in fp32, one 4-byte store at
// the pair's place.  The pairs that were not retained are zeroed by gate_zero;
// gate_grad_kernel is launched dependently and waits for it only before its first
// store, so that the zeroing costs no time of its own.  87204 rows of 768 take
// 40.7 us (6.6 TB/s).
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

template <int L>
__global__ void __launch_bounds__(GG_THREADS) gate_grad_kernel(const uint4* __restrict__ dphi,
                                                               const uint4* __restrict__ phi,
                                                               const int32_t* __restrict__ sel_offsets, int E,
                                                               const int32_t* __restrict__ sel_ids, int max_rows,
                                                               int N, int iv, float* __restrict__ dgate,
                                                               unsigned int* status) {
  constexpr int PER_WARP = 32 / L;
  const int lane = threadIdx.x & 31, q = lane % L;
  const int rows = min(max(__ldg(sel_offsets + E), 0), max_rows);
  const long long step = static_cast<long long>(gridDim.x) * GG_WARPS * PER_WARP;
  bool zeroed = false;
  // r0: the warp's first row; its groups take the rows after it
  for (long long r0 = (static_cast<long long>(blockIdx.x) * GG_WARPS + (threadIdx.x >> 5)) * PER_WARP; r0 < rows;
       r0 += step) {
    const long long r = r0 + lane / L;
    const bool here = L == 32 || r < rows;
    const uint4* x = dphi + static_cast<size_t>(r) * iv;
    const uint4* y = phi + static_cast<size_t>(r) * iv;
    const int u = here ? __ldg(sel_ids + r) : 0;
    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int v0 = q; v0 < iv; v0 += L * GG_BATCH) {
      uint4 xs[GG_BATCH], ys[GG_BATCH];
#pragma unroll
      for (int j = 0; j < GG_BATCH; ++j) {
        const int v = v0 + L * j;
        const bool in = here && v < iv;
        xs[j] = in ? ld_stream(x + v) : make_uint4(0u, 0u, 0u, 0u);
        ys[j] = in ? ld_stream(y + v) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < GG_BATCH; ++j) acc_dot8(xs[j], ys[j], a);
    }
    float s = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (!zeroed) {
      grid_dependency_wait();
      zeroed = true;
    }
    if (q == 0 && here) {
      if (u >= 0 && u < N)
        dgate[u] = s;
      else
        raise_flag(status, LRM_ERR_INDEX);
    }
  }
  if (!zeroed) grid_dependency_wait();
}

struct GateArgs {
  const uint4 *dphi, *phi;
  const int32_t* sel_offsets;
  int E;
  const int32_t* sel_ids;
  int max_rows, N, iv;
  float* dgate;
};

template <int L>
lrm_status launch_gate(lrm_ctx* ctx, const GateArgs& a, cudaStream_t s) {
  static thread_local int dev = -1, grid = 0;
  if (dev != ctx->device) {
    grid = resident_grid(ctx, gate_grad_kernel<L>, GG_THREADS, 0);
    dev = ctx->device;
  }
  constexpr long long pass = GG_WARPS * (32 / L);
  const long long need = (a.max_rows + pass - 1) / pass;
  return launch_dependent(gate_grad_kernel<L>, static_cast<int>(need < grid ? need : grid), GG_THREADS, 0, 1, s, a.dphi,
                          a.phi, a.sel_offsets, a.E, a.sel_ids, a.max_rows, a.N, a.iv, a.dgate, ctx->d_status);
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
  const GateArgs a{reinterpret_cast<const uint4*>(dphi_c), reinterpret_cast<const uint4*>(phi_c), sel_offsets, dims.E,
                   sel_ids, max_rows, N, dims.I / 8, dgate};
  // lanes a row: two loads of each operand a lane where the row has them
  if (a.iv <= 8) return launch_gate<4>(ctx, a, s);
  if (a.iv <= 16) return launch_gate<8>(ctx, a, s);
  if (a.iv <= 32) return launch_gate<16>(ctx, a, s);
  return launch_gate<32>(ctx, a, s);
}
