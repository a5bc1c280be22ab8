// The inverse mapping of LRMoE (sec. 1 and 3.3; Alg. 1, ScatterWithZeros;
// sec. 3.4): every kept row returns to the slot its pair had before
// compaction, and the slots of dropped pairs are filled with zeros so that
// the next dense layer sees the layout it expects.
// lrm_grouped_dgrad_scatter writes every retained row of the input gradient
// to its pair's row; this file zeroes the rows of the pairs that were not
// retained.  Two launches:
//   mark_kernel   one thread per retained row sets bit sel_ids[r] of an
//                 N-bit map (the map is cleared on the stream first);
//   zero_kernel   one warp per pair row: rows whose bit is clear are written
//                 with zeros (16-byte stores; HBM-bound, no reads but the map).
//
// lrm_counted_rows is the same for whole tokens: counted_kernel copies the rows
// of the tokens that the router counted and writes zeros for the others, whose
// rows it does not read (a product of such a row, NaN or infinity, with a zero
// gradient would not be zero).  One warp per row, HBM-bound: 32768 rows of 2048, a
// tenth of them padding, 42.7 us (6.0 TB/s).
#include "lrm_internal.cuh"
#include "vec.cuh"

namespace lrm {
namespace {

constexpr int ZR_THREADS = 256;
constexpr int ZR_WARPS = ZR_THREADS / 32;

__global__ void __launch_bounds__(ZR_THREADS) mark_kernel(const int32_t* __restrict__ sel_offsets, int E,
                                                          const int32_t* __restrict__ sel_ids, int max_rows, int N,
                                                          uint32_t* __restrict__ bits, unsigned int* status) {
  const int total = min(max(__ldg(sel_offsets + E), 0), max_rows);
  for (int r = blockIdx.x * ZR_THREADS + threadIdx.x; r < total; r += gridDim.x * ZR_THREADS) {
    const int u = __ldg(sel_ids + r);
    if (u < 0 || u >= N) {
      raise_flag(status, LRM_ERR_INDEX);
      continue;
    }
    atomicOr(bits + (u >> 5), 1u << (u & 31));
  }
}

__global__ void __launch_bounds__(ZR_THREADS) zero_kernel(const uint32_t* __restrict__ bits, int N, int iv,
                                                          uint4* __restrict__ rows) {
  const int lane = threadIdx.x & 31;
  const int warps_total = gridDim.x * ZR_WARPS;
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  for (int u = blockIdx.x * ZR_WARPS + (threadIdx.x >> 5); u < N; u += warps_total) {
    if ((__ldg(bits + (u >> 5)) >> (u & 31)) & 1u) continue;  // retained: dgrad wrote it
    uint4* row = rows + static_cast<size_t>(u) * iv;
    for (int v = lane; v < iv; v += 32) row[v] = z;
  }
}

__global__ void __launch_bounds__(ZR_THREADS) counted_kernel(const uint4* __restrict__ rows,
                                                             const float2* __restrict__ row_stats, int T, int wv,
                                                             uint4* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * ZR_WARPS;
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  for (long long t = static_cast<long long>(blockIdx.x) * ZR_WARPS + (threadIdx.x >> 5); t < T; t += step) {
    const bool counted = __ldg(row_stats + t).y != 0.f;
    const uint4* from = rows + static_cast<size_t>(t) * wv;
    uint4* to = out + static_cast<size_t>(t) * wv;
#pragma unroll 4
    for (int v = lane; v < wv; v += 32) to[v] = counted ? ld_stream(from + v) : z;
  }
}

}  // namespace

size_t zero_dropped_workspace_bytes(const lrm_dims& d) {
  const size_t N = static_cast<size_t>(d.T) * d.k;
  return ((N + 31) / 32) * sizeof(uint32_t);
}

}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_zero_dropped_rows(lrm_ctx* ctx, const int32_t* sel_offsets, const int32_t* sel_ids,
                                            lrm_dims dims, int32_t max_rows, uint16_t* rows, void* ws,
                                            size_t ws_bytes, void* stream) {
  if (ctx == nullptr) return LRM_ERR_INVALID_ARG;
  lrm_status st = check_dims(dims);
  if (st != LRM_OK) return st;
  if (max_rows < 0 || sel_offsets == nullptr) return LRM_ERR_INVALID_ARG;
  const int N = dims.T * dims.k;
  if (N == 0) return LRM_OK;
  if (rows == nullptr || ws == nullptr || (max_rows > 0 && sel_ids == nullptr)) return LRM_ERR_INVALID_ARG;
  if (ws_bytes < zero_dropped_workspace_bytes(dims)) return LRM_ERR_WORKSPACE;
  if (!aligned(rows, 16) || !aligned(ws, 4) || !aligned(sel_offsets, 4) || (sel_ids && !aligned(sel_ids, 4)))
    return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t* bits = static_cast<uint32_t*>(ws);
  LRM_CHECK_CUDA(cudaMemsetAsync(bits, 0, zero_dropped_workspace_bytes(dims), s));
  if (max_rows > 0) {
    const int need = (max_rows + ZR_THREADS - 1) / ZR_THREADS;
    const int cap = ctx->sm_count * 4;
    mark_kernel<<<need < cap ? need : cap, ZR_THREADS, 0, s>>>(sel_offsets, dims.E, sel_ids, max_rows, N, bits,
                                                               ctx->d_status);
    if ((st = launch_status()) != LRM_OK) return st;
  }
  static thread_local int cap_device = -1, cap = 0;
  if (cap_device != ctx->device) {
    cap = resident_grid(ctx, zero_kernel, ZR_THREADS, 0);
    cap_device = ctx->device;
  }
  const int need = (N + ZR_WARPS - 1) / ZR_WARPS;
  zero_kernel<<<need < cap ? need : cap, ZR_THREADS, 0, s>>>(bits, N, dims.I / 8, reinterpret_cast<uint4*>(rows));
  return launch_status();
}

extern "C" lrm_status lrm_counted_rows(lrm_ctx* ctx, const uint16_t* rows, const float* row_stats, lrm_dims dims,
                                       int32_t width, uint16_t* out, void* stream) {
  if (ctx == nullptr) return LRM_ERR_INVALID_ARG;
  lrm_status st = check_dims(dims);
  if (st != LRM_OK) return st;
  if (width < 8 || width % 8 != 0 || width > 65536) return LRM_ERR_INVALID_ARG;
  if (dims.T == 0) return LRM_OK;
  if (rows == nullptr || row_stats == nullptr || out == nullptr) return LRM_ERR_INVALID_ARG;
  if (!aligned(rows, 16) || !aligned(out, 16) || !aligned(row_stats, 8)) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  static thread_local int cap_device = -1, cap = 0;
  if (cap_device != ctx->device) {
    cap = resident_grid(ctx, counted_kernel, ZR_THREADS, 0);
    cap_device = ctx->device;
  }
  const int need = static_cast<int>((static_cast<long long>(dims.T) + ZR_WARPS - 1) / ZR_WARPS);
  counted_kernel<<<need < cap ? need : cap, ZR_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
      reinterpret_cast<const uint4*>(rows), reinterpret_cast<const float2*>(row_stats), dims.T, width / 8,
      reinterpret_cast<uint4*>(out));
  return launch_status();
}
