// The router of the layer: gates and balance loss of a batch of logits, and
// the logits' gradient ("Expert Parallel Math Deep": importance P_e, load f_e
// and the auxiliary loss E sum f_e P_e; the z loss is the mean squared
// log-partition).
//
//   rf_rows    one warp per token.  The k largest logits are taken in k
//              rounds of a warp-wide maximum over order-preserving integer
//              keys (ties to the lower expert); the softmax of the same
//              registers is summed per lane for P, so the logits are read
//              once.  Every block leaves its sums of p, its counts, its sum
//              of lse^2 and its number of counted tokens in the workspace.
//   rf_sums    adds the blocks' sums in a fixed order and writes counts, f, P
//              and the losses.
//   rb_rows    one warp per token: p again from the saved (max, sum), the
//              balance term needs sum_e f_e p_e over the row, and the gates'
//              part touches k experts, which are placed through a row of
//              shared memory.
#include <math.h>

#include "lrm_internal.cuh"
#include "vec.cuh"

namespace lrm {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;
constexpr int RT_MAX_BLOCKS_PER_SM = 2;  // the grid of rf_rows, and so the workspace

struct RouterLayout {
  int nblk;  // blocks of rf_rows
  size_t p_off, cnt_off, z_off, tok_off, bytes;
};

RouterLayout router_layout(const lrm_ctx* ctx, const lrm_dims& d) {
  RouterLayout L;
  const long long need = (static_cast<long long>(d.T) + RT_WARPS - 1) / RT_WARPS;
  const long long cap = static_cast<long long>(ctx->sm_count) * RT_MAX_BLOCKS_PER_SM;
  L.nblk = static_cast<int>(need < cap ? need : cap);
  const size_t cells = static_cast<size_t>(L.nblk) * d.E;
  L.p_off = 0;
  L.cnt_off = L.p_off + cells * sizeof(float);
  L.z_off = (L.cnt_off + cells * sizeof(int32_t) + 15) / 16 * 16;
  L.tok_off = L.z_off + L.nblk * sizeof(double);
  L.bytes = L.tok_off + L.nblk * sizeof(int32_t);
  return L;
}

__device__ __forceinline__ float load_elem(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_elem(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A key that orders like the value: NaN is 1, -inf the next, -0 like +0.  0 is
// left for places that hold no logit.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  const uint32_t key = b ^ ((b & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
  return v != v ? 1u : key;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename TL, int VPL>
__global__ void __launch_bounds__(RT_THREADS) rf_rows(const TL* __restrict__ logits,
                                                      const uint8_t* __restrict__ valid, int T, int E, int k,
                                                      int renorm, int32_t* __restrict__ expert_idx,
                                                      float* __restrict__ alpha, float2* __restrict__ row_stats,
                                                      float* __restrict__ ws_p, int32_t* __restrict__ ws_cnt,
                                                      double* __restrict__ ws_z, int32_t* __restrict__ ws_tok) {
  extern __shared__ float rt_smem[];
  float* sp = rt_smem;                                        // [RT_WARPS][E]
  int* hist = reinterpret_cast<int*>(rt_smem + RT_WARPS * E);  // [E]
  __shared__ double s_z[RT_WARPS];
  __shared__ int s_tok[RT_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < E; i += RT_THREADS) hist[i] = 0;
  __syncthreads();

  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
  double z = 0.0;
  int tokens = 0;
  const long long step = static_cast<long long>(gridDim.x) * RT_WARPS;
  for (long long t = static_cast<long long>(blockIdx.x) * RT_WARPS + warp; t < T; t += step) {
    const TL* row = logits + static_cast<size_t>(t) * E;
    float v[VPL];
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < E ? load_elem(row + e) : -INFINITY;
      key[i] = e < E ? order_key(v[i]) : 0u;
    }
    float m = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    const float base = m == -INFINITY ? 0.f : m;
    float p[VPL], s = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = expf(v[i] - base);
      s += p[i];
    }
    s = warp_sum(s);
    const bool counted = s != 0.f && (valid == nullptr || valid[t] != 0);

    // slot j's expert and exponential go to lane j
    int my_e = 0;
    float my_p = 0.f;
    for (int j = 0; j < k; ++j) {
      uint32_t best = key[0];
      int e = lane;
      float pe = p[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i)
        if (key[i] > best) best = key[i], e = lane + 32 * i, pe = p[i];
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const int win = static_cast<int>(__reduce_min_sync(0xffffffffu, best == top ? static_cast<unsigned>(e) : ~0u));
      const float wp = __shfl_sync(0xffffffffu, pe, win & 31);
      if (lane == j) my_e = win, my_p = wp;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (win == lane + 32 * i) key[i] = 0u;
    }
    const float sel = warp_sum(my_p);  // lanes beyond k hold 0
    if (lane < k) {
      const size_t u = static_cast<size_t>(t) * k + lane;
      expert_idx[u] = my_e;
      alpha[u] = counted ? my_p / (renorm ? sel : s) : 0.f;
      if (counted) atomicAdd(&hist[my_e], 1);
    }
    if (lane == 0) row_stats[t] = counted ? make_float2(base, s) : make_float2(0.f, 0.f);
    if (counted) {
      const float inv = 1.f / s;
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += p[i] * inv;
      const float lse = base + logf(s);
      z += static_cast<double>(lse) * lse;
      ++tokens;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    if (e < E) sp[warp * E + e] = acc[i];
  }
  if (lane == 0) s_z[warp] = z, s_tok[warp] = tokens;
  __syncthreads();
  for (int e = tid; e < E; e += RT_THREADS) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < RT_WARPS; ++w) a += sp[w * E + e];
    ws_p[static_cast<size_t>(blockIdx.x) * E + e] = a;
    ws_cnt[static_cast<size_t>(blockIdx.x) * E + e] = hist[e];
  }
  if (tid == 0) {
    double a = 0.0;
    int n = 0;
    for (int w = 0; w < RT_WARPS; ++w) a += s_z[w], n += s_tok[w];
    ws_z[blockIdx.x] = a;
    ws_tok[blockIdx.x] = n;
  }
}

// One block of 1024 threads: thread e owns expert e.
__global__ void __launch_bounds__(1024) rf_sums(const float* __restrict__ ws_p, const int32_t* __restrict__ ws_cnt,
                                                const double* __restrict__ ws_z, const int32_t* __restrict__ ws_tok,
                                                int nblk, int E, int k, float aux_coef, float z_coef,
                                                int32_t* __restrict__ counts, float* __restrict__ f,
                                                float* __restrict__ P, lrm_router_losses* __restrict__ losses) {
  __shared__ double s_red[32];
  __shared__ double s_z;
  __shared__ int s_tok;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    double z = 0.0;
    int n = 0;
    for (int b = lane; b < nblk; b += 32) z += ws_z[b], n += ws_tok[b];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (lane == 0) s_z = z, s_tok = n;
  }
  __syncthreads();
  const int tokens = s_tok;
  double fp = 0.0;
  for (int e = tid; e < E; e += 1024) {
    double a = 0.0;
    int n = 0;
    for (int b = 0; b < nblk; ++b) {
      a += ws_p[static_cast<size_t>(b) * E + e];
      n += ws_cnt[static_cast<size_t>(b) * E + e];
    }
    const float Pe = tokens > 0 ? static_cast<float>(a / tokens) : 0.f;
    const float fe = tokens > 0 ? static_cast<float>(static_cast<double>(n) / (static_cast<double>(tokens) * k)) : 0.f;
    counts[e] = n;
    P[e] = Pe;
    f[e] = fe;
    fp += static_cast<double>(fe) * Pe;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) fp += __shfl_xor_sync(0xffffffffu, fp, o);
  if (lane == 0) s_red[warp] = fp;
  __syncthreads();
  if (tid == 0) {
    double a = 0.0;
    for (int w = 0; w < 32; ++w) a += s_red[w];
    const double aux = a * E, zl = tokens > 0 ? s_z / tokens : 0.0;
    lrm_router_losses r;
    r.aux = static_cast<float>(aux);
    r.z = static_cast<float>(zl);
    r.loss = static_cast<float>(aux_coef * aux + z_coef * zl);
    r.tokens = tokens;
    *losses = r;
  }
}

template <typename TL, typename TO, int VPL>
__global__ void __launch_bounds__(RT_THREADS) rb_rows(const TL* __restrict__ logits,
                                                      const int32_t* __restrict__ expert_idx,
                                                      const float* __restrict__ alpha,
                                                      const float2* __restrict__ row_stats,
                                                      const float* __restrict__ dgate, const float* __restrict__ f,
                                                      const lrm_router_losses* __restrict__ losses, int T, int E,
                                                      int k, int renorm, float aux_coef, float z_coef,
                                                      TO* __restrict__ dlogits, unsigned int* status) {
  extern __shared__ float rt_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* add = rt_smem + warp * E;  // the gates' part of this warp's row
  for (int e = lane; e < E; e += 32) add[e] = 0.f;
  float fe[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) fe[i] = lane + 32 * i < E ? f[lane + 32 * i] : 0.f;
  const float tokens = static_cast<float>(max(1, losses->tokens));
  const float ca = aux_coef * static_cast<float>(E) / tokens, cz = 2.f * z_coef / tokens;
  __syncwarp();
  const long long step = static_cast<long long>(gridDim.x) * RT_WARPS;
  for (long long t = static_cast<long long>(blockIdx.x) * RT_WARPS + warp; t < T; t += step) {
    TO* out = dlogits + static_cast<size_t>(t) * E;
    const float2 ms = row_stats[t];
    if (ms.y == 0.f) {  // not counted
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < E) store_elem(out + lane + 32 * i, 0.f);
      continue;
    }
    const TL* row = logits + static_cast<size_t>(t) * E;
    const float inv = 1.f / ms.y;
    float p[VPL], fp = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = lane + 32 * i < E ? expf(load_elem(row + lane + 32 * i) - ms.x) * inv : 0.f;
      fp = fmaf(fe[i], p[i], fp);
    }
    fp = warp_sum(fp);
    float S = 0.f;
    int my_e = -1;
    if (dgate != nullptr) {
      const size_t u = static_cast<size_t>(t) * k + lane;
      float dg = 0.f;
      int e = -1 - lane;  // distinct among the lanes
      if (lane < k) {
        const int id = expert_idx[u];
        if (id >= 0 && id < E) e = id, dg = dgate[u];
      }
      const unsigned peers = __match_any_sync(0xffffffffu, e);
      const bool first = (peers & ((1u << lane) - 1u)) == 0;
      if (lane < k && (e < 0 || !first)) raise_flag(status, LRM_ERR_INDEX);
      if (!first) dg = 0.f;
      S = warp_sum(dg);
      if (e >= 0 && first) {
        my_e = e;
        add[e] = renorm ? dg - alpha[u] * S : dg;
      }
      __syncwarp();
    }
    const float zt = cz * (ms.x + logf(ms.y)) - (renorm ? 0.f : S);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E) store_elem(out + e, fmaf(p[i], fmaf(ca, fe[i] - fp, zt), add[e]));
    }
    __syncwarp();
    if (my_e >= 0) add[my_e] = 0.f;
    __syncwarp();
  }
}

struct ForwardArgs {
  const uint8_t* valid;
  lrm_dims d;
  int renorm;
  int32_t* expert_idx;
  float* alpha;
  float2* row_stats;
  float* ws_p;
  int32_t* ws_cnt;
  double* ws_z;
  int32_t* ws_tok;
};

template <typename TL, int VPL>
lrm_status launch_rf(const TL* logits, const ForwardArgs& a, int nblk, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(RT_WARPS + 1) * a.d.E * sizeof(float);
  rf_rows<TL, VPL><<<nblk, RT_THREADS, smem, s>>>(logits, a.valid, a.d.T, a.d.E, a.d.k, a.renorm, a.expert_idx,
                                                  a.alpha, a.row_stats, a.ws_p, a.ws_cnt, a.ws_z, a.ws_tok);
  return launch_status();
}

template <typename TL>
lrm_status dispatch_rf(const void* logits, const ForwardArgs& a, int nblk, cudaStream_t s) {
  const TL* l = static_cast<const TL*>(logits);
  const int vpl = (a.d.E + 31) / 32;
  if (vpl <= 1) return launch_rf<TL, 1>(l, a, nblk, s);
  if (vpl <= 2) return launch_rf<TL, 2>(l, a, nblk, s);
  if (vpl <= 4) return launch_rf<TL, 4>(l, a, nblk, s);
  if (vpl <= 8) return launch_rf<TL, 8>(l, a, nblk, s);
  if (vpl <= 16) return launch_rf<TL, 16>(l, a, nblk, s);
  return launch_rf<TL, 32>(l, a, nblk, s);
}

struct BackwardArgs {
  const int32_t* expert_idx;
  const float* alpha;
  const float2* row_stats;
  const float* dgate;
  const float* f;
  const lrm_router_losses* losses;
  lrm_dims d;
  int renorm;
  float aux_coef, z_coef;
  unsigned int* status;
};

template <typename TL, typename TO, int VPL>
lrm_status launch_rb(const TL* logits, TO* dlogits, const BackwardArgs& a, int grid, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(RT_WARPS) * a.d.E * sizeof(float);
  rb_rows<TL, TO, VPL><<<grid, RT_THREADS, smem, s>>>(logits, a.expert_idx, a.alpha, a.row_stats, a.dgate, a.f,
                                                      a.losses, a.d.T, a.d.E, a.d.k, a.renorm, a.aux_coef, a.z_coef,
                                                      dlogits, a.status);
  return launch_status();
}

template <typename TL, typename TO>
lrm_status dispatch_rb(const void* logits, void* dlogits, const BackwardArgs& a, int grid, cudaStream_t s) {
  const TL* l = static_cast<const TL*>(logits);
  TO* o = static_cast<TO*>(dlogits);
  const int vpl = (a.d.E + 31) / 32;
  if (vpl <= 1) return launch_rb<TL, TO, 1>(l, o, a, grid, s);
  if (vpl <= 2) return launch_rb<TL, TO, 2>(l, o, a, grid, s);
  if (vpl <= 4) return launch_rb<TL, TO, 4>(l, o, a, grid, s);
  if (vpl <= 8) return launch_rb<TL, TO, 8>(l, o, a, grid, s);
  if (vpl <= 16) return launch_rb<TL, TO, 16>(l, o, a, grid, s);
  return launch_rb<TL, TO, 32>(l, o, a, grid, s);
}

bool dtype_ok(int32_t t) { return t == LRM_F32 || t == LRM_BF16; }
// fp32 arrays at 4 bytes, bf16 arrays at 16 (the library's rule)
bool dtype_aligned(const void* p, int32_t t) { return aligned(p, t == LRM_F32 ? 4 : 16); }

}  // namespace

size_t router_workspace_bytes(const lrm_ctx* ctx, const lrm_dims& d) { return router_layout(ctx, d).bytes; }

}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_router_forward(lrm_ctx* ctx, const void* logits, int32_t logits_dtype, const uint8_t* valid,
                                         lrm_dims dims, int32_t renorm, float aux_coef, float z_coef,
                                         int32_t* expert_idx, float* alpha, float* row_stats, int32_t* counts,
                                         float* f, float* P, lrm_router_losses* losses, void* ws, size_t ws_bytes,
                                         void* stream) {
  if (ctx == nullptr) return LRM_ERR_INVALID_ARG;
  lrm_status st = check_dims(dims);
  if (st != LRM_OK) return st;
  if (!dtype_ok(logits_dtype) || renorm < 0 || renorm > 1) return LRM_ERR_INVALID_ARG;
  if (counts == nullptr || f == nullptr || P == nullptr || losses == nullptr) return LRM_ERR_INVALID_ARG;
  if (dims.T > 0 && (logits == nullptr || expert_idx == nullptr || alpha == nullptr || row_stats == nullptr))
    return LRM_ERR_INVALID_ARG;
  if (!dtype_aligned(logits, logits_dtype) || !aligned(row_stats, 8)) return LRM_ERR_ALIGN;
  const void* ptrs[] = {expert_idx, alpha, counts, f, P, losses};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return LRM_ERR_ALIGN;
  const RouterLayout L = router_layout(ctx, dims);
  if (L.nblk > 0 && (ws == nullptr || ws_bytes < L.bytes)) return LRM_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  ForwardArgs a{valid, dims, renorm, expert_idx, alpha, reinterpret_cast<float2*>(row_stats),
                reinterpret_cast<float*>(w + L.p_off), reinterpret_cast<int32_t*>(w + L.cnt_off),
                reinterpret_cast<double*>(w + L.z_off), reinterpret_cast<int32_t*>(w + L.tok_off)};
  if (L.nblk > 0) {
    st = logits_dtype == LRM_F32 ? dispatch_rf<float>(logits, a, L.nblk, s)
                                 : dispatch_rf<__nv_bfloat16>(logits, a, L.nblk, s);
    if (st != LRM_OK) return st;
  }
  rf_sums<<<1, 1024, 0, s>>>(a.ws_p, a.ws_cnt, a.ws_z, a.ws_tok, L.nblk, dims.E, dims.k, aux_coef, z_coef, counts, f,
                             P, losses);
  return launch_status();
}

extern "C" lrm_status lrm_router_backward(lrm_ctx* ctx, const void* logits, int32_t logits_dtype,
                                          const int32_t* expert_idx, const float* alpha, const float* row_stats,
                                          const float* dgate, const float* f, const lrm_router_losses* losses,
                                          lrm_dims dims, int32_t renorm, float aux_coef, float z_coef, void* dlogits,
                                          int32_t dlogits_dtype, void* stream) {
  if (ctx == nullptr) return LRM_ERR_INVALID_ARG;
  lrm_status st = check_dims(dims);
  if (st != LRM_OK) return st;
  if (!dtype_ok(logits_dtype) || !dtype_ok(dlogits_dtype) || renorm < 0 || renorm > 1) return LRM_ERR_INVALID_ARG;
  if (dims.T == 0) return LRM_OK;
  if (logits == nullptr || expert_idx == nullptr || alpha == nullptr || row_stats == nullptr || f == nullptr ||
      losses == nullptr || dlogits == nullptr)
    return LRM_ERR_INVALID_ARG;
  if (!dtype_aligned(logits, logits_dtype) || !dtype_aligned(dlogits, dlogits_dtype) || !aligned(row_stats, 8))
    return LRM_ERR_ALIGN;
  const void* ptrs[] = {expert_idx, alpha, dgate, f, losses};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  BackwardArgs a{expert_idx, alpha, reinterpret_cast<const float2*>(row_stats), dgate, f, losses, dims, renorm,
                 aux_coef, z_coef, ctx->d_status};
  const long long need = (static_cast<long long>(dims.T) + RT_WARPS - 1) / RT_WARPS;
  const int cap = ctx->sm_count * 4;
  const int grid = static_cast<int>(need < cap ? need : cap);
  using bf = __nv_bfloat16;
  if (logits_dtype == LRM_F32)
    return dlogits_dtype == LRM_F32 ? dispatch_rb<float, float>(logits, dlogits, a, grid, s)
                                    : dispatch_rb<float, bf>(logits, dlogits, a, grid, s);
  return dlogits_dtype == LRM_F32 ? dispatch_rb<bf, float>(logits, dlogits, a, grid, s)
                                  : dispatch_rb<bf, bf>(logits, dlogits, a, grid, s);
}
