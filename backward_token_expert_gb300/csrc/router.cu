// The router of the layer: gates and balance loss of a batch of logits, and
// the logits' gradient ("Expert Parallel Math Deep": importance P_e, load f_e
// and the auxiliary loss E sum f_e P_e; the z loss is the mean squared
// log-partition).
//
//   rf_rows    G lanes per token, 4 C logits a lane, so a warp holds 32 / G
//              tokens (E = 128: four; E = 8: eight).
//              The logits are read once, a token ahead.  From the same
//              registers come the maximum, the softmax (summed per lane for
//              P) and the k largest.  Every block leaves its sums of p, its
//              counts, its sum of lse^2 and its counted tokens in the
//              workspace.
//   rf_sums    one cluster adds the blocks' sums in a fixed order and writes
//              counts, f, P and the losses; launched dependently, so that
//              only its work and not its launch follows rf_rows.  A batch of
//              one block is finished inside rf_rows.
//   rb_rows    the same lanes: p again from the saved (max, sum), the balance
//              term needs sum_e f_e p_e over the row, and the gates' part
//              touches k experts, which are placed through shared memory.
//
// The k largest: a lane sorts its logits as 32-bit keys whose top bits order
// like the value and whose low bits hold the expert, inverted, so that
// keys are unique and equal values go to the lower expert.  Few slots are
// found by rounds of a group-wide maximum, the lane that owns it moving up its
// list; more by merging the lanes' lists of eight pairwise.  For bf16 logits the
// cut-off bits are zero and the order is exact.  For fp32 the keys are made of
// l - m, and the order is checked against the logits: where a logit left out has a
// key that agrees with the last slot's in all the bits kept, the logits up to the
// last slot are counted; more than k of them, slots out of order, NaN and rows of
// -inf send the warp to an exact selection on full keys (131072 x 128, k = 8:
// random logits 35 us, logits of bf16 precision, where ties abound, 38 us, all
// logits equal 44 us; 53 and 82 without the count).
//
// The forward is bound by instruction issue: 131072 x 128 fp32 logits take 35 us,
// of which the 77 MB to move need 11; 32768 x 128 take 16 us, half of it launch,
// first load and rf_sums.  The backward is bound by memory: 131072 x 128 fp32 in
// 25 us, 5.8 TB/s.
#include <math.h>

#include <type_traits>

#include "lrm_internal.cuh"
#include "vec.cuh"

namespace lrm {
namespace {

constexpr int RF_ONE_BLOCK_PASSES = 2;  // batches of up to this many passes of one block use one block
// Up to this k, and above 8, the slots are found by rounds of a maximum, between
// them by merging the lanes' lists of eight (131072 x 128, rounds against merges: k = 2 28.7 / 32.5 us,
// k = 4 31.2 / 33.2, k = 8 37.4 / 34.3).
constexpr int RF_ROUNDS = 4;
constexpr int RS_SUM_THREADS = 1024;
constexpr int RB_THREADS = 128;  // 131072 x 128 fp32: 24.8 us; measured when it was 25.3: blocks of 256 26.5, of 512 27.2
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// Lanes per token (G) and groups of four logits per lane (C): the fewest lanes
// that have a slot each and at most 16 logits (32 for the widest layers), so
// that what a token costs once (reductions, slots, addresses) is shared by the
// tokens of a warp.  From 8 lanes on C is 1, 2, 3 or 4: three groups where two do not reach and
// four would be a quarter empty (65536 tokens, k = 6, forward / backward with three and with four:
// E = 96 fp32 19.1 / 11.6 and 21.2 / 11.8 us, bf16 16.8 / 7.9 and 19.0 / 8.5; E = 160 fp32 32.3 / 18.0
// and 36.3 / 18.3, bf16 29.6 / 14.1 and 33.7 / 16.0; E = 384 fp32 44.3 / 33.8 and 51.0 / 35.6, bf16
// 44.9 / 25.6 and 52.9 / 28.4).  At E = 128 a warp a token took 346 instructions a token in
// the forward (45 us for 131072 tokens) and 31.3 us in the backward; four tokens a
// warp take 175 (37 us; 35 with merged lists) and 25 us.
template <int N>
using Int = std::integral_constant<int, N>;

struct Split {
  int G, C;
};
constexpr Split kSplits[] = {{4, 1}, {8, 1}, {8, 2}, {8, 3}, {8, 4}, {16, 1}, {16, 2}, {16, 3}, {16, 4},
                              {32, 1}, {32, 2}, {32, 3}, {32, 4}, {32, 8}};
Split split_of(int E, int k) {
  for (const Split& s : kSplits)
    if (E <= 4 * s.G * s.C && k <= s.G) return s;
  return {32, 8};
}

// Calls run(std::integral_constant...) with the layer's G and C.
template <typename Run>
lrm_status with_split(int E, int k, Run run) {
  const Split s = split_of(E, k);
  const auto pick = [&](auto g, auto c) { return run(g, c); };
  switch (s.G * 16 + s.C) {
    case 4 * 16 + 1: return pick(Int<4>{}, Int<1>{});
    case 8 * 16 + 1: return pick(Int<8>{}, Int<1>{});
    case 8 * 16 + 2: return pick(Int<8>{}, Int<2>{});
    case 8 * 16 + 3: return pick(Int<8>{}, Int<3>{});
    case 8 * 16 + 4: return pick(Int<8>{}, Int<4>{});
    case 16 * 16 + 1: return pick(Int<16>{}, Int<1>{});
    case 16 * 16 + 2: return pick(Int<16>{}, Int<2>{});
    case 16 * 16 + 3: return pick(Int<16>{}, Int<3>{});
    case 16 * 16 + 4: return pick(Int<16>{}, Int<4>{});
    case 32 * 16 + 1: return pick(Int<32>{}, Int<1>{});
    case 32 * 16 + 2: return pick(Int<32>{}, Int<2>{});
    case 32 * 16 + 3: return pick(Int<32>{}, Int<3>{});
    case 32 * 16 + 4: return pick(Int<32>{}, Int<4>{});
  }
  return pick(Int<32>{}, Int<8>{});
}

// Threads of a block of rf_rows, one block an SM: as many as the registers of C
// groups allow (three instantiations of C = 4 spill one to three of them).  640
// threads of 96 registers at C = 4 gain 1 % at 131072 x 128 and lose 10 % at
// 16384 x 128; blocks sized to the batch, so that a small one has a warp on every
// SM, lose 4 % at 8192 x 128: rf_sums then adds more rows.
__host__ __device__ constexpr int rf_threads(int C) { return C == 1 ? 768 : C <= 4 ? 512 : 256; }

struct RouterLayout {
  int nblk;  // blocks of rf_rows
  size_t p_off, cnt_off, z_off, tok_off, bytes;
};

RouterLayout router_layout(const lrm_ctx* ctx, const lrm_dims& d) {
  RouterLayout L;
  const Split sp = split_of(d.E, d.k);
  const long long pass = rf_threads(sp.C) / sp.G;  // tokens of a block in flight
  long long need = (static_cast<long long>(d.T) + pass - 1) / pass;
  if (need <= RF_ONE_BLOCK_PASSES) need = need > 0 ? 1 : 0;
  const long long cap = ctx->sm_count;
  L.nblk = static_cast<int>(need < cap ? need : cap);
  const size_t cells = static_cast<size_t>(L.nblk) * d.E;
  L.p_off = 0;
  L.cnt_off = L.p_off + cells * sizeof(float);
  L.z_off = (L.cnt_off + cells * sizeof(int32_t) + 15) / 16 * 16;
  L.tok_off = L.z_off + L.nblk * sizeof(float);
  L.bytes = L.tok_off + L.nblk * sizeof(int32_t);
  return L;
}

// ---------------------------------------------------------------------------
// elements

template <typename T>
constexpr bool is_bf16 = sizeof(T) == 2;

__device__ __forceinline__ float load_elem(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_elem(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four consecutive logits as they lie in memory.  load() leaves the places
// beyond the row as they are: -inf, from clear().  V: the elements that rows
// start at a multiple of, 4, 2 or 1 (bf16 backward of 80000 x 210: 22.7 us in
// pairs, 38.9 one by one).
template <typename TL>
struct Four {
  uint32_t w[sizeof(TL)];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(TL)); ++i) w[i] = is_bf16<TL> ? 0xFF80FF80u : 0xFF800000u;
  }
  template <int V>
  __device__ __forceinline__ void load(const TL* __restrict__ row, int e0, int E) {
#pragma unroll
    for (int i = 0; i < 4; i += V) {
      if (e0 + i >= E) continue;
      const TL* p = row + e0 + i;
      if constexpr (V == 4 && is_bf16<TL>) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = x.x;
        w[1] = x.y;
      } else if constexpr (V == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        w[3] = x.w;
      } else if constexpr (V == 2 && is_bf16<TL>) {
        w[i / 2] = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else if constexpr (V == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
        w[i] = x.x;
        w[i + 1] = x.y;
      } else if constexpr (is_bf16<TL>) {
        const uint32_t x = __ldg(reinterpret_cast<const uint16_t*>(p));
        w[i / 2] = (i & 1) ? (w[i / 2] & 0xFFFFu) | x << 16 : (w[i / 2] & 0xFFFF0000u) | x;
      } else {
        w[i] = __float_as_uint(__ldg(reinterpret_cast<const float*>(p)));
      }
    }
  }
};

// A lane's logits: C groups of four, G groups apart, so that
// the lanes of a token read consecutive 16-byte pieces.
template <typename TL, int G, int C>
struct Pieces {
  Four<TL> f[C];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int c = 0; c < C; ++c) f[c].clear();
  }
  template <int V>
  __device__ __forceinline__ void load_by(const TL* __restrict__ row, int q, int E) {
#pragma unroll
    for (int c = 0; c < C; ++c) f[c].template load<V>(row, 4 * (q + G * c), E);
  }
  __device__ __forceinline__ void load(const TL* __restrict__ row, int q, int E, int vec) {
    if (vec == 4)
      load_by<4>(row, q, E);
    else if (vec == 2)
      load_by<2>(row, q, E);
    else
      load_by<1>(row, q, E);
  }
  __device__ __forceinline__ float get(int c, int i) const {
    if constexpr (is_bf16<TL>)
      return (i & 1) ? bf16_hi(f[c].w[i / 2]) : bf16_lo(f[c].w[i / 2]);
    else
      return __uint_as_float(f[c].w[i]);
  }
};

template <typename TO>
__device__ __forceinline__ void store_four(TO* __restrict__ row, int e0, int E, int vec, const float (&v)[4]) {
  if (vec == 4) {
    if (e0 >= E) return;
    if constexpr (is_bf16<TO>) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(row + e0) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      *reinterpret_cast<float4*>(row + e0) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else if (vec == 2) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      if (e0 + i >= E) continue;
      if constexpr (is_bf16<TO>)
        *reinterpret_cast<__nv_bfloat162*>(row + e0 + i) = __floats2bfloat162_rn(v[i], v[i + 1]);
      else
        *reinterpret_cast<float2*>(row + e0 + i) = make_float2(v[i], v[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < E) store_elem(row + e0 + i, v[i]);
  }
}

// e^x for x <= 0 as 2^(x log2 e): the product's rounding is 2^-24 |x| log2 e in
// the exponent and the constant's 1.3e-8 |x| log2 e, so the relative error is up to
// 7.3e-8 |x| + 2 ulp, largest where the term itself is smallest; results below
// 2^-126 are 0.
__device__ __forceinline__ float exp_neg(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * LOG2E));
  return r;
}

// ---------------------------------------------------------------------------
// keys and group reductions

// A key that orders like the value (-0 like +0; NaN has no place).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// The value of a key that holds at least its upper 16 bits, a bf16's.
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key ^ (static_cast<int32_t>(key) < 0 ? 0x80000000u : 0xffffffffu)) & 0xffff0000u);
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The group's largest value, NaN left out unless there is nothing else.
template <int G>
__device__ __forceinline__ float group_fmax(float v) {
  if constexpr (G == 32) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (G == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum over a group whose lanes from k on hold 0, valid in the lanes below k.
template <int G>
__device__ __forceinline__ float slot_sum(float v, int k) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1)
    if (o < k) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Descending sort of a lane's keys: Batcher's odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&a)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int k = p; k >= 1; k /= 2) {
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(a[i + j], a[i + j + k]), lo = min(a[i + j], a[i + j + k]);
            a[i + j] = hi;
            a[i + j + k] = lo;
          }
        }
      }
    }
  }
}

// a: the eight largest of two descending lists of eight, descending.  The
// larger of a[i] and b[7 - i] are those eight, as a bitonic list.
__device__ __forceinline__ void merge_top8(uint32_t* a, const uint32_t* b) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
#pragma unroll
  for (int d = 4; d >= 1; d /= 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i & d) == 0) {
        const uint32_t hi = max(a[i], a[i + d]), lo = min(a[i], a[i + d]);
        a[i] = hi;
        a[i + d] = lo;
      }
    }
  }
}

// The keys' LIST largest in front, descending.
template <int N, int LIST>
__device__ __forceinline__ void sort_top(uint32_t (&a)[N]) {
  if constexpr (LIST >= N) {
    sort_desc(a);
  } else {
    static_assert(LIST == 8 && N % 8 == 0, "lists of eight");
#pragma unroll
    for (int b = 0; b < N / 8; ++b) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a[8 * b + i];
      sort_desc(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[8 * b + i] = v[i];
      if (b > 0) merge_top8(a, a + 8 * b);
    }
  }
}

// Whether no more than k of the token's logits come before or at the last slot's
// (v, e): larger, or equal in an expert up to e.  Slots in order are then the k
// largest.
template <typename TL, int G, int C>
__device__ __noinline__ bool is_last(const TL* row, int E, int k, int vec, float v, int e) {
  const int q = threadIdx.x % G;
  Pieces<TL, G, C> raw;
  raw.clear();
  raw.load(row, q, E, vec);
  int n = 0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = raw.get(c, i);
      n += x > v || (x == v && 4 * (q + G * c) + i <= e);
    }
#pragma unroll
  for (int o = 1; o < G; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n == k;
}

// The exact selection: k rounds over full keys, NaN below -inf, equal keys to
// the lower expert.  Returns slot q's expert.
template <typename TL, int G, int C>
__device__ __noinline__ int select_exact(const TL* row, int E, int k, int vec) {
  const int lane = threadIdx.x & 31, q = lane % G;
  Pieces<TL, G, C> raw;
  raw.clear();
  raw.load(row, q, E, vec);
  uint32_t key[C][4];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = raw.get(c, i);
      key[c][i] = 4 * (q + G * c) + i >= E ? 0u : v != v ? 1u : order_key(v);
    }
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (key[c][i] > best) best = key[c][i], at = 4 * (q + G * c) + i;
    const uint32_t top = group_max<G>(best);
    const int e = static_cast<int>(~group_max<G>(best == top ? ~static_cast<uint32_t>(at) : 0u));
    if (q == j) mine = e;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * (q + G * c) + i == e) key[c][i] = 0u;
  }
  return mine;
}

// ---------------------------------------------------------------------------
// forward

struct ForwardArgs {
  const uint8_t* valid;
  int T, E, k, renorm;
  float aux_coef, z_coef;
  int32_t* expert_idx;
  float* alpha;
  float2* row_stats;
  float* ws_p;
  int32_t* ws_cnt;
  float* ws_z;
  int32_t* ws_tok;
  int32_t* counts;
  float *f, *P;
  lrm_router_losses* losses;
};

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void st_cluster_f32(const float* p, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(p, rank)), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float warp_sum(float v) { return group_sum<32>(v); }

// counts, P and f of expert e from its sums; returns f P.
__device__ __forceinline__ float write_expert(const ForwardArgs& a, int e, float p, int c, int tokens) {
  const float Pe = tokens > 0 ? __fdiv_rn(p, static_cast<float>(tokens)) : 0.f;
  const long long pairs = static_cast<long long>(tokens) * a.k;
  float fe = 0.f;
  if (tokens > 0)  // correctly rounded: fp32 holds integers up to 2^24
    fe = pairs <= (1 << 24) ? __fdiv_rn(static_cast<float>(c), static_cast<float>(pairs))
                            : static_cast<float>(static_cast<double>(c) / static_cast<double>(pairs));
  a.counts[e] = c;
  a.P[e] = Pe;
  a.f[e] = fe;
  return fe * Pe;
}

__device__ __forceinline__ void write_losses(const ForwardArgs& a, float fp, float z, int tokens) {
  lrm_router_losses r;
  r.aux = static_cast<float>(a.E) * fp;
  r.z = tokens > 0 ? __fdiv_rn(z, static_cast<float>(tokens)) : 0.f;
  r.loss = fmaf(a.aux_coef, r.aux, a.z_coef * r.z);
  r.tokens = tokens;
  *a.losses = r;
}

// Adds nblk blocks' sums.  The cluster's CTAs share the experts; a warp adds
// every 32nd row of 32 experts, then warp w the warps' sums of the w-th
// expert.  The CTAs push their sums of f P to CTA 0.
__global__ void __launch_bounds__(RS_SUM_THREADS) rf_sums(ForwardArgs a, int nblk) {
  constexpr int NW = RS_SUM_THREADS / 32, BATCH = 5;  // rows a warp has in flight: all of 152 blocks
  __shared__ float s_p[NW][33];
  __shared__ int s_c[NW][33];
  __shared__ float s_fp[NW];
  __shared__ float s_total[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), ranks = static_cast<int>(cluster_nctarank());
  const int per = (a.E + ranks - 1) / ranks;
  const int e0 = min(a.E, rank * per), e1 = min(a.E, e0 + per);
  if (ranks > 1) cluster_arrive();  // waited for before the push: CTA 0 has started by then
  grid_dependency_wait();
  float z = 0.f, fp = 0.f;
  int tokens = 0;
  for (int b = lane; b < nblk; b += 32) z += __ldcg(a.ws_z + b), tokens += __ldcg(a.ws_tok + b);
  for (int c0 = e0; c0 < e1; c0 += 32) {
    const int e = c0 + lane;
    float p = 0.f;
    int c = 0;
    for (int b0 = warp; b0 < nblk; b0 += BATCH * NW) {
      float pv[BATCH];
      int cv[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const int b = b0 + j * NW;
        const bool in = b < nblk && e < e1;
        pv[j] = in ? __ldcg(a.ws_p + static_cast<size_t>(b) * a.E + e) : 0.f;
        cv[j] = in ? __ldcg(a.ws_cnt + static_cast<size_t>(b) * a.E + e) : 0;
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) p += pv[j], c += cv[j];
    }
    if (c0 == e0) {
      z = warp_sum(z);
      tokens = __reduce_add_sync(0xffffffffu, tokens);
    }
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    __syncthreads();
    p = warp_sum(s_p[lane][warp]);
    c = __reduce_add_sync(0xffffffffu, s_c[lane][warp]);
    if (c0 + warp < e1 && lane == 0) fp += write_expert(a, c0 + warp, p, c, tokens);
    __syncthreads();
  }
  if (lane == 0) s_fp[warp] = fp;
  __syncthreads();
  if (warp == 0) fp = warp_sum(s_fp[lane]);
  if (ranks > 1) {
    cluster_wait();
    if (rank != 0 && threadIdx.x == 0) st_cluster_f32(&s_total[rank], 0, fp);
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
    if (warp == 0) fp = warp_sum(lane == 0 ? fp : lane < ranks ? s_total[lane] : 0.f);
  }
  if (threadIdx.x == 0) write_losses(a, fp, z, tokens);
}

template <typename TL, int G, int C>
__global__ void __launch_bounds__(rf_threads(C), 1) rf_rows(const TL* __restrict__ logits, ForwardArgs a, int vec) {
  constexpr int NT = rf_threads(C), NW = NT / 32, PER_WARP = 32 / G, N = 4 * C;
  constexpr int NK = C == 3 ? 16 : N;    // keys of a lane, a power of two
  // those it keeps for the selection, more slots than that included (80000 x 208, k = 12: 55 us, 80 with lists of 16)
  constexpr int LIST = NK < 8 ? NK : 8;
  constexpr uint32_t LOW = G * NK - 1;  // the key's bits that hold the expert
  extern __shared__ float rt_smem[];
  float* sp = rt_smem;                                     // [NW][E]
  int* hist = reinterpret_cast<int*>(rt_smem + NW * a.E);  // [E]
  __shared__ __align__(16) uint32_t s_sel[NW][32];                     // the slots' keys
  __shared__ float s_z[NW];
  __shared__ int s_tok[NW];
  __shared__ float s_fp[NW];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = lane % G;
  const int T = a.T, E = a.E, k = a.k;
  uint32_t* sel = s_sel[warp] + (lane - q);
  grid_dependency_launch();
  for (int i = tid; i < E; i += NT) hist[i] = 0;
  __syncthreads();

  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  // (m, s) of the group's counted tokens are kept a lane each until G are there
  float z = 0.f, km = 0.f, ks = 1.f;
  int held = 0, tokens = 0;
  const long long step = static_cast<long long>(gridDim.x) * NW * PER_WARP;
  long long t = (static_cast<long long>(blockIdx.x) * NW + warp) * PER_WARP + lane / G;
  // a group without a token of its own (here false) reads a row that another has
  const TL* next_row = logits + static_cast<size_t>(t < T ? t : 0) * E;
  const size_t row_step = static_cast<size_t>(step) * E;
  Pieces<TL, G, C> next;
  next.clear();
  if (T > 0) next.load(next_row, q, E, vec);
  for (; t - lane / G < T; t += step) {
    const bool here = G == 32 || t < T;
    const TL* row = next_row;
    const Pieces<TL, G, C> raw = next;
    if (t + step < T) next_row += row_step;
    next.load(next_row, q, E, vec);
    bool ok = here;
    if (a.valid != nullptr && here) ok = a.valid[t] != 0;

    float m = raw.get(0, 0);
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, raw.get(i / 4, i % 4));
    m = group_fmax<G>(m);
    // -0 takes both zeros to d = +0, so that they tie
    const float base = m == -INFINITY ? 0.f : m == 0.f ? -0.f : m;
    uint32_t key[NK] = {};
    float p[N], s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = raw.get(i / 4, i % 4), d = v - base;  // <= 0: the larger its bits, the smaller it is
      const uint32_t order = is_bf16<TL> ? order_key(v) : ~__float_as_uint(d);
      key[i] = (order & ~LOW) | (LOW - static_cast<uint32_t>(4 * (q + G * (i / 4)) + i % 4));
      p[i] = exp_neg(d);
      s += p[i];
    }
    s = group_sum<G>(s);
    const bool counted = ok && s != 0.f;

    sort_top<NK, LIST>(key);
    bool crowded = false;  // a logit left out may be larger than the last one kept
    if (LIST == 8 && G <= 16 && k > RF_ROUNDS && (G <= LIST || k <= LIST)) {
      // the lanes' lists merged pairwise: every lane ends with the token's eight largest
      uint32_t own[LIST];
#pragma unroll
      for (int i = 0; i < LIST; ++i) own[i] = key[i];
      if constexpr (LIST == 8 && G <= 16) {  // (the condition above, for the compiler)
#pragma unroll
        for (int o = 1; o < G; o <<= 1) {
          uint32_t other[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(0xffffffffu, key[i], o);
          merge_top8(key, other);
        }
        if (q == 0) {
          *reinterpret_cast<uint4*>(sel) = make_uint4(key[0], key[1], key[2], key[3]);
          *reinterpret_cast<uint4*>(sel + 4) = make_uint4(key[4], key[5], key[6], key[7]);
        }
      }
      __syncwarp();
      if constexpr (!is_bf16<TL>) {
        const uint32_t last = sel[k - 1] & ~LOW;
        int n = 0;
#pragma unroll
        for (int i = 0; i < LIST; ++i) n += own[i] >= last;
        crowded = NK > LIST && n == LIST;
#pragma unroll
        for (int o = 1; o < G; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        crowded = crowded || n != k;
      }
    } else {
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        const uint32_t top = group_max<G>(key[0]);
        const bool hit = key[0] == top;
        if (hit) sel[j] = top;
#pragma unroll
        for (int i = 0; i + 1 < LIST; ++i) key[i] = hit ? key[i + 1] : key[i];
        key[LIST - 1] = hit ? 0u : key[LIST - 1];
      }
      __syncwarp();
      // a lane whose list ran out may hold more (with 16 lanes and 16 random slots one token in 30000)
      if constexpr (!is_bf16<TL>)
        crowded = (sel[k - 1] ^ group_max<G>(key[0])) <= LOW || (NK > LIST && key[0] == 0u);
      else
        crowded = NK > LIST && k > LIST && key[0] == 0u;
    }
    const bool slot = q < k && here;
    const uint32_t mine = sel[q];
    int e = min(static_cast<int>(LOW - (mine & LOW)), E - 1);
    float v = 0.f;
    if constexpr (is_bf16<TL>)
      v = key_value(mine);  // saves a dependent load: 65536 x 256, k = 8: 34.7 -> 34.0 us
    else if (slot)
      v = load_elem(row + e);
    if constexpr (!is_bf16<TL>) {
      if (__any_sync(0xffffffffu, crowded && here)) {
        const int at = lane - q + k - 1;
        crowded = !is_last<TL, G, C>(row, E, k, vec, __shfl_sync(0xffffffffu, v, at), __shfl_sync(0xffffffffu, e, at));
      }
    }
    bool unclear = here && (crowded || !(s > 0.f));
    if constexpr (!is_bf16<TL>) {
      const float vn = __shfl_down_sync(0xffffffffu, v, 1, G);
      unclear = unclear || (q < k - 1 && here && v < vn);
    }
    if (__any_sync(0xffffffffu, unclear)) {
      e = select_exact<TL, G, C>(row, E, k, vec);
      if (slot) v = load_elem(row + e);
    }
    __syncwarp();  // sel is read before the next token writes it

    const float pj = slot ? exp_neg(v - base) : 0.f;
    const float den = a.renorm ? slot_sum<G>(pj, k) : s;
    if (slot) {
      const size_t u = static_cast<size_t>(t) * k + q;
      a.expert_idx[u] = e;
      a.alpha[u] = counted ? pj * rcp(den) : 0.f;
      if (counted) atomicAdd(&hist[e], 1);
    }
    if (q == 0 && here) a.row_stats[t] = counted ? make_float2(base + 0.f, s) : make_float2(0.f, 0.f);
    if (counted) {
      const float inv = rcp(s);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(p[i], inv, acc[i]);
      if (q == held) km = base, ks = s;
      ++tokens;
      if (++held == G) {
        const float lse = km + logf(ks);
        z = fmaf(lse, lse, z);
        held = 0;
      }
    }
  }
  if (q < held) {
    const float lse = km + logf(ks);
    z = fmaf(lse, lse, z);
  }

  // the block's sums, in a fixed order
  z = warp_sum(z);
  tokens = __reduce_add_sync(0xffffffffu, q == 0 ? tokens : 0);
  if (lane == 0) s_z[warp] = z, s_tok[warp] = tokens;
#pragma unroll
  for (int o = G; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  }
  if (lane < G) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = 4 * (q + G * (i / 4)) + i % 4;
      if (e < E) sp[warp * E + e] = acc[i];
    }
  }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  z = warp_sum(lane < NW ? s_z[lane] : 0.f);
  tokens = __reduce_add_sync(0xffffffffu, lane < NW ? s_tok[lane] : 0);
  float fp = 0.f;
  for (int e = tid; e < E; e += NT) {
    float own = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) own += sp[w * E + e];
    if (alone) {
      fp += write_expert(a, e, own, hist[e], tokens);
    } else {
      a.ws_p[static_cast<size_t>(blockIdx.x) * E + e] = own;
      a.ws_cnt[static_cast<size_t>(blockIdx.x) * E + e] = hist[e];
    }
  }
  if (!alone) {
    if (tid == 0) a.ws_z[blockIdx.x] = z, a.ws_tok[blockIdx.x] = tokens;
    return;
  }
  fp = warp_sum(fp);
  if (lane == 0) s_fp[warp] = fp;
  __syncthreads();
  if (warp == 0) {
    fp = warp_sum(lane < NW ? s_fp[lane] : 0.f);
    if (lane == 0) write_losses(a, fp, z, tokens);
  }
}

// ---------------------------------------------------------------------------
// backward

struct BackwardArgs {
  const int32_t* expert_idx;
  const float* alpha;
  const float2* row_stats;
  const float* dgate;
  const float* f;
  const lrm_router_losses* losses;
  int T, E, k, renorm;
  float aux_coef, z_coef;
  unsigned int* status;
};

// What a lane reads of one token.
template <typename TL, int G, int C>
struct TokenIn {
  Pieces<TL, G, C> raw;
  float2 ms;  // (max, sum); sum 0: not counted
  int id;
  float dg, al;
};

template <typename TL, typename TO, int G, int C>
__global__ void __launch_bounds__(RB_THREADS) rb_rows(const TL* __restrict__ logits, TO* __restrict__ dlogits,
                                                      BackwardArgs a, int vec_in, int vec_out) {
  constexpr int NW = RB_THREADS / 32, PER_WARP = 32 / G;
  __shared__ float4 s_add[NW][32 * C];         // the gates' part of the warp's tokens
  __shared__ uint8_t s_slot[NW][32 * 4 * C];   // the slot that named an expert last
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane % G;
  const int T = a.T, E = a.E, k = a.k;
  float4* own = s_add[warp] + (lane - q) * C + q;  // the group's row, at the lane's first piece
  float* add = reinterpret_cast<float*>(s_add[warp] + (lane - q) * C);
  uint8_t* slot_of = s_slot[warp] + (lane - q) * C * 4;
  const bool gates = a.dgate != nullptr;
  const long long step = static_cast<long long>(gridDim.x) * NW * PER_WARP;
  long long t = (static_cast<long long>(blockIdx.x) * NW + warp) * PER_WARP + lane / G;
  const bool slot = gates && q < k;
  // a group without a token of its own reads the first one's and stores nothing
  const auto load = [&](TokenIn<TL, G, C>& x, long long at) {
    const bool in = at < T;
    const long long from = in ? at : 0;
    x.raw.load(logits + static_cast<size_t>(from) * E, q, E, vec_in);
    x.ms = __ldg(a.row_stats + from);
    if (slot) {
      const size_t u = static_cast<size_t>(from) * k + q;
      x.id = __ldg(a.expert_idx + u);
      x.dg = __ldg(a.dgate + u);
      x.al = __ldg(a.alpha + u);
    }
  };
  TokenIn<TL, G, C> next;
  next.raw.clear();
  next.ms = make_float2(0.f, 0.f);
  next.id = -1;
  next.dg = next.al = 0.f;
  load(next, t);  // before the rest of the set-up, which it hides: 32768 x 128 fp32 8.7 -> 8.2 us
#pragma unroll
  for (int c = 0; c < C; ++c) own[c * G] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float tc = static_cast<float>(max(1, a.losses->tokens));
  const float ca = a.aux_coef * static_cast<float>(E) / tc, cz = 2.f * a.z_coef / tc;
  float cf[C][4];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * (q + G * c) + i;
      cf[c][i] = e < E ? ca * a.f[e] : 0.f;
    }
  __syncwarp();

  for (; t - lane / G < T; t += step) {
    const TokenIn<TL, G, C> x = next;
    load(next, t + step);
    const bool counted = x.ms.y != 0.f;
    const bool rare = __any_sync(0xffffffffu, !counted);  // a token of the warp that gets zeros, or none
    const float inv = rcp(x.ms.y);
    float p[C][4], dg = x.dg;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) p[c][i] = exp_neg(x.raw.get(c, i) - x.ms.x) * inv;
    int e = x.id;  // -1 in lanes without a slot
    if (rare && !counted) {
      e = -1;
      dg = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[c][i] = 0.f;
    }
    float fp = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) fp = fmaf(cf[c][i], p[c][i], fp);
    if (gates) {
      const bool in = static_cast<unsigned>(e) < static_cast<unsigned>(E);
      if (in) slot_of[e] = static_cast<uint8_t>(q);
      __syncwarp();
      const bool lost = in && slot_of[e] != q, bad = !in && slot && counted;
      if (__any_sync(0xffffffffu, bad || lost)) {  // an id out of range, or one named by several slots
        const unsigned peers = __match_any_sync(0xffffffffu, in ? ((lane - q) << 16) | e : -1 - lane);
        if (bad || (in && (peers & ((1u << lane) - 1u)) != 0)) {
          raise_flag(a.status, LRM_ERR_INDEX);
          e = -1;
          dg = 0.f;
        }
      }
      if (a.renorm) {
        const float S = slot_sum<G>(dg, k);
        if (e >= 0) add[e] = fmaf(-x.al, S, dg);
      } else {
        fp += dg;  // p_e takes off S = sum dg like the balance term's sum
        if (e >= 0) add[e] = dg;
      }
      __syncwarp();
    }
    float w = -group_sum<G>(fp);
    if (cz != 0.f) w = counted ? fmaf(cz, x.ms.x + __log2f(x.ms.y) * LN2, w) : 0.f;
    TO* row = dlogits + static_cast<size_t>(t) * E;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float4 g = own[c * G];
      float out[4];
      out[0] = fmaf(p[c][0], cf[c][0] + w, g.x);
      out[1] = fmaf(p[c][1], cf[c][1] + w, g.y);
      out[2] = fmaf(p[c][2], cf[c][2] + w, g.z);
      out[3] = fmaf(p[c][3], cf[c][3] + w, g.w);
      if (rare && !counted) out[0] = out[1] = out[2] = out[3] = 0.f;
      if (t < T) store_four<TO>(row, 4 * (q + G * c), E, vec_out, out);
    }
    __syncwarp();
    if (e >= 0) add[e] = 0.f;
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// launches

template <typename TL, int G, int C>
lrm_status launch_rf(const TL* logits, const ForwardArgs& a, int nblk, int vec, cudaStream_t s) {
  constexpr int NT = rf_threads(C);
  const size_t smem = static_cast<size_t>(NT / 32 + 1) * a.E * sizeof(float);
  rf_rows<TL, G, C><<<nblk, NT, smem, s>>>(logits, a, vec);
  return launch_status();
}

// The elements of a group that every row starts on the bytes of.
template <typename T>
int rows_vec(const T* p, int E) {
  return E % 4 == 0 && aligned(p, 4 * sizeof(T)) ? 4 : E % 2 == 0 && aligned(p, 2 * sizeof(T)) ? 2 : 1;
}

template <typename TL>
lrm_status dispatch_rf(const void* logits, const ForwardArgs& a, int nblk, cudaStream_t s) {
  const TL* l = static_cast<const TL*>(logits);
  const int vec = rows_vec(l, a.E);
  return with_split(a.E, a.k, [&](auto g, auto c) {
    return launch_rf<TL, decltype(g)::value, decltype(c)::value>(l, a, nblk, vec, s);
  });
}

template <typename TL, typename TO, int G, int C>
lrm_status launch_rb(lrm_ctx* ctx, const TL* logits, TO* dlogits, const BackwardArgs& a, cudaStream_t s) {
  static thread_local int dev = -1, grid = 0;
  if (dev != ctx->device) {
    grid = resident_grid(ctx, rb_rows<TL, TO, G, C>, RB_THREADS, 0);
    dev = ctx->device;
  }
  const long long pass = RB_THREADS / G, need = (a.T + pass - 1) / pass;
  rb_rows<TL, TO, G, C><<<static_cast<int>(need < grid ? need : grid), RB_THREADS, 0, s>>>(
      logits, dlogits, a, rows_vec(logits, a.E), rows_vec(dlogits, a.E));
  return launch_status();
}

template <typename TL, typename TO>
lrm_status dispatch_rb(lrm_ctx* ctx, const void* logits, void* dlogits, const BackwardArgs& a, cudaStream_t s) {
  return with_split(a.E, a.k, [&](auto g, auto c) {
    return launch_rb<TL, TO, decltype(g)::value, decltype(c)::value>(ctx, static_cast<const TL*>(logits),
                                                                      static_cast<TO*>(dlogits), a, s);
  });
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
  ForwardArgs a{valid, dims.T, dims.E, dims.k, renorm, aux_coef, z_coef, expert_idx, alpha,
                reinterpret_cast<float2*>(row_stats), reinterpret_cast<float*>(w + L.p_off),
                reinterpret_cast<int32_t*>(w + L.cnt_off), reinterpret_cast<float*>(w + L.z_off),
                reinterpret_cast<int32_t*>(w + L.tok_off), counts, f, P, losses};
  if (L.nblk > 0) {
    st = logits_dtype == LRM_F32 ? dispatch_rf<float>(logits, a, L.nblk, s)
                                 : dispatch_rf<__nv_bfloat16>(logits, a, L.nblk, s);
    if (st != LRM_OK || L.nblk == 1) return st;
  }
  const int cluster = dims.E > 128 ? 8 : dims.E > 64 ? 4 : dims.E > 32 ? 2 : 1;
  return launch_dependent(rf_sums, cluster, RS_SUM_THREADS, 0, cluster, s, a, L.nblk);
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
  const BackwardArgs a{expert_idx, alpha, reinterpret_cast<const float2*>(row_stats), dgate, f, losses, dims.T,
                       dims.E, dims.k, renorm, aux_coef, z_coef, ctx->d_status};
  using bf = __nv_bfloat16;
  if (logits_dtype == LRM_F32)
    return dlogits_dtype == LRM_F32 ? dispatch_rb<float, float>(ctx, logits, dlogits, a, s)
                                    : dispatch_rb<float, bf>(ctx, logits, dlogits, a, s);
  return dlogits_dtype == LRM_F32 ? dispatch_rb<bf, float>(ctx, logits, dlogits, a, s)
                                  : dispatch_rb<bf, bf>(ctx, logits, dlogits, a, s);
}
