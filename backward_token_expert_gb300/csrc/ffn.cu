// Forward of the routed experts: the gated feed-forward block
//   up    [a | b] = W1_e x_t, phi_u = silu(a) b       (lrm_ffn_up, one kernel)
//   down  row_u = W_e phi_u                           (lrm_ffn_down)
//   y_t = sum over the k pairs u of t of alpha_u row_u (lrm_ffn_combine)
// for the pairs u = t k + j of every expert's segment of `ids`.
//
// Both products are one kernel template: persistent clusters of one CTA pair, whose
// even CTA issues tcgen05.mma.cta_group::2 with M = 256 rows of the weight and N =
// up to 256 pairs of the routing (fp32 accumulators in TMEM, double-buffered), K
// blocks of 64.  The routed pairs are the N dimension because N is cut to multiples
// of 32 at a segment's end, where M would be rounded up to 256.  Both operands are K-major:
//   A  weight rows, one TMA box a CTA and stage.  Up interleaves eight gate rows
//      with the eight up rows of the same features (a 5-D view of W1 does that in
//      the box), so that a thread of the epilogue that reads TMEM in 16-lane
//      fragments gets a and b of its features.
//   B  the routed pairs' rows, gathered by their ids with gather4 TMA loads into
//      the swizzled tile: x and phi are never copied into expert order.  The 32
//      gathers of a CTA and stage take the TMA unit longer than its products' 512
//      cycles (up of the layer: some 670 a stage), so they bound full tiles.
//   warp 0        TMA producer of the weights
//   warp 1        MMA issuer (even CTAs), one elected thread
//   warps 2-9     epilogue, two a TMEM lane quarter, half of the tile's pairs
//                 each: fragments of 8 features x 8 pairs are transposed by
//                 stmatrix into shared memory, from where a pair's features are
//                 stored 16 bytes a lane, 32 or 64 contiguous bytes a row.  (The
//                 operands take nearly all of the shared memory's bandwidth, 32
//                 KB written and 32 KB read a stage, so the epilogue's share
//                 costs products' time.)
//   warps 10-17   TMA producers of the pairs' rows, four for the even stages and
//                 four for the odd ones
// Layer of 32768 x 8 pairs, h = 2048, I = 768: up 1.07 to 1.10 ms (1.50 to 1.54 PFLOP/s), down
// 0.65 to 0.72 ms (1.15 to 1.27), the clock at 1.7 to 1.85 GHz under the power cap.  Four
// gather warps: 1.16 and 0.70 ms.  Rows copied by cp.async and handed over with a
// proxy fence took 2.4 and 1.7 where gathers took 1.25 and 0.70; two blocks of M =
// 256 over 128 pairs (half the gathers, but operands of N = 128 products need more
// of the shared memory than it gives) 1.56 and 0.85.
// Every wait is bounded as in the other grouped products (grouped_gemm.cu).
//
// Roundings to bf16: phi (the second product's operand, saved for the backward), the
// pairs' rows and y.  y is off by 2.9e-3 of its size for it, sqrt(3) of one rounding.
// Rows in fp32 would leave 2.3e-3 and double the bytes that down writes and combine
// reads, 2 x 1.07 GB or 0.3 of the layer's 1.80 ms.
#include <cuda_bf16.h>

#include "f32x2.cuh"
#include "grouped.cuh"
#include "lrm_internal.cuh"
#include "swiglu.cuh"
#include "vec.cuh"

namespace lrm {
namespace {

struct CfgFfn {
  static constexpr int BN = 256;                      // pairs of a tile
  static constexpr int BKS = 64;                      // K of a stage: one 128-byte swizzle row, 4 MMAs
  static constexpr int A_BYTES = 128 * BKS * 2;       // this CTA's 128 weight rows
  static constexpr int B_BYTES = (BN / 2) * BKS * 2;  // this CTA's half of the pairs
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int EPI_WARPS = 8;
  static constexpr int GATHER_WARPS = 8;
  static constexpr int ROUND = 32;  // a tile's pairs are a multiple: each gather warp has four rows at least
  static constexpr int THREADS = 64 + 32 * EPI_WARPS + 32 * GATHER_WARPS;
  static constexpr int BUF_BYTES = 32 * 64;  // a warp's: 32 pairs, 32 bf16 values each
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_WARPS * BUF_BYTES + 1024;
  static_assert(ROUND % (4 * GATHER_WARPS) == 0, "half a tile is cut into the shares of half the gather warps, in fours");
  static_assert(ROUND % 32 == 0, "N of an M = 256 pair MMA is a multiple of 32");
};

template <bool UP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(CfgFfn::THREADS, 1)
    ffn_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const int32_t* __restrict__ offsets, const int32_t* __restrict__ ids, int E, int K, int M, int N,
               int div, int max_rows, uint16_t* __restrict__ out, uint16_t* __restrict__ ab, unsigned int* status,
               unsigned long long budget_ns) {
  using C = CfgFfn;
  extern __shared__ uint8_t dsmem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~uintptr_t(1023));

  __shared__ __align__(8) uint64_t full_bar[C::STAGES];
  __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ int s_len[MAX_E];
  __shared__ int s_start[MAX_E];
  __shared__ int s_prefix[MAX_E + 1];  // first pair tile of each expert

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  constexpr int TILE_M = UP ? 128 : 256;  // features of a tile: up has a gate and an up row for each
  const int tiles_m = (M + TILE_M - 1) / TILE_M;

  if (tid == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    s_abort = 0;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full_bar[i], 2);  // both arrivals come from the even CTA's weight producer
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 2 * C::EPI_WARPS);
    }
    mbar_init(&drain_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem_base, C::TMEM_COLS);
    tmem_relinquish_pair();
  }
  grid_dependency_wait();  // the segments, the rows and the buffers written below may be an earlier kernel's
  for (int e = tid; e < E; e += C::THREADS) {
    int st, ln;
    segment(offsets, e, max_rows, st, ln);
    s_len[e] = ln;
    s_start[e] = st;
  }
  __syncthreads();
  if (warp == 0) {
    // pair tiles per expert: a run of experts a lane, then a warp scan
    const int per = (E + 31) / 32;
    const int i0 = lane * per, i1 = min(E, i0 + per);
    int local = 0;
    for (int i = i0; i < i1; ++i) local += ((s_len[i] + C::BN - 1) / C::BN) * tiles_m;
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    int run = incl - local;
    for (int i = i0; i < i1; ++i) {
      s_prefix[i] = run;
      run += ((s_len[i] + C::BN - 1) / C::BN) * tiles_m;
    }
    if (lane == 31) s_prefix[E] = incl;
    if (lane == 0 && blockIdx.x == 0 && __ldg(offsets + E) > max_rows) raise_flag(status, LRM_ERR_SHAPE);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  grid_dependency_launch();
  const uint32_t tmem_base = s_tmem_base;
  const int total_tiles = s_prefix[E];
  volatile int* abort_flag = &s_abort;
  auto fail = [&]() {
    *abort_flag = 1;
    raise_flag(status, LRM_ERR_TIMEOUT);
  };
  // tile -> expert, row tile nt (over the segment), feature tile mt; the row tiles of one feature tile run side by
  // side, so neighbouring CTA pairs share its weights through L2
  int e = 0;  // a warp's tiles come in order: the expert of its last one
  auto decode = [&](int tile, int& nt, int& mt) {
    for (;;) {  // the last expert with s_prefix <= tile, 32 at a time
      const int i = e + 1 + lane;
      const unsigned m = __ballot_sync(0xffffffffu, i < E && s_prefix[i] <= tile);
      e += __popc(m);
      if (m != 0xffffffffu) break;
    }
    const int rem = tile - s_prefix[e];
    const int n_nt = (s_len[e] + C::BN - 1) / C::BN;
    mt = rem / n_nt;
    nt = rem - mt * n_nt;
  };
  // pairs of a row tile that the MMA computes: the remainder rounded up
  auto tile_rows = [&](int len, int nt) {
    return min(C::BN, (len - nt * C::BN + C::ROUND - 1) / C::ROUND * C::ROUND);
  };
  const int nkb = (K + C::BKS - 1) / C::BKS;  // K past the end reads as zeros (tensor bounds)

  if (warp == 0) {
    // ------------------------------------------------------------ weights
    const uint32_t full0 = mapa_shared(&full_bar[0], 0);  // the even CTA's full barriers
    uint32_t it = 0;
    bool ok = true;
    for (int tile = pair; tile < total_tiles && ok; tile += npairs) {
      int nt, mt;
      decode(tile, nt, mt);
      if (elect_one()) {
        const int m0 = mt * TILE_M + static_cast<int>(rank) * (TILE_M / 2);
        const int rows = tile_rows(s_len[e], nt);
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % C::STAGES;
          const uint32_t ph = (it / C::STAGES) & 1u;
          ok = mbar_wait_suspended(&empty_bar[s], ph ^ 1u, budget_ns, abort_flag);
          if (!ok) {
            fail();
            break;
          }
          if (leader) {
            mbar_arrive_expect_tx(&full_bar[s], 2 * (C::A_BYTES + rows / 2 * C::BKS * 2));
            mbar_arrive(&full_bar[s]);
          }
          tma_load_5d_pair(smem + s * C::STAGE_BYTES, &tmA, full0 + s * 8, kb * C::BKS, 0, 0, m0 / 8, e);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    // the even CTAs' commits arrive on these barriers asynchronously: wait for the release of the last STAGES stages,
    // whose copies have landed then, before the block can exit
    if (elect_one())
      for (uint32_t j = it; j < it + C::STAGES; ++j)
        if (!mbar_wait_suspended(&empty_bar[j % C::STAGES], ((j / C::STAGES) & 1u) ^ 1u, budget_ns,
                                 ok ? abort_flag : nullptr))
          break;
    __syncwarp();
  } else if (warp >= 2 + C::EPI_WARPS) {
    // ------------------------------------------------------------ gather
    // A gather takes its operands from uniform registers, so a warp's are issued one after the other, some 75 cycles
    // each by as many lanes (150 by one lane with all the rows).  Four warps share a stage's 32, the other four have the
    // next stage's, so that a warp's wait falls into the time of the others' gathers (two at each: up of 65536 pairs 286
    // us instead of 251).  A tile's ids are loaded while the rows of the one before are gathered.
    const int g = warp - 2 - C::EPI_WARPS;
    const uint32_t par = g & 1, part = g >> 1;
    const uint32_t full0 = mapa_shared(&full_bar[0], 0);
    // this warp's gathers of a tile, one for each of its first n lanes
    int n = 0, id[4] = {0, 0, 0, 0};
    auto first = [&](int n) { return static_cast<int>(part) * n + lane; };  // in fours
    auto look = [&](int tile) {
      if (tile >= total_tiles) return;
      int nt, mt;
      decode(tile, nt, mt);
      const int len = s_len[e];
      const int half = tile_rows(len, nt) / 2;
      n = half / (2 * C::GATHER_WARPS);
      if (lane < n) {
        const int at = nt * C::BN + static_cast<int>(rank) * half + 4 * first(n);
#pragma unroll
        for (int i = 0; i < 4; ++i)  // rows past the segment repeat its last one: computed for nothing, never stored
          id[i] = __ldg(ids + s_start[e] + min(at + i, len - 1));
      }
    };
    uint32_t it0 = 0;
    bool ok = true;
    look(pair);
    for (int tile = pair; tile < total_tiles && ok; tile += npairs, it0 += nkb) {
      const bool mine = lane < n;
      const uint32_t dst = C::A_BYTES + first(n) * 512;
      int row[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)  // the epilogue flags a bad id and stores nothing for it
        row[i] = id[i] >= 0 && id[i] < N ? id[i] / div : 0;
      look(tile + npairs);
      for (int kb = (it0 & 1u) != par ? 1 : 0; kb < nkb; kb += 2) {
        const uint32_t s = (it0 + kb) % C::STAGES;
        const uint32_t ph = ((it0 + kb) / C::STAGES) & 1u;
        if (!__all_sync(0xffffffffu, mbar_wait_suspended(&empty_bar[s], ph ^ 1u, budget_ns, abort_flag))) {
          if (lane == 0) fail();
          ok = false;
          break;
        }
        if (mine)
          tma_gather4_pair(smem + s * C::STAGE_BYTES + dst, &tmB, full0 + s * 8, kb * C::BKS, row);
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // One thread, whose own time has to stay short of the products' (a stage's four take 512 cycles, the tensor core
    // holds only a few ahead): the warp finds the next tile's shape before it issues a tile.  (With the products issued
    // by lane 0 after a wait of the whole warp and its vote: up of the same tokens 562 thousand cycles instead of 470.)
    uint32_t it = 0, acc_it = 0;
    bool ok = leader;
    int rows = 0;
    auto look = [&](int tile) {
      if (tile >= total_tiles) return;
      int nt, mt;
      decode(tile, nt, mt);
      rows = tile_rows(s_len[e], nt);
    };
    look(pair);
    for (int tile = pair; tile < total_tiles && ok; tile += npairs, ++acc_it) {
      const uint32_t idesc = idesc_bf16_f32(256, static_cast<uint32_t>(rows), 0u, 0u);
      look(tile + npairs);
      const uint32_t acc = acc_it & 1u;
      const uint32_t d_tmem = tmem_base + acc * C::BN;
      if (elect_one()) {
        ok = mbar_wait_suspended<true>(&tempty_bar[acc], ((acc_it >> 1) & 1u) ^ 1u, budget_ns, abort_flag);
        tc_fence_after();
        for (int kb = 0; kb < nkb && ok; ++kb, ++it) {
          const uint32_t s = it % C::STAGES;
          ok = mbar_wait_suspended(&full_bar[s], (it / C::STAGES) & 1u, budget_ns, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + s * C::STAGE_BYTES);
          const uint64_t adesc = smem_desc_sw128(a_addr, 16, 1024);
          const uint64_t bdesc = smem_desc_sw128(a_addr + C::A_BYTES, 16, 1024);
          // 16 K are 32 bytes of the swizzled row, 2 in the descriptors' address field
#pragma unroll
          for (int kk = 0; kk < C::BKS / 16; ++kk)
            mma_bf16_ss_pair(d_tmem, adesc + kk * 2, bdesc + kk * 2, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          mma_commit_pair_multicast(&empty_bar[s]);
        }
        if (ok)
          mma_commit_pair_multicast(&tfull_bar[acc]);
        else
          fail();
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (leader) {
      if (elect_one()) {
        mma_commit_pair_local(&drain_bar);
        if (!mbar_wait_suspended(&drain_bar, 0, budget_ns, nullptr)) raise_flag(status, LRM_ERR_TIMEOUT);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                               // TMEM lane quarter this warp may access
    const int hf = (warp - 2) >> 2;                       // its half of the tile's pairs
    const int c_begin = hf * (C::BN / 2);
    constexpr int CHUNKS = C::BN / 2 / 32;
    uint8_t* buf = smem + C::STAGES * C::STAGE_BYTES + (warp - 2) * C::BUF_BYTES;
    // 16-byte chunks of a pair's row in the buffer, swizzled so that neither eight rows of a chunk nor a warp's
    // contiguous reads share banks
    auto at4 = [&](int row, int chunk) { return buf + row * 64 + ((chunk ^ (row >> 1)) & 3) * 16; };
    auto at2 = [&](int row, int chunk) { return buf + row * 32 + ((chunk ^ (row >> 2)) & 1) * 16; };
    const uint32_t tempty0 = mapa_shared(&tempty_bar[0], 0);
    uint32_t acc_it = 0;
    for (int tile = pair; tile < total_tiles; tile += npairs) {
      int nt, mt;
      decode(tile, nt, mt);
      const int n_cols = tile_rows(s_len[e], nt);
      const int rows_valid = s_len[e] - nt * C::BN;  // pairs of this tile inside the segment
      int ids_of[CHUNKS];  // ids of pairs c_begin + 32 i + lane, -1: nothing to store
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        const int c = c_begin + 32 * i + lane;
        ids_of[i] = -1;
        if (c < rows_valid) {
          const int u = __ldg(ids + s_start[e] + nt * C::BN + c);
          if (u >= 0 && u < N)
            ids_of[i] = u;
          else
            raise_flag(status, LRM_ERR_INDEX);
        }
      }
      const uint32_t acc = acc_it & 1u;
      const uint32_t aph = (acc_it >> 1) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait_suspended(&tfull_bar[acc], aph, budget_ns, abort_flag))) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      constexpr int COLS = UP ? 16 : 32;  // features of this warp
      const int col0 = mt * TILE_M + static_cast<int>(rank) * (TILE_M / 2) + q * COLS;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * C::BN;
      const int c_end = min(n_cols, c_begin + C::BN / 2);
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        const int c = c_begin + 32 * i;
        if (c >= c_end) break;
        // v[hh][4 n + x]: TMEM lane 16 hh + lane / 4 (x < 2) or 8 further, pair c + 8 n + 2 (lane % 4) + x % 2
        uint32_t v[2][16];
        tmem_ld_16x256b_x4(taddr + c, v[0]);
        tmem_ld_16x256b_x4(taddr + (16u << 16) + c, v[1]);
        tmem_ld_wait();
        pin_registers(v[0]);
        pin_registers(v[1]);
        auto val = [&](int hh, int n, int x) { return __uint_as_float(v[hh][4 * n + x]); };
        __syncwarp();  // the previous chunk's reads of the buffer are done
        if (!UP || ab != nullptr) {
          // four groups of 8 features: down 8 f .. of this warp's, up a and a, b and b
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int hh = UP ? f & 1 : f >> 1, o = UP ? f & 2 : 2 * (f & 1);
            uint32_t m[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) m[n] = pack_bf16x2(val(hh, n, o), val(hh, n, o + 1));
            stmatrix_x4_trans(at4(lane, f), m);
          }
          __syncwarp();
          const int chunk = lane & 3;
          const int col = col0 + (UP ? chunk & 1 : chunk) * 8;
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int row = it * 8 + (lane >> 2);
            const int u = __shfl_sync(0xffffffffu, ids_of[i], row);
            if (u >= 0 && col < M) {
              uint16_t* o = UP ? ab + (2 * static_cast<size_t>(u) + (chunk >> 1)) * M + col
                               : out + static_cast<size_t>(u) * M + col;
              *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(at4(row, chunk));
            }
          }
          if (UP) __syncwarp();
        }
        if (UP) {  // the activation in fp32, of the unrounded sums
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t m[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
              m[n] = pack_bf16x2(mul2(silu2(F2(val(hh, n, 0), val(hh, n, 1))), F2(val(hh, n, 2), val(hh, n, 3))));
            stmatrix_x4_trans(at2(lane, hh), m);
          }
          __syncwarp();
          const int chunk = lane & 1, col = col0 + chunk * 8;
#pragma unroll
          for (int it = 0; it < 2; ++it) {
            const int row = it * 16 + (lane >> 1);
            const int u = __shfl_sync(0xffffffffu, ids_of[i], row);
            if (u >= 0 && col < M)
              *reinterpret_cast<uint4*>(out + static_cast<size_t>(u) * M + col) =
                  *reinterpret_cast<const uint4*>(at2(row, chunk));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(&tempty_bar[acc]);
        else
          mbar_arrive_cluster(tempty0 + acc * 8);
      }
      ++acc_it;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) let_copies_land();
  cluster_sync_all();  // no CTA leaves while another may still read or write its shared memory or TMEM
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
}

// ---------------------------------------------------------------------------
// Few pairs (a token or a few): the products are bound by the bytes of the weights, and the tiles above leave half of
// the SMs without one (48 tiles for eight pairs of 768 features) and spend their time in set-up and barriers.  Here a
// warp takes four weight rows (up: gate and up of two features; down: four features) for one pair: its lanes stream
// the rows 16 bytes at a time, K in steps of 256, with two or three steps in flight, and read the pair's row out of L1;
// the sums are fp32 and are added over the lanes at the end.  Pairs of one expert read its weights again, out of the L2.
//
// Measured against the tiles, up and down together, us.  Pairs of one expert cost its bytes once more each, at some 18
// TB/s out of the L2 (an expert of h = 2048, I = 768 has 9.4 MB, of 5120, 1536 47 MB); the tiles cost their set-up, some
// 9 to 14 more than the bytes.
//   pairs spread over          1 expert       2              4              8              128
//   2048, 768:    8 pairs   11.3 | 16.9   11.4 | 17.3   12.4 | 18.3   16.2 | 22.4   17.0 | 23.3
//                16         15.6 | 16.9   16.0 | 17.4   17.2 | 18.4   20.2 | 22.4   27.8 | 37.1
//                24         21.0 | 16.9   21.2 | 17.5   22.2 | 18.5   24.8 | 22.6   38.3 | 45.0
//                32         26.1 | 17.0   26.2 | 17.5   26.9 | 18.5   28.9 | 22.7   48.6 | 57.4
//   5120, 1536:   4         21.5 | 29.0   23.2 | 31.6   32.9 | 45.0   33.8 | 45.0   33.9 | 44.8
//                 8         31.2 | 29.1   33.7 | 31.9   41.4 | 45.1   58.5 | 77.8   60.0 | 77.8
//                12         42.5 | 29.0   46.1 | 31.9   51.9 | 45.5   66.1 | 77.6   85.8 | 97.9
//                16         53.8 | 29.0   57.2 | 31.6   63.9 | 45.6   75.5 | 78.0    112 | 127
//   1024, 512:   16          9.1 | 13.1    9.4 | 13.5   10.0 | 13.9   11.4 | 14.7   14.4 | 18.0
// The call knows the pairs' number and the experts', not who shares one: with 16 pairs of 128 experts all on one the
// first line's times hold.
constexpr int FEW_PAIRS = 32;  // at most
constexpr int FEW_ANYWAY = 16;  // also where several pairs are sure to share an expert, up to the bytes read again of
constexpr int FEW_SHARED = 3;    // pairs and
constexpr long long FEW_SHARED_BYTES = 120ll << 20;  // more
constexpr int FEW_THREADS = 256;

// Whether a call of max_rows pairs takes the kernel for few of them: both products, by their weights together.
bool few_pairs(const lrm_dims& d, int max_rows) {
  if (max_rows <= d.E) return max_rows <= FEW_PAIRS;
  const long long expert = 3ll * d.h * d.I * sizeof(uint16_t);
  return max_rows <= FEW_ANYWAY && (max_rows - d.E - FEW_SHARED) * expert <= FEW_SHARED_BYTES;
}

template <bool UP>
__global__ void __launch_bounds__(FEW_THREADS, UP ? 3 : 2)
    ffn_few_kernel(const uint16_t* __restrict__ in, const uint16_t* __restrict__ weight,
                   const int32_t* __restrict__ offsets, const int32_t* __restrict__ ids, int E, int K, int M, int N,
                   int div, int max_rows, uint16_t* __restrict__ out, uint16_t* __restrict__ ab,
                   unsigned int* status) {
  __shared__ int s_expert[FEW_PAIRS], s_ids[FEW_PAIRS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < max_rows) s_expert[threadIdx.x] = -1;
  __syncthreads();
  grid_dependency_wait();
  if (threadIdx.x < max_rows) s_ids[threadIdx.x] = __ldg(ids + threadIdx.x);
  for (int e = threadIdx.x; e < E; e += FEW_THREADS) {
    int st, ln;
    segment(offsets, e, max_rows, st, ln);
    for (int i = 0; i < ln; ++i) s_expert[st + i] = e;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(offsets + E) > max_rows) raise_flag(status, LRM_ERR_SHAPE);
  __syncthreads();
  grid_dependency_launch();
  constexpr int FEATURES = UP ? 2 : 4;  // of a warp's task
  const int groups = M / FEATURES;      // M is a multiple of 8
  const int tasks = max_rows * groups;
  const int kv = K / 8;  // 16-byte vectors of a row
  // tasks go round the blocks first: what is left after whole rounds is spread over the SMs
  for (int task = warp * gridDim.x + blockIdx.x; task < tasks; task += gridDim.x * (FEW_THREADS / 32)) {
    const int r = task / groups, f = (task - r * groups) * FEATURES;
    const int e = s_expert[r], u = s_ids[r];
    if (e < 0) continue;  // beyond the total
    if (u < 0 || u >= N) {
      if (lane == 0) raise_flag(status, LRM_ERR_INDEX);
      continue;
    }
    // rows f (+ 1; up: and those of the up projection; down: + 2, + 3) of the expert
    const uint4* w0 = reinterpret_cast<const uint4*>(weight + (static_cast<size_t>(e) * (UP ? 2 : 1) * M + f) * K) + lane;
    const size_t far = static_cast<size_t>(UP ? M : 2) * kv;
    const uint4* x0 = reinterpret_cast<const uint4*>(in + static_cast<size_t>(u / div) * K) + lane;
    F2 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = F2(0.0f, 0.0f);
    // of 32 vectors, in flight (down of one token with two and three blocks an SM: 7.5 us instead of 6.4; up with four
    // and two blocks: 10.5 instead of 9.9)
    constexpr int STEPS = UP ? 2 : 3;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    for (int v = lane; v < kv; v += 32 * STEPS, w0 += 32 * STEPS, x0 += 32 * STEPS) {
      uint4 w[STEPS][4], x[STEPS];
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const bool in_k = v + 32 * s < kv;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[s][i] = in_k ? ld_stream(w0 + 32 * s + (i & 1) * kv + (i >> 1) * far) : none;
        x[s] = in_k ? __ldg(x0 + 32 * s) : none;
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const F2 xa(bf16_lo(x[s].x), bf16_hi(x[s].x)), xb(bf16_lo(x[s].y), bf16_hi(x[s].y));
        const F2 xc(bf16_lo(x[s].z), bf16_hi(x[s].z)), xd(bf16_lo(x[s].w), bf16_hi(x[s].w));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4& q = w[s][i];
          acc[i] = fma2(F2(bf16_lo(q.x), bf16_hi(q.x)), xa, acc[i]);
          acc[i] = fma2(F2(bf16_lo(q.y), bf16_hi(q.y)), xb, acc[i]);
          acc[i] = fma2(F2(bf16_lo(q.z), bf16_hi(q.z)), xc, acc[i]);
          acc[i] = fma2(F2(bf16_lo(q.w), bf16_hi(q.w)), xd, acc[i]);
        }
      }
    }
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = acc[i].get();
      s[i] = a.x + a.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if (lane != 0) continue;
    if (UP) {  // a of both features, then b
      *reinterpret_cast<uint32_t*>(out + static_cast<size_t>(u) * M + f) =
          pack_bf16x2(mul2(silu2(F2(s[0], s[1])), F2(s[2], s[3])));
      if (ab != nullptr) {
        uint16_t* o = ab + static_cast<size_t>(u) * 2 * M + f;
        *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(s[0], s[1]);
        *reinterpret_cast<uint32_t*>(o + M) = pack_bf16x2(s[2], s[3]);
      }
    } else {
      *reinterpret_cast<uint2*>(out + static_cast<size_t>(u) * M + f) =
          make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    }
  }
}

constexpr int CB_THREADS = 256;

// y_t = sum_j alpha_tj row_tj in fp32, one thread per token and 8 columns; a pair with gate 0 is not read.  One wave of
// blocks that go round the rows: 185 us for 32768 tokens of 8 rows of 2048 values (0.96 of the HBM's rate), a block for
// every 256 items 208; eight rows in flight instead of four 239.
__global__ void __launch_bounds__(CB_THREADS) ffn_combine_kernel(const uint4* __restrict__ rows,
                                                                 const float* __restrict__ alpha, long long items,
                                                                 int k, int wv, uint4* __restrict__ out) {
  grid_dependency_wait();
  for (long long i = static_cast<long long>(blockIdx.x) * CB_THREADS + threadIdx.x; i < items;
       i += static_cast<long long>(gridDim.x) * CB_THREADS) {
    const long long t = i / wv;
    const int v = static_cast<int>(i - t * wv);
    const float* at = alpha + t * k;
    const uint4* rt = rows + t * k * wv + v;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < k; j0 += 4) {
      float a[4];
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = j0 + j < k ? __ldg(at + j0 + j) : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = a[j] != 0.0f ? ld_stream(rt + static_cast<long long>(j0 + j) * wv) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (a[j] != 0.0f) {
          acc[0] = fmaf(a[j], bf16_lo(x[j].x), acc[0]);
          acc[1] = fmaf(a[j], bf16_hi(x[j].x), acc[1]);
          acc[2] = fmaf(a[j], bf16_lo(x[j].y), acc[2]);
          acc[3] = fmaf(a[j], bf16_hi(x[j].y), acc[3]);
          acc[4] = fmaf(a[j], bf16_lo(x[j].z), acc[4]);
          acc[5] = fmaf(a[j], bf16_hi(x[j].z), acc[5]);
          acc[6] = fmaf(a[j], bf16_lo(x[j].w), acc[6]);
          acc[7] = fmaf(a[j], bf16_hi(x[j].w), acc[7]);
        }
      }
    }
    out[i] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                        pack_bf16x2(acc[6], acc[7]));
  }
}

// Weights [E][parts][rows][K] bf16, rows a multiple of 8, as a 5-D tensor (K, 8 rows, parts, rows / 8, E): a box of
// 128 rows holds 8 rows of each part in turn.
lrm_status encode_weight(lrm_ctx* ctx, CUtensorMap* map, const void* base, uint64_t K, uint64_t rows, uint64_t parts,
                         uint64_t E) {
  const cuuint64_t dims[5] = {K, 8, parts, rows / 8, E};
  const cuuint64_t strides[4] = {K * 2, rows * K * 2, 8 * K * 2, parts * rows * K * 2};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(parts), static_cast<cuuint32_t>(16 / parts), 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = ctx->encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides,
                                 box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? LRM_OK : LRM_ERR_CUDA;
}

// Both products: rows of in [in_rows, K] gathered by id / div, weights [E][parts][M][K], out [N, M].
template <bool UP>
lrm_status launch_ffn(lrm_ctx* ctx, const uint16_t* in, uint64_t in_rows, const uint16_t* weight,
                      const int32_t* offsets, const int32_t* ids, const lrm_dims& d, int max_rows, uint16_t* out,
                      uint16_t* ab, cudaStream_t s) {
  using C = CfgFfn;
  const int K = UP ? d.h : d.I, M = UP ? d.I : d.h, N = d.T * d.k;
  if (few_pairs(d, max_rows)) {
    auto few = ffn_few_kernel<UP>;
    static thread_local int few_device = -1, grid = 0;
    if (few_device != ctx->device) {
      grid = resident_grid(ctx, few, FEW_THREADS, 0);
      few_device = ctx->device;
    }
    const long long tasks = static_cast<long long>(max_rows) * (M / (UP ? 2 : 4));
    const long long need = (tasks + FEW_THREADS / 32 - 1) / (FEW_THREADS / 32);
    return launch_dependent(few, static_cast<int>(need < grid ? need : grid), FEW_THREADS, 0, 0, s, in, weight,
                            offsets, ids, d.E, K, M, N, UP ? d.k : 1, max_rows, out, ab, ctx->d_status);
  }
  auto kern = ffn_kernel<UP>;
  static thread_local int configured_device = -1;
  static thread_local int clusters = 0;
  if (configured_device != ctx->device) {
    if (ctx->smem_optin < C::SMEM_BYTES + 14 * 1024) return LRM_ERR_ARCH;
    LRM_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctx->sm_count & ~1, 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    int n = 0;
    LRM_CHECK_CUDA(cudaOccupancyMaxActiveClusters(&n, kern, &cfg));
    if (n < 1) return LRM_ERR_ARCH;
    clusters = n;
    configured_device = ctx->device;
  }
  alignas(64) CUtensorMap ma, mb;
  lrm_status st = encode_weight(ctx, &ma, weight, K, M, UP ? 2 : 1, d.E);
  if (st != LRM_OK) return st;
  if ((st = encode_2d(ctx, &mb, in, K, in_rows, 1)) != LRM_OK) return st;
  return launch_dependent(kern, 2 * clusters, C::THREADS, C::SMEM_BYTES, 0, s, ma, mb, offsets, ids, d.E, K, M, N,
                          UP ? d.k : 1, max_rows, out, ab, ctx->d_status, ctx->wait_budget_ns);
}

lrm_status check_ffn(const lrm_ctx* ctx, const lrm_dims& dims, int max_rows, const void* in, const void* weight,
                     const int32_t* offsets, const int32_t* ids, const void* out, const void* ab, bool& empty) {
  empty = false;
  if (ctx == nullptr) return LRM_ERR_INVALID_ARG;
  const lrm_status st = check_dims(dims);
  if (st != LRM_OK) return st;
  if (max_rows < 0 || offsets == nullptr) return LRM_ERR_INVALID_ARG;
  if (max_rows == 0 || dims.T == 0) {
    empty = true;
    return LRM_OK;
  }
  if (in == nullptr || weight == nullptr || ids == nullptr || out == nullptr) return LRM_ERR_INVALID_ARG;
  if (!aligned(in, 16) || !aligned(weight, 16) || !aligned(out, 16) || (ab != nullptr && !aligned(ab, 16)) ||
      !aligned(offsets, 4) || !aligned(ids, 4))
    return LRM_ERR_ALIGN;
  return LRM_OK;
}

}  // namespace
}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_ffn_up(lrm_ctx* ctx, const uint16_t* x, const uint16_t* W1, const int32_t* offsets,
                                 const int32_t* ids, lrm_dims dims, int32_t max_rows, uint16_t* ab, uint16_t* phi,
                                 void* stream) {
  bool empty;
  const lrm_status st = check_ffn(ctx, dims, max_rows, x, W1, offsets, ids, phi, ab, empty);
  if (st != LRM_OK || empty) return st;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  return launch_ffn<true>(ctx, x, dims.T, W1, offsets, ids, dims, max_rows, phi, ab,
                          static_cast<cudaStream_t>(stream));
}

extern "C" lrm_status lrm_ffn_down(lrm_ctx* ctx, const uint16_t* phi, const uint16_t* W, const int32_t* offsets,
                                   const int32_t* ids, lrm_dims dims, int32_t max_rows, uint16_t* rows,
                                   void* stream) {
  bool empty;
  const lrm_status st = check_ffn(ctx, dims, max_rows, phi, W, offsets, ids, rows, nullptr, empty);
  if (st != LRM_OK || empty) return st;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  return launch_ffn<false>(ctx, phi, static_cast<uint64_t>(dims.T) * dims.k, W, offsets, ids, dims, max_rows, rows,
                           nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" lrm_status lrm_ffn_combine(lrm_ctx* ctx, const uint16_t* rows, const float* alpha, lrm_dims dims,
                                      uint16_t* out, void* stream) {
  if (ctx == nullptr) return LRM_ERR_INVALID_ARG;
  const lrm_status st = check_dims(dims);
  if (st != LRM_OK) return st;
  if (dims.T == 0) return LRM_OK;
  if (rows == nullptr || alpha == nullptr || out == nullptr) return LRM_ERR_INVALID_ARG;
  if (!aligned(rows, 16) || !aligned(out, 16) || !aligned(alpha, 4)) return LRM_ERR_ALIGN;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return LRM_ERR_CUDA;
  const int wv = dims.h / 8;
  const long long items = static_cast<long long>(dims.T) * wv;
  const long long need = (items + CB_THREADS - 1) / CB_THREADS;
  static thread_local int device = -1, cap = 0;
  if (device != ctx->device) {
    cap = resident_grid(ctx, ffn_combine_kernel, CB_THREADS, 0);
    device = ctx->device;
  }
  return launch_dependent(ffn_combine_kernel, static_cast<int>(need < cap ? need : cap), CB_THREADS, 0, 0,
                          static_cast<cudaStream_t>(stream), reinterpret_cast<const uint4*>(rows), alpha, items,
                          dims.k, wv, reinterpret_cast<uint4*>(out));
}
