// k_gemm_mx4.cu -- MXFP4 linear layer: y = epi(deq(A) deq(W)^T + b) with E2M1
// codes and one E8M0 scale per 32 elements of K on both sides (OCP
// Microscaling v1.0), fp32 accumulation in tensor memory, bf16 output.
//
// Structure (persistent over output tiles; the roles of gemm_tc_kernel and
// gemm_tc2_kernel): per 256-column k-block the producer brings 128 rows of A
// codes and the tile's rows of W codes (128 bytes a row, one 128-byte swizzle
// atom) and their scale blocks; the MMA lane copies the scales into TMEM
// (tcgen05.cp, 512 bytes per 128 rows x 128 columns) and issues four K = 64
// block-scaled MMAs.  MMA k reads bytes 2 (k & 1) and 2 (k & 1) + 1 of each
// row's scale word of the 128-column half k / 2.  MMAs that start past K are
// left out: their scale half need not exist.  Two accumulators let the
// epilogue of a tile overlap the next tile's main loop.  Where tiles are few and K
// is long, gemm_mx4_split_kernel spreads a tile's k-blocks over a cluster.
//
// Bound: an SM's share of the work is small at these sizes (3900 x 4304 x 1152 is
// 3.7 tiles of 256 x 256 a pair, 0.3 us of MMA each), so no single unit is: with
// the stores, the loads or the MMAs left out the 15.3 us become 13.9, 14.8 and
// 14.6.  The start (first operands from DRAM, 1.3 us), the drain of the last tile's
// stores (1.6 us) and GELU's hardware tanh (one in 16 a clock and SM) remain.  At
// 8192 x 4096 x 8192 the tensor core is: 5570 TFLOP/s, 3.3 times cuBLAS's bf16 rate.
//
// PAIR: a cluster of two CTAs computes 256-row tiles (cta_group::2, M = 256):
// each loads its own 128 rows of A, half of the tile's W rows, the scales of
// its own A rows and of all W rows (the MMA reads those from both CTAs'
// tensor memory), completing on the leader's barriers; the leader issues.
//
// Two accumulators of 256 columns and the 24 scale columns do not fit in the
// 512 TMEM columns, so the 256-wide accumulators share 24 columns: the next tile's
// MMAs start once the epilogue's warps have read their 64 columns each into
// registers, before they finish and store them.
#include <cuda_bf16.h>
#include <stdio.h>
#include <stdlib.h>

#include <atomic>

#include "gemm_common.cuh"
#include "kernels.h"
#include "mx4.h"
#include "sm100_mx4.cuh"

namespace vit {

namespace {

constexpr int BM = 128;
constexpr int kBK = 256;                       // E2M1 elements per k-block: 128 bytes
constexpr uint32_t kATileBytes = BM * kBK / 2; // 16 KB
constexpr uint32_t kSfBytes = 1024;            // scales of 128 rows x 256 columns
constexpr int kCols = 64;                      // columns of an epilogue warp
constexpr int kMaxEpiWarps = 16;
constexpr uint32_t kBufBytes = 32 * kCols * 2; // its staged 32 x 64 bf16 results
constexpr int kMaxDevices = 64;                // per-device cache of the launch size
constexpr uint32_t kPrefetchBytes = 4096;
constexpr size_t kPrefetchMost = 32u << 20;    // operands beyond this are streamed from DRAM
constexpr size_t kSmemLimit = 232448;          // dynamic shared memory of one CTA (227 KB)

struct __align__(16) Bars {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t res_full[kMaxEpiWarps];  // residual chunks
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

template <int BN, bool PAIR>
struct Cfg {
  static constexpr int kSfbBlocks = (BN + 127) / 128;  // 128-row blocks a tile's W rows touch
  static constexpr int kBRows = PAIR ? BN / 2 : BN;  // W rows this CTA loads
  static constexpr uint32_t kSfOff = kATileBytes + kBRows * kBK / 2;
  static constexpr uint32_t kStageBytes = kSfOff + kSfBytes * (1 + kSfbBlocks);
  // epilogue warps: one per TMEM lane quarter and 64 columns
  static constexpr int kEpiWarps = 4 * BN / kCols;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  // barriers, the epilogue warps' bias slots (fp32), their staging buffers
  static constexpr uint32_t kBufOff = 1024 + kMaxEpiWarps * kCols * 4;
  static constexpr uint32_t kAfterRing = kBufOff + kEpiWarps * kBufBytes;
  static constexpr int kFit = int((kSmemLimit - 1024 - kAfterRing) / kStageBytes);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr size_t kSmemBytes = size_t(kStages) * kStageBytes + 1024 + kAfterRing;
  static constexpr uint32_t kTmemCols = 512;
  // scales: 4 columns per 128-column half of A's rows, then 4 per half and 128
  // rows of W, at the end of TMEM; the second accumulator ends before them
  static constexpr uint32_t kSfaCol = kTmemCols - 8 - 8 * kSfbBlocks;
  static constexpr uint32_t kSfbCol = kSfaCol + 8;
  static constexpr bool kShared = 2 * BN > int(kSfaCol);
  static constexpr uint32_t kAcc1 = kShared ? kSfaCol - BN : BN;
  static_assert(kStageBytes % 1024 == 0, "stages keep the 1 KB alignment of the swizzled tiles");
  static_assert(sizeof(Bars) <= 1024 && kStages >= 3, "barrier block, operand ring");
};

// GELU (tanh form) of two values in packed fp32: u/2 (1 + tanh(u (k0 + k0 k1
// u^2))) with the hardware tanh.
__device__ __forceinline__ uint64_t gelu_x2(uint64_t u) {
  const uint64_t k0 = f2_pack(0.7978845608f, 0.7978845608f);
  const uint64_t k01 = f2_pack(0.7978845608f * 0.044715f, 0.7978845608f * 0.044715f);
  const uint64_t z = f2_mul(u, f2_fma(f2_mul(u, u), k01, k0));
  float z0, z1;
  f2_unpack(z, z0, z1);
  const uint64_t h = f2_mul(u, f2_pack(0.5f, 0.5f));
  return f2_fma(h, f2_pack(gemm::tanh_fast(z0), gemm::tanh_fast(z1)), h);
}

// 8 columns of one row: accumulator r -> bias b, GELU or residual -> bf16, two
// columns at a time (packed fp32 halves the instructions of the epilogue).
template <int EPI>
__device__ __forceinline__ uint4 finish8(const uint32_t *r, const float4 *b, const uint4 &res) {
  const uint32_t rw[4] = {res.x, res.y, res.z, res.w};
  const float4 b0 = b[0], b1 = b[1];
  const float bw[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint64_t v = f2_add(f2_pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])),
                        f2_pack(bw[2 * e], bw[2 * e + 1]));
    if constexpr (EPI == kEpiGelu) v = gelu_x2(v);
    if constexpr (EPI == kEpiResidual) v = f2_add(v, f2_pack(bf16_lo(rw[e]), bf16_hi(rw[e])));
    float lo, hi;
    f2_unpack(v, lo, hi);
    o[e] = pack_bf16x2(lo, hi);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// One k-block of MMAs from a ring stage: scales to TMEM, then up to four K = 64
// MMAs (`left`: columns of K from here on).  sfb_n: the TMEM columns by which the
// tile's first W row lies inside its first scale block.
template <int BN, bool PAIR>
__device__ __forceinline__ void issue_k_block(uint32_t stage, uint32_t d_tmem, uint32_t sfa_t,
                                              uint32_t sfb_t, uint32_t sfb_n, int left,
                                              bool first) {
  using CF = Cfg<BN, PAIR>;
  const uint32_t sb = stage + kATileBytes, ssf = stage + CF::kSfOff;
  const int mmas = min(4, (left + 63) / 64);
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // 128-column halves
    if (2 * j >= mmas) break;
    tmem_cp_scales<PAIR>(sfa_t + 4 * j, smem_desc(ssf + 512 * j, 0, 128, 0));
#pragma unroll
    for (int i = 0; i < CF::kSfbBlocks; ++i)
      tmem_cp_scales<PAIR>(sfb_t + 4 * (j * CF::kSfbBlocks + i),
                           smem_desc(ssf + kSfBytes * (1 + i) + 512 * j, 0, 128, 0));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k >= mmas) break;
    const uint64_t ad = smem_desc(stage + k * 32, 16, 1024, 2);
    const uint64_t bd = smem_desc(sb + k * 32, 16, 1024, 2);
    const int j = k >> 1, sf = 2 * (k & 1);
    mma_mx4_ss<PAIR>(d_tmem, ad, bd, idesc_mx4(PAIR ? 2 * BM : BM, BN, sf),
                     (sfa_t + 4 * j) | (uint32_t(sf) << 30),
                     (sfb_t + sfb_n + 4 * j * CF::kSfbBlocks) | (uint32_t(sf) << 30),
                     !first || k > 0);
  }
}

// The codes of A and W, for the L2 prefetch at a kernel's start (bytes; 0: none).
struct Prefetch {
  const uint8_t *p[2];
  size_t bytes[2];
};

template <int BN, int EPI, bool PAIR>
__global__ void __launch_bounds__((Cfg<BN, PAIR>::kThreads), 1)
    gemm_mx4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSa,
                    const __grid_constant__ CUtensorMap tmSb,
                    const __grid_constant__ CUtensorMap tmR, const __grid_constant__ CUtensorMap tmY,
                    const __nv_bfloat16 *__restrict__ bias, int M, int N, int K, int *status,
                    const __grid_constant__ Prefetch pre, uint32_t lost_tx) {
  using CF = Cfg<BN, PAIR>;
  constexpr int kCtas = PAIR ? 2 : 1, kRows = kCtas * BM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  Bars *bars = reinterpret_cast<Bars *>(smem + size_t(CF::kStages) * CF::kStageBytes);
  volatile int *abort_flag = &bars->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? int(cluster_cta_rank()) : 0;
  const int worker = blockIdx.x / kCtas, workers = gridDim.x / kCtas;
  const int num_m = (M + kRows - 1) / kRows, num_n = (N + BN - 1) / BN;
  const int num_tiles = num_m * num_n;
  const int k_blocks = (K + kBK - 1) / kBK;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < CF::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bars->acc_full[a], 1);
      mbar_init(&bars->acc_empty[a], kCtas * CF::kEpiWarps);
    }
    for (int w = 0; w < CF::kEpiWarps; ++w) mbar_init(&bars->res_full[w], 1);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSa);
    tma_prefetch_desc(&tmSb);
    tma_prefetch_desc(&tmY);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&bars->tmem_base, CF::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&bars->tmem_base, CF::kTmemCols);
      tmem_relinquish();
    }
  }
  if (warp == 2) {
    // Every CTA asks for its share of the operands at once: many CTAs wait for
    // the same cold rows, and a tile's loads are only a few k-blocks ahead (3900
    // x 3456 x 1152: 13.2 -> 12.5 us).  A prefetch changes no value, so it need
    // not wait for the kernel before.
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const size_t chunks = pre.bytes[o] / kPrefetchBytes;
      for (size_t i = blockIdx.x * 32 + lane; i < chunks; i += gridDim.x * 32)
        prefetch_l2(pre.p[o] + i * kPrefetchBytes, kPrefetchBytes);
    }
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();  // both CTAs' barriers exist before remote use
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int tile = worker; tile < num_tiles && ok; tile += workers) {
        const int mb = (tile % num_m) * kCtas + rank, nb = tile / num_m;
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait(&bars->empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
          uint8_t *sa = smem + size_t(stage) * CF::kStageBytes;
          const int n0 = nb * BN + rank * CF::kBRows;
          uint32_t full = smem_u32(&bars->full[stage]);
          // lost_tx > 0 only under fault injection (vit_debug_lost_tx): the stage then
          // waits for bytes that no copy delivers
          if (rank == 0)
            mbar_arrive_expect_tx(&bars->full[stage], kCtas * CF::kStageBytes + lost_tx);
          if constexpr (PAIR) {
            full = map_to_cta(&bars->full[stage], 0);
            tma_load_2d_pair(sa, &tmA, full, kb * (kBK / 2), mb * BM);
            tma_load_2d_pair(sa + kATileBytes, &tmB, full, kb * (kBK / 2), n0);
          } else {
            tma_load_2d(sa, &tmA, &bars->full[stage], kb * (kBK / 2), mb * BM);
            tma_load_2d(sa + kATileBytes, &tmB, &bars->full[stage], kb * (kBK / 2), n0);
          }
          tma_load_3d<PAIR>(sa + CF::kSfOff, &tmSa, full, 0, 2 * kb, mb);
          tma_load_3d<PAIR>(sa + CF::kSfOff + kSfBytes, &tmSb, full, 0, 2 * kb,
                            nb * BN / 128);
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == CF::kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok && rank == 0)
        for (int s = 0; s < CF::kStages; ++s)
          if (issued_mask & (1u << s)) gemm::drain_wait(&bars->full[s], (issued_parity >> s) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0 && elect_one()) {
      auto commit = [&](uint64_t *bar) {
        if constexpr (PAIR) mma_commit_pair_mc(bar, 0x3);
        else mma_commit(bar);
      };
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      bool any_mma = false;
      const uint32_t sfa_t = tmem + CF::kSfaCol, sfb_t = tmem + CF::kSfbCol;
      for (int tile = worker; tile < num_tiles && ok; tile += workers, ++it) {
        const int a = it & 1;
        // what frees accumulator a for this tile: the epilogue has read tile
        // it - 2, or (shared columns) tile it - 1
        const int freed = CF::kShared ? it - 1 : it - 2;
        if (freed >= 0 && !mbar_wait(&bars->acc_empty[a], (freed >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + (a ? CF::kAcc1 : 0u);
        // a tile of 192 columns may start in the middle of a 128-row scale block:
        // its first 64 rows there are two of the block's four TMEM columns
        const uint32_t sfb_n = uint32_t(tile / num_m * BN % 128 / 32);
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait(&bars->full[stage], phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          issue_k_block<BN, PAIR>(smem_u32(smem + size_t(stage) * CF::kStageBytes), d_tmem, sfa_t,
                                  sfb_t, sfb_n, K - kb * kBK, kb == 0);
          any_mma = true;
          commit(&bars->empty[stage]);
          if (++stage == CF::kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        commit(&bars->acc_full[a]);
      }
      if (!ok && any_mma) {
        if constexpr (PAIR) mma_commit_pair_mc(&bars->drain, 0x1);
        else mma_commit(&bars->drain);
        gemm::drain_wait(&bars->drain, 0);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // warp ew drains 32 rows (TMEM lane quarter warp & 3) of 64 columns
    const int ew = warp - 2, quarter = warp & 3, cg = (ew >> 2) * kCols;
    uint8_t *buf = reinterpret_cast<uint8_t *>(bars) + CF::kBufOff + ew * kBufBytes;
    uint4 *rowp = reinterpret_cast<uint4 *>(buf + lane * (kCols * 2));
    const int sw = lane & 7;  // 128-byte swizzle: 16-byte unit u ^ (row & 7)
    float *bias_s =
        reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(bars) + 1024) + ew * kCols;
    auto tile_row = [&](int tile) { return ((tile % num_m) * kCtas + rank) * BM + quarter * 32; };
    auto tile_col = [&](int tile) { return tile / num_m * BN + cg; };
    // bias (two columns a lane) and residual of a tile are asked for a tile ahead
    auto load_bias = [&](int tile) {
      const int col = tile_col(tile) + 2 * lane;
      return bias != nullptr && tile < num_tiles && col < N
                 ? __ldg(reinterpret_cast<const uint32_t *>(bias + col))
                 : 0u;
    };
    auto load_res = [&](int tile) {
      if (EPI == kEpiResidual && tile < num_tiles && lane == 0) {
        mbar_arrive_expect_tx(&bars->res_full[ew], kBufBytes);
        tma_load_2d(buf, &tmR, &bars->res_full[ew], tile_col(tile), tile_row(tile));
      }
    };
    uint32_t bias_next = load_bias(worker);
    load_res(worker);
    int it = 0;
    bool ok = true;
    for (int tile = worker; tile < num_tiles; tile += workers, ++it) {
      const int row0 = tile_row(tile), col0 = tile_col(tile);
      const int a = it & 1;
      __syncwarp();
      reinterpret_cast<float2 *>(bias_s)[lane] = make_float2(bf16_lo(bias_next), bf16_hi(bias_next));
      __syncwarp();
      bias_next = load_bias(tile + workers);
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_full[a], (it >> 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t r[kCols];
      tmem_ld_cols<kCols>(tmem + (a ? CF::kAcc1 : 0u) + (uint32_t(quarter * 32) << 16) + cg, r);
      tmem_ld_wait();
      // this warp's part of the accumulator is read: a relaxed arrival, which
      // does not wait for the stores
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        uint64_t *bar = &bars->acc_empty[CF::kShared ? a ^ 1 : a];
        if constexpr (PAIR) mbar_arrive_cluster_relaxed(map_to_cta(bar, 0));
        else mbar_arrive_relaxed(bar);
      }
      if constexpr (EPI == kEpiResidual) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->res_full[ew], it & 1, abort_flag));
        if (!ok) break;
      } else {
        if (lane == 0) bulk_wait_group_read<0>();  // the last tile's copy has read the buffer
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < kCols / 8; ++u) {
        const uint4 res = EPI == kEpiResidual ? rowp[u ^ sw] : make_uint4(0, 0, 0, 0);
        rowp[u ^ sw] = finish8<EPI>(r + 8 * u, reinterpret_cast<const float4 *>(bias_s) + 2 * u, res);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {  // one copy, clipped at M and N
        if (row0 < M && col0 < N) tma_store_2d(&tmY, buf, col0, row0);
        bulk_commit_group();
        if (EPI == kEpiResidual) bulk_wait_group_read<0>();
      }
      load_res(tile + workers);
    }
    // after an abort, the residual copy still in flight
    if (EPI == kEpiResidual && !ok && lane == 0) gemm::drain_wait(&bars->res_full[ew], it & 1);
    // the copies have read the buffers; their writes complete before the grid does
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }

  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();  // no CTA leaves while the pair's MMAs may read its memory
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, CF::kTmemCols);
    else tmem_dealloc(tmem, CF::kTmemCols);
  }
  if (threadIdx.x == 0 && bars->abort_flag) {
    // The CTA stays for copies that nobody has waited for: those that a producer had
    // issued before another role gave up, and rank 1's, which complete on the
    // leader's barriers.  (If the leader gives up, rank 1 does: it misses a tile.)
    gemm::settle();
    report_status(status, kDevTimeout);
  }
}

// Few tiles and a long K: a cluster of SPLIT CTAs shares one 128 x 128 tile, each
// over its own run of k-blocks.  Every CTA leaves its partial sums (the rows that
// exist, fp32) in its shared memory, where the operand ring was; then CTA r
// finishes columns [r, r + 1) 128 / SPLIT, adding the partials of all CTAs in
// rank order over the cluster's shared memory, so the result does not depend on
// which CTA is done first.  A CTA that gave up (a lost arrival) leaves kGaveUp in
// place of its sums, and what they belong to is not written.  No CTA is persistent:
// the grid is one cluster a tile.
constexpr uint32_t kGaveUp = 0xFFC0DEADu;  // a NaN that no MMA produces (theirs is 7FFFFFFF)
template <int EPI, int SPLIT>
__global__ void __launch_bounds__((Cfg<128, false>::kThreads), 1)
    gemm_mx4_split_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmSa,
                          const __grid_constant__ CUtensorMap tmSb,
                          const __nv_bfloat16 *__restrict__ bias, const __nv_bfloat16 *res,
                          __nv_bfloat16 *y, int M, int N, int K, int *status, uint32_t lost_tx) {
  constexpr int BN = 128;
  using CF = Cfg<BN, false>;
  constexpr int kPitch = BN + 4;  // floats of a partial row: lanes on different banks
  static_assert(size_t(CF::kStages) * CF::kStageBytes >= size_t(BM) * kPitch * 4, "partial sums");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  Bars *bars = reinterpret_cast<Bars *>(smem + size_t(CF::kStages) * CF::kStageBytes);
  volatile int *abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_cta_rank()), tile = blockIdx.x / SPLIT;
  const int num_m = (M + BM - 1) / BM, mb = tile % num_m, nb = tile / num_m;
  const int k_blocks = (K + kBK - 1) / kBK;
  const int kb0 = k_blocks * rank / SPLIT, kb1 = k_blocks * (rank + 1) / SPLIT;  // not empty

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < CF::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->acc_full[0], 1);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSa);
    tma_prefetch_desc(&tmSb);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, CF::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  pdl_wait();

  const int rows = min(BM, M - mb * BM);
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&bars->empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
        uint8_t *sa = smem + size_t(stage) * CF::kStageBytes;
        const uint32_t full = smem_u32(&bars->full[stage]);
        // lost_tx > 0 only under fault injection (vit_debug_lost_tx): the last CTA of
        // the cluster then waits for bytes that no copy delivers
        mbar_arrive_expect_tx(&bars->full[stage],
                              CF::kStageBytes + (rank == SPLIT - 1 ? lost_tx : 0u));
        tma_load_2d(sa, &tmA, &bars->full[stage], kb * (kBK / 2), mb * BM);
        tma_load_2d(sa + kATileBytes, &tmB, &bars->full[stage], kb * (kBK / 2), nb * BN);
        tma_load_3d<false>(sa + CF::kSfOff, &tmSa, full, 0, 2 * kb, mb);
        tma_load_3d<false>(sa + CF::kSfOff + kSfBytes, &tmSb, full, 0, 2 * kb, nb);
        issued_mask |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == CF::kStages) { stage = 0; phase ^= 1; }
      }
      if (!ok)
        for (int s = 0; s < CF::kStages; ++s)
          if (issued_mask & (1u << s)) gemm::drain_wait(&bars->full[s], (issued_parity >> s) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, any_mma = false;
      const uint32_t sfa_t = tmem + CF::kSfaCol, sfb_t = tmem + CF::kSfbCol;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&bars->full[stage], phase, abort_flag)) { ok = false; break; }
        tc_fence_after();
        issue_k_block<BN, false>(smem_u32(smem + size_t(stage) * CF::kStageBytes), tmem, sfa_t,
                                 sfb_t, 0, K - kb * kBK, kb == kb0);
        any_mma = true;
        mma_commit(&bars->empty[stage]);
        if (++stage == CF::kStages) { stage = 0; phase ^= 1; }
      }
      if (ok) {
        mma_commit(&bars->acc_full[0]);
      } else if (any_mma) {
        mma_commit(&bars->drain);
        gemm::drain_wait(&bars->drain, 0);
      }
    }
  } else {
    // ------------------------------------------------------------ partial sums
    const int ew = warp - 2, quarter = warp & 3, cg = (ew >> 2) * kCols;
    const int row = quarter * 32 + lane;
    const bool ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_full[0], 0, abort_flag));
    if (quarter * 32 < rows) {
      uint32_t r[kCols];
      if (ok) {
        tc_fence_after();
        tmem_ld_cols<kCols>(tmem + (uint32_t(quarter * 32) << 16) + cg, r);
        tmem_ld_wait();
      } else {
        gemm::settle();  // the operands' copies land where the sums go
#pragma unroll
        for (int c = 0; c < kCols; ++c) r[c] = kGaveUp;
      }
      if (row < rows) {
        uint4 *p = reinterpret_cast<uint4 *>(smem) + (row * kPitch + cg) / 4;
#pragma unroll
        for (int u = 0; u < kCols / 4; ++u)
          p[u] = make_uint4(r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // every CTA's partial sums are in place
  if (!*abort_flag) {
    constexpr int kUnits = BN / SPLIT / 8;  // 8-column pieces of this CTA's columns
    const uint32_t base = smem_u32(smem);
    for (int u = threadIdx.x; u < rows * kUnits; u += CF::kThreads) {
      const int row = u / kUnits, c = rank * (BN / SPLIT) + u % kUnits * 8;
      const int col = nb * BN + c;
      if (col >= N) continue;
      const size_t at = size_t(mb * BM + row) * N + col;
      const uint4 rv = EPI == kEpiResidual ? __ldcg(reinterpret_cast<const uint4 *>(res + at))
                                           : make_uint4(0, 0, 0, 0);
      const uint4 b4 = bias != nullptr ? __ldg(reinterpret_cast<const uint4 *>(bias + col))
                                       : make_uint4(0, 0, 0, 0);
      const float4 b[2] = {make_float4(bf16_lo(b4.x), bf16_hi(b4.x), bf16_lo(b4.y), bf16_hi(b4.y)),
                           make_float4(bf16_lo(b4.z), bf16_hi(b4.z), bf16_lo(b4.w), bf16_hi(b4.w))};
      float4 s[SPLIT][2];
#pragma unroll
      for (int q = 0; q < SPLIT; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          s[q][e] = ld_cluster(map_addr_to_cta(base + uint32_t(row * kPitch + c + 4 * e) * 4, q));
      bool lost = false;
#pragma unroll
      for (int q = 0; q < SPLIT; ++q) lost |= __float_as_uint(s[q][0].x) == kGaveUp;
      float v[8] = {};
#pragma unroll
      for (int q = 0; q < SPLIT; ++q) {
        v[0] += s[q][0].x; v[1] += s[q][0].y; v[2] += s[q][0].z; v[3] += s[q][0].w;
        v[4] += s[q][1].x; v[5] += s[q][1].y; v[6] += s[q][1].z; v[7] += s[q][1].w;
      }
      uint32_t r[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(v[e]);
      const uint4 out = finish8<EPI>(r, b, rv);  // before the test: 960 x 1152 x 4304 11.5 -> 10.6 us
      if (!lost) *reinterpret_cast<uint4 *>(y + at) = out;
    }
  }
  cluster_sync_all();  // no CTA leaves while another may read its partial sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, CF::kTmemCols);
  }
  if (threadIdx.x == 0 && bars->abort_flag) {
    gemm::settle();  // as above
    report_status(status, kDevTimeout);
  }
}

struct Args {
  const uint8_t *a_codes, *a_scales, *w_codes, *w_scales;
  const __nv_bfloat16 *bias, *res;
  __nv_bfloat16 *y;
  int M, N, K, num_sms;
  int *status;
  cudaStream_t st;
  uint32_t lost_tx;
};

// Codes as [rows, bytes] with 128-byte boxes, scales as [block rows][k blocks]
// [512 bytes] with boxes of two k blocks, residual and output in 32 x 64 boxes.
struct Maps {
  CUtensorMap a, b, sa, sb, res, y;
};
bool encode_maps(Maps &m, const Args &g, int b_rows, int sb_blocks, bool residual) {
  const uint64_t kb = (uint64_t(g.K) + 127) / 128, bytes = (uint64_t(g.K) + 1) / 2;
  auto codes = [&](CUtensorMap *t, const uint8_t *p, int rows, int box) {
    return encode_tensor_map_2d(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, bytes, rows,
                                mx4_row_bytes(g.K), kBK / 2, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  auto scales = [&](CUtensorMap *t, const uint8_t *p, int rows, int box) {
    return encode_tensor_map_3d(t, CU_TENSOR_MAP_DATA_TYPE_UINT32, p, 128, kb,
                                (uint64_t(rows) + 127) / 128, 512, kb * 512, 128, 2, box,
                                CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  auto chunks = [&](CUtensorMap *t, const __nv_bfloat16 *p) {
    return encode_tensor_map_2d(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, g.N, g.M,
                                uint64_t(g.N) * 2, kCols, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (codes(&m.a, g.a_codes, g.M, BM) || codes(&m.b, g.w_codes, g.N, b_rows) ||
      scales(&m.sa, g.a_scales, g.M, 1) || scales(&m.sb, g.w_scales, g.N, sb_blocks) ||
      chunks(&m.y, g.y) || (residual && chunks(&m.res, g.res)))
    return false;
  if (!residual) m.res = m.y;  // not read
  return true;
}

// The device's cache slot of a kernel's launch size, or null.
std::atomic<int> *launch_slot(std::atomic<int> *slots) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  return &slots[dev < kMaxDevices ? dev : kMaxDevices];
}

template <int BN, int EPI, bool PAIR>
cudaError_t run(const Args &g) {
  using CF = Cfg<BN, PAIR>;
  constexpr int kCtas = PAIR ? 2 : 1;
  Maps m;
  if (!encode_maps(m, g, CF::kBRows, CF::kSfbBlocks, EPI == kEpiResidual))
    return cudaErrorInvalidValue;
  const size_t na = size_t(g.M) * mx4_row_bytes(g.K), nw = size_t(g.N) * mx4_row_bytes(g.K);
  const bool warm = na + nw <= kPrefetchMost;
  const Prefetch pre{{g.a_codes, g.w_codes}, {warm ? na : 0, warm ? nw : 0}};
  auto kern = gemm_mx4_kernel<BN, EPI, PAIR>;
  // asked for once per device: the kernel's shared memory and, for pairs, how
  // many run at once (clusters live inside a GPC, so perhaps not one per two SMs;
  // concurrent first calls find the same)
  static std::atomic<int> slots[kMaxDevices + 1];
  std::atomic<int> *slot = launch_slot(slots);
  if (slot == nullptr) return cudaErrorInvalidDevice;
  int most = slot < slots + kMaxDevices ? slot->load(std::memory_order_acquire) : 0;
  if (most <= 0) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(CF::kSmemBytes));
    if (e != cudaSuccess) return e;
    most = g.num_sms;
    if constexpr (PAIR) {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(g.num_sms / 2 * 2);
      cfg.blockDim = dim3(CF::kThreads);
      cfg.dynamicSmemBytes = CF::kSmemBytes;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&most, kern, &cfg) != cudaSuccess || most <= 0) {
        cudaGetLastError();
        most = g.num_sms / 2;
      }
    }
    slot->store(most, std::memory_order_release);
  }
  const long long tiles =
      ((long long)g.M + kCtas * BM - 1) / (kCtas * BM) * ((g.N + BN - 1) / BN);
  if (tiles > 0x7FFFFFFFll - 4ll * g.num_sms) return cudaErrorInvalidValue;
  const int workers = int(std::min<long long>(tiles, most));
  return launch_pdl(kern, dim3(workers * kCtas), dim3(CF::kThreads), CF::kSmemBytes, g.st, kCtas, m.a,
                    m.b, m.sa, m.sb, m.res, m.y, g.bias, g.M, g.N, g.K, g.status, pre, g.lost_tx);
}

template <int EPI, int SPLIT>
cudaError_t run_split(const Args &g) {
  using CF = Cfg<128, false>;
  Maps m;
  if (!encode_maps(m, g, 128, 1, false)) return cudaErrorInvalidValue;
  auto kern = gemm_mx4_split_kernel<EPI, SPLIT>;
  static std::atomic<int> slots[kMaxDevices + 1];
  std::atomic<int> *slot = launch_slot(slots);
  if (slot == nullptr) return cudaErrorInvalidDevice;
  if (slot == slots + kMaxDevices || slot->load(std::memory_order_acquire) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(CF::kSmemBytes));
    if (e != cudaSuccess) return e;
    slot->store(1, std::memory_order_release);
  }
  const int tiles = (g.M + BM - 1) / BM * ((g.N + 127) / 128);  // at most the SMs
  return launch_pdl(kern, dim3(tiles * SPLIT), dim3(CF::kThreads), CF::kSmemBytes, g.st, SPLIT,
                    m.a, m.b, m.sa, m.sb, g.bias, g.res, g.y, g.M, g.N, g.K, g.status, g.lost_tx);
}

template <int SPLIT>
cudaError_t run_split_epi(const Args &g, int epi) {
  switch (epi) {
    case kEpiGelu: return run_split<kEpiGelu, SPLIT>(g);
    case kEpiResidual: return run_split<kEpiResidual, SPLIT>(g);
    default: return run_split<kEpiBias, SPLIT>(g);
  }
}

template <int BN, bool PAIR>
cudaError_t run_epi(const Args &g, int epi) {
  switch (epi) {
    case kEpiGelu: return run<BN, kEpiGelu, PAIR>(g);
    case kEpiResidual: return run<BN, kEpiResidual, PAIR>(g);
    default: return run<BN, kEpiBias, PAIR>(g);
  }
}

// The tile's shape by a cost model.  Its constants (microseconds) are fitted to the
// order of the shapes over 3900 x {1152, 3456, 4304} x {1152, 4304}, 960 x 4304 x
// 1152, 10936 x 1152 x 4304 and 8192 x 4096 x 8192; its sums are not times (3900 x
// 4304 x 1152: 11.2 for 15.4 us; 10936 x 1152 x 4304: 26.6 for 35.9; 8192 x 4096 x
// 8192: 106 for 100), since the launch and rows that straddle lines are not in them.
// A round over the SMs takes a tile's k-blocks or its
// epilogue, whichever is longer (accumulators that share columns add a wait); the
// first round's k-blocks and the last one's epilogue are not overlapped, a pair
// starts later, and joining a split tile takes time by its rows and parts.
//  - One CTA wins with few k-blocks and tiles (960 x 4304 x 1152: 6.9 us, pairs
//    7.7 to 8.2; 3900 x 1152 x 1152: 9.1 against 9.4);
//  - 192 columns for the wide projections (3900 x 4304 x 1152: 15.4, 128 columns
//    17.9, 256 15.8, one CTA 18.1);
//  - 256 for the most work per byte (10936 x 1152 x 4304: 35.9, 192 columns 36.7, 128
//    41.7; 8192 x 4096 x 8192: 100, 109, 123);
//  - where it errs: 960 x 1152 x 4304 takes 10.6 us split over 2 CTAs, pairs of 128
//    columns 9.3; 10936 x 4304 x 1152 35.4 with 192 columns, 256 34.4;
//  - split tiles for few rows over a long K (1 x 1152 x 4304: 7.8, over 8 CTAs 4.1;
//    64 rows: 9.0, over 4 CTAs 7.3, over 8 8.6; 1 x 3456 x 1152: 3.7 either way).
struct Shape {
  int ctas, bn, split;
  float kblock, epilogue, wait, start;
};
constexpr Shape kShapes[] = {{1, 128, 1, 0.33f, 1.4f, 0.0f, 0.0f},
                             {1, 128, 2, 0.33f, 1.4f, 0.0f, 0.6f},
                             {1, 128, 4, 0.33f, 1.4f, 0.0f, 0.6f},
                             {1, 128, 8, 0.33f, 1.4f, 0.0f, 0.6f},
                             {2, 128, 1, 0.29f, 1.4f, 0.0f, 0.7f},
                             {2, 192, 1, 0.36f, 1.5f, 0.0f, 0.7f},
                             {2, 256, 1, 0.45f, 2.0f, 0.5f, 0.7f}};

const Shape &choose(int M, int N, int K, int num_sms) {
  const Shape *best = nullptr;
  float least = 0.f;
  const int k_blocks = (K + kBK - 1) / kBK;
  auto tiles_of = [&](const Shape &s) {
    return ((long long)M + s.ctas * BM - 1) / (s.ctas * BM) * ((N + s.bn - 1) / s.bn);
  };
  // a split tile's CTAs run at once, and each has a k-block
  auto fits = [&](const Shape &s) {
    return s.split == 1 || (s.split <= k_blocks && tiles_of(s) * s.split <= num_sms);
  };
  if (const char *f = getenv("VIT_MX4_TILE")) {  // e.g. "2x192": tuning and tests
    int c = 0, n = 0, k = 1;
    if (sscanf(f, "%dx%dx%d", &c, &n, &k) >= 2)
      for (const Shape &s : kShapes)
        if (s.ctas == c && s.bn == n && s.split == k && fits(s)) return s;
  }
  for (const Shape &s : kShapes) {
    if ((s.ctas == 2 && M <= BM) || !fits(s)) continue;  // one row of tiles: nothing to share
    const long long tiles = tiles_of(s);
    const float kb = float((k_blocks + s.split - 1) / s.split);
    const long long rounds = (tiles + num_sms / s.ctas - 1) / (num_sms / s.ctas);
    const float main = kb * s.kblock, period = std::max(main + s.wait, s.epilogue);
    const float join = s.split > 1 ? 0.0072f * float(std::min(M, BM) * s.split) : 0.f;
    const float cost = s.start + main + float(rounds - 1) * period + s.epilogue + join;
    if (best == nullptr || cost < least) {
      best = &s;
      least = cost;
    }
  }
  return *best;
}

}  // namespace

cudaError_t launch_gemm_mx4(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                            const uint8_t *w_scales, const void *b, const void *res, void *y, int M,
                            int N, int K, int epi, int num_sms, int *status, cudaStream_t st,
                            uint32_t lost_tx) {
  const Args g{a_codes, a_scales, w_codes, w_scales, static_cast<const __nv_bfloat16 *>(b),
               static_cast<const __nv_bfloat16 *>(res), static_cast<__nv_bfloat16 *>(y),
               M, N, K, num_sms, status, st, lost_tx};
  const Shape &s = choose(M, N, K, num_sms);
  if (s.split == 2) return run_split_epi<2>(g, epi);
  if (s.split == 4) return run_split_epi<4>(g, epi);
  if (s.split == 8) return run_split_epi<8>(g, epi);
  if (s.ctas == 1) return run_epi<128, false>(g, epi);
  if (s.bn == 128) return run_epi<128, true>(g, epi);
  return s.bn == 192 ? run_epi<192, true>(g, epi) : run_epi<256, true>(g, epi);
}

}  // namespace vit
