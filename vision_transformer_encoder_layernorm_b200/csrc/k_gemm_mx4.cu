// k_gemm_mx4.cu -- MXFP4 linear layer: y = epi(deq(A) deq(W)^T + b) with E2M1
// codes and one E8M0 scale per 32 elements of K on both sides (OCP
// Microscaling v1.0), fp32 accumulation in tensor memory, bf16 output.
//
// Structure (persistent over output tiles, one CTA per SM; the roles of
// gemm_tc_kernel): per 256-column k-block the producer brings 128 rows of A
// codes and the tile's rows of W codes (128 bytes a row, one 128-byte swizzle
// atom) and their scale blocks; the MMA lane copies the scales into TMEM
// (tcgen05.cp, 512 bytes per 128 rows x 128 columns) and issues four K = 64
// block-scaled MMAs.  MMA k reads bytes 2 (k & 1) and 2 (k & 1) + 1 of each
// row's scale word of the 128-column half k / 2.  MMAs that start past K are
// left out: their scale half need not exist.  Two accumulators let the
// epilogue of a tile overlap the next tile's main loop.
#include <cuda_bf16.h>

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
constexpr int kThreads = 320;                  // 2 role warps + 8 epilogue warps
constexpr int kEpiWarps = 8;
constexpr uint32_t kBufBytes = 2048;           // one staged 32 x 32 bf16 chunk
constexpr size_t kSmemLimit = 232448;          // dynamic shared memory of one CTA (227 KB)

struct __align__(16) Bars {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

template <int BN>
struct Cfg {
  static constexpr int kSfbBlocks = BN / 128;
  static constexpr uint32_t kSfOff = kATileBytes + BN * kBK / 2;
  static constexpr uint32_t kStageBytes = kSfOff + kSfBytes * (1 + kSfbBlocks);
  static constexpr uint32_t kAfterRing = 1024 + kEpiWarps * kBufBytes;  // barriers, staging
  static constexpr int kFit = int((kSmemLimit - 1024 - kAfterRing) / kStageBytes);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr size_t kSmemBytes = size_t(kStages) * kStageBytes + 1024 + kAfterRing;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kSfaCol = 2 * BN;      // 4 columns per 128-column half
  static constexpr uint32_t kSfbCol = 2 * BN + 8;  // 4 columns per half and 128 rows of W
  static_assert(kStageBytes % 1024 == 0, "stages keep the 1 KB alignment of the swizzled tiles");
  static_assert(kSfbCol + 8 * kSfbBlocks <= kTmemCols, "TMEM columns");
  static_assert(sizeof(Bars) <= 1024, "barrier block");
};

struct Epi {
  const __nv_bfloat16 *bias;  // [N] or null
  const __nv_bfloat16 *res;   // [M, N] (kEpiResidual)
};

// 32 columns of one row: accumulator r -> bias, GELU or residual -> bf16.
template <int EPI>
__device__ __forceinline__ void finish_chunk(const uint32_t (&r)[32], const uint4 (&bv)[4],
                                             const uint4 (&rv)[4], uint4 (&o)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t bw[4] = {bv[q].x, bv[q].y, bv[q].z, bv[q].w};
    const uint32_t rw[4] = {rv[q].x, rv[q].y, rv[q].z, rv[q].w};
    uint32_t ow[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo = __uint_as_float(r[8 * q + 2 * e]) + bf16_lo(bw[e]);
      float hi = __uint_as_float(r[8 * q + 2 * e + 1]) + bf16_hi(bw[e]);
      if constexpr (EPI == kEpiGelu) {
        lo = gemm::gelu_fast(lo);
        hi = gemm::gelu_fast(hi);
      }
      if constexpr (EPI == kEpiResidual) {
        lo += bf16_lo(rw[e]);
        hi += bf16_hi(rw[e]);
      }
      ow[e] = pack_bf16x2(lo, hi);
    }
    o[q] = make_uint4(ow[0], ow[1], ow[2], ow[3]);
  }
}

template <int BN, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_mx4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSa, const __grid_constant__ CUtensorMap tmSb,
                    const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Epi ep, int M,
                    int N, int K, int *status) {
  using CF = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  Bars *bars = reinterpret_cast<Bars *>(smem + size_t(CF::kStages) * CF::kStageBytes);
  volatile int *abort_flag = &bars->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_m = (M + BM - 1) / BM, num_n = (N + BN - 1) / BN;
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
      mbar_init(&bars->acc_empty[a], kEpiWarps);
    }
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
    tmem_alloc(&bars->tmem_base, CF::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
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
      for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
        const int mb = tile % num_m, nb = tile / num_m;
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait(&bars->empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
          uint8_t *sa = smem + size_t(stage) * CF::kStageBytes;
          mbar_arrive_expect_tx(&bars->full[stage], CF::kStageBytes);
          tma_load_2d(sa, &tmA, &bars->full[stage], kb * (kBK / 2), mb * BM);
          tma_load_2d(sa + kATileBytes, &tmB, &bars->full[stage], kb * (kBK / 2), nb * BN);
          const uint32_t full = smem_u32(&bars->full[stage]);
          tma_load_3d<false>(sa + CF::kSfOff, &tmSa, full, 0, 2 * kb, mb);
          tma_load_3d<false>(sa + CF::kSfOff + kSfBytes, &tmSb, full, 0, 2 * kb,
                             nb * CF::kSfbBlocks);
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == CF::kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) {
        for (int s = 0; s < CF::kStages; ++s)
          if (issued_mask & (1u << s)) gemm::drain_wait(&bars->full[s], (issued_parity >> s) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      bool any_mma = false;
      const uint32_t sfa_t = tmem + CF::kSfaCol, sfb_t = tmem + CF::kSfbCol;
      for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x, ++it) {
        const int a = it & 1;
        const uint32_t aphase = (it >> 1) & 1;
        if (!mbar_wait(&bars->acc_empty[a], aphase ^ 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem + uint32_t(a * BN);
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait(&bars->full[stage], phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + size_t(stage) * CF::kStageBytes);
          const uint32_t sb = sa + kATileBytes;
          const uint32_t ssf = sa + CF::kSfOff;
          const int mmas = min(4, (K - kb * kBK + 63) / 64);
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // 128-column halves
            if (2 * j >= mmas) break;
            tmem_cp_scales<false>(sfa_t + 4 * j, smem_desc(ssf + 512 * j, 0, 128, 0));
#pragma unroll
            for (int i = 0; i < CF::kSfbBlocks; ++i)
              tmem_cp_scales<false>(sfb_t + 4 * (j * CF::kSfbBlocks + i),
                                    smem_desc(ssf + kSfBytes * (1 + i) + 512 * j, 0, 128, 0));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= mmas) break;
            const uint64_t ad = smem_desc(sa + k * 32, 16, 1024, 2);
            const uint64_t bd = smem_desc(sb + k * 32, 16, 1024, 2);
            const int j = k >> 1, sf = 2 * (k & 1);
            mma_mx4_ss<false>(d_tmem, ad, bd, idesc_mx4(BM, BN, sf),
                              (sfa_t + 4 * j) | (uint32_t(sf) << 30),
                              (sfb_t + 4 * j * CF::kSfbBlocks) | (uint32_t(sf) << 30),
                              (kb | k) != 0);
          }
          any_mma = true;
          mma_commit(&bars->empty[stage]);
          if (++stage == CF::kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        mma_commit(&bars->acc_full[a]);
      }
      if (!ok && any_mma) {
        mma_commit(&bars->drain);
        gemm::drain_wait(&bars->drain, 0);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t *buf = reinterpret_cast<uint8_t *>(bars) + 1024 + (warp - 2) * kBufBytes;
    int it = 0;
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++it) {
      const int mb = tile % num_m, nb = tile / num_m;
      const int a = it & 1;
      const uint32_t aphase = (it >> 1) & 1;
      const int row0 = mb * BM + quarter * 32, row = row0 + lane;
      if (!mbar_wait(&bars->acc_full[a], aphase, abort_flag)) break;
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < BN / 64; ++i) {
        const int c = half * (BN / 64) + i;
        const int col0 = nb * BN + c * 32;
        uint32_t r[32];
        __syncwarp();
        tmem_ld32(tmem + uint32_t(a * BN) + (uint32_t(quarter * 32) << 16) + uint32_t(c * 32), r);
        uint4 bv[4] = {}, rv[4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (col0 + 8 * q < N) {  // N % 8 == 0: whole vectors
            if (ep.bias) bv[q] = __ldg(reinterpret_cast<const uint4 *>(ep.bias + col0) + q);
            if (EPI == kEpiResidual && row < M)
              rv[q] = __ldg(reinterpret_cast<const uint4 *>(ep.res + size_t(row) * N + col0) + q);
          }
        }
        tmem_ld_wait();
        uint4 o[4];
        finish_chunk<EPI>(r, bv, rv, o);
        // one 32 x 32 chunk through the warp's buffer (64-byte swizzle), then
        // one copy, clipped at M and N
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        const int sw = (lane >> 1) & 3;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4 *>(buf + lane * 64 + ((q ^ sw) << 4)) = o[q];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < M && col0 < N) {
          tma_store_2d(&tmY, buf, col0, row0);
          bulk_commit_group();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(&bars->acc_empty[a]);  // TMEM reads complete
    }
    if (lane == 0) bulk_wait_group<0>();  // the TMA stores have completed
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, CF::kTmemCols);
  }
  if (threadIdx.x == 0 && bars->abort_flag) report_status(status, kDevTimeout);
}

struct Maps {
  CUtensorMap a, b, sa, sb, y;
};

// Codes as [rows, bytes] with 128-byte boxes, scales as [block rows][k blocks]
// [512 bytes] with boxes of two k blocks, the output in 32 x 32 boxes.
bool encode_maps(Maps &m, const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                 const uint8_t *w_scales, void *y, int M, int N, int K, int b_rows, int sb_blocks) {
  const uint64_t kb = (uint64_t(K) + 127) / 128, bytes = (uint64_t(K) + 1) / 2;
  auto codes = [&](CUtensorMap *t, const uint8_t *p, int rows, int box) {
    return encode_tensor_map_2d(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, bytes, rows, mx4_row_bytes(K),
                                kBK / 2, box, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
  };
  auto scales = [&](CUtensorMap *t, const uint8_t *p, int rows, int box) {
    return encode_tensor_map_3d(t, CU_TENSOR_MAP_DATA_TYPE_UINT32, p, 128, kb,
                                (uint64_t(rows) + 127) / 128, 512, kb * 512, 128, 2, box,
                                CU_TENSOR_MAP_SWIZZLE_NONE) == CUDA_SUCCESS;
  };
  return codes(&m.a, a_codes, M, BM) && codes(&m.b, w_codes, N, b_rows) &&
         scales(&m.sa, a_scales, M, 1) && scales(&m.sb, w_scales, N, sb_blocks) &&
         encode_tensor_map_2d(&m.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, uint64_t(N) * 2, 32,
                              32, CU_TENSOR_MAP_SWIZZLE_64B) == CUDA_SUCCESS;
}

template <int BN, int EPI>
cudaError_t run(const Maps &m, const Epi &ep, int M, int N, int K, int num_sms, int *status,
                cudaStream_t st) {
  using CF = Cfg<BN>;
  auto kern = gemm_mx4_kernel<BN, EPI>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(CF::kSmemBytes));
  if (e != cudaSuccess) return e;
  const long long tiles = ((long long)M + BM - 1) / BM * ((N + BN - 1) / BN);
  if (tiles > 0x7FFFFFFFll - num_sms) return cudaErrorInvalidValue;
  const int grid = int(std::min<long long>(tiles, num_sms));
  return launch_pdl(kern, dim3(grid), dim3(kThreads), CF::kSmemBytes, st, 1, m.a, m.b, m.sa, m.sb,
                    m.y, ep, M, N, K, status);
}

}  // namespace

cudaError_t launch_gemm_mx4(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                            const uint8_t *w_scales, const void *b, const void *res, void *y, int M,
                            int N, int K, int epi, int num_sms, int *status, cudaStream_t st) {
  constexpr int BN = 128;
  Maps m;
  if (!encode_maps(m, a_codes, a_scales, w_codes, w_scales, y, M, N, K, BN, BN / 128))
    return cudaErrorInvalidValue;
  const Epi ep{static_cast<const __nv_bfloat16 *>(b), static_cast<const __nv_bfloat16 *>(res)};
  switch (epi) {
    case kEpiGelu: return run<BN, kEpiGelu>(m, ep, M, N, K, num_sms, status, st);
    case kEpiResidual: return run<BN, kEpiResidual>(m, ep, M, N, K, num_sms, status, st);
    default: return run<BN, kEpiBias>(m, ep, M, N, K, num_sms, status, st);
  }
}

}  // namespace vit
