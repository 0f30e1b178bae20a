// k_mx4.cu -- bf16 <-> MXFP4 (OCP Microscaling v1.0: E2M1 elements two a
// byte, one E8M0 scale per 32 consecutive elements of a row).
//   X = floor(log2(amax)) - 2 (2 = exponent of E2M1's largest value, 6),
//       clamped to [-127, 127]; an all-zero group gets -127, a group with a
//       NaN the scale byte 255;
//   code = E2M1(x * 2^-X), round to nearest even, saturating at +-6.
// x * 2^-X is exact in fp32, so a code is decided as an exact reference
// decides it.
//
// Bound: HBM (2 bytes read, 17/32 written an element; the other way round for
// the dequantiser), with instructions close behind: at 6.4 TB/s an SM has about
// 16 issue slots an element.  The quantiser gives a thread a whole group, so the
// scale is found once for 32 elements; the dequantiser gives it 8 columns (a word
// of codes, 16 bytes out), so that its stores are whole lines.
#include <cuda_bf16.h>

#include "kernels.h"
#include "mx4.h"
#include "sm100.cuh"

namespace vit {

namespace {

constexpr int kBatch = 4;  // vectors of 8 columns a dequantising thread has in flight

// 8 columns from k0 (a multiple of 8) of a row of K; zeros past K.  ALIGN:
// elements that are sure to be aligned together at the row's start.
template <int ALIGN>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16 *row, int k0, int K) {
  if constexpr (ALIGN == 8) {  // K % 8 == 0: whole vectors
    return k0 < K ? __ldg(reinterpret_cast<const uint4 *>(row + k0)) : make_uint4(0, 0, 0, 0);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = k0 + 2 * q;
      if constexpr (ALIGN == 2) {
        w[q] = k < K ? __ldg(reinterpret_cast<const uint32_t *>(row + k)) : 0u;
      } else {
        const unsigned short *p = reinterpret_cast<const unsigned short *>(row + k);
        w[q] = (k < K ? uint32_t(__ldg(p)) : 0u) | (k + 1 < K ? uint32_t(__ldg(p + 1)) << 16 : 0u);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int ALIGN>
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int k0, int K, const uint32_t (&w)[4]) {
  if constexpr (ALIGN == 8) {
    if (k0 < K) *reinterpret_cast<uint4 *>(row + k0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = k0 + 2 * q;
      if constexpr (ALIGN == 2) {
        if (k < K) *reinterpret_cast<uint32_t *>(row + k) = w[q];
      } else {
        unsigned short *p = reinterpret_cast<unsigned short *>(row + k);
        if (k < K) p[0] = (unsigned short)(w[q]);
        if (k + 1 < K) p[1] = (unsigned short)(w[q] >> 16);
      }
    }
  }
}

// Four fp32 pairs as eight E2M1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t v) {
  return *reinterpret_cast<const __nv_bfloat162 *>(&v);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t *>(&v);
}

// A block takes rows_per_block rows, a thread one 32-column group at a time of
// their padded groups (4 per 128 columns, so that every scale byte is written).
template <int ALIGN>
__global__ void __launch_bounds__(512)
    mx4_quantize_kernel(const __nv_bfloat16 *__restrict__ x, int rows, int K, size_t row_bytes,
                        int k_blocks, int rows_per_block, uint8_t *__restrict__ codes,
                        uint8_t *__restrict__ scales) {
  pdl_trigger();
  pdl_wait();
  const int groups = (K + 31) / 32, pgroups = 4 * k_blocks;
  const long long row0 = (long long)blockIdx.x * rows_per_block;
  const long long prows = ((long long)rows + 127) / 128 * 128;
  const float inv_groups = 1.0f / float(pgroups);
  for (int u = threadIdx.x; u < rows_per_block * pgroups; u += blockDim.x) {
    // u / pgroups: one row, or few rows of few groups (below 2^10, exact in fp32)
    const int lr = rows_per_block == 1 ? 0 : int((float(u) + 0.5f) * inv_groups);
    const int j = u - lr * pgroups;
    const long long row = row0 + lr;
    if (row >= prows) return;
    const int rr = int(row & 127);
    uint8_t &scale = scales[(size_t(row >> 7) * k_blocks + (j >> 2)) * 512 + (rr & 31) * 16 +
                            (rr >> 5) * 4 + (j & 3)];
    if (row >= rows || j >= groups) {
      scale = 127;
      continue;
    }
    const __nv_bfloat16 *xr = x + size_t(row) * K;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load8<ALIGN>(xr, j * 32 + 8 * i, K);
    __nv_bfloat162 m = as_bf16x2(0u);  // largest magnitudes; NaN stays
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m = __hmax2_nan(m, __habs2(as_bf16x2(v[i].x)));
      m = __hmax2_nan(m, __habs2(as_bf16x2(v[i].y)));
      m = __hmax2_nan(m, __habs2(as_bf16x2(v[i].z)));
      m = __hmax2_nan(m, __habs2(as_bf16x2(v[i].w)));
    }
    const uint32_t amax = max(as_u32(m) & 0x7FFFu, (as_u32(m) >> 16) & 0x7FFFu);
    const bool nan = amax > 0x7F80u;
    const int byte = max(int(amax >> 7) - 2, 0);  // X + 127
    const float inv = __uint_as_float(uint32_t(254 - byte) << 23);
    const uint64_t inv2 = f2_pack(inv, inv);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      float f[8];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        f2_unpack(f2_mul(f2_pack(bf16_lo(w[q]), bf16_hi(w[q])), inv2), f[2 * q], f[2 * q + 1]);
      c[i] = nan ? 0u : e2m1x8(f);
    }
    *reinterpret_cast<uint4 *>(codes + size_t(row) * row_bytes + j * 16) =
        make_uint4(c[0], c[1], c[2], c[3]);
    scale = uint8_t(nan ? 255 : byte);
  }
}

// Four E2M1 codes (16 bits) as two bf16 words, times s (a power of two, twice).
// A magnitude's high and low byte are looked up by byte permutation (codes 0..7
// have bf16 bits 0000 3F00 3F80 3FC0 4000 4040 4080 40C0).  A third permutation
// takes the codes whole: a nibble's top bit makes it replicate the picked byte's
// top bit, FF for a negative code and 80 for a positive one, which shifted by one
// has the sign where the high byte wants it.
__device__ __forceinline__ void e2m1_to_bf16(uint32_t code, __nv_bfloat162 s, uint32_t &w0,
                                             uint32_t &w1) {
  const uint32_t c = code & 0x7777u;
  uint32_t sign;  // (the intrinsic ignores the selectors' top bits)
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(code));
  const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, c);
  const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, c) | ((sign << 1) & 0x80808080u);
  w0 = as_u32(__hmul2_rn(as_bf16x2(__byte_perm(lo, hi, 0x5140u)), s));
  w1 = as_u32(__hmul2_rn(as_bf16x2(__byte_perm(lo, hi, 0x7362u)), s));
}

// blockDim.y rows a block; a row's blockDim.x threads take 8 columns at a time,
// four loads in flight.
template <int ALIGN>
__global__ void __launch_bounds__(512)
    mx4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                          int rows, int K, size_t row_bytes, int k_blocks,
                          __nv_bfloat16 *__restrict__ y) {
  pdl_trigger();
  pdl_wait();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= rows) return;
  const int nvec = (K + 7) / 8, step = blockDim.x, rr = int(row & 127);
  const uint32_t *cr = reinterpret_cast<const uint32_t *>(codes + size_t(row) * row_bytes);
  const uint8_t *sr = scales + size_t(row >> 7) * k_blocks * 512 + (rr & 31) * 16 + (rr >> 5) * 4;
  __nv_bfloat16 *yr = y + size_t(row) * K;
  for (int j0 = threadIdx.x; j0 < nvec; j0 += kBatch * step) {
    uint32_t c[kBatch], sc[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i * step;
      c[i] = j < nvec ? __ldg(cr + j) : 0u;
      sc[i] = j < nvec ? __ldg(sr + size_t(j >> 4) * 512 + ((j >> 2) & 3)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i * step;
      if (j >= nvec) break;
      // 2^X in bf16: the byte is its exponent field (2^-127 is subnormal)
      const uint32_t b = sc[i] == 255u ? 0x7FC0u : sc[i] == 0u ? 0x0040u : sc[i] << 7;
      const __nv_bfloat162 s = as_bf16x2(b * 0x10001u);
      uint32_t w[4];
      e2m1_to_bf16(c[i], s, w[0], w[1]);
      e2m1_to_bf16(c[i] >> 16, s, w[2], w[3]);
      store8<ALIGN>(yr, j * 8, K, w);
    }
  }
}

// Rows of a block and its threads for rows of `units` thread-sized pieces: about
// `most` pieces a block, threads in whole warps with little left over.
struct Split {
  int rows, threads;
  Split(int units, int most) {
    rows = std::max(1, most / units);
    const int all = rows * units, turns = (all + 511) / 512;
    threads = std::min(512, ((all + turns - 1) / turns + 31) / 32 * 32);
  }
};

}  // namespace

cudaError_t launch_mx4_quantize(const void *x, int rows, int K, uint8_t *codes, uint8_t *scales,
                                cudaStream_t st) {
  const int k_blocks = (K + 127) / 128;
  const Split sp(4 * k_blocks, 512);
  const long long grid = (((long long)rows + 127) / 128 * 128 + sp.rows - 1) / sp.rows;
  auto kern = K % 8 == 0 ? mx4_quantize_kernel<8>
                         : K % 2 == 0 ? mx4_quantize_kernel<2> : mx4_quantize_kernel<1>;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(sp.threads), 0, st, 1,
                    static_cast<const __nv_bfloat16 *>(x), rows, K, mx4_row_bytes(K), k_blocks,
                    sp.rows, codes, scales);
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int rows, int K,
                                  void *y, cudaStream_t st) {
  // four vectors a thread, or two where that leaves a row under a warp of threads
  const int nvec = (K + 7) / 8, per = nvec >= 32 * kBatch ? kBatch : 2;
  const int tx = std::min(512, (nvec + per - 1) / per), ty = std::max(1, 256 / tx);
  const long long grid = ((long long)rows + ty - 1) / ty;
  auto kern = K % 8 == 0 ? mx4_dequantize_kernel<8>
                         : K % 2 == 0 ? mx4_dequantize_kernel<2> : mx4_dequantize_kernel<1>;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(tx, ty), 0, st, 1, codes, scales, rows, K,
                    mx4_row_bytes(K), (K + 127) / 128, static_cast<__nv_bfloat16 *>(y));
}

}  // namespace vit
