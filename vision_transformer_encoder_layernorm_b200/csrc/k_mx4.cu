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
// of codes, 16 bytes out), so that its stores are whole lines.  10936 x 4304: 20.2
// us (5910 GB/s, 92% of the measured copy rate) and 23.3 us (5120 GB/s, 72% of the
// issue slots).
#include <cuda_bf16.h>

#include "kernels.h"
#include "mx4.h"
#include "sm100.cuh"

namespace vit {

namespace {

constexpr int kBatch = 4;  // vectors of 8 columns a dequantising thread has in flight

// Rows of K % 8 != 0 columns start anywhere in a 16-byte vector.  Memory is still
// read and written in whole aligned vectors, and shifted in registers: 3900 x 1151
// takes 4.6 and 5.8 us (3900 x 1152: 4.2 and 3.7), by accesses of one bf16 at a time
// 10.1 and 20.3.

// 32 elements from element `at` of x (n elements in all, 16-byte aligned), the ones
// past n zero.
__device__ __forceinline__ void load_group(const __nv_bfloat16 *x, size_t at, size_t n,
                                           uint32_t (&w)[16]) {
  const int e = int(at & 7);
  const uint4 *p = reinterpret_cast<const uint4 *>(x) + at / 8;
  uint32_t a[20];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const size_t first = at - e + 8 * i;  // of the vector
    uint4 v = make_uint4(0, 0, 0, 0);
    if (first + 8 <= n) {
      if (i < 4 || e) v = __ldg(p + i);
    } else if (first < n) {  // the tensor's last, unfinished vector
      uint32_t t[4] = {};
      for (int q = 0; q < int(n - first); ++q) {
        const uint32_t h = reinterpret_cast<const uint16_t *>(x)[first + q];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u == q / 2) t[u] |= h << (16 * (q & 1));
      }
      v = make_uint4(t[0], t[1], t[2], t[3]);
    }
    a[4 * i] = v.x; a[4 * i + 1] = v.y; a[4 * i + 2] = v.z; a[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < 18; ++i) a[i] = (e & 4) ? a[i + 2] : a[i];
#pragma unroll
  for (int i = 0; i < 17; ++i) a[i] = (e & 2) ? a[i + 1] : a[i];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = __byte_perm(a[i], a[i + 1], (e & 1) ? 0x5432u : 0x3210u);
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
template <bool ALIGNED>
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
    uint32_t v[16];
    const size_t at = size_t(row) * K + j * 32;
    const int n = K - j * 32;
    if constexpr (ALIGNED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 r = 8 * i < n ? __ldg(reinterpret_cast<const uint4 *>(x + at) + i)
                                  : make_uint4(0, 0, 0, 0);
        v[4 * i] = r.x; v[4 * i + 1] = r.y; v[4 * i + 2] = r.z; v[4 * i + 3] = r.w;
      }
    } else {
      load_group(x, at, size_t(rows) * K, v);
      if (n < 32) {  // what follows is the next row's
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[i] = 2 * i + 1 < n ? v[i] : 2 * i < n ? v[i] & 0xFFFFu : 0u;
      }
    }
    __nv_bfloat162 m = as_bf16x2(0u);  // largest magnitudes; NaN stays
#pragma unroll
    for (int i = 0; i < 16; ++i) m = __hmax2_nan(m, __habs2(as_bf16x2(v[i])));
    const uint32_t amax = max(as_u32(m) & 0x7FFFu, (as_u32(m) >> 16) & 0x7FFFu);
    const bool nan = amax > 0x7F80u;
    const int byte = max(int(amax >> 7) - 2, 0);  // X + 127
    const float inv = __uint_as_float(uint32_t(254 - byte) << 23);
    const uint64_t inv2 = f2_pack(inv, inv);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[8];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        f2_unpack(f2_mul(f2_pack(bf16_lo(v[4 * i + q]), bf16_hi(v[4 * i + q])), inv2), f[2 * q],
                  f[2 * q + 1]);
      c[i] = nan ? 0u : e2m1x8(f);
    }
    *reinterpret_cast<uint4 *>(codes + size_t(row) * row_bytes + j * 16) =
        make_uint4(c[0], c[1], c[2], c[3]);
    scale = uint8_t(nan ? 255 : byte);
  }
}

// Four E2M1 codes (16 bits) as two bf16 words, times s0 and s1 (powers of two for
// the two values of a word each).  A magnitude's high and low byte are looked up
// by byte permutation (codes 0..7 have bf16 bits 0000 3F00 3F80 3FC0 4000 4040 4080
// 40C0).  A third permutation takes the codes whole: a nibble's top bit makes it
// replicate the picked byte's top bit, FF for a negative code and 80 for a positive
// one, which shifted by one has the sign where the high byte wants it.
__device__ __forceinline__ void e2m1_to_bf16(uint32_t code, uint32_t s0, uint32_t s1, uint32_t &w0,
                                             uint32_t &w1) {
  const uint32_t c = code & 0x7777u;
  uint32_t sign;  // (the intrinsic ignores the selectors' top bits)
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(code));
  const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, c);
  const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, c) | ((sign << 1) & 0x80808080u);
  w0 = as_u32(__hmul2_rn(as_bf16x2(__byte_perm(lo, hi, 0x5140u)), as_bf16x2(s0)));
  w1 = as_u32(__hmul2_rn(as_bf16x2(__byte_perm(lo, hi, 0x7362u)), as_bf16x2(s1)));
}

// 2^X in bf16, twice: the scale byte is its exponent field (2^-127 is subnormal,
// 255 is NaN).
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t byte) {
  return (byte == 255u ? 0x7FC0u : byte == 0u ? 0x0040u : byte << 7) * 0x10001u;
}

// blockDim.y rows a block; a row's blockDim.x threads take its 16-byte vectors, four
// loads in flight.  With the row's first column e elements into a vector, vector m
// holds columns 8 m - e on: its codes are those of word m and the e nibbles before
// it, which may belong to the group before.
template <bool ALIGNED>
__global__ void __launch_bounds__(512)
    mx4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                          int rows, int K, size_t row_bytes, int k_blocks,
                          __nv_bfloat16 *__restrict__ y) {
  pdl_trigger();
  pdl_wait();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= rows) return;
  const size_t r0 = size_t(row) * K;
  const int e = ALIGNED ? 0 : int(r0 & 7);
  const int nvec = (K + e + 7) / 8, words = (K + 7) / 8, step = blockDim.x, rr = int(row & 127);
  const uint32_t *cr = reinterpret_cast<const uint32_t *>(codes + size_t(row) * row_bytes);
  const uint8_t *sr = scales + size_t(row >> 7) * k_blocks * 512 + (rr & 31) * 16 + (rr >> 5) * 4;
  auto scale_at = [&](int m) {
    return uint32_t(__ldg(sr + size_t(m >> 4) * 512 + ((m >> 2) & 3)));
  };
  // which values of a vector are the e of the word before
  uint32_t before[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) before[q] = 2 * q + 1 < e ? ~0u : 2 * q < e ? 0xFFFFu : 0u;
  __nv_bfloat16 *yr = y + r0 - e;
  for (int j0 = threadIdx.x; j0 < nvec; j0 += kBatch * step) {
    uint32_t c[kBatch], sc[kBatch], sp[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int m = j0 + i * step;
      c[i] = m < words ? __ldg(cr + m) : 0u;
      sp[i] = sc[i] = m < nvec ? scale_at(min(m, words - 1)) : 0u;
      if (!ALIGNED && e && m < nvec) {
        c[i] = __funnelshift_rc(m > 0 ? __ldg(cr + m - 1) : 0u, c[i], 4 * (8 - e));
        if ((m & 3) == 0 && m > 0) sp[i] = scale_at(m - 1);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int m = j0 + i * step;
      if (m >= nvec) break;
      const uint32_t cur = scale_bf16x2(sc[i]);
      uint32_t s[4] = {cur, cur, cur, cur};
      if constexpr (!ALIGNED) {
        const uint32_t prev = scale_bf16x2(sp[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] = (prev & before[q]) | (cur & ~before[q]);
      }
      uint32_t w[4];
      e2m1_to_bf16(c[i], s[0], s[1], w[0], w[1]);
      e2m1_to_bf16(c[i] >> 16, s[2], s[3], w[2], w[3]);
      const int k0 = 8 * m - e;
      if (ALIGNED || (k0 >= 0 && k0 + 8 <= K)) {
        *reinterpret_cast<uint4 *>(yr + 8 * m) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {  // a vector that the row shares with its neighbours
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (k0 + q >= 0 && k0 + q < K)
            reinterpret_cast<uint16_t *>(yr)[8 * m + q] = uint16_t(w[q / 2] >> (16 * (q & 1)));
      }
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
  auto kern = K % 8 == 0 ? mx4_quantize_kernel<true> : mx4_quantize_kernel<false>;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(sp.threads), 0, st, 1,
                    static_cast<const __nv_bfloat16 *>(x), rows, K, mx4_row_bytes(K), k_blocks,
                    sp.rows, codes, scales);
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int rows, int K,
                                  void *y, cudaStream_t st) {
  // four vectors a thread, or two where that leaves a row under a warp of threads
  const int nvec = (K + 7) / 8, per = nvec >= 32 * kBatch ? kBatch : 2;
  int tx = std::min(512, (nvec + per - 1) / per);
  if (K % 8) tx = (tx + 31) / 32 * 32;  // a warp's threads share a row's shift
  const int ty = std::max(1, 256 / tx);
  const long long grid = ((long long)rows + ty - 1) / ty;
  auto kern = K % 8 == 0 ? mx4_dequantize_kernel<true> : mx4_dequantize_kernel<false>;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(tx, ty), 0, st, 1, codes, scales, rows, K,
                    mx4_row_bytes(K), (K + 127) / 128, static_cast<__nv_bfloat16 *>(y));
}

}  // namespace vit
