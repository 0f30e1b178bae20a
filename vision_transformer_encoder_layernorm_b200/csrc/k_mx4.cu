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
// the dequantiser).  A thread takes 8 columns at a time: 16 bytes of bf16 are
// one word of codes, 4 threads a group (two shuffles for its maximum), 16
// threads the 128 columns whose four scale bytes are one word.  A warp takes a
// segment of a row, at most 1024 columns, its loads issued together; a row's
// segments are of equal length, in 128-column blocks.
#include <cuda_bf16.h>
#include <cuda_fp4.h>

#include "kernels.h"
#include "mx4.h"

namespace vit {

namespace {

constexpr int kVecs = 4;  // 8-column vectors a thread holds: 1024 columns a warp

// Where a warp works: its row and its 128-column blocks [kb0, kb1).
struct Segment {
  long long row;
  int kb0, kb1;
};
__device__ __forceinline__ Segment segment_of(int k_blocks, int n_seg, int per) {
  const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  Segment s;
  s.row = w / n_seg;
  s.kb0 = int(w - s.row * n_seg) * per;
  s.kb1 = min(s.kb0 + per, k_blocks);
  return s;
}

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

template <int ALIGN>
__global__ void __launch_bounds__(256)
    mx4_quantize_kernel(const __nv_bfloat16 *__restrict__ x, int rows, int K, size_t row_bytes,
                        int k_blocks, int n_seg, int per, uint8_t *__restrict__ codes,
                        uint8_t *__restrict__ scales) {
  pdl_trigger();
  pdl_wait();
  const Segment s = segment_of(k_blocks, n_seg, per);
  if (s.row >= ((long long)rows + 127) / 128 * 128) return;  // whole warps
  const int lane = threadIdx.x & 31;
  const bool active = s.row < rows;  // the other rows only have padding scales
  const __nv_bfloat16 *xr = x + size_t(active ? s.row : 0) * K;
  uint8_t *cr = codes + size_t(active ? s.row : 0) * row_bytes;
  const int rr = int(s.row & 127);
  uint8_t *sr = scales + size_t(s.row >> 7) * k_blocks * 512 + (rr & 31) * 16 + (rr >> 5) * 4;
  uint4 v[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k0 = s.kb0 * 128 + (lane + 32 * i) * 8;
    v[i] = active && k0 < s.kb1 * 128 ? load8<ALIGN>(xr, k0, K) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k0 = s.kb0 * 128 + (lane + 32 * i) * 8;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    // magnitudes compare as integers, a NaN above all
    uint32_t m2 = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) m2 = __vmaxu2(m2, w[q] & 0x7FFF7FFFu);
    m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
    m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
    const uint32_t amax = max(m2 & 0xFFFFu, m2 >> 16);
    const int ef = int(amax >> 7);
    const bool nan = amax > 0x7F80u;
    const int byte = max(ef - 2, 0);  // X + 127
    const float inv = __uint_as_float(uint32_t(254 - byte) << 23);
    uint32_t code = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = make_float2(bf16_lo(w[q]) * inv, bf16_hi(w[q]) * inv);
      code |= uint32_t(__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest)) << (8 * q);
    }
    if (nan) code = 0;
    const bool in_row = active && (k0 & ~31) < K;  // the group has a column
    uint32_t word = uint32_t(!in_row ? 127 : nan ? 255 : byte) << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (k0 < s.kb1 * 128) {
      if (in_row) *reinterpret_cast<uint32_t *>(cr + k0 / 2) = code;
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(sr + size_t(k0 >> 7) * 512) = word;
    }
  }
}

// Eight E2M1 codes (one word) as bf16 words: a magnitude's high and low byte
// are looked up by byte permutation (codes 0..7 have bf16 bits 0000 3F00 3F80
// 3FC0 4000 4040 4080 40C0), the sign is the nibble's top bit.
__device__ __forceinline__ void e2m1_to_bf16(uint32_t code, uint32_t (&w)[4]) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t c = p == 0 ? code & 0xFFFFu : code >> 16;
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, c & 0x7777u);
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, c & 0x7777u);
    const uint32_t a = __byte_perm(lo, hi, 0x5140u), b = __byte_perm(lo, hi, 0x7362u);
    w[2 * p] = a | ((c & 0x8u) << 12) | ((c & 0x80u) << 24);
    w[2 * p + 1] = b | ((c & 0x800u) << 4) | ((c & 0x8000u) << 16);
  }
}

template <int ALIGN>
__global__ void __launch_bounds__(256)
    mx4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                          int rows, int K, size_t row_bytes, int k_blocks, int n_seg, int per,
                          __nv_bfloat16 *__restrict__ y) {
  pdl_trigger();
  pdl_wait();
  const Segment s = segment_of(k_blocks, n_seg, per);
  if (s.row >= rows) return;
  const int lane = threadIdx.x & 31;
  const uint8_t *cr = codes + size_t(s.row) * row_bytes;
  __nv_bfloat16 *yr = y + size_t(s.row) * K;
  const int rr = int(s.row & 127);
  const uint8_t *sr = scales + size_t(s.row >> 7) * k_blocks * 512 + (rr & 31) * 16 + (rr >> 5) * 4 +
                      ((lane >> 2) & 3);
  uint32_t v[kVecs], sc[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k0 = s.kb0 * 128 + (lane + 32 * i) * 8;
    const bool ok = k0 < s.kb1 * 128 && k0 < K;
    v[i] = ok ? __ldg(reinterpret_cast<const uint32_t *>(cr + k0 / 2)) : 0u;
    sc[i] = ok ? __ldg(sr + size_t(k0 >> 7) * 512) : 0u;
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k0 = s.kb0 * 128 + (lane + 32 * i) * 8;
    if (k0 >= s.kb1 * 128 || k0 >= K) break;
    // 2^X in bf16: the byte is its exponent field (2^-127 is subnormal)
    const uint32_t b = sc[i] == 255u ? 0x7FC0u : sc[i] == 0u ? 0x0040u : sc[i] << 7;
    const float f = __uint_as_float(b << 16);
    uint32_t w[4];
    e2m1_to_bf16(v[i], w);
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = pack_bf16x2(bf16_lo(w[q]) * f, bf16_hi(w[q]) * f);
    store8<ALIGN>(yr, k0, K, w);
  }
}

// Segments of a row: as few as hold it at 8 blocks of 128 columns each, their
// lengths equal to a block (1152 columns: 5 and 4 blocks, not 8 and 1).
struct Split {
  int k_blocks, n_seg, per;
  explicit Split(int K) {
    k_blocks = (K + 127) / 128;
    n_seg = (k_blocks + 2 * kVecs - 1) / (2 * kVecs);
    per = (k_blocks + n_seg - 1) / n_seg;
    n_seg = (k_blocks + per - 1) / per;
  }
};

}  // namespace

cudaError_t launch_mx4_quantize(const void *x, int rows, int K, uint8_t *codes, uint8_t *scales,
                                cudaStream_t st) {
  const Split sp(K);
  const long long warps = ((long long)rows + 127) / 128 * 128 * sp.n_seg;
  const long long grid = (warps + 7) / 8;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  auto kern = K % 8 == 0 ? mx4_quantize_kernel<8>
                         : K % 2 == 0 ? mx4_quantize_kernel<2> : mx4_quantize_kernel<1>;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(256), 0, st, 1,
                    static_cast<const __nv_bfloat16 *>(x), rows, K, mx4_row_bytes(K), sp.k_blocks,
                    sp.n_seg, sp.per, codes, scales);
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int rows, int K,
                                  void *y, cudaStream_t st) {
  const Split sp(K);
  const long long grid = ((long long)rows * sp.n_seg + 7) / 8;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  auto kern = K % 8 == 0 ? mx4_dequantize_kernel<8>
                         : K % 2 == 0 ? mx4_dequantize_kernel<2> : mx4_dequantize_kernel<1>;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(256), 0, st, 1, codes, scales, rows, K,
                    mx4_row_bytes(K), sp.k_blocks, sp.n_seg, sp.per,
                    static_cast<__nv_bfloat16 *>(y));
}

}  // namespace vit
