// mx4.h -- host-side declarations of the MXFP4 (block-scaled E2M1) kernels.
//
// Layouts (OCP Microscaling v1.0, MXFP4):
//   codes  [rows, mx4_row_bytes(K)] uint8, two elements a byte: element (r, k)
//          in the low (even k) or high (odd k) nibble of byte
//          r * row_bytes + k / 2.  A code is sign | 2 exponent bits (bias 1)
//          | 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.
//          Nibbles at k >= K are zero.
//   scales one E8M0 byte (2^(s-127)) per 32 consecutive elements of a row, in
//          the 512-byte blocks of the MXFP8 scales (mx8.h).  255 (NaN) marks a
//          group that holds a NaN, which E2M1 cannot express.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace vit {

inline size_t mx4_row_bytes(int K) { return (size_t(K) + 31) / 32 * 16; }
inline size_t mx4_scale_bytes(int rows, int K) {
  return (size_t(rows) + 127) / 128 * ((size_t(K) + 127) / 128) * 512;
}

// bf16 [rows, K] (row stride K) -> codes and scales, and back to bf16.
cudaError_t launch_mx4_quantize(const void *x, int rows, int K, uint8_t *codes, uint8_t *scales,
                                cudaStream_t st);
cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int rows, int K,
                                  void *y, cudaStream_t st);

// y[M, N] (bf16) = epi(deq(A) . deq(W)^T + b): A codes/scales [M, K], W
// codes/scales [N, K]; epi: kEpiBias, kEpiGelu or kEpiResidual.  lost_tx: fault
// injection for the watchdog tests (0 in normal use), the bytes that a stage barrier
// expects beyond those that arrive.
cudaError_t launch_gemm_mx4(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                            const uint8_t *w_scales, const void *b, const void *res, void *y, int M,
                            int N, int K, int epi, int num_sms, int *status, cudaStream_t st,
                            uint32_t lost_tx = 0);

}  // namespace vit
