// gemm_common.cuh -- device helpers shared by the tensor-core GEMM kernels.
#pragma once
#include "sm100.cuh"

namespace vit {
namespace gemm {

__device__ __forceinline__ float tanh_fast(float x) {
  float y;
  asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float gelu_fast(float u) {
  const float k0 = 0.7978845608028654f, k1 = 0.044715f;
  return 0.5f * u * (1.0f + tanh_fast(k0 * fmaf(k1 * u, u * u, u)));
}

// Waits bounded by time only (used while draining after an abort).
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > 200000000ull) break;  // 200 ms
  }
}

// After an abort: time for copies into shared memory that no barrier is waited on for.
__device__ __forceinline__ void settle() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 2000000ull) {  // 2 ms
  }
}

}  // namespace gemm
}  // namespace vit
