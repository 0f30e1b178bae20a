// k_rmsnorm.cu -- root-mean-square norm with the residual's addition, its
// output in the context's type or as MXFP8:
//   h = x + residual (rounded once to the type, as a separate addition stores it)
//   y = h gamma / sqrt(mean(h^2) + eps)
//
// Bound: HBM.  x and residual are read once, h and y written once (8 bytes a
// bf16 element, 7 with MXFP8 codes); the row stays in registers between the
// sum of squares and the output.
//
// Numerics.  The squares are summed in fp64 (one conversion and one DFMA an
// element, far below the fp64 rate at this bandwidth), so neither large rows
// overflow nor long ones lose bits, and a bf16 output is the correctly rounded
// value of the formula for the stored h: the product h gamma is exact in fp32
// (8 + 8 significant bits), times fp32 1/rms it is within 2 ulp, and the few
// values that close to a bf16 rounding border are recomputed in fp64.  The
// MXFP8 codes are those of the bf16 output (mx8_quantize_kernel's rule), so
// they do not depend on how the sum is split over threads either.
#include <cuda_fp8.h>

#include "kernels.h"
#include "mx8.h"

namespace vit {

namespace {

template <typename T>
struct RowVec;  // 16 bytes of a row as floats
template <>
struct RowVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &r, float (&f)[8]) {
    f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
    f[4] = bf16_lo(r.z); f[5] = bf16_hi(r.z); f[6] = bf16_lo(r.w); f[7] = bf16_hi(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct RowVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

// An fp32 value that rounds to the same bf16 as v does: v rounded to fp32,
// moved off a bf16 midpoint to the side v lies on.
__device__ __noinline__ float bf16_side(double v) {
  const float f = __double2float_rn(v);
  uint32_t u = __float_as_uint(f);
  if ((u & 0xFFFFu) == 0x8000u) {
    const double b = fabs(double(f)), a = fabs(v);
    u += a > b ? 1u : 0u;
    u -= a < b ? 1u : 0u;
  }
  return __uint_as_float(u);
}

// TPR threads per row (a divisor of the block), thread t holding the 16-byte
// vectors t, t + TPR, ... (V at most).  MX8: y goes out as codes and scales;
// four neighbouring threads hold a 32-column group, sixteen the 128 columns
// whose four scale bytes make one word of the scale blocks.  The MX8 grid
// covers the padded rows of the last block row, whose scale bytes are 127.
// x, res, h and y may be the same buffers row by row: a thread reads its
// vectors before it writes them, and no other thread touches them.
template <typename T, bool MX8, int TPR, int V>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    rmsnorm_kernel(const T *x, const T *res, const T *__restrict__ gamma, T *h, T *y, int rows,
                   int cols, float eps, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                   size_t row_bytes, int k_blocks) {
  using R = RowVec<T>;
  constexpr int N = R::N;
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  __shared__ double red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x % TPR, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  const bool active = row < rows;
  const int nvec = cols / N;
  const size_t base = size_t(active ? row : 0) * nvec;
  const uint4 *xr = reinterpret_cast<const uint4 *>(x) + base;
  const uint4 *rr = reinterpret_cast<const uint4 *>(res) + base;
  uint4 hv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + TPR * i;
    hv[i] = active && c < nvec ? xr[c] : make_uint4(0, 0, 0, 0);
  }
  if (res != nullptr) {
    uint4 rv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + TPR * i;
      rv[i] = active && c < nvec ? rr[c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float a[N], b[N];
      R::unpack(hv[i], a);
      R::unpack(rv[i], b);
#pragma unroll
      for (int e = 0; e < N; ++e) a[e] += b[e];
      hv[i] = R::pack(a);
    }
  }
  if (h != nullptr && active) {
    uint4 *hr = reinterpret_cast<uint4 *>(h) + base;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + TPR * i;
      if (c < nvec) hr[c] = hv[i];
    }
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float a[N];
    R::unpack(hv[i], a);
#pragma unroll
    for (int e = 0; e < N; ++e) ss = fma(double(a[e]), double(a[e]), ss);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if constexpr (TPR > 32) {
    if (lane == 0) red[threadIdx.x >> 5] = ss;
    __syncthreads();
    const int w0 = threadIdx.x / TPR * (TPR / 32);
    ss = 0.0;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) ss += red[w0 + w];
  }
  const double rstd = rsqrt(ss / double(cols) + double(eps));
  const float rh = float(rstd);
  // rows so large or small that h gamma might leave the fp32 range (and a row
  // of zeros without eps, or one with an infinity or NaN) take fp64 throughout
  const bool wide = !(rh > 0x1p-100f && rh < 0x1p100f);
  if constexpr (MX8) {
    if (row >= ((long long)rows + 127) / 128 * 128) return;  // whole row groups of threads
  } else {
    if (!active) return;
  }
  const uint4 *gr = reinterpret_cast<const uint4 *>(gamma);
  uint4 *yr = reinterpret_cast<uint4 *>(y) + base;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + TPR * i;
    if (MX8 ? (c & ~15) * N >= k_blocks * 128 : c >= nvec) break;
    const bool ok = active && c < nvec;
    float a[N], g[N], o[N];
    R::unpack(hv[i], a);
    R::unpack(ok ? __ldg(gr + c) : make_uint4(0, 0, 0, 0), g);
    if constexpr (N == 8) {
      bool near = wide;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        o[e] = (a[e] * g[e]) * rh;
        near |= ((__float_as_uint(o[e]) - 0x7FFDu) & 0xFFFFu) <= 6u;  // 3 ulp about a midpoint
      }
      if (near) {
#pragma unroll 1
        for (int e = 0; e < N; ++e) {
          float v = 0.f;  // o[e] by a runtime index would spill the arrays
#pragma unroll
          for (int q = 0; q < N; ++q)
            if (q == e) v = bf16_side(double(a[q]) * double(g[q]) * rstd);
#pragma unroll
          for (int q = 0; q < N; ++q)
            if (q == e) o[q] = v;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        o[e] = wide ? float(double(a[e]) * double(g[e]) * rstd) : (a[e] * rh) * g[e];
    }
    const uint4 packed = R::pack(o);
    if constexpr (!MX8) {
      yr[c] = packed;
    } else {
      float q[N];
      R::unpack(ok ? packed : make_uint4(0, 0, 0, 0), q);
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) amax = fmaxf(amax, fabsf(q[e]));
      // sixteen lanes hold 128 columns and none of them has left the loop
      const uint32_t mask = 0xFFFFu << (lane & 16);
      amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 2));
      const int ef = int(__float_as_uint(amax) >> 23) & 0xFF;
      const int X = ef == 0 ? -127 : max(ef - 127 - 8, -127);
      const float inv = __uint_as_float(uint32_t(127 - X) << 23);
      if (ok) {
        uint32_t w[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(
              make_float2(q[4 * p] * inv, q[4 * p + 1] * inv), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(
              make_float2(q[4 * p + 2] * inv, q[4 * p + 3] * inv), __NV_SATFINITE, __NV_E4M3);
          w[p] = (lo & 0xFFFFu) | ((hi & 0xFFFFu) << 16);
        }
        reinterpret_cast<uint2 *>(codes + size_t(row) * row_bytes)[c] = make_uint2(w[0], w[1]);
      }
      const bool group = active && (c & ~3) < nvec;  // the group has a column
      uint32_t word = uint32_t(group ? X + 127 : 127) << (8 * ((lane >> 2) & 3));
      word |= __shfl_xor_sync(mask, word, 4);
      word |= __shfl_xor_sync(mask, word, 8);
      if ((lane & 15) == 0) {
        const int r = int(row & 127);
        uint8_t *block = scales + (size_t(row >> 7) * k_blocks + (c >> 4)) * 512;
        *reinterpret_cast<uint32_t *>(block + (r & 31) * 16 + (r >> 5) * 4) = word;
      }
    }
  }
}

template <typename T, bool MX8, int TPR, int V>
cudaError_t run(const void *x, const void *res, const void *gamma, void *h, void *y, int rows,
                int cols, float eps, uint8_t *codes, uint8_t *scales, cudaStream_t st) {
  constexpr int threads = TPR > 256 ? TPR : 256;
  const long long all = MX8 ? ((long long)rows + 127) / 128 * 128 : rows;
  const long long grid = (all + threads / TPR - 1) / (threads / TPR);
  return launch_pdl(rmsnorm_kernel<T, MX8, TPR, V>, dim3(unsigned(grid)), dim3(threads), 0, st, 1,
                    static_cast<const T *>(x), static_cast<const T *>(res),
                    static_cast<const T *>(gamma), static_cast<T *>(h), static_cast<T *>(y), rows,
                    cols, eps, codes, scales, MX8 ? mx8_row_bytes(cols) : size_t(0),
                    (cols + 127) / 128);
}

// Threads per row by the row's vectors: a warp up to 160 (1280 bf16 columns),
// then 128 and 512 threads, so that a thread holds at most 5 (8 for the
// widest rows) and has all its loads in flight at once.
template <typename T, bool MX8>
cudaError_t pick(const void *x, const void *res, const void *gamma, void *h, void *y, int rows,
                 int cols, float eps, uint8_t *codes, uint8_t *scales, cudaStream_t st) {
  // MX8 threads also cover the padding columns of the last 128-column block
  const int nvec = MX8 ? (cols + 127) / 128 * 16 : cols / RowVec<T>::N;
#define VIT_RMS(TPR, V) return run<T, MX8, TPR, V>(x, res, gamma, h, y, rows, cols, eps, codes, scales, st)
  if (nvec <= 64) VIT_RMS(32, 2);
  if (nvec <= 160) VIT_RMS(32, 5);
  if (nvec <= 384) VIT_RMS(128, 3);
  if (nvec <= 640) VIT_RMS(128, 5);
  if (nvec <= 2048) VIT_RMS(512, 4);
  if constexpr (RowVec<T>::N == 4) VIT_RMS(512, 8);
#undef VIT_RMS
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rmsnorm(int dtype, const void *x, const void *res, const void *gamma, void *h,
                           void *y, int rows, int cols, float eps, cudaStream_t st) {
  return dtype == kF32
             ? pick<float, false>(x, res, gamma, h, y, rows, cols, eps, nullptr, nullptr, st)
             : pick<__nv_bfloat16, false>(x, res, gamma, h, y, rows, cols, eps, nullptr, nullptr, st);
}

cudaError_t launch_rmsnorm_mx8(const void *x, const void *res, const void *gamma, void *h, int rows,
                               int cols, float eps, uint8_t *codes, uint8_t *scales,
                               cudaStream_t st) {
  return pick<__nv_bfloat16, true>(x, res, gamma, h, nullptr, rows, cols, eps, codes, scales, st);
}

}  // namespace vit
