// k_rmsnorm.cu -- root-mean-square norm with the residual's addition, its
// output in the context's type or as MXFP8:
//   h = x + residual (rounded once to the type, as a separate addition stores it)
//   y = h gamma / sqrt(mean(h^2) + eps)
//
// Bound: HBM.  x and residual are read once, h and y written once (8 bytes a
// bf16 element, 7 with MXFP8 codes); the row stays in registers between the
// sum of squares and the output.  10936 x 1152 with residual takes 19.9 us (5070
// GB/s, 79% of the measured copy rate), 3900 x 1152 to MXFP8 10.7 us: there all rows
// are resident at once, and a warp's 1250 instructions after its loads are what is
// left.
//
// Numerics.  The squares are summed in fp64, so neither large rows overflow nor
// long ones lose bits, and a bf16 output is the correctly rounded value of the
// formula for the stored h (ties to even, within 2^-40).  For rows of rms 2^-40 to 2^20 h 2^40 stays finite, and
// p = (h 2^40) gamma is exact in fp32 (8 + 8 significant bits) unless the output is
// below fp32's normal range too; times fp32 2^-40 / rms it is within 2 ulp, and a
// vector with a value that close to a bf16 border is redone with the product's
// rounding error and the second half of 1/rms.  Other rows, and vectors with an
// infinite result (p may overflow where the output does not), take fp64.  The
// MXFP8 codes are those of the bf16 output (mx8_quantize_kernel's rule), so they do
// not depend on how the sum is split over threads either.
// fp64 costs little here: a bf16 value becomes an fp64 one by moving its bits (a
// conversion instruction an element cost 1.3 us on 3900 x 1152 rows).
#include <cuda_fp8.h>

#include "kernels.h"
#include "mx8.h"
#include "sm100.cuh"

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
  // rounded once: for two bf16 values that is what rounding their fp32 sum gives
  // (where that sum is inexact one of them is below 2^-16 of the other, far from
  // moving it by half a step)
  static __device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 s = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                        *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&s);
  }
  static __device__ __forceinline__ uint4 add(const uint4 &a, const uint4 &b) {
    return make_uint4(add2(a.x, b.x), add2(a.y, b.y), add2(a.z, b.z), add2(a.w, b.w));
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
  static __device__ __forceinline__ uint4 add(const uint4 &a, const uint4 &b) {
    float u[4], v[4];
    unpack(a, u);
    unpack(b, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] += v[e];
    return pack(u);
  }
};

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t v) {
  return *reinterpret_cast<const __nv_bfloat162 *>(&v);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t *>(&v);
}

// The largest magnitudes of 8 bf16 values, in two halves; NaN drops out.
__device__ __forceinline__ __nv_bfloat162 max8(const uint4 &v) {
  return __hmax2(__hmax2(__habs2(as_bf16x2(v.x)), __habs2(as_bf16x2(v.y))),
                 __hmax2(__habs2(as_bf16x2(v.z)), __habs2(as_bf16x2(v.w))));
}

// 8 bf16 values times 2^40.
__device__ __forceinline__ uint4 scaled8(const uint4 &v) {
  const __nv_bfloat162 s = as_bf16x2(((127u + 40u) << 7) * 0x10001u);
  return make_uint4(as_u32(__hmul2_rn(as_bf16x2(v.x), s)), as_u32(__hmul2_rn(as_bf16x2(v.y), s)),
                    as_u32(__hmul2_rn(as_bf16x2(v.z), s)), as_u32(__hmul2_rn(as_bf16x2(v.w), s)));
}

// Closer to a bf16 midpoint than this, relative, a value counts as half-way: 1/rms
// is known to about 2^-43, so that exact ties arrive a little off.
constexpr float kTie = 0x1p-40f;

// An fp32 value that rounds to the same bf16 as v does: v rounded to fp32,
// moved off a bf16 midpoint to the side v lies on.
__device__ __forceinline__ float bf16_side(double v) {
  const float f = __double2float_rn(v);
  uint32_t u = __float_as_uint(f);
  if ((u & 0xFFFFu) == 0x8000u) {
    const double b = fabs(double(f)), a = fabs(v);
    u += a - b > b * kTie ? 1u : 0u;
    u -= b - a > b * kTie ? 1u : 0u;
  }
  return __uint_as_float(u);
}

// h gamma rstd of 8 bf16 columns, correctly rounded, for rows and values whose
// fp32 products leave the range.  Out of line: rarely taken, and
// inlined its registers halve the occupancy.
__device__ __noinline__ uint4 exact8(uint4 h, uint4 gamma, double rstd) {
  float a[8], g[8], o[8];
  RowVec<__nv_bfloat16>::unpack(h, a);
  RowVec<__nv_bfloat16>::unpack(gamma, g);
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = bf16_side(double(a[e]) * double(g[e]) * rstd);
  return RowVec<__nv_bfloat16>::pack(o);
}

// p (rh + rl), rounded to fp32 and moved off a bf16 midpoint to its own side; p
// exact, the product's error recovered by fused multiply-add.
__device__ __forceinline__ float bf16_side2(float p, float rh, float rl) {
  const float hi = p * rh;
  const float err = fmaf(p, rl, fmaf(p, rh, -hi));
  const float s = hi + err, rest = err - (s - hi);
  uint32_t u = __float_as_uint(s);
  if ((u & 0xFFFFu) == 0x8000u && fabsf(rest) > kTie * fabsf(s))
    u += (rest > 0.f) == (s > 0.f) ? 1u : ~0u;
  return __uint_as_float(u | (__float_as_uint(p) & 0x80000000u));  // -0 + 0 is 0
}

// Sum of squares of 16 bytes of a row.
template <typename T>
__device__ __noinline__ double exact_squares(uint4 v) {
  float a[RowVec<T>::N];
  RowVec<T>::unpack(v, a);
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < RowVec<T>::N; ++e) s = fma(double(a[e]), double(a[e]), s);
  return s;
}

// The same of a thread's vectors, times kSquareScale.  A normal bf16 value's
// magnitude times 2^128 is an fp64 one with its bits moved and one exponent bit
// set; what that makes of zeros and subnormals (below 2^-126) and of infinities
// and NaN (2^128 and up) the caller sees by the size of the row's sum, and asks
// for exact_squares.
template <typename T>
constexpr double kSquareScale = sizeof(T) == 2 ? 0x1p256 : 1.0;
template <typename T, int V>
__device__ __forceinline__ double moved_squares(const uint4 (&hv)[V]) {
  double part[4] = {};  // four chains
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t w[4] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (sizeof(T) == 2) {
        const double lo = __hiloint2double(int(((w[q] << 13) & 0x0FFFE000u) | 0x40000000u), 0);
        const double hi = __hiloint2double(int(((w[q] >> 3) & 0x0FFFE000u) | 0x40000000u), 0);
        part[(2 * q) & 3] = fma(lo, lo, part[(2 * q) & 3]);
        part[(2 * q + 1) & 3] = fma(hi, hi, part[(2 * q + 1) & 3]);
      } else {
        const double a = double(__uint_as_float(w[q]));
        part[q] = fma(a, a, part[q]);
      }
    }
  }
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// 1 / sqrt(v): fp32's, and one Newton step in fp64 (its error squared, 2^-44);
// the library's where v leaves the fp32 range.
__device__ __forceinline__ double inverse_root(double v) {
  if (!(v > 0x1p-100 && v < 0x1p100)) return rsqrt(v);
  const double r = double(rsqrtf(float(v)));
  return fma(0.5 * r, fma(-v * r, r, 1.0), r);
}

// A row takes blockDim.x threads (whole warps), thread t holding the 16-byte
// vectors t, t + blockDim.x, ... (V at most); blockDim.y rows a block.  MX8: y
// goes out as codes and scales; four neighbouring threads hold a 32-column group.
// The MX8 grid covers the padded rows of the last block row, whose scale
// bytes are 127.  x, res, h and y may be the same buffers row by row: a thread
// reads its vectors before it writes them, and no other thread touches them.
template <typename T, bool MX8, int V>
__global__ void __launch_bounds__(V == 5 ? 512 : 1024, V == 5 ? 2 : 1)
    rmsnorm_kernel(const T *x, const T *res, const T *__restrict__ gamma, T *h, T *y, int rows,
                   int cols, double inv_cols, float eps, uint8_t *__restrict__ codes,
                   uint8_t *__restrict__ scales, size_t row_bytes, int k_blocks) {
  using R = RowVec<T>;
  constexpr int N = R::N;
  __shared__ double red[32];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x, tpr = blockDim.x, lane = t & 31, row_warps = tpr >> 5;
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool active = row < rows;
  const int nvec = cols / N;
  const size_t base = size_t(active ? row : 0) * nvec;
  const uint4 *xr = reinterpret_cast<const uint4 *>(x) + base;
  const uint4 *rr = reinterpret_cast<const uint4 *>(res) + base;
  uint4 hv[V], rv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + tpr * i;
    hv[i] = rv[i] = make_uint4(0, 0, 0, 0);
    if (active && c < nvec) {
      hv[i] = xr[c];
      if (res != nullptr) rv[i] = rr[c];
    }
  }
  if (res != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      hv[i] = R::add(hv[i], rv[i]);
    }
  }
  if (h != nullptr && active) {
    uint4 *hr = reinterpret_cast<uint4 *>(h) + base;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + tpr * i;
      if (c < nvec) hr[c] = hv[i];
    }
  }
  double ss, mean;
  for (int pass = 0;; ++pass) {
    if (pass == 0) {
      ss = moved_squares<T, V>(hv);
    } else {
      ss = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) ss += exact_squares<T>(hv[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (row_warps > 1) {
      const int w0 = threadIdx.y * row_warps;
      if (lane == 0) red[w0 + (t >> 5)] = ss;
      __syncthreads();
      ss = 0.0;
      for (int w = 0; w < row_warps; ++w) ss += red[w0 + w];
    }
    mean = ss * (pass == 0 ? inv_cols * (1.0 / kSquareScale<T>) : inv_cols);
    if (sizeof(T) == 4 || pass > 0) break;
    // moved bits stand for the values where the sum is between these (padding
    // and zeros count 2^-254 each); a block's rows go together
    const bool fine = ss > kSquareScale<T> * 0x1p-180 && ss < kSquareScale<T> * 0x1p250;
    if (row_warps > 1 ? __syncthreads_and(fine) : fine) break;
  }
  const double rstd = inverse_root(mean + double(eps));
  const float r1 = float(rstd);
  // rows so large or small that their products might leave the fp32 range (and a
  // row of zeros without eps, or one with an infinity or NaN) take fp64 throughout
  const bool wide = sizeof(T) == 2 ? !(r1 > 0x1p-20f && r1 < 0x1p40f)
                                   : !(r1 > 0x1p-100f && r1 < 0x1p100f);
  // 1/rms in two halves, without the 2^40 that bf16 products have
  constexpr float kUnscale = sizeof(T) == 2 ? 0x1p-40f : 1.f;
  const float rh = r1 * kUnscale, rl = float(rstd - double(r1)) * kUnscale;
  const uint64_t rh2 = f2_pack(rh, rh);
  if constexpr (MX8) {
    if (row >= ((long long)rows + 127) / 128 * 128) return;  // whole row groups of threads
  } else {
    if (!active) return;
  }
  const uint4 *gr = reinterpret_cast<const uint4 *>(gamma);
  uint4 *yr = reinterpret_cast<uint4 *>(y) + base;
  uint8_t *crow = codes + (active ? size_t(row) * row_bytes : 0);
  uint8_t *srow = scales + size_t(row >> 7) * k_blocks * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + tpr * i;
    if (MX8 ? (c & ~31) >= 16 * k_blocks : c >= nvec) break;  // MX8: whole warps
    const bool ok = active && c < nvec;
    const uint4 gv = ok ? __ldg(gr + c) : make_uint4(0, 0, 0, 0);
    float a[N], g[N], o[N];
    R::unpack(gv, g);
    uint4 packed;
    __nv_bfloat162 m;
    if constexpr (N == 8) {
      R::unpack(scaled8(hv[i]), a);
      // o is less than 2 ulp off (1/rms and the product are rounded): only one
      // that is within 1 ulp of a bf16 midpoint may round to another bf16 than
      // the formula's value
      // (tested on the low halves of two values a word; the upper may take the
      // lower one's carry)
      uint32_t least = 0xFFFFFFFFu;
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const uint64_t p = f2_mul(f2_pack(a[e], a[e + 1]), f2_pack(g[e], g[e + 1]));  // exact
        f2_unpack(p, a[e], a[e + 1]);
        f2_unpack(f2_mul(p, rh2), o[e], o[e + 1]);
        least = __vminu2(least, __byte_perm(__float_as_uint(o[e]), __float_as_uint(o[e + 1]),
                                            0x5410) + 0x80018001u);
      }
      packed = R::pack(o);
      m = max8(packed);
      const bool inf = !__hblt2(m, as_bf16x2(0x7F807F80u));
      const bool near = wide || inf || min(least & 0xFFFFu, least >> 16) <= 3u;
      if (near) {
        bool out = wide || inf;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          out |= o[e] != 0.f && fabsf(o[e]) < 0x1p-90f;  // the error terms would be subnormal
          o[e] = bf16_side2(a[e], rh, rl);
        }
        packed = out ? exact8(hv[i], gv, rstd) : R::pack(o);
        m = max8(packed);
      }
    } else {
      R::unpack(hv[i], a);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float u = a[e] * rh;  // at most sqrt(cols)
        const bool far = fabsf(u) < 0x1p-126f && a[e] != 0.f;  // it has lost bits, and g may be large
        o[e] = wide || far ? float(double(a[e]) * double(g[e]) * rstd) : u * g[e];
      }
      packed = R::pack(o);
    }
    if constexpr (!MX8) {
      yr[c] = packed;
    } else {
      if (!ok) m = as_bf16x2(0u);  // its codes are not stored
      float q[N];
      R::unpack(packed, q);
      m = __hmax2(m, as_bf16x2(0u));  // NaN drops out, as in the quantiser
      const uint32_t mw = as_u32(m);
      uint32_t amax = max(mw & 0xFFFFu, mw >> 16);  // bf16 magnitudes order as integers
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int ef = int(amax >> 7);
      const int X = ef == 0 ? -127 : max(ef - 127 - 8, -127);
      const float inv = __uint_as_float(uint32_t(127 - X) << 23);
      if (ok) {
        uint32_t w[2];
#pragma unroll
        for (int e = 0; e < N; e += 2)
          f2_unpack(f2_mul(f2_pack(q[e], q[e + 1]), f2_pack(inv, inv)), q[e], q[e + 1]);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(
              make_float2(q[4 * p], q[4 * p + 1]), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(
              make_float2(q[4 * p + 2], q[4 * p + 3]), __NV_SATFINITE, __NV_E4M3);
          w[p] = (lo & 0xFFFFu) | ((hi & 0xFFFFu) << 16);
        }
        reinterpret_cast<uint2 *>(crow)[c] = make_uint2(w[0], w[1]);
      }
      if ((lane & 3) == 0 && c < 16 * k_blocks)
        srow[size_t(c >> 4) * 512 + ((c >> 2) & 3)] = ok ? uint8_t(X + 127) : uint8_t(127);
    }
  }
}

template <typename T, bool MX8, int V>
cudaError_t run(const void *x, const void *res, const void *gamma, void *h, void *y, int rows,
                int cols, float eps, uint8_t *codes, uint8_t *scales, int nvec, cudaStream_t st) {
  const int tpr = ((nvec + V - 1) / V + 31) / 32 * 32;
  const int rpb = std::max(1, 256 / tpr);  // rows of a block
  const long long all = MX8 ? ((long long)rows + 127) / 128 * 128 : rows;
  const long long grid = (all + rpb - 1) / rpb;
  return launch_pdl(rmsnorm_kernel<T, MX8, V>, dim3(unsigned(grid)), dim3(tpr, rpb), 0, st, 1,
                    static_cast<const T *>(x), static_cast<const T *>(res),
                    static_cast<const T *>(gamma), static_cast<T *>(h), static_cast<T *>(y), rows,
                    cols, 1.0 / cols, eps, codes, scales, MX8 ? mx8_row_bytes(cols) : size_t(0),
                    (cols + 127) / 128);
}

// Vectors a thread holds.  With few rows, one (the fewest a block of 1024 threads
// allows): each thread's code is short (1 row of 1152 columns 1.9 us, with five
// 3.0).  Where the rows need more threads than the SMs hold at once, five: the
// row's reduction and its root are then shared by more columns (10936 x 1152: 19.9
// us, with one 27.9, with three 20.6).
template <typename T, bool MX8>
cudaError_t pick(const void *x, const void *res, const void *gamma, void *h, void *y, int rows,
                 int cols, float eps, uint8_t *codes, uint8_t *scales, int num_sms,
                 cudaStream_t st) {
  // MX8 threads also cover the padding columns of the last 128-column block
  const int nvec = MX8 ? (cols + 127) / 128 * 16 : cols / RowVec<T>::N;
#define VIT_RMS(V) return run<T, MX8, V>(x, res, gamma, h, y, rows, cols, eps, codes, scales, nvec, st)
  if constexpr (sizeof(T) == 2) {
    const bool many = (long long)rows * nvec > 1024ll * num_sms;
    if (many && nvec > 64) VIT_RMS(5);
    if (many) VIT_RMS(2);
  }
  if (nvec <= 1024) VIT_RMS(1);
  if (nvec <= 2048) VIT_RMS(2);
  if constexpr (RowVec<T>::N == 4)
    if (nvec <= 4096) VIT_RMS(4);
#undef VIT_RMS
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rmsnorm(int dtype, const void *x, const void *res, const void *gamma, void *h,
                           void *y, int rows, int cols, float eps, int num_sms, cudaStream_t st) {
  return dtype == kF32 ? pick<float, false>(x, res, gamma, h, y, rows, cols, eps, nullptr, nullptr,
                                            num_sms, st)
                       : pick<__nv_bfloat16, false>(x, res, gamma, h, y, rows, cols, eps, nullptr,
                                                    nullptr, num_sms, st);
}

cudaError_t launch_rmsnorm_mx8(const void *x, const void *res, const void *gamma, void *h, int rows,
                               int cols, float eps, uint8_t *codes, uint8_t *scales, int num_sms,
                               cudaStream_t st) {
  return pick<__nv_bfloat16, true>(x, res, gamma, h, nullptr, rows, cols, eps, codes, scales,
                                   num_sms, st);
}

}  // namespace vit
