// k_rope3d.cu -- rotary positions over three axes (time, row, column), for
// images and video.
//
// Pair p of a head (d/2 of them) has an axis and a frequency w_p; at position
// pos[axis] it is turned by the angle pos[axis] w_p:
//   (a, b) -> (a cos - b sin, b cos + a sin).
//
// Angles.  A frequency is held as w / 2 pi in 64-bit fixed point, in turns:
// pos times it, modulo 2^64, is the angle's fraction of a turn.  The host's
// fp64 frequency is what limits it (2^-23 turns at position 2^31; an fp32
// product is off by a radian at 10^7).  The top 32 bits become fp32 and go
// through sincospif.
//
// Bound: HBM, each element read once and written once.  A thread holds VEC
// pairs (up to 16 bytes of each half) of one token and keeps their cos and sin
// in registers over the token's heads, four heads' loads in flight at a time;
// the block's cos/sin table (tokens x d/2) is computed while the first four
// are on their way.
#include "kernels.h"

namespace vit {

namespace {

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[VEC]) {
  if constexpr (VEC * sizeof(T) == 2) {
    f[0] = to_f32(p[0]);
  } else {
    constexpr int W = VEC * int(sizeof(T)) / 4;
    uint32_t w[W];
    if constexpr (W == 4) {
      const uint4 r = *reinterpret_cast<const uint4 *>(p);
      w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
    } else if constexpr (W == 2) {
      const uint2 r = *reinterpret_cast<const uint2 *>(p);
      w[0] = r.x; w[1] = r.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      f[i] = sizeof(T) == 4 ? __uint_as_float(w[i * W / VEC])
                            : (i & 1) ? bf16_hi(w[i * W / VEC]) : bf16_lo(w[i * W / VEC]);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[VEC]) {
  if constexpr (VEC * sizeof(T) == 2) {
    p[0] = from_f32<T>(f[0]);
  } else {
    constexpr int W = VEC * int(sizeof(T)) / 4;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
    if constexpr (W == 4) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (W == 2) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(p) = w[0];
  }
}

constexpr int kHeadBatch = 4;  // heads a thread has in flight

// Threads of a block: (token, head group, vector of VEC pairs); thread (t, g,
// v) takes heads g, g + groups, ...  x and y may be the same buffer: an
// element is read and written by one thread.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
    rope3d_kernel(const T *x, long long xs, T *y, long long ys, const int32_t *__restrict__ pos,
                  int tokens, int heads, int d, int groups, int tok_per_block,
                  const __grid_constant__ Rope3dTable tab) {
  extern __shared__ float2 cs[];  // [tok_per_block][d / 2] = (cos, sin)
  pdl_trigger();
  pdl_wait();
  const int pairs = d / 2, nv = pairs / VEC, per_tok = nv * groups;
  const int lt = threadIdx.x / per_tok, u = threadIdx.x - lt * per_tok;
  const int g = u / nv, p0 = (u - g * nv) * VEC;
  const long long tok0 = (long long)blockIdx.x * tok_per_block;
  const long long t = tok0 + lt;
  const bool active = lt < tok_per_block && t < tokens;
  const int lo = tab.lo[p0], hi = tab.hi[p0];
  const T *xt = x + (active ? t : 0) * xs;
  T *yt = y + (active ? t : 0) * ys;
  float a[kHeadBatch][VEC], b[kHeadBatch][VEC];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kHeadBatch; ++k) {
      const int h = h0 + k * groups;
      if (active && h < heads) {
        load_vec<T, VEC>(xt + (long long)h * d + lo, a[k]);
        load_vec<T, VEC>(xt + (long long)h * d + hi, b[k]);
      }
    }
  };
  load(g);
  for (int i = threadIdx.x; i < tok_per_block * pairs; i += blockDim.x) {
    const int tt = i / pairs, p = i - tt * pairs;
    if (tok0 + tt < tokens) {
      const long long m = pos[3 * (tok0 + tt) + tab.axis[p]];
      const uint64_t turns = uint64_t(m) * tab.turn[p];  // modulo one turn
      float sn, c;
      sincospif(float(int32_t(turns >> 32)) * 0x1p-31f, &sn, &c);
      cs[i] = make_float2(c, sn);
    }
  }
  __syncthreads();
  if (!active) return;
  float c[VEC], sn[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float2 v = cs[lt * pairs + p0 + i];
    c[i] = v.x;
    sn[i] = v.y;
  }
  for (int h0 = g;;) {
#pragma unroll
    for (int k = 0; k < kHeadBatch; ++k) {
      const int h = h0 + k * groups;
      if (h < heads) {
        float oa[VEC], ob[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          oa[i] = a[k][i] * c[i] - b[k][i] * sn[i];
          ob[i] = b[k][i] * c[i] + a[k][i] * sn[i];
        }
        store_vec<T, VEC>(yt + (long long)h * d + lo, oa);
        store_vec<T, VEC>(yt + (long long)h * d + hi, ob);
      }
    }
    h0 += kHeadBatch * groups;
    if (h0 >= heads) break;
    load(h0);
  }
}

template <typename T, int VEC>
cudaError_t run(const void *x, long long xs, void *y, long long ys, const int32_t *pos, int tokens,
                int heads, int d, const Rope3dTable &tab, cudaStream_t st) {
  const int nv = d / 2 / VEC;
  // four heads a thread where the block's 256 threads allow it
  const int groups = std::max(1, std::min((heads + kHeadBatch - 1) / kHeadBatch, 256 / nv));
  const int tpb = std::max(1, 256 / (nv * groups));
  const int threads = (tpb * nv * groups + 31) / 32 * 32;
  const long long blocks = ((long long)tokens + tpb - 1) / tpb;
  return launch_pdl(rope3d_kernel<T, VEC>, dim3(unsigned(blocks)), dim3(threads),
                    sizeof(float2) * tpb * (d / 2), st, 1, static_cast<const T *>(x), xs,
                    static_cast<T *>(y), ys, pos, tokens, heads, d, groups, tpb, tab);
}

}  // namespace

// VEC: the widest access of at most 16 bytes that stays inside every pair
// block (vec, from the table) and keeps the rows' alignment.
cudaError_t launch_rope3d(int dtype, const void *x, long long xs, void *y, long long ys,
                          const int32_t *pos, int tokens, int heads, int d, const Rope3dTable &tab,
                          int vec, cudaStream_t st) {
  const int es = dtype == kF32 ? 4 : 2;
  const uint64_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) |
                        uint64_t(xs * es) | uint64_t(ys * es) | uint64_t(vec * es) |
                        uint64_t(d * es) | 16u;
  const int bytes = int(bits & (~bits + 1));  // largest power of two that divides all
#define VIT_ROPE3(T, V) return run<T, V>(x, xs, y, ys, pos, tokens, heads, d, tab, st)
  if (dtype == kF32) {
    if (bytes >= 16) VIT_ROPE3(float, 4);
    if (bytes >= 8) VIT_ROPE3(float, 2);
    VIT_ROPE3(float, 1);
  }
  if (bytes >= 16) VIT_ROPE3(__nv_bfloat16, 8);
  if (bytes >= 8) VIT_ROPE3(__nv_bfloat16, 4);
  if (bytes >= 4) VIT_ROPE3(__nv_bfloat16, 2);
  VIT_ROPE3(__nv_bfloat16, 1);
#undef VIT_ROPE3
}

}  // namespace vit
