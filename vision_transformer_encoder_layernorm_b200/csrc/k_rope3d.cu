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
// are on their way.  16384 tokens x 32 heads of 128: 43.4 us (6200 GB/s, 96% of the
// measured copy rate); kept as fp32 in flight, the heads took 128 registers, left two
// blocks an SM and took 81 us.
#include "kernels.h"

namespace vit {

namespace {

// VEC elements in one access of up to 16 bytes, as they are stored.
template <typename T, int VEC>
struct Raw {
  static constexpr int W = VEC * int(sizeof(T)) / 4;  // 32-bit words; 0: one bf16
  uint32_t w[W ? W : 1];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (W == 4) {
      const uint4 r = *reinterpret_cast<const uint4 *>(p);
      w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
    } else if constexpr (W == 2) {
      const uint2 r = *reinterpret_cast<const uint2 *>(p);
      w[0] = r.x; w[1] = r.y;
    } else if constexpr (W == 1) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (W == 4) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (W == 2) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else if constexpr (W == 1) *reinterpret_cast<uint32_t *>(p) = w[0];
    else *reinterpret_cast<uint16_t *>(p) = uint16_t(w[0]);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (VEC == 1) {
      w[0] = pack_bf16x2(f[0], 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
  }
};

constexpr int kHeadBatch = 4;  // heads a thread has in flight

// Thread (v, g, t) takes VEC pairs of token t's heads g, g + groups, ...  x and y
// may be the same buffer: an element is read and written by one thread.
template <typename T, int VEC>
__global__ void __launch_bounds__(256, 3)
    rope3d_kernel(const T *x, long long xs, T *y, long long ys, const int32_t *__restrict__ pos,
                  int tokens, int heads, int d, const __grid_constant__ Rope3dTable tab) {
  extern __shared__ float2 cs[];  // [tok_per_block][d / 2] = (cos, sin)
  pdl_trigger();
  pdl_wait();
  // blockDim = (vectors of a head, head groups, tokens)
  const int pairs = d / 2, groups = blockDim.y, tok_per_block = blockDim.z;
  const int p0 = threadIdx.x * VEC, g = threadIdx.y, lt = threadIdx.z;
  const long long tok0 = (long long)blockIdx.x * tok_per_block;
  const long long t = tok0 + lt;
  const bool active = t < tokens;
  const int lo = tab.lo[p0], hi = tab.hi[p0];
  const T *xt = x + (active ? t : 0) * xs;
  T *yt = y + (active ? t : 0) * ys;
  Raw<T, VEC> a[kHeadBatch], b[kHeadBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kHeadBatch; ++k) {
      const int h = h0 + k * groups;
      if (active && h < heads) {
        a[k].load(xt + h * d + lo);
        b[k].load(xt + h * d + hi);
      }
    }
  };
  load(g);
  // a thread keeps to one pair, so that the table in the kernel's parameters,
  // where a warp's 32 different entries are 32 accesses, is read once
  const int tid = (lt * groups + g) * blockDim.x + threadIdx.x;
  const float inv = 1.0f / float(pairs);  // quotients of small integers, exact
  const int table_toks = int((float(blockDim.x * groups * tok_per_block) + 0.5f) * inv);
  const int first = int((float(tid) + 0.5f) * inv), p = tid - first * pairs;
  if (first < table_toks) {  // tokens the block fills at a time
    const uint64_t turn = tab.turn[p];
    const int32_t *pp = pos + 3 * tok0 + tab.axis[p];
#pragma unroll 1
    for (int tt = first; tt < tok_per_block; tt += table_toks) {
      if (tok0 + tt >= tokens) break;
      const uint64_t turns = uint64_t((long long)__ldg(pp + 3 * tt)) * turn;  // modulo one turn
      float sn, c;
      sincospif(float(int32_t(turns >> 32)) * 0x1p-31f, &sn, &c);
      cs[tt * pairs + p] = make_float2(c, sn);
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
          const float p = a[k].get(i), q = b[k].get(i);
          oa[i] = p * c[i] - q * sn[i];
          ob[i] = q * c[i] + p * sn[i];
        }
        a[k].set(oa);
        b[k].set(ob);
        a[k].store(yt + h * d + lo);
        b[k].store(yt + h * d + hi);
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
  const int tpb = std::min(64, std::max(1, 256 / (nv * groups)));  // 64: the most a block's z takes
  const long long blocks = ((long long)tokens + tpb - 1) / tpb;
  return launch_pdl(rope3d_kernel<T, VEC>, dim3(unsigned(blocks)), dim3(nv, groups, tpb),
                    sizeof(float2) * tpb * (d / 2), st, 1, static_cast<const T *>(x), xs,
                    static_cast<T *>(y), ys, pos, tokens, heads, d, tab);
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
