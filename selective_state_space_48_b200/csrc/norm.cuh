// norm.cuh -- shared parts of the RMS norm kernels (norm_fwd.cu,
// norm_bwd.cu): parameters, the mapping of a row onto threads, vector loads
// and the sums over a row.
//
// A row is one (token, group) pair of gs channels.  Its threads hold it in
// registers, NV pieces of 8 channels each, so every input is read once:
// vectors of 8 neighbouring channels where sizes, strides and addresses
// allow (VEC), else channels as far apart as there are threads, so that a
// warp's scalar accesses still fall into whole sectors.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device_math.cuh"
#include "norm.h"

namespace sss48 {
namespace norm {

constexpr int kGateAfter = 0, kGateBefore = 1, kAdd = 2;  // MODE
constexpr int64_t kMaxGroup = 16384;

struct Params {
  int64_t rows;
  int ng, gs;   // groups of a row, channels of a group (add: 1, width)
  int shared;   // one weight for every group
  float eps, inv;  // 1 / gs
  const void *x, *z;      // add: x, residual
  const float *weight, *scale;
  void *y, *res;          // res: residual_out
  const void *dy, *dres;  // dres: dresidual_out
  void *dx, *dz;          // add: dx, dresidual
  int64_t sx, sz, sy, sres, sdy, sdres, sdx, sdz;
  float *part, *part2;    // partial sums of dweight, dscale
};

// How a row lies on threads.  Up to 512 channels: TPR threads of a warp or a
// part of one, so that sums are shuffles alone, NV pieces each, several rows to
// a block of 128.  Longer rows (TPR 0): a block per row, as many threads as it
// takes at NV pieces each, at most 512 (2560 channels are 160 threads: with a
// power of two the spare ones cost a third of the time).
// MAXT: the most threads of a block per row; kVector: for rows of vectors only.
template <int TPR_, int NV_, int MAXT_ = 512> struct Shape {
  static constexpr int TPR = TPR_, NV = NV_;
  static constexpr int kMaxThreads = TPR_ ? 128 : MAXT_;
  static constexpr bool kVector = MAXT_ < 512;
  static constexpr int kRows = TPR_ ? 128 / (TPR_ ? TPR_ : 1) : 1;  // rows of a block
  static int threads(int64_t gs) {
    return TPR_ ? 128 : static_cast<int>(((gs + 8 * NV_ - 1) / (8 * NV_) + 31) / 32 * 32);
  }
};
// Two pieces of a thread from 1024 channels on where rows move as vectors
// (16384 rows of 4096 in bf16: forward 66 us, 82 with one piece, backward 129,
// 157 with one), one where they are scalar (4096 rows of 1155: backward 33 us,
// 38 with two).
template <typename F> auto by_shape(int64_t gs, bool vec, F f) {
  if (gs <= 64) return f(Shape<8, 1>());
  if (gs <= 128) return f(Shape<16, 1>());
  if (gs <= 512) return f(Shape<32, 2>());
  if (gs <= (vec ? 1024 : 4096)) return f(Shape<0, 1>());
  if (vec && gs <= 4096) return f(Shape<0, 2, 256>());
  if (vec && gs <= 6144) return f(Shape<0, 2, 384>());
  if (gs <= 8192) return f(Shape<0, 2>());
  return f(Shape<0, 4>());
}

// eight channels as they lie in memory
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void set(int e, float v) { reinterpret_cast<float *>(this)[e] = v; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    a = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void set(int e, __nv_bfloat16 v) {
    reinterpret_cast<__nv_bfloat16 *>(this)[e] = v;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// this thread's place in its row, the row's place in the block, and the
// threads of a row
template <typename S> struct Place {
  int lane, sub, tpr;
  __device__ __forceinline__ Place() {
    tpr = S::TPR ? S::TPR : static_cast<int>(blockDim.x);
    lane = S::TPR ? static_cast<int>(threadIdx.x) % (S::TPR ? S::TPR : 1)
                  : static_cast<int>(threadIdx.x);
    sub = S::TPR ? static_cast<int>(threadIdx.x) / (S::TPR ? S::TPR : 1) : 0;
  }
  // channel e of piece i
  template <bool VEC> __device__ __forceinline__ int column(int i, int e) const {
    return VEC ? (i * tpr + lane) * 8 + e : (i * 8 + e) * tpr + lane;
  }
};

// piece i of a row of gs channels (zeros past its end)
template <bool VEC, typename T, typename S>
__device__ __forceinline__ Raw8<T> load8(const T *row, int i, const Place<S> &at, int gs,
                                         bool valid) {
  Raw8<T> r;
  if constexpr (VEC) {
    const int c = at.template column<true>(i, 0);
    if (valid && c < gs) {
      r.load(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.set(e, from_f32<T>(0.f));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = at.template column<false>(i, e);
      r.set(e, valid && c < gs ? row[c] : from_f32<T>(0.f));
    }
  }
  return r;
}

__device__ __forceinline__ void store_vec8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_vec8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&t);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool VEC, typename T, typename S>
__device__ __forceinline__ void store8(T *row, int i, const Place<S> &at, int gs,
                                       const float (&v)[8]) {
  if constexpr (VEC) {
    const int c = at.template column<true>(i, 0);
    if (c < gs) store_vec8(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = at.template column<false>(i, e);
      if (c < gs) row[c] = from_f32<T>(v[e]);
    }
  }
}

// Sums of NS values over the threads of a row, given to all of them.  `sm`
// holds 16 NS floats, another place each time in turn.
template <int TPR, int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], float *sm) {
#pragma unroll
  for (int o = (TPR ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int s = 0; s < NS; ++s) v[s] += __shfl_xor_sync(0xffffffffu, v[s], o);
  if constexpr (TPR == 0) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int s = 0; s < NS; ++s) sm[s * 16 + (threadIdx.x >> 5)] = v[s];
    __syncthreads();
    const int warps = static_cast<int>(blockDim.x) >> 5;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      float t = 0.f;
      for (int w = 0; w < warps; ++w) t += sm[s * 16 + w];
      v[s] = t;
    }
  }
}

// Argument checks of a call (norm_bwd.cu): fills *p, and *vec with whether
// every row can be moved as 16-byte vectors.
mss_status resolve(const mss_gated_norm_args *a, bool bwd, Params *p, bool *vec);
mss_status resolve(const mss_add_norm_args *a, bool bwd, Params *p, bool *vec);

inline bool al(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t esize(mss_dtype t) { return t == MSS_BF16 ? 2 : 4; }

}  // namespace norm
}  // namespace sss48
