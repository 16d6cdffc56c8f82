// norm_bwd.cu -- gradients of the RMS norms before and after a block, and
// the argument checks of all their entry points.
//
// With n = a rstd, dn = (the upstream gradient of n) o weight and means over
// the group's channels,
//   da = rstd (dn - n mean(dn o n)),
// so one pass over a row gives both sums it needs (a^2 and dn o a), taken
// together, and its gradients; every input is read once and every gradient
// written once, which bounds the kernel.  A block walks over rows of one
// group, the next rows' inputs on their way into shared memory meanwhile (each
// thread copies and reads places of its own, so nothing but the sums
// synchronises), and keeps its rows' sums for dweight (and dscale) in
// registers; they end in the workspace as one line per warp or block, and a
// second launch adds the lines in a fixed order.  There are about as many
// blocks as fit the SMs, so the lines stay few beside the rows.
#include <algorithm>

#include "norm.cuh"
#include "nvtx_range.cuh"

namespace sss48 {
namespace norm {
namespace {

// lines of partial sums that a block leaves
template <typename S> constexpr int kLines = S::TPR ? 4 : 1;

// 16-byte pieces of a thread's share of a row, and the rows on their way at a
// time: about 100 KB of a block of 512 threads, so that two fit an SM
template <typename T, typename R, int MODE, typename S> struct Ring {
  static constexpr int kT = sizeof(T) / 2, kR = sizeof(R) / 2;  // of 8 channels
  static constexpr int kPiece = 2 * kT + (MODE == kAdd ? 2 : 1) * kR;
  static constexpr int kPieces = S::NV * kPiece;
  static constexpr int kStages = kPieces <= 3 ? 4 : 2;
  static constexpr bool kUsed = 16 * S::kMaxThreads * kPieces * kStages <= 200 * 1024;
};

// Blocks that an SM's registers hold.  Two pieces of a thread want 111
// registers; where every tensor is bf16 three blocks of 256 threads at 80 are
// faster than two (16384 rows of 4096: 129 us, 136; four at 64: 134), with fp32
// residuals two (2560 channels: 136 us, 150 with three).
template <typename T, typename R, typename S>
constexpr int kResident = S::TPR ? 4
                          : S::NV == 1 ? (sizeof(T) == 2 ? 2 : 1)
                          : S::kMaxThreads == 256 ? (sizeof(R) == 2 ? 3 : 2)
                          : S::kMaxThreads == 384 ? 2
                                                  : 1;

__device__ __forceinline__ float rcp_mufu(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}

template <typename T, typename R, int MODE, typename S, bool VEC>
__global__ void __launch_bounds__(S::kMaxThreads, kResident<T, R, S>)
    norm_bwd_kernel(const Params p) {
  constexpr int NV = S::NV;
  using Rg = Ring<T, R, MODE, S>;
  constexpr bool kRing = VEC && Rg::kUsed;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float sm[2][32];
  const Place<S> at;
  const int c0 = static_cast<int>(blockIdx.y) * p.gs;
  const float *wr = p.weight + (p.shared ? 0 : c0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * S::kRows;

  // add: the stored residual in zv, its upstream gradient in rv, x in xv only
  // for dscale; gated: x in xv, z in zv
  Raw8<T> xv[NV], gv[NV];
  Raw8<R> zv[NV], rv[MODE == kAdd ? NV : 1];
  const T *xp = static_cast<const T *>(p.x) + (MODE == kAdd ? 0 : c0);
  const T *gp = static_cast<const T *>(p.dy) + c0;
  const R *zp = MODE == kAdd ? static_cast<const R *>(p.res) : static_cast<const R *>(p.z) + c0;
  const int64_t sz = MODE == kAdd ? p.sres : p.sz;
  const bool has_x = MODE != kAdd || p.part2, has_r = MODE == kAdd && p.dres;
  const uint32_t slot = smem_addr(ring), pitch = blockDim.x * 16;
  // fp32 rows are copied so that neighbouring lanes of a row take neighbouring
  // 16 bytes (a thread's own 32 would leave half of every sector to a second
  // request): lane l of the W that share a row or a warp of it
  constexpr int W = S::TPR ? S::TPR : 32;
  const int l = threadIdx.x % W;
  // row's inputs towards stage `st` (zeros behind the last row and channel)
  auto fetch = [&](int64_t row, int st) {
    if constexpr (kRing) {
      uint32_t d = slot + st * Rg::kPieces * pitch;
      const bool ok = row < p.rows;
      const int64_t q = ok ? row : 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = at.template column<true>(i, 0);
        auto put = [&](auto *base, bool on) {
          if constexpr (sizeof(*base) == 2) {
            const bool in = ok && c < p.gs && on;
            copy16(d + threadIdx.x * 16, base + (in ? c : 0), in);
            d += pitch;
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int ck = c - 8 * l + 4 * (k * W + l);
              const bool in = ok && ck < p.gs && on;
              copy16(d + (threadIdx.x - l) * 32 + (k * W + l) * 16, base + (in ? ck : 0), in);
            }
            d += 2 * pitch;
          }
        };
        put(has_x ? xp + q * p.sx : gp, has_x);
        put(gp + q * p.sdy, true);
        put(zp + q * sz, true);
        if constexpr (MODE == kAdd)
          put(has_r ? static_cast<const R *>(p.dres) + q * p.sdres : zp, has_r);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  auto load = [&](int64_t row, int st) {
    if constexpr (kRing) {
      const unsigned char *d = ring + st * Rg::kPieces * pitch;
      auto get = [&](auto &raw) {
        constexpr int n = sizeof(raw) / 16;
#pragma unroll
        for (int k = 0; k < n; ++k)
          reinterpret_cast<uint4 *>(&raw)[k] =
              *reinterpret_cast<const uint4 *>(d + threadIdx.x * 16 * n + 16 * k);
        d += n * pitch;
      };
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        get(xv[i]);
        get(gv[i]);
        get(zv[i]);
        if constexpr (MODE == kAdd) get(rv[i]);
      }
    } else {
      const bool ok = row < p.rows;
      const int64_t q = ok ? row : 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xv[i] = load8<VEC>(xp + q * p.sx, i, at, p.gs, ok && has_x);
        gv[i] = load8<VEC>(gp + q * p.sdy, i, at, p.gs, ok);
        zv[i] = load8<VEC>(zp + q * sz, i, at, p.gs, ok);
        if constexpr (MODE == kAdd)
          rv[i] = load8<VEC>(static_cast<const R *>(p.dres) + q * p.sdres, i, at, p.gs, ok && has_r);
      }
    }
  };

  float dw[NV][8], ds[MODE == kAdd ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[i][e] = 0.f;
      if constexpr (MODE == kAdd) ds[i][e] = 0.f;
    }

  const int64_t first = static_cast<int64_t>(blockIdx.x) * S::kRows;
  if constexpr (kRing) {
#pragma unroll
    for (int k = 0; k < Rg::kStages; ++k) fetch(first + at.sub + k * step, k);
  }
  int turn = 0, st = 0;
  // the block's rows together: every thread of it takes part in the sums
  for (int64_t base = first; base < p.rows; base += step, turn ^= 1) {
    const int64_t row = base + at.sub;
    const bool valid = row < p.rows;
    if constexpr (kRing) {
      asm volatile("cp.async.wait_group %0;" ::"n"(Rg::kStages - 1) : "memory");
      __syncwarp();  // the other lanes' copies
    }
    load(row, st);
    float sg[MODE == kAdd ? 1 : NV][8], sum[2] = {0.f, 0.f};  // sg: sigmoid(z)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], d[8], w[8], z[8];
      gv[i].get(d);
      load8<VEC>(wr, i, at, p.gs, true).get(w);  // (from the L1: not worth its registers)
      zv[i].get(z);
      xv[i].get(a);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (MODE == kAdd) {
          a[e] = z[e];
        } else {
          sg[i][e] = rcp_mufu(1.0f + ex2_mufu(-z[e] * kLog2e));
          if (MODE == kGateAfter) a[e] *= z[e] * sg[i][e];
          else d[e] *= z[e] * sg[i][e];
        }
        sum[0] = fmaf(a[e], a[e], sum[0]);
        sum[1] = fmaf(d[e] * w[e], a[e], sum[1]);
      }
    }
    row_sum<S::TPR, 2>(sum, sm[turn]);
    // (0 behind the last row: with eps 0 its zeros would give NaN to dweight)
    const float r = valid ? rsqrtf(fmaf(sum[0], p.inv, p.eps)) : 0.f;
    // da = r dn - a r^2 mean(dn n) r, with n mean(dn n) = a r * r mean(dn a)
    const float nm = -sum[1] * p.inv * r * r * r;
    if constexpr (kRing) load(row, st);  // (again: not kept in registers)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float d[8], w[8], x[8], z[8], da[8], dz[8];
      gv[i].get(d);
      load8<VEC>(wr, i, at, p.gs, true).get(w);
      zv[i].get(z);
      xv[i].get(x);
      if constexpr (MODE == kAdd) {
        float up[8], sc[8];
        rv[i].get(up);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float dr = d[e] * r;
          dw[i][e] = fmaf(dr, z[e], dw[i][e]);
          dz[e] = fmaf(z[e], nm, fmaf(dr, w[e], up[e]));
          ds[i][e] = fmaf(dz[e], x[e], ds[i][e]);
          da[e] = dz[e];
        }
        if (p.scale) {
          load8<VEC>(p.scale, i, at, p.gs, true).get(sc);
#pragma unroll
          for (int e = 0; e < 8; ++e) da[e] *= sc[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = sg[i][e], g = z[e] * s, dr = d[e] * r;
          const float dg = fmaf(s, z[e] - g, s);  // silu'(z) = s (1 + z - z s)
          if constexpr (MODE == kGateAfter) {
            const float a = x[e] * g;
            dw[i][e] = fmaf(dr, a, dw[i][e]);
            const float o = fmaf(a, nm, dr * w[e]);
            dz[e] = o * x[e] * dg;
            da[e] = o * g;
          } else {
            const float xr = dr * x[e], gw = g * w[e];
            dw[i][e] = fmaf(xr, g, dw[i][e]);
            dz[e] = xr * w[e] * dg;
            da[e] = fmaf(x[e], nm, dr * gw);
          }
        }
      }
      if (valid) {
        if (MODE != kAdd || p.dz)
          store8<VEC>(static_cast<R *>(p.dz) + row * p.sdz + c0, i, at, p.gs, dz);
        store8<VEC>(static_cast<T *>(p.dx) + row * p.sdx + c0, i, at, p.gs, da);
      }
    }
    if constexpr (kRing) {
      __syncwarp();  // read: the place may be written again
      fetch(row + Rg::kStages * step, st);
      st = st == Rg::kStages - 1 ? 0 : st + 1;
    }
  }

  // (no copy may land in the memory of a block that has ended)
  if constexpr (kRing) asm volatile("cp.async.wait_all;" ::: "memory");

  // this block's lines of the sums over rows
  auto lines = [&](float *part, float (&v)[NV][8]) {
    if (!part) return;
    const int64_t width = static_cast<int64_t>(p.ng) * p.gs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (S::TPR != 0) {  // rows of a warp
#pragma unroll
        for (int o = S::TPR; o < 32; o <<= 1)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] += __shfl_xor_sync(0xffffffffu, v[i][e], o);
      }
      if (S::TPR == 0 || (threadIdx.x & 31) < S::TPR) {
        const int line = S::TPR ? static_cast<int>(threadIdx.x >> 5) : 0;
        float *dst = part + (static_cast<int64_t>(blockIdx.x) * kLines<S> + line) * width + c0;
        // (the workspace is 16-byte aligned; a vector path has gs % 8 == 0)
        store8<VEC>(dst, i, at, p.gs, v[i]);
      }
    }
  };
  lines(p.part, dw);
  if constexpr (MODE == kAdd) lines(p.part2, ds);
}

// out[c] = sum over n lines of `width` values; blockIdx.y chooses the pair.
// 32 columns of a block, 16 threads down the lines.
__global__ void __launch_bounds__(512) line_sum_kernel(const float *pa, float *oa, const float *pb,
                                                       float *ob, int64_t n, int width) {
  __shared__ float sm[16][33];
  const float *part = blockIdx.y ? pb : pa;
  float *out = blockIdx.y ? ob : oa;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float s = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int64_t i = ry; i < n; i += 16) s += part[i * width + c];
  }
  sm[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && c < width) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sm[i][cx];
    out[c] = t;
  }
}

// Row blocks of a backward call: as many in all as are on the SMs at once, by
// their threads and their shared memory (of blocks of 128 threads with several
// rows, 6 were best of 4 .. 16; rows that are not vectors are better off with
// fewer lines: 1000 rows of 1155 in fp32 took 12.6 us with 512 threads to an
// SM, 15.3 with 1024).
template <typename S>
int64_t row_blocks(int64_t rows, int64_t ng, int64_t gs, int sm_threads, int ring, int sms) {
  int per = S::TPR ? 6 : std::min(8, sm_threads / S::threads(gs));
  per = std::max(1, std::min(per, ring > 0 ? 220 * 1024 / (ring + 1024) : per));
  const int64_t want = std::max<int64_t>(1, sms * per / ng);
  return std::min<int64_t>(want, (rows + S::kRows - 1) / S::kRows);
}

mss_status sm_count(int *sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MSS_ERR_CUDA;
  return MSS_OK;
}

// floats that one set of partial sums takes at most, whatever the types
int64_t part_floats(int64_t rows, int64_t ng, int64_t gs, int sms) {
  return by_shape(gs, true, [&](auto s) {
    using S = decltype(s);
    return row_blocks<S>(rows, ng, gs, 1024, 0, sms) * kLines<S> * ng * gs;
  });
}

template <typename T, typename R, int MODE>
cudaError_t launch(const Params &p, bool vec, int sms, float *dw, float *ds, cudaStream_t stream) {
  return by_shape(p.gs, vec, [&](auto shape) {
    using S = decltype(shape);
    const int threads = S::threads(p.gs);
    using Rg = Ring<T, R, MODE, S>;
    const int smem = vec && Rg::kUsed ? threads * 16 * Rg::kPieces * Rg::kStages : 0;
    const int sm_threads = !vec ? 512 : S::kVector ? S::kMaxThreads * kResident<T, R, S> : 1024;
    const int64_t rb = row_blocks<S>(p.rows, p.ng, p.gs, sm_threads, smem, sms);
    const dim3 grid(static_cast<unsigned>(rb), static_cast<unsigned>(p.ng));
    auto kernel = norm_bwd_kernel<T, R, MODE, S, true>;
    if constexpr (!S::kVector) {
      if (!vec) kernel = norm_bwd_kernel<T, R, MODE, S, false>;
    }
    if (smem > 40 * 1024) {  // (48 KB with the static part) per launch: the current device's
      const cudaError_t a =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (a != cudaSuccess) return a;
    }
    kernel<<<grid, threads, smem, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!dw && !ds)) return e;
    // with a shared weight the groups of a line are lines of their own
    const int64_t lines = rb * kLines<S> * (p.shared ? p.ng : 1);
    const int width = p.shared ? p.gs : p.ng * p.gs;
    const float *pa = dw ? p.part : p.part2;
    line_sum_kernel<<<dim3((width + 31) / 32, dw && ds ? 2 : 1), 512, 0, stream>>>(
        pa, dw ? dw : ds, p.part2, ds, lines, width);
    return cudaGetLastError();
  });
}

bool valid_dtype(mss_dtype t) { return t == MSS_F32 || t == MSS_BF16; }

mss_status check_sizes(int64_t rows, int64_t ng, int64_t gs) {
  if (rows < 1 || ng < 1 || gs < 1) return MSS_ERR_INVALID_ARG;
  const int64_t lim = int64_t(1) << 30;
  if (gs > kMaxGroup || ng > 65535 || rows > lim / ng) return MSS_ERR_UNSUPPORTED;
  return MSS_OK;
}

// one (rows, width) tensor: present, aligned to its elements, with a sane
// stride; clears *vec where rows cannot be read as 16-byte vectors
bool tensor_ok(const void *ptr, int64_t stride, mss_dtype t, int64_t rows, int64_t width,
               bool output, bool *vec) {
  const size_t es = esize(t);
  if (!ptr || !al(ptr, es) || stride < 0 || stride > (int64_t(1) << 40)) return false;
  if (output && rows > 1 && stride < width) return false;
  if (!al(ptr, 16) || (rows > 1 && (stride * es) % 16 != 0)) *vec = false;
  return true;
}
bool vector_ok(const float *ptr, bool *vec) {
  if (!al(ptr, 4)) return false;
  if (!al(ptr, 16)) *vec = false;
  return true;
}

}  // namespace

mss_status resolve(const mss_gated_norm_args *a, bool bwd, Params *p, bool *vec) {
  if (!a || a->group_size < 1 || a->width < 1 || a->width % a->group_size != 0)
    return MSS_ERR_INVALID_ARG;
  const int64_t ng = a->width / a->group_size;
  const mss_status st = check_sizes(a->rows, ng, a->group_size);
  if (st != MSS_OK) return st;
  if (!valid_dtype(a->dtype) || !(a->eps >= 0.f)) return MSS_ERR_INVALID_ARG;
  *vec = a->group_size % 8 == 0;
  const auto ok = [&](const void *ptr, int64_t stride, bool out) {
    return tensor_ok(ptr, stride, a->dtype, a->rows, a->width, out, vec);
  };
  if (!ok(a->x, a->stride_x, false) || !ok(a->z, a->stride_z, false) || !a->weight ||
      !vector_ok(a->weight, vec))
    return MSS_ERR_INVALID_ARG;
  if (!bwd && !ok(a->y, a->stride_y, true)) return MSS_ERR_INVALID_ARG;
  if (bwd && (!ok(a->dy, a->stride_dy, false) || !ok(a->dx, a->stride_dx, true) ||
              !ok(a->dz, a->stride_dz, true) || !al(a->dweight, 4)))
    return MSS_ERR_INVALID_ARG;
  *p = Params();
  p->rows = a->rows;
  p->ng = static_cast<int>(ng);
  p->gs = static_cast<int>(a->group_size);
  p->shared = a->shared_weight ? 1 : 0;
  p->eps = a->eps;
  p->inv = 1.0f / static_cast<float>(p->gs);
  p->x = a->x;
  p->z = a->z;
  p->weight = a->weight;
  p->y = a->y;
  p->dy = a->dy;
  p->dx = a->dx;
  p->dz = a->dz;
  p->sx = a->stride_x;
  p->sz = a->stride_z;
  p->sy = a->stride_y;
  p->sdy = a->stride_dy;
  p->sdx = a->stride_dx;
  p->sdz = a->stride_dz;
  return MSS_OK;
}

mss_status resolve(const mss_add_norm_args *a, bool bwd, Params *p, bool *vec) {
  if (!a) return MSS_ERR_INVALID_ARG;
  const mss_status st = check_sizes(a->rows, 1, a->width);
  if (st != MSS_OK) return st;
  if (!valid_dtype(a->dtype) || !valid_dtype(a->res_dtype) || !(a->eps >= 0.f))
    return MSS_ERR_INVALID_ARG;
  if (a->dtype == MSS_F32 && a->res_dtype != MSS_F32) return MSS_ERR_UNSUPPORTED;
  *vec = a->width % 8 == 0;
  const auto ok = [&](const void *ptr, int64_t stride, mss_dtype t, bool out) {
    return tensor_ok(ptr, stride, t, a->rows, a->width, out, vec);
  };
  const bool need_x = !bwd || a->dscale;
  if ((need_x && !ok(a->x, a->stride_x, a->dtype, false)) || !a->weight ||
      !vector_ok(a->weight, vec) || !vector_ok(a->scale, vec) ||
      !ok(a->residual_out, a->stride_residual_out, a->res_dtype, !bwd))
    return MSS_ERR_INVALID_ARG;
  if (!bwd && ((a->residual && !ok(a->residual, a->stride_residual, a->res_dtype, false)) ||
               !ok(a->y, a->stride_y, a->dtype, true)))
    return MSS_ERR_INVALID_ARG;
  if (bwd &&
      (!ok(a->dy, a->stride_dy, a->dtype, false) || !ok(a->dx, a->stride_dx, a->dtype, true) ||
       (a->dresidual_out &&
        !ok(a->dresidual_out, a->stride_dresidual_out, a->res_dtype, false)) ||
       (a->dresidual && !ok(a->dresidual, a->stride_dresidual, a->res_dtype, true)) ||
       !al(a->dweight, 4) || !al(a->dscale, 4)))
    return MSS_ERR_INVALID_ARG;
  *p = Params();
  p->rows = a->rows;
  p->ng = 1;
  p->gs = static_cast<int>(a->width);
  p->eps = a->eps;
  p->inv = 1.0f / static_cast<float>(p->gs);
  p->x = a->x;
  p->z = a->residual;
  p->scale = a->scale;
  p->weight = a->weight;
  p->y = a->y;
  p->res = a->residual_out;
  p->dy = a->dy;
  p->dres = a->dresidual_out;
  p->dx = a->dx;
  p->dz = a->dresidual;
  p->sx = a->stride_x;
  p->sz = a->stride_residual;
  p->sy = a->stride_y;
  p->sres = a->stride_residual_out;
  p->sdy = a->stride_dy;
  p->sdres = a->stride_dresidual_out;
  p->sdx = a->stride_dx;
  p->sdz = a->stride_dresidual;
  return MSS_OK;
}

}  // namespace norm
}  // namespace sss48

using namespace sss48;
using namespace sss48::norm;

namespace {

// the partial sums in the workspace, after its size is checked
mss_status partials(void *ws, size_t have, bool dw, bool ds, int sms, Params *p) {
  if (!dw && !ds) return MSS_OK;
  const int64_t n = part_floats(p->rows, p->ng, p->gs, sms);
  if (!ws || have < static_cast<size_t>(n) * 4 * ((dw ? 1 : 0) + (ds ? 1 : 0)))
    return MSS_ERR_WORKSPACE;
  if (!al(ws, 16)) return MSS_ERR_INVALID_ARG;
  float *f = static_cast<float *>(ws);
  if (dw) {
    p->part = f;
    f += n;
  }
  if (ds) p->part2 = f;
  return MSS_OK;
}

}  // namespace

extern "C" mss_status mss_gated_rmsnorm_bwd_workspace_size(const mss_gated_norm_args *a,
                                                           size_t *bytes) {
  if (!a || !bytes || a->group_size < 1 || a->width < 1 || a->width % a->group_size != 0)
    return MSS_ERR_INVALID_ARG;
  const int64_t ng = a->width / a->group_size;
  mss_status st = check_sizes(a->rows, ng, a->group_size);
  if (st != MSS_OK) return st;
  *bytes = 0;
  if (!a->dweight) return MSS_OK;
  int sms = 0;
  if ((st = sm_count(&sms)) != MSS_OK) return st;
  *bytes = static_cast<size_t>(part_floats(a->rows, ng, a->group_size, sms)) * 4;
  return MSS_OK;
}

extern "C" mss_status mss_add_rmsnorm_bwd_workspace_size(const mss_add_norm_args *a,
                                                         size_t *bytes) {
  if (!a || !bytes) return MSS_ERR_INVALID_ARG;
  mss_status st = check_sizes(a->rows, 1, a->width);
  if (st != MSS_OK) return st;
  *bytes = 0;
  const int sets = (a->dweight ? 1 : 0) + (a->dscale ? 1 : 0);
  if (!sets) return MSS_OK;
  int sms = 0;
  if ((st = sm_count(&sms)) != MSS_OK) return st;
  *bytes = static_cast<size_t>(part_floats(a->rows, 1, a->width, sms)) * 4 * sets;
  return MSS_OK;
}

extern "C" mss_status gated_rmsnorm_bwd(const mss_gated_norm_args *a, void *stream) {
  sss48::NvtxRange range("gated_rmsnorm_bwd");
  Params p;
  bool vec = false;
  mss_status st = resolve(a, true, &p, &vec);
  if (st != MSS_OK) return st;
  int sms = 0;
  if ((st = sm_count(&sms)) != MSS_OK) return st;
  st = partials(a->workspace, a->workspace_bytes, a->dweight != nullptr, false, sms, &p);
  if (st != MSS_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto run = [&](auto t) {
    using T = decltype(t);
    return a->norm_before_gate ? launch<T, T, kGateBefore>(p, vec, sms, a->dweight, nullptr, s)
                               : launch<T, T, kGateAfter>(p, vec, sms, a->dweight, nullptr, s);
  };
  return (a->dtype == MSS_BF16 ? run(__nv_bfloat16()) : run(float())) == cudaSuccess
             ? MSS_OK
             : MSS_ERR_CUDA;
}

extern "C" mss_status add_rmsnorm_bwd(const mss_add_norm_args *a, void *stream) {
  sss48::NvtxRange range("add_rmsnorm_bwd");
  Params p;
  bool vec = false;
  mss_status st = resolve(a, true, &p, &vec);
  if (st != MSS_OK) return st;
  int sms = 0;
  if ((st = sm_count(&sms)) != MSS_OK) return st;
  st = partials(a->workspace, a->workspace_bytes, a->dweight != nullptr, a->dscale != nullptr,
                sms, &p);
  if (st != MSS_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == MSS_F32)
    e = launch<float, float, kAdd>(p, vec, sms, a->dweight, a->dscale, s);
  else if (a->res_dtype == MSS_F32)
    e = launch<__nv_bfloat16, float, kAdd>(p, vec, sms, a->dweight, a->dscale, s);
  else
    e = launch<__nv_bfloat16, __nv_bfloat16, kAdd>(p, vec, sms, a->dweight, a->dscale, s);
  return e == cudaSuccess ? MSS_OK : MSS_ERR_CUDA;
}
