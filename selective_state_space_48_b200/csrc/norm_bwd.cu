// norm_bwd.cu -- gradients of the RMS norms before and after a block, and
// the argument checks of all their entry points.
//
// With n = a rstd, dn = (the upstream gradient of n) o weight and means over
// the group's channels,
//   da = rstd (dn - n mean(dn o n)),
// so one pass over a row gives both sums it needs (a^2 and dn o a), taken
// together, and its gradients; every input is read once and every gradient
// written once, which bounds the kernel.  A block walks over rows of one
// group, the next row's inputs loaded while the current one is summed, and
// keeps its rows' sums for dweight (and dscale) in registers; they end in the
// workspace as one line per warp or block, and a second launch adds the lines
// in a fixed order.  There are about as many blocks as fit the SMs, so the
// lines stay few beside the rows.
#include <algorithm>

#include "norm.cuh"
#include "nvtx_range.cuh"

namespace sss48 {
namespace norm {
namespace {

// lines of partial sums that a block leaves
template <typename S> constexpr int kLines = S::TPR < 32 ? 4 : S::kRows;

template <typename T, typename R, int MODE, typename S, bool VEC>
__global__ void __launch_bounds__(S::kThreads) norm_bwd_kernel(const Params p) {
  constexpr int TPR = S::TPR, NV = S::NV;
  constexpr bool kAhead = VEC && NV <= 2;  // registers for the next row's inputs
  __shared__ float sm[2][32];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int c0 = static_cast<int>(blockIdx.y) * p.gs;
  const float *wr = p.weight + (p.shared ? 0 : c0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * S::kRows;

  Raw8<T> xn[NV], gn[NV];
  Raw8<R> zn[NV], rn[MODE == kAdd ? NV : 1];
  // add: the stored residual in zn, its upstream gradient in rn, x in xn only
  // for dscale; gated: x in xn, z in zn
  auto load = [&](int64_t row) {
    const bool ok = row < p.rows;
    const int64_t q = ok ? row : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (MODE == kAdd) {
        zn[i] = load8<R, TPR, VEC>(static_cast<const R *>(p.res) + q * p.sres, i, lane, p.gs, ok);
        rn[i] = load8<R, TPR, VEC>(static_cast<const R *>(p.dres) + q * p.sdres, i, lane, p.gs,
                                   ok && p.dres);
        xn[i] = load8<T, TPR, VEC>(static_cast<const T *>(p.x) + q * p.sx, i, lane, p.gs,
                                   ok && p.part2);
      } else {
        xn[i] = load8<T, TPR, VEC>(static_cast<const T *>(p.x) + q * p.sx + c0, i, lane, p.gs, ok);
        zn[i] = load8<R, TPR, VEC>(static_cast<const R *>(p.z) + q * p.sz + c0, i, lane, p.gs, ok);
      }
      gn[i] = load8<T, TPR, VEC>(static_cast<const T *>(p.dy) + q * p.sdy + c0, i, lane, p.gs, ok);
    }
  };

  float w[NV][8], sc[MODE == kAdd ? NV : 1][8], dw[NV][8], ds[MODE == kAdd ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load8<float, TPR, VEC>(wr, i, lane, p.gs, true).get(w[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    if constexpr (MODE == kAdd) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ds[i][e] = 0.f;
        sc[i][e] = 1.f;
      }
      if (p.scale) load8<float, TPR, VEC>(p.scale, i, lane, p.gs, true).get(sc[i]);
    }
  }

  const int64_t first = static_cast<int64_t>(blockIdx.x) * S::kRows;
  if (kAhead) load(first + sub);
  int turn = 0;
  // the block's rows together: every thread of it takes part in the sums
  for (int64_t base = first; base < p.rows; base += step, turn ^= 1) {
    const int64_t row = base + sub;
    const bool valid = row < p.rows;
    if (!kAhead) load(row);
    // a: the normed values; d: dy times the gate after the norm, if any
    float a[NV][8], d[NV][8], sum[2] = {0.f, 0.f};
    Raw8<T> xv[NV];
    Raw8<R> zv[NV], rv[MODE == kAdd ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xv[i] = xn[i];
      zv[i] = zn[i];
      if constexpr (MODE == kAdd) rv[i] = rn[i];
      gn[i].get(d[i]);
      if constexpr (MODE == kAdd) {
        zv[i].get(a[i]);
      } else {
        float z[8];
        xv[i].get(a[i]);
        zv[i].get(z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float g = silu_f(z[e]);
          if (MODE == kGateAfter) a[i][e] *= g;
          else d[i][e] *= g;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[0] = fmaf(a[i][e], a[i][e], sum[0]);
        sum[1] = fmaf(d[i][e] * w[i][e], a[i][e], sum[1]);
      }
    }
    Raw8<T> dyv[MODE == kGateBefore ? NV : 1];
    if constexpr (MODE == kGateBefore) {
#pragma unroll
      for (int i = 0; i < NV; ++i) dyv[i] = gn[i];
    }
    if (kAhead) load(row + step);
    row_sum<TPR, 2>(sum, sm[turn]);
    const float r = rsqrtf(fmaf(sum[0], p.inv, p.eps));
    const float m = sum[1] * r * r * p.inv;  // n mean(dn n) = a rstd * rstd mean(dn a)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float da[8], dz[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = a[i][e] * r;
        dw[i][e] = fmaf(d[i][e], n, dw[i][e]);
        da[e] = r * fmaf(-a[i][e], m, d[i][e] * w[i][e]);
      }
      if constexpr (MODE == kAdd) {
        float up[8], x[8];
        rv[i].get(up);
        xv[i].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dz[e] = da[e] + up[e];
          ds[i][e] = fmaf(dz[e], x[e], ds[i][e]);
          da[e] = dz[e] * sc[i][e];
        }
        if (valid && p.dz)
          store8<R, TPR, VEC>(static_cast<R *>(p.dz) + row * p.sdz, i, lane, p.gs, dz);
      } else {
        float z[8], x[8], g[8];
        zv[i].get(z);
        if constexpr (MODE == kGateBefore) dyv[i].get(g);
        else xv[i].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = __fdividef(1.0f, 1.0f + ex2_mufu(-z[e] * kLog2e));
          const float dg = s * fmaf(z[e], 1.0f - s, 1.0f);
          if (MODE == kGateBefore) {
            dz[e] = g[e] * a[i][e] * r * w[i][e] * dg;
          } else {
            dz[e] = da[e] * x[e] * dg;
            da[e] *= z[e] * s;
          }
        }
        if (valid)
          store8<R, TPR, VEC>(static_cast<R *>(p.dz) + row * p.sdz + c0, i, lane, p.gs, dz);
      }
      if (valid)
        store8<T, TPR, VEC>(static_cast<T *>(p.dx) + row * p.sdx + c0, i, lane, p.gs, da);
    }
  }

  // this block's lines of the sums over rows
  auto lines = [&](float *part, float (&v)[NV][8]) {
    if (!part) return;
    const int64_t width = static_cast<int64_t>(p.ng) * p.gs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (TPR < 32) {
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] += __shfl_xor_sync(0xffffffffu, v[i][e], o);
      }
      if (TPR >= 32 || (threadIdx.x & 31) < TPR) {
        const int line = TPR < 32 ? static_cast<int>(threadIdx.x >> 5) : sub;
        float *dst = part + (static_cast<int64_t>(blockIdx.x) * kLines<S> + line) * width + c0;
        // (the workspace is 16-byte aligned; a vector path has gs % 8 == 0)
        store8<float, TPR, VEC>(dst, i, lane, p.gs, v[i]);
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

// Row blocks of a backward call: about 1024 threads of every SM in all.
template <typename S> int64_t row_blocks(int64_t rows, int64_t ng, int sms) {
  const int64_t want = std::max<int64_t>(1, sms * (1024 / S::kThreads) / ng);
  return std::min<int64_t>(want, (rows + S::kRows - 1) / S::kRows);
}

mss_status sm_count(int *sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MSS_ERR_CUDA;
  return MSS_OK;
}

// floats of one set of partial sums
int64_t part_floats(int64_t rows, int64_t ng, int64_t gs, int sms) {
  return by_shape(gs, [&](auto s) {
    using S = decltype(s);
    return row_blocks<S>(rows, ng, sms) * kLines<S> * ng * gs;
  });
}

template <typename T, typename R, int MODE>
cudaError_t launch(const Params &p, bool vec, int sms, float *dw, float *ds, cudaStream_t stream) {
  return by_shape(p.gs, [&](auto shape) {
    using S = decltype(shape);
    const int64_t rb = row_blocks<S>(p.rows, p.ng, sms);
    const dim3 grid(static_cast<unsigned>(rb), static_cast<unsigned>(p.ng));
    if (vec)
      norm_bwd_kernel<T, R, MODE, S, true><<<grid, S::kThreads, 0, stream>>>(p);
    else
      norm_bwd_kernel<T, R, MODE, S, false><<<grid, S::kThreads, 0, stream>>>(p);
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
