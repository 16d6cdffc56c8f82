// norm_fwd.cu -- RMS norms before a block (fused with the residual sum) and
// after it (fused with the silu gate), forward.
//
// y = n o weight with n = a / sqrt(mean(a^2) + eps), where a is the new
// residual, x, or x o silu(z).  One pass: a row's inputs are read once into
// registers, its sum of squares is taken there and the outputs are written
// from there, so the kernel is bound by the bytes of its inputs and outputs.
#include "norm.cuh"
#include "nvtx_range.cuh"

namespace sss48 {
namespace norm {
namespace {

template <typename T, typename R, int MODE, typename S, bool VEC>
__global__ void __launch_bounds__(S::kMaxThreads) norm_fwd_kernel(const Params p) {
  constexpr int NV = S::NV;
  __shared__ float sm[16];
  const Place<S> at;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * S::kRows + at.sub;
  const bool valid = unit < p.rows * p.ng;  // every thread takes part in the shuffles
  const int64_t row = valid ? unit / p.ng : 0;
  const int c0 = valid ? static_cast<int>(unit - row * p.ng) * p.gs : 0;
  const T *xr = static_cast<const T *>(p.x) + row * p.sx + c0;
  const R *zr = p.z ? static_cast<const R *>(p.z) + row * p.sz + c0 : nullptr;
  const float *wr = p.weight + (p.shared ? 0 : c0);

  Raw8<T> xv[NV];
  Raw8<R> zv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    xv[i] = load8<VEC>(xr, i, at, p.gs, valid);
    zv[i] = load8<VEC>(zr, i, at, p.gs, valid && zr);
  }
  float a[NV][8], gate[NV][8], ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float z[8];
    xv[i].get(a[i]);
    zv[i].get(z);
    if constexpr (MODE == kAdd) {
      if (p.scale) {
        float sc[8];
        load8<VEC>(p.scale, i, at, p.gs, true).get(sc);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] *= sc[e];
      }
      // the norm is of the residual as it is stored, the value that the
      // backward and the next block read
#pragma unroll
      for (int e = 0; e < 8; ++e) a[i][e] = to_f32<R>(from_f32<R>(a[i][e] + z[e]));
      if (valid) store8<VEC>(static_cast<R *>(p.res) + row * p.sres, i, at, p.gs, a[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        gate[i][e] = silu_f(z[e]);
        if (MODE == kGateAfter) a[i][e] *= gate[i][e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[0] = fmaf(a[i][e], a[i][e], ss[0]);
  }
  row_sum<S::TPR, 1>(ss, sm);
  const float r = rsqrtf(fmaf(ss[0], p.inv, p.eps));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[8];
    load8<VEC>(wr, i, at, p.gs, true).get(w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[i][e] *= r * w[e];
      if (MODE == kGateBefore) a[i][e] *= gate[i][e];
    }
    if (valid)
      store8<VEC>(static_cast<T *>(p.y) + row * p.sy + c0, i, at, p.gs, a[i]);
  }
}

template <typename T, typename R, int MODE>
cudaError_t launch(const Params &p, bool vec, cudaStream_t stream) {
  return by_shape(p.gs, vec, [&](auto shape) {
    using S = decltype(shape);
    const unsigned grid = static_cast<unsigned>((p.rows * p.ng + S::kRows - 1) / S::kRows);
    const int threads = S::threads(p.gs);
    auto kernel = norm_fwd_kernel<T, R, MODE, S, true>;
    if constexpr (!S::kVector) {
      if (!vec) kernel = norm_fwd_kernel<T, R, MODE, S, false>;
    }
    kernel<<<grid, threads, 0, stream>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace
}  // namespace norm
}  // namespace sss48

using namespace sss48;
using namespace sss48::norm;

extern "C" mss_status gated_rmsnorm_fwd(const mss_gated_norm_args *a, void *stream) {
  sss48::NvtxRange range("gated_rmsnorm_fwd");
  Params p;
  bool vec = false;
  const mss_status st = resolve(a, false, &p, &vec);
  if (st != MSS_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto run = [&](auto t) {
    using T = decltype(t);
    return a->norm_before_gate ? launch<T, T, kGateBefore>(p, vec, s)
                               : launch<T, T, kGateAfter>(p, vec, s);
  };
  return (a->dtype == MSS_BF16 ? run(__nv_bfloat16()) : run(float())) == cudaSuccess
             ? MSS_OK
             : MSS_ERR_CUDA;
}

extern "C" mss_status add_rmsnorm_fwd(const mss_add_norm_args *a, void *stream) {
  sss48::NvtxRange range("add_rmsnorm_fwd");
  Params p;
  bool vec = false;
  const mss_status st = resolve(a, false, &p, &vec);
  if (st != MSS_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == MSS_F32)
    e = launch<float, float, kAdd>(p, vec, s);
  else if (a->res_dtype == MSS_F32)
    e = launch<__nv_bfloat16, float, kAdd>(p, vec, s);
  else
    e = launch<__nv_bfloat16, __nv_bfloat16, kAdd>(p, vec, s);
  return e == cudaSuccess ? MSS_OK : MSS_ERR_CUDA;
}
