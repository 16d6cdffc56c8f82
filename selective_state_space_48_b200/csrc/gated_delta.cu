// gated_delta.cu -- the gated delta rule step by step, and its C ABI.
//
//   u_t = b_t (v_t - a_t S k_t),  S <- a_t S + u_t k_t^T,  y_t = scale S q_t
//
// Eight lanes share a row of S (headdim x dstate) and hold its columns in
// registers, four neighbouring columns of every 32; a thread holds RPT rows.
// Both readouts are taken from the state before the step,
//
//   S_t q = a S_{t-1} q + u (k . q),
//
// so the two dot products of a row run beside each other and one round of
// shuffles over the eight lanes sums both.  A sequence of one token is the
// decode step: it is bound by reading and writing the fp32 state (8 headdim
// dstate bytes per head), every load of which is issued before the arithmetic.
// Over more steps the chain of a step (dots, three shuffles, update) bounds
// it; the next step's inputs are loaded a step ahead.
#include "gated_delta.cuh"

#include <cuda_bf16.h>

#include <algorithm>

#include "gated_delta.h"
#include "nvtx_range.cuh"

namespace sss48 {
namespace {

constexpr int kThreads = 128;
// steps of a sequence (packed ones: on average) from which the chunked
// evaluation runs
constexpr int64_t kChunkSteps = 32;
constexpr int kGroups = kThreads / 8;  // rows of a block side by side

// Four columns from `col` of a row of n columns: one vector load where VEC,
// else element by element with zeros past the end.
template <typename T, bool VEC>
__device__ __forceinline__ float4 row4(const T *row, int col, int n) {
  if constexpr (VEC) {
    return col < n ? load4_f32(row + col) : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = col + e < n ? to_f32<T>(row[col + e]) : 0.f;
    return make_float4(v[0], v[1], v[2], v[3]);
  }
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}
__device__ __forceinline__ float sum8(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 4);
}

template <typename InT, typename OutT, int NV, int RPT, bool VEC>
__global__ void __launch_bounds__(kThreads) delta_recurrent_kernel(const DeltaParams p) {
  const int nrb = static_cast<int>((p.P + kGroups * RPT - 1) / (kGroups * RPT));
  const int64_t sh = blockIdx.x / nrb;
  const int rb = static_cast<int>(blockIdx.x - sh * nrb);
  const int64_t s = sh / p.H;
  const int h = static_cast<int>(sh - s * p.H);
  const int g = h / static_cast<int>(p.H / p.G);
  const int lane8 = threadIdx.x & 7;
  const int row0 = rb * kGroups * RPT + (threadIdx.x >> 3);
  const int N = static_cast<int>(p.N), P = static_cast<int>(p.P);
  int64_t b, t0, t1;
  delta_span(p, s, b, t0, t1);

  const int64_t base = sh * p.P * p.N;
  float4 S[RPT][NV];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = row0 + r * kGroups;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = c * 32 + lane8 * 4;
      S[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.h0 && row < P) {
        const float *src = p.h0 + base + static_cast<int64_t>(row) * N;
        if constexpr (VEC) {
          // read once and written once: streaming accesses keep the state
          // from displacing the other inputs in the caches
          if (col < N) S[r][c] = __ldcs(reinterpret_cast<const float4 *>(src + col));
        } else {
          S[r][c] = row4<float, false>(src, col, N);
        }
      }
    }
  }

  const float A2 = p.A[h] * kLog2e;
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  const InT *qp = static_cast<const InT *>(p.q) + b * p.sq[0] + g * p.sq[2];
  const InT *kp = static_cast<const InT *>(p.k) + b * p.sk[0] + g * p.sk[2];
  const InT *vp = static_cast<const InT *>(p.v) + b * p.sv[0] + h * p.sv[2];
  const InT *dtp = static_cast<const InT *>(p.dt) + b * p.sdt[0] + h * p.sdt[2];
  const InT *bp = static_cast<const InT *>(p.beta) + b * p.sbeta[0] + h * p.sbeta[2];
  OutT *yp = static_cast<OutT *>(p.y) + b * p.sy[0] + h * p.sy[2];

  float4 kn[NV], qn[NV];
  float vn[RPT], dtn = 0.f, bn = 0.f;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      kn[c] = row4<InT, VEC>(kp + t * p.sk[1], c * 32 + lane8 * 4, N);
      qn[c] = row4<InT, VEC>(qp + t * p.sq[1], c * 32 + lane8 * 4, N);
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r)
      vn[r] = row0 + r * kGroups < P ? to_f32<InT>(vp[t * p.sv[1] + row0 + r * kGroups]) : 0.f;
    dtn = to_f32<InT>(dtp[t * p.sdt[1]]);
    bn = to_f32<InT>(bp[t * p.sbeta[1]]);
  };
  if (t0 < t1) load(t0);

  for (int64_t t = t0; t < t1; ++t) {
    float4 k[NV], q[NV];
    float v[RPT];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      k[c] = kn[c];
      q[c] = qn[c];
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) v[r] = vn[r];
    float g2, beta;
    delta_gates<InT>(p, dtn, bn, A2, bias, g2, beta);
    if (t + 1 < t1) load(t + 1);
    const float a = ex2_mufu(g2);
    float kq = 0.f, sk[RPT], sq[RPT];
#pragma unroll
    for (int c = 0; c < NV; ++c) kq = dot4(k[c], q[c], kq);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      sk[r] = 0.f;
      sq[r] = 0.f;
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        sk[r] = dot4(S[r][c], k[c], sk[r]);
        sq[r] = dot4(S[r][c], q[c], sq[r]);
      }
    }
    kq = sum8(kq);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      sk[r] = sum8(sk[r]);
      sq[r] = sum8(sq[r]);
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const float u = beta * (v[r] - a * sk[r]);
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        S[r][c].x = fmaf(u, k[c].x, a * S[r][c].x);
        S[r][c].y = fmaf(u, k[c].y, a * S[r][c].y);
        S[r][c].z = fmaf(u, k[c].z, a * S[r][c].z);
        S[r][c].w = fmaf(u, k[c].w, a * S[r][c].w);
      }
      const int row = row0 + r * kGroups;
      if (lane8 == 0 && row < P)
        yp[t * p.sy[1] + row] = from_f32<OutT>(p.scale * fmaf(a, sq[r], u * kq));
    }
  }

  if (!p.last) return;
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = row0 + r * kGroups;
    if (row >= P) continue;
    float *dst = p.last + base + static_cast<int64_t>(row) * N;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = c * 32 + lane8 * 4;
      if constexpr (VEC) {
        if (col < N) __stcs(reinterpret_cast<float4 *>(dst + col), S[r][c]);
      } else {
        const float v[4] = {S[r][c].x, S[r][c].y, S[r][c].z, S[r][c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < N) dst[col + e] = v[e];
      }
    }
  }
}

bool al(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename InT, typename OutT, int NV, int RPT, bool VEC>
cudaError_t go(const DeltaParams &p, cudaStream_t stream) {
  const int64_t nrb = (p.P + kGroups * RPT - 1) / (kGroups * RPT);
  delta_recurrent_kernel<InT, OutT, NV, RPT, VEC>
      <<<static_cast<unsigned>(p.seqs * p.H * nrb), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename InT, typename OutT, bool VEC>
cudaError_t by_size(const DeltaParams &p, cudaStream_t stream) {
  if (p.N <= 64) return go<InT, OutT, 2, 2, VEC>(p, stream);
  if (p.N <= 128) return go<InT, OutT, 4, 2, VEC>(p, stream);
  return go<InT, OutT, 8, 1, VEC>(p, stream);
}

// four-column vectors everywhere: the state's rows and the q, k rows
bool vectors(const DeltaParams &p, size_t es) {
  if (p.N % 4 || !al(p.h0, 16) || !al(p.last, 16) || !al(p.q, 4 * es) || !al(p.k, 4 * es))
    return false;
  for (int i = 0; i < 3; ++i)
    if (p.sq[i] % 4 || p.sk[i] % 4) return false;
  return true;
}

bool valid_dtype(mss_dtype t) { return t == MSS_F32 || t == MSS_BF16; }

// Batch, step and head strides of a (batch, steps, heads, width) tensor:
// non-negative and sane; rows of an output must not overlap.
bool strides_ok(const int64_t (&s)[3], const int64_t (&n)[3], int64_t width, bool output) {
  const int64_t lim = int64_t(1) << 44;
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] > lim) return false;
  if (!output) return true;
  // dimensions of size above one, by stride: each has to step over what the
  // smaller ones span
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return s[a] < s[b]; });
  int64_t span = width;
  for (int i : order) {
    if (n[i] < 2) continue;
    if (s[i] < span) return false;
    span += (n[i] - 1) * s[i];
  }
  return true;
}

mss_status check_sizes(int64_t batch, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N,
                       mss_dtype in, mss_dtype out) {
  if (batch < 1 || L < 1 || H < 1 || P < 1 || G < 1 || N < 1 || H % G != 0)
    return MSS_ERR_INVALID_ARG;
  if (!valid_dtype(in) || !valid_dtype(out)) return MSS_ERR_INVALID_ARG;
  if (N > 256) return MSS_ERR_UNSUPPORTED;
  // sizes whose grid, 32-bit tensor coordinates or row index would overflow
  const int64_t lim = int64_t(1) << 30;
  if (P > lim || H > lim || L > lim || batch > lim || batch > lim / H ||
      batch * H > lim / ((P + 15) / 16))
    return MSS_ERR_UNSUPPORTED;
  return MSS_OK;
}


}  // namespace

cudaError_t launch_delta_recurrent(const DeltaParams &p, bool in_bf16, bool out_bf16,
                                   cudaStream_t stream) {
  const bool vec = vectors(p, in_bf16 ? 2 : 4);
  auto run = [&](auto in, auto out) {
    using I = decltype(in);
    using O = decltype(out);
    return vec ? by_size<I, O, true>(p, stream) : by_size<I, O, false>(p, stream);
  };
  if (in_bf16)
    return out_bf16 ? run(__nv_bfloat16(), __nv_bfloat16()) : run(__nv_bfloat16(), float());
  return out_bf16 ? run(float(), __nv_bfloat16()) : run(float(), float());
}

}  // namespace sss48

using namespace sss48;

extern "C" mss_status gated_delta_fwd(const mss_delta_args *a, void *stream) {
  sss48::NvtxRange range("gated_delta_fwd");
  if (!a) return MSS_ERR_INVALID_ARG;
  const bool packed = a->cu_seqlens != nullptr;
  if (packed ? (a->num_seqs < 1 || a->batch != 1 || !al(a->cu_seqlens, 4)) : a->num_seqs != 0)
    return MSS_ERR_INVALID_ARG;
  const int64_t seqs = packed ? a->num_seqs : a->batch;
  const mss_status st = check_sizes(seqs, a->seqlen, a->nheads, a->headdim, a->ngroups, a->dstate,
                                    a->in_dtype, a->out_dtype);
  if (st != MSS_OK) return st;
  if (!a->q || !a->k || !a->v || !a->dt || !a->A || !a->beta || !a->y) return MSS_ERR_INVALID_ARG;
  if (a->plan < MSS_DELTA_AUTO || a->plan > MSS_DELTA_CHUNKED) return MSS_ERR_INVALID_ARG;
  const size_t ie = a->in_dtype == MSS_BF16 ? 2 : 4, oe = a->out_dtype == MSS_BF16 ? 2 : 4;
  if (!al(a->q, ie) || !al(a->k, ie) || !al(a->v, ie) || !al(a->dt, ie) || !al(a->beta, ie) ||
      !al(a->y, oe) || !al(a->A, 4) || !al(a->dt_bias, 4) || !al(a->h0, 4) ||
      !al(a->last_state, 4))
    return MSS_ERR_INVALID_ARG;
  const int64_t ng[3] = {a->batch, a->seqlen, a->ngroups}, nh[3] = {a->batch, a->seqlen, a->nheads};
  if (!strides_ok(a->stride_q, ng, a->dstate, false) ||
      !strides_ok(a->stride_k, ng, a->dstate, false) ||
      !strides_ok(a->stride_v, nh, a->headdim, false) || !strides_ok(a->stride_dt, nh, 1, false) ||
      !strides_ok(a->stride_beta, nh, 1, false) || !strides_ok(a->stride_y, nh, a->headdim, true))
    return MSS_ERR_INVALID_ARG;
  DeltaParams p{};
  p.seqs = seqs;
  p.batch = a->batch;
  p.L = a->seqlen;
  p.H = a->nheads;
  p.P = a->headdim;
  p.G = a->ngroups;
  p.N = a->dstate;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.dt = a->dt;
  p.beta = a->beta;
  p.A = a->A;
  p.dt_bias = a->dt_bias;
  p.softplus = a->dt_softplus ? 1 : 0;
  p.sigmoid = a->beta_sigmoid ? 1 : 0;
  p.scale = a->scale;
  p.h0 = a->h0;
  p.y = a->y;
  p.last = a->last_state;
  for (int i = 0; i < 3; ++i) {
    p.sq[i] = a->stride_q[i];
    p.sk[i] = a->stride_k[i];
    p.sv[i] = a->stride_v[i];
    p.sdt[i] = a->stride_dt[i];
    p.sbeta[i] = a->stride_beta[i];
    p.sy[i] = a->stride_y[i];
  }
  p.cu = a->cu_seqlens;
  p.spin_ns = a->spin_timeout_ns ? a->spin_timeout_ns : 2000000000ull;
  const bool bf16 = a->in_dtype == MSS_BF16;
  const bool applies = delta_chunk_applies(p, bf16);
  if (a->plan == MSS_DELTA_CHUNKED && !applies) return MSS_ERR_UNSUPPORTED;
  if (applies && (a->plan == MSS_DELTA_CHUNKED ||
                  (a->plan == MSS_DELTA_AUTO && p.L / (packed ? seqs : 1) >= kChunkSteps))) {
    p.status = delta_status_word();
    if (!p.status) return MSS_ERR_CUDA;
    return launch_delta_chunk(p, a->out_dtype == MSS_BF16, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MSS_OK
               : MSS_ERR_CUDA;
  }
  return launch_delta_recurrent(p, a->in_dtype == MSS_BF16, a->out_dtype == MSS_BF16,
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MSS_OK
             : MSS_ERR_CUDA;
}

extern "C" mss_status gated_delta_update(const mss_delta_update_args *a, void *stream) {
  sss48::NvtxRange range("gated_delta_update");
  if (!a) return MSS_ERR_INVALID_ARG;
  const mss_status st = check_sizes(a->batch, 1, a->nheads, a->headdim, a->ngroups, a->dstate,
                                    a->in_dtype, a->out_dtype);
  if (st != MSS_OK) return st;
  if (!a->state || !a->q || !a->k || !a->v || !a->dt || !a->A || !a->beta || !a->y)
    return MSS_ERR_INVALID_ARG;
  const size_t ie = a->in_dtype == MSS_BF16 ? 2 : 4, oe = a->out_dtype == MSS_BF16 ? 2 : 4;
  if (!al(a->q, ie) || !al(a->k, ie) || !al(a->v, ie) || !al(a->dt, ie) || !al(a->beta, ie) ||
      !al(a->y, oe) || !al(a->A, 4) || !al(a->dt_bias, 4) || !al(a->state, 4))
    return MSS_ERR_INVALID_ARG;
  DeltaParams p{};
  auto three = [](const int64_t (&s)[2], int64_t (&o)[3]) {
    o[0] = s[0];
    o[1] = 0;
    o[2] = s[1];
  };
  three(a->stride_q, p.sq);
  three(a->stride_k, p.sk);
  three(a->stride_v, p.sv);
  three(a->stride_dt, p.sdt);
  three(a->stride_beta, p.sbeta);
  three(a->stride_y, p.sy);
  const int64_t ng[3] = {a->batch, 1, a->ngroups}, nh[3] = {a->batch, 1, a->nheads};
  if (!strides_ok(p.sq, ng, a->dstate, false) || !strides_ok(p.sk, ng, a->dstate, false) ||
      !strides_ok(p.sv, nh, a->headdim, false) || !strides_ok(p.sdt, nh, 1, false) ||
      !strides_ok(p.sbeta, nh, 1, false) || !strides_ok(p.sy, nh, a->headdim, true))
    return MSS_ERR_INVALID_ARG;
  p.seqs = p.batch = a->batch;
  p.L = 1;
  p.H = a->nheads;
  p.P = a->headdim;
  p.G = a->ngroups;
  p.N = a->dstate;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.dt = a->dt;
  p.beta = a->beta;
  p.A = a->A;
  p.dt_bias = a->dt_bias;
  p.softplus = a->dt_softplus ? 1 : 0;
  p.sigmoid = a->beta_sigmoid ? 1 : 0;
  p.scale = a->scale;
  p.h0 = a->state;
  p.y = a->y;
  p.last = a->state;
  return launch_delta_recurrent(p, a->in_dtype == MSS_BF16, a->out_dtype == MSS_BF16,
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MSS_OK
             : MSS_ERR_CUDA;
}

extern "C" mss_status mss_gated_delta_status(void *stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return MSS_ERR_CUDA;
  unsigned *word = delta_status_word();
  unsigned v = 0;
  const unsigned zero = 0;
  if (!word || cudaMemcpy(&v, word, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess)
    return MSS_ERR_CUDA;
  if (v && cudaMemcpy(word, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
    return MSS_ERR_CUDA;
  return v ? MSS_ERR_TIMEOUT : MSS_OK;
}
