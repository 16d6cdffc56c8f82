// gated_delta.cu -- the gated delta rule step by step, and its C ABI.
//
//   u_t = b_t (v_t - a_t S k_t),  S <- a_t S + u_t k_t^T,  y_t = scale S q_t
//
// Eight lanes share a row of S (headdim x dstate) and hold its columns in
// registers, four neighbouring columns of every 32; a thread holds one row or
// two.  Both readouts are taken from the state before the step,
//
//   S_t q = a S_{t-1} q + u (k . q),
//
// so the two dot products of a row run beside each other and one round of
// shuffles over the eight lanes sums both.
//
// One token (the decode step) is bound by reading and writing the fp32 state
// (8 headdim dstate bytes per head), every load of which is issued before the
// arithmetic: 192 sequences of 32 heads of 128 x 128 take 124 to 127 us, 97 to
// 99 % of the copy bandwidth.
//
// Over more steps the chain of a step (dots, three shuffles, update) bounds it.
// What does not hang on the state is kept out of that chain: a tile of TB steps
// of q, k, v is loaded into registers while the tile before is worked on, then
// put into shared memory as fp32, where the gates and k . q of its steps are
// taken by one thread or eight lanes each.  (Loading one step ahead into
// registers left a step waiting for memory: 227 us for 2 x 517 steps of 6
// heads of 64 x 64 in fp32, 90 us this way.)
#include "gated_delta.cuh"

#include <cuda_bf16.h>

#include <algorithm>

#include "gated_delta.h"
#include "nvtx_range.cuh"

namespace sss48 {
namespace {

constexpr int kThreads = 128;
// Steps of a sequence (packed ones: on average, their lengths are on the device;
// a pack of one long sequence and many short ones is therefore worth an explicit
// plan: 8000 steps beside 300 single ones 3719 us, 1570 in chunks) from which the
// chunked evaluation runs.  Steps against chunks, us, 32 heads of 128 x 128 in
// bf16: of one sequence 10.4 / 15.4 at 16 steps, 14.6 / 14.8 at 32, 27 / 15 at
// 64; of 8 sequences 25 / 30, 44 / 29, 82 / 29; of 32 84 / 97, 156 / 95, 304 / 95.
constexpr int64_t kChunkSteps = 32;
// ... and where q, k, v are copied for it first (sizes, strides or addresses
// that tensor maps do not take): one sequence of 32 heads of 100 x 100, steps
// against copy and chunks, us: 21 / 20 at 48 steps, 27 / 21 at 64, 50 / 25 at
// 128; 8 of 2048 2608 / 525.
constexpr int64_t kCopySteps = 48;

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
template <int LANES> __device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// How rows of the state lie on a block: LANES threads share a row and hold NV
// vectors of four columns each, LANES vectors apart; a thread holds RPT rows,
// kSide apart.
template <int LANES_, int NV_, int RPT_> struct Layout {
  static constexpr int LANES = LANES_, NV = NV_, RPT = RPT_;
  static constexpr int kSide = kThreads / LANES, kRows = kSide * RPT;  // of a block
  static constexpr int kCols = 4 * LANES * NV;
  static __device__ __forceinline__ int column(int c, int lane) { return 4 * (c * LANES + lane); }
};

// the thread's part of the state at `src` (NULL: zeros).  It is read once and
// written once: streaming accesses keep it from displacing the other inputs in
// the caches.
template <typename Y, bool VEC>
__device__ __forceinline__ void load_state(float4 (&S)[Y::RPT][Y::NV], const float *src, int row0,
                                           int P, int N, int lane) {
#pragma unroll
  for (int r = 0; r < Y::RPT; ++r) {
    const int row = row0 + r * Y::kSide;
#pragma unroll
    for (int c = 0; c < Y::NV; ++c) {
      const int col = Y::column(c, lane);
      S[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (src && row < P) {
        const float *at = src + static_cast<int64_t>(row) * N;
        if constexpr (VEC) {
          if (col < N) S[r][c] = __ldcs(reinterpret_cast<const float4 *>(at + col));
        } else {
          S[r][c] = row4<float, false>(at, col, N);
        }
      }
    }
  }
}
template <typename Y, bool VEC>
__device__ __forceinline__ void store_state(const float4 (&S)[Y::RPT][Y::NV], float *dst, int row0,
                                            int P, int N, int lane) {
  if (!dst) return;
#pragma unroll
  for (int r = 0; r < Y::RPT; ++r) {
    const int row = row0 + r * Y::kSide;
    if (row >= P) continue;
    float *at = dst + static_cast<int64_t>(row) * N;
#pragma unroll
    for (int c = 0; c < Y::NV; ++c) {
      const int col = Y::column(c, lane);
      if constexpr (VEC) {
        if (col < N) __stcs(reinterpret_cast<float4 *>(at + col), S[r][c]);
      } else {
        const float v[4] = {S[r][c].x, S[r][c].y, S[r][c].z, S[r][c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < N) at[col + e] = v[e];
      }
    }
  }
}

// k . q, and S k and S q of the thread's rows, over the lanes of each
template <int LANES, int NV>
__device__ __forceinline__ float inner(const float4 (&k)[NV], const float4 (&q)[NV]) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < NV; ++c) s = dot4(k[c], q[c], s);
  return sum_lanes<LANES>(s);
}
template <typename Y>
__device__ __forceinline__ void readouts(const float4 (&S)[Y::RPT][Y::NV],
                                         const float4 (&k)[Y::NV], const float4 (&q)[Y::NV],
                                         float (&sk)[Y::RPT], float (&sq)[Y::RPT]) {
#pragma unroll
  for (int r = 0; r < Y::RPT; ++r) {
    // (two sums of each: half the chain)
    float a[2] = {0.f, 0.f}, b[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < Y::NV; ++c) {
      a[c & 1] = dot4(S[r][c], k[c], a[c & 1]);
      b[c & 1] = dot4(S[r][c], q[c], b[c & 1]);
    }
    sk[r] = a[0] + a[1];
    sq[r] = b[0] + b[1];
  }
#pragma unroll
  for (int r = 0; r < Y::RPT; ++r) {
    sk[r] = sum_lanes<Y::LANES>(sk[r]);
    sq[r] = sum_lanes<Y::LANES>(sq[r]);
  }
}
// S <- a S + u k
template <int NV>
__device__ __forceinline__ void write_row(float4 (&S)[NV], const float4 (&k)[NV], float a,
                                          float u) {
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    S[c].x = fmaf(u, k[c].x, a * S[c].x);
    S[c].y = fmaf(u, k[c].y, a * S[c].y);
    S[c].z = fmaf(u, k[c].z, a * S[c].z);
    S[c].w = fmaf(u, k[c].w, a * S[c].w);
  }
}

// the place of a thread and the tensors of its sequence and head
template <typename InT, typename OutT, typename Y> struct Seat {
  int h, lane, row0;
  int64_t base, t0, t1;
  float A2, bias;
  const InT *q, *k, *v, *dt, *beta;
  OutT *y;
  __device__ __forceinline__ explicit Seat(const DeltaParams &p) {
    const int nrb = static_cast<int>((p.P + Y::kRows - 1) / Y::kRows);
    const int64_t sh = blockIdx.x / nrb;
    const int rb = static_cast<int>(blockIdx.x - sh * nrb);
    const int64_t s = sh / p.H;
    h = static_cast<int>(sh - s * p.H);
    const int g = h / static_cast<int>(p.H / p.G);
    lane = threadIdx.x % Y::LANES;
    row0 = rb * Y::kRows + threadIdx.x / Y::LANES;
    base = sh * p.P * p.N;
    int64_t b;
    delta_span(p, s, b, t0, t1);
    A2 = p.A[h] * kLog2e;
    bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    q = static_cast<const InT *>(p.q) + b * p.sq[0] + g * p.sq[2];
    k = static_cast<const InT *>(p.k) + b * p.sk[0] + g * p.sk[2];
    v = static_cast<const InT *>(p.v) + b * p.sv[0] + h * p.sv[2];
    dt = static_cast<const InT *>(p.dt) + b * p.sdt[0] + h * p.sdt[2];
    beta = static_cast<const InT *>(p.beta) + b * p.sbeta[0] + h * p.sbeta[2];
    y = static_cast<OutT *>(p.y) + b * p.sy[0] + h * p.sy[2];
  }
};

// one token of every sequence (not packed)
template <typename InT, typename OutT, typename Y, bool VEC>
__global__ void __launch_bounds__(kThreads) delta_token_kernel(const DeltaParams p) {
  constexpr int NV = Y::NV, RPT = Y::RPT;
  const int N = static_cast<int>(p.N), P = static_cast<int>(p.P);
  const Seat<InT, OutT, Y> at(p);
  float4 S[RPT][NV], k[NV], q[NV];
  load_state<Y, VEC>(S, p.h0 ? p.h0 + at.base : nullptr, at.row0, P, N, at.lane);
  float v[RPT], sk[RPT], sq[RPT], g2, beta;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    k[c] = row4<InT, VEC>(at.k, Y::column(c, at.lane), N);
    q[c] = row4<InT, VEC>(at.q, Y::column(c, at.lane), N);
  }
#pragma unroll
  for (int r = 0; r < RPT; ++r)
    v[r] = at.row0 + r * Y::kSide < P ? to_f32<InT>(at.v[at.row0 + r * Y::kSide]) : 0.f;
  delta_gates<InT>(p, to_f32<InT>(*at.dt), to_f32<InT>(*at.beta), at.A2, at.bias, g2, beta);
  const float a = ex2_mufu(g2), kq = inner<Y::LANES>(k, q);
  readouts<Y>(S, k, q, sk, sq);
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const float u = beta * (v[r] - a * sk[r]);
    write_row<NV>(S[r], k, a, u);
    const int row = at.row0 + r * Y::kSide;
    if (at.lane == 0 && row < P) at.y[row] = from_f32<OutT>(p.scale * fmaf(a, sq[r], u * kq));
  }
  store_state<Y, VEC>(S, p.last ? p.last + at.base : nullptr, at.row0, P, N, at.lane);
}

// sequences of any length
template <typename InT, typename OutT, typename Y, bool VEC>
__global__ void __launch_bounds__(kThreads) delta_steps_kernel(const DeltaParams p) {
  constexpr int NV = Y::NV, RPT = Y::RPT, kCols = Y::kCols, kRows = Y::kRows;
  constexpr int TB = kCols == 256 ? 8 : 16;                       // steps of a tile
  constexpr int kItems = TB * kCols / 4 / kThreads;               // vectors of a thread, of q and of k
  constexpr int kVals = TB * kRows / kThreads;
  __shared__ __align__(16) float ks[2][TB][kCols], qs[2][TB][kCols];
  __shared__ float vs[2][TB][kRows], gate[2][TB][4];  // gate: a, b, k . q
  const int N = static_cast<int>(p.N), P = static_cast<int>(p.P), tid = threadIdx.x;
  const Seat<InT, OutT, Y> at(p);
  const int side = tid / Y::LANES, block0 = at.row0 - side;

  float4 kn[kItems], qn[kItems];
  float vn[kVals], dtn = 0.f, bn = 0.f;
  // a tile's part of a thread, towards registers (zeros behind the sequence)
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int item = tid + i * kThreads, col = item % (kCols / 4) * 4;
      const int64_t r = t + item / (kCols / 4);
      const bool in = r < at.t1;
      kn[i] = row4<InT, VEC>(at.k + (in ? r * p.sk[1] : 0), col, in ? N : 0);
      qn[i] = row4<InT, VEC>(at.q + (in ? r * p.sq[1] : 0), col, in ? N : 0);
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int item = tid + i * kThreads, row = block0 + item % kRows;
      const int64_t r = t + item / kRows;
      vn[i] = r < at.t1 && row < P ? to_f32<InT>(at.v[r * p.sv[1] + row]) : 0.f;
    }
    if (tid < TB && t + tid < at.t1) {
      dtn = to_f32<InT>(at.dt[(t + tid) * p.sdt[1]]);
      bn = to_f32<InT>(at.beta[(t + tid) * p.sbeta[1]]);
    }
  };
  // ... and from there into the buffer, with what follows from them
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int item = tid + i * kThreads;
      *reinterpret_cast<float4 *>(&ks[buf][0][0] + item * 4) = kn[i];
      *reinterpret_cast<float4 *>(&qs[buf][0][0] + item * 4) = qn[i];
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i) (&vs[buf][0][0])[tid + i * kThreads] = vn[i];
    if (tid < TB) {
      float g2, b;
      delta_gates<InT>(p, dtn, bn, at.A2, at.bias, g2, b);
      gate[buf][tid][0] = ex2_mufu(g2);
      gate[buf][tid][1] = b;
    }
    __syncthreads();
    if ((tid >> 3) < TB) {  // k . q, eight lanes to a step (whole warps)
      constexpr int n = kCols / 32;
      float4 k[n], q[n];
#pragma unroll
      for (int c = 0; c < n; ++c) {
        k[c] = *reinterpret_cast<const float4 *>(&ks[buf][tid >> 3][32 * c + 4 * (tid & 7)]);
        q[c] = *reinterpret_cast<const float4 *>(&qs[buf][tid >> 3][32 * c + 4 * (tid & 7)]);
      }
      const float kq = inner<8>(k, q);
      if ((tid & 7) == 0) gate[buf][tid >> 3][2] = kq;
    }
    __syncthreads();
  };

  if (at.t0 < at.t1) load(at.t0);
  float4 S[RPT][NV];
  load_state<Y, VEC>(S, p.h0 ? p.h0 + at.base : nullptr, at.row0, P, N, at.lane);
  if (at.t0 < at.t1) put(0);
  int buf = 0;
  for (int64_t t = at.t0; t < at.t1; t += TB, buf ^= 1) {
    if (t + TB < at.t1) load(t + TB);
    const int n = at.t1 - t < TB ? static_cast<int>(at.t1 - t) : TB;
    OutT *yp = at.y + t * p.sy[1];
#pragma unroll 2
    for (int j = 0; j < n; ++j) {
      float4 k[NV], q[NV];
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        k[c] = *reinterpret_cast<const float4 *>(&ks[buf][j][Y::column(c, at.lane)]);
        q[c] = *reinterpret_cast<const float4 *>(&qs[buf][j][Y::column(c, at.lane)]);
      }
      const float a = gate[buf][j][0], beta = gate[buf][j][1], kq = gate[buf][j][2];
      float sk[RPT], sq[RPT];
      readouts<Y>(S, k, q, sk, sq);
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const float u = beta * (vs[buf][j][side + r * Y::kSide] - a * sk[r]);
        write_row<NV>(S[r], k, a, u);
        const int row = at.row0 + r * Y::kSide;
        if (at.lane == 0 && row < P)
          yp[j * p.sy[1] + row] = from_f32<OutT>(p.scale * fmaf(a, sq[r], u * kq));
      }
    }
    // (its own syncs order the tiles: the buffer written here was read before
    // the ones of the last tile)
    if (t + TB < at.t1) put(buf ^ 1);
  }
  store_state<Y, VEC>(S, p.last ? p.last + at.base : nullptr, at.row0, P, N, at.lane);
}

bool al(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename Y> unsigned blocks(const DeltaParams &p) {
  return static_cast<unsigned>(p.seqs * p.H * ((p.P + Y::kRows - 1) / Y::kRows));
}

// Eight lanes read 128 bytes of a row of the state at a time.  Two rows of a
// thread share its k and q (steps, 8 sequences of 64 of 32 heads of 128 x 128:
// 80 us, 111 with one row in twice the blocks, 107 with four lanes to a row; few
// blocks gain 5 % from one row); at dstate 256 two would not fit.
template <typename InT, typename OutT, bool VEC>
cudaError_t by_size(const DeltaParams &p, cudaStream_t stream) {
  const bool token = p.L == 1 && !p.cu;
  auto go = [&](auto layout) {
    using Y = decltype(layout);
    if (token)
      delta_token_kernel<InT, OutT, Y, VEC><<<blocks<Y>(p), kThreads, 0, stream>>>(p);
    else
      delta_steps_kernel<InT, OutT, Y, VEC><<<blocks<Y>(p), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  };
  if (p.N <= 64) return go(Layout<8, 2, 2>());
  if (p.N <= 128) return go(Layout<8, 4, 2>());
  return go(Layout<8, 8, 1>());
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

bool chunked(const DeltaParams &p, int plan, int64_t steps) {
  return plan == MSS_DELTA_CHUNKED ||
         (plan == MSS_DELTA_AUTO && p.L / (p.cu ? p.seqs : 1) >= steps);
}

// What a call does with a workspace: copies of q, k, v that tensor maps can
// read, and the segments of its sequences (p.segs, p.seg_chunks; on the current
// device).
struct Room {
  int64_t copies = 0, segments = 0;  // bytes
  int64_t bytes() const { return copies + segments; }
};
mss_status workspace(DeltaParams &p, int plan, bool bf16, bool applies, Room *room) {
  const bool copies = !applies && bf16 && p.N <= 128 && chunked(p, plan, kCopySteps);
  if (copies) room->copies = (delta_copy_bytes(p) + 15) / 16 * 16;
  if (!p.cu && (copies || (applies && chunked(p, plan, kChunkSteps)))) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return MSS_ERR_CUDA;
    int64_t floats = 0;
    p.segs = delta_segments(p, sms, &p.seg_chunks, &floats);
    room->segments = 4 * floats;
  }
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

namespace {

// sizes, strides and pointers of a call's tensors
mss_status sizes(const mss_delta_args *a, DeltaParams *p) {
  if (!a) return MSS_ERR_INVALID_ARG;
  const bool packed = a->cu_seqlens != nullptr;
  if (packed ? (a->num_seqs < 1 || a->batch != 1 || !al(a->cu_seqlens, 4)) : a->num_seqs != 0)
    return MSS_ERR_INVALID_ARG;
  if (a->plan < MSS_DELTA_AUTO || a->plan > MSS_DELTA_CHUNKED) return MSS_ERR_INVALID_ARG;
  p->seqs = packed ? a->num_seqs : a->batch;
  const mss_status st = check_sizes(p->seqs, a->seqlen, a->nheads, a->headdim, a->ngroups,
                                    a->dstate, a->in_dtype, a->out_dtype);
  if (st != MSS_OK) return st;
  p->batch = a->batch;
  p->L = a->seqlen;
  p->H = a->nheads;
  p->P = a->headdim;
  p->G = a->ngroups;
  p->N = a->dstate;
  p->q = a->q;
  p->k = a->k;
  p->v = a->v;
  p->h0 = a->h0;
  p->last = a->last_state;
  p->cu = a->cu_seqlens;
  for (int i = 0; i < 3; ++i) {
    p->sq[i] = a->stride_q[i];
    p->sk[i] = a->stride_k[i];
    p->sv[i] = a->stride_v[i];
  }
  return MSS_OK;
}

}  // namespace

extern "C" mss_status gated_delta_fwd(const mss_delta_args *a, void *stream) {
  sss48::NvtxRange range("gated_delta_fwd");
  DeltaParams p{};
  const mss_status st = sizes(a, &p);
  if (st != MSS_OK) return st;
  if (!a->q || !a->k || !a->v || !a->dt || !a->A || !a->beta || !a->y) return MSS_ERR_INVALID_ARG;
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
  p.dt = a->dt;
  p.beta = a->beta;
  p.A = a->A;
  p.dt_bias = a->dt_bias;
  p.softplus = a->dt_softplus ? 1 : 0;
  p.sigmoid = a->beta_sigmoid ? 1 : 0;
  p.scale = a->scale;
  p.y = a->y;
  for (int i = 0; i < 3; ++i) {
    p.sdt[i] = a->stride_dt[i];
    p.sbeta[i] = a->stride_beta[i];
    p.sy[i] = a->stride_y[i];
  }
  p.spin_ns = a->spin_timeout_ns ? a->spin_timeout_ns : 2000000000ull;
  const bool bf16 = a->in_dtype == MSS_BF16;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  const bool applies = delta_chunk_applies(p, bf16);
  if (a->plan == MSS_DELTA_CHUNKED && !applies) return MSS_ERR_UNSUPPORTED;
  Room room;
  if (a->workspace) {
    const mss_status w = workspace(p, a->plan, bf16, applies, &room);
    if (w != MSS_OK) return w;
    if (!al(a->workspace, 16)) return MSS_ERR_INVALID_ARG;
    if (a->workspace_bytes < static_cast<size_t>(room.bytes())) return MSS_ERR_WORKSPACE;
  }
  if (room.copies || (applies && chunked(p, a->plan, kChunkSteps))) {
    p.status = delta_status_word();
    if (!p.status) return MSS_ERR_CUDA;
    char *ws = static_cast<char *>(a->workspace);
    if (room.copies && launch_delta_copy(&p, ws, on) != cudaSuccess) return MSS_ERR_CUDA;
    if (p.segs) {
      p.ends = reinterpret_cast<float *>(ws + room.copies);
      p.moves = p.ends + (p.segs - 1) * p.seqs * p.H * p.P * p.N;
    }
    return launch_delta_chunk(p, a->out_dtype == MSS_BF16, on) == cudaSuccess ? MSS_OK
                                                                            : MSS_ERR_CUDA;
  }
  return launch_delta_recurrent(p, a->in_dtype == MSS_BF16, a->out_dtype == MSS_BF16,
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MSS_OK
             : MSS_ERR_CUDA;
}

extern "C" mss_status mss_gated_delta_workspace_size(const mss_delta_args *a, size_t *bytes) {
  if (!bytes) return MSS_ERR_INVALID_ARG;
  DeltaParams p{};
  mss_status st = sizes(a, &p);
  if (st != MSS_OK) return st;
  const bool bf16 = a->in_dtype == MSS_BF16;
  Room room;
  if ((st = workspace(p, a->plan, bf16, delta_chunk_applies(p, bf16), &room)) != MSS_OK) return st;
  *bytes = static_cast<size_t>(room.bytes());
  return MSS_OK;
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
