// gated_delta.cuh -- parameters and launchers of the gated delta rule's two
// evaluations (gated_delta.cu: recurrent and the C ABI; gated_delta_chunk.cu:
// 64-step chunks on the tensor cores).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "device_math.cuh"

namespace sss48 {

struct DeltaParams {
  int64_t seqs;  // independent sequences: batch rows, or the packed ones
  int64_t batch, L, H, P, G, N;
  const void *q, *k, *v, *dt, *beta;
  const float *A, *dt_bias;
  int softplus, sigmoid;
  float scale;
  const float *h0;
  void *y;
  float *last;
  int64_t sq[3], sk[3], sv[3], sdt[3], sbeta[3], sy[3];  // {batch, step, head}
  const int32_t *cu;
  unsigned *status;
  uint64_t spin_ns;
  // sequences cut into `segs` segments of seg_chunks chunks (segs 0: whole);
  // pass 1 or 2 of the two that then run (gated_delta_chunk.cu)
  int segs, seg_chunks, pass;
  float *ends, *moves;  // (segs - 1) states, (segs - 2) transitions of every head
};

// Steps [t0, t1) of sequence s in batch row b.  Packed offsets come from the
// device and are clamped to the tensor, so a bad one cannot lead outside it.
__device__ __forceinline__ void delta_span(const DeltaParams &p, int64_t s, int64_t &b,
                                           int64_t &t0, int64_t &t1) {
  if (p.cu) {
    b = 0;
    const int64_t lo = p.cu[s], hi = p.cu[s + 1];
    t0 = lo < 0 ? 0 : (lo > p.L ? p.L : lo);
    t1 = hi < t0 ? t0 : (hi > p.L ? p.L : hi);
  } else {
    b = s;
    t0 = 0;
    t1 = p.L;
  }
}

// log2 of the decay and the writing strength of one step
template <typename InT>
__device__ __forceinline__ void delta_gates(const DeltaParams &p, float dt, float beta, float A2,
                                            float bias, float &g2, float &b) {
  const float x = dt + bias;
  g2 = (p.softplus ? softplus_f(x) : x) * A2;
  b = p.sigmoid ? __fdividef(1.0f, 1.0f + ex2_mufu(-beta * kLog2e)) : beta;
}

cudaError_t launch_delta_recurrent(const DeltaParams &p, bool in_bf16, bool out_bf16,
                                   cudaStream_t stream);
// true where the chunked kernel applies to these types, sizes and addresses
bool delta_chunk_applies(const DeltaParams &p, bool in_bf16);
cudaError_t launch_delta_chunk(const DeltaParams &p, bool out_bf16, cudaStream_t stream);
// bytes of copies of q, k, v that tensor maps can read, and the launch that
// makes them at `to` and points p at them
int64_t delta_copy_bytes(const DeltaParams &p);
cudaError_t launch_delta_copy(DeltaParams *p, void *to, cudaStream_t stream);
// segments that sequences of these sizes are best cut into on `sms` SMs (0:
// none), their length in chunks, and the floats of workspace that takes
int delta_segments(const DeltaParams &p, int sms, int *seg_chunks, int64_t *floats);
unsigned *delta_status_word();

}  // namespace sss48
