// gated_delta_chunk.cu -- the gated delta rule in chunks of C = 64 steps on
// the sm_100a tensor cores.
//
// Inside a chunk, with c_t the running sum of log2 a, D[t,s] = 2^(c_t - c_s)
// for s <= t, and H the state (headdim x dstate) before the chunk, the
// written rows U solve
//
//   (I + A) U = diag(b) (V - diag(2^c) K H^T),  A[t,s] = b_t D[t,s] k_t.k_s
//                                               for s < t.
//
// T = (I + A)^-1 does not depend on H, so with M = T diag(b) and
// W = T diag(b 2^c) K only one product with H and one with U lie on the
// chain from chunk to chunk:
//
//   U^T = V^T M^T - H W^T                   M = headdim, N = t
//   H  <- 2^(c_last) H + (U^T diag(2^(c_last - c))) K       N = dstate
//   Y^T = H Q^T diag(2^c) + U^T (Q K^T o D)^T               N = t
//
// Everything runs transposed, headdim (128 of it per block) on the lanes of
// tensor memory, so that H and U enter their products as the operand in
// tensor memory, straight from the registers of the thread that owns the row.
//
// Precision.  q, k and v are bf16 and enter exactly.  M, W, H, U and
// Q K^T o D are fp32 values given as hi + lo, two bf16 values (off by 2^-18
// at most): a product with an exact operand takes two products, one of two
// such pairs three (lo lo is left out).  H itself stays in fp32 registers and
// is added to there, not in the tensor cores' accumulators.
//
// Roles (18 warps, one block per SM: the sequence, head and 128 rows):
//   warp 0        TMA loads of the K, Q tiles (three stages) and V (two)
//   warp 1        issues every product, in one order
//   warps 2-9     the chain: H in registers (64 columns a thread), its pairs
//                 and those of U into tensor memory
//   warps 10-17   what does not depend on H, one chunk ahead: gates, A, its
//                 inverse, M, Q K^T o D, W; and the output
// The inverse: two 32 x 32 triangles by substitution, a column per lane, and
// the block below them as two 32^3 products of 3 x tf32 mma.sync.
//
// Shared memory tiles are rows of 128 bytes with the 128-byte swizzle.  Every
// wait is bounded as in tcgen05.cuh, so no block can hang.
#include <cuda_bf16.h>

#include "device_math.cuh"
#include "gated_delta.cuh"
#include "tcgen05.cuh"

namespace sss48 {
namespace {

constexpr int C = 64;                 // steps of a chunk
constexpr int kThreads = 576;
constexpr int kGroup = 256;           // threads of the chain, and of the rest
constexpr int kBarAux = 1;            // named barrier of warps 10-17

constexpr int kHalf = 64 * 128;       // 64 rows of 128 bytes
constexpr int kStageKQ = 4 * kHalf;   // K, Q of dstate 0..63, K, Q of 64..127
constexpr int kStageV = 2 * kHalf;
constexpr int oKQ = 0;
constexpr int oV = 3 * kStageKQ;
constexpr int oW = oV + 2 * kStageV;  // W^T hi, lo: [dstate][t]
constexpr int oM = oW + 4 * kHalf;    // M hi, lo, -M diag(2^c) hi, lo: [t][s]
constexpr int oP = oM + 4 * kHalf;    // two of (Q K^T o D) hi, lo: [t][s]
constexpr int oArr = oP + 4 * kHalf;  // float beta, colf, cum [C]; 2 x (du, eo)
constexpr int oBar = oArr + 7 * C * 4;
constexpr int kBars = 21;
constexpr int oTmemSlot = oBar + kBars * 8;
constexpr int oAbort = oTmemSlot + 4;
constexpr int kSmemBytes = oAbort + 4 + 1024;  // room to align the base
static_assert(kSmemBytes <= 232448, "shared memory above the per-block limit");

// the inverse's scratch lies where M is written afterwards: 32 x 32 blocks of
// rows of 40 floats (8 rows start on 8 different groups of banks)
constexpr int kLd = 40, kBlk = 32 * kLd;
constexpr int bA11 = 0, bA22 = 1, bA21 = 2, bT11 = 3, bT22 = 4, bZ = 5;
static_assert(6 * kBlk * 4 <= 4 * kHalf, "scratch of the inverse");

// tensor memory columns
constexpr uint32_t kColH = 0;     // H pairs / the update U'^T K (128)
constexpr uint32_t kColU = 128;   // U, then its pairs
constexpr uint32_t kColUd = 192;  // pairs of U diag(2^(c_last - c))
constexpr uint32_t kColO1 = 256, kColO2 = 320;
constexpr uint32_t kColS = 384;   // K K^T (lanes 0..63), Q K^T (64..127)
constexpr uint32_t kColW = 448;   // -W^T
constexpr uint32_t kTmemCols = 512;

// barriers: tiles landed and released; then, per chunk, products done (S, W,
// U, O1, the update, O) and operands ready (M and P; W; H; U; O drained)
constexpr int kFullKQ = 0, kFullV = 3, kEmptyKQ = 5, kEmptyV = 8, kDoneS = 10, kDoneW = 11,
              kDoneU = 12, kDoneO1 = 13, kDoneH = 14, kDoneO = 15, kReadyM = 16, kReadyW = 17,
              kReadyH = 18, kReadyU = 19, kFreeO = 20;

struct Maps {
  CUtensorMap q, k, v;
};

__device__ unsigned g_delta_status;

// x = hi + lo for a pair of values, packed two to a register
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(a, b);
  lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}

// c += a b, m16n8k8, tf32 operands (bits below tf32's are not read)
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4],
                                         const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// One 16 x 8 tile (rows r0.., columns n0..) of X Y, 32 deep, as three tf32
// products; X[r][k] at xa + r * xr + k * xk, Y[k][n] at yb + k * kLd + n.
__device__ __forceinline__ void tile32(const float *xa, int xr, int xk, const float *yb, int r0,
                                       int n0, int lane, float (&out)[4]) {
  const int g = lane >> 2, t = lane & 3;
  float c0[4] = {}, c1[4] = {}, c2[4] = {};
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      split_tf32(xa[(r0 + g + 8 * (i & 1)) * xr + (k + t + 4 * (i >> 1)) * xk], ah[i], al[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) split_tf32(yb[(k + t + 4 * i) * kLd + n0 + g], bh[i], bl[i]);
    mma_tf32(c0, ah, bh);
    mma_tf32(c1, al, bh);
    mma_tf32(c2, ah, bl);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = c0[i] + (c1[i] + c2[i]);
}

template <typename OutT>
__global__ void __launch_bounds__(kThreads, 1)
    delta_chunk_kernel(const __grid_constant__ Maps maps, const DeltaParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + oBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + oTmemSlot);
  volatile int *abort = reinterpret_cast<volatile int *>(sm + oAbort);
  float *beta_s = reinterpret_cast<float *>(sm + oArr);
  float *colf_s = beta_s + C, *cum_s = colf_s + C;
  float *dueo_s = cum_s + C;  // [2][du, eo][C]
  const Sync sy{bar, abort, p.status, p.spin_ns};

  if (tid == 0) {
    for (int i = 0; i < kReadyM; ++i) mbar_init(bar + i, 1);
    for (int i = kReadyM; i < kBars; ++i) mbar_init(bar + i, kGroup);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int slices = static_cast<int>((p.P + 127) / 128);
  const int64_t sh = blockIdx.x / slices;
  const int p0 = static_cast<int>(blockIdx.x - sh * slices) * 128;
  const int64_t s = sh / p.H;
  const int h = static_cast<int>(sh - s * p.H);
  const int g = h / static_cast<int>(p.H / p.G);
  const int N = static_cast<int>(p.N), P = static_cast<int>(p.P);
  int64_t b64, t0, t1;
  delta_span(p, s, b64, t0, t1);
  const int b = static_cast<int>(b64);
  const int nc = static_cast<int>((t1 - t0 + C - 1) / C);

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      for (int i = 0; i < nc; ++i) {
        const int t = static_cast<int>(t0) + i * C;
        const int a = i % 3, v = i & 1;
        if (i >= 3) sy.wait(kEmptyKQ + a, (i / 3 - 1) & 1);
        unsigned char *d = sm + oKQ + a * kStageKQ;
        mbar_expect_tx(bar + kFullKQ + a, kStageKQ);
        tma_load_4d(d, &maps.k, 0, g, t, b, bar + kFullKQ + a);
        tma_load_4d(d + kHalf, &maps.q, 0, g, t, b, bar + kFullKQ + a);
        tma_load_4d(d + 2 * kHalf, &maps.k, 64, g, t, b, bar + kFullKQ + a);
        tma_load_4d(d + 3 * kHalf, &maps.q, 64, g, t, b, bar + kFullKQ + a);
        if (i >= 2) sy.wait(kEmptyV + v, (i / 2 - 1) & 1);
        d = sm + oV + v * kStageV;
        mbar_expect_tx(bar + kFullV + v, kStageV);
        tma_load_4d(d, &maps.v, p0, h, t, b, bar + kFullV + v);
        tma_load_4d(d + kHalf, &maps.v, p0 + 64, h, t, b, bar + kFullV + v);
      }
      // no copy may still be landing when the block exits
      for (int i = nc > 3 ? nc - 3 : 0; i < nc; ++i) sy.drain(kFullKQ + i % 3, (i / 3) & 1);
      for (int i = nc > 2 ? nc - 2 : 0; i < nc; ++i) sy.drain(kFullV + (i & 1), (i / 2) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------- tensor-core issue
    if (lane == 0 && nc > 0) {
      constexpr uint32_t idKK = idesc_bf16(128, 64, 0, 0);   // both K-major
      constexpr uint32_t idTK = idesc_bf16(128, 64, 1, 0);   // A as stored by step
      constexpr uint32_t idKT = idesc_bf16(128, 64, 0, 1);   // B as stored by step
      const uint32_t idH = idesc_bf16(128, N <= 64 ? 64 : 128, 0, 1);
      const int nk = (N + 15) >> 4;  // 16-wide slices of dstate
      const uint64_t dW = smem_desc(sbase + oW, 16, 1024);
      const uint64_t dM = smem_desc(sbase + oM, 16, 1024);
      constexpr uint64_t kLo = 2 * kHalf >> 4;  // hi -> lo of W; M to M diag(2^c)
      constexpr uint64_t kLoM = kHalf >> 4;     // hi -> lo of M and P
      auto stage = [&](int i) { return sbase + oKQ + (i % 3) * kStageKQ; };
      // slice k of a K-major tile in 64-wide halves `half` bytes apart
      auto kslice = [](int k, uint64_t half) {
        return static_cast<uint64_t>(k >> 2) * (half >> 4) + (k & 3) * 2;
      };
      auto scores = [&](int i) {  // [K; Q] K^T
        sy.wait(kFullKQ + i % 3, (i / 3) & 1);
        tc_fence_after();
        if (!*abort) {
          const uint64_t d = smem_desc(stage(i), 16, 1024);
          for (int k = 0; k < nk; ++k) {
            const uint64_t o = kslice(k, 2 * kHalf);
            umma_bf16(tmem + kColS, d + o, d + o, idKK, k > 0);
          }
        }
        umma_commit(bar + kDoneS);
      };
      // -W^T = K^T (-M diag(2^c))^T and U^T = V^T M^T of chunk i
      auto ahead = [&](int i) {
        sy.wait(kReadyM, i & 1);
        tc_fence_after();
        if (!*abort) {
          const uint64_t dK = smem_desc(stage(i), 2 * kHalf, 1024);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_bf16(tmem + kColW, dK + (k & 3) * 128, dM + kLo + (k >> 2) * kLoM + (k & 3) * 2,
                      idTK, k > 0);
        }
        umma_commit(bar + kDoneW);
        if (i > 0) sy.wait(kDoneO, (i - 1) & 1);  // U of chunk i - 1 has been read
        sy.wait(kFullV + (i & 1), (i / 2) & 1);
        tc_fence_after();
        if (!*abort) {
          const uint64_t dV = smem_desc(sbase + oV + (i & 1) * kStageV, kHalf, 1024);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_bf16(tmem + kColU, dV + (k & 3) * 128, dM + (k >> 2) * kLoM + (k & 3) * 2, idTK,
                      k > 0);
        }
        umma_commit(bar + kEmptyV + (i & 1));
      };
      scores(0);
      ahead(0);
      if (nc > 1) scores(1);
      for (int i = 0; i < nc; ++i) {
        const uint32_t st = stage(i);
        sy.wait(kReadyW, i & 1);
        sy.wait(kReadyH, i & 1);
        tc_fence_after();
        if (!*abort) {  // U^T -= H W^T
          for (int k = 0; k < nk; ++k) {
            const uint32_t hi = tmem + kColH + (k >> 2) * 64 + (k & 3) * 8;
            umma_bf16_ts(tmem + kColU, hi, dW + k * 128, idKT, 1);
            umma_bf16_ts(tmem + kColU, hi + 32, dW + k * 128, idKT, 1);
            umma_bf16_ts(tmem + kColU, hi, dW + kLo + k * 128, idKT, 1);
          }
        }
        umma_commit(bar + kDoneU);
        if (i > 0) {
          sy.wait(kFreeO, (i - 1) & 1);
          tc_fence_after();
        }
        if (!*abort) {  // O1 = H Q^T
          const uint64_t dQ = smem_desc(st + kHalf, 16, 1024);
          for (int k = 0; k < nk; ++k) {
            const uint32_t hi = tmem + kColH + (k >> 2) * 64 + (k & 3) * 8;
            const uint64_t o = dQ + kslice(k, 2 * kHalf);
            umma_bf16_ts(tmem + kColO1, hi, o, idKK, k > 0);
            umma_bf16_ts(tmem + kColO1, hi + 32, o, idKK, 1);
          }
        }
        umma_commit(bar + kDoneO1);
        sy.wait(kReadyU, i & 1);
        sy.wait(kDoneO1, i & 1);  // the update overwrites the pairs of H
        tc_fence_after();
        if (!*abort) {  // U'^T K
          const uint64_t dK = smem_desc(st, 2 * kHalf, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t hi = tmem + kColUd + (k >> 1) * 32 + (k & 1) * 8;
            umma_bf16_ts(tmem + kColH, hi, dK + k * 128, idH, k > 0);
            umma_bf16_ts(tmem + kColH, hi + 16, dK + k * 128, idH, 1);
          }
        }
        umma_commit(bar + kDoneH);
        umma_commit(bar + kEmptyKQ + i % 3);
        if (!*abort) {  // O2 = U^T (Q K^T o D)^T
          const uint64_t dP = smem_desc(sbase + oP + (i & 1) * 2 * kHalf, 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t hi = tmem + kColU + (k >> 1) * 32 + (k & 1) * 8;
            umma_bf16_ts(tmem + kColO2, hi, dP + k * 2, idKK, k > 0);
            umma_bf16_ts(tmem + kColO2, hi + 16, dP + k * 2, idKK, 1);
            umma_bf16_ts(tmem + kColO2, hi, dP + kLoM + k * 2, idKK, 1);
          }
        }
        umma_commit(bar + kDoneO);
        if (i + 1 < nc) ahead(i + 1);
        if (i + 2 < nc) scores(i + 2);
      }
      // every product done before the tensor memory is freed
      sy.drain(kDoneO, (nc - 1) & 1);
    }
    __syncwarp();
  } else if (warp < 10) {
    // -------------------------------------------------------- the chain
    const int q = warp & 3, e = (warp - 2) >> 2;
    const int row = p0 + 32 * q + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int64_t base = (sh * p.P + row) * p.N + 64 * e;
    float H[64];
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.h0 && row < P && 64 * e + j < N)
        v = __ldcs(reinterpret_cast<const float4 *>(p.h0 + base + j));
      H[j] = v.x;
      H[j + 1] = v.y;
      H[j + 2] = v.z;
      H[j + 3] = v.w;
    }
    float gam = 1.0f;
    for (int i = 0; i < nc; ++i) {
      if (i > 0) {
        sy.wait(kDoneH, (i - 1) & 1);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[16];
          tmem_ld16(tl + kColH + 64 * e + 16 * c, v);
          tmem_wait_ld(v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            H[16 * c + j] = fmaf(gam, H[16 * c + j], __uint_as_float(v[j]));
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) split2(H[16 * c + 2 * j], H[16 * c + 2 * j + 1], hi[j], lo[j]);
        tmem_st8(tl + kColH + 64 * e + 8 * c, hi);
        tmem_st8(tl + kColH + 64 * e + 32 + 8 * c, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar + kReadyH);

      sy.wait(kReadyW, i & 1);  // (the gates' arrays, too)
      const float *du = dueo_s + (i & 1) * 2 * C, *eo = du + C;
      gam = eo[C - 1];
      sy.wait(kDoneU, i & 1);
      tc_fence_after();
      {
        // 32 steps of a thread, their pairs in the columns they came from
        uint32_t v[2][16];
        tmem_ld16(tl + kColU + 32 * e, v[0]);
        tmem_ld16(tl + kColU + 32 * e + 16, v[1]);
        tmem_wait_ld(v[0]);
        tmem_wait_ld(v[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            split2(__uint_as_float(v[c][2 * j]) * du[32 * e + 16 * c + 2 * j],
                   __uint_as_float(v[c][2 * j + 1]) * du[32 * e + 16 * c + 2 * j + 1], hi[j],
                   lo[j]);
          tmem_st8(tl + kColUd + 32 * e + 8 * c, hi);
          tmem_st8(tl + kColUd + 32 * e + 16 + 8 * c, lo);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            split2(__uint_as_float(v[c][2 * j]), __uint_as_float(v[c][2 * j + 1]), hi[j], lo[j]);
          tmem_st8(tl + kColU + 32 * e + 8 * c, hi);
          tmem_st8(tl + kColU + 32 * e + 16 + 8 * c, lo);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar + kReadyU);
    }
    if (nc > 0) {
      sy.wait(kDoneH, (nc - 1) & 1);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[16];
        tmem_ld16(tl + kColH + 64 * e + 16 * c, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          H[16 * c + j] = fmaf(gam, H[16 * c + j], __uint_as_float(v[j]));
      }
    }
    if (p.last && row < P) {
#pragma unroll
      for (int j = 0; j < 64; j += 4)
        if (64 * e + j < N)
          __stcs(reinterpret_cast<float4 *>(p.last + base + j),
                 make_float4(H[j], H[j + 1], H[j + 2], H[j + 3]));
    }
  } else {
    // --------------------------------- what does not depend on H; output
    const int q = warp & 3, e = (warp - 10) >> 2, at = tid - 320, aw = at >> 5;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float *scr = reinterpret_cast<float *>(sm + oM);
    const __nv_bfloat16 *dtp = static_cast<const __nv_bfloat16 *>(p.dt) + b * p.sdt[0] + h * p.sdt[2];
    const __nv_bfloat16 *bp =
        static_cast<const __nv_bfloat16 *>(p.beta) + b * p.sbeta[0] + h * p.sbeta[2];
    const float A2 = p.A[h] * kLog2e, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    OutT *yp = static_cast<OutT *>(p.y) + b * p.sy[0] + h * p.sy[2] + t0 * p.sy[1];
    const int row = p0 + 32 * q + lane;

    // the blocks of P above the diagonal stay zero
    for (int k = at; k < 2 * 2 * 32 * 4; k += kGroup)
      *reinterpret_cast<uint4 *>(sm + oP + (k >> 7) * kHalf + swz((k >> 2) & 31, 4 + (k & 3))) =
          make_uint4(0u, 0u, 0u, 0u);

    // raw gates of two steps of a lane (warp 0 of the group), a chunk ahead
    unsigned short rd[2] = {0, 0}, rb[2] = {0, 0};
    auto raw = [&](int j) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t t = t0 + static_cast<int64_t>(j) * C + 32 * k + lane;
        if (t < t1) {
          rd[k] = *reinterpret_cast<const unsigned short *>(dtp + t * p.sdt[1]);
          rb[k] = *reinterpret_cast<const unsigned short *>(bp + t * p.sbeta[1]);
        }
      }
    };
    if (aw == 0 && nc > 0) raw(0);

    // y rows of chunk i: scale (2^c O1 + O2)
    auto output = [&](int i) {
      sy.wait(kDoneO, i & 1);
      tc_fence_after();
      const float *eo = dueo_s + (i & 1) * 2 * C + C;
      const int64_t left = t1 - t0 - static_cast<int64_t>(i) * C;
      OutT *yr = yp + (static_cast<int64_t>(i) * C + 32 * e) * p.sy[1] + row;
      float o[32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[16], w[16];
        tmem_ld16(tl + kColO1 + 32 * e + 16 * c, v);
        tmem_ld16(tl + kColO2 + 32 * e + 16 * c, w);
        tmem_wait_ld(v);
        tmem_wait_ld(w);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          o[16 * c + j] = p.scale * fmaf(eo[32 * e + 16 * c + j], __uint_as_float(v[j]),
                                         __uint_as_float(w[j]));
      }
      tc_fence_before();
      mbar_arrive(bar + kFreeO);
      if (row < P) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (32 * e + j < left) yr[j * p.sy[1]] = from_f32<OutT>(o[j]);
      }
    };

    for (int i = 0; i < nc; ++i) {
      const int64_t left = t1 - t0 - static_cast<int64_t>(i) * C;
      const int len = left < C ? static_cast<int>(left) : C;
      float *du = dueo_s + (i & 1) * 2 * C, *eo = du + C;
      if (aw == 0) {
        // these arrays' last readers: the output of chunk i - 2
        if (i > 1) sy.wait(kFreeO, i & 1);
        float g2[2], bt[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          g2[k] = bt[k] = 0.f;
          if (32 * k + lane < len)
            delta_gates<__nv_bfloat16>(p, __uint_as_float(static_cast<uint32_t>(rd[k]) << 16),
                                       __uint_as_float(static_cast<uint32_t>(rb[k]) << 16), A2,
                                       bias, g2[k], bt[k]);
        }
        raw(i + 1);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x0 = __shfl_up_sync(0xffffffffu, g2[0], o);
          const float x1 = __shfl_up_sync(0xffffffffu, g2[1], o);
          if (lane >= o) {
            g2[0] += x0;
            g2[1] += x1;
          }
        }
        const float end0 = __shfl_sync(0xffffffffu, g2[0], 31);
        g2[1] += end0;
        const float end1 = __shfl_sync(0xffffffffu, g2[1], 31);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = 32 * k + lane;
          cum_s[t] = g2[k];
          beta_s[t] = bt[k];
          colf_s[t] = ex2_mufu((k ? end1 : end0) - g2[k]);
          du[t] = ex2_mufu(end1 - g2[k]);
          eo[t] = ex2_mufu(g2[k]);
        }
      }
      // M of the chunk before has been read: its place is free
      if (i > 0) sy.wait(kEmptyV + ((i - 1) & 1), ((i - 1) >> 1) & 1);
      sy.wait(kDoneS, i & 1);
      tc_fence_after();
      bar_sync(kBarAux, kGroup);

      if (len < C) {
        // steps of whatever lies behind the sequence: nothing of them may
        // enter a product (zero times a NaN would)
        sy.wait(kFullKQ + i % 3, (i / 3) & 1);
        sy.wait(kFullV + (i & 1), (i / 2) & 1);
        const int rows = C - len;
        for (int k = at; k < rows * 32; k += kGroup) {
          const int r = len + (k >> 5), c = k & 31;
          unsigned char *d = c < 16 ? sm + oKQ + (i % 3) * kStageKQ + (c >> 3) * 2 * kHalf
                                    : sm + oV + (i & 1) * kStageV + ((c >> 3) & 1) * kHalf;
          *reinterpret_cast<uint4 *>(d + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }

      // rows of A (lanes 0..63 of S) and of Q K^T o D (64..127), 32 columns
      // of a thread: below the diagonal 2^(c_t - c_end) colf[s], c_end the
      // end of s's block of 32, both at most 1; in a diagonal block the same
      // two factors unless the first could overflow, else one 2^x each
      if (e <= (q & 1)) {
        const int blk = q & 1, t = 32 * blk + lane;
        const bool diag = e == blk, isA = q < 2;
        uint32_t v[32];
        tmem_ld32(tl + kColS + 32 * e, v);
        const float cend = cum_s[32 * e + 31], ct = cum_s[t];
        const float rowf = isA ? beta_s[t] : 1.0f;
        const bool fact = !diag || cum_s[32 * e] - cend < 64.0f;
        const float rf = rowf * ex2_mufu(ct - cend);
        const int last = diag ? (isA ? lane : lane + 1) : 32;  // columns kept
        tmem_wait_ld(v);
        float f[32];
        if (fact) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            f[j] = j < last && t < len ? __uint_as_float(v[j]) * (rf * colf_s[32 * e + j]) : 0.f;
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            f[j] = j < last && t < len
                       ? __uint_as_float(v[j]) * (rowf * ex2_mufu(ct - cum_s[32 * e + j]))
                       : 0.f;
        }
        if (isA) {  // transposed: the substitution reads columns of A
          float *d = scr + (diag ? (blk ? bA22 : bA11) : bA21) * kBlk + lane;
#pragma unroll
          for (int j = 0; j < 32; ++j) d[j * kLd] = f[j];
        } else {
          unsigned char *d = sm + oP + (i & 1) * 2 * kHalf;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) split2(f[8 * c + 2 * k], f[8 * c + 2 * k + 1], hi[k], lo[k]);
            const uint32_t o = swz(t, 4 * e + c);
            *reinterpret_cast<uint4 *>(d + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(d + kHalf + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      }
      tc_fence_before();
      bar_sync(kBarAux, kGroup);

      if (aw < 2) {
        // column `lane` of T11 / T22: x_s is final once the steps before it
        // have been taken out of it
        const float *a = scr + (aw ? bA22 : bA11) * kBlk;
        float *d = scr + (aw ? bT22 : bT11) * kBlk + lane;
        float2 x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          x[j] = make_float2(lane == 2 * j ? 1.f : 0.f, lane == 2 * j + 1 ? 1.f : 0.f);
#pragma unroll
        for (int t = 0; t < 32; ++t) {
          const float xt = t & 1 ? x[t >> 1].y : x[t >> 1].x;
          d[t * kLd] = xt;
          const float2 m = make_float2(-xt, -xt);
#pragma unroll
          for (int j = (t + 1) >> 2; j < 8; ++j) {
            // A is zero on and above the diagonal, so the pair that holds
            // row t itself keeps it
            const float4 av = *reinterpret_cast<const float4 *>(a + t * kLd + 4 * j);
            x[2 * j] = __ffma2_rn(make_float2(av.x, av.y), m, x[2 * j]);
            x[2 * j + 1] = __ffma2_rn(make_float2(av.z, av.w), m, x[2 * j + 1]);
          }
        }
      }
      bar_sync(kBarAux, kGroup);
      // T21 = -T22 (A21 T11)
      const int r0 = 16 * (aw >> 2), n0 = 8 * (aw & 3), fr = r0 + (lane >> 2),
                fc = n0 + 2 * (lane & 3);
      float z[4];
      tile32(scr + bA21 * kBlk, 1, kLd, scr + bT11 * kBlk, r0, n0, lane, z);
      *reinterpret_cast<float2 *>(scr + bZ * kBlk + fr * kLd + fc) = make_float2(z[0], z[1]);
      *reinterpret_cast<float2 *>(scr + bZ * kBlk + (fr + 8) * kLd + fc) = make_float2(z[2], z[3]);
      bar_sync(kBarAux, kGroup);
      tile32(scr + bT22 * kBlk, kLd, 1, scr + bZ * kBlk, r0, n0, lane, z);
      float *t21 = scr + bA21 * kBlk;
      *reinterpret_cast<float2 *>(t21 + fr * kLd + fc) = make_float2(-z[0], -z[1]);
      *reinterpret_cast<float2 *>(t21 + (fr + 8) * kLd + fc) = make_float2(-z[2], -z[3]);
      bar_sync(kBarAux, kGroup);
      {
        // M = T diag(b) and -M diag(2^c): row t, columns 16c .. 16c + 15
        const int t = at >> 2, c = at & 3;
        float f[16];
        const bool upper = t < 32 && c >= 2;
        const float *src = scr + (t < 32 ? bT11 : (c < 2 ? bA21 : bT22)) * kBlk + (t & 31) * kLd +
                           16 * (c & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 v = *reinterpret_cast<const float4 *>(src + 4 * j);
          f[4 * j] = v.x;
          f[4 * j + 1] = v.y;
          f[4 * j + 2] = v.z;
          f[4 * j + 3] = v.w;
        }
        bar_sync(kBarAux, kGroup);  // the scratch has been read
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = upper ? 0.f : f[j] * beta_s[16 * c + j];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          unsigned char *d = sm + oM + w * 2 * kHalf;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              split2(f[8 * k + 2 * j], f[8 * k + 2 * j + 1], hi[j], lo[j]);
            const uint32_t o = swz(t, 2 * c + k);
            *reinterpret_cast<uint4 *>(d + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(d + kHalf + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] *= -eo[16 * c + j];
        }
      }
      fence_async_smem();
      mbar_arrive(bar + kReadyM);

      // -W^T rows n = 32 q + lane, steps 32 e .. 32 e + 31
      if (i > 0) sy.wait(kDoneU, (i - 1) & 1);  // W of the chunk before has been read
      sy.wait(kDoneW, i & 1);
      tc_fence_after();
      {
        uint32_t v[32];
        tmem_ld32(tl + kColW + 32 * e, v);
        tmem_wait_ld(v);
        unsigned char *d = sm + oW;
        const int n = 32 * q + lane;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            split2(__uint_as_float(v[8 * c + 2 * k]), __uint_as_float(v[8 * c + 2 * k + 1]), hi[k],
                   lo[k]);
          const uint32_t o = swz(n, 4 * e + c);
          *reinterpret_cast<uint4 *>(d + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4 *>(d + 2 * kHalf + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(bar + kReadyW);
      if (i > 0) output(i - 1);
    }
    if (nc > 0) output(nc - 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------ host side

bool al16(const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; }

// strides of a bf16 tensor (batch, steps, heads, width) that a tensor map
// takes: multiples of 16 bytes, and no broadcast dimension
bool map_strides(const int64_t (&s)[3], int64_t batch, int64_t L, int64_t heads) {
  const int64_t n[3] = {batch, L, heads};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] <= 0 || s[i] % 8 || s[i] >= (int64_t(1) << 39))) return false;
  return true;
}

// box {64, 1, C, 1}, 128-byte swizzle; channels and steps past the end read
// as zeros
bool encode(CUtensorMap *m, const void *ptr, int64_t width, int64_t heads, int64_t L,
            int64_t batch, const int64_t (&s)[3]) {
  auto enc = encoder();
  if (!enc) return false;
  const auto st = [](int64_t n, int64_t stride) {
    return static_cast<cuuint64_t>(n > 1 ? stride * 2 : 16);
  };
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(batch)};
  cuuint64_t strides[3] = {st(heads, s[2]), st(L, s[1]), st(batch, s[0])};
  cuuint32_t box[4] = {64, 1, C, 1}, estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

unsigned *delta_status_word() {
  unsigned *w = nullptr;
  return cudaGetSymbolAddress(reinterpret_cast<void **>(&w), g_delta_status) == cudaSuccess
             ? w
             : nullptr;
}

bool delta_chunk_applies(const DeltaParams &p, bool in_bf16) {
  return in_bf16 && p.N <= 128 && p.N % 8 == 0 && p.P % 8 == 0 && al16(p.q) && al16(p.k) &&
         al16(p.v) && al16(p.h0) && al16(p.last) && map_strides(p.sq, p.batch, p.L, p.G) &&
         map_strides(p.sk, p.batch, p.L, p.G) && map_strides(p.sv, p.batch, p.L, p.H);
}

cudaError_t launch_delta_chunk(const DeltaParams &p, bool out_bf16, cudaStream_t stream) {
  Maps maps;
  if (!encode(&maps.q, p.q, p.N, p.G, p.L, p.batch, p.sq) ||
      !encode(&maps.k, p.k, p.N, p.G, p.L, p.batch, p.sk) ||
      !encode(&maps.v, p.v, p.P, p.H, p.L, p.batch, p.sv))
    return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(p.seqs * p.H * ((p.P + 127) / 128));
  auto run = [&](auto kernel) {
    // per launch: the attribute belongs to the current device
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, kSmemBytes, stream>>>(maps, p);
    return cudaGetLastError();
  };
  return out_bf16 ? run(delta_chunk_kernel<__nv_bfloat16>) : run(delta_chunk_kernel<float>);
}

}  // namespace sss48
