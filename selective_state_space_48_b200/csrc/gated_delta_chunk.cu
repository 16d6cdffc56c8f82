// gated_delta_chunk.cu -- the gated delta rule in chunks of C = 64 steps on
// the sm_100a tensor cores.
//
// Inside a chunk, with c_t the running sum of log2 a, D[t,s] = 2^(c_t - c_s)
// for s <= t, and H the state (headdim x dstate) before the chunk, the
// written rows U solve
//
//   (I + A) U = diag(b) (V - diag(2^c) K H^T),
//   A[t,s] = b_t D[t,s] k_t.k_s  for s < t,
//
// and with T = (I + A)^-1 diag(b), which does not depend on H,
//
//   R^T = -(H K^T) diag(2^c)                                N = t
//   U^T = V^T T^T + R^T T^T                                 N = t, K = s
//   H  <- 2^(c_last) H + (U^T diag(2^(c_last - c))) K       N = dstate, K = s
//   Y^T = (H Q^T) diag(2^c) + U^T (Q K^T o D)^T             N = t
//
// Everything runs transposed, headdim (128 of it per block) on the lanes of
// tensor memory, so that H, R and U enter their products as the operand in
// tensor memory, straight from the registers of the thread that owns the row.
// (T diag(2^c) K as an operand instead of R would take one product less on
// the chain from chunk to chunk, but more in all, and the tensor cores were
// the limit of that form.)
//
// Precision.  q, k and v are bf16 and enter exactly.  H, R, T, U and
// Q K^T o D are fp32 values given as hi + lo, two bf16 values (off by 2^-18
// at most): a product with an exact operand takes two products, one of two
// such pairs three (lo lo is left out).  H itself stays in fp32 registers and
// is added to there, not in the tensor cores' accumulators.  Two of the pairs
// made nearly all of the final state's error, 3.6e-6 of its size (U' 2.6e-6, T
// 2.1e-6, H and R 2e-8 each): U' = U diag(2^(c_last - c)) therefore has a third
// piece, and so has the diagonal of T, which is b.  That leaves 6.0e-7 (5.4e-7
// with third pieces of T's 16 x 16 diagonal blocks, for 2 to 3 % of the time)
// and takes 1 to 2.5 %.  The pairs of the output (U, Q K^T o D) leave y 5e-6
// off, nothing beside a bf16 y's 2^-9; an fp32 y has third pieces of U and of
// the 16 x 16 diagonal blocks of Q K^T o D as well, and the product lo lo:
// 1.3e-6, for 3.5 %.  States that grow old bring H's and R's pairs to the fore:
// 2.6e-6 for decays about 0.999, where the step form is 1.3e-6 off.
// The sums c are pairs of fp32 values: a decay is the power of the difference
// of two of them, and one word alone, rounded to 2^-24 of its size, takes that
// from every decay behind a hard one (after a step of log2 a = -2300 outputs
// were off by 2e-4 up to the chunk's end, after one of -2.3e6 by 8 %).
//
// Roles (28 warps, one block per SM: the sequence, head and 128 rows):
//   warps 0, 3    TMA loads of the K, Q tiles (three stages); of V (one), and
//                 the stores of y
//   warp 1        issues every product, those that are not on the chain in the
//                 shadow of its other work
//   warp 2        the gates: running sums of log2 a and what follows from them
//   warps 4-19    the chain: H in registers (32 columns a thread), its pairs
//                 and those of R and U into tensor memory; the output of the
//                 chunk before, while products run
//   warps 20-27   what does not depend on H: A, its inverse T, Q K^T o D; two
//                 groups of four that take chunks in turn, since a chunk takes
//                 them longer than the chain takes for one
// The inverse: 16 x 16 triangles by substitution, a column per lane, then the
// blocks below them as products, -T22 (A21 T11), in fp32 (2 x 4 values of a
// thread; as three tf32 mma.sync products they made a chunk 2.2 us longer).
//
// Shared memory tiles are rows of 128 bytes with the 128-byte swizzle.  Every
// wait is bounded as in tcgen05.cuh, so no block can hang.
#include <cuda_bf16.h>

#include <type_traits>

#include "device_math.cuh"
#include "gated_delta.cuh"
#include "tcgen05.cuh"

namespace sss48 {
namespace {

constexpr int C = 64;                 // steps of a chunk
constexpr int kThreads = 896;
constexpr int kChainWarps = 16, kAuxWarps = 4;  // kAuxWarps of each group
constexpr int kAux = kAuxWarps * 32;
// named barriers of a group (+ its number): all of it; the A22 block handed on
constexpr int kBarAux = 1, kBarA22 = 3;

constexpr int kHalf = 64 * 128;       // 64 rows of 128 bytes
constexpr int kStageKQ = 4 * kHalf;   // K, Q of dstate 0..63, K, Q of 64..127
constexpr int kStageV = 2 * kHalf;
constexpr int oKQ = 0;
constexpr int oV = 3 * kStageKQ;
constexpr int oP = oV + kStageV;      // two of (Q K^T o D) hi, lo: [t][s]
constexpr int oT = oP + 4 * kHalf;    // two of T hi, lo: [t][s]
constexpr int oScr = oT + 4 * kHalf;  // scratch of the inverse, for each group
// 32 x 32 blocks, rows of 40 floats (8 rows start on 8 groups of banks): A,
// transposed, then T in the diagonal ones; A21 T11
constexpr int kLd = 40, kBlk = 32 * kLd;
constexpr int bA11 = 0, bA22 = 1, bA21 = 2, bZ = 3, kScr = 4 * kBlk;
constexpr int oGate = oScr + 2 * kScr * 4;  // two of (b, -c hi, -c lo) [C]
constexpr int kGate = 3 * C * 4;
constexpr int oDecay = oGate + 2 * kGate;  // three of (2^(c_last - c), 2^c, scale 2^c) [C]
constexpr int kDecay = 3 * C * 4;
constexpr int oBar = oDecay + 3 * kDecay;
constexpr int kBars = 37;
constexpr int oTmemSlot = oBar + kBars * 8;
constexpr int oAbort = oTmemSlot + 4;
constexpr int oSeq = oAbort + 4;
constexpr int kSmemBytes = oSeq + 4;
static_assert(kSmemBytes <= 232448, "shared memory above the per-block limit");
static_assert(oGate % 16 == 0 && kGate % 16 == 0 && oDecay % 16 == 0, "16-byte vectors");

// tensor memory columns (all 512 are allocated, so they start at 0)
constexpr uint32_t kColH = 0;     // H pairs / the update U'^T K (128)
constexpr uint32_t kColX = 128;   // H K^T, then the pairs of R, then those of
                                  // U' = U diag(2^(c_last - c))
constexpr uint32_t kColU = 192;   // U, then its pairs
constexpr uint32_t kColO1 = 256;  // two; third pieces of U', U in the one not in use
constexpr uint32_t kColO2 = 384;
constexpr uint32_t kColS = 448;   // K K^T (lanes 0..63), Q K^T (64..127)
constexpr uint32_t kTmemCols = 512;

// Barriers.  Tiles landed and released; per chunk, products done (S, X, U, O1,
// the update, O) and operands ready (H; R; U'; U; T and P), S and O drained; y
// staged (two: nothing but time keeps the chain from staging a chunk's y before
// the warp that stores it has looked for the one before); the two P buffers
// released; the gates written (the decays have three
// buffers, the rest two) and their two and three buffers released; every
// product done.  A waiter may not fall two phases behind: where it could, the
// barriers are a ring.  The groups arrive one lane per warp.  (H, R and U' in
// four parts, so that a product starts with the first of them, cost more in
// waits than they gained: 618 us against 482 for 8192 steps.)
constexpr int kFullKQ = 0, kFullV = 3, kEmptyKQ = 5, kEmptyV = 8, kDoneS = 9, kDoneX = 11,
              kDoneU = 12, kDoneO1 = 13, kDoneH = 14, kDoneO = 15, kReadyH = 16, kReadyR = 17,
              kReadyU = 18, kReadyO = 19, kFreeO = 20, kReadyY = 21, kFreeS = 23, kReadyT = 24,
              kFreeP = 26, kReadyG = 28, kFreeG = 31, kFreeD = 33,
              kEnd = 36;
// arrivals that complete a barrier's phase
__device__ __forceinline__ int bar_count(int i) {
  if (i == kFreeS || i == kReadyT || i == kReadyT + 1 || i == kFreeG || i == kFreeG + 1)
    return kAuxWarps;
  if ((i >= kReadyH && i <= kReadyY + 1) || (i >= kFreeD && i < kEnd)) return kChainWarps;
  return 1;
}

// Bounded waits, short since every one is inlined: instructions from beyond
// the instruction caches bound this kernel where every SM runs it (108 KB of
// code took twice the time; 8 x 2048 steps with the products unrolled 292 us,
// with them in loops, 7 KB less, 275, though alone on its SMs the longer form is
// 2 % faster).  It is 81 KB.  A try suspends the thread for up to 4.0 us
// (measured: hints of 1 ns to 1 ms gave the same), and a wait gives up after
// `limit` of them (read off the clock instead, the limit made the kernel 2 to 3
// % slower by its size).  Then, and once any wait of the block has given up,
// every wait that is not complete returns after one try (the results are
// garbage, but nothing hangs: products run on whatever their operands hold),
// and the block's end records the timeout.
constexpr uint32_t kTryNs = 4000;
constexpr uint32_t kDrainTries = 2000000000u / kTryNs;  // 2 s
struct Waits {
  uint32_t bar;  // shared-memory address of the barriers
  volatile int *abort;
  uint32_t limit;
  __device__ __forceinline__ bool try_wait(int i, uint32_t parity) const {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar + 8 * i), "r"(parity), "r"(kTryNs)
        : "memory");
    return ok != 0;
  }
  // Whether the phase is complete, without waiting.
  __device__ __forceinline__ bool test(int i, uint32_t parity) const {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar + 8 * i), "r"(parity)
        : "memory");
    return ok != 0;
  }
  // (every lane tries: about 110 cycles for a phase that is complete, 250 and
  // more for one lane and a __syncwarp)
  __device__ __forceinline__ void wait(int i, uint32_t parity) const {
    if (__builtin_expect(try_wait(i, parity), 1)) return;
    uint32_t n = 0;
    do {
      if (*abort) break;
      if (++n >= limit) *abort = 1;
    } while (!try_wait(i, parity));
  }
  // for copies and products still in flight at the end, which no block may
  // leave behind: neither cut short by another wait's timeout nor by a caller's
  // short limit
  __device__ __forceinline__ void drain(int i, uint32_t parity) const {
    uint32_t n = 0;
#pragma unroll 1
    while (!try_wait(i, parity))
      if (++n >= kDrainTries) {
        *abort = 1;
        break;
      }
  }
};

struct Maps {
  CUtensorMap q, k, v, y;
};

// A step's log2 decay is taken as at least this: two to it times any fp32 value
// is 0, and 64 of them leave the pairs of the sums exact to 2^-30.  (As a
// comparison that lets NaN pass.)
constexpr float kLeastLog2 = -300.f;

// s = a + b; returned: what that rounded off
__device__ __forceinline__ float two_sum(float a, float b, float &s) {
  s = a + b;
  const float t = s - a;
  return (a - (s - t)) + (b - t);
}

__device__ unsigned g_delta_status;

// what a pair of bf16 values leaves of two fp32 ones (exact)
__device__ __forceinline__ float2 left2(float a, float b, uint32_t p) {
  float2 r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n fma.rn.f32.bf16 %0, l, %5, %3;\n"
      " fma.rn.f32.bf16 %1, h, %5, %4;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "r"(p), "f"(a), "f"(b), "h"(static_cast<unsigned short>(0xbf80)));
  return r;
}
// x = hi + lo for a pair of values, packed two to a register
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(a, b);
  const float2 r = left2(a, b, hi);
  lo = pack_bf16(r.x, r.y);
}
// ... and what that leaves, as a third
__device__ __forceinline__ uint32_t third2(float a, float b, uint32_t hi, uint32_t lo) {
  float2 r = left2(a, b, hi);
  r = left2(r.x, r.y, lo);
  return pack_bf16(r.x, r.y);
}
__device__ __forceinline__ uint4 third8(const float *f, uint4 hi, uint4 lo) {
  return make_uint4(third2(f[0], f[1], hi.x, lo.x), third2(f[2], f[3], hi.y, lo.y),
                    third2(f[4], f[5], hi.z, lo.z), third2(f[6], f[7], hi.w, lo.w));
}
__device__ __forceinline__ void split8(const float *f, uint4 &hi, uint4 &lo) {
  split2(f[0], f[1], hi.x, lo.x);
  split2(f[2], f[3], hi.y, lo.y);
  split2(f[4], f[5], hi.z, lo.z);
  split2(f[6], f[7], hi.w, lo.w);
}

// 16 columns of this thread's lane (and 16 more from `b`), waited for: with
// the wait in the same statement the registers are free to be any
__device__ __forceinline__ void tmem_get16(uint32_t a, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_get16x2(uint32_t a, uint32_t b, float (&v)[16],
                                             float (&w)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]), "=f"(w[6]), "=f"(w[7]), "=f"(w[8]), "=f"(w[9]), "=f"(w[10]), "=f"(w[11]), "=f"(w[12]), "=f"(w[13]), "=f"(w[14]), "=f"(w[15])
      : "r"(a), "r"(b)
      : "memory");
}

// 4 columns of this thread's lane
__device__ __forceinline__ void tmem_st4(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// one arrival for the warp, after all its lanes' writes
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// The products are issued by one lane (`go`: elect_one's), but the whole warp
// runs the issuing code, so that descriptors stay in uniform registers: 35
// cycles a product of 128 x 64 x 16 with an operand in tensor memory, 52 with
// both in shared memory; from a branch of one lane it was 50 and 52, with a
// lane index for the predicate 65.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r));
  return r;
}
// A descriptor is given as its low word (address, leading offset); the high
// word is the same for all: rows of 8 groups 1024 bytes apart, version 1,
// 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFF) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t acc, uint32_t go) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n"
      " setp.ne.b32 q, %5, 0;\n mov.b64 da, {%1, %6};\n mov.b64 db, {%2, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(go), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t acc, uint32_t go) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n"
      " setp.ne.b32 q, %5, 0;\n mov.b64 db, {%2, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(go), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar, uint32_t go) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_addr(bar)),
      "r"(go)
      : "memory");
}

// z += x y for two rows of four columns
__device__ __forceinline__ void fma24(float2 (&z)[2][2], float x0, float x1, float4 y) {
  z[0][0] = __ffma2_rn(make_float2(x0, x0), make_float2(y.x, y.y), z[0][0]);
  z[0][1] = __ffma2_rn(make_float2(x0, x0), make_float2(y.z, y.w), z[0][1]);
  z[1][0] = __ffma2_rn(make_float2(x1, x1), make_float2(y.x, y.y), z[1][0]);
  z[1][1] = __ffma2_rn(make_float2(x1, x1), make_float2(y.z, y.w), z[1][1]);
}
// Rows r, r + 1, columns c .. c + 3 of X Y, DEPTH deep: X given transposed (x
// points to its row r of values r, y to columns c), ...
template <int DEPTH>
__device__ __forceinline__ void prod_t(const float *x, const float *y, float2 (&z)[2][2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i >> 1][i & 1] = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < DEPTH; ++k) {
    const float2 v = *reinterpret_cast<const float2 *>(x + k * kLd);
    fma24(z, v.x, v.y, *reinterpret_cast<const float4 *>(y + k * kLd));
  }
}
// ... or as it is (x points to its row r)
template <int DEPTH>
__device__ __forceinline__ void prod_n(const float *x, const float *y, float2 (&z)[2][2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i >> 1][i & 1] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < DEPTH; k += 4) {
    const float4 v = *reinterpret_cast<const float4 *>(x + k);
    const float4 w = *reinterpret_cast<const float4 *>(x + kLd + k);
    fma24(z, v.x, w.x, *reinterpret_cast<const float4 *>(y + k * kLd));
    fma24(z, v.y, w.y, *reinterpret_cast<const float4 *>(y + (k + 1) * kLd));
    fma24(z, v.z, w.z, *reinterpret_cast<const float4 *>(y + (k + 2) * kLd));
    fma24(z, v.w, w.w, *reinterpret_cast<const float4 *>(y + (k + 3) * kLd));
  }
}
__device__ __forceinline__ void store24(float *d, const float2 (&z)[2][2], float sign) {
  *reinterpret_cast<float4 *>(d) =
      make_float4(sign * z[0][0].x, sign * z[0][0].y, sign * z[0][1].x, sign * z[0][1].y);
  *reinterpret_cast<float4 *>(d + kLd) =
      make_float4(sign * z[1][0].x, sign * z[1][0].y, sign * z[1][1].x, sign * z[1][1].y);
}

// (I + A)^-1 of a 32 x 32 block in place, by one warp; `a` holds A transposed
// on entry.  Two 16 x 16 triangles at once: lane j of a half has column j, and
// x_s is final once the steps before it have been taken out of it; then
// T21 = -T22 (A21 T11), with A21 in the upper right 16 x 16 of `a`, and its
// products in the lower left.
__device__ __forceinline__ void invert32(float *a, int lane) {
  const int off = (lane >> 4) * (16 * kLd + 16), j = lane & 15;
  float2 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = make_float2(j == 2 * i ? 1.f : 0.f, j == 2 * i + 1 ? 1.f : 0.f);
#pragma unroll
  for (int s = 0; s < 16; ++s) {
    const float xs = s & 1 ? x[s >> 1].y : x[s >> 1].x;
    const float2 m = make_float2(-xs, -xs);
    float4 v[4];
#pragma unroll
    for (int i = (s + 1) >> 2; i < 4; ++i)
      v[i] = *reinterpret_cast<const float4 *>(a + off + s * kLd + 4 * i);
    __syncwarp();  // the row has been read: x_s takes its place
    a[off + s * kLd + j] = xs;
#pragma unroll
    for (int i = (s + 1) >> 2; i < 4; ++i) {
      // A is zero on and above the diagonal: the pair that holds row s keeps it
      x[2 * i] = __ffma2_rn(make_float2(v[i].x, v[i].y), m, x[2 * i]);
      x[2 * i + 1] = __ffma2_rn(make_float2(v[i].z, v[i].w), m, x[2 * i + 1]);
    }
  }
  __syncwarp();
  const int r = 2 * (lane >> 2), c = 4 * (lane & 3);
  float2 z[2][2];
  prod_t<16>(a + 16 + r, a + c, z);
  store24(a + (16 + r) * kLd + c, z, 1.f);
  __syncwarp();
  prod_n<16>(a + (16 + r) * kLd + 16, a + 16 * kLd + c, z);
#pragma unroll
  for (int i = 0; i < 2; ++i)  // above the diagonal T is zero
    *reinterpret_cast<float4 *>(a + (lane >> 1) * kLd + 16 + 8 * (lane & 1) + 4 * i) =
        make_float4(0.f, 0.f, 0.f, 0.f);
  __syncwarp();
  store24(a + (16 + r) * kLd + c, z, -1.f);
}

constexpr uint32_t kIdKK = idesc_bf16(128, 64, 0, 0);  // both operands K-major
constexpr uint32_t kIdTK = idesc_bf16(128, 64, 1, 0);  // the first as stored by step
constexpr uint32_t kLoTile = kHalf >> 4;               // hi -> lo of T and P
// T and P are lower triangular: slice k (s = 16 k ..) meets the rows and output
// columns t from 16 k on, so that far into the tile and N that much smaller.
constexpr uint32_t kTriN = 2u << 17;
__device__ __forceinline__ constexpr uint32_t tri(int k) { return static_cast<uint32_t>(k * 130); }
// Third pieces of their 16 x 16 diagonal blocks lie in the hi tile above the
// diagonal: block k in rows 16 (k / 2) .., columns 32 + 16 (k % 2) ..
// (of T's only the diagonal is not 0)
constexpr uint32_t kId16KK = idesc_bf16(128, 16, 0, 0), kId16TK = idesc_bf16(128, 16, 1, 0);
__device__ __forceinline__ constexpr uint32_t diag3(int k) {
  return static_cast<uint32_t>((k >> 1) * 128 + 4 + 2 * (k & 1));
}
// slice k of a K-major tile whose 64-wide halves lie 2 kHalf apart
__device__ __forceinline__ constexpr uint32_t kslice(int k) {
  return static_cast<uint32_t>((k >> 2) * (2 * kHalf >> 4) + (k & 3) * 2);
}

// NK: 16-wide slices of dstate (4 up to 64, else 8; TMA pads with zeros).
// y_tma: whole chunks of y go out through their Q tile and a TMA store (bf16
// rows that a tensor map takes): 16 two-byte stores of a thread straight to
// memory took 1.3 us of a chunk's 4.5.
// VEC: states in rows of 16-byte vectors.
template <typename OutT, int NK, bool VEC>
__global__ void __launch_bounds__(kThreads, 1)
    delta_chunk_kernel(const __grid_constant__ Maps maps, const DeltaParams p, const int y_tma) {
  constexpr uint32_t idH = idesc_bf16(128, 16 * NK, 0, 1);  // the second as stored by step
  // an fp32 output: its products with third pieces too
  constexpr bool kWide = sizeof(OutT) == 4;
  // the swizzle needs 1024-byte tiles; a block without static shared memory
  // has its dynamic memory on such a boundary
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t sbase = smem_addr(sm);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler

  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + oBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + oTmemSlot);
  volatile int *abort = reinterpret_cast<volatile int *>(sm + oAbort);
  const uint64_t tries = p.spin_ns / kTryNs + 1;
  const Waits sy{smem_addr(bar), abort,
                 tries < 0xffffffffull ? static_cast<uint32_t>(tries) : 0xffffffffu};

  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bar + i, bar_count(i));
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  // the sequence, head and 128 rows; of a cut sequence the segment, and in its
  // first pass whether this block takes the transition's rows (`move`)
  int slices = static_cast<int>((p.P + 127) / 128), seg = 0;
  int64_t task = blockIdx.x;
  bool move = false;
  if (p.segs) {
    const int64_t heads = p.seqs * p.H, of_rows = (p.segs - 1) * heads * slices;
    move = task >= of_rows;
    if (move) {
      task -= of_rows;
      slices = 1;
    }
    seg = static_cast<int>(task / (heads * slices));
    task -= seg * heads * slices;
    if (move || p.pass == 2) ++seg;
  }
  const int64_t sh = task / slices;
  const int p0 = static_cast<int>(task - sh * slices) * 128;
  int64_t seq = sh / p.H;
  const int h = static_cast<int>(sh - seq * p.H);
  const int N = static_cast<int>(p.N), P = static_cast<int>(move ? p.N : p.P);
  const bool write_y = p.pass != 1 || seg == 0;
  if (move) {  // no values
    for (int k = tid; k < kStageV / 16; k += kThreads)
      *reinterpret_cast<uint4 *>(sm + oV + 16 * k) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
  }
  // Packed sequences are taken longest first (the n-th of the grid is the n-th
  // longest): a long one that starts among the last runs on alone.  24 of 0 to
  // 1362 steps: 222 us, 263 in their own order.
  const bool ranked = p.cu && p.seqs <= kThreads;
  int *len = reinterpret_cast<int *>(sm + oScr), *slot = reinterpret_cast<int *>(sm + oSeq);
  if (ranked && tid < p.seqs) {
    int64_t none, lo, hi;
    delta_span(p, tid, none, lo, hi);
    len[tid] = static_cast<int>(hi - lo);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (ranked) {
    if (tid < p.seqs) {
      const int mine = len[tid], n = static_cast<int>(p.seqs);
      int before = 0;
      for (int k = 0; k < n; ++k) before += len[k] > mine || (len[k] == mine && k < tid);
      if (before == seq) *slot = tid;
    }
    __syncthreads();
    seq = __shfl_sync(0xffffffffu, *slot, 0);
  }
  // (an allocation of every column starts at 0; the addresses below rely on it)
  if (*tmem_slot != 0) *abort = 1;

  const int g = h / static_cast<int>(p.H / p.G);
  int64_t b64, t0, t1;
  delta_span(p, seq, b64, t0, t1);
  const float *h0 = p.h0;
  float *last = p.last;
  if (p.segs) {
    const int64_t states = p.seqs * p.H * p.P * p.N, len = static_cast<int64_t>(p.seg_chunks) * C;
    t0 = seg * len;
    t1 = t1 - t0 > len ? t0 + len : t1;
    if (p.pass == 2) {
      h0 = p.ends + (seg - 1) * states;
      if (seg < p.segs - 1) last = nullptr;
    } else {
      if (seg > 0) h0 = nullptr;
      last = move ? p.moves + (seg - 1) * p.seqs * p.H * p.N * p.N : p.ends + seg * states;
    }
  }
  const int b = static_cast<int>(b64);
  const int total = static_cast<int>(t1 - t0);
  const int nc = __shfl_sync(0xffffffffu, (total + C - 1) / C, 0);

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      int i = 0;
      for (; i < nc; ++i) {
        const int t = static_cast<int>(t0) + i * C;
        const int a = i % 3;
        if (i >= 3) sy.wait(kEmptyKQ + a, (i / 3 - 1) & 1);
        if (*abort) break;  // (the waits are no order any more)
        unsigned char *d = sm + oKQ + a * kStageKQ;
        mbar_expect_tx(bar + kFullKQ + a, kStageKQ);
        tma_load_4d(d, &maps.k, 0, g, t, b, bar + kFullKQ + a);
        tma_load_4d(d + kHalf, &maps.q, 0, g, t, b, bar + kFullKQ + a);
        tma_load_4d(d + 2 * kHalf, &maps.k, 64, g, t, b, bar + kFullKQ + a);
        tma_load_4d(d + 3 * kHalf, &maps.q, 64, g, t, b, bar + kFullKQ + a);
      }
      // no copy may still be landing when the block exits
      for (int j = i > 3 ? i - 3 : 0; j < i; ++j) sy.drain(kFullKQ + j % 3, (j / 3) & 1);
    }
    __syncwarp();
  } else if (warp == 3) {
    // (V waits for its one place, while K and Q run ahead)
    if (lane == 0) {
      int i = 0;  // V of chunk i, y of the one before
      for (; i <= nc; ++i) {
        if (i > 0) sy.wait(kEmptyV, (i - 1) & 1);
        if (*abort) break;
        if (i < nc && move) {
          mbar_arrive(bar + kFullV + (i & 1));
        } else if (i < nc) {
          const int t = static_cast<int>(t0) + i * C;
          uint64_t *full = bar + kFullV + (i & 1);
          mbar_expect_tx(full, kStageV);
          tma_load_4d(sm + oV, &maps.v, p0, h, t, b, full);
          tma_load_4d(sm + oV + kHalf, &maps.v, p0 + 64, h, t, b, full);
        }
        if (i == 0 || !y_tma || i * C > total) continue;
        // y of chunk i - 1, a whole one, staged in its Q tile; then the stage
        // is free
        sy.wait(kReadyY + ((i - 1) & 1), ((i - 1) / 2) & 1);
        const int t = static_cast<int>(t0) + (i - 1) * C, a = (i - 1) % 3;
        const unsigned char *y = sm + oKQ + a * kStageKQ + kHalf;
        if (write_y && !*abort) {
          tma_store_4d(&maps.y, y, p0, h, t, b);
          if (p0 + 64 < P) tma_store_4d(&maps.y, y + 2 * kHalf, p0 + 64, h, t, b);
        }
        tma_store_wait_read();
        mbar_arrive(bar + kEmptyKQ + a);
      }
      const int loads = min(i, nc);
      for (int j = loads > 2 ? loads - 2 : 0; j < loads; ++j)
        sy.drain(kFullV + (j & 1), (j / 2) & 1);
      tma_store_wait_all();
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------- tensor-core issue
    const uint32_t on = elect_one();
    auto ready = [&](int i, uint32_t parity) {
      return __shfl_sync(0xffffffffu, sy.test(i, parity), 0) != 0;
    };
    int ns = 0, sst = 0;  // the next chunk whose S = [K; Q] K^T is due, ns % 3
    auto issue_scores = [&]() {
      tc_fence_after();
      const uint32_t d = desc_lo(sbase + oKQ + sst * kStageKQ, 16);
#pragma unroll 1
      for (int k = 0; k < NK; ++k) mma_ss(kColS, d + kslice(k), d + kslice(k), kIdKK, k > 0, on);
      mma_commit(bar + kDoneS + (ns & 1), on);
      ++ns;
      sst = sst == 2 ? 0 : sst + 1;
    };
    // S as early as its tiles and its place allow, without waiting
    auto try_scores = [&]() {
      if (ns < nc && (ns == 0 || ready(kFreeS, (ns - 1) & 1)) && ready(kFullKQ + sst, (ns / 3) & 1))
        issue_scores();
    };
    int st = 0;  // i % 3
    for (int i = 0; i < nc; ++i, st = st == 2 ? 0 : st + 1) {
      const uint32_t kq = sbase + oKQ + st * kStageKQ;
      while (ns <= i) {
        if (ns > 0) sy.wait(kFreeS, (ns - 1) & 1);
        sy.wait(kFullKQ + sst, (ns / 3) & 1);
        issue_scores();
      }
      sy.wait(kReadyH, i & 1);
      tc_fence_after();
      {  // X = H K^T
        const uint32_t dK = desc_lo(kq, 16);
#pragma unroll 2  // (rolled: what the instruction caches hold, see the waits)
        for (int k = 0; k < NK; ++k) {
          const uint32_t hi = kColH + (k >> 1) * 32 + (k & 1) * 8;
          mma_ts(kColX, hi, dK + kslice(k), kIdKK, k > 0, on);
          mma_ts(kColX, hi + 16, dK + kslice(k), kIdKK, 1, on);
        }
      }
      mma_commit(bar + kDoneX, on);
      // T of this chunk may hang on the S of the next having been issued
      for (uint32_t n = 0; !ready(kReadyT + (i & 1), (i / 2) & 1); ++n) {
        if (ns == nc || n == 1000) {
          sy.wait(kReadyT + (i & 1), (i / 2) & 1);
          break;
        }
        try_scores();
      }
      const uint32_t dT = desc_lo(sbase + oT + (i & 1) * 2 * kHalf, 16);
      sy.wait(kFullV + (i & 1), (i / 2) & 1);
      if (i > 0) sy.wait(kDoneO, (i - 1) & 1);  // U of the chunk before has been read
      tc_fence_after();
      {  // U^T = V^T T^T
        const uint32_t dV = desc_lo(sbase + oV, kHalf);
#pragma unroll 2
        for (int k = 0; k < 4; ++k) {
          const uint32_t d = kColU + 16 * k, id = kIdTK - k * kTriN;
          mma_ss(d, dV + k * 128, dT + tri(k), id, k > 0, on);
          mma_ss(d, dV + k * 128, dT + kLoTile + tri(k), id, 1, on);
          mma_ss(d, dV + k * 128, dT + diag3(k), kId16TK, 1, on);
        }
      }
      mma_commit(bar + kEmptyV, on);
      sy.wait(kReadyR, i & 1);
      tc_fence_after();
      {  // U^T += R^T T^T
#pragma unroll 2
        for (int k = 0; k < 4; ++k) {
          const uint32_t d = kColU + 16 * k, id = kIdKK - k * kTriN;
          mma_ts(d, kColX + 16 * k, dT + tri(k), id, 1, on);
          mma_ts(d, kColX + 16 * k + 8, dT + tri(k), id, 1, on);
          mma_ts(d, kColX + 16 * k, dT + kLoTile + tri(k), id, 1, on);
        }
      }
      mma_commit(bar + kDoneU, on);
      {  // O1 = H Q^T
        const uint32_t dQ = desc_lo(kq + kHalf, 16), o1 = kColO1 + (i & 1) * 64;
#pragma unroll 2
        for (int k = 0; k < NK; ++k) {
          const uint32_t hi = kColH + (k >> 1) * 32 + (k & 1) * 8;
          mma_ts(o1, hi, dQ + kslice(k), kIdKK, k > 0, on);
          mma_ts(o1, hi + 16, dQ + kslice(k), kIdKK, 1, on);
        }
      }
      mma_commit(bar + kDoneO1, on);
      try_scores();
      sy.wait(kDoneO1, i & 1);  // the update overwrites the pairs of H
      sy.wait(kReadyU, i & 1);
      tc_fence_after();
      const uint32_t col3 = kColO1 + (~i & 1) * 64;  // third pieces of U', U
      {  // U'^T K
        const uint32_t dK = desc_lo(kq, 2 * kHalf);
#pragma unroll 2
        for (int k = 0; k < 4; ++k) {
          mma_ts(kColH, kColX + 16 * k, dK + k * 128, idH, k > 0, on);
          mma_ts(kColH, kColX + 16 * k + 8, dK + k * 128, idH, 1, on);
        }
#pragma unroll 2
        for (int k = 0; k < 4; ++k) mma_ts(kColH, col3 + 16 * k, dK + k * 128, idH, 1, on);
      }
      mma_commit(bar + kDoneH, on);
      if (!y_tma) mma_commit(bar + kEmptyKQ + st, on);
      if (i > 0) sy.wait(kFreeO, (i - 1) & 1);
      sy.wait(kReadyO, i & 1);
      tc_fence_after();
      {  // O2 = U^T (Q K^T o D)^T
        const uint32_t dP = desc_lo(sbase + oP + (i & 1) * 2 * kHalf, 16);
#pragma unroll 2
        for (int k = 0; k < 4; ++k) {
          const uint32_t d = kColO2 + 16 * k, u = kColU + 16 * k, id = kIdKK - k * kTriN;
          mma_ts(d, u, dP + tri(k), id, k > 0, on);
          mma_ts(d, u + 8, dP + tri(k), id, 1, on);
          mma_ts(d, u, dP + kLoTile + tri(k), id, 1, on);
          if constexpr (kWide) {
            mma_ts(d, u + 8, dP + kLoTile + tri(k), id, 1, on);
            mma_ts(d, col3 + 16 * k + 8, dP + tri(k), id, 1, on);
            mma_ts(d, u, dP + diag3(k), kId16KK, 1, on);
          }
        }
      }
      mma_commit(bar + kDoneO, on);
      mma_commit(bar + kFreeP + (i & 1), on);
      try_scores();
    }
    // every product done before the tensor memory is freed, and every commit
    // arrived, those too that nobody waits for: an arrival at the shared
    // memory of a block that has ended is an illegal access
    if (nc > 0) {
      // (after a timeout the waits above were no order any more: this one,
      // used once, is behind everything)
      mma_commit(bar + kEnd, on);
      sy.drain(kEnd, 0);
      sy.drain(kDoneO, (nc - 1) & 1);
      sy.drain(kEmptyV, (nc - 1) & 1);
      for (int i = y_tma ? nc : (nc > 3 ? nc - 3 : 0); i < nc; ++i)
        sy.drain(kEmptyKQ + i % 3, (i / 3) & 1);
      for (int i = nc > 2 ? nc - 2 : 0; i < nc; ++i) sy.drain(kFreeP + (i & 1), (i / 2) & 1);
    }
  } else if (warp == 2) {
    // --------------------------------------------------------- the gates
    const __nv_bfloat16 *dtp = static_cast<const __nv_bfloat16 *>(p.dt) + b * p.sdt[0] + h * p.sdt[2];
    const __nv_bfloat16 *bp =
        static_cast<const __nv_bfloat16 *>(p.beta) + b * p.sbeta[0] + h * p.sbeta[2];
    const float A2 = p.A[h] * kLog2e, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    // raw values of two steps of a lane, a chunk ahead
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
    if (nc > 0) raw(0);
    for (int i = 0; i < nc; ++i) {
      const int left = total - i * C;
      float g2[2], lo[2], bt[2];  // g2 + lo: the running sums
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        g2[k] = lo[k] = bt[k] = 0.f;
        if (32 * k + lane < left)
          delta_gates<__nv_bfloat16>(p, __uint_as_float(static_cast<uint32_t>(rd[k]) << 16),
                                     __uint_as_float(static_cast<uint32_t>(rb[k]) << 16), A2, bias,
                                     g2[k], bt[k]);
        if (g2[k] < kLeastLog2) g2[k] = kLeastLog2;
      }
      raw(i + 1);
      auto add = [&](int k, float hi_before, float lo_before) {
        const float r = two_sum(hi_before, g2[k], g2[k]);
        lo[k] += lo_before + r;
      };
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = __shfl_up_sync(0xffffffffu, g2[k], o);
          const float xl = __shfl_up_sync(0xffffffffu, lo[k], o);
          if (lane >= o) add(k, x, xl);
        }
      }
      add(1, __shfl_sync(0xffffffffu, g2[0], 31), __shfl_sync(0xffffffffu, lo[0], 31));
      const float end1 = __shfl_sync(0xffffffffu, g2[1], 31);
      const float end1l = __shfl_sync(0xffffffffu, lo[1], 31);
      if (i >= 2) sy.wait(kFreeG + (i & 1), (i / 2 - 1) & 1);
      if (i >= 3) sy.wait(kFreeD + i % 3, (i / 3 - 1) & 1);
      float *beta_s = reinterpret_cast<float *>(sm + oGate + (i & 1) * kGate), *neg_s = beta_s + C;
      float *du = reinterpret_cast<float *>(sm + oDecay + (i % 3) * kDecay);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = 32 * k + lane;
        const float eo = ex2_mufu(g2[k] + lo[k]);
        neg_s[t] = -g2[k];
        neg_s[C + t] = -lo[k];
        beta_s[t] = bt[k];
        du[t] = ex2_mufu((end1 - g2[k]) + (end1l - lo[k]));
        du[C + t] = eo;
        du[2 * C + t] = p.scale * eo;
      }
      warp_arrive(bar + kReadyG + i % 3, lane);
    }
  } else if (warp >= 4 && warp < 20) {
    // -------------------------------------------------------- the chain
    const int q = warp & 3, e = (warp - 4) >> 2;
    const int row = p0 + 32 * q + lane;
    const uint32_t tl = static_cast<uint32_t>(32 * q) << 16;
    const int64_t base = ((seq * p.H + h) * P + row) * p.N + 32 * e;
    OutT *yp = static_cast<OutT *>(p.y) + b * p.sy[0] + h * p.sy[2] + t0 * p.sy[1] + row;
    float H[32];
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (h0 && row < P && 32 * e + j < N) {
        if constexpr (VEC) {
          v = __ldcs(reinterpret_cast<const float4 *>(h0 + base + j));
        } else {
          float *f = reinterpret_cast<float *>(&v);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (32 * e + j + k < N) f[k] = h0[base + j + k];
        }
      }
      H[j] = v.x;
      H[j + 1] = v.y;
      H[j + 2] = v.z;
      H[j + 3] = v.w;
    }
    if (move) {  // the transition: where the unit rows go
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (32 * e + j == row) H[j] = 1.f;
    }
    float gam = 1.0f;
    // H <- 2^(c_last) H + U'^T K of chunk i
    auto update = [&](int i) {
      sy.wait(kDoneH, i & 1);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v[16];
        tmem_get16(tl + kColH + 32 * e + 16 * c, v);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 n = __ffma2_rn(make_float2(gam, gam),
                                      make_float2(H[16 * c + j], H[16 * c + j + 1]),
                                      make_float2(v[j], v[j + 1]));
          H[16 * c + j] = n.x;
          H[16 * c + j + 1] = n.y;
        }
      }
    };
    // column `row` of a 64-step tile in two halves of 64 columns: 16-byte
    // chunk (row % 64) / 8 of a step's 128 bytes, swizzled by the step
    const uint32_t ycol = (q >> 1) * 2 * kHalf + 2048 * e + (((32 * q + lane) & 63) << 1);
    // y rows of chunk i, 16 steps of a thread: scale 2^c O1 + O2 (P holds the
    // scale of O2)
    auto output = [&](int i) {
      sy.wait(kDoneO, i & 1);
      tc_fence_after();
      const float *eo =
          reinterpret_cast<const float *>(sm + oDecay + (i % 3) * kDecay) + 2 * C + 16 * e;
      float v[16], o[16];
      tmem_get16x2(tl + kColO1 + (i & 1) * 64 + 16 * e, tl + kColO2 + 16 * e, v, o);
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(eo + j);
        o[j] = fmaf(x.x, v[j], o[j]);
        o[j + 1] = fmaf(x.y, v[j + 1], o[j + 1]);
        o[j + 2] = fmaf(x.z, v[j + 2], o[j + 2]);
        o[j + 3] = fmaf(x.w, v[j + 3], o[j + 3]);
      }
      tc_fence_before();
      warp_arrive(bar + kFreeO, lane);
      if (lane == 0) mbar_arrive(bar + kFreeD + i % 3);
      const int left = total - i * C - 16 * e;
      if (y_tma && (i + 1) * C <= total) {
        if constexpr (sizeof(OutT) == 2) {
          unsigned char *d = sm + oKQ + (i % 3) * kStageKQ + kHalf;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            *reinterpret_cast<OutT *>(d + (ycol ^ ((j & 7) << 4)) + j * 128) = from_f32<OutT>(o[j]);
          fence_async_smem();
        }
        warp_arrive(bar + kReadyY + (i & 1), lane);
      } else if (write_y && row < P) {
        OutT *yr = yp + static_cast<int64_t>(i * C + 16 * e) * p.sy[1];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j < left) yr[j * p.sy[1]] = from_f32<OutT>(o[j]);
      }
    };
    for (int i = 0;; ++i) {
      if (i > 0) update(i - 1);
      if (i < nc) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            split2(H[16 * c + 2 * j], H[16 * c + 2 * j + 1], hi[j], lo[j]);
          tmem_st8(tl + kColH + 32 * e + 8 * c, hi);
          tmem_st8(tl + kColH + 32 * e + 16 + 8 * c, lo);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar + kReadyH, lane);
        sy.wait(kReadyG + i % 3, (i / 3) & 1);
      }
      if (i > 0) output(i - 1);
      if (i >= nc) break;

      const float *du = reinterpret_cast<const float *>(sm + oDecay + (i % 3) * kDecay);
      sy.wait(kDoneX, i & 1);
      tc_fence_after();
      {
        // R = -2^c x, 16 steps of a thread, its pairs in the columns that x
        // came from; nothing of the steps behind the sequence
        float x[16];
        uint32_t hi[8], lo[8];
        const int left = total - i * C - 16 * e;
        const float *ec = du + C + 16 * e;
        tmem_get16(tl + kColX + 16 * e, x);
        if (left < 16) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j >= left) x[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 w = *reinterpret_cast<const float4 *>(ec + j);
          split2(-w.x * x[j], -w.y * x[j + 1], hi[j / 2], lo[j / 2]);
          split2(-w.z * x[j + 2], -w.w * x[j + 3], hi[j / 2 + 1], lo[j / 2 + 1]);
        }
        tmem_st8(tl + kColX + 16 * e, hi);
        tmem_st8(tl + kColX + 16 * e + 8, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bar + kReadyR, lane);

      sy.wait(kDoneU, i & 1);
      gam = du[2 * C - 1];
      tc_fence_after();
      {
        // (third pieces go into the columns of the O1 before, which this warp has
        // read and O1 of the next chunk takes after O2 of this one; 8 steps at
        // a time, for the registers)
        const uint32_t col3 = tl + kColO1 + (~i & 1) * 64 + 16 * e;
        float v[16];
        tmem_get16(tl + kColU + 16 * e, v);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t hi[4], lo[4], t[4];
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 d = *reinterpret_cast<const float4 *>(du + 16 * e + 8 * c + j);
            const float a0 = v[8 * c + j] * d.x, a1 = v[8 * c + j + 1] * d.y;
            const float a2 = v[8 * c + j + 2] * d.z, a3 = v[8 * c + j + 3] * d.w;
            split2(a0, a1, hi[j / 2], lo[j / 2]);
            split2(a2, a3, hi[j / 2 + 1], lo[j / 2 + 1]);
            t[j / 2] = third2(a0, a1, hi[j / 2], lo[j / 2]);
            t[j / 2 + 1] = third2(a2, a3, hi[j / 2 + 1], lo[j / 2 + 1]);
          }
          tmem_st4(tl + kColX + 16 * e + 4 * c, hi);
          tmem_st4(tl + kColX + 16 * e + 8 + 4 * c, lo);
          tmem_st4(col3 + 4 * c, t);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar + kReadyU, lane);
        // (the pieces that only the output needs)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t hi[4], lo[4], t[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float a = v[8 * c + 2 * j], b = v[8 * c + 2 * j + 1];
            split2(a, b, hi[j], lo[j]);
            if (kWide) t[j] = third2(a, b, hi[j], lo[j]);
          }
          tmem_st4(tl + kColU + 16 * e + 4 * c, hi);
          tmem_st4(tl + kColU + 16 * e + 8 + 4 * c, lo);
          if (kWide) tmem_st4(col3 + 8 + 4 * c, t);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bar + kReadyO, lane);
    }
    if (last && row < P) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (32 * e + j >= N) continue;
        if constexpr (!VEC)
          last[base + j] = H[j];
        else if (j % 4 == 0)
          __stcs(reinterpret_cast<float4 *>(last + base + j),
                 make_float4(H[j], H[j + 1], H[j + 2], H[j + 3]));
      }
    }
  } else if (warp >= 20) {
    // ------------------------------------- what does not depend on H
    // group gr takes the chunks of its parity
    const int q = warp & 3, gr = (warp - 20) >> 2, at = tid - 640 - gr * kAux;
    const uint32_t tl = static_cast<uint32_t>(32 * q) << 16;
    float *scr = reinterpret_cast<float *>(sm + oScr) + gr * kScr;
    unsigned char *pt = sm + oP + gr * 2 * kHalf, *tt = sm + oT + gr * 2 * kHalf;
    const float *beta_s = reinterpret_cast<const float *>(sm + oGate + gr * kGate);
    const float *neg_s = beta_s + C;  // -c: the high words, then the low ones

    *reinterpret_cast<uint4 *>(tt + swz(at >> 2, 4 + (at & 3))) = make_uint4(0u, 0u, 0u, 0u);

    for (int i = gr; i < nc; i += 2) {
      const int st = i % 3;
      const int len = min(total - i * C, C);
      sy.wait(kReadyG + st, (i / 3) & 1);
      sy.wait(kDoneS + gr, (i / 2) & 1);
      tc_fence_after();

      if (len < C) {
        // keys and values of whatever lies behind the sequence: nothing of
        // them may enter a product over steps (zero times a NaN would)
        sy.wait(kFullKQ + st, (i / 3) & 1);
        sy.wait(kFullV + gr, (i / 2) & 1);
        const int rows = C - len;
        for (int k = at; k < rows * 32; k += kAux) {
          const int r = len + (k >> 5), c = k & 31;
          unsigned char *d = c < 16 ? sm + oKQ + st * kStageKQ + (c >> 3) * 2 * kHalf
                                    : sm + oV + ((c >> 3) & 1) * kHalf;
          *reinterpret_cast<uint4 *>(d + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }

      // rows of A (lanes 0..63 of S) and of scale Q K^T o D (64..127) in
      // blocks of 32 columns, the diagonal one first, 16 columns at a time
      const int blk = q & 1, t = 32 * blk + lane;
      const bool isA = q < 2;
      const float ch = -neg_s[t], cl = -neg_s[C + t], rowf = isA ? beta_s[t] : p.scale;
      // U and O2 of chunk i - 2 have read the T and P in this one's place (the
      // other warps write T behind a barrier with these)
      if (!isA && i >= 2) sy.wait(kFreeP + gr, (i / 2 - 1) & 1);
#pragma unroll 1
      for (int part = 0; part <= 2 * blk + 1; ++part) {
        const bool diag = part < 2;
        const int e = diag ? blk : 0, c = part & 1;
        // columns kept
        const int last = t >= len ? 0 : (diag ? (isA ? lane : lane + 1) - 16 * c : 16);
        const float *cs = neg_s + 32 * e + 16 * c;
        float v[16], f[16];
        const auto diff = [&](float h0, float h1, float l0, float l1) {
          return __fadd2_rn(__fadd2_rn(make_float2(ch, ch), make_float2(h0, h1)),
                            __fadd2_rn(make_float2(cl, cl), make_float2(l0, l1)));
        };
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 x = *reinterpret_cast<const float4 *>(cs + j);
          const float4 y = *reinterpret_cast<const float4 *>(cs + C + j);
          const float2 a = diff(x.x, x.y, y.x, y.y), b = diff(x.z, x.w, y.z, y.w);
          f[j] = ex2_mufu(a.x);
          f[j + 1] = ex2_mufu(a.y);
          f[j + 2] = ex2_mufu(b.x);
          f[j + 3] = ex2_mufu(b.y);
        }
        tmem_get16(tl + kColS + 32 * e + 16 * c, v);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 y =
              __fmul2_rn(make_float2(f[j], f[j + 1]),
                         __fmul2_rn(make_float2(rowf, rowf), make_float2(v[j], v[j + 1])));
          f[j] = j < last ? y.x : 0.f;
          f[j + 1] = j + 1 < last ? y.y : 0.f;
        }
        if (isA) {  // transposed: the substitution reads columns of A
          float *da = scr + (diag ? (blk ? bA22 : bA11) : bA21) * kBlk + lane + 16 * c * kLd;
#pragma unroll
          for (int j = 0; j < 16; ++j) da[j * kLd] = f[j];
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint4 hi, lo;
            split8(f + 8 * k, hi, lo);
            const uint32_t o = swz(t, 4 * e + 2 * c + k);
            *reinterpret_cast<uint4 *>(pt + o) = hi;
            *reinterpret_cast<uint4 *>(pt + kHalf + o) = lo;
            if (kWide && diag && c == lane >> 4)
              *reinterpret_cast<uint4 *>(pt + swz(16 * blk + (lane & 15), 4 + 2 * c + k)) =
                  third8(f + 8 * k, hi, lo);
          }
        }
        // A22 is there for the warp of q = 2
        if (q == 1 && part == 1) bar_arrive(kBarA22 + gr, 64);
      }
      tc_fence_before();
      warp_arrive(bar + kFreeS, lane);
      if (!blk) {
        if (q) bar_sync(kBarA22 + gr, 64);
        invert32(scr + (q ? bA22 : bA11) * kBlk, lane);
      }
      bar_sync(kBarAux + gr, kAux);
      // T21 = -T22 (A21 T11)
      const int r2 = 2 * (at >> 3), c4 = 4 * (at & 7);
      float2 z[2][2];
      prod_t<32>(scr + bA21 * kBlk + r2, scr + bA11 * kBlk + c4, z);
      store24(scr + bZ * kBlk + r2 * kLd + c4, z, 1.f);
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {
        // pairs of T11 and T22, times b: 8 columns of a row
        const int r = at >> 2, c = at & 3;
        const float *src = scr + (w ? bA22 : bA11) * kBlk + r * kLd + 8 * c;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const float4 v = *reinterpret_cast<const float4 *>(src + j);
          const float4 x = *reinterpret_cast<const float4 *>(beta_s + 32 * w + 8 * c + j);
          f[j] = v.x * x.x;
          f[j + 1] = v.y * x.y;
          f[j + 2] = v.z * x.z;
          f[j + 3] = v.w * x.w;
        }
        uint4 hi, lo;
        split8(f, hi, lo);
        const uint32_t o = swz(32 * w + r, 4 * w + c);
        *reinterpret_cast<uint4 *>(tt + o) = hi;
        *reinterpret_cast<uint4 *>(tt + kHalf + o) = lo;
      }
      if (at < C) {  // the third piece of T's diagonal
        const float b = beta_s[at];
        const uint32_t hi = pack_bf16(b, 0.f), lo = pack_bf16(b - __uint_as_float(hi << 16), 0.f);
        *reinterpret_cast<__nv_bfloat16 *>(
            tt + swz(16 * (at >> 5) + (at & 15), 4 + ((at >> 3) & 3)) + 2 * (at & 7)) =
            __float2bfloat16_rn((b - __uint_as_float(hi << 16)) - __uint_as_float(lo << 16));
      }
      bar_sync(kBarAux + gr, kAux);
      prod_n<32>(scr + bA22 * kBlk + r2 * kLd, scr + bZ * kBlk + c4, z);
      {
        const float4 nb = *reinterpret_cast<const float4 *>(beta_s + c4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint2 hi, lo;
          split2(-nb.x * z[k][0].x, -nb.y * z[k][0].y, hi.x, lo.x);
          split2(-nb.z * z[k][1].x, -nb.w * z[k][1].y, hi.y, lo.y);
          const uint32_t o = swz(32 + r2 + k, c4 >> 3) + 2 * (c4 & 4);
          *reinterpret_cast<uint2 *>(tt + o) = hi;
          *reinterpret_cast<uint2 *>(tt + kHalf + o) = lo;
        }
      }
      fence_async_smem();
      // Where the group's next chunk is a tail, its wait for V there is for the
      // phase after this chunk's V, which has to be over by then: with V of
      // this chunk still on its way, the parity would be that of the phase
      // before, and the wait would pass.  Here, before T is handed over, the V
      // that is to come next cannot have been loaded yet, so this wait is sure
      // of its phase; V is behind the product before, long before T is due.
      if (i + 2 == nc - 1 && total < nc * C) sy.wait(kFullV + gr, (i / 2) & 1);
      warp_arrive(bar + kReadyT + gr, lane);
      if (lane == 0) mbar_arrive(bar + kFreeG + gr);
      // (the next chunk's A overwrites what the last product read)
      bar_sync(kBarAux + gr, kAux);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort) atomicOr(p.status, static_cast<unsigned>(MSS_ERR_TIMEOUT));
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, kTmemCols);
  }
}

// The states that segments start from: ends[s] <- ends[s] + ends[s - 1] M_s, in
// order, with ends[0] the state after the first segment and ends[s] on entry
// what segment s makes of a zero state.  kJoinRows rows of a head's state to a
// block, 2 rows of 4 columns to a thread; the next M is on its way into shared
// memory meanwhile (read where it is used, M's latency made a segment 6 us).
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(256) delta_join_kernel(const DeltaParams p) {
  extern __shared__ __align__(16) float ms[];  // one or two of M
  __shared__ __align__(8) float rows[128][kJoinRows + 2];
  const int N = static_cast<int>(p.N), c = 4 * (threadIdx.x & 31), r0 = 2 * (threadIdx.x >> 5);
  const int64_t sh = blockIdx.x, states = p.seqs * p.H * p.P * p.N;
  const int row0 = kJoinRows * blockIdx.y + r0;
  float *at = p.ends + (sh * p.P + row0) * N + c;
  auto in = [&](int r) { return row0 + r < p.P && c < N; };
  auto fetch = [&](int s) {
    const float *m = p.moves + ((s - 1) * p.seqs * p.H + sh) * N * N;
    const uint32_t d = smem_addr(ms + ((s - 1) & 1) * N * N);
    for (int k = threadIdx.x; k < N * N / 4; k += 256)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + 16 * k), "l"(m + 4 * k)
                   : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float4 v[2], next[2];
  auto load = [&](float4 (&e)[2], int s) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      e[r] = in(r) ? *reinterpret_cast<const float4 *>(at + s * states + r * N)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  fetch(1);
  load(v, 0);
  load(next, 1);
  for (int s = 1;; ++s) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      rows[c][r0 + r] = v[r].x;
      rows[c + 1][r0 + r] = v[r].y;
      rows[c + 2][r0 + r] = v[r].z;
      rows[c + 3][r0 + r] = v[r].w;
      v[r] = next[r];
    }
    if (s == p.segs - 1) break;
    if (s < p.segs - 2) {
      fetch(s + 1);
      load(next, s + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const float *m = ms + ((s - 1) & 1) * N * N + (c < N ? c : 0);
#pragma unroll 8
    for (int n = 0; n < N; ++n) {
      const float2 h = *reinterpret_cast<const float2 *>(&rows[n][r0]);
      const float4 x = *reinterpret_cast<const float4 *>(m + n * N);
      v[0] = make_float4(fmaf(h.x, x.x, v[0].x), fmaf(h.x, x.y, v[0].y), fmaf(h.x, x.z, v[0].z),
                         fmaf(h.x, x.w, v[0].w));
      v[1] = make_float4(fmaf(h.y, x.x, v[1].x), fmaf(h.y, x.y, v[1].y), fmaf(h.y, x.z, v[1].z),
                         fmaf(h.y, x.w, v[1].w));
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (in(r)) *reinterpret_cast<float4 *>(at + s * states + r * N) = v[r];
  }
}

// Copies of q, k, v (blockIdx.y) whose rows start on 16 bytes, for sizes and
// views that tensor maps do not take: a warp four rows, two channels of a lane.
// Rows end in zeros up to the next 16 bytes: a map's width then cuts inside
// them, and what is behind it is 0 whether the copy engine cuts there or not.
constexpr int kCopyWarps = 8, kCopyRows = 4;
__global__ void __launch_bounds__(32 * kCopyWarps)
    delta_copy_kernel(const __grid_constant__ DeltaParams p, __nv_bfloat16 *q, __nv_bfloat16 *k,
                      __nv_bfloat16 *v) {
  const int which = blockIdx.y, lane = threadIdx.x & 31;
  const __nv_bfloat16 *src =
      static_cast<const __nv_bfloat16 *>(which == 0 ? p.q : which == 1 ? p.k : p.v);
  __nv_bfloat16 *dst = which == 0 ? q : which == 1 ? k : v;
  const int64_t *st = which == 0 ? p.sq : which == 1 ? p.sk : p.sv;
  const int64_t heads = which == 2 ? p.H : p.G, width = which == 2 ? p.P : p.N;
  const int64_t pitch = (width + 7) / 8 * 8, rows = p.batch * p.L * heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyWarps * kCopyRows;
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5)) * kCopyRows;
       r0 < rows; r0 += step) {
    const __nv_bfloat16 *from[kCopyRows];
#pragma unroll
    for (int i = 0; i < kCopyRows; ++i) {
      const int64_t r = r0 + i < rows ? r0 + i : rows - 1, t = r / heads, b = t / p.L;
      from[i] = src + b * st[0] + (t - b * p.L) * st[1] + (r - t * heads) * st[2];
    }
    for (int64_t c = 2 * lane; c < pitch; c += 64) {
      __nv_bfloat162 two[kCopyRows];
#pragma unroll
      for (int i = 0; i < kCopyRows; ++i) {
        two[i].x = c < width ? from[i][c] : __float2bfloat16(0.f);
        two[i].y = c + 1 < width ? from[i][c + 1] : __float2bfloat16(0.f);
      }
#pragma unroll
      for (int i = 0; i < kCopyRows; ++i)
        if (r0 + i < rows)
          *reinterpret_cast<__nv_bfloat162 *>(dst + (r0 + i) * pitch + c) = two[i];
    }
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

// box {64, 1, steps, 1}, 128-byte swizzle; channels and steps past the end read
// as zeros
bool encode(CUtensorMap *m, const void *ptr, int64_t width, int64_t heads, int64_t L,
            int64_t batch, const int64_t (&s)[3], cuuint32_t steps) {
  auto enc = encoder();
  if (!enc) return false;
  const auto st = [](int64_t n, int64_t stride) {
    return static_cast<cuuint64_t>(n > 1 ? stride * 2 : 16);
  };
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(batch)};
  cuuint64_t strides[3] = {st(heads, s[2]), st(L, s[1]), st(batch, s[0])};
  cuuint32_t box[4] = {64, 1, steps, 1}, estr[4] = {1, 1, 1, 1};
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

namespace {
int64_t copy_pitch(int64_t width) { return (width + 7) / 8 * 8; }
}  // namespace

int64_t delta_copy_bytes(const DeltaParams &p) {
  return 2 * p.batch * p.L * (2 * p.G * copy_pitch(p.N) + p.H * copy_pitch(p.P));
}

cudaError_t launch_delta_copy(DeltaParams *p, void *to, cudaStream_t stream) {
  const int64_t n = copy_pitch(p->N), w = copy_pitch(p->P), rows = p->batch * p->L;
  __nv_bfloat16 *q = static_cast<__nv_bfloat16 *>(to), *k = q + rows * p->G * n,
                *v = k + rows * p->G * n;
  const int64_t per = kCopyWarps * kCopyRows, blocks = (rows * p->H + per - 1) / per;
  delta_copy_kernel<<<dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 3),
                      32 * kCopyWarps, 0, stream>>>(*p, q, k, v);
  p->q = q;
  p->k = k;
  p->v = v;
  const auto dense = [&](int64_t (&s)[3], int64_t heads, int64_t pitch) {
    s[0] = p->L * heads * pitch;
    s[1] = heads * pitch;
    s[2] = pitch;
  };
  dense(p->sq, p->G, n);
  dense(p->sk, p->G, n);
  dense(p->sv, p->H, w);
  return cudaGetLastError();
}

// A long sequence of few heads leaves SMs idle while its chain runs.  Cut into
// segments, the first pass runs the first of them, and every other one but the
// last from a zero state and from the unit rows: H_end = H_start M + B, B the
// end from zero and M the transition.  The join gives every segment's start,
// from which the second pass runs all but the first.  That is three times the
// work on two chains of 1 / segs the length.
// Times in chunks, a block's start taken as 3 of them and the join as 2.5 and
// one more for every further segment.  8192 steps of 32 heads of 128 x 128 take
// 389 us, 492 whole; of 8 heads 168, 478 whole; 2048 of 32 heads 117 and 130.
int delta_segments(const DeltaParams &p, int sms, int *seg_chunks, int64_t *floats) {
  const int64_t heads = p.seqs * p.H, tasks = heads * ((p.P + 127) / 128), nc = (p.L + C - 1) / C;
  const auto waves = [&](int64_t blocks) { return (blocks + sms - 1) / sms; };
  double best = 0.9 * waves(tasks) * (nc + 3);
  int segs = 0;
  // (the join moves rows of vectors)
  for (int s = 3; s <= 32 && s <= nc && tasks < sms && p.N % 4 == 0; ++s) {
    const int64_t len = (nc + s - 1) / s;
    if ((s - 1) * len >= nc) continue;  // an empty segment
    const double t = (waves((s - 1) * tasks + (s - 2) * heads) + waves((s - 1) * tasks)) *
                         (len + 3.0) + 2.5 + (s - 3);
    if (t < best) {
      best = t;
      segs = s;
      *seg_chunks = static_cast<int>(len);
    }
  }
  *floats = segs ? heads * p.N * ((segs - 1) * p.P + (segs - 2) * p.N) : 0;
  return segs;
}

cudaError_t launch_delta_chunk(const DeltaParams &p, bool out_bf16, cudaStream_t stream) {
  Maps maps;
  if (!encode(&maps.q, p.q, p.N, p.G, p.L, p.batch, p.sq, C) ||
      !encode(&maps.k, p.k, p.N, p.G, p.L, p.batch, p.sk, C) ||
      !encode(&maps.v, p.v, p.P, p.H, p.L, p.batch, p.sv, C))
    return cudaErrorInvalidValue;
  // y through tensor maps: bf16, rows that start and end on 16-byte boundaries
  // (a store writes whole 16 bytes, past a width that does not)
  const int y_tma = out_bf16 && p.P % 8 == 0 && al16(p.y) && map_strides(p.sy, p.batch, p.L, p.H) &&
                    encode(&maps.y, p.y, p.P, p.H, p.L, p.batch, p.sy, C);
  const int64_t heads = p.seqs * p.H, tasks = heads * ((p.P + 127) / 128);
  auto run = [&](auto kernel) {
    // per launch: the attribute belongs to the current device
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    auto pass = [&](int n, int64_t grid) {
      DeltaParams q = p;
      q.pass = n;
      kernel<<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(maps, q, y_tma);
      return cudaGetLastError();
    };
    if (!p.segs) return pass(0, tasks);
    cudaError_t f = pass(1, (p.segs - 1) * tasks + (p.segs - 2) * heads);
    if (f != cudaSuccess) return f;
    const int join_smem = static_cast<int>(p.N * p.N) * 4 * (p.segs > 3 ? 2 : 1);
    f = cudaFuncSetAttribute(delta_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             join_smem);
    if (f != cudaSuccess) return f;
    const dim3 join(static_cast<unsigned>(heads),
                    static_cast<unsigned>((p.P + kJoinRows - 1) / kJoinRows));
    delta_join_kernel<<<join, 256, join_smem, stream>>>(p);
    if ((f = cudaGetLastError()) != cudaSuccess) return f;
    return pass(2, (p.segs - 1) * tasks);
  };
  auto by_state = [&](auto out, auto nk) {
    using O = decltype(out);
    constexpr int NK = decltype(nk)::value;
    return p.N % 4 == 0 && al16(p.h0) && al16(p.last) ? run(delta_chunk_kernel<O, NK, true>)
                                                      : run(delta_chunk_kernel<O, NK, false>);
  };
  auto by_width = [&](auto nk) {
    return out_bf16 ? by_state(__nv_bfloat16(), nk) : by_state(float(), nk);
  };
  return p.N <= 64 ? by_width(std::integral_constant<int, 4>())
                   : by_width(std::integral_constant<int, 8>());
}

}  // namespace sss48
