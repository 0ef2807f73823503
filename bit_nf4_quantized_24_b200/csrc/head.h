// What the two translation units of the head losses share: head.cu (the call, and
// the products for many tokens) and head_few.cu (those for at most 128).
#pragma once

#include "internal.h"

namespace qn {

constexpr float kHeadFits = 64.0f;  // |reference| (log2) up to which e is stored without it
constexpr int kHeadFewTokens = 128;
// Tokens up to which a teacher's p - q are stored in two parts, the bf16 value and
// what its rounding left (in rows of its own behind the tokens'): the values of one
// token often share a mantissa (a flat teacher's are all near -1 / k), so that their
// roundings add up instead of cancelling.  dX of single tokens at T = 4: error 2.6e-3
// with one part, 1.7e-3 (its own rounding to bf16) with two.  Over many tokens the
// roundings differ (at most 2.2e-3 with one part), and the second part costs the more
// the wider the products get: 32000 x 4096, 64 slots, one / two parts: 16 tokens 105 /
// 106 us (NF4 head 95 / 100), 32 tokens 108 / 115 us.
constexpr int kHeadTwoParts = 16;

// The frozen head: W, or (W null) the NF4 weight.
struct HeadWeight {
  const uint16_t* W;
  const uint8_t* codes;
  const uint8_t* absmax_q;
  const float* dq_scale;
  int block, dq_block;
  int64_t N, K;
};

// Parts of a logit's contraction of K: a part fills an accumulator, which the
// epilogue then adds up in fp32.  The tensor core truncates every addition to an
// accumulator, always towards 0, so a long sum drifts with its length: products of
// one sign, in units of 2^-24 of the logit, by 5 after 32 steps of 16, 17 after 64,
// 24 after 85, 54 after 128 and 176 after 256.  fp32's own additions round to
// nearest.  What that does to a loss grows with the logits' spread, so with K: parts
// have at most 85 steps (1365 of K), above K = 8192 64.  Largest error of the losses
// over drawn calls of up to 8192 x 131072 x 8192 (2-norm, relative): parts of 85
// steps 1.0e-6, of 128 1.5e-6; time of the losses / the step of 4096 x 32000 x 4096
// with 64, 85 and 128 steps: 760 / 1691, 758 / 1688, 748 / 1687 us under the power
// cap, and of its distillation step (64 slots) 1742, 1706, 1706 us.
__host__ __device__ constexpr int parts_of(int K) { return K <= 8192 ? (3 * K + 4095) / 4096 : (K + 1023) / 1024; }

// log2 of a block's weights (32, 64, 128 or 256).
inline int block_log2(int block) { return block == 32 ? 5 : block == 64 ? 6 : block == 128 ? 7 : 8; }

// What the products' epilogues read and write (MODE 0: logits, MODE 1: gradient).
struct HeadEpi {
  int rows;         // token rows of the piece
  int cols;         // MODE 0: N; MODE 1: K
  // MODE 0
  float c;                   // log2(e) / T
  float2* part;              // [segments][rows], per column segment: (reference n, sum of exp2(z c - n))
  uint16_t* e;               // [rows][lde] (nullable)
  uint16_t* e_low;           // few tokens: [rows][lde] to be written as zeros (nullable)
  int64_t lde;
  const int64_t* labels;     // [rows] (cross entropy), or
  const int* sidx;           // [rows][k] targets in ascending order, and
  const uint16_t* off;       // [rows][segments + 1] first target of each column segment
  int k;
  const uint16_t* X;         // few tokens: the labels' logits are computed beside the products
  float* zlabel;             // [rows]
  float2* ztgt;              // [rows][k] the teacher's slots' logits: (z c - n, n)
  // MODE 1: dX = sums x y + z W[w]; y = 0: the row is written as zeros; w < 0: no such term
  const float4* rscale;      // [rows] (x, y, z, w as int)
  const uint16_t* W;         // both modes: bf16 head (few tokens on an NF4 head: null)
  uint16_t* out;             // [rows][cols]
  float* split;              // fp32 sums of the split tiles' pieces
  bool two_parts;            // few tokens: the sums of row i have a second part in row rows + i
};

// exp2 on the special-function unit: relative error about 2^-22, which is far
// below the bf16 rounding of e and of the order of the fp32 sums' own rounding.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A logit times c = log2(e) / T as the sum of a whole number, .y, and what is left
// of it, .x.  A logit of -inf (or one that 1 / T takes there) has .y = -inf and
// .x = 0, so that differences from .y stay numbers; +inf and NaN give NaN.
__device__ __forceinline__ float2 log2_parts(float z, float c) {
  const float n = rintf(z * c);
  return make_float2(n == -INFINITY ? 0.0f : fmaf(z, c, -n), n);
}

// s + the products of eight bf16, with additions rounded to nearest.
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s = fmaf(__uint_as_float(x[j] << 16), __uint_as_float(y[j] << 16), s);
    s = fmaf(__uint_as_float(x[j] & 0xffff0000u), __uint_as_float(y[j] & 0xffff0000u), s);
  }
  return s;
}
__device__ __forceinline__ float warp_sum(float z) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}
// x . w over K bf16 by a warp.
__device__ __forceinline__ float dot_row(const uint16_t* x, const uint16_t* w, int K, int lane) {
  float z = 0.0f;
#pragma unroll 4
  for (int j = lane; j < K / 8; j += 32)
    z = dot8(reinterpret_cast<const uint4*>(x)[j], reinterpret_cast<const uint4*>(w)[j], z);
  return warp_sum(z);
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// True in one lane of a converged warp.  The single-thread roles (TMA, MMA) run
// with the whole warp and issue from the elected lane: their addresses and
// descriptors are then the same in all lanes, as those instructions want them.
// In code that only one lane runs, a stage's MMAs took 800 cycles to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// wait_bounded by a whole warp: true if all lanes saw the phase complete.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort, status));
}
__device__ __forceinline__ bool wait_warp_cluster(uint32_t bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xffffffffu, wait_bounded_cluster(bar, parity, abort, status));
}

// A position in a ring of stages.  Kept as slot and phase: dividing a running
// count by the ring's length took longer than the MMAs of a narrow stage.
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance(int by, int stages) {  // by may exceed the ring's length
    slot += by;
    while (slot >= stages) {
      slot -= stages;
      phase ^= 1u;
    }
  }
};

// At most kHeadFewTokens tokens.  Column segments are tiles of few_tile_rows(N)
// entries; the gradient's p.split holds few_splits(N, K) x rows x K sums.
int few_tile_rows(int64_t N);
int few_splits(int64_t N, int64_t K);
cudaError_t launch_few_logits(const HeadWeight& h, const uint16_t* X, int br, const HeadEpi& p, cudaStream_t st);
cudaError_t launch_few_grad(const HeadWeight& h, const uint16_t* P, int64_t ldp, int nsplit, const HeadEpi& p,
                            cudaStream_t st);

}  // namespace qn
