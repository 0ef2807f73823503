// The two products of the head losses for a few tokens (at most 128), where the
// head's bytes from HBM are the bound: the roles of the operands are swapped
// against head.cu.  The head's rows (logits) or columns (gradient) are the 128
// MMA rows of a CTA, and the tokens are the narrow N side, so a stage of the ring
// is nearly all head (16 KB of it beside 128 bytes per token), and the whole
// ring is in flight.
//
//   MODE 0, logits:    D[v, m] = sum_k W[v, k] X[m, k]     (W K-major)
//   MODE 1, gradient:  D[k, m] = sum_v W[v, k] P[m, v]     (W MN-major)
//
// An NF4 head is expanded in shared memory, one stage at a time, as the fused
// GEMM of the layer does, so that its 4 bits are all that HBM moves.
#include <algorithm>

#include "head.h"

namespace qn {

namespace {

constexpr int UM = 128;              // MMA rows: vocabulary entries (MODE 0) or hidden columns (MODE 1)
constexpr int BK = 64;                // contraction of a sub-stage (a 128-byte row of each operand)
constexpr int SUB = 2;                // sub-stages per stage: waits and commits are paid per stage
constexpr int W_BYTES = UM * BK * 2;  // head tile of a sub-stage, in bf16
constexpr int MAX_STAGES = 6;
constexpr int DQ_GROUPS = 4;          // groups of 4 warps that take turns at expanding the stages
constexpr int BUF_PITCH = UM + 4;     // floats per token in the epilogue's buffer
constexpr int BUF_TOKENS = 16;
constexpr int BUF_BYTES = 2 * BUF_TOKENS * BUF_PITCH * 4;  // per set of epilogue warps
// Sets of four epilogue warps, which take turns at 16 tokens: two on a bf16 head
// (128 tokens, 8000 x 1024 / 32000 x 2048 with the gradient, on the GPU: 38 / 73 us
// with one set, 32 / 66 us with two; now 64 us); an NF4 head's block has no threads to
// spare.
__host__ __device__ constexpr int epi_sets(bool nf4) { return nf4 ? 1 : 2; }
constexpr int BAR_BYTES = 512;
constexpr int SMEM_MAX = 232448;

__host__ __device__ constexpr int threads_of(bool nf4) { return 64 + epi_sets(nf4) * 128 + (nf4 ? DQ_GROUPS * 128 : 0); }

struct FewBars {
  uint64_t full[MAX_STAGES];   // head tile and token tile landed (or were written)
  uint64_t empty[MAX_STAGES];  // MMAs of the stage completed
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(FewBars) <= BAR_BYTES, "barrier block");

struct FewGrid {
  int tiles;   // tiles along the MMA rows
  int br;      // MMA rows of a tile (MODE 0: vocabulary entries, a multiple of 8 up to 128; MODE 1: 128)
  int nsplit;  // pieces of the contraction (MODE 1)
  int numK;    // stages of the contraction (SUB x 64 each)
  int tp;      // tokens, rounded up to 16
  int stages;
  int parts;   // accumulators that a round of the contraction fills in turn
  int rounds;  // rounds (MODE 0), joined in tp more columns of TMEM if there are several
  int cols;    // TMEM columns
};

__device__ __forceinline__ void epilogue_barrier(int set) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");
}
// The same barrier; tells all 128 threads whether ok holds for every one of them.
__device__ __forceinline__ bool epilogue_all(int set, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "r"(1 + set)
      : "memory");
  return r != 0;
}

// KIND 0: bf16 head; 1: NF4 in the default format (64-weight blocks, double
// quantization); 2: NF4 with 2^lg-weight blocks, double quantization if dq.
//   warp 0       TMA producer
//   warp 1       TMEM allocation, MMA issue
//   warps 2-9    KIND 0: epilogue in two sets of four (two accumulators alternate)
//   warps 2-5    KIND > 0: epilogue
//   warps 6-21   KIND > 0: expansion of the codes
// Every wait is bounded; on expiry the kernel records kDevTimeout, drains what
// it issued, frees TMEM and returns.
template <int MODE, int KIND>
__global__ void __launch_bounds__(threads_of(KIND > 0), 1)
    k_few(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, FewGrid g, HeadEpi p,
          const uint8_t* __restrict__ codes, const uint8_t* __restrict__ absmax_q, const float* __restrict__ dq_scale, Nf4Levels lv, int N, int K, int lg,
          int dq, int* status) {
  constexpr bool NF4 = KIND > 0, GEN = KIND == 2;
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int x_tile = g.tp * BK * 2, stage_bytes = SUB * (W_BYTES + x_tile);
  const uint32_t buf = base + g.stages * stage_bytes;
  constexpr int SETS = epi_sets(NF4);
  const uint32_t bar0 = buf + SETS * BUF_BYTES;
  FewBars* bars = reinterpret_cast<FewBars*>(smem_raw + (bar0 - raw));
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
  auto acc_full = [&](int a) { return bar0 + 8u * (2 * MAX_STAGES + a); };
  auto acc_empty = [&](int a) { return bar0 + 8u * (2 * MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * MAX_STAGES + 4);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nitems = g.tiles * g.nsplit, tokens = MODE == 1 && p.two_parts ? 2 * p.rows : p.rows;

  // Item i: piece z of tile nt; pieces of one range of the contraction follow
  // one another, so the CTAs walk it together.
  auto item = [&](int i, int& nt, int& z, int& kbeg, int& kend) {
    z = i / g.tiles;
    nt = i - z * g.tiles;
    kbeg = static_cast<int>(static_cast<int64_t>(z) * g.numK / g.nsplit);
    kend = static_cast<int>(static_cast<int64_t>(z + 1) * g.numK / g.nsplit);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(full(s), NF4 ? 1 + 4 : 1);  // the producer, and the four warps that expand the stage
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full(a), 1);
      mbar_init(acc_empty(a), 4 * SETS);
    }
    mbar_init(drain_bar, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    if (!NF4) tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (tokens < g.tp) {  // the token rows that no copy writes hold zeros
    const int n = (g.tp - tokens) * BK * 2 / 16;
    for (int s = 0; s < g.stages * SUB; ++s)
      for (int i = threadIdx.x; i < n; i += blockDim.x)
        st_shared_v4(base + s / SUB * stage_bytes + SUB * W_BYTES + s % SUB * x_tile + tokens * BK * 2 + 16 * i, 0u, 0u,
                     0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(bar0 + static_cast<uint32_t>(offsetof(FewBars, tmem_base)), g.cols);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0) {
    // --------------------------------------------------------- TMA producer
    const uint32_t x_bytes = tokens * BK * 2, w_bytes = NF4 ? 0 : MODE == 0 ? g.br * BK * 2 : W_BYTES;
    bool ok = true, issued = false;
    RingPos r;
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
      int nt, z, kbeg, kend;
      item(i, nt, z, kbeg, kend);
      for (int k = kbeg; k < kend; ++k, r.advance(1, g.stages)) {
        if (!(ok = wait_warp(empty(r.slot), r.phase ^ 1, abort, status))) break;
        issued = true;
        if (elect_one()) {
          const uint32_t bar = full(r.slot), w_s = base + r.slot * stage_bytes;
          mbar_arrive_expect_tx(bar, SUB * (w_bytes + x_bytes));
#pragma unroll
          for (int u = 0; u < SUB; ++u) {  // past the end of the contraction: zeros
            const int at = (k * SUB + u) * BK;
            if (!NF4 && MODE == 0) {
              tma_load_2d(w_s + u * W_BYTES, &tm_w, bar, at, nt * g.br);
            } else if (!NF4) {
              tma_load_2d(w_s + u * W_BYTES, &tm_w, bar, nt * UM, at);
              tma_load_2d(w_s + u * W_BYTES + 8192, &tm_w, bar, nt * UM + 64, at);
            }
            tma_load_2d(w_s + SUB * W_BYTES + u * x_tile, &tm_x, bar, at, 0);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && issued) {  // the copies already issued land well within this time
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 20000000ull) {
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    const uint32_t idesc = idesc_bf16(UM, g.tp, MODE == 1, false);
    bool ok = true, committed = false;
    RingPos r;
    int t = 0;
    for (int i = blockIdx.x, rd = 0; i < nitems && ok; ++t) {
      int nt, z, ibeg, iend;
      item(i, nt, z, ibeg, iend);
      const int kbeg = MODE == 0 ? ibeg + rd * (iend - ibeg) / g.rounds : ibeg;
      const int kend = MODE == 0 ? ibeg + (rd + 1) * (iend - ibeg) / g.rounds : iend;
      if (MODE == 1 || ++rd == g.rounds) {
        rd = 0;
        i += gridDim.x;
      }
      if (!(ok = wait_warp(acc_empty(t & 1), ((t >> 1) & 1) ^ 1, abort, status))) break;
      tc_fence_after();
      const uint32_t d0 = tmem + (t & 1) * g.parts * g.tp;
      int part = 0, start = kbeg;
      for (int k = kbeg; k < kend; ++k, r.advance(1, g.stages)) {
        if (!(ok = wait_warp(full(r.slot), r.phase, abort, status))) break;
        tc_fence_after();
        const uint32_t w_s = base + r.slot * stage_bytes, x_s = w_s + SUB * W_BYTES;
        const uint64_t ad = MODE == 0 ? desc_sw128(w_s, 16, 1024) : desc_sw128(w_s, 8192, 1024);
        const uint64_t bd = desc_sw128(x_s, 16, 1024);
        if (part + 1 < g.parts && k == kbeg + (part + 1) * (kend - kbeg) / g.parts) {
          ++part;
          start = k;
        }
        const uint32_t d = d0 + part * g.tp;
        if (elect_one()) {
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)  // a descriptor's low bits are the address / 16
              tc_mma_f16(d, ad + u * (W_BYTES / 16) + kk * (MODE == 0 ? 2 : 128), bd + u * (x_tile / 16) + kk * 2, idesc,
                         (k > start || u + kk > 0) ? 1u : 0u);
          tc_commit(empty(r.slot));
        }
        __syncwarp();
        committed = true;
      }
      if (ok && elect_one()) tc_commit(acc_full(t & 1));
      __syncwarp();
    }
    if (!ok && committed && elect_one()) {
      tc_commit(drain_bar);
      wait_drain(drain_bar, 0);
    }
    __syncwarp();
  } else if (warp < 2 + 4 * SETS) {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3, ew = (warp - 2) & 3, set = (warp - 2) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    // The labels' logits, a token per warp: fp32 dot products with additions rounded
    // to nearest, while the first tile's products run.  (Taken from the accumulators,
    // which truncate, they made the loss of a single confident token up to 9e-6 off,
    // of 128 tokens and K = 8192 2e-6; in the statistics kernel they took 1 to 8 us.)
    if (MODE == 0 && p.labels) {
      for (int row = blockIdx.x + gridDim.x * (warp - 2); row < tokens; row += gridDim.x * 4 * SETS) {
        const int64_t y = p.labels[row];
        if (y < 0 || y >= p.cols) continue;
        const uint4* x = reinterpret_cast<const uint4*>(p.X + static_cast<int64_t>(row) * K);
        float z = 0.0f;
        for (int j = lane; j < K / 32; j += 32) {  // 32 weights, of one block
          const int64_t at = y * K + 32 * j, blk = at >> lg;
          uint4 w[4];
          if (!NF4) {
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = ldg_nc_v4(p.W + at + 8 * q);
          } else {
            const uint4 c = ldg_nc_v4(codes + at / 2);
            const Nf4Lut lut = make_lut(
                lv, dq ? __fmul_rn(static_cast<float>(absmax_q[blk]), dq_scale[blk >> 8]) : dq_scale[blk]);
            deq8(c.x, lut, w[0].x, w[0].y, w[0].z, w[0].w);
            deq8(c.y, lut, w[1].x, w[1].y, w[1].z, w[1].w);
            deq8(c.z, lut, w[2].x, w[2].y, w[2].z, w[2].w);
            deq8(c.w, lut, w[3].x, w[3].y, w[3].z, w[3].w);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) z = dot8(x[4 * j + q], w[q], z);
        }
        z = warp_sum(z);
        if (lane == 0) p.zlabel[row] = z;
      }
    }
    int t = 0, filled = 0;
    // A round that is not the contraction's last leaves its sums, with those of the
    // rounds before, in TMEM, where the same threads find them again.
    const uint32_t total = tmem + lane_base + 2 * g.parts * g.tp;
    for (int i = blockIdx.x, rd = 0; i < nitems; ++t) {
      int nt, z, kbeg, kend;
      item(i, nt, z, kbeg, kend);
      // a set's four warps leave together: they meet at barriers
      if (!epilogue_all(set, wait_bounded(acc_full(t & 1), (t >> 1) & 1, abort, status))) break;
      tc_fence_after();
      const uint32_t acc = tmem + lane_base + (t & 1) * g.parts * g.tp;
      auto sums = [&](int m, uint32_t (&x)[16]) {  // of 16 tokens, as the bits of floats
        tmem_ld_x16((rd > 0 ? total : acc) + m, x);
        tmem_ld_wait();
#pragma unroll 1
        for (int q = rd > 0 ? 0 : 1; q < g.parts; ++q) {
          uint32_t v[16];
          tmem_ld_x16(acc + q * g.tp + m, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) + __uint_as_float(v[j]));
        }
      };
      if (MODE == 0 && rd + 1 < g.rounds) {
#pragma unroll 1
        for (int m = 16 * set; m < tokens; m += 16 * SETS) {
          uint32_t x[16];
          sums(m, x);
          tmem_st_x16(total + m, x);
        }
        tmem_st_wait();
        ++rd;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(t & 1));
        continue;
      }
      if (MODE == 1) {
        const int k = nt * UM + quad * 32 + lane;
        float* dst = p.split + static_cast<int64_t>(z) * tokens * p.cols + k;
#pragma unroll 1
        for (int m = 16 * set; m < tokens; m += 16 * SETS) {
          uint32_t v[16];
          tmem_ld_x16(acc + m, v);
          tmem_ld_wait();
          if (k < p.cols) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (m + j < tokens) dst[static_cast<int64_t>(m + j) * p.cols] = __uint_as_float(v[j]);
          }
        }
      } else {
        const int v0 = nt * g.br;                                 // first vocabulary entry
        const int ncols = min(g.br, p.cols - v0);                 // entries of the tile
        const int ewidth = static_cast<int>(min(static_cast<int64_t>(g.br), p.lde - v0));
#pragma unroll 1
        for (int m = BUF_TOKENS * set; m < tokens; m += BUF_TOKENS * SETS, ++filled) {
          // 16 tokens x 128 entries into shared memory, token by token; then a warp
          // has a token's entries side by side
          const uint32_t b = buf + set * BUF_BYTES + (filled & 1) * (BUF_BYTES / 2);
          float* bp = reinterpret_cast<float*>(smem_raw + (b - raw));
          {
            uint32_t x[BUF_TOKENS];
            sums(m, x);
#pragma unroll
            for (int j = 0; j < BUF_TOKENS; ++j) bp[j * BUF_PITCH + quad * 32 + lane] = __uint_as_float(x[j]);
          }
          epilogue_barrier(set);
          // The warp's four tokens together: each step is a chain of shuffles.
          constexpr int TW = BUF_TOKENS / 4;
          const int j0 = ew * TW, c0 = 4 * lane;
          float e[TW][4], ref[TW], top[TW], sum[TW], mx[TW];
          int label[TW];  // the token's label in this tile, or -1
#pragma unroll
          for (int u = 0; u < TW; ++u) {
            label[u] = -1;
            if (p.labels && m + j0 + u < tokens) {
              const int64_t y = p.labels[m + j0 + u] - v0;
              if (y >= 0 && y < ncols) label[u] = static_cast<int>(y);
            }
          }
#pragma unroll
          for (int u = 0; u < TW; ++u) {
            const float4 x = *reinterpret_cast<const float4*>(bp + (j0 + u) * BUF_PITCH + c0);
            e[u][0] = x.x, e[u][1] = x.y, e[u][2] = x.z, e[u][3] = x.w;
            mx[u] = -INFINITY;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (c0 + q >= ncols || c0 + q == label[u]) e[u][q] = -INFINITY;  // a label stays out of the sums
              mx[u] = fmaxf(mx[u], e[u][q]);
            }
          }
#pragma unroll
          for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int u = 0; u < TW; ++u) mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], d));
#pragma unroll
          for (int u = 0; u < TW; ++u) {
            top[u] = rintf(mx[u] * p.c);  // as in head.cu
            ref[u] = top[u] == -INFINITY ? 0.0f : top[u];
#pragma unroll
            for (int q = 0; q < 4; ++q) e[u][q] = exp2_fast(fmaf(e[u][q], p.c, -ref[u]));
            sum[u] = (e[u][0] + e[u][1]) + (e[u][2] + e[u][3]);
          }
#pragma unroll
          for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int u = 0; u < TW; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], d);
#pragma unroll
          for (int u = 0; u < TW; ++u) {
            const int j = j0 + u, row = m + j;
            if (row >= tokens) break;
            if (lane == 0)
              p.part[static_cast<int64_t>(nt) * tokens + row] = make_float2(top[u], sum[u]);
            if (p.e) {
              uint16_t* er = p.e + static_cast<int64_t>(row) * p.lde + v0;
              const float back = exp2f(fabsf(ref[u]) <= kHeadFits ? ref[u] : 0.0f);
              if (c0 < ewidth)  // groups of four entries are whole: br % 8 == 0, lde % 64 == 0
                *reinterpret_cast<uint2*>(er + c0) = make_uint2(bf16x2_bits(e[u][0] * back, e[u][1] * back),
                                                                bf16x2_bits(e[u][2] * back, e[u][3] * back));
              uint16_t* el = p.e_low ? p.e_low + static_cast<int64_t>(row) * p.lde + v0 : nullptr;
              if (el && c0 < ewidth) *reinterpret_cast<uint2*>(el + c0) = make_uint2(0u, 0u);
              if (nt == g.tiles - 1)  // the pitch may reach past the last tile
                for (int64_t c = g.br + c0; c < p.lde - v0; c += 128) {
                  *reinterpret_cast<uint2*>(er + c) = make_uint2(0u, 0u);
                  if (el) *reinterpret_cast<uint2*>(el + c) = make_uint2(0u, 0u);
                }
            }
            if (!p.labels) {
              const uint16_t* o = p.off + static_cast<int64_t>(row) * (g.tiles + 1) + nt;
              for (int s = o[0] + lane; s < o[1]; s += 32) {
                const int64_t at = static_cast<int64_t>(row) * p.k + s;
                p.ztgt[at] = make_float2(fmaf(bp[j * BUF_PITCH + p.sidx[at] - v0], p.c, -ref[u]), ref[u]);
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(t & 1));
      rd = 0;
      i += gridDim.x;
    }
  } else if (NF4) {
    // ----------------------------------------------- expansion of the codes
    // Never more groups than stages: a group that has expanded stage n knows that
    // stage n - stages is consumed, and no more; stage n + groups must not lie two
    // turns of the ring past the last stage known to be consumed, because a phase's
    // parity cannot tell the two turns apart.
    const int groups = min(DQ_GROUPS, g.stages);
    const int e = warp - 6, grp = e >> 2;
    // A stage is 128 rows of W (MODE 0: of the tile; MODE 1: of the contraction) by
    // two groups of 64 columns.  A thread expands one group of two rows, 16 apart,
    // its neighbour the other group: their codes are 64 contiguous bytes, and a load
    // touches 16 rows (a load instruction costs a cycle per 128-byte line; 16 tokens
    // on a 32000 x 4096 head with the gradient, when this was chosen: 108 us, with a
    // row per lane 117; now 90 us).
    const int row0 = (e & 3) * 32 + (lane >> 1), half = lane & 1;
    struct Walk {
      int i, nt, z, k, kend;
    };
    auto start = [&](Walk& w) {
      if (w.i < nitems) item(w.i, w.nt, w.z, w.k, w.kend);
    };
    auto advance = [&](Walk& w, int by) {  // by stages; an item may be shorter than that
      w.k += by;
      while (w.i < nitems && w.k >= w.kend) {
        const int over = w.k - w.kend;
        w.i += gridDim.x;
        start(w);
        w.k += over;
      }
    };
    // The codes go from global memory to registers (32 bytes: a whole sector), one of
    // the group's stages ahead, with the one or two scales of their blocks.  Each row
    // has its own registers: handing them on by moves would wait for the loads.
    struct Part {
      uint32_t c[8];
      uint32_t q0, q1;
      float s0, s1;
      bool valid, zero;  // has weights; must hold zeros
    };
    auto fetch = [&](const Walk& w, int row, Part& f) {
      f.valid = f.zero = false;
      if (w.i >= nitems) return;
      const int wrow = MODE == 0 ? w.nt * g.br + row : w.k * (SUB * BK) + row;
      const int kcol = MODE == 0 ? (w.k * SUB + half) * BK : w.nt * UM + 64 * half;
      // Past the end of the contraction the token tile is zero, and the head must be
      // finite; MMA rows without an output may hold anything.
      f.zero = MODE == 0 ? kcol >= K : wrow >= N;
      if (wrow >= N || kcol >= K || (MODE == 0 && row >= g.br)) return;
      f.valid = true;
      const int64_t at = static_cast<int64_t>(wrow) * K + kcol;
      ldg_nc_v8(codes + at / 2, f.c);
      if (!GEN) {
        f.q0 = __ldg(absmax_q + (at >> 6));
        f.s0 = __ldg(dq_scale + (at >> 14));
      } else {
        const int64_t blk = at >> lg;
        if (dq) {
          f.q0 = __ldg(absmax_q + blk);
          f.s0 = __ldg(dq_scale + (blk >> 8));
          if (lg == 5) {
            f.q1 = __ldg(absmax_q + blk + 1);
            f.s1 = __ldg(dq_scale + ((blk + 1) >> 8));
          }
        } else {
          f.s0 = __ldg(dq_scale + blk);
          if (lg == 5) f.s1 = __ldg(dq_scale + blk + 1);
        }
      }
    };
    RingPos r;
    auto expand = [&](int row, Part& f) {
      const uint32_t row_s = base + r.slot * stage_bytes +
                             (MODE == 0 ? half * W_BYTES + row * 128
                                        : (row >> 6) * W_BYTES + half * 8192 + (row & 63) * 128);
      // Neighbours write the same row of two tiles, so the same banks: the second one
      // starts with its other four chunks.
      const uint32_t sw = (row & 7) ^ (half << 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = f.c[j], y = f.c[j + 4];
        f.c[j] = half ? y : x;
        f.c[j + 4] = half ? x : y;
      }
      if (f.valid) {
        const float a0 = (GEN && !dq) ? f.s0 : __fmul_rn(static_cast<float>(f.q0), f.s0);
        if (GEN && lg == 5) {
          const float a1 = dq ? __fmul_rn(static_cast<float>(f.q1), f.s1) : f.s1;
          const Nf4Lut lut = make_lut(lv, half ? a1 : a0), lut1 = make_lut(lv, half ? a0 : a1);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t o0, o1, o2, o3;
            deq8(f.c[j], j < 4 ? lut : lut1, o0, o1, o2, o3);
            st_shared_v4(row_s + ((j ^ sw) << 4), o0, o1, o2, o3);
          }
        } else {
          const Nf4Lut lut = make_lut(lv, a0);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t o0, o1, o2, o3;
            deq8(f.c[j], lut, o0, o1, o2, o3);
            st_shared_v4(row_s + ((j ^ sw) << 4), o0, o1, o2, o3);
          }
        }
      } else if (f.zero) {
#pragma unroll
        for (int j = 0; j < 8; ++j) st_shared_v4(row_s + ((j ^ sw) << 4), 0u, 0u, 0u, 0u);
      }
    };
    static_assert(SUB == 2, "two groups of 64 columns, or two sets of 64 rows, per stage");
    Walk w{grp < groups ? static_cast<int>(blockIdx.x) : nitems, 0, 0, 0, 0};
    start(w);
    advance(w, grp);
    r.advance(grp, g.stages);
    Part a, b;
    fetch(w, row0, a);
    fetch(w, row0 + 16, b);
    while (w.i < nitems) {
      if (!wait_warp(empty(r.slot), r.phase ^ 1, abort, status)) break;
      advance(w, groups);
      expand(row0, a);
      expand(row0 + 16, b);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(r.slot));
      r.advance(groups, g.stages);
      fetch(w, row0, a);  // after both: the second expansion would wait for these loads too
      fetch(w, row0 + 16, b);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, g.cols);
  }
}

// Sum of the gradient's pieces in piece order, times the row's factors, plus the
// label's term, rounded once to bf16.  Thread: 4 consecutive outputs of a token.
__global__ void __launch_bounds__(128) k_few_join(const float* __restrict__ split, int nsplit, HeadEpi p,
                                                  const uint8_t* __restrict__ codes,
                                                  const uint8_t* __restrict__ absmax_q,
                                                  const float* __restrict__ dq_scale, Nf4Levels lv, int lg, int dq) {
  pdl_wait();  // the call's last kernel: it lets nothing start early (see k_head)
  const int c = (blockIdx.x * 128 + threadIdx.x) * 4, row = blockIdx.y;
  if (c >= p.cols) return;
  const int64_t at = static_cast<int64_t>(row) * p.cols + c, part = static_cast<int64_t>(p.rows) * p.cols;
  const int64_t piece = p.two_parts ? 2 * part : part;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int z = 0; z < nsplit; ++z) {
    const float4 x = *reinterpret_cast<const float4*>(split + at + z * piece);
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
  }
  if (p.two_parts) {
    float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int z = 0; z < nsplit; ++z) {
      const float4 x = *reinterpret_cast<const float4*>(split + at + part + z * piece);
      b.x += x.x; b.y += x.y; b.z += x.z; b.w += x.w;
    }
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  const float4 f = p.rscale[row];
  const int label = __float_as_int(f.w);
  float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // of the label's row of the head
  if (label >= 0) {
    const int64_t from = static_cast<int64_t>(label) * p.cols + c;
    if (p.W) {
      const uint2 b = *reinterpret_cast<const uint2*>(p.W + from);
      w[0] = __uint_as_float(b.x << 16), w[1] = __uint_as_float(b.x & 0xffff0000u);
      w[2] = __uint_as_float(b.y << 16), w[3] = __uint_as_float(b.y & 0xffff0000u);
    } else {  // the four weights lie in one block
      const int64_t blk = from >> lg;
      const float scale = dq ? __fmul_rn(static_cast<float>(absmax_q[blk]), dq_scale[blk >> 8]) : dq_scale[blk];
      const uint32_t b = *reinterpret_cast<const uint16_t*>(codes + from / 2);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = __bfloat162float(__float2bfloat16_rn(__fmul_rn(lv.v[(b >> (4 * j)) & 15u], scale)));
    }
  }
  uint2 o = make_uint2(0u, 0u);
  if (f.y != 0.0f)
    o = make_uint2(bf16x2_bits(fmaf(f.z, w[0], a.x * f.x * f.y), fmaf(f.z, w[1], a.y * f.x * f.y)),
                   bf16x2_bits(fmaf(f.z, w[2], a.z * f.x * f.y), fmaf(f.z, w[3], a.w * f.x * f.y)));
  *reinterpret_cast<uint2*>(p.out + at) = o;
}

// Ring depth and shared memory for `tokens` tokens.
int few_stages(int tp, bool nf4) {
  const int room = SMEM_MAX - 1024 - BAR_BYTES - epi_sets(nf4) * BUF_BYTES;
  return std::min(MAX_STAGES, room / (SUB * (W_BYTES + tp * BK * 2)));
}
int few_smem(const FewGrid& g, bool nf4) {
  return 1024 + g.stages * SUB * (W_BYTES + g.tp * BK * 2) + epi_sets(nf4) * BUF_BYTES + BAR_BYTES;
}

// contraction: that of a logit, K (0: the gradient's, which is not divided: its
// terms have both signs and its result is rounded to bf16).
FewGrid few_grid(int64_t tokens, int64_t contraction, bool nf4) {
  FewGrid g{};
  g.tp = static_cast<int>((tokens + 15) / 16 * 16);
  g.stages = few_stages(g.tp, nf4);
  g.parts = g.rounds = 1;
  if (contraction > 0) {
    // A logit's contraction fills several accumulators in turn, which the epilogue
    // adds up (the tensor core's additions truncate, see parts_of): as many as two
    // sets of them leave room for in TMEM, up to 8 of at least 256 of the
    // contraction, or 16 of 512.  Where these are too few for parts_of, it goes in
    // rounds, with room for one set's total.  (One round left errors of 2.5e-6 in the
    // losses of 128 tokens at K = 8192.  On 32000 entries, one round / three: 128
    // tokens, NF4 head, K = 4096 59.1 / 62.8 us; one / six: 128 tokens, bf16 head, K =
    // 8192 102 / 105 us, with the gradient 232 / 235 us.)
    const int64_t want = std::max(std::min<int64_t>((contraction + 255) / 256, 8),
                                  std::min<int64_t>((contraction + 511) / 512, 16));
    const int64_t need = parts_of(static_cast<int>(contraction));
    g.parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, 256 / g.tp)));
    if (g.parts < need) {
      g.parts = (512 / g.tp - 1) / 2;
      g.rounds = static_cast<int>((need + g.parts - 1) / g.parts);
    }
  }
  const int used = (2 * g.parts + (g.rounds > 1 ? 1 : 0)) * g.tp;
  g.cols = 32;
  while (g.cols < used) g.cols *= 2;
  return g;
}

template <int MODE, int KIND>
cudaError_t launch_kind(const CUtensorMap& w, const CUtensorMap& x, const FewGrid& g, const HeadEpi& p,
                        const HeadWeight& h, cudaStream_t st) {
  cudaError_t e = smem_limit_once<k_few<MODE, KIND>>(SMEM_MAX);
  if (e != cudaSuccess) return e;
  const int lg = block_log2(h.block);
  const int grid = std::min(g.tiles * g.nsplit, device_sm_count());
  return launch_ex(k_few<MODE, KIND>, dim3(grid), dim3(threads_of(KIND > 0)), few_smem(g, KIND > 0), st,
                   true, w, x, g, p, h.codes, h.absmax_q, h.dq_scale, host_codebook().levels, static_cast<int>(h.N),
                   static_cast<int>(h.K), lg, h.dq_block ? 1 : 0, device_status_ptr());
}
template <int MODE>
cudaError_t launch_few(const CUtensorMap& w, const CUtensorMap& x, const FewGrid& g, const HeadEpi& p,
                       const HeadWeight& h, cudaStream_t st) {
  if (h.W) return launch_kind<MODE, 0>(w, x, g, p, h, st);
  if (h.block == 64 && h.dq_block == 256) return launch_kind<MODE, 1>(w, x, g, p, h, st);
  return launch_kind<MODE, 2>(w, x, g, p, h, st);
}

const auto BF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
const auto SW128 = CU_TENSOR_MAP_SWIZZLE_128B;

}  // namespace

// Vocabulary entries per tile: the multiple of 8 up to 128 with which the CTAs'
// largest share of the head is smallest (32000 entries on 148 CTAs: two tiles of
// 112 each, instead of two of 128).
int few_tile_rows(int64_t N) {
  const int P = device_sm_count();
  int best = UM;
  int64_t cost = 0;
  for (int br = UM; br >= 32; br -= 8) {
    // a tile costs its rows, and its start and epilogue about what 16 rows cost (an
    // estimate, as is the 2 in few_splits)
    const int64_t c = ((N + br - 1) / br + P - 1) / P * (br + 16);
    if (br == UM || c < cost) {
      cost = c;
      best = br;
    }
  }
  return best;
}

int few_splits(int64_t N, int64_t K) {
  const int64_t tiles = (K + UM - 1) / UM, numK = (N + SUB * BK - 1) / (SUB * BK);
  const int P = device_sm_count();
  int best = 1;
  double cost = 0.0;
  for (int64_t S = 1; S <= std::min<int64_t>(std::max<int64_t>(numK / 4, 1), 64); ++S) {
    const double rounds = static_cast<double>((tiles * S + P - 1) / P);
    // rounds of S-ths of the vocabulary, each with its start and epilogue (about 2 stages)
    const double c = rounds * (static_cast<double>(numK) / static_cast<double>(S) + 2.0);
    if (S == 1 || c < cost) {
      cost = c;
      best = static_cast<int>(S);
    }
  }
  return best;
}

cudaError_t launch_few_logits(const HeadWeight& h, const uint16_t* X, int br, const HeadEpi& p, cudaStream_t st) {
  FewGrid g = few_grid(p.rows, h.K, !h.W);
  g.br = br;
  g.tiles = static_cast<int>((h.N + br - 1) / br);
  g.nsplit = 1;
  g.numK = static_cast<int>((h.K + SUB * BK - 1) / (SUB * BK));
  CUtensorMap w{}, x;
  if ((h.W && !make_map(&w, BF16, h.W, h.K, h.N, h.K * 2, BK, br, SW128)) ||
      !make_map(&x, BF16, X, h.K, p.rows, h.K * 2, BK, p.rows, SW128)) return cudaErrorInvalidValue;
  return launch_few<0>(w, x, g, p, h, st);
}

cudaError_t launch_few_grad(const HeadWeight& h, const uint16_t* P, int64_t ldp, int nsplit, const HeadEpi& p,
                            cudaStream_t st) {
  const int64_t rows = p.two_parts ? 2 * p.rows : p.rows;
  FewGrid g = few_grid(rows, 0, !h.W);
  g.br = UM;
  g.tiles = static_cast<int>((h.K + UM - 1) / UM);
  g.nsplit = nsplit;
  g.numK = static_cast<int>((h.N + SUB * BK - 1) / (SUB * BK));
  CUtensorMap w{}, x;
  if ((h.W && !make_map(&w, BF16, h.W, h.K, h.N, h.K * 2, 64, BK, SW128)) ||
      !make_map(&x, BF16, P, ldp, rows, ldp * 2, BK, rows, SW128)) return cudaErrorInvalidValue;
  const int lg = block_log2(h.block);
  cudaError_t e = launch_few<1>(w, x, g, p, h, st);
  if (e != cudaSuccess) return e;
  return launch_ex(k_few_join, dim3(static_cast<unsigned>((p.cols + 511) / 512), static_cast<unsigned>(p.rows)),
                   dim3(128), 0, st, true, static_cast<const float*>(p.split), nsplit, p, h.codes, h.absmax_q, h.dq_scale,
                   host_codebook().levels, lg, h.dq_block ? 1 : 0);
}

}  // namespace qn
