// The head losses: softmax cross entropy and distillation from a teacher's top
// logits, through a frozen output head W [N, K] (N = vocabulary, K = hidden
// width), with the gradient of the head's input X [M, K].
//
//   z = X W^T / T,  lse_i = log sum_j exp z_ij,  p_ij = exp(z_ij - lse_i)
//   loss_i = T^2 sum_s q_is (log q_is - (z_i,idx(s) - lse_i))
//   dX_i   = dloss_i T (sum_j p_ij w_j - sum_s q_is w_idx(s))
// with one target per row (q = 1, T = 1) for cross entropy, and the softmax of
// the teacher's kept logits over T for distillation.
//
// The logits never reach memory.  A product kernel (k_head<0>) leaves, for each
// row and each column segment of its tiles, a reference near the segment's
// maximum and the sum of exponentials relative to it, and the logits of the
// teacher's slots it meets, all in fp32 straight from the accumulator; k_head_stats
// joins them into lse and loss.  For the gradient the same kernel also writes e = exp(z) in bf16
// for a piece of the tokens, and k_head<1> multiplies e by W once lse is known:
// p = e exp(-lse) is a factor of the whole row, so it waits for the epilogue,
// and only the target columns of e change in between, because p - q from a rounded
// p would be noise for a confident token: the teacher's hold p - q, computed from
// their fp32 logits and rounded once (the largest stays in fp32).  A label stays out of e and of the sums: its
// p - 1 times its row of W is added in fp32 (it is most of the gradient, and p - 1
// is -1 for most tokens: rounded after the row's factor it alone made the error of
// dX 1.5 times that of a bf16 result), and the loss is log1p(exp(lse of the others
// - label's logit)), which keeps the digits of a small loss.  So a loss with its gradient costs two products and no pass over the
// exponentials.
//  - Computing p from the logits a second time would need three products.
//  - Keeping the logits themselves in bf16 would cost accuracy: a rounding error
//    of 2^-9 of a logit near 20 is 4 % of its p; the same rounding of e is 2^-9 of
//    p.
//  - e needs no maximum subtracted as long as it fits the exponent of bf16, which
//    is that of fp32: a segment whose maximum is within 2^-64 .. 2^64 is stored as
//    it is.  A segment outside (a logit past 44) is stored relative to its own
//    reference, and k_head_stats then brings the rows that have one to a common
//    reference, by exact powers of two.
#include <algorithm>
#include <atomic>

#include "head.h"

namespace qn {

namespace {

constexpr int UM = 128;      // token rows of each CTA of a pair
constexpr int TM = 2 * UM;   // token rows of a tile
constexpr int TN = 256;      // largest width of one accumulator (vocabulary entries or outputs)
constexpr int BK = 64;       // contraction per stage
constexpr int A_BYTES = UM * BK * 2;
constexpr int B_BYTES = TN / 2 * BK * 2;  // per accumulator
constexpr int RING_BYTES = 192 * 1024;    // 6 stages of 32 KB (NH = 1) or 4 of 48 KB (NH = 2)
constexpr int MAX_STAGES = 6;
constexpr int EPI_WARPS = 8;
constexpr int SEG = TN / 2;               // columns of a segment (one epilogue group's) of the logits
constexpr int E_BYTES = 32 * 64;          // 32 rows of 32 bf16 on their way out, two buffers per warp
constexpr int OFF_E = RING_BYTES;
constexpr int OFF_BAR = OFF_E + EPI_WARPS * 2 * E_BYTES;
constexpr int SMEM_ALLOC = OFF_BAR + 256 + 1024;  // slack for 1024-byte alignment
constexpr int NUM_THREADS = 64 + EPI_WARPS * 32;
constexpr int TMEM_COLS = 512;  // two accumulators of 256 columns
constexpr int kNoTarget = 0x7fffffff;

static_assert(SMEM_ALLOC <= 232448, "shared memory budget");

struct HeadBars {
  uint64_t full[MAX_STAGES];   // leader: both CTAs' tiles landed
  uint64_t empty[MAX_STAGES];  // MMAs of the stage completed (multicast by the leader)
  uint64_t acc_full[2];    // accumulator complete (multicast by the leader)
  uint64_t acc_empty[2];   // leader: both CTAs' epilogue warps have read it
  uint64_t drain;          // leader: used only when aborting
  uint64_t dealloc;        // the other CTA finished with the pair's TMEM
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(HeadBars) <= 256, "barrier block");

// Work items: whole tiles, then nsplit pieces (of the contraction) of each of
// the last ntail tiles, as in the fused NF4 GEMM.
struct HeadGrid {
  int mtiles, ntiles;         // token tiles of 256, output tiles of tn
  int nwhole, ntail, nsplit;
  int band;                   // token tiles walked together
  int nh;                     // accumulators per tile, side by side along the outputs (2: MODE 1 only)
  int bn;                     // outputs per accumulator (a multiple of 32; 256 in MODE 1)
  int tn;                     // outputs per tile, nh bn
  int sw;                     // outputs of the first of a tile's two column segments (one per epilogue group)
};

__device__ __forceinline__ void tile_of(const HeadGrid& g, int L, int& mt, int& nt) {
  const int per_band = g.band * g.ntiles;
  const int b = L / per_band, rem = L - b * per_band;
  const int in_band = min(g.band, g.mtiles - b * g.band);
  nt = rem / in_band;
  mt = b * g.band + (rem - nt * in_band);
}

// Two gradient values of a row with factors f (rscale): sums v0, v1 and a pair of
// bf16 of the label's row of W.
__device__ __forceinline__ uint32_t grad_pair(float v0, float v1, const float4& f, uint32_t w) {
  if (f.y == 0.0f) return 0u;
  return bf16x2_bits(fmaf(f.z, __uint_as_float(w << 16), v0 * f.x * f.y),
                     fmaf(f.z, __uint_as_float(w & 0xffff0000u), v1 * f.x * f.y));
}

// Arrival at a barrier of the other CTA that orders no memory of this thread: what
// it reports are TMEM loads, which have completed.  The releasing form waits for
// the thread's earlier stores first.
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// D = A B^T by pairs of CTAs (cta_group::2): 256 tokens x NH accumulators of up
// to 256 outputs per tile, each CTA holding 128 token rows and half of the
// output rows of each stage, both brought by TMA.  MODE 0: A = X, B = W
// (K-major).  MODE 1: A = p - q [rows, N], B = W with its rows as the
// contraction (MN-major).
//
// A persistent pair walks its items.  NH = 1: two accumulators alternate, so the
// epilogue of one runs under the products of the next.  NH = 2 (MODE 1): the two
// accumulators make one tile of 512 outputs, which brings a quarter fewer bytes
// from L2 per product.
//   warp 0     TMA producer
//   warp 1     TMEM allocation; the leader issues the MMAs
//   warps 2-9  epilogue in two groups of four, one column segment each, a warp
//              one TMEM lane quarter: a thread owns a token row
// Every wait is bounded; on expiry the kernel records kDevTimeout, drains what
// it issued, frees TMEM and returns.
template <int MODE, int NH>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_head(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
           const __grid_constant__ CUtensorMap tm_e, int numK, HeadGrid g, HeadEpi p, int* status) {
  constexpr int STAGE_BYTES = A_BYTES + NH * B_BYTES;
  constexpr int STAGES = RING_BYTES / STAGE_BYTES;
  static_assert(STAGES <= MAX_STAGES, "barrier block");
  // The last kernel of a call lets nothing start early: whatever follows waits for
  // its outputs first.
  if (MODE == 0 || g.ntail > 0) pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  HeadBars* bars = reinterpret_cast<HeadBars*>(smem_raw + (base - raw) + OFF_BAR);
  const uint32_t bar0 = base + OFF_BAR;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
  auto acc_full = [&](int a) { return bar0 + 8u * (2 * MAX_STAGES + a); };
  auto acc_empty = [&](int a) { return bar0 + 8u * (2 * MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * MAX_STAGES + 4);
  const uint32_t dealloc_bar = drain_bar + 8u;
  volatile int* abort = &bars->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0 = leader, 1 = peer
  const bool leader = rank == 0;
  const int bnl = g.bn >> 1;
  const int nitems = g.nwhole + g.ntail * g.nsplit;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  // Item i: its tile, and the stages [kbeg, kend) of the contraction it covers.
  auto item = [&](int i, int& mt, int& nt, int& kbeg, int& kend, int& tail, int& z) {
    int L = i;
    tail = -1;
    z = 0;
    kbeg = 0;
    kend = numK;
    if (i >= g.nwhole) {
      const int j = i - g.nwhole;
      tail = j / g.nsplit;
      z = j - tail * g.nsplit;
      L = g.nwhole + tail;
      kbeg = static_cast<int>(static_cast<int64_t>(z) * numK / g.nsplit);
      kend = static_cast<int>(static_cast<int64_t>(z + 1) * numK / g.nsplit);
    }
    tile_of(g, L, mt, nt);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full(a), 1);
      // NH = 1: both groups read each accumulator; NH = 2: one group each
      mbar_init(acc_empty(a), 2 * EPI_WARPS / NH);
    }
    mbar_init(drain_bar, 1);
    mbar_init(dealloc_bar, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(bar0 + static_cast<uint32_t>(offsetof(HeadBars, tmem_base)), TMEM_COLS);
    tmem_relinquish_pair();
  }
  pdl_wait();  // everything above is local to the pair
  tc_fence_before();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0) {
    // --------------------------------------------------------- TMA producer
    const uint32_t bytes = 2 * (UM + NH * bnl) * static_cast<uint32_t>(BK * 2);  // of both CTAs
    const uint32_t full_at_leader = mapa_shared(full(0), 0);
    bool ok = true, issued = false;
    RingPos r;
    for (int i = first; i < nitems && ok; i += step) {
      int mt, nt, kbeg, kend, tail, z;
      item(i, mt, nt, kbeg, kend, tail, z);
      const int m0 = mt * TM + static_cast<int>(rank) * UM, n0 = nt * g.tn + static_cast<int>(rank) * bnl;
      for (int k = kbeg; k < kend; ++k, r.advance(1, STAGES)) {
        if (!(ok = wait_warp(empty(r.slot), r.phase ^ 1, abort, status))) break;
        issued = true;
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(full(r.slot), bytes);
          const uint32_t bar = full_at_leader + 8u * r.slot, a_s = base + r.slot * STAGE_BYTES, b_s = a_s + A_BYTES;
          tma_load_2d_pair(a_s, &tm_a, bar, k * BK, m0);
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            if (MODE == 0) {
              tma_load_2d_pair(b_s + h * B_BYTES, &tm_b, bar, k * BK, n0 + h * TN);
            } else {
              tma_load_2d_pair(b_s + h * B_BYTES, &tm_b, bar, n0 + h * TN, k * BK);
              tma_load_2d_pair(b_s + h * B_BYTES + 8192, &tm_b, bar, n0 + h * TN + 64, k * BK);
            }
          }
        }
        __syncwarp();
      }
    }
    // Let the copies already issued land before the CTA exits.  They report to
    // the leader, which cannot see the end of a stage that only one CTA has
    // issued, so each CTA gives its own the time they can need at most.
    if (!ok && issued) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 20000000ull) {
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    if (leader) {
      const uint32_t idesc = idesc_bf16(TM, g.bn, false, MODE == 1);
      bool ok = true, committed = false;
      RingPos r;
      int t = 0;  // accumulators filled so far
      for (int i = first; i < nitems && ok; i += step) {
        int mt, nt, kbeg, kend, tail, z;
        item(i, mt, nt, kbeg, kend, tail, z);
        const int parts = MODE == 0 ? parts_of((kend - kbeg) * BK) : 1;
        for (int q = 0, k = kbeg; q < parts && ok; ++q, ++t) {
          const int stop = kbeg + (q + 1) * (kend - kbeg) / parts, start = k;
          if (NH == 1) {
            ok = wait_warp_cluster(acc_empty(t & 1), ((t >> 1) & 1) ^ 1, abort, status);
          } else {
            ok = wait_warp_cluster(acc_empty(0), (t & 1) ^ 1, abort, status) &&
                 wait_warp_cluster(acc_empty(1), (t & 1) ^ 1, abort, status);
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = NH == 1 ? tmem + 256u * (t & 1) : tmem;
          for (; k < stop; ++k, r.advance(1, STAGES)) {
            if (!(ok = wait_warp_cluster(full(r.slot), r.phase, abort, status))) break;
            tc_fence_after();
            const uint32_t a_s = base + r.slot * STAGE_BYTES, b_s = a_s + A_BYTES;
            const uint64_t ad = desc_sw128(a_s, 16, 1024);
            const uint64_t bd = MODE == 0 ? desc_sw128(b_s, 16, 1024) : desc_sw128(b_s, 8192, 1024);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk) {  // a descriptor's low bits are the address / 16
                const uint64_t a_k = ad + kk * 2, b_k = bd + kk * (MODE == 0 ? 2 : 128);
                const uint32_t more = (k > start || kk > 0) ? 1u : 0u;
                if (NH == 1) {
                  tc_mma_f16_pair(d, a_k, b_k, idesc, more);
                } else {
                  tc_mma_f16_pair_fill_a(d, a_k, b_k, idesc, more);
                  tc_mma_f16_pair_last_a(d + 256u, a_k, b_k + B_BYTES / 16, idesc, more);
                }
              }
              tc_commit_pair(empty(r.slot));
            }
            __syncwarp();
            committed = true;
          }
          if (ok && elect_one()) {
            if (NH == 1) {
              tc_commit_pair(acc_full(t & 1));
            } else {
              tc_commit_pair(acc_full(0));
              tc_commit_pair(acc_full(1));
            }
          }
          __syncwarp();
        }
      }
      if (!ok && committed && elect_one()) {  // wait for MMAs in flight before TMEM is freed
        tc_commit_pair(drain_bar);
        wait_drain(drain_bar, 0);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3;         // TMEM lanes 32 quad .. 32 quad + 31
    const int h = (warp - 2) >> 2;     // column segment
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t empty_at_leader = mapa_shared(acc_empty(0), 0);
    const int cseg = h * g.sw;                         // the segment's first column in the tile
    const int cwidth = h == 0 ? g.sw : g.tn - g.sw;    // and its width
    const uint32_t e_buf = base + OFF_E + static_cast<uint32_t>(warp - 2) * 2 * E_BYTES;
    int t = 0, stored = 0;
    // Waits for the next accumulator, and gives it back.
    auto take = [&](int& a) {
      a = NH == 1 ? (t & 1) : h;
      const bool landed = wait_warp(acc_full(a), NH == 1 ? (t >> 1) & 1 : t & 1, abort, status);
      ++t;
      tc_fence_after();
      return landed;
    };
    auto give = [&](int a) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(acc_empty(a));
        else arrive_remote_relaxed(empty_at_leader + 8u * a);
      }
    };
    bool ok = true;
    for (int i = first; i < nitems && ok; i += step) {
      int mt, nt, kbeg, kend, tail, zp;
      item(i, mt, nt, kbeg, kend, tail, zp);
      const int row0 = mt * TM + static_cast<int>(rank) * UM + quad * 32;  // the warp's first row
      const int row = row0 + lane;
      const int n0 = nt * g.tn + cseg;  // the segment's first output
      const bool used = row0 < p.rows, live = row < p.rows;
      int a;
      if (MODE == 0) {
        const int ncols = max(0, min(cwidth, p.cols - n0));
        // The row's label in this segment, or its teacher's slots in ascending order.
        int label = kNoTarget, first_t = 0, end_t = 0;
        if (live && p.labels) {
          const int64_t y = p.labels[row] - n0;
          if (y >= 0 && y < ncols) label = static_cast<int>(y);
        } else if (live) {
          const uint16_t* o = p.off + static_cast<int64_t>(row) * (2 * g.ntiles + 1) + 2 * nt + h;
          first_t = o[0];
          end_t = o[1];
        }
        float z[SEG];
        const int parts = parts_of((kend - kbeg) * BK);
        for (int q = 0; q < parts; ++q) {
          if (!(ok = take(a))) break;
          const uint32_t acc = tmem + lane_base + 256u * a + cseg;
          if (used) {
#pragma unroll
            for (int c = 0; c < SEG; c += 16) {
              if (c < cwidth) {
                uint32_t v[16];
                tmem_ld_x16(acc + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  z[c + j] = q == 0 ? __uint_as_float(v[j]) : z[c + j] + __uint_as_float(v[j]);
              }
            }
          }
          give(a);  // the rest runs beside the products of the next accumulator
        }
        if (!ok) break;
        if (!used) continue;
        if (ncols < SEG) {
#pragma unroll
          for (int j = 0; j < SEG; ++j)
            if (j >= ncols) z[j] = -INFINITY;
        }
        if (__any_sync(0xffffffffu, label != kNoTarget)) {
#pragma unroll
          for (int j = 0; j < SEG; ++j)
            if (label == j) z[j] = -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < SEG; ++j) mx = fmaxf(mx, z[j]);
        // The segment's reference in units of log2 is a whole number, so taking it
        // off and putting it back are exact.  (A segment whose logits are all -inf,
        // times 1 / T, or NaN has none and is summed around 0.)
        const float top = rintf(mx * p.c), ref = top == -INFINITY ? 0.0f : top;
        const float back = exp2f(fabsf(ref) <= kHeadFits ? ref : 0.0f);  // e is stored relative to 0, or to ref
        const __nv_bfloat162 back2 = __float2bfloat162_rn(back);
        // The teacher's slots, from the registers: only a warp with a slot in this
        // segment looks for them.
        if (__any_sync(0xffffffffu, first_t < end_t)) {
          const int* idx = p.sidx + static_cast<int64_t>(row) * p.k;
          int cur = first_t, want = cur < end_t ? idx[cur] - n0 : kNoTarget;
#pragma unroll
          for (int j = 0; j < SEG; ++j) {
            while (want == j) {  // more than once for an entry in several slots
              p.ztgt[static_cast<int64_t>(row) * p.k + cur] = make_float2(fmaf(z[j], p.c, -ref), ref);
              ++cur;
              want = cur < end_t ? idx[cur] - n0 : kNoTarget;
            }
          }
        }
        float sum = 0.0f;
        const int ewidth = static_cast<int>(min(static_cast<int64_t>(cwidth), p.lde - n0));
#pragma unroll
        for (int col = 0; col < SEG; col += 32) {
          if (col >= ewidth) break;
          float* e = z + col;
#pragma unroll
          for (int j = 0; j < 32; ++j) e[j] = exp2_fast(fmaf(e[j], p.c, -ref));
          if (p.e) {
            // 32 rows x 32 columns through shared memory (64-byte swizzle) and out by
            // TMA: written from the registers, every 16 bytes of a lane would be a
            // line of their own.  Rows past the piece are not written.
            const uint32_t buf = e_buf + static_cast<uint32_t>(stored & 1) * E_BYTES;
            if (lane == 0) bulk_wait_read<1>();  // the store before the last has left this buffer
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 x = __hmul2(__floats2bfloat162_rn(e[8 * q + 2 * j], e[8 * q + 2 * j + 1]), back2);
                w[j] = *reinterpret_cast<const uint32_t*>(&x);
              }
              st_shared_v4(buf + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tm_e, buf, n0 + col, row0);
              bulk_commit();
            }
            ++stored;
          }
          // As a tree: a column with p near 1 then meets the small rest in 9
          // additions at most per segment, not in one for each of them (a loss of
          // 1e-5 is the difference of the sum from 1).
#pragma unroll
          for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int j = 0; j < d; ++j) e[j] += e[j + d];
          sum += e[0];
        }
        if (p.e && live && h == 1 && nt == g.ntiles - 1)  // the pitch may reach past the last tile
          for (int64_t col = n0 + cwidth; col < p.lde; col += 8)
            *reinterpret_cast<uint4*>(p.e + static_cast<int64_t>(row) * p.lde + col) = make_uint4(0u, 0u, 0u, 0u);
        if (live)
          p.part[(2 * static_cast<int64_t>(nt) + h) * p.rows + row] = make_float2(top, sum);
      } else {
        const float4 f = live && tail < 0 ? p.rscale[row] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int label = live && tail < 0 ? __float_as_int(f.w) : -1;
        const int width = min(cwidth, p.cols - n0);  // a multiple of 64, as both are; may be negative
        const uint16_t* wl = label >= 0 ? p.W + static_cast<int64_t>(label) * p.cols + n0 : nullptr;
        // The label's row of W, 64 columns at a time and 64 ahead of their use (the
        // first before the accumulator is complete): a row per lane takes a
        // microsecond to come.
        auto fetch = [&](int col, uint4 (&w)[8]) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            w[q] = wl && col < width ? ldg_nc_v4(wl + col + 8 * q) : make_uint4(0u, 0u, 0u, 0u);
        };
        uint4 w0[8], w1[8];
        fetch(0, w0);
        fetch(64, w1);
        if (!(ok = take(a))) break;
        const uint32_t acc = tmem + lane_base + (NH == 1 ? 256u * a + cseg : 256u * h);
        auto emit = [&](int col, const uint4 (&w)[8]) {
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const int at = col + 32 * part;
            uint32_t v[32];
            tmem_ld_32x32b_x32(acc + at, v);
            tmem_ld_wait();
            if (tail >= 0) {  // a piece of a split tile: fp32 sums, joined by k_head_join
              float4* dst = reinterpret_cast<float4*>(
                  p.split + ((static_cast<int64_t>(tail) * g.nsplit + zp) * TM + rank * UM + quad * 32 + lane) * g.tn +
                  cseg + at);
#pragma unroll
              for (int q = 0; q < 8; ++q)
                dst[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                     __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
            } else if (live) {
              uint4* dst = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(row) * p.cols + n0 + at);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint4 x = w[4 * part + q];
                const uint32_t wq[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  o[j] = grad_pair(__uint_as_float(v[8 * q + 2 * j]), __uint_as_float(v[8 * q + 2 * j + 1]), f, wq[j]);
                dst[q] = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
          }
        };
        if (used) {
#pragma unroll 1
          for (int col = 0; col < width; col += 128) {
            emit(col, w0);
            fetch(col + 128, w0);
            if (col + 64 < width) emit(col + 64, w1);
            fetch(col + 192, w1);
          }
        }
        give(a);
      }
    }
    if (MODE == 0 && lane == 0) bulk_wait_all();  // the stores have left shared memory and are visible
  }

  // Both CTAs must be done with the pair's TMEM, and with each other's
  // barriers, before either leaves: each tells the other and waits (bounded).
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) {
      mbar_arrive_remote(mapa_shared(dealloc_bar, rank ^ 1u));
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait_cluster(dealloc_bar, 0)) {
        if (global_timer_ns() - t0 > 2 * kWaitLimitNs) {
          atomicExch(status, kDevTimeout);
          break;
        }
      }
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// Sum of the pieces of the split gradient tiles in piece order, times the row's
// factor, rounded once to bf16.  Thread: 8 consecutive outputs of a row.
__global__ void __launch_bounds__(256) k_head_join(const float* __restrict__ split, HeadGrid g, HeadEpi p) {
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int groups = g.tn / 8, per_tile = TM * groups;
  const int t = static_cast<int>(i / per_tile), w = static_cast<int>(i % per_tile);
  if (t >= g.ntail) return;
  const int r = w / groups, c = (w % groups) * 8;
  int mt, nt;
  tile_of(g, g.nwhole + t, mt, nt);
  const int row = mt * TM + r, n = nt * g.tn + c;
  if (row >= p.rows || n >= p.cols) return;
  const float* src = split + (static_cast<int64_t>(t) * g.nsplit * TM + r) * g.tn + c;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
#pragma unroll 4
  for (int z = 0; z < g.nsplit; ++z) {
    const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + 4);
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
    src += TM * g.tn;
  }
  const float4 f = p.rscale[row];
  const int label = __float_as_int(f.w);
  uint4 lw = make_uint4(0u, 0u, 0u, 0u);
  if (label >= 0) lw = ldg_nc_v4(p.W + static_cast<int64_t>(label) * p.cols + n);
  *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(row) * p.cols + n) =
      make_uint4(grad_pair(a.x, a.y, f, lw.x), grad_pair(a.z, a.w, f, lw.y), grad_pair(b.x, b.y, f, lw.z),
                 grad_pair(b.z, b.w, f, lw.w));
}

// The teacher's slots of one row per block: the softmax of the kept logits over
// T (as logarithms), in ascending order of their vocabulary index (ties in slot
// order), and where each column segment's targets begin.  A slot whose index
// is outside [0, N) or whose logit is -inf holds nothing: it sorts last.  k is
// at most 256, so each thread ranks its slot by comparing it with the others.
constexpr int TARGET_THREADS = 128;
template <typename T>
__global__ void __launch_bounds__(TARGET_THREADS) k_head_targets(const int64_t* __restrict__ idx, const T* __restrict__ logit,
                                                      int k, int N, float inv_t, int tn, int sw, int nseg,
                                                      int* __restrict__ sidx, float* __restrict__ logq,
                                                      uint16_t* __restrict__ off) {
  pdl_trigger();
  pdl_wait();
  __shared__ int key[256], sorted[256];
  __shared__ float val[256];
  const int64_t row = blockIdx.x;
  const int s = threadIdx.x;
  for (int j = s; j < k; j += TARGET_THREADS) {
    const int64_t y = idx[row * k + j];
    const float x = static_cast<float>(logit[row * k + j]);
    const bool kept = y >= 0 && y < N && x != -INFINITY;
    key[j] = kept ? static_cast<int>(y) : kNoTarget;
    val[j] = x;
  }
  __syncthreads();
  // maximum and sum over the block, in a fixed order
  __shared__ float red[2][4];
  const int lane = s & 31, warp = s >> 5;
  float mx = -INFINITY, sum = 0.0f;
  for (int j = s; j < k; j += TARGET_THREADS)
    if (key[j] != kNoTarget) mx = fmaxf(mx, val[j]);
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  if (lane == 0) red[0][warp] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  for (int j = s; j < k; j += TARGET_THREADS)
    if (key[j] != kNoTarget) sum += expf((val[j] - mx) * inv_t);
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) red[1][warp] = sum;
  __syncthreads();
  sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  const float lsum = logf(sum);
  for (int j = s; j < k; j += TARGET_THREADS) {
    const int mine = key[j];
    int rank = 0;
    for (int o = 0; o < k; ++o) rank += (key[o] < mine || (key[o] == mine && o < j)) ? 1 : 0;
    sorted[rank] = mine;
    sidx[row * k + rank] = mine;
    logq[row * k + rank] = mine == kNoTarget ? -INFINITY : (val[j] - mx) * inv_t - lsum;
  }
  __syncthreads();
  for (int t = s; t <= nseg; t += TARGET_THREADS) {
    const int64_t bound = min(static_cast<int64_t>(t >> 1) * tn + (t & 1) * sw, static_cast<int64_t>(N));
    int lo = 0, hi = k;  // first slot with sorted >= bound
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < bound) lo = mid + 1;
      else hi = mid;
    }
    off[row * (nseg + 1) + t] = static_cast<uint16_t>(lo);
  }
}

constexpr float kLn2 = 0.69314718055994530942f;

// Factor that takes a sum of exponentials from reference x to reference top.
__device__ __forceinline__ float shift2(float x, float top) { return x == -INFINITY ? 0.0f : exp2f(x - top); }

// A row's log2 of the sum of exponentials, m + l2s, and the reference r that its
// stored exponentials have.  The parts stay apart: their sum would round off
// digits of z - lse.
struct RowStat {
  float m, l2s, r;
};

// Writes p - q, relative to reference r, into the columns of the row's teacher
// slots (one warp per row; what the rounding leaves into el, if given), all but the
// largest one: that one stays in fp32 (*d, and its entry as the result) and is added
// in the gradient's epilogue as a label's is.
// (The slots' rounding to bf16 alone makes the error of dX 1.4 times that of a bf16
// result, and the largest slot has most of it.)
__device__ __forceinline__ int write_targets(uint16_t* er, uint16_t* el, const RowStat& st, int lane, int row,
                                             const int* sidx, const float* logq, int k, const float2* ztgt,
                                             float* d_out) {
  const float up = exp2f((st.m - st.r) + st.l2s);
  const int64_t at = static_cast<int64_t>(row) * k;
  float best = 0.0f;
  int entry = -1;
  for (int j = lane; j < k; j += 32) {
    const int y = sidx[at + j];
    if (y == kNoTarget) break;
    if (j > 0 && sidx[at + j - 1] == y) continue;  // the first of equal entries takes them all
    const float2 z = ztgt[at + j];
    float d = exp2f((z.x + (z.y - st.m)) - st.l2s);
    for (int o = j; o < k && sidx[at + o] == y; ++o) d -= expf(logq[at + o]);
    const uint32_t hi = bf16x2_bits(d * up, 0.0f);
    er[y] = static_cast<uint16_t>(hi);
    if (el) el[y] = static_cast<uint16_t>(bf16x2_bits(d * up - __uint_as_float(hi << 16), 0.0f));
    if (fabsf(d) > fabsf(best)) {
      best = d;
      entry = y;
    }
  }
  // the largest over the warp, the lowest entry among equals
  float d = best;
  int y = entry;
  for (int o = 16; o > 0; o >>= 1) {
    const float d2 = __shfl_xor_sync(0xffffffffu, d, o);
    const int y2 = __shfl_xor_sync(0xffffffffu, y, o);
    if (fabsf(d2) > fabsf(d) || (fabsf(d2) == fabsf(d) && y2 >= 0 && (y < 0 || y2 < y))) {
      d = d2;
      y = y2;
    }
  }
  if (y >= 0 && entry == y) {
    er[y] = 0;
    if (el) el[y] = 0;
  }
  *d_out = d;
  return y;
}

// What k_head_stats reads and writes.
struct StatArgs {
  const float2* part;  // [nseg][rows]
  int nseg, rows, N, K;
  const int64_t* labels;           // cross entropy, with
  const uint16_t *X, *W;           //   the label's logit computed here from these, or (null)
  const float* zlabel;             //   taken from here
  const int* sidx;                 // distillation
  const float* logq;
  int k;
  const float2* ztgt;
  float c, temp;
  const float* dloss;
  float *loss, *lse;
  float4* rscale;
  uint16_t* e;  // null: no gradient
  uint16_t* e_low;  // the second part of a teacher's p - q (nullable)
  int64_t lde;
  int tn, sw;   // column segments of e (see Segments)
};

__device__ __forceinline__ uint32_t scale_pair(uint32_t v, float f) {
  return bf16x2_bits(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
}

// Brings a row that holds a segment with its own reference to the common one, r,
// by powers of two (one warp; such rows are rare, and if all are, their warps
// together are bound by HBM like any other pass).
__device__ __noinline__ void rescale_row(const StatArgs& p, int row, float r, int lane) {
  uint4* v = reinterpret_cast<uint4*>(p.e + row * p.lde);
  const int n = static_cast<int>(p.lde / 8), per_tile = p.tn / 8, per_seg = p.sw / 8;
  for (int c = lane; c < n; c += 32) {
    const int q = c / per_tile, t = min(2 * q + (c - q * per_tile >= per_seg ? 1 : 0), p.nseg - 1);
    const float ref = p.part[static_cast<int64_t>(t) * p.rows + row].x;
    const float f = exp2f((fabsf(ref) <= kHeadFits ? 0.0f : ref) - r);
    uint4 x = v[c];
    x.x = scale_pair(x.x, f);
    x.y = scale_pair(x.y, f);
    x.z = scale_pair(x.z, f);
    x.w = scale_pair(x.w, f);
    v[c] = x;
  }
  __syncwarp();
}

// Joins the segments' (reference, sum) pairs of SROWS rows per block: first thread
// (r, j) takes row r and segments j, j + SLANES, ..., then warp r joins its row's
// values, adds the label's logit or the teacher's terms of the loss, and writes the
// teacher's columns of e.  The orders are fixed.  The label's logit is one more dot
// product of X and W with fp32 additions rounded to nearest (12 us for 4096 x 4096,
// read from HBM; few tokens: beside k_few's products): the tensor core's truncating
// sum alone made the loss of 2047 x 50003 x 2048 1.4e-6 off instead of 4e-7.
// 16 rows per block where there are many (4096 tokens: 18 us, with 8 21 us), 4 where
// a row's chain of segments counts.
constexpr int STAT_THREADS = 512;
template <int SROWS>
__global__ void __launch_bounds__(STAT_THREADS) k_head_stats(const __grid_constant__ StatArgs p) {
  constexpr int SLANES = STAT_THREADS / SROWS;
  if (p.e) pdl_trigger();  // without a gradient this is the call's last kernel
  pdl_wait();
  __shared__ float2 sh[SROWS][SLANES + 1];
  __shared__ int own[SROWS];
  const int row0 = blockIdx.x * SROWS;
  float m = -INFINITY, s = 0.0f;
  bool big = false;
  const int r = threadIdx.x % SROWS, seg0 = threadIdx.x / SROWS;
  if (threadIdx.x < SROWS) own[threadIdx.x] = 0;
  __syncthreads();
  if (row0 + r < p.rows) {
#pragma unroll 4
    for (int t = seg0; t < p.nseg; t += SLANES) {
      const float2 v = p.part[static_cast<int64_t>(t) * p.rows + row0 + r];
      const float top = fmaxf(m, v.x);
      s = s * shift2(m, top) + v.y * shift2(v.x, top);
      m = top;
      big = big || (fabsf(v.x) > kHeadFits && v.x != -INFINITY);
    }
  }
  sh[r][seg0] = make_float2(m, s);
  if (big) own[r] = 1;
  __syncthreads();
  const int a = threadIdx.x & 31, b = threadIdx.x >> 5;
  const int row = row0 + b;
  if (b >= SROWS || row >= p.rows) return;
  m = -INFINITY;
#pragma unroll
  for (int j = a; j < SLANES; j += 32) m = fmaxf(m, sh[b][j].x);
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  s = 0.0f;
#pragma unroll
  for (int j = a; j < SLANES; j += 32) s += sh[b][j].y * shift2(sh[b][j].x, m);
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  big = own[b] != 0;
  RowStat st{m, 0.0f, big ? m : 0.0f};
  float total = 0.0f, d = 0.0f;  // the loss / T^2, and the label's p - 1
  bool any = false;
  int label = -1;
  if (p.labels) {
    const int64_t y = p.labels[row];
    any = y >= 0 && y < p.N;
    if (any) {
      label = static_cast<int>(y);
      const float z = p.X ? dot_row(p.X + static_cast<int64_t>(row) * p.K, p.W + y * p.K, p.K, a) : p.zlabel[row];
      const float2 zn = log2_parts(z, p.c);
      const float zy = zn.x, ny = zn.y;  // the label's logit times c, relative to ny
      // log2 of p / (1 - p): the sums hold the other entries alone.  (A label at -inf
      // has p = 0 and the loss +inf; if the others are there too, NaN.)
      const float odds = (zy + (ny - m)) - log2f(s);
      total = log1pf(exp2f(-fabsf(odds))) + (odds < 0.0f ? -odds * kLn2 : 0.0f);
      d = expm1f(-total);
      const float top = fmaxf(m, ny);
      s = s * shift2(m, top) + (ny == -INFINITY ? 0.0f : exp2f(zy + (ny - top)));
      st.m = top;
    }
    st.l2s = log2f(s);
  } else {
    // loss = T^2 sum_s q_s (log q_s + (lse - z_s)); lse - z_s in units of log2 is
    // (m - n) - (z - n) + log2(sum), which keeps the digits of a small loss.
    st.l2s = log2f(s);
    const int64_t at = static_cast<int64_t>(row) * p.k;
    any = p.sidx[at] != kNoTarget;
    for (int j = a; j < p.k; j += 32) {
      if (p.sidx[at + j] == kNoTarget) break;
      const float lq = p.logq[at + j], q = expf(lq);
      const float2 z = p.ztgt[at + j];
      if (q != 0.0f) total += q * (lq + (((m - z.y) - z.x) + st.l2s) * kLn2);
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  const float g = any ? (p.dloss ? p.dloss[row] : 1.0f) * p.temp : 0.0f;
  if (p.e && g != 0.0f) {  // otherwise the row's gradient is written as zeros
    if (big) rescale_row(p, row, st.r, a);
    if (!p.labels)
      label = write_targets(p.e + row * p.lde, p.e_low ? p.e_low + row * p.lde : nullptr, st, a, row, p.sidx, p.logq,
                            p.k, p.ztgt, &d);
  }
  if (a == 0) {
    p.loss[row] = any ? total * (p.temp * p.temp) : 0.0f;
    p.lse[row] = (st.m + st.l2s) * kLn2;
    if (p.e) {
      p.rscale[row] = make_float4(exp2f(-((st.m - st.r) + st.l2s)), g, d * g, __int_as_float(label));
    }
  }
}

// ------------------------------------------------------------ host side

cudaLaunchConfig_t pair_config(int pairs, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_ALLOC;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Pairs of CTAs resident at once on the current device (0: unknown).
int head_pairs() {
  constexpr int kDev = 64;
  static std::atomic<int> cache[kDev];  // 0: not yet asked; -1: unknown
  int d = -1;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kDev) {
    cudaGetLastError();
    return 0;
  }
  int v = cache[d].load(std::memory_order_relaxed);
  if (v == 0) {
    cudaLaunchAttribute attr[2];
    int a = 0, b = 0;
    const cudaLaunchConfig_t cfg = pair_config(1, nullptr, attr);
    if (smem_limit_once<k_head<0, 1>>(SMEM_ALLOC) == cudaSuccess &&
        smem_limit_once<k_head<1, 1>>(SMEM_ALLOC) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&a, k_head<0, 1>, &cfg) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&b, k_head<1, 1>, &cfg) == cudaSuccess && std::min(a, b) > 0) {
      v = std::min(a, b);
    } else {
      cudaGetLastError();
      v = -1;
    }
    cache[d].store(v, std::memory_order_relaxed);
  }
  return v > 0 ? v : 0;
}

// Token tiles walked together: their A rows (256 rows of the contraction each)
// stay near 48 MB, so they stay in L2 while the other operand streams past.
int band_of(int64_t mtiles, int64_t contraction) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(mtiles, (48ll << 20) / (TM * contraction * 2))));
}

// Tiles of the logits product.  Their width is the one whose rounds over the
// resident pairs cost least, 256 if nothing is clearly better.  A stage of a
// tile costs the bytes a CTA brings from L2 for it (128 token rows and bn / 2 of
// the head): a pair's MMA of width 256 takes 512 cycles per stage, and its 32 KB
// per CTA are 64 B per cycle, about what L2 delivers, so narrower tiles only pay
// where they save a round.  With a single token tile the head's rows alone count
// (they come from HBM): 32000 entries are two rounds of 256 on 74 pairs, or two
// of 224.
HeadGrid logits_grid(int64_t rows, int64_t N, int64_t K) {
  HeadGrid g{};
  g.mtiles = static_cast<int>((rows + TM - 1) / TM);
  g.bn = TN;
  const int P = head_pairs();
  g.nh = 1;
  if (P > 0) {
    double best = 0.0;
    for (int bn = TN; bn >= 128; bn -= 32) {
      const int64_t rounds = (g.mtiles * ((N + bn - 1) / bn) + P - 1) / P;
      const double cost = static_cast<double>(rounds) * (g.mtiles == 1 ? bn : UM + bn / 2);
      if (bn == TN || cost < 0.97 * best) {
        best = cost;
        g.bn = bn;
      }
    }
  }
  g.tn = g.nh * g.bn;
  g.sw = std::min(g.bn, SEG);
  g.ntiles = static_cast<int>((N + g.tn - 1) / g.tn);
  g.nwhole = g.mtiles * g.ntiles;
  g.nsplit = 1;
  g.band = band_of(g.mtiles, K);
  return g;
}

// Tiles of the gradient product of width 256 nh; the tiles of a partial last
// wave are split along the vocabulary where that saves time.  *cost: estimated
// time in stages of a 256-wide tile.
HeadGrid grad_tiles(int64_t rows, int64_t N, int64_t K, int nh, double* cost) {
  HeadGrid g{};
  g.mtiles = static_cast<int>((rows + TM - 1) / TM);
  g.bn = TN;
  g.nh = nh;
  g.tn = nh * TN;
  g.sw = g.tn / 2;
  g.ntiles = static_cast<int>((K + g.tn - 1) / g.tn);
  g.nwhole = g.mtiles * g.ntiles;
  g.nsplit = 1;
  g.band = g.mtiles;
  const int64_t numK = (N + BK - 1) / BK;
  const int P = head_pairs();
  *cost = 0.0;
  if (P <= 0) return g;
  // Two accumulators side by side bring 48 KB per CTA for twice the products of
  // 32 KB: 2.79 against 2.99 ms for 2048 x 128000 x 8192, where both divide the
  // pairs alike.
  const double stage = nh == 2 ? 1.87 : 1.0;
  const int64_t w = g.nwhole % P, full = g.nwhole / P;
  double tail = w ? static_cast<double>(numK) * stage : 0.0;
  // Split in S, the w tiles of the last wave take ceil(w S / P) rounds of S-ths;
  // their fp32 sums (256 KB per piece and accumulator, written and read again)
  // cost about 0.2 of a stage each, and every round the filling and emptying of
  // the pipeline, about 8 (both are estimates).
  for (int64_t S = 2; w && S <= std::min<int64_t>(numK / 8, 64); ++S) {
    const double rounds = static_cast<double>((w * S + P - 1) / P);
    const double t = rounds / static_cast<double>(S) * static_cast<double>(numK) * stage +
                     0.2 * nh * static_cast<double>(w * S) + 8.0 * nh * rounds;
    if (t < tail) {
      tail = t;
      g.nsplit = static_cast<int>(S);
    }
  }
  if (g.nsplit > 1) {
    g.ntail = static_cast<int>(w);
    g.nwhole -= g.ntail;
  }
  *cost = static_cast<double>(full) * static_cast<double>(numK) * stage + tail;
  return g;
}
// The cheaper width's tiles.  A call asks for them several times (the workspace's
// layout and the launch), and finding them takes a microsecond or two: the last
// answer is kept per host thread.
HeadGrid grad_grid(int64_t rows, int64_t N, int64_t K) {
  struct Plan {
    int64_t rows = -1, N = 0, K = 0;
    int pairs = 0;
    HeadGrid g{};
  };
  thread_local Plan last;
  const int P = head_pairs();
  if (last.rows != rows || last.N != N || last.K != K || last.pairs != P) {
    double one = 0.0, two = 0.0;
    const HeadGrid a = grad_tiles(rows, N, K, 1, &one), b = grad_tiles(rows, N, K, 2, &two);
    last.g = two < one ? b : a;
    last.rows = rows;
    last.N = N;
    last.K = K;
    last.pairs = P;
  }
  return last.g;
}

// The column segments of a piece's statistics: the first of a tile's two has sw
// columns, a tile tn.
struct Segments {
  int tn, sw, count;
};
Segments segments(int64_t rows, int64_t N, int64_t K) {
  if (rows <= kHeadFewTokens) {
    const int br = few_tile_rows(N);
    return {2 * br, br, static_cast<int>((N + br - 1) / br)};
  }
  const HeadGrid g = logits_grid(rows, N, K);
  return {g.tn, g.sw, 2 * g.ntiles};
}

bool two_parts(int64_t rows, bool distill) { return distill && rows <= kHeadTwoParts; }

// Bytes of the gradient's fp32 sums of split tiles.
size_t split_bytes(int64_t rows, int64_t N, int64_t K, bool distill) {
  if (rows <= 0) return 0;
  if (rows <= kHeadFewTokens)
    return static_cast<size_t>(few_splits(N, K)) * (two_parts(rows, distill) ? 2 * rows : rows) * K * 4;
  const HeadGrid d = grad_grid(rows, N, K);
  return static_cast<size_t>(d.ntail) * d.nsplit * d.tn * TM * 4;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace of a call of M tokens whose pieces hold `rows` (the last one M % rows).
struct HeadSpace {
  uint16_t* w16;
  float2* part;
  float2* ztgt;
  float4* rscale;
  float *zlabel, *logq, *split;
  int* sidx;
  uint16_t *off, *e;
  size_t bytes;
};
int64_t e_pitch(int64_t N) { return (N + 63) / 64 * 64; }

HeadSpace head_space(void* ws, int64_t rows, int64_t M, int64_t N, int64_t K, int k, bool distill, bool grad, bool nf4) {
  HeadSpace s{};
  size_t at = 0;
  auto take = [&](size_t n) -> void* {
    uint8_t* q = ws ? static_cast<uint8_t*>(ws) + at : nullptr;
    at += up256(n);
    return q;
  };
  // The last piece's tiles may be narrower (few tokens), and then more.
  const int64_t last = M % rows;
  const size_t segs = static_cast<size_t>(rows) * segments(rows, N, K).count,
               last_segs = last ? static_cast<size_t>(last) * segments(last, N, K).count : 0;
  if (nf4 && rows > kHeadFewTokens) s.w16 = static_cast<uint16_t*>(take(static_cast<size_t>(N) * K * 2));
  s.part = static_cast<float2*>(take(std::max(segs, last_segs) * 8));
  if (!distill) s.zlabel = static_cast<float*>(take(kHeadFewTokens * 4));
  if (distill) {
    s.ztgt = static_cast<float2*>(take(static_cast<size_t>(rows) * k * 8));
    s.sidx = static_cast<int*>(take(static_cast<size_t>(rows) * k * 4));
    s.logq = static_cast<float*>(take(static_cast<size_t>(rows) * k * 4));
    s.off = static_cast<uint16_t*>(take((std::max(segs, last_segs) + rows) * 2));
  }
  if (grad) {
    s.rscale = static_cast<float4*>(take(static_cast<size_t>(rows) * 16));
    // (a last piece that is stored in two parts is shorter than half of the others)
    const size_t e_rows = two_parts(rows, distill) ? 2 * rows : rows;
    s.e = static_cast<uint16_t*>(take(e_rows * e_pitch(N) * 2));
    s.split = static_cast<float*>(take(std::max(split_bytes(rows, N, K, distill), split_bytes(last, N, K, distill))));
  }
  s.bytes = at;
  return s;
}

// Tokens per piece when the caller leaves the choice to the library: as many as
// e (with a gradient) or the segments' statistics and targets (without) hold in
// 1 GB, one tile at least, and 16384 at most where only statistics are kept.
// Pieces of a call are alike, in whole tiles.
int64_t default_piece(int64_t M, int64_t N, int k, bool distill, bool grad) {
  const int64_t segs = (N + 63) / 64 + 2;  // never more: tiles of 128 entries, two segments each
  const int64_t token = grad ? e_pitch(N) * 2 : segs * (distill ? 10 : 8) + (distill ? int64_t(k) * 16 : 0);
  int64_t most = std::max<int64_t>(TM, (1ll << 30) / token / TM * TM);
  if (!grad) most = std::min<int64_t>(most, 64 * TM);
  const int64_t pieces = std::max<int64_t>(1, (M + most - 1) / most);
  return std::max<int64_t>(1, std::min<int64_t>(M, ((M + pieces - 1) / pieces + TM - 1) / TM * TM));
}

template <int MODE, int NH>
cudaError_t launch_pairs(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& out, int64_t contraction,
                         const HeadGrid& g, const HeadEpi& p, cudaStream_t st) {
  cudaError_t e = smem_limit_once<k_head<MODE, NH>>(SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  const int64_t items = int64_t(g.nwhole) + int64_t(g.ntail) * g.nsplit;
  int P = head_pairs();
  if (P <= 0) P = std::max(1, device_sm_count() / 2);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pair_config(static_cast<int>(std::min<int64_t>(items, P)), st, attr);
  return cudaLaunchKernelEx(&cfg, k_head<MODE, NH>, a, b, out, static_cast<int>((contraction + BK - 1) / BK), g, p,
                            device_status_ptr());
}
}  // namespace

// Pieces are the library's choice or a smaller number of whole tiles (all of M, if
// that is less than one).
size_t head_workspace_bytes(int64_t piece, int64_t M, int64_t N, int64_t K, int k, bool distill, bool grad,
                            bool nf4) {
  int64_t rows = default_piece(M, N, k, distill, grad);
  if (piece > 0) rows = std::min(rows, std::max<int64_t>(piece / TM * TM, TM));
  return std::max<size_t>(256, head_space(nullptr, rows, M, N, K, k, distill, grad, nf4).bytes);
}

int64_t head_piece(size_t bytes, int64_t M, int64_t N, int64_t K, int k, bool distill, bool grad, bool nf4) {
  int64_t rows = default_piece(M, N, k, distill, grad);
  while (rows > 0 && head_space(nullptr, rows, M, N, K, k, distill, grad, nf4).bytes > bytes)
    rows = (rows - 1) / TM * TM;
  return rows;
}

cudaError_t launch_head_loss(const HeadArgs& a, cudaStream_t st) {
  const bool distill = a.labels == nullptr, grad = a.dX != nullptr, nf4 = a.W == nullptr;
  const HeadSpace s = head_space(a.workspace, a.piece, a.M, a.N, a.K, a.k, distill, grad, nf4);
  const auto BF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto SW = CU_TENSOR_MAP_SWIZZLE_128B;
  cudaError_t err = cudaSuccess;
  // An NF4 head is expanded once for the pieces of many tokens (its bf16 values
  // are then read by several tiles); few tokens expand it as they go.  The last
  // piece may be of the other kind.
  HeadWeight h{a.W, a.codes, a.absmax_q, a.dq_scale, a.block, a.dq_block, a.N, a.K};
  if (nf4 && a.piece > kHeadFewTokens) {
    err = launch_dequantize(a.codes, a.absmax_q, a.dq_scale, a.N * a.K, a.block, a.dq_block, s.w16, st);
    if (err != cudaSuccess) return err;
    h.W = s.w16;
  }
  const uint16_t* W = h.W;
  const int64_t lde = e_pitch(a.N);
  for (int64_t r0 = 0; r0 < a.M; r0 += a.piece) {
    const int64_t rows = std::min(a.piece, a.M - r0);
    const bool few = rows <= kHeadFewTokens;
    const HeadGrid g = logits_grid(rows, a.N, a.K);
    const Segments seg = segments(rows, a.N, a.K);
    const uint16_t* X = a.X + r0 * a.K;
    CUtensorMap ma, mb, me{};  // me: e as the logits product writes it
    if (!few && (!make_map(&ma, BF16, X, a.K, rows, a.K * 2, BK, UM, SW) ||
                 !make_map(&mb, BF16, W, a.K, a.N, a.K * 2, BK, g.bn / 2, SW) ||
                 (grad && !make_map(&me, BF16, s.e, lde, rows, lde * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))))
      return cudaErrorInvalidValue;
    HeadEpi p{};
    p.rows = static_cast<int>(rows);
    p.cols = static_cast<int>(a.N);
    p.c = 1.4426950408889634f / a.temperature;
    p.part = s.part;
    p.e = s.e;
    p.e_low = grad && two_parts(rows, distill) ? s.e + rows * lde : nullptr;
    p.lde = lde;
    p.labels = distill ? nullptr : a.labels + r0;
    p.sidx = s.sidx;
    p.off = s.off;
    p.k = a.k;
    p.ztgt = s.ztgt;
    p.X = X;
    p.W = W;
    p.zlabel = s.zlabel;
    if (distill) {
      const dim3 grid(static_cast<unsigned>(rows)), block(TARGET_THREADS);
      const int64_t* idx = a.teacher_idx + r0 * a.k;
      const float inv_t = 1.0f / a.temperature;
      if (a.teacher_bf16)
        err = launch_ex(k_head_targets<__nv_bfloat16>, grid, block, 0, st, true, idx,
                        static_cast<const __nv_bfloat16*>(a.teacher_logits) + r0 * a.k, a.k, p.cols, inv_t, seg.tn,
                        seg.sw, seg.count, s.sidx, s.logq, s.off);
      else
        err = launch_ex(k_head_targets<float>, grid, block, 0, st, true, idx,
                        static_cast<const float*>(a.teacher_logits) + r0 * a.k, a.k, p.cols, inv_t, seg.tn,
                        seg.sw, seg.count, s.sidx, s.logq, s.off);
      if (err != cudaSuccess) return err;
    }
    if (few) err = launch_few_logits(h, X, seg.sw, p, st);
    else err = launch_pairs<0, 1>(ma, mb, me, a.K, g, p, st);
    if (err != cudaSuccess) return err;
    StatArgs t{};
    t.part = s.part;
    t.nseg = seg.count;
    t.rows = p.rows;
    t.N = p.cols;
    t.K = static_cast<int>(a.K);
    t.labels = p.labels;
    t.X = few ? nullptr : X;
    t.W = W;
    t.zlabel = s.zlabel;
    t.sidx = s.sidx;
    t.logq = s.logq;
    t.k = a.k;
    t.ztgt = s.ztgt;
    t.c = p.c;
    t.temp = a.temperature;
    t.dloss = a.dloss ? a.dloss + r0 : nullptr;
    t.loss = a.loss + r0;
    t.lse = a.lse + r0;
    t.rscale = s.rscale;
    t.e = s.e;
    t.e_low = p.e_low;
    t.lde = lde;
    t.tn = seg.tn;
    t.sw = seg.sw;
    if (rows > 1024)
      err = launch_ex(k_head_stats<16>, dim3(static_cast<unsigned>((rows + 15) / 16)), dim3(STAT_THREADS), 0, st, true, t);
    else
      err = launch_ex(k_head_stats<4>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(STAT_THREADS), 0, st, true, t);
    if (err != cudaSuccess) return err;
    if (!grad) continue;
    HeadEpi q{};
    q.rows = p.rows;
    q.cols = static_cast<int>(a.K);
    q.rscale = s.rscale;
    q.W = h.W;
    q.out = a.dX + r0 * a.K;
    q.split = s.split;
    q.two_parts = p.e_low != nullptr;
    if (few) {
      err = launch_few_grad(h, s.e, lde, few_splits(a.N, a.K), q, st);
      if (err != cudaSuccess) return err;
      continue;
    }
    const HeadGrid d = grad_grid(rows, a.N, a.K);
    if (!make_map(&ma, BF16, s.e, lde, rows, lde * 2, BK, UM, SW) ||
        !make_map(&mb, BF16, W, a.K, a.N, a.K * 2, 64, BK, SW))
      return cudaErrorInvalidValue;
    err = d.nh == 2 ? launch_pairs<1, 2>(ma, mb, me, a.N, d, q, st) : launch_pairs<1, 1>(ma, mb, me, a.N, d, q, st);
    if (err == cudaSuccess && d.ntail)
      err = launch_ex(k_head_join, dim3(static_cast<unsigned>(d.ntail * (TM * (d.tn / 8) / 256))), dim3(256), 0, st,
                      true, static_cast<const float*>(s.split), d, q);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace qn
