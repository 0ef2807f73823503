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
constexpr int BK = 64;
constexpr int W_BYTES = UM * BK * 2;  // expanded head tile of a stage
constexpr int C_BYTES = UM * BK / 2;  // its NF4 codes
constexpr int MAX_STAGES = 12;
constexpr int CSTAGES = 12;           // NF4 code ring
constexpr int DQ_GROUPS = 4;          // groups of 4 warps, each expanding every fourth stage
constexpr int BUF_PITCH = UM + 4;     // floats per token in the epilogue's buffer
constexpr int BUF_TOKENS = 16;
constexpr int BUF_BYTES = 2 * BUF_TOKENS * BUF_PITCH * 4;
constexpr int BAR_BYTES = 512;
constexpr int SMEM_MAX = 232448;

struct FewBars {
  uint64_t full[MAX_STAGES];   // head tile and token tile landed (or were written)
  uint64_t empty[MAX_STAGES];  // MMAs of the stage completed
  uint64_t full_c[CSTAGES];    // NF4: code tile landed
  uint64_t empty_c[CSTAGES];   // NF4: code tile expanded
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
  int numK;    // stages of the contraction
  int tp;      // tokens, rounded up to 16
  int stages;
  int cols;    // TMEM columns
};

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same barrier; tells all 128 threads whether ok holds for every one of them.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// KIND 0: bf16 head; 1: NF4 in the default format (64-weight blocks, double
// quantization); 2: NF4 with 2^lg-weight blocks, double quantization if dq.
//   warp 0       TMA producer
//   warp 1       TMEM allocation, MMA issue
//   warps 2-5    epilogue (two accumulators alternate)
//   warps 6-21   KIND > 0: expansion of the codes
// Every wait is bounded; on expiry the kernel records kDevTimeout, drains what
// it issued, frees TMEM and returns.
template <int MODE, int KIND>
__global__ void __launch_bounds__(KIND ? 192 + DQ_GROUPS * 128 : 192, 1)
    k_few(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, FewGrid g, HeadEpi p,
          const uint8_t* __restrict__ absmax_q, const float* __restrict__ dq_scale, Nf4Levels lv, int N, int K, int lg,
          int dq, int* status) {
  constexpr bool NF4 = KIND > 0, GEN = KIND == 2;
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int stage_bytes = W_BYTES + g.tp * BK * 2;
  const uint32_t codes = base + g.stages * stage_bytes;
  const uint32_t buf = codes + (NF4 ? CSTAGES * C_BYTES : 0);
  const uint32_t bar0 = buf + BUF_BYTES;
  FewBars* bars = reinterpret_cast<FewBars*>(smem_raw + (bar0 - raw));
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
  auto full_c = [&](int s) { return bar0 + 8u * (2 * MAX_STAGES + s); };
  auto empty_c = [&](int s) { return bar0 + 8u * (2 * MAX_STAGES + CSTAGES + s); };
  auto acc_full = [&](int a) { return bar0 + 8u * (2 * MAX_STAGES + 2 * CSTAGES + a); };
  auto acc_empty = [&](int a) { return bar0 + 8u * (2 * MAX_STAGES + 2 * CSTAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * MAX_STAGES + 2 * CSTAGES + 4);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nitems = g.tiles * g.nsplit, tokens = p.rows;

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
    for (int s = 0; s < CSTAGES; ++s) {
      mbar_init(full_c(s), 1);
      mbar_init(empty_c(s), 4);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full(a), 1);
      mbar_init(acc_empty(a), 4);
    }
    mbar_init(drain_bar, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (tokens < g.tp) {  // the token rows that no copy writes hold zeros
    const int n = (g.tp - tokens) * BK * 2 / 16;
    for (int s = 0; s < g.stages; ++s)
      for (int i = threadIdx.x; i < n; i += blockDim.x)
        st_shared_v4(base + s * stage_bytes + W_BYTES + tokens * BK * 2 + 16 * i, 0u, 0u, 0u, 0u);
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
    if (lane == 0) {
      const uint32_t x_bytes = tokens * BK * 2, w_bytes = MODE == 0 ? g.br * BK * 2 : W_BYTES;
      bool ok = true;
      int n = 0;
      if (!NF4) {
        for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
          int nt, z, kbeg, kend;
          item(i, nt, z, kbeg, kend);
          for (int k = kbeg; k < kend; ++k, ++n) {
            const int s = n % g.stages;
            if (!(ok = wait_bounded(empty(s), ((n / g.stages) & 1) ^ 1, abort, status))) break;
            const uint32_t w_s = base + s * stage_bytes;
            mbar_arrive_expect_tx(full(s), w_bytes + x_bytes);
            if (MODE == 0) {
              tma_load_2d(w_s, &tm_w, full(s), k * BK, nt * g.br);
            } else {
              tma_load_2d(w_s, &tm_w, full(s), nt * UM, k * BK);
              tma_load_2d(w_s + 8192, &tm_w, full(s), nt * UM + 64, k * BK);
            }
            tma_load_2d(w_s + W_BYTES, &tm_x, full(s), k * BK, 0);
          }
        }
      } else {
        // Two walks over the same stages: the codes run ahead as far as their ring
        // allows, the token tiles follow the expanded stages.
        struct Walk {
          int i, nt, z, k, kend, n;
        };
        auto start = [&](Walk& w) {
          if (w.i < nitems) item(w.i, w.nt, w.z, w.k, w.kend);
        };
        auto advance = [&](Walk& w) {
          ++w.n;
          if (++w.k == w.kend) {
            w.i += gridDim.x;
            start(w);
          }
        };
        Walk c{static_cast<int>(blockIdx.x), 0, 0, 0, 0, 0}, x = c;
        start(c);
        start(x);
        while (x.i < nitems && ok) {
          while (c.i < nitems && c.n < x.n + CSTAGES - 1 && ok) {
            const int s = c.n % CSTAGES;
            if (!(ok = wait_bounded(empty_c(s), ((c.n / CSTAGES) & 1) ^ 1, abort, status))) break;
            mbar_arrive_expect_tx(full_c(s), MODE == 0 ? g.br * (BK / 2) : C_BYTES);
            if (MODE == 0) tma_load_2d(codes + s * C_BYTES, &tm_w, full_c(s), c.k * (BK / 2), c.nt * g.br);
            else tma_load_2d(codes + s * C_BYTES, &tm_w, full_c(s), c.nt * (UM / 2), c.k * BK);
            advance(c);
          }
          if (!ok) break;
          const int s = x.n % g.stages;
          if (!(ok = wait_bounded(empty(s), ((x.n / g.stages) & 1) ^ 1, abort, status))) break;
          mbar_arrive_expect_tx(full(s), x_bytes);
          tma_load_2d(base + s * stage_bytes + W_BYTES, &tm_x, full(s), x.k * BK, 0);
          advance(x);
        }
        n = c.n;
      }
      if (!ok && n > 0) {  // the copies already issued land well within this time
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 20000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(UM, g.tp, MODE == 1, false);
      bool ok = true, committed = false;
      int n = 0, t = 0;
      for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x, ++t) {
        int nt, z, kbeg, kend;
        item(i, nt, z, kbeg, kend);
        if (!(ok = wait_bounded(acc_empty(t & 1), ((t >> 1) & 1) ^ 1, abort, status))) break;
        tc_fence_after();
        const uint32_t d = tmem + (t & 1) * g.tp;
        for (int k = kbeg; k < kend; ++k, ++n) {
          const int s = n % g.stages;
          if (!(ok = wait_bounded(full(s), (n / g.stages) & 1, abort, status))) break;
          tc_fence_after();
          const uint32_t w_s = base + s * stage_bytes, x_s = w_s + W_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = MODE == 0 ? desc_sw128(w_s + kk * 32, 16, 1024) : desc_sw128(w_s + kk * 2048, 8192, 1024);
            tc_mma_f16(d, ad, desc_sw128(x_s + kk * 32, 16, 1024), idesc, (k > kbeg || kk > 0) ? 1u : 0u);
          }
          tc_commit(empty(s));
          committed = true;
        }
        if (ok) tc_commit(acc_full(t & 1));
      }
      if (!ok && committed) {
        tc_commit(drain_bar);
        wait_drain(drain_bar, 0);
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3, ew = warp - 2;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    int t = 0, filled = 0;
    for (int i = blockIdx.x; i < nitems; i += gridDim.x, ++t) {
      int nt, z, kbeg, kend;
      item(i, nt, z, kbeg, kend);
      // the four warps leave together: they meet at barriers
      if (!epilogue_all(wait_bounded(acc_full(t & 1), (t >> 1) & 1, abort, status))) break;
      tc_fence_after();
      const uint32_t acc = tmem + lane_base + (t & 1) * g.tp;
      if (MODE == 1) {
        const int k = nt * UM + quad * 32 + lane;
        float* dst = p.split + static_cast<int64_t>(z) * tokens * p.cols + k;
#pragma unroll 1
        for (int m = 0; m < tokens; m += 16) {
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
        for (int m = 0; m < tokens; m += BUF_TOKENS, ++filled) {
          // 16 tokens x 128 entries into shared memory, token by token; then a warp
          // has a token's entries side by side
          const uint32_t b = buf + (filled & 1) * (BUF_BYTES / 2);
          float* bp = reinterpret_cast<float*>(smem_raw + (b - raw));
          uint32_t v[16];
          tmem_ld_x16(acc + m, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < BUF_TOKENS; ++j) bp[j * BUF_PITCH + quad * 32 + lane] = __uint_as_float(v[j]);
          epilogue_barrier();
          for (int j = ew * (BUF_TOKENS / 4); j < (ew + 1) * (BUF_TOKENS / 4) && m + j < tokens; ++j) {
            const int row = m + j, c0 = 4 * lane;
            const float4 x4 = *reinterpret_cast<const float4*>(bp + j * BUF_PITCH + c0);
            const float x[4] = {x4.x, x4.y, x4.z, x4.w};
            float mx = -INFINITY;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (c0 + q < ncols) mx = fmaxf(mx, x[q]);
            for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float ref = mx == -INFINITY ? 0.0f : rintf(mx * p.c);  // as in head.cu
            float e[4], sum;
#pragma unroll
            for (int q = 0; q < 4; ++q) e[q] = c0 + q < ncols ? exp2_fast(fmaf(x[q], p.c, -ref)) : 0.0f;
            sum = (e[0] + e[1]) + (e[2] + e[3]);
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (lane == 0)
              p.part[static_cast<int64_t>(nt) * tokens + row] = make_float2(mx == -INFINITY ? mx : ref, sum);
            if (p.e) {
              uint16_t* er = p.e + static_cast<int64_t>(row) * p.lde + v0;
              const float back = exp2f(fabsf(ref) <= kHeadFits ? ref : 0.0f);
              if (c0 < ewidth)  // groups of four entries are whole: br % 8 == 0, lde % 64 == 0
                *reinterpret_cast<uint2*>(er + c0) =
                    make_uint2(bf16x2_bits(e[0] * back, e[1] * back), bf16x2_bits(e[2] * back, e[3] * back));
              if (nt == g.tiles - 1)  // the pitch may reach past the last tile
                for (int64_t c = v0 + g.br + c0; c < p.lde; c += 128)
                  *reinterpret_cast<uint2*>(er + (c - v0)) = make_uint2(0u, 0u);
            }
            if (p.labels) {
              const int64_t y = p.labels[row];
              if (lane == 0 && y >= v0 && y < v0 + ncols)
                p.ztgt[row] = make_float2(fmaf(bp[j * BUF_PITCH + static_cast<int>(y - v0)], p.c, -ref), ref);
            } else {
              const uint16_t* o = p.off + static_cast<int64_t>(row) * (g.tiles + 1) + nt;
              for (int s = o[0] + lane; s < o[1]; s += 32) {
                const int64_t at = static_cast<int64_t>(row) * p.k + s;
                p.ztgt[at] = make_float2(fmaf(bp[j * BUF_PITCH + p.sidx[at] - v0], p.c, -ref), ref);
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(t & 1));
    }
  } else if (NF4) {
    // ----------------------------------------------- expansion of the codes
    const int e = warp - 6, grp = e >> 2;
    const int t = (e & 3) * 32 + lane;  // row of the 128-byte rows of the stage
    const int KB = K / 64;
    // Which (row, 64-weight group) of W this thread expands: MODE 0, row t of the
    // tile; MODE 1, row t % 64 of the stage, columns 64 (t / 64) of the tile.
    struct Walk {
      int i, nt, z, k, kend, n;
    };
    auto start = [&](Walk& w) {
      if (w.i < nitems) item(w.i, w.nt, w.z, w.k, w.kend);
    };
    auto advance = [&](Walk& w, int by) {  // by stages; an item may be shorter than that
      w.n += by;
      w.k += by;
      while (w.i < nitems && w.k >= w.kend) {
        const int over = w.k - w.kend;
        w.i += gridDim.x;
        start(w);
        w.k += over;
      }
    };
    struct Scale {
      uint32_t q0, q1;
      float s0, s1;
      bool valid;
    };
    auto fetch = [&](const Walk& w) {
      Scale sc{0u, 0u, 0.0f, 0.0f, false};
      if (w.i >= nitems) return sc;
      const int wrow = MODE == 0 ? w.nt * g.br + t : w.k * BK + (t & 63);
      const int kcol = MODE == 0 ? w.k * BK : w.nt * UM + 64 * (t >> 6);
      if (wrow < N && kcol < K && (MODE == 1 || t < g.br)) {
        if (!GEN) {
          const int64_t blk = static_cast<int64_t>(wrow) * KB + (kcol >> 6);
          sc.q0 = __ldg(absmax_q + blk);
          sc.s0 = __ldg(dq_scale + (blk >> 8));
        } else {
          const int64_t blk = (static_cast<int64_t>(wrow) * K + kcol) >> lg;
          if (dq) {
            sc.q0 = __ldg(absmax_q + blk);
            sc.s0 = __ldg(dq_scale + (blk >> 8));
            if (lg == 5) {
              sc.q1 = __ldg(absmax_q + blk + 1);
              sc.s1 = __ldg(dq_scale + ((blk + 1) >> 8));
            }
          } else {
            sc.s0 = __ldg(dq_scale + blk);
            if (lg == 5) sc.s1 = __ldg(dq_scale + blk + 1);
          }
        }
        sc.valid = true;
      }
      return sc;
    };
    // The scales are loaded two of this group's stages ahead.
    Walk w{static_cast<int>(blockIdx.x), 0, 0, 0, 0, 0};
    start(w);
    advance(w, grp);
    Walk a1 = w;
    Scale p0 = fetch(a1);
    advance(a1, DQ_GROUPS);
    Scale p1 = fetch(a1);
    Walk a2 = a1;
    bool ok = true;
    while (w.i < nitems && ok) {
      advance(a2, DQ_GROUPS);
      const Scale p2 = fetch(a2);
      const int cs = w.n % CSTAGES, s = w.n % g.stages;
      if (!(ok = wait_bounded(full_c(cs), (w.n / CSTAGES) & 1, abort, status))) break;
      const uint32_t c_s = codes + cs * C_BYTES;
      uint4 q0, q1;
      if (MODE == 0) {  // code tile [br rows][32 B], 32-byte swizzle
        const uint32_t sw = (static_cast<uint32_t>(t) >> 2) & 1u;
        q0 = ld_shared_v4(c_s + t * 32 + ((0u ^ sw) << 4));
        q1 = ld_shared_v4(c_s + t * 32 + ((1u ^ sw) << 4));
      } else {  // code tile [64 rows][64 B], 64-byte swizzle
        const uint32_t row = t & 63, j = t >> 6, sw = (row >> 1) & 3u;
        q0 = ld_shared_v4(c_s + row * 64 + (((2 * j) ^ sw) << 4));
        q1 = ld_shared_v4(c_s + row * 64 + (((2 * j + 1) ^ sw) << 4));
      }
      if (!(ok = wait_bounded(empty(s), ((w.n / g.stages) & 1) ^ 1, abort, status))) break;
      const uint32_t row_s = base + s * stage_bytes + t * 128;
      const uint32_t sw = t & 7;
      if (p0.valid) {
        const float a0 = (GEN && !dq) ? p0.s0 : __fmul_rn(static_cast<float>(p0.q0), p0.s0);
        const Nf4Lut lut = make_lut(lv, a0);
        const uint32_t c[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        if (GEN && lg == 5) {
          const float a1s = dq ? __fmul_rn(static_cast<float>(p0.q1), p0.s1) : p0.s1;
          const Nf4Lut lut1 = make_lut(lv, a1s);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t o0, o1, o2, o3;
            deq8(c[j], j < 4 ? lut : lut1, o0, o1, o2, o3);
            st_shared_v4(row_s + ((j ^ sw) << 4), o0, o1, o2, o3);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t o0, o1, o2, o3;
            deq8(c[j], lut, o0, o1, o2, o3);
            st_shared_v4(row_s + ((j ^ sw) << 4), o0, o1, o2, o3);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) st_shared_v4(row_s + (j << 4), 0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(empty_c(cs));
        mbar_arrive(full(s));
      }
      advance(w, DQ_GROUPS);
      p0 = p1;
      p1 = p2;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, g.cols);
  }
}

// Sum of the gradient's pieces in piece order, times the row's factors, rounded
// once to bf16.  Thread: 4 consecutive outputs of a token.
__global__ void __launch_bounds__(128) k_few_join(const float* __restrict__ split, int nsplit, HeadEpi p) {
  pdl_trigger();
  pdl_wait();
  const int c = (blockIdx.x * 128 + threadIdx.x) * 4, row = blockIdx.y;
  if (c >= p.cols) return;
  const int64_t at = static_cast<int64_t>(row) * p.cols + c, piece = static_cast<int64_t>(p.rows) * p.cols;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int z = 0; z < nsplit; ++z) {
    const float4 x = *reinterpret_cast<const float4*>(split + at + z * piece);
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
  }
  const float2 f = p.rscale[row];
  uint2 o = make_uint2(0u, 0u);
  if (f.y != 0.0f) o = make_uint2(bf16x2_bits(a.x * f.x * f.y, a.y * f.x * f.y), bf16x2_bits(a.z * f.x * f.y, a.w * f.x * f.y));
  *reinterpret_cast<uint2*>(p.out + at) = o;
}

// Ring depth and shared memory for `tokens` tokens.
int few_stages(int tp, bool nf4) {
  const int room = SMEM_MAX - 1024 - BAR_BYTES - BUF_BYTES - (nf4 ? CSTAGES * C_BYTES : 0);
  return std::min(MAX_STAGES, room / (W_BYTES + tp * BK * 2));
}
int few_smem(const FewGrid& g, bool nf4) {
  return 1024 + g.stages * (W_BYTES + g.tp * BK * 2) + (nf4 ? CSTAGES * C_BYTES : 0) + BUF_BYTES + BAR_BYTES;
}

FewGrid few_grid(int64_t tokens, bool nf4) {
  FewGrid g{};
  g.tp = static_cast<int>((tokens + 15) / 16 * 16);
  g.stages = few_stages(g.tp, nf4);
  g.cols = 32;
  while (g.cols < 2 * g.tp) g.cols *= 2;
  return g;
}

template <int MODE, int KIND>
cudaError_t launch_kind(const CUtensorMap& w, const CUtensorMap& x, const FewGrid& g, const HeadEpi& p,
                        const HeadWeight& h, cudaStream_t st) {
  cudaError_t e = smem_limit_once<k_few<MODE, KIND>>(SMEM_MAX);
  if (e != cudaSuccess) return e;
  int lg = 0;
  while ((1 << lg) < h.block) ++lg;
  const int grid = std::min(g.tiles * g.nsplit, device_sm_count());
  return launch_ex(k_few<MODE, KIND>, dim3(grid), dim3(KIND ? 192 + DQ_GROUPS * 128 : 192), few_smem(g, KIND > 0), st,
                   true, w, x, g, p, h.absmax_q, h.dq_scale, host_codebook().levels, static_cast<int>(h.N),
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
const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
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
    // a tile costs its rows, and its start and epilogue about what 16 rows cost
    const int64_t c = ((N + br - 1) / br + P - 1) / P * (br + 16);
    if (br == UM || c < cost) {
      cost = c;
      best = br;
    }
  }
  return best;
}

int few_splits(int64_t N, int64_t K) {
  const int64_t tiles = (K + UM - 1) / UM, numK = (N + BK - 1) / BK;
  const int P = device_sm_count();
  int best = 1;
  double cost = 0.0;
  for (int64_t S = 1; S <= std::min<int64_t>(std::max<int64_t>(numK / 8, 1), 64); ++S) {
    const double rounds = static_cast<double>((tiles * S + P - 1) / P);
    // rounds of S-ths of the vocabulary, each with its start and epilogue (about 4 stages)
    const double c = rounds * (static_cast<double>(numK) / static_cast<double>(S) + 4.0);
    if (S == 1 || c < cost) {
      cost = c;
      best = static_cast<int>(S);
    }
  }
  return best;
}

cudaError_t launch_few_logits(const HeadWeight& h, const uint16_t* X, int br, const HeadEpi& p, cudaStream_t st) {
  FewGrid g = few_grid(p.rows, !h.W);
  g.br = br;
  g.tiles = static_cast<int>((h.N + br - 1) / br);
  g.nsplit = 1;
  g.numK = static_cast<int>(h.K / BK);
  CUtensorMap w, x;
  const bool ok = h.W ? make_map(&w, BF16, h.W, h.K, h.N, h.K * 2, BK, br, SW128)
                      : make_map(&w, U8, h.codes, h.K / 2, h.N, h.K / 2, BK / 2, br, CU_TENSOR_MAP_SWIZZLE_32B);
  if (!ok || !make_map(&x, BF16, X, h.K, p.rows, h.K * 2, BK, p.rows, SW128)) return cudaErrorInvalidValue;
  return launch_few<0>(w, x, g, p, h, st);
}

cudaError_t launch_few_grad(const HeadWeight& h, const uint16_t* P, int64_t ldp, int nsplit, const HeadEpi& p,
                            cudaStream_t st) {
  FewGrid g = few_grid(p.rows, !h.W);
  g.br = UM;
  g.tiles = static_cast<int>((h.K + UM - 1) / UM);
  g.nsplit = nsplit;
  g.numK = static_cast<int>((h.N + BK - 1) / BK);
  CUtensorMap w, x;
  const bool ok = h.W ? make_map(&w, BF16, h.W, h.K, h.N, h.K * 2, 64, BK, SW128)
                      : make_map(&w, U8, h.codes, h.K / 2, h.N, h.K / 2, UM / 2, BK, CU_TENSOR_MAP_SWIZZLE_64B);
  if (!ok || !make_map(&x, BF16, P, ldp, p.rows, ldp * 2, BK, p.rows, SW128)) return cudaErrorInvalidValue;
  cudaError_t e = launch_few<1>(w, x, g, p, h, st);
  if (e != cudaSuccess) return e;
  return launch_ex(k_few_join, dim3(static_cast<unsigned>((p.cols + 511) / 512), static_cast<unsigned>(p.rows)),
                   dim3(128), 0, st, true, static_cast<const float*>(p.split), nsplit, p);
}

}  // namespace qn
