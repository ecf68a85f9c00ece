// gemm_fp8.cu -- grouped GEMM of e4m3 operands with an fp32 scale per 128 columns of a
// row (activations) and per 128 x 128 block (weights), on tcgen05 kind::f8f6f4.
//
//   acc[r, n] = sum_b xs[r, b] ws[n / 128, b] D_b[r, n],   D_b = sum_{k in block b} xq[r, k] wq[n, k]
//
// The tensor cores form D_b as an fp32 accumulation over one block of K (four K = 32
// steps) in tensor memory; the scales differ from block to block and row to row, so each
// D_b is read back and added to an fp32 accumulator with its scale product.  Rows are the
// MMA's M: a thread of an epilogue warp owns one row and 64 columns of one weight block, so
// a block of K costs it one scale product and 64 multiply-adds, and the accumulators live
// in its registers for the whole K loop.  (With the weights as M the row scales would
// differ from register to register and each multiply-add would need an operand from shared
// memory.)  Tensor memory is a ring of four quarters of 128 columns; a block of K is two MMA
// groups of N = 128 (one per weight block), each handed over by itself, so that the adds of
// one quarter run beside the products of the others: with two halves of 256 columns the
// chain product - hand-over - adds - hand-over of a buffer was longer than two products.
//
// Work: tiles of 128 rows by 256 weight rows (128 gate and their 128 up rows, or 256 plain
// rows); persistent CTAs, one per SM; the tile list is made on the device from the groups'
// row counts.  (On CTA pairs, 256 rows by 256 weight rows, an earlier form of the kernel
// loaded a third less and was no faster: 8192 rows of 8 experts of 4096 x 14336 took 1.81 ms
// against 1.71.)  Warps of a CTA:
//   0     TMA producer (128-byte swizzle, one block of K per stage);
//   1, 3  MMA issue, blocks of K in turn; 1: TMEM, too;
//   2     the products of row and weight scales, a ring of blocks ahead in shared memory
//         (read by the epilogue itself they cost it a memory latency per block);
//   4-19  epilogue: TMEM lane quadrant x 64 columns.  Sixteen warps of 64 accumulators each
//         fit 96 registers a thread, and four per scheduler hide the tensor memory reads
//         (eight of 128 with registers handed over from the first four: 4096 rows 368 us
//         against 366, 77 rows 119 against 123).
// Large batches: a block of K takes some 1200 clocks for 512 of products, and no unit is full
// (6001 rows of 4096 x 4096: tensor pipe 47%, L2 39%, issue slots 57%, DRAM 23%); what is left
// is the latency of the chain commit - barrier - reads and adds - hand-back, and the power
// limit (clocks of 1.3 to 1.65 GHz): 8192 rows of 8 experts of 4096 x 14336 1.80 ms, 1.6 PFLOP/s; 4096 rows of 32
// experts of 7168 x 2048 0.37 ms; 8 rows by their weights, 59 us for 201 MB.
// Every wait is bounded (2 s) and reports MOE_ERR_TIMEOUT.  No asynchronous write into a
// CTA's shared memory outlives it: its producer waits for every load and for the last commit
// on every stage's barrier.  Launched in plain stream order, and nothing starts before its
// end: as programmatic launches, without that wait, a GEMM's CTAs started on SMs that the
// GEMM before it left free, and 8 rows of 32 experts in a loop of calls ended in an illegal
// address.
#include "fp8.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int BM = kFp8BM;
constexpr int BK = kFp8Block;     // bytes of K per stage: one scale block
constexpr int BNB = 256;          // weight rows per tile
constexpr int BNH = 128;          // of them per MMA group: one of the tile's two weight blocks
constexpr int kQuarters = 4;      // accumulators of BNH columns in tensor memory
constexpr int TMEM_COLS = kQuarters * BNH;
constexpr int kEpiWarps = 16;     // tensor memory lane quadrant x 64 of the 256 columns
constexpr int kFirstEpiWarp = 4;
constexpr int kThreads = (kFirstEpiWarp + kEpiWarps) * 32;
constexpr int kMaxStages = 6;
constexpr int kScaleBatch = 8;    // blocks of K whose scale products are handed over together
constexpr int kScaleSlots = 2 * kScaleBatch;
constexpr int kSmemLimit = 232448;
// kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A and B e4m3 (format 0), K-major, N >> 3
// in bits 17-22, M >> 4 in 24-28.
constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(BNH >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);

// Shared memory after the stages: scale products, barriers, the row maxima the two column
// halves of a tile exchange, the groups' first rows and tile prefixes.  The quarters'
// barriers are aligned so that quarters 0, 1 and 2, 3 differ by one address bit.
struct alignas(64) Meta {
  float2 scale[kScaleSlots][BM];  // [block of K mod slots][row]: times the two weight blocks' scales
  float amax[4][BM];              // [quarter of the tile's columns][row]
  uint64_t tfull[kQuarters], tempty[kQuarters];
  uint64_t full[kMaxStages], empty[kMaxStages], sfull[2], sempty[2], drain;
  uint32_t tmem_slot;
  int abort_flag;
};

constexpr int stage_bytes(int abox) { return (abox + BNB) * BK; }
constexpr int meta_bytes(int E) { return (int)sizeof(Meta) + 2 * (E + 1) * 4; }
constexpr int stages_for(int abox, int E) {
  const int n = (kSmemLimit - 1024 - meta_bytes(E)) / stage_bytes(abox);
  return n > kMaxStages ? kMaxStages : n;
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(IDESC), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Waits for the thread's TMEM loads; r is in place after it (and not read before).
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// True in one lane of a converged warp.  The compiler knows that the branch on it runs in
// one thread: issuing MMAs and commits there takes a third of the cycles that a branch on
// the lane number takes (4 MMAs and 2 commits: about 200 cycles instead of 450).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// The four warps of a tensor memory lane quadrant meet.
__device__ __forceinline__ void quadrant_sync(int q) { asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory"); }

// The same value in every lane, in a form that the compiler knows to be uniform: loops and
// branches on it need no reconvergence around the whole-warp tensor memory loads (with
// bounds read from shared memory by every lane, those cost the K loop much of its time).
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Barriers by shared-memory address: a loop keeps one register per role, not a pointer per
// barrier.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {  // suspends for some microseconds at most
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {  // does not suspend
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The rest of a wait whose first attempt was in vain: until the phase completes, another
// role gives up (*abort) or 2 s have passed.
__device__ __forceinline__ bool keep_waiting(uint32_t bar, uint32_t parity, uint32_t abort, int* status) {
  const uint64_t t0 = global_timer();
  while (!try_wait(bar, parity)) {
    int stop;
    asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(stop) : "r"(abort) : "memory");
    if (stop) return false;
    if (global_timer() - t0 > kTimeoutNs) {
      asm volatile("st.volatile.shared.s32 [%0], %1;" ::"r"(abort), "r"(1) : "memory");
      set_status(status, MOE_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint32_t abort, int* status) {  // one thread
  return try_wait(bar, parity) || keep_waiting(bar, parity, abort, status);
}
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, uint32_t abort, int* status) {
  if (!__all_sync(0xffffffffu, try_wait(bar, parity))) {
    keep_waiting(bar, parity, abort, status);
    __syncwarp();
  }
}
// One lane arrives, without a branch.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(lane)
      : "memory");
}
struct Unit {
  int e, m0, n_blk, rows, row0, sp, kb0, kb1;
};

// Unit u of the list: split-fastest, then row tile, then N block, then group.
__device__ __forceinline__ Unit unit_of(const Fp8GemmArgs& p, const int32_t* row0, const int32_t* tiles, int u, int nkb) {
  Unit r;
  const int tile = u / p.splits;
  r.sp = u % p.splits;
  int lo = 0, hi = p.E - 1;  // last group with tiles[g] <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tiles[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  r.e = lo;
  r.row0 = row0[lo];
  r.rows = row0[lo + 1] - r.row0;
  const int mt = (r.rows + BM - 1) / BM;
  const int local = tile - tiles[lo];
  r.n_blk = local / mt;
  r.m0 = (local % mt) * BM;
  r.kb0 = r.sp * nkb / p.splits;
  r.kb1 = (r.sp + 1) * nkb / p.splits;
  return r;
}

// Scale rows of a tile's two weight blocks: [ceil(K / 128)] each.
struct BlockScales {
  const float *w0, *w1;
};
template <int MODE>
__device__ __forceinline__ BlockScales block_scales(const Fp8GemmArgs& p, const Unit& t, int nbn, int nkb) {
  BlockScales b;
  if (MODE == FP8_GATED) {
    const bool cat = p.layout != MOE_GU_UNFUSED;
    b.w0 = cat ? p.ws + ((int64_t)t.e * 2 * nbn + t.n_blk) * nkb : p.wgs + ((int64_t)t.e * nbn + t.n_blk) * nkb;
    b.w1 = cat ? b.w0 + (int64_t)nbn * nkb : p.ws + ((int64_t)t.e * nbn + t.n_blk) * nkb;
  } else {
    b.w0 = p.ws + ((int64_t)t.e * nbn + 2 * t.n_blk) * nkb;
    b.w1 = 2 * t.n_blk + 1 < nbn ? b.w0 + nkb : b.w0;
  }
  return b;
}

// Features f0 .. f0 + 15 of a row: gate (or plain) sums in g, up sums in u -> activated
// values in g; returns their largest magnitude.  One activation per instance: the values
// run a short straight piece of code.
template <bool GATED, int ACT>
__device__ __forceinline__ float activate(float (&g)[16], const float (&u)[16], ActParams a, int f0, int N) {
  a.act = ACT;
  if (ACT == MOE_ACT_SILU && GATED && a.limit > 0.f) {
#pragma unroll
    for (int i = 0; i < 16; i++) g[i] = fminf(g[i], a.limit);
  }
  a.limit = ACT == MOE_ACT_SILU && GATED && a.limit > 0.f ? a.limit : INFINITY;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    g[i] = fp8_act(a, g[i], false);
    if (GATED) g[i] *= (ACT == MOE_ACT_SILU ? fminf(fmaxf(u[i], -a.limit), a.limit) : u[i]) + a.beta;
    m = fmaxf(m, fabsf(g[i]));
  }
  return f0 < N ? m : 0.f;  // N is a multiple of 16
}
template <bool GATED>
__device__ __forceinline__ float activate(float (&g)[16], const float (&u)[16], const ActParams& act, int f0, int N) {
  switch (act.act) {
    case MOE_ACT_SILU: return activate<GATED, MOE_ACT_SILU>(g, u, act, f0, N);
    case MOE_ACT_GELU_ERF: return activate<GATED, MOE_ACT_GELU_ERF>(g, u, act, f0, N);
    case MOE_ACT_GELU_TANH: return activate<GATED, MOE_ACT_GELU_TANH>(g, u, act, f0, N);
    case MOE_ACT_RELU: return activate<GATED, MOE_ACT_RELU>(g, u, act, f0, N);
    default: return activate<GATED, MOE_ACT_IDENTITY>(g, u, act, f0, N);
  }
}

// v[i] += bias[c0 + i] for the columns below N (a multiple of 8).
__device__ __forceinline__ void add_bias(float (&v)[16], const uint16_t* bias, int c0, int N) {
#pragma unroll
  for (int i = 0; i < 16; i++)
    if (c0 + i < N) v[i] += bf16_to_f32(__ldg(bias + c0 + i));
}

template <int MODE, int ABOX>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmG, const Fp8GemmArgs p, const int stages) {
  constexpr int STAGE_BYTES = stage_bytes(ABOX), A_BYTES = ABOX * BK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Meta& meta = *reinterpret_cast<Meta*>(smem + stages * STAGE_BYTES);
  int32_t* row0 = reinterpret_cast<int32_t*>(&meta + 1);  // [E + 1]
  int32_t* tiles = row0 + p.E + 1;                         // [E + 1]
  volatile int* abort_flag = &meta.abort_flag;

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; s++) {
      mbar_init(&meta.full[s], 1);
      mbar_init(&meta.empty[s], 1);
    }
    for (int b = 0; b < kQuarters; b++) {
      mbar_init(&meta.tfull[b], 1);
      mbar_init(&meta.tempty[b], kEpiWarps / 2);  // the warps of that weight block
    }
    for (int s = 0; s < 2; s++) {
      mbar_init(&meta.sfull[s], 1);
      mbar_init(&meta.sempty[s], kEpiWarps);
    }
    mbar_init(&meta.drain, 2);  // both MMA issuers
    meta.abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    if (MODE == FP8_GATED && p.layout == MOE_GU_UNFUSED) prefetch_tmap(&tmG);
  }
  if (warp == 1) {
    tmem_alloc(&meta.tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  // (no pdl_enter(): launched when everything before has ended, and nothing starts before its end)
  if (p.clear_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_OK;
  for (int e = threadIdx.x; e < p.E; e += kThreads) row0[e] = p.cnt ? p.cnt[e] : p.R;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int nt = (p.N + (MODE == FP8_GATED ? 127 : 255)) / (MODE == FP8_GATED ? 128 : 256);
  if (warp == 2) {
    // first rows (counts cut off at R) and tile prefixes of the groups
    int64_t rows_before = 0;
    int32_t tiles_before = 0;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      const int64_t c = e < p.E ? max(row0[e], 0) : 0;
      int64_t incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int32_t first = (int32_t)min(rows_before + incl - c, (int64_t)p.R);
      const int32_t end = (int32_t)min(rows_before + incl, (int64_t)p.R);
      const int32_t mt = (end - first + BM - 1) / BM * nt;
      int32_t tincl = mt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, tincl, o);
        if (lane >= o) tincl += v;
      }
      __syncwarp();
      if (e < p.E) {
        row0[e] = first;
        tiles[e] = tiles_before + tincl - mt;
      }
      rows_before += __shfl_sync(0xffffffffu, incl, 31);
      tiles_before += __shfl_sync(0xffffffffu, tincl, 31);
    }
    if (lane == 0) {
      row0[p.E] = (int32_t)min(rows_before, (int64_t)p.R);
      tiles[p.E] = tiles_before;
    }
  }
  __syncthreads();
  // Addresses in shared memory; what every role needs is formed again where it is used
  // (kept across the roles it would be spilled).
  const uint32_t abort = smem_u32(&meta.abort_flag);

  if (warp < kFirstEpiWarp) {
    if (warp == 0 && elect_one()) {
      // ---------------------------------------------------------- TMA producer
      const int nkb = (p.K + BK - 1) / BK, total = tiles[p.E] * p.splits;
      const uint32_t full = smem_u32(meta.full), empty = smem_u32(meta.empty);
      int s = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit t = unit_of(p, row0, tiles, u, nkb);
        const int arow = t.row0 + t.m0;
        for (int kb = t.kb0; kb < t.kb1; kb++) {
          if (!wait(empty + 8 * s, phase ^ 1, abort, p.status)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * STAGE_BYTES;
          uint8_t* sb = sa + A_BYTES;
          const int k0 = kb * BK;
          mbar_arrive_expect_tx(&meta.full[s], STAGE_BYTES);
          tma_load_2d(&tmA, &meta.full[s], sa, k0, arow);
          if (MODE == FP8_GATED && p.layout == MOE_GU_UNFUSED) {
            tma_load_3d(&tmG, &meta.full[s], sb, k0, t.n_blk * 128, t.e);
            tma_load_3d(&tmB, &meta.full[s], sb + BNH * BK, k0, t.n_blk * 128, t.e);
          } else if (MODE == FP8_GATED) {  // [E][2][N][K]: gate rows, then up rows
            tma_load_4d(&tmB, &meta.full[s], sb, k0, t.n_blk * 128, 0, t.e);
            tma_load_4d(&tmB, &meta.full[s], sb + BNH * BK, k0, t.n_blk * 128, 1, t.e);
          } else {
            tma_load_3d(&tmB, &meta.full[s], sb, k0, t.n_blk * BNB, t.e);
          }
          issued++;
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // Before the CTA may exit: every load issued has landed, and the last commit on every
      // stage's barrier has arrived (the drain barrier tells that the MMAs have ended, not
      // that the arrivals of other commits have been made), also after a role has given up.
      const uint32_t n = issued < (uint32_t)stages ? issued : (uint32_t)stages;
      const uint64_t t0 = global_timer();
      for (uint32_t j = issued - n; j < issued; j++) {
        const uint32_t at = 8 * (j % stages), parity = (j / stages) & 1;
        while (!(try_wait(full + at, parity) && try_wait(empty + at, parity))) {
          if (global_timer() - t0 > kTimeoutNs) {
            set_status(p.status, MOE_ERR_TIMEOUT);
            break;
          }
        }
      }
    } else if ((warp == 1 || warp == 3) && elect_one()) {
      // ---------------------------------------------------------- MMA issuers
      // Warp 1 takes the even blocks of K (quarters 0, 1), warp 3 the odd ones (2, 3): a
      // barrier answers after some hundred cycles on a busy SM, and one thread's waits for a
      // stage and two quarters took longer than the block's products.
      const int nkb = (p.K + BK - 1) / BK, total = tiles[p.E] * p.splits;
      const uint32_t odd = warp >> 1, q0 = 2 * odd;
      const uint32_t full = smem_u32(meta.full), tempty = smem_u32(meta.tempty) + 8 * q0;
      const uint32_t tmem_base = meta.tmem_slot + q0 * BNH;
      const uint64_t ad0 = sdesc_k_sw128(smem_u32(smem)), bd0 = sdesc_k_sw128(smem_u32(smem) + A_BYTES);
      int s = odd;
      uint32_t phase = 0, par = 1, n = 0;  // n: blocks of K so far
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit t = unit_of(p, row0, tiles, u, nkb);
        const int len = t.kb1 - t.kb0;
        for (int i = (n ^ odd) & 1; i < len; i += 2) {
          // all three are asked before the first answer is awaited
          const bool loaded = test_wait(full + 8 * s, phase), free0 = test_wait(tempty, par), free1 = test_wait(tempty + 8, par);
          if (!(loaded || wait(full + 8 * s, phase, abort, p.status)) || !(free0 || wait(tempty, par, abort, p.status))) {
            ok = false;
            break;
          }
          const uint64_t ad = ad0 + s * (STAGE_BYTES / 16), bd = bd0 + s * (STAGE_BYTES / 16);
#pragma unroll
          for (int h = 0; h < 2; h++) {
            if (h == 1 && !(free1 || wait(tempty + 8, par, abort, p.status))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t bh = bd + h * (BNH * BK / 16);  // rows 128 h .. of the stage's weights
#pragma unroll
            for (int kk = 0; kk < BK / 32; kk++) mma_f8(tmem_base + h * BNH, ad + 2 * kk, bh + 2 * kk, kk > 0);
            mma_commit(&meta.tfull[q0 + h]);
          }
          if (!ok) break;
          mma_commit(&meta.empty[s]);
          par ^= 1;
          if ((s += 2) >= stages) {
            s -= stages;
            phase ^= 1;
          }
        }
        n += len;
      }
      // all issued MMAs complete before the tensor memory is released
      mma_commit(&meta.drain);
      const uint64_t t0 = global_timer();
      while (!mbar_try_wait(&meta.drain, 0) && global_timer() - t0 < kTimeoutNs) {
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- scale products
      constexpr int kLoad = 4;  // blocks of K whose scales are loaded together, of four rows per lane
      const int nkb = (p.K + BK - 1) / BK, nbn = (p.N + 127) / 128, total = uniform(tiles[p.E] * p.splits);
      const uint32_t sfull = smem_u32(meta.sfull), sempty = smem_u32(meta.sempty);
      const bool vec = p.as_kb == 1 && p.as_row % 4 == 0 && (reinterpret_cast<uintptr_t>(p.as) & 15u) == 0;
      uint32_t n = 0;  // blocks of K so far
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit t = unit_of(p, row0, tiles, u, nkb);
        const BlockScales w = block_scales<MODE>(p, t, nbn, nkb);
        const int m0 = t.m0 + lane, kb1 = uniform(t.kb1);
        int row[4];  // rows past the last: any
#pragma unroll
        for (int r = 0; r < 4; r++) row[r] = t.row0 + min(m0 + 32 * r, t.rows - 1);
        for (int kb = uniform(t.kb0); ok && kb < kb1; kb += kLoad) {
          float xs[4][kLoad], wa[kLoad], wb[kLoad];
#pragma unroll
          for (int i = 0; i < kLoad; i++) {
            const int k = min(kb + i, kb1 - 1);
            wa[i] = __ldg(w.w0 + k);
            wb[i] = __ldg(w.w1 + k);
          }
          if (vec && kb % 4 == 0 && kb + kLoad <= kb1) {
#pragma unroll
            for (int r = 0; r < 4; r++) {
              const float4 a = __ldg(reinterpret_cast<const float4*>(p.as + row[r] * p.as_row + kb));
              xs[r][0] = a.x, xs[r][1] = a.y, xs[r][2] = a.z, xs[r][3] = a.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < kLoad; i++) {
              const int64_t k = (int64_t)min(kb + i, kb1 - 1) * p.as_kb;
#pragma unroll
              for (int r = 0; r < 4; r++) xs[r][i] = __ldg(p.as + row[r] * p.as_row + k);
            }
          }
#pragma unroll
          for (int i = 0; i < kLoad; i++) {
            if (kb + i < kb1) {
              const uint32_t g = (n / kScaleBatch) & 1;  // half of the ring
              if (n % kScaleBatch == 0) warp_wait(sempty + 8 * g, ((n / kScaleSlots) & 1) ^ 1, abort, p.status);
#pragma unroll
              for (int r = 0; r < 4; r++)
                meta.scale[n % kScaleSlots][lane + 32 * r] = make_float2(xs[r][i] * wa[i], xs[r][i] * wb[i]);
              if (++n % kScaleBatch == 0) {
                __syncwarp();
                warp_arrive(sfull + 8 * g, lane);
              }
            }
          }
          ok = __all_sync(0xffffffffu, *abort_flag == 0);
        }
      }
      if (n % kScaleBatch != 0) {  // the last blocks
        __syncwarp();
        warp_arrive(sfull + 8 * ((n / kScaleBatch) & 1), lane);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int nkb = (p.K + BK - 1) / BK, nbn = (p.N + 127) / 128, units = uniform(tiles[p.E] * p.splits);
    const int q = warp & 3, part = (warp - kFirstEpiWarp) >> 2;
    const int wb = part >> 1, half = part & 1;  // 64 columns of one of the tile's two weight blocks
    const int r_in_tile = q * 32 + lane;
    // The current block's quarter for this weight block and its barriers: quarters wb and
    // wb + 2 take turns by one address bit.
    const uint32_t lanes0 = meta.tmem_slot + ((uint32_t)(q * 32) << 16);
    uint32_t tq = lanes0 + wb * BNH + half * 64;
    uint32_t fq = smem_u32(meta.tfull) + 8 * wb, eq = smem_u32(meta.tempty) + 8 * wb;
    const uint32_t sfull = smem_u32(meta.sfull), sempty = smem_u32(meta.sempty);
    const uint32_t srow = smem_u32(meta.scale) + r_in_tile * 8 + wb * 4;
    uint32_t n = 0;  // blocks of K so far
    // A wait that gives up does not leave the loop: the warps of a quadrant meet in every
    // unit, so they walk the same list to its end (the waits then return at once).
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Unit t = unit_of(p, row0, tiles, u, nkb);
      const int kb0 = uniform(t.kb0), kb1 = uniform(t.kb1);
      const int m = uniform(t.m0);
      const bool valid = m + r_in_tile < t.rows;
      const int64_t grow = (int64_t)t.row0 + m + r_in_tile;
      const bool live = m + q * 32 < uniform(t.rows);  // the whole quadrant: some row of it exists
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; i++) acc[i] = 0.f;
      for (int left = kb1 - kb0; left > 0; left--, n++) {
        // this row's scale product of the block
        const uint32_t g = 8 * ((n / kScaleBatch) & 1);
        if (n % kScaleBatch == 0) warp_wait(sfull + g, (n / kScaleSlots) & 1, abort, p.status);
        float f;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(srow + (n % kScaleSlots) * (BM * 8)) : "memory");
        if ((n + 1) % kScaleBatch == 0) {
          __syncwarp();
          warp_arrive(sempty + g, lane);
        }
        warp_wait(fq, (n >> 1) & 1, abort, p.status);
        if (live) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; c++) {
            uint32_t v[16];
            tmem_ld16(tq + c * 16, v);
            tmem_ld_wait16(v);
            if (c == 3) {
              tc_fence_before();
              if (left > 1) warp_arrive(eq, lane);  // the last block's quarter is kept
            }
#pragma unroll
            for (int i = 0; i < 16; i++) acc[c * 16 + i] = fmaf(__uint_as_float(v[i]), f, acc[c * 16 + i]);
          }
        } else {
          warp_arrive(eq, lane);
        }
        tq ^= 2 * BNH;
        fq ^= 16;
        eq ^= 16;
      }
      // The sums go back to tensor memory, to this thread's columns of the quarter kept, for
      // the loops below to walk: unrolled over registers, what follows was some 2500
      // instructions, 6 to 17 thousand cycles for a tile, most of them waiting for code.
      if (live) {
#pragma unroll
        for (int i = 0; i < 4; i++) tmem_st16((tq ^ (2 * BNH)) + i * 16, &acc[i * 16]);
        tmem_st_wait();
      }

      // Columns of the kept quarters (weight block b's from column 0) in this thread's lane;
      // this warp's own 64 in runs of 16.
      const uint32_t kept = (tq ^ (2 * BNH)) - (wb * BNH + half * 64), el = eq ^ 16;
      auto fetch = [&](uint32_t at, float (&v)[16]) {
        uint32_t r[16];
        tmem_ld16(at, r);
        tmem_ld_wait16(r);
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
      };
      const int c0 = wb * BNH + half * 64;  // the warp's first column of the tile's 256
      if (p.splits > 1) {
        if (live) {
          float* out = p.partial + ((int64_t)t.sp * p.R + grow) * p.pitch + t.n_blk * BNB + c0;
#pragma unroll 1
          for (int c = 0; c < 4; c++) {
            float v[16];
            fetch(kept + c0 + c * 16, v);
            if (valid) {
              float4* o = reinterpret_cast<float4*>(out + c * 16);
#pragma unroll
              for (int i = 0; i < 4; i++) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
          }
          tc_fence_before();
          warp_arrive(el, lane);
        }
        continue;
      }
      if (MODE == FP8_LINEAR) {
        if (live) {
          const float w = p.roww && valid ? p.roww[grow] : 1.f;
          int64_t orow = grow;
          bool stored = valid;
          if (p.y_row && valid) {
            orow = p.y_row[grow];
            if (orow < 0 || orow >= p.R) {
              set_status(p.status, MOE_ERR_SHAPE);
              stored = false;
            }
          }
          const uint16_t* bias = p.bias ? p.bias + (int64_t)t.e * p.N : nullptr;
#pragma unroll 1
          for (int c = 0; c < 4; c++) {
            float v[16];
            fetch(kept + c0 + c * 16, v);
            const int n0 = t.n_blk * BNB + c0 + c * 16;
            if (bias) add_bias(v, bias, n0, p.N);
            uint16_t* out = p.y + orow * p.N + n0;
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
              if (stored && n0 + i < p.N)  // N is a multiple of 8
                *reinterpret_cast<uint4*>(out + i) =
                    make_uint4(pack_bf16x2(v[i] * w, v[i + 1] * w), pack_bf16x2(v[i + 2] * w, v[i + 3] * w),
                               pack_bf16x2(v[i + 4] * w, v[i + 5] * w), pack_bf16x2(v[i + 6] * w, v[i + 7] * w));
            }
          }
          tc_fence_before();
          warp_arrive(el, lane);
        }
        continue;
      }
      // gated / plain: activate (back into tensor memory), agree on each row's largest
      // magnitude per 128 features, round.  Gated: block 0 holds the gate sums and block 1
      // the up sums of 128 features, 32 of them for each of the quadrant's four warps;
      // plain: 128 features per block, 64 for each of its two.
      constexpr bool kGated = MODE == FP8_GATED;
      constexpr int kRuns = kGated ? 2 : 4;  // of 16 features
      const int col = kGated ? part * 32 : c0;
      const int grp = kGated ? t.n_blk : 2 * t.n_blk + wb;
      const int f_first = kGated ? t.n_blk * 128 + col : t.n_blk * BNB + col;
      if (live) {
        tc_fence_before();
        quadrant_sync(q);  // the quadrant's sums are in tensor memory
        tc_fence_after();
        const Fp8Bias bias = fp8_bias(MODE, p.layout, t.e, p.N, p.bias, p.gate_bias);
        float m = 0.f;
#pragma unroll 1
        for (int c = 0; c < kRuns; c++) {
          float g[16], u[16];
          fetch(kept + col + c * 16, g);
          if (kGated) fetch(kept + BNH + col + c * 16, u);
          const int f0 = f_first + c * 16;
          if (bias.g) add_bias(g, bias.g, f0, p.N);
          if (bias.u) add_bias(u, bias.u, f0, p.N);
          m = fmaxf(m, activate<kGated>(g, u, p.act, f0, p.N));
          tmem_st16(kept + col + c * 16, g);
        }
        meta.amax[part][r_in_tile] = m;
        tmem_st_wait();
        quadrant_sync(q);
        m = fmaxf(meta.amax[part][r_in_tile], meta.amax[part ^ 1][r_in_tile]);
        if (kGated) m = fmaxf(m, fmaxf(meta.amax[part ^ 2][r_in_tile], meta.amax[part ^ 3][r_in_tile]));
        const Fp8Scale s = fp8_scale_of(m);
        if (valid && (kGated ? part == 0 : half == 0) && grp < nbn) p.hs[grow * p.hs_row + (int64_t)grp * p.hs_grp] = s.s;
#pragma unroll 1
        for (int c = 0; c < kRuns; c++) {
          float h[16];
          fetch(kept + col + c * 16, h);
          const int f0 = f_first + c * 16;
          if (valid && f0 < p.N)  // N is a multiple of 16
            *reinterpret_cast<uint4*>(p.hq + grow * p.N + f0) =
                make_uint4(fp8_round4(h, s), fp8_round4(h + 4, s), fp8_round4(h + 8, s), fp8_round4(h + 12, s));
        }
        tc_fence_before();
        quadrant_sync(q);  // both quarters and the maxima are read before they are written again
        warp_arrive(el, lane);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(meta.tmem_slot, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side
bool map_bytes(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
               const uint32_t* box) {
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Weight stack [E, N, K], `rows` rows per box.
bool map_stack(CUtensorMap* m, const void* base, uint64_t K, uint64_t N, uint64_t E, uint32_t rows) {
  const uint64_t dims[3] = {K, N, E};
  const uint64_t strides[2] = {K, N * K};
  const uint32_t box[3] = {BK, rows, 1};
  return map_bytes(m, base, 3, dims, strides, box);
}

template <int MODE, int ABOX>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& g, const Fp8GemmArgs& p, cudaStream_t st) {
  const int stages = stages_for(ABOX, p.E);
  const int smem = 1024 + stages * stage_bytes(ABOX) + meta_bytes(p.E);
  // (the most, whatever E needs: another thread may launch the same kernel for more groups)
  cudaError_t e =
      cudaFuncSetAttribute(fp8_gemm_kernel<MODE, ABOX>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.max_tiles * p.splits;
  const unsigned grid = (unsigned)(units < p.num_sms ? units : p.num_sms);
  return launch_ordered(fp8_gemm_kernel<MODE, ABOX>, grid, kThreads, smem, st, a, b, g, p, stages);
}

template <int MODE>
cudaError_t launch_mode(const Fp8GemmArgs& p, cudaStream_t st) {
  // no group has more than R rows: small batches load a shorter row tile and leave room
  // for more weight stages (the accumulator rows past it are never stored); 16 experts of
  // 2880 x 2880, against tiles of 128: 32 rows 117, 123 us, 64 rows 119, 121
  const uint32_t abox = p.R <= 32 ? 32 : p.R <= 64 ? 64 : 128;
  constexpr uint32_t brows = MODE == FP8_GATED ? BNH : BNB;  // weight rows per box
  CUtensorMap a, b, g;
  const uint64_t dims[2] = {(uint64_t)p.K, (uint64_t)p.R};
  const uint64_t strides[1] = {(uint64_t)p.K};
  const uint32_t box[2] = {BK, abox};
  bool ok = map_bytes(&a, p.a, 2, dims, strides, box);
  if (MODE == FP8_GATED && p.layout == MOE_GU_UNFUSED) {
    ok = ok && map_stack(&b, p.w, p.K, p.N, p.E, brows) && map_stack(&g, p.wg, p.K, p.N, p.E, brows);
  } else if (MODE == FP8_GATED) {
    const uint64_t K = p.K, N = p.N;
    const uint64_t d4[4] = {K, N, 2, (uint64_t)p.E};
    const uint64_t s4[3] = {K, N * K, 2 * N * K};
    const uint32_t b4[4] = {BK, brows, 1, 1};
    ok = ok && map_bytes(&b, p.w, 4, d4, s4, b4);
    g = b;
  } else {
    ok = ok && map_stack(&b, p.w, p.K, p.N, p.E, brows);
    g = b;
  }
  if (!ok) return cudaErrorInvalidValue;
  if (abox == 32) return launch<MODE, 32>(a, b, g, p, st);
  if (abox == 64) return launch<MODE, 64>(a, b, g, p, st);
  return launch<MODE, 128>(a, b, g, p, st);
}

}  // namespace

int fp8_splits(int mode, int64_t R, int64_t E, int64_t N, int64_t K, int sms) {
  // In blocks of K of one tile (0.47 us): a unit's fixed cost, the reduction's launch, and the
  // partial sums written and read at 4.2 TB/s.  Split and whole: 1 row of 7168 x 4096 22.5,
  // 32.8 us; 384 rows 32.8, 41.0; 1 row through experts of 4096 x 2048 41, 47; 512 rows of
  // 4096 x 4096 (not split by this) 33, 29.
  constexpr int kUnit = 8, kReduce = 8, kMost = 8;
  constexpr double kBytes = 2e6;
  const int64_t tiles = fp8_m_tiles(R, E) * fp8_n_tiles(mode, N), nkb = (K + BK - 1) / BK;
  if (tiles <= 0 || tiles >= sms) return 1;
  const double sums = (double)R * fp8_n_tiles(mode, N) * BNB * 8 / kBytes;
  int best = 1;
  double best_cost = nkb + kUnit;
  for (int s = 2; s <= kMost && 2 * s <= nkb; s++) {
    const double cost = (double)((tiles * s + sms - 1) / sms * ((nkb + s - 1) / s + kUnit) + kReduce) + s * sums;
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& p, cudaStream_t st) {
  if (p.max_tiles == 0) return cudaSuccess;
  if (p.mode == FP8_GATED) return launch_mode<FP8_GATED>(p, st);
  if (p.mode == FP8_PLAIN) return launch_mode<FP8_PLAIN>(p, st);
  return launch_mode<FP8_LINEAR>(p, st);
}

}  // namespace moe
