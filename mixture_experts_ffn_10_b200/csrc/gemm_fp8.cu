// gemm_fp8.cu -- grouped GEMM of e4m3 operands with an fp32 scale per 128 columns of a
// row (activations) and per 128 x 128 block (weights), on tcgen05 kind::f8f6f4.
//
//   acc[r, n] = sum_b xs[r, b] ws[n / 128, b] D_b[r, n],   D_b = sum_{k in block b} xq[r, k] wq[n, k]
//
// The tensor cores form D_b exactly as an fp32 accumulation over one block of K (four
// K = 32 steps) in tensor memory; the scales differ from block to block and row to row,
// so each D_b is read back and added to an fp32 accumulator with its scale product.  Rows
// are the MMA's M: a thread of an epilogue warp owns one row and 128 columns of two
// weight blocks, so a block costs it two scale products and 128 multiply-adds (64
// packed ones), and the accumulators live in its registers for the whole K loop.
// (With the weights as M the row scales would differ from register to register and each
// multiply-add would need an operand from shared memory.)  Two 256-column halves of
// tensor memory alternate: while block b is added up, block b + 1 is multiplied.
//
// Work: tiles of 128 rows x 256 weight rows (128 gate and their 128 up rows, or 256 plain
// rows), persistent CTAs, one per SM; the tile list is made on the device from the
// groups' row counts.  Warps: 0 TMA producer (128 x 128 and 256 x 128 bytes per stage,
// 128-byte swizzle), 1 TMEM and MMA issue, 4-11 epilogue (TMEM lane quadrant x column
// half).  The epilogue's 128 accumulators a thread do not fit the 168 registers that
// twelve warps leave each: the first four warps hand theirs over (setmaxnreg, 56 + 2 x
// 224 = 3 x 168).  Every wait is bounded (2 s) and reports MOE_ERR_TIMEOUT.
#include "fp8.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int BM = kFp8BM;
constexpr int BK = kFp8Block;     // bytes of K per stage: one scale block
constexpr int BNB = 256;          // weight rows per tile
constexpr int B_BYTES = BNB * BK;
constexpr int ACC_COLS = BNB;
constexpr int TMEM_COLS = 2 * ACC_COLS;
constexpr int kEpiWarps = 8;
constexpr int kFirstEpiWarp = 4;
constexpr int kThreads = (kFirstEpiWarp + kEpiWarps) * 32;
constexpr int kControlRegs = 56, kEpiRegs = 224;  // of 168 at launch: 4 x 56 + 8 x 224 = 12 x 168
constexpr int kMaxStages = 6;
constexpr int kSmemLimit = 232448;
// kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A and B e4m3 (format 0), K-major, N >> 3
// in bits 17-22, M >> 4 in 24-28.
constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(BNB >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);

// Shared memory after the stages: barriers, the row maxima the two column halves of a
// tile exchange, the groups' first rows and tile prefixes.
struct Meta {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
  uint32_t tmem_slot;
  int abort_flag;
  float amax[2][2][BM];  // [group of 128 columns][column half][row]
};

constexpr int stage_bytes(int abox) { return abox * BK + B_BYTES; }
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

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// acc (two floats) += {a, b} * f (two floats)
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t a, uint32_t b, uint64_t f) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(a), "r"(b), "l"(f));
}
__device__ __forceinline__ uint64_t twice(float f) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(f));
  return r;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// The two column halves (warps w and w + 4) of a TMEM lane quadrant meet.
__device__ __forceinline__ void quadrant_sync(int q) { asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory"); }

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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; s++) {
      mbar_init(&meta.full[s], 1);
      mbar_init(&meta.empty[s], 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(&meta.tfull[b], 1);
      mbar_init(&meta.tempty[b], kEpiWarps);
    }
    mbar_init(&meta.drain, 1);
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
  pdl_enter();
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
  const uint32_t tmem_base = meta.tmem_slot;
  const int nkb = (p.K + BK - 1) / BK;
  const int total = tiles[p.E] * p.splits;

  if (warp < kFirstEpiWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- TMA producer
      int s = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit t = unit_of(p, row0, tiles, u, nkb);
        for (int kb = t.kb0; kb < t.kb1; kb++) {
          if (!mbar_wait(&meta.empty[s], phase ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&meta.full[s], STAGE_BYTES);
          uint8_t* sa = smem + s * STAGE_BYTES;
          uint8_t* sb = sa + A_BYTES;
          const int k0 = kb * BK;
          tma_load_2d(&tmA, &meta.full[s], sa, k0, t.row0 + t.m0);
          if (MODE == FP8_GATED && p.layout == MOE_GU_UNFUSED) {
            tma_load_3d(&tmG, &meta.full[s], sb, k0, t.n_blk * 128, t.e);
            tma_load_3d(&tmB, &meta.full[s], sb + B_BYTES / 2, k0, t.n_blk * 128, t.e);
          } else if (MODE == FP8_GATED) {  // [E][2][N][K]: gate rows, then up rows
            tma_load_4d(&tmB, &meta.full[s], sb, k0, t.n_blk * 128, 0, t.e);
            tma_load_4d(&tmB, &meta.full[s], sb + B_BYTES / 2, k0, t.n_blk * 128, 1, t.e);
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
      // every load issued has landed before the CTA may exit: the last `stages` of them
      const uint32_t n = issued < (uint32_t)stages ? issued : (uint32_t)stages;
      for (uint32_t j = issued - n; j < issued; j++) {
        const uint64_t t0 = global_timer();
        while (!mbar_try_wait(&meta.full[j % stages], (j / stages) & 1) && global_timer() - t0 < kTimeoutNs) {
        }
      }
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      int s = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit t = unit_of(p, row0, tiles, u, nkb);
        for (int kb = t.kb0; kb < t.kb1; kb++, it++) {
          const int acc = it & 1;
          if (!mbar_wait(&meta.tempty[acc], ((it >> 1) & 1) ^ 1, abort_flag, p.status) ||
              !mbar_wait(&meta.full[s], phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * STAGE_BYTES);
          const uint64_t ad = sdesc_k_sw128(sa), bd = sdesc_k_sw128(sa + A_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 32; kk++) mma_f8(tmem_base + acc * ACC_COLS, ad + 2 * kk, bd + 2 * kk, kk > 0);
          mma_commit(&meta.empty[s]);
          mma_commit(&meta.tfull[acc]);
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // all issued MMAs complete before the tensor memory is released
      mma_commit(&meta.drain);
      const uint64_t t0 = global_timer();
      while (!mbar_try_wait(&meta.drain, 0) && global_timer() - t0 < kTimeoutNs) {
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - kFirstEpiWarp) >> 2;
    const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + half * 64;
    const int nbn = (p.N + 127) / 128;
    uint32_t it = 0;
    // A wait that gives up does not leave the loop: both halves of a quadrant meet in
    // every unit, so they walk the same list to its end (the waits then return at once).
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
      const Unit t = unit_of(p, row0, tiles, u, nkb);
      const int r_in_tile = q * 32 + lane;
      const bool valid = t.m0 + r_in_tile < t.rows;
      const int64_t grow = (int64_t)t.row0 + t.m0 + r_in_tile;
      const bool live = t.m0 + q * 32 < t.rows;  // whole warp: some row of this quadrant exists
      // scales: this row's, and those of the tile's two weight blocks
      const float* as = p.as + (valid ? grow : (int64_t)t.row0) * nkb;
      const float *w0, *w1;
      if (MODE == FP8_GATED) {
        const bool cat = p.layout != MOE_GU_UNFUSED;
        w0 = cat ? p.ws + ((int64_t)t.e * 2 * nbn + t.n_blk) * nkb : p.wgs + ((int64_t)t.e * nbn + t.n_blk) * nkb;
        w1 = cat ? w0 + (int64_t)nbn * nkb : p.ws + ((int64_t)t.e * nbn + t.n_blk) * nkb;
      } else {
        w0 = p.ws + ((int64_t)t.e * nbn + 2 * t.n_blk) * nkb;
        w1 = 2 * t.n_blk + 1 < nbn ? w0 + nkb : w0;
      }
      uint64_t acc[2][32];  // two sets of 64 columns: half * 64 .. of each weight block
#pragma unroll
      for (int i = 0; i < 32; i++) acc[0][i] = acc[1][i] = 0;
      float xs = 0.f, s0 = 0.f, s1 = 0.f;
      if (live && t.kb0 < t.kb1) {
        xs = __ldg(as + t.kb0);
        s0 = __ldg(w0 + t.kb0);
        s1 = __ldg(w1 + t.kb0);
      }
      for (int kb = t.kb0; kb < t.kb1; kb++, it++) {
        const int buf = it & 1;
        const uint64_t f[2] = {twice(xs * s0), twice(xs * s1)};
        if (live && kb + 1 < t.kb1) {
          xs = __ldg(as + kb + 1);
          s0 = __ldg(w0 + kb + 1);
          s1 = __ldg(w1 + kb + 1);
        }
        mbar_wait(&meta.tfull[buf], (it >> 1) & 1, abort_flag, p.status);
        __syncwarp();
        tc_fence_after();
        if (live) {
#pragma unroll
          for (int c = 0; c < 4; c++) {
            uint32_t v[32];
            tmem_ld32(tb + buf * ACC_COLS + (c >> 1) * 128 + (c & 1) * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i++) fma2(acc[c >> 1][(c & 1) * 16 + i], v[2 * i], v[2 * i + 1], f[c >> 1]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&meta.tempty[buf]);
      }

      if (p.splits > 1) {
        if (valid) {
#pragma unroll
          for (int j = 0; j < 2; j++) {
            float4* out = reinterpret_cast<float4*>(p.partial + ((int64_t)t.sp * p.R + grow) * p.pitch + t.n_blk * BNB +
                                                    j * 128 + half * 64);
#pragma unroll
            for (int i = 0; i < 16; i++)
              out[i] = make_float4(lo_of(acc[j][2 * i]), hi_of(acc[j][2 * i]), lo_of(acc[j][2 * i + 1]),
                                   hi_of(acc[j][2 * i + 1]));
          }
        }
        continue;
      }
      if (MODE == FP8_LINEAR) {
        if (valid) {
          const float w = p.roww ? p.roww[grow] : 1.f;
#pragma unroll
          for (int j = 0; j < 2; j++) {
            const int n0 = t.n_blk * BNB + j * 128 + half * 64;
            const uint16_t* bias = p.bias ? p.bias + (int64_t)t.e * p.N : nullptr;
            uint16_t* out = p.y + grow * p.N;
#pragma unroll
            for (int i = 0; i < 8; i++) {
              if (n0 + 8 * i >= p.N) break;  // N is a multiple of 8
              float b[8];
#pragma unroll
              for (int c = 0; c < 8; c++) b[c] = bias ? bf16_to_f32(__ldg(bias + n0 + 8 * i + c)) : 0.f;
              uint32_t o[4];
#pragma unroll
              for (int c = 0; c < 4; c++)
                o[c] = pack_bf16x2((lo_of(acc[j][4 * i + c]) + b[2 * c]) * w, (hi_of(acc[j][4 * i + c]) + b[2 * c + 1]) * w);
              *reinterpret_cast<uint4*>(out + n0 + 8 * i) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        continue;
      }
      // gated / plain: activate, agree on each row's largest magnitude per 128 features,
      // round.  Gated: one group per tile (set 0 gate, set 1 up); plain: two.
      constexpr int kGroups = MODE == FP8_GATED ? 1 : 2;
      float h[kGroups][64];
#pragma unroll
      for (int j = 0; j < kGroups; j++) {
        const int f0 = (MODE == FP8_GATED ? t.n_blk * 128 : t.n_blk * BNB + j * 128) + half * 64;
        float m = 0.f;
        const Fp8Bias b = fp8_bias(MODE, p.layout, t.e, p.N, p.bias, p.gate_bias);
#pragma unroll
        for (int i = 0; i < 64; i++) {
          const float a0 = i & 1 ? hi_of(acc[j][i / 2]) : lo_of(acc[j][i / 2]);
          const bool in = f0 + i < p.N;
          const float g = a0 + (in && b.g ? bf16_to_f32(__ldg(b.g + f0 + i)) : 0.f);
          if (MODE == FP8_GATED) {
            const float a1 = i & 1 ? hi_of(acc[1][i / 2]) : lo_of(acc[1][i / 2]);
            const float up = a1 + (in && b.u ? bf16_to_f32(__ldg(b.u + f0 + i)) : 0.f);
            h[j][i] = fp8_act(p.act, g, true) * (fp8_up(p.act, up) + p.act.beta);
          } else {
            h[j][i] = fp8_act(p.act, g, false);
          }
          if (!in) h[j][i] = 0.f;
          m = fmaxf(m, fabsf(h[j][i]));
        }
        meta.amax[j][half][r_in_tile] = m;
      }
      quadrant_sync(q);
#pragma unroll
      for (int j = 0; j < kGroups; j++) {
        const int grp = MODE == FP8_GATED ? t.n_blk : 2 * t.n_blk + j;
        const int f0 = grp * 128 + half * 64;
        const float s = fp8_scale(fmaxf(meta.amax[j][0][r_in_tile], meta.amax[j][1][r_in_tile]));
        const float inv = __frcp_rn(s);
        if (valid && grp < nbn) {
          if (half == 0) p.hs[grow * nbn + grp] = s;
          uint8_t* out = p.hq + grow * p.N + f0;
#pragma unroll
          for (int c = 0; c < 4; c++) {
            if (f0 + 16 * c >= p.N) break;  // N is a multiple of 16
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const float* x = &h[j][16 * c + 4 * i];
              o[i] = fp8_pack4(fp8_quotient(x[0], s, inv), fp8_quotient(x[1], s, inv), fp8_quotient(x[2], s, inv),
                               fp8_quotient(x[3], s, inv));
            }
            *reinterpret_cast<uint4*>(out + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      quadrant_sync(q);  // the maxima are read before the next tile's are written
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
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
  cudaError_t e = cudaFuncSetAttribute(fp8_gemm_kernel<MODE, ABOX>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.max_tiles * p.splits;
  const unsigned grid = (unsigned)(units < p.num_sms ? units : p.num_sms);
  return launch_pdl(fp8_gemm_kernel<MODE, ABOX>, grid, kThreads, smem, st, a, b, g, p, stages);
}

template <int MODE>
cudaError_t launch_mode(const Fp8GemmArgs& p, cudaStream_t st) {
  // no group has more than R rows: small batches load a shorter row tile and leave room
  // for more weight stages (the accumulator rows past it are never stored)
  const uint32_t abox = p.R <= 32 ? 32 : p.R <= 64 ? 64 : 128;
  CUtensorMap a, b, g;
  const uint64_t dims[2] = {(uint64_t)p.K, (uint64_t)p.R};
  const uint64_t strides[1] = {(uint64_t)p.K};
  const uint32_t box[2] = {BK, abox};
  bool ok = map_bytes(&a, p.a, 2, dims, strides, box);
  if (MODE == FP8_GATED && p.layout == MOE_GU_UNFUSED) {
    ok = ok && map_stack(&b, p.w, p.K, p.N, p.E, 128) && map_stack(&g, p.wg, p.K, p.N, p.E, 128);
  } else if (MODE == FP8_GATED) {
    const uint64_t K = p.K, N = p.N;
    const uint64_t d4[4] = {K, N, 2, (uint64_t)p.E};
    const uint64_t s4[3] = {K, N * K, 2 * N * K};
    const uint32_t b4[4] = {BK, 128, 1, 1};
    ok = ok && map_bytes(&b, p.w, 4, d4, s4, b4);
    g = b;
  } else {
    ok = ok && map_stack(&b, p.w, p.K, p.N, p.E, BNB);
    g = b;
  }
  if (!ok) return cudaErrorInvalidValue;
  if (abox == 32) return launch<MODE, 32>(a, b, g, p, st);
  if (abox == 64) return launch<MODE, 64>(a, b, g, p, st);
  return launch<MODE, 128>(a, b, g, p, st);
}

}  // namespace

int fp8_splits(int mode, int64_t R, int64_t E, int64_t N, int64_t K, int sms) {
  if (R > kSplitMaxRows) return 1;
  return choose_splits(fp8_m_tiles(R, E) * fp8_n_tiles(mode, N), (int)((K + BK - 1) / BK), sms);
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& p, cudaStream_t st) {
  if (p.max_tiles == 0) return cudaSuccess;
  if (p.mode == FP8_GATED) return launch_mode<FP8_GATED>(p, st);
  if (p.mode == FP8_PLAIN) return launch_mode<FP8_PLAIN>(p, st);
  return launch_mode<FP8_LINEAR>(p, st);
}

}  // namespace moe
