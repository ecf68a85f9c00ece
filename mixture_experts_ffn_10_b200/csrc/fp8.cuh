// fp8.cuh -- e4m3 operands with an fp32 scale per block of 128: the rounding to e4m3,
// and the launchers of the FP8 kernels (quantisation, grouped products, reductions).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

constexpr int kFp8Block = 128;    // columns (and weight rows) that share a scale
constexpr int kFp8BM = 128;       // rows per tile of the FP8 grouped GEMM (UMMA M)
// Routed rows that one block sorts: one launch for three, but one warp places the rows one
// after the other.  The layer of 32 experts of 1024 x 512 with one expert a token, sorted by
// one block and by three launches: 77 rows 33.0, 35.1 us, 128 rows 33.0, 33.0, 256 rows 34.2,
// 33.0, 512 rows 40.2, 33.7.
constexpr int kFp8OneBlockRows = 128;
constexpr int kFp8MinNK = 16;     // K (and F) multiple: 16-byte rows

// SMs of the current device.
int device_sms();

// Where an FP8 layer keeps its operands in the workspace (bytes from the region's start).
struct Fp8Regions {
  size_t xq, xs, hq, hs, tiles, total;  // tiles: the shared expert's tile prefix [E + 2]
};
inline Fp8Regions fp8_regions(int64_t R, int64_t d, int64_t F, int64_t E) {
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  Fp8Regions r;
  r.xq = 0;
  r.xs = up(r.xq + (size_t)R * d);
  r.hq = up(r.xs + (size_t)R * ((d + 127) / 128) * 4);
  r.hs = up(r.hq + (size_t)R * F);
  r.tiles = up(r.hs + (size_t)R * ((F + 127) / 128) * 4);
  r.total = up(r.tiles + (size_t)(E + 2) * 4);
  return r;
}
// tiles[0 .. E] = 0, tiles[E + 1] = n: the prefix of a tile list that holds the shared
// segment's n tiles alone (the bf16 shared expert beside FP8 experts).
cudaError_t launch_shared_tiles(int32_t* tiles, int E, int n, cudaStream_t st);

// ---------------------------------------------------------------- rounding to e4m3
// The scale of a block of largest magnitude amax, max(amax, 2^-100) / 448 correctly rounded:
// a quotient by the rounded reciprocal, corrected once by its exact remainder (Markstein's
// division; a fifth of the instructions of __fdiv_rn, which the tests find it equal to).
// An infinite amax gives an infinite scale.
__device__ __forceinline__ float fp8_scale(float amax) {
  constexpr float r = 1.f / 448.f;
  const float a = fmaxf(amax, 0x1p-100f);
  const float q = a * r;
  const float rem = fmaf(-448.f, q, a);
  return rem == rem ? fmaf(rem, r, q) : q;
}

// What rounding a block needs: its scale and the scale's reciprocal, a little too small and
// a little too large (2^-21 relative; the instruction's own error is 2^-23).
struct Fp8Scale {
  float s, lo, hi;
};
__device__ __forceinline__ Fp8Scale fp8_scale_of(float amax) {
  const float s = fp8_scale(amax);
  const uint32_t u = __float_as_uint(s);
  if ((u & 0x7fffffu) == 0 && u < 0x7f800000u) {
    // 2^k: the quotients by it are exact as they are (and ties are frequent)
    const float inv = __uint_as_float(0x7f000000u - u);
    return Fp8Scale{s, inv, inv};
  }
  const float inv = __fdividef(1.f, s);
  return Fp8Scale{s, inv * (1.f - 0x1p-21f), inv * (1.f + 0x1p-21f)};
}

// A float that the hardware conversion (nearest even, saturating) takes to the e4m3 value
// nearest to the real quotient x / s.  t = x hi is within eight units in the last place of
// x / s, so the two round alike unless a point halfway between e4m3 values is that near.
// Such points (and the e4m3 values) have at most four fraction bits: their low 19 bits are
// zero.  Next to one, m, the residual x - m s (exact in sign in one fma: m s has 29 bits)
// tells on which side of m the quotient is.
__device__ __forceinline__ float fp8_quotient(float x, float s, float hi) {
  float t = x * hi;
  const uint32_t u = __float_as_uint(t) + 16u;
  if ((u & 0x7ffffu) < 32u) {
    const uint32_t m = u & ~0x7ffffu;
    const float r = fmaf(-__uint_as_float(m), s, x);  // NaN (t stays) for NaN x and for infinite s
    const bool neg = (m >> 31) != 0;
    if (r == 0.f) t = __uint_as_float(m);
    if (r > 0.f) t = __uint_as_float(neg ? m - 1u : m + 1u);
    if (r < 0.f) t = __uint_as_float(neg ? m + 1u : m - 1u);
  }
  return t;
}

// Four floats as e4m3, the first in the low byte.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// x[0 .. 3] / s as e4m3.  The real quotients lie between x lo and x hi; rounding is
// monotone, so where both round to the same value, that is the answer (all but a few in ten
// thousand: no test of each value for the neighbourhood of a halfway point is needed).
__device__ __forceinline__ uint32_t fp8_round4(const float* x, const Fp8Scale& f) {
  const uint32_t lo = fp8_pack4(x[0] * f.lo, x[1] * f.lo, x[2] * f.lo, x[3] * f.lo);
  const uint32_t hi = fp8_pack4(x[0] * f.hi, x[1] * f.hi, x[2] * f.hi, x[3] * f.hi);
  if (lo == hi) return hi;
  return fp8_pack4(fp8_quotient(x[0], f.s, f.hi), fp8_quotient(x[1], f.s, f.hi), fp8_quotient(x[2], f.s, f.hi),
                   fp8_quotient(x[3], f.s, f.hi));
}

// Rounding bf16 values, whose block's largest magnitude is a bf16 value (or the floor
// 2^-100): no bracket is needed.  With eight-bit significands p of x and a of amax, 448 x /
// amax = 7 p 2^i / a equals a halfway point odd 2^j (odd < 32) or differs from it by 1 / (31 *
// 255) > 2^-13 relative at least.  And x / s differs from 448 x / amax by the rounding of s
// alone, a common factor 1 - d, |d| <= 2^-24: if s was rounded, every tie of the block falls to
// the same side, which a factor 1 +- 2^-16 on the quotients decides without touching any
// other value; if s is exact, ties go to the even value, for which the quotient itself has
// to be: x inv, corrected by its remainder.  (Such ties are one value in two hundred of
// normal data, one warp in two meets some.)
struct Fp8ScaleBf16 {
  float s, inv, fix;  // fix: factor of the remainder's correction, 0 where none is due
};
__device__ __forceinline__ Fp8ScaleBf16 fp8_scale_of_bf16(float amax) {
  const float s = fp8_scale(amax), inv = __fdividef(1.f, s);
  const float rem = fmaf(-448.f, s, fmaxf(amax, 0x1p-100f));  // exact; > 0: s was rounded down
  if (rem == 0.f) return Fp8ScaleBf16{s, inv, inv};
  return Fp8ScaleBf16{s, inv * (rem > 0.f ? 1.f + 0x1p-16f : 1.f - 0x1p-16f), 0.f};
}
// Whole warp (lanes may hold different blocks): 16 values.
__device__ __forceinline__ void fp8_round16_bf16(const float (&x)[16], const Fp8ScaleBf16& f, uint32_t (&w)[4]) {
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; i++) t[i] = x[i] * f.inv;
  if (__any_sync(0xffffffffu, f.fix != 0.f)) {
#pragma unroll
    for (int i = 0; i < 16; i++) {
      // (keeps -0; a lane without a correction keeps its quotients: 0 times an infinite scale is no 0)
      const float c = fmaf(-fmaf(t[i], f.s, -x[i]), f.fix, t[i]);
      if (f.fix != 0.f) t[i] = c;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++) w[i] = fp8_pack4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
}

// ---------------------------------------------------------------- activation
// act(g) in fp32 (h is rounded to e4m3 next to it, a step of 2^-4: the hardware tanh of the
// bf16 epilogues, 5e-4 off, would move too many values over a rounding border); the SiLU
// limit applies to gated experts only.
__device__ __forceinline__ float fp8_act(const ActParams& a, float g, bool gated) {
  switch (a.act) {
    case MOE_ACT_SILU:
      if (gated && a.limit > 0.f) g = fminf(g, a.limit);
      return __fdividef(g, 1.f + __expf(-a.alpha * g));
    case MOE_ACT_GELU_ERF: return 0.5f * g * (1.f + erff(g * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH: {  // 0.5 (1 + tanh z) = sigmoid(2 z)
      const float z2 = 2.f * 0.79788456080286536f * fmaf(0.044715f * g, g * g, g);
      return __fdividef(g, 1.f + __expf(-z2));
    }
    case MOE_ACT_RELU: return fmaxf(g, 0.f);
    default: return g;
  }
}
__device__ __forceinline__ float fp8_up(const ActParams& a, float u) {
  return a.act == MOE_ACT_SILU && a.limit > 0.f ? fminf(fmaxf(u, -a.limit), a.limit) : u;
}

// Bias rows of group e: of the gate (or plain) and of the up values; null if absent.
struct Fp8Bias {
  const uint16_t *g, *u;
};
__device__ __forceinline__ Fp8Bias fp8_bias(int mode, int layout, int e, int64_t N, const uint16_t* bias,
                                            const uint16_t* gate_bias) {
  if (mode != 0 /*FP8_GATED*/) return Fp8Bias{bias ? bias + e * N : nullptr, nullptr};
  if (layout == MOE_GU_UNFUSED)
    return Fp8Bias{gate_bias ? gate_bias + e * N : nullptr, bias ? bias + e * N : nullptr};
  return Fp8Bias{bias ? bias + 2 * e * N : nullptr, bias ? bias + (2 * e + 1) * N : nullptr};
}

// ---------------------------------------------------------------- quantisation
cudaError_t launch_fp8_quantize(int bf16, int64_t rows, int64_t K, const void* x, int64_t pitch, uint8_t* q,
                                float* scales, cudaStream_t st);
cudaError_t launch_fp8_quantize_weights(int bf16, int64_t E, int64_t N, int64_t K, const void* w, uint8_t* q,
                                        float* scales, cudaStream_t st);

// Row pos[t, j] of xq / xs = x[t] quantised (times the row's weight for weigh-inputs).
struct Fp8GatherArgs {
  const uint16_t* x;    // [T, d] bf16
  const int32_t* pos;   // [T, k]
  const float* roww;    // [R]
  uint8_t* xq;          // [R, d]
  float* xs;            // [ceil(d / 128), R]
  int R, d, T, k, weigh_inputs;
  int* status;
  uint16_t* y;          // k = 1 with rows written in place: [T, d], zeros for a token without an expert; or null
};
cudaError_t launch_fp8_gather(const Fp8GatherArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- grouped products
enum { FP8_GATED = 0, FP8_PLAIN = 1, FP8_LINEAR = 2 };  // what the epilogue makes of the accumulators

// One grouped GEMM: rows of group e are the cnt[e] rows after those of groups 0 .. e-1.
//   GATED   h = act(W_gate x + b) (W_up x + b), quantised per 128 features
//   PLAIN   h = act(W x + b), quantised likewise
//   LINEAR  y = (W x + b) * roww, bf16
// With splits > 1 the K blocks of a tile are divided among that many work units, which
// write fp32 partial sums partial[split][row][column] (pitch floats per row; column
// 256 n_blk + c is accumulator column c of tile column n_blk) for a reduction kernel.
struct Fp8GemmArgs {
  int mode;
  int E, R, K, N;             // N: features (gated, plain) or outputs (linear)
  const int32_t* cnt;         // [E], or null: one group of R rows
  const uint8_t* a;           // [R, K]
  const float* as;            // scale of row r and block b of K at r * as_row + b * as_kb
  int64_t as_row, as_kb;
  int layout;                 // gated: MOE_GU_CONCAT or MOE_GU_UNFUSED
  const uint8_t* w;           // [E, N, K]; concat: [E, 2N, K]; unfused: the up rows
  const float* ws;            // [E, ceil(N / 128), ceil(K / 128)]; concat: [E, 2 ceil(N / 128), ceil(K / 128)]
  const uint8_t* wg;          // unfused: the gate rows [E, N, K]
  const float* wgs;
  const uint16_t* bias;       // bf16, rows as w; or null
  const uint16_t* gate_bias;  // unfused: [E, N] or null
  ActParams act;
  const float* roww;          // linear: [R] or null (1)
  uint8_t* hq;                // [R, N]
  float* hs;                  // scale of row r and group g of h at r * hs_row + g * hs_grp
  int64_t hs_row, hs_grp;
  uint16_t* y;                // [R, N]
  const int32_t* y_row;       // linear: row r goes to row y_row[r] of y, or null (row r)
  int splits;
  float* partial;
  int pitch;
  int max_tiles;              // upper bound of the tile count
  int num_sms;
  int* status;
  int clear_status;           // the kernel starts by clearing *status (a timeout comes seconds later)
};
cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t st);

// N tiles of a GEMM: 256 accumulator columns (128 gated features).
inline int fp8_n_tiles(int mode, int64_t N) { return (int)((N + (mode == FP8_GATED ? 127 : 255)) / (mode == FP8_GATED ? 128 : 256)); }
// Upper bound of the row tiles of R rows in E groups: r rows fill at most (r + 127) / 128.
inline int64_t fp8_m_tiles(int64_t R, int64_t E) { return (R + (E < R ? E : R) * (kFp8BM - 1)) / kFp8BM; }
// Ordinary launch: the FP8 GEMMs, and what reads their results, start when everything before
// them has ended (no programmatic launch: see gemm_fp8.cu).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_ordered(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// The split factor of a GEMM (1: none).
int fp8_splits(int mode, int64_t R, int64_t E, int64_t N, int64_t K, int sms);

// ---------------------------------------------------------------- reductions of split products
// h of rows 0 .. R-1 from the partial sums of a gated or plain GEMM (same arguments).
// off [E + 1]: first row of each group (for the biases).
cudaError_t launch_fp8_reduce_h(const Fp8GemmArgs& a, const int32_t* off, cudaStream_t st);
// y of a linear GEMM (rows past the groups' sum stay as they were).
cudaError_t launch_fp8_reduce_y(const Fp8GemmArgs& a, cudaStream_t st);
// The layer's combine from the partial sums of its down product:
// y[t] = sum_j w_j (sum_s partial[s][pos[t, j]] + bias) + gate_t Y_shared[t] + shared_output[t]
struct Fp8CombineArgs {
  const float* partial;
  int splits, pitch;
  const int32_t* pos;         // [T, k]
  const int32_t* idx;         // [T, k] experts (for the bias)
  const float* roww;          // [R] or null
  const uint16_t* bias;       // [E, d] or null
  const float* sgate;         // [T] or null
  const uint16_t* Ys;         // [T, d] shared expert rows, or null
  const uint16_t* shared_output;  // [T, d] or null
  uint16_t* y;
  int T, d, k, R, E;
  int* status;
};
cudaError_t launch_fp8_combine(const Fp8CombineArgs& a, cudaStream_t st);

}  // namespace moe
