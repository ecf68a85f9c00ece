// fp8_quant.cu -- quantisation to e4m3 with an fp32 scale per 128 columns (rows of
// activations) or per 128 x 128 block (weights), and the gather that quantises the
// layer's tokens into expert order.
//
//   s = max(amax, 2^-100) / 448,  q = e4m3(x / s)   (fp8_scale, fp8_round4)
//
// One pass: the 128 columns of a block stay in the registers of eight lanes between the
// maximum and the rounding, so each value is read once and its byte written once.
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// 16 neighbouring values of a row in one lane, as loaded: two (bf16) or four (fp32)
// vectors of 16 bytes, zeros past K.
template <bool BF16>
struct Sixteen {
  static constexpr int kVecs = BF16 ? 2 : 4, kPer = 16 / kVecs;  // vectors, values in each
  uint4 v[kVecs];

  __device__ __forceinline__ void load(const void* row, int col, int K) {  // col: the lane's first column
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (int64_t)col * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < kVecs; i++) v[i] = col + i * kPer < K ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kVecs; i++) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void unpack(float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < kVecs; i++) {
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int c = 0; c < 4; c++) {
        if constexpr (BF16) {
          f[8 * i + 2 * c] = __uint_as_float(u[c] << 16);
          f[8 * i + 2 * c + 1] = __uint_as_float(u[c] & 0xffff0000u);
        } else {
          f[4 * i + c] = __uint_as_float(u[c]);
        }
      }
    }
  }
};

__device__ __forceinline__ float amax16(const float (&f)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i++) m = fmaxf(m, fabsf(f[i]));  // (a NaN is left out)
  return m;
}

// Largest value over the LANES neighbouring lanes that hold a block.
template <int LANES>
__device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The lane's 16 values rounded under the block's largest magnitude; returns the scale.
// Whole warp.
template <bool BF16>
__device__ __forceinline__ float round16(const float (&f)[16], float amax, uint32_t (&w)[4]) {
  if constexpr (BF16) {
    const Fp8ScaleBf16 s = fp8_scale_of_bf16(amax);
    fp8_round16_bf16(f, s, w);
    return s.s;
  } else {
    const Fp8Scale s = fp8_scale_of(amax);
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = fp8_round4(f + 4 * i, s);
    return s.s;
  }
}

// Sixteen rounded values to q (the lane's first column's place): whole, or (rows of a
// multiple of 8 or 4 values) the vectors below K.
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store16(uint8_t* q, int col, int K, const uint32_t (&w)[4]) {
  if constexpr (WHOLE) {
    if (col < K) *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if constexpr (BF16) {
    if (col < K) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    if (col + 8 < K) *reinterpret_cast<uint2*>(q + 8) = make_uint2(w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (col + 4 * i < K) *reinterpret_cast<uint32_t*>(q + 4 * i) = w[i];
  }
}

// Rows in vectors: eight lanes per block of 128 columns, so that a block's maximum and
// scale are worked out by eight lanes for 16 values each; two blocks in flight.  16384 rows
// of 7168 bf16 take 62 us, 5.7 TB/s (with a test of every value for a near tie and eight
// values per lane it was bound by instructions, 183 per eight values: 113 us).
constexpr int kLanes = 8, kGroups = kThreads / kLanes, kBatch = 2;
template <bool BF16, bool WHOLE>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const uint8_t* x, int64_t pitch_bytes, int K, int nb,
                                                                 int step_row, int step_blk, int64_t blocks, uint8_t* q,
                                                                 float* scales) {
  pdl_enter();
  const int64_t b0 = (int64_t)blockIdx.x * (kGroups * kBatch) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  // one division, then steps of kGroups blocks
  int64_t row[kBatch];
  int col[kBatch];
  row[0] = b0 / nb;
  int blk = (int)(b0 - row[0] * nb);
  Sixteen<BF16> v[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; i++) {
    col[i] = blk * 128 + lane * 16;
    if (b0 + i * kGroups < blocks) v[i].load(x + row[i] * pitch_bytes, col[i], K);
    else v[i].clear();
    if (i + 1 < kBatch) {
      blk += step_blk;
      row[i + 1] = row[i] + step_row;
      if (blk >= nb) {
        blk -= nb;
        row[i + 1]++;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kBatch; i++) {
    const int64_t b = b0 + i * kGroups;
    float f[16];
    v[i].unpack(f);
    uint32_t w[4];
    const float s = round16<BF16>(f, lanes_max<kLanes>(amax16(f)), w);
    if (b < blocks) {
      store16<BF16, WHOLE>(q + row[i] * K + col[i], col[i], K, w);
      if (lane == 0) scales[b] = s;
    }
  }
}

__device__ __forceinline__ float load_any(const void* x, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(((const uint16_t*)x)[i]) : ((const float*)x)[i];
}

// Rows of any size and alignment: one warp per block, a value at a time.
__global__ void __launch_bounds__(kThreads) quantize_rows_any_kernel(const void* x, int bf16, int64_t pitch, int K, int nb,
                                                                     int64_t blocks, uint8_t* q, float* scales) {
  pdl_enter();
  const int64_t b = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (b >= blocks) return;
  const int64_t row = b / nb;
  const int c0 = (int)(b - row * nb) * 128 + lane;
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; i++) f[i] = c0 + 32 * i < K ? load_any(x, bf16, row * pitch + c0 + 32 * i) : 0.f;
  const Fp8Scale s = fp8_scale_of(lanes_max<32>(fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])))));
  const uint32_t w = fp8_round4(f, s);
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (c0 + 32 * i < K) q[row * K + c0 + 32 * i] = (uint8_t)(w >> (8 * i));
  if (lane == 0) scales[b] = s.s;
}

// One 128 x 128 weight block per thread block, held in registers between the maximum and
// the rounding (64 values per thread).
template <bool BF16, bool WHOLE>
__global__ void __launch_bounds__(kThreads) quantize_weights_kernel(const uint8_t* w, int64_t N, int64_t K, int nbn, int nbk,
                                                                    uint8_t* q, float* scales) {
  pdl_enter();
  __shared__ float warp_max[kThreads / 32];
  constexpr int kIter = 128 / kGroups;  // steps of kGroups rows
  const int64_t blk = blockIdx.x;
  const int kb = (int)(blk % nbk);
  const int64_t en = blk / nbk, e = en / nbn;
  const int64_t n0 = (en - e * nbn) * 128;
  const int col = kb * 128 + (threadIdx.x % kLanes) * 16, r0 = threadIdx.x / kLanes;
  Sixteen<BF16> v[kIter];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kIter; i++) {
    const int64_t n = n0 + r0 + i * kGroups;
    if (n < N) v[i].load(w + (e * N + n) * K * (BF16 ? 2 : 4), col, (int)K);
    else v[i].clear();
  }
#pragma unroll
  for (int i = 0; i < kIter; i++) {
    float f[16];
    v[i].unpack(f);
    m = fmaxf(m, amax16(f));
  }
  m = lanes_max<32>(m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = warp_max[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; i++) m = fmaxf(m, warp_max[i]);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kIter; i++) {
    const int64_t n = n0 + r0 + i * kGroups;
    float f[16];
    uint32_t o[4];
    v[i].unpack(f);
    s = round16<BF16>(f, m, o);
    if (n < N) store16<BF16, WHOLE>(q + (e * N + n) * K + col, col, (int)K, o);
  }
  if (threadIdx.x == 0) scales[blk] = s;
}

// The same for rows of any size and alignment, reading the block twice.
__global__ void __launch_bounds__(kThreads) quantize_weights_any_kernel(const void* w, int bf16, int64_t N, int64_t K, int nbn,
                                                                        int nbk, uint8_t* q, float* scales) {
  pdl_enter();
  __shared__ float warp_max[kThreads / 32];
  const int64_t blk = blockIdx.x;
  const int kb = (int)(blk % nbk);
  const int64_t en = blk / nbk, e = en / nbn;
  const int64_t n0 = (en - e * nbn) * 128;
  const int cols = (int)min((int64_t)128, K - kb * 128), rows = (int)min((int64_t)128, N - n0);
  const int64_t base = (e * N + n0) * K + kb * 128;
  float m = 0.f;
  for (int i = threadIdx.x; i < rows * cols; i += kThreads)
    m = fmaxf(m, fabsf(load_any(w, bf16, base + (int64_t)(i / cols) * K + i % cols)));
  m = lanes_max<32>(m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = warp_max[0];
  for (int i = 1; i < kThreads / 32; i++) m = fmaxf(m, warp_max[i]);
  const Fp8Scale s = fp8_scale_of(m);
  for (int i = threadIdx.x; i < rows * cols; i += kThreads) {
    const int64_t at = base + (int64_t)(i / cols) * K + i % cols;
    q[at] = (uint8_t)fp8_pack4(fp8_quotient(load_any(w, bf16, at), s.s, s.hi), 0.f, 0.f, 0.f);
  }
  if (threadIdx.x == 0) scales[blk] = s.s;
}

// Tokens into expert order: eight lanes per (token, block of 128 columns), which is read
// and rounded once and written to the token's k rows (rounded per row for weigh-inputs,
// whose rows differ by their weight); B blocks in flight per group of lanes.
template <int B>
__global__ void __launch_bounds__(kThreads) gather_quantize_kernel(Fp8GatherArgs a, int nb, int step_t, int step_blk) {
  pdl_enter();
  const int64_t b0 = (int64_t)blockIdx.x * (kGroups * B) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  int tok[B], at[B];
  tok[0] = (int)(b0 / nb);
  at[0] = (int)(b0 - (int64_t)tok[0] * nb);
  Sixteen<true> v[B];
#pragma unroll
  for (int i = 0; i < B; i++) {
    if (tok[i] < a.T) v[i].load(a.x + (int64_t)tok[i] * a.d, at[i] * 128 + lane * 16, a.d);
    else v[i].clear();
    if (i + 1 < B) {
      at[i + 1] = at[i] + step_blk;
      tok[i + 1] = tok[i] + step_t;
      if (at[i + 1] >= nb) {
        at[i + 1] -= nb;
        tok[i + 1]++;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < B; i++) {
    const int col = at[i] * 128 + lane * 16;
    float f[16];
    v[i].unpack(f);
    const float m = lanes_max<kLanes>(amax16(f));
    uint32_t w[4] = {};
    float s = 0.f;
    if (!a.weigh_inputs) s = round16<true>(f, m, w);
    if (tok[i] >= a.T) continue;
    for (int j = 0; j < a.k; j++) {
      const int row = a.pos[(int64_t)tok[i] * a.k + j];
      if (row < 0 || row >= a.R) {
        set_status(a.status, MOE_ERR_SHAPE);
        // no row of the down product is this token's: its output is the empty sum, as a combine's
        if (a.y && col < a.d) {
          uint4* out = reinterpret_cast<uint4*>(a.y + (int64_t)tok[i] * a.d + col);
          out[0] = out[1] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      if (a.weigh_inputs) {
        // the largest |w x| is |w| times the largest |x| (rounding is monotone)
        const float wt = a.roww[row];
        float g[16];
#pragma unroll
        for (int c = 0; c < 16; c++) g[c] = f[c] * wt;
        s = round16<false>(g, fabsf(m * wt), w);
      }
      // d is a multiple of 16
      if (col < a.d) *reinterpret_cast<uint4*>(a.xq + (int64_t)row * a.d + col) = make_uint4(w[0], w[1], w[2], w[3]);
      if (lane == 0) a.xs[(int64_t)at[i] * a.R + row] = s;
    }
  }
}

__global__ void shared_tiles_kernel(int32_t* tiles, int E, int n) {
  pdl_enter();
  for (int i = threadIdx.x; i < E + 2; i += blockDim.x) tiles[i] = i == E + 1 ? n : 0;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

cudaError_t launch_fp8_quantize(int bf16, int64_t rows, int64_t K, const void* x, int64_t pitch, uint8_t* q, float* scales,
                                cudaStream_t st) {
  const int nb = (int)((K + 127) / 128);
  const int64_t blocks = rows * nb;
  const int V = bf16 ? 8 : 4, elt = bf16 ? 2 : 4;
  // sixteen bytes per load: whole vectors in every row of x, whole words of q
  if (K % V == 0 && (pitch * elt) % 16 == 0 && aligned(x, 16) && aligned(q, V)) {
    const bool whole = K % 16 == 0 && aligned(q, 16);
    const auto kernel = bf16 ? (whole ? quantize_rows_kernel<true, true> : quantize_rows_kernel<true, false>)
                             : (whole ? quantize_rows_kernel<false, true> : quantize_rows_kernel<false, false>);
    const int per = kGroups * kBatch;
    return launch_pdl(kernel, (unsigned)((blocks + per - 1) / per), kThreads, 0, st, (const uint8_t*)x, pitch * elt, (int)K, nb,
                      kGroups / nb, kGroups % nb, blocks, q, scales);
  }
  const unsigned grid = (unsigned)((blocks + kThreads / 32 - 1) / (kThreads / 32));
  return launch_pdl(quantize_rows_any_kernel, grid, kThreads, 0, st, x, bf16, pitch, (int)K, nb, blocks, q, scales);
}

cudaError_t launch_fp8_quantize_weights(int bf16, int64_t E, int64_t N, int64_t K, const void* w, uint8_t* q, float* scales,
                                        cudaStream_t st) {
  const int nbn = (int)((N + 127) / 128), nbk = (int)((K + 127) / 128);
  const unsigned grid = (unsigned)(E * nbn * nbk);
  if (K % (bf16 ? 8 : 4) == 0 && aligned(w, 16) && aligned(q, bf16 ? 8 : 4)) {
    const bool whole = K % 16 == 0 && aligned(q, 16);
    const auto kernel = bf16 ? (whole ? quantize_weights_kernel<true, true> : quantize_weights_kernel<true, false>)
                             : (whole ? quantize_weights_kernel<false, true> : quantize_weights_kernel<false, false>);
    return launch_pdl(kernel, grid, kThreads, 0, st, (const uint8_t*)w, N, K, nbn, nbk, q, scales);
  }
  return launch_pdl(quantize_weights_any_kernel, grid, kThreads, 0, st, w, bf16, N, K, nbn, nbk, q, scales);
}

cudaError_t launch_shared_tiles(int32_t* tiles, int E, int n, cudaStream_t st) {
  return launch_ordered(shared_tiles_kernel, 1, kThreads, 0, st, tiles, E, n);
}

cudaError_t launch_fp8_gather(const Fp8GatherArgs& a, cudaStream_t st) {
  if (a.R == 0) return cudaSuccess;
  const int nb = (a.d + 127) / 128;
  // two blocks in flight once that leaves every SM several thread blocks
  const int64_t work = (int64_t)a.T * nb;
  const int sr = kGroups / nb, sb = kGroups % nb;
  if (work >= kGroups * 2 * 592)
    return launch_pdl(gather_quantize_kernel<2>, (unsigned)((work + 2 * kGroups - 1) / (2 * kGroups)), kThreads, 0, st, a, nb, sr, sb);
  return launch_pdl(gather_quantize_kernel<1>, (unsigned)((work + kGroups - 1) / kGroups), kThreads, 0, st, a, nb, sr, sb);
}

}  // namespace moe
