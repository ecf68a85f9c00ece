// fp8_quant.cu -- quantisation to e4m3 with an fp32 scale per 128 columns (rows of
// activations) or per 128 x 128 block (weights), and the gather that quantises the
// layer's tokens into expert order.
//
//   s = max(amax, 2^-100) / 448,  q = e4m3(x / s)   (fp8_scale, fp8_quotient)
//
// One pass: the 128 columns of a block stay in the registers of 16 lanes (bf16, eight
// values each) or 32 lanes (fp32, four each) between the maximum and the rounding, so
// each value is read once and its byte written once.  Bound by memory.
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// A lane's 16 bytes as floats: V = 8 bf16 or 4 fp32.
template <int V>
__device__ __forceinline__ void unpack16(const uint4& q, float (&f)[V]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (V == 8) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(u[i]);
    }
  }
}

template <int V>
__device__ __forceinline__ float amax_of(const float (&f)[V]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < V; i++) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// Largest value over the LANES neighbouring lanes that hold a block.
template <int LANES>
__device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

template <int V>
__device__ __forceinline__ void store_q(uint8_t* dst, const float (&f)[V], float s, float inv) {
  if constexpr (V == 8)
    *reinterpret_cast<uint2*>(dst) = fp8_round8(f, s, inv);
  else
    *reinterpret_cast<uint32_t*>(dst) = fp8_pack4(fp8_quotient(f[0], s, inv), fp8_quotient(f[1], s, inv),
                                                  fp8_quotient(f[2], s, inv), fp8_quotient(f[3], s, inv));
}

// Vectorised rows: 128 / V lanes per block, kBatch blocks in flight per group of lanes.
constexpr int kBatch = 4;
template <int V>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const uint8_t* x, int64_t pitch_bytes, int K, int nb,
                                                                 int64_t blocks, uint8_t* q, float* scales) {
  pdl_enter();
  constexpr int L = 128 / V;
  constexpr int kGroups = kThreads / L;
  const int sub = threadIdx.x / L, lane = threadIdx.x % L;
  const int64_t b0 = (int64_t)blockIdx.x * (kGroups * kBatch) + sub;
  uint4 v[kBatch];
  int64_t row[kBatch];
  int col[kBatch];
  const int64_t first = b0 / nb;  // one division, then steps of kGroups blocks
  int down = 0, blk = (int)(b0 - first * nb);
#pragma unroll
  for (int i = 0; i < kBatch; i++) {
    const int64_t b = b0 + i * kGroups;
    row[i] = first + down;
    col[i] = blk * 128 + lane * V;
    blk += kGroups;
    while (blk >= nb) {
      blk -= nb;
      down++;
    }
    v[i] = make_uint4(0, 0, 0, 0);
    if (b < blocks && col[i] < K)
      v[i] = __ldg(reinterpret_cast<const uint4*>(x + row[i] * pitch_bytes + (int64_t)col[i] * (16 / V)));
  }
#pragma unroll
  for (int i = 0; i < kBatch; i++) {
    const int64_t b = b0 + i * kGroups;
    float f[V];
    unpack16<V>(v[i], f);
    const float s = fp8_scale(lanes_max<L>(amax_of<V>(f)));
    const float inv = __frcp_rn(s);
    if (b < blocks) {
      if (col[i] < K) store_q<V>(q + row[i] * K + col[i], f, s, inv);
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
  const float s = fp8_scale(lanes_max<32>(amax_of<4>(f)));
  const float inv = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (c0 + 32 * i < K)
      q[row * K + c0 + 32 * i] = (uint8_t)fp8_pack4(fp8_quotient(f[i], s, inv), 0.f, 0.f, 0.f);
  if (lane == 0) scales[b] = s;
}

// One 128 x 128 weight block per thread block.  Vectorised rows are held in registers
// between the maximum and the rounding (64 values per thread).
template <int V>
__global__ void __launch_bounds__(kThreads) quantize_weights_kernel(const uint8_t* w, int64_t N, int64_t K, int nbn, int nbk,
                                                                    uint8_t* q, float* scales) {
  pdl_enter();
  __shared__ float warp_max[kThreads / 32];
  constexpr int L = 128 / V, kRows = kThreads / L, kIter = 128 / kRows;  // rows per step, steps
  const int64_t blk = blockIdx.x;
  const int kb = (int)(blk % nbk);
  const int64_t en = blk / nbk, e = en / nbn;
  const int64_t n0 = (en - e * nbn) * 128;
  const int col = kb * 128 + (threadIdx.x % L) * V, r0 = threadIdx.x / L;
  uint4 v[kIter];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kIter; i++) {
    const int64_t n = n0 + r0 + i * kRows;
    v[i] = make_uint4(0, 0, 0, 0);
    if (n < N && col < K) v[i] = __ldg(reinterpret_cast<const uint4*>(w + ((e * N + n) * K + col) * (16 / V)));
  }
#pragma unroll
  for (int i = 0; i < kIter; i++) {
    float f[V];
    unpack16<V>(v[i], f);
    m = fmaxf(m, amax_of<V>(f));
  }
  m = lanes_max<32>(m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = warp_max[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; i++) m = fmaxf(m, warp_max[i]);
  const float s = fp8_scale(m), inv = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < kIter; i++) {
    const int64_t n = n0 + r0 + i * kRows;
    float f[V];
    unpack16<V>(v[i], f);
    if (n < N && col < K) store_q<V>(q + (e * N + n) * K + col, f, s, inv);
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
  const float s = fp8_scale(m), inv = __frcp_rn(s);
  for (int i = threadIdx.x; i < rows * cols; i += kThreads) {
    const int64_t at = base + (int64_t)(i / cols) * K + i % cols;
    q[at] = (uint8_t)fp8_pack4(fp8_quotient(load_any(w, bf16, at), s, inv), 0.f, 0.f, 0.f);
  }
  if (threadIdx.x == 0) scales[blk] = s;
}

// Tokens into expert order: 16 lanes per (token, block of 128 columns), which is read
// and rounded once and written to the token's k rows (rounded per row for weigh-inputs,
// whose rows differ by their weight); B blocks in flight per group of lanes.
template <int B>
__global__ void __launch_bounds__(kThreads) gather_quantize_kernel(Fp8GatherArgs a, int nb) {
  pdl_enter();
  constexpr int kGroups = kThreads / 16;
  const int64_t b0 = (int64_t)blockIdx.x * (kGroups * B) + threadIdx.x / 16;
  const int lane = threadIdx.x & 15;
  const int first = (int)(b0 / nb);  // one division, then steps of kGroups blocks
  int blk = (int)(b0 - (int64_t)first * nb), t = first;
  uint4 v[B];
  int tok[B], at[B];
#pragma unroll
  for (int i = 0; i < B; i++) {
    tok[i] = t;
    at[i] = blk;
    const int col = blk * 128 + lane * 8;
    v[i] = make_uint4(0, 0, 0, 0);
    if (t < a.T && col < a.d) v[i] = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.d + col));
    blk += kGroups;
    while (blk >= nb) {
      blk -= nb;
      t++;
    }
  }
#pragma unroll
  for (int i = 0; i < B; i++) {
    const int col = at[i] * 128 + lane * 8;
    float f[8];
    unpack16<8>(v[i], f);
    const float m = lanes_max<16>(amax_of<8>(f));
    if (tok[i] >= a.T) continue;  // (the shuffles are behind: lanes of a group agree, groups need not)
    float s = fp8_scale(m), inv = __frcp_rn(s);
    uint2 w = make_uint2(0, 0);
    if (!a.weigh_inputs) w = fp8_round8(f, s, inv);
    for (int j = 0; j < a.k; j++) {
      const int row = a.pos[(int64_t)tok[i] * a.k + j];
      if (row < 0 || row >= a.R) {
        set_status(a.status, MOE_ERR_SHAPE);
        continue;
      }
      if (a.weigh_inputs) {
        // the largest |w x| is |w| times the largest |x| (rounding is monotone)
        const float wt = a.roww[row];
        float g[8];
#pragma unroll
        for (int c = 0; c < 8; c++) g[c] = f[c] * wt;
        s = fp8_scale(fabsf(m * wt));
        inv = __frcp_rn(s);
        w = fp8_round8(g, s, inv);
      }
      if (col < a.d) *reinterpret_cast<uint2*>(a.xq + (int64_t)row * a.d + col) = w;
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
  // sixteen bytes per lane: whole vectors in every row of x, whole words of q
  if (K % V == 0 && (pitch * elt) % 16 == 0 && aligned(x, 16) && aligned(q, V)) {
    const int per = kThreads / (128 / V) * kBatch;
    const unsigned grid = (unsigned)((blocks + per - 1) / per);
    return launch_pdl(bf16 ? quantize_rows_kernel<8> : quantize_rows_kernel<4>, grid, kThreads, 0, st, (const uint8_t*)x,
                      pitch * elt, (int)K, nb, blocks, q, scales);
  }
  const unsigned grid = (unsigned)((blocks + kThreads / 32 - 1) / (kThreads / 32));
  return launch_pdl(quantize_rows_any_kernel, grid, kThreads, 0, st, x, bf16, pitch, (int)K, nb, blocks, q, scales);
}

cudaError_t launch_fp8_quantize_weights(int bf16, int64_t E, int64_t N, int64_t K, const void* w, uint8_t* q, float* scales,
                                        cudaStream_t st) {
  const int nbn = (int)((N + 127) / 128), nbk = (int)((K + 127) / 128);
  const unsigned grid = (unsigned)(E * nbn * nbk);
  if (K % (bf16 ? 8 : 4) == 0 && aligned(w, 16) && aligned(q, bf16 ? 8 : 4))
    return launch_pdl(bf16 ? quantize_weights_kernel<8> : quantize_weights_kernel<4>, grid, kThreads, 0, st,
                      (const uint8_t*)w, N, K, nbn, nbk, q, scales);
  return launch_pdl(quantize_weights_any_kernel, grid, kThreads, 0, st, w, bf16, N, K, nbn, nbk, q, scales);
}

cudaError_t launch_shared_tiles(int32_t* tiles, int E, int n, cudaStream_t st) {
  return launch_pdl(shared_tiles_kernel, 1, kThreads, 0, st, tiles, E, n);
}

cudaError_t launch_fp8_gather(const Fp8GatherArgs& a, cudaStream_t st) {
  if (a.R == 0) return cudaSuccess;
  const int nb = (a.d + 127) / 128;
  // four blocks in flight once that leaves every SM several thread blocks
  const int64_t work = (int64_t)a.T * nb, per = kThreads / 16;
  if (work >= per * 4 * 592)
    return launch_pdl(gather_quantize_kernel<4>, (unsigned)((work + 4 * per - 1) / (4 * per)), kThreads, 0, st, a, nb);
  return launch_pdl(gather_quantize_kernel<1>, (unsigned)((work + per - 1) / per), kThreads, 0, st, a, nb);
}

}  // namespace moe
