// fp8_reduce.cu -- the sums of a split FP8 product and what follows them: activation and
// quantisation of h, the plain rounding to bf16, or the layer's combine.
//
// A product of few rows is split along K so that every SM streams weights; each split
// leaves fp32 partial sums [split][row][column].  These kernels add them in split order
// (the result does not depend on timing).  They read splits * R * columns floats, a few
// MB at most, from L2: with the launch 4 us for 1 row of 7168 x 4096 in 8 splits.
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Sum over the splits of four neighbouring columns; loads of four splits in flight.
__device__ __forceinline__ float4 sum4(const float* p, int64_t stride, int splits) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < splits; s0 += 4) {
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
      v[i] = s0 + i < splits ? __ldcg(reinterpret_cast<const float4*>(p + (s0 + i) * stride)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (s0 + i < splits) {
        a.x += v[i].x;
        a.y += v[i].y;
        a.z += v[i].z;
        a.w += v[i].w;
      }
  }
  return a;
}

__device__ __forceinline__ int group_of_row(const int32_t* off, int E, int r) {
  int lo = 0, hi = E - 1;  // last group with off[g] <= r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One warp per (row, 128 features): four features per lane.
__global__ void __launch_bounds__(kThreads) reduce_h_kernel(Fp8GemmArgs a, const int32_t* off, int nb) {
  pdl_enter();
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (int64_t)a.R * nb) return;
  const int row = (int)(w / nb), grp = (int)(w - (int64_t)row * nb);
  const int f0 = grp * 128 + lane * 4;
  const bool in = f0 < a.N;  // N is a multiple of 16
  const int64_t stride = (int64_t)a.R * a.pitch;
  const bool gated = a.mode == FP8_GATED;
  const float* src = a.partial + (int64_t)row * a.pitch + grp * (gated ? 256 : 128) + lane * 4;
  float g[4] = {}, u[4] = {}, h[4] = {};
  if (in) {
    const float4 x = sum4(src, stride, a.splits);
    g[0] = x.x, g[1] = x.y, g[2] = x.z, g[3] = x.w;
    if (gated) {
      const float4 y = sum4(src + 128, stride, a.splits);
      u[0] = y.x, u[1] = y.y, u[2] = y.z, u[3] = y.w;
    }
    if (a.bias || a.gate_bias) {
      const Fp8Bias b = fp8_bias(a.mode, a.layout, group_of_row(off, a.E, row), a.N, a.bias, a.gate_bias);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if (b.g) g[i] += bf16_to_f32(__ldg(b.g + f0 + i));
        if (b.u) u[i] += bf16_to_f32(__ldg(b.u + f0 + i));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
      h[i] = fp8_act(a.act, g[i], gated) * (gated ? fp8_up(a.act, u[i]) + a.act.beta : 1.f);
  }
  float m = fmaxf(fmaxf(fabsf(h[0]), fabsf(h[1])), fmaxf(fabsf(h[2]), fabsf(h[3])));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const Fp8Scale s = fp8_scale_of(m);
  if (in) *reinterpret_cast<uint32_t*>(a.hq + (int64_t)row * a.N + f0) = fp8_round4(h, s);
  if (lane == 0) a.hs[row * a.hs_row + grp * a.hs_grp] = s.s;
}

// Four outputs per thread; the rows of the groups only.
__global__ void __launch_bounds__(kThreads) reduce_y_kernel(Fp8GemmArgs a) {
  pdl_enter();
  __shared__ int32_t rows;
  if (threadIdx.x < 32) {
    int64_t sum = 0;
    if (a.cnt)
      for (int e = threadIdx.x; e < a.E; e += 32) sum += max(a.cnt[e], 0);
    else
      sum = threadIdx.x == 0 ? a.R : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x == 0) rows = (int32_t)min(sum, (int64_t)a.R);
  }
  __syncthreads();
  const int n4 = a.N / 4;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = i / n4;
  if (row >= rows) return;
  const int col = (int)(i - row * n4) * 4;
  const float4 v = sum4(a.partial + row * a.pitch + col, (int64_t)a.R * a.pitch, a.splits);
  *reinterpret_cast<uint2*>(a.y + row * a.N + col) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

__device__ __forceinline__ void add_bf16x4(float4& acc, const uint16_t* p, float f) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
  acc.x = fmaf(f, bf16_to_f32(v.x & 0xffff), acc.x);
  acc.y = fmaf(f, bf16_to_f32(v.x >> 16), acc.y);
  acc.z = fmaf(f, bf16_to_f32(v.y & 0xffff), acc.z);
  acc.w = fmaf(f, bf16_to_f32(v.y >> 16), acc.w);
}

// acc += bias[0 .. 3], which is aligned to its elements: a caller's bias may start anywhere
// in a larger buffer, and its rows are a multiple of 16 long.
__device__ __forceinline__ void add_bias4(float4& acc, const uint16_t* bias) {
  if ((reinterpret_cast<uintptr_t>(bias) & 7u) == 0) {
    add_bf16x4(acc, bias, 1.f);
  } else {
    acc.x += bf16_to_f32(__ldg(bias));
    acc.y += bf16_to_f32(__ldg(bias + 1));
    acc.z += bf16_to_f32(__ldg(bias + 2));
    acc.w += bf16_to_f32(__ldg(bias + 3));
  }
}

// Four outputs of one token per thread, slots in order.
__global__ void __launch_bounds__(kThreads) combine_splits_kernel(Fp8CombineArgs a) {
  pdl_enter();
  const int t = blockIdx.x;
  const int c = (blockIdx.y * kThreads + threadIdx.x) * 4;
  if (c >= a.d) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < a.k; j++) {
    const int row = a.pos[(int64_t)t * a.k + j];
    if (row < 0 || row >= a.R) {
      set_status(a.status, MOE_ERR_SHAPE);
      continue;
    }
    float4 v = sum4(a.partial + (int64_t)row * a.pitch + c, (int64_t)a.R * a.pitch, a.splits);
    if (a.bias) {
      const int e = a.idx[(int64_t)t * a.k + j];
      if (e >= 0 && e < a.E) add_bias4(v, a.bias + (int64_t)e * a.d + c);
    }
    const float w = a.roww ? a.roww[row] : 1.f;
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  if (a.Ys) add_bf16x4(acc, a.Ys + (int64_t)t * a.d + c, a.sgate ? a.sgate[t] : 1.f);
  if (a.shared_output) add_bf16x4(acc, a.shared_output + (int64_t)t * a.d + c, 1.f);
  *reinterpret_cast<uint2*>(a.y + (int64_t)t * a.d + c) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

}  // namespace

cudaError_t launch_fp8_reduce_h(const Fp8GemmArgs& a, const int32_t* off, cudaStream_t st) {
  const int nb = (a.N + 127) / 128;
  const int64_t blocks = ((int64_t)a.R * nb + kThreads / 32 - 1) / (kThreads / 32);
  return launch_ordered(reduce_h_kernel, (unsigned)blocks, kThreads, 0, st, a, off, nb);
}

cudaError_t launch_fp8_reduce_y(const Fp8GemmArgs& a, cudaStream_t st) {
  const int64_t blocks = ((int64_t)a.R * (a.N / 4) + kThreads - 1) / kThreads;
  return launch_ordered(reduce_y_kernel, (unsigned)blocks, kThreads, 0, st, a);
}

cudaError_t launch_fp8_combine(const Fp8CombineArgs& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const dim3 grid(a.T, (a.d / 4 + kThreads - 1) / kThreads);
  return launch_ordered(combine_splits_kernel, grid, kThreads, 0, st, a);
}

}  // namespace moe
