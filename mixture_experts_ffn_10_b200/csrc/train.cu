// train.cu -- the router's training kernels: balance loss with per-expert counts, and the
// gradient of routing weights and balance loss with respect to the logits.
//
// A token's E logits lie in the registers of a group of G lanes (G a power of two), each
// with NV vectors of V neighbouring experts: one 16-byte load per vector where the rows
// are 16-byte aligned, else single values.  Maximum, sums and shares (softmax, or sigmoids
// divided by their sum) are fp32 and never leave the registers; the row is read once.
//
// Balance loss, two launches:
//   partial: one block per chunk of tokens; per sequence that meets the chunk, the sum of
//     the shares (per lane over its tokens, then over the lanes and warps in fixed order)
//     and a histogram of the slots, to row chunk + sequence of the partial sums (both
//     indices grow along the tokens, so every (chunk, sequence) pair has a row of its own);
//   finish: 32 experts of a sequence per block: sums over its chunks (double), the counts,
//     its part of the loss; the last block to finish adds the parts in order.
// Backward, one launch: dl = J_w^T dw + A J_p^T c, with
//   softmax:  dp/dl = p (1 - p'),  sigmoid: ds/dl = s (1 - s), p = s / Z,
// the k slots of a token being added to its row in shared memory.
// Bound by memory for large batches, by latency (two launches, one) for small ones.
#include "train.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- a token's row
template <int BF16, int V, int NV>
struct Row {
  uint4 v[V > 1 ? NV : 1];
  float s[V > 1 ? 1 : NV];

  // Experts (i G + lane) V .. + V - 1 for i < NV.
  __device__ __forceinline__ void load(const void* base, int64_t t, int E, int G, int lane) {
    if constexpr (V > 1) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + t * E * (16 / V));
#pragma unroll
      for (int i = 0; i < NV; i++)
        if ((i * G + lane) * V < E) v[i] = __ldg(p + i * G + lane);
    } else {
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const int e = i * G + lane;
        if (e < E)
          s[i] = BF16 ? bf16_to_f32(__ldg(static_cast<const uint16_t*>(base) + t * E + e))
                      : __ldg(static_cast<const float*>(base) + t * E + e);
      }
    }
  }
  __device__ __forceinline__ float get(int n) const {
    if constexpr (V == 1) return s[n];
    const uint4& q = v[n / V];
    const int c = n % V;
    if constexpr (BF16) {
      const uint32_t u = c < 2 ? q.x : c < 4 ? q.y : c < 6 ? q.z : q.w;
      return __uint_as_float(c & 1 ? u & 0xffff0000u : u << 16);
    } else {
      return __uint_as_float(c == 0 ? q.x : c == 1 ? q.y : c == 2 ? q.z : q.w);
    }
  }
};

template <int V>
__device__ __forceinline__ int expert_of(int n, int G, int lane) {
  return ((n / V) * G + lane) * V + n % V;
}

__device__ __forceinline__ float group_sum(float x, int G) {
  for (int o = G >> 1; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float group_max(float x, int G) {
  for (int o = G >> 1; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ float bias_of(const RouterTrainArgs& a, int e) {
  if (!a.router_bias) return 0.f;
  return a.bf16 ? bf16_to_f32(__ldg(static_cast<const uint16_t*>(a.router_bias) + e))
                : __ldg(static_cast<const float*>(a.router_bias) + e);
}
__device__ __forceinline__ float logit_of(const RouterTrainArgs& a, int64_t t, int e) {
  const int64_t i = t * a.E + e;
  return (a.bf16 ? bf16_to_f32(__ldg(static_cast<const uint16_t*>(a.logits) + i))
                 : __ldg(static_cast<const float*>(a.logits) + i)) + bias_of(a, e);
}

// sigma(l) and 1 - sigma(l), both to full relative precision.
__device__ __forceinline__ void sigmoid_pair(float l, float* s, float* r) {
  const float x = expf(-fabsf(l)), d = 1.f / (1.f + x);
  *s = l >= 0.f ? d : x * d;
  *r = l >= 0.f ? x * d : d;
  if (l != l) *s = *r = l;
}

// What turns a logit into its score: softmax s = exp(l - m) inv_z, sigmoid s = sigma(l);
// the share is s (softmax) or s inv_z.
struct Norm {
  float m, inv_z;
};

// l' of the row in l[], scores in s[] (0 past E).  Whole warp.
template <int BF16, int V, int NV>
__device__ __forceinline__ Norm scores(const RouterTrainArgs& a, const Row<BF16, V, NV>& row, int G, int lane,
                                       float (&l)[V * NV], float (&s)[V * NV]) {
  constexpr int N = V * NV;
#pragma unroll
  for (int n = 0; n < N; n++) {
    const int e = expert_of<V>(n, G, lane);
    l[n] = e < a.E ? row.get(n) + bias_of(a, e) : -INFINITY;
  }
  Norm z{0.f, 0.f};
  float sum = 0.f;
  if (a.score == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int n = 0; n < N; n++) m = fmaxf(m, l[n]);
    m = group_max(m, G);
    z.m = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int n = 0; n < N; n++) {
      s[n] = expf(l[n] - z.m);
      sum += s[n];
    }
  } else {
#pragma unroll
    for (int n = 0; n < N; n++) {
      float r;
      sigmoid_pair(l[n], &s[n], &r);
      sum += s[n];
    }
  }
  sum = group_sum(sum, G);
  z.inv_z = sum == 0.f ? 0.f : 1.f / sum;
  if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int n = 0; n < N; n++) s[n] *= z.inv_z;
  }
  return z;
}

__device__ __forceinline__ int seq_at(const RouterTrainArgs& a, int b) {
  if (!a.seq) return b == 0 ? 0 : a.T;
  const int v = __ldg(a.seq + b);
  return v < 0 ? 0 : v > a.T ? a.T : v;
}
// The last sequence with seq[b] <= t, -1 if none; B if t is behind the last.
__device__ __forceinline__ int seq_of(const RouterTrainArgs& a, int t) {
  int lo = -1, hi = a.B;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_at(a, mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ---------------------------------------------------------------- balance loss
constexpr int partial_threads(int n) { return n >= 32 ? 256 : 512; }  // n values of a row per lane
constexpr int kPartialRows = 16384;  // floats of the block's sums: a row of E per warp

template <int BF16, int V, int NV>
__global__ void __launch_bounds__(partial_threads(V * NV)) balance_partial_kernel(RouterTrainArgs a, int G) {
  constexpr int N = V * NV;
  extern __shared__ float sums[];  // [warps][E], then the histogram [E]
  int32_t* hist = reinterpret_cast<int32_t*>(sums + (blockDim.x >> 5) * a.E);
  pdl_enter();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int lane = threadIdx.x & (G - 1), group = threadIdx.x / G, groups = blockDim.x / G;
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  for (int b = max(0, seq_of(a, t0)); b < a.B; b++) {
    const int s0 = max(t0, seq_at(a, b)), s1 = min(t1, seq_at(a, b + 1));
    if (s0 >= t1) break;
    if (s0 >= s1) continue;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    float acc[N];
#pragma unroll
    for (int n = 0; n < N; n++) acc[n] = 0.f;
    Row<BF16, V, NV> next;
    int t = s0 + group;
    if (t < s1) next.load(a.logits, t, a.E, G, lane);
    // the whole warp takes every step (the sums are shuffles)
    for (int base = s0; base < s1; base += groups, t += groups) {
      const Row<BF16, V, NV> row = next;
      if (t + groups < s1) next.load(a.logits, t + groups, a.E, G, lane);
      float l[N], s[N];
      const Norm z = scores<BF16, V, NV>(a, row, G, lane, l, s);
      const float f = a.score == MOE_SCORE_SOFTMAX ? 1.f : z.inv_z;
      if (t < s1) {
#pragma unroll
        for (int n = 0; n < N; n++) acc[n] += s[n] * f;
      }
    }
    __syncthreads();  // the histogram is clear
    for (int i = threadIdx.x; i < (s1 - s0) * a.k; i += blockDim.x) {
      const int e = __ldg(a.idx + (int64_t)s0 * a.k + i);
      if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
    }
    // over the groups of the warp, then the warps
#pragma unroll
    for (int n = 0; n < N; n++) {
      for (int o = G; o < 32; o <<= 1) acc[n] += __shfl_xor_sync(0xffffffffu, acc[n], o);
      const int e = expert_of<V>(n, G, lane);
      if ((threadIdx.x & 31) < G && e < a.E) sums[warp * a.E + e] = acc[n];
    }
    __syncthreads();
    const int64_t at = ((int64_t)blockIdx.x + b) * a.E;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
      float x = 0.f;
      for (int w = 0; w < warps; w++) x += sums[w * a.E + e];
      a.psum[at + e] = x;
      a.pcnt[at + e] = hist[e];
    }
    __syncthreads();
  }
}

// Block (b, y): experts 32 y .. + 31 of sequence b; blockDim.x / 32 warps share its chunks.
__global__ void __launch_bounds__(1024) balance_finish_kernel(RouterTrainArgs a) {
  __shared__ double ps[32][33];
  __shared__ int32_t cs[32][33];
  __shared__ int last;
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int b = blockIdx.x, e = blockIdx.y * 32 + lane;
  const int o0 = seq_at(a, b), o1 = seq_at(a, b + 1);
  double p = 0.0;
  int32_t c = 0;
  if (o1 > o0 && e < a.E) {
    const int c1 = (o1 - 1) / a.chunk;
    int i = o0 / a.chunk + warp;
    for (; i + 3 * warps <= c1; i += 4 * warps) {
      float x[4];
      int32_t y[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int64_t at = ((int64_t)i + u * warps + b) * a.E + e;
        x[u] = a.psum[at];
        y[u] = a.pcnt[at];
      }
#pragma unroll
      for (int u = 0; u < 4; u++) {
        p += x[u];
        c += y[u];
      }
    }
    for (; i <= c1; i += warps) {
      const int64_t at = ((int64_t)i + b) * a.E + e;
      p += a.psum[at];
      c += a.pcnt[at];
    }
  }
  ps[warp][lane] = p;
  cs[warp][lane] = c;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < warps; w++) {
      p += ps[w][lane];
      c += cs[w][lane];
    }
    if (e < a.E) a.counts[(int64_t)b * a.E + e] = c;
    double f = (double)c * p;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
    if (lane == 0) {
      const double n = o1 > o0 ? (double)(o1 - o0) : 1.0;
      a.part[(int64_t)b * gridDim.y + blockIdx.y] = f * a.E / (a.k * n * n);
      __threadfence();
      last = atomicAdd(a.ticket, 1) == (int)(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  // the last block: every part is written; added in a fixed order
  __threadfence();
  double sum = 0.0;
  int live = 0;
  const int64_t parts = (int64_t)gridDim.x * gridDim.y;
  for (int64_t i = threadIdx.x; i < parts; i += blockDim.x) sum += __ldcg(a.part + i);
  for (int i = threadIdx.x; i < a.B; i += blockDim.x) live += seq_at(a, i + 1) > seq_at(a, i);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    live += __shfl_xor_sync(0xffffffffu, live, o);
  }
  if (lane == 0) {
    ps[0][warp] = sum;
    cs[0][warp] = live;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < warps; w++) {
      sum += ps[0][w];
      live += cs[0][w];
    }
    *a.loss = live > 0 ? (float)(a.coef * sum / live) : 0.f;
  }
}

// ---------------------------------------------------------------- backward
constexpr int kBackThreads = 256;

template <int BF16, int V, int NV>
__global__ void __launch_bounds__(kBackThreads) router_backward_kernel(RouterTrainArgs a, int G) {
  constexpr int N = V * NV;
  extern __shared__ float rows[];  // [groups][G N]
  __shared__ int live_seqs;
  pdl_enter();
  const int lane = threadIdx.x & (G - 1), group = threadIdx.x / G, groups = blockDim.x / G;
  float* mine = rows + group * G * N;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  float lead = 0.f;  // dloss coef E / k / B'
  if (a.counts) {
    if (threadIdx.x == 0) live_seqs = 0;
    __syncthreads();
    int live = 0;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) live += seq_at(a, b + 1) > seq_at(a, b);
    live = __reduce_add_sync(0xffffffffu, live);
    if ((threadIdx.x & 31) == 0) atomicAdd(&live_seqs, live);
    __syncthreads();
    lead = (a.dloss ? *a.dloss : 1.f) * a.coef * (float)a.E / ((float)a.k * (float)max(live_seqs, 1));
  }
  const int rounds = (a.k + G - 1) / G;
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t t = (int64_t)blockIdx.x * groups + group;
  Row<BF16, V, NV> next;
  if (t < a.T) next.load(a.logits, t, a.E, G, lane);
  // the whole block takes every step (shuffles and warp barriers)
  for (int64_t base = (int64_t)blockIdx.x * groups; base < a.T; base += step, t += step) {
    const bool in = t < a.T;
    const Row<BF16, V, NV> row = next;
    if (t + step < a.T) next.load(a.logits, t + step, a.E, G, lane);
    float l[N], s[N];
    const Norm z = scores<BF16, V, NV>(a, row, G, lane, l, s);

    // balance: A (c_e - sum c p), A = 0 for tokens outside every sequence
    float amp = 0.f, mean = 0.f;
    const int32_t* c = nullptr;
    if (a.counts) {
      if (in) {
        const int b = seq_of(a, (int)t);
        if (b >= 0 && b < a.B) {
          const int o0 = seq_at(a, b), o1 = seq_at(a, b + 1);
          if (t < o1) {
            const float n = (float)(o1 - o0);
            amp = lead / (n * n);
            c = a.counts + (int64_t)b * a.E;
          }
        }
      }
      if (c) {
#pragma unroll
        for (int n = 0; n < N; n++) {
          const int e = expert_of<V>(n, G, lane);
          if (e < a.E) mean += s[n] * (float)__ldg(c + e);
        }
      }
      mean = group_sum(mean, G) * (soft ? 1.f : z.inv_z);
    }

    // routing: sums over the slots
    float kept = 0.f, dot = 0.f;
    if (a.dw) {
      for (int j = lane; in && j < a.k; j += G) {
        const int e = __ldg(a.idx + t * a.k + j);
        if (e >= 0 && e < a.E) {
          const float le = logit_of(a, t, e);
          float se, r;
          if (soft) se = expf(le - z.m) * z.inv_z;
          else sigmoid_pair(le, &se, &r);
          kept += se;
          dot += se * __ldg(a.dw + t * a.k + j);
        }
      }
      kept = group_sum(kept, G);
      dot = group_sum(dot, G);
    }
    // w_j = S s_j / den: ds_j = S / den (dw_j - [not clamped] dot / den)
    float inv_den = 1.f, shift = 0.f;
    if (a.renorm) {
      inv_den = 1.f / fmaxf(kept, 0x1p-14f);
      if (!(kept < 0x1p-14f)) shift = dot * inv_den;
    }
    const float f = a.scale * inv_den;
    // softmax: dl_e = s_e (ds_e - sum_e s ds); the sum is 0 when the weights are renormalised
    const float drop = soft ? f * (dot - shift * kept) : 0.f;

    // the dense part to the row in shared memory, the slots added there
#pragma unroll
    for (int n = 0; n < N; n++) {
      const int e = expert_of<V>(n, G, lane);
      float d = 0.f;
      if (e < a.E) {
        const float g = c ? amp * ((float)__ldg(c + e) - mean) : 0.f;
        if (soft) {
          d = s[n] * (g - drop);
        } else if (c) {
          float se, r;
          sigmoid_pair(l[n], &se, &r);
          d = g * z.inv_z * se * r;
        }
      }
      mine[(n / V) * G * V + lane * V + n % V] = d;
    }
    if (a.dw) {
      for (int q = 0; q < rounds; q++) {
        const int j = q * G + lane;
        int e = -1;
        float add = 0.f;
        if (in && j < a.k) {
          e = __ldg(a.idx + t * a.k + j);
          if (e < 0 || e >= a.E) e = -1;
        }
        if (e >= 0) {
          const float le = logit_of(a, t, e);
          float se, r = 1.f;
          if (soft) se = expf(le - z.m) * z.inv_z;
          else sigmoid_pair(le, &se, &r);
          add = f * (__ldg(a.dw + t * a.k + j) - shift) * se * r;
        }
        // slots of one token that name the same expert are added in slot order
        const unsigned same = __match_any_sync(0xffffffffu, e >= 0 ? (group & 31) * a.E + e : -1 - (int)(threadIdx.x & 31));
        __syncwarp();
        if (__any_sync(0xffffffffu, __popc(same) > 1)) {
          for (int g = 0; g < G; g++) {
            if (lane == g && e >= 0) mine[e] += add;
            __syncwarp();
          }
        } else if (e >= 0) {
          mine[e] += add;
        }
        __syncwarp();
      }
    } else {
      __syncwarp();
    }
    if (in) {
      if constexpr (V > 1) {
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.dlogits) + t * a.E * (16 / V));
#pragma unroll
        for (int i = 0; i < NV; i++) {
          if ((i * G + lane) * V >= a.E) continue;
          const float4* m = reinterpret_cast<const float4*>(mine + (i * G + lane) * V);
          if constexpr (BF16) {
            const float4 x = m[0], y = m[1];
            out[i * G + lane] = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y),
                                           pack_bf16x2(y.z, y.w));
          } else {
            out[i * G + lane] = *reinterpret_cast<const uint4*>(m);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; i++) {
          const int e = i * G + lane;
          if (e >= a.E) continue;
          if constexpr (BF16) static_cast<uint16_t*>(a.dlogits)[t * a.E + e] = f32_to_bf16_rn(mine[e]);
          else static_cast<float*>(a.dlogits)[t * a.E + e] = mine[e];
        }
      }
    }
    __syncwarp();  // the row is read before the next token's is written
  }
}

// ---------------------------------------------------------------- dispatch
// Lanes per token: the fewest (a power of two) that hold the row in one vector each.
int lanes_for(int E, int V) {
  int G = 1;
  while (G < 32 && G * V < E) G *= 2;
  return G;
}

template <int BF16, int V, int NV>
cudaError_t run_partial(const RouterTrainArgs& a, int G, cudaStream_t st) {
  int threads = partial_threads(V * NV);
  while (threads > 32 && threads / 32 * a.E > kPartialRows / 2) threads /= 2;  // at most 32 KiB of sums
  // no more groups of lanes than the chunk has tokens
  while (threads > 128 && threads / 2 / G >= a.chunk) threads /= 2;
  const size_t smem = (size_t)(threads / 32 + 1) * a.E * 4;
  return launch_pdl(balance_partial_kernel<BF16, V, NV>, (unsigned)a.nchunks, threads, smem, st, a, G);
}

template <int BF16, int V, int NV>
cudaError_t run_backward(const RouterTrainArgs& a, int G, int num_sms, cudaStream_t st) {
  const int groups = kBackThreads / G;
  const int64_t blocks = ((int64_t)a.T + groups - 1) / groups, most = (int64_t)num_sms * 8;
  return launch_pdl(router_backward_kernel<BF16, V, NV>, (unsigned)(blocks < most ? blocks : most), kBackThreads,
                    (size_t)kBackThreads * V * NV * 4, st, a, G);
}

template <template <int, int, int> class Run, typename... Args>
cudaError_t by_row(const RouterTrainArgs& a, Args... rest) {
  const int V = a.vec ? (a.bf16 ? 8 : 4) : 1;
  const int G = lanes_for(a.E, V), nv = (a.E + G * V - 1) / (G * V);
  if (a.vec && a.bf16) {
    if (nv <= 1) return Run<1, 8, 1>::go(a, G, rest...);
    if (nv <= 2) return Run<1, 8, 2>::go(a, G, rest...);
    return Run<1, 8, 4>::go(a, G, rest...);
  }
  if (a.vec) {
    if (nv <= 1) return Run<0, 4, 1>::go(a, G, rest...);
    if (nv <= 2) return Run<0, 4, 2>::go(a, G, rest...);
    if (nv <= 4) return Run<0, 4, 4>::go(a, G, rest...);
    return Run<0, 4, 8>::go(a, G, rest...);
  }
  if (a.bf16) {
    if (nv <= 2) return Run<1, 1, 2>::go(a, G, rest...);
    if (nv <= 8) return Run<1, 1, 8>::go(a, G, rest...);
    return Run<1, 1, 32>::go(a, G, rest...);
  }
  if (nv <= 2) return Run<0, 1, 2>::go(a, G, rest...);
  if (nv <= 8) return Run<0, 1, 8>::go(a, G, rest...);
  return Run<0, 1, 32>::go(a, G, rest...);
}

template <int BF16, int V, int NV>
struct Partial {
  static cudaError_t go(const RouterTrainArgs& a, int G, cudaStream_t st) { return run_partial<BF16, V, NV>(a, G, st); }
};
template <int BF16, int V, int NV>
struct Backward {
  static cudaError_t go(const RouterTrainArgs& a, int G, int sms, cudaStream_t st) {
    return run_backward<BF16, V, NV>(a, G, sms, st);
  }
};

}  // namespace

cudaError_t launch_balance_loss(const RouterTrainArgs& a, cudaStream_t st) {
  const cudaError_t e = by_row<Partial>(a, st);
  if (e != cudaSuccess) return e;
  // as many warps per block as a sequence has chunks on average
  int warps = 1;
  while (warps < 32 && warps * a.B < a.nchunks + a.B) warps *= 2;
  return launch_pdl(balance_finish_kernel, dim3((unsigned)a.B, (unsigned)((a.E + 31) / 32)), dim3(warps * 32), 0, st, a);
}

cudaError_t launch_router_backward(const RouterTrainArgs& a, int num_sms, cudaStream_t st) {
  return by_row<Backward>(a, num_sms, st);
}

}  // namespace moe
