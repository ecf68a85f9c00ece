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
// Large batches are bound by instructions, some 30 a value for the exponential, the sums and
// the slots' detour, in half of the issue slots with a quarter to a third of the warps in
// flight: the loss of 32768 tokens and 256 experts 16.8 us on the device (2.8 at the memory's
// rate; 5 of them the second launch), the gradient of 65536 tokens and 128 experts 18.0 us
// (softmax; 22.6 sigmoid; 5.8).  Small ones by latency: 100 tokens 9.0 and 3.8 us.
#include "train.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- a token's row
// A token's row in G lanes: lane g holds experts (i G + g) V .. + V - 1, i < NV.
template <int BF16_, int V_, int NV_, int G_>
struct Layout {
  static constexpr int BF16 = BF16_, V = V_, NV = NV_, G = G_, N = V_ * NV_;
};

template <class L>
struct Row {
  uint4 v[L::V > 1 ? L::NV : 1];
  float s[L::V > 1 ? 1 : L::NV];

  // (-inf past E: those values take part in maxima and sums as nothing)
  __device__ __forceinline__ void load(const void* base, int64_t t, int E, int lane) {
    if constexpr (L::V > 1) {
      constexpr uint32_t inf = L::BF16 ? 0xff80ff80u : 0xff800000u;
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + t * E * (16 / L::V));
#pragma unroll
      for (int i = 0; i < L::NV; i++)
        v[i] = (i * L::G + lane) * L::V < E ? __ldg(p + i * L::G + lane) : make_uint4(inf, inf, inf, inf);
    } else {
#pragma unroll
      for (int i = 0; i < L::NV; i++) {
        const int e = i * L::G + lane;
        s[i] = -INFINITY;
        if (e < E)
          s[i] = L::BF16 ? bf16_to_f32(__ldg(static_cast<const uint16_t*>(base) + t * E + e))
                         : __ldg(static_cast<const float*>(base) + t * E + e);
      }
    }
  }
  __device__ __forceinline__ float get(int n) const {
    if constexpr (L::V == 1) return s[n];
    const uint4& q = v[n / L::V];
    const int c = n % L::V;
    if constexpr (L::BF16) {
      const uint32_t u = c < 2 ? q.x : c < 4 ? q.y : c < 6 ? q.z : q.w;
      return __uint_as_float(c & 1 ? u & 0xffff0000u : u << 16);
    } else {
      return __uint_as_float(c == 0 ? q.x : c == 1 ? q.y : c == 2 ? q.z : q.w);
    }
  }
};

// Expert of a lane's n-th value; a vector is whole or past E (E is a multiple of V).
template <class L>
__device__ __forceinline__ int expert_of(int n, int lane) {
  return ((n / L::V) * L::G + lane) * L::V + n % L::V;
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G >> 1; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int G>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
  for (int o = G >> 1; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ float load_one(const void* p, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(__ldg(static_cast<const uint16_t*>(p) + i)) : __ldg(static_cast<const float*>(p) + i);
}

// The router bias of a lane's experts (0 without one, and past E).
template <class L>
__device__ __forceinline__ void load_bias(const RouterTrainArgs& a, int lane, float (&b)[L::N]) {
#pragma unroll
  for (int n = 0; n < L::N; n++) {
    const int e = expert_of<L>(n, lane);
    b[n] = a.router_bias && e < a.E ? load_one(a.router_bias, L::BF16, e) : 0.f;
  }
}

// exp and 1 / x by the hardware instructions: 2^-22 relative, exp 2^-24 |x| more (its
// argument is scaled by log2 e in fp32).
__device__ __forceinline__ float fast_exp(float x) { return __expf(x); }
__device__ __forceinline__ float fast_rcp(float x) { return __fdividef(1.f, x); }

// The same where results below 2^-126 may be 0: exp(x + y) = 2^(x log2 e + y2) for y2 = y log2 e
// (2^-24 (|x| + |y|) from the argument), and 1 / x.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_ftz(float x, float y2) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(x, kLog2e, y2)));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sigma(l) and 1 - sigma(l), both to full relative precision.
__device__ __forceinline__ void sigmoid_pair(float l, float* s, float* r) {
  const float x = fast_exp(-fabsf(l)), d = fast_rcp(1.f + x);
  *s = l >= 0.f ? d : x * d;
  *r = l >= 0.f ? x * d : d;
  if (l != l) *s = *r = l;
}

// What turns a logit into its score: softmax s = exp(l - m) inv_z, the share, m the row's
// largest logit; sigmoid s = sigma(l) exp(-m), m = min(the largest, 0), and the share s inv_z.
// (sigma alone leaves fp32 from -87 down, and with it the shares of a row of such logits.
// Rows apart, by a branch, cost the other rows registers: loss of 65536 tokens and 32 experts
// 14.2 us as it is, 17.7 with the branch; of 32768 and 256 16.8 and 16.9.)
struct Norm {
  float inv_z, m;
};
// Sigmoid rows that lie below this throughout have no shares: the type's lowest value is a mask.
constexpr float kMaskedLogit = -700.f;

// l' of the row in l[], scores in s[] (0 past E).  Whole warp.
template <class L>
__device__ __forceinline__ Norm scores(const RouterTrainArgs& a, const Row<L>& row, const float (&bias)[L::N],
                                       float (&l)[L::N], float (&s)[L::N]) {
#pragma unroll
  for (int n = 0; n < L::N; n++) l[n] = row.get(n);
  if (a.router_bias) {
#pragma unroll
    for (int n = 0; n < L::N; n++) l[n] += bias[n];
  }
  float m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int n = 0; n < L::N; n++) m = fmaxf(m, l[n]);
  m = group_max<L::G>(m);
  if (a.score == MOE_SCORE_SOFTMAX) {
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int n = 0; n < L::N; n++) {
      s[n] = fast_exp(l[n] - m);
      sum += s[n];
    }
  } else {
    m = m < kMaskedLogit ? 0.f : fminf(m, 0.f);  // (masked: every score 0)
    const float em = fast_exp(m), m2 = m * kLog2e;
#pragma unroll
    for (int n = 0; n < L::N; n++) {
      s[n] = rcp_ftz(em + exp_ftz(-l[n], m2));  // 0 from 87 below m down; em + .. >= 1
      sum += s[n];
    }
  }
  sum = group_sum<L::G>(sum);
  const Norm z{sum == 0.f ? 0.f : 1.f / sum, m};
  if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int n = 0; n < L::N; n++) s[n] *= z.inv_z;
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
constexpr int partial_threads(int n) { return n >= 16 ? 256 : 512; }  // n values of a row per lane
constexpr int kPartialSums = 8192;  // floats of a block's sums: a row of E per warp

template <class L>
__global__ void __launch_bounds__(partial_threads(L::N)) balance_partial_kernel(RouterTrainArgs a) {
  constexpr int G = L::G, N = L::N;
  extern __shared__ float sums[];  // [warps][E], then the histogram [E]
  int32_t* hist = reinterpret_cast<int32_t*>(sums + (blockDim.x >> 5) * a.E);
  pdl_enter();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int lane = threadIdx.x % G, group = threadIdx.x / G, groups = blockDim.x / G;
  float bias[N];
  load_bias<L>(a, lane, bias);
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  for (int b = max(0, seq_of(a, t0)); b < a.B; b++) {
    const int s0 = max(t0, seq_at(a, b)), s1 = min(t1, seq_at(a, b + 1));
    if (s0 >= t1) break;
    if (s0 >= s1) continue;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    float acc[N];
#pragma unroll
    for (int n = 0; n < N; n++) acc[n] = 0.f;
    Row<L> next;
    int t = s0 + group;
    if (t < s1) next.load(a.logits, t, a.E, lane);
    // the whole warp takes every step (the sums are shuffles)
    for (int base = s0; base < s1; base += groups, t += groups) {
      const Row<L> row = next;
      if (t + groups < s1) next.load(a.logits, t + groups, a.E, lane);
      float l[N], s[N];
      const Norm z = scores<L>(a, row, bias, l, s);
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
#pragma unroll
      for (int o = G; o < 32; o <<= 1) acc[n] += __shfl_xor_sync(0xffffffffu, acc[n], o);
      const int e = expert_of<L>(n, lane);
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
constexpr int back_blocks(int n) { return n <= 8 ? 4 : n <= 16 ? 2 : 1; }  // per SM, n values of a row per lane

template <class L>
__global__ void __launch_bounds__(kBackThreads, back_blocks(L::N)) router_backward_kernel(RouterTrainArgs a) {
  constexpr int G = L::G, N = L::N, V = L::V;
  constexpr int kSlots = N < 32 / G ? N : 32 / G;  // slots per lane: k <= E, k <= 32
  constexpr int groups = kBackThreads / G;
  extern __shared__ float4 rows4[];  // [groups][G N] floats
  __shared__ int live_seqs;
  pdl_enter();
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  float* mine = reinterpret_cast<float*>(rows4) + group * G * N;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  float lead = 0.f;  // dloss coef E / k / B'
  if (a.counts) {
    if (threadIdx.x == 0) live_seqs = 0;
    __syncthreads();
    int live = 0;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) live += seq_at(a, b + 1) > seq_at(a, b);
    live = __reduce_add_sync(0xffffffffu, live);
    if ((threadIdx.x & 31) == 0 && live) atomicAdd(&live_seqs, live);
    __syncthreads();
    lead = (a.dloss ? *a.dloss : 1.f) * a.coef * (float)a.E / ((float)a.k * (float)max(live_seqs, 1));
  }
  float bias[N];
  load_bias<L>(a, lane, bias);
  // this block's tokens are neighbours: the sequence and its counts change rarely and stay
  // in registers
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk, c1 = min((int64_t)a.T, c0 + a.chunk);
  int seq_end = -1;    // tokens below it have the amplitude and counts held
  float amp = 0.f, cnt[N];
#pragma unroll
  for (int n = 0; n < N; n++) cnt[n] = 0.f;
  auto store_row = [&](const float (&x)[N]) {
#pragma unroll
    for (int n = 0; n < N; n += V >= 4 ? 4 : 1) {
      const int e = (n / V) * G * V + lane * V + n % V;
      if constexpr (V >= 4) *reinterpret_cast<float4*>(mine + e) = make_float4(x[n], x[n + 1], x[n + 2], x[n + 3]);
      else mine[e] = x[n];
    }
  };
  struct Slots {
    int e[kSlots];
    float dw[kSlots];
  } slots, next_slots;
  auto load_slots = [&](int64_t t, Slots& s) {
    if (!a.dw) return;
#pragma unroll
    for (int q = 0; q < kSlots; q++) {
      const int j = q * G + lane;
      s.e[q] = -1;
      s.dw[q] = 0.f;
      if (q > 0 && q * G >= a.k) continue;  // (uniform: no lane has such a slot)
      if (t < c1 && j < a.k) {
        const int64_t at = t * a.k + j;
        const int e = __ldg(a.idx + at);
        const float dw = __ldg(a.dw + at);
        // (a slot without an expert has no weight: its gradient may be anything, a NaN too)
        s.e[q] = (unsigned)e < (unsigned)a.E ? e : -1;
        s.dw[q] = s.e[q] >= 0 ? dw : 0.f;
      }
    }
  };
  int64_t t = c0 + group;
  Row<L> next;
  if (t < c1) next.load(a.logits, t, a.E, lane);
  load_slots(t, next_slots);
  // the whole block takes every step (shuffles and warp barriers)
  for (int64_t base = c0; base < c1; base += groups, t += groups) {
    const bool in = t < c1;
    const Row<L> row = next;
    slots = next_slots;
    if (t + groups < c1) next.load(a.logits, t + groups, a.E, lane);
    load_slots(t + groups, next_slots);
    float l[N], s[N];
    const Norm z = scores<L>(a, row, bias, l, s);

    // balance: A (c_e - sum c p), A = 0 for tokens outside every sequence
    float mean = 0.f;
    if (a.counts) {
      if (in && t >= seq_end) {
        const int b = seq_of(a, (int)t);
        amp = 0.f;
        if (b < 0 || b >= a.B) {
          seq_end = b < 0 ? seq_at(a, 0) : a.T;
        } else {
          const int o0 = seq_at(a, b);
          seq_end = seq_at(a, b + 1);
          if (t < seq_end) amp = lead / ((float)(seq_end - o0) * (float)(seq_end - o0));
          const int32_t* c = a.counts + (int64_t)b * a.E;
#pragma unroll
          for (int n = 0; n < N; n++) {
            const int e = expert_of<L>(n, lane);
            cnt[n] = e < a.E ? (float)__ldg(c + e) : 0.f;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < N; n++) mean = fmaf(s[n], cnt[n], mean);
      mean = group_sum<G>(mean) * (soft ? 1.f : z.inv_z);
    }

    // routing: the slots' scores (softmax) or logits (sigmoid) through the row in shared
    // memory, and their sums
    float kept = 0.f, dot = 0.f, ss[kSlots], sr[kSlots];
    bool twice[kSlots];
    if (a.dw) {
      store_row(soft ? s : l);
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kSlots; q++) {
        ss[q] = 0.f;
        sr[q] = 1.f;
        if (q > 0 && q * G >= a.k) continue;
        if (slots.e[q] >= 0) {
          ss[q] = mine[slots.e[q]];
          if (!soft) sigmoid_pair(ss[q], &ss[q], &sr[q]);
        }
        kept += ss[q];
        dot = fmaf(ss[q], slots.dw[q], dot);
      }
      kept = group_sum<G>(kept);
      dot = group_sum<G>(dot);
      // does another lane's slot name the same expert?  Each leaves its number there.
#pragma unroll
      for (int q = 0; q < kSlots; q++) {
        twice[q] = false;
        if (q > 0 && q * G >= a.k) break;
        __syncwarp();
        if (slots.e[q] >= 0) reinterpret_cast<int*>(mine)[slots.e[q]] = lane;
        __syncwarp();
        if (slots.e[q] >= 0) twice[q] = reinterpret_cast<int*>(mine)[slots.e[q]] != lane;
      }
      __syncwarp();
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
    float d[N];
    if (soft) {
      const float less = fmaf(amp, mean, drop);
#pragma unroll
      for (int n = 0; n < N; n++) d[n] = s[n] * fmaf(amp, cnt[n], -less);
      // nothing of the row enters, whatever its logits (a padding token's may be a NaN)
      const bool inert = amp == 0.f && drop == 0.f;
      if (__any_sync(0xffffffffu, inert)) {
#pragma unroll
        for (int n = 0; n < N; n++) d[n] = inert ? 0.f : d[n];
      }
    } else {
#pragma unroll
      for (int n = 0; n < N; n++) d[n] = 0.f;
      if (a.counts && amp != 0.f) {
        // s = sigma(l) exp(-m) and r = 1 - sigma(l), both to full relative precision; all l <= m for m < 0
        const float g = amp * z.inv_z, em = fast_exp(z.m), m2 = -z.m * kLog2e;
#pragma unroll
        for (int n = 0; n < N; n++) {
          const float x = exp_ftz(-fabsf(l[n]), m2), xe = x * em, q = rcp_ftz(1.f + xe);
          const float se = l[n] >= 0.f ? q : x * q, r = l[n] >= 0.f ? xe * q : q;
          d[n] = g * (cnt[n] - mean) * se * r;
        }
      }
    }
    if (a.dw) {
      store_row(d);
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kSlots; q++) {
        if (q > 0 && q * G >= a.k) break;
        const int e = slots.e[q];
        const float add = f * (slots.dw[q] - shift) * ss[q] * sr[q];
        // slots of one token that name the same expert are added in slot order
        if (__any_sync(0xffffffffu, twice[q])) {
          for (int g = 0; g < G; g++) {
            if (lane == g && e >= 0) mine[e] += add;
            __syncwarp();
          }
        } else if (e >= 0) {
          mine[e] += add;
        }
        __syncwarp();
      }
#pragma unroll
      for (int n = 0; n < N; n += V >= 4 ? 4 : 1) {
        const int e = (n / V) * G * V + lane * V + n % V;
        if constexpr (V >= 4) {
          const float4 x = *reinterpret_cast<const float4*>(mine + e);
          d[n] = x.x, d[n + 1] = x.y, d[n + 2] = x.z, d[n + 3] = x.w;
        } else {
          d[n] = mine[e];
        }
      }
      __syncwarp();  // the row is read before the next token's is written
    }
    if (in) {
      if constexpr (V > 1) {
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.dlogits) + t * a.E * (16 / V));
#pragma unroll
        for (int i = 0; i < L::NV; i++) {
          if ((i * G + lane) * V >= a.E) continue;
          const float* x = &d[i * V];
          if constexpr (L::BF16)
            out[i * G + lane] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                           pack_bf16x2(x[6], x[7]));
          else
            out[i * G + lane] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                           __float_as_uint(x[3]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < L::NV; i++) {
          const int e = i * G + lane;
          if (e >= a.E) continue;
          if constexpr (L::BF16) static_cast<uint16_t*>(a.dlogits)[t * a.E + e] = f32_to_bf16_rn(d[i]);
          else static_cast<float*>(a.dlogits)[t * a.E + e] = d[i];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- dispatch
// Vectors of a row per lane, of rows of w vectors of v values.  Fewer lanes per token share
// the shuffles and the slots among fewer, and more values per lane cost registers and so
// warps in flight.
// Loss: two.  65536 x 64 / 65536 x 128 / 32768 x 256 bf16, one, two, four per lane:
// 18.4 / 21.2 / 22.5, 16.6 / 18.6 / 18.5, 22.8 / 22.6 / 23.1 us.
template <class L>
struct Partial {
  static constexpr int vectors(int w, int) { return w > 1 ? 2 : 1; }
  static cudaError_t go(const RouterTrainArgs& a, cudaStream_t st) {
    int threads = partial_threads(L::N);
    while (threads > 32 && threads / 32 * a.E > kPartialSums) threads /= 2;
    // no more groups of lanes than the chunk has tokens
    while (threads > 128 && threads / 2 / L::G >= a.chunk) threads /= 2;
    const size_t smem = (size_t)(threads / 32 + 1) * a.E * 4;
    return launch_pdl(balance_partial_kernel<L>, (unsigned)a.nchunks, threads, smem, st, a);
  }
};
// Backward: eight lanes per token, from 128 experts on 16 values per lane.  The same sizes, 8
// and 16 values per lane: 18.6 / 24.7 / 22.6, 18.5 / 22.3 / 20.6 us; 65536 x 32 fp32, 4 and 8:
// 16.4, 20.6 us.
template <class L>
struct Backward {
  static constexpr int vectors(int w, int v) { return w <= 8 ? 1 : w / 8 < 16 / v ? w / 8 : 16 / v; }
  static cudaError_t go(const RouterTrainArgs& a, int sms, cudaStream_t st) {
    // neighbouring tokens to a block, whole steps of its groups, one wave
    constexpr int groups = kBackThreads / L::G;
    RouterTrainArgs b = a;
    const int64_t blocks = (int64_t)sms * back_blocks(L::N), per = (a.T + blocks - 1) / blocks;
    b.chunk = (int)((per + groups - 1) / groups * groups);
    return launch_pdl(router_backward_kernel<L>, (unsigned)((a.T + b.chunk - 1) / b.chunk), kBackThreads,
                      (size_t)kBackThreads * L::N * 4, st, b);
  }
};

// Rows of up to W vectors (a power of two), Run's share of them per lane and what 32 lanes
// cannot share otherwise.
template <template <class> class Run, int BF16, int W, typename... Args>
cudaError_t by_vectors(const RouterTrainArgs& a, Args... rest) {
  constexpr int V = BF16 ? 8 : 4;
  if constexpr (W < kMaxE / V) {
    if (a.E > W * V) return by_vectors<Run, BF16, 2 * W>(a, rest...);
  }
  constexpr int share = Run<Layout<BF16, V, 1, 1>>::vectors(W, V), NV = share > W / 32 ? share : W / 32;
  return Run<Layout<BF16, V, NV, W / NV>>::go(a, rest...);
}
template <template <class> class Run, int BF16, typename... Args>
cudaError_t by_values(const RouterTrainArgs& a, Args... rest) {
  if (a.E <= 32) return Run<Layout<BF16, 1, 1, 32>>::go(a, rest...);
  if (a.E <= 64) return Run<Layout<BF16, 1, 2, 32>>::go(a, rest...);
  if (a.E <= 256) return Run<Layout<BF16, 1, 8, 32>>::go(a, rest...);
  return Run<Layout<BF16, 1, 32, 32>>::go(a, rest...);
}
template <template <class> class Run, typename... Args>
cudaError_t by_row(const RouterTrainArgs& a, Args... rest) {
  if (a.vec) return a.bf16 ? by_vectors<Run, 1, 1>(a, rest...) : by_vectors<Run, 0, 1>(a, rest...);
  return a.bf16 ? by_values<Run, 1>(a, rest...) : by_values<Run, 0>(a, rest...);
}

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
