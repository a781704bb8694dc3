// Balance loss of a router and its gradient.  Over the n_q tokens of sequence q, with counts_qe the
// (token, slot) pairs that chose expert e, s the scores and coef the loss's weight:
//   f_qe = counts_qe E / (k n_q)          1 for a balanced expert
//   R_t  = sum_e s_te,  p_te = s_te / R_t
//   D_t  = sum_e p_te f_qe                (q the sequence of token t)
//   w_q  = coef / (S' n_q)                (S' the number of sequences that have tokens)
//   L    = coef / S' sum_q sum_e f_qe mean_{t in q} p_te  =  sum_t w_q D_t
// The choice is piecewise constant, so f has no gradient, and
//   dL/ds_te = w_q (f_qe - D_t) / R_t.
// With the counts known, the loss and its gradient need one pass over the scores, a warp a token: the
// mean probabilities are never formed.  It is bound by that pass (scores read, gradient written).
#pragma once

#include "common.cuh"

namespace lmoe {

constexpr int kBalThreads = 256;
constexpr int kBalMaxBlocks = 2048;

struct BalanceParams {
  const float* scores;   // [T, E]
  const int* idx;        // [T, k]
  const int* cu;         // [S + 1] or null (one sequence of all T tokens)
  int T, E, k, S;
  float coef;
  int* counts;           // [S, E]
  float* loss;           // [1]
  float* dscores;        // [T, E] or null
  double* partial;       // scratch: [blocks]
  unsigned* done;        // scratch: blocks that finished
  uint32_t* status;
  int chunk;             // tokens a block
};

__device__ __forceinline__ int bal_cu(const BalanceParams& p, int q) {
  return p.cu ? min(max(p.cu[q], 0), p.T) : (q ? p.T : 0);
}
// The last sequence that begins at or before token t (-1: none does).
__device__ __forceinline__ int bal_seq(const BalanceParams& p, int t) {
  int lo = -1, hi = p.S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (bal_cu(p, mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// counts: a block counts a run of tokens in shared memory, sequence by sequence, and adds what it
// found (integer atomics: the order does not matter).
__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(const BalanceParams p) {
  extern __shared__ int hist[];
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) *p.done = 0;
    if (p.cu)
      for (int q = threadIdx.x; q <= p.S; q += kBalThreads)
        if (p.cu[q] < 0 || p.cu[q] > p.T || (q && p.cu[q] < p.cu[q - 1])) set_status(p.status, LMOE_STATUS_BAD_INDEX);
  }
  for (int q = max(bal_seq(p, t0), 0); q < p.S; ++q) {
    const int lo = max(t0, bal_cu(p, q)), hi = min(t1, bal_cu(p, q + 1));
    if (bal_cu(p, q) >= t1) break;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < p.E; e += kBalThreads) hist[e] = 0;
    __syncthreads();
    for (long long i = (long long)lo * p.k + threadIdx.x; i < (long long)hi * p.k; i += kBalThreads) {
      const int e = p.idx[i];
      if ((unsigned)e < (unsigned)p.E) atomicAdd(&hist[e], 1);
      else if (e != -1) set_status(p.status, LMOE_STATUS_BAD_INDEX);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kBalThreads)
      if (hist[e]) atomicAdd(&p.counts[(long long)q * p.E + e], hist[e]);
    __syncthreads();
  }
}

// loss and gradient, a warp a token; lane l holds experts VEC (l + 32 j) .. + VEC - 1.
template <int NJ, int VEC>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(const BalanceParams p) {
  __shared__ float wsum[kBalThreads / 32];
  __shared__ int filled;
  __shared__ bool last;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) filled = 0;
  __syncthreads();
  int mine = 0;
  for (int q = threadIdx.x; q < p.S; q += kBalThreads) mine += bal_cu(p, q + 1) > bal_cu(p, q);
  if (mine) atomicAdd(&filled, mine);
  __syncthreads();
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  float f[NJ * VEC];
  float acc = 0.f, wq = 0.f;
  int q_lo = 0, q_hi = 0;  // token range for which f and wq hold
  bool inside = false, nan = false;
  for (int t = t0 + warp; t < t1; t += kBalThreads / 32) {
    if (t >= q_hi || t < q_lo) {
      const int q = bal_seq(p, t);
      inside = q >= 0 && t < bal_cu(p, q + 1);
      q_lo = t;
      q_hi = t + 1;
      if (inside) {
        q_hi = bal_cu(p, q + 1);
        const int n = q_hi - bal_cu(p, q);
        const float fs = (float)p.E / ((float)p.k * (float)n);
        wq = p.coef / ((float)filled * (float)n);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int e = (lane + 32 * j) * VEC + i;
            f[j * VEC + i] = e < p.E ? (float)p.counts[(long long)q * p.E + e] * fs : 0.f;
          }
      }
    }
    const float* srow = p.scores + (long long)t * p.E;
    float* drow = p.dscores ? p.dscores + (long long)t * p.E : nullptr;
    float s[NJ * VEC];
    float R = 0.f, D = 0.f;
    if (inside) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = (lane + 32 * j) * VEC;
        if constexpr (VEC == 4) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (e < p.E) v = __ldcs(reinterpret_cast<const float4*>(srow + e));
          s[4 * j] = v.x; s[4 * j + 1] = v.y; s[4 * j + 2] = v.z; s[4 * j + 3] = v.w;
        } else {
          s[j] = e < p.E ? __ldcs(srow + e) : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < NJ * VEC; ++i) {
        R += s[i];
        D = fmaf(s[i], f[i], D);
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        R += __shfl_xor_sync(0xffffffffu, R, off);
        D += __shfl_xor_sync(0xffffffffu, D, off);
      }
      nan |= R != R;
    }
    // a row of zeros has no probabilities: it adds nothing and gets no gradient
    const float inv = inside && R != 0.f ? 1.f / R : 0.f;
    D *= inv;
    const float g = wq * inv;
    if (inside) acc = fmaf(wq, D, acc);
    if (drow) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = (lane + 32 * j) * VEC;
        if (e >= p.E) continue;
        if constexpr (VEC == 4) {
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          if (inside)
            o = make_float4(g * (f[4 * j] - D), g * (f[4 * j + 1] - D), g * (f[4 * j + 2] - D), g * (f[4 * j + 3] - D));
          *reinterpret_cast<float4*>(drow + e) = o;
        } else {
          drow[e] = inside ? g * (f[j] - D) : 0.f;
        }
      }
    }
  }
  if (nan && lane == 0) set_status(p.status, LMOE_STATUS_NAN_SCORE);
  // the blocks' sums are added in their order by the last block to finish, in 64 bits
  if (lane == 0) wsum[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double b = 0;
    for (int w = 0; w < kBalThreads / 32; ++w) b += wsum[w];
    p.partial[blockIdx.x] = b;
    __threadfence();
    last = atomicAdd(p.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (last && warp == 0) {
    __threadfence();
    double b = 0;
    for (int i = lane; i < (int)gridDim.x; i += 32) b += reinterpret_cast<volatile double*>(p.partial)[i];
#pragma unroll
    for (int off = 16; off; off >>= 1) b += __shfl_xor_sync(0xffffffffu, b, off);
    if (lane == 0) *p.loss = (float)b;
  }
}

}  // namespace lmoe
