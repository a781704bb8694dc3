// Balance loss of a router and its gradient.  Over the n_q tokens of sequence q, with counts_qe the
// (token, slot) pairs that chose expert e, s the scores and coef the loss's weight:
//   f_qe = counts_qe E / (k n_q)          1 for a balanced expert
//   R_t  = sum_e s_te,  p_te = s_te / R_t
//   D_t  = sum_e p_te f_qe                (q the sequence of token t)
//   w_q  = coef / (S' n_q)                (S' the number of sequences that have tokens)
//   L    = coef / S' sum_q sum_e f_qe mean_{t in q} p_te  =  sum_t w_q D_t
// The choice is piecewise constant, so f has no gradient, and
//   dL/ds_te = w_q (f_qe - D_t) / R_t.
// With the counts known, the loss and its gradient need one pass over the scores: the mean
// probabilities are never formed.  The pass is bound by memory (scores read, gradient written).
// Near balance f and D are both close to 1 and f - D cancels, so both are held as what they differ from
// 1 by, f from whole numbers: f_qe - 1 = (counts_qe E - k n_q) / (k n_q), D_t - 1 = sum_e p_te (f_qe - 1).
// A token whose probabilities lie on experts that few chose has a D near 0, where D - 1 cancels in its
// turn: rows of D < 1/2 are taken again with f and D themselves.
//
// Two forms.  A batch whose scores a few SMs can stream takes one launch of one cluster of CTAs, which
// count their own tokens, add the counts up through distributed shared memory and go on to the pass.
// A larger one takes two launches over the whole GPU, counting (integer atomics: their order does not
// matter) and the pass.  Either way the loss's partial sums are added in a fixed order, in 64 bits.
#pragma once

#include "common.cuh"

namespace lmoe {

constexpr int kBalThreads = 512;
constexpr int kBalMaxBlocks = 1024;
constexpr int kBalHistInts = 8192;   // shared counters of a block
constexpr int kBalMaxCluster = 16;
constexpr int kBalMaxE = 1024;

struct BalanceParams {
  const float* scores;   // [T, E]
  const int* idx;        // [T, k]
  const int* cu;         // [S + 1] or null (one sequence of all T tokens)
  int T, E, k, S;
  const int* total;      // [1] or null: S' where it is more than 0 (a batch spread over ranks)
  float coef;
  int* counts;           // [S, E]
  float* loss;           // [1]
  float* dscores;        // [T, E] or null
  double* partial;       // scratch: [blocks]
  unsigned* done;        // scratch: blocks that finished
  uint32_t* status;
  int chunk;             // tokens a block
};

// CTAs of the one-launch form, at most `most`: a round of rows each, and at most some two sequences each,
// which a CTA takes in turn (a few microseconds each).
constexpr int bal_ctas(int T, int S, int round, int most) {
  int ctas = 1;
  while (ctas < most && (ctas * round < T || 2 * ctas < (S < T ? S : T))) ctas *= 2;
  return ctas;
}
static_assert(bal_ctas(64, 1, 64, 16) == 1 && bal_ctas(65, 1, 64, 16) == 2, "a round of rows each");
static_assert(bal_ctas(8192, 1, 64, 16) == 16 && bal_ctas(8192, 1, 64, 8) == 8, "at most as many as the device places");
static_assert(bal_ctas(64, 16, 64, 16) == 8 && bal_ctas(3, 900, 64, 16) == 2, "two sequences each");

// Sequence bounds a block needs, checked: cu that decreases or leaves [0, T] is reported and counts as
// no sequence at all.  Up to kBalSeqCache sequences' bounds are kept in shared memory, where looking a
// token's sequence up does not wait for memory step by step.
constexpr int kBalSeqCache = 1023;
struct BalSeqs {
  const int* cu;   // shared or global
  int S, filled;   // sequences; S'
  __device__ __forceinline__ int begin(int q) const { return cu[q]; }
  // The last sequence behind lo that begins at or before token t (lo: none does).
  __device__ __forceinline__ int at(int t, int lo = -1) const {
    int hi = S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (begin(mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
  }
  // The sequence after q to look at: a run of empty ones, which may be millions, is stepped over at once.
  // Always past q, also where the caller's bounds change under the kernel: its loops end.
  __device__ __forceinline__ int next(int q) const {
    ++q;
    return q < S && begin(q) == begin(q + 1) ? at(begin(q), q) : q;
  }
};
struct BalSeqSmem {
  int cu[kBalSeqCache + 1];
  int filled, bad;
};
// The whole block takes part.
__device__ __forceinline__ BalSeqs bal_seqs(const BalanceParams& p, BalSeqSmem& m) {
  if (threadIdx.x == 0) m.filled = m.bad = 0;
  const int total = p.total ? *p.total : 0;
  __syncthreads();
  int mine = 0, bad = 0;
  for (int q = threadIdx.x; q < p.S; q += kBalThreads) {
    const int a = p.cu ? p.cu[q] : 0, b = p.cu ? p.cu[q + 1] : p.T;
    mine += b > a;
    bad |= a < 0 || b > p.T || b < a;
    if (p.S <= kBalSeqCache) {
      m.cu[q] = a;
      if (q == p.S - 1) m.cu[p.S] = b;
    }
  }
  if (mine) atomicAdd(&m.filled, mine);
  if (bad) m.bad = 1;
  __syncthreads();
  if (m.bad && threadIdx.x == 0) set_status(p.status, LMOE_STATUS_BAD_INDEX);
  return BalSeqs{p.S <= kBalSeqCache ? m.cu : p.cu, m.bad ? 0 : p.S, total > 0 ? total : m.filled};
}

// Copies of each of n shared counters: a power of two up to 32, one a lane where there are few, so that
// few experts' counters do not make the lanes wait for each other (many experts' hardly meet).
__device__ __forceinline__ int bal_copies(int n) {
  int c = 32;
  while (c > 1 && n * c > 4096) c >>= 1;
  return c;
}
// Adds the choices of tokens [lo, hi) to hist (copies of each expert side by side).
__device__ __forceinline__ void bal_count(const BalanceParams& p, int lo, int hi, int* hist, int copies) {
  const int mine = threadIdx.x & (copies - 1);
  const int end = hi * p.k;  // T k is at most 2^30
#pragma unroll 4
  for (int i = lo * p.k + threadIdx.x; i < end; i += kBalThreads) {
    const int e = p.idx[i];
    if ((unsigned)e < (unsigned)p.E) atomicAdd(&hist[e * copies + mine], 1);
    else if (e != -1) set_status(p.status, LMOE_STATUS_BAD_INDEX);
  }
}

// Sums between these bounds have a reciprocal that every product here stays finite with; the rows of other
// sums, and those of D < 1/2, are left to bal_row_alone.
constexpr float kBalSumMin = 0x1p-60f, kBalSumMax = 0x1p60f;

// One row by itself, LANES lanes a row (`there` is false for lanes without one).  f: shared, f - 1 and,
// kBalMaxE further, f.  Scores so small that 1 / R overflows or so large that R does are taken again times c, a
// power of two, which D does not see and the gradient's 1 / R gives back.  D < 1/2 is summed as it is, D
// above as D - 1.  A gradient past fp32 saturates at its largest value; a row of zeros has no
// probabilities: it adds nothing and gets no gradient.  Returns D in the row's first lane.  A batch of
// such rows alone takes 50 us at 16384 x 896 for 29 of ordinary ones, 16.5 us at 8192 x 256 for 12.5.
template <int LANES>
__device__ __forceinline__ double bal_row_alone(const float* srow, float* drow, int E, const float* f, float wq,
                                                bool there, bool& nan) {
  const int lane = threadIdx.x & (LANES - 1), end = there ? E : 0;
  float c = 1.f, sum, dot, whole;
  for (bool again = false;; again = true) {
    sum = dot = whole = 0.f;
#pragma unroll 4
    for (int e = lane; e < end; e += LANES) {
      const float v = srow[e] * c;
      sum += v;
      dot = fmaf(v, f[e], dot);
      whole = fmaf(v, f[kBalMaxE + e], whole);
    }
#pragma unroll
    for (int off = LANES / 2; off; off >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, off);
      dot += __shfl_xor_sync(0xffffffffu, dot, off);
      whole += __shfl_xor_sync(0xffffffffu, whole, off);
    }
    const bool inside = sum >= kBalSumMin && sum <= kBalSumMax;
    if (again || !__any_sync(0xffffffffu, there && !inside)) break;
    if (!inside) c = sum < kBalSumMin ? 0x1p64f : 0x1p-64f;
  }
  nan |= !(fabsf(sum) <= 3.4028234e38f);
  const bool some = sum != 0.f, low = dot < -0.5f * sum;
  const float d = some ? (low ? whole : dot) / sum : 0.f;
  if (low) f += kBalMaxE;
  const float w = some ? wq / sum : 0.f;
  if (drow) {
#pragma unroll 4
    for (int e = lane; e < end; e += LANES) {
      const float g = w * (f[e] - d) * c;
      drow[e] = isinf(g) ? copysignf(3.4028234e38f, g) : g;
    }
  }
  return some && lane == 0 ? (low ? 0.0 : 1.0) + (double)d : 0.0;
}

// The pass over tokens [lo, hi) of one sequence: f (shared) holds f_qe - 1 and, kBalMaxE further, f_qe.
// LANES lanes share a row (a warp takes 32 / LANES rows side by side) and R such sets of rows are in flight;
// lane l of a row holds experts VEC (l + LANES j) .. + VEC - 1.  Returns the lane's sum of D (lane 0 of
// each row's); nan: some score was a NaN or infinite (such a row's sum is one too, which leaves it to
// bal_row_alone).
template <int NJ, int VEC, int R, int LANES>
__device__ __forceinline__ double bal_rows(const BalanceParams& p, int lo, int hi, const float* f, float wq, bool& nan) {
  constexpr int kSide = 32 / LANES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & (LANES - 1), side = (threadIdx.x & 31) / LANES;
  // D is summed as the rows' number and what theirs differ from 1 by, in 64 bits but for the R rows of a set: a
  // lane's sets may be thousands
  double acc = 0, alone = 0;
  int n = 0;
  for (int t0 = lo + warp * R * kSide + side; t0 - side < hi; t0 += kBalThreads / 32 * R * kSide) {
    float s[R][NJ * VEC], sum[R], dot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float* srow = p.scores + (long long)min(t0 + r * kSide, hi - 1) * p.E;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = (lane + LANES * j) * VEC;
        if constexpr (VEC == 4) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (e < p.E) v = __ldcs(reinterpret_cast<const float4*>(srow + e));
          s[r][4 * j] = v.x; s[r][4 * j + 1] = v.y; s[r][4 * j + 2] = v.z; s[r][4 * j + 3] = v.w;
        } else {
          s[r][j] = e < p.E ? __ldcs(srow + e) : 0.f;
        }
      }
    }
    auto fval = [&](int j) {
      const int e = (lane + LANES * j) * VEC;
      if constexpr (VEC == 4) return e < p.E ? *reinterpret_cast<const float4*>(f + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      else return make_float4(e < p.E ? f[e] : 0.f, 0.f, 0.f, 0.f);
    };
#pragma unroll
    for (int r = 0; r < R; ++r) sum[r] = dot[r] = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const float4 fv = fval(j);
      const float fe[4] = {fv.x, fv.y, fv.z, fv.w};
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          sum[r] += s[r][j * VEC + i];
          dot[r] = fmaf(s[r][j * VEC + i], fe[i], dot[r]);
        }
    }
#pragma unroll
    for (int off = LANES / 2; off; off >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], off);
        dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], off);
      }
    float g[R];
    unsigned skip = 0, left = 0;  // sets in which this lane's row is not there or left to bal_row_alone; is left
    float part = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool there = t0 + r * kSide < hi;
      const bool ok = sum[r] >= kBalSumMin && sum[r] <= kBalSumMax && dot[r] >= -0.5f * sum[r];
      const float inv = 1.f / sum[r];
      dot[r] *= inv;
      g[r] = wq * inv;
      if (there && ok) part += dot[r];
      else skip |= 1u << r;
      if (there && !ok) left |= 1u << r;
    }
    acc += (double)part;
    n += R - __popc(skip);
    if (p.dscores) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = (lane + LANES * j) * VEC;
        if (e >= p.E) continue;
        const float4 fv = fval(j);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if ((skip >> r) & 1) continue;
          float* d = p.dscores + (long long)(t0 + r * kSide) * p.E + e;
          if constexpr (VEC == 4)
            *reinterpret_cast<float4*>(d) = make_float4(g[r] * (fv.x - dot[r]), g[r] * (fv.y - dot[r]),
                                                        g[r] * (fv.z - dot[r]), g[r] * (fv.w - dot[r]));
          else
            *d = g[r] * (fv.x - dot[r]);
        }
      }
    }
    const unsigned rare = __reduce_or_sync(0xffffffffu, left);
#pragma unroll 1
    for (int r = 0; rare >> r; ++r) {
      if (!((rare >> r) & 1)) continue;
      const long long at = (long long)(t0 + r * kSide) * p.E;
      alone += bal_row_alone<LANES>(p.scores + at, p.dscores ? p.dscores + at : nullptr, p.E, f, wq, (left >> r) & 1, nan);
    }
  }
  return lane == 0 ? acc + (double)n + alone : 0.0;
}

// The pass over tokens [t0, t1), sequence by sequence (counts known): the block's share of the loss, for
// thread 0.  f: shared, [2 kBalMaxE]; wsum: shared, [kBalThreads / 32] doubles.
template <int NJ, int VEC, int R, int LANES>
__device__ __forceinline__ double bal_pass(const BalanceParams& p, const BalSeqs& sq, int t0, int t1, float* f,
                                           double* wsum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double acc = 0;
  bool nan = false;
  // tokens before the first sequence and behind the last
  if (p.dscores) {
    const int first = sq.S ? sq.begin(0) : p.T, end = sq.S ? sq.begin(sq.S) : p.T;
    const long long a1 = (long long)min(t1, first) * p.E, b0 = (long long)max(t0, end) * p.E, b1 = (long long)t1 * p.E;
    for (long long i = (long long)t0 * p.E + threadIdx.x; i < a1; i += kBalThreads) p.dscores[i] = 0.f;
    for (long long i = b0 + threadIdx.x; i < b1; i += kBalThreads) p.dscores[i] = 0.f;
  }
  for (int q = max(sq.at(t0), 0); q < sq.S; q = sq.next(q)) {
    const int b = sq.begin(q), e = sq.begin(q + 1);
    if (b >= t1) break;
    if (max(b, t0) >= min(e, t1)) continue;
    const long long kn = (long long)p.k * (e - b);
    const float per = 1.f / (float)kn, wq = p.coef / ((float)sq.filled * (float)(e - b));
    __syncthreads();  // the sequence before is done with f
    for (int i = threadIdx.x; i < p.E; i += kBalThreads) {
      const long long c = (long long)p.counts[(long long)q * p.E + i] * p.E;
      f[i] = (float)(c - kn) * per;
      f[kBalMaxE + i] = (float)c * per;
    }
    __syncthreads();
    acc += wq * bal_rows<NJ, VEC, R, LANES>(p, max(b, t0), min(e, t1), f, wq, nan);
  }
  if (__any_sync(0xffffffffu, nan) && lane == 0) set_status(p.status, LMOE_STATUS_NAN_SCORE);
#pragma unroll
  for (int off = 16; off; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (lane == 0) wsum[warp] = acc;
  __syncthreads();
  double sum = 0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kBalThreads / 32; ++w) sum += wsum[w];
  return sum;
}

// Counts of the second form: a block counts a run of tokens, sequence by sequence.
__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(const BalanceParams p) {
  __shared__ int hist[kBalHistInts];
  __shared__ BalSeqSmem seqs;
  pdl_wait();
  pdl_trigger();
  const BalSeqs sq = bal_seqs(p, seqs);
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
  const int copies = bal_copies(p.E);
  for (int q = max(sq.at(t0), 0); q < sq.S; q = sq.next(q)) {
    const int b = sq.begin(q), lo = max(t0, b), hi = min(t1, sq.begin(q + 1));
    if (b >= t1) break;
    if (lo >= hi) continue;
    for (int i = threadIdx.x; i < p.E * copies; i += kBalThreads) hist[i] = 0;
    __syncthreads();
    bal_count(p, lo, hi, hist, copies);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kBalThreads) {
      int c = 0;
      for (int i = 0; i < copies; ++i) c += hist[e * copies + ((i + e) & (copies - 1))];
      if (c) atomicAdd(&p.counts[(long long)q * p.E + e], c);
    }
    __syncthreads();
  }
}

// The pass of the second form.
template <int NJ, int VEC, int R, int LANES>
__global__ void __launch_bounds__(kBalThreads, 2) balance_kernel(const BalanceParams p) {
  __shared__ __align__(16) float f[2 * kBalMaxE];
  __shared__ double wsum[kBalThreads / 32];
  __shared__ BalSeqSmem seqs;
  __shared__ bool last;
  pdl_wait();
  pdl_trigger();
  const BalSeqs sq = bal_seqs(p, seqs);
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  const double sum = bal_pass<NJ, VEC, R, LANES>(p, sq, t0, t1, f, wsum);
  // the blocks' sums are added in their order by the last block to finish
  if (threadIdx.x == 0) {
    p.partial[blockIdx.x] = sum;
    __threadfence();
    last = atomicAdd(p.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (last && threadIdx.x < 32) {
    __threadfence();
    double b = 0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += 32) b += reinterpret_cast<volatile double*>(p.partial)[i];
#pragma unroll
    for (int off = 16; off; off >>= 1) b += __shfl_xor_sync(0xffffffffu, b, off);
    if (threadIdx.x == 0) *p.loss = (float)b;
  }
}

// The first form: one cluster, S E at most kBalHistInts.
__device__ __forceinline__ int ld_cluster_int(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)));
  return v;
}
__device__ __forceinline__ double ld_cluster_double(const double* p, uint32_t rank) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(mapa_shared(smem_u32(p), rank)));
  return v;
}
template <int NJ, int VEC, int R, int LANES>
__global__ void __launch_bounds__(kBalThreads, 1) balance_cluster_kernel(const BalanceParams p) {
  __shared__ int hist[kBalHistInts];
  __shared__ __align__(16) float f[2 * kBalMaxE];
  __shared__ double wsum[kBalThreads / 32], total;
  __shared__ BalSeqSmem seqs;
  pdl_wait();
  pdl_trigger();
  const int n = p.S * p.E, copies = bal_copies(n), ctas = gridDim.x, rank = blockIdx.x;
  for (int i = threadIdx.x; i < n * copies; i += kBalThreads) hist[i] = 0;
  const BalSeqs sq = bal_seqs(p, seqs);  // ends with a barrier
  const int t0 = min(p.T, rank * p.chunk), t1 = min(p.T, t0 + p.chunk);
  if (t0 < t1)
    for (int q = max(sq.at(t0), 0); q < sq.S; q = sq.next(q)) {
      const int b = sq.begin(q), lo = max(t0, b), hi = min(t1, sq.begin(q + 1));
      if (b >= t1) break;
      if (lo < hi) bal_count(p, lo, hi, hist + q * p.E * copies, copies);
    }
  __syncthreads();
  // each counter's copies into the first
  if (copies > 1) {
    for (int i = threadIdx.x; i < n; i += kBalThreads) {
      int c = 0;
      for (int j = 0; j < copies; ++j) c += hist[i * copies + ((j + i) & (copies - 1))];
      hist[i * copies] = c;
    }
  }
  __syncthreads();
  cluster_sync_all();
  for (int i = rank * kBalThreads + threadIdx.x; i < n; i += ctas * kBalThreads) {
    int c[kBalMaxCluster];
#pragma unroll
    for (int r = 0; r < kBalMaxCluster; ++r) c[r] = r < ctas ? ld_cluster_int(&hist[i * copies], r) : 0;
    int sum = 0;
#pragma unroll
    for (int r = 0; r < kBalMaxCluster; ++r) sum += c[r];
    p.counts[i] = sum;
  }
  __syncthreads();
  cluster_sync_all();  // every CTA sees the counts
  const double sum = bal_pass<NJ, VEC, R, LANES>(p, sq, t0, t1, f, wsum);
  if (threadIdx.x == 0) total = sum;
  __syncthreads();
  cluster_sync_all();
  if (rank == 0 && threadIdx.x == 0) {
    double b = 0;
    for (int r = 0; r < ctas; ++r) b += ld_cluster_double(&total, r);
    *p.loss = (float)b;
  }
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its sum is being read
}

}  // namespace lmoe
