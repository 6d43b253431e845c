// Attention with modified scores: what its kernels share.
//
// For query position i and key position j of one sequence (n valid positions)
// and head h, with s = q_i . k_j:
//   u = scale * s;  with a cap: u = cap * tanh(u / cap)
//   t = u - slopes[h] * |j - i| + table[bucket(j - i)][h]
//   j is visible to i where i, j < n, where a causal mask has j <= i or
//   j < prefix, and where doc[i] == doc[j].
// The causal, prefix and length masks leave each query the keys [0, jlim_i):
// jlim_i = min(n, max(i + 1, prefix)) (n without the causal mask); and each key
// the queries [ilow_j, n): ilow_j = j where the causal mask holds and
// j >= prefix, else 0.  The kernels work on t in units of log2 (t2 = t log2 e),
// so that exp is one ex2.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace enc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// tanh(x) / x on |x| <= kTanhSmall in powers of x^2: a least-maximum fit of the relative error, found by reweighted least
// squares (2.9e-8; the form 1 - 2 / (1 + 2^(2 x log2 e)) is off by 2^-22 or so however small x is).
constexpr float kTanhSmall = 0.5f;
struct TanhSmall {
  float c[5] = {1.f, -0.33333075046539307f, 0.13324907422065735f, -0.0529942512512207f, 0.017151331529021263f};
};

// Bucket of the relative position rel = key - query.
__host__ __device__ __forceinline__ int score_bucket(const ScoreArgs& s, int rel) {
  const int nb = s.both ? s.buckets >> 1 : s.buckets;
  const int a = s.both ? (rel < 0 ? -rel : rel) : (rel < 0 ? -rel : 0);
  const int exact = nb >> 1;
  int c = a;
  if (a >= exact) {
    c = nb - 1;                             // from the last bound on
    if (a < s.reach) {
      c = exact;                            // and how many bounds are <= a (the same ones for every lane)
#pragma unroll 8
      for (int k = 0; k < s.num_bounds; ++k) c += s.bounds[k] <= a;
    }
  }
  return c + (s.both && rel > 0 ? nb : 0);
}

// The relative positions [lo, hi] of bucket c, within +-reach (empty where lo > hi).
__device__ __forceinline__ void bucket_range(const ScoreArgs& s, int c, int& lo, int& hi) {
  const int nb = s.both ? s.buckets >> 1 : s.buckets, exact = nb >> 1;
  const bool ahead = s.both && c >= nb;                    // positive relative positions
  const int cc = ahead ? c - nb : c;
  const int a0 = cc < exact ? cc : cc == exact ? exact : s.bounds[cc - exact - 1];
  const int a1 = cc < exact ? cc : cc == nb - 1 ? s.reach : s.bounds[cc - exact] - 1;
  lo = ahead ? max(a0, 1) : -a1;
  hi = ahead ? a1 : -a0;
  if (!s.both && cc == 0) hi = s.reach;                    // one direction: every key ahead
}

// The part of t2 that depends on the distance alone; column: the head's column of the table.
__device__ __forceinline__ float score_bias2(const ScoreArgs& s, const float* column, float slope, int rel) {
  float b = -slope * fabsf(static_cast<float>(rel));
  if (s.table) b += column[score_bucket(s, rel)];
  return b * kLog2e;
}
// Copies the head's column of the table to shared memory; a barrier must follow.
__device__ __forceinline__ void load_column(const ScoreArgs& s, float* column, int nh, int h, int t, int threads) {
  if (s.table)
    for (int c = t; c < s.buckets; c += threads) column[c] = s.table[static_cast<size_t>(c) * nh + h];
}

__device__ __forceinline__ int score_len(const int32_t* valid_len, int b, int S) {
  const int n = valid_len[b];
  return n < 0 ? 0 : (n > S ? S : n);
}

__device__ __forceinline__ int score_prefix(const ScoreArgs& s, int b) { return s.prefix ? s.prefix[b] : 0; }

// First key that query i does not see for its position, and first query that
// sees key j.
__device__ __forceinline__ int score_jlim(const ScoreArgs& s, int i, int n, int prefix) {
  return s.causal ? min(n, max(i + 1, prefix)) : n;
}
__device__ __forceinline__ int score_ilow(const ScoreArgs& s, int j, int prefix) {
  return s.causal && j >= prefix ? j : 0;
}

// A grid that starts before the one ahead of it has ended (dK/dV beside dQ) reads what a still earlier grid wrote (the
// row statistics).  Its own griddepcontrol.wait would make that visible, but would also wait for the whole dQ grid.  So
// every dQ block, once past its wait, adds one to a counter with release order before it lets the next grid start, and
// a dK/dV block that acquires the full count sees all that the dQ blocks saw.  One that does not (no block has to wait
// for another one here) takes its griddepcontrol.wait at its start instead of its end.  The statistics grid, which
// starts after every earlier reader has ended, sets the counter to zero.
__device__ __forceinline__ void count_block(unsigned* counter) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
}
// Called by every thread of a block; a barrier.  The bulk copies that follow read through the asynchronous proxy.
__device__ __forceinline__ bool all_blocks_counted(const unsigned* counter, unsigned blocks) {
  unsigned v = 0;
  if (threadIdx.x == 0) asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
  const bool all = __syncthreads_or(threadIdx.x == 0 && v == blocks);
  asm volatile("fence.proxy.async;" ::: "memory");
  return all;
}

// Persistent CTAs over `items`: CTA c of `ctas` takes [first_item(c), first_item(c + 1)).
__host__ __device__ __forceinline__ int first_item(int c, int items, int ctas) {
  return static_cast<int>(static_cast<long long>(items) * c / ctas);
}
__host__ __device__ __forceinline__ int cta_of_item(int item, int items, int ctas) {
  return static_cast<int>((static_cast<long long>(item + 1) * ctas - 1) / items);
}

}  // namespace enc
