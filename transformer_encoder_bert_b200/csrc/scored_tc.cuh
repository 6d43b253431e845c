// What the tensor-core kernels of attention with modified scores share: tensor
// maps, descriptors, and the arithmetic of a row of scores.
#pragma once

#include <type_traits>

#include "scored.cuh"
#include "sm100.cuh"

namespace enc {
namespace scored_tc {

using namespace sm100;

constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Head-split operands [*, S, d] as {d, S, planes} and merged ones [B, S, H] as
// {H, S, B}; boxes of 64 columns (128 bytes, 128-byte swizzle).  A box over
// heads of 32 is wider than the tensor (head-split: zeros) or reaches into the
// next head (merged): only its first 32 columns are used.
bool encode_operand_map(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t planes,
                        uint32_t box_cols, uint32_t box_rows);

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Contiguous bytes (a multiple of 16, both addresses 16-byte aligned), counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// MN-major operand, 128-byte swizzle: rows of 64 MN elements, K rows in groups
// of 8 that are 1 KB apart; the second group of 64 MN elements `mn_bytes` on.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t mn_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(mn_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// A descriptor `bytes` further on (a multiple of 16; the address field does not overflow within shared memory).  An
// MMA's address costs the issuing thread one addition this way, where forming each descriptor anew took longer than
// the MMA itself.
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
__host__ __device__ constexpr uint32_t idesc_bmn(int m, int n) { return idesc_f16_f32(m, n) | (1u << 16); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Bounded waits: by every lane of a warp (no divergence, no broadcast; true in all lanes or in none), and by a
// single thread.  A waiting thread sleeps up to kSleepNs at a time, so that it leaves its issue slots to others.
constexpr uint32_t kSleepNs = 20000;
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  bool got = mbar_try_wait<kSleepNs>(bar, parity);
  if (!__all_sync(0xffffffffu, got)) got = mbar_wait<kSleepNs>(bar, parity, kWaitLimitNs);
  return __all_sync(0xffffffffu, got);
}
__device__ __forceinline__ bool one_wait(uint32_t bar, uint32_t parity) {
  return mbar_wait<kSleepNs>(bar, parity, kWaitLimitNs);
}
// One lane of the warp.  The warps that issue MMAs and TMA loads run their loops with all lanes and elect a lane for
// the instructions alone: descriptors and addresses are then the same in every lane and stay in uniform registers,
// where a loop run by one lane has to move each operand there first (measured: 60 to 90 cycles an MMA).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 r;\n\t"
      "elect.sync r|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool any_warp(bool p) { return __any_sync(0xffffffffu, p); }

// Distance bias of a 128-row tile of positions against a block of positions.
// The bias is a function of the distance alone, and past +-reach it is a
// constant plus the slope's linear part.  A block that lies past the reach on
// one side adds `base + step * column`; the others read a table in shared
// memory that holds the bias of every distance within reach of such a block
// (score_bias2 at index distance + off), neighbouring lanes at neighbouring
// addresses.
struct Bias {
  const float* lut;     // shared memory
  int off;              // index of distance 0
  int reach;            // s.reach with a table, else 0
  float slope2;         // slopes[h] log2 e
  float right, left;    // table bias of far keys on either side, in log2 units
};

// The LUT spans distances that blocks within reach can hold: 128 rows against `block` columns.
__host__ __device__ constexpr int lut_half(int reach, int block) { return reach + 128 + block; }
__host__ __device__ inline int lut_floats(const ScoreArgs& s, int block) {
  return s.table || s.slopes ? (2 * lut_half(s.table ? s.reach : 0, block) + 1 + 3) / 4 * 4 : 0;
}

// Called by `threads` threads (t = 0 ..) that share named barrier 1.  Distances outside [rel_min, rel_max] are not
// filled: no visible key is read there.
__device__ __forceinline__ Bias make_bias(const ScoreArgs& s, float* column, float* lut, int nh, int h, int block,
                                          int rel_min, int rel_max, int t, int threads) {
  Bias b;
  b.lut = lut;
  b.reach = s.table ? s.reach : 0;
  b.off = lut_half(b.reach, block);
  const float slope = s.slopes ? s.slopes[h] : 0.f;
  b.slope2 = slope * kLog2e;
  b.right = b.left = 0.f;
  if (s.table) {
    load_column(s, column, nh, h, t, threads);
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
    b.right = column[score_bucket(s, s.reach)] * kLog2e;
    b.left = column[score_bucket(s, -s.reach)] * kLog2e;
  }
  if (s.table || s.slopes) {
    const int last = min(2 * b.off, rel_max + b.off);
    for (int k = max(0, rel_min + b.off) + t; k <= last; k += threads)
      lut[k] = score_bias2(s, column, slope, k - b.off);
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
  }
  return b;
}

// The cap, t2 = cap2 tanh(x) with x = s * in = u / cap.  1 - 2 / (1 + 2^(2 x log2 e)) costs two special-function
// operations a score (a quarter of the FMA rate each, besides the softmax's own).  Where every |x| of a warp's block is
// at most kCapPoly, a polynomial x P(x^2) of degree 8 in x^2 does it on the FMA pipe, and where every one is at most
// kTanhSmall, one of degree 4 with in and cap2 taken into its coefficients (s.cap_small), 6 operations a score where the
// other costs 12.  Both are least-maximum fits of the relative error, found by reweighted least squares: 1.9e-8 and
// 2.9e-8, with FP32 rounding 1.1e-7 and 1e-7 (fits of the absolute error take a term less, but are off by 2e-6 of a
// small score, which the table's gradient shows).  In the other blocks a score is off by about 2^-22 of the cap however
// small it is.  Up to a cap of 64 that is a thirtieth of what rounding P to FP16 does to it; larger caps have kernels of
// their own, in which scores up to kTanhSmall take the short polynomial there too (8 heads of 128, 8 sequences of 2048, a
// cap of 8, where most blocks hold a larger score: 412 us, and 534 with that).
constexpr float kCapPoly = 1.25f, kCapCoarse = 64.f;
struct Cap {
  float in, cap2;
  float neg_inv2;           // -1 / cap2^2: 1 - tanh^2 of a capped score
  bool on;
};
__device__ __forceinline__ Cap make_cap(const ScoreArgs& s) {
  Cap c;
  c.on = s.cap > 0.f;
  c.in = c.on ? s.scale / s.cap : 0.f;
  c.cap2 = s.cap * kLog2e;
  c.neg_inv2 = c.on ? -1.f / (c.cap2 * c.cap2) : 0.f;
  return c;
}
// tanh(x) / x of two scores from x^2, |x| <= kCapPoly.
__device__ __forceinline__ uint64_t tanh_over_x2(uint64_t z) {
  constexpr float c[9] = {1.f,
                          -0.33333247900009155f,
                          0.13331784307956696f,
                          -0.053858835250139236f,
                          0.021475467830896378f,
                          -0.00804087147116661f,
                          0.002523908857256174f,
                          -0.0005492825293913484f,
                          5.841381425852887e-05f};
  uint64_t p = f2_pack(c[8], c[8]);
#pragma unroll
  for (int k = 7; k >= 0; --k) p = f2_fma(p, z, f2_pack(c[k], c[k]));
  return p;
}
// t2 of two scores by s.cap_small.
__device__ __forceinline__ uint64_t small_cap2(const ScoreArgs& s, uint64_t x) {
  const uint64_t z = f2_mul(x, x);
  uint64_t p = f2_pack(s.cap_small[4], s.cap_small[4]);
#pragma unroll
  for (int k = 3; k >= 0; --k) p = f2_fma(p, z, f2_pack(s.cap_small[k], s.cap_small[k]));
  return f2_mul(x, p);
}
// The backward's P, at most 1, is rounded to FP16 for dV = P^T dO as P 2^13: otherwise a weight below 2^-14 would lose
// digits, and one below 2^-25 would be nothing, which is all that a key gets that is seldom attended to.  The statistics
// hold 13 - lse2, dU's scale takes the factor back, and dV's output does; the three bits left allow for a P above 1 by
// the rounding of large scores.
constexpr int kPBits = 13;
constexpr float kPScale = 1 << kPBits, kPInverse = 1.f / kPScale;

// What the forward adds to t2 before the exponential: `raise` less the row's reference.  References past 2^17 do not
// take the raise, which their rounding could multiply beyond FP16's range.
__device__ __forceinline__ float raised(float raise, float reference) {
  return fabsf(reference) < 131072.f ? raise - reference : -reference;
}

// What a kernel does about the cap (its template argument).
constexpr int kNoCap = 0, kCap = 1, kLargeCap = 2;
inline int cap_kind(const ScoreArgs& s) { return s.cap > kCapCoarse ? kLargeCap : s.cap > 0.f ? kCap : kNoCap; }
template <typename F>
cudaError_t with_cap(const ScoreArgs& s, F f) {            // f(integral constant)
  switch (cap_kind(s)) {
    case kNoCap: return f(std::integral_constant<int, kNoCap>());
    case kCap: return f(std::integral_constant<int, kCap>());
  }
  return f(std::integral_constant<int, kLargeCap>());
}
// The forms of the cap; any: also when there is none.
constexpr int kAny = 0, kPoly = 1, kSmall = 2, kCareful = 3;
// tanh(s in) of any size; in2 = 2 in log2 e.
__device__ __forceinline__ float tanh_of(float s, float in2) { return fmaf(-2.f, rcp(1.f + ex2(s * in2)), 1.f); }
// The same of two scores, with the polynomial for those up to kTanhSmall.
__device__ __forceinline__ uint64_t tanh_careful2(uint64_t s, float in) {
  constexpr TanhSmall fit;
  const uint64_t x = f2_mul(s, f2_pack(in, in)), z = f2_mul(x, x);
  uint64_t p = f2_pack(fit.c[4], fit.c[4]);
#pragma unroll
  for (int k = 3; k >= 0; --k) p = f2_fma(p, z, f2_pack(fit.c[k], fit.c[k]));
  float x0, x1, p0, p1;
  f2_unpack(x, x0, x1);
  f2_unpack(f2_mul(x, p), p0, p1);
  return f2_pack(fabsf(x0) <= kTanhSmall ? p0 : tanh_of(x0, 2.f * kLog2e),
                 fabsf(x1) <= kTanhSmall ? p1 : tanh_of(x1, 2.f * kLog2e));
}

// The gradient's: tanh and 1 - tanh^2 of two scores times in, of any size.  From E = 2^(-2 |x| log2 e), r = 1 / (1 + E):
// tanh |x| = 1 - 2 E r and 1 - tanh^2 = 4 E r^2, which keeps its precision where tanh is near 1 (1 - tanh^2 from tanh
// itself is off by 2^-23, a hundredth of it at x = 6).
template <bool CAREFUL>
__device__ __forceinline__ uint64_t tanh_slope2(uint64_t s, float in, uint64_t& slope) {
  const uint64_t x = f2_mul(s, f2_pack(in, in));
  float x0, x1;
  f2_unpack(x, x0, x1);
  const float e0 = ex2(fabsf(x0) * (-2.f * kLog2e)), e1 = ex2(fabsf(x1) * (-2.f * kLog2e));
  const uint64_t r = f2_pack(rcp(1.f + e0), rcp(1.f + e1)), er = f2_mul(f2_pack(e0, e1), r);
  slope = f2_mul(er, f2_mul(r, f2_pack(4.f, 4.f)));
  float t0, t1;
  f2_unpack(f2_fma(er, f2_pack(-2.f, -2.f), f2_pack(1.f, 1.f)), t0, t1);
  t0 = copysignf(t0, x0);
  t1 = copysignf(t1, x1);
  if (CAREFUL) {
    constexpr TanhSmall fit;
    const uint64_t z = f2_mul(x, x);
    uint64_t p = f2_pack(fit.c[4], fit.c[4]);
#pragma unroll
    for (int k = 3; k >= 0; --k) p = f2_fma(p, z, f2_pack(fit.c[k], fit.c[k]));
    float p0, p1;
    f2_unpack(f2_mul(x, p), p0, p1);
    t0 = fabsf(x0) <= kTanhSmall ? p0 : t0;
    t1 = fabsf(x1) <= kTanhSmall ? p1 : t1;
  }
  return f2_pack(t0, t1);
}

// (Two predicated additions; a choice of addends costs two more instructions a score.)
__device__ __forceinline__ void add_either(bool first, float v, float& a, float& b) {
  asm("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\t@p add.f32 %0, %0, %3;\n\t@!p add.f32 %1, %1, %3;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"((int)first), "f"(v));
}

// Adds 32 lanes' values to the warp's bucket sums.  The lanes' distances are consecutive (up or down), so a
// bucket's lanes are neighbours: a segmented scan, then the last lane of each run adds.
__device__ __forceinline__ void add_by_bucket(float v, int bucket, float* sums, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float w = __shfl_up_sync(0xffffffffu, v, off);
    const int bk = __shfl_up_sync(0xffffffffu, bucket, off);
    if (lane >= off && bk == bucket) v += w;
  }
  const int after = __shfl_down_sync(0xffffffffu, bucket, 1);
  if (lane == 31 || after != bucket) sums[bucket] += v;
  __syncwarp();
}

}  // namespace scored_tc
}  // namespace enc
