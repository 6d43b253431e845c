// Backward of attention with modified scores on the 5th-generation tensor
// cores, FP16: one kernel in two modes.
//
// With dT = P (dP - D), dP = dO V^T, D_i = dO_i . O_i, dU = dT (1 - tanh^2):
//   dQ mode   rows = 128 queries, blocks of 64 keys:  dQ += dU K
//   dKV mode  rows = 128 keys, blocks of 64 queries:  dV += P^T dO, dK += dU^T Q
// Either mode keeps two operands of its rows in shared memory (Q and dO, or K
// and V) and streams the two of the columns, and both form the same two score
// tiles with the rows in TMEM lanes, so one thread owns one row:
//   S  = A0 B0^T, dP = A1 B1^T        M = 128, N = 64, K = D, shared memory
//   acc0 += dU B0, (dKV) acc1 += P B1   M = 128, N = D, K = 64, dU and P in TMEM
// S and dP are computed twice (once a mode) instead of adding dQ up with
// atomics from the dKV mode: 7 products instead of 5, but no FP32 traffic of dQ
// through memory and the same result on every run.
//
// Warps: two warpgroups of threads that own rows, one MMA warp, one TMA warp.
// Heads up to 64 run two CTAs per SM (256 TMEM columns each), so that one CTA's
// exponentials run under the other's products, and the warpgroups share a
// block's columns: its scores are the chain that the products wait for, and half
// the columns to a thread shorten it.  Heads of 128 fill the TMEM with one CTA:
// its warpgroups take the blocks in turn, each with S and dP columns of its own.
//
// P and dU are rounded to FP16 for the products, P as P 2^13 (kPBits).  dU is scaled
// by a power of two e per (sequence, head): |dT| <= 2 max|dO_i| max|v_j|, and e
// puts that product of norms between 2^13 and 2^14, so that no dU leaves FP16's
// range and small gradients keep their bits.  e is exact and is taken out of
// the FP32 results.
//
// The table's gradient (dQ mode) is the sum of dT over every diagonal of equal
// distance, then over a bucket's distances.  A warp owns 32 rows: with one
// shuffle a column the 32 values of a column go to 32 lanes by diagonal (see
// row_chunk), each of which adds up the diagonals of its number in a fixed order;
// a block whose distances all share a bucket only adds its values up.
//
// Measured, full lengths, counted as five products: 8 heads of 128, 37 sequences
// of 2048: 2.69 ms, 592 TF/s (829 as the seven that run; table 2.79, cap 3.02
// ms); 16 heads of 64, 37 of 1024: 1.13 ms, 351 TF/s (table 1.27, cap 1.40 ms).
// What bounds a block is the chain S and dP -> a row's arithmetic -> the products
// -> the next S and dP in the same columns.  In dKV mode TMEM holds no third pair of
// buffers beside the accumulators; in dQ mode a quarter of it and more is free, but dU
// lies over dP there too, so the next scores wait for the product.
#include "scored_tc.cuh"

namespace enc {
namespace scored_tc {
namespace {

constexpr int kBN = 64;                        // columns of a block
constexpr int kDQ = 0, kDKV = 1;

template <int D, int MODE>
struct BCfg {
  static constexpr int NB = D > 64 ? 2 : 1;                // S and dP buffers
  static constexpr int kShare = 2 / NB;                    // warpgroups that share a block
  static constexpr int kRowWarps = 8, kRowThreads = 256, kThreads = kRowThreads + 64;
  static constexpr int kChunk = D > 64 ? 32 : 16;          // columns in registers at a time (168 or 96 registers)
  static constexpr int kSub = D > 64 ? D / 64 : 1;
  static constexpr int kABytes = kSub * 128 * 128;         // one operand of the rows
  static constexpr int kBSub = kBN * 128;
  static constexpr int kBBytes = kSub * kBSub;             // one operand of a block's columns
  static constexpr int kStages = 3;
  static constexpr int kStage = 2 * kBBytes;
  static constexpr int kB = 2 * kABytes;
  static constexpr int kCol = kB + kStages * kStage;       // dKV: kPBits - lse2 and D of a block's queries, per stage
  static constexpr int kColBytes = 2 * kBN * 4;
  static constexpr int kBars = kCol + (MODE == kDKV ? kStages * kColBytes : 0);
  // a_full, drain, b_full, b_empty (kStages each), s_full, p_full, done (NB each)
  static constexpr int kNumBars = 2 + 2 * kStages + 3 * NB;
  static constexpr int kSlot = kBars + kNumBars * 8;
  static constexpr int kSums = (kSlot + 16 + 15) / 16 * 16;   // dQ: per row warp, bucket sums
  static constexpr int kColumn = kSums + (MODE == kDQ ? kRowWarps * kMaxScoreBuckets * 4 : 0);   // of the bias table
  static constexpr int kLut = kColumn + kMaxScoreBuckets * 4;
  static constexpr int kS = 0, kDP = NB * kBN, kAcc = 2 * NB * kBN;
  static constexpr int kTmemUsed = kAcc + (MODE == kDKV ? 2 : 1) * D;
  static constexpr int kTmemCols = kTmemUsed <= 256 ? 256 : 512;
  static size_t smem(const ScoreArgs& s, int seq, bool table) {
    return 1024 + kLut + (size_t)lut_floats(s, kBN) * 4 + (table ? (size_t)(2 * s.reach + 1) : 0) +
           (s.docs ? (size_t)(seq + kBN - 1) / kBN : 0);
  }
};

// One row's block of 64 columns, 32 at a time: from S and dP to P and dU.
struct RowBlock {
  uint32_t t_s, t_dp;       // TMEM addresses of the row warp's S and dP columns
  float base, step;         // bias (plus kPBits - lse2 in dQ mode): base, base + step * column, or base + lut
  const float* lut;         // at column 0
  uint32_t see[2];          // bits: visible columns
  float e, de;              // what dT's dP - D is scaled by (dU's scale over P's), and D times that (dQ mode)
  const float* col;         // dKV mode: kPBits - lse2 [64], D [64] of the columns (shared memory)
  int valid;                // columns that are valid positions (any number)
  bool mine;                // the row is one
  int p_at;                 // P and dU of column c go to column p_at + c / 2 (of S, of dP)
};

// CH columns of it from column c, two at a time in packed FP32 arithmetic.  NEAR 0: constant bias; 1: bias from the
// table in shared memory; 2: that, and the diagonals' sums: for column k, lane t takes dT of row (k - t) mod 32, which
// lies on the diagonal whose column less row is t (pos) or t - 32 (neg); else pos += dT.  NEAR 3: linear bias.
// FORM: of the cap.
template <int MODE, int CH, bool CAP, int NEAR, bool MASK, int FORM>
__device__ __forceinline__ void row_chunk(const ScoreArgs& s, const RowBlock& rb, const Cap& cap, float scale2, int lane, int c,
                                          const uint32_t (&sv)[CH], const uint32_t (&dp)[CH], float& pos, float& neg) {
  uint32_t pp[CH / 2], pu[CH / 2];
  const int k0 = c & 31;                                   // column of a 32 x 32 block
  const float* lut = MODE == kDQ ? rb.lut + c : rb.lut - c;
  const float base = NEAR == 3 ? fmaf((float)c, rb.step, rb.base) : rb.base;
  const uint64_t base2 = f2_pack(base, base), e2 = f2_pack(rb.e, rb.e), neg_e2 = f2_pack(-rb.e, -rb.e);
  const uint64_t mul = CAP ? f2_pack(cap.cap2, cap.cap2) : f2_pack(scale2, scale2), one2 = f2_pack(1.f, 1.f);
  const uint64_t row_d2 = f2_pack(-rb.de, -rb.de);
  const uint32_t see = (c < 32 ? rb.see[0] : rb.see[1]) >> (c & 31);
  uint64_t far2 = 0;                                       // two partial sums of dT (0.0f, 0.0f)
#pragma unroll
  for (int k = 0; k < CH; k += 4) {
    ulonglong2 nl = make_ulonglong2(0, 0), dc = make_ulonglong2(0, 0);       // kPBits - lse2 and D of four columns
    if (MODE == kDKV) {
      nl = *reinterpret_cast<const ulonglong2*>(rb.col + c + k);
      dc = *reinterpret_cast<const ulonglong2*>(rb.col + kBN + c + k);
    }
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const int at = k + q;
      uint64_t x = f2_pack(__uint_as_float(sv[at]), __uint_as_float(sv[at + 1]));
      uint64_t slope2 = 0;                                 // 1 - tanh^2
      if constexpr (CAP) {
        if (FORM == kSmall) {
          x = small_cap2(s, x);
        } else if (FORM == kPoly) {
          const uint64_t y = f2_mul(x, f2_pack(cap.in, cap.in));
          x = f2_mul(y, tanh_over_x2(f2_mul(y, y)));
        } else {
          x = tanh_slope2<FORM == kCareful>(x, cap.in, slope2);
        }
      }
      uint64_t add = base2;
      if (NEAR == 3) add = f2_pack(fmaf((float)at, rb.step, base), fmaf((float)(at + 1), rb.step, base));
      if (NEAR == 1 || NEAR == 2) {
        add = MODE == kDQ ? f2_pack(lut[at], lut[at + 1]) : f2_pack(lut[-at], lut[-(at + 1)]);
        if (MODE == kDQ) add = f2_add(add, base2);
      }
      if (MODE == kDKV) add = f2_add(add, q ? nl.y : nl.x);
      float t0, t1;
      f2_unpack(CAP && FORM == kSmall ? f2_add(x, add) : f2_fma(x, mul, add), t0, t1);
      float p0 = ex2(t0), p1 = ex2(t1);
      const uint64_t d2 = MODE == kDKV ? f2_mul(q ? dc.y : dc.x, neg_e2) : row_d2;
      const uint64_t dt2 =
          f2_mul(f2_pack(p0, p1), f2_fma(f2_pack(__uint_as_float(dp[at]), __uint_as_float(dp[at + 1])), e2, d2));
      uint64_t u2 = dt2;
      if constexpr (CAP) {                                 // dU = dT (1 - tanh^2)
        const float f = FORM == kSmall ? cap.neg_inv2 : -1.f;
        if (FORM == kSmall || FORM == kPoly) slope2 = f2_fma(f2_mul(x, f2_pack(f, f)), x, one2);
        u2 = f2_mul(dt2, slope2);
      }
      float u0, u1, a0, a1;
      f2_unpack(u2, u0, u1);
      f2_unpack(dt2, a0, a1);
      if (MASK) {                                          // (hidden scores may be NaN)
        const bool see0 = see & (1u << at), see1 = see & (2u << at);
        p0 = see0 ? p0 : 0.f;
        p1 = see1 ? p1 : 0.f;
        a0 = see0 ? a0 : 0.f;
        a1 = see1 ? a1 : 0.f;
        u0 = see0 ? u0 : 0.f;
        u1 = see1 ? u1 : 0.f;
      }
      if (MODE == kDQ) {
        if (NEAR == 2) {
          add_either(k0 + at >= lane, __shfl_sync(0xffffffffu, a0, k0 + at - lane), pos, neg);
          add_either(k0 + at + 1 >= lane, __shfl_sync(0xffffffffu, a1, k0 + at + 1 - lane), pos, neg);
        } else {
          far2 = f2_add(far2, f2_pack(a0, a1));
        }
      }
      if (MODE == kDKV) pp[at / 2] = half2_of(p0, p1);
      pu[at / 2] = half2_of(u0, u1);
    }
  }
  if (MODE == kDQ && NEAR != 2) {
    float a0, a1;
    f2_unpack(far2, a0, a1);
    pos += a0 + a1;
  }
  // Over columns that this lane has read.
  if constexpr (CH == 32) {
    if constexpr (MODE == kDKV) tmem_st_32x32b_x16_async(rb.t_s + rb.p_at + c / 2, pp);
    tmem_st_32x32b_x16_async(rb.t_dp + rb.p_at + c / 2, pu);
  } else {
    if constexpr (MODE == kDKV) tmem_st_32x32b_x8_async(rb.t_s + rb.p_at + c / 2, pp);
    tmem_st_32x32b_x8_async(rb.t_dp + rb.p_at + c / 2, pu);
  }
}

// Columns [first, last).  sums: NEAR 2: the lane's diagonals, k: columns less rows lane + 32 (k - 1), from the first
// column and the warp's first row; else sums[1] += dT.
template <int MODE, int CH, int CAP, int NEAR, bool MASK>
__device__ __forceinline__ void row_block(const ScoreArgs& s, const RowBlock& rb, int first, int last, const Cap& cap, float scale2,
                                          int lane, float (&sums)[3]) {
  constexpr bool kOn = CAP != kNoCap;
  float pos = 0.f, neg = 0.f;
#pragma unroll 1
  for (int c = first; c < last; c += CH) {
    uint32_t sv[CH], dp[CH];
    if constexpr (CH == 32) {
      tmem_ld_32x32b_x32_async(rb.t_s + c, sv);
      tmem_ld_32x32b_x32_async(rb.t_dp + c, dp);
    } else {
      tmem_ld_32x32b_x16_async(rb.t_s + c, sv);
      tmem_ld_32x32b_x16_async(rb.t_dp + c, dp);
    }
    tmem_wait_ld(sv);
    tmem_wait_ld(dp);
    int form = kAny;
    if constexpr (kOn) {
      float top = 0.f;                                     // (of valid rows and columns, so that no other decides)
      if (MASK && c + CH > rb.valid) {
#pragma unroll
        for (int k = 0; k < CH; ++k) top = fmaxf(top, c + k < rb.valid ? fabsf(__uint_as_float(sv[k])) : 0.f);
      } else {
#pragma unroll
        for (int k = 0; k < CH; k += 2)
          top = fmaxf(fmaxf(top, fabsf(__uint_as_float(sv[k]))), fabsf(__uint_as_float(sv[k + 1])));
      }
      form = !any_warp(rb.mine && top > s.cap_small_top) ? kSmall
             : !any_warp(rb.mine && top * fabsf(cap.in) > kCapPoly) ? kPoly : kAny;
    }
    if (kOn && form == kSmall)
      row_chunk<MODE, CH, kOn, NEAR, MASK, kOn ? kSmall : kAny>(s, rb, cap, scale2, lane, c, sv, dp, pos, neg);
    else if (kOn && form == kPoly)
      row_chunk<MODE, CH, kOn, NEAR, MASK, kOn ? kPoly : kAny>(s, rb, cap, scale2, lane, c, sv, dp, pos, neg);
    else
      row_chunk<MODE, CH, kOn, NEAR, MASK, CAP == kLargeCap ? kCareful : kAny>(s, rb, cap, scale2, lane, c, sv, dp, pos, neg);
    if (NEAR == 2 && c + CH == first + 32) {
      sums[0] = neg;
      neg = pos;                                           // the first 32 columns' lane is the next ones' lane - 32
      pos = 0.f;
    }
  }
  if (NEAR == 2) {
    sums[1] = neg;
    sums[2] = pos;
  } else {
    sums[1] += pos;
  }
}

// Columns [first, last) of a warp none of whose rows sees them: P = dU = 0, nothing to sum.
template <int MODE>
__device__ __forceinline__ void hidden_rows(const RowBlock& rb, int first, int last) {
  uint32_t zero[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) zero[k] = 0;
  for (int c = first; c < last; c += 32) {
    if constexpr (MODE == kDKV) tmem_st_32x32b_x16_async(rb.t_s + rb.p_at + c / 2, zero);
    tmem_st_32x32b_x16_async(rb.t_dp + rb.p_at + c / 2, zero);
  }
}

template <int MODE, int CH, int CAP, int NEAR>
__device__ __forceinline__ void row_block_m(const ScoreArgs& s, bool mask, const RowBlock& rb, int first, int last, const Cap& cap,
                                            float scale2, int lane, float (&sums)[3]) {
  if (mask)
    row_block<MODE, CH, CAP, NEAR, true>(s, rb, first, last, cap, scale2, lane, sums);
  else
    row_block<MODE, CH, CAP, NEAR, false>(s, rb, first, last, cap, scale2, lane, sums);
}

// LARGE: for caps above kCapCoarse.
template <int D, int MODE, bool LARGE>
__global__ void __launch_bounds__(BCfg<D, MODE>::kThreads, D > 64 ? 1 : 2)
    scored_tc_bwd_kernel(const __grid_constant__ ScoreArgs s, const __grid_constant__ CUtensorMap tm_a0,
                         const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b0,
                         const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ CUtensorMap tm_out,
                         const int32_t* valid_len, const float* rows2, int Sp, const float* norms, unsigned* counter,
                         float* partial, __half* dqkv, int B, int S, int NH, int* status) {
  // (Pointers without __restrict__: no load may go through the read-only path, or move above the acquire.)
  using C = BCfg<D, MODE>;
  constexpr int kCapped = LARGE ? kLargeCap : kCap;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBars;
  const uint32_t a_full = bar0, drain = bar0 + 8;
  auto b_full = [&](int st) { return bar0 + 16 + 8 * st; };
  auto b_empty = [&](int st) { return bar0 + 16 + 8 * (C::kStages + st); };
  const uint32_t buf_bars = bar0 + 16 + 16 * C::kStages;
  auto s_full = [&](int w) { return buf_bars + 8 * w; };
  auto p_full = [&](int w) { return buf_bars + 8 * (C::NB + w); };
  auto done = [&](int w) { return buf_bars + 8 * (2 * C::NB + w); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kSlot);
  float* column = reinterpret_cast<float*>(smem + C::kColumn);
  float* lut = reinterpret_cast<float*>(smem + C::kLut);
  uint8_t* bucket_of = reinterpret_cast<uint8_t*>(lut + lut_floats(s, kBN));   // by distance + reach
  uint8_t* cls = bucket_of + (partial ? 2 * s.reach + 1 : 0);   // documents: 0 skip, 1 whole, 2 mask per element

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int blk = MODE == kDQ ? gridDim.x - 1 - blockIdx.x : blockIdx.x;    // long causal rows first
  const int r0 = blk * 128;
  const size_t bh = (size_t)b * NH + h;
  const int planes = B * NH;
  // The dKV grid needs nothing of the dQ grid before it (all_blocks_counted has how it sees what both read).  So its
  // blocks fill the SMs that the dQ grid's last ones leave idle, and wait for the end of that grid at their own end, so
  // that what follows finds both complete (8 heads of 128, 4093 tokens, causal: 222 -> 200 us; 8 sequences of 512 and
  // 16 heads of 64: 80 -> 71 us).
  if (MODE == kDQ) {
    pdl_wait();
    if (tid == 0) count_block(counter);
  } else if (!all_blocks_counted(counter, gridDim.x * gridDim.y * gridDim.z)) {
    pdl_wait();
  }
  const int n = score_len(valid_len, b, S), prefix = score_prefix(s, b);
  if (r0 >= n) {                                           // padding: zero gradients
    const int rows = min(128, S - r0);
    for (int part = MODE == kDQ ? 0 : 1; part < (MODE == kDQ ? 1 : 3); ++part)
      for (int k = tid; k < rows * (D / 8); k += C::kThreads)
        *reinterpret_cast<uint4*>(dqkv + (((size_t)part * planes + bh) * S + r0) * D + (size_t)k * 8) =
            make_uint4(0, 0, 0, 0);
    if (MODE == kDQ && partial)
      for (int k = tid; k < s.buckets; k += C::kThreads) partial[(bh * gridDim.x + blk) * s.buckets + k] = 0.f;
    if (MODE == kDKV) pdl_wait();
    return;
  }
  // Blocks of columns that some row sees, as far as length and causality go.
  const int r_last = min(r0 + 127, n - 1);
  const int jb0 = MODE == kDQ ? 0 : score_ilow(s, r0, prefix) / kBN;
  const int jb1 = ((MODE == kDQ ? score_jlim(s, r_last, n, prefix) : n) + kBN - 1) / kBN;

  if (tid == 0) {
    for (int k = 0; k < C::kNumBars; ++k) mbar_init(bar0 + 8 * k, 1);
    for (int w = 0; w < C::NB; ++w) mbar_init(p_full(w), 4 * C::kShare);
    fence_barrier_init();
  }
  if (warp == C::kRowWarps) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  const int32_t* docs = s.docs ? s.docs + (size_t)b * S : nullptr;
  if (docs) {
    int rlo = INT32_MAX, rhi = INT32_MIN;
    for (int k = r0 + lane; k <= r_last; k += 32) {
      const int v = docs[k];
      rlo = min(rlo, v);
      rhi = max(rhi, v);
    }
    rlo = __reduce_min_sync(0xffffffffu, rlo);
    rhi = __reduce_max_sync(0xffffffffu, rhi);
    for (int jb = jb0 + warp; jb < jb1; jb += C::kThreads / 32) {
      int lo = INT32_MAX, hi = INT32_MIN;
#pragma unroll
      for (int c = 0; c < kBN; c += 32) {
        const int j = jb * kBN + c + lane;
        if (j < n) {
          const int v = docs[j];
          lo = min(lo, v);
          hi = max(hi, v);
        }
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (lane == 0) cls[jb] = hi < rlo || lo > rhi ? 0 : (lo == hi && rlo == rhi ? 1 : 2);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  pdl_trigger();                                           // after taking TMEM
  auto next_block = [&](int jb) {
    if (docs)
      while (jb < jb1 && cls[jb] == 0) ++jb;
    return jb;
  };

  bool ok = true;
  if (warp == C::kRowWarps + 1) {
    if (lane == 0) {                                       // TMA
      const int a0 = MODE == kDQ ? (int)bh : planes + (int)bh;               // plane of Q or K
      const int b0 = MODE == kDQ ? planes + (int)bh : (int)bh;               // plane of K or Q
      mbar_arrive_expect_tx(a_full, 2 * C::kABytes);
      for (int u = 0; u < C::kSub; ++u) {
        tma_load_3d(&tm_a0, sbase + u * 16384, a_full, 64 * u, r0, a0);
        if (MODE == kDQ)
          tma_load_3d(&tm_a1, sbase + C::kABytes + u * 16384, a_full, h * D + 64 * u, r0, b);       // dO
        else
          tma_load_3d(&tm_a1, sbase + C::kABytes + u * 16384, a_full, 64 * u, r0, 2 * planes + (int)bh);   // V
      }
      int it = 0;
      for (int jb = next_block(jb0); jb < jb1; jb = next_block(jb + 1), ++it) {
        const int st = it % C::kStages, c0 = jb * kBN;
        if (it >= C::kStages && !(ok = one_wait(b_empty(st), ((it / C::kStages) & 1) ^ 1))) break;
        const uint32_t dst = sbase + C::kB + st * C::kStage;
        mbar_arrive_expect_tx(b_full(st), C::kStage + (MODE == kDKV ? C::kColBytes : 0));
        for (int u = 0; u < C::kSub; ++u) {
          tma_load_3d(&tm_b0, dst + u * C::kBSub, b_full(st), 64 * u, c0, b0);
          if (MODE == kDQ)
            tma_load_3d(&tm_b1, dst + C::kBBytes + u * C::kBSub, b_full(st), 64 * u, c0, 2 * planes + (int)bh);   // V
          else
            tma_load_3d(&tm_b1, dst + C::kBBytes + u * C::kBSub, b_full(st), h * D + 64 * u, c0, b);   // dO
        }
        if (MODE == kDKV)                                  // rows of rows2 are padded to whole blocks
          for (int k = 0; k < 2; ++k)
            bulk_load(sbase + C::kCol + st * C::kColBytes + k * kBN * 4, rows2 + ((size_t)k * planes + bh) * Sp + c0,
                      kBN * 4, b_full(st));
      }
      one_wait(a_full, 0);                  // every load has landed before the CTA exits
      for (int k = it > C::kStages ? it - C::kStages : 0; k < it; ++k)
        one_wait(b_full(k % C::kStages), (k / C::kStages) & 1);
    }
  } else if (warp == C::kRowWarps) {                       // MMA
    constexpr uint32_t idesc_s = idesc_f16_f32(128, kBN);
    constexpr uint32_t idesc_o = idesc_bmn(128, D);
    const uint64_t a_desc = smem_desc_sw128(sbase), b_desc = smem_desc_sw128(sbase + C::kB);
    const uint64_t bt_desc = desc_mn_sw128(sbase + C::kB, C::kBSub);           // the columns' operands, transposed
    auto p_of = [](int kk) { return 8 * kk + (C::kShare == 2 ? 16 * (kk >> 1) : 0); };   // columns of 16 of P or dU
    auto issue_scores = [&](int w, int st) {               // S and dP of the block in stage st, for warpgroup w
      tc_fence_after();
      if (elect_one()) {
        const uint64_t b_st = desc_at(b_desc, st * C::kStage);
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t u = kk / 4, o = (kk % 4) * 32;
            mma_f16_ss(tmem + (a ? C::kDP : C::kS) + w * kBN, desc_at(a_desc, a * C::kABytes + u * 16384 + o),
                       desc_at(b_st, a * C::kBBytes + u * C::kBSub + o), idesc_s, kk > 0 ? 1u : 0u);
          }
        mma_commit(s_full(w));
      }
      __syncwarp();
    };
    ok = warp_wait(a_full, 0);
    int jb = next_block(jb0), ahead = jb;                  // block of `it`, and the next whose scores are not issued
    int issued = 0, st_issue = 0, st = 0;                  // blocks whose scores are issued; stages of both
    for (; issued < C::NB && ok && ahead < jb1; ++issued, ++st_issue) {
      if (!(ok = warp_wait(b_full(st_issue), 0))) break;
      issue_scores(issued, st_issue);
      ahead = next_block(ahead + 1);
    }
    for (int it = 0; ok && jb < jb1; ++it, jb = next_block(jb + 1)) {
      const int w = it % C::NB;
      if (!(ok = warp_wait(p_full(w), (it / C::NB) & 1))) break;
      tc_fence_after();
      const int columns = n - jb * kBN;
      if (elect_one()) {
        const uint64_t bt = desc_at(bt_desc, st * C::kStage);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          if (16 * kk < columns)
            mma_f16_ts(tmem + C::kAcc, tmem + C::kDP + w * kBN + p_of(kk), desc_at(bt, kk * 2048), idesc_o,
                       it > 0 || kk > 0 ? 1u : 0u);
        if (MODE == kDKV) {
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            if (16 * kk < columns)
              mma_f16_ts(tmem + C::kAcc + D, tmem + C::kS + w * kBN + p_of(kk), desc_at(bt, C::kBBytes + kk * 2048),
                         idesc_o, it > 0 || kk > 0 ? 1u : 0u);
        }
        mma_commit(done(w));
        mma_commit(b_empty(st));
      }
      __syncwarp();
      if (ahead < jb1) {                                   // S and dP may be overwritten once P and dU have been read
        if (!(ok = warp_wait(b_full(st_issue), (issued / C::kStages) & 1))) break;
        if (!(ok = warp_wait(done(w), (it / C::NB) & 1))) break;
        issue_scores(w, st_issue);
        ++issued;
        st_issue = st_issue + 1 == C::kStages ? 0 : st_issue + 1;
        ahead = next_block(ahead + 1);
      }
      st = st + 1 == C::kStages ? 0 : st + 1;
    }
    if (elect_one()) mma_commit(drain);                    // every MMA issued here has completed
    __syncwarp();
    warp_wait(drain, 0);
  } else {
    const int w = warp >> 2, quad = warp & 3, r = quad * 32 + lane;   // warpgroup; row of the tile = TMEM lane
    const int pos = r0 + r;                                // the row's position
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int c_end = jb1 * kBN - 1, row_end = min(r0 + 127, n - 1);
    const Bias bias = MODE == kDQ ? make_bias(s, column, lut, NH, h, kBN, -row_end, c_end - r0, tid, C::kRowThreads)
                                  : make_bias(s, column, lut, NH, h, kBN, r0 - c_end, row_end, tid, C::kRowThreads);
    float* sums = reinterpret_cast<float*>(smem + C::kSums) + warp * kMaxScoreBuckets;
    if (MODE == kDQ && partial) {
      for (int k = tid; k <= 2 * s.reach; k += C::kRowThreads)
        bucket_of[k] = static_cast<uint8_t>(score_bucket(s, k - s.reach));
      for (int k = lane; k < s.buckets; k += 32) sums[k] = 0.f;
    }
    // dU's scale: norms holds the largest |dO_i|^2 and |v_j|^2 of every 128 rows.
    float mo = 0.f, mv = 0.f;
    for (int k = lane; k < (n + 127) / 128; k += 32) {
      mo = fmaxf(mo, norms[bh * (Sp / 128) + k]);
      mv = fmaxf(mv, norms[((size_t)planes + bh) * (Sp / 128) + k]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      mo = fmaxf(mo, __shfl_xor_sync(0xffffffffu, mo, off));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, off));
    }
    const float prod = sqrtf(mo) * sqrtf(mv);
    int ex = 0;
    if (prod > 0.f && prod < INFINITY) frexpf(prod, &ex);  // prod in [2^(ex-1), 2^ex)
    ex = max(-100, min(100, 14 - ex));
    const float e = exp2f((float)ex), inv_e = exp2f((float)-ex);
    asm volatile("bar.sync 1, %0;" ::"n"(C::kRowThreads) : "memory");

    const Cap cap = make_cap(s);
    const float scale2 = s.scale * kLog2e;
    const bool mine = pos < n;
    float neg_lse2 = 0.f, dsum = 0.f;
    if (MODE == kDQ) {                                     // (-inf where the row sees nothing)
      neg_lse2 = rows2[bh * Sp + pos];
      dsum = rows2[((size_t)planes + bh) * Sp + pos];
    }
    const int r_end = r0 + 127;
    // The columns that the row sees, and those that every row of the tile sees.
    const int lo = MODE == kDQ ? 0 : score_ilow(s, pos, prefix);
    const int hi = !mine ? 0 : MODE == kDQ ? score_jlim(s, pos, n, prefix) : n;
    const int lo_all = MODE == kDQ ? 0 : score_ilow(s, r_end, prefix);
    const int hi_all = MODE == kDQ ? score_jlim(s, r0, n, prefix) : n;
    RowBlock rb;
    const int doc = docs && mine ? docs[pos] : 0;
    rb.mine = mine;
    rb.e = e * kPInverse;
    rb.de = dsum * rb.e;
    const int buf = C::NB == 2 ? w : 0, first = C::kShare == 2 ? 32 * w : 0, last = C::kShare == 2 ? first + 32 : kBN;
    rb.t_s = t_lane + C::kS + buf * kBN;
    rb.t_dp = t_lane + C::kDP + buf * kBN;
    rb.p_at = C::kShare == 2 ? 16 * w : 0;                 // within the columns that the warpgroup reads itself
    float far_right = 0.f, far_left = 0.f;                 // sums of dT past the table's reach
    const bool biased = s.table || s.slopes;
    int it = 0;
    for (int jb = next_block(jb0); jb < jb1; jb = next_block(jb + 1), ++it) {
      if (it % C::NB != buf) continue;
      const int c0 = jb * kBN, st = it % C::kStages;
      const uint32_t ph = (it / C::NB) & 1;
      const bool cut = lo_all > c0 || c0 + kBN > hi_all || r_end >= n;
      const bool by_doc = docs && cls[jb] == 2;
      rb.valid = n - c0;
      // The row's visible columns among those that its warpgroup takes.  Documents: each id that the warp's rows
      // hold, against the columns'.
      bool mask = cut || by_doc, hidden = false;
      if (mask) {
        uint32_t some = 0, all = ~0u;
#pragma unroll
        for (int c = 0; c < kBN / 32; ++c) {
          if (C::kShare == 2 && c != w) continue;
          auto below = [](int x) { return x >= 32 ? ~0u : x <= 0 ? 0u : (1u << x) - 1; };
          uint32_t see = below(hi - c0 - 32 * c) & ~below(lo - c0 - 32 * c);
          if (by_doc) {
            const int j = c0 + 32 * c + lane, dj = j < n ? docs[j] : 0;
            uint32_t left = __ballot_sync(0xffffffffu, mine), eq = 0;
            while (left) {
              const int d = __shfl_sync(0xffffffffu, doc, __ffs(left) - 1);
              const bool same = doc == d;
              const uint32_t here = __ballot_sync(0xffffffffu, dj == d);
              left &= ~__ballot_sync(0xffffffffu, same);
              if (same) eq = here;
            }
            see &= eq;
          }
          rb.see[c] = see;
          some |= see;
          all &= see;
        }
        hidden = !any_warp(some != 0);                     // (rows past n see nothing)
        mask = any_warp(all != ~0u);
      }
      // Distances key - query of the block, and its bias.
      const int rel0 = MODE == kDQ ? c0 - pos : pos - c0;  // at column 0
      const int rel_min = MODE == kDQ ? c0 - r_end : r0 - (c0 + kBN - 1);
      const int rel_max = MODE == kDQ ? c0 + kBN - 1 - r0 : r_end - c0;
      const bool ahead = rel_min >= bias.reach;
      const bool near = biased && !ahead && rel_max > -bias.reach;
      const float sl = ahead ? -bias.slope2 : bias.slope2;
      rb.step = MODE == kDQ ? sl : -sl;
      rb.base = near ? neg_lse2 : (biased ? (ahead ? bias.right : bias.left) + sl * (float)rel0 : 0.f) + neg_lse2;
      rb.lut = bias.lut + bias.off + rel0;
      rb.col = reinterpret_cast<const float*>(smem + C::kCol + st * C::kColBytes);
      if (!(ok = warp_wait(s_full(buf), ph))) break;
      if (MODE == kDKV && !(ok = warp_wait(b_full(st), (it / C::kStages) & 1))) break;   // the columns' lse2 and D
      tc_fence_after();
      float sum[3] = {};
      if (hidden) {
        hidden_rows<MODE>(rb, first, last);
      } else if (near) {
        if (MODE == kDQ && partial) {
          if (LARGE || cap.on)
            row_block_m<MODE, C::kChunk, kCapped, MODE == kDQ ? 2 : 1>(s, mask, rb, first, last, cap, scale2, lane, sum);
          else
            row_block_m<MODE, C::kChunk, kNoCap, MODE == kDQ ? 2 : 1>(s, mask, rb, first, last, cap, scale2, lane, sum);
        } else if (LARGE || cap.on) {
          row_block_m<MODE, C::kChunk, kCapped, 1>(s, mask, rb, first, last, cap, scale2, lane, sum);
        } else {
          row_block_m<MODE, C::kChunk, kNoCap, 1>(s, mask, rb, first, last, cap, scale2, lane, sum);
        }
      } else if (s.slopes) {
        if (LARGE || cap.on)
          row_block_m<MODE, C::kChunk, kCapped, 3>(s, mask, rb, first, last, cap, scale2, lane, sum);
        else
          row_block_m<MODE, C::kChunk, kNoCap, 3>(s, mask, rb, first, last, cap, scale2, lane, sum);
      } else if (LARGE || cap.on) {
        row_block_m<MODE, C::kChunk, kCapped, 0>(s, mask, rb, first, last, cap, scale2, lane, sum);
      } else {
        row_block_m<MODE, C::kChunk, kNoCap, 0>(s, mask, rb, first, last, cap, scale2, lane, sum);
      }
      // Rows of the columns' operands in [n, n rounded up to 16) are read by the products: zeros.
      const int lim = n - c0, lim16 = (min(kBN, lim) + 15) & ~15;
      if (lim < lim16 && quad == 0 && (C::kShare == 1 || w == 0)) {
        const int units = (lim16 - lim) * 8;
        for (int k = lane; k < units * C::kSub * (MODE == kDKV ? 2 : 1); k += 32) {
          const int plane = k / units, rr = lim + k % units / 8;             // sub-tiles of B0, then of B1
          *reinterpret_cast<uint4*>(smem + C::kB + st * C::kStage + plane * C::kBSub + rr * 128 + (k % 8) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(buf));
      if (MODE == kDQ && partial) {
        if (near) {
          const int rel = c0 + first - (r0 + quad * 32);   // of the first column to the warp's first row
          auto bucket_at = [&](int x) { return (int)bucket_of[max(-s.reach, min(s.reach, x)) + s.reach]; };
#pragma unroll
          for (int k = 0; k < (C::kShare == 2 ? 2 : 3); ++k) add_by_bucket(sum[k], bucket_at(rel + lane + 32 * (k - 1)), sums, lane);
        } else if (ahead) {
          far_right += sum[1];
        } else {
          far_left += sum[1];
        }
      }
    }
    if (MODE == kDQ && partial) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        far_right += __shfl_xor_sync(0xffffffffu, far_right, off);
        far_left += __shfl_xor_sync(0xffffffffu, far_left, off);
      }
      if (lane == 0) {
        sums[score_bucket(s, s.reach)] += far_right;
        sums[score_bucket(s, -s.reach)] += far_left;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(C::kRowThreads) : "memory");
      const float* all = reinterpret_cast<const float*>(smem + C::kSums);
      for (int k = tid; k < s.buckets; k += C::kRowThreads) {
        float total = 0.f;
#pragma unroll
        for (int v = 0; v < C::kRowWarps; ++v) total += all[v * kMaxScoreBuckets + k];
        partial[(bh * gridDim.x + blk) * s.buckets + k] = total * inv_e;
      }
    }
    // Accumulators: 32 columns at a time to the warpgroups in turn, staged over the rows' operands (their
    // last reader has completed) in the store's swizzle, one TMA store per 64 columns of a warp's 32 rows.
    if (ok)
      for (int k = max(0, it - C::NB); k < it && ok; ++k) ok = warp_wait(done(k % C::NB), (k / C::NB) & 1);
    if (it == 0) one_wait(a_full, 0);
    if (ok) {
      tc_fence_after();
      constexpr int kCols = D < 64 ? D : 64, kRowBytes = 2 * kCols;
      constexpr int kParts = (MODE == kDKV ? 2 : 1) * C::kSub;               // pieces of up to 64 columns
#pragma unroll 1
      for (int part = w; part < kParts; part += 2) {
        const int acc = part / C::kSub, u = part % C::kSub;                  // acc 0: dQ or dK; 1: dV
        const float f = !mine ? 0.f : acc == 0 ? s.scale * inv_e : kPInverse;
        uint8_t* tile = smem + part * 16384 + quad * 32 * kRowBytes;
#pragma unroll 1
        for (int c = 0; c < kCols; c += 32) {
          uint32_t oa[32];
          if (it > 0) tmem_ld_32x32b_x32(t_lane + C::kAcc + acc * D + u * 64 + c, oa);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = mine && it > 0 ? half2_of(__uint_as_float(oa[8 * q + 2 * k]) * f, __uint_as_float(oa[8 * q + 2 * k + 1]) * f)
                                    : 0u;
            const int unit = c / 8 + q;
            const int sw = D < 64 ? unit ^ ((lane >> 1) & 3) : unit ^ (lane & 7);
            *reinterpret_cast<uint4*>(tile + lane * kRowBytes + 16 * sw) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        const int row = r0 + quad * 32;
        if (lane == 0 && row < S) {
          tma_store_3d(&tm_out, smem_u32(tile), 64 * u, row, (MODE == kDQ ? 0 : 1 + acc) * planes + (int)bh);
          bulk_commit_group();
        }
      }
      if (lane == 0) bulk_wait_group_all();
    }
  }

  if (!ok) atomicCAS(status, 0, kStatusWaitTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == C::kRowWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (MODE == kDKV) pdl_wait();
}

// Per row i: kPBits - lse in units of log2 (-inf where the row sees nothing or is past
// n, which makes P zero) and D_i, in rows padded to Sp; per 128 rows, the
// largest |dO_i|^2 and |v_j|^2.  D / 8 lanes read a row with 16-byte loads.
constexpr int kStatThreads = 256;
template <int D>
__global__ void __launch_bounds__(kStatThreads)
    scored_stats_kernel(const __half* __restrict__ qkv, const __half* __restrict__ ctx,
                        const __half* __restrict__ dctx, const float* __restrict__ lse,
                        const int32_t* __restrict__ valid_len, float* __restrict__ rows2, float* __restrict__ norms,
                        unsigned* __restrict__ counter, int B, int S, int Sp, int NH) {
  constexpr int kLanes = D / 8, kRows = kStatThreads / kLanes;
  __shared__ float wo[kStatThreads / 32], wv[kStatThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y, b = blockIdx.z, r0 = blockIdx.x * 128;
  if (blockIdx.x + h + b == 0 && threadIdx.x == 0) *counter = 0;
  const size_t bh = (size_t)b * NH + h, planes = (size_t)B * NH;
  const int n = score_len(valid_len, b, S);
  const int gl = threadIdx.x % kLanes;
  float mo = 0.f, mv = 0.f;
  auto widen = [](uint4 w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
      f[2 * k] = v.x;
      f[2 * k + 1] = v.y;
    }
  };
#pragma unroll 2
  for (int rr = threadIdx.x / kLanes; rr < 128; rr += kRows) {
    const int i = r0 + rr;
    float dot = 0.f, oo = 0.f, vv = 0.f;
    if (i < n) {
      float o[8], g[8], v[8];
      const size_t at = ((size_t)b * S + i) * NH * D + (size_t)h * D + gl * 8;
      widen(*reinterpret_cast<const uint4*>(ctx + at), o);
      widen(*reinterpret_cast<const uint4*>(dctx + at), g);
      widen(*reinterpret_cast<const uint4*>(qkv + ((2 * planes + bh) * S + i) * D + gl * 8), v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dot = fmaf(o[k], g[k], dot);
        oo = fmaf(g[k], g[k], oo);
        vv = fmaf(v[k], v[k], vv);
      }
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) {
      dot += __shfl_xor_sync(0xffffffffu, dot, off);
      oo += __shfl_xor_sync(0xffffffffu, oo, off);
      vv += __shfl_xor_sync(0xffffffffu, vv, off);
    }
    mo = fmaxf(mo, oo);
    mv = fmaxf(mv, vv);
    if (gl == 0) {
      const float l = i < n ? lse[bh * S + i] * kLog2e : -INFINITY;
      rows2[bh * Sp + i] = l == -INFINITY ? -INFINITY : kPBits - l;
      rows2[(planes + bh) * Sp + i] = dot;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    mo = fmaxf(mo, __shfl_xor_sync(0xffffffffu, mo, off));
    mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, off));
  }
  if (threadIdx.x % 32 == 0) {
    wo[threadIdx.x / 32] = mo;
    wv[threadIdx.x / 32] = mv;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kStatThreads / 32; ++k) {
      mo = fmaxf(mo, wo[k]);
      mv = fmaxf(mv, wv[k]);
    }
    norms[bh * (Sp / 128) + blockIdx.x] = mo;
    norms[(planes + bh) * (Sp / 128) + blockIdx.x] = mv;
  }
}

template <int D, int MODE, bool LARGE>
cudaError_t launch_mode(const ScoreArgs& s, const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0,
                        const CUtensorMap& b1, const CUtensorMap& out, const int32_t* vl, const float* rows2, int Sp,
                        const float* norms, unsigned* counter, float* partial, __half* dqkv, const ScoredShape& sh,
                        int* status, cudaStream_t stream) {
  using C = BCfg<D, MODE>;
  auto kern = scored_tc_bwd_kernel<D, MODE, LARGE>;
  static const cudaError_t attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (attr != cudaSuccess) return attr;
  const dim3 grid((sh.seq + 127) / 128, sh.head_num, sh.batch);
  return launch_kernel(kern, grid, dim3(C::kThreads), C::smem(s, sh.seq, partial != nullptr), stream, nullptr, 0, s, a0, a1,
                       b0, b1, out, vl, rows2, Sp, norms, counter, partial, dqkv, sh.batch, sh.seq, sh.head_num, status);
}

template <int D>
cudaError_t launch_d(const ScoreArgs& s, const __half* qkv, const int32_t* vl, const __half* ctx, const float* lse,
                     const __half* dctx, __half* dqkv, float* partial, void* scratch, const ScoredShape& sh, int* status,
                     cudaStream_t stream) {
  const uint64_t planes = (uint64_t)sh.batch * sh.head_num, H = (uint64_t)sh.head_num * D;
  const int Sp = (sh.seq + 127) / 128 * 128;
  float* rows2 = static_cast<float*>(scratch);
  float* norms = rows2 + 2 * planes * Sp;
  unsigned* counter = reinterpret_cast<unsigned*>(norms + 2 * planes * (Sp / 128));
  const dim3 grid(Sp / 128, sh.head_num, sh.batch);
  cudaError_t e = launch_kernel(scored_stats_kernel<D>, grid, dim3(kStatThreads), 0, stream, nullptr, 0, qkv, ctx, dctx,
                                lse, vl, rows2, norms, counter, sh.batch, sh.seq, Sp, sh.head_num);
  if (e != cudaSuccess) return e;
  CUtensorMap rows, cols, drows, dcols, out;
  if (!encode_operand_map(&rows, qkv, D, sh.seq, 3 * planes, 64, 128) ||
      !encode_operand_map(&cols, qkv, D, sh.seq, 3 * planes, 64, kBN) ||
      !encode_operand_map(&drows, dctx, H, sh.seq, sh.batch, 64, 128) ||
      !encode_operand_map(&dcols, dctx, H, sh.seq, sh.batch, 64, kBN) ||
      !encode_operand_map(&out, dqkv, D, sh.seq, 3 * planes, D < 64 ? D : 64, 32))
    return cudaErrorInvalidValue;
  auto both = [&](auto large) {
    constexpr bool LARGE = decltype(large)::value;
    const cudaError_t first = launch_mode<D, kDQ, LARGE>(s, rows, drows, cols, cols, out, vl, rows2, Sp, norms, counter,
                                                         partial, dqkv, sh, status, stream);
    if (first != cudaSuccess) return first;
    return launch_mode<D, kDKV, LARGE>(s, rows, rows, cols, dcols, out, vl, rows2, Sp, norms, counter, nullptr, dqkv, sh,
                                       status, stream);
  };
  return cap_kind(s) == kLargeCap ? both(std::true_type()) : both(std::false_type());
}

}  // namespace
}  // namespace scored_tc

size_t scored_backward_tc_scratch(const ScoredShape& sh) {
  const size_t planes = (size_t)sh.batch * sh.head_num, blocks = ((size_t)sh.seq + 127) / 128;
  return (planes * blocks * (2 * 128 + 2) + 1) * 4;
}

cudaError_t launch_scored_backward_tc(const ScoreArgs& s, const __half* qkv, const int32_t* valid_len,
                                      const __half* ctx, const float* lse, const __half* dctx, __half* dqkv,
                                      float* partial, void* scratch, const ScoredShape& sh, int* status,
                                      cudaStream_t stream) {
  using namespace scored_tc;
  switch (sh.size_per_head) {
    case 32: return launch_d<32>(s, qkv, valid_len, ctx, lse, dctx, dqkv, partial, scratch, sh, status, stream);
    case 64: return launch_d<64>(s, qkv, valid_len, ctx, lse, dctx, dqkv, partial, scratch, sh, status, stream);
    case 128: return launch_d<128>(s, qkv, valid_len, ctx, lse, dctx, dqkv, partial, scratch, sh, status, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace enc
