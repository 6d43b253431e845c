// Backward of attention with modified scores for sequences of at most 128: one
// pass that forms the scores once, persistent CTAs over (sequence, head) items.
//
// With one block of keys and one of queries, dQ needs no sum over blocks, so
// all five products run on one pair of score tiles (formulas in
// scored_tc_bwd.cu):
//   S^T = K Q^T, dP^T = V dO^T        M = 128 keys, N = 128 queries, K = D
//   dV = P^T dO                       A = P^T from TMEM
//   dK = dU^T Q                       A = dU^T from shared memory
//   dQ = dU K                         A = the same tile, read M-major
// Threads own key rows (TMEM lanes); two warpgroups share the 128 columns, w
// taking queries 64 g + 32 w .. + 31 for g = 0, 1, so that the FP16 P^T of each
// lands over S columns that it has read itself: P^T in columns [0, 64) of S, and
// dV's accumulator in [64, 128); dK and dQ go over dP (heads of 128: dV and dQ
// have columns of their own).  dU^T goes to shared memory as rows of keys, 64
// queries (128 bytes) to a swizzled row, which is a K-major operand for dK and
// an M-major one for dQ.
//
// The row statistics that the long kernels take from a kernel of their own (D_i
// and the norms for dU's scale) are worked out here from the tiles and a row of
// O, under the first two products.  The chain of an item's latencies is again
// what counts: two CTAs share an SM (one for heads of 128), and once the last
// products are done the next item's tiles load (and its O, into registers) and,
// as soon as the accumulators have been read, its first products run, under the
// output of this one, which goes through dU^T's tile.
//
// The table's gradient leaves the kernel as sums of dT by distance (255 floats
// for each head that a CTA has items of, at the place of the first of them).  For a column k of a 32 x 32 block, lane t takes the value of row
// (t + k) mod 32: all 32 lie on distinct diagonals, and over the columns lane t
// adds up the two diagonals whose row less column is t and t - 32, with no
// shuffle that waits for the one before (a partial sum passed from lane to lane
// along the diagonal took 64 dependent steps a row: 8,400 cycles an item against
// 2,400 without the sums).
//
// Measured, 12 heads of 64: 64 sequences of 64 to 128 with a table 50 us against
// 13 us of bytes; 148 full sequences of 128 59 us, 318 TF/s (table 80, cap 67 us).
// Bound by an item's chain of latencies: with two items to an SM, 5,000 cycles
// each with the table's sums, of which 630 are loads and stores at full bandwidth.
#include "scored_tc.cuh"

namespace enc {
namespace scored_tc {
namespace {

constexpr int kRowWarps = 8;
constexpr int kThreads = 32 * (kRowWarps + 1);

template <int D>
struct SBCfg {
  static constexpr int kCtasPerSm = D > 64 ? 1 : 2;
  static constexpr int kSub = D > 64 ? D / 64 : 1;
  static constexpr int kTile = kSub * 128 * 128;
  static constexpr int kQ = 0, kK = kTile, kDO = 2 * kTile, kV = 3 * kTile;
  static constexpr int kDU = 4 * kTile;                    // dU^T: 2 sub-tiles of 64 queries
  static constexpr int kBars = kDU + 2 * 16384;
  // full, s_full, p_full, acc_full, free, group, drain
  static constexpr int kSlot = kBars + 64;
  static constexpr int kMax = kSlot + 16;                  // per row warp: norms of dO and V
  static constexpr int kCol = kMax + 2 * kRowWarps * 4;    // kPBits - lse2 [128], D [128]
  static constexpr int kDocs = kCol + 256 * 4;
  static constexpr int kColumn = kDocs + 128 * 4;          // the head's column of the bias table
  static constexpr int kLut = kColumn + kMaxScoreBuckets * 4;   // bias of distance k - 127
  static constexpr int kDiag = kLut + 256 * 4;             // per row warp and g: 64 diagonals
  static constexpr int kSmem = 1024 + kDiag + kRowWarps * 2 * 64 * 4;
  // TMEM: S [0, 128) with P^T in [0, 64), dP [128, 256).
  static constexpr int kDP = 128, kDK = 128;
  static constexpr int kDQ = D > 64 ? 256 : 192, kDV = D > 64 ? 384 : 64;
  static constexpr int kTmemCols = D > 64 ? 512 : 256;
  static_assert(kCtasPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// 16 queries of a key row: from S^T and dP^T to P^T (TMEM) and dU^T (shared memory).
struct BwdChunk {
  uint32_t t_s, t_dp, t_p;  // TMEM addresses
  const float* lut;         // the row's bias at the chunk's first query; falls with the query
  const float* col;         // kPBits - lse2 [128] and D [128] at the first query
  int lo, hi;               // visible queries, as far as length and causality go
  const int* docs;          // documents of the queries, or nullptr
  int doc;
  float e;                  // dU's scale over P's
  uint8_t* du;              // the row of dU^T (64 queries), and the swizzle and 16-byte unit of the chunk
  int swizzle, unit;
  int valid;                // queries that are valid positions (any number)
  bool mine;                // the row is one
};

// DIAG: adds dT to the lane's two diagonals of the 32 x 32 block (k0: the chunk's first column in it).
// FORM: of the cap.
template <bool CAP, bool BIAS, bool DIAG, bool MASK, int FORM>
__device__ __forceinline__ void bwd_scores(const ScoreArgs& s, const BwdChunk& ch, const Cap& cap, float scale2, int lane, int k0,
                                           const uint32_t (&sv)[16], const uint32_t (&dp)[16], float& pos, float& neg) {
  uint32_t pp[8], pu[8];
  const uint64_t e2 = f2_pack(ch.e, ch.e), neg_e2 = f2_pack(-ch.e, -ch.e), one2 = f2_pack(1.f, 1.f);
  const uint64_t mul = CAP ? f2_pack(cap.cap2, cap.cap2) : f2_pack(scale2, scale2);
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(ch.col + k);
    const ulonglong2 dc = *reinterpret_cast<const ulonglong2*>(ch.col + 128 + k);
    int4 dj = make_int4(0, 0, 0, 0);
    if (MASK && ch.docs) dj = *reinterpret_cast<const int4*>(ch.docs + k);
    const int djs[4] = {dj.x, dj.y, dj.z, dj.w};
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
      uint64_t add = q ? nl.y : nl.x;
      if (BIAS) add = f2_add(add, f2_pack(ch.lut[-at], ch.lut[-(at + 1)]));
      float t0, t1;
      f2_unpack(CAP && FORM == kSmall ? f2_add(x, add) : f2_fma(x, mul, add), t0, t1);
      float p0 = ex2(t0), p1 = ex2(t1);
      const uint64_t dt2 =
          f2_mul(f2_pack(p0, p1), f2_fma(f2_pack(__uint_as_float(dp[at]), __uint_as_float(dp[at + 1])), e2,
                                         f2_mul(q ? dc.y : dc.x, neg_e2)));
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
        const bool see0 = at >= ch.lo && at < ch.hi && (!ch.docs || djs[q] == ch.doc);
        const bool see1 = at + 1 >= ch.lo && at + 1 < ch.hi && (!ch.docs || djs[q + 1] == ch.doc);
        p0 = see0 ? p0 : 0.f;
        p1 = see1 ? p1 : 0.f;
        a0 = see0 ? a0 : 0.f;
        a1 = see1 ? a1 : 0.f;
        u0 = see0 ? u0 : 0.f;
        u1 = see1 ? u1 : 0.f;
      }
      if (DIAG) {
        const int row = lane + k0 + at;                    // (mod 32)
        add_either(row < 32, __shfl_sync(0xffffffffu, a0, row), pos, neg);
        add_either(row + 1 < 32, __shfl_sync(0xffffffffu, a1, row + 1), pos, neg);
      }
      pp[at / 2] = half2_of(p0, p1);
      pu[at / 2] = half2_of(u0, u1);
    }
  }
  tmem_st_32x32b_x8_async(ch.t_p, pp);                     // over columns that this lane has read
  *reinterpret_cast<uint4*>(ch.du + 16 * (ch.unit ^ ch.swizzle)) = make_uint4(pu[0], pu[1], pu[2], pu[3]);
  *reinterpret_cast<uint4*>(ch.du + 16 * ((ch.unit + 1) ^ ch.swizzle)) = make_uint4(pu[4], pu[5], pu[6], pu[7]);
}

template <int CAP, bool BIAS, bool DIAG, bool MASK>
__device__ __forceinline__ void bwd_chunk(const ScoreArgs& s, const BwdChunk& ch, const Cap& cap, float scale2, int lane,
                                          int k0, float& pos, float& neg) {
  constexpr bool kOn = CAP != kNoCap;
  uint32_t sv[16], dp[16];
  tmem_ld_32x32b_x16_async(ch.t_s, sv);
  tmem_ld_32x32b_x16_async(ch.t_dp, dp);
  tmem_wait_ld(sv);
  tmem_wait_ld(dp);
  int form = kAny;
  if constexpr (kOn) {
    float top = 0.f;                                       // (of valid rows and queries, so that no other decides)
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, !MASK || k < ch.valid ? fabsf(__uint_as_float(sv[k])) : 0.f);
    form = !any_warp(ch.mine && top > s.cap_small_top) ? kSmall
           : !any_warp(ch.mine && top * fabsf(cap.in) > kCapPoly) ? kPoly : kAny;
  }
  if (kOn && form == kSmall)
    bwd_scores<kOn, BIAS, DIAG, MASK, kOn ? kSmall : kAny>(s, ch, cap, scale2, lane, k0, sv, dp, pos, neg);
  else if (kOn && form == kPoly)
    bwd_scores<kOn, BIAS, DIAG, MASK, kOn ? kPoly : kAny>(s, ch, cap, scale2, lane, k0, sv, dp, pos, neg);
  else
    bwd_scores<kOn, BIAS, DIAG, MASK, CAP == kLargeCap ? kCareful : kAny>(s, ch, cap, scale2, lane, k0, sv, dp, pos, neg);
}

template <int D, int CAP, bool BIAS, bool DIAG>
__global__ void __launch_bounds__(kThreads, SBCfg<D>::kCtasPerSm)
    scored_tc_bwd_short_kernel(const __grid_constant__ ScoreArgs s, const __grid_constant__ CUtensorMap tm_qkv,
                               const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_out,
                               const int32_t* __restrict__ valid_len, const __half* __restrict__ ctx,
                               const float* __restrict__ lse, __half* __restrict__ dqkv, float* __restrict__ partial,
                               int B, int S, int NH, int* __restrict__ status) {
  using C = SBCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBars;
  const uint32_t full = bar0, s_full = bar0 + 8, p_full = bar0 + 16, acc_full = bar0 + 24, acc_free = bar0 + 32,
                 group = bar0 + 40, drain = bar0 + 48;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kSlot);
  float* warp_max = reinterpret_cast<float*>(smem + C::kMax);
  float* col = reinterpret_cast<float*>(smem + C::kCol);
  int* pos_docs = reinterpret_cast<int*>(smem + C::kDocs);
  float* column = reinterpret_cast<float*>(smem + C::kColumn);
  float* lut = reinterpret_cast<float*>(smem + C::kLut);

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (tid == 0) {
    for (int k = 0; k < 7; ++k) {
      const uint32_t bar = bar0 + 8 * k;
      mbar_init(bar, bar == p_full || bar == acc_free || bar == group ? kRowWarps : 1);
    }
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == kRowWarps) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  pdl_trigger();                                           // after taking TMEM

  // Items [first, last) of B * NH, item = head * B + sequence.
  const int items = B * NH;
  const int first = first_item(blockIdx.x, items, gridDim.x), last = first_item(blockIdx.x + 1, items, gridDim.x);
  auto length = [&](int item) { return score_len(valid_len, item % B, S); };
  bool ok = true;
  if (warp == kRowWarps) {
    prefetch_tmap(&tm_qkv);
    prefetch_tmap(&tm_do);
    constexpr uint32_t idesc_s = idesc_f16_f32(128, 128);
    constexpr uint32_t idesc_o = idesc_bmn(128, D);        // A K-major (or in TMEM), B N-major
    constexpr uint32_t idesc_q = idesc_o | (1u << 15);     // A M-major too
    const uint64_t q_desc = smem_desc_sw128(sbase + C::kQ), k_desc = smem_desc_sw128(sbase + C::kK);
    const uint64_t v_desc = smem_desc_sw128(sbase + C::kV), do_desc = smem_desc_sw128(sbase + C::kDO);
    const uint64_t du_desc = smem_desc_sw128(sbase + C::kDU);
    const uint64_t du_m = desc_mn_sw128(sbase + C::kDU, 16384);
    const uint64_t q_n = desc_mn_sw128(sbase + C::kQ, 16384), k_n = desc_mn_sw128(sbase + C::kK, 16384);
    const uint64_t do_n = desc_mn_sw128(sbase + C::kDO, 16384);
    auto next_loaded = [&](int item) {
      while (item < last && length(item) == 0) ++item;
      return item;
    };
    auto load = [&](int item) {
      const int b = item % B, h = item / B;
      mbar_arrive_expect_tx(full, 4 * C::kTile);
      for (int part = 0; part < 3; ++part)
        for (int u = 0; u < C::kSub; ++u)
          tma_load_3d(&tm_qkv, sbase + (part == 0 ? C::kQ : part == 1 ? C::kK : C::kV) + u * 16384, full, 64 * u, 0,
                      (part * B + b) * NH + h);
      for (int u = 0; u < C::kSub; ++u) tma_load_3d(&tm_do, sbase + C::kDO + u * 16384, full, h * D + 64 * u, 0, b);
    };
    int loads = 0, it = 0;
    int cur = next_loaded(first);
    if (cur < last) {
      if (elect_one()) load(cur);
      loads = 1;
    }
    for (; cur < last; ++it) {
      const uint32_t ph = it & 1;
      const int n = length(cur), nxt = next_loaded(cur + 1);
      if (!(ok = warp_wait(full, ph))) break;
      if (it > 0 && !(ok = warp_wait(acc_free, ph ^ 1))) break;              // the previous item's accumulators
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = (kk / 4) * 16384 + (kk % 4) * 32;
          mma_f16_ss(tmem, desc_at(k_desc, o), desc_at(q_desc, o), idesc_s, kk > 0 ? 1u : 0u);
        }
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = (kk / 4) * 16384 + (kk % 4) * 32;
          mma_f16_ss(tmem + C::kDP, desc_at(v_desc, o), desc_at(do_desc, o), idesc_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(s_full);
      }
      __syncwarp();
      if (!(ok = warp_wait(p_full, ph))) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)                     // 16 queries: their P^T is in warpgroup (kk / 2) % 2's columns
          if (16 * kk < n)
            mma_f16_ts(tmem + C::kDV, tmem + 32 * ((kk >> 1) & 1) + 16 * (kk >> 2) + 8 * (kk & 1),
                       desc_at(do_n, kk * 2048), idesc_o, kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (16 * kk < n)
            mma_f16_ss(tmem + C::kDK, desc_at(du_desc, (kk / 4) * 16384 + (kk % 4) * 32), desc_at(q_n, kk * 2048), idesc_o,
                       kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)                     // 16 keys
          if (16 * kk < n)
            mma_f16_ss(tmem + C::kDQ, desc_at(du_m, kk * 2048), desc_at(k_n, kk * 2048), idesc_q, kk > 0 ? 1u : 0u);
        mma_commit(acc_full);
      }
      __syncwarp();
      if (nxt < last) {                                    // the tiles have been read
        if (!(ok = warp_wait(acc_full, ph))) break;
        if (elect_one()) load(nxt);
        ++loads;
      }
      cur = nxt;
    }
    if (elect_one()) mma_commit(drain);                    // every MMA issued here has completed
    __syncwarp();
    warp_wait(drain, 0);
    if (loads) warp_wait(full, (loads - 1) & 1);           // and every load has landed
  } else {
    const int w = warp >> 2, quad = warp & 3, r = quad * 32 + lane;          // warpgroup; key row = TMEM lane
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const Cap cap = make_cap(s);
    const float scale2 = s.scale * kLog2e;
    float* diag = reinterpret_cast<float*>(smem + C::kDiag);     // [row warp][g][64]: row less column + 32
    int it = 0, built = -1;
    uint32_t group_ph = 0;
    auto group_sync = [&] {                                // the row warps, bounded
      __syncwarp();
      if (lane == 0) mbar_arrive(group);
      ok = ok && warp_wait(group, group_ph);
      group_ph ^= 1;
    };
    // Half a row of O, and the row's lse, of an item (two threads to a row), asked for one item ahead.
    constexpr int kUnits = D / 16;                         // 16-byte units of half a row
    const int srow = tid >> 1, shalf = tid & 1;
    uint4 o_row[kUnits];
    float lse_row = 0.f;
    auto ask = [&](int item) {
      const int b = item % B, h = item / B;
      if (item >= last || srow >= score_len(valid_len, b, S)) return;
      const uint4* at = reinterpret_cast<const uint4*>(ctx + ((size_t)b * S + srow) * NH * D + (size_t)h * D) + shalf * kUnits;
#pragma unroll
      for (int k = 0; k < kUnits; ++k) o_row[k] = at[k];
      lse_row = lse[((size_t)b * NH + h) * S + srow];
    };
    ask(first);
    float by_distance = 0.f;                               // of distance tid - 127, over a head's items here
    for (int item = first; item < last; ++item) {
      const int b = item % B, h = item / B;
      if (DIAG && item > first && b == 0) {
        partial[(size_t)max(first, item - B) * 256 + tid] = by_distance;
        by_distance = 0.f;
      }
      const size_t bh = (size_t)b * NH + h;
      const int n = score_len(valid_len, b, S), prefix = score_prefix(s, b);
      if (BIAS && h != built) {                            // the head's bias, for distances within the sequence
        built = h;
        group_sync();                                      // the previous head's has been read
        load_column(s, column, NH, h, tid, 32 * kRowWarps);
        group_sync();
        const float slope = s.slopes ? s.slopes[h] : 0.f;
        for (int k = 128 - S + tid; k <= 126 + S; k += 32 * kRowWarps) lut[k] = score_bias2(s, column, slope, k - 127);
        group_sync();
        if (!ok) break;
      }
      if (n == 0) {                                        // zero gradients
        for (int part = 0; part < 3; ++part) {
          uint4* out = reinterpret_cast<uint4*>(dqkv + (((size_t)part * B * NH + bh) * S) * D);
          for (int k = tid; k < S * (D / 8); k += 32 * kRowWarps) out[k] = make_uint4(0, 0, 0, 0);
        }
        ask(item + 1);
        continue;
      }
      const uint32_t ph = it & 1;
      ++it;
      // Row statistics: two threads to a row.
      {
        const float l = srow < n ? lse_row * kLog2e : -INFINITY;
        if (s.docs && shalf == 0) pos_docs[srow] = srow < n ? s.docs[(size_t)b * S + srow] : 0;
        if (!(ok = warp_wait(full, ph))) break;
        float dot = 0.f, oo = 0.f, vv = 0.f;
        if (srow < n) {
#pragma unroll
          for (int k = 0; k < kUnits; ++k) {
            const int u = shalf * kUnits + k, at = (u / 8) * 16384 + srow * 128 + 16 * ((u % 8) ^ (srow & 7));
            const uint4 g4 = *reinterpret_cast<const uint4*>(smem + C::kDO + at);
            const uint4 v4 = *reinterpret_cast<const uint4*>(smem + C::kV + at);
            const uint32_t ow[4] = {o_row[k].x, o_row[k].y, o_row[k].z, o_row[k].w}, gw[4] = {g4.x, g4.y, g4.z, g4.w},
                           vw[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 o = __half22float2(*reinterpret_cast<const __half2*>(&ow[q]));
              const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&gw[q]));
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&vw[q]));
              dot = fmaf(o.x, g.x, fmaf(o.y, g.y, dot));
              oo = fmaf(g.x, g.x, fmaf(g.y, g.y, oo));
              vv = fmaf(v.x, v.x, fmaf(v.y, v.y, vv));
            }
          }
        }
        dot += __shfl_xor_sync(0xffffffffu, dot, 1);
        float mo = oo + __shfl_xor_sync(0xffffffffu, oo, 1), mv = vv + __shfl_xor_sync(0xffffffffu, vv, 1);
        if (shalf == 0) {
          col[srow] = l == -INFINITY ? -INFINITY : kPBits - l;
          col[128 + srow] = dot;
        }
#pragma unroll
        for (int off = 16; off > 1; off >>= 1) {
          mo = fmaxf(mo, __shfl_xor_sync(0xffffffffu, mo, off));
          mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, off));
        }
        if (lane == 0) {
          warp_max[warp] = mo;
          warp_max[kRowWarps + warp] = mv;
        }
        if (lane == 0) bulk_wait_group_read<0>();          // the last output rows have left dU^T's tile
        group_sync();
        if (!ok) break;
      }
      float mo = 0.f, mv = 0.f;
#pragma unroll
      for (int k = 0; k < kRowWarps; ++k) {
        mo = fmaxf(mo, warp_max[k]);
        mv = fmaxf(mv, warp_max[kRowWarps + k]);
      }
      const float prod = sqrtf(mo) * sqrtf(mv);
      int ex = 0;
      if (prod > 0.f && prod < INFINITY) frexpf(prod, &ex);                  // prod in [2^(ex-1), 2^ex)
      ex = max(-100, min(100, 14 - ex));
      const float e = exp2f((float)ex), inv_e = exp2f((float)-ex);

      const bool mine = r < n;
      const int w0 = quad * 32, w1 = w0 + 31;              // the warp's keys
      const int ilow = score_ilow(s, r, prefix), ilow_first = score_ilow(s, w0, prefix);
      const int ilow_all = max(score_ilow(s, w1, prefix), ilow_first);
      BwdChunk ch;
      ch.doc = s.docs ? pos_docs[r] : 0;
      ch.e = e * kPInverse;
      ch.swizzle = r & 7;
      if (!(ok = warp_wait(s_full, ph))) break;
      tc_fence_after();
#pragma unroll 1
      for (int g = 0; g < 2; ++g) {
        float pos = 0.f, neg = 0.f;                        // diagonals lane and lane - 32
        const int i0 = 64 * g + 32 * w;
        const bool none = w0 >= n || i0 >= n || i0 + 32 <= min(ilow_first, score_ilow(s, min(w1, n - 1), prefix));
#pragma unroll 1
        for (int c = 0; c < 32; c += 16) {
          const int i = i0 + c;
          ch.t_s = t_row + i;
          ch.t_dp = t_row + C::kDP + i;
          ch.t_p = t_row + 32 * w + 16 * g + c / 2;
          ch.lut = lut + 127 + r - i;
          ch.col = col + i;
          ch.lo = ilow - i;
          ch.hi = mine ? n - i : 0;
          ch.docs = s.docs ? pos_docs + i : nullptr;
          ch.du = smem + C::kDU + g * 16384 + r * 128;
          ch.unit = 4 * w + c / 8;
          ch.valid = n - i;
          ch.mine = mine;
          if (none) {
            const uint32_t zero[8] = {};
            tmem_st_32x32b_x8_async(ch.t_p, zero);
            *reinterpret_cast<uint4*>(ch.du + 16 * (ch.unit ^ ch.swizzle)) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(ch.du + 16 * ((ch.unit + 1) ^ ch.swizzle)) = make_uint4(0, 0, 0, 0);
          } else if (s.docs || w1 >= n || i + 16 > n || i < ilow_all) {
            bwd_chunk<CAP, BIAS, DIAG, true>(s, ch, cap, scale2, lane, c, pos, neg);
          } else {
            bwd_chunk<CAP, BIAS, DIAG, false>(s, ch, cap, scale2, lane, c, pos, neg);
          }
        }
        if (DIAG) {
          diag[(warp * 2 + g) * 64 + 32 + lane] = pos;
          diag[(warp * 2 + g) * 64 + lane] = neg;
        }
      }
      // Rows in [n, n rounded up to 16) of the operands that the last three products sum over: zeros, whatever
      // memory holds there.
      const int n16 = (n + 15) & ~15;
      if (n < n16 && quad == (n >> 5)) {
        const int units = (n16 - n) * 8;
        for (int k = w * 32 + lane; k < units * C::kSub * 3; k += 64) {
          const int plane = k / units, rr = n + k % units / 8;               // sub-tiles of Q, K, dO
          *reinterpret_cast<uint4*>(smem + plane * 16384 + rr * 128 + (k % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();                            // dU^T and the zeros visible to the tensor core
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
      if (DIAG) {
        group_sync();
        if (!ok) break;
        // Distance tid - 127: block (quad, i0 / 32) has it at row less column tid - 127 - 32 (quad - i0 / 32).
        float total = 0.f;
#pragma unroll
        for (int v = 0; v < kRowWarps * 2; ++v) {          // row warp v / 2, g = v % 2
          const int d = tid - 127 - 32 * ((v / 2) % 4 - (2 * (v % 2) + v / 8));
          if (d >= -32 && d < 32) total += diag[v * 64 + 32 + d];
        }
        by_distance += total * inv_e;                      // (the 256th is not used)
      }
      ask(item + 1);
      if (!(ok = warp_wait(acc_full, ph))) break;
      tc_fence_after();
      // 32 columns of an accumulator at a time, the warpgroups in turn: FP16 rows of 64 bytes in the store's swizzle
      // over dU^T's tile, in one of the warp's two places in turn, and a TMA store for its 32 rows.
      constexpr int kPieces = 3 * (D / 32);
#pragma unroll 1
      for (int piece = w; piece < kPieces; piece += 2) {
        const int part = piece / (D / 32), c = piece % (D / 32) * 32;        // 0: dQ, 1: dK, 2: dV
        const float f = !mine ? 0.f : part == 2 ? kPInverse : s.scale * inv_e;
        uint32_t oa[32];
        tmem_ld_32x32b_x32(t_row + (part == 0 ? C::kDQ : part == 1 ? C::kDK : C::kDV) + c, oa);
        uint8_t* tile = smem + C::kDU + warp * 4096 + ((piece >> 1) & 1) * 2048;
        if (piece >= 4) {
          if (lane == 0) bulk_wait_group_read<1>();
          __syncwarp();
        }
        if (piece + 2 >= kPieces) {                        // all that this warp reads has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_free);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = mine ? half2_of(__uint_as_float(oa[8 * q + 2 * k]) * f, __uint_as_float(oa[8 * q + 2 * k + 1]) * f) : 0u;
          *reinterpret_cast<uint4*>(tile + lane * 64 + 16 * (q ^ ((lane >> 1) & 3))) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && w0 < S) {                         // rows at or past S are outside the map
          tma_store_3d(&tm_out, smem_u32(tile), c, w0, part * B * NH + (int)bh);
          bulk_commit_group();
        }
      }
    }
    if (DIAG && first < last) partial[(size_t)max(first, (last - 1) / B * B) * 256 + tid] = by_distance;
    if (lane == 0) bulk_wait_group_read<0>();
  }

  if (!ok) atomicCAS(status, 0, kStatusWaitTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == kRowWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int CAP, bool BIAS, bool DIAG>
cudaError_t launch_v(const ScoreArgs& s, const __half* qkv, const int32_t* vl, const __half* ctx, const float* lse,
                     const __half* dctx, __half* dqkv, float* partial, const ScoredShape& sh, int* status, int num_sms,
                     cudaStream_t stream) {
  using C = SBCfg<D>;
  auto kern = scored_tc_bwd_short_kernel<D, CAP, BIAS, DIAG>;
  static const cudaError_t attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (attr != cudaSuccess) return attr;
  const uint64_t planes = 3ull * sh.batch * sh.head_num;
  CUtensorMap tq, td, to;
  if (!encode_operand_map(&tq, qkv, D, sh.seq, planes, 64, 128) ||
      !encode_operand_map(&td, dctx, (uint64_t)sh.head_num * D, sh.seq, sh.batch, 64, 128) ||
      !encode_operand_map(&to, dqkv, D, sh.seq, planes, 32, 32))
    return cudaErrorInvalidValue;
  return launch_kernel(kern, dim3(scored_short_ctas(sh, num_sms)), dim3(kThreads), C::kSmem, stream,
                       nullptr, 0, s, tq, td, to, vl, ctx, lse, dqkv, partial, sh.batch, sh.seq, sh.head_num,
                       status);
}

template <int D, int CAP>
cudaError_t launch_d(const ScoreArgs& s, const __half* qkv, const int32_t* vl, const __half* ctx, const float* lse,
                     const __half* dctx, __half* dqkv, float* partial, const ScoredShape& sh, int* status, int num_sms,
                     cudaStream_t stream) {
  if (partial) return launch_v<D, CAP, true, true>(s, qkv, vl, ctx, lse, dctx, dqkv, partial, sh, status, num_sms, stream);
  return s.table || s.slopes
             ? launch_v<D, CAP, true, false>(s, qkv, vl, ctx, lse, dctx, dqkv, partial, sh, status, num_sms, stream)
             : launch_v<D, CAP, false, false>(s, qkv, vl, ctx, lse, dctx, dqkv, partial, sh, status, num_sms, stream);
}

}  // namespace
}  // namespace scored_tc

int scored_short_ctas(const ScoredShape& sh, int num_sms) {
  const long items = (long)sh.batch * sh.head_num, resident = (sh.size_per_head > 64 ? 1L : 2L) * num_sms;
  return (int)(items < resident ? items : resident);
}

cudaError_t launch_scored_backward_tc_short(const ScoreArgs& s, const __half* qkv, const int32_t* valid_len,
                                            const __half* ctx, const float* lse, const __half* dctx, __half* dqkv,
                                            float* partial, const ScoredShape& sh, int* status, int num_sms,
                                            cudaStream_t stream) {
  using namespace scored_tc;
  auto run = [&](auto d, auto cap) {
    return launch_d<decltype(d)::value, decltype(cap)::value>(s, qkv, valid_len, ctx, lse, dctx, dqkv, partial, sh, status,
                                                              num_sms, stream);
  };
  auto capped = [&](auto d) { return with_cap(s, [&](auto cap) { return run(d, cap); }); };
  switch (sh.size_per_head) {
    case 32: return capped(std::integral_constant<int, 32>());
    case 64: return capped(std::integral_constant<int, 64>());
    case 128: return capped(std::integral_constant<int, 128>());
  }
  return cudaErrorInvalidValue;
}

}  // namespace enc
