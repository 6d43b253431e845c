// Forward of attention with modified scores for sequences of at most 128, where
// one block of 128 keys holds every key: persistent CTAs, each taking a run of
// (sequence, head) items.
//
// At these lengths an item is two small products and 128 rows of softmax, and
// the chain of an item's latencies (its loads, S, the softmax, P V, the output)
// is several times its work.  So four CTAs share an SM (two for heads of 128),
// and each overlaps its items: the next item's Q and K load as soon as S is
// done, its V once the output rows have left the V tile.  Items are numbered
// head by head, and a CTA takes consecutive ones, so that the bias table in
// shared memory is built once for a run of sequences.
//
//   warps 0..3  softmax: thread r owns query row r = TMEM lane r
//   warp 4      TMA loads and MMAs
//                 S = Q K^T   M = 128, N = 128, K = D
//                 O = P V     M = 128, N = D, K = 16 per group of 16 valid keys
// TMEM: S in columns [0, 128); t2 is written back over S in the first pass (scale,
// cap, bias, masks, row maximum), so that the row needs no registers, and P over
// columns [0, 64) in the second; O in [64, 64 + D) for heads up to 64, else in
// [128, 256).  Chunks of 32 keys that no row of a warp sees cost nothing but a
// store of zeros, and warps whose rows are all padding do no work.
//
// Measured: 12 heads of 64, 256 sequences of 64 to 128, a table: 41 us, 44 with a
// cold L2, 0.57 of the measured bandwidth on the 165 MB of its valid rows (the boxes
// hold 128 rows whatever n is: 201 MB move); 148 full sequences of 128: 28 us with a
// table, 32 with a cap.  The encoder's plain attention kernel takes 40 us on the
// data of the first.
#include "scored_tc.cuh"

namespace enc {
namespace scored_tc {
namespace {

constexpr int kSoftmax = 4;                                // warps
constexpr int kThreads = 32 * (kSoftmax + 1);
constexpr float kRaiseLog2 = 15.f;                         // P = 2^(t2 - maximum + 15), in the upper half of FP16's range

template <int D>
struct SCfg {
  static constexpr int kCtasPerSm = D > 64 ? 2 : 4;
  static constexpr int kSub = D > 64 ? D / 64 : 1;
  static constexpr int kTile = kSub * 128 * 128;           // an operand
  static constexpr int kQ = 0, kK = kTile, kV = 2 * kTile; // V tile, then the output rows
  static constexpr int kBars = 3 * kTile;                  // qk_full, v_full, s_full, p_full, o_full, o_free, v_free, drain, group
  static constexpr int kSlot = kBars + 80;
  static constexpr int kDocs = kSlot + 16;
  static constexpr int kColumn = kDocs + 128 * 4;
  static constexpr int kLut = kColumn + kMaxScoreBuckets * 4;  // bias of distance k - 127
  static constexpr int kSmem = 1024 + kLut + 256 * 4;
  static constexpr int kO = D > 64 ? 128 : 64;
  static constexpr int kTmemCols = D > 64 ? 256 : 128;
  static_assert(kCtasPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// 32 keys of a row, first pass: S in TMEM becomes t2; returns the maximum over the visible ones.
struct ShortChunk {
  uint32_t t_s;             // TMEM address of the chunk in the row
  uint64_t scale2, cap2;    // pairs
  float cap_in;
  const float* lut;         // the row's bias at the chunk's first key
  int lim;                  // visible keys of the chunk, as far as length and causality go
  const int* docs;          // documents of the keys (shared memory), or nullptr
  int doc;
  int keys;                 // valid keys of the chunk (any number)
  bool mine;                // the row is a valid query
};
template <int CAP, bool BIAS, bool MASK>
__device__ __forceinline__ float first_pass(const ScoreArgs& s, const ShortChunk& ch, float mx) {
  uint32_t sv[32];
  tmem_ld_32x32b_x32(ch.t_s, sv);
  uint64_t x[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = f2_pack(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1]));
  uint64_t mul = CAP != kNoCap ? ch.cap2 : ch.scale2;
  if constexpr (CAP != kNoCap) {
    float top = 0.f;                                       // (of valid rows and keys, so that no other decides)
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float a, c;
      f2_unpack(x[k], a, c);
      if (MASK) {
        a = 2 * k < ch.keys ? a : 0.f;
        c = 2 * k + 1 < ch.keys ? c : 0.f;
      }
      top = fmaxf(fmaxf(top, fabsf(a)), fabsf(c));
    }
    if (!any_warp(ch.mine && top > s.cap_small_top)) {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = small_cap2(s, x[k]);
      mul = f2_pack(1.f, 1.f);
    } else if (!any_warp(ch.mine && top * fabsf(ch.cap_in) > kCapPoly)) {
      const uint64_t in = f2_pack(ch.cap_in, ch.cap_in);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint64_t y = f2_mul(x[k], in);
        x[k] = f2_mul(y, tanh_over_x2(f2_mul(y, y)));
      }
    } else if constexpr (CAP == kLargeCap) {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = tanh_careful2(x[k], ch.cap_in);
    } else {
      const float in2 = 2.f * kLog2e * ch.cap_in;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float a, c;
        f2_unpack(x[k], a, c);
        x[k] = f2_pack(tanh_of(a, in2), tanh_of(c, in2));
      }
    }
  }
  float m2[2] = {mx, mx};
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    x[k] = BIAS ? f2_fma(x[k], mul, f2_pack(ch.lut[2 * k], ch.lut[2 * k + 1])) : f2_mul(x[k], mul);
    float a, c;
    f2_unpack(x[k], a, c);
    if constexpr (MASK) {
      a = 2 * k < ch.lim && (!ch.docs || ch.docs[2 * k] == ch.doc) ? a : -INFINITY;
      c = 2 * k + 1 < ch.lim && (!ch.docs || ch.docs[2 * k + 1] == ch.doc) ? c : -INFINITY;
    }
    m2[k & 1] = fmaxf(fmaxf(m2[k & 1], a), c);
    sv[2 * k] = __float_as_uint(a);
    sv[2 * k + 1] = __float_as_uint(c);
  }
  tmem_st_32x32b_x32(ch.t_s, sv);
  return fmaxf(m2[0], m2[1]);
}

template <int D, int CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, SCfg<D>::kCtasPerSm)
    scored_tc_short_kernel(const __grid_constant__ ScoreArgs s, const __grid_constant__ CUtensorMap tm_qkv,
                           const __grid_constant__ CUtensorMap tm_ctx, const int32_t* __restrict__ valid_len,
                           __half* __restrict__ ctx, float* __restrict__ lse, int B, int S, int NH, int* __restrict__ status) {
  using C = SCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBars;
  const uint32_t qk_full = bar0, v_full = bar0 + 8, s_full = bar0 + 16, p_full = bar0 + 24, o_full = bar0 + 32,
                 o_free = bar0 + 40, v_free = bar0 + 48, drain = bar0 + 56, group = bar0 + 64;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kSlot);
  float* column = reinterpret_cast<float*>(smem + C::kColumn);
  float* lut = reinterpret_cast<float*>(smem + C::kLut);
  int* key_docs = reinterpret_cast<int*>(smem + C::kDocs);

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (tid == 0) {
    for (int k = 0; k < 9; ++k) {
      const uint32_t bar = bar0 + 8 * k;
      mbar_init(bar, bar == p_full || bar == o_free || bar == v_free || bar == group ? kSoftmax : 1);
    }
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == kSoftmax) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  pdl_trigger();                                           // after taking TMEM

  // Items [first, last) of B * NH, item = head * B + sequence.
  const int items = B * NH, ctas = gridDim.x, cta = blockIdx.x;
  const int first = (int)((long long)items * cta / ctas), last = (int)((long long)items * (cta + 1) / ctas);
  auto length = [&](int item) { return score_len(valid_len, item % B, S); };
  bool ok = true;
  if (warp == kSoftmax) {
    prefetch_tmap(&tm_qkv);
    constexpr uint32_t idesc_s = idesc_f16_f32(128, 128), idesc_o = idesc_bmn(128, D);
    const uint64_t q_desc = smem_desc_sw128(sbase + C::kQ), k_desc = smem_desc_sw128(sbase + C::kK);
    const uint64_t v_desc = desc_mn_sw128(sbase + C::kV, 16384);
    auto next_loaded = [&](int item) {                     // items with no valid key load nothing
      while (item < last && length(item) == 0) ++item;
      return item;
    };
    auto load = [&](int item, int part, uint32_t dst, uint32_t bar) {        // part 0: Q, 1: K, 2: V
      const int plane = (part * B + item % B) * NH + item / B;
      for (int u = 0; u < C::kSub; ++u) tma_load_3d(&tm_qkv, dst + u * 16384, bar, 64 * u, 0, plane);
    };
    auto load_qk = [&](int item) {
      mbar_arrive_expect_tx(qk_full, 2 * C::kTile);
      load(item, 0, sbase + C::kQ, qk_full);
      load(item, 1, sbase + C::kK, qk_full);
    };
    auto load_v = [&](int item) {
      mbar_arrive_expect_tx(v_full, C::kTile);
      load(item, 2, sbase + C::kV, v_full);
    };
    int qk_loads = 0, v_loads = 0, it = 0;
    int cur = next_loaded(first);
    if (cur < last) {
      if (elect_one()) {
        load_qk(cur);
        load_v(cur);
      }
      qk_loads = v_loads = 1;
    }
    for (; cur < last; ++it) {
      const uint32_t ph = it & 1;
      const int n = length(cur), nxt = next_loaded(cur + 1);
      if (!(ok = warp_wait(qk_full, ph))) break;
      if (it > 0 && !(ok = warp_wait(o_free, ph ^ 1))) break;                // S goes over the previous item's O
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = (kk / 4) * 16384 + (kk % 4) * 32;
          mma_f16_ss(tmem, desc_at(q_desc, o), desc_at(k_desc, o), idesc_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(s_full);
      }
      __syncwarp();
      if (it > 0) {                                        // the V tile held the previous item's output rows
        if (!(ok = warp_wait(v_free, ph ^ 1))) break;
        if (elect_one()) load_v(cur);
        ++v_loads;
      }
      if (nxt < last) {                                    // the next Q and K, once S has read these
        if (!(ok = warp_wait(s_full, ph))) break;
        if (elect_one()) load_qk(nxt);
        ++qk_loads;
      }
      if (!(ok = warp_wait(p_full, ph))) break;
      if (!(ok = warp_wait(v_full, ph))) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (16 * kk < n)
            mma_f16_ts(tmem + C::kO, tmem + 8 * kk, desc_at(v_desc, kk * 2048), idesc_o, kk > 0 ? 1u : 0u);
        mma_commit(o_full);
      }
      __syncwarp();
      cur = nxt;
    }
    if (elect_one()) mma_commit(drain);                    // every MMA issued here has completed
    __syncwarp();
    warp_wait(drain, 0);
    if (qk_loads) warp_wait(qk_full, (qk_loads - 1) & 1);  // and every load has landed
    if (v_loads) warp_wait(v_full, (v_loads - 1) & 1);
  } else {
    const int r = warp * 32 + lane;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const Cap cap = make_cap(s);
    ShortChunk ch;
    ch.scale2 = f2_pack(s.scale * kLog2e, s.scale * kLog2e);
    ch.cap2 = f2_pack(cap.cap2, cap.cap2);
    ch.cap_in = cap.in;
    constexpr int kCols = D < 64 ? D : 64, kRowBytes = 2 * kCols;
    int it = 0, built = -1;
    uint32_t group_ph = 0;
    auto group_sync = [&] {                                // the softmax warps; bounded, unlike a named barrier
      __syncwarp();
      if (lane == 0) mbar_arrive(group);
      ok = ok && warp_wait(group, group_ph);
      group_ph ^= 1;
    };
    for (int item = first; item < last; ++item) {
      const int b = item % B, h = item / B;
      const int n = score_len(valid_len, b, S), prefix = score_prefix(s, b);
      if (BIAS && h != built) {                            // the head's bias, for distances within the sequence
        built = h;
        group_sync();                                      // the previous head's has been read
        load_column(s, column, NH, h, r, 128);
        group_sync();
        const float slope = s.slopes ? s.slopes[h] : 0.f;
        for (int k = 128 - S + r; k <= 126 + S; k += 128) lut[k] = score_bias2(s, column, slope, k - 127);
        group_sync();
        if (!ok) break;
      }
      if (n == 0) {                                        // ctx = 0, lse = -inf
        if (r < S) {
          uint4* out = reinterpret_cast<uint4*>(ctx + ((size_t)b * S + r) * NH * D + h * D);
          for (int u = 0; u < D / 8; ++u) out[u] = make_uint4(0, 0, 0, 0);
          if (lse) lse[((size_t)b * NH + h) * S + r] = -INFINITY;
        }
        continue;
      }
      const uint32_t ph = it & 1;
      ++it;
      if (s.docs) {
        group_sync();                                      // the previous item's have been read
        key_docs[r] = r < n ? s.docs[(size_t)b * S + r] : 0;
        group_sync();
        if (!ok) break;
      }
      const int w0 = warp * 32;                            // the warp's first row
      // Keys that the row, the warp's last valid row and its first row see, as far as length and causality go.
      const int jlim = r < n ? score_jlim(s, r, n, prefix) : 0;
      const int wlim = w0 < n ? score_jlim(s, min(w0 + 31, n - 1), n, prefix) : 0;
      const int jall = w0 + 31 < n && !s.docs ? score_jlim(s, w0, n, prefix) : 0;
      const int chunks = (wlim + 31) >> 5, stored = (n + 31) >> 5;
      ch.doc = s.docs ? key_docs[r] : 0;
      ch.mine = r < n;
      if (!(ok = warp_wait(s_full, ph))) break;
      tc_fence_after();
      float mx = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        ch.t_s = t_row + 32 * c;
        ch.lut = lut + 127 + 32 * c - r;
        ch.lim = jlim - 32 * c;
        ch.docs = s.docs ? key_docs + 32 * c : nullptr;
        ch.keys = n - 32 * c;
        mx = 32 * c + 32 <= jall ? first_pass<CAP, BIAS, false>(s, ch, mx) : first_pass<CAP, BIAS, true>(s, ch, mx);
      }
      const float mu = mx == -INFINITY ? 0.f : mx;
      const float neg_m = raised(kRaiseLog2, mu);
      const uint64_t neg_m2 = f2_pack(neg_m, neg_m);
      uint64_t sum2 = 0;                                   // two partial row sums (0.0f, 0.0f)
#pragma unroll 1
      for (int c = 0; c < stored; ++c) {
        uint32_t pk[16];
        if (c < chunks) {
          uint32_t sv[32];
          tmem_ld_32x32b_x32(t_row + 32 * c, sv);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float t0, t1;
            f2_unpack(f2_add(f2_pack(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), neg_m2), t0, t1);
            const float p0 = ex2(t0), p1 = ex2(t1);
            sum2 = f2_add(sum2, f2_pack(p0, p1));
            pk[k] = half2_of(p0, p1);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) pk[k] = 0;
        }
        tmem_st_32x32b_x16_async(t_row + 16 * c, pk);
      }
      // V rows of keys in [n, n rounded up to 16) are read by P V: zeros, whatever memory holds there.
      const int n16 = (n + 15) & ~15;
      if (n < n16 && warp == (n >> 5)) {
        if (!(ok = warp_wait(v_full, ph))) break;
        if (r >= n && r < n16)
          for (int u = 0; u < 8 * C::kSub; ++u)
            *reinterpret_cast<uint4*>(smem + C::kV + (u / 8) * 16384 + r * 128 + (u % 8) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();                          // visible to the tensor core
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
      float s0, s1;
      f2_unpack(sum2, s0, s1);
      const float l = s0 + s1;
      const bool seen = r < n && l > 0.f;
      const float inv = seen ? 1.f / l : 0.f;
      if (lse && r < S) lse[((size_t)b * NH + h) * S + r] = seen ? (log2f(l) - neg_m) * kLn2 : -INFINITY;
      if (!(ok = warp_wait(o_full, ph))) break;
      tc_fence_after();
      // The row of O as FP16 into the V tile (P V has read it), in the store's swizzle.
      uint8_t* out = smem + C::kV + warp * 32 * kRowBytes + lane * kRowBytes;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t oa[32];
        tmem_ld_32x32b_x32(t_row + C::kO + c, oa);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = seen ? half2_of(__uint_as_float(oa[8 * u + 2 * k]) * inv, __uint_as_float(oa[8 * u + 2 * k + 1]) * inv)
                        : 0u;
          const int unit = (c % 64) / 8 + u;
          const int sw = D < 64 ? unit ^ ((lane >> 1) & 3) : unit ^ (lane & 7);
          *reinterpret_cast<uint4*>(out + (c / 64) * 16384 + 16 * sw) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();                            // the rows visible to the TMA store
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_free);                               // the next S may overwrite O
        if (w0 < S) {                                      // rows at or past S are outside the map
          for (int u = 0; u < C::kSub; ++u)
            tma_store_3d(&tm_ctx, sbase + C::kV + u * 16384 + w0 * kRowBytes, h * D + 64 * u, w0, b);
          bulk_commit_group();
          bulk_wait_group_read<0>();
        }
        mbar_arrive(v_free);
      }
    }
  }

  if (!ok) atomicCAS(status, 0, kStatusWaitTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmax) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int CAP, bool BIAS>
cudaError_t launch_v(const ScoreArgs& s, const __half* qkv, const int32_t* vl, __half* ctx, float* lse,
                     const ScoredShape& sh, int* status, int num_sms, cudaStream_t stream) {
  using C = SCfg<D>;
  static const cudaError_t attr = cudaFuncSetAttribute(scored_tc_short_kernel<D, CAP, BIAS>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (attr != cudaSuccess) return attr;
  CUtensorMap tq, tc;
  if (!encode_operand_map(&tq, qkv, D, sh.seq, 3ull * sh.batch * sh.head_num, 64, 128) ||
      !encode_operand_map(&tc, ctx, (uint64_t)sh.head_num * D, sh.seq, sh.batch, D < 64 ? D : 64, 32))
    return cudaErrorInvalidValue;
  const long items = (long)sh.batch * sh.head_num, resident = (long)C::kCtasPerSm * num_sms;
  return launch_kernel(scored_tc_short_kernel<D, CAP, BIAS>, dim3((unsigned)(items < resident ? items : resident)),
                       dim3(kThreads), C::kSmem, stream, nullptr, 0, s, tq, tc, vl, ctx, lse, sh.batch, sh.seq,
                       sh.head_num, status);
}

template <int D>
cudaError_t launch_d(const ScoreArgs& s, const __half* qkv, const int32_t* vl, __half* ctx, float* lse,
                     const ScoredShape& sh, int* status, int num_sms, cudaStream_t stream) {
  const bool bias = s.table || s.slopes;
  auto run = [&](auto cap) {
    constexpr int CAP = decltype(cap)::value;
    return bias ? launch_v<D, CAP, true>(s, qkv, vl, ctx, lse, sh, status, num_sms, stream)
                : launch_v<D, CAP, false>(s, qkv, vl, ctx, lse, sh, status, num_sms, stream);
  };
  return with_cap(s, run);
}

}  // namespace
}  // namespace scored_tc

cudaError_t launch_scored_tc_short(const ScoreArgs& s, const __half* qkv, const int32_t* valid_len, __half* ctx,
                                   float* lse, const ScoredShape& sh, int* status, int num_sms, cudaStream_t stream) {
  using namespace scored_tc;
  switch (sh.size_per_head) {
    case 32: return launch_d<32>(s, qkv, valid_len, ctx, lse, sh, status, num_sms, stream);
    case 64: return launch_d<64>(s, qkv, valid_len, ctx, lse, sh, status, num_sms, stream);
    case 128: return launch_d<128>(s, qkv, valid_len, ctx, lse, sh, status, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace enc
