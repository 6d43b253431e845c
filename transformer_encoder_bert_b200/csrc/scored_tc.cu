// Forward of attention with modified scores on the 5th-generation tensor cores
// (tcgen05 + TMEM + TMA), FP16.
//
// A CTA takes TILES tiles of 128 query rows of one (sequence, head) and walks
// the blocks of BN keys that some row sees.  Warps:
//   TILES x 4   softmax: thread r of a tile owns query row r = TMEM lane r
//   TILES       one thread per tile issues its MMAs
//                 S = Q K^T    M = 128, N = BN, both operands in shared memory
//                 O += P V     M = 128, N = D, K = 16 per step, P read from TMEM
//   1           one thread issues the TMA loads (Q once; K and V through rings)
// A softmax thread reads its whole row of S into registers and releases S, so
// that the next block's S is computed during this block's exponentials; it
// turns the row into t (scale, cap, bias, masks), takes the maximum, writes
// P = 2^(t2 - m + 7) as FP16 to TMEM and adds up l in FP32.  m is a reference
// maximum: it moves only when a block exceeds it by 2^8, and then the thread
// scales its row of O first.  O / l does not depend on m.  The 7 uses up FP16's
// range above 2^8: a weight counts for nothing in O below 2^-32 of the row's
// largest, not already below 2^-25, where 65,536 of them would be a five-hundredth
// of the row.
//
// What bounds a block is the softmax, not the products: 8 cycles of the
// special-function unit a score and warp, and a chain of waits and dependent
// steps around them.  So as many tiles share an SM as TMEM holds: three CTAs of
// one tile for heads up to 64, one CTA of two tiles (which share K and V) for
// heads of 128.
//
// Keys hidden by length, causal or prefix masks are a suffix of the row, so a
// block past every row's limit is not visited and only blocks that a row's limit
// cuts are masked per element.  With documents the CTA first takes the least and
// largest id of every block: blocks whose range does not meet the rows' range
// are not visited, and blocks that hold only the rows' one document are not
// masked.  In a masked block each row's visible keys are a bit set that its
// thread has before S arrives; a warp whose rows see none of the block writes
// P = 0 and leaves it.
//
// Measured, full lengths: 8 heads of 128, 37 sequences of 2048: 731 to 755 us
// between runs, 840 to 870 TF/s (slopes 890, table 805, cap 965 us); 16 heads of 64,
// 37 of 1024: 300 us, 530 TF/s (slopes 385, table 401, cap 450 us), where a block of 64 keys takes the three
// tiles of an SM some 2,600 cycles against 1,536 of exponentials alone: the rest is
// loads from and stores to TMEM, the arithmetic of t and P, and waits.  The document
// mask costs about as much as the blocks that it hides: 16 heads of 64, 32 sequences
// of 256 to 512, four documents each: 82 us against 76 without, 126 against 115 with
// a cap of 30.
#include <cmath>
#include <mutex>

#include <cudaTypedefs.h>

#include "scored_tc.cuh"

namespace enc {
namespace scored_tc {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}
}  // namespace

bool encode_operand_map(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t planes,
                        uint32_t box_cols, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, planes};
  const cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1}, estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr float kRescaleLog2 = 8.f;                // 2^(t2 - m) stays below 2^8 between moves of the reference maximum
constexpr float kRaiseLog2 = 7.f;                  // and P below 2^15

constexpr int BN = 64;                             // keys of a block

template <int D, int TILES>
struct Cfg {
  static constexpr int kCtasPerSm = D > 64 ? 1 : 3;
  static constexpr int kSoftmaxThreads = TILES * 128;
  static constexpr int kMmaWarp = TILES * 4, kTmaWarp = TILES * 5;
  // The MMA and TMA warps are filled up to a warpgroup, whose registers the softmax warps take.
  static constexpr int kThreads = kSoftmaxThreads + 128;
  static constexpr int kRegs = 65536 / kCtasPerSm / kThreads / 8 * 8;          // a thread at launch
  static constexpr int kOtherRegs = D > 64 ? 72 : 40;
  static constexpr int kSoftmaxRegs =
      (kRegs * kThreads - 128 * kOtherRegs) / kSoftmaxThreads / 8 * 8 < 216
          ? (kRegs * kThreads - 128 * kOtherRegs) / kSoftmaxThreads / 8 * 8
          : 216;
  static constexpr int kSub = D > 64 ? D / 64 : 1;         // 64-column sub-tiles of an operand
  static constexpr int kQBytes = kSub * 128 * 128;
  static constexpr int kKVSub = BN * 128;
  static constexpr int kKVBytes = kSub * kKVSub;
  static constexpr int kStages = 3;
  static constexpr int kK = TILES * kQBytes;
  static constexpr int kV = kK + kStages * kKVBytes;
  static constexpr int kBars = kV + kStages * kKVBytes;
  // q_full, k_full, k_empty, v_full, v_empty (kStages each), s_full, s_free, p_full, o_done, drain (TILES each)
  static constexpr int kNumBars = 1 + 4 * kStages + 5 * TILES;
  static constexpr int kSlot = kBars + kNumBars * 8;
  static constexpr int kColumn = (kSlot + 16 + 15) / 16 * 16;          // the head's column of the bias table
  static constexpr int kLut = kColumn + kMaxScoreBuckets * 4;
  // TMEM columns of tile t: S at t * BN, O at kO + t * D, P at kP + t * BN / 2; for heads of 64 P is an allocation
  // of its own, as 128 + 32 columns fit an SM three times where 160 would be rounded up to 256.
  static constexpr bool kOwnP = D == 64;
  static constexpr int kP = kOwnP ? 0 : TILES * BN, kO = kP + (kOwnP ? BN : TILES * BN / 2);
  static constexpr int kTmemUsed = kO + TILES * D;
  static constexpr int kTmemCols = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(!kOwnP || TILES == 1, "one tile");
  static_assert((kTmemCols + (kOwnP ? 32 : 0)) * kCtasPerSm <= 512 && kTmemUsed <= kTmemCols, "TMEM");
  static size_t smem(const ScoreArgs& s, int seq) {
    return 1024 + kLut + (size_t)lut_floats(s, BN) * 4 + (s.docs ? (size_t)(seq + BN - 1) / BN : 0);
  }
};

// One row's block of BN keys: from S in TMEM to P in TMEM, the reference maximum
// and the row's sum.  BIAS 0: none; 1: base; 2: base + step * column; 3: from the
// table in shared memory.  Every variant is a body of its own from the load to the store:
// with the row in registers, each place where two ways of preparing it join costs
// moves of the whole row (when the bodies were split, heads of 64 and 1024 keys, no bias:
// 456 us with branches inside one body, 286 us with a body each).
struct SoftmaxBlock {
  uint32_t t_s, t_p, t_o;   // TMEM addresses of the row's S, P and O
  uint32_t s_free, o_done;  // barriers: S has been read; P V is done
  int it;                   // blocks before this one
  uint64_t scale2, cap2;    // pairs: of the scores; cap log2 e
  float cap_in;
  float base, step;
  const float* lut;         // at column 0
  uint32_t see[BN / 32];    // bits: visible columns
  int keys;                 // columns that are valid keys (any number)
  bool mine;                // the row is a valid query
};

// CAP 0: none; 1: small scores; 2: by polynomial; 3: of any size; 4: that, with a large cap.  x: the row, two scores to a register pair.
template <int D, int CAP, int BIAS, bool MASK>
__device__ __forceinline__ bool softmax_row(const ScoreArgs& s, const SoftmaxBlock& sb, uint64_t (&x)[BN / 2], float& m_ref,
                                            uint64_t& sum2) {
  // t2 of the row: x * mul + bias.
  if constexpr (CAP == 1) {
#pragma unroll
    for (int k = 0; k < BN / 2; ++k) x[k] = small_cap2(s, x[k]);
  } else if constexpr (CAP == 2) {
    const uint64_t in = f2_pack(sb.cap_in, sb.cap_in);
#pragma unroll
    for (int k = 0; k < BN / 2; ++k) {
      const uint64_t y = f2_mul(x[k], in);
      x[k] = f2_mul(y, tanh_over_x2(f2_mul(y, y)));
    }
  } else if constexpr (CAP == 3) {
    const float in2 = 2.f * kLog2e * sb.cap_in;
#pragma unroll
    for (int k = 0; k < BN / 2; ++k) {
      float a, c;
      f2_unpack(x[k], a, c);
      x[k] = f2_pack(tanh_of(a, in2), tanh_of(c, in2));
    }
  } else if constexpr (CAP == 4) {
#pragma unroll
    for (int k = 0; k < BN / 2; ++k) x[k] = tanh_careful2(x[k], sb.cap_in);
  }
  const uint64_t mul = CAP ? sb.cap2 : sb.scale2;
#pragma unroll
  for (int k = 0; k < BN / 2; ++k) {
    if (BIAS == 0) {
      if (CAP != 1) x[k] = f2_mul(x[k], mul);
      continue;
    }
    const uint64_t add =
        BIAS == 1   ? f2_pack(sb.base, sb.base)
        : BIAS == 2 ? f2_pack(fmaf((float)(2 * k), sb.step, sb.base), fmaf((float)(2 * k + 1), sb.step, sb.base))
                    : f2_pack(sb.lut[2 * k], sb.lut[2 * k + 1]);
    x[k] = CAP == 1 ? f2_add(x[k], add) : f2_fma(x[k], mul, add);
  }
  if constexpr (MASK) {
#pragma unroll
    for (int k = 0; k < BN; k += 2) {
      float a, c;
      f2_unpack(x[k / 2], a, c);
      a = sb.see[k / 32] & (1u << k % 32) ? a : -INFINITY;
      c = sb.see[k / 32] & (2u << k % 32) ? c : -INFINITY;
      x[k / 2] = f2_pack(a, c);
    }
  }
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < BN / 2; ++k) {
    float a, c;
    f2_unpack(x[k], a, c);
    m4[k & 3] = fmaxf(fmaxf(m4[k & 3], a), c);
  }
  const float bmax = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));

  // P's columns are free, and O is whole, once the previous P V has completed.
  if (sb.it > 0 && !warp_wait(sb.o_done, (sb.it - 1) & 1)) return false;
  // Until a key has been seen m_ref is -inf, and O and l are zeros.
  const bool moved = bmax > m_ref + kRescaleLog2;
  if (any_warp(moved)) {
    const float alpha = moved ? ex2(raised(kRaiseLog2, bmax) - raised(kRaiseLog2, m_ref)) : 1.f;
    if (moved) m_ref = bmax;
    if (sb.it > 0) {
      tc_fence_after();
      uint32_t oa[32];
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        tmem_ld_32x32b_x32(sb.t_o + c, oa);
#pragma unroll
        for (int k = 0; k < 32; ++k) oa[k] = __float_as_uint(__uint_as_float(oa[k]) * alpha);
        tmem_st_32x32b_x32(sb.t_o + c, oa);
      }
    }
    sum2 = f2_mul(sum2, f2_pack(alpha, alpha));
  }
  const float mu = m_ref == -INFINITY ? 0.f : m_ref;
  const float neg_m = raised(kRaiseLog2, mu);
  const uint64_t neg_m2 = f2_pack(neg_m, neg_m);
#pragma unroll
  for (int c = 0; c < BN; c += 32) {
    uint32_t pk[16];
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      float t0, t1;
      f2_unpack(f2_add(x[(c + k) / 2], neg_m2), t0, t1);
      const float p0 = ex2(t0), p1 = ex2(t1);
      sum2 = f2_add(sum2, f2_pack(p0, p1));
      pk[k / 2] = half2_of(p0, p1);
    }
    tmem_st_32x32b_x16_async(sb.t_p + c / 2, pk);
  }
  return true;
}

template <int D, int CAP, int BIAS, bool MASK>
__device__ __forceinline__ bool softmax_block(const ScoreArgs& s, const SoftmaxBlock& sb, int lane, float& m_ref, uint64_t& sum2) {
  uint64_t x[BN / 2];
  {
    uint32_t sv[BN / 32][32];
#pragma unroll
    for (int c = 0; c < BN / 32; ++c) tmem_ld_32x32b_x32_async(sb.t_s + 32 * c, sv[c]);
#pragma unroll
    for (int c = 0; c < BN / 32; ++c) tmem_wait_ld(sv[c]);
#pragma unroll
    for (int k = 0; k < BN; k += 2)
      x[k / 2] = f2_pack(__uint_as_float(sv[k / 32][k % 32]), __uint_as_float(sv[k / 32][k % 32 + 1]));
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(sb.s_free);
  if constexpr (CAP == kNoCap) {
    return softmax_row<D, 0, BIAS, MASK>(s, sb, x, m_ref, sum2);
  } else {
    float top = 0.f;                                       // (of valid rows and keys, so that no other decides)
    if (MASK && sb.keys < BN) {
#pragma unroll
      for (int k = 0; k < BN / 2; ++k) {
        float a, c;
        f2_unpack(x[k], a, c);
        top = fmaxf(fmaxf(top, 2 * k < sb.keys ? fabsf(a) : 0.f), 2 * k + 1 < sb.keys ? fabsf(c) : 0.f);
      }
    } else {
      float t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < BN / 2; ++k) {
        float a, c;
        f2_unpack(x[k], a, c);
        t4[k & 3] = fmaxf(fmaxf(t4[k & 3], fabsf(a)), fabsf(c));
      }
      top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
    }
    if (!any_warp(sb.mine && top > s.cap_small_top)) return softmax_row<D, 1, BIAS, MASK>(s, sb, x, m_ref, sum2);
    if (!any_warp(sb.mine && top * fabsf(sb.cap_in) > kCapPoly))
      return softmax_row<D, 2, BIAS, MASK>(s, sb, x, m_ref, sum2);
    return softmax_row<D, CAP == kLargeCap ? 4 : 3, BIAS, MASK>(s, sb, x, m_ref, sum2);
  }
}

// The same for a warp none of whose rows sees the block: P = 0, and nothing else changes.
__device__ __forceinline__ bool hidden_block(const SoftmaxBlock& sb, int lane) {
  if (lane == 0) mbar_arrive(sb.s_free);
  if (sb.it > 0 && !warp_wait(sb.o_done, (sb.it - 1) & 1)) return false;
  uint32_t zero[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) zero[k] = 0;
#pragma unroll
  for (int c = 0; c < BN; c += 32) tmem_st_32x32b_x16_async(sb.t_p + c / 2, zero);
  return true;
}

// BIAS 0: none; 1: a table; 2: slopes, with or without a table.
template <int D, int TILES, int CAP, int BIAS>
__global__ void __launch_bounds__(Cfg<D, TILES>::kThreads, Cfg<D, TILES>::kCtasPerSm)
    scored_tc_kernel(const __grid_constant__ ScoreArgs s, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_ctx,
                     const int32_t* __restrict__ valid_len, __half* __restrict__ ctx, float* __restrict__ lse, int B,
                     int S, int NH, int* __restrict__ status) {
  using C = Cfg<D, TILES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBars;
  const uint32_t q_full = bar0;
  auto k_full = [&](int st) { return bar0 + 8 + 8 * st; };
  auto k_empty = [&](int st) { return bar0 + 8 + 8 * (C::kStages + st); };
  auto v_full = [&](int st) { return bar0 + 8 + 8 * (2 * C::kStages + st); };
  auto v_empty = [&](int st) { return bar0 + 8 + 8 * (3 * C::kStages + st); };
  const uint32_t tile_bars = bar0 + 8 + 32 * C::kStages;
  auto s_full = [&](int t) { return tile_bars + 8 * t; };
  auto s_free = [&](int t) { return tile_bars + 8 * (TILES + t); };
  auto p_full = [&](int t) { return tile_bars + 8 * (2 * TILES + t); };
  auto o_done = [&](int t) { return tile_bars + 8 * (3 * TILES + t); };
  auto drain = [&](int t) { return tile_bars + 8 * (4 * TILES + t); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kSlot);
  float* column = reinterpret_cast<float*>(smem + C::kColumn);
  float* lut = reinterpret_cast<float*>(smem + C::kLut);
  uint8_t* cls = reinterpret_cast<uint8_t*>(lut + lut_floats(s, BN));   // documents: 0 skip, 1 whole, 2 mask per element

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int q0 = (gridDim.x - 1 - blockIdx.x) * (128 * TILES);          // long causal rows first
  const int H = NH * D;
  pdl_wait();
  const int n = score_len(valid_len, b, S), prefix = score_prefix(s, b);
  if (q0 >= n) {                                           // no query here: ctx = 0, lse = -inf
    const int rows = min(128 * TILES, S - q0);
    for (int k = tid; k < rows * (D / 8); k += C::kThreads)
      *reinterpret_cast<uint4*>(ctx + ((size_t)b * S + q0 + k / (D / 8)) * H + h * D + (k % (D / 8)) * 8) =
          make_uint4(0, 0, 0, 0);
    if (lse)
      for (int k = tid; k < rows; k += C::kThreads) lse[((size_t)b * NH + h) * S + q0 + k] = -INFINITY;
    return;
  }
  // Keys that the last row of tile t sees (its blocks: [0, nb[t])).
  int klim[TILES], nb[TILES], nbmax = 0;
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    const int first = q0 + 128 * t, last = min(first + 127, n - 1);
    klim[t] = first < n ? score_jlim(s, last, n, prefix) : 0;
    nb[t] = (klim[t] + BN - 1) / BN;
    nbmax = max(nbmax, nb[t]);
  }

  if (tid == 0) {
    for (int k = 0; k < C::kNumBars; ++k) mbar_init(bar0 + 8 * k, 1);
    for (int t = 0; t < TILES; ++t) {
      mbar_init(s_free(t), 4);
      mbar_init(p_full(t), 4);
    }
    for (int st = 0; st < C::kStages; ++st) {
      mbar_init(k_empty(st), TILES);
      mbar_init(v_empty(st), TILES);
    }
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    if constexpr (C::kOwnP) tmem_alloc(smem_u32(tmem_slot) + 4, 32);
    tmem_relinquish();
  }
  const int32_t* docs = s.docs ? s.docs + (size_t)b * S : nullptr;
  if (docs) {                                              // one warp per block of keys
    const int rows_end = min(q0 + 128 * TILES, n);
    int rlo = INT32_MAX, rhi = INT32_MIN;
    for (int k = q0 + lane; k < rows_end; k += 32) {
      const int v = docs[k];
      rlo = min(rlo, v);
      rhi = max(rhi, v);
    }
    rlo = __reduce_min_sync(0xffffffffu, rlo);
    rhi = __reduce_max_sync(0xffffffffu, rhi);
    for (int jb = warp; jb < nbmax; jb += C::kThreads / 32) {
      int lo = INT32_MAX, hi = INT32_MIN;
#pragma unroll
      for (int c = 0; c < BN; c += 32) {
        const int j = jb * BN + c + lane;
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
  const uint32_t tmem = uniform(tmem_slot[0]), tmem_p = C::kOwnP ? uniform(tmem_slot[1]) : tmem + C::kP;
  pdl_trigger();                                           // after taking TMEM
  auto next_block = [&](int jb) {                          // first block at or after jb that is visited
    if (docs)
      while (jb < nbmax && cls[jb] == 0) ++jb;
    return jb;
  };

  bool ok = true;
  if (warp >= TILES * 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == C::kTmaWarp && lane == 0) {                // TMA
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_kv);
      const int bh = b * NH + h, plane = B * NH;
      mbar_arrive_expect_tx(q_full, TILES * C::kQBytes);
      for (int t = 0; t < TILES; ++t)
        for (int u = 0; u < C::kSub; ++u)
          tma_load_3d(&tm_q, sbase + t * C::kQBytes + u * 16384, q_full, 64 * u, q0 + 128 * t, bh);
      int it = 0;
      for (int jb = next_block(0); jb < nbmax; jb = next_block(jb + 1), ++it) {
        const int st = it % C::kStages;
        const uint32_t ph = ((it / C::kStages) & 1) ^ 1;
        if (it >= C::kStages && !(ok = one_wait(k_empty(st), ph))) break;
        mbar_arrive_expect_tx(k_full(st), C::kKVBytes);
        for (int u = 0; u < C::kSub; ++u)
          tma_load_3d(&tm_kv, sbase + C::kK + st * C::kKVBytes + u * C::kKVSub, k_full(st), 64 * u, jb * BN, plane + bh);
        if (it >= C::kStages && !(ok = one_wait(v_empty(st), ph))) {
          one_wait(k_full(st), ph ^ 1);
          break;
        }
        mbar_arrive_expect_tx(v_full(st), C::kKVBytes);
        for (int u = 0; u < C::kSub; ++u)
          tma_load_3d(&tm_kv, sbase + C::kV + st * C::kKVBytes + u * C::kKVSub, v_full(st), 64 * u, jb * BN,
                      2 * plane + bh);
      }
      // Every load has landed before the CTA exits.
      one_wait(q_full, 0);
      for (int k = it > C::kStages ? it - C::kStages : 0; k < it; ++k) {
        one_wait(k_full(k % C::kStages), (k / C::kStages) & 1);
        one_wait(v_full(k % C::kStages), (k / C::kStages) & 1);
      }
    } else if (warp < C::kTmaWarp) {                       // MMA of tile t
      const int t = warp - C::kMmaWarp;
      int nbt = nb[0];
      if (TILES > 1 && t > 0) nbt = nb[TILES - 1];
      const int kl = TILES > 1 && t > 0 ? klim[TILES - 1] : klim[0];
      constexpr uint32_t idesc_s = idesc_f16_f32(128, BN);
      constexpr uint32_t idesc_o = idesc_bmn(128, D);
      const uint64_t q_desc = smem_desc_sw128(sbase + t * C::kQBytes), k_desc = smem_desc_sw128(sbase + C::kK);
      const uint64_t v_desc = desc_mn_sw128(sbase + C::kV, C::kKVSub);
      const uint32_t t_s = tmem + t * BN, t_p = tmem_p + t * (BN / 2), t_o = tmem + C::kO + t * D;
      // Waits for K of block number `it` and for S's columns to have been read, then issues S; a tile that is past its last block only releases.
      auto scores = [&](int it, int st, bool active) {
        if (!warp_wait(k_full(st), (it / C::kStages) & 1)) return false;
        if (!active) {
          if (elect_one()) mbar_arrive(k_empty(st));
          return true;
        }
        if (it > 0 && !warp_wait(s_free(t), (it - 1) & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t k_st = desc_at(k_desc, st * C::kKVBytes);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t u = kk / 4, o = (kk % 4) * 32;
            mma_f16_ss(t_s, desc_at(q_desc, u * 16384 + o), desc_at(k_st, u * C::kKVSub + o), idesc_s, kk > 0 ? 1u : 0u);
          }
          mma_commit(s_full(t));
          mma_commit(k_empty(st));
        }
        __syncwarp();
        return true;
      };
      int jb = next_block(0), st = 0;
      ok = warp_wait(q_full, 0) && scores(0, 0, jb < nbt);
      for (int it = 0; ok && jb < nbmax; ++it) {
        const int nxt = next_block(jb + 1), st_next = st + 1 == C::kStages ? 0 : st + 1;
        if (nxt < nbmax && !(ok = scores(it + 1, st_next, nxt < nbt))) break;
        if (!(ok = warp_wait(v_full(st), (it / C::kStages) & 1))) break;
        if (jb < nbt) {
          if (!(ok = warp_wait(p_full(t), it & 1))) break;
          tc_fence_after();
          const int keys = kl - jb * BN;
          if (elect_one()) {
            const uint64_t v_st = desc_at(v_desc, st * C::kKVBytes);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              if (16 * kk < keys)
                mma_f16_ts(t_o, t_p + 8 * kk, desc_at(v_st, kk * 2048), idesc_o, it > 0 || kk > 0 ? 1u : 0u);
            mma_commit(o_done(t));
            mma_commit(v_empty(st));
          }
          __syncwarp();
        } else if (elect_one()) {
          mbar_arrive(v_empty(st));
        }
        jb = nxt;
        st = st_next;
      }
      if (elect_one()) mma_commit(drain(t));               // every MMA issued here has completed
      __syncwarp();
      warp_wait(drain(t), 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;   // tile, row of the tile = TMEM lane
    const int i = q0 + 128 * t + r;
    const uint32_t lane_bits = static_cast<uint32_t>((warp & 3) * 32) << 16, t_lane = tmem + lane_bits;
    const uint32_t t_s = t_lane + t * BN, t_p = tmem_p + lane_bits + t * (BN / 2), t_o = t_lane + C::kO + t * D;
    const Bias bias = make_bias(s, column, lut, NH, h, BN, -min(q0 + 128 * TILES - 1, n - 1), nbmax * BN - 1 - q0, tid,
                                C::kSoftmaxThreads);
    const Cap cap = make_cap(s);
    const int jlim = i < n ? score_jlim(s, i, n, prefix) : 0;
    const int i_first = q0 + 128 * t, i_last = i_first + 127;
    // Keys that every valid row of the tile sees (as far as length and causality go).
    const int jall = i_first < n ? score_jlim(s, i_first, n, prefix) : 0;
    SoftmaxBlock sb;
    sb.t_s = t_s;
    sb.t_p = t_p;
    sb.t_o = t_o;
    sb.s_free = s_free(t);
    sb.o_done = o_done(t);
    sb.scale2 = f2_pack(s.scale * kLog2e, s.scale * kLog2e);
    sb.cap2 = f2_pack(cap.cap2, cap.cap2);
    sb.cap_in = cap.in;
    sb.mine = i < n;
    const int doc = docs && i < n ? docs[i] : 0;
    float m_ref = -INFINITY;
    uint64_t sum2 = 0;                                     // two partial row sums (0.0f, 0.0f)
    const int nb_mine = TILES == 2 && t == 1 ? nb[TILES - 1] : nb[0];
    int it = 0;
    for (int jb = next_block(0); jb < nb_mine; jb = next_block(jb + 1), ++it) {
      const int j0 = jb * BN;
      // The row's visible keys.  Documents: each id that the warp's rows hold, against the block's keys.
      const bool by_doc = docs && cls[jb] == 2;
      bool mask = j0 + BN > jall || by_doc, hidden = false;
      if (mask) {
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) {
          const int lim = jlim - j0 - 32 * c;
          sb.see[c] = lim >= 32 ? ~0u : lim <= 0 ? 0u : (1u << lim) - 1;
        }
        if (by_doc) {
          int dj[BN / 32];
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) {
            const int j = j0 + 32 * c + lane;
            dj[c] = j < n ? docs[j] : 0;
          }
          uint32_t left = __ballot_sync(0xffffffffu, sb.mine);
          while (left) {
            const int d = __shfl_sync(0xffffffffu, doc, __ffs(left) - 1);
            const bool same = doc == d;
            left &= ~__ballot_sync(0xffffffffu, same);
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
              const uint32_t eq = __ballot_sync(0xffffffffu, dj[c] == d);
              if (same) sb.see[c] &= eq;
            }
          }
        }
        hidden = !any_warp(sb.mine && (sb.see[0] | sb.see[BN / 32 - 1]) != 0);
        mask = any_warp(sb.mine && (sb.see[0] & sb.see[BN / 32 - 1]) != ~0u);
      }
      if (!(ok = warp_wait(s_full(t), it & 1))) break;
      tc_fence_after();
      // How the block is biased.
      sb.it = it;
      const bool near = BIAS && j0 - i_last < bias.reach && j0 + BN - 1 - i_first > -bias.reach;
      const bool ahead = j0 - i_last >= bias.reach;
      sb.step = ahead ? -bias.slope2 : bias.slope2;
      sb.base = (ahead ? bias.right : bias.left) + sb.step * (float)(j0 - i);
      sb.lut = bias.lut + bias.off + (j0 - i);
      sb.keys = n - j0;
      if (hidden)
        ok = hidden_block(sb, lane);
      else if (BIAS && near)
        ok = mask ? softmax_block<D, CAP, BIAS ? 3 : 0, true>(s, sb, lane, m_ref, sum2)
                  : softmax_block<D, CAP, BIAS ? 3 : 0, false>(s, sb, lane, m_ref, sum2);
      else
        ok = mask ? softmax_block<D, CAP, BIAS, true>(s, sb, lane, m_ref, sum2)
                  : softmax_block<D, CAP, BIAS, false>(s, sb, lane, m_ref, sum2);
      if (!ok) break;
      // V rows of keys in [n, n rounded up to 16) are read by P V: zeros, whatever memory holds there.
      const int lim = n - j0, lim16 = (min(BN, klim[t] - j0) + 15) & ~15;
      if (lim < lim16 && (warp & 3) == 0) {
        const int st = it % C::kStages;
        if (!(ok = warp_wait(v_full(st), (it / C::kStages) & 1))) break;
        for (int k = lane; k < (lim16 - lim) * 8 * C::kSub; k += 32) {
          const int u = k / ((lim16 - lim) * 8), rr = lim + k % ((lim16 - lim) * 8) / 8;
          *reinterpret_cast<uint4*>(smem + C::kV + st * C::kKVBytes + u * C::kKVSub + rr * 128 + (k % 8) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();                          // visible to the tensor core
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(t));
    }
    if (ok && it > 0) ok = warp_wait(o_done(t), (it - 1) & 1);
    if (ok && i_first < S) {
      tc_fence_after();
      float s0, s1;
      f2_unpack(sum2, s0, s1);
      const float l = s0 + s1;
      const bool seen = it > 0 && i < n && l > 0.f;        // (rows i >= n may have been computed from anything)
      const float inv = seen ? 1.f / l : 0.f;
      // The row as FP16 into the Q tile (its readers, the MMAs of S, have completed), swizzled as the
      // store's box is; then one TMA store per 64 columns of the warp's 32 rows.
      constexpr int kCols = D < 64 ? D : 64, kRowBytes = 2 * kCols;
      if (it == 0) one_wait(q_full, 0);     // no MMA read Q: its load must have landed
      uint8_t* out = smem + t * C::kQBytes;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t oa[32];
        if (it > 0) tmem_ld_32x32b_x32(t_o + c, oa);
        uint8_t* orow = out + (c / 64) * 16384 + (warp & 3) * 32 * kRowBytes + lane * kRowBytes;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = seen ? half2_of(__uint_as_float(oa[8 * u + 2 * k]) * inv, __uint_as_float(oa[8 * u + 2 * k + 1]) * inv)
                        : 0u;
          const int unit = (c % 64) / 8 + u;
          const int sw = D < 64 ? unit ^ ((lane >> 1) & 3) : unit ^ (lane & 7);
          *reinterpret_cast<uint4*>(orow + 16 * sw) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      const int row0 = i_first + (warp & 3) * 32;
      if (lane == 0 && row0 < S) {                         // rows at or past S are outside the map
        for (int u = 0; u < C::kSub; ++u)
          tma_store_3d(&tm_ctx, smem_u32(out) + u * 16384 + (warp & 3) * 32 * kRowBytes, h * D + 64 * u, row0, b);
        bulk_commit_group();
      }
      if (lse && i < S) lse[((size_t)b * NH + h) * S + i] = seen ? (log2f(l) - raised(kRaiseLog2, m_ref)) * kLn2 : -INFINITY;
      if (lane == 0) bulk_wait_group_read<0>();            // shared memory has been read
    }
  }

  if (!ok) atomicCAS(status, 0, kStatusWaitTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
    if constexpr (C::kOwnP) tmem_dealloc(tmem_p, 32);
  }
}

template <int D, int TILES, int CAP, int BIAS>
cudaError_t launch_v(const ScoreArgs& s, const __half* qkv, const int32_t* vl, __half* ctx, float* lse,
                     const ScoredShape& sh, int* status, cudaStream_t stream) {
  using C = Cfg<D, TILES>;
  static const cudaError_t attr = cudaFuncSetAttribute(scored_tc_kernel<D, TILES, CAP, BIAS>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (attr != cudaSuccess) return attr;
  const uint64_t planes = 3ull * sh.batch * sh.head_num;
  CUtensorMap tq, tkv, tc;
  if (!encode_operand_map(&tq, qkv, D, sh.seq, planes, 64, 128) ||
      !encode_operand_map(&tkv, qkv, D, sh.seq, planes, 64, BN) ||
      !encode_operand_map(&tc, ctx, (uint64_t)sh.head_num * D, sh.seq, sh.batch, D < 64 ? D : 64, 32))
    return cudaErrorInvalidValue;
  const dim3 grid((sh.seq + 128 * TILES - 1) / (128 * TILES), sh.head_num, sh.batch);
  return launch_kernel(scored_tc_kernel<D, TILES, CAP, BIAS>, grid, dim3(C::kThreads), C::smem(s, sh.seq), stream,
                       nullptr, 0, s, tq, tkv, tc, vl, ctx, lse, sh.batch, sh.seq, sh.head_num, status);
}

template <int D, int TILES>
cudaError_t launch_d(const ScoreArgs& s, const __half* qkv, const int32_t* vl, __half* ctx, float* lse,
                     const ScoredShape& sh, int* status, cudaStream_t stream) {
  auto run = [&](auto cap) {
    constexpr int CAP = decltype(cap)::value;
    return s.slopes  ? launch_v<D, TILES, CAP, 2>(s, qkv, vl, ctx, lse, sh, status, stream)
           : s.table ? launch_v<D, TILES, CAP, 1>(s, qkv, vl, ctx, lse, sh, status, stream)
                     : launch_v<D, TILES, CAP, 0>(s, qkv, vl, ctx, lse, sh, status, stream);
  };
  return with_cap(s, run);
}

}  // namespace
}  // namespace scored_tc

// TanhSmall's coefficients with x = in q.k: multiplied by in^(2k + 1) cap2.
// Beyond the factors here a coefficient could leave FP32's range, and no score takes this form.
void fold_cap(ScoreArgs* s) {
  constexpr TanhSmall fit;
  const double in = (double)s->scale / s->cap;
  s->cap_small_top = -1.f;
  if (!(s->cap > 0.f) || !(fabs(in) >= 1e-4 && fabs(in) <= 1e4)) return;
  double f = in * s->cap * 1.4426950408889634;
  for (int k = 0; k < 5; ++k, f *= in * in) s->cap_small[k] = (float)(fit.c[k] * f);
  s->cap_small_top = (float)(kTanhSmall / fabs(in));
}

cudaError_t launch_scored_tc(const ScoreArgs& s, const __half* qkv, const int32_t* valid_len, __half* ctx, float* lse,
                             const ScoredShape& sh, int* status, cudaStream_t stream) {
  using namespace scored_tc;
  switch (sh.size_per_head) {
    case 32: return launch_d<32, 1>(s, qkv, valid_len, ctx, lse, sh, status, stream);
    case 64: return launch_d<64, 1>(s, qkv, valid_len, ctx, lse, sh, status, stream);
    case 128: return launch_d<128, 2>(s, qkv, valid_len, ctx, lse, sh, status, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace enc
