// Attention with modified scores for one new token per sequence: its key and
// value go into the cache at position p, its query attends to positions 0..p.
//
// The work is one pass over (p + 1) rows of K and of V, with 4 d flops per pair
// of rows, so the cache's bytes bound it; at small batches there are too few
// (sequence, head) pairs to fill the GPU, and the latency of one load chain
// bounds it.  A cluster of C CTAs shares a (sequence, head): CTA r takes the
// r-th part of the p + 1 positions (split by the actual length, not by the
// capacity), and the parts meet in the cluster's shared memory, added in rank
// order: no scratch in memory, no second launch, and the same result on every
// run.
//
// Inside a CTA a row is read by D * sizeof(T) / 16 neighbouring lanes, 16 bytes
// each.  A lane group takes kU rows of K and the same rows of V at a time,
// through a ring of kStages stages in shared memory that cp.async fills: every
// thread reads back only what it asked for itself, so the ring needs no barrier
// and the next stage's loads stay in flight under the arithmetic, with three CTAs
// of 256 threads (32 KB a stage) to an SM.  Measured at 16 heads of 64, 32
// sequences, capacity 4096, caches half to wholly full, with a cap and a table: 87
// us, 92 with a cold L2, 4.4 TB/s of the measured 6.56; the same total in caches of
// one length 79 us, so a third of the gap is the longest caches' clusters, which end
// last.  Two CTAs with three stages took 100 us where this took 85.
// The kU dot products are added up over the group by halving: each exchange
// passes half of the rows on, so that a lane ends with the score of one row and
// bias, cap and exponential are worked out once per row.  The group keeps a
// running maximum, sum and output (the softmax in one pass); groups, then
// warps, then CTAs are merged at the end.
#include "scored.cuh"
#include "sm100.cuh"

namespace enc {
namespace {

constexpr int kU = 4;                                      // rows of K and of V per lane group and stage
constexpr int kStages = 2;
constexpr int kShortCache = 512;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Vec;                                                // the 16 bytes of a lane as floats
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  // 1 - 2 / (1 + 2^(2 x log2 e)) is off by about 2^-22 however small x is, which a cap multiplies (by 2e-3 of a score at
  // a cap of 1e4); small x take the polynomial, so that a score is off by less than 2^-20 of itself at every cap.
  static __device__ __forceinline__ float tanh_of(float x) {
    constexpr TanhSmall fit;
    const float z = x * x;
    float p = fit.c[4];
#pragma unroll
    for (int k = 3; k >= 0; --k) p = fmaf(p, z, fit.c[k]);
    return fabsf(x) <= kTanhSmall ? x * p : 1.f - __fdividef(2.f, 1.f + ex2(x * (2.f * kLog2e)));
  }
  static __device__ __forceinline__ void widen(const uint4& w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float tanh_of(float x) { return tanhf(x); }
  static __device__ __forceinline__ void widen(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  }
};
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// 2^(m - to), 0 for a part that has seen nothing.
__device__ __forceinline__ float weight2(float m, float to) { return m == -INFINITY ? 0.f : ex2(m - to); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool read) {   // zeros where not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
               : "memory");
  return v;
}

template <typename T, int D, int kThreads>
__global__ void __launch_bounds__(kThreads, 768 / kThreads)
    scored_step_kernel(const __grid_constant__ ScoreArgs s, const T* __restrict__ qkv, T* __restrict__ cache,
                       const int32_t* __restrict__ len, T* __restrict__ ctx, int B, int C, int NH) {
  constexpr int N = Vec<T>::N;
  constexpr int kWarps = kThreads / 32, kStageBytes = 2 * kU * kThreads * 16;
  constexpr int kLanes = D / N;                            // lanes of a row
  constexpr int kGroups = kThreads / kLanes;
  static_assert(kU == 4 && kLanes >= kU && kLanes <= 32, "a lane of the group per row");
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float wm[kWarps], wl[kWarps];
  __shared__ __align__(16) float wo[kWarps][D];
  __shared__ float part_o[D], part_ml[2], column[kMaxScoreBuckets];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y, b = blockIdx.z;
  const int rank = blockIdx.x, ranks = gridDim.x;          // the cluster spans the grid's x
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t bh = (size_t)b * NH + h, part = (size_t)B * NH * D;
  const int p = len[b];
  const bool held = p >= 0 && p < C;                       // no room for the token: ctx = 0, the cache stays
  const int keys = held ? p + 1 : 0;
  const int per = (keys + ranks - 1) / ranks;
  const int lo = min(keys, rank * per), hi = min(keys, lo + per);

  const T* qg = qkv + bh * D;
  T* kc = cache + bh * (size_t)C * D;
  T* vc = kc + (size_t)B * NH * C * D;
  const int gl = lane % kLanes, group = tid / kLanes;
  const uint32_t mine = sm100::smem_u32(ring) + tid * 16;
  constexpr int kStep = kGroups * kU;                      // rows of a stage
  auto request = [&](int j0, int stage) {                  // position p itself comes from the new token
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = j0 + u * kGroups + group;
      const bool read = j < hi;
      const T* k = j == p ? qg + part : kc + (size_t)(read ? j : 0) * D;
      const T* v = j == p ? qg + 2 * part : vc + (size_t)(read ? j : 0) * D;
      copy16(mine + stage * kStageBytes + (2 * u) * kThreads * 16, k + gl * N, read);
      copy16(mine + stage * kStageBytes + (2 * u + 1) * kThreads * 16, v + gl * N, read);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int st = 0; st < kStages - 1; ++st) request(lo + st * kStep, st);

  load_column(s, column, NH, h, tid, kThreads);
  float q[N];
  Vec<T>::widen(*reinterpret_cast<const uint4*>(qg + gl * N), q);
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] *= s.scale;
  const float slope = s.slopes ? s.slopes[h] : 0.f;
  const int doc = s.docs && held ? s.docs[(size_t)b * C + p] : 0;
  __syncthreads();

  const float inv_cap = s.cap > 0.f ? 1.f / s.cap : 0.f;
  float m = -INFINITY, l = 0.f, o[N] = {};                 // l: of the rows that this lane scored
  int stage = 0;
  for (int j0 = lo; j0 < hi; j0 += kStep) {
    const int next = stage == 0 ? kStages - 1 : stage - 1;
    request(j0 + (kStages - 1) * kStep, next);             // rows past hi read nothing
    // Bias and visibility of the lane's row, number gl % kU of the group's.
    const int jb = j0 + (gl % kU) * kGroups + group;
    float bias = -INFINITY;
    if (jb < hi && (!s.docs || s.docs[(size_t)b * C + jb] == doc)) {
      bias = -slope * static_cast<float>(p - jb);
      if (s.table) bias += column[score_bucket(s, jb - p)];
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    const uint32_t at = mine + stage * kStageBytes;
    float dot[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint4 kr = shared16(at + (2 * u) * kThreads * 16);
      const int j = j0 + u * kGroups + group;
      if (j == p && j < hi) {                              // (not a later CTA's row past this one's end)
        *reinterpret_cast<uint4*>(kc + (size_t)j * D + gl * N) = kr;
        *reinterpret_cast<uint4*>(vc + (size_t)j * D + gl * N) = shared16(at + (2 * u + 1) * kThreads * 16);
      }
      float kf[N];
      Vec<T>::widen(kr, kf);
      dot[u] = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) dot[u] = fmaf(q[i], kf[i], dot[u]);
    }
    const bool up2 = lane & 2, up1 = lane & 1;
    float k0 = up2 ? dot[2] : dot[0], k1 = up2 ? dot[3] : dot[1];
    k0 += __shfl_xor_sync(0xffffffffu, up2 ? dot[0] : dot[2], 2);
    k1 += __shfl_xor_sync(0xffffffffu, up2 ? dot[1] : dot[3], 2);
    float t = (up1 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, up1 ? k0 : k1, 1);
#pragma unroll
    for (int off = 4; off < kLanes; off <<= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    if (s.cap > 0.f) t = s.cap * Vec<T>::tanh_of(t * inv_cap);
    // A row that is not seen has t = -inf, whatever its K and V hold.
    t = bias == -INFINITY ? -INFINITY : (t + bias) * kLog2e;
    float mx = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
    mx = fmaxf(m, fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)));
    const float a = weight2(m, mx), w = weight2(t, mx);
    m = mx;
    l = fmaf(l, a, w);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] *= a;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float wu = __shfl_sync(0xffffffffu, w, (lane & ~3) | u);
      if (wu == 0.f) continue;
      float vf[N];
      Vec<T>::widen(shared16(at + (2 * u + 1) * kThreads * 16), vf);
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = fmaf(wu, vf[i], o[i]);
    }
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  // Groups of a warp.
#pragma unroll
  for (int off = kLanes; off < 32; off <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, off), mx = fmaxf(m, m2);
    const float a = weight2(m, mx), a2 = weight2(m2, mx);
    l = l * a + __shfl_xor_sync(0xffffffffu, l, off) * a2;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * a + __shfl_xor_sync(0xffffffffu, o[i], off) * a2;
    m = mx;
  }
  if (lane == 0) { wm[warp] = m; wl[warp] = l; }
  if (lane < kLanes)
#pragma unroll
    for (int i = 0; i < N; ++i) wo[warp][gl * N + i] = o[i];
  __syncthreads();
  // Warps of the CTA.
  if (tid < D) {
    float mx = -INFINITY, ls = 0.f, os = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, wm[w]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = weight2(wm[w], mx);
      ls = fmaf(wl[w], a, ls);
      os = fmaf(wo[w][tid], a, os);
    }
    part_o[tid] = os;
    if (tid == 0) { part_ml[0] = mx; part_ml[1] = ls; }
  }
  // CTAs of the cluster.
  sm100::cluster_sync();
  if (rank == 0 && tid < D) {
    float mx = -INFINITY, ls = 0.f, os = 0.f;
    for (int r = 0; r < ranks; ++r)
      mx = fmaxf(mx, sm100::ld_cluster_f32(sm100::mapa_shared(sm100::smem_u32(&part_ml[0]), r)));
    for (int r = 0; r < ranks; ++r) {
      const float a = weight2(sm100::ld_cluster_f32(sm100::mapa_shared(sm100::smem_u32(&part_ml[0]), r)), mx);
      ls = fmaf(sm100::ld_cluster_f32(sm100::mapa_shared(sm100::smem_u32(&part_ml[1]), r)), a, ls);
      os = fmaf(sm100::ld_cluster_f32(sm100::mapa_shared(sm100::smem_u32(&part_o[tid]), r)), a, os);
    }
    put(ctx + bh * D + tid, ls > 0.f ? os / ls : 0.f);
  }
  sm100::cluster_sync();                                   // the parts stay until rank 0 has read them
}

template <typename T, int D, int kThreads>
cudaError_t step_t(const ScoreArgs& s, const void* qkv, void* cache, const int32_t* len, void* ctx, int ranks,
                   const ScoredShape& sh, cudaStream_t stream) {
  constexpr int kBytes = kStages * 2 * kU * kThreads * 16;
  auto kern = scored_step_kernel<T, D, kThreads>;
  static const cudaError_t attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (attr != cudaSuccess) return attr;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = (unsigned)ranks;
  cluster.val.clusterDim.y = 1;
  cluster.val.clusterDim.z = 1;
  return launch_kernel(kern, dim3((unsigned)ranks, sh.head_num, sh.batch), dim3(kThreads), kBytes, stream, &cluster, 1, s, static_cast<const T*>(qkv), static_cast<T*>(cache), len,
                       static_cast<T*>(ctx), sh.batch, sh.seq, sh.head_num);
}

// Short caches leave 256 threads few rows each: 128 threads a CTA, six CTAs an SM (12 heads of 64, 200 sequences,
// capacity 128: 31 -> 23 us); long ones stream better with 256 (16 heads of 64, 32 sequences, 4096: 96 -> 85 us).
template <typename T, int D>
cudaError_t step_d(const ScoreArgs& s, const void* qkv, void* cache, const int32_t* len, void* ctx, int ranks,
                   const ScoredShape& sh, cudaStream_t stream) {
  return sh.seq <= kShortCache ? step_t<T, D, 128>(s, qkv, cache, len, ctx, ranks, sh, stream)
                               : step_t<T, D, 256>(s, qkv, cache, len, ctx, ranks, sh, stream);
}

}  // namespace

cudaError_t launch_scored_step(const ScoreArgs& s, const void* qkv, void* cache, const int32_t* len, void* ctx,
                               const ScoredShape& sh, bool half, int num_sms, cudaStream_t stream) {
  // About four CTAs per SM and more, so that sequences of different lengths even out (with one or two CTAs to an
  // item, 512 items of 4096 took 106 us; with two to four, 85; with eight, 141), but at least 128 positions of a full
  // cache to a CTA; 8 is the portable cluster size.
  const long items = (long)sh.batch * sh.head_num;
  int ranks = 1;
  while (ranks < 8 && items * ranks < 4L * num_sms && sh.seq >= 256 * ranks) ranks *= 2;
  switch (sh.size_per_head) {
    case 32:
      return half ? step_d<__half, 32>(s, qkv, cache, len, ctx, ranks, sh, stream)
                  : step_d<float, 32>(s, qkv, cache, len, ctx, ranks, sh, stream);
    case 64:
      return half ? step_d<__half, 64>(s, qkv, cache, len, ctx, ranks, sh, stream)
                  : step_d<float, 64>(s, qkv, cache, len, ctx, ranks, sh, stream);
    case 128:
      return half ? step_d<__half, 128>(s, qkv, cache, len, ctx, ranks, sh, stream)
                  : step_d<float, 128>(s, qkv, cache, len, ctx, ranks, sh, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace enc
