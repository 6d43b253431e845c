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
// Inside a CTA a row is read by D * sizeof(T) / 16 neighbouring lanes with one
// 16-byte load each.  A lane group takes kU rows of K and the same rows of V at
// a time (2 kU loads in flight), forms the kU scores with shuffles, and keeps a
// running maximum, sum and output (the softmax in one pass); groups, then
// warps, then CTAs are merged at the end.
#include "scored.cuh"
#include "sm100.cuh"

namespace enc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kU = 4;                                      // rows of K and of V in flight per lane group

template <typename T>
struct Vec;                                                // the 16 bytes of a lane as floats
template <>
struct Vec<__half> {
  static constexpr int N = 8;
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
  static __device__ __forceinline__ void widen(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  }
};
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// 2^(m - to), 0 for a part that has seen nothing.
__device__ __forceinline__ float weight2(float m, float to) { return m == -INFINITY ? 0.f : exp2f(m - to); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2)
    scored_step_kernel(const __grid_constant__ ScoreArgs s, const T* __restrict__ qkv, T* __restrict__ cache,
                       const int32_t* __restrict__ len, T* __restrict__ ctx, int B, int C, int NH) {
  constexpr int N = Vec<T>::N;
  constexpr int kLanes = D / N;                            // lanes of a row
  constexpr int kGroups = kThreads / kLanes;
  static_assert(kLanes >= kU && kLanes <= 32, "a lane of the group per score");
  __shared__ float wm[kWarps], wl[kWarps];
  __shared__ __align__(16) float wo[kWarps][D];
  __shared__ float part_o[D], part_ml[2];
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
  float q[N];
  Vec<T>::widen(*reinterpret_cast<const uint4*>(qg + gl * N), q);
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] *= s.scale;
  const float slope = s.slopes ? s.slopes[h] : 0.f;
  const int doc = s.docs && held ? s.docs[(size_t)b * C + p] : 0;

  float m = -INFINITY, l = 0.f, o[N] = {};
  for (int j0 = lo; j0 < hi; j0 += kGroups * kU) {
    uint4 kr[kU], vr[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {                         // position p itself comes from the new token
      const int j = j0 + u * kGroups + group;
      kr[u] = vr[u] = make_uint4(0, 0, 0, 0);
      if (j < hi) {
        const T* k = j == p ? qg + part : kc + (size_t)j * D;
        const T* v = j == p ? qg + 2 * part : vc + (size_t)j * D;
        kr[u] = *reinterpret_cast<const uint4*>(k + gl * N);
        vr[u] = *reinterpret_cast<const uint4*>(v + gl * N);
        if (j == p) {
          *reinterpret_cast<uint4*>(kc + (size_t)j * D + gl * N) = kr[u];
          *reinterpret_cast<uint4*>(vc + (size_t)j * D + gl * N) = vr[u];
        }
      }
    }
    // Lane gl % kU of the group works out the bias and visibility of the group's row gl % kU.
    const int jb = j0 + (gl % kU) * kGroups + group;
    float bias = -INFINITY;
    if (jb < hi && (!s.docs || s.docs[(size_t)b * C + jb] == doc))
      bias = s.table || s.slopes ? score_bias2(s, NH, h, slope, jb - p) : 0.f;
    float t[kU], mx = m;                                   // a row that is not seen has t = -inf
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float kf[N], dot = 0.f;
      Vec<T>::widen(kr[u], kf);
#pragma unroll
      for (int i = 0; i < N; ++i) dot = fmaf(q[i], kf[i], dot);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      if (s.cap > 0.f) dot = s.cap * tanhf(dot / s.cap);
      const float bu = __shfl_sync(0xffffffffu, bias, (lane - gl) + u);
      t[u] = bu == -INFINITY ? -INFINITY : fmaf(dot, kLog2e, bu);
      mx = fmaxf(mx, t[u]);
    }
    const float a = weight2(m, mx);
    m = mx;
    l *= a;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] *= a;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (t[u] == -INFINITY) continue;                     // whatever its V holds
      const float w = exp2f(t[u] - m);
      float vf[N];
      Vec<T>::widen(vr[u], vf);
      l += w;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = fmaf(w, vf[i], o[i]);
    }
  }
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

template <typename T, int D>
cudaError_t step_d(const ScoreArgs& s, const void* qkv, void* cache, const int32_t* len, void* ctx, int ranks,
                   const ScoredShape& sh, cudaStream_t stream) {
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = (unsigned)ranks;
  cluster.val.clusterDim.y = 1;
  cluster.val.clusterDim.z = 1;
  return launch_kernel(scored_step_kernel<T, D>, dim3((unsigned)ranks, sh.head_num, sh.batch), dim3(kThreads), 0,
                       stream, &cluster, 1, s, static_cast<const T*>(qkv), static_cast<T*>(cache), len,
                       static_cast<T*>(ctx), sh.batch, sh.seq, sh.head_num);
}

}  // namespace

cudaError_t launch_scored_step(const ScoreArgs& s, const void* qkv, void* cache, const int32_t* len, void* ctx,
                               const ScoredShape& sh, bool half, int num_sms, cudaStream_t stream) {
  // Enough CTAs for two per SM, each with at least 64 positions of a full cache; 8 is the portable cluster size.
  const long items = (long)sh.batch * sh.head_num;
  int ranks = 1;
  while (ranks < 8 && items * ranks < 2L * num_sms && sh.seq >= 128 * ranks) ranks *= 2;
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
