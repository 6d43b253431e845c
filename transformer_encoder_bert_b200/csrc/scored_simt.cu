// Attention with modified scores on the CUDA cores: forward, and backward in
// two passes (dQ and the table's gradient with the queries fixed, then dK and
// dV with the keys fixed).  FP32 mode runs these kernels; FP16 runs them where
// the tensor-core kernels are switched off.  Everything is computed in FP32.
//
// Every pass works on tiles of 64 x 64 scores with 256 threads: thread
// (ty, tx) = (tid / 16, tid % 16) owns scores of rows 4 ty .. 4 ty + 3 and
// columns tx + 16 c.  Operand tiles lie in shared memory with rows of D + 4
// floats, which makes the float4 reads of 8 consecutive rows hit all 32 banks;
// a dot-product step of 4 elements costs a thread 8 float4 reads for 64 FMAs.
// The second products (P V, dS K, ...) read the score tile back from shared
// memory, 4 columns at a time.  Rows of a tile at or past the valid length are
// zeros, whatever memory holds there.
//
// The backward pass computes the scores twice instead of adding to dQ with
// atomics, so that its results do not depend on the order of the blocks.
//
// Bound by shared memory: a step of 64 FMAs reads 8 float4 (and the second
// products as many), and short sequences by the latency of a block's few tiles.
// Measured, FP32, 12 heads of 64, 8 sequences of 256 to 512: forward 165 us, 23 TF/s
// of the visible pairs' products (table 194 us), backward 444 us, 21 TF/s (table 583
// us).  Tiles are copied under the arithmetic of the ones before (forward 186,
// backward 549 us without), a last tile of at most 16 columns forms those alone (4
// heads of 32, 16 sequences of up to 131, a table: forward 22.6 -> 20.3 us), and the
// dK/dV grid runs beside the dQ grid (the same sequences' backward 63.5 -> 44.0 us).
#include "scored.cuh"

namespace enc {
namespace {

constexpr int kT = 64;                 // rows and columns of a tile
constexpr int kThreads = 256;
constexpr int kPs = kT + 4;            // row stride of the score tile

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// Rows [row0, row0 + 64) of a [rows, stride] operand into shared memory; rows at or past `rows` are zeros.  FP32
// copies are asynchronous (one group; wait_copies), so that the next tile loads under this one's arithmetic.
template <typename T, int D>
__device__ __forceinline__ void load_tile(float* dst, const T* src, int row0, int rows, size_t stride) {
  for (int i = threadIdx.x; i < kT * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    const bool read = row0 + r < rows;
    if constexpr (sizeof(T) == 4) {
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * (D + 4) + c));
      const T* from = src + (read ? (size_t)(row0 + r) * stride + c : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(read ? 16 : 0) : "memory");
    } else {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (read) v = load4<T>(src + (size_t)(row0 + r) * stride + c);
      *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = v;
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the last N tiles asked for by this thread have arrived (a barrier makes the others' visible).
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// acc[a][c] = A[4 ty + a] . B[tx + 16 c] for c < N; zeros past that.
template <int D, int N>
__device__ __forceinline__ void dot_columns(const float* A, const float* B, float (&acc)[4][4]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = 0.f;
#pragma unroll 4
  for (int k = 0; k < D; k += 4) {
    float4 x[4], y[N];
#pragma unroll
    for (int a = 0; a < 4; ++a) x[a] = *reinterpret_cast<const float4*>(A + (4 * ty + a) * (D + 4) + k);
#pragma unroll
    for (int c = 0; c < N; ++c) y[c] = *reinterpret_cast<const float4*>(B + (tx + 16 * c) * (D + 4) + k);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < N; ++c) {
        acc[a][c] = fmaf(x[a].x, y[c].x, acc[a][c]);
        acc[a][c] = fmaf(x[a].y, y[c].y, acc[a][c]);
        acc[a][c] = fmaf(x[a].z, y[c].z, acc[a][c]);
        acc[a][c] = fmaf(x[a].w, y[c].w, acc[a][c]);
      }
  }
}
// The same for the first `live` columns of a tile (the others are hidden; a last tile of at most 16 is common).
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int live, float (&acc)[4][4]) {
  if (live <= 16)
    dot_columns<D, 1>(A, B, acc);
  else
    dot_columns<D, 4>(A, B, acc);
}

// Column of a thread's e-th output element (D / 16 of them).
template <int D>
__device__ __forceinline__ int out_col(int e) {
  const int tx = threadIdx.x & 15;
  return D == 32 ? tx * 2 + e : (e / 4) * 64 + tx * 4 + e % 4;
}

// out[a][e] += sum over k < live of P[4 ty + a][k] B[k][out_col(e)] (P = 0 from there to a multiple of 4)
template <int D>
__device__ __forceinline__ void accumulate(const float* P, const float* B, int live, float (&out)[4][D / 16]) {
  const int ty = threadIdx.x >> 4;
#pragma unroll 2
  for (int k = 0; k < live; k += 4) {
    float p[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float4 v = *reinterpret_cast<const float4*>(P + (4 * ty + a) * kPs + k);
      p[a][0] = v.x; p[a][1] = v.y; p[a][2] = v.z; p[a][3] = v.w;
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      float b[D / 16];
      const float* row = B + (k + kk) * (D + 4);
      if constexpr (D == 32) {
        const float2 v = *reinterpret_cast<const float2*>(row + out_col<D>(0));
        b[0] = v.x; b[1] = v.y;
      } else {
#pragma unroll
        for (int e = 0; e < D / 16; e += 4) {
          const float4 v = *reinterpret_cast<const float4*>(row + out_col<D>(e));
          b[e] = v.x; b[e + 1] = v.y; b[e + 2] = v.z; b[e + 3] = v.w;
        }
      }
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) out[a][e] = fmaf(p[a][kk], b[e], out[a][e]);
    }
  }
}

// The biases of the 127 distances of a tile (rel = rel0 + index - 63) and the
// documents of its rows and columns.
struct TileInfo {
  float bias2[2 * kT], column[kMaxScoreBuckets];
  int row_doc[kT], col_doc[kT];
};

__device__ __forceinline__ void fill_bias(TileInfo* ti, const ScoreArgs& s, float slope, int rel0) {
  if (threadIdx.x < 2 * kT - 1)
    ti->bias2[threadIdx.x] =
        s.table || s.slopes ? score_bias2(s, ti->column, slope, rel0 + (int)threadIdx.x - (kT - 1)) : 0.f;
}

__device__ __forceinline__ void fill_docs(int* dst, const ScoreArgs& s, int b, int S, int pos0) {
  const int t = threadIdx.x;
  if (s.docs && t < kT) dst[t] = pos0 + t < S ? s.docs[(size_t)b * S + pos0 + t] : 0;
}

// u in units of log2, and 1 - tanh^2 (1 without a cap).
__device__ __forceinline__ float capped2(const ScoreArgs& s, float inv_cap, float dot, float& slope) {
  const float u = dot * s.scale;
  slope = 1.f;
  if (s.cap <= 0.f) return u * kLog2e;
  const float x = u * inv_cap, th = tanhf(x);
  slope = fmaf(-th, th, 1.f);
  if (fabsf(th) > 0.75f) {               // near 1 that difference loses its digits: from E = e^(-2 |x|)
    const float e = exp2f(fabsf(x) * (-2.f * kLog2e)), r = 1.f / (1.f + e);
    slope = 4.f * e * r * r;
  }
  return s.cap * th * kLog2e;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    scored_fwd_kernel(const __grid_constant__ ScoreArgs s, const T* __restrict__ qkv,
                      const int32_t* __restrict__ valid_len, T* __restrict__ ctx, float* __restrict__ lse, int B, int S,
                      int NH) {
  extern __shared__ __align__(16) float smem[];
  float* Qs = smem;
  float* Ks = Qs + kT * (D + 4);
  float* Vs = Ks + kT * (D + 4);
  float* Ps = Vs + kT * (D + 4);
  TileInfo* ti = reinterpret_cast<TileInfo*>(Ps + kT * kPs);
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, h = blockIdx.y, q0 = (gridDim.x - 1 - blockIdx.x) * kT;   // long causal rows first
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = score_len(valid_len, b, S), prefix = score_prefix(s, b);
  const size_t head = (size_t)S * D, part = (size_t)B * NH * head;
  const T* Qg = qkv + ((size_t)b * NH + h) * head;
  const float slope = s.slopes ? s.slopes[h] : 0.f, inv_cap = s.cap > 0.f ? 1.f / s.cap : 0.f;
  float out[4][D / 16] = {};
  float m[4], l[4] = {};
  for (int a = 0; a < 4; ++a) m[a] = -INFINITY;
  const int rows = min(kT, n - q0);      // valid queries of the tile
  const int klim = rows > 0 ? score_jlim(s, q0 + rows - 1, n, prefix) : 0;
  load_tile<T, D>(Qs, Qg, q0, n, D);
  load_tile<T, D>(Ks, Qg + part, 0, n, D);
  load_tile<T, D>(Vs, Qg + 2 * part, 0, n, D);
  fill_docs(ti->row_doc, s, b, S, q0);
  load_column(s, ti->column, NH, h, threadIdx.x, kThreads);
  __syncthreads();
  for (int j0 = 0; j0 < klim; j0 += kT) {
    fill_bias(ti, s, slope, j0 - q0);
    fill_docs(ti->col_doc, s, b, S, j0);
    wait_copies<1>();
    __syncthreads();
    const int live = min(kT, klim - j0);
    float acc[4][4];
    dot_tile<D>(Qs, Ks, live, acc);
    __syncthreads();
    load_tile<T, D>(Ks, Qg + part, j0 + kT, n, D);         // the next tile's, under the softmax
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = 4 * ty + a, i = q0 + r;
      const int jlim = i < n ? score_jlim(s, i, n, prefix) : 0;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c, j = j0 + col;
        float unused;
        const float t = capped2(s, inv_cap, acc[a][c], unused) + ti->bias2[col - r + kT - 1];
        acc[a][c] = j < jlim && (!s.docs || ti->row_doc[r] == ti->col_doc[col]) ? t : -INFINITY;
        mx = fmaxf(mx, acc[a][c]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[a], mx), mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m[a] - mu);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = exp2f(acc[a][c] - mu);
        sum += p;
        Ps[r * kPs + tx + 16 * c] = p;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[a] = l[a] * alpha + sum;
      m[a] = mn;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) out[a][e] *= alpha;
    }
    wait_copies<1>();
    __syncthreads();
    accumulate<D>(Ps, Vs, live, out);
    __syncthreads();
    load_tile<T, D>(Vs, Qg + 2 * part, j0 + kT, n, D);
  }
  wait_copies<0>();
  const int H = NH * D;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = q0 + 4 * ty + a;
    if (i >= S) continue;
    const float inv = l[a] > 0.f ? 1.f / l[a] : 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) put(ctx + ((size_t)b * S + i) * H + h * D + out_col<D>(e), out[a][e] * inv);
    if (lse && tx == 0) lse[((size_t)b * NH + h) * S + i] = l[a] > 0.f ? (m[a] + log2f(l[a])) * kLn2 : -INFINITY;
  }
}

// dT of one score: p (dP - D); t2 is masked to -inf where the key is not
// visible.  lse2 = +inf marks a row that sees nothing.
__device__ __forceinline__ float prob2(float t2, float lse2) { return exp2f(t2 - lse2); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    scored_dq_kernel(const __grid_constant__ ScoreArgs s, const T* __restrict__ qkv,
                     const int32_t* __restrict__ valid_len, const T* __restrict__ dctx, const float* __restrict__ lse,
                     const float* __restrict__ rowsum, unsigned* __restrict__ counter, T* __restrict__ dq,
                     float* __restrict__ partial, int B, int S, int NH) {
  extern __shared__ __align__(16) float smem[];
  float* Qs = smem;
  float* dOs = Qs + kT * (D + 4);
  float* Ks = dOs + kT * (D + 4);
  float* Vs = Ks + kT * (D + 4);
  float* Ps = Vs + kT * (D + 4);
  TileInfo* ti = reinterpret_cast<TileInfo*>(Ps + kT * kPs);
  // Sums of dT by distance within +-reach (index distance + reach), and past it on either side.
  float* by_distance = reinterpret_cast<float*>(ti + 1);
  float far_left = 0.f, far_right = 0.f;
  __shared__ float far[2][2 * kT];
  pdl_wait();
  if (threadIdx.x == 0) count_block(counter);
  pdl_trigger();
  const int b = blockIdx.z, h = blockIdx.y, qb = gridDim.x - 1 - blockIdx.x, q0 = qb * kT;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = score_len(valid_len, b, S), prefix = score_prefix(s, b);
  const size_t head = (size_t)S * D, part = (size_t)B * NH * head, bh = (size_t)b * NH + h;
  const T* Qg = qkv + bh * head;
  const int H = NH * D;
  const float slope = s.slopes ? s.slopes[h] : 0.f, inv_cap = s.cap > 0.f ? 1.f / s.cap : 0.f;
  float out[4][D / 16] = {};
  const bool busy = q0 + 8 * (ty >> 1) < n;                // some row of the warp's eight is valid
  const int rows = min(kT, n - q0);
  const int klim = rows > 0 ? score_jlim(s, q0 + rows - 1, n, prefix) : 0;
  load_tile<T, D>(Qs, Qg, q0, n, D);
  load_tile<T, D>(dOs, dctx + (size_t)b * S * H + h * D, q0, n, H);
  load_tile<T, D>(Ks, Qg + part, 0, n, D);
  load_tile<T, D>(Vs, Qg + 2 * part, 0, n, D);
  fill_docs(ti->row_doc, s, b, S, q0);
  load_column(s, ti->column, NH, h, threadIdx.x, kThreads);
  __syncthreads();
  if (partial)
    for (int k = threadIdx.x; k <= 2 * s.reach; k += kThreads) by_distance[k] = 0.f;
  float lse2[4], dsum[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = q0 + 4 * ty + a;
    lse2[a] = i < n ? lse[bh * S + i] * kLog2e : INFINITY;
    if (lse2[a] == -INFINITY) lse2[a] = INFINITY;
    dsum[a] = i < n ? rowsum[bh * S + i] : 0.f;
  }
  for (int j0 = 0; j0 < klim; j0 += kT) {
    fill_bias(ti, s, slope, j0 - q0);
    fill_docs(ti->col_doc, s, b, S, j0);
    wait_copies<0>();
    __syncthreads();
    const int live = min(kT, klim - j0);
    float acc[4][4] = {}, dp[4][4] = {};
    if (busy) {
      dot_tile<D>(Qs, Ks, live, acc);
      dot_tile<D>(dOs, Vs, live, dp);
    }
    __syncthreads();
    load_tile<T, D>(Vs, Qg + 2 * part, j0 + kT, n, D);     // the next tile's
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = 4 * ty + a, i = q0 + r;
      const int jlim = i < n ? score_jlim(s, i, n, prefix) : 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c, j = j0 + col;
        float sl;
        const float t = capped2(s, inv_cap, acc[a][c], sl) + ti->bias2[col - r + kT - 1];
        const bool see = j < jlim && (!s.docs || ti->row_doc[r] == ti->col_doc[col]);
        const float dt = see ? prob2(t, lse2[a]) * (dp[a][c] - dsum[a]) : 0.f;
        Ps[r * kPs + col] = dt;
        acc[a][c] = dt * sl;
      }
    }
    if (partial) {                       // the tile's 127 diagonals, a thread each
      __syncthreads();
      const int d0 = (int)threadIdx.x - (kT - 1), rel = j0 - q0 + d0;
      if (d0 < kT) {
        float sum = 0.f;
#pragma unroll 8
        for (int r = max(0, -d0); r < min(kT, kT - d0); ++r) sum += Ps[r * kPs + r + d0];
        if (rel <= -s.reach)
          far_left += sum;
        else if (rel >= s.reach)
          far_right += sum;
        else
          by_distance[rel + s.reach] += sum;
      }
      if (s.cap > 0.f) __syncthreads();
    }
    if (s.cap > 0.f) {
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int c = 0; c < 4; ++c) Ps[(4 * ty + a) * kPs + tx + 16 * c] = acc[a][c];
    }
    __syncthreads();
    if (busy) accumulate<D>(Ps, Ks, live, out);
    __syncthreads();
    load_tile<T, D>(Ks, Qg + part, j0 + kT, n, D);
  }
  wait_copies<0>();
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = q0 + 4 * ty + a;
    if (i >= S) continue;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) put(dq + (bh * S + i) * D + out_col<D>(e), out[a][e] * s.scale);
  }
  if (partial) {
    if (threadIdx.x < 2 * kT) {
      far[0][threadIdx.x] = far_left;
      far[1][threadIdx.x] = far_right;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < 2) {                      // both ends
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * kT; k += 32) sum += far[warp][k + lane];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) by_distance[warp * 2 * s.reach] = sum;
    }
    __syncthreads();
    for (int c = warp; c < s.buckets; c += kThreads / 32) {
      int lo, hi;
      bucket_range(s, c, lo, hi);
      float sum = 0.f;
      for (int k = lo + lane; k <= hi; k += 32) sum += by_distance[k + s.reach];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) partial[(bh * gridDim.x + qb) * s.buckets + c] = sum;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    scored_dkv_kernel(const __grid_constant__ ScoreArgs s, const T* qkv, const int32_t* valid_len, const T* dctx,
                      const float* lse, const float* rowsum, const unsigned* counter, T* dqkv, int B, int S, int NH) {
  // (Pointers without __restrict__: no load may go through the read-only path, or move above the acquire.)
  extern __shared__ __align__(16) float smem[];
  float* Ks = smem;
  float* Vs = Ks + kT * (D + 4);
  float* Qs = Vs + kT * (D + 4);
  float* dOs = Qs + kT * (D + 4);
  float* Ps = dOs + kT * (D + 4);
  TileInfo* ti = reinterpret_cast<TileInfo*>(Ps + kT * kPs);
  __shared__ float lse2[kT], dsum[kT];
  // The dQ grid before it makes nothing that this one reads: it runs beside that grid (all_blocks_counted has how it
  // sees what both read), and waits for it at the end so that what follows finds both complete.
  if (!all_blocks_counted(counter, gridDim.x * gridDim.y * gridDim.z)) pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, h = blockIdx.y, j0 = blockIdx.x * kT;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = score_len(valid_len, b, S), prefix = score_prefix(s, b);
  const size_t head = (size_t)S * D, part = (size_t)B * NH * head, bh = (size_t)b * NH + h;
  const T* Qg = qkv + bh * head;
  const int H = NH * D;
  const float slope = s.slopes ? s.slopes[h] : 0.f, inv_cap = s.cap > 0.f ? 1.f / s.cap : 0.f;
  float dk[4][D / 16] = {}, dv[4][D / 16] = {};
  load_tile<T, D>(Ks, Qg + part, j0, n, D);
  load_tile<T, D>(Vs, Qg + 2 * part, j0, n, D);
  const bool busy = j0 + 8 * (ty >> 1) < n;                // some row of the warp's eight is valid
  const int qfirst = j0 < n ? score_ilow(s, j0, prefix) / kT * kT : n;
  const T* dOg = dctx + (size_t)b * S * H + h * D;
  load_tile<T, D>(Qs, Qg, qfirst, n, D);
  load_tile<T, D>(dOs, dOg, qfirst, n, H);
  fill_docs(ti->row_doc, s, b, S, j0);
  load_column(s, ti->column, NH, h, threadIdx.x, kThreads);
  __syncthreads();
  for (int q0 = qfirst; q0 < n; q0 += kT) {
    fill_bias(ti, s, slope, j0 - q0);
    fill_docs(ti->col_doc, s, b, S, q0);
    if (threadIdx.x < kT) {
      const int i = q0 + threadIdx.x;
      const float v = i < n ? lse[bh * S + i] * kLog2e : INFINITY;
      lse2[threadIdx.x] = v == -INFINITY ? INFINITY : v;
      dsum[threadIdx.x] = i < n ? rowsum[bh * S + i] : 0.f;
    }
    wait_copies<0>();
    __syncthreads();
    const int live = min(kT, n - q0);
    float acc[4][4], dp[4][4];
    if (busy) {
      dot_tile<D>(Ks, Qs, live, acc);    // rows are keys, columns queries
      dot_tile<D>(Vs, dOs, live, dp);
    }
#pragma unroll
    for (int a = 0; a < 4 && busy; ++a) {
      const int r = 4 * ty + a, j = j0 + r;
      const int ilow = score_ilow(s, j, prefix);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = tx + 16 * c, i = q0 + col;
        float sl;
        const float t = capped2(s, inv_cap, acc[a][c], sl) + ti->bias2[r - col + kT - 1];
        const bool see = j < n && i >= ilow && i < n && (!s.docs || ti->row_doc[r] == ti->col_doc[col]);
        const float p = see ? prob2(t, lse2[col]) : 0.f;
        Ps[r * kPs + col] = p;
        acc[a][c] = p * (dp[a][c] - dsum[col]) * sl;
      }
    }
    __syncthreads();
    if (busy) accumulate<D>(Ps, dOs, live, dv);
    __syncthreads();
    load_tile<T, D>(dOs, dOg, q0 + kT, n, H);              // the next tile's
#pragma unroll
    for (int a = 0; a < 4 && busy; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) Ps[(4 * ty + a) * kPs + tx + 16 * c] = acc[a][c];
    __syncthreads();
    if (busy) accumulate<D>(Ps, Qs, live, dk);
    __syncthreads();
    load_tile<T, D>(Qs, Qg, q0 + kT, n, D);
  }
  wait_copies<0>();
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int j = j0 + 4 * ty + a;
    if (j >= S) continue;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
      put(dqkv + part + (bh * S + j) * D + out_col<D>(e), dk[a][e] * s.scale);
      put(dqkv + 2 * part + (bh * S + j) * D + out_col<D>(e), dv[a][e]);
    }
  }
  pdl_wait();
}

// One warp per (token, head).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    scored_rowsum_kernel(const T* __restrict__ ctx, const T* __restrict__ dctx, const int32_t* __restrict__ valid_len,
                         float* __restrict__ rowsum, unsigned* __restrict__ counter, int B, int S, int NH) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;
  const size_t item = (size_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= (size_t)B * S * NH) return;
  const int h = (int)(item % NH);
  const size_t token = item / NH;
  const int b = (int)(token / S), i = (int)(token % S);
  float sum = 0.f;
  if (i < score_len(valid_len, b, S)) {
    if (lane < D / 4) {
      const size_t at = token * NH * D + (size_t)h * D + lane * 4;
      const float4 x = load4<T>(ctx + at), y = load4<T>(dctx + at);
      sum = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  if (lane == 0) rowsum[((size_t)b * NH + h) * S + i] = sum;
}

// Block (head, bucket): the bucket's entries of the partial sums, added up by threads in a fixed order.  They are
// [B, nh, blocks, buckets], or with short_ctas sums by distance (entry distance + 127 of 256) at the first item of
// each CTA's run of the head's items; a bucket's distances are consecutive entries.
__global__ void __launch_bounds__(kThreads)
    scored_table_grad_kernel(const __grid_constant__ ScoreArgs s, const float* __restrict__ partial,
                             float* __restrict__ dtable, int B, int blocks, int short_ctas, int S, int NH) {
  __shared__ double sums[kThreads / 32];
  const int h = blockIdx.x, c = blockIdx.y, t = threadIdx.x;
  double sum = 0.0;
  if (short_ctas) {
    int lo, hi;
    bucket_range(s, c, lo, hi);
    // (past +-reach the bias does not change: the bucket takes the rest)
    lo = lo <= -s.reach ? 1 - S : max(lo, 1 - S);
    hi = hi >= s.reach ? S - 1 : min(hi, S - 1);
    const int at = lo + 127, count = max(0, hi - lo + 1), items = B * NH;
    const int first = cta_of_item(h * B, items, short_ctas), last = cta_of_item(h * B + B - 1, items, short_ctas);
    pdl_wait();
    pdl_trigger();
    const int total = (last - first + 1) * count;
#pragma unroll 4
    for (int k = t; k < total; k += kThreads) {
      const int item = max(h * B, first_item(first + k / count, items, short_ctas));
      sum += partial[(size_t)item * 256 + at + k % count];
    }
  } else {
    pdl_wait();
    pdl_trigger();
#pragma unroll 4
    for (int k = t; k < B * blocks; k += kThreads)
      sum += partial[(((size_t)(k / blocks) * NH + h) * blocks + k % blocks) * s.buckets + c];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (t % 32 == 0) sums[t / 32] = sum;
  __syncthreads();
  if (t == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) sum += sums[w];
    dtable[(size_t)c * NH + h] = static_cast<float>(sum);
  }
}

template <int D>
constexpr size_t smem_bytes(int tiles) {
  return (size_t)(tiles * kT * (D + 4) + kT * kPs) * sizeof(float) + sizeof(TileInfo);
}

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int D>
cudaError_t fwd_d(const ScoreArgs& s, const void* qkv, const int32_t* vl, void* ctx, float* lse,
                  const ScoredShape& sh, cudaStream_t stream) {
  static const cudaError_t attr = allow_smem(scored_fwd_kernel<T, D>, smem_bytes<D>(3));
  if (attr != cudaSuccess) return attr;
  const dim3 grid((sh.seq + kT - 1) / kT, sh.head_num, sh.batch);
  return launch_kernel(scored_fwd_kernel<T, D>, grid, dim3(kThreads), smem_bytes<D>(3), stream, nullptr, 0, s,
                       static_cast<const T*>(qkv), vl, static_cast<T*>(ctx), lse, sh.batch, sh.seq, sh.head_num);
}

template <typename T, int D>
cudaError_t bwd_d(const ScoreArgs& s, const void* qkv, const int32_t* vl, const void* dctx, const float* lse,
                  const float* rowsum, unsigned* counter, void* dqkv, float* partial, const ScoredShape& sh,
                  cudaStream_t stream) {
  const size_t dq_smem = smem_bytes<D>(4) + (partial ? (2 * s.reach + 1) * sizeof(float) : 0);
  static const cudaError_t attr1 =
      allow_smem(scored_dq_kernel<T, D>, smem_bytes<D>(4) + (2 * kMaxScoreDistance + 1) * sizeof(float));
  static const cudaError_t attr2 = allow_smem(scored_dkv_kernel<T, D>, smem_bytes<D>(4));
  if (attr1 != cudaSuccess) return attr1;
  if (attr2 != cudaSuccess) return attr2;
  const dim3 grid((sh.seq + kT - 1) / kT, sh.head_num, sh.batch);
  cudaError_t e = launch_kernel(scored_dq_kernel<T, D>, grid, dim3(kThreads), dq_smem, stream, nullptr, 0, s,
                                static_cast<const T*>(qkv), vl, static_cast<const T*>(dctx), lse, rowsum, counter,
                                static_cast<T*>(dqkv), partial, sh.batch, sh.seq, sh.head_num);
  if (e != cudaSuccess) return e;
  return launch_kernel(scored_dkv_kernel<T, D>, grid, dim3(kThreads), smem_bytes<D>(4), stream, nullptr, 0, s,
                       static_cast<const T*>(qkv), vl, static_cast<const T*>(dctx), lse, rowsum, counter,
                       static_cast<T*>(dqkv), sh.batch, sh.seq, sh.head_num);
}

template <typename T, int D>
cudaError_t rowsum_d(const void* ctx, const void* dctx, const int32_t* vl, float* rowsum, unsigned* counter,
                     const ScoredShape& sh, cudaStream_t stream) {
  const size_t items = (size_t)sh.batch * sh.seq * sh.head_num;
  return launch_kernel(scored_rowsum_kernel<T, D>, dim3((unsigned)((items + 7) / 8)), dim3(kThreads), 0, stream,
                       nullptr, 0, static_cast<const T*>(ctx), static_cast<const T*>(dctx), vl, rowsum, counter, sh.batch,
                       sh.seq, sh.head_num);
}

// f(type tag, integral constant of the head size)
template <typename F>
cudaError_t dispatch(bool half, int d, F f) {
  switch (d) {
    case 32: return half ? f(__half(), std::integral_constant<int, 32>()) : f(0.f, std::integral_constant<int, 32>());
    case 64: return half ? f(__half(), std::integral_constant<int, 64>()) : f(0.f, std::integral_constant<int, 64>());
    case 128: return half ? f(__half(), std::integral_constant<int, 128>()) : f(0.f, std::integral_constant<int, 128>());
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_scored_simt(const ScoreArgs& s, const void* qkv, const int32_t* valid_len, void* ctx, float* lse,
                               const ScoredShape& sh, bool half, cudaStream_t stream) {
  return dispatch(half, sh.size_per_head, [&](auto t, auto d) {
    return fwd_d<decltype(t), decltype(d)::value>(s, qkv, valid_len, ctx, lse, sh, stream);
  });
}

cudaError_t launch_scored_rowsum(const void* ctx, const void* dctx, const int32_t* valid_len, float* rowsum,
                                 unsigned* counter, const ScoredShape& sh, bool half, cudaStream_t stream) {
  return dispatch(half, sh.size_per_head, [&](auto t, auto d) {
    return rowsum_d<decltype(t), decltype(d)::value>(ctx, dctx, valid_len, rowsum, counter, sh, stream);
  });
}

cudaError_t launch_scored_backward_simt(const ScoreArgs& s, const void* qkv, const int32_t* valid_len,
                                        const void* dctx, const float* lse, const float* rowsum, unsigned* counter,
                                        void* dqkv, float* partial, const ScoredShape& sh, bool half,
                                        cudaStream_t stream) {
  return dispatch(half, sh.size_per_head, [&](auto t, auto d) {
    return bwd_d<decltype(t), decltype(d)::value>(s, qkv, valid_len, dctx, lse, rowsum, counter, dqkv, partial, sh,
                                                        stream);
  });
}

cudaError_t launch_scored_table_grad(const ScoreArgs& s, const float* partial, float* dtable, int blocks, int short_ctas,
                                     const ScoredShape& sh, cudaStream_t stream) {
  return launch_kernel(scored_table_grad_kernel, dim3(sh.head_num, s.buckets), dim3(kThreads), 0, stream, nullptr, 0, s,
                       partial, dtable, sh.batch, blocks, short_ctas, sh.seq, sh.head_num);
}

}  // namespace enc
