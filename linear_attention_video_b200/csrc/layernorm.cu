// Layer norm over the last axis and its backward pass.
//
//   mu = mean_c x,  r = (mean_c (x - mu)^2 + eps)^(-1/2),  h = (x - mu) r,  y = w h + b
//   g = w dy:  dx = r (g - mean_c g - h mean_c (g h)),  dw = sum_rows dy h,  db = sum_rows dy
//
// Bound by memory: x in, y out (backward: dy and x in, dx out).  A row lives in the registers of the 1 to 32
// warps that own it, so it is read once: the mean, then the squares around the mean (no cancellation), then
// the output.  Columns of a thread are the same for every row it takes, so the backward pass sums dw and db
// in registers over the rows of a persistent grid, writes one partial per row group, and a second launch adds
// the partials in a fixed order: the result does not depend on timing.
#include <algorithm>

#include "common.cuh"

namespace kda {
namespace {

template <typename T, int V> struct Pack;   // V elements as one access
template <> struct Pack<float, 4> { using U = uint4; };
template <> struct Pack<__nv_bfloat16, 8> { using U = uint4; };
template <> struct Pack<float, 1> { using U = float; };
template <> struct Pack<__nv_bfloat16, 1> { using U = unsigned short; };

template <typename T, int V> __device__ __forceinline__ void load_vec(const T* p, float* f) {
  const typename Pack<T, V>::U u = *reinterpret_cast<const typename Pack<T, V>::U*>(p);
  const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f32(e[i]);
}
template <typename T, int V> __device__ __forceinline__ void store_vec(T* p, const float* f) {
  typename Pack<T, V>::U u;
  T* e = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = from_f32<T>(f[i]);
  *reinterpret_cast<typename Pack<T, V>::U*>(p) = u;
}
// V fp32 parameters (weight, bias): 16-byte loads where V allows them.
template <int V> __device__ __forceinline__ void load_par(const float* p, float* f) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(p + i);
      f[i] = u.x; f[i + 1] = u.y; f[i + 2] = u.z; f[i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = p[i];
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Sum of K values over the W warps of a row (all threads of the CTA call it: rows of one CTA run in step).
template <int W, int K>
__device__ __forceinline__ void row_sum(float (&x)[K], float* scratch, int group, int wg) {
#pragma unroll
  for (int i = 0; i < K; ++i) x[i] = warp_sum(x[i]);
  if constexpr (W > 1) {
    float* sc = scratch + group * W * K;
    __syncthreads();   // the previous sums have been read
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) sc[wg * K + i] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) t += sc[w * K + i];
      x[i] = t;
    }
  }
}

// W warps per row, E elements per thread in vectors of V.
template <typename T, int V, int E, int W>
struct Shape {
  static constexpr int threads = W * 32 < 128 ? 128 : W * 32;
  static constexpr int groups = threads / (W * 32);   // rows per CTA at a time
};

template <typename T, int V, int E, int W>
__global__ void __launch_bounds__(Shape<T, V, E, W>::threads) norm_fwd_kernel(NormFwdArgs a) {
  using S = Shape<T, V, E, W>;
  __shared__ float scratch[S::groups * W];
  const int group = threadIdx.x / (W * 32), lane = threadIdx.x % (W * 32), wg = lane / 32;
  const int64_t row = (int64_t)blockIdx.x * S::groups + group;
  const bool live = row < a.rows;
  const T* x = static_cast<const T*>(a.x) + row * a.cols;
  float v[E];
#pragma unroll
  for (int i = 0; i < E / V; ++i) {
    const int c = (i * W * 32 + lane) * V;
    if (live && c < a.cols) load_vec<T, V>(x + c, v + i * V);
    else
#pragma unroll
      for (int j = 0; j < V; ++j) v[i * V + j] = 0.f;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < E; ++i) s[0] += v[i];
  row_sum<W>(s, scratch, group, wg);
  const float mean = s[0] / (float)a.cols;
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < E / V; ++i)
    if ((i * W * 32 + lane) * V < a.cols)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float t = v[i * V + j] - mean;
        q[0] += t * t;
      }
  row_sum<W>(q, scratch, group, wg);
  const float rstd = 1.f / sqrtf(q[0] / (float)a.cols + a.eps);
  if (!live) return;
  if (lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.cols;
#pragma unroll
  for (int i = 0; i < E / V; ++i) {
    const int c = (i * W * 32 + lane) * V;
    if (c >= a.cols) continue;
    float w[V], b[V], o[V];
    if (a.weight) load_par<V>(a.weight + c, w);
    if (a.bias) load_par<V>(a.bias + c, b);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float h = (v[i * V + j] - mean) * rstd;
      o[j] = (a.weight ? h * w[j] : h) + (a.bias ? b[j] : 0.f);
    }
    store_vec<T, V>(y + c, o);
  }
}

template <typename T, int V, int E, int W>
__global__ void __launch_bounds__(Shape<T, V, E, W>::threads) norm_bwd_kernel(NormBwdArgs a) {
  using S = Shape<T, V, E, W>;
  __shared__ float scratch[S::groups * W * 2];
  const int group = threadIdx.x / (W * 32), lane = threadIdx.x % (W * 32), wg = lane / 32;
  const int64_t stride = (int64_t)gridDim.x * S::groups;
  const float inv = 1.f / (float)a.cols;
  float w[E], dw[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) w[i] = 1.f, dw[i] = 0.f, db[i] = 0.f;
  if (a.weight) {
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const int c = (i * W * 32 + lane) * V;
      if (c < a.cols) load_par<V>(a.weight + c, w + i * V);
    }
  }
  for (int64_t row0 = (int64_t)blockIdx.x * S::groups; row0 < a.rows; row0 += stride) {
    const int64_t row = row0 + group;
    const bool live = row < a.rows;
    const T* x = static_cast<const T*>(a.x) + row * a.cols;
    const T* dy = static_cast<const T*>(a.dy) + row * a.cols;
    float h[E], g[E];
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const int c = (i * W * 32 + lane) * V;
      if (live && c < a.cols) {
        load_vec<T, V>(x + c, h + i * V);
        load_vec<T, V>(dy + c, g + i * V);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) h[i * V + j] = 0.f, g[i * V + j] = 0.f;
      }
    }
    const float mean = live ? a.mean[row] : 0.f, rstd = live ? a.rstd[row] : 0.f;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) {   // columns past the row have g = 0
      h[i] = (h[i] - mean) * rstd;
      dw[i] += g[i] * h[i];
      db[i] += g[i];
      g[i] *= w[i];
      s[0] += g[i];
      s[1] += g[i] * h[i];
    }
    row_sum<W>(s, scratch, group, wg);
    if (!live) continue;
    const float mg = s[0] * inv, mgh = s[1] * inv;
    T* dx = static_cast<T*>(a.dx) + row * a.cols;
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const int c = (i * W * 32 + lane) * V;
      if (c >= a.cols) continue;
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = rstd * (g[i * V + j] - mg - h[i * V + j] * mgh);
      store_vec<T, V>(dx + c, o);
    }
  }
  if (!a.parts) return;
  float* part = a.parts + ((int64_t)blockIdx.x * S::groups + group) * 2 * a.cols;
#pragma unroll
  for (int i = 0; i < E / V; ++i) {
    const int c = (i * W * 32 + lane) * V;
    if (c >= a.cols) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      part[c + j] = dw[i * V + j];
      part[a.cols + c + j] = db[i * V + j];
    }
  }
}

// Adds the partials of 32 columns: 8 strands of rows, joined in a fixed order.
__global__ void __launch_bounds__(256) norm_sum_kernel(const float* parts, int n_parts, int cols, float* dw, float* db) {
  __shared__ float sm[8][32];
  const int cx = threadIdx.x % 32, ry = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + cx;   // over 2 * cols: the weight's sums, then the bias's
  float s = 0.f;
  if (c < 2 * cols)
    for (int r = ry; r < n_parts; r += 8) s += parts[(int64_t)r * 2 * cols + c];
  sm[ry][cx] = s;
  __syncthreads();
  if (ry || c >= 2 * cols) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) s += sm[r][cx];
  if (c < cols) { if (dw) dw[c] = s; }
  else if (db) db[c - cols] = s;
}

constexpr int kFwdE = 32, kBwdE = 16;   // elements of a row per thread

int warps_for(int cols, int e) {
  int w = 1;
  while (w * 32 * e < cols) w *= 2;
  return w;
}

template <typename T, int V>
cudaError_t fwd(const NormFwdArgs& a, cudaStream_t s) {
  const int W = warps_for(a.cols, kFwdE);
  auto go = [&](auto kernel, int threads, int groups) {
    kernel<<<(unsigned)((a.rows + groups - 1) / groups), threads, 0, s>>>(a);
    return cudaGetLastError();
  };
#define KDA_NORM(w) \
  case w: return go(norm_fwd_kernel<T, V, kFwdE, w>, Shape<T, V, kFwdE, w>::threads, Shape<T, V, kFwdE, w>::groups)
  switch (W) {
    KDA_NORM(1);
    KDA_NORM(2);
    KDA_NORM(4);
    KDA_NORM(8);
    KDA_NORM(16);
  }
#undef KDA_NORM
  return cudaErrorInvalidValue;
}

template <typename T, int V>
cudaError_t bwd(const NormBwdArgs& a, int grid, cudaStream_t s) {
  const int W = warps_for(a.cols, kBwdE);
#define KDA_NORM(w) \
  case w: norm_bwd_kernel<T, V, kBwdE, w><<<grid, Shape<T, V, kBwdE, w>::threads, 0, s>>>(a); return cudaGetLastError()
  switch (W) {
    KDA_NORM(1);
    KDA_NORM(2);
    KDA_NORM(4);
    KDA_NORM(8);
    KDA_NORM(16);
    KDA_NORM(32);
  }
#undef KDA_NORM
  return cudaErrorInvalidValue;
}

int bwd_groups(int cols) { return std::max(1, 4 / warps_for(cols, kBwdE)); }

// CTAs of the backward pass: enough to fill the GPU, no more than there are row groups.
int bwd_grid(int64_t rows, int cols) {
  const int threads = std::max(128, 32 * warps_for(cols, kBwdE));
  const int64_t need = (rows + bwd_groups(cols) - 1) / bwd_groups(cols);
  return (int)std::min<int64_t>(need, (int64_t)148 * (1024 / threads));
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwdArgs& a, kda_dtype dt, cudaStream_t s, int* launches) {
  if (a.rows == 0) return cudaSuccess;
  cudaError_t e;
  if (dt == KDA_DT_BF16) e = a.cols % 8 == 0 ? fwd<__nv_bfloat16, 8>(a, s) : fwd<__nv_bfloat16, 1>(a, s);
  else e = a.cols % 4 == 0 ? fwd<float, 4>(a, s) : fwd<float, 1>(a, s);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

size_t norm_bwd_parts(int64_t rows, int cols) {
  return (size_t)bwd_grid(rows, cols) * bwd_groups(cols) * 2 * cols * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, kda_dtype dt, float* dw, float* db, cudaStream_t s, int* launches) {
  cudaError_t e;
  if (a.rows == 0) {   // no rows: the sums are zero
    if (dw && (e = cudaMemsetAsync(dw, 0, (size_t)a.cols * sizeof(float), s)) != cudaSuccess) return e;
    if (db && (e = cudaMemsetAsync(db, 0, (size_t)a.cols * sizeof(float), s)) != cudaSuccess) return e;
    return cudaSuccess;
  }
  const int grid = bwd_grid(a.rows, a.cols);
  if (dt == KDA_DT_BF16) e = a.cols % 8 == 0 ? bwd<__nv_bfloat16, 8>(a, grid, s) : bwd<__nv_bfloat16, 1>(a, grid, s);
  else e = a.cols % 4 == 0 ? bwd<float, 4>(a, grid, s) : bwd<float, 1>(a, grid, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (!dw && !db) return cudaSuccess;
  norm_sum_kernel<<<(2 * a.cols + 31) / 32, 256, 0, s>>>(a.parts, grid * bwd_groups(a.cols), a.cols, dw, db);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  *launches += 1;
  return cudaSuccess;
}

}  // namespace kda
