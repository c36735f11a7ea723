// Layer norm over the last axis and its backward pass.
//
//   mu = mean_c x,  r = (mean_c (x - mu)^2 + eps)^(-1/2),  h = (x - mu) r,  y = w h + b
//   g = w dy:  dx = r (g - mean_c g - h mean_c (g h)),  dw = sum_rows dy h,  db = sum_rows dy
//
// Bound by memory: x in, y out (backward: dy and x in, dx out).  A row lives in the registers of the lanes that
// own it, so it is read once: the mean, then the squares around the mean (no cancellation), then the output.
// Columns of a thread are the same for every row it takes, so the backward pass sums dw and db in registers
// over the rows of a persistent grid, writes one partial per CTA, and a second launch adds the partials in a
// fixed order: the result does not depend on timing.
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace kda {
namespace {

// V elements as one access (16 bytes, 8, or one element): as fetched, and as fp32.
template <typename T, int V> struct Raw;
template <> struct Raw<float, 4> { using type = uint4; };
template <> struct Raw<__nv_bfloat16, 8> { using type = uint4; };
template <> struct Raw<__nv_bfloat16, 4> { using type = uint2; };
template <typename T> struct Raw<T, 1> { using type = T; };
template <typename T, int V> using raw_t = typename Raw<T, V>::type;

__device__ __forceinline__ void widen(const uint4& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void widen(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const uint2& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void widen(float u, float (&f)[1]) { f[0] = u; }
__device__ __forceinline__ void widen(__nv_bfloat16 u, float (&f)[1]) { f[0] = __bfloat162float(u); }
__device__ __forceinline__ void clear(uint2& u) { u = make_uint2(0, 0); }
__device__ __forceinline__ void clear(uint4& u) { u = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void clear(float& u) { u = 0.f; }
__device__ __forceinline__ void clear(__nv_bfloat16& u) { u = __nv_bfloat16(0.f); }
template <int V> __device__ __forceinline__ void store_vec(float* p, const float (&f)[V]) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  else p[0] = f[0];
}
template <int V> __device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    p[0] = __float2bfloat16_rn(f[0]);
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = reinterpret_cast<const uint32_t&>(v);
    }
    if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}
// V fp32 parameters (weight, bias); `none` where there are none.
template <int V> __device__ __forceinline__ void load_par(const float* p, int c, float none, float (&f)[V]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = none;
  } else if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(p + c + i);
      f[i] = u.x; f[i + 1] = u.y; f[i + 2] = u.z; f[i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = p[c + i];
  }
}

// Two fp32 operations in one instruction: half the issue slots.  With them the backward pass of bf16 rows issues in 55%
// of its cycles and waits for memory: a row prefetched in registers is 32 KB in flight per SM.
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
// (x, y) = (a, b) * (c, d) + (x, y)
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float c, float d) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 r, {%4, %5};\n\t"
      "fma.rn.f32x2 p, q, r, p;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b), "f"(c), "f"(d));
}
// The same over V elements, single ones where V is odd.  x += y; x *= y; z += x y.
template <int V> __device__ __forceinline__ void add_v(float (&x)[V], const float (&y)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) add2(x[j], x[j + 1], y[j], y[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] += y[j];
  }
}
template <int V> __device__ __forceinline__ void add_s(float (&x)[V], float y) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) add2(x[j], x[j + 1], y, y);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] += y;
  }
}
template <int V> __device__ __forceinline__ void mul_v(float (&x)[V], const float (&y)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) mul2(x[j], x[j + 1], y[j], y[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] *= y[j];
  }
}
template <int V> __device__ __forceinline__ void mul_s(float (&x)[V], float y) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) mul2(x[j], x[j + 1], y, y);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] *= y;
  }
}
template <int V> __device__ __forceinline__ void fma_v(float (&z)[V], const float (&x)[V], const float (&y)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) fma2(z[j], z[j + 1], x[j], x[j + 1], y[j], y[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = fmaf(x[j], y[j], z[j]);
  }
}
template <int V> __device__ __forceinline__ void fma_s(float (&z)[V], const float (&x)[V], float y) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) fma2(z[j], z[j + 1], x[j], x[j + 1], y, y);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = fmaf(x[j], y, z[j]);
  }
}
// Two strands of a lane's sum: sum over V elements into (lo, hi), x or x y each.
template <int V> __device__ __forceinline__ void sum_v(float (&s)[2], const float (&x)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) add2(s[0], s[1], x[j], x[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) s[0] += x[j];
  }
}
template <int V> __device__ __forceinline__ void dot_v(float (&s)[2], const float (&x)[V], const float (&y)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) fma2(s[0], s[1], x[j], x[j + 1], y[j], y[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) s[0] = fmaf(x[j], y[j], s[0]);
  }
}

// A row belongs to G lanes (a power of two, 8..1024) with E elements each, in vectors of V, and a group of lanes
// takes R rows at a time: R rows' loads are in flight together and share one reading of the weight.
template <int G> struct Shape {
  static constexpr int threads = G < 128 ? 128 : G;
  static constexpr int groups = threads / G;
};
// Resident threads per SM that registers must allow.  Backward: 640 would spill (33,272 x 2048 bf16: 123 us against 83).
// Rows of more than 8192 columns take 1024 threads, whose 64 registers each do spill: 4000 x 16,384 bf16 backward 213 us
// (1.85 TB/s; 10,000 x 8192: 112 us, 4.4 TB/s), fp32 402 us.
constexpr int kFwdThreads = 1024, kBwdThreads = 512;
constexpr int ctas_of(int threads, int resident) { return threads < resident ? resident / threads : 1; }

// Sums of K values over the G lanes of a group; every thread of the CTA calls it.
template <int G, int K>
__device__ __forceinline__ void group_sum(float (&x)[K], float* scratch, int group, int lane) {
#pragma unroll
  for (int m = (G < 32 ? G : 32) / 2; m; m >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], m);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    float* sc = scratch + group * W * K;
    __syncthreads();   // the sums before have been read
    if ((lane & 31) == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) sc[i * W + lane / 32] = x[i];
    }
    __syncthreads();
    if constexpr (W <= 8) {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        float t = sc[i * W];
#pragma unroll
        for (int w = 1; w < W; ++w) t += sc[i * W + w];
        x[i] = t;
      }
    } else {   // 16 or 32 partial sums: one per lane
#pragma unroll
      for (int i = 0; i < K; ++i) {
        float t = sc[i * W + (lane & (W - 1))];
#pragma unroll
        for (int m = W / 2; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
        x[i] = t;
      }
    }
  }
}

// This lane's elements of rows row0 .. row0 + R - 1; zeros past the columns and the rows.
template <typename T, int V, int E, int G, int R>
__device__ __forceinline__ void fetch(const void* base, int64_t row0, int64_t rows, int cols, int lane,
                                      raw_t<T, V> (&v)[R][E / V]) {
  const T* p = static_cast<const T*>(base) + row0 * cols;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const int c = (i * G + lane) * V;
      if (row0 + r < rows && c < cols) v[r][i] = *reinterpret_cast<const raw_t<T, V>*>(p + (int64_t)r * cols + c);
      else clear(v[r][i]);
    }
}

// Forward: a row stays as fetched and is widened in each of the three passes over it: one instruction per element and
// pass, against twice the registers.  A lane takes four columns at a time, whose weights and biases are one 16-byte
// access each (of eight they would be two, half a line apart: the L1 cache, which serves them for every row, is then
// 75% busy).  One row per group and many CTAs: 33,272 x 2048 bf16 in 51 us, the same with two rows at a time, 55 to 57
// with a warp per row and 54 with a persistent grid that fetches ahead; fp32 runs at a copy's bandwidth (84 us).
template <typename T, int V, int NV, int G, int R>
__global__ void __launch_bounds__(Shape<G>::threads, ctas_of(Shape<G>::threads, kFwdThreads)) norm_fwd_kernel(NormFwdArgs a) {
  using S = Shape<G>;
  __shared__ float scratch[S::groups * (G / 32 + 1) * R];
  const int group = threadIdx.x / G, lane = threadIdx.x % G;
  const float inv = 1.f / (float)a.cols;
  const int64_t row0 = ((int64_t)blockIdx.x * S::groups + group) * R;
  raw_t<T, V> cur[R][NV];
  fetch<T, V, V * NV, G, R>(a.x, row0, a.rows, a.cols, lane, cur);
  float s[R], mean[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float t[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[V];
      widen(cur[r][i], v);
      sum_v<V>(t, v);
    }
    s[r] = t[0] + t[1];
  }
  group_sum<G>(s, scratch, group, lane);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mean[r] = s[r] * inv;
    float t[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * G + lane) * V < a.cols) {
        float v[V];
        widen(cur[r][i], v);
        add_s<V>(v, -mean[r]);
        dot_v<V>(t, v, v);
      }
    s[r] = t[0] + t[1];
  }
  group_sum<G>(s, scratch, group, lane);
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = 1.f / sqrtf(fmaf(s[r], inv, a.eps));
  if (lane == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (row0 + r < a.rows) {
        if (a.mean) a.mean[row0 + r] = mean[r];
        if (a.rstd) a.rstd[row0 + r] = s[r];
      }
  }
  T* y = static_cast<T*>(a.y) + row0 * a.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + lane) * V;
    if (c >= a.cols) continue;
    float w[V], b[V];
    load_par<V>(a.weight, c, 1.f, w);
    load_par<V>(a.bias, c, 0.f, b);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= a.rows) break;
      float v[V], o[V];
      widen(cur[r][i], v);
      add_s<V>(v, -mean[r]);
      mul_s<V>(v, s[r]);
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = b[j];
      fma_v<V>(o, v, w);
      store_vec<V>(y + (int64_t)r * a.cols + c, o);
    }
  }
}

// Backward: a persistent grid; the rows of the next turn are fetched before the sums of this one, so the loads do not
// wait for reductions and stores.
template <typename T, int V, int E, int G, int R>
__global__ void __launch_bounds__(Shape<G>::threads, ctas_of(Shape<G>::threads, kBwdThreads)) norm_bwd_kernel(NormBwdArgs a) {
  using S = Shape<G>;
  constexpr int NV = E / V;
  __shared__ float scratch[S::groups * (G / 32 + 1) * 2 * R];
  __shared__ float sums[S::groups > 1 ? S::groups * G * E : 1];
  const int group = threadIdx.x / G, lane = threadIdx.x % G;
  const int64_t stride = (int64_t)gridDim.x * S::groups * R;
  const float inv = 1.f / (float)a.cols;
  float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + lane) * V;
    load_par<V>(c < a.cols ? a.weight : nullptr, c, 1.f, w[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  raw_t<T, V> nx[R][NV], ny[R][NV];
  float nm[R], nr[R];
  auto get = [&](int64_t row0) {
    fetch<T, V, E, G, R>(a.x, row0, a.rows, a.cols, lane, nx);
    fetch<T, V, E, G, R>(a.dy, row0, a.rows, a.cols, lane, ny);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = row0 + r < a.rows;
      nm[r] = live ? a.mean[row0 + r] : 0.f;
      nr[r] = live ? a.rstd[row0 + r] : 0.f;
    }
  };
  get(((int64_t)blockIdx.x * S::groups + group) * R);
  for (int64_t base = (int64_t)blockIdx.x * S::groups * R; base < a.rows; base += stride) {
    const int64_t row0 = base + group * R;
    float h[R][NV][V], g[R][NV][V], rstd[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mean = nm[r];
      rstd[r] = nr[r];
      float t[2] = {0.f, 0.f}, u[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {   // columns past the row have dy = 0
        widen(nx[r][i], h[r][i]);
        widen(ny[r][i], g[r][i]);
        add_s<V>(h[r][i], -mean);
        mul_s<V>(h[r][i], rstd[r]);
        fma_v<V>(dw[i], g[r][i], h[r][i]);
        add_v<V>(db[i], g[r][i]);
        mul_v<V>(g[r][i], w[i]);
        sum_v<V>(t, g[r][i]);
        dot_v<V>(u, g[r][i], h[r][i]);
      }
      s[2 * r] = t[0] + t[1];
      s[2 * r + 1] = u[0] + u[1];
    }
    get(row0 + stride);
    group_sum<G>(s, scratch, group, lane);
    T* dx = static_cast<T*>(a.dx) + row0 * a.cols;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= a.rows) break;
      const float mg = -s[2 * r] * inv * rstd[r], mgh = -s[2 * r + 1] * inv * rstd[r];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + lane) * V;
        if (c >= a.cols) continue;
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = mg;
        fma_s<V>(o, h[r][i], mgh);
        fma_s<V>(o, g[r][i], rstd[r]);
        store_vec<V>(dx + (int64_t)r * a.cols + c, o);
      }
    }
  }
  if (!a.parts) return;
  float* part = a.parts + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
  for (int which = 0; which < 2; ++which) {   // the CTA's groups, added in order
    float(&acc)[NV][V] = which ? db : dw;
    if constexpr (S::groups > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) sums[(group * NV * V + i * V + j) * G + lane] = acc[i][j];
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j)
            for (int k = 1; k < S::groups; ++k) acc[i][j] += sums[(k * NV * V + i * V + j) * G + lane];
      }
    }
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + lane) * V;
        if (c >= a.cols) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) part[which * a.cols + c + j] = acc[i][j];
      }
    }
  }
}

// Adds the partials of 32 columns: 32 strands of rows, joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_sum_kernel(const float* parts, int n_parts, int cols, float* dw, float* db, uint32_t* status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  __shared__ float sm[32][33];
  const int cx = threadIdx.x % 32, ry = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + cx;   // over 2 * cols: the weight's sums, then the bias's
  float s = 0.f;
  if (c < 2 * cols) {
#pragma unroll 4
    for (int r = ry; r < n_parts; r += 32) s += parts[(int64_t)r * 2 * cols + c];
  }
  sm[ry][cx] = s;
  __syncthreads();
  float t = sm[cx][ry];   // warp ry adds column ry
#pragma unroll
  for (int m = 16; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
  const int k = blockIdx.x * 32 + ry;
  if (cx || k >= 2 * cols) return;
  if (k < cols) { if (dw) dw[k] = t; }
  else if (db) db[k - cols] = t;
}

template <int N> using Const = std::integral_constant<int, N>;

template <typename T, int V, int NV, int G, int R>
cudaError_t fwd_shape(const NormFwdArgs& a, cudaStream_t s) {
  using S = Shape<G>;
  constexpr int per = S::groups * R;
  norm_fwd_kernel<T, V, NV, G, R><<<(unsigned)((a.rows + per - 1) / per), S::threads, 0, s>>>(a);
  return cudaGetLastError();
}
// Vectors of a row: up to 4 per lane and 32 lanes, then 8 (scalars: 16) per lane, then more warps.  Narrow rows come
// in pairs, which keeps 64 bytes per lane in flight and shares a reading of the weights.
template <typename T, int V>
cudaError_t fwd(const NormFwdArgs& a, cudaStream_t s) {
  const int n = (a.cols + V - 1) / V;
  if (n <= 8) return fwd_shape<T, V, 1, 8, 4>(a, s);
  if (n <= 16) return fwd_shape<T, V, 2, 8, 2>(a, s);
  if (n <= 32) return fwd_shape<T, V, 4, 8, 2>(a, s);
  if (n <= 64) return fwd_shape<T, V, 4, 16, 2>(a, s);
  if (n <= 128) return fwd_shape<T, V, 4, 32, 2>(a, s);
  if (n <= 256) return fwd_shape<T, V, 8, 32, 1>(a, s);
  if (n <= 512) return fwd_shape<T, V, 8, 64, 1>(a, s);
  if (n <= 1024) return fwd_shape<T, V, 8, 128, 1>(a, s);
  if (n <= 2048) return fwd_shape<T, V, 8, 256, 1>(a, s);
  if (n <= 4096) return fwd_shape<T, V, 8, 512, 1>(a, s);
  if constexpr (V == 1) {
    if (n <= 8192) return fwd_shape<T, V, 16, 512, 1>(a, s);
    return fwd_shape<T, V, 16, 1024, 1>(a, s);
  }
  return cudaErrorInvalidValue;
}

// Backward: 16 elements of a row per lane and one row at a time (33,272 x 2048 bf16: 83 us with the sums' 5; 8 and two
// rows 84 us, the reductions then cost a third of the instructions; 16 and two rows 137 us, out of registers).  Scalar
// accesses take 8 and two rows (2047 columns: 116 us against 163).
int lanes_for(int cols, int e) {
  int g = 8;
  while (g < 1024 && g * e < cols) g *= 2;
  return g;
}
constexpr int groups_for(int g) { return g < 128 ? 128 / g : 1; }

template <typename T, int V, int E, int R>
cudaError_t bwd_shape(const NormBwdArgs& a, int grid, cudaStream_t s) {
#define KDA_NORM(g) \
  case g: norm_bwd_kernel<T, V, E, g, R><<<grid, Shape<g>::threads, 0, s>>>(a); break
  switch (lanes_for(a.cols, E)) {
    KDA_NORM(8);
    KDA_NORM(16);
    KDA_NORM(32);
    KDA_NORM(64);
    KDA_NORM(128);
    KDA_NORM(256);
    KDA_NORM(512);
    KDA_NORM(1024);
  }
#undef KDA_NORM
  return cudaGetLastError();
}
// CTAs of lanes with e elements and r rows at a time: as many as are resident at once, no more than there are row groups.
int bwd_grid(int64_t rows, int cols, int e, int r) {
  const int g = lanes_for(cols, e), per = groups_for(g) * r;
  return (int)std::min<int64_t>((rows + per - 1) / per, (int64_t)148 * ctas_of(std::max(128, g), kBwdThreads));
}
bool narrow_scalar(int cols, int v) { return v == 1 && cols <= 8 * 512; }
// Of accesses of v elements.
int bwd_grid(int64_t rows, int cols, int v) {
  return narrow_scalar(cols, v) ? bwd_grid(rows, cols, 8, 2) : bwd_grid(rows, cols, 16, 1);
}
template <typename T, int V>
cudaError_t bwd(const NormBwdArgs& a, int grid, cudaStream_t s) {
  if constexpr (V == 1)
    if (narrow_scalar(a.cols, V)) return bwd_shape<T, V, 8, 2>(a, grid, s);
  return bwd_shape<T, V, 16, 1>(a, grid, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwdArgs& a, kda_dtype dt, cudaStream_t s, int* launches) {
  if (a.rows == 0) return cudaSuccess;
  cudaError_t e;
  if (dt == KDA_DT_BF16) e = a.cols % 4 == 0 ? fwd<__nv_bfloat16, 4>(a, s) : fwd<__nv_bfloat16, 1>(a, s);
  else e = a.cols % 4 == 0 ? fwd<float, 4>(a, s) : fwd<float, 1>(a, s);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

// What no problem with fewer rows or columns exceeds.  The shape of 16 elements has the larger grid of the two (the other
// has as many or twice as many lanes and rows at a time), and its grid shrinks behind 2048 and 4096 columns alone.
size_t norm_bwd_parts(int64_t rows, int cols) {
  size_t most = (size_t)bwd_grid(rows, cols, 16, 1) * cols;
  for (int c : {2048, 4096})
    if (c < cols) most = std::max(most, (size_t)bwd_grid(rows, c, 16, 1) * c);
  return most * 2 * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, kda_dtype dt, float* dw, float* db, uint32_t* status, cudaStream_t s, int* launches) {
  cudaError_t e;
  if (a.rows == 0) {   // no rows: the sums are zero
    if (dw && (e = cudaMemsetAsync(dw, 0, (size_t)a.cols * sizeof(float), s)) != cudaSuccess) return e;
    if (db && (e = cudaMemsetAsync(db, 0, (size_t)a.cols * sizeof(float), s)) != cudaSuccess) return e;
    return cudaSuccess;
  }
  const int v = dt == KDA_DT_BF16 ? (a.cols % 8 == 0 ? 8 : 1) : (a.cols % 4 == 0 ? 4 : 1);
  const int grid = bwd_grid(a.rows, a.cols, v);
  if (dt == KDA_DT_BF16) e = v == 8 ? bwd<__nv_bfloat16, 8>(a, grid, s) : bwd<__nv_bfloat16, 1>(a, grid, s);
  else e = v == 4 ? bwd<float, 4>(a, grid, s) : bwd<float, 1>(a, grid, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (!dw && !db) return cudaMemsetAsync(status, 0, sizeof(uint32_t), s);
  norm_sum_kernel<<<(2 * a.cols + 31) / 32, 1024, 0, s>>>(a.parts, grid, a.cols, dw, db, status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  *launches += 1;
  return cudaSuccess;
}

}  // namespace kda
