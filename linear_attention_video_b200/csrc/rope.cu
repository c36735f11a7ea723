// Rotary positions with three axes (time, height, width) on q and k.
//
// Pair j of a head's d/2 pairs turns by the angle position[axis(j)] * inv_freq[j]:
//   y_a = x_a cos - x_b sin,  y_b = x_a sin + x_b cos      (the backward pass turns by minus the angle).
// A turn is orthogonal, so the gradient's map is the turn back and nothing of the forward pass is kept.
//
// The angle's error must stay below the fp32 cosine's for positions of a long stream, so position *
// inv_freq / (2 pi) is formed in fp64 and only its fraction of a turn, in [-1/2, 1/2], goes to fp32.
//
// Bound by memory: 2 reads and 2 writes of every element, 32 (head, tensor) rows sharing the angles of a
// token.  A CTA takes the tokens that give each of its threads one angle (256 / (d/2)), so the cost of the
// angles is 1/(2H) of an evaluation per pair, and keeps them in shared memory as (cos, sin).
#include "common.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // vectors in flight per thread and half

// Elements of one 16-byte vector.
template <typename T> struct Vec { static constexpr int n = 16 / sizeof(T); };

template <typename T> __device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < Vec<T>::n; ++i) f[i] = to_f32(e[i]);
}
template <typename T> __device__ __forceinline__ uint4 pack(const float* f) {
  uint4 u;
  T* e = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int i = 0; i < Vec<T>::n; ++i) e[i] = from_f32<T>(f[i]);
  return u;
}

// kHalves: pair j is (j, j + D/2); otherwise (2j, 2j + 1).
template <typename T, int D, bool kHalves>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a) {
  constexpr int P = D / 2, TOK = kThreads / P, V = Vec<T>::n;
  constexpr int UNITS = P / V;   // a unit: two vectors holding V whole pairs
  __shared__ float2 turn[TOK * P];
  const int tid = threadIdx.x;
  const int64_t tok0 = (int64_t)blockIdx.x * TOK;
  const int n_tok = (int)min((int64_t)TOK, a.tokens - tok0);
  const int per_tok = a.n_tensors * a.H * UNITS;
  const int items = n_tok * per_tok;

  // item i: token, tensor, head, unit, innermost last
  auto locate = [&](int i, int& tok, int& unit, const T*& src, T*& dst) {
    tok = i / per_tok;
    int r = i - tok * per_tok;
    const int tensor = r >= a.H * UNITS;
    r -= tensor * a.H * UNITS;
    unit = r % UNITS;
    const int64_t off = ((tok0 + tok) * a.H + r / UNITS) * D;
    src = static_cast<const T*>(tensor ? a.x[1] : a.x[0]) + off;
    dst = static_cast<T*>(tensor ? a.y[1] : a.y[0]) + off;
  };
  constexpr int LO_STEP = kHalves ? V : 2 * V;   // first vector of unit u at u * LO_STEP
  constexpr int HI_OFF = kHalves ? P : V;        // the second one, from the first

  for (int base = 0; base < items; base += kThreads * kUnroll) {
    uint4 lo[kUnroll], hi[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kThreads + tid;
      if (i >= items) continue;
      int tok, unit;
      const T* src;
      T* dst;
      locate(i, tok, unit, src, dst);
      const uint4* s = reinterpret_cast<const uint4*>(src + unit * LO_STEP);
      lo[u] = s[0];
      hi[u] = s[HI_OFF / V];
    }
    if (base == 0) {   // the angles, while the first loads are in flight
      const int tok = tid / P, j = tid % P;
      if (tok < n_tok) {
        const int axis = j < a.pairs_t ? 0 : (j < a.pairs_t + a.pairs_h ? 1 : 2);
        const int64_t t = tok0 + tok;
        int64_t pos;
        if (a.positions) {
          pos = a.positions[t * 3 + axis];
        } else {
          pos = t % a.N;
          if (pos >= a.text) {
            const int64_t m = pos - a.text;
            const int64_t hw = (int64_t)a.Hg * a.Wg;
            pos = a.text + (axis == 0 ? m / hw : (axis == 1 ? m % hw / a.Wg : m % a.Wg));
          }
        }
        const double turns = (double)pos * ((double)a.inv_freq[j] * 0.15915494309189533577);   // 1 / (2 pi)
        float sn, cs;
        sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
        turn[tid] = make_float2(cs, a.inverse ? -sn : sn);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kThreads + tid;
      if (i >= items) continue;
      int tok, unit;
      const T* src;
      T* dst;
      locate(i, tok, unit, src, dst);
      const float2* cs = turn + tok * P + unit * V;
      float x[2 * V], y[2 * V];
      unpack<T>(lo[u], x);
      unpack<T>(hi[u], x + V);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int ia = kHalves ? j : 2 * j, ib = kHalves ? V + j : 2 * j + 1;
        y[ia] = x[ia] * cs[j].x - x[ib] * cs[j].y;
        y[ib] = x[ia] * cs[j].y + x[ib] * cs[j].x;
      }
      uint4* o = reinterpret_cast<uint4*>(dst + unit * LO_STEP);
      o[0] = pack<T>(y);
      o[HI_OFF / V] = pack<T>(y + V);
    }
  }
}

template <typename T, int D>
cudaError_t launch(const RopeArgs& a, bool interleaved, cudaStream_t s) {
  constexpr int TOK = kThreads / (D / 2);
  const unsigned grid = (unsigned)((a.tokens + TOK - 1) / TOK);
  if (interleaved) rope_kernel<T, D, false><<<grid, kThreads, 0, s>>>(a);
  else rope_kernel<T, D, true><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, kda_dtype dt, int d, bool interleaved, cudaStream_t s, int* launches) {
  if (a.tokens == 0) return cudaSuccess;
  cudaError_t e;
  if (dt == KDA_DT_BF16)
    e = d == 128 ? launch<__nv_bfloat16, 128>(a, interleaved, s) : launch<__nv_bfloat16, 64>(a, interleaved, s);
  else
    e = d == 128 ? launch<float, 128>(a, interleaved, s) : launch<float, 64>(a, interleaved, s);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace kda
