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

// 16 bytes as fp32 values and back (bf16 in pairs: one instruction per element in, half of one out).
template <typename T> struct Vec { static constexpr int n = 16 / sizeof(T); };
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = reinterpret_cast<const uint32_t&>(v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kHalves: pair j is (j, j + D/2); otherwise (2j, 2j + 1).
template <typename T, int D, bool kHalves>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(RopeArgs a) {
  constexpr int P = D / 2, TOK = kThreads / P, V = Vec<T>::n;
  // A unit is two vectors, V elements at u V and at P + u V, which hold V whole pairs either way; neighbouring threads'
  // vectors are neighbours (interleaved pairs taken as 2 V elements in a row: 109 us for 33,272 tokens, so 82).
  constexpr int UNITS = P / V;
  constexpr int LINES = kThreads / UNITS;        // lines (token, tensor, head) per sweep of the CTA
  // (cos, sin) of a token's pairs, two pairs to 16 bytes, in the order in which neighbouring threads read neighbouring
  // 16 bytes (by pair number their reads meet in a quarter of the banks: 94 us for 33,272 tokens, so 83).
  __shared__ float2 turn[TOK * P];
  auto slot = [](int j) {
    if constexpr (kHalves) return (j % V / 2 * UNITS + j / V) * 2 + j % 2;
    const int r = j % (P / 2);
    return ((j / (P / 2) * (V / 4) + r % (V / 2) / 2) * UNITS + r / (V / 2)) * 2 + j % 2;
  };
  const int tid = threadIdx.x, unit = tid % UNITS;
  const uint32_t tok0 = blockIdx.x * (uint32_t)TOK;
  const int n_tok = min(TOK, (int)(a.tokens - tok0)), per_tok = a.n_tensors * a.H;
  // this thread's next line: token tok, line r of its tensors' heads; offset of its first element
  int tok = 0, r = tid / UNITS;
  auto settle = [&] { while (r >= per_tok) r -= per_tok, ++tok; };
  auto offset = [&](int& tensor) {
    tensor = r >= a.H;
    return ((int64_t)(tok0 + tok) * a.H + (tensor ? r - a.H : r)) * D + unit * V;
  };
  settle();
  bool first = true;
  while (true) {
    uint4 lo[kUnroll], hi[kUnroll];
    int64_t off[kUnroll];
    int which[kUnroll];   // -1: no line; else 2 * token + tensor
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      which[u] = -1;
      if (tok < n_tok) {
        int tensor;
        off[u] = offset(tensor);
        which[u] = 2 * tok + tensor;
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const T*>(tensor ? a.x[1] : a.x[0]) + off[u]);
        lo[u] = s[0];
        hi[u] = s[P / V];
        r += LINES;
        settle();
      }
    }
    if (first) {   // the angles, while the first loads are in flight
      first = false;
      const int j = tid % P;
      if (tid / P < n_tok) {
        const int axis = j < a.pairs_t ? 0 : (j < a.pairs_t + a.pairs_h ? 1 : 2);
        const uint32_t t = tok0 + tid / P;
        double pos;
        if (a.positions) {
          pos = (double)a.positions[(int64_t)t * 3 + axis];
        } else {
          uint32_t n = t % (uint32_t)a.N;
          if (n >= (uint32_t)a.text) {
            const uint32_t m = n - (uint32_t)a.text, row = m / (uint32_t)a.Wg;
            n = (uint32_t)a.text + (axis == 2 ? m - row * a.Wg : axis == 1 ? row % (uint32_t)a.Hg : row / (uint32_t)a.Hg);
          }
          pos = (double)n;
        }
        const double turns = pos * ((double)a.inv_freq[j] * 0.15915494309189533577);   // 1 / (2 pi)
        float sn, cs;
        sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
        turn[tid / P * P + slot(j)] = make_float2(cs, a.inverse ? -sn : sn);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (which[u] < 0) continue;
      const float4* cs = reinterpret_cast<const float4*>(turn + (which[u] >> 1) * P) + unit;
      float xl[V], xh[V], yl[V], yh[V];
      unpack(lo[u], xl);
      unpack(hi[u], xh);
      if constexpr (kHalves) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const float4 t = cs[j / 2 * UNITS];   // cos, sin of pairs j and j + 1
          yl[j] = xl[j] * t.x - xh[j] * t.y;
          yh[j] = xl[j] * t.y + xh[j] * t.x;
          yl[j + 1] = xl[j + 1] * t.z - xh[j + 1] * t.w;
          yh[j + 1] = xl[j + 1] * t.w + xh[j + 1] * t.z;
        }
      } else {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          float(&x)[V] = v ? xh : xl;
          float(&y)[V] = v ? yh : yl;
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const float4 t = cs[(v * (V / 4) + i / 4) * UNITS];
            y[i] = x[i] * t.x - x[i + 1] * t.y;
            y[i + 1] = x[i] * t.y + x[i + 1] * t.x;
            y[i + 2] = x[i + 2] * t.z - x[i + 3] * t.w;
            y[i + 3] = x[i + 2] * t.w + x[i + 3] * t.z;
          }
        }
      }
      uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(which[u] & 1 ? a.y[1] : a.y[0]) + off[u]);
      o[0] = pack(yl);
      o[P / V] = pack(yh);
    }
    if (which[kUnroll - 1] < 0 || tok >= n_tok) break;
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
