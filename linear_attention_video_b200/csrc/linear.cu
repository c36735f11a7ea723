// Linear attention with a fixed decay per head: S_t = lam S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.
//
// The token axis is cut into segments of L tokens.  With s0 the first token of i's segment, n its tokens and S
// the state entering it,
//   o_i  = lam^(i-s0+1) S^T q_i + sum_{s0 <= j <= i} lam^(i-j) (q_i . k_j) v_j
// and with G the gradient that reaches the state leaving the segment
//   dq_i = lam^(i-s0+1) S do_i     + sum_{j <= i} lam^(i-j) (do_i . v_j) k_j
//   dk_j = lam^(s0+n-1-j) G v_j    + sum_{i >= j} lam^(i-j) (v_j . do_i) q_i
//   dv_j = lam^(s0+n-1-j) G^T k_j  + sum_{i >= j} lam^(i-j) (k_j . q_i) do_i
// so all four are one map over (a, b, c, state) in one of two directions:
//   out_i = lam^e(i) X^(T) a_i + sum_j lam^|i-j| (a_i . b_j) c_j.
// Three launches: every segment's own contribution sum_t w_t x_t y_t^T to the state behind it (before it, for
// G); the recurrence over segments, element by element; the map, whose tiles are then independent.
//
// The local sums and the map run on the tensor cores, in linear_tc.cu for bf16 problems and linear_tc32.cu for fp32
// ones; here are the recurrence of fp32 problems, the single token and the passes over a problem.
#include <initializer_list>
#include <type_traits>

#include "linear_tc.cuh"

namespace kda {
namespace {

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(&u)[0]);
  const float2 b = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(&u)[1]);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// ---------------------------------------------------------------------------
// recurrence over segments, in place: local contributions become what enters each segment
// ---------------------------------------------------------------------------
template <bool ONE>
__global__ void __launch_bounds__(128) lin_scan_kernel(const __grid_constant__ LinScanSets sets) {
  const int per_set = ONE ? gridDim.x : gridDim.x / sets.n, which = ONE ? 0 : blockIdx.x / per_set;
  const LinScanArgs& a = sets.set[which];
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = (int64_t)b * a.H + h;
  const int64_t e = ((int64_t)(blockIdx.x - which * per_set) * 128 + threadIdx.x) * 4;   // element of the D x D state
  const int64_t dd = a.dd, len = item_tokens(a.lengths, b, a.N);
  const float ld = a.log_decay[h];
  const int64_t last = len / a.seg;   // the segment that holds the end, if it is not whole
  const Factor whole = segment_factor(ld, a.seg), part = segment_factor(ld, len % a.seg);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.initial) S = *reinterpret_cast<const float4*>(a.initial + bh * dd + e);
  float* p = a.states + bh * a.n_seg * dd + e;
  // States fetched at once.  33,272 x 16 x 128: 6 92 us, 4 104, 8 197; 16 x 64: 49, 62, 57; 2 x 16,000 x 16 x 128: 84, 83,
  // 134; two sets of 33,272 x 16 x 128: 4 177, 8 285.
  constexpr int U = ONE ? 6 : 4;
  for (int c0 = 0; c0 < a.n_seg; c0 += U) {
    float4 loc[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u < a.n_seg)
        loc[u] = *reinterpret_cast<const float4*>(p + (int64_t)(a.reverse ? a.n_seg - 1 - c0 - u : c0 + u) * dd);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u >= a.n_seg) break;
      const int c = a.reverse ? a.n_seg - 1 - c0 - u : c0 + u;
      *reinterpret_cast<float4*>(p + (int64_t)c * dd) = S;
      if (c > last) continue;   // behind the end: no tokens
      const Factor f = c == last ? part : whole;
      S.x = fmaf(f.hi, S.x, fmaf(f.lo, S.x, loc[u].x));
      S.y = fmaf(f.hi, S.y, fmaf(f.lo, S.y, loc[u].y));
      S.z = fmaf(f.hi, S.z, fmaf(f.lo, S.z, loc[u].z));
      S.w = fmaf(f.hi, S.w, fmaf(f.lo, S.w, loc[u].w));
    }
  }
  if (a.final) *reinterpret_cast<float4*>(a.final + bh * dd + e) = S;
}

// ---------------------------------------------------------------------------
// one token: state out = lam state in + k v^T, o = (state out)^T q
// Bound by the state's 8 D^2 bytes per (item, head).  Columns of the state are independent: a CTA takes 32 of
// them, 8 lanes x 16 bytes per row, and has all its loads in flight before the first product.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(256) lin_step_kernel(LinStepArgs a) {
  constexpr int R = D / 32;   // rows per thread
  __shared__ float4 part[8][8];
  const int tid = threadIdx.x, cx = tid % 8, ry = tid / 8;
  const int64_t bh = (int64_t)blockIdx.z * a.H + blockIdx.y;
  const int col = blockIdx.x * 32 + cx * 4;
  const float* in = a.state_in + bh * D * D + col;
  float* out = a.state_out + bh * D * D + col;
  float4 S[R];
#pragma unroll
  for (int i = 0; i < R; ++i) S[i] = *reinterpret_cast<const float4*>(in + (ry + 32 * i) * D);
  const float lam = decay_pow(a.log_decay[blockIdx.y], 1);
  const float4 v = load4(static_cast<const T*>(a.v) + bh * D + col);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = ry + 32 * i;
    const float k = to_f32(static_cast<const T*>(a.k)[bh * D + r]), q = to_f32(static_cast<const T*>(a.q)[bh * D + r]);
    S[i].x = fmaf(k, v.x, lam * S[i].x);
    S[i].y = fmaf(k, v.y, lam * S[i].y);
    S[i].z = fmaf(k, v.z, lam * S[i].z);
    S[i].w = fmaf(k, v.w, lam * S[i].w);
    *reinterpret_cast<float4*>(out + r * D) = S[i];
    o.x = fmaf(q, S[i].x, o.x);
    o.y = fmaf(q, S[i].y, o.y);
    o.z = fmaf(q, S[i].z, o.z);
    o.w = fmaf(q, S[i].w, o.w);
  }
#pragma unroll
  for (int m = 8; m < 32; m *= 2) {   // the four rows of a warp
    o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
  }
  if (tid % 32 < 8) part[tid / 32][cx] = o;
  __syncthreads();
  if (tid >= 8) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) {
    const float4 x = part[w][cx];
    o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
  }
  T* y = static_cast<T*>(a.o) + bh * D + col;
  store2(y, o.x, o.y);
  store2(y + 2, o.z, o.w);
}

// Calls f with a value of the problem's element type and its head dim as a constant.
template <typename F> cudaError_t dispatch(const Dims& d, kda_dtype dt, F f) {
  using std::integral_constant;
  if (dt == KDA_DT_BF16)
    return d.dk == 128 ? f(__nv_bfloat16(), integral_constant<int, 128>()) : f(__nv_bfloat16(), integral_constant<int, 64>());
  return d.dk == 128 ? f(float(), integral_constant<int, 128>()) : f(float(), integral_constant<int, 64>());
}

cudaError_t launch_scan(const Dims& d, const LinScanSets& a, cudaStream_t s) {
  const auto kernel = a.n == 1 ? lin_scan_kernel<true> : lin_scan_kernel<false>;
  kernel<<<dim3((unsigned)(a.set[0].dd / 512 * a.n), d.H, d.B), 128, 0, s>>>(a);
  return cudaGetLastError();
}

// Of the states in one direction: the sums w x y^T, what they start from, and where they go.
struct States {
  const void *x, *y;
  float* out;             // what enters every segment
  const float* initial;
  float* last;            // what leaves the last one, or NULL
  bool reverse;
};
// What a pass over one problem needs to know: its kernels' segment length, and the three launches.
struct Pass {
  const Dims& d;
  bool bf16;   // the states between the launches are images (linear_tc.cu), not fp32 matrices
  int seg, n_seg;
  const float* log_decay;
  const int32_t* lengths;
  uint32_t* status;
  cudaStream_t s;
  int* launches;

  Pass(const Dims& d_, kda_dtype dt, const float* ld, const int32_t* len, uint32_t* st, cudaStream_t s_, int* l)
      : d(d_), bf16(dt == KDA_DT_BF16), seg(bf16 ? linear_tc_segment(d_) : linear_tc32_segment()),
        n_seg((int)((d_.N + seg - 1) / seg)), log_decay(ld), lengths(len), status(st), s(s_), launches(l) {}

  size_t state_floats() const { return (size_t)d.B * d.H * n_seg * d.dk * d.dv; }

  cudaError_t states(std::initializer_list<States> all) {
    LinLocalSets l = {};
    LinScanSets c = {};
    for (const States& w : all) {
      const bool local = n_seg > 1 || (n_seg == 1 && w.last);
      if (!local && !w.last && !(bf16 && w.initial)) continue;   // nothing enters, or the initial state as it is
      if (local) l.set[l.n++] = {w.x, w.y, log_decay, lengths, w.out, d.N, d.H, n_seg, seg, w.reverse};
      c.set[c.n++] = {w.out, w.initial, w.last, log_decay, lengths, d.N, (int64_t)d.dk * d.dv, seg, d.H, n_seg, w.reverse, local};
    }
    cudaError_t e;
    if (l.n) {
      if ((e = bf16 ? launch_linear_tc_local(d, l, status, s) : launch_linear_tc32_local(d, l, status, s)) != cudaSuccess) return e;
      *launches += 1;
    }
    if (c.n) {
      if ((e = bf16 ? launch_linear_tc_scan(d, c, s) : launch_scan(d, c, s)) != cudaSuccess) return e;
      *launches += 1;
    }
    return cudaSuccess;
  }

  LinMapArgs one(const void* a, const void* b, const void* c, void* out, const float* st, const float* initial,
                 bool reverse, bool transposed) const {
    return {a, b, c, out, st, initial, log_decay, lengths, d.N, d.H, n_seg, seg, reverse, transposed};
  }
  cudaError_t map(const LinMapSets& m) {
    if (n_seg == 0) return cudaSuccess;
    const cudaError_t e = bf16 ? launch_linear_tc_map(d, m, status, s) : launch_linear_tc32_map(d, m, status, s);
    if (e == cudaSuccess) *launches += 1;
    return e;
  }
};

// Of the states between the launches, for every problem up to this one's size.
size_t state_bytes(const Dims& d, kda_dtype dt) {
  if (dt == KDA_DT_BF16) return (size_t)linear_tc_most_states(d) * d.dk * d.dv * sizeof(float);
  return Pass(d, dt, nullptr, nullptr, nullptr, nullptr, nullptr).state_floats() * sizeof(float);
}

}  // namespace

size_t linear_fwd_scratch(const Dims& d, kda_dtype dt) { return state_bytes(d, dt); }
size_t linear_bwd_scratch(const Dims& d, kda_dtype dt) { return 2 * state_bytes(d, dt); }

cudaError_t launch_linear_fwd(const Dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                              const float* log_decay, const int32_t* lengths, const float* S0, void* o, float* SN,
                              void* scratch, uint32_t* status, cudaStream_t s, int* launches) {
  Pass p(d, dt, log_decay, lengths, status, s, launches);
  float* states = static_cast<float*>(scratch);
  cudaError_t e;
  if ((e = p.states({{k, v, states, S0, SN, false}})) != cudaSuccess) return e;
  return p.map({{p.one(q, k, v, o, states, S0, false, false)}, 1});
}

cudaError_t launch_linear_bwd(const Dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                              const float* log_decay, const int32_t* lengths, const float* S0, const void* d_o,
                              const float* dSN, void* dq, void* dk, void* dv, float* dS0, void* scratch,
                              uint32_t* status, cudaStream_t s, int* launches) {
  Pass p(d, dt, log_decay, lengths, status, s, launches);
  float* states = static_cast<float*>(scratch);
  float* grads = states + p.state_floats();
  cudaError_t e;
  if ((e = p.states({{k, v, states, S0, nullptr, false}, {q, d_o, grads, dSN, dS0, true}})) != cudaSuccess) return e;
  return p.map({{p.one(d_o, v, k, dq, states, S0, false, true), p.one(v, d_o, q, dk, grads, dSN, true, true),
                 p.one(k, q, d_o, dv, grads, dSN, true, false)}, 3});
}

cudaError_t launch_linear_step(const Dims& d, kda_dtype dt, const LinStepArgs& a, cudaStream_t s, int* launches) {
  const cudaError_t e = dispatch(d, dt, [&](auto t, auto D) {
    lin_step_kernel<decltype(t), decltype(D)::value><<<dim3(d.dv / 32, d.H, d.B), 256, 0, s>>>(a);
    return cudaGetLastError();
  });
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace kda
