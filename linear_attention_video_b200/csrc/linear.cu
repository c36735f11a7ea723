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
// bf16 problems run these launches on tcgen05 (linear_tc.cu).  The matrix products here, of fp32 problems, run on
// mma.sync in tf32 with each operand split into two terms (three products, 2^-22 relative): fp32 accuracy.
// Decays are lam^n = exp(n log lam) of whole n >= 0: never above 1, so nothing overflows however fast a head
// forgets, and the fp32 error of n log lam, 2^-25 |n log lam|, is largest beside e^-1.
#include <type_traits>

#include "common.cuh"

namespace kda {
namespace {

// lam^n; 1 at n = 0 whatever the decay.
__device__ __forceinline__ float decay_pow(float log_decay, int64_t n) {
  return n == 0 ? 1.f : expf((float)n * log_decay);
}
__device__ __forceinline__ int64_t item_tokens(const int32_t* lengths, int b, int64_t N) {
  if (!lengths) return N;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n > N ? N : n);
}

// ---------------------------------------------------------------------------
// tf32 products
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
// x = hi + lo to 22 bits.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = tf32(x);
  lo = tf32(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// The tensor cores truncate as they add to an accumulator, so a long chain drifts by 2^-24 per link; every 32-deep
// product starts from zero (12 links) and is added to its running sum by an ordinary rounded addition.
//
// d += A B, both operands in two terms (lo lo, 2^-22 of the product, is left out).
__device__ __forceinline__ void mma3(float (&d)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], float b0, float b1) {
  uint32_t bh[2], bl[2];
  split(b0, bh[0], bl[0]);
  split(b1, bh[1], bl[1]);
  mma8(d, ah, bl);
  mma8(d, al, bh);
  mma8(d, ah, bh);
}
__device__ __forceinline__ void split4(const float (&x)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) split(x[i], hi[i], lo[i]);
}

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

constexpr int TK = 32;       // tokens per shared-memory tile
constexpr int TQ = 64;       // output rows per CTA
// Tokens per segment.  These kernels are bound by their products, and a token's share of them grows with the segment
// (128: D + 64..128 columns of scores per row; 256: up to 256), while a state's traffic is small beside fp32 inputs.
constexpr int kSeg = 128;

// ---------------------------------------------------------------------------
// a segment's own contribution: local[x][y] = sum_t w_t x_t y_t^T
// w_t = lam^(s0+n-1-t) (state behind it), or lam^(t-s0+1) (gradient before it)
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) lin_local_kernel(LinLocalArgs a) {
  constexpr int LD = D + 8;            // rows 8 banks apart: A and B fragments without conflicts
  constexpr int RG = D / 16, CG = 8 / RG, NT = D / CG / 8;
  __shared__ float xs[TK * LD], ys[TK * LD];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int seg = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t s0 = (int64_t)seg * kSeg, end = min(item_tokens(a.lengths, b, a.N), s0 + kSeg);
  const float ld = a.log_decay[h];
  const int64_t stride = (int64_t)a.H * D;
  const float* x = static_cast<const float*>(a.x) + (int64_t)b * a.N * stride + (int64_t)h * D;
  const float* y = static_cast<const float*>(a.y) + (int64_t)b * a.N * stride + (int64_t)h * D;
  const int m0 = (warp % RG) * 16, n0 = (warp / RG) * (D / CG);
  float acc[NT][4] = {};
  for (int64_t t0 = s0; t0 < end; t0 += TK) {
    __syncthreads();
    for (int i = tid; i < TK * D / 4; i += 256) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      float4 fx = make_float4(0.f, 0.f, 0.f, 0.f), fy = fx;
      if (t0 + r < end) {
        fx = load4(x + (t0 + r) * stride + c);
        fy = load4(y + (t0 + r) * stride + c);
        const float w = decay_pow(ld, a.reverse ? t0 + r - s0 + 1 : end - 1 - t0 - r);
        fy.x *= w; fy.y *= w; fy.z *= w; fy.w *= w;
      }
      *reinterpret_cast<float4*>(xs + r * LD + c) = fx;
      *reinterpret_cast<float4*>(ys + r * LD + c) = fy;
    }
    __syncthreads();
    uint32_t ah[TK / 8][4], al[TK / 8][4];
#pragma unroll
    for (int k8 = 0; k8 < TK / 8; ++k8) {
      const float* xr = xs + (k8 * 8 + t) * LD + m0 + g;
      const float av[4] = {xr[0], xr[8], xr[4 * LD], xr[4 * LD + 8]};
      split4(av, ah[k8], al[k8]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float d[4] = {};
#pragma unroll
      for (int k8 = 0; k8 < TK / 8; ++k8) {
        const float* yr = ys + (k8 * 8 + t) * LD + n0 + n * 8 + g;
        mma3(d, ah[k8], al[k8], yr[0], yr[4 * LD]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] += d[e];
    }
  }
  float* out = a.local + (((int64_t)b * a.H + h) * a.n_seg + seg) * D * D;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    store2(out + (m0 + g) * D + n0 + n * 8 + 2 * t, acc[n][0], acc[n][1]);
    store2(out + (m0 + g + 8) * D + n0 + n * 8 + 2 * t, acc[n][2], acc[n][3]);
  }
}

// ---------------------------------------------------------------------------
// recurrence over segments, in place: local contributions become what enters each segment
// ---------------------------------------------------------------------------
// The decay of a whole segment multiplies a state again and again, so its fp32 rounding would add up; it is kept
// in two fp32 terms of the fp64 power.
struct Factor { float hi, lo; };
__device__ __forceinline__ Factor segment_factor(float log_decay, int64_t n) {
  const double f = n == 0 ? 1.0 : exp((double)n * (double)log_decay);
  const float hi = (float)f;
  return {hi, (float)(f - (double)hi)};
}

__global__ void __launch_bounds__(128) lin_scan_kernel(LinScanArgs a) {
  const int bh = blockIdx.y, h = bh % a.H, b = bh / a.H;
  const int64_t e = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 4;   // element of the D x D state
  const int64_t dd = a.dd, len = item_tokens(a.lengths, b, a.N);
  const float ld = a.log_decay[h];
  const int64_t last = len / a.seg;   // the segment that holds the end, if it is not whole
  const Factor whole = segment_factor(ld, a.seg), part = segment_factor(ld, len % a.seg);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.initial) S = *reinterpret_cast<const float4*>(a.initial + bh * dd + e);
  float* p = a.states + (int64_t)bh * a.n_seg * dd + e;
  constexpr int U = 4;
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
// the map: out_i = lam^e(i) X^(T) a_i + sum_j lam^|i-j| (a_i . b_j) c_j over i's segment
// ---------------------------------------------------------------------------
template <int D> struct MapSmem {
  static constexpr int LDA = D + 8;    // a, b: pairs of columns read as 8 bytes, rows 8 banks apart
  static constexpr int LDC = D + 4;    // c, X: rows 2t read by lane t, 8 banks apart
  static constexpr int LDX = TK + 8;   // X transposed: D rows of 32 columns, read as b
  static constexpr int stage = TK * LDA + TK * LDC;
  static_assert(stage >= D * LDX, "");
  static constexpr int floats = TQ * LDA + 2 * stage + kSeg;
  static constexpr int bytes = floats * (int)sizeof(float);
};

// 16 bytes global -> shared, zeros where `live` is false.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// The state's D rows and then the segment's tokens pass through two stages of 32 rows each: 32 rows of X are a tile
// of c whose scores are the rows of a themselves, scaled.  The k index of a product is permuted (2t, 2t+1 for t, t+4),
// which makes the scores' accumulators A operands as they are.
template <int D>
__global__ void __launch_bounds__(128) lin_map_kernel(LinMapArgs a) {
  using L = MapSmem<D>;
  constexpr int LDA = L::LDA, LDC = L::LDC, NT = D / 8, KT = TK / 8;
  extern __shared__ float sm[];
  float* as = sm;
  float* stages = as + TQ * LDA;
  float* pw = stages + 2 * L::stage;   // lam^n, n < kSeg
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t i0 = (int64_t)blockIdx.x * TQ;
  const int seg = (int)(i0 / kSeg);
  const int64_t s0 = (int64_t)seg * kSeg, len = item_tokens(a.lengths, b, a.N), end = min(len, s0 + kSeg);
  const float ld = a.log_decay[h];
  const int64_t stride = (int64_t)a.H * D, off = (int64_t)b * a.N * stride + (int64_t)h * D;
  const float *pa = static_cast<const float*>(a.a) + off, *pb = static_cast<const float*>(a.b) + off,
              *pc = static_cast<const float*>(a.c) + off;
  const bool has_state = i0 < end && (a.initial || (a.reverse ? seg != a.n_seg - 1 : seg != 0));
  const float* X = a.n_seg == 1 ? a.initial + ((int64_t)b * a.H + h) * D * D
                                : a.states + (((int64_t)b * a.H + h) * a.n_seg + seg) * D * D;
  const int64_t jb = a.reverse ? i0 : s0, je = a.reverse ? end : min(end, i0 + TQ);
  const int n_x = has_state ? D / TK : 0, n_kv = je > jb ? (int)((je - jb + TK - 1) / TK) : 0, n = n_x + n_kv;
  auto fetch = [&](int u) {
    float* bs = stages + (u & 1) * L::stage;
    float* cs = bs + TK * LDA;
    if (u >= n) {
    } else if (u >= n_x) {
      const int64_t j0 = jb + (int64_t)(u - n_x) * TK;
      for (int i = tid; i < TK * D / 4; i += 128) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        const bool live = j0 + r < end;   // tokens behind the end: zeros, whatever stands there
        const int64_t at = live ? (j0 + r) * stride + c : 0;
        copy16(bs + r * LDA + c, pb + at, live);
        copy16(cs + r * LDC + c, pc + at, live);
      }
    } else if (!a.transposed) {
      for (int i = tid; i < TK * D / 4; i += 128) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        copy16(cs + r * LDC + c, X + (u * TK + r) * D + c, true);
      }
    } else {
      for (int i = tid; i < TK * D / 4; i += 128) {
        const int r = i / (TK / 4), c = (i % (TK / 4)) * 4;
        copy16(bs + r * L::LDX + c, X + r * D + u * TK + c, true);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = tid; i < TQ * D / 4; i += 128) {   // rows behind the end: zero, and so is their output
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    const bool live = i0 + r < end;
    copy16(as + r * LDA + c, pa + (live ? (i0 + r) * stride + c : 0), live);
  }
  fetch(0);
  for (int i = tid; i < kSeg; i += 128) pw[i] = decay_pow(ld, i);
  const int r0 = warp * 16 + g;   // this thread's rows: r0 and r0 + 8
  float acc[NT][4] = {};
  const float w0 = decay_pow(ld, a.reverse ? max((int64_t)0, end - 1 - (i0 + r0)) : i0 + r0 - s0 + 1);
  const float w1 = decay_pow(ld, a.reverse ? max((int64_t)0, end - 1 - (i0 + r0 + 8)) : i0 + r0 + 8 - s0 + 1);
  for (int u = 0; u < n; ++u) {
    fetch(u + 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const float* bs = stages + (u & 1) * L::stage;
    const float* cs = bs + TK * LDA;
    uint32_t ph[KT][4], pl[KT][4];
    if (u < n_x) {
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const float2 x = *reinterpret_cast<const float2*>(as + r0 * LDA + u * TK + k * 8 + 2 * t);
        const float2 y = *reinterpret_cast<const float2*>(as + (r0 + 8) * LDA + u * TK + k * 8 + 2 * t);
        const float av[4] = {x.x * w0, y.x * w1, x.y * w0, y.y * w1};
        split4(av, ph[k], pl[k]);
      }
    } else {
      const int64_t j0 = jb + (int64_t)(u - n_x) * TK;
      float p[KT][4] = {}, q[KT][4];
#pragma unroll
      for (int k8 = 0; k8 < D / 8; ++k8) {
        if (k8 % 4 == 0) {
#pragma unroll
          for (int m = 0; m < KT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[m][e] = 0.f;
        }
        const float2 x = *reinterpret_cast<const float2*>(as + r0 * LDA + k8 * 8 + 2 * t);
        const float2 y = *reinterpret_cast<const float2*>(as + (r0 + 8) * LDA + k8 * 8 + 2 * t);
        const float av[4] = {x.x, y.x, x.y, y.y};
        uint32_t ah[4], al[4];
        split4(av, ah, al);
#pragma unroll
        for (int m = 0; m < KT; ++m) {
          const float2 w = *reinterpret_cast<const float2*>(bs + (m * 8 + g) * LDA + k8 * 8 + 2 * t);
          mma3(q[m], ah, al, w.x, w.y);
        }
        if (k8 % 4 == 3) {
#pragma unroll
          for (int m = 0; m < KT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[m][e] += q[m][e];
        }
      }
#pragma unroll
      for (int m = 0; m < KT; ++m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ahead = (int)(i0 - j0) + r0 + (e / 2) * 8 - m * 8 - 2 * t - (e & 1);
          const int dist = a.reverse ? -ahead : ahead;
          p[m][e] = dist < 0 ? 0.f : p[m][e] * pw[dist];
        }
        const float av[4] = {p[m][0], p[m][2], p[m][1], p[m][3]};
        split4(av, ph[m], pl[m]);
      }
    }
    const bool as_b = u < n_x && a.transposed;   // X transposed lies as b does: columns 2t, 2t+1 of row n
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      float d[4] = {};
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        float2 w;
        if (as_b) w = *reinterpret_cast<const float2*>(bs + (m * 8 + g) * L::LDX + k * 8 + 2 * t);
        else w = make_float2(cs[(k * 8 + 2 * t) * LDC + m * 8 + g], cs[(k * 8 + 2 * t + 1) * LDC + m * 8 + g]);
        mma3(d, ph[k], pl[k], w.x, w.y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][e] += d[e];
    }
    __syncthreads();   // this stage is fetched into again
  }
  float* out = static_cast<float*>(a.out) + off;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int64_t i = i0 + r0 + half * 8;
    if (i >= a.N) continue;
#pragma unroll
    for (int m = 0; m < NT; ++m) store2(out + i * stride + m * 8 + 2 * t, acc[m][2 * half], acc[m][2 * half + 1]);
  }
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

template <int D>
cudaError_t map(const LinMapArgs& m, const Dims& d, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(lin_map_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       MapSmem<D>::bytes);
  if (e != cudaSuccess) return e;
  lin_map_kernel<D><<<dim3((unsigned)((d.N + TQ - 1) / TQ), d.H, d.B), 128, MapSmem<D>::bytes, s>>>(m);
  return cudaGetLastError();
}

// Calls f with a value of the problem's element type and its head dim as a constant.
template <typename F> cudaError_t dispatch(const Dims& d, kda_dtype dt, F f) {
  using std::integral_constant;
  if (dt == KDA_DT_BF16)
    return d.dk == 128 ? f(__nv_bfloat16(), integral_constant<int, 128>()) : f(__nv_bfloat16(), integral_constant<int, 64>());
  return d.dk == 128 ? f(float(), integral_constant<int, 128>()) : f(float(), integral_constant<int, 64>());
}

cudaError_t launch_local(const Dims& d, const LinLocalArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.n_seg, d.H, d.B);
  if (d.dk == 128) lin_local_kernel<128><<<grid, 256, 0, s>>>(a);
  else lin_local_kernel<64><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_scan(const Dims& d, const LinScanArgs& a, cudaStream_t s) {
  lin_scan_kernel<<<dim3((unsigned)(a.dd / 512), d.B * d.H), 128, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_map(const Dims& d, const LinMapArgs& a, cudaStream_t s) {
  return d.dk == 128 ? map<128>(a, d, s) : map<64>(a, d, s);
}

// What a pass over one problem needs to know: its kernels' segment length, and the three launches.
struct Pass {
  const Dims& d;
  bool tc;
  int seg, n_seg;
  const float* log_decay;
  const int32_t* lengths;
  uint32_t* status;
  cudaStream_t s;
  int* launches;

  Pass(const Dims& d_, kda_dtype dt, const float* ld, const int32_t* len, uint32_t* st, cudaStream_t s_, int* l)
      : d(d_), tc(dt == KDA_DT_BF16), seg(tc ? linear_tc_segment(d_) : kSeg),
        n_seg((int)((d_.N + seg - 1) / seg)), log_decay(ld), lengths(len), status(st), s(s_), launches(l) {}

  size_t state_floats() const { return (size_t)d.B * d.H * n_seg * d.dk * d.dv; }

  // What enters every segment (in the direction of the pass) of sum w x y^T; `last`: what leaves the last one.
  cudaError_t states(const void* x, const void* y, float* out, const float* initial, float* last, bool reverse) {
    const bool local = n_seg > 1 || (n_seg == 1 && last);
    if (!local && !last && !(tc && initial)) return cudaSuccess;   // nothing enters, or the initial state as it is
    cudaError_t e;
    if (local) {
      const LinLocalArgs a{x, y, log_decay, lengths, out, d.N, d.H, n_seg, reverse};
      if ((e = tc ? launch_linear_tc_local(d, a, status, s) : launch_local(d, a, s)) != cudaSuccess) return e;
      *launches += 1;
    }
    const LinScanArgs a{out, initial, last, log_decay, lengths, d.N, (int64_t)d.dk * d.dv, seg, d.H, n_seg, reverse};
    if ((e = tc ? launch_linear_tc_scan(d, a, local, s) : launch_scan(d, a, s)) != cudaSuccess) return e;
    *launches += 1;
    return cudaSuccess;
  }

  cudaError_t map(const void* a, const void* b, const void* c, void* out, const float* st, const float* initial,
                  bool reverse, bool transposed) {
    if (n_seg == 0) return cudaSuccess;
    const LinMapArgs m{a, b, c, out, st, initial, log_decay, lengths, d.N, d.H, n_seg, reverse, transposed};
    const cudaError_t e = tc ? launch_linear_tc_map(d, m, status, s) : launch_map(d, m, s);
    if (e == cudaSuccess) *launches += 1;
    return e;
  }
};

size_t state_bytes(const Dims& d, kda_dtype dt) {
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
  if ((e = p.states(k, v, states, S0, SN, false)) != cudaSuccess) return e;
  return p.map(q, k, v, o, states, S0, false, false);
}

cudaError_t launch_linear_bwd(const Dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                              const float* log_decay, const int32_t* lengths, const float* S0, const void* d_o,
                              const float* dSN, void* dq, void* dk, void* dv, float* dS0, void* scratch,
                              uint32_t* status, cudaStream_t s, int* launches) {
  Pass p(d, dt, log_decay, lengths, status, s, launches);
  float* states = static_cast<float*>(scratch);
  float* grads = states + p.state_floats();
  cudaError_t e;
  if ((e = p.states(k, v, states, S0, nullptr, false)) != cudaSuccess) return e;
  if ((e = p.states(q, d_o, grads, dSN, dS0, true)) != cudaSuccess) return e;
  if ((e = p.map(d_o, v, k, dq, states, S0, false, true)) != cudaSuccess) return e;
  if ((e = p.map(v, d_o, q, dk, grads, dSN, true, true)) != cudaSuccess) return e;
  return p.map(k, q, d_o, dv, grads, dSN, true, false);
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
