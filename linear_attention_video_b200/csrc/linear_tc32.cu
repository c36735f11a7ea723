// Linear attention with a fixed decay per head on the tensor cores (tcgen05), fp32 problems.
//
// The local sums and the map of linear.cu with every fp32 operand as three bf16 terms (24 bits): a product is the six
// products of terms i, j with i + j <= 4 (from 1), what is left out being 2^-24 of it.  On these units that is fp32
// accuracy at a sixth of the bf16 rate; tf32 would need three products at half the rate and take as long.
// The tensor cores truncate as they add, so the small products are added first, and sums over many tiles keep them in
// an accumulator of their own.
//
// Copies pass through registers, where eight warps split them on the way to the operand images; the next tile's loads
// are in flight meanwhile.
#include "linear_tc.cuh"

namespace kda {
namespace {

using namespace tc;

// Tokens per segment: 2 x 1237 x 6 x 64 forward 29 us (256: 39), 33,272 x 16 x 128 1.01 ms (256: 1.00): a shorter
// segment has fewer tiles in a row per CTA, a longer one fewer states.
constexpr int kSeg = 128;
constexpr int TM = 128;        // rows per CTA of the map
constexpr int TK = 64;         // tokens per tile
constexpr int kThreads = 288;  // eight working warps, one for the products

// Eight fp32 as three bf16 terms: 16 bytes each at off, off + stride, off + 2 stride.
__device__ __forceinline__ void store_terms(uint8_t* img, int stride, const float4& u, const float4& v) {
  uint64_t f[4] = {pair2(u.x, u.y), pair2(u.z, u.w), pair2(v.x, v.y), pair2(v.z, v.w)};
  uint4 a, b, c;
  uint32_t *pa = &a.x, *pb = &b.x, *pc = &c.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    pa[j] = take2(f[j]);
    pb[j] = take2(f[j]);
    pc[j] = pack2(f[j]);
  }
  *reinterpret_cast<uint4*>(img) = a;
  *reinterpret_cast<uint4*>(img + stride) = b;
  *reinterpret_cast<uint4*>(img + 2 * stride) = c;
}
__device__ __forceinline__ float4 scaled(const float4& u, float w) { return make_float4(u.x * w, u.y * w, u.z * w, u.w * w); }
__device__ __forceinline__ float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }

// The six products of three terms each, the smallest first: (0, 2) (2, 0) (1, 1) (0, 1) (1, 0) (0, 0).
__device__ __forceinline__ uint32_t term_a(int p) { return (0x010120u >> (4 * p)) & 15u; }
__device__ __forceinline__ uint32_t term_b(int p) { return (0x001102u >> (4 * p)) & 15u; }

// ---------------------------------------------------------------------------
// local: one CTA per (segment, 128 channels, item), two heads of 64 side by side as in the bf16 kernel
// ---------------------------------------------------------------------------
constexpr int kLocalSmem = 1024 + 6 * 16384;

template <int D, bool ONE>
__global__ void __launch_bounds__(kThreads, 2) lin_tc32_local_kernel(const __grid_constant__ LinLocalSets sets, uint32_t* status) {
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t ready, done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_slot;
  uint8_t* xs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* ys = xs + 3 * 16384;
  volatile int* abort_flag = &abort_slot;
  const int tid = threadIdx.x, warp = tid / 32;
  constexpr int HP = 128 / D;   // heads per CTA
  const int per_set = ONE ? gridDim.x : gridDim.x / sets.n, which = ONE ? 0 : blockIdx.x / per_set;
  const LinLocalArgs& a = sets.set[which];
  const int seg = blockIdx.x - which * per_set, h0 = blockIdx.y * HP, b = blockIdx.z;
  const int64_t s0 = (int64_t)seg * kSeg, len = item_tokens(a.lengths, b, a.N);
  const int n_tok = (int)max((int64_t)0, min(len - s0, (int64_t)kSeg)), n_tiles = (n_tok + TK - 1) / TK;
  if (tid == 0) {
    mbar_init(&ready, 256);
    mbar_init(&done, 1);
    abort_slot = 0;
    fence_mbar_init();
  }
  if (warp == 8) { tmem_alloc(&tmem_slot, 256); tmem_relinquish(); }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = tmem_slot;
  bool ok = true;

  if (warp == 8) {
    if (tid == 256) {
      constexpr uint32_t id = idesc_bf16(128, 128, true, true);
      const uint64_t dx = mdesc0(smem_u32(xs), 8192), dy = mdesc0(smem_u32(ys), 8192);
      for (int t = 0; t < n_tiles; ++t) {
        ok = wait_or_abort(&ready, t & 1, abort_flag);
        if (!ok) break;
        fence_after_sync();
#pragma unroll 1
        for (int p = 0; p < 6; ++p) {   // the products of the first terms to one accumulator, the rest to the other
          const uint64_t da = dx + term_a(p) * (16384 >> 4), db = dy + term_b(p) * (16384 >> 4);
#pragma unroll
          for (int k = 0; k < TK / 16; ++k) mma_ss(p == 5 ? tm : tm + 128, da + mstep(k), db + mstep(k), id, t || k || (p && p < 5));
        }
        mma_commit(&done);
      }
    }
    __syncwarp();
  } else {
    const int c8 = tid % 16, r0 = tid / 16;   // this thread's 8 channels, its tokens r0 + 16 i
    const bool there = D == 128 || h0 + c8 / 8 < a.H;
    const int h = D == 128 ? h0 : min(h0 + c8 / 8, a.H - 1), ch = D == 128 ? c8 * 8 : (c8 % 8) * 8;
    const float ld = a.log_decay[h];
    const int64_t stride = (int64_t)a.H * D, off = ((int64_t)b * a.N + s0) * stride + (int64_t)h * D + ch;
    const float *x = static_cast<const float*>(a.x) + off, *y = static_cast<const float*>(a.y) + off;
    float roww[4];   // the weight of a token of a whole tile: its row's power times the tile's
#pragma unroll
    for (int i = 0; i < 4; ++i) roww[i] = decay_pow(ld, a.reverse ? r0 + 16 * i + 1 : TK - 1 - r0 - 16 * i);
    float4 fx[4][2], fy[4][2];
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = t * TK + r0 + 16 * i;
        if (there && tok < n_tok) {   // behind the end: zeros, whatever stands there
          const float4 *px = reinterpret_cast<const float4*>(x + tok * stride), *py = reinterpret_cast<const float4*>(y + tok * stride);
          fx[i][0] = px[0], fx[i][1] = px[1], fy[i][0] = py[0], fy[i][1] = py[1];
        } else {
          fx[i][0] = fx[i][1] = fy[i][0] = fy[i][1] = zero4();
        }
      }
    };
    fetch(0);
    for (int t = 0; t < n_tiles; ++t) {
      const int left = n_tok - t * TK;   // tokens from this tile on
      const float tilew = decay_pow(ld, a.reverse ? t * TK : max(0, left - TK));
      if (t > 0) ok = warp_wait(&done, (t - 1) & 1, abort_flag);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 16 * i;
        const uint32_t at = image_off(TK, r, c8);
        const float w = !a.reverse && left < TK ? decay_pow(ld, max(0, left - 1 - r)) : roww[i] * tilew;
        store_terms(xs + at, 16384, fx[i][0], fx[i][1]);
        store_terms(ys + at, 16384, scaled(fy[i][0], w), scaled(fy[i][1], w));
      }
      fence_proxy_async();
      mbar_arrive(&ready);
      if (t + 1 < n_tiles) fetch(t + 1);
    }
    if (ok && n_tiles) ok = warp_wait(&done, (n_tiles - 1) & 1, abort_flag);
    if (ok) {
      fence_after_sync();
      // lane = row of the 128 x 128 block; head = row / D owns columns of the same block
      const int row = (warp & 3) * 32 + (tid & 31), hp = row / D, r = row % D;
      constexpr int COLS = D / 2;   // columns of this warp: a half of its head's
      const int c0 = (warp >> 2) * COLS;
      const uint32_t at = tm + ((uint32_t)((warp & 3) * 32) << 16) + hp * (D % 128) + c0;
      float* out = a.local + ((((int64_t)b * a.H + h0 + hp) * a.n_seg + seg) * D + r) * D + c0;
#pragma unroll 1
      for (int c = 0; c < COLS; c += 16) {
        float v[16], w[16];
        if (n_tiles) {
          tmem_ld16(at + c, v);
          tmem_ld16(at + 128 + c, w);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = w[i] = 0.f;
        }
        if (h0 + hp < a.H) {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(out + c + i) = make_float4(v[i] + w[i], v[i + 1] + w[i + 1], v[i + 2] + w[i + 2], v[i + 3] + w[i + 3]);
        }
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(status, KDA_ERR_TIMEOUT);
  fence_after_sync();
  if (warp == 8) tmem_dealloc(tm, 256);
}

// ---------------------------------------------------------------------------
// map
// ---------------------------------------------------------------------------
// One CTA per 128 output rows.  The D rows of the state and then the segment's tokens pass in tiles of 64:
//   a tile of tokens: S = a b^T, P = S * decay;  a tile of the state: P = the rows of a themselves, scaled by lam^e(i);
//   then O += P c, where c is the tile of tokens or of X.
// P goes to tensor memory as three terms, two of them over S.  Two threads share a row, a group of 32 columns each; b of the next tile is
// split while O += P c runs, c while S = a b^T does.
template <int D> struct MapSmem {
  static constexpr int a_term = TM * D * 2, t_term = TK * D * 2;   // one term's image of a; of b, c or X
  static constexpr int bytes = 1024 + 3 * a_term + 6 * t_term;
};
// S, and P's first two terms over it, 64 columns; P's third term 32; O of the first terms' product and of the others
template <int D> constexpr uint32_t kMapTmem = D == 128 ? 512 : 256;

template <int D, bool REV>
__device__ __forceinline__ void map_tile(const CUtensorMap& out_map, const LinMapArgs& a, int tile, uint32_t* status) {
  using L = MapSmem<D>;
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t bar_b, bar_s, bar_p, bar_o;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_slot;
  __shared__ float diag[64];               // lam^n at 32 + n, zeros below
  __shared__ float power32[2 * kSeg / 64];   // lam^(32 n)
  uint8_t* as = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* bs = as + 3 * L::a_term;
  uint8_t* cs = bs + 3 * L::t_term;
  volatile int* abort_flag = &abort_slot;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t i0 = (int64_t)tile * TM, len = item_tokens(a.lengths, b, a.N);
  const int seg = (int)(i0 / kSeg);
  const int64_t s0 = (int64_t)seg * kSeg, end = min(len, s0 + kSeg), stride = (int64_t)a.H * D;
  const int64_t head = (int64_t)b * a.N * stride + (int64_t)h * D;
  if (i0 >= len) {   // behind the item's end: zeros
    float* out = static_cast<float*>(a.out) + head + i0 * stride;
    const int n = (int)min((int64_t)TM, a.N - i0) * (D / 4);
    for (int i = tid; i < n; i += kThreads) *reinterpret_cast<float4*>(out + (i / (D / 4)) * stride + (i % (D / 4)) * 4) = zero4();
    return;
  }
  const bool has_state = a.initial || (REV ? seg != a.n_seg - 1 : seg != 0);
  const int64_t j_first = REV ? i0 : s0;
  const int to_end = (int)((REV ? end : min(end, i0 + TM)) - j_first);   // tokens that the rows look at
  const int n_x = has_state ? D / 64 : 0, n = n_x + (to_end + TK - 1) / TK;
  const float ld = a.log_decay[h];
  if (tid == 0) {
    mbar_init(&bar_b, 256);
    mbar_init(&bar_s, 1);
    mbar_init(&bar_p, 256);
    mbar_init(&bar_o, 1);
    abort_slot = 0;
    fence_mbar_init();
  }
  if (tid < 64) diag[tid] = tid < 32 ? 0.f : decay_pow(ld, tid - 32);
  else if (tid < 64 + 2 * kSeg / 64) power32[tid - 64] = decay_pow(ld, 32 * (tid - 64));
  if (warp == 8) { tmem_alloc(&tmem_slot, kMapTmem<D>); tmem_relinquish(); }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm_s = tmem_slot, tm_p2 = tm_s + 64, tm_o = tm_s + 96, tm_r = tm_o + D;
  bool ok = true;

  if (warp == 8) {
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16(128, TK, false, false);
      const uint64_t da = kdesc0(smem_u32(as)), db = kdesc0(smem_u32(bs));
      const uint64_t dc_mn = mdesc0(smem_u32(cs), TK * 128), dc_k = kdesc0(smem_u32(cs));
      for (int u = 0; ok && u < n; ++u) {
        if (u >= n_x) {
          ok = wait_or_abort(&bar_b, (u - n_x) & 1, abort_flag);
          if (ok && u > 0) ok = wait_or_abort(&bar_o, (u - 1) & 1, abort_flag);   // P over S has been read
          if (!ok) break;
          fence_after_sync();
#pragma unroll 1
          for (int p = 0; p < 6; ++p) {
            const uint64_t pa = da + term_a(p) * (L::a_term >> 4), pb = db + term_b(p) * (L::t_term >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) mma_ss(tm_s, pa + kstep(k, TM * 128), pb + kstep(k, TK * 128), id_s, p || k);
          }
          mma_commit(&bar_s);
        }
        ok = wait_or_abort(&bar_p, u & 1, abort_flag);
        if (!ok) break;
        fence_after_sync();
        const bool k_major = u < n_x && a.transposed;   // X transposed lies with its columns along k
        const uint32_t id = idesc_bf16(128, D, false, !k_major);
#pragma unroll 1
        for (int p = 0; p < 6; ++p) {
          const uint64_t pc = (k_major ? dc_k : dc_mn) + term_b(p) * (L::t_term >> 4);
#pragma unroll
          for (int k = 0; k < TK / 16; ++k) {
            const uint32_t pa = term_a(p) == 2 ? tm_p2 + 8 * k : tm_s + 32 * (k >> 1) + 16 * term_a(p) + 8 * (k & 1);
            mma_ts(p == 5 ? tm_o : tm_r, pa, pc + (k_major ? kstep(k, 0) : mstep(k)), id, u || k || (p && p < 5));
          }
        }
        mma_commit(&bar_o);
      }
    }
    __syncwarp();
  } else {
    const int row = tid & 127, half = tid >> 7, quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float *pa = static_cast<const float*>(a.a) + head, *pb = static_cast<const float*>(a.b) + head,
                *pc = static_cast<const float*>(a.c) + head;
    const float* X = a.n_seg == 1 ? a.initial + ((int64_t)b * a.H + h) * D * D
                                  : a.states + (((int64_t)b * a.H + h) * a.n_seg + seg) * D * D;
    constexpr int CH = D / 8, UN = TK * CH / 256;   // 16-byte chunks of a row; (row, chunk) pairs of a tile per thread
    float4 fb[UN][2], fc[UN][2];
    auto fetch = [&](int u) {
      if (u >= n) return;
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int e = tid + 256 * i;
        const float4* src;
        if (u >= n_x) {
          const int tok = (u - n_x) * TK + e / CH;
          fb[i][0] = fb[i][1] = fc[i][0] = fc[i][1] = zero4();
          if (j_first + tok >= end) continue;   // behind the end: zeros, whatever stands there
          const int64_t at = (j_first + tok) * stride + (e % CH) * 8;
          const float4* q = reinterpret_cast<const float4*>(pb + at);
          fb[i][0] = q[0], fb[i][1] = q[1];
          src = reinterpret_cast<const float4*>(pc + at);
        } else if (!a.transposed) {   // rows 64 u .. of X
          src = reinterpret_cast<const float4*>(X + (u * TK + e / CH) * D + (e % CH) * 8);
        } else {                      // columns 64 u .. of X, rows of 8 chunks
          src = reinterpret_cast<const float4*>(X + (e / 8) * D + u * TK + (e % 8) * 8);
        }
        fc[i][0] = src[0], fc[i][1] = src[1];
      }
    };
    {   // a, zeros behind the end; all of a thread's loads before the first store
      float4 fa[2 * UN][2];
#pragma unroll
      for (int i = 0; i < 2 * UN; ++i) {
        const int e = tid + 256 * i, r = e / CH;
        fa[i][0] = fa[i][1] = zero4();
        if (i0 + r < end) {
          const float4* q = reinterpret_cast<const float4*>(pa + (i0 + r) * stride + (e % CH) * 8);
          fa[i][0] = q[0], fa[i][1] = q[1];
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * UN; ++i) {
        const int e = tid + 256 * i;
        store_terms(as + image_off(TM, e / CH, e % CH), L::a_term, fa[i][0], fa[i][1]);
      }
    }
    fetch(0);
    // a row's distance to the nearest column of an earlier (later) group is rowf's plus a multiple of 32
    const float rowf = decay_pow(ld, REV ? 32 - lane : lane + 1);
    const bool live = i0 + row < end;
    for (int u = 0; ok && u < n; ++u) {
      const bool kv = u >= n_x;
      if (kv) {   // the products that read b before are over: their scores have been taken
#pragma unroll
        for (int i = 0; i < UN; ++i) {
          const int e = tid + 256 * i;
          store_terms(bs + image_off(TK, e / CH, e % CH), L::t_term, fb[i][0], fb[i][1]);
        }
        fence_proxy_async();
        mbar_arrive(&bar_b);
      }
      if (u > 0) ok = warp_wait(&bar_o, (u - 1) & 1, abort_flag);   // c and P have been read
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int e = tid + 256 * i;
        const uint32_t at = !kv && a.transposed ? image_off(D, e / 8, e % 8) : image_off(TK, e / CH, e % CH);
        store_terms(cs + at, L::t_term, fc[i][0], fc[i][1]);
      }
      fetch(u + 1);
      float s[32];
      if (kv) {
        ok = warp_wait(&bar_s, (u - n_x) & 1, abort_flag);
        if (!ok) break;
        fence_after_sync();
        tmem_ld32(tm_s + lanes + 32 * half, s);
        tmem_wait_ld();
        const int off = (int)(i0 - j_first) - (u - n_x) * TK;   // from the tile's first column to the first row
        const int ahead = REV ? half - quarter - off / 32 : off / 32 + quarter - half;   // groups from column to row
        if (ahead > 0) {
          const float f = rowf * power32[ahead - 1];
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] *= f * diag[32 + (REV ? i : 31 - i)];
        } else if (ahead == 0) {
          const float* d = diag + 32 + (REV ? -lane : lane);
#pragma unroll
          for (int i = 0; i < 32; ++i) {   // zeros of the table for columns that the row does not see
            const float v = s[i] * d[REV ? i : -i];
            s[i] = (REV ? i >= lane : i <= lane) ? v : 0.f;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = 0.f;
        }
      } else {
        const int e = REV ? (int)(end - 1 - i0) - row : (int)(i0 - s0) + row + 1;
        const float w = decay_pow(ld, max(0, e));
        const float4* q = reinterpret_cast<const float4*>(pa + (i0 + row) * stride + u * TK + 32 * half);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 v = live ? scaled(q[i], w) : zero4();
          s[4 * i] = v.x, s[4 * i + 1] = v.y, s[4 * i + 2] = v.z, s[4 * i + 3] = v.w;
        }
      }
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        float p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint64_t f = pair2(s[2 * i], s[2 * i + 1]);
          p[i] = __uint_as_float(take2(f));
          asm("mov.b64 {%0, %1}, %2;" : "=f"(s[2 * i]), "=f"(s[2 * i + 1]) : "l"(f));
        }
        tmem_st16((term == 2 ? tm_p2 + 16 * half : tm_s + 32 * half + 16 * term) + lanes, p);
      }
      tmem_wait_st();
      fence_proxy_async();
      fence_before_sync();
      mbar_arrive(&bar_p);
    }
    // O, through a's images
    if (ok) ok = warp_wait(&bar_o, (n - 1) & 1, abort_flag);
    if (ok) {
      fence_after_sync();
#pragma unroll 1
      for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
        float v[32], w[32];
        tmem_ld32(tm_o + lanes + c, v);
        tmem_ld32(tm_r + lanes + c, w);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(as + image_off(TM, row, (c + i) / 4)) =
              live ? make_float4(v[i] + w[i], v[i + 1] + w[i + 1], v[i + 2] + w[i + 2], v[i + 3] + w[i + 3]) : zero4();
      }
      fence_proxy_async();
    }
    ok = named_sync_and(1, 256, ok);
    if (ok && tid == 0) {
#pragma unroll
      for (int p = 0; p < D / 32; ++p) tma_store_4d(&out_map, as + p * TM * 128, 32 * p, h, (int)i0, b);
      bulk_commit();
      bulk_wait_read();
    }
  }
  fence_before_sync();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(status, KDA_ERR_TIMEOUT);
  fence_after_sync();
  if (warp == 8) tmem_dealloc(tm_s, kMapTmem<D>);
}

struct OutMaps { CUtensorMap set[3]; };

// ONE: the forward pass's map alone; otherwise the backward pass's three.
template <int D, bool ONE>
__global__ void __launch_bounds__(kThreads, D == 128 ? 1 : 2) lin_tc32_map_kernel(const __grid_constant__ OutMaps outs,
                                                                                 const __grid_constant__ LinMapSets sets,
                                                                                 uint32_t* status) {
  if constexpr (ONE) {
    map_tile<D, false>(outs.set[0], sets.set[0], blockIdx.x, status);
  } else {
    const int per_set = gridDim.x / sets.n, which = blockIdx.x / per_set, tile = blockIdx.x % per_set;
    if (sets.set[which].reverse) map_tile<D, true>(outs.set[which], sets.set[which], tile, status);
    else map_tile<D, false>(outs.set[which], sets.set[which], tile, status);
  }
}

template <int D>
cudaError_t local(const Dims& d, const LinLocalSets& a, uint32_t* status, cudaStream_t s) {
  const auto kernel = a.n == 1 ? lin_tc32_local_kernel<D, true> : lin_tc32_local_kernel<D, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLocalSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.set[0].n_seg * a.n), (d.H * D + 127) / 128, d.B);
  kernel<<<grid, kThreads, kLocalSmem, s>>>(a, status);
  return cudaGetLastError();
}

template <int D>
cudaError_t map(const Dims& d, const LinMapSets& a, uint32_t* status, cudaStream_t s) {
  // out [B][N][H][D] seen as a 4D tensor; box: 32 channels x 1 head x 128 tokens x 1 item
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return cudaErrorInvalidValue;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)d.H, (cuuint64_t)d.N, (cuuint64_t)d.B};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 4, (cuuint64_t)d.H * D * 4, (cuuint64_t)d.N * d.H * D * 4};
  const cuuint32_t box[4] = {32u, 1u, (cuuint32_t)TM, 1u}, estr[4] = {1u, 1u, 1u, 1u};
  OutMaps m;
  for (int i = 0; i < a.n; ++i)
    if (enc(&m.set[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.set[i].out, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  const auto kernel = a.n == 1 ? lin_tc32_map_kernel<D, true> : lin_tc32_map_kernel<D, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MapSmem<D>::bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((d.N + TM - 1) / TM * a.n), d.H, d.B);
  kernel<<<grid, kThreads, MapSmem<D>::bytes, s>>>(m, a, status);
  return cudaGetLastError();
}

}  // namespace

int linear_tc32_segment() { return kSeg; }

cudaError_t launch_linear_tc32_local(const Dims& d, const LinLocalSets& a, uint32_t* status, cudaStream_t s) {
  return d.dk == 128 ? local<128>(d, a, status, s) : local<64>(d, a, status, s);
}
cudaError_t launch_linear_tc32_map(const Dims& d, const LinMapSets& a, uint32_t* status, cudaStream_t s) {
  return d.dk == 128 ? map<128>(d, a, status, s) : map<64>(d, a, status, s);
}

}  // namespace kda
