// Linear attention with a fixed decay per head on the tensor cores (tcgen05), bf16 problems.
//
// The three launches of linear.cu, for bf16 inputs:
//   local: each segment's own sum_t w_t x_t y_t^T, [D x tokens] x [tokens x D] products;
//   scan:  the recurrence over segments, element by element in fp32;
//   map:   out_i = lam^e(i) X^(T) a_i + sum_j lam^|i-j| (a_i . b_j) c_j, 128 rows per CTA.
// The decay is a constant of the head, so no tile needs a running maximum or an exponential of its own: with a
// column's place cc in its group of 32, lam^(i-j) = lam^(i - group's last) * lam^(31-cc), a factor per (row, group)
// times one of 32 registers, both at most 1.  Only the 32 x 32 blocks on the diagonal look lam^(i-j) up.
//
// What is rounded: an output, once, to bf16.  A decayed score and a state that enters a segment go into their products
// with c and a as two bf16 terms, which leaves 2^-16 of each (a state is an fp32 argument and the past of every later
// token, and the single-token call reads it in fp32).  The error against fp64 is that of rounding the exact outputs,
// 1.66e-3 of their norm at random.  One term each would give 2.35e-3; 33,272 x 16 x 128 forward took 292 us as it is,
// 270 with scores of one term, 278 with states of one, 258 with both (in segments of 512 tokens).  The states stay fp32
// from segment to segment, and the sums that become a state are taken of three bf16 terms (24 bits), because states are
// fp32 results.  All sums are fp32.
//
// State images.  Between scan and map a state is two bf16 matrices, its first and second terms, in the
// 128-byte-swizzled panels that the tensor core reads, so a CTA fetches each with one bulk copy.  Of a segment's fp32
// local state, four of eight columns lie where the first image's eight will be and four where the second's will be, so
// the scan works in place.
#include "linear_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kMaxSeg = 256;   // tokens per segment, at most; always a multiple of TM
constexpr int TM = 128;       // tokens per tile of the map
constexpr int TL = 64;        // tokens per tile of the local sums

// ---------------------------------------------------------------------------
// local
// ---------------------------------------------------------------------------
// One CTA per (segment, 128 channels, item): one head of 128, or two of 64 side by side (a 64-channel head is a
// panel of the operand, so the pair's products are the diagonal blocks of a 128 x 128 one).  Per 64-token tile eight
// warps turn y into the three bf16 terms of w y, hi over y itself; D[x][y] += x^T hi goes to one accumulator, the
// mid and lo terms to another, so the main one sees one addition per 16 tokens.  Two stages of x and y and the
// mid and lo images are 96 KB: two CTAs per SM, one's products under the other's roundings.
constexpr int kLocalThreads = 288;
constexpr int kLocalSmem = 1024 + 2 * 32768 + 32768;

struct LocalMaps { CUtensorMap x, y; };
struct LocalMapSets { LocalMaps set[2]; };

template <int D, bool ONE>
__global__ void __launch_bounds__(kLocalThreads, 2) lin_tc_local_kernel(const __grid_constant__ LocalMapSets map_sets,
                                                                       const __grid_constant__ LinLocalSets sets,
                                                                       uint32_t* status) {
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t full[2], ready, done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_slot;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* mid = sm + 65536;
  uint8_t* lo = mid + 16384;
  volatile int* abort_flag = &abort_slot;
  const int tid = threadIdx.x, warp = tid / 32;
  constexpr int HP = 128 / D;   // heads per CTA
  const int per_set = ONE ? gridDim.x : gridDim.x / sets.n, which = ONE ? 0 : blockIdx.x / per_set;
  const LocalMaps& maps = map_sets.set[which];
  const LinLocalArgs& a = sets.set[which];
  const int seg = blockIdx.x - which * per_set, h0 = blockIdx.y * HP, b = blockIdx.z;
  const int64_t s0 = (int64_t)seg * a.seg, len = item_tokens(a.lengths, b, a.N), end = min(len, s0 + a.seg);
  const int n_tok = (int)max((int64_t)0, end - s0), n_tiles = (n_tok + TL - 1) / TL;
  if (tid == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
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
      auto load = [&](int t) {
        uint8_t* x = sm + (t & 1) * 32768;
        mbar_arrive_expect_tx(&full[t & 1], 32768);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int c = D == 128 ? 64 * p : 0, h = D == 128 ? h0 : h0 + p, tok = (int)(s0 + t * TL);
          tma_load_4d(x + p * 8192, &maps.x, c, h, tok, b, &full[t & 1]);
          tma_load_4d(x + 16384 + p * 8192, &maps.y, c, h, tok, b, &full[t & 1]);
        }
      };
      constexpr uint32_t id = idesc_bf16(128, 128, true, true);
      int loaded = 0;
      while (loaded < min(2, n_tiles)) load(loaded++);
      for (int t = 0; ok && t < n_tiles; ++t) {
        ok = wait_or_abort(&ready, t & 1, abort_flag);
        if (!ok) break;
        fence_after_sync();
        const uint32_t xs = smem_u32(sm + (t & 1) * 32768);
        const uint64_t dx = mdesc0(xs, 8192), dh = mdesc0(xs + 16384, 8192), dm = mdesc0(smem_u32(mid), 8192),
                       dl = mdesc0(smem_u32(lo), 8192);
#pragma unroll
        for (int k = 0; k < TL / 16; ++k) {
          mma_ss(tm, dx + mstep(k), dh + mstep(k), id, t || k);
          mma_ss(tm + 128, dx + mstep(k), dl + mstep(k), id, t || k);
          mma_ss(tm + 128, dx + mstep(k), dm + mstep(k), id, 1u);
        }
        mma_commit(&done);
        if (loaded < n_tiles) {
          ok = wait_or_abort(&done, t & 1, abort_flag);
          if (ok) load(loaded++);
        }
      }
      if (!ok)   // copies in flight end before the CTA does
        for (int t = max(0, loaded - 2); t < loaded; ++t) mbar_wait(&full[t & 1], (t >> 1) & 1, 100000000ull);
    }
    __syncwarp();
  } else {
    const int c8 = tid % 16, r0 = tid / 16;   // this thread's 8 channels, its tokens r0 + 16 i
    const int h = D == 128 ? h0 : min(h0 + c8 / 8, a.H - 1);
    const float ld = a.log_decay[h];
    // the weight of a token of a whole tile: its row's power times the tile's, both at most 1
    float roww[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) roww[i] = decay_pow(ld, a.reverse ? r0 + 16 * i + 1 : TL - 1 - r0 - 16 * i);
    for (int t = 0; ok && t < n_tiles; ++t) {
      const int left = n_tok - t * TL;   // tokens from this tile on
      const float tilew = decay_pow(ld, a.reverse ? t * TL : max(0, left - TL));
      ok = warp_wait(&full[t & 1], (t >> 1) & 1, abort_flag);
      if (ok && t > 0) ok = warp_wait(&done, (t - 1) & 1, abort_flag);   // mid and lo free
      if (!ok) break;
      uint8_t* x = sm + (t & 1) * 32768;
      uint8_t* y = x + 16384;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 16 * i;
        const uint32_t off = image_off(TL, r, c8);
        uint4 hi, m, l;
        if (r < left) {
          const float w = !a.reverse && left < TL ? decay_pow(ld, left - 1 - r) : roww[i] * tilew;
          const uint64_t ww = pair2(w, w);
          const uint4 u = *reinterpret_cast<const uint4*>(y + off);
          const uint32_t e[4] = {u.x, u.y, u.z, u.w};
          uint32_t *ph = &hi.x, *pm = &m.x, *pl = &l.x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint64_t f = mul2(wide2(e[j]), ww);
            ph[j] = take2(f);
            pm[j] = take2(f);
            pl[j] = pack2(f);
          }
        } else {   // behind the end, whatever stands there
          hi = m = l = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(x + off) = hi;
        }
        *reinterpret_cast<uint4*>(y + off) = hi;
        *reinterpret_cast<uint4*>(mid + off) = m;
        *reinterpret_cast<uint4*>(lo + off) = l;
      }
      fence_proxy_async();
      mbar_arrive(&ready);
    }
    if (ok && n_tiles) ok = warp_wait(&done, (n_tiles - 1) & 1, abort_flag);
    if (ok) {
      fence_after_sync();
      // lane = row of the 128 x 128 block; head = row / D owns columns of the same block.  The heads' images are put
      // together over the x and y stages and leave as whole.
      const int row = (warp & 3) * 32 + (tid & 31), hp = row / D, r = row % D;
      constexpr int COLS = D / 2;   // columns of this warp: a half of its head's
      const int c0 = (warp >> 2) * COLS;
      const uint32_t at = tm + ((uint32_t)((warp & 3) * 32) << 16) + hp * (D % 128) + c0;
      uint8_t* img = sm + hp * D * D * 4;
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
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          const uint32_t off = image_off(D, r, (c0 + c + i) / 8);
          *reinterpret_cast<float4*>(img + off) = make_float4(v[i] + w[i], v[i + 1] + w[i + 1], v[i + 2] + w[i + 2], v[i + 3] + w[i + 3]);
          *reinterpret_cast<float4*>(img + D * D * 2 + off) =
              make_float4(v[i + 4] + w[i + 4], v[i + 5] + w[i + 5], v[i + 6] + w[i + 6], v[i + 7] + w[i + 7]);
        }
      }
      fence_proxy_async();
    }
    ok = named_sync_and(1, 256, ok);
    if (ok && tid == 0) {
#pragma unroll
      for (int p = 0; p < HP; ++p)
        if (h0 + p < a.H)
          bulk_s2g(a.local + (((int64_t)b * a.H + h0 + p) * a.n_seg + seg) * D * D, sm + p * D * D * 4, D * D * 4);
      bulk_commit();
      bulk_wait_read();
    }
  }
  fence_before_sync();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(status, KDA_ERR_TIMEOUT);
  fence_after_sync();
  if (warp == 8) tmem_dealloc(tm, 256);
}

// ---------------------------------------------------------------------------
// scan
// ---------------------------------------------------------------------------
// A thread takes 8 columns of one row: 32 bytes of the local state, 16 each of the two images over them.
// U local states are fetched at once: 8 where the CTAs do not fill the GPU twice over (33,272 tokens x 16 x 128 forward:
// 45 us, with 4 51; 4 x 8192 x 16 x 64: 11, with 4 12), else 4, whose fewer registers let more CTAs run at once
// (4 x 8192 x 16 x 128: 40 us, with 8 43; 8 prompts of up to 2000: 18.5, with 8 22; 33,272 tokens backward: 86, with 8 93).
template <int D, bool ONE, int U>
__global__ void __launch_bounds__(128) lin_tc_scan_kernel(const __grid_constant__ LinScanSets sets) {
  constexpr int kPerSet = D * D / 8 / 128;
  const LinScanArgs& a = sets.set[ONE ? 0 : blockIdx.x / kPerSet];
  const bool local = a.local;
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = (int64_t)b * a.H + h;
  const int e = blockIdx.x % kPerSet * 128 + threadIdx.x, r = e / (D / 8), c8 = e % (D / 8);
  const int64_t len = item_tokens(a.lengths, b, a.N), last = len / a.seg;
  const float ld = a.log_decay[h];
  const Factor whole = segment_factor(ld, a.seg), part = segment_factor(ld, len % a.seg);
  float S[8] = {};
  if (a.initial) {
    const float4* p = reinterpret_cast<const float4*>(a.initial + bh * D * D + r * D + c8 * 8);
    const float4 u = p[0], v = p[1];
    S[0] = u.x; S[1] = u.y; S[2] = u.z; S[3] = u.w; S[4] = v.x; S[5] = v.y; S[6] = v.z; S[7] = v.w;
  }
  uint8_t* p = reinterpret_cast<uint8_t*>(a.states + bh * a.n_seg * D * D) + image_off(D, r, c8);
  constexpr int LO = D * D * 2;
  for (int c0 = 0; c0 < a.n_seg; c0 += U) {
    float4 x[U], y[U];
    if (local) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u < a.n_seg) {
          const uint8_t* s = p + (int64_t)(a.reverse ? a.n_seg - 1 - c0 - u : c0 + u) * D * D * 4;
          x[u] = *reinterpret_cast<const float4*>(s);
          y[u] = *reinterpret_cast<const float4*>(s + LO);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u >= a.n_seg) break;
      const int c = a.reverse ? a.n_seg - 1 - c0 - u : c0 + u;
      uint8_t* s = p + (int64_t)c * D * D * 4;
      uint4 hi, lo;
      uint32_t *ph = &hi.x, *pl = &lo.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint64_t f = pair2(S[2 * i], S[2 * i + 1]);
        ph[i] = take2(f);
        pl[i] = pack2(f);
      }
      *reinterpret_cast<uint4*>(s) = hi;
      *reinterpret_cast<uint4*>(s + LO) = lo;
      if (c > last || !local) continue;   // behind the end: no tokens
      const Factor f = c == last ? part : whole;
      const float l[8] = {x[u].x, x[u].y, x[u].z, x[u].w, y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) S[i] = fmaf(f.hi, S[i], fmaf(f.lo, S[i], l[i]));
    }
  }
  if (a.final) {
    float4* q = reinterpret_cast<float4*>(a.final + bh * D * D + r * D + c8 * 8);
    q[0] = make_float4(S[0], S[1], S[2], S[3]);
    q[1] = make_float4(S[4], S[5], S[6], S[7]);
  }
}

// ---------------------------------------------------------------------------
// map
// ---------------------------------------------------------------------------
// One CTA per 128 output rows: warps 0-3 hold a row per thread, one thread of warp 4 issues copies and products.
//   O = a X, scaled row by row by lam^e(i); then per tile of 128 tokens S = a b^T, P = S * decay as two bf16 terms
//   written over S in tensor memory, O += P c.
// S and O take 256 columns of tensor memory and a, b, c 96 KB of shared memory, so two CTAs share an SM and one's
// products run under the other's decays; before their own tiles, X's first term passes through c's buffer and, once the
// first scores have read b, its second through b's.  What was tried against it: one persistent CTA with two lanes of 128
// rows, copies fetched ahead and separate warps for the outputs, whose larger code ran at the same speed (a fifth of the
// cycles waiting for instructions).
constexpr int kMapThreads = 160;
template <int D> struct MapSmem {
  static constexpr int tile = TM * D * 2, panel = TM * 128;
  // below 77 KB a third CTA would fit the shared memory but not the tensor memory
  static constexpr int bytes = 1024 + (3 * tile < 78 * 1024 ? 78 * 1024 : 3 * tile);
};

struct MapMaps { CUtensorMap a, b, c, out; };
struct MapMapSets { MapMaps set[3]; };

// The map's 128 rows of tile `tile`; REV: columns behind the rows instead of before them.
template <int D, bool REV>
__device__ __forceinline__ void map_tile(const MapMaps& maps, const LinMapArgs& a, int tile, uint32_t* status) {
  using L = MapSmem<D>;
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t bar_a, full_b, full_c, bar_s, bar_x, bar_o, bar_p;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_slot;
  __shared__ float diag[64];                // lam^n at 32 + n, zeros below
  __shared__ float power32[4 * kMaxSeg / TM];   // lam^(32 n)
  uint8_t* as = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* bs = as + L::tile;
  uint8_t* cs = bs + L::tile;
  volatile int* abort_flag = &abort_slot;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t i0 = (int64_t)tile * TM, len = item_tokens(a.lengths, b, a.N);
  const int seg = (int)(i0 / a.seg);
  const int64_t s0 = (int64_t)seg * a.seg, end = min(len, s0 + a.seg);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)b * a.N * a.H + h) * D;
  if (i0 >= len) {   // behind the item's end: zeros
    const int n = (int)min((int64_t)TM, a.N - i0) * (D / 8);
    for (int i = tid; i < n; i += kMapThreads)
      *reinterpret_cast<uint4*>(out + (i0 + i / (D / 8)) * a.H * D + (i % (D / 8)) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const bool has_state = a.initial || (REV ? seg != a.n_seg - 1 : seg != 0);
  const int64_t j_first = REV ? i0 : s0;
  const int n_tiles = (int)((REV ? end - i0 + TM - 1 : i0 - s0 + TM) / TM);
  const float ld = a.log_decay[h];
  if (tid == 0) {
    mbar_init(&bar_a, 1);
    mbar_init(&full_b, 1);
    mbar_init(&full_c, 1);
    mbar_init(&bar_s, 1);
    mbar_init(&bar_x, 1);
    mbar_init(&bar_o, 1);
    mbar_init(&bar_p, 128);
    abort_slot = 0;
    fence_mbar_init();
  }
  if (tid < 64) diag[tid] = tid < 32 ? 0.f : decay_pow(ld, tid - 32);
  else if (tid < 64 + 4 * kMaxSeg / TM) power32[tid - 64] = decay_pow(ld, 32 * (tid - 64));
  if (warp == 4) { tmem_alloc(&tmem_slot, 256); tmem_relinquish(); }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm_s = tmem_slot, tm_o = tm_s + 128;
  bool ok = true;

  if (warp == 4) {
    if (lane == 0) {
      auto load = [&](uint8_t* dst, const CUtensorMap* m, int64_t tok, uint64_t* bar) {
        mbar_arrive_expect_tx(bar, L::tile);
#pragma unroll
        for (int p = 0; p < D / 64; ++p) tma_load_4d(dst + p * L::panel, m, 64 * p, h, (int)tok, b, bar);
      };
      int nb = 0, nc = 0;   // loads issued into b's and c's buffers
      load(as, &maps.a, i0, &bar_a);
      load(bs, &maps.b, j_first, &full_b);
      const uint8_t* X = reinterpret_cast<const uint8_t*>(a.states + (((int64_t)b * a.H + h) * a.n_seg + seg) * D * D);
      if (has_state) {
        mbar_arrive_expect_tx(&full_c, D * D * 2);
        bulk_g2s(cs, X, D * D * 2, &full_c);
      } else {
        load(cs, &maps.c, j_first, &full_c);
      }
      ++nb, ++nc;
      const uint32_t sa = smem_u32(as), sb = smem_u32(bs), sc = smem_u32(cs);
      const uint64_t da = kdesc0(sa), db = kdesc0(sb), dc = mdesc0(sc, L::panel);
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false), id_o = idesc_bf16(128, D, false, true);
      int no = 0;   // phases of bar_o that have been waited for
      ok = wait_or_abort(&bar_a, 0, abort_flag);
      for (int t = 0; ok && t < n_tiles; ++t) {
        if (t > 0) {   // P and c of the tile before have been read
          ok = wait_or_abort(&bar_o, no++ & 1, abort_flag);
          if (!ok) break;
          load(cs, &maps.c, j_first + t * TM, &full_c);
          ++nc;
        }
        ok = wait_or_abort(&full_b, (nb - 1) & 1, abort_flag);
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) mma_ss(tm_s, da + kstep(k, L::panel), db + kstep(k, L::panel), id_s, k > 0);
        mma_commit(&bar_s);
        // X as stored has a's channel along rows; transposed, along columns
        auto state_product = [&](uint32_t x, bool first) {
          const uint32_t id = idesc_bf16(128, D, false, !a.transposed);
          const uint64_t dx = a.transposed ? kdesc0(x) : mdesc0(x, D * 128);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tm_o, da + kstep(k, L::panel), dx + (a.transposed ? kstep(k, D * 128) : mstep(k)), id, !first || k > 0);
        };
        const bool state = t == 0 && has_state;
        if (state) {   // X's first term, in c's buffer
          ok = wait_or_abort(&full_c, 0, abort_flag);
          if (!ok) break;
          state_product(sc, true);
          mma_commit(&bar_x);
        }
        ok = wait_or_abort(&bar_s, t & 1, abort_flag);
        if (!ok) break;
        if (state) {   // its second, through b's
          mbar_arrive_expect_tx(&full_b, D * D * 2);
          bulk_g2s(bs, X + D * D * 2, D * D * 2, &full_b);
          ++nb;
          ok = wait_or_abort(&bar_x, 0, abort_flag);
          if (!ok) break;
          load(cs, &maps.c, j_first, &full_c);
          ++nc;
          ok = wait_or_abort(&full_b, (nb - 1) & 1, abort_flag);
          if (!ok) break;
          state_product(sb, false);
          mma_commit(&bar_o);
          ok = wait_or_abort(&bar_o, no++ & 1, abort_flag);
          if (!ok) break;
        }
        if (t + 1 < n_tiles) {
          load(bs, &maps.b, j_first + (t + 1) * TM, &full_b);
          ++nb;
        }
        ok = wait_or_abort(&bar_p, t & 1, abort_flag) && wait_or_abort(&full_c, (nc - 1) & 1, abort_flag);
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int k = 0; k < TM / 16; ++k) {   // P's terms: 16 columns each of a group of 32 tokens
          const uint32_t p = tm_s + 32 * (k >> 1) + 8 * (k & 1);
          mma_ts(tm_o, p + 16, dc + mstep(k), id_o, has_state || t || k);
          mma_ts(tm_o, p, dc + mstep(k), id_o, 1u);
        }
        mma_commit(&bar_o);
      }
      if (!ok) {   // copies in flight end before the CTA does
        mbar_wait(&bar_a, 0, 100000000ull);
        mbar_wait(&full_b, (nb - 1) & 1, 100000000ull);
        mbar_wait(&full_c, (nc - 1) & 1, 100000000ull);
      }
    }
    __syncwarp();
  } else {
    const int row = tid;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    uint64_t col[16];   // lam^(31-cc), or lam^cc in the reverse direction, in pairs
#pragma unroll
    for (int i = 0; i < 16; ++i)
      col[i] = REV ? pair2(diag[32 + 2 * i], diag[33 + 2 * i]) : pair2(diag[63 - 2 * i], diag[62 - 2 * i]);
    // a row's distance to the nearest column of an earlier (later) group is rowf's plus a multiple of 32
    const float rowf = decay_pow(ld, REV ? 32 - lane : lane + 1);
    const int to_end = (int)min((int64_t)a.seg, len - j_first);   // tokens of the sequence from j_first on
    for (int t = 0; ok && t < n_tiles; ++t) {
      ok = warp_wait(&bar_s, t & 1, abort_flag);
      if (!ok) break;
      fence_after_sync();
      const int m = REV ? t : n_tiles - 1 - t;   // tiles between the rows and the columns
      const int n_valid = to_end - t * TM;       // columns within the sequence (below TM at its end only)
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {   // P of 32 columns: s * factor(row, group) * col[cc]; on the diagonal block s * lam^|i-j|
        const int ahead = 4 * m + (REV ? g - warp : warp - g);   // groups from column to row
        float s[32];
        uint32_t p[32];   // the first terms of 32 columns, the second terms
        tmem_ld32(tm_s + lanes + 32 * g, s);
        tmem_wait_ld();
        auto put = [&](int i, uint64_t f) {
          p[i] = take2(f);
          p[16 + i] = pack2(f);
        };
        if (ahead > 0) {
          const float f = rowf * power32[ahead - 1];
          const uint64_t ff = pair2(f, f);
#pragma unroll
          for (int i = 0; i < 16; ++i) put(i, mul2(pair2(s[2 * i], s[2 * i + 1]), mul2(ff, col[i])));
        } else if (ahead == 0) {
          const float* d = diag + 32 + (REV ? -lane : lane);
#pragma unroll
          for (int i = 0; i < 16; ++i) {   // zeros of the table for columns that the row does not see
            const float u = s[2 * i] * d[REV ? 2 * i : -2 * i], v = s[2 * i + 1] * d[REV ? 2 * i + 1 : -2 * i - 1];
            put(i, pair2((REV ? 2 * i >= lane : 2 * i <= lane) ? u : 0.f, (REV ? 2 * i + 1 >= lane : 2 * i + 1 <= lane) ? v : 0.f));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) p[i] = 0;
        }
        if (n_valid < TM) {   // columns behind the end, whatever their scores
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = 32 * g + 2 * i;
            const uint32_t keep = (c < n_valid ? 0xffffu : 0u) | (c + 1 < n_valid ? 0xffff0000u : 0u);
            p[i] &= keep;
            p[16 + i] &= keep;
          }
        }
        tmem_st32(tm_s + lanes + 32 * g, p);
      }
      if (t == 0 && has_state) {   // O = a X, row by row lam^e(i) of it, before the tiles are added
        const float w = decay_pow(ld, REV ? max((int64_t)0, end - 1 - (i0 + row)) : i0 + row - s0 + 1);
        ok = warp_wait(&bar_o, 0, abort_flag);
        if (!ok) { tmem_wait_st(); break; }
        fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          uint32_t u[32];
          tmem_ld32(tm_o + lanes + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i] * w);
          tmem_st32(tm_o + lanes + c, u);
        }
      }
      // A wait for a phase holds only once the phase before is over.  Of full_c, load 0 is X where there is a state and
      // c of tile t is load has_state + t.  Load has_state + t - 1 is over here: at t = 0 it is X, which the product
      // behind bar_o has read (waited for above); at t > 0 the scores of this tile, whose bar_s every row has waited
      // for, were issued after O += P c of the tile before.
      if (n_valid < TM) {   // c behind the end may hold anything, and 0 x NaN is NaN
        ok = warp_wait(&full_c, (has_state + t) & 1, abort_flag);
        if (!ok) { tmem_wait_st(); break; }
        for (int i = tid + n_valid * (D / 8); i < TM * (D / 8); i += 128)
          *reinterpret_cast<uint4*>(cs + image_off(TM, i / (D / 8), i % (D / 8))) = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
      }
      tmem_wait_st();
      fence_before_sync();
      mbar_arrive(&bar_p);
    }
    // O of the last tile: to bf16 in a's buffer, then out
    if (ok) ok = warp_wait(&bar_o, (has_state + n_tiles - 1) & 1, abort_flag);
    if (ok) {
      fence_after_sync();
      const bool live = i0 + row < len;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float v[32];
        tmem_ld32(tm_o + lanes + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint4 u;
          u.x = pack2(v[i], v[i + 1]);
          u.y = pack2(v[i + 2], v[i + 3]);
          u.z = pack2(v[i + 4], v[i + 5]);
          u.w = pack2(v[i + 6], v[i + 7]);
          if (!live) u = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(as + image_off(TM, row, (c + i) / 8)) = u;
        }
      }
      fence_proxy_async();
    }
    ok = named_sync_and(1, 128, ok);
    if (ok && tid == 0) {
#pragma unroll
      for (int p = 0; p < D / 64; ++p) tma_store_4d(&maps.out, as + p * L::panel, 64 * p, h, (int)i0, b);
      bulk_commit();
      bulk_wait_read();
    }
  }
  fence_before_sync();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(status, KDA_ERR_TIMEOUT);
  fence_after_sync();
  if (warp == 4) tmem_dealloc(tm_s, 256);
}

// ONE: the forward pass's map alone; otherwise the backward pass's three.
template <int D, bool ONE>
__global__ void __launch_bounds__(kMapThreads, 2) lin_tc_map_kernel(const __grid_constant__ MapMapSets map_sets,
                                                                   const __grid_constant__ LinMapSets sets, uint32_t* status) {
  if constexpr (ONE) {
    map_tile<D, false>(map_sets.set[0], sets.set[0], blockIdx.x, status);
  } else {
    const int per_set = gridDim.x / sets.n, which = blockIdx.x / per_set, tile = blockIdx.x % per_set;
    if (sets.set[which].reverse) map_tile<D, true>(map_sets.set[which], sets.set[which], tile, status);
    else map_tile<D, false>(map_sets.set[which], sets.set[which], tile, status);
  }
}

// [B][N][H][D] bf16 seen as a 4D tensor (channel, head, token, item); box: 64 channels x 1 head x `tokens` x 1 item.
// Tokens past N and heads past H read as zero.
bool encode(CUtensorMap* m, const void* base, const Dims& d, int tokens) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d.dk, (cuuint64_t)d.H, (cuuint64_t)d.N, (cuuint64_t)d.B};
  const cuuint64_t strides[3] = {(cuuint64_t)d.dk * 2, (cuuint64_t)d.H * d.dk * 2, (cuuint64_t)d.N * d.H * d.dk * 2};
  const cuuint32_t box[4] = {64u, 1u, (cuuint32_t)tokens, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t local(const Dims& d, const LinLocalSets& a, uint32_t* status, cudaStream_t s) {
  LocalMapSets m;
  for (int i = 0; i < a.n; ++i)
    if (!encode(&m.set[i].x, a.set[i].x, d, TL) || !encode(&m.set[i].y, a.set[i].y, d, TL)) return cudaErrorInvalidValue;
  const auto kernel = a.n == 1 ? lin_tc_local_kernel<D, true> : lin_tc_local_kernel<D, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLocalSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.set[0].n_seg * a.n), (d.H * D + 127) / 128, d.B);
  kernel<<<grid, kLocalThreads, kLocalSmem, s>>>(m, a, status);
  return cudaGetLastError();
}

template <int D>
cudaError_t map(const Dims& d, const LinMapSets& a, uint32_t* status, cudaStream_t s) {
  MapMapSets m;
  for (int i = 0; i < a.n; ++i)
    if (!encode(&m.set[i].a, a.set[i].a, d, TM) || !encode(&m.set[i].b, a.set[i].b, d, TM) ||
        !encode(&m.set[i].c, a.set[i].c, d, TM) || !encode(&m.set[i].out, a.set[i].out, d, TM))
      return cudaErrorInvalidValue;
  const auto kernel = a.n == 1 ? lin_tc_map_kernel<D, true> : lin_tc_map_kernel<D, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MapSmem<D>::bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((d.N + TM - 1) / TM * a.n), d.H, d.B);
  kernel<<<grid, kMapThreads, MapSmem<D>::bytes, s>>>(m, a, status);
  return cudaGetLastError();
}

}  // namespace

// Tokens per segment.  A longer one costs the map more tiles of scores per row, a shorter one costs states.  33,272
// tokens x 16 x 128: forward 296 us with 256, 292 with 512, 353 with 1024; backward 684, 714 and 930.  8 ragged prompts
// of up to 2000: 128 us with 256 and 123 with 512, their backward pass 281 and 284; 4 x 8192 x 16 x 64: 169 us with 256
// and 188 with 512, backward 467 and 540.  Where the segments would not give every SM its two CTAs of the local sums,
// shorter ones take less time in a row.
int linear_tc_segment(const Dims& d) {
  int seg = kMaxSeg;
  while (seg > TM && (int64_t)d.B * d.H * ((d.N + seg - 1) / seg) < 2 * 148) seg /= 2;
  return seg;
}
// States that a workspace holds: what no problem with fewer items, heads or tokens exceeds.  A halved segment means
// fewer than 2 x 148 of the longer ones, so at most twice as many less two.
int64_t linear_tc_most_states(const Dims& d) {
  static_assert(kMaxSeg == 2 * TM, "one halving");
  const int64_t pairs = (int64_t)d.B * d.H, whole = pairs * ((d.N + kMaxSeg - 1) / kMaxSeg), halves = pairs * ((d.N + TM - 1) / TM);
  return std::max(whole, std::min<int64_t>(halves, 2 * (2 * 148 - 1)));
}

cudaError_t launch_linear_tc_local(const Dims& d, const LinLocalSets& a, uint32_t* status, cudaStream_t s) {
  return d.dk == 128 ? local<128>(d, a, status, s) : local<64>(d, a, status, s);
}
template <int D>
static cudaError_t scan(const Dims& d, const LinScanSets& a, cudaStream_t s) {
  const dim3 grid(D * D / 8 / 128 * a.n, d.H, d.B);
  const bool four = a.set[0].n_seg <= 4 || (int64_t)grid.x * d.H * d.B >= 2 * 148;
  const auto kernel = a.n == 1 ? (four ? lin_tc_scan_kernel<D, true, 4> : lin_tc_scan_kernel<D, true, 8>)
                               : (four ? lin_tc_scan_kernel<D, false, 4> : lin_tc_scan_kernel<D, false, 8>);
  kernel<<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_linear_tc_scan(const Dims& d, const LinScanSets& a, cudaStream_t s) {
  return d.dk == 128 ? scan<128>(d, a, s) : scan<64>(d, a, s);
}
cudaError_t launch_linear_tc_map(const Dims& d, const LinMapSets& a, uint32_t* status, cudaStream_t s) {
  return d.dk == 128 ? map<128>(d, a, status, s) : map<64>(d, a, status, s);
}

}  // namespace kda
