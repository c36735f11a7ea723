// C-ABI layer of the operators beside the KDA scan: rotary positions, layer norm, linear attention with a decay
// per head.  Argument validation, workspace layout and dispatch; the operations are documented in include/kda.h.
#include <limits.h>

#include <initializer_list>

#include "common.cuh"

namespace {

constexpr size_t kStatusBytes = 256;

struct Span {   // an argument's address range
  const void* p;
  size_t bytes;
};

// A required argument has an address, unless the problem has none of its elements (an empty tensor has no address).
int check_aligned(std::initializer_list<Span> required, std::initializer_list<Span> optional) {
  for (const Span& s : required)
    if (!s.p && s.bytes) return KDA_ERR_INVALID_ARG;
  for (const auto* list : {&required, &optional})
    for (const Span& s : *list)
      if (reinterpret_cast<uintptr_t>(s.p) & 15u) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// Outputs share no byte with an input or with one another.  Output i may be the same range as the input whose place in
// `ins` in_place[i] gives (-1: none), and as that one alone: another argument at the same address is still read.
int check_alias(std::initializer_list<Span> outs, std::initializer_list<Span> ins, std::initializer_list<int> in_place = {}) {
  int i = 0;
  for (const Span& o : outs) {
    int j = 0;
    for (const Span& in : ins) {
      const bool own = i < (int)in_place.size() && in_place.begin()[i] == j;
      if (!(own && o.p == in.p && o.bytes == in.bytes) && overlap(o, in)) return KDA_ERR_INVALID_ARG;
      ++j;
    }
    for (const Span* p = outs.begin(); p != &o; ++p)
      if (overlap(*p, o)) return KDA_ERR_INVALID_ARG;
    ++i;
  }
  return KDA_OK;
}

int check_workspace(void* ws, size_t have, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || have < need) return KDA_ERR_WORKSPACE;
  return KDA_OK;
}

size_t elem_size(kda_dtype dt) { return dt == KDA_DT_BF16 ? 2 : 4; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

int finish(cudaError_t e, int launches) {
  const int st = cuda_status(e);
  if (!st) kda::set_last_launch_count(launches);
  return st;
}

// The problem's shape alone: its conv and scan options do not concern these operators.
int make_shape(const kda_problem* p, kda_dtype dt, kda::Dims* d) {
  const int st = kda::validate_problem(p, dt, d);
  if (st) return st;
  if (d->reuse_records || d->qkv_f16) return KDA_ERR_INVALID_ARG;
  if (d->B > 65535 || d->H > 65535) return KDA_ERR_UNSUPPORTED;   // grid axes
  return KDA_OK;
}

size_t act_bytes(const kda::Dims& d, kda_dtype dt) { return (size_t)d.B * d.N * d.H * d.dk * elem_size(dt); }
size_t one_state(const kda::Dims& d) { return (size_t)d.B * d.H * d.dk * d.dv * sizeof(float); }

int run_rope(const kda_problem* p, const kda_rope* r, kda_dtype dt, const void* q, const void* k,
             const float* inv_freq, const int32_t* positions, void* qo, void* ko, void* stream, bool inverse) {
  kda::set_last_launch_count(0);
  kda::Dims d;
  int st = make_shape(p, dt, &d);
  if (st) return st;
  if (!r || r->pairs_t < 0 || r->pairs_h < 0 || r->pairs_w < 0 || (r->flags & ~KDA_ROPE_INTERLEAVED))
    return KDA_ERR_INVALID_ARG;
  if ((int64_t)r->pairs_t + r->pairs_h + r->pairs_w != d.dk / 2) return KDA_ERR_INVALID_ARG;
  if (!k != !ko) return KDA_ERR_INVALID_ARG;
  const int64_t tokens = (int64_t)d.B * d.N;
  if (tokens > (int64_t)INT_MAX) return KDA_ERR_UNSUPPORTED;
  const size_t n = act_bytes(d, dt);
  const Span sq{q, n}, sk{k, n}, oq{qo, n}, ok{ko, n}, fr{inv_freq, (size_t)d.dk / 2 * 4}, ps{positions, (size_t)tokens * 12};
  if ((st = check_aligned({sq, oq, fr}, {sk, ok, ps}))) return st;
  if ((st = check_alias({oq, ok}, {sq, sk, fr, ps}, {0, 1}))) return st;
  const kda::RopeArgs a{{q, k}, {qo, ko}, inv_freq, positions, tokens, d.N, d.L, d.H, d.Hg, d.Wg,
                        k ? 2 : 1, r->pairs_t, r->pairs_h, inverse};
  int launches = 0;
  return finish(kda::launch_rope(a, dt, d.dk, (r->flags & KDA_ROPE_INTERLEAVED) != 0,
                                 static_cast<cudaStream_t>(stream), &launches), launches);
}

int check_norm(int64_t rows, int32_t cols, kda_dtype dt) {
  if (dt != KDA_DT_BF16 && dt != KDA_DT_F32) return KDA_ERR_INVALID_ARG;
  if (rows < 0 || cols < 1) return KDA_ERR_INVALID_ARG;
  if (cols > kda::kNormMaxCols || rows > (int64_t)INT_MAX) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace

extern "C" {

int kda_rope_fwd(const kda_problem* p, const kda_rope* rope, kda_dtype dtype, const void* q, const void* k,
                 const float* inv_freq, const int32_t* positions, void* q_out, void* k_out, void* stream) {
  return run_rope(p, rope, dtype, q, k, inv_freq, positions, q_out, k_out, stream, false);
}

int kda_rope_bwd(const kda_problem* p, const kda_rope* rope, kda_dtype dtype, const void* d_q_out,
                 const void* d_k_out, const float* inv_freq, const int32_t* positions, void* dq, void* dk,
                 void* stream) {
  return run_rope(p, rope, dtype, d_q_out, d_k_out, inv_freq, positions, dq, dk, stream, true);
}

int kda_layernorm_fwd(int64_t rows, int32_t cols, kda_dtype dtype, const void* x, const float* weight,
                      const float* bias, float eps, void* y, float* mean, float* rstd, void* stream) {
  kda::set_last_launch_count(0);
  int st = check_norm(rows, cols, dtype);
  if (st) return st;
  if (!(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
  const size_t n = (size_t)rows * cols * elem_size(dtype), c = (size_t)cols * 4, r = (size_t)rows * 4;
  const Span sx{x, n}, sw{weight, c}, sb{bias, c}, oy{y, n}, om{mean, r}, orr{rstd, r};
  if ((st = check_aligned({sx, oy}, {sw, sb, om, orr}))) return st;
  if ((st = check_alias({oy, om, orr}, {sx, sw, sb}))) return st;
  int launches = 0;
  return finish(kda::launch_norm_fwd({x, weight, bias, y, mean, rstd, rows, cols, eps}, dtype,
                                     static_cast<cudaStream_t>(stream), &launches), launches);
}

size_t kda_layernorm_bwd_workspace_bytes(int64_t rows, int32_t cols) {
  if (check_norm(rows, cols, KDA_DT_F32)) return 0;
  return kStatusBytes + kda::norm_bwd_parts(rows, cols);
}

int kda_layernorm_bwd(int64_t rows, int32_t cols, kda_dtype dtype, const void* dy, const void* x,
                      const float* weight, const float* mean, const float* rstd, void* dx, float* d_weight,
                      float* d_bias, void* workspace, size_t workspace_bytes, void* stream) {
  kda::set_last_launch_count(0);
  int st = check_norm(rows, cols, dtype);
  if (st) return st;
  const size_t n = (size_t)rows * cols * elem_size(dtype), c = (size_t)cols * 4, r = (size_t)rows * 4;
  const Span sdy{dy, n}, sx{x, n}, sw{weight, c}, sm{mean, r}, sr{rstd, r}, odx{dx, n}, odw{d_weight, c}, odb{d_bias, c};
  if ((st = check_aligned({sdy, sx, sm, sr, odx}, {sw, odw, odb}))) return st;
  const size_t need = kda_layernorm_bwd_workspace_bytes(rows, cols);
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  if ((st = check_alias({odx, odw, odb, {workspace, need}}, {sdy, sx, sw, sm, sr}))) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* parts = d_weight || d_bias ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kStatusBytes) : nullptr;
  int launches = 0;
  return finish(kda::launch_norm_bwd({dy, x, weight, mean, rstd, dx, parts, rows, cols}, dtype, d_weight, d_bias,
                                     static_cast<uint32_t*>(workspace), s, &launches), launches);
}

size_t kda_linear_workspace_bytes(const kda_problem* p, kda_dtype dtype) {
  kda::Dims d;
  if (make_shape(p, dtype, &d)) return 0;
  return kStatusBytes + kda::linear_fwd_scratch(d, dtype);
}

int kda_linear_fwd(const kda_problem* p, kda_dtype dtype, const void* q, const void* k, const void* v,
                   const float* log_decay, const int32_t* lengths, const float* initial_state, void* o,
                   float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  kda::set_last_launch_count(0);
  kda::Dims d;
  int st = make_shape(p, dtype, &d);
  if (st) return st;
  const size_t n = act_bytes(d, dtype), m = one_state(d);
  const Span sq{q, n}, sk{k, n}, sv{v, n}, sl{log_decay, (size_t)d.H * 4}, sn{lengths, (size_t)d.B * 4},
      s0{initial_state, m}, so{o, n}, sf{final_state, m};
  if ((st = check_aligned({sq, sk, sv, sl, so}, {sn, s0, sf}))) return st;
  const size_t need = kStatusBytes + kda::linear_fwd_scratch(d, dtype);
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  if ((st = check_alias({so, sf, {workspace, need}}, {sq, sk, sv, sl, sn, s0}))) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = cuda_status(cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s)))) return st;
  int launches = 0;
  return finish(kda::launch_linear_fwd(d, dtype, q, k, v, log_decay, lengths, initial_state, o, final_state,
                                       static_cast<char*>(workspace) + kStatusBytes, static_cast<uint32_t*>(workspace), s,
                                       &launches), launches);
}

size_t kda_linear_bwd_workspace_bytes(const kda_problem* p, kda_dtype dtype) {
  kda::Dims d;
  if (make_shape(p, dtype, &d)) return 0;
  return kStatusBytes + kda::linear_bwd_scratch(d, dtype);
}

int kda_linear_bwd(const kda_problem* p, kda_dtype dtype, const void* q, const void* k, const void* v,
                   const float* log_decay, const int32_t* lengths, const float* initial_state, const void* d_o,
                   const float* d_final_state, void* dq, void* dk, void* dv, float* d_initial_state,
                   void* workspace, size_t workspace_bytes, void* stream) {
  kda::set_last_launch_count(0);
  kda::Dims d;
  int st = make_shape(p, dtype, &d);
  if (st) return st;
  const size_t n = act_bytes(d, dtype), m = one_state(d);
  const Span sq{q, n}, sk{k, n}, sv{v, n}, sl{log_decay, (size_t)d.H * 4}, sn{lengths, (size_t)d.B * 4},
      s0{initial_state, m}, sdo{d_o, n}, sdf{d_final_state, m}, odq{dq, n}, odk{dk, n}, odv{dv, n}, od0{d_initial_state, m};
  if ((st = check_aligned({sq, sk, sv, sl, sdo, odq, odk, odv}, {sn, s0, sdf, od0}))) return st;
  const size_t need = kStatusBytes + kda::linear_bwd_scratch(d, dtype);
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  if ((st = check_alias({odq, odk, odv, od0, {workspace, need}}, {sq, sk, sv, sl, sn, s0, sdo, sdf}))) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = cuda_status(cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s)))) return st;
  int launches = 0;
  return finish(kda::launch_linear_bwd(d, dtype, q, k, v, log_decay, lengths, initial_state, d_o, d_final_state, dq,
                                       dk, dv, d_initial_state, static_cast<char*>(workspace) + kStatusBytes,
                                       static_cast<uint32_t*>(workspace), s, &launches), launches);
}

int kda_linear_step(const kda_problem* p, kda_dtype dtype, const void* q, const void* k, const void* v,
                    const float* log_decay, const float* state_in, void* o, float* state_out, void* stream) {
  kda::set_last_launch_count(0);
  kda::Dims d;
  int st = make_shape(p, dtype, &d);
  if (st) return st;
  if (d.N != 1) return KDA_ERR_INVALID_ARG;
  const size_t n = act_bytes(d, dtype), m = one_state(d);
  const Span sq{q, n}, sk{k, n}, sv{v, n}, sl{log_decay, (size_t)d.H * 4}, si{state_in, m}, so{o, n}, su{state_out, m};
  if ((st = check_aligned({sq, sk, sv, sl, si, so, su}, {}))) return st;
  if ((st = check_alias({so, su}, {sq, sk, sv, sl, si}, {-1, 4}))) return st;
  int launches = 0;
  return finish(kda::launch_linear_step(d, dtype, {q, k, v, log_decay, state_in, o, state_out, d.H},
                                        static_cast<cudaStream_t>(stream), &launches), launches);
}

}  // extern "C"
