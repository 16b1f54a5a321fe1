// gdn2_linattn_api.hip -- C entry points of the linear attention with a decay for each head and of the q/k head norms
// with rotation: argument checks, workspace sizing, dispatch. No allocation, no host synchronisation, no state.

#include <stdint.h>

#include <initializer_list>
#include <utility>

#include "gdn2.h"
#include "gdn2_linattn.h"
#include "gdn2_qk_norm.h"

namespace {

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
int hip_status(hipError_t e) { return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP; }

int check_ptrs(std::initializer_list<const void*> required, std::initializer_list<const void*> optional) {
  for (const void* p : required)
    if (p == nullptr) return GDN2_ERR_NULL;
  for (const void* p : required)
    if (!aligned(p, 16)) return GDN2_ERR_ALIGN;
  for (const void* p : optional)
    if (!aligned(p, 16)) return GDN2_ERR_ALIGN;
  return GDN2_OK;
}

int check_sizes(int N, int T, int Hk, int H, int Dk, int Dv, int dt) {
  if (dt != GDN2_F32 && dt != GDN2_BF16) return GDN2_ERR_DTYPE;
  if (N < 0 || T < 0 || Hk < 0 || H < 0 || Dk < 0 || Dv < 0) return GDN2_ERR_SHAPE;
  if (T > (1 << 30)) return GDN2_ERR_SHAPE;  // token indices are int32 inside the kernels
  if (!dim_ok(Dk) || !dim_ok(Dv)) return GDN2_ERR_UNSUPPORTED;
  if (H > 0 && (Hk == 0 || H % Hk != 0)) return GDN2_ERR_SHAPE;
  return GDN2_OK;
}

// Sizes of a call: the pieces its sequences are cut into, and its workspace
// [tables of a packed batch][piece states of each sweep][fp32 dq and dk of shared heads].
struct Plan {
  int seg_tok, max_segs;
  bool pieces;
  size_t states, state_bytes, partial, partial_bytes, need;  // offsets, and sizes of one
  bool fits;                                                 // every launch within the grid's limits
};

Plan plan(bool bwd, int N, int T, int Hk, int H, int Dk, int Dv, bool packed, int dt) {
  Plan p{};
  const int sweeps = bwd ? 3 : 1;
  const int E = bwd && Dk < Dv ? Dk : Dv;  // the sweeps' columns (the backward's: Dk and Dv)
  p.seg_tok = gdn2::linattn_seg_tokens(N, T, H, E, bwd ? 2 : 1, packed, dt == GDN2_F32);
  p.max_segs = gdn2::linattn_max_segs(N, T, p.seg_tok, packed);
  p.pieces = packed ? p.seg_tok < T : p.max_segs > 1;
  p.states = packed ? gdn2::linattn_table_bytes(N, p.max_segs) : 0;
  const size_t slots = (size_t)p.max_segs * (packed ? 1 : N);
  p.state_bytes = p.pieces ? al256(slots * H * Dk * Dv * 4) : 0;
  p.partial = p.states + sweeps * p.state_bytes;
  p.partial_bytes = bwd && H != Hk ? al256((size_t)(packed ? 1 : N) * T * H * Dk * 4) : 0;
  p.need = p.partial + 2 * p.partial_bytes;
  const int wide = (Dk > Dv ? Dk : Dv) <= 64 ? 1 : 2;
  // a grid holds fewer than 2^32 threads: 512 a workgroup of the sweeps, 256 and up to 16 workgroups a state to join
  p.fits = slots * H * wide * sweeps < ((size_t)1 << 23) - 64 && (size_t)N * H < (size_t)1 << 20;
  return p;
}

struct Call {
  const void *q, *k, *v;
  const float* log_decay;
  const long long* cu;
  const float* S0;
  int N, T, Hk, H, Dk, Dv;
  float scale;
  int dt;
  char* ws;
  size_t ws_bytes;
  hipStream_t stream;
};

// Checks that come after the sizes', and the packed batch's tables. done: nothing (more) to do, return st.
int begin(const Call& c, bool bwd, Plan& p, gdn2::LinArgs& a) {
  p = plan(bwd, c.N, c.T, c.Hk, c.H, c.Dk, c.Dv, c.cu != nullptr, c.dt);
  if (!p.fits) return GDN2_ERR_SHAPE;
  if (p.need > 0) {
    if (c.ws == nullptr || c.ws_bytes < p.need) return GDN2_ERR_WORKSPACE;
    if (!aligned(c.ws, 256)) return GDN2_ERR_ALIGN;
  }
  a = gdn2::LinArgs{};
  a.log_decay = c.log_decay;
  a.N = c.N;
  a.T = c.T;
  a.H = c.H;
  a.f32 = c.dt == GDN2_F32;
  a.pieces = p.pieces;
  a.seg_tok = p.seg_tok;
  a.max_segs = p.max_segs;
  if (c.cu) return hip_status(gdn2::launch_linattn_plan(reinterpret_cast<const int64_t*>(c.cu), c.ws, a, c.stream));
  return GDN2_OK;
}

int forward(const Call& c, void* o, float* S_final) {
  int st = check_sizes(c.N, c.T, c.Hk, c.H, c.Dk, c.Dv, c.dt);
  if (st != GDN2_OK || c.N == 0 || c.H == 0) return st;
  const int64_t state = (int64_t)c.N * c.H * c.Dk * c.Dv;
  if (c.T == 0) {
    st = check_ptrs({}, {c.S0, S_final});
    if (st != GDN2_OK || S_final == nullptr) return st;
    return hip_status(gdn2::launch_copy_or_zero(S_final, c.S0, state, c.stream));
  }
  st = check_ptrs({c.q, c.k, c.v, o}, {c.S0, S_final});
  if (st == GDN2_OK && c.log_decay == nullptr) st = GDN2_ERR_NULL;
  if (st == GDN2_OK && !aligned(c.log_decay, 4)) st = GDN2_ERR_ALIGN;
  if (st != GDN2_OK) return st;
  Plan p;
  gdn2::LinArgs a;
  st = begin(c, false, p, a);
  if (st != GDN2_OK) return st;
  const int G = c.H / c.Hk;
  a.A = c.Dk;
  a.E = c.Dv;
  a.sw[0] = gdn2::LinSweep{c.q, c.k, c.v, o, G, G, 1, false, false, 1, 1.f, c.scale, c.S0, c.Dv, 1, S_final,
                           reinterpret_cast<float*>(c.ws + p.states)};
  a.sweeps = 1;
  return hip_status(gdn2::launch_linattn_sweeps(a, c.stream));
}

int backward(const Call& c, const void* dO, const float* dS_final, void* dq, void* dk, void* dv, float* dS0) {
  int st = check_sizes(c.N, c.T, c.Hk, c.H, c.Dk, c.Dv, c.dt);
  if (st != GDN2_OK || c.N == 0 || c.H == 0) return st;
  const int64_t state = (int64_t)c.N * c.H * c.Dk * c.Dv;
  if (c.T == 0) {
    st = check_ptrs({}, {dS_final, dS0});
    if (st != GDN2_OK || dS0 == nullptr) return st;
    return hip_status(gdn2::launch_copy_or_zero(dS0, dS_final, state, c.stream));
  }
  st = check_ptrs({c.q, c.k, c.v, dO, dq, dk, dv}, {c.S0, dS_final, dS0});
  if (st == GDN2_OK && c.log_decay == nullptr) st = GDN2_ERR_NULL;
  if (st == GDN2_OK && !aligned(c.log_decay, 4)) st = GDN2_ERR_ALIGN;
  if (st != GDN2_OK) return st;
  Plan p;
  gdn2::LinArgs a;
  st = begin(c, true, p, a);
  if (st != GDN2_OK) return st;
  const int G = c.H / c.Hk;
  const int64_t rows = c.cu ? c.T : (int64_t)c.N * c.T;
  const auto at = [&](size_t offset) { return reinterpret_cast<float*>(c.ws + offset); };
  void* const dq_to = G == 1 ? dq : at(p.partial);
  void* const dk_to = G == 1 ? dk : at(p.partial + p.partial_bytes);
  // dq: the forward recurrence of S^T, over (dO, v, k)
  const gdn2::LinSweep sq{dO, c.v, c.k, dq_to, 1, 1, G, G > 1, false, 1, 1.f, c.scale,
                          c.S0, 1, c.Dv, nullptr, at(p.states)};
  // dk: the reversed recurrence of the state's gradient, transposed, over (v, dO, q)
  const gdn2::LinSweep sk{c.v, dO, c.q, dk_to, 1, 1, G, G > 1, true, 0, c.scale, 1.f,
                          dS_final, 1, c.Dv, nullptr, at(p.states + p.state_bytes)};
  // dv: the same state, over (k, q, dO); its last value is dS0
  const gdn2::LinSweep sv{c.k, c.q, dO, dv, G, G, 1, false, true, 0, c.scale, 1.f,
                          dS_final, c.Dv, 1, dS0, at(p.states + 2 * p.state_bytes)};
  hipError_t e = hipSuccess;
  // dS0 may be S0 or dS_final: with pieces all entering states are read before the last are written, else they are
  // not when dk's and dv's sweeps run side by side
  const bool apart = dS0 != nullptr && (dS0 == c.S0 || dS0 == dS_final) && !p.pieces;
  a.A = c.Dv;
  a.E = c.Dk;
  a.sw[0] = sq;
  a.sw[1] = sk;
  a.sw[2] = sv;
  a.sweeps = c.Dk == c.Dv && !apart ? 3 : 2;
  e = gdn2::launch_linattn_sweeps(a, c.stream);
  if (e == hipSuccess && a.sweeps == 2) {
    a.A = c.Dk;
    a.E = c.Dv;
    a.sw[0] = sv;
    a.sweeps = 1;
    e = gdn2::launch_linattn_sweeps(a, c.stream);
  }
  if (G > 1) {
    for (auto x : {std::pair<void*, void*>{dq_to, dq}, {dk_to, dk}})
      if (e == hipSuccess)
        e = gdn2::launch_linattn_group_sum(static_cast<float*>(x.first), x.second, rows, c.Hk, G, c.Dk, a.f32, a.cu,
                                           c.N, c.stream);
  }
  return hip_status(e);
}

int decode(const void* q, const void* k, const void* v, const float* log_decay, float* S, const int* slots,
           int num_slots, void* o, int B, int Hk, int H, int Dk, int Dv, float scale, int dt, void* stream) {
  int st = check_sizes(B, 1, Hk, H, Dk, Dv, dt);
  if (st != GDN2_OK || B == 0 || H == 0) return st;
  if ((int64_t)B * H >= (int64_t)1 << 24) return GDN2_ERR_SHAPE;  // a grid holds fewer than 2^32 threads
  st = check_ptrs({q, k, v, S, o}, {});
  if (st == GDN2_OK && log_decay == nullptr) st = GDN2_ERR_NULL;
  if (st == GDN2_OK && (!aligned(log_decay, 4) || !aligned(slots, 4))) st = GDN2_ERR_ALIGN;
  if (st != GDN2_OK) return st;
  const gdn2::LinDecodeArgs a{q, k, v, log_decay, S, o, slots, num_slots, B, Hk, H, Dk, Dv, scale, dt == GDN2_F32};
  return hip_status(gdn2::launch_linattn_decode(a, static_cast<hipStream_t>(stream)));
}

Call call(const void* q, const void* k, const void* v, const float* log_decay, const long long* cu, const float* S0,
          int N, int T, int Hk, int H, int Dk, int Dv, float scale, int dt, void* ws, size_t ws_bytes, void* stream) {
  return Call{q, k, v, log_decay, cu, S0, N, T, Hk, H, Dk, Dv, scale, dt, static_cast<char*>(ws), ws_bytes,
              static_cast<hipStream_t>(stream)};
}

// --- head norms with rotation
int norm_sizes(int64_t tokens, int64_t period, int Hq, int Hk, int D, int rot, float eps, int dt, unsigned flags) {
  if (dt != GDN2_F32 && dt != GDN2_BF16) return GDN2_ERR_DTYPE;
  if (tokens < 0 || Hq < 1 || Hk < 0 || D < 0 || rot < 0 || rot > D) return GDN2_ERR_SHAPE;
  if (tokens > 0 && period < 1) return GDN2_ERR_SHAPE;
  if (!(eps >= 0.f)) return GDN2_ERR_SHAPE;
  // the grid as above: 256 threads for every four tokens, fewer than 2^32 in all
  if ((int64_t)Hq + Hk > (1 << 20) || tokens > ((int64_t)1 << 26) - 4) return GDN2_ERR_SHAPE;
  if (!dim_ok(D) || rot % 16 != 0) return GDN2_ERR_UNSUPPORTED;
  if ((flags & ~(GDN2_FLAG_L2_NORM | GDN2_FLAG_INTERLEAVED)) != 0) return GDN2_ERR_UNSUPPORTED;
  return GDN2_OK;
}

int norm_stride(int64_t stride, int heads, int D, int dt) {
  if (heads == 0) return GDN2_OK;
  if (stride < (int64_t)heads * D) return GDN2_ERR_SHAPE;
  return stride % (dt == GDN2_F32 ? 4 : 8) == 0 ? GDN2_OK : GDN2_ERR_ALIGN;
}

int norm_ptrs(int Hk, const long long* positions, const float* inv_freq, int rot,
              std::initializer_list<const void*> q_side, std::initializer_list<const void*> k_side,
              std::initializer_list<const void*> weights) {
  int st = check_ptrs(q_side, weights);
  if (st == GDN2_OK && Hk > 0) st = check_ptrs(k_side, {});
  if (st == GDN2_OK && rot > 0 && inv_freq == nullptr) st = GDN2_ERR_NULL;
  if (st == GDN2_OK && (!aligned(positions, 8) || !aligned(inv_freq, 4))) st = GDN2_ERR_ALIGN;
  return st;
}

}  // namespace

extern "C" {

size_t gdn2_linattn_workspace_bytes(int op, int N, int T, int Hk, int H, int Dk, int Dv, int packed, int dt) {
  if (op != GDN2_OP_FWD && op != GDN2_OP_BWD) return 0;
  if (check_sizes(N, T, Hk, H, Dk, Dv, dt) != GDN2_OK || N == 0 || T == 0 || H == 0) return 0;
  return plan(op == GDN2_OP_BWD, N, T, Hk, H, Dk, Dv, packed != 0, dt).need;
}

int gdn2_linattn_fwd_chunked(const void* q, const void* k, const void* v, const float* log_decay, const float* S0,
                             void* o, float* S_final, void* workspace, size_t workspace_bytes, int B, int T, int Hk,
                             int H, int Dk, int Dv, float scale, int dt, void* stream) {
  return forward(call(q, k, v, log_decay, nullptr, S0, B, T, Hk, H, Dk, Dv, scale, dt, workspace, workspace_bytes,
                      stream), o, S_final);
}

int gdn2_linattn_bwd_chunked(const void* q, const void* k, const void* v, const float* log_decay, const float* S0,
                             const void* dO, const float* dS_final, void* dq, void* dk, void* dv, float* dS0,
                             void* workspace, size_t workspace_bytes, int B, int T, int Hk, int H, int Dk, int Dv,
                             float scale, int dt, void* stream) {
  return backward(call(q, k, v, log_decay, nullptr, S0, B, T, Hk, H, Dk, Dv, scale, dt, workspace, workspace_bytes,
                       stream), dO, dS_final, dq, dk, dv, dS0);
}

int gdn2_linattn_fwd_varlen(const void* q, const void* k, const void* v, const float* log_decay,
                            const long long* cu_seqlens, int N, const float* S0, void* o, float* S_final,
                            void* workspace, size_t workspace_bytes, int T, int Hk, int H, int Dk, int Dv, float scale,
                            int dt, void* stream) {
  if (cu_seqlens == nullptr) return GDN2_ERR_NULL;
  if (!aligned(cu_seqlens, 8)) return GDN2_ERR_ALIGN;
  return forward(call(q, k, v, log_decay, cu_seqlens, S0, N, T, Hk, H, Dk, Dv, scale, dt, workspace, workspace_bytes,
                      stream), o, S_final);
}

int gdn2_linattn_bwd_varlen(const void* q, const void* k, const void* v, const float* log_decay,
                            const long long* cu_seqlens, int N, const float* S0, const void* dO,
                            const float* dS_final, void* dq, void* dk, void* dv, float* dS0, void* workspace,
                            size_t workspace_bytes, int T, int Hk, int H, int Dk, int Dv, float scale, int dt,
                            void* stream) {
  if (cu_seqlens == nullptr) return GDN2_ERR_NULL;
  if (!aligned(cu_seqlens, 8)) return GDN2_ERR_ALIGN;
  return backward(call(q, k, v, log_decay, cu_seqlens, S0, N, T, Hk, H, Dk, Dv, scale, dt, workspace, workspace_bytes,
                       stream), dO, dS_final, dq, dk, dv, dS0);
}

int gdn2_varlen_zero_outside(void* x, const long long* cu_seqlens, int N, int T, size_t row_bytes, void* stream) {
  if (N < 0 || T < 0) return GDN2_ERR_SHAPE;
  if (N == 0 || T == 0 || row_bytes == 0) return GDN2_OK;
  if (x == nullptr || cu_seqlens == nullptr) return GDN2_ERR_NULL;
  if (!aligned(x, 16) || !aligned(cu_seqlens, 8) || row_bytes % 16 != 0) return GDN2_ERR_ALIGN;
  return hip_status(gdn2::launch_linattn_outside(x, reinterpret_cast<const int64_t*>(cu_seqlens), N, T,
                                                 (int64_t)row_bytes, static_cast<hipStream_t>(stream)));
}

int gdn2_linattn_decode_step(const void* q, const void* k, const void* v, const float* log_decay, float* S, void* o,
                             int B, int Hk, int H, int Dk, int Dv, float scale, int dt, void* stream) {
  return decode(q, k, v, log_decay, S, nullptr, 0, o, B, Hk, H, Dk, Dv, scale, dt, stream);
}

int gdn2_linattn_decode_step_slots(const void* q, const void* k, const void* v, const float* log_decay, float* S_pool,
                                   const int* slots, int num_slots, void* o, int B, int Hk, int H, int Dk, int Dv,
                                   float scale, int dt, void* stream) {
  if (num_slots < 0) return GDN2_ERR_SHAPE;
  if (B > 0 && H > 0 && slots == nullptr) return GDN2_ERR_NULL;
  return decode(q, k, v, log_decay, S_pool, slots, num_slots, o, B, Hk, H, Dk, Dv, scale, dt, stream);
}

int gdn2_qk_norm_rope_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                          const long long* positions, const float* inv_freq, void* q_out, void* k_out,
                          long long tokens, long long period, int Hq, int Hk, int D, int rot, long long q_stride,
                          long long k_stride, long long q_out_stride, long long k_out_stride, float eps, float q_scale,
                          int dt, unsigned flags, void* stream) {
  int st = norm_sizes(tokens, period, Hq, Hk, D, rot, eps, dt, flags);
  if (st != GDN2_OK || tokens == 0) return st;
  st = norm_ptrs(Hk, positions, inv_freq, rot, {q, q_out}, {k, k_out}, {q_weight, k_weight});
  for (const auto& s : {norm_stride(q_stride, Hq, D, dt), norm_stride(q_out_stride, Hq, D, dt),
                        norm_stride(k_stride, Hk, D, dt), norm_stride(k_out_stride, Hk, D, dt)})
    if (st == GDN2_OK) st = s;
  if (st != GDN2_OK) return st;
  gdn2::QkNormArgs a{};
  a.s[0] = gdn2::QkNormSide{q, nullptr, q_out, q_weight, nullptr, Hq, q_stride, q_out_stride, q_scale};
  a.s[1] = gdn2::QkNormSide{k, nullptr, k_out, k_weight, nullptr, Hk, k_stride, k_out_stride, 1.f};
  a.pos = reinterpret_cast<const int64_t*>(positions);
  a.inv_freq = inv_freq;
  a.tokens = tokens;
  a.period = period;
  a.D = D;
  a.rot = rot;
  a.eps = eps;
  a.inv_count = (flags & GDN2_FLAG_L2_NORM) ? 1.f : 1.f / (float)D;
  a.interleaved = (flags & GDN2_FLAG_INTERLEAVED) != 0;
  a.f32 = dt == GDN2_F32;
  return hip_status(gdn2::launch_qk_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t gdn2_qk_norm_rope_workspace_bytes(long long tokens, int Hq, int Hk, int D) {
  if (norm_sizes(tokens, 1, Hq, Hk, D, 0, 0.f, GDN2_F32, 0) != GDN2_OK || tokens == 0) return 0;
  return (size_t)gdn2::qk_norm_bwd_workgroups(tokens, Hq, Hk, D) * 2 * D * sizeof(float);
}

int gdn2_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, const float* q_weight,
                          const float* k_weight, const long long* positions, const float* inv_freq, void* dq, void* dk,
                          float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                          long long tokens, long long period, int Hq, int Hk, int D, int rot, long long q_stride,
                          long long k_stride, long long q_grad_stride, long long k_grad_stride, float eps,
                          float q_scale, int dt, int dt_grad, unsigned flags, void* stream) {
  int st = norm_sizes(tokens, period, Hq, Hk, D, rot, eps, dt, flags);
  if (st != GDN2_OK) return st;
  if (dt_grad != dt && dt_grad != GDN2_F32) return GDN2_ERR_DTYPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (tokens == 0) {
    st = check_ptrs({}, {dq_weight, dk_weight});
    if (st == GDN2_OK && dq_weight) st = hip_status(gdn2::launch_copy_or_zero(dq_weight, nullptr, D, s));
    if (st == GDN2_OK && dk_weight) st = hip_status(gdn2::launch_copy_or_zero(dk_weight, nullptr, D, s));
    return st;
  }
  st = norm_ptrs(Hk, positions, inv_freq, rot, {q, dq_out, dq}, {k, dk_out, dk},
                 {q_weight, k_weight, dq_weight, dk_weight});
  for (const auto& x : {norm_stride(q_stride, Hq, D, dt), norm_stride(q_grad_stride, Hq, D, dt),
                        norm_stride(k_stride, Hk, D, dt), norm_stride(k_grad_stride, Hk, D, dt)})
    if (st == GDN2_OK) st = x;
  if (st != GDN2_OK) return st;
  gdn2::QkNormArgs a{};
  a.s[0] = gdn2::QkNormSide{q, dq_out, dq, q_weight, dq_weight, Hq, q_stride, q_grad_stride, q_scale};
  a.s[1] = gdn2::QkNormSide{k, dk_out, dk, k_weight, dk_weight, Hk, k_stride, k_grad_stride, 1.f};
  a.pos = reinterpret_cast<const int64_t*>(positions);
  a.inv_freq = inv_freq;
  a.tokens = tokens;
  a.period = period;
  a.D = D;
  a.rot = rot;
  a.eps = eps;
  a.inv_count = (flags & GDN2_FLAG_L2_NORM) ? 1.f : 1.f / (float)D;
  a.interleaved = (flags & GDN2_FLAG_INTERLEAVED) != 0;
  a.f32 = dt == GDN2_F32;
  a.f32_dy = dt_grad == GDN2_F32;
  if (dq_weight || dk_weight) {
    if (workspace == nullptr || workspace_bytes < gdn2_qk_norm_rope_workspace_bytes(tokens, Hq, Hk, D))
      return GDN2_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return GDN2_ERR_ALIGN;
    a.partial = static_cast<float*>(workspace);
  }
  return hip_status(gdn2::launch_qk_norm_bwd(a, s));
}

}  // extern "C"
