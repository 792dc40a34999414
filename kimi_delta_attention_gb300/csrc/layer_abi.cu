// layer_abi.cu -- C ABI of the gated linear recurrence, of group norm and of the AdamW step
// (include/kda.h): host-side validation, workspace sizing and dispatch.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "../../include/kda.h"
#include "layer_ops.cuh"
#include "wait_limit.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
  const void* p;
  size_t n;
};

bool overlaps(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

bool is_dtype(int64_t d) { return d == KDA_F32 || d == KDA_BF16; }
size_t size_of(int64_t d) { return d == KDA_BF16 ? 2 : 4; }

constexpr int kMostChannels = 1 << 30;  // channels, and steps past the last one, are counted in 32 bits on the device

// ------------------------------------------------------------ linear recurrence --
struct GlrSizes {
  size_t ns, tokens, io, gate, state;  // sequences, tokens, bytes
};

kda_status check_glr(const kda_glr_shape* s, bool packed, GlrSizes& z) {
  if (!s || s->B < 0 || s->T < 0 || s->D < 1 || s->num_seqs < 0) return KDA_ERR_INVALID_ARG;
  if (!is_dtype(s->io_dtype) || !is_dtype(s->gate_dtype)) return KDA_ERR_INVALID_ARG;
  if (packed ? (s->B != 1 || s->num_seqs < 1) : s->num_seqs != 0) return KDA_ERR_INVALID_ARG;
  z.ns = packed ? static_cast<size_t>(s->num_seqs) : static_cast<size_t>(s->B);
  z.tokens = static_cast<size_t>(s->B) * s->T;
  if (z.tokens > INT32_MAX || s->D > kMostChannels) return KDA_ERR_UNSUPPORTED;  // tokens are counted in 32 bits on the device
  z.io = z.tokens * s->D * size_of(s->io_dtype);
  z.gate = z.tokens * s->D * size_of(s->gate_dtype);
  z.state = z.ns * s->D * 4;
  return KDA_OK;
}

size_t glr_workspace_size(const kda_glr_shape* s) {
  GlrSizes z;
  return check_glr(s, s && s->num_seqs > 0, z) == KDA_OK ? kda::kWorkspaceBytes : 0;   // the status word
}

// Both directions: `ins` inputs, `outs` outputs (the last one may be the array `same`).
kda_status run_glr(const kda_glr_shape* s, const GlrSizes& z, kda::glr::Params p, bool backward, const Span* ins, int n_ins,
                   const Span* outs, int n_outs, const void* same, void* workspace, size_t workspace_bytes, void* stream) {
  if (!workspace || workspace_bytes < kda::kWorkspaceBytes) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return KDA_ERR_ALIGNMENT;
  const Span w{workspace, workspace_bytes};
  for (int i = 0; i < n_outs; ++i) {
    for (int j = 0; j < n_ins; ++j)
      if (overlaps(outs[i], ins[j]) && !(i == n_outs - 1 && outs[i].p == same && ins[j].p == same)) return KDA_ERR_INVALID_ARG;
    for (int j = i + 1; j < n_outs; ++j)
      if (overlaps(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
    if (overlaps(outs[i], w)) return KDA_ERR_INVALID_ARG;
  }
  for (int j = 0; j < n_ins; ++j)
    if (overlaps(ins[j], w)) return KDA_ERR_INVALID_ARG;
  if (z.ns == 0) return KDA_OK;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  p.status = static_cast<uint32_t*>(workspace);
  p.wait_ns = kda::wait_limit_ns();
  p.tokens = static_cast<long>(z.tokens);
  p.T = s->T;
  p.D = s->D;
  p.num_seqs = static_cast<int>(z.ns);
  return kda::glr::launch(p, backward, s->io_dtype == KDA_BF16, s->gate_dtype == KDA_BF16, cs) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// ------------------------------------------------------------------- group norm --
kda_status check_gn(int64_t N, int64_t L, int C, int groups) {
  if (N < 0 || L < 1 || C < 1 || groups < 1 || C % groups != 0) return KDA_ERR_INVALID_ARG;
  // rows (samples x positions) are counted in 32 bits on the device
  if (N > INT32_MAX || L > INT32_MAX || N * L > INT32_MAX || N * groups > INT32_MAX || C > kMostChannels) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

bool is_activation(int a) { return a == KDA_ACT_NONE || a == KDA_ACT_SILU; }

// ------------------------------------------------------------------------ AdamW --
struct Range {
  uintptr_t at, end;
  bool written;
};

// Whether a range that is written overlaps any other.
bool clash(Range* r, int n) {
  std::sort(r, r + n, [](const Range& a, const Range& b) { return a.at < b.at; });
  uintptr_t any = 0, written = 0;  // furthest end of the ranges before
  for (int i = 0; i < n; ++i) {
    if (r[i].at < written || (r[i].written && r[i].at < any)) return true;
    any = std::max(any, r[i].end);
    if (r[i].written) written = std::max(written, r[i].end);
  }
  return false;
}

}  // namespace

extern "C" {

size_t kda_glr_fwd_workspace_size(const kda_glr_shape* s) { return glr_workspace_size(s); }
size_t kda_glr_bwd_workspace_size(const kda_glr_shape* s) { return glr_workspace_size(s); }

kda_status kda_glr_fwd(const kda_glr_shape* s, const void* x, const void* g, const float* initial_state,
                       const int32_t* cu_seqlens, void* y, float* final_state, void* workspace, size_t workspace_bytes,
                       void* stream) {
  GlrSizes z;
  const kda_status st = check_glr(s, cu_seqlens != nullptr, z);
  if (st != KDA_OK) return st;
  if (z.tokens > 0 && (!x || !g || !y)) return KDA_ERR_INVALID_ARG;
  const size_t es = size_of(s->io_dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(g, size_of(s->gate_dtype)) || !aligned(initial_state, 4) ||
      !aligned(final_state, 4) || !aligned(cu_seqlens, 4))
    return KDA_ERR_ALIGNMENT;
  const Span ins[] = {{x, z.io}, {g, z.gate}, {initial_state, z.state}, {cu_seqlens, (z.ns + 1) * 4}};
  const Span outs[] = {{y, z.io}, {final_state, z.state}};
  kda::glr::Params p{};
  p.x = x; p.g = g; p.h0 = p.init = initial_state; p.cu = cu_seqlens; p.out = y; p.fin = final_state;
  return run_glr(s, z, p, false, ins, 4, outs, 2, initial_state, workspace, workspace_bytes, stream);
}

kda_status kda_glr_bwd(const kda_glr_shape* s, const void* g, const void* y, const void* d_out, const float* initial_state,
                       const int32_t* cu_seqlens, const float* d_final_state, void* dx, void* dg, float* d_initial_state,
                       void* workspace, size_t workspace_bytes, void* stream) {
  GlrSizes z;
  const kda_status st = check_glr(s, cu_seqlens != nullptr, z);
  if (st != KDA_OK) return st;
  if (z.tokens > 0 && (!g || !y || !d_out || !dx || !dg)) return KDA_ERR_INVALID_ARG;
  const size_t es = size_of(s->io_dtype), gs = size_of(s->gate_dtype);
  if (!aligned(y, es) || !aligned(d_out, es) || !aligned(dx, es) || !aligned(g, gs) || !aligned(dg, gs) ||
      !aligned(initial_state, 4) || !aligned(d_final_state, 4) || !aligned(d_initial_state, 4) || !aligned(cu_seqlens, 4))
    return KDA_ERR_ALIGNMENT;
  const Span ins[] = {{g, z.gate}, {y, z.io}, {d_out, z.io}, {initial_state, z.state}, {cu_seqlens, (z.ns + 1) * 4},
                      {d_final_state, z.state}};
  const Span outs[] = {{dx, z.io}, {dg, z.gate}, {d_initial_state, z.state}};
  kda::glr::Params p{};
  p.x = d_out; p.g = g; p.y = y; p.h0 = initial_state; p.init = d_final_state; p.cu = cu_seqlens;
  p.out = dx; p.dg = dg; p.fin = d_initial_state;
  return run_glr(s, z, p, true, ins, 6, outs, 3, d_final_state, workspace, workspace_bytes, stream);
}

kda_status kda_glr_step(const kda_glr_shape* s, const void* x, const void* g, float* state, const int32_t* slots,
                        int num_slots, void* y, uint32_t* status_word, void* stream) {
  GlrSizes z;
  const kda_status st = check_glr(s, false, z);
  if (st != KDA_OK) return st;
  if (num_slots < 0) return KDA_ERR_INVALID_ARG;
  if (z.ns == 0 || z.tokens == 0) return KDA_OK;  // (no live request: an empty `slots` has no address)
  if (!slots && num_slots != 0) return KDA_ERR_INVALID_ARG;
  if (!x || !g || !state || !y) return KDA_ERR_INVALID_ARG;
  const size_t es = size_of(s->io_dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(g, size_of(s->gate_dtype)) || !aligned(state, 4) ||
      !aligned(slots, 4) || !aligned(status_word, 4))
    return KDA_ERR_ALIGNMENT;
  const Span o{y, z.io}, f{state, slots ? static_cast<size_t>(num_slots) * s->D * 4 : z.state};
  const Span ins[] = {{x, z.io}, {g, z.gate}, {slots, z.ns * 4}, {status_word, 4}};
  for (const Span& i : ins)
    if (overlaps(o, i) || overlaps(f, i)) return KDA_ERR_INVALID_ARG;
  if (overlaps(o, f)) return KDA_ERR_INVALID_ARG;
  const kda::glr::StepParams p{x, g, state, slots, y, status_word, s->B, s->T, s->D, num_slots};
  return kda::glr::launch_step(p, s->io_dtype == KDA_BF16, s->gate_dtype == KDA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK
             : KDA_ERR_CUDA;
}

size_t kda_group_norm_fwd_workspace_size(int64_t N, int64_t L, int C, int groups) {
  return check_gn(N, L, C, groups) == KDA_OK ? 256 + kda::gn::fwd_workspace_bytes(N, L, C, groups) : 0;
}

kda_status kda_group_norm_fwd(int64_t N, int64_t L, int C, int groups, kda_dtype io_dtype, kda_activation act, const void* x,
                              const float* weight, const float* bias, float eps, void* y, float* mean, float* rstd,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const kda_status st = check_gn(N, L, C, groups);
  if (st != KDA_OK) return st;
  if (!is_dtype(io_dtype) || !is_activation(act) || !(eps >= 0.f) || !std::isfinite(eps)) return KDA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kda_group_norm_fwd_workspace_size(N, L, C, groups)) return KDA_ERR_WORKSPACE;
  if (N > 0 && (!x || !y)) return KDA_ERR_INVALID_ARG;
  const size_t es = size_of(io_dtype), n = static_cast<size_t>(N) * L * C * es, stats = static_cast<size_t>(N) * groups * 4;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(workspace, 16))
    return KDA_ERR_ALIGNMENT;
  const Span ins[] = {{x, n}, {weight, size_t(C) * 4}, {bias, size_t(C) * 4}};
  const Span outs[] = {{y, n}, {mean, stats}, {rstd, stats}, {workspace, workspace_bytes}};
  for (int i = 0; i < 4; ++i) {
    for (const Span& j : ins)
      if (overlaps(outs[i], j)) return KDA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
  }
  if (N == 0) return KDA_OK;
  const kda::gn::Params p{x, nullptr, weight, bias, y, mean, rstd, nullptr, nullptr, static_cast<uint8_t*>(workspace),
                          N, L, C, groups, eps, act == KDA_ACT_SILU};
  return kda::gn::launch_fwd(p, io_dtype == KDA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_group_norm_bwd_workspace_size(int64_t N, int64_t L, int C, int groups) {
  return check_gn(N, L, C, groups) == KDA_OK ? 256 + kda::gn::bwd_workspace_bytes(N, L, C, groups) : 0;
}

kda_status kda_group_norm_bwd(int64_t N, int64_t L, int C, int groups, kda_dtype io_dtype, kda_activation act, const void* x,
                              const void* dy, const float* weight, const float* bias, const float* mean, const float* rstd,
                              void* dx, float* dweight, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  const kda_status st = check_gn(N, L, C, groups);
  if (st != KDA_OK) return st;
  if (!is_dtype(io_dtype) || !is_activation(act)) return KDA_ERR_INVALID_ARG;
  if (!dx && !dweight && !dbias) return KDA_ERR_INVALID_ARG;
  if (N > 0 && (!x || !dy || !mean || !rstd)) return KDA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kda_group_norm_bwd_workspace_size(N, L, C, groups)) return KDA_ERR_WORKSPACE;
  const size_t es = size_of(io_dtype), n = static_cast<size_t>(N) * L * C * es, stats = static_cast<size_t>(N) * groups * 4;
  if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(workspace, 16))
    return KDA_ERR_ALIGNMENT;
  const Span ins[] = {{x, n}, {dy, n}, {weight, size_t(C) * 4}, {bias, size_t(C) * 4}, {mean, stats}, {rstd, stats}};
  const Span outs[] = {{dx, n}, {dweight, size_t(C) * 4}, {dbias, size_t(C) * 4}, {workspace, workspace_bytes}};
  for (int i = 0; i < 4; ++i) {
    for (const Span& j : ins)
      if (overlaps(outs[i], j)) return KDA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
  }
  const kda::gn::Params p{x, dy, weight, bias, dx, const_cast<float*>(mean), const_cast<float*>(rstd), dweight, dbias,
                          static_cast<uint8_t*>(workspace), N, L, C, groups, 0.f, act == KDA_ACT_SILU};
  return kda::gn::launch_bwd(p, io_dtype == KDA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_adamw_step(const kda_adamw_tensor* tensors, int count, const kda_adamw_config* c, void* stream) {
  if (count < 0 || count > (1 << 20) || (count > 0 && !tensors) || !c) return KDA_ERR_INVALID_ARG;
  if (c->state_bits != 8 && c->state_bits != 32) return KDA_ERR_INVALID_ARG;
  const bool packed = c->state_bits == 8;
  auto good = [](double v) { return v >= 0 && std::isfinite(static_cast<float>(v)); };   // (the step is one in fp32)
  // an eps that fp32 holds as a subnormal, or not at all, would be nothing beside a v of 0, and m = 0 over it NaN
  if (!good(c->lr) || !good(c->eps) || !good(c->weight_decay) || (c->eps > 0 && c->eps < FLT_MIN) || !(c->beta1 >= 0 && c->beta1 < 1) ||
      !(c->beta2 >= 0 && c->beta2 < 1))
    return KDA_ERR_INVALID_ARG;
  if (!c->step_device && (c->step < 1 || c->step > INT32_MAX)) return KDA_ERR_INVALID_ARG;
  if (!aligned(c->step_device, 4) || !aligned(c->lr_device, 4) || !aligned(c->grad_scale, 4) || !aligned(c->skip, 4))
    return KDA_ERR_ALIGNMENT;
  if (count == 0) return KDA_OK;
  Range* r = static_cast<Range*>(std::malloc((7 * static_cast<size_t>(count) + 4) * sizeof(Range)));
  if (!r) return KDA_ERR_INVALID_ARG;
  int n = 0;
  kda_status st = KDA_OK;
  auto add = [&](const void* p, size_t bytes, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    r[n++] = {a, a + bytes, written};
  };
  for (int i = 0; i < count && st == KDA_OK; ++i) {
    const kda_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t(1) << 40) || !is_dtype(t.param_dtype) || !is_dtype(t.grad_dtype)) st = KDA_ERR_INVALID_ARG;
    if (st != KDA_OK || t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (packed ? !t.m_scale || !t.v_scale : t.m_scale || t.v_scale)) st = KDA_ERR_INVALID_ARG;
    const size_t ps = size_of(t.param_dtype), gs = size_of(t.grad_dtype), ss = packed ? 1 : 4, len = static_cast<size_t>(t.n);
    if (!aligned(t.param, ps) || !aligned(t.grad, gs) || !aligned(t.m, ss) || !aligned(t.v, ss) || !aligned(t.m_scale, 4) ||
        !aligned(t.v_scale, 4) || !aligned(t.master, 4))
      st = st != KDA_OK ? st : KDA_ERR_ALIGNMENT;
    if (st != KDA_OK) continue;
    add(t.param, len * ps, true);
    add(t.grad, len * gs, false);
    add(t.m, len * ss, true);
    add(t.v, len * ss, true);
    const size_t blocks = (len + KDA_ADAMW_BLOCK - 1) / KDA_ADAMW_BLOCK;
    if (packed) {
      add(t.m_scale, blocks * 4, true);
      add(t.v_scale, blocks * 4, true);
    }
    if (t.master) add(t.master, len * 4, true);
  }
  const void* words[] = {c->step_device, c->lr_device, c->grad_scale, c->skip};
  for (const void* w : words)
    if (w) add(w, 4, false);
  if (st == KDA_OK && clash(r, n)) st = KDA_ERR_INVALID_ARG;
  std::free(r);
  if (st != KDA_OK) return st;
  return kda::adamw::launch(tensors, count, *c, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
