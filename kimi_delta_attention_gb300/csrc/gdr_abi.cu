// gdr_abi.cu -- C ABI of the gated delta rule with a scalar gate and of layer norm
// (include/kda.h): host-side validation, workspace sizing and dispatch.
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "../../include/kda.h"
#include "gdr_common.cuh"

namespace kda {
namespace gdr {
cudaError_t launch_step(const Params& p, float* state, const int32_t* slots, int num_slots, int K, int V, bool bf16,
                        cudaStream_t stream);
cudaError_t launch_recurrent(const Params& p, int K, int V, bool bf16, cudaStream_t stream);
size_t chunk_slots(size_t tokens, size_t ns, bool packed, int T);
size_t chunk_fwd_bytes(size_t slots, int HV);
cudaError_t launch_chunk_fwd(const Params& p, uint8_t* rec, unsigned long long wait_ns, int K, int V, cudaStream_t st);
size_t chunk_bwd_bytes(size_t slots, int HV, int K, int V);
cudaError_t launch_chunk_bwd(const Params& p, const void* dout, const float* dfin, void* dq, void* dk, void* dv,
                             float* dg, float* dbeta, float* ds0, uint8_t* ws, float* shares,
                             unsigned long long wait_ns, int K, int V, cudaStream_t st);
}  // namespace gdr
namespace ln {
size_t bwd_workspace_bytes(long rows, int D);
cudaError_t launch_fwd(const void* x, long ldx, const float* w, const float* b, float eps, void* y, float* mean,
                       float* rstd, long rows, int D, bool bf16, cudaStream_t st);
cudaError_t launch_bwd(const void* x, long ldx, const void* dy, long lddy, const float* w, const float* mean,
                       const float* rstd, void* dx, float* dw, float* db, float* ws, long rows, int D, bool bf16,
                       cudaStream_t st);
}  // namespace ln
}  // namespace kda

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

// Sizes of the arguments of a shape, after the checks every delta-rule entry shares.
struct Sizes {
  size_t ns, tokens, qk, v, gate, state;  // sequences, tokens, bytes
};

kda_status check_shape(const kda_shape* s, bool packed, Sizes& z) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->B < 0 || s->T < 0 || s->H < 1 || s->HV < 1 || s->K < 1 || s->V < 1 || s->num_seqs < 0)
    return KDA_ERR_INVALID_ARG;
  if (s->HV % s->H != 0) return KDA_ERR_INVALID_ARG;
  if (s->io_dtype != KDA_F32 && s->io_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (packed ? (s->B != 1 || s->num_seqs < 1) : s->num_seqs != 0) return KDA_ERR_INVALID_ARG;
  if ((s->K != 64 && s->K != 128) || (s->V != 64 && s->V != 128)) return KDA_ERR_UNSUPPORTED;
  const size_t es = s->io_dtype == KDA_BF16 ? 2 : 4;
  z.ns = packed ? static_cast<size_t>(s->num_seqs) : static_cast<size_t>(s->B);
  z.tokens = static_cast<size_t>(s->B) * s->T;
  // (sequence, value head) pairs and 64-token chunks are counted in 32 bits on the device
  if (z.ns * s->HV > (1u << 28) || (z.tokens / 64 + z.ns) * s->HV > (1u << 28)) return KDA_ERR_UNSUPPORTED;
  z.qk = z.tokens * s->H * s->K * es;
  z.v = z.tokens * s->HV * s->V * es;
  z.gate = z.tokens * s->HV * 4;
  z.state = z.ns * s->HV * s->K * s->V * 4;
  return KDA_OK;
}

// Limit of the kernels' bounded waits: 2 s, or KDA_WAIT_LIMIT_NS (read at each call).
unsigned long long wait_limit_ns() {
  const char* e = std::getenv("KDA_WAIT_LIMIT_NS");
  if (e) {
    char* end = nullptr;
    const unsigned long long v = std::strtoull(e, &end, 10);
    if (end != e && v > 0) return v;
  }
  return 2000000000ull;
}

// The chunk kernels' part of a workspace: 128-byte aligned, after the status word.
constexpr size_t kChunkAlign = 128;
uint8_t* chunk_part(void* workspace) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(workspace) + kda::kWorkspaceBytes;
  return reinterpret_cast<uint8_t*>((at + kChunkAlign - 1) & ~(kChunkAlign - 1));
}

// bf16 I/O runs the chunk kernels; fp32 I/O the token recurrence (its q, k and v are not
// exact tensor-core operands).
bool chunked(const kda_shape* s, const Sizes& z) { return s->io_dtype == KDA_BF16 && z.tokens > 0; }

bool good_scale(float scale) { return scale > 0.f && std::isfinite(scale); }

}  // namespace

extern "C" {

size_t kda_gdr_fwd_workspace_size(const kda_shape* s) {
  Sizes z;
  if (check_shape(s, s && s->num_seqs > 0, z) != KDA_OK) return 0;
  if (!chunked(s, z)) return kda::kWorkspaceBytes;
  return kda::kWorkspaceBytes + kChunkAlign +
         kda::gdr::chunk_fwd_bytes(kda::gdr::chunk_slots(z.tokens, z.ns, s->num_seqs > 0, s->T), s->HV);
}

kda_status kda_gdr_fwd(const kda_shape* s, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, float scale, const float* initial_state, const int32_t* cu_seqlens,
                       void* out, float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  Sizes z;
  const kda_status st = check_shape(s, cu_seqlens != nullptr, z);
  if (st != KDA_OK) return st;
  if (!good_scale(scale)) return KDA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kda_gdr_fwd_workspace_size(s)) return KDA_ERR_WORKSPACE;
  if (z.tokens > 0 && (!q || !k || !v || !g || !beta || !out)) return KDA_ERR_INVALID_ARG;
  const void* ptrs16[] = {q, k, v, out, initial_state, final_state, workspace};
  for (const void* p : ptrs16)
    if (p && !aligned(p, 16)) return KDA_ERR_ALIGNMENT;
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_ALIGNMENT;
  const Span o{out, z.v}, f{final_state, z.state}, w{workspace, workspace_bytes};
  const Span ins[] = {{q, z.qk}, {k, z.qk}, {v, z.v}, {g, z.gate}, {beta, z.gate}, {initial_state, z.state}, {cu_seqlens, cu_seqlens ? (z.ns + 1) * 4 : 0}};
  for (int i = 0; i < 7; ++i) {
    if (overlaps(o, ins[i]) || overlaps(w, ins[i])) return KDA_ERR_INVALID_ARG;
    if (overlaps(f, ins[i]) && !(i == 5 && final_state == initial_state)) return KDA_ERR_INVALID_ARG;
  }
  if (overlaps(o, f) || overlaps(w, o) || overlaps(w, f)) return KDA_ERR_INVALID_ARG;
  if (z.ns == 0) return KDA_OK;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint32_t* status = static_cast<uint32_t*>(workspace);
  const kda::gdr::Params p{q, k, v, g, beta, initial_state, cu_seqlens, out, final_state, status, scale, s->T,
                           s->H, s->HV, static_cast<int>(z.ns)};
  if (!chunked(s, z) && cudaMemsetAsync(status, 0, sizeof(uint32_t), cs) != cudaSuccess) return KDA_ERR_CUDA;
  const cudaError_t e =
      chunked(s, z) ? kda::gdr::launch_chunk_fwd(p, chunk_part(workspace), wait_limit_ns(), s->K, s->V, cs)
                    : kda::gdr::launch_recurrent(p, s->K, s->V, s->io_dtype == KDA_BF16, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

namespace {
// Workspace of the backward: the status word, the chunks' intermediates, and with grouped
// value heads their fp32 shares of dq and dk.
size_t bwd_shares_at(const kda_shape* s, const Sizes& z) {  // from chunk_part()
  return kda::gdr::chunk_bwd_bytes(kda::gdr::chunk_slots(z.tokens, z.ns, s->num_seqs > 0, s->T),
                                                          s->HV, s->K, s->V);
}
size_t bwd_bytes(const kda_shape* s, const Sizes& z) {
  if (z.tokens == 0) return kda::kWorkspaceBytes;
  return kda::kWorkspaceBytes + kChunkAlign + bwd_shares_at(s, z) + (s->HV != s->H ? 2 * z.tokens * s->HV * s->K * sizeof(float) : 0);
}
}  // namespace

size_t kda_gdr_bwd_workspace_size(const kda_shape* s) {
  Sizes z;
  if (check_shape(s, s && s->num_seqs > 0, z) != KDA_OK || s->io_dtype != KDA_BF16) return 0;
  return bwd_bytes(s, z);
}

kda_status kda_gdr_bwd(const kda_shape* s, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, float scale, const float* initial_state, const int32_t* cu_seqlens,
                       const void* d_out, const float* d_final_state, void* dq, void* dk, void* dv, float* dg,
                       float* dbeta, float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
  Sizes z;
  const kda_status st = check_shape(s, cu_seqlens != nullptr, z);
  if (st != KDA_OK) return st;
  if (!good_scale(scale)) return KDA_ERR_INVALID_ARG;
  if (s->io_dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < bwd_bytes(s, z)) return KDA_ERR_WORKSPACE;
  if (z.tokens > 0 && (!q || !k || !v || !g || !beta || !d_out || !dq || !dk || !dv || !dg || !dbeta))
    return KDA_ERR_INVALID_ARG;
  const void* ptrs16[] = {q, k, v, initial_state, d_out, d_final_state, dq, dk, dv, d_initial_state, workspace};
  for (const void* p : ptrs16)
    if (p && !aligned(p, 16)) return KDA_ERR_ALIGNMENT;
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(dg, 4) || !aligned(dbeta, 4) || !aligned(cu_seqlens, 4))
    return KDA_ERR_ALIGNMENT;
  const Span ins[] = {{q, z.qk}, {k, z.qk}, {v, z.v}, {g, z.gate}, {beta, z.gate}, {initial_state, z.state},
                      {d_out, z.v}, {d_final_state, z.state}, {cu_seqlens, cu_seqlens ? (z.ns + 1) * 4 : 0}};
  const Span outs[] = {{dq, z.qk}, {dk, z.qk}, {dv, z.v}, {dg, z.gate}, {dbeta, z.gate}, {d_initial_state, z.state},
                       {workspace, workspace_bytes}};
  for (int i = 0; i < 7; ++i) {
    for (const Span& j : ins)
      if (overlaps(outs[i], j)) return KDA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 7; ++j)
      if (overlaps(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
  }
  if (z.ns == 0) return KDA_OK;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint32_t* status = static_cast<uint32_t*>(workspace);
  if (z.tokens == 0) {  // no tokens: the state's gradient passes through
    if (cudaMemsetAsync(status, 0, sizeof(uint32_t), cs) != cudaSuccess) return KDA_ERR_CUDA;
    if (!d_initial_state) return KDA_OK;
    const cudaError_t e = d_final_state ? cudaMemcpyAsync(d_initial_state, d_final_state, z.state, cudaMemcpyDeviceToDevice, cs)
                                        : cudaMemsetAsync(d_initial_state, 0, z.state, cs);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
  }
  const kda::gdr::Params p{q, k, v, g, beta, initial_state, cu_seqlens, nullptr, nullptr, status, scale, s->T,
                           s->H, s->HV, static_cast<int>(z.ns)};
  uint8_t* ws = chunk_part(workspace);
  return kda::gdr::launch_chunk_bwd(p, d_out, d_final_state, dq, dk, dv, dg, dbeta, d_initial_state, ws, reinterpret_cast<float*>(ws + bwd_shares_at(s, z)),
                                    wait_limit_ns(), s->K, s->V, cs) == cudaSuccess
             ? KDA_OK
             : KDA_ERR_CUDA;
}

kda_status kda_gdr_step(const kda_shape* s, const void* q, const void* k, const void* v, const float* g,
                        const float* beta, float scale, float* state, const int32_t* slots, int num_slots, void* out,
                        uint32_t* status_word, void* stream) {
  Sizes z;
  const kda_status st = check_shape(s, false, z);
  if (st != KDA_OK) return st;
  if (!good_scale(scale)) return KDA_ERR_INVALID_ARG;
  if (num_slots < 0) return KDA_ERR_INVALID_ARG;
  if (z.ns == 0 || z.tokens == 0) return KDA_OK;   // (no live request: an empty `slots` has no address)
  if (!slots && num_slots != 0) return KDA_ERR_INVALID_ARG;
  if (!state || !q || !k || !v || !g || !beta || !out) return KDA_ERR_INVALID_ARG;
  const void* ptrs16[] = {q, k, v, out, state};
  for (const void* p : ptrs16)
    if (!aligned(p, 16)) return KDA_ERR_ALIGNMENT;
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(slots, 4) || !aligned(status_word, 4)) return KDA_ERR_ALIGNMENT;
  const size_t pool = slots ? static_cast<size_t>(num_slots) * s->HV * s->K * s->V * 4 : z.state;
  const Span o{out, z.v}, f{state, pool};
  const Span ins[] = {{q, z.qk}, {k, z.qk}, {v, z.v}, {g, z.gate}, {beta, z.gate}, {slots, z.ns * 4}, {status_word, 4}};
  for (const Span& i : ins)
    if (overlaps(o, i) || overlaps(f, i)) return KDA_ERR_INVALID_ARG;
  if (overlaps(o, f)) return KDA_ERR_INVALID_ARG;
  const kda::gdr::Params p{q, k, v, g, beta, nullptr, nullptr, out, nullptr, status_word, scale, s->T,
                           s->H, s->HV, static_cast<int>(z.ns)};
  return kda::gdr::launch_step(p, state, slots, num_slots, s->K, s->V, s->io_dtype == KDA_BF16,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK
             : KDA_ERR_CUDA;
}

kda_status kda_layer_norm_fwd(int64_t rows, int D, kda_dtype io_dtype, const void* x, int64_t x_stride,
                              const float* weight, const float* bias, float eps, void* y, float* mean, float* rstd,
                              void* stream) {
  if (rows < 0 || rows > INT32_MAX || D < 1 || x_stride < D) return KDA_ERR_INVALID_ARG;
  if (io_dtype != KDA_F32 && io_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return KDA_ERR_INVALID_ARG;
  if (rows == 0) return KDA_OK;
  if (!x || !y) return KDA_ERR_INVALID_ARG;
  const size_t es = io_dtype == KDA_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return KDA_ERR_ALIGNMENT;
  const size_t n_x = (static_cast<size_t>(rows - 1) * x_stride + D) * es, n_y = static_cast<size_t>(rows) * D * es;
  const Span ins[] = {{x, n_x}, {weight, size_t(D) * 4}, {bias, size_t(D) * 4}};
  const Span outs[] = {{y, n_y}, {mean, size_t(rows) * 4}, {rstd, size_t(rows) * 4}};
  for (int i = 0; i < 3; ++i) {
    for (const Span& j : ins)
      if (overlaps(outs[i], j)) return KDA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
  }
  return kda::ln::launch_fwd(x, x_stride, weight, bias, eps, y, mean, rstd, rows, D, io_dtype == KDA_BF16,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK
             : KDA_ERR_CUDA;
}

size_t kda_layer_norm_bwd_workspace_size(int64_t rows, int D) {
  if (rows < 0 || rows > INT32_MAX || D < 1) return 0;
  return 256 + kda::ln::bwd_workspace_bytes(rows, D);
}

kda_status kda_layer_norm_bwd(int64_t rows, int D, kda_dtype io_dtype, const void* x, int64_t x_stride,
                              const void* dy, int64_t dy_stride, const float* weight, const float* mean,
                              const float* rstd, void* dx, float* dweight, float* dbias, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (rows < 0 || rows > INT32_MAX || D < 1 || x_stride < D || dy_stride < D) return KDA_ERR_INVALID_ARG;
  if (io_dtype != KDA_F32 && io_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !dy || !mean || !rstd)) return KDA_ERR_INVALID_ARG;
  if (!dx && !dweight && !dbias) return KDA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kda_layer_norm_bwd_workspace_size(rows, D)) return KDA_ERR_WORKSPACE;
  const size_t es = io_dtype == KDA_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(weight, 4) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(workspace, 16))
    return KDA_ERR_ALIGNMENT;
  const size_t r1 = rows > 0 ? static_cast<size_t>(rows - 1) : 0;
  const Span ins[] = {{x, (r1 * x_stride + D) * es}, {dy, (r1 * dy_stride + D) * es}, {weight, size_t(D) * 4},
                      {mean, size_t(rows) * 4},      {rstd, size_t(rows) * 4}};
  const Span outs[] = {{dx, static_cast<size_t>(rows) * D * es}, {dweight, size_t(D) * 4}, {dbias, size_t(D) * 4},
                       {workspace, workspace_bytes}};
  for (int i = 0; i < 4; ++i) {
    for (const Span& j : ins)
      if (overlaps(outs[i], j)) return KDA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
  }
  return kda::ln::launch_bwd(x, x_stride, dy, dy_stride, weight, mean, rstd, dx, dweight, dbias,
                             reinterpret_cast<float*>(workspace), rows, D, io_dtype == KDA_BF16,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK
             : KDA_ERR_CUDA;
}

}  // extern "C"
