// glr.cu -- gated linear recurrence, per channel:  h_t = e^{g_t} h_{t-1} + x_t,  y_t = h_t,
// and its gradients:  lam_t = dy_t + mu_{t+1},  mu_t = e^{g_t} lam_t,  dx_t = lam_t,
// dg_t = mu_t h_{t-1}  (mu behind the last token: d_final; d_initial: mu of the first).
#include "layer_ops.cuh"

namespace kda {
namespace glr {
namespace {

// One thread per (sequence, channel), token after token.
template <typename IO, typename G, bool BWD>
__global__ void __launch_bounds__(128) glr_kernel(const Params p) {
  const int c = blockIdx.x * 128 + threadIdx.x, seq = blockIdx.y;
  if (c >= p.D) return;
  long tok0 = static_cast<long>(seq) * p.T;
  int len = p.T;
  if (p.cu) {
    const int a = p.cu[seq], b = p.cu[seq + 1];
    tok0 = a;
    len = b - a;
    if (a < 0 || b < a || b > p.tokens || (seq == 0 && a != 0) || (seq == p.num_seqs - 1 && b != p.tokens)) {
      atomicOr(p.status, kStatusBounds);
      len = 0;
    }
  }
  const IO* x = static_cast<const IO*>(p.x);
  const G* g = static_cast<const G*>(p.g);
  IO* out = static_cast<IO*>(p.out);
  const size_t st = static_cast<size_t>(seq) * p.D + c;
  float h = p.init ? p.init[st] : 0.f;
  for (int i = 0; i < len; ++i) {
    const size_t t = tok0 + (BWD ? len - 1 - i : i), at = t * p.D + c;
    const float a = expf(to_f32(g[at]));
    if constexpr (BWD) {
      const float lam = to_f32(x[at]) + h;
      h = a * lam;
      const float before = i + 1 < len ? to_f32(static_cast<const IO*>(p.y)[at - p.D]) : p.h0 ? p.h0[st] : 0.f;
      out[at] = from_f32<IO>(lam);
      static_cast<G*>(p.dg)[at] = from_f32<G>(h * before);
    } else {
      h = fmaf(a, h, to_f32(x[at]));
      out[at] = from_f32<IO>(h);
    }
  }
  if (p.fin) p.fin[st] = h;
}

template <typename IO, typename G>
__global__ void __launch_bounds__(128) glr_step_kernel(const StepParams p) {
  const int c = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
  if (c >= p.D) return;
  const IO* x = static_cast<const IO*>(p.x);
  const G* g = static_cast<const G*>(p.g);
  IO* y = static_cast<IO*>(p.y);
  long slot = b;
  if (p.slots) {
    slot = p.slots[b];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot >= p.num_slots && p.status && threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
      for (int t = 0; t < p.T; ++t) y[(static_cast<size_t>(b) * p.T + t) * p.D + c] = from_f32<IO>(0.f);
      return;
    }
  }
  float h = p.state[slot * p.D + c];
  for (int t = 0; t < p.T; ++t) {
    const size_t at = (static_cast<size_t>(b) * p.T + t) * p.D + c;
    h = fmaf(expf(to_f32(g[at])), h, to_f32(x[at]));
    y[at] = from_f32<IO>(h);
  }
  p.state[slot * p.D + c] = h;
}

template <typename IO, typename G>
cudaError_t launch_types(const Params& p, bool backward, cudaStream_t st) {
  const dim3 grid((p.D + 127) / 128, p.num_seqs);
  if (backward) glr_kernel<IO, G, true><<<grid, 128, 0, st>>>(p);
  else glr_kernel<IO, G, false><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename IO, typename G>
cudaError_t launch_step_types(const StepParams& p, cudaStream_t st) {
  glr_step_kernel<IO, G><<<dim3((p.D + 127) / 128, p.B), 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t workspace_bytes(long, int, bool, int) { return 0; }

cudaError_t launch(const Params& p, bool backward, bool bf16, bool gate_bf16, cudaStream_t st) {
  const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st);
  if (e != cudaSuccess) return e;
  if (bf16) return gate_bf16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(p, backward, st) : launch_types<__nv_bfloat16, float>(p, backward, st);
  return gate_bf16 ? launch_types<float, __nv_bfloat16>(p, backward, st) : launch_types<float, float>(p, backward, st);
}

cudaError_t launch_step(const StepParams& p, bool bf16, bool gate_bf16, cudaStream_t st) {
  if (bf16) return gate_bf16 ? launch_step_types<__nv_bfloat16, __nv_bfloat16>(p, st) : launch_step_types<__nv_bfloat16, float>(p, st);
  return gate_bf16 ? launch_step_types<float, __nv_bfloat16>(p, st) : launch_step_types<float, float>(p, st);
}

}  // namespace glr
}  // namespace kda
