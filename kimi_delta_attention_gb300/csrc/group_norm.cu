// group_norm.cu -- group norm with an activation, channels last, forward and backward.
//
// Per sample and group of n = L C / groups values:  xh = (x - mu) r,  z = xh w + b,  y = act(z),
// r = (var + eps)^{-1/2}.  Backward, with dz = dy act'(z) and a = dz w:
//     dx = r (a - mean(a) - xh mean(a xh)),   dw = sum dz xh,   db = sum dz   (over samples and positions).
#include "layer_ops.cuh"

namespace kda {
namespace gn {
namespace {

__device__ __forceinline__ float silu(float z) { return z / (1.f + expf(-z)); }
// act'(z) of silu: s (1 + z (1 - s))
__device__ __forceinline__ float silu_slope(float z) {
  const float s = 1.f / (1.f + expf(-z));
  return s * (1.f + z * (1.f - s));
}

__device__ __forceinline__ float block_sum(float x) {
  __shared__ float red[32];
  for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) s += red[w];
  return s;
}

// One block per (sample, group).
template <typename IO, bool BWD>
__global__ void __launch_bounds__(256) group_norm_kernel(const Params p) {
  const long sample = blockIdx.x / p.groups;
  const int grp = blockIdx.x % p.groups, width = p.C / p.groups;
  const size_t base = static_cast<size_t>(sample) * p.L * p.C + static_cast<size_t>(grp) * width;
  const long n = p.L * width;
  const IO* x = static_cast<const IO*>(p.x) + base;
  IO* out = static_cast<IO*>(p.out) + base;
  auto at = [&](long i) { return static_cast<size_t>(i / width) * p.C + i % width; };
  auto weight = [&](long i) { return p.w ? p.w[grp * width + i % width] : 1.f; };
  auto bias = [&](long i) { return p.b ? p.b[grp * width + i % width] : 0.f; };
  if constexpr (!BWD) {
    float s = 0.f;
    for (long i = threadIdx.x; i < n; i += 256) s += to_f32(x[at(i)]);
    const float mu = block_sum(s) / n;
    s = 0.f;
    for (long i = threadIdx.x; i < n; i += 256) {
      const float d = to_f32(x[at(i)]) - mu;
      s = fmaf(d, d, s);
    }
    const float r = 1.f / sqrtf(block_sum(s) / n + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[blockIdx.x] = mu;
      if (p.rstd) p.rstd[blockIdx.x] = r;
    }
    for (long i = threadIdx.x; i < n; i += 256) {
      const float z = fmaf((to_f32(x[at(i)]) - mu) * r, weight(i), bias(i));
      out[at(i)] = from_f32<IO>(p.silu ? silu(z) : z);
    }
  } else {
    const IO* dy = static_cast<const IO*>(p.dy) + base;
    const float mu = p.mean[blockIdx.x], r = p.rstd[blockIdx.x];
    auto value = [&](long i, float& xh) {
      xh = (to_f32(x[at(i)]) - mu) * r;
      const float d = to_f32(dy[at(i)]);
      return (p.silu ? d * silu_slope(fmaf(xh, weight(i), bias(i))) : d) * weight(i);
    };
    float s0 = 0.f, s1 = 0.f, xh;
    for (long i = threadIdx.x; i < n; i += 256) {
      const float a = value(i, xh);
      s0 += a;
      s1 = fmaf(a, xh, s1);
    }
    s0 = block_sum(s0) / n;
    s1 = block_sum(s1) / n;
    for (long i = threadIdx.x; i < n; i += 256) {
      const float a = value(i, xh);
      out[at(i)] = from_f32<IO>(r * (a - s0 - xh * s1));
    }
  }
}

// dw and db: one block per channel, over the rows.
template <typename IO>
__global__ void __launch_bounds__(256) group_norm_weights_kernel(const Params p) {
  const int c = blockIdx.x, grp = c / (p.C / p.groups);
  const float w = p.w ? p.w[c] : 1.f, b = p.b ? p.b[c] : 0.f;
  float sw = 0.f, sb = 0.f;
  for (long row = threadIdx.x; row < p.N * p.L; row += 256) {
    const long st = row / p.L * p.groups + grp;
    const float xh = (to_f32(static_cast<const IO*>(p.x)[row * p.C + c]) - p.mean[st]) * p.rstd[st];
    float d = to_f32(static_cast<const IO*>(p.dy)[row * p.C + c]);
    if (p.silu) d *= silu_slope(fmaf(xh, w, b));
    sw = fmaf(d, xh, sw);
    sb += d;
  }
  sw = block_sum(sw);
  sb = block_sum(sb);
  if (threadIdx.x == 0) {
    if (p.dw) p.dw[c] = sw;
    if (p.db) p.db[c] = sb;
  }
}

}  // namespace

size_t fwd_workspace_bytes(long, long, int, int) { return 0; }
size_t bwd_workspace_bytes(long, long, int, int) { return 0; }

cudaError_t launch_fwd(const Params& p, bool bf16, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.N * p.groups);
  if (bf16) group_norm_kernel<__nv_bfloat16, false><<<grid, 256, 0, st>>>(p);
  else group_norm_kernel<float, false><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_bwd(const Params& p, bool bf16, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.N * p.groups);
  if (p.out && grid > 0) {
    if (bf16) group_norm_kernel<__nv_bfloat16, true><<<grid, 256, 0, st>>>(p);
    else group_norm_kernel<float, true><<<grid, 256, 0, st>>>(p);
  }
  if (p.dw || p.db) {
    if (bf16) group_norm_weights_kernel<__nv_bfloat16><<<p.C, 256, 0, st>>>(p);
    else group_norm_weights_kernel<float><<<p.C, 256, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace gn
}  // namespace kda
