// layer_norm.cu -- layer norm over the last dimension, forward and backward.
//
// Per row of D values:  y = (x - mu) r w + b,  mu = mean(x),  r = (mean((x - mu)^2) + eps)^{-1/2}.
// Backward, with xh = (x - mu) r and a = dy w:
//     dx = r (a - mean(a) - xh mean(a xh)),   dw = sum over rows of dy xh,   db = sum over rows of dy.
// Both passes are bound by HBM: 2 and 3 passes over the rows.  A row stays in the registers
// of its threads between the sums and the result, so it is read once.  The second moment is
// taken around the mean already known (no cancellation of large squares); all sums are fp32.
#include <cstddef>
#include <cstdint>

#include "kda_common.cuh"

namespace kda {
namespace ln {
namespace {

struct Params {
  const void* x;
  const void* dy;       // backward
  const float* w;       // [D] or null (ones)
  const float* b;       // [D] or null (zeros)
  void* y;              // forward: y; backward: dx
  float* mean;          // forward: written; backward: read
  float* rstd;
  float* pw;            // backward: [parts, D] partial dw, or null
  float* pb;            // backward: [parts, D] partial db, or null
  long rows;
  long ldx, lddy;       // elements from one row to the next
  int D;
  float eps;
};

template <typename IO, int VEC>
struct Vec {
  float v[VEC];
  __device__ __forceinline__ void load(const IO* p) {
    if constexpr (VEC == 1) {
      v[0] = to_f32(*p);
    } else if constexpr (sizeof(IO) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
      const float4 u = *reinterpret_cast<const float4*>(p);
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
  }
  __device__ __forceinline__ void store(IO* p) const {
    if constexpr (VEC == 1) {
      *p = from_f32<IO>(v[0]);
    } else if constexpr (sizeof(IO) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  // fp32 parameters at the same positions
  __device__ __forceinline__ void load_f32(const float* p) {
    if constexpr (VEC == 1) {
      v[0] = *p;
    } else {
#pragma unroll
      for (int j = 0; j < VEC / 4; ++j) {
        const float4 u = reinterpret_cast<const float4*>(p)[j];
        v[4 * j] = u.x; v[4 * j + 1] = u.y; v[4 * j + 2] = u.z; v[4 * j + 3] = u.w;
      }
    }
  }
};

// Sums of N values over the TPR threads of a row (TPR a multiple of 32; `red` holds one
// slot per warp and value, of this row's group).
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float* red, int t) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xFFFFFFFFu, x[i], m);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    if ((t & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * W + (t >> 5)] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[i * W + w];
      x[i] = s;
    }
    __syncthreads();
  }
}

// One row per TPR threads, NV vectors of VEC values a thread (vector j of thread t at
// column VEC (t + TPR j)).
template <typename IO, int VEC, int NV, int TPR, int NT>
__global__ void __launch_bounds__(NT) layer_norm_kernel(const Params p) {
  __shared__ float red[NT / 32];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const long row = static_cast<long>(blockIdx.x) * (NT / TPR) + grp;
  const bool live = row < p.rows;
  const IO* x = static_cast<const IO*>(p.x) + row * p.ldx;
  Vec<IO, VEC> a[NV];
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = VEC * (t + TPR * j);
    if (live && c < p.D) a[j].load(x + c);
    else
#pragma unroll
      for (int e = 0; e < VEC; ++e) a[j].v[e] = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[0] += a[j].v[e];
  }
  row_sum<TPR>(s, red + grp * (TPR / 32), t);
  const float mu = s[0] / p.D;
  s[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (VEC * (t + TPR * j) < p.D)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = a[j].v[e] - mu;
        s[0] = fmaf(d, d, s[0]);
      }
  }
  row_sum<TPR>(s, red + grp * (TPR / 32), t);
  const float r = 1.f / sqrtf(s[0] / p.D + p.eps);
  if (!live) return;
  if (t == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = r;
  }
  IO* y = static_cast<IO*>(p.y) + row * p.D;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = VEC * (t + TPR * j);
    if (c < p.D) {
      Vec<IO, VEC> w, b;
      if (p.w) w.load_f32(p.w + c);
      if (p.b) b.load_f32(p.b + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (a[j].v[e] - mu) * r;
        a[j].v[e] = fmaf(xh, p.w ? w.v[e] : 1.f, p.b ? b.v[e] : 0.f);
      }
      a[j].store(y + c);
    }
  }
}

// Rows wider than the register kernels hold: the block reads its row three times.
template <typename IO>
__global__ void __launch_bounds__(1024) layer_norm_wide_kernel(const Params p) {
  __shared__ float red[32];
  const IO* x = static_cast<const IO*>(p.x) + static_cast<long>(blockIdx.x) * p.ldx;
  IO* y = static_cast<IO*>(p.y) + static_cast<long>(blockIdx.x) * p.D;
  float s[1] = {0.f};
  for (int c = threadIdx.x; c < p.D; c += 1024) s[0] += to_f32(x[c]);
  row_sum<1024>(s, red, threadIdx.x);
  const float mu = s[0] / p.D;
  s[0] = 0.f;
  for (int c = threadIdx.x; c < p.D; c += 1024) {
    const float d = to_f32(x[c]) - mu;
    s[0] = fmaf(d, d, s[0]);
  }
  row_sum<1024>(s, red, threadIdx.x);
  const float r = 1.f / sqrtf(s[0] / p.D + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[blockIdx.x] = mu;
    if (p.rstd) p.rstd[blockIdx.x] = r;
  }
  for (int c = threadIdx.x; c < p.D; c += 1024)
    y[c] = from_f32<IO>(fmaf((to_f32(x[c]) - mu) * r, p.w ? p.w[c] : 1.f, p.b ? p.b[c] : 0.f));
}

// Backward: the block's rows are blockIdx.x * (NT / TPR) + group, then every gridDim.x *
// (NT / TPR) further; a thread meets the same columns in every row, so its share of dw and
// db stays in registers and is written once, as part (block, group) of [parts, D].
template <typename IO, int VEC, int NV, int TPR, int NT>
__global__ void __launch_bounds__(NT) layer_norm_bwd_kernel(const Params p) {
  __shared__ float red[2 * (NT / 32)];
  constexpr int G = NT / TPR;
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  float* rd = red + grp * (2 * TPR / 32);
  Vec<IO, VEC> dw[NV], db[NV], w[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = VEC * (t + TPR * j);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      dw[j].v[e] = db[j].v[e] = 0.f;
      w[j].v[e] = 1.f;
    }
    if (p.w && c < p.D) w[j].load_f32(p.w + c);
  }
  // every thread of the block makes the same number of steps (row_sum has block barriers)
  for (long base = static_cast<long>(blockIdx.x) * G; base < p.rows; base += static_cast<long>(gridDim.x) * G) {
    const long row = base + grp;
    const bool live = row < p.rows;
    const IO* x = static_cast<const IO*>(p.x) + row * p.ldx;
    const IO* dy = static_cast<const IO*>(p.dy) + row * p.lddy;
    const float mu = live ? p.mean[row] : 0.f, r = live ? p.rstd[row] : 0.f;
    Vec<IO, VEC> xh[NV], a[NV];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = VEC * (t + TPR * j);
      if (live && c < p.D) {
        xh[j].load(x + c);
        a[j].load(dy + c);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xh[j].v[e] = mu;
          a[j].v[e] = 0.f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float h = (xh[j].v[e] - mu) * r, d = a[j].v[e];
        dw[j].v[e] = fmaf(d, h, dw[j].v[e]);
        db[j].v[e] += d;
        xh[j].v[e] = h;
        a[j].v[e] = d * w[j].v[e];
        s[0] += a[j].v[e];
        s[1] = fmaf(a[j].v[e], h, s[1]);
      }
    row_sum<TPR>(s, rd, t);
    const float c0 = s[0] / p.D, c1 = s[1] / p.D;
    if (live && p.y) {
      IO* dx = static_cast<IO*>(p.y) + row * p.D;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = VEC * (t + TPR * j);
        if (c < p.D) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) a[j].v[e] = r * (a[j].v[e] - c0 - xh[j].v[e] * c1);
          a[j].store(dx + c);
        }
      }
    }
  }
  const size_t part = (static_cast<size_t>(blockIdx.x) * G + grp) * p.D;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = VEC * (t + TPR * j);
    if (c < p.D)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (p.pw) p.pw[part + c + e] = dw[j].v[e];
        if (p.pb) p.pb[part + c + e] = db[j].v[e];
      }
  }
}

// Rows wider than that: two sums, then dx; dw and db of a block's rows accumulate in its part.
template <typename IO>
__global__ void __launch_bounds__(1024) layer_norm_bwd_wide_kernel(const Params p) {
  __shared__ float red[64];
  bool first = true;
  for (long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const IO* x = static_cast<const IO*>(p.x) + row * p.ldx;
    const IO* dy = static_cast<const IO*>(p.dy) + row * p.lddy;
    IO* dx = static_cast<IO*>(p.y) + row * p.D;
    const float mu = p.mean[row], r = p.rstd[row];
    float s[2] = {0.f, 0.f};
    const size_t part = static_cast<size_t>(blockIdx.x) * p.D;
    for (int c = threadIdx.x; c < p.D; c += 1024) {
      const float h = (to_f32(x[c]) - mu) * r, d = to_f32(dy[c]), aw = d * (p.w ? p.w[c] : 1.f);
      s[0] += aw;
      s[1] = fmaf(aw, h, s[1]);
      if (p.pw) p.pw[part + c] = first ? d * h : fmaf(d, h, p.pw[part + c]);
      if (p.pb) p.pb[part + c] = first ? d : p.pb[part + c] + d;
    }
    first = false;
    row_sum<1024>(s, red, threadIdx.x);
    const float c0 = s[0] / p.D, c1 = s[1] / p.D;
    if (p.y)
      for (int c = threadIdx.x; c < p.D; c += 1024) {
        const float h = (to_f32(x[c]) - mu) * r, aw = to_f32(dy[c]) * (p.w ? p.w[c] : 1.f);
        dx[c] = from_f32<IO>(r * (aw - c0 - h * c1));
      }
  }
}

// The parts' sum, in their order: 32 columns x 8 shares of the parts a block.
__global__ void __launch_bounds__(256) layer_norm_parts_kernel(const float* pw, const float* pb, float* dw, float* db,
                                                               int parts, int D) {
  __shared__ float sh[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), share = threadIdx.x >> 5;
  const float* src = blockIdx.y == 0 ? pw : pb;
  float* dst = blockIdx.y == 0 ? dw : db;
  if (!dst) return;
  float s = 0.f;
  if (c < D)
    for (int i = share; i < parts; i += 8) s += src[static_cast<size_t>(i) * D + c];
  sh[share][threadIdx.x & 31] = s;
  __syncthreads();
  if (share == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sh[i][threadIdx.x];
    dst[c] = s;
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

constexpr int kMaxRegD = 16384;  // widest row the register kernels hold

// Threads of a row so that each holds at most 16 values.
int threads_per_row(int D) {
  int t = 32;
  while (t * 16 < D) t *= 2;
  return t;
}

// Blocks of the backward: two of 256 threads (or the equal in larger ones) an SM keep the
// rows streaming while the parts stay few.
constexpr int kMaxParts = 2048;

template <typename IO, int VEC, int TPR, bool BWD>
void launch_tpr(const Params& p, int grid, cudaStream_t st) {
  constexpr int NT = TPR < 256 ? 256 : TPR, NV = 16 / VEC;
  if constexpr (BWD)
    layer_norm_bwd_kernel<IO, VEC, NV, TPR, NT><<<grid, NT, 0, st>>>(p);
  else
    layer_norm_kernel<IO, VEC, NV, TPR, NT>
        <<<static_cast<unsigned>((p.rows + NT / TPR - 1) / (NT / TPR)), NT, 0, st>>>(p);
}

template <typename IO, int VEC, bool BWD>
void launch_vec(const Params& p, int grid, cudaStream_t st) {
  switch (threads_per_row(p.D)) {
    case 32: return launch_tpr<IO, VEC, 32, BWD>(p, grid, st);
    case 64: return launch_tpr<IO, VEC, 64, BWD>(p, grid, st);
    case 128: return launch_tpr<IO, VEC, 128, BWD>(p, grid, st);
    case 256: return launch_tpr<IO, VEC, 256, BWD>(p, grid, st);
    case 512: return launch_tpr<IO, VEC, 512, BWD>(p, grid, st);
    default: return launch_tpr<IO, VEC, 1024, BWD>(p, grid, st);
  }
}

template <typename IO, bool BWD>
void launch_io(const Params& p, int grid, cudaStream_t st) {
  constexpr int E = 16 / sizeof(IO);
  auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool vec = p.D % E == 0 && p.ldx % E == 0 && al(p.x) && al(p.y) && al(p.w) && al(p.b) &&
                   (!BWD || (p.lddy % E == 0 && al(p.dy)));
  if (p.D > kMaxRegD) {
    if constexpr (BWD)
      layer_norm_bwd_wide_kernel<IO><<<grid, 1024, 0, st>>>(p);
    else
      layer_norm_wide_kernel<IO><<<static_cast<unsigned>(p.rows), 1024, 0, st>>>(p);
  } else if (vec) {
    launch_vec<IO, E, BWD>(p, grid, st);
  } else {
    launch_vec<IO, 1, BWD>(p, grid, st);
  }
}

// Blocks of the backward and the parts of dw and db that they write.
void bwd_grid(long rows, int D, int sms, int& grid, int& parts) {
  const int tpr = D > kMaxRegD ? 1024 : threads_per_row(D);
  const int nt = tpr < 256 ? 256 : tpr, groups = nt / tpr;
  const long want = (rows + groups - 1) / groups, most = static_cast<long>(sms) * (nt <= 256 ? 4 : nt <= 512 ? 2 : 1);
  grid = static_cast<int>(want < most ? want : most);
  if (static_cast<long>(grid) * groups > kMaxParts) grid = kMaxParts / groups;
  parts = grid * groups;
}

}  // namespace

size_t bwd_workspace_bytes(long rows, int D) {
  int grid, parts;
  bwd_grid(rows, D, sm_count(), grid, parts);
  return 2 * static_cast<size_t>(parts) * D * sizeof(float);
}

cudaError_t launch_fwd(const void* x, long ldx, const float* w, const float* b, float eps, void* y, float* mean,
                       float* rstd, long rows, int D, bool bf16, cudaStream_t st) {
  Params p{x, nullptr, w, b, y, mean, rstd, nullptr, nullptr, rows, ldx, 0, D, eps};
  if (bf16) launch_io<__nv_bfloat16, false>(p, 0, st);
  else launch_io<float, false>(p, 0, st);
  return cudaGetLastError();
}

cudaError_t launch_bwd(const void* x, long ldx, const void* dy, long lddy, const float* w, const float* mean,
                       const float* rstd, void* dx, float* dw, float* db, float* ws, long rows, int D, bool bf16,
                       cudaStream_t st) {
  int grid, parts;
  bwd_grid(rows, D, sm_count(), grid, parts);
  float* pw = dw ? ws : nullptr;
  float* pb = db ? ws + static_cast<size_t>(parts) * D : nullptr;
  if (rows > 0) {
    Params p{x, dy, w, nullptr, dx, const_cast<float*>(mean), const_cast<float*>(rstd), pw, pb, rows, ldx, lddy, D, 0.f};
    if (bf16) launch_io<__nv_bfloat16, true>(p, grid, st);
    else launch_io<float, true>(p, grid, st);
  }
  if (dw || db)
    layer_norm_parts_kernel<<<dim3((D + 31) / 32, 2), 256, 0, st>>>(pw, pb, dw, db, rows > 0 ? parts : 0, D);
  return cudaGetLastError();
}

}  // namespace ln
}  // namespace kda
