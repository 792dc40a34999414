// layer_norm.cu -- layer norm over the last dimension, forward and backward.
//
// Per row of D values:  y = (x - mu) r w + b,  mu = mean(x),  r = (mean((x - mu)^2) + eps)^{-1/2}.
// Backward, with xh = (x - mu) r and a = dy w:
//     dx = r (a - mean(a) - xh mean(a xh)),   dw = sum over rows of dy xh,   db = sum over rows of dy.
// Both passes are bound by HBM: 2 and 3 passes over the rows.  A row stays in the registers
// of its threads between the sums and the result, so it is read once.  The second moment is
// taken around the mean already known (no cancellation of large squares); all sums are fp32.
// 16384 rows of 4096 bf16: forward 44 us (268 MB, 90 % of the copy bandwidth), backward 72 us
// (403 MB, 83 %: between two rows a block waits for its sums) and 6 for the sums over its
// blocks; calls among others take 46 and 80.
#include <cstddef>
#include <cstdint>

#include "kda_common.cuh"
#include "pairs.cuh"

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
  float* pw;            // backward: [blocks, D] partial dw, or null
  float* pb;            // backward: [blocks, D] partial db, or null
  long rows;
  long ldx, lddy;       // elements from one row to the next
  int D;
  float eps;
};

// VEC values of a row as they lie in memory (one 16-byte load, or one element), so that the
// next row's can be in flight in few registers.
template <typename IO, int VEC>
struct Raw {
  uint4 u;
  __device__ __forceinline__ void load(const IO* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void to(float (&v)[VEC]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(IO) == 2) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        v[j] = __uint_as_float(w[j]);
      }
    }
  }
  static __device__ __forceinline__ void store(IO* p, const float (&v)[VEC]) {
    if constexpr (sizeof(IO) == 2) {
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
};
template <typename IO>
struct Raw<IO, 1> {
  IO u;
  __device__ __forceinline__ void load(const IO* p) { u = *p; }
  __device__ __forceinline__ void zero() { u = from_f32<IO>(0.f); }
  __device__ __forceinline__ void to(float (&v)[1]) const { v[0] = to_f32(u); }
  static __device__ __forceinline__ void store(IO* p, const float (&v)[1]) { *p = from_f32<IO>(v[0]); }
};
// fp32 parameters at the same columns; `def` where there are none
template <int VEC>
__device__ __forceinline__ void load_param(float (&v)[VEC], const float* p, int c, int D, float def) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = def;
  if (!p || c >= D) return;
  if constexpr (VEC == 1) {
    v[0] = p[c];
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const float4 u = reinterpret_cast<const float4*>(p + c)[j];
      v[4 * j] = u.x; v[4 * j + 1] = u.y; v[4 * j + 2] = u.z; v[4 * j + 3] = u.w;
    }
  }
}

// Sums of N values over the TPR threads of a row (TPR a multiple of 32; `red`: one slot per
// warp and value of this row's group, another buffer from one call to the next, so that one
// barrier is enough).
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
  }
}

// 16 or 4 bytes to shared memory without passing through registers; the issuing thread alone
// reads them, so waiting for its own groups is all it needs.  Zeros where there is nothing to
// copy (nothing is read then).
template <typename T>
__device__ __forceinline__ void copy_async(T* dst, const void* src, bool there) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst)), bytes = there ? sizeof(T) : 0;
  if constexpr (sizeof(T) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// One row per TPR threads, NV vectors of VEC values a thread (vector j of thread t at
// column VEC (t + TPR j)).  A block walks over rows with its columns' weights in registers
// (read per row they were 4 times the row's own bytes from L2: 65 us for 16384 rows of 4096
// in bf16) and the rows to come on their way in a ring in shared memory of RING rows a group,
// each thread's own vectors or elements (RING = 0, for single bf16 elements, and 49 us a call for
// 46 with vectors too: the next row's in registers).
template <typename IO, int VEC, int NV, int TPR, int NT, int RING>
__global__ void __launch_bounds__(NT) layer_norm_kernel(const Params p) {
  constexpr int G = NT / TPR;
  using Slot = decltype(Raw<IO, VEC>::u);
  extern __shared__ __align__(16) uint4 dynamic[];
  Slot* ring = reinterpret_cast<Slot*>(dynamic);  // [RING][NV][NT]
  __shared__ float red[2][NT / 32];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  float* rd[2] = {red[0] + grp * (TPR / 32), red[1] + grp * (TPR / 32)};
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = VEC * (t + TPR * j);
    load_param<VEC>(w[j], p.w, c, p.D, 1.f);
    load_param<VEC>(b[j], p.b, c, p.D, 0.f);
  }
  Raw<IO, VEC> raw[NV];
  auto fetch = [&](long row, int slot) {
    const IO* x = static_cast<const IO*>(p.x) + row * p.ldx;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = VEC * (t + TPR * j);
      if constexpr (RING > 0) {
        const bool there = row < p.rows && c < p.D;
        copy_async(&ring[(slot * NV + j) * NT + threadIdx.x], there ? x + c : static_cast<const IO*>(p.x), there);
      } else if (row < p.rows && c < p.D) {
        raw[j].load(x + c);
      } else {
        raw[j].zero();
      }
    }
    if constexpr (RING > 0) copies_close();
  };
  const long step = static_cast<long>(gridDim.x) * G;
  long base = static_cast<long>(blockIdx.x) * G;
  int slot = 0;
  if constexpr (RING > 0) {
#pragma unroll
    for (int n = 0; n < RING; ++n) fetch(base + grp + n * step, n);
  } else {
    fetch(base + grp, 0);
  }
  for (; base < p.rows; base += step) {  // (the whole block: row_sum has block barriers)
    const long row = base + grp;
    float a[NV][VEC], s[1] = {0.f};
    if constexpr (RING > 0) copies_wait<RING - 1>();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (RING > 0) raw[j].u = ring[(slot * NV + j) * NT + threadIdx.x];
      raw[j].to(a[j]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += a[j][e];
    }
    fetch(row + (RING > 0 ? RING : 1) * step, slot);
    if (++slot >= RING) slot = 0;
    row_sum<TPR>(s, rd[0], t);
    const float mu = s[0] / p.D;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (VEC * (t + TPR * j) < p.D)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          a[j][e] -= mu;
          s[0] = fmaf(a[j][e], a[j][e], s[0]);
        }
    }
    row_sum<TPR>(s, rd[1], t);
    const float r = 1.f / sqrtf(s[0] / p.D + p.eps);
    if (row >= p.rows) continue;
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = r;
    }
    IO* y = static_cast<IO*>(p.y) + row * p.D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = VEC * (t + TPR * j);
      if (c < p.D) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[j][e] = fmaf(a[j][e] * r, w[j][e], b[j][e]);
        Raw<IO, VEC>::store(y + c, a[j]);
      }
    }
  }
  if constexpr (RING > 0) copies_wait<0>();   // (zeros, past the last row: they land before the block's memory goes)
}

// Rows wider than the register kernels hold: the block reads its row three times.
template <typename IO>
__global__ void __launch_bounds__(1024) layer_norm_wide_kernel(const Params p) {
  __shared__ float red[2][32];
  const IO* x = static_cast<const IO*>(p.x) + static_cast<long>(blockIdx.x) * p.ldx;
  IO* y = static_cast<IO*>(p.y) + static_cast<long>(blockIdx.x) * p.D;
  float s[1] = {0.f};
  for (int c = threadIdx.x; c < p.D; c += 1024) s[0] += to_f32(x[c]);
  row_sum<1024>(s, red[0], threadIdx.x);
  const float mu = s[0] / p.D;
  s[0] = 0.f;
  for (int c = threadIdx.x; c < p.D; c += 1024) {
    const float d = to_f32(x[c]) - mu;
    s[0] = fmaf(d, d, s[0]);
  }
  row_sum<1024>(s, red[1], threadIdx.x);
  const float r = 1.f / sqrtf(s[0] / p.D + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[blockIdx.x] = mu;
    if (p.rstd) p.rstd[blockIdx.x] = r;
  }
  for (int c = threadIdx.x; c < p.D; c += 1024)
    y[c] = from_f32<IO>(fmaf((to_f32(x[c]) - mu) * r, p.w ? p.w[c] : 1.f, p.b ? p.b[c] : 0.f));
}

// Backward: the block's rows are blockIdx.x G + group, then every gridDim.x G further; a
// thread meets the same columns in every row, so its share of dw and db stays in registers.
// The groups' shares are added in their order and written once, as the block's part of
// [blocks, D].  The ring is the forward's (with the next row's loads in registers alone 32 KB an
// SM were in flight, a call of 16384 rows of 4096 took 88 us, with the ring 84).  The arithmetic is in pairs of values (84 -> 82).
template <typename IO, int VEC, int NV, int TPR, int NT, int RING>
__global__ void __launch_bounds__(NT, NT == 256 ? 2 : 1) layer_norm_bwd_kernel(const Params p) {
  constexpr int G = NT / TPR;
  using Slot = decltype(Raw<IO, VEC>::u);
  extern __shared__ __align__(16) uint4 dynamic[];
  Slot* ring = reinterpret_cast<Slot*>(dynamic);  // [RING][2 NV][NT]
  __shared__ float red[2][2 * (NT / 32)];
  __shared__ float share[G > 1 ? TPR * 16 : 1];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  // a thread's 16 values in pairs: value n = VEC j + e is element e of vector j
  constexpr int NP = NV * VEC / 2;
  uint64_t dw[NP], db[NP], w[NP];
  {
    float v[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_param<VEC>(v[j], p.w, VEC * (t + TPR * j), p.D, 1.f);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      w[n] = pack2f(v[2 * n / VEC][2 * n % VEC], v[(2 * n + 1) / VEC][(2 * n + 1) % VEC]);
      dw[n] = db[n] = 0ull;
    }
  }
  Raw<IO, VEC> rx[NV], ry[NV];
  float mu, r;
  const long step = static_cast<long>(gridDim.x) * G;
  long base = static_cast<long>(blockIdx.x) * G;
  auto fetch = [&](long row, int slot) {
    const bool live = row < p.rows;
    const IO* x = static_cast<const IO*>(p.x) + row * p.ldx;
    const IO* dy = static_cast<const IO*>(p.dy) + row * p.lddy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = VEC * (t + TPR * j);
      if constexpr (RING > 0) {
        const bool there = live && c < p.D;
        copy_async(&ring[(slot * 2 * NV + 2 * j) * NT + threadIdx.x], there ? x + c : static_cast<const IO*>(p.x), there);
        copy_async(&ring[(slot * 2 * NV + 2 * j + 1) * NT + threadIdx.x], there ? dy + c : static_cast<const IO*>(p.dy), there);
      } else if (live && c < p.D) {
        rx[j].load(x + c);
        ry[j].load(dy + c);
      } else {
        rx[j].zero();
        ry[j].zero();
      }
    }
    if constexpr (RING > 0) copies_close();
  };
  auto stats = [&](long row) {
    mu = row < p.rows ? p.mean[row] : 0.f;
    r = row < p.rows ? p.rstd[row] : 0.f;
  };
  int buf = 0, slot = 0;
  if constexpr (RING > 0) {
#pragma unroll
    for (int n = 0; n < RING; ++n) fetch(base + grp + n * step, n);
  } else {
    fetch(base + grp, 0);
  }
  stats(base + grp);
  for (; base < p.rows; base += step) {
    const long row = base + grp;
    float vx[NV][VEC], vy[NV][VEC];
    const float rr = r;
    if constexpr (RING > 0) copies_wait<RING - 1>();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (RING > 0) {
        rx[j].u = ring[(slot * 2 * NV + 2 * j) * NT + threadIdx.x];
        ry[j].u = ring[(slot * 2 * NV + 2 * j + 1) * NT + threadIdx.x];
      }
      rx[j].to(vx[j]);
      ry[j].to(vy[j]);   // (0 past D, which keeps these columns out of every sum)
    }
    uint64_t xh[NP], a[NP], s0 = 0ull, s1 = 0ull;
    {
      const uint64_t mm = pack2f(-mu, -mu), r2 = pack2f(r, r);
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        const uint64_t x = pack2f(vx[2 * n / VEC][2 * n % VEC], vx[(2 * n + 1) / VEC][(2 * n + 1) % VEC]);
        const uint64_t d = pack2f(vy[2 * n / VEC][2 * n % VEC], vy[(2 * n + 1) / VEC][(2 * n + 1) % VEC]);
        xh[n] = mul2(add2(x, mm), r2);
        dw[n] = fma2(d, xh[n], dw[n]);
        db[n] = add2(db[n], d);
        a[n] = mul2(d, w[n]);
        s0 = add2(s0, a[n]);
        s1 = fma2(a[n], xh[n], s1);
      }
    }
    float s[2], half;
    unpack2f(s0, s[0], half);
    s[0] += half;
    unpack2f(s1, s[1], half);
    s[1] += half;
    fetch(row + (RING > 0 ? RING : 1) * step, slot);
    stats(row + step);
    if (++slot >= RING) slot = 0;
    row_sum<TPR>(s, red[buf] + grp * (2 * TPR / 32), t);
    buf ^= 1;
    const float c0 = s[0] / p.D, c1 = s[1] / p.D;
    if (row < p.rows && p.y) {
      IO* dx = static_cast<IO*>(p.y) + row * p.D;
      const uint64_t n0 = pack2f(-c0, -c0), n1 = pack2f(-c1, -c1), r2 = pack2f(rr, rr);
#pragma unroll
      for (int n = 0; n < NP; ++n)
        unpack2f(mul2(r2, fma2(xh[n], n1, add2(a[n], n0))), vx[2 * n / VEC][2 * n % VEC], vx[(2 * n + 1) / VEC][(2 * n + 1) % VEC]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = VEC * (t + TPR * j);
        if (c < p.D) Raw<IO, VEC>::store(dx + c, vx[j]);
      }
    }
  }
  auto write = [&](const uint64_t (&sums)[NP], float* part) {
    if (!part) return;
    float x[NV][VEC];
#pragma unroll
    for (int n = 0; n < NP; ++n) unpack2f(sums[n], x[2 * n / VEC][2 * n % VEC], x[(2 * n + 1) / VEC][(2 * n + 1) % VEC]);
    for (int g = 0; g < G; ++g) {
      if (grp == g) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = VEC * (t + TPR * j);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float sum = x[j][e];
            if (G > 1) {
              if (g > 0) sum += share[c + e];
              if (g < G - 1) share[c + e] = sum;
            }
            if (g == G - 1 && c + e < p.D) part[static_cast<size_t>(blockIdx.x) * p.D + c + e] = sum;
          }
        }
      }
      if (G > 1) __syncthreads();
    }
  };
  if constexpr (RING > 0) copies_wait<0>();   // (zeros, past the last row)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  write(dw, p.pw);
  write(db, p.pb);
}

// Rows wider than that: two sums, then dx; dw and db of a block's rows accumulate in its part.
template <typename IO>
__global__ void __launch_bounds__(1024) layer_norm_bwd_wide_kernel(const Params p) {
  __shared__ float red[2][64];
  bool first = true;
  int buf = 0;
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
    row_sum<1024>(s, red[buf], threadIdx.x);
    buf ^= 1;
    const float c0 = s[0] / p.D, c1 = s[1] / p.D;
    if (p.y)
      for (int c = threadIdx.x; c < p.D; c += 1024) {
        const float h = (to_f32(x[c]) - mu) * r, aw = to_f32(dy[c]) * (p.w ? p.w[c] : 1.f);
        dx[c] = from_f32<IO>(r * (aw - c0 - h * c1));
      }
  }
}

// The parts' sum, in a fixed order: 32 columns x 32 shares of the parts a block.
__global__ void __launch_bounds__(1024) layer_norm_parts_kernel(const float* pw, const float* pb, float* dw, float* db,
                                                                int parts, int D) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float* src = blockIdx.y == 0 ? pw : pb;
  float* dst = blockIdx.y == 0 ? dw : db;
  if (!dst) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the parts: this kernel starts under the one that writes them
  float s = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int i = share; i < parts; i += 32) s += src[static_cast<size_t>(i) * D + c];
  }
  sh[share][lane] = s;
  __syncthreads();
  s = sh[lane][share];  // column blockIdx.x 32 + share, share `lane` of the parts
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
  if (lane == 0 && blockIdx.x * 32 + share < D) dst[blockIdx.x * 32 + share] = s;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

// Widest row that the kernels of a row in registers take.  Up to 8192 columns they hold it (but for
// some 80 bytes a thread of single elements); above, a row takes 1024 threads, which leaves 64 registers
// each, and the backward spills 436 to 716 bytes a thread (the forward 72 at most).
constexpr int kMaxRegD = 16384;

// Threads of a row so that each holds at most 16 values.
int threads_per_row(int D) {
  int t = 32;
  while (t * 16 < D) t *= 2;
  return t;
}

template <typename IO, int VEC, int TPR, bool BWD>
cudaError_t launch_tpr(const Params& p, int grid, cudaStream_t st) {
  constexpr int NT = TPR < 256 ? 256 : TPR, NV = 16 / VEC;
  // the ring: as many rows, up to 4, as 192 KB an SM hold
  constexpr size_t row = (BWD ? 2 : 1) * static_cast<size_t>(NV) * NT * sizeof(Raw<IO, VEC>);
  constexpr size_t fit = 192 * 1024 / (row * (NT > 256 ? 1 : BWD ? 2 : 3));
  constexpr int RING = sizeof(Raw<IO, VEC>) == 2 ? 0 : fit < 4 ? fit : 4;
  constexpr size_t bytes = RING * row;
  void (*kernel)(Params);
  if constexpr (BWD) kernel = layer_norm_bwd_kernel<IO, VEC, NV, TPR, NT, RING>;
  else kernel = layer_norm_kernel<IO, VEC, NV, TPR, NT, RING>;
  if constexpr (bytes > 40 * 1024) {
    static bool raised[64] = {};       // (a race raises it twice, to the same value)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !raised[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) raised[dev] = true;
    }
  }
  kernel<<<grid, NT, bytes, st>>>(p);
  return cudaGetLastError();
}

template <typename IO, int VEC, bool BWD>
cudaError_t launch_vec(const Params& p, int grid, cudaStream_t st) {
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
cudaError_t launch_io(const Params& p, int grid, cudaStream_t st) {
  constexpr int E = 16 / sizeof(IO);
  auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool vec = p.D % E == 0 && p.ldx % E == 0 && al(p.x) && al(p.y) && al(p.w) && al(p.b) &&
                   (!BWD || (p.lddy % E == 0 && al(p.dy)));
  if (p.D > kMaxRegD) {
    if constexpr (BWD)
      layer_norm_bwd_wide_kernel<IO><<<grid, 1024, 0, st>>>(p);
    else
      layer_norm_wide_kernel<IO><<<static_cast<unsigned>(p.rows), 1024, 0, st>>>(p);
    return cudaGetLastError();
  }
  return vec ? launch_vec<IO, E, BWD>(p, grid, st) : launch_vec<IO, 1, BWD>(p, grid, st);
}

// Blocks for `rows` rows with at most `threads` threads an SM: 512 in the backward (each thread
// holds three rows' worth of values beside those in flight, and every block costs a part of dw
// and db), 768 in the forward.
int grid_for(long rows, int D, int threads) {
  const int tpr = D > kMaxRegD ? 1024 : threads_per_row(D);
  const int nt = tpr < 256 ? 256 : tpr, groups = nt / tpr;
  const long want = (rows + groups - 1) / groups, per = threads / nt, most = static_cast<long>(sm_count()) * (per < 1 ? 1 : per);
  return static_cast<int>(want < most ? want : most);
}
int bwd_grid(long rows, int D) { return grid_for(rows, D, 512); }

}  // namespace

size_t bwd_workspace_bytes(long rows, int D) {
  return 2 * static_cast<size_t>(bwd_grid(rows, D)) * D * sizeof(float);
}

cudaError_t launch_fwd(const void* x, long ldx, const float* w, const float* b, float eps, void* y, float* mean,
                       float* rstd, long rows, int D, bool bf16, cudaStream_t st) {
  Params p{x, nullptr, w, b, y, mean, rstd, nullptr, nullptr, rows, ldx, 0, D, eps};
  const int grid = grid_for(rows, D, 768);
  return bf16 ? launch_io<__nv_bfloat16, false>(p, grid, st) : launch_io<float, false>(p, grid, st);
}

cudaError_t launch_bwd(const void* x, long ldx, const void* dy, long lddy, const float* w, const float* mean,
                       const float* rstd, void* dx, float* dw, float* db, float* ws, long rows, int D, bool bf16,
                       cudaStream_t st) {
  const int grid = bwd_grid(rows, D);
  float* pw = dw ? ws : nullptr;
  float* pb = db ? ws + static_cast<size_t>(grid) * D : nullptr;
  if (rows > 0) {
    Params p{x, dy, w, nullptr, dx, const_cast<float*>(mean), const_cast<float*>(rstd), pw, pb, rows, ldx, lddy, D, 0.f};
    const cudaError_t e = bf16 ? launch_io<__nv_bfloat16, true>(p, grid, st) : launch_io<float, true>(p, grid, st);
    if (e != cudaSuccess) return e;
  }
  if (dw || db) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((D + 31) / 32, 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = rows > 0 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, layer_norm_parts_kernel, static_cast<const float*>(pw), static_cast<const float*>(pb),
                                             dw, db, rows > 0 ? grid : 0, D);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace ln
}  // namespace kda
