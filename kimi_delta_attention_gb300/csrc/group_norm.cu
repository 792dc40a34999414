// group_norm.cu -- group norm with an activation, channels last, forward and backward.
//
// Per sample and group of n = L C / groups values:  xh = (x - mu) r,  z = xh w + b,  y = act(z),
// r = (var + eps)^{-1/2}.  Backward, with dz = dy act'(z) and a = dz w:
//     dx = r (a - mean(a) - xh mean(a xh)),   dw = sum dz xh,   db = sum dz   (over samples and positions).
// Bound by HBM: 2 passes over the values forward, 3 backward.  Three ways, by the group's shape:
//   rows   L = 1 and a group of 1 to 128 vectors of 16 bytes, a power of two (heads): the group lies in
//          the registers of a few neighbouring lanes, is read once, and its sums are shuffles.
//   warps  other groups of at most 2048 values: up to 512 in the registers of 1 to 32 lanes, more by a warp each that
//          reads its group again from L1.
//   chunks larger groups: blocks sum up chunks of a sample's positions, then blocks finish the sums and
//          write; the second reading comes from L2 where that holds the samples (it begins with
//          the chunks that were read last).
// Measured (bf16): 16384 rows of 32 heads of 128 with SiLU 55 us (268 MB, 73 % of the copy rate; loads are what its
// warps wait for most, and 19 instructions a value use 62 % of the issue slots), backward 93 (403 MB, 64 %;
// latency of the rows' sums at 24 warps an SM, and 7 for the parts' sum); 4 samples of 4096 x 4096 74 (268 MB and a
// second reading of 134), backward 134.
// Statistics and sums are fp32; deviations are taken around a value of the group's own (no
// cancellation of large squares), and every sum is taken in a fixed order.
#include "layer_ops.cuh"
#include "pairs.cuh"

namespace kda {
namespace gn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }
// act'(z) of silu: s (1 + z (1 - s))
__device__ __forceinline__ float silu_slope(float z) {
  const float s = __fdividef(1.f, 1.f + __expf(-z));
  return s * fmaf(z, 1.f - s, 1.f);
}

// Two values at once: 1 / (1 + e^-z), with e^-z as 2^(-z log2 e) and the hardware's reciprocal (0 for an infinite one)
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z) {
  float a, b;
  unpack2f(mul2(z, pack2f(-1.44269504f, -1.44269504f)), a, b);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(a));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(b));
  unpack2f(add2(pack2f(a, b), pack2f(1.f, 1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(a));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(b));
  return pack2f(a, b);
}
__device__ __forceinline__ uint64_t slope2(uint64_t z) {
  const uint64_t s = sigmoid2(z), one = pack2f(1.f, 1.f);
  return mul2(s, fma2(z, fma2(s, pack2f(-1.f, -1.f), one), one));
}
__device__ __forceinline__ float both(uint64_t v) {
  float a, b;
  unpack2f(v, a, b);
  return a + b;
}

// VEC values: a load of 16 bytes, or one element
template <typename IO, int VEC>
struct Raw {
  uint4 u;
  __device__ __forceinline__ void load(const IO* p) { u = *reinterpret_cast<const uint4*>(p); }
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
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(IO) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[j] = __float_as_uint(v[j]);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <typename IO>
struct Raw<IO, 1> {
  IO u;
  __device__ __forceinline__ void load(const IO* p) { u = *p; }
  __device__ __forceinline__ void to(float (&v)[1]) const { v[0] = to_f32(u); }
  static __device__ __forceinline__ void store(IO* p, const float (&v)[1]) { *p = from_f32<IO>(v[0]); }
};
template <int VEC>
__device__ __forceinline__ void load_param(float (&v)[VEC], const float* p, int c, float def) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = p ? p[c + e] : def;
}

// In pairs (a single value's partner is 0).
template <int VEC>
__device__ __forceinline__ void pack(const float (&f)[VEC], uint64_t (&v)[(VEC + 1) / 2]) {
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) v[i] = pack2f(f[2 * i], VEC > 1 ? f[(2 * i + 1) % VEC] : 0.f);
}
template <int VEC>
__device__ __forceinline__ void unpack(const uint64_t (&v)[(VEC + 1) / 2], float (&f)[VEC]) {
  float none;
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) {
    if constexpr (VEC > 1) unpack2f(v[i], f[2 * i], f[2 * i + 1]);
    else unpack2f(v[i], f[0], none);
  }
}
template <typename IO, int VEC>
__device__ __forceinline__ void to_pairs(const Raw<IO, VEC>& raw, uint64_t (&v)[(VEC + 1) / 2]) {
  float f[VEC];
  raw.to(f);
  pack<VEC>(f, v);
}

__device__ __forceinline__ float dz_of(float dy, float z, bool act) { return act ? dy * silu_slope(z) : dy; }

// The sums of n values with deviations from `shift`: their mean and the sum of squares around it.
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments join(const Moments& a, const Moments& b) {
  const float n = a.n + b.n;
  if (n == 0.f) return a;
  const float d = b.mean - a.mean, f = __fdividef(b.n, n);
  return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}
__device__ __forceinline__ Moments warp_join(Moments m) {
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    const Moments o{__shfl_down_sync(0xFFFFFFFFu, m.n, s), __shfl_down_sync(0xFFFFFFFFu, m.mean, s),
                    __shfl_down_sync(0xFFFFFFFFu, m.m2, s)};
    m = join(m, o);
  }
  return {__shfl_sync(0xFFFFFFFFu, m.n, 0), __shfl_sync(0xFFFFFFFFu, m.mean, 0), __shfl_sync(0xFFFFFFFFu, m.m2, 0)};
}
__device__ __forceinline__ float2 warp_sum(float2 v) {
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, s);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, s);
  }
  return v;
}

// -------------------------------------------------------------------- rows --
// Threads of a block over the groups of a row, TPU a group, NV vectors each (vector j of thread t at
// (t + TPU j) VEC of its group): several rows a block where there are few groups, else blocks side by
// side (blockIdx.x).  A block walks over rows with its columns' weights in registers.
struct RowLayout {
  int groups_each;   // groups of a row that a block takes
  int rows_each;     // rows of a block at once
};
__host__ __device__ inline RowLayout row_layout(int groups, int tpu) {
  const int all = kThreads / tpu;
  return groups >= all ? RowLayout{all, 1} : RowLayout{groups, all / groups};
}

template <int NV, int VEC, int TPU>
__device__ __forceinline__ void load_pairs(uint64_t (&v)[NV][VEC / 2], const float* p, int c0, float def) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[VEC];
    load_param<VEC>(f, p, c0 + TPU * VEC * j, def);
    pack<VEC>(f, v[j]);
  }
}

// Values go two at a time (16384 x 4096 62.7 -> 56 us).
template <typename IO, int VEC, int NV, int TPU, bool ACT>
__global__ void __launch_bounds__(kThreads) group_rows_kernel(const Params p) {
  constexpr int W = TPU * NV * VEC;              // values of a group
  const RowLayout lay = row_layout(p.groups, TPU);
  const int unit = threadIdx.x / TPU, t = threadIdx.x % TPU;
  const int grp = blockIdx.x * lay.groups_each + unit % lay.groups_each;
  const bool on = unit < lay.groups_each * lay.rows_each && grp < p.groups;
  const int c0 = grp * W + t * VEC;
  constexpr int NP = VEC / 2;                    // arithmetic on pairs of values
  uint64_t w[NV][NP], b[NV][NP];
  load_pairs<NV, VEC, TPU>(w, on ? p.w : nullptr, c0, 1.f);
  load_pairs<NV, VEC, TPU>(b, on ? p.b : nullptr, c0, 0.f);
  const long step = static_cast<long>(gridDim.y) * lay.rows_each;
  long row = static_cast<long>(blockIdx.y) * lay.rows_each + unit / lay.groups_each;
  Raw<IO, VEC> next[NV];
  auto fetch = [&](long r) {
    const IO* x = static_cast<const IO*>(p.x) + r * p.C + c0;
    if (on && r < p.N)
#pragma unroll
      for (int j = 0; j < NV; ++j) next[j].load(x + TPU * VEC * j);
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) next[j].u = {};
  fetch(row);
  // (a warp's lanes go on together: its groups may be of two rows)
  for (; __any_sync(0xFFFFFFFFu, on && row < p.N); row += step) {
    uint64_t v[NV][NP], s2 = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      to_pairs(next[j], v[j]);
#pragma unroll
      for (int i = 0; i < NP; ++i) s2 = add2(s2, v[j][i]);
    }
    fetch(row + step);
    float s = both(s2);
#pragma unroll
    for (int m = TPU / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
    const float mu = s * (1.f / W);
    s2 = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        v[j][i] = add2(v[j][i], pack2f(-mu, -mu));
        s2 = fma2(v[j][i], v[j][i], s2);
      }
    s = both(s2);
#pragma unroll
    for (int m = TPU / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
    const float r = rsqrtf(fmaf(s, 1.f / W, p.eps));
    if (!on || row >= p.N) continue;
    if (t == 0) {
      if (p.mean) p.mean[row * p.groups + grp] = mu;
      if (p.rstd) p.rstd[row * p.groups + grp] = r;
    }
    IO* y = static_cast<IO*>(p.out) + row * p.C + c0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float out[VEC];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint64_t z = fma2(mul2(v[j][i], pack2f(r, r)), w[j][i], b[j][i]);
        if (ACT) z = mul2(z, sigmoid2(z));
        unpack2f(z, out[2 * i], out[2 * i + 1]);
      }
      Raw<IO, VEC>::store(y + TPU * VEC * j, out);
    }
  }
}

// Backward: a thread meets the same columns in every row, so its shares of dw and db stay in registers; the
// block's rows' shares are added in their order and written as the block's part of [blocks, C].
template <typename IO, int VEC, int NV, int TPU, bool ACT>
__global__ void __launch_bounds__(kThreads, NV > 2 ? 1 : NV == 2 ? 2 : 3) group_rows_bwd_kernel(const Params p, float* pw, float* pb) {
  constexpr int W = TPU * NV * VEC;
  extern __shared__ float share[];               // [rows_each][groups_each W] where there are several rows
  const RowLayout lay = row_layout(p.groups, TPU);
  const int unit = threadIdx.x / TPU, t = threadIdx.x % TPU, line = unit / lay.groups_each;
  const int grp = blockIdx.x * lay.groups_each + unit % lay.groups_each;
  const bool on = unit < lay.groups_each * lay.rows_each && grp < p.groups;
  const int c0 = grp * W + t * VEC;
  constexpr int NP = VEC / 2;                    // arithmetic on pairs of values
  uint64_t w[NV][NP], b[NV][NP], dw[NV][NP], db[NV][NP];
  load_pairs<NV, VEC, TPU>(w, on ? p.w : nullptr, c0, 1.f);
  load_pairs<NV, VEC, TPU>(b, on ? p.b : nullptr, c0, 0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < NP; ++i) dw[j][i] = db[j][i] = 0ull;
  const long step = static_cast<long>(gridDim.y) * lay.rows_each;
  long row = static_cast<long>(blockIdx.y) * lay.rows_each + line;
  Raw<IO, VEC> nx[NV], ny[NV];
  float nmu = 0.f, nr = 0.f;
  auto fetch = [&](long r) {
    const size_t at = r * p.C + c0;
    if (on && r < p.N) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        nx[j].load(static_cast<const IO*>(p.x) + at + TPU * VEC * j);
        ny[j].load(static_cast<const IO*>(p.dy) + at + TPU * VEC * j);
      }
      nmu = p.mean[r * p.groups + grp];
      nr = p.rstd[r * p.groups + grp];
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) nx[j].u = ny[j].u = {};
  fetch(row);
  for (; __any_sync(0xFFFFFFFFu, on && row < p.N); row += step) {
    const bool live = on && row < p.N;
    uint64_t xh[NV][NP], a[NV][NP], s0 = 0ull, s1 = 0ull;
    const float mu = nmu, r = live ? nr : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      to_pairs(nx[j], xh[j]);
      to_pairs(ny[j], a[j]);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        xh[j][i] = mul2(add2(xh[j][i], pack2f(-mu, -mu)), pack2f(r, r));
        if (ACT) a[j][i] = mul2(a[j][i], slope2(fma2(xh[j][i], w[j][i], b[j][i])));
        if (live) {
          dw[j][i] = fma2(a[j][i], xh[j][i], dw[j][i]);
          db[j][i] = add2(db[j][i], a[j][i]);
        }
        a[j][i] = mul2(a[j][i], w[j][i]);
        s0 = add2(s0, a[j][i]);
        s1 = fma2(a[j][i], xh[j][i], s1);
      }
    }
    fetch(row + step);
    float m0 = both(s0), m1 = both(s1);
#pragma unroll
    for (int m = TPU / 2; m >= 1; m >>= 1) {
      m0 += __shfl_xor_sync(0xFFFFFFFFu, m0, m);
      m1 += __shfl_xor_sync(0xFFFFFFFFu, m1, m);
    }
    if (!live || !p.out) continue;
    m0 *= -1.f / W;
    m1 *= -1.f / W;
    IO* dx = static_cast<IO*>(p.out) + row * p.C + c0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float out[VEC];
#pragma unroll
      for (int i = 0; i < NP; ++i)
        unpack2f(mul2(pack2f(r, r), fma2(xh[j][i], pack2f(m1, m1), add2(a[j][i], pack2f(m0, m0)))), out[2 * i], out[2 * i + 1]);
      Raw<IO, VEC>::store(dx + TPU * VEC * j, out);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto write = [&](const uint64_t (&sums)[NV][NP], float* part) {
    if (!part) return;
    float v[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < NP; ++i) unpack2f(sums[j][i], v[j][2 * i], v[j][2 * i + 1]);
    float* to = part + static_cast<size_t>(blockIdx.y) * p.C;
    if (lay.rows_each == 1) {
      if (on)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) to[c0 + TPU * VEC * j + e] = v[j][e];
      return;
    }
    const int width = lay.groups_each * W;       // (every group: one block over the columns)
    __syncthreads();
    if (on)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) share[line * width + c0 + TPU * VEC * j + e] = v[j][e];
    __syncthreads();
    for (int c = threadIdx.x; c < width; c += kThreads) {
      float s = 0.f;
      for (int k = 0; k < lay.rows_each; ++k) s += share[k * width + c];
      to[c] = s;
    }
  };
  write(dw, pw);
  write(db, pb);
}

// ------------------------------------------------------------------- small --
// Groups of at most OWN values a lane, LANES neighbouring lanes each: a group is read once and stays in
// registers.  (A warp for every group, as larger ones have: 5990 rows of 71 groups of 9 in bf16 164 us.)
// FLAT: L = 1, a group's values lie side by side.
constexpr int kMostSmall = 512;

template <typename IO, int LANES, int OWN, bool FLAT, bool BWD>
__global__ void __launch_bounds__(kThreads) group_small_kernel(const Params p) {
  const long unit = (static_cast<long>(blockIdx.x) * kThreads + threadIdx.x) / LANES;
  const bool on = unit < p.N * p.groups;         // (idle lanes go along: their neighbours' shuffles need them)
  const int t = threadIdx.x % LANES, width = p.C / p.groups, n = static_cast<int>(p.L) * width;
  const int grp = on ? static_cast<int>(unit % p.groups) : 0;
  const size_t base = on ? unit / p.groups * p.L * p.C + static_cast<size_t>(grp) * width : 0;
  const float* w = p.w ? p.w + grp * width : nullptr;
  const float* b = p.b ? p.b + grp * width : nullptr;
  // f(i, offset, channel) for the lane's values i: value t + LANES i of the group lies at position / width
  auto each = [&](auto f) {
    if constexpr (FLAT) {
#pragma unroll
      for (int i = 0; i < OWN; ++i)
        if (on && t + LANES * i < n) f(i, base + t + LANES * i, t + LANES * i);
    } else {
      int c = t % width;
      size_t at = base + static_cast<size_t>(t / width) * p.C + c;
      const int dl = LANES / width, dc = LANES % width;
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        if (on && t + LANES * i < n) f(i, at, c);
        at += static_cast<size_t>(dl) * p.C + dc;
        c += dc;
        if (c >= width) {
          c -= width;
          at += p.C - width;
        }
      }
    }
  };
  auto sum = [](float x) {
#pragma unroll
    for (int m = LANES / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
    return x;
  };
  const IO* x = static_cast<const IO*>(p.x);
  IO* out = static_cast<IO*>(p.out);
  float v[OWN];
#pragma unroll
  for (int i = 0; i < OWN; ++i) v[i] = 0.f;
  each([&](int i, size_t at, int) { v[i] = to_f32(x[at]); });
  const float inv = 1.f / n;
  if constexpr (!BWD) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < OWN; ++i) s += v[i];
    const float mu = sum(s) * inv;
    s = 0.f;
    each([&](int i, size_t, int) {
      v[i] -= mu;
      s = fmaf(v[i], v[i], s);
    });
    const float r = rsqrtf(fmaf(sum(s), inv, p.eps));
    if (on && t == 0) {
      if (p.mean) p.mean[unit] = mu;
      if (p.rstd) p.rstd[unit] = r;
    }
    each([&](int i, size_t at, int c) {
      const float z = fmaf(v[i] * r, w ? w[c] : 1.f, b ? b[c] : 0.f);
      out[at] = from_f32<IO>(p.silu ? silu(z) : z);
    });
  } else {
    const IO* dy = static_cast<const IO*>(p.dy);
    const float mu = on ? p.mean[unit] : 0.f, r = on ? p.rstd[unit] : 0.f;
    float a[OWN], s0 = 0.f, s1 = 0.f;
    each([&](int i, size_t at, int c) {
      const float wc = w ? w[c] : 1.f;
      v[i] = (v[i] - mu) * r;
      a[i] = dz_of(to_f32(dy[at]), fmaf(v[i], wc, b ? b[c] : 0.f), p.silu) * wc;
      s0 += a[i];
      s1 = fmaf(a[i], v[i], s1);
    });
    const float m0 = sum(s0) * inv, m1 = sum(s1) * inv;
    each([&](int i, size_t at, int) { out[at] = from_f32<IO>(r * (a[i] - m0 - v[i] * m1)); });
  }
}

template <typename IO, bool FLAT, bool BWD>
cudaError_t launch_small(const Params& p, cudaStream_t st) {
  const long n = p.L * (p.C / p.groups), units = p.N * p.groups;
  auto blocks = [&](int lanes) { return static_cast<unsigned>((units * lanes + kThreads - 1) / kThreads); };
  if (n <= 8) group_small_kernel<IO, 1, 8, FLAT, BWD><<<blocks(1), kThreads, 0, st>>>(p);
  else if (n <= 32) group_small_kernel<IO, 4, 8, FLAT, BWD><<<blocks(4), kThreads, 0, st>>>(p);
  else if (n <= 128) group_small_kernel<IO, 16, 8, FLAT, BWD><<<blocks(16), kThreads, 0, st>>>(p);
  else if (n <= 256) group_small_kernel<IO, 32, 8, FLAT, BWD><<<blocks(32), kThreads, 0, st>>>(p);
  else group_small_kernel<IO, 32, 16, FLAT, BWD><<<blocks(32), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename IO, bool BWD>
cudaError_t small_way(const Params& p, cudaStream_t st) {
  return p.L == 1 ? launch_small<IO, true, BWD>(p, st) : launch_small<IO, false, BWD>(p, st);
}

// ------------------------------------------------------------------- warps --
template <typename IO, bool BWD>
__global__ void __launch_bounds__(kThreads) group_warp_kernel(const Params p) {
  const long unit = static_cast<long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  if (unit >= p.N * p.groups) return;
  const int lane = threadIdx.x & 31, width = p.C / p.groups, n = static_cast<int>(p.L) * width;
  const int grp = static_cast<int>(unit % p.groups);
  const size_t base = unit / p.groups * p.L * p.C + static_cast<size_t>(grp) * width;
  const IO* x = static_cast<const IO*>(p.x) + base;
  IO* out = static_cast<IO*>(p.out) + base;
  const float* w = p.w ? p.w + grp * width : nullptr;
  const float* b = p.b ? p.b + grp * width : nullptr;
  // element i lies at position i / width and channel i % width; a lane's steps of 32 keep both
  auto each = [&](auto f) {
    int c = lane % width;
    size_t at = static_cast<size_t>(lane / width) * p.C + c;
    const int dl = 32 / width, dc = 32 % width;
    for (int i = lane; i < n; i += 32) {
      f(at, c);
      at += static_cast<size_t>(dl) * p.C + dc;
      c += dc;
      if (c >= width) {
        c -= width;
        at += p.C - width;
      }
    }
  };
  if constexpr (!BWD) {
    float s = 0.f;
    each([&](size_t at, int) { s += to_f32(x[at]); });
    const float mu = warp_sum({s, 0.f}).x / n;
    s = 0.f;
    each([&](size_t at, int) {
      const float d = to_f32(x[at]) - mu;
      s = fmaf(d, d, s);
    });
    const float r = 1.f / sqrtf(warp_sum({s, 0.f}).x / n + p.eps);
    if (lane == 0) {
      if (p.mean) p.mean[unit] = mu;
      if (p.rstd) p.rstd[unit] = r;
    }
    each([&](size_t at, int c) {
      const float z = fmaf((to_f32(x[at]) - mu) * r, w ? w[c] : 1.f, b ? b[c] : 0.f);
      out[at] = from_f32<IO>(p.silu ? silu(z) : z);
    });
  } else {
    const IO* dy = static_cast<const IO*>(p.dy) + base;
    const float mu = p.mean[unit], r = p.rstd[unit];
    auto value = [&](size_t at, int c, float& xh) {
      const float wc = w ? w[c] : 1.f;
      xh = (to_f32(x[at]) - mu) * r;
      return dz_of(to_f32(dy[at]), fmaf(xh, wc, b ? b[c] : 0.f), p.silu) * wc;
    };
    float2 s{0.f, 0.f};
    each([&](size_t at, int c) {
      float xh;
      const float a = value(at, c, xh);
      s.x += a;
      s.y = fmaf(a, xh, s.y);
    });
    s = warp_sum(s);
    const float m0 = s.x / n, m1 = s.y / n;
    each([&](size_t at, int c) {
      float xh;
      const float a = value(at, c, xh);
      out[at] = from_f32<IO>(r * (a - m0 - xh * m1));
    });
  }
}

// dw and db of these: 32 columns and a share of the rows a block, 8 rows at once; parts as above.
template <typename IO>
__global__ void __launch_bounds__(kThreads) group_weights_kernel(const Params p, long rows_each, float* pw, float* pb) {
  __shared__ float sh[2][kThreads / 32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const long rows = p.N * p.L, from = blockIdx.y * rows_each, to = from + rows_each < rows ? from + rows_each : rows;
  float sw = 0.f, sb = 0.f;
  if (c < p.C) {
    const int grp = c / (p.C / p.groups);
    const float w = p.w ? p.w[c] : 1.f, b = p.b ? p.b[c] : 0.f;
#pragma unroll 4
    for (long row = from + warp; row < to; row += kThreads / 32) {
      const long st = (p.L == 1 ? row : row / p.L) * p.groups + grp;
      const float xh = (to_f32(static_cast<const IO*>(p.x)[row * p.C + c]) - p.mean[st]) * p.rstd[st];
      const float dz = dz_of(to_f32(static_cast<const IO*>(p.dy)[row * p.C + c]), fmaf(xh, w, b), p.silu);
      sw = fmaf(dz, xh, sw);
      sb += dz;
    }
  }
  sh[0][warp][lane] = sw;
  sh[1][warp][lane] = sb;
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp < 2 && c < p.C) {
    float s = 0.f;
    for (int k = 0; k < kThreads / 32; ++k) s += sh[warp][k][lane];
    float* part = warp == 0 ? pw : pb;
    if (part) part[static_cast<size_t>(blockIdx.y) * p.C + c] = s;
  }
}

// ------------------------------------------------------------------ chunks --
// A block takes some whole groups' columns of some of a sample's positions: `across` threads over the
// column vectors and `down` over the positions; a group wider than the block's threads is walked over.
struct ChunkLayout {
  int groups_each, blocks;       // groups of a block; blocks over the channels
  int vectors, across, down;     // of a block's columns; its threads
  int chunks;                    // of a sample's positions
  long rows_each;                // positions of a chunk
};

ChunkLayout chunk_layout(long N, long L, int C, int groups, int vec, int sms) {
  ChunkLayout l;
  const int width = C / groups / vec;            // a group's vectors
  l.groups_each = width >= kThreads ? 1 : kThreads / width < groups ? kThreads / width : groups;
  l.blocks = (groups + l.groups_each - 1) / l.groups_each;
  l.vectors = l.groups_each * width;
  l.across = l.vectors < kThreads ? l.vectors : kThreads;
  l.down = kThreads / l.across;
  // 3 blocks an SM, all of which run at once (4 samples of 4096 x 4096 in 2, 3, 4, 6, 8 and 16: 83, 76, 76, 89, 90, 118
  // us forward, 155, 134, 167, 149, 163, 186 backward), each with several positions a thread
  long want = (3l * sms + N * l.blocks - 1) / (N * l.blocks);
  const long most = (L + 4l * l.down - 1) / (4l * l.down);
  want = want < 1 ? 1 : want > most ? most : want;
  l.rows_each = (L + want - 1) / want;
  l.chunks = static_cast<int>((L + l.rows_each - 1) / l.rows_each);
  return l;
}

struct ChunkArgs {
  Params p;
  ChunkLayout l;
  float2* sums;                  // [N][groups][chunks]: mean and squares around it, or the sums of a and a xh
  float* pw;                     // backward: [N chunks][C] parts of dw and db, or null
  float* pb;
  int first = 0;                 // blocks over the channels in the launches before this one
};

// What a block of either pass works on.
struct Work {
  int tc, tr, g0, chunk;         // its thread's place, its first group
  long sample, r0, r1;           // positions [r0, r1)
  __device__ __forceinline__ Work(const ChunkArgs& a, unsigned block)
      : tc(threadIdx.x % a.l.across), tr(threadIdx.x / a.l.across), g0((a.first + static_cast<int>(blockIdx.y)) * a.l.groups_each),
        chunk(block % a.l.chunks), sample(block / a.l.chunks), r0(chunk * a.l.rows_each), r1(r0 + a.l.rows_each < a.p.L ? r0 + a.l.rows_each : a.p.L) {}
  // how many of the positions r0 + tr, + down, ... are below r1
  __device__ __forceinline__ int rows(int down) const { return r0 + tr < r1 ? static_cast<int>((r1 - r0 - tr - 1) / down) + 1 : 0; }
};

// f(row) for n rows from the loads of `at`, `stride` values from one to the next; U loads at once.
template <int U, typename IO, int VEC, typename F>
__device__ __forceinline__ void walk(const IO* at, long stride, int n, F f) {
  for (; n >= U; n -= U) {
    Raw<IO, VEC> raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i].load(at + i * stride);
#pragma unroll
    for (int i = 0; i < U; ++i) f(raw[i]);
    at += U * stride;
  }
  for (; n > 0; --n, at += stride) {
    Raw<IO, VEC> raw;
    raw.load(at);
    f(raw);
  }
}
// The same over x and dy side by side, with the values' offset.
template <int U, typename IO, int VEC, typename F>
__device__ __forceinline__ void walk2(const IO* x, const IO* dy, size_t at, long stride, int n, F f) {
  for (; n >= U; n -= U) {
    Raw<IO, VEC> rx[U], ry[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      rx[i].load(x + at + i * stride);
      ry[i].load(dy + at + i * stride);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) f(rx[i], ry[i], at + i * stride);
    at += U * stride;
  }
  for (; n > 0; --n, at += stride) {
    Raw<IO, VEC> rx, ry;
    rx.load(x + at);
    ry.load(dy + at);
    f(rx, ry, at);
  }
}

// The group k of a block over its threads' shares, a warp a group: `of` entries of thread numbers.
struct Shares {
  int each, of;                  // a group's threads along the columns, and in all
  __device__ __forceinline__ Shares(const ChunkLayout& l, int width) : each(width < l.across ? width : l.across), of(each * l.down) {}
  __device__ __forceinline__ int thread(const ChunkLayout& l, int k, int i) const { return i / each * l.across + k * each + i % each; }
};

template <typename IO, int VEC>
__global__ void __launch_bounds__(kThreads, 4) group_moments_kernel(const ChunkArgs a) {
  constexpr int NP = (VEC + 1) / 2;
  __shared__ Moments sh[kThreads];
  const Params& p = a.p;
  const ChunkLayout& l = a.l;
  const Work k(a, blockIdx.x);
  const int width = p.C / p.groups / VEC, n = k.rows(l.down);
  const IO* base = static_cast<const IO*>(p.x) + (static_cast<size_t>(k.sample) * p.L + k.r0 + k.tr) * p.C;
  Moments mine{0.f, 0.f, 0.f};
  for (int v = k.tc; v < l.vectors && k.tr < l.down && n > 0; v += l.across) {
    if (k.g0 + v / width >= p.groups) break;
    const IO* x = base + (static_cast<size_t>(k.g0) * width + v) * VEC;
    uint64_t shift[NP], s1[NP], s2[NP];          // deviations from the thread's first value of the column
    {
      Raw<IO, VEC> first;
      first.load(x);
      to_pairs(first, shift);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        shift[i] ^= 0x8000000080000000ull;
        s1[i] = s2[i] = 0ull;
      }
    }
    walk<4, IO, VEC>(x, static_cast<long>(l.down) * p.C, n, [&](const Raw<IO, VEC>& raw) {
      uint64_t f[NP];
      to_pairs(raw, f);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        f[i] = add2(f[i], shift[i]);
        s1[i] = add2(s1[i], f[i]);
        s2[i] = fma2(f[i], f[i], s2[i]);
      }
    });
    float f0[VEC], f1[VEC], f2[VEC];
    unpack<VEC>(shift, f0);
    unpack<VEC>(s1, f1);
    unpack<VEC>(s2, f2);
    const float inv = 1.f / n;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float m = f1[e] * inv, m2 = fmaf(-m, f1[e], f2[e]);
      mine = join(mine, {static_cast<float>(n), m - f0[e], m2 < 0.f ? 0.f : m2});
    }
  }
  sh[threadIdx.x] = mine;
  __syncthreads();
  const Shares of(l, width);
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < l.groups_each && k.g0 + g < p.groups; g += kThreads / 32) {
    Moments m{0.f, 0.f, 0.f};
    for (int i = lane; i < of.of; i += 32) m = join(m, sh[of.thread(l, g, i)]);
    m = warp_join(m);
    if (lane == 0) a.sums[(k.sample * p.groups + k.g0 + g) * l.chunks + k.chunk] = make_float2(m.mean, m.m2);
  }
}

template <typename IO, int VEC>
__global__ void __launch_bounds__(kThreads, 3) group_sums_kernel(const ChunkArgs a) {
  constexpr int NP = (VEC + 1) / 2;
  __shared__ float2 sh[kThreads];
  __shared__ float cols[2][kThreads * VEC];
  const Params& p = a.p;
  const ChunkLayout& l = a.l;
  const Work k(a, blockIdx.x);
  const int width = p.C / p.groups / VEC;
  const size_t base = static_cast<size_t>(k.sample) * p.L * p.C;
  const size_t part = (static_cast<size_t>(k.sample) * l.chunks + k.chunk) * p.C;
  float2 s{0.f, 0.f};
  for (int v = k.tc; v < l.vectors && k.tr < l.down; v += l.across) {
    const int grp = k.g0 + v / width, c = (k.g0 * width + v) * VEC;
    if (grp >= p.groups) break;
    const float mu = p.mean[k.sample * p.groups + grp], r = p.rstd[k.sample * p.groups + grp];
    float w[VEC], b[VEC], dw[VEC], db[VEC];
    load_param<VEC>(w, p.w, c, 1.f);
    load_param<VEC>(b, p.b, c, 0.f);
    uint64_t w2[NP], b2[NP], sw[NP], sb[NP];
    pack<VEC>(w, w2);
    pack<VEC>(b, b2);
#pragma unroll
    for (int i = 0; i < NP; ++i) sw[i] = sb[i] = 0ull;
    walk2<2, IO, VEC>(static_cast<const IO*>(p.x), static_cast<const IO*>(p.dy), base + (k.r0 + k.tr) * p.C + c,
                      static_cast<long>(l.down) * p.C, k.rows(l.down), [&](const Raw<IO, VEC>& rx, const Raw<IO, VEC>& ry, size_t) {
      uint64_t xh[NP], dz[NP];
      to_pairs(rx, xh);
      to_pairs(ry, dz);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        xh[i] = mul2(add2(xh[i], pack2f(-mu, -mu)), pack2f(r, r));
        if (p.silu) dz[i] = mul2(dz[i], slope2(fma2(xh[i], w2[i], b2[i])));
        sw[i] = fma2(dz[i], xh[i], sw[i]);
        sb[i] = add2(sb[i], dz[i]);
      }
    });
    unpack<VEC>(sw, dw);
    unpack<VEC>(sb, db);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {              // the group's sums of a = dz w and a xh are its columns'
      s.x = fmaf(db[e], w[e], s.x);
      s.y = fmaf(dw[e], w[e], s.y);
      if (l.down == 1) {
        if (a.pw) a.pw[part + c + e] = dw[e];
        if (a.pb) a.pb[part + c + e] = db[e];
      } else {                                   // (each thread has one vector)
        cols[0][threadIdx.x * VEC + e] = dw[e];
        cols[1][threadIdx.x * VEC + e] = db[e];
      }
    }
  }
  sh[threadIdx.x] = s;
  __syncthreads();
  const Shares of(l, width);
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < l.groups_each && k.g0 + g < p.groups; g += kThreads / 32) {
    float2 m{0.f, 0.f};
    for (int i = lane; i < of.of; i += 32) {
      const float2 o = sh[of.thread(l, g, i)];
      m.x += o.x;
      m.y += o.y;
    }
    m = warp_sum(m);
    if (lane == 0) a.sums[(k.sample * p.groups + k.g0 + g) * l.chunks + k.chunk] = m;
  }
  if (l.down > 1 && (a.pw || a.pb)) {
    const int n = l.across * VEC, most = (p.groups - k.g0) * width * VEC;
    for (int c = threadIdx.x; c < n && c < most; c += kThreads) {
      float sw = 0.f, sb = 0.f;
      for (int t = 0; t < l.down; ++t) {
        sw += cols[0][t * n + c];
        sb += cols[1][t * n + c];
      }
      if (a.pw) a.pw[part + k.g0 * width * VEC + c] = sw;
      if (a.pb) a.pb[part + k.g0 * width * VEC + c] = sb;
    }
  }
}

// The second pass of both directions.
template <typename IO, int VEC, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 3 : 4) group_finish_kernel(const ChunkArgs a) {
  constexpr int NP = (VEC + 1) / 2;
  __shared__ float4 stats[kThreads];             // a group's mean, rstd and, backward, minus the means of a and a xh
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the sums: this kernel starts under the one that writes them
  const Params& p = a.p;
  const ChunkLayout& l = a.l;
  const Work k(a, gridDim.x - 1 - blockIdx.x);   // what was read last first
  const int width = p.C / p.groups / VEC, lane = threadIdx.x & 31;
  const float n = static_cast<float>(p.L) * (width * VEC);
  for (int g = threadIdx.x >> 5; g < l.groups_each && k.g0 + g < p.groups; g += kThreads / 32) {
    const long st = k.sample * p.groups + k.g0 + g;
    const float2* sums = a.sums + st * l.chunks;
    if constexpr (BWD) {
      float2 m{0.f, 0.f};
      for (int i = lane; i < l.chunks; i += 32) {
        m.x += sums[i].x;
        m.y += sums[i].y;
      }
      m = warp_sum(m);
      if (lane == 0) stats[g] = make_float4(p.mean[st], p.rstd[st], -m.x / n, -m.y / n);
    } else {
      Moments m{0.f, 0.f, 0.f};
      for (int i = lane; i < l.chunks; i += 32) {
        const long rows = (i + 1) * l.rows_each < p.L ? l.rows_each : p.L - i * l.rows_each;
        m = join(m, {static_cast<float>(rows) * (width * VEC), sums[i].x, sums[i].y});
      }
      m = warp_join(m);
      const float r = rsqrtf(m.m2 / n + p.eps);
      if (lane == 0) {
        stats[g] = make_float4(m.mean, r, 0.f, 0.f);
        if (k.chunk == 0) {
          if (p.mean) p.mean[st] = m.mean;
          if (p.rstd) p.rstd[st] = r;
        }
      }
    }
  }
  __syncthreads();
  const long stride = static_cast<long>(l.down) * p.C;
  const size_t base = (static_cast<size_t>(k.sample) * p.L + k.r0 + k.tr) * p.C;
  for (int v = k.tc; v < l.vectors && k.tr < l.down; v += l.across) {
    const int g = v / width, c = (k.g0 * width + v) * VEC;
    if (k.g0 + g >= p.groups) break;
    const float4 st = stats[g];
    const uint64_t mu = pack2f(-st.x, -st.x), r = pack2f(st.y, st.y);
    uint64_t w[NP], b[NP];
    {
      float f[VEC];
      load_param<VEC>(f, p.w, c, 1.f);
      pack<VEC>(f, w);
      load_param<VEC>(f, p.b, c, 0.f);
      pack<VEC>(f, b);
    }
    IO* out = static_cast<IO*>(p.out);
    if constexpr (BWD) {
      walk2<2, IO, VEC>(static_cast<const IO*>(p.x), static_cast<const IO*>(p.dy), base + c, stride, k.rows(l.down),
                        [&](const Raw<IO, VEC>& rx, const Raw<IO, VEC>& ry, size_t at) {
        uint64_t xh[NP], d[NP];
        float f[VEC];
        to_pairs(rx, xh);
        to_pairs(ry, d);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          xh[i] = mul2(add2(xh[i], mu), r);
          if (p.silu) d[i] = mul2(d[i], slope2(fma2(xh[i], w[i], b[i])));
          d[i] = mul2(r, fma2(xh[i], pack2f(st.w, st.w), fma2(d[i], w[i], pack2f(st.z, st.z))));
        }
        unpack<VEC>(d, f);
        Raw<IO, VEC>::store(out + at, f);
      });
    } else {
      out += base + c;
      walk<4, IO, VEC>(static_cast<const IO*>(p.x) + base + c, stride, k.rows(l.down), [&](const Raw<IO, VEC>& raw) {
        uint64_t z[NP];
        float f[VEC];
        to_pairs(raw, z);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          z[i] = fma2(mul2(add2(z[i], mu), r), w[i], b[i]);
          if (p.silu) z[i] = mul2(z[i], sigmoid2(z[i]));
        }
        unpack<VEC>(z, f);
        Raw<IO, VEC>::store(out, f);
        out += stride;
      });
    }
  }
}

// The parts' sum, in a fixed order: 32 columns x 32 shares of the parts a block.
__global__ void __launch_bounds__(1024) group_parts_kernel(const float* pw, const float* pb, float* dw, float* db, int parts, int C) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float* src = blockIdx.y == 0 ? pw : pb;
  float* dst = blockIdx.y == 0 ? dw : db;
  if (!dst) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int i = share; i < parts; i += 32) s += src[static_cast<size_t>(i) * C + c];
  }
  sh[share][lane] = s;
  __syncthreads();
  s = sh[lane][share];
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
  if (lane == 0 && blockIdx.x * 32 + share < C) dst[blockIdx.x * 32 + share] = s;
}

// -------------------------------------------------------------------- host --
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

constexpr int kMostY = 65535;          // of a grid's second dimension

enum class Way { rows, warps, chunks };
constexpr long kWarpValues = 2048;     // of a group that one warp takes

// vec: values of a vector where rows and parameters are aligned, else 1
Way way(long L, int C, int groups, int vec) {
  const int width = C / groups;
  if (L == 1 && vec > 1 && width % vec == 0) {
    const int n = width / vec;
    if (n <= 128 && (n & (n - 1)) == 0) return Way::rows;
  }
  return L * width <= kWarpValues ? Way::warps : Way::chunks;
}

unsigned row_blocks(long N, int groups, int tpu, int per_sm, unsigned& across) {
  const RowLayout lay = row_layout(groups, tpu);
  across = (groups + lay.groups_each - 1) / lay.groups_each;
  const long want = (N + lay.rows_each - 1) / lay.rows_each, most = (static_cast<long>(per_sm) * sm_count() + across - 1) / across;
  return static_cast<unsigned>(want < most ? want : most < kMostY ? most : kMostY);
}
int lanes_of(int vectors) { return vectors < 32 ? vectors : 32; }
// Blocks an SM, walking over the rows: 16384 x 4096 forward 57.2 us for 4, 58.5 for 8, 61.2 for 16; backward 105 for 2, 94
// for 3, 98 for 6.
constexpr int kRowsPerSm = 4, kBwdRowsPerSm = 3;

long weight_blocks(long rows, int C) {                     // shares of the rows for group_weights_kernel
  const long want = 8l * sm_count() / ((C + 31) / 32) + 1, most = (rows + 31) / 32;
  return want < most ? want : most < 1 ? 1 : most;
}
// Whether the chunks' first pass leaves the parts of dw and db too: 8 bytes a channel and chunk, so with chunks of 4
// positions as much workspace as a bf16 x, and with fewer positions more than that, which is where
// group_weights_kernel takes over although it is slower (128 M values, parts against that kernel: 32768 samples of 4 x
// 1024 741 us, 1153; of 8 465, 905; of 1024 317, 835; 16384 of 2 x 4096 823, 1012).
bool chunk_parts(const ChunkLayout& l) { return l.rows_each >= 4; }

size_t up16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }
size_t chunk_sums_bytes(long N, int groups, const ChunkLayout& l) { return up16(static_cast<size_t>(N) * groups * l.chunks * sizeof(float2)); }

template <typename F, typename... A>
cudaError_t with_launch(F kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, bool after, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename IO, int VEC, int NV, int TPU>
cudaError_t launch_rows(const Params& p, bool bwd, float* pw, float* pb, unsigned& parts, cudaStream_t st) {
  unsigned across;
  const unsigned down = row_blocks(p.N, p.groups, TPU, bwd ? kBwdRowsPerSm : kRowsPerSm, across);
  const dim3 grid(across, down);
  parts = down;
  if (!bwd) {
    if (p.silu) group_rows_kernel<IO, VEC, NV, TPU, true><<<grid, kThreads, 0, st>>>(p);
    else group_rows_kernel<IO, VEC, NV, TPU, false><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  const RowLayout lay = row_layout(p.groups, TPU);
  const size_t smem = lay.rows_each > 1 ? static_cast<size_t>(lay.rows_each) * lay.groups_each * TPU * NV * VEC * sizeof(float) : 0;
  if (p.silu) group_rows_bwd_kernel<IO, VEC, NV, TPU, true><<<grid, kThreads, smem, st>>>(p, pw, pb);
  else group_rows_bwd_kernel<IO, VEC, NV, TPU, false><<<grid, kThreads, smem, st>>>(p, pw, pb);
  return cudaGetLastError();
}

template <typename IO, int VEC>
cudaError_t rows_way(const Params& p, bool bwd, float* pw, float* pb, unsigned& parts, cudaStream_t st) {
  switch (p.C / p.groups / VEC) {
    case 1: return launch_rows<IO, VEC, 1, 1>(p, bwd, pw, pb, parts, st);
    case 2: return launch_rows<IO, VEC, 1, 2>(p, bwd, pw, pb, parts, st);
    case 4: return launch_rows<IO, VEC, 1, 4>(p, bwd, pw, pb, parts, st);
    case 8: return launch_rows<IO, VEC, 1, 8>(p, bwd, pw, pb, parts, st);
    case 16: return launch_rows<IO, VEC, 1, 16>(p, bwd, pw, pb, parts, st);
    case 32: return launch_rows<IO, VEC, 1, 32>(p, bwd, pw, pb, parts, st);
    case 64: return launch_rows<IO, VEC, 2, 32>(p, bwd, pw, pb, parts, st);
    default: return launch_rows<IO, VEC, 4, 32>(p, bwd, pw, pb, parts, st);
  }
}

template <typename IO, int VEC, bool BWD>
cudaError_t chunks_way(ChunkArgs a, cudaStream_t st) {
  const Params& p = a.p;
  for (; a.first < a.l.blocks; a.first += kMostY) {
    // (samples x chunks are no more than samples x positions)
    const dim3 grid(static_cast<unsigned>(p.N * a.l.chunks), a.l.blocks - a.first < kMostY ? a.l.blocks - a.first : kMostY);
    if constexpr (BWD) group_sums_kernel<IO, VEC><<<grid, kThreads, 0, st>>>(a);
    else group_moments_kernel<IO, VEC><<<grid, kThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.out) e = with_launch(group_finish_kernel<IO, VEC, BWD>, grid, kThreads, 0, st, true, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename IO>
int vector_of(const Params& p) {
  constexpr int E = 16 / sizeof(IO);
  return p.C / p.groups % E == 0 && aligned(p.x) && aligned(p.dy) && aligned(p.out) ? E : 1;
}

template <typename IO>
cudaError_t fwd(const Params& p, cudaStream_t st) {
  constexpr int E = 16 / sizeof(IO);
  const int vec = vector_of<IO>(p);
  unsigned parts;
  switch (way(p.L, p.C, p.groups, vec)) {
    case Way::rows: return rows_way<IO, E>(p, false, nullptr, nullptr, parts, st);
    case Way::warps:
      if (p.L * (p.C / p.groups) <= kMostSmall) return small_way<IO, false>(p, st);
      group_warp_kernel<IO, false><<<static_cast<unsigned>((p.N * p.groups + 7) / 8), kThreads, 0, st>>>(p);
      return cudaGetLastError();
    default: break;
  }
  const ChunkArgs a{p, chunk_layout(p.N, p.L, p.C, p.groups, vec, sm_count()), reinterpret_cast<float2*>(p.work), nullptr, nullptr};
  return vec > 1 ? chunks_way<IO, E, false>(a, st) : chunks_way<IO, 1, false>(a, st);
}

template <typename IO>
cudaError_t bwd(const Params& p, cudaStream_t st) {
  constexpr int E = 16 / sizeof(IO);
  const int vec = vector_of<IO>(p);
  const Way by = way(p.L, p.C, p.groups, vec);
  float* ws = reinterpret_cast<float*>(p.work);
  float *pw = nullptr, *pb = nullptr;
  unsigned parts = 0;
  cudaError_t e = cudaSuccess;
  auto place = [&](float* at, unsigned n) {
    parts = n;
    pw = p.dw ? at : nullptr;
    pb = p.db ? at + static_cast<size_t>(n) * p.C : nullptr;
  };
  bool weights = p.dw || p.db;                   // still to be found by a kernel of their own
  if (p.N > 0 && by == Way::rows) {
    unsigned across;
    place(ws, row_blocks(p.N, p.groups, lanes_of(p.C / p.groups / E), kBwdRowsPerSm, across));
    e = rows_way<IO, E>(p, true, pw, pb, parts, st);
    weights = false;
  } else if (p.N > 0 && by == Way::warps) {
    if (p.out) {
      if (p.L * (p.C / p.groups) <= kMostSmall) small_way<IO, true>(p, st);
      else group_warp_kernel<IO, true><<<static_cast<unsigned>((p.N * p.groups + 7) / 8), kThreads, 0, st>>>(p);
    }
    e = cudaGetLastError();
  } else if (p.N > 0) {
    ChunkArgs a{p, chunk_layout(p.N, p.L, p.C, p.groups, vec, sm_count()), reinterpret_cast<float2*>(ws), nullptr, nullptr};
    ws += chunk_sums_bytes(p.N, p.groups, a.l) / sizeof(float);
    const bool here = weights && chunk_parts(a.l);
    if (here) {
      place(ws, static_cast<unsigned>(p.N * a.l.chunks));
      a.pw = pw;
      a.pb = pb;
      weights = false;
    }
    if (p.out || here) e = vec > 1 ? chunks_way<IO, E, true>(a, st) : chunks_way<IO, 1, true>(a, st);
  }
  if (e != cudaSuccess) return e;
  if (weights && p.N > 0) {
    const long rows = p.N * p.L, blocks = weight_blocks(rows, p.C), each = (rows + blocks - 1) / blocks;
    place(ws, static_cast<unsigned>((rows + each - 1) / each));
    group_weights_kernel<IO><<<dim3((p.C + 31) / 32, parts), kThreads, 0, st>>>(p, each, pw, pb);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!p.dw && !p.db) return cudaSuccess;
  // (under the chunks' second pass it would start too early: that one does not wait for the parts' kernel's end by itself)
  return with_launch(group_parts_kernel, dim3((p.C + 31) / 32, 2), 1024, 0, st, p.N > 0 && by != Way::chunks,
                     static_cast<const float*>(pw), static_cast<const float*>(pb), p.dw, p.db, static_cast<int>(parts), p.C);
}

}  // namespace

size_t fwd_workspace_bytes(long N, long L, int C, int groups) {
  size_t most = 0;
  if (N == 0) return 0;                // (no samples: no layout, and nothing to keep)
  for (int vec : {1, 4, 8})            // (the call's types and alignment are not known here)
    if (C / groups % vec == 0 && way(L, C, groups, vec) == Way::chunks) {
      const size_t n = chunk_sums_bytes(N, groups, chunk_layout(N, L, C, groups, vec, sm_count()));
      most = n > most ? n : most;
    }
  return most;
}

size_t bwd_workspace_bytes(long N, long L, int C, int groups) {
  if (N == 0) return 0;
  const size_t row = 2 * static_cast<size_t>(C) * sizeof(float), weights = weight_blocks(N * L, C) * row;
  size_t most = 0;
  for (int vec : {1, 4, 8}) {
    if (C / groups % vec != 0) continue;
    size_t n = weights;
    const Way by = way(L, C, groups, vec);
    if (by == Way::rows) {
      unsigned across;
      n = row_blocks(N, groups, lanes_of(C / groups / vec), kBwdRowsPerSm, across) * row;
    } else if (by == Way::chunks) {
      const ChunkLayout l = chunk_layout(N, L, C, groups, vec, sm_count());
      n = chunk_sums_bytes(N, groups, l) + (chunk_parts(l) ? static_cast<size_t>(N) * l.chunks * row : weights);
    }
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_fwd(const Params& p, bool bf16, cudaStream_t st) { return bf16 ? fwd<__nv_bfloat16>(p, st) : fwd<float>(p, st); }
cudaError_t launch_bwd(const Params& p, bool bf16, cudaStream_t st) { return bf16 ? bwd<__nv_bfloat16>(p, st) : bwd<float>(p, st); }

}  // namespace gn
}  // namespace kda
