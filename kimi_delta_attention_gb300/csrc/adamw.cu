// adamw.cu -- one AdamW step over many tensors, states in fp32 or in e4m3 with a scale for 256 values.
//
//     m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//     p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Every value is read once and written once.  The tensors' addresses travel in the launch's own
// parameters, so a step needs no table in device memory, and a captured one keeps its own.
#include <cuda_fp8.h>

#include <cmath>

#include "layer_ops.cuh"

namespace kda {
namespace adamw {
namespace {

constexpr int kThreads = 256, kEach = 8;             // a thread's values: a warp holds a block of 256
constexpr int kChunk = kThreads * kEach;             // values a thread block takes at once
constexpr int kBlock = KDA_ADAMW_BLOCK;
static_assert(kBlock == 32 * kEach, "a warp holds a block of values that share a scale");

struct Entry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  long n;
};
enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2, kVector = 4 };

struct Scalars {
  float lr, wd, b1, c1, b2, c2, eps;   // c = 1 - b
  double log_b1, log_b2;               // for the step's bias corrections
  int step;
  uint32_t seed_lo, seed_hi;
  const int32_t* step_device;
  const float* lr_device;
  const float* grad_scale;
  const float* skip;
};

// What a launch takes: up to CAP tensors (launch parameters hold 32764 bytes).
template <int CAP>
struct Batch {
  Scalars s;
  int count, number;        // tensors here, and the first one's number in the call
  uint32_t first[CAP + 1];  // first thread block of each tensor
  uint32_t flags[CAP];
  Entry t[CAP];
};

// A 32-bit mix of shifts and odd multiplications (each input bit turns over half of the output's).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x71C61315u;
  x = (x ^ (x >> 15)) * 0x189C32BFu;
  return x ^ (x >> 16);
}
constexpr uint32_t kSpread = 0x9E3779B1u;

template <typename T>
__device__ __forceinline__ void load8(float (&x)[kEach], const T* src, int left, bool vector) {
  if (vector && left >= kEach) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(src);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 u = reinterpret_cast<const float4*>(src)[i];
        x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = i < left ? to_f32(src[i]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[kEach], int left, bool vector) {
  if (vector && left >= kEach) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        reinterpret_cast<float4*>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < left) dst[i] = from_f32<T>(x[i]);
  }
}

__device__ __forceinline__ float decode(uint8_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__device__ __forceinline__ void load_codes(float (&x)[kEach], const uint8_t* src, float scale, int left, bool vector) {
  uint8_t c[kEach];
  if (vector && left >= kEach) {
    *reinterpret_cast<uint2*>(c) = *reinterpret_cast<const uint2*>(src);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) c[i] = i < left ? src[i] : uint8_t(0);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) x[i] = __fmul_rn(decode(c[i]), scale);
}

// The codes of a warp's 256 values, by random numbers in [0, 1) (16 bits of each hash from `shift`),
// and their scale.  Each operation is rounded by itself, so the result is that of the formula in
// fp32 operations whatever the compiler.  KEEP: a value above 0 keeps a code above 0.
template <bool KEEP>
__device__ __forceinline__ float store_codes(uint8_t* dst, const float (&x)[kEach], const uint32_t (&hash)[kEach], int shift,
                                             int left, bool vector) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) top = fmaxf(top, isfinite(x[i]) ? fabsf(x[i]) : 0.f);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
  const bool some = top >= 0x1p-100f;
  const float scale = some ? __fmul_rn(top, static_cast<float>(1.0 / 448)) : 0.f;
  const float up0 = some ? __fmul_rn(__frcp_rn(top), 448.f) : 0.f;
  uint8_t c[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const float a = fabsf(x[i]), y = __fmul_rn(a, up0);
    const int e = min(max((__float_as_int(y) >> 23) - 127, -6), 8);        // (subnormal codes share their step)
    const float u = static_cast<float>((hash[i] >> shift) & 0xFFFFu) * 0x1p-16f;
    float q = __fmul_rn(floorf(__fadd_rn(__fmul_rn(y, __int_as_float((130 - e) << 23)), u)), __int_as_float((124 + e) << 23));
    q = fminf(q, 448.f);
    if (KEEP && a > 0.f && q == 0.f) q = 0x1p-9f;
    if (!isfinite(a)) q = __int_as_float(0x7FFFFFFF);
    c[i] = __nv_cvt_float_to_fp8(copysignf(q, x[i]), __NV_SATFINITE, __NV_E4M3);
  }
  if (vector && left >= kEach) {
    *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(c);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < left) dst[i] = c[i];
  }
  return scale;
}

template <int CAP, bool BITS8>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Batch<CAP> b) {
  __shared__ float sh[5];
  __shared__ uint32_t sh_key;
  const Scalars& s = b.s;
  if (s.skip && *s.skip != 0.f) return;
  int lo = 0, hi = b.count;            // the tensor of this block: first[lo] <= blockIdx.x < first[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (b.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  if (threadIdx.x == 0) {
    const int step = s.step_device ? *s.step_device : s.step;
    const float lr = s.lr_device ? *s.lr_device : s.lr;
    const float bc1 = static_cast<float>(-expm1(step * s.log_b1)), bc2 = static_cast<float>(-expm1(step * s.log_b2));
    sh[0] = 1.f - lr * s.wd;
    sh[1] = lr / bc1;
    sh[2] = 1.f / sqrtf(bc2);
    sh[3] = s.grad_scale ? *s.grad_scale : 1.f;
    const uint32_t key = mix(s.seed_lo ^ mix(s.seed_hi ^ mix(static_cast<uint32_t>(step))));
    sh_key = mix(key + static_cast<uint32_t>(b.number + lo) * kSpread);
  }
  __syncthreads();
  const float keep = sh[0], rate = sh[1], inv = sh[2], gs = sh[3];
  const Entry& t = b.t[lo];
  const uint32_t flags = b.flags[lo];
  const bool vector = flags & kVector;
  const long at = static_cast<long>(blockIdx.x - b.first[lo]) * kChunk + threadIdx.x * kEach;
  if ((at & ~static_cast<long>(kBlock - 1)) >= t.n) return;            // (whole warps)
  const long rest = t.n - at;
  const int left = rest < 0 ? 0 : rest > kEach ? kEach : static_cast<int>(rest);
  const long blk = at / kBlock;
  float p[kEach], g[kEach], m[kEach], v[kEach];
  if (t.master) load8(p, t.master + at, left, vector);
  else if (flags & kParamBf16) load8(p, static_cast<const __nv_bfloat16*>(t.p) + at, left, vector);
  else load8(p, static_cast<const float*>(t.p) + at, left, vector);
  if (flags & kGradBf16) load8(g, static_cast<const __nv_bfloat16*>(t.g) + at, left, vector);
  else load8(g, static_cast<const float*>(t.g) + at, left, vector);
  if constexpr (BITS8) {
    load_codes(m, static_cast<const uint8_t*>(t.m) + at, t.m_scale[blk], left, vector);
    load_codes(v, static_cast<const uint8_t*>(t.v) + at, t.v_scale[blk], left, vector);
  } else {
    load8(m, static_cast<const float*>(t.m) + at, left, vector);
    load8(v, static_cast<const float*>(t.v) + at, left, vector);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const float d = s.grad_scale ? __fmul_rn(g[i], gs) : g[i];
    m[i] = __fadd_rn(__fmul_rn(m[i], s.b1), __fmul_rn(d, s.c1));
    v[i] = __fadd_rn(__fmul_rn(v[i], s.b2), __fmul_rn(__fmul_rn(d, d), s.c2));
    p[i] = p[i] * keep - rate * (m[i] / fmaf(sqrtf(v[i]), inv, s.eps));
  }
  if (t.master) store8(t.master + at, p, left, vector);
  if (flags & kParamBf16) store8(static_cast<__nv_bfloat16*>(t.p) + at, p, left, vector);
  else store8(static_cast<float*>(t.p) + at, p, left, vector);
  if constexpr (BITS8) {
    uint32_t hash[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      hash[i] = mix((static_cast<uint32_t>(at + i) * kSpread) ^ sh_key);
      if (i >= left) m[i] = v[i] = 0.f;
    }
    const float ms = store_codes<false>(static_cast<uint8_t*>(t.m) + at, m, hash, 0, left, vector);
    const float vs = store_codes<true>(static_cast<uint8_t*>(t.v) + at, v, hash, 16, left, vector);
    if ((threadIdx.x & 31) == 0) {
      t.m_scale[blk] = ms;
      t.v_scale[blk] = vs;
    }
  } else {
    store8(static_cast<float*>(t.m) + at, m, left, vector);
    store8(static_cast<float*>(t.v) + at, v, left, vector);
  }
}

template <int CAP>
cudaError_t launch_batch(const kda_adamw_tensor* tensors, int from, int to, const Scalars& s, bool bits8, cudaStream_t st) {
  static_assert(sizeof(Batch<CAP>) <= 32764, "launch parameters");
  Batch<CAP> b;
  b.s = s;
  b.count = 0;
  b.number = from;
  uint64_t blocks = 0;
  for (int i = from; i < to; ++i) {
    const kda_adamw_tensor& t = tensors[i];
    const uintptr_t state = bits8 ? 7 : 15;
    auto off = [](const void* q, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(q) & mask) != 0; };
    const bool vector = !off(t.param, 15) && !off(t.grad, 15) && !off(t.m, state) && !off(t.v, state) && !off(t.master, 15);
    b.first[b.count] = static_cast<uint32_t>(blocks);
    b.flags[b.count] = (t.param_dtype == KDA_BF16 ? kParamBf16 : 0u) | (t.grad_dtype == KDA_BF16 ? kGradBf16 : 0u) |
                       (vector ? kVector : 0u);
    b.t[b.count++] = Entry{t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.master, static_cast<long>(t.n)};
    blocks += (static_cast<uint64_t>(t.n) + kChunk - 1) / kChunk;
  }
  if (blocks == 0) return cudaSuccess;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  b.first[b.count] = static_cast<uint32_t>(blocks);
  if (bits8) adamw_kernel<CAP, true><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(b);
  else adamw_kernel<CAP, false><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(b);
  return cudaGetLastError();
}

constexpr int kMany = 440, kFew = 24;

}  // namespace

cudaError_t launch(const kda_adamw_tensor* tensors, int count, const kda_adamw_config& c, cudaStream_t st) {
  const Scalars s{static_cast<float>(c.lr), static_cast<float>(c.weight_decay), static_cast<float>(c.beta1),
                  static_cast<float>(1 - c.beta1), static_cast<float>(c.beta2), static_cast<float>(1 - c.beta2),
                  static_cast<float>(c.eps), std::log(c.beta1), std::log(c.beta2), static_cast<int>(c.step),
                  static_cast<uint32_t>(c.seed), static_cast<uint32_t>(c.seed >> 32), c.step_device, c.lr_device,
                  c.grad_scale, c.skip};
  for (int from = 0; from < count; from += kMany) {
    const int to = count - from < kMany ? count : from + kMany;
    const cudaError_t e = to - from <= kFew ? launch_batch<kFew>(tensors, from, to, s, c.state_bits == 8, st)
                                            : launch_batch<kMany>(tensors, from, to, s, c.state_bits == 8, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace adamw
}  // namespace kda
