// adamw.cu -- one AdamW step over many tensors, states in fp32 or in e4m3 with a scale for 256 values.
//
//     m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//     p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Every value is read once and written once.  With 32-bit states that is all there is to it (22 bytes a
// value in bf16, 28 in fp32 and in bf16 with masters): 134 M values 440 us, 551 and 559, 6.7 to 6.8 TB/s, the copy rate.
// With 8-bit states (10 bytes) the instructions count as much: 403 M values 1035 us, 58 % of the copy rate, 71 % of the
// issue slots used, 87 instructions a value: 37 for
// the rounding, 12 for its random numbers, 9 for the step, the rest loads, decoding, averages and stores.
// So codes are made in integer arithmetic on the bits of the scaled value, and what is rare (subnormal codes,
// values that are not finite, ragged ends) lies aside of the common path.  The tensors' addresses travel in the
// launch's own parameters, so a step needs no table in device memory, and a captured one keeps its own.
#include <cuda_fp8.h>

#include <cmath>

#include "layer_ops.cuh"

namespace kda {
namespace adamw {
namespace {

constexpr int kThreads = 256, kEach = 8;             // a thread's values: a warp holds a block of 256
constexpr int kPass = kThreads * kEach;              // values a thread block takes at once
constexpr int kChunk = 8 * kPass;                    // and in all
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

// What learning rate and step number give, the same from either side.
struct Rates {
  float keep, rate, inv;               // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};
__host__ __device__ __forceinline__ Rates rates(float lr, double wd, double log_b1, double log_b2, int step) {
  return {static_cast<float>(1 - lr * wd), static_cast<float>(lr / -expm1(step * log_b1)),
          static_cast<float>(1 / sqrt(-expm1(step * log_b2)))};
}

struct Scalars {
  Rates r;
  float lr, b1, c1, b2, c2, eps;       // c = 1 - b
  double wd, log_b1, log_b2;
  int step;
  uint32_t key, seed_lo, seed_hi;      // key: of seed and step
  const int32_t* step_device;          // with either of these two, r and key are found on the device
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

// A 32-bit mix: shifts, odd multiplications and exclusive ors, each of which can be undone, so no two inputs meet.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x71C61315u;
  x = (x ^ (x >> 15)) * 0x189C32BFu;
  return x ^ (x >> 16);
}
constexpr uint32_t kSpread = 0x9E3779B1u;
__host__ __device__ __forceinline__ uint32_t step_key(uint32_t lo, uint32_t hi, int step) {
  return mix(lo ^ mix(hi ^ mix(static_cast<uint32_t>(step))));
}

// FULL: a whole pass of values at aligned addresses; else `left` of a thread's own, one by one.
template <bool FULL, typename T>
__device__ __forceinline__ void load8(float (&x)[kEach], const T* src, int left) {
  if constexpr (FULL) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(src);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      // (32 bytes in one load: two of 16 would leave half of each sector to the other)
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                   : "l"(src));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = i < left ? to_f32(src[i]) : 0.f;
  }
}

template <bool FULL, typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[kEach], int left) {
  if constexpr (FULL) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
                   "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "l"(dst)
                   : "memory");
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < left) dst[i] = from_f32<T>(x[i]);
  }
}

template <bool FULL>
__device__ __forceinline__ void load_codes(float (&x)[kEach], const uint8_t* src, float scale, int left) {
  uint32_t c[2] = {0u, 0u};
  if constexpr (FULL) {
    const uint2 u = *reinterpret_cast<const uint2*>(src);
    c[0] = u.x;
    c[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < left) c[i / 4] |= static_cast<uint32_t>(src[i]) << 8 * (i % 4);
  }
#pragma unroll
  for (int i = 0; i < kEach / 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(c[i / 2] >> 16 * (i % 2)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = __fmul_rn(f.x, scale);
    x[2 * i + 1] = __fmul_rn(f.y, scale);
  }
}

// The codes of a warp's 256 values, by 16 bits of each value's hash from `SHIFT` on, and their scale.  With y =
// |x| 448 / top, a code's step in y is 2^(e - 3) for 2^e <= y < 2^(e + 1), and 2^-9 below 2^-6; the random
// number, in steps, is added and the rest cut off.  On the bits of y that is one integer addition
// (the exponent follows the mantissa, in fp32 as in the code).
// KEEP: a value above 0 keeps a code above 0.
// Logic, shifts, compares and selections run at half the rate of multiplications and additions and bound this
// kernel, so what can be a multiplication is one.
template <bool FULL, int SHIFT, bool KEEP>
__device__ __forceinline__ float store_codes(uint8_t* dst, const float (&x)[kEach], const uint32_t (&hash)[kEach], int left) {
  float largest = 0.f, odd = 0.f;      // (odd becomes NaN by a value that is not finite)
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    largest = fmaxf(largest, fabsf(x[i]));
    odd = fmaf(x[i], 0.f, odd);
  }
  const bool bad = __any_sync(0xFFFFFFFFu, odd != 0.f);
  if (bad) {                           // (the whole warp) such values count for no scale
    largest = 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) largest = fmaxf(largest, isfinite(x[i]) ? fabsf(x[i]) : 0.f);
  }
  largest = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(largest)));   // magnitudes compare as their bits do
  const bool some = largest >= 0x1p-100f;
  const float scale = some ? __fmul_rn(largest, static_cast<float>(1.0 / 448)) : 0.f;
  const float up = some ? __fmul_rn(__frcp_rn(largest), 448.f) : 0.f;
  uint32_t code[kEach];
  float least = 448.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const float y = fabsf(__fmul_rn(x[i], up));
    least = fminf(least, y);
    const uint32_t u = SHIFT == 0 ? hash[i] & 0xFFFFu : hash[i] >> 16;
    code[i] = static_cast<uint32_t>(min(static_cast<int>((__float_as_uint(y) + u * 16u) >> 20) - 960, 126));   // 960: the exponents' offset
  }
  if (__any_sync(0xFFFFFFFFu, least < 0x1p-6f)) {      // below: the codes' own subnormals
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const float y = fabsf(__fmul_rn(x[i], up));
      const uint32_t u = SHIFT == 0 ? hash[i] & 0xFFFFu : hash[i] >> 16;
      // floor(512 y + random number): the sum rounded down at 2^23 has it in its last bits
      const float z = fmaf(y, 512.f, __uint_as_float(u * 128u + 0x3F800000u) - 1.f);
      if (y < 0x1p-6f) code[i] = __float_as_uint(__fadd_rd(z, 0x1p23f)) - 0x4B000000u;
      if (KEEP && x[i] > 0.f) code[i] = max(code[i], 1u);
    }
  }
  if (bad)
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (!isfinite(x[i])) code[i] = 0x7Fu;
  uint32_t c[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    c[k] = code[4 * k] + code[4 * k + 1] * 0x100u + code[4 * k + 2] * 0x10000u + code[4 * k + 3] * 0x1000000u;
    if (!KEEP) {                       // the signs: the values' top bytes side by side
      const uint32_t a = __byte_perm(__float_as_uint(x[4 * k]), __float_as_uint(x[4 * k + 1]), 0x0073);
      const uint32_t b = __byte_perm(__float_as_uint(x[4 * k + 2]), __float_as_uint(x[4 * k + 3]), 0x0073);
      c[k] |= __byte_perm(a, b, 0x5410) & 0x80808080u;
    }
  }
  if constexpr (FULL) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < left) dst[i] = static_cast<uint8_t>(c[i / 4] >> 8 * (i % 4));
  }
  return scale;
}

// Where a block's values begin: what is alike for all its threads is worked out once, and a thread adds a
// 32-bit offset.
struct Chunk {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
};

// A thread's values from the chunk's `at` on; place: the first one's in its tensor.
template <bool BITS8, bool FULL>
__device__ __forceinline__ void update(const Scalars& s, const Rates& r, float gs, uint32_t key, const Chunk& t, uint32_t flags,
                                       uint32_t at, uint32_t place, int left) {
  const uint32_t blk = at / kBlock;
  float p[kEach], g[kEach], m[kEach], v[kEach];
  if (t.master) load8<FULL>(p, t.master + at, left);
  else if (flags & kParamBf16) load8<FULL>(p, static_cast<const __nv_bfloat16*>(t.p) + at, left);
  else load8<FULL>(p, static_cast<const float*>(t.p) + at, left);
  if (flags & kGradBf16) load8<FULL>(g, static_cast<const __nv_bfloat16*>(t.g) + at, left);
  else load8<FULL>(g, static_cast<const float*>(t.g) + at, left);
  if constexpr (BITS8) {
    load_codes<FULL>(m, static_cast<const uint8_t*>(t.m) + at, t.m_scale[blk], left);
    load_codes<FULL>(v, static_cast<const uint8_t*>(t.v) + at, t.v_scale[blk], left);
  } else {
    load8<FULL>(m, static_cast<const float*>(t.m) + at, left);
    load8<FULL>(v, static_cast<const float*>(t.v) + at, left);
  }
  // m and v: each operation rounded by itself, as the formula's (the codes go by their bits)
  if (s.grad_scale)
#pragma unroll
    for (int i = 0; i < kEach; ++i) g[i] = __fmul_rn(g[i], gs);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    m[i] = __fadd_rn(__fmul_rn(m[i], s.b1), __fmul_rn(g[i], s.c1));
    v[i] = __fadd_rn(__fmul_rn(v[i], s.b2), __fmul_rn(__fmul_rn(g[i], g[i]), s.c2));
  }
  // part: 1 / (sqrt(v) / sqrt(1 - b2^t) + eps), never so small or large that ftz counts.  A root below 1e-19 is nothing
  // beside an eps of 1e-15, so it may be flushed to 0 there, which is three instructions less.
  float part[kEach];
  if (s.eps >= 1e-15f) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(part[i]) : "f"(v[i]));
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) asm("sqrt.approx.f32 %0, %1;" : "=f"(part[i]) : "f"(v[i]));
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(part[i]) : "f"(fmaf(part[i], r.inv, s.eps)));
    p[i] = fmaf(p[i], r.keep, -r.rate * (m[i] * part[i]));
  }
  if (t.master) store8<FULL>(t.master + at, p, left);
  if (flags & kParamBf16) store8<FULL>(static_cast<__nv_bfloat16*>(t.p) + at, p, left);
  else store8<FULL>(static_cast<float*>(t.p) + at, p, left);
  if constexpr (BITS8) {
    uint32_t hash[kEach];
    const uint32_t h0 = place * kSpread;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      hash[i] = mix((h0 + i * kSpread) ^ key);
      if (!FULL && i >= left) m[i] = v[i] = 0.f;
    }
    const float ms = store_codes<FULL, 0, false>(static_cast<uint8_t*>(t.m) + at, m, hash, left);
    const float vs = store_codes<FULL, 16, true>(static_cast<uint8_t*>(t.v) + at, v, hash, left);
    if ((threadIdx.x & 31) == 0) {
      t.m_scale[blk] = ms;
      t.v_scale[blk] = vs;
    }
  } else {
    store8<FULL>(static_cast<float*>(t.m) + at, m, left);
    store8<FULL>(static_cast<float*>(t.v) + at, v, left);
  }
}

// A block takes up to 8 passes of one tensor.  Five blocks an SM: 385 us for 134 M values with 8-bit states, 418 for
// four, 461 for three (more registers hide less than more warps).
template <int CAP, bool BITS8>
__global__ void __launch_bounds__(kThreads, 5) adamw_kernel(const __grid_constant__ Batch<CAP> b) {
  __shared__ Rates sh;
  __shared__ uint32_t sh_key;
  const Scalars& s = b.s;
  if (s.skip && *s.skip != 0.f) return;
  int lo = 0, hi = b.count;            // the tensor of this block: first[lo] <= blockIdx.x < first[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (b.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  Rates r = s.r;
  uint32_t key = s.key;
  if (s.step_device || s.lr_device) {
    if (threadIdx.x == 0) {
      const int step = s.step_device ? *s.step_device : s.step;
      sh = rates(s.lr_device ? *s.lr_device : s.lr, s.wd, s.log_b1, s.log_b2, step);
      sh_key = step_key(s.seed_lo, s.seed_hi, step);
    }
    __syncthreads();
    r = sh;
    key = sh_key;
  }
  key = mix(key + static_cast<uint32_t>(b.number + lo) * kSpread);
  const float gs = s.grad_scale ? *s.grad_scale : 1.f;
  const Entry& e = b.t[lo];
  const uint32_t flags = b.flags[lo];
  const long from = static_cast<long>(blockIdx.x - b.first[lo]) * kChunk;
  const long rest = e.n - from;
  const uint32_t n = rest < kChunk ? static_cast<uint32_t>(rest) : kChunk;      // values of this block (at least one)
  const long p_size = flags & kParamBf16 ? 2 : 4, g_size = flags & kGradBf16 ? 2 : 4, state_size = BITS8 ? 1 : 4;
  const Chunk t{static_cast<char*>(e.p) + from * p_size,
                static_cast<const char*>(e.g) + from * g_size,
                static_cast<char*>(e.m) + from * state_size,
                static_cast<char*>(e.v) + from * state_size,
                BITS8 ? e.m_scale + from / kBlock : nullptr,
                BITS8 ? e.v_scale + from / kBlock : nullptr,
                e.master ? e.master + from : nullptr};
  const uint32_t place = static_cast<uint32_t>(from);
#pragma unroll 1
  for (uint32_t pass = 0; pass < n; pass += kPass) {
    const uint32_t at = pass + threadIdx.x * kEach;
    if ((flags & kVector) && pass + kPass <= n) {
      update<BITS8, true>(s, r, gs, key, t, flags, at, place + at, kEach);
    } else if ((at & ~static_cast<uint32_t>(kBlock - 1)) < n) {                  // (whole warps)
      update<BITS8, false>(s, r, gs, key, t, flags, at, place + at, at >= n ? 0 : min(static_cast<int>(n - at), kEach));
    }
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
    // (vectors of 8 values: 32 bytes in fp32, 16 in bf16, 8 of codes; a tensor elsewhere goes value by value)
    const uintptr_t state = bits8 ? 7 : 31, param = t.param_dtype == KDA_BF16 ? 15 : 31, grad = t.grad_dtype == KDA_BF16 ? 15 : 31;
    auto off = [](const void* q, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(q) & mask) != 0; };
    const bool vector = !off(t.param, param) && !off(t.grad, grad) && !off(t.m, state) && !off(t.v, state) && !off(t.master, 31);
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

// Most tensors of a launch, and of one with small parameters, which the host copies for every launch: a call of 4
// tensors 21.6 us for 23.8, of 24 50.7 for 53.1 (on the device, in a graph, both are alike: 2.7 and 2.9 us of 1000 values each).
constexpr int kMany = 440, kFew = 24;

}  // namespace

cudaError_t launch(const kda_adamw_tensor* tensors, int count, const kda_adamw_config& c, cudaStream_t st) {
  Scalars s{};
  s.lr = static_cast<float>(c.lr);
  s.wd = c.weight_decay;
  s.b1 = static_cast<float>(c.beta1);
  s.c1 = static_cast<float>(1 - c.beta1);
  s.b2 = static_cast<float>(c.beta2);
  s.c2 = static_cast<float>(1 - c.beta2);
  s.eps = static_cast<float>(c.eps);
  s.log_b1 = std::log(c.beta1);
  s.log_b2 = std::log(c.beta2);
  s.step = static_cast<int>(c.step);
  s.r = rates(s.lr, s.wd, s.log_b1, s.log_b2, s.step);
  s.seed_lo = static_cast<uint32_t>(c.seed);
  s.seed_hi = static_cast<uint32_t>(c.seed >> 32);
  s.key = step_key(s.seed_lo, s.seed_hi, s.step);
  s.step_device = c.step_device;
  s.lr_device = c.lr_device;
  s.grad_scale = c.grad_scale;
  s.skip = c.skip;
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
