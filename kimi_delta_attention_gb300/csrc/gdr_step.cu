// gdr_step.cu -- the gated delta rule token by token, fp32 on CUDA cores: the serving step
// (states read and updated in place, optionally in a pool) and the forward for fp32 I/O.
//
// Per sequence and value head, with one gate per token (scalar e^{g_t}):
//     P   = e^{g_t} S_{t-1}
//     S_t = P + beta_t k_t (v_t - P^T k_t)^T
//     o_t = scale S_t^T q_t
// A column of S meets only its own column of v and o, so the columns are split freely: a
// warp owns 16 value columns of one head and needs no other warp.  Thread (r, c) of a warp
// (r = lane / 4, c = lane % 4) holds rows r K/8 .. and columns 4 c .. 4 c + 3 in registers;
// the two sums over rows per token are 3 shuffle steps over r.  All the state's loads are
// issued before the first use, 256 B a thread at K = 128.
// Bound: at T = 1 a call moves the state once each way, 128 KiB per (sequence, value head)
// at K = V = 128, and next to nothing else: HBM bandwidth, or latency for a few heads.
#include "gdr_common.cuh"

namespace kda {
namespace gdr {
namespace {

constexpr int COLS = 16;  // value columns of a warp

struct StepParams {
  Params p;
  float* state;          // serving step: [B or num_slots, HV, K, V], in place; else null
  const int32_t* slots;  // [B] or null
  int num_slots;
};

template <typename IO, int N>
__device__ __forceinline__ void load_row(float (&x)[N], const IO* src) {
  constexpr int E = 16 / sizeof(IO);
#pragma unroll
  for (int i = 0; i < N / E; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(src)[i];
    if constexpr (sizeof(IO) == 4) {
      x[4 * i] = __uint_as_float(u.x);
      x[4 * i + 1] = __uint_as_float(u.y);
      x[4 * i + 2] = __uint_as_float(u.z);
      x[4 * i + 3] = __uint_as_float(u.w);
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}

template <typename IO, int K>
__global__ void __launch_bounds__(256) gdr_recurrent_kernel(const StepParams a, int V) {
  constexpr int R = K / 8;  // rows of a thread
  const Params& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int slices = V / COLS;                       // warps per (sequence, value head)
  const long w = static_cast<long>(blockIdx.x) * warps + warp;
  const long unit = w / slices;
  if (unit >= static_cast<long>(p.num_seqs) * p.HV) return;
  const int seq = static_cast<int>(unit / p.HV), hv = static_cast<int>(unit % p.HV), hk = hv / (p.HV / p.H);
  const int r0 = (lane >> 2) * R, col = static_cast<int>(w % slices) * COLS + 4 * (lane & 3);

  const IO* q = static_cast<const IO*>(p.q);
  const IO* k = static_cast<const IO*>(p.k);
  const IO* v = static_cast<const IO*>(p.v);
  IO* out = static_cast<IO*>(p.out);
  long tok0;
  int len;
  seq_tokens(p.cu, p.T, p.num_seqs, p.status, seq, tok0, len);

  const float* src = p.s0;
  float* dst = p.sfin;
  long at = seq;
  bool live = true;
  if (a.state) {
    src = dst = a.state;
    if (a.slots) {
      at = a.slots[seq];
      live = at >= 0 && at < a.num_slots;  // a negative slot is an empty row: no state, o = 0
      if (at >= a.num_slots && p.status && lane == 0) atomicOr(p.status, kStatusBounds);
    }
  }
  if (!live) {
    if ((lane >> 2) == 0)
      for (int t = 0; t < len; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) out[(static_cast<size_t>(tok0 + t) * p.HV + hv) * V + col + c] = from_f32<IO>(0.f);
    return;
  }
  const size_t off = (static_cast<size_t>(at) * p.HV + hv) * K * V + static_cast<size_t>(r0) * V + col;
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    s[i] = src ? *reinterpret_cast<const float4*>(src + off + static_cast<size_t>(i) * V) : make_float4(0.f, 0.f, 0.f, 0.f);

  auto sum_rows = [](float4 x) {  // over the warp's 8 row groups
#pragma unroll
    for (int m = 4; m < 32; m <<= 1) {
      x.x += __shfl_xor_sync(0xFFFFFFFFu, x.x, m);
      x.y += __shfl_xor_sync(0xFFFFFFFFu, x.y, m);
      x.z += __shfl_xor_sync(0xFFFFFFFFu, x.z, m);
      x.w += __shfl_xor_sync(0xFFFFFFFFu, x.w, m);
    }
    return x;
  };
  for (int t = 0; t < len; ++t) {
    const size_t tok = static_cast<size_t>(tok0 + t);
    float kr[R], qr[R];
    load_row<IO, R>(kr, k + (tok * p.H + hk) * K + r0);
    load_row<IO, R>(qr, q + (tok * p.H + hk) * K + r0);
    const float e = expf(p.g[tok * p.HV + hv]), b = p.beta[tok * p.HV + hv];
    float vv[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) vv[c] = to_f32(v[(tok * p.HV + hv) * V + col + c]);
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i].x *= e; s[i].y *= e; s[i].z *= e; s[i].w *= e;
      u.x = fmaf(kr[i], s[i].x, u.x); u.y = fmaf(kr[i], s[i].y, u.y);
      u.z = fmaf(kr[i], s[i].z, u.z); u.w = fmaf(kr[i], s[i].w, u.w);
    }
    u = sum_rows(u);
    const float4 d = make_float4(b * (vv[0] - u.x), b * (vv[1] - u.y), b * (vv[2] - u.z), b * (vv[3] - u.w));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i].x = fmaf(kr[i], d.x, s[i].x); s[i].y = fmaf(kr[i], d.y, s[i].y);
      s[i].z = fmaf(kr[i], d.z, s[i].z); s[i].w = fmaf(kr[i], d.w, s[i].w);
      o.x = fmaf(qr[i], s[i].x, o.x); o.y = fmaf(qr[i], s[i].y, o.y);
      o.z = fmaf(qr[i], s[i].z, o.z); o.w = fmaf(qr[i], s[i].w, o.w);
    }
    o = sum_rows(o);
    if ((lane >> 2) == 0) {
      IO* op = out + (tok * p.HV + hv) * V + col;
      op[0] = from_f32<IO>(p.scale * o.x);
      op[1] = from_f32<IO>(p.scale * o.y);
      op[2] = from_f32<IO>(p.scale * o.z);
      op[3] = from_f32<IO>(p.scale * o.w);
    }
  }
  if (dst) {
#pragma unroll
    for (int i = 0; i < R; ++i) *reinterpret_cast<float4*>(dst + off + static_cast<size_t>(i) * V) = s[i];
  }
}

cudaError_t launch(const StepParams& a, int K, int V, bool bf16, cudaStream_t stream) {
  const long warps = static_cast<long>(a.p.num_seqs) * a.p.HV * (V / COLS);
  if (warps == 0) return cudaSuccess;
  const int per = 8;
  const unsigned grid = static_cast<unsigned>((warps + per - 1) / per);
  if (bf16) {
    if (K == 128) gdr_recurrent_kernel<__nv_bfloat16, 128><<<grid, 32 * per, 0, stream>>>(a, V);
    else gdr_recurrent_kernel<__nv_bfloat16, 64><<<grid, 32 * per, 0, stream>>>(a, V);
  } else {
    if (K == 128) gdr_recurrent_kernel<float, 128><<<grid, 32 * per, 0, stream>>>(a, V);
    else gdr_recurrent_kernel<float, 64><<<grid, 32 * per, 0, stream>>>(a, V);
  }
  return cudaGetLastError();
}

}  // namespace

// The serving step: p.num_seqs = B sequences of p.T tokens.
cudaError_t launch_step(const Params& p, float* state, const int32_t* slots, int num_slots, int K, int V, bool bf16,
                        cudaStream_t stream) {
  return launch(StepParams{p, state, slots, num_slots}, K, V, bf16, stream);
}

// The forward token by token (initial state -> final state).
cudaError_t launch_recurrent(const Params& p, int K, int V, bool bf16, cudaStream_t stream) {
  return launch(StepParams{p, nullptr, nullptr, 0}, K, V, bf16, stream);
}

}  // namespace gdr
}  // namespace kda
