// gdr_step.cu -- the gated delta rule token by token, fp32 on CUDA cores: the serving step
// (states read and updated in place, optionally in a pool) and the forward for fp32 I/O.
//
// Per sequence and value head, with one gate per token (scalar e^{g_t}):
//     P   = e^{g_t} S_{t-1}
//     S_t = P + beta_t k_t (v_t - P^T k_t)^T
//     o_t = scale S_t^T q_t
// One CTA of 8 warps per (sequence, value head): a warp reads whole rows of the state (512
// contiguous bytes at V = 128; a thread holds 4 columns of K / 8 or K / 16 rows in
// registers, every load issued before the first use), sums over its rows in registers and
// over the warps through shared memory, two barriers a token.
// Bound: at T = 1 a call moves the state once each way, 128 KiB per (sequence, value head)
// at K = V = 128, and next to nothing else: HBM bandwidth, or latency for a few heads.  128
// sequences x 32 heads, 537 MB: 89 us, 89 % of the copy bandwidth.  (A
// warp per 16 columns, with no barrier at all, reads 64-byte pieces of the rows and reached
// 72 % of the copy bandwidth at 128 sequences x 32 heads, 111.5 us.)
#include "gdr_common.cuh"

namespace kda {
namespace gdr {
namespace {

constexpr int NW = 8;  // warps of a CTA

struct StepParams {
  Params p;
  float* state;          // serving step: [B or num_slots, HV, K, V], in place; else null
  const int32_t* slots;  // [B] or null
  int num_slots;
};

template <typename IO, int K, int V>
__global__ void __launch_bounds__(32 * NW) gdr_recurrent_kernel(const StepParams a) {
  constexpr int TPR = V / 4;            // threads of a row
  constexpr int RPW = 32 / TPR;         // rows of a warp at once
  constexpr int G = NW * RPW;           // row groups of the CTA
  constexpr int R = K / G;              // rows of a thread
  __shared__ __align__(16) float sk[2][K], sq[2][K], sv[2][V], part[2][NW][V];
  __shared__ float sg[2][2];
  const Params& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.x / p.HV, hv = blockIdx.x % p.HV, hk = hv / (p.HV / p.H);
  const int grp = warp * RPW + lane / TPR, col = 4 * (lane % TPR);

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
  if (a.state) {
    src = dst = a.state;
    if (a.slots) {
      at = a.slots[seq];
      if (at < 0 || at >= a.num_slots) {  // an empty row: no state, o = 0
        if (at >= a.num_slots && p.status && tid == 0) atomicOr(p.status, kStatusBounds);
        for (int t = 0; t < len; ++t)
          for (int c = tid; c < V; c += 32 * NW) out[(static_cast<size_t>(tok0 + t) * p.HV + hv) * V + c] = from_f32<IO>(0.f);
        return;
      }
    }
  }
  // thread's rows: grp + G i
  const size_t off = (static_cast<size_t>(at) * p.HV + hv) * K * V + static_cast<size_t>(grp) * V + col;
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    s[i] = src ? *reinterpret_cast<const float4*>(src + off + static_cast<size_t>(i) * G * V) : make_float4(0.f, 0.f, 0.f, 0.f);

  // a token's inputs into buffer b; staged one token ahead
  auto stage = [&](int t, int b) {
    const size_t tok = static_cast<size_t>(tok0 + t);
    if (tid < K) {
      sk[b][tid] = to_f32(k[(tok * p.H + hk) * K + tid]);
      sq[b][tid] = to_f32(q[(tok * p.H + hk) * K + tid]);
    }
    if (tid >= 32 * NW - V) sv[b][tid - (32 * NW - V)] = to_f32(v[(tok * p.HV + hv) * V + tid - (32 * NW - V)]);
    if (tid == 0) sg[b][0] = expf(p.g[tok * p.HV + hv]);
    if (tid == 32) sg[b][1] = p.beta[tok * p.HV + hv];
  };
  // the warp's sum over its rows, then the CTA's share
  auto put_sum = [&](float4 x, float (&to)[NW][V]) {
    if constexpr (RPW == 2) {
      x.x += __shfl_xor_sync(0xFFFFFFFFu, x.x, 16);
      x.y += __shfl_xor_sync(0xFFFFFFFFu, x.y, 16);
      x.z += __shfl_xor_sync(0xFFFFFFFFu, x.z, 16);
      x.w += __shfl_xor_sync(0xFFFFFFFFu, x.w, 16);
    }
    if (lane < TPR) *reinterpret_cast<float4*>(&to[warp][col]) = x;
  };
  auto total = [&](const float (&from)[NW][V]) {
    float4 x = *reinterpret_cast<const float4*>(&from[0][col]);
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(&from[w][col]);
      x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
    }
    return x;
  };
  auto emit = [&](int t) {
    if (warp != 0 || lane >= TPR) return;
    const float4 o = total(part[1]);
    IO* op = out + (static_cast<size_t>(tok0 + t) * p.HV + hv) * V + col;
    op[0] = from_f32<IO>(p.scale * o.x);
    op[1] = from_f32<IO>(p.scale * o.y);
    op[2] = from_f32<IO>(p.scale * o.z);
    op[3] = from_f32<IO>(p.scale * o.w);
  };
  if (len > 0) stage(0, 0);
  __syncthreads();
  for (int t = 0; t < len; ++t) {
    const int b = t & 1;
    const float e = sg[b][0], be = sg[b][1];
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float kd = sk[b][grp + G * i];
      s[i].x *= e; s[i].y *= e; s[i].z *= e; s[i].w *= e;
      u.x = fmaf(kd, s[i].x, u.x); u.y = fmaf(kd, s[i].y, u.y);
      u.z = fmaf(kd, s[i].z, u.z); u.w = fmaf(kd, s[i].w, u.w);
    }
    put_sum(u, part[0]);
    if (t + 1 < len) stage(t + 1, b ^ 1);
    if (t > 0) emit(t - 1);
    __syncthreads();
    u = total(part[0]);
    const float4 vv = *reinterpret_cast<const float4*>(&sv[b][col]);
    const float4 d = make_float4(be * (vv.x - u.x), be * (vv.y - u.y), be * (vv.z - u.z), be * (vv.w - u.w));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float kd = sk[b][grp + G * i], qd = sq[b][grp + G * i];
      s[i].x = fmaf(kd, d.x, s[i].x); s[i].y = fmaf(kd, d.y, s[i].y);
      s[i].z = fmaf(kd, d.z, s[i].z); s[i].w = fmaf(kd, d.w, s[i].w);
      o.x = fmaf(qd, s[i].x, o.x); o.y = fmaf(qd, s[i].y, o.y);
      o.z = fmaf(qd, s[i].z, o.z); o.w = fmaf(qd, s[i].w, o.w);
    }
    put_sum(o, part[1]);
    __syncthreads();
  }
  if (len > 0) emit(len - 1);
  if (dst) {
#pragma unroll
    for (int i = 0; i < R; ++i) *reinterpret_cast<float4*>(dst + off + static_cast<size_t>(i) * G * V) = s[i];
  }
}

template <typename IO>
void launch_io(const StepParams& a, int K, int V, unsigned grid, cudaStream_t st) {
  if (K == 128 && V == 128) gdr_recurrent_kernel<IO, 128, 128><<<grid, 32 * NW, 0, st>>>(a);
  else if (K == 128) gdr_recurrent_kernel<IO, 128, 64><<<grid, 32 * NW, 0, st>>>(a);
  else if (V == 128) gdr_recurrent_kernel<IO, 64, 128><<<grid, 32 * NW, 0, st>>>(a);
  else gdr_recurrent_kernel<IO, 64, 64><<<grid, 32 * NW, 0, st>>>(a);
}

cudaError_t launch(const StepParams& a, int K, int V, bool bf16, cudaStream_t st) {
  const long units = static_cast<long>(a.p.num_seqs) * a.p.HV;
  if (units == 0) return cudaSuccess;
  if (bf16) launch_io<__nv_bfloat16>(a, K, V, static_cast<unsigned>(units), st);
  else launch_io<float>(a, K, V, static_cast<unsigned>(units), st);
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
