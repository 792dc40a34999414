// glr.cu -- gated linear recurrence, per channel:  h_t = e^{g_t} h_{t-1} + x_t,  y_t = h_t,
// and its gradients:  lam_t = dy_t + mu_{t+1},  mu_t = e^{g_t} lam_t,  dx_t = lam_t,
// dg_t = mu_t h_{t-1}  (mu behind the last token: d_final; d_initial: mu of the first).
//
// Both are one scan  c -> e^{g_t} c + x_t  (backward, from the last token to the first:
// c -> e^{g_t} (c + dy_t)) over all tokens laid end to end, which starts anew at each sequence's
// first token from its initial value.  Bound by HBM: each input is read and each output
// written once, 8 bytes an element forward (bf16 with an fp32 gate), 14 backward.
//
// A CTA owns 32 channels and walks over the tokens in tiles of 128, the next tile on its way by TMA:
// 8 threads a row with 4 channels each, 8 neighbouring tokens a thread.  Any stretch of tokens
// acts on what enters it as c -> A c + H.  Each thread finds its stretch's (A, H), one warp folds
// the 16 of a channel in their order, and each thread goes through its tokens again, still in
// registers, from what enters them.  Where there are fewer channel tiles than places for CTAs, a
// cluster takes its step's tiles side by side, and the folding warps send each other their
// tile's (A, H) into shared memory.  Every fold goes over the same terms in the same order on
// every call, and the recurrence never leaves the chip.  All waits are bounded (2 s, or KDA_WAIT_LIMIT_NS, then the
// status says so; 2 s more for what is under way).
//
// Measured: 4 x 4096 x 4096 backward 152 us (939 MB, 91 % of the copy rate); 4096 x 4096 forward 34.5 (134 MB, 57 %;
// a kernel that only streams the same arrays 26); 46402 packed x 2048 forward with a bf16 gate 169 (570 MB, 50 %).
// What is short of the copy rate is a step's latency: 20 instructions a value by 8 to 12 warps an SM, two
// barriers, the fold and the exchange, some 1.7 us a step of two to three CTAs.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "layer_ops.cuh"
#include "pairs.cuh"
#include "sm103.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int kThreads = 128;
constexpr int kChannels = 32;              // of a tile: 4 a thread, 8 threads a row
constexpr int kEach = 8;                   // neighbouring tokens of a thread
constexpr int kSegs = kThreads / 8;        // threads along the tokens
constexpr int kTile = kSegs * kEach;       // tokens of a tile
constexpr int kMaxCluster = 16;

// 4 channels as they lie in memory
template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ float get(int j) const {
    const uint32_t w = j < 2 ? u.x : u.y;
    return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
  }
  __device__ __forceinline__ uint64_t pair(int i) const { return pack2f(get(2 * i), get(2 * i + 1)); }
};
template <>
struct Raw4<float> {
  float4 u;
  __device__ __forceinline__ float get(int j) const { return j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w; }
  __device__ __forceinline__ uint64_t pair(int i) const { return pack2f(get(2 * i), get(2 * i + 1)); }
};

// e^x of two values, x <= 88: 2^(x log2 e) with the product's rounding error put back to first order
// (without it a strong decay loses |x| 2^-24 of itself).  Below some -87.3, where e^x is no normal number any
// more, it is 0, as for -inf (expf, in the step, keeps the subnormals: 1e-38 of a state at most); NaN stays.
// Half the instructions of two calls of expf, and with them a fifth of the kernel's.
// The hardware's 2^y comes out low in the mean, by 0.27 of 2^-24 for x from -0.01 to -0.001 and by 0.32 down to -0.3,
// which a state that remembers hundreds of tokens adds up.  With kShift (0.42 of 2^-24) on y that is +0.03 and -0.03
// (expf: +0.08), and errors of states and gradients over some hundred tokens are half of what they were.  e^0 is
// 1 all the same, and for larger |x| the product's error takes the shift off again.
__device__ __forceinline__ uint64_t exp_pair(uint64_t x) {
  constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.925963e-8f, kLn2 = 0.693147181f, kShift = 0x1.bp-26f;
  float a, b;
  unpack2f(x, a, b);
  asm("max.NaN.f32 %0, %1, 0fC2D00000;" : "=f"(a) : "f"(a));
  asm("max.NaN.f32 %0, %1, 0fC2D00000;" : "=f"(b) : "f"(b));
  x = pack2f(a, b);
  const uint64_t L = pack2f(kLog2e, kLog2e);
  const uint64_t hi = fma2(x, L, pack2f(kShift, kShift));
  const uint64_t lo = fma2(x, pack2f(kLog2eRest, kLog2eRest), fma2(x, L, hi ^ 0x8000000080000000ull));
  unpack2f(hi, a, b);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(a));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(b));
  const uint64_t r = pack2f(a, b);
  return fma2(mul2(r, lo), pack2f(kLn2, kLn2), r);
}

// A thread's channels: c0 .. c0 + 3 (VEC: D % 4 = 0 and aligned rows), else c0, c0 + GAP, ...
template <bool VEC, int GAP, typename T>
__device__ __forceinline__ Raw4<T> load4(const T* row, int c0, int D) {
  Raw4<T> r;
  if constexpr (VEC) {
    if (c0 < D) r.u = __ldcs(reinterpret_cast<const decltype(r.u)*>(row + c0));
    else r.u = {};
  } else if constexpr (sizeof(T) == 2) {
    uint16_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = c0 + GAP * j < D ? __ldcs(reinterpret_cast<const unsigned short*>(row) + c0 + GAP * j) : uint16_t(0);
    r.u = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
  } else {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = c0 + GAP * j < D ? __ldcs(row + c0 + GAP * j) : 0.f;
    r.u = make_float4(v[0], v[1], v[2], v[3]);
  }
  return r;
}

template <bool VEC, int GAP, typename T>
__device__ __forceinline__ void store4(T* row, int c0, int D, const float (&v)[4]) {
  if constexpr (VEC) {
    if (c0 >= D) return;
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(row + c0) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      *reinterpret_cast<float4*>(row + c0) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + GAP * j < D) row[c0 + GAP * j] = from_f32<T>(v[j]);
  }
}

// A state row's 4 channels (fp32; zeros without one); through element loads, as states need 4-byte
// alignment only and a sequence has one.
template <bool VEC, int GAP>
__device__ __forceinline__ void load_state(float (&v)[4], const float* states, int seq, int c0, int D) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = VEC ? c0 + j : c0 + GAP * j;
    v[j] = states && c < D ? states[static_cast<size_t>(seq) * D + c] : 0.f;
  }
}
template <bool VEC, int GAP>
__device__ __forceinline__ void store_state(float* states, int seq, int c0, int D, const float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = VEC ? c0 + j : c0 + GAP * j;
    if (c < D) states[static_cast<size_t>(seq) * D + c] = v[j];
  }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// 2 floats into the same place of another CTA of the cluster, counted by the barrier at `bar` there (a
// store and a releasing arrive would first wait for every store to HBM that the thread has under way)
__device__ __forceinline__ void store_remote(float2* mine, uint64_t* bar, uint32_t rank, float2 v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                   mapa_shared(smem_u32(mine), rank)),
               "f"(v.x), "f"(v.y), "r"(mapa_shared(smem_u32(bar), rank))
               : "memory");
}

// A wait for what is under way and comes by itself (copies that were issued, a step's maps, which every CTA of a
// cluster sends).  Longer than the call's limit it is reported, and waited for all the same, so that nothing is
// left under way when a block ends; false if it has not come kDrainNs later either, which takes a
// fault of the device.  try_wait may suspend a thread until the phase completes, so a limit below kPollNs is
// kept by looks that do not; the timer advances in steps of up to kTickNs, so one below that is over at once.
constexpr unsigned long long kDrainNs = 2000000000ull, kPollNs = 20000ull, kTickNs = 1000ull;
template <bool CLUSTER>
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, unsigned long long limit_ns, uint32_t* status) {
  const unsigned long long t0 = globaltimer_ns();
  bool late = false;
#pragma unroll 1
  do {
    const unsigned long long t = globaltimer_ns() - t0;
    if (t + kTickNs > limit_ns && !late) {
      late = true;
      atomicOr(status, kStatusTimeout);
    }
    if (t > kDrainNs && t - kDrainNs > limit_ns) return false;
  } while (!(limit_ns < kPollNs ? (CLUSTER ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity))
                                : (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))));
  return true;
}
template <bool CLUSTER>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, unsigned long long limit_ns, uint32_t* status) {
  if (limit_ns >= kPollNs && (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) return true;
  return wait_longer<CLUSTER>(bar, parity, limit_ns, status);
}

// The sequence around a token: its number and tokens [begin, end); empty where the token is in none.
struct Span {
  int seq, begin, end;
};
constexpr int kMostCu = 2048;              // entries of cu_seqlens that a CTA keeps in shared memory
__device__ __forceinline__ void locate(Span& s, const Params& p, const int32_t* cu, int t) {
  if (cu == nullptr) {
    s.seq = t / p.T;
    s.begin = s.seq * p.T;
    s.end = s.begin + p.T;
    return;
  }
  int lo = 0, hi = p.num_seqs;               // the last one that starts at or before t, whatever cu holds
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  s.seq = lo;
  s.begin = cu[lo];
  s.end = cu[lo + 1];
  if (t < s.begin || t >= s.end) s.begin = s.end = -1;
}

// The number of the sequence that holds token t, for threads with several starts or ends.  (A function, as it
// stands at each of a thread's tokens in both passes: written out, 4096 x 4096 took 35.1 us for 34.3, 46402 packed x 2048 171 for 167.5.)
__device__ __noinline__ int sequence_of(const int32_t* cu, int num_seqs, int T, int t) {
  if (cu == nullptr) return t / T;
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

constexpr uint64_t kOnes = 0x3F8000003F800000ull;
// An A of -1 marks a stretch in which the scan started anew, so that nothing of what enters it gets
// through (an A is a product of exponentials, never below 0; multiplying by 0 would let a NaN through).
constexpr float kClosed = -1.f;
__device__ __forceinline__ float apply(float A, float c, float H) { return A == kClosed ? H : fmaf(A, c, H); }

struct Args {
  Params p;
  int cluster;
  CUtensorMap g, x, y;   // boxes of 32 channels x 128 tokens
};

template <typename IO, typename G, bool BWD>
constexpr int stage_bytes() { return kTile * kChannels * static_cast<int>(sizeof(G) + (BWD ? 2 : 1) * sizeof(IO)); }
constexpr int maps_bytes(int cluster) { return 2 * cluster * kChannels * static_cast<int>(sizeof(float2)); }
// CTAs an SM: what registers (a thread's tokens) and two stages each leave room for.
template <typename IO, bool BWD>
constexpr int ctas_each() { return sizeof(IO) == 2 ? (BWD ? 3 : 4) : (BWD ? 2 : 3); }

// TMA: rows are multiples of 16 bytes and aligned; else threads load their own elements, a tile at a time.
template <typename IO, typename G, bool BWD, bool TMA>
__global__ void __launch_bounds__(kThreads, ctas_each<IO, BWD>()) glr_scan_kernel(const __grid_constant__ Args args) {
  constexpr int R = kEach, GAP = 8;
  using RawIO = decltype(Raw4<IO>::u);
  using RawG = decltype(Raw4<G>::u);
  extern __shared__ __align__(128) uint8_t stages[];        // [2] of g, x, y: [128 tokens][32 channels]
  __shared__ __align__(16) float seg_a[kSegs][kChannels], seg_h[kSegs][kChannels];   // then what enters a stretch, over its H
  __shared__ uint64_t full[2], arrived[2];
  const Params& p = args.p;
  const int cluster = args.cluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, seg = tid >> 3, cq = lane & 7;
  const int rank = blockIdx.x % cluster, ct = blockIdx.x / cluster;
  const int c0 = ct * kChannels + (TMA ? 4 * cq : cq), D = p.D;
  const int total = static_cast<int>(p.tokens);
  const int steps = static_cast<int>((p.tokens + static_cast<long>(cluster) * kTile - 1) / (static_cast<long>(cluster) * kTile));
  const G* pg = static_cast<const G*>(p.g);
  const IO* px = static_cast<const IO*>(p.x);
  const IO* py = static_cast<const IO*>(p.y);
  auto tile_at = [&](int n) { return (static_cast<long>(n) * cluster + rank) * kTile; };   // in scan order
  auto stage_g = [&](int n) { return reinterpret_cast<G*>(stages + (n & 1) * stage_bytes<IO, G, BWD>()); };
  auto stage_x = [&](int n) { return reinterpret_cast<IO*>(stage_g(n) + kTile * kChannels); };
  auto stage_y = [&](int n) { return stage_x(n) + kTile * kChannels; };
  auto maps = [&](int n, int q) {                            // the cluster's tiles of a step: [2][cluster][32 channels]
    return reinterpret_cast<float2*>(stages + (TMA ? 2 * stage_bytes<IO, G, BWD>() : 0)) + ((n & 1) * cluster + q) * kChannels;
  };
  auto issue = [&](int n) {                                  // one thread: a tile's inputs on their way
    const long at = tile_at(n);
    if (n >= steps || at >= total) return;
    const int row = static_cast<int>(BWD ? total - at - kTile : at), col = ct * kChannels;
    uint64_t* bar = &full[n & 1];
    mbar_arrive_expect_tx(bar, stage_bytes<IO, G, BWD>());
    tma_load_2d(stage_g(n), &args.g, bar, col, row);
    tma_load_2d(stage_x(n), &args.x, bar, col, row);
    if constexpr (BWD) tma_load_2d(stage_y(n), &args.y, bar, col, row - 1);   // (each token's state before it)
  };

  const int32_t* cu = p.cu;
  if (cu && p.num_seqs < kMostCu) {
    int32_t* kept = reinterpret_cast<int32_t*>(maps(0, 0) + 2 * cluster * kChannels);
    for (int i = tid; i <= p.num_seqs; i += kThreads) kept[i] = p.cu[i];
    cu = kept;
  }
  bool lost = false;                           // a wait has been given up: no more copies, and no exchange
  if (tid == 0) {
    if (blockIdx.x == 0) *p.status = 0u;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&arrived[i], 1);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (cluster > 1) cluster_arrive();           // (every CTA is ready before another one writes into it)
  if (TMA && tid == 0) {
    issue(0);
    issue(1);
  }
  if (cluster > 1) cluster_wait();
  float carry = 0.f;                           // the folding warp's: what enters the step, a channel a lane
  Span span{0, -1, -1};
  for (int n = 0; n < steps; ++n) {
    const long pos = tile_at(n) + seg * R;
    auto token = [&](int r) { return static_cast<int>(BWD ? total - 1 - pos - r : pos + r); };
    if (TMA && !lost && tile_at(n) < total && !wait_phase<false>(&full[n & 1], n >> 1 & 1, p.wait_ns, p.status)) lost = true;
    Raw4<IO> x[R], y[BWD ? R : 1];
    Raw4<G> g[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (TMA) {
        const int at = (BWD ? kTile - 1 - seg * R - r : seg * R + r) * kChannels + 4 * cq;
        g[r].u = *reinterpret_cast<const RawG*>(stage_g(n) + at);
        x[r].u = *reinterpret_cast<const RawIO*>(stage_x(n) + at);
        if constexpr (BWD) y[r].u = *reinterpret_cast<const RawIO*>(stage_y(n) + at);
      } else {
        const bool there = pos + r < total;
        const size_t row = static_cast<size_t>(there ? token(r) : 0) * D;
        g[r] = load4<false, GAP>(pg + row, c0, there ? D : 0);
        x[r] = load4<false, GAP>(px + row, c0, there ? D : 0);
        if constexpr (BWD) y[r] = load4<false, GAP>(py + (row > 0 ? row - D : 0), c0, there && row > 0 ? D : 0);
      }
    }
    // Tokens of a sequence's inside need no look at where sequences start and end.  Else, a bit each:
    // the scan starts anew at a token, ends with it, and the token is one of a sequence.
    uint32_t starts = 0, ends = 0, live = 0;
    int start_seq = 0, end_seq = 0;                          // of the thread's last start and end
    const int t_lo = BWD ? token(R - 1) : token(0), t_hi = BWD ? token(0) : token(R - 1);
    if (pos < total && (token(0) < span.begin || token(0) >= span.end)) locate(span, p, cu, token(0));
    const bool plain = __all_sync(0xFFFFFFFFu, pos + R <= total && t_lo > span.begin && t_hi < span.end - 1);
    if (!plain) {
      for (int r = 0; r < R && pos + r < total; ++r) {
        const int t = token(r);
        if (t < span.begin || t >= span.end) locate(span, p, cu, t);
        if (span.end < 0) continue;
        live |= 1u << r;
        if (t == (BWD ? span.end - 1 : span.begin)) {
          starts |= 1u << r;
          start_seq = span.seq;
        }
        if (t == (BWD ? span.begin : span.end - 1)) {
          ends |= 1u << r;
          end_seq = span.seq;
        }
      }
    }

    // (the last value that the scan started from is kept: where that sequence goes on beyond this thread, its
    // array may hold the final state by the time the tokens are gone through again)
    uint64_t a[R][2], A[2] = {kOnes, kOnes}, H[2] = {0ull, 0ull}, from[2] = {0ull, 0ull};
    if (plain) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[r][i] = exp_pair(g[r].pair(i));
          A[i] = r == 0 ? a[r][i] : mul2(A[i], a[r][i]);
          if constexpr (BWD) H[i] = mul2(a[r][i], r == 0 ? x[r].pair(i) : add2(H[i], x[r].pair(i)));
          else H[i] = r == 0 ? x[r].pair(i) : fma2(a[r][i], H[i], x[r].pair(i));
        }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!(live >> r & 1)) {                // (a token of no sequence leaves everything as it is)
          a[r][0] = a[r][1] = kOnes;
          continue;
        }
        if (starts >> r & 1) {
          Span s{start_seq, 0, 0};
          if (starts >> r != 1u) s.seq = sequence_of(cu, p.num_seqs, p.T, token(r));
          float h[4];
          load_state<TMA, GAP>(h, p.init, s.seq, c0, D);
          H[0] = from[0] = pack2f(h[0], h[1]);
          H[1] = from[1] = pack2f(h[2], h[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[r][i] = exp_pair(g[r].pair(i));
          A[i] = mul2(A[i], a[r][i]);
          H[i] = BWD ? mul2(a[r][i], add2(H[i], x[r].pair(i))) : fma2(a[r][i], H[i], x[r].pair(i));
        }
      }
      if (starts) A[0] = A[1] = pack2f(kClosed, kClosed);
    }
    *reinterpret_cast<ulonglong2*>(&seg_a[seg][4 * cq]) = make_ulonglong2(A[0], A[1]);
    *reinterpret_cast<ulonglong2*>(&seg_h[seg][4 * cq]) = make_ulonglong2(H[0], H[1]);
    __syncthreads();
    if (TMA && tid == kThreads - 1 && !lost) issue(n + 2);   // (the stage has been read)
    if (warp == 0) {
      float c = carry, sa[kSegs], sh[kSegs];
#pragma unroll
      for (int i = 0; i < kSegs; ++i) {
        sa[i] = seg_a[i][lane];
        sh[i] = seg_h[i][lane];
      }
      if (cluster > 1) {
        float TA = 1.f, TH = 0.f;
#pragma unroll
        for (int i = 0; i < kSegs; ++i) {
          TH = apply(sa[i], TH, sh[i]);
          TA = sa[i] == kClosed || TA == kClosed ? kClosed : TA * sa[i];
        }
        if (!lost) {                             // (after a wait that gave up, the others' waits give up too)
          for (int q = 0; q < cluster; ++q) store_remote(maps(n, rank) + lane, &arrived[n & 1], q, make_float2(TA, TH));
          if (lane == 0) mbar_arrive_expect_tx_relaxed(&arrived[n & 1], cluster * kChannels * sizeof(float2));
        }
        if (!lost && !wait_phase<true>(&arrived[n & 1], n >> 1 & 1, p.wait_ns, p.status)) lost = true;
        for (int q = 0; q < cluster; ++q) {
          const float2 m = maps(n, q)[lane];
          if (q == rank) c = carry;
          carry = apply(m.x, carry, m.y);
        }
      }
#pragma unroll
      for (int i = 0; i < kSegs; ++i) {
        seg_h[i][lane] = c;
        c = apply(sa[i], c, sh[i]);
      }
      if (cluster == 1) carry = c;
    }
    __syncthreads();

    // the tokens again, from what enters them
    const ulonglong2 in = *reinterpret_cast<const ulonglong2*>(&seg_h[seg][4 * cq]);
    uint64_t c[2] = {in.x, in.y};
    if (plain) {
      long at = static_cast<long>(token(0)) * D;
      const long stride = BWD ? -static_cast<long>(D) : D;
#pragma unroll
      for (int r = 0; r < R; ++r, at += stride) {
        float out[4];
        if constexpr (BWD) {
          float dg[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t lam = add2(c[i], x[r].pair(i));
            unpack2f(lam, out[2 * i], out[2 * i + 1]);
            c[i] = mul2(a[r][i], lam);
            unpack2f(mul2(c[i], y[r].pair(i)), dg[2 * i], dg[2 * i + 1]);
          }
          store4<TMA, GAP>(static_cast<G*>(p.dg) + at, c0, D, dg);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            c[i] = fma2(a[r][i], c[i], x[r].pair(i));
            unpack2f(c[i], out[2 * i], out[2 * i + 1]);
          }
        }
        store4<TMA, GAP>(static_cast<IO*>(p.out) + at, c0, D, out);
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!(live >> r & 1)) continue;
        const size_t row = static_cast<size_t>(token(r)) * D;
        const bool end = ends >> r & 1;
        Span s{end_seq, 0, 0};
        if ((end && ends >> r != 1u) || (starts >> r & 1 && starts >> r != 1u)) s.seq = sequence_of(cu, p.num_seqs, p.T, token(r));
        if (starts >> r == 1u) {
          c[0] = from[0];
          c[1] = from[1];
        } else if (starts >> r & 1) {
          float h[4];
          load_state<TMA, GAP>(h, p.init, s.seq, c0, D);
          c[0] = pack2f(h[0], h[1]);
          c[1] = pack2f(h[2], h[3]);
        }
        float out[4], last[4];
        if constexpr (BWD) {
          float dg[4];
          uint64_t before[2] = {y[r].pair(0), y[r].pair(1)};
          if (end) {
            float h[4];
            load_state<TMA, GAP>(h, p.h0, s.seq, c0, D);
            before[0] = pack2f(h[0], h[1]);
            before[1] = pack2f(h[2], h[3]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t lam = add2(c[i], x[r].pair(i));
            unpack2f(lam, out[2 * i], out[2 * i + 1]);
            c[i] = mul2(a[r][i], lam);
            unpack2f(mul2(c[i], before[i]), dg[2 * i], dg[2 * i + 1]);
            unpack2f(c[i], last[2 * i], last[2 * i + 1]);
          }
          store4<TMA, GAP>(static_cast<G*>(p.dg) + row, c0, D, dg);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            c[i] = fma2(a[r][i], c[i], x[r].pair(i));
            unpack2f(c[i], out[2 * i], out[2 * i + 1]);
            unpack2f(c[i], last[2 * i], last[2 * i + 1]);
          }
        }
        store4<TMA, GAP>(static_cast<IO*>(p.out) + row, c0, D, out);
        if (end && p.fin) store_state<TMA, GAP>(p.fin, s.seq, c0, D, last);
      }
    }
  }

  // sequences without tokens keep their initial value; one block checks cu_seqlens
  if (p.cu) {
    for (int s0 = (rank * (kThreads / 32) + warp) * 32; s0 < p.num_seqs; s0 += kThreads * cluster) {
      const int q = s0 + lane;
      const bool none = q < p.num_seqs && p.cu[q + 1] <= p.cu[q] && p.fin;
      const int c = ct * kChannels + lane;
      for (uint32_t m = __ballot_sync(0xFFFFFFFFu, none); m; m &= m - 1) {
        const size_t at = static_cast<size_t>(s0 + __ffs(m) - 1) * D + c;
        if (c < D) p.fin[at] = p.init ? p.init[at] : 0.f;
      }
    }
    if (blockIdx.x == 0) {
      bool bad = false;
      for (int q = tid; q < p.num_seqs; q += kThreads) {
        const int b = p.cu[q], e = p.cu[q + 1];
        bad |= b < 0 || e < b || e > total || (q == 0 && b != 0) || (q == p.num_seqs - 1 && e != total);
      }
      if (bad) atomicOr(p.status, kStatusBounds);
    }
  }
  if (cluster > 1) {                           // (nobody writes into a CTA that has ended)
    cluster_arrive();
    cluster_wait();
  }
}

// The serving step: 4 channels a thread, the state in registers between its load and its store.  Bound by HBM for
// thousands of requests, by the call itself below (128 x 4096, 8 MB: 12 us among others, 1.2 at the copy rate).
template <typename IO, typename G, bool VEC>
__global__ void __launch_bounds__(128) glr_step_kernel(const StepParams p) {
  const int b = blockIdx.y, D = p.D;
  const int c0 = VEC ? 4 * (blockIdx.x * 128 + threadIdx.x) : blockIdx.x * 512 + (threadIdx.x >> 5) * 128 + (threadIdx.x & 31);
  const size_t row0 = static_cast<size_t>(b) * p.T * D;
  const IO* x = static_cast<const IO*>(p.x) + row0;
  const G* g = static_cast<const G*>(p.g) + row0;
  IO* y = static_cast<IO*>(p.y) + row0;
  Raw4<IO> xr = load4<VEC, 32>(x, c0, D);
  Raw4<G> gr = load4<VEC, 32>(g, c0, D);
  int slot = b;
  if (p.slots) {
    slot = p.slots[b];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot >= p.num_slots && p.status && threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
      const float zero[4] = {};
      for (int t = 0; t < p.T; ++t) store4<VEC, 32>(y + static_cast<size_t>(t) * D, c0, D, zero);
      return;
    }
  }
  float* state = p.state + static_cast<size_t>(slot) * D;
  float h[4];
  if constexpr (VEC) {
    const float4 u = c0 < D ? *reinterpret_cast<const float4*>(state + c0) : make_float4(0.f, 0.f, 0.f, 0.f);
    h[0] = u.x; h[1] = u.y; h[2] = u.z; h[3] = u.w;
  } else {
    load_state<false, 32>(h, state, 0, c0, D);
  }
  for (int t = 0; t < p.T; ++t) {
    const Raw4<IO> xt = xr;
    const Raw4<G> gt = gr;
    if (t + 1 < p.T) {
      xr = load4<VEC, 32>(x + static_cast<size_t>(t + 1) * D, c0, D);
      gr = load4<VEC, 32>(g + static_cast<size_t>(t + 1) * D, c0, D);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = fmaf(expf(gt.get(j)), h[j], xt.get(j));
    store4<VEC, 32>(y + static_cast<size_t>(t) * D, c0, D, h);
  }
  if constexpr (VEC) {
    if (c0 < D) *reinterpret_cast<float4*>(state + c0) = make_float4(h[0], h[1], h[2], h[3]);
  } else {
    store_state<false, 32>(state, 0, c0, D, h);
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

template <typename T>
bool make_map(CUtensorMap* m, const void* base, int D, long tokens) {
  const auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * sizeof(T)};
  const cuuint32_t box[2] = {kChannels, kTile}, step[2] = {1, 1};
  return enc(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base),
             dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename IO, typename G, bool BWD, bool TMA>
cudaError_t launch_scan(const Params& p, cudaStream_t st) {
  constexpr int ring = TMA ? 2 * stage_bytes<IO, G, BWD>() : 0;
  const auto kernel = glr_scan_kernel<IO, G, BWD, TMA>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  {
    static bool raised[64] = {};       // (a race raises it twice, to the same value)
    if (dev < 0 || dev >= 64 || !raised[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring + maps_bytes(kMaxCluster) + kMostCu * sizeof(int32_t));
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) raised[dev] = true;
    }
  }
  Args args{};
  args.p = p;
  if (TMA && p.tokens > 0 &&
      (!make_map<G>(&args.g, p.g, p.D, p.tokens) || !make_map<IO>(&args.x, p.x, p.D, p.tokens) ||
       (BWD && !make_map<IO>(&args.y, p.y, p.D, p.tokens))))
    return cudaErrorInvalidValue;
  const size_t cu_bytes = p.cu && p.num_seqs < kMostCu ? (p.num_seqs + 1) * sizeof(int32_t) : 0;
  const long cts = (p.D + kChannels - 1) / kChannels, tiles = (p.tokens + kTile - 1) / kTile;
  args.cluster = 1;
  if (tiles > 1) {
    // CTAs of a cluster share a channel tile's tokens: as many as can all run at once, up to 8 CTAs for 3 SMs,
    // and with more bytes an element (fp32, backward) 2 an SM.  us a call for 1, 2, 3, 4, 6 and 8 CTAs a cluster:
    // 4096 x 4096 bf16 (128 channel tiles) 46, 39, 36.5, 34.4; 46402 x 2048 (64) 356, 249, 208, 152, 133, 139;
    // 8192 x 8192 (256) 100, 108; 16384 x 4096 backward 190, 161, 184, 191; 65536 x 128 (4) 489, 342, 245, 178,
    // 129, 98 and 61 for 16.
    const long most = sizeof(IO) == 2 && !BWD ? 8 * sms / 3 : 2 * sms;
    // clusters of a size that run at once, by device and by the KB that cu_seqlens takes beside the tiles (fp32
    // backward: two CTAs an SM in clusters of 16 with 4 KB of it, of 9 with 8 KB)
    static int room[64][kMostCu / 256 + 1][kMaxCluster + 1] = {};
    const int kb = static_cast<int>((cu_bytes + 1023) / 1024);
    for (int c = tiles < kMaxCluster ? static_cast<int>(tiles) : kMaxCluster; c > 1; --c) {
      if (cts * c > most) continue;
      int fit = dev >= 0 && dev < 64 ? room[dev][kb][c] : 0;
      if (fit == 0) {
        cudaLaunchAttribute shape;
        shape.id = cudaLaunchAttributeClusterDimension;
        shape.val.clusterDim.x = c;
        shape.val.clusterDim.y = shape.val.clusterDim.z = 1;
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(c);
        q.blockDim = dim3(kThreads);
        q.dynamicSmemBytes = ring + maps_bytes(c) + kb * 1024;
        q.attrs = &shape;
        q.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&fit, kernel, &q);
        if (e != cudaSuccess) return e;
        if (fit == 0) fit = -1;
        if (dev >= 0 && dev < 64) room[dev][kb][c] = fit;
      }
      if (fit >= cts) {
        args.cluster = c;
        break;
      }
    }
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = args.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cts * args.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = ring + maps_bytes(args.cluster) + cu_bytes;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

template <typename IO, typename G>
cudaError_t launch_types(const Params& p, bool backward, cudaStream_t st) {
  const bool tma = p.D * sizeof(IO) % 16 == 0 && p.D * sizeof(G) % 16 == 0 && aligned(p.x, 16) && aligned(p.y, 16) &&
                   aligned(p.out, 16) && aligned(p.g, 16) && aligned(p.dg, 16);
  if (backward) return tma ? launch_scan<IO, G, true, true>(p, st) : launch_scan<IO, G, true, false>(p, st);
  return tma ? launch_scan<IO, G, false, true>(p, st) : launch_scan<IO, G, false, false>(p, st);
}

template <typename IO, typename G>
cudaError_t launch_step_types(const StepParams& p, cudaStream_t st) {
  const bool vec = p.D % 4 == 0 && aligned(p.x, 4 * sizeof(IO)) && aligned(p.y, 4 * sizeof(IO)) && aligned(p.g, 4 * sizeof(G)) &&
                   aligned(p.state, 16);
  for (long b = 0; b < p.B; b += 65535) {       // (a grid's second dimension)
    StepParams q = p;
    const size_t row = static_cast<size_t>(b) * p.T * p.D;
    q.x = static_cast<const IO*>(p.x) + row;
    q.g = static_cast<const G*>(p.g) + row;
    q.y = static_cast<IO*>(p.y) + row;
    if (p.slots) q.slots = p.slots + b;
    else q.state = p.state + static_cast<size_t>(b) * p.D;
    q.B = static_cast<int>(p.B - b < 65535 ? p.B - b : 65535);
    const dim3 grid((p.D + 511) / 512, q.B);
    if (vec) glr_step_kernel<IO, G, true><<<grid, 128, 0, st>>>(q);
    else glr_step_kernel<IO, G, false><<<grid, 128, 0, st>>>(q);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch(const Params& p, bool backward, bool bf16, bool gate_bf16, cudaStream_t st) {
  if (p.tokens == 0 && !p.cu) {       // no tokens: the initial values pass through
    const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st);
    if (e != cudaSuccess || !p.fin || p.fin == p.init) return e;
    const size_t n = static_cast<size_t>(p.num_seqs) * p.D * sizeof(float);
    return p.init ? cudaMemcpyAsync(p.fin, p.init, n, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(p.fin, 0, n, st);
  }
  if (bf16) return gate_bf16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(p, backward, st) : launch_types<__nv_bfloat16, float>(p, backward, st);
  return gate_bf16 ? launch_types<float, __nv_bfloat16>(p, backward, st) : launch_types<float, float>(p, backward, st);
}

cudaError_t launch_step(const StepParams& p, bool bf16, bool gate_bf16, cudaStream_t st) {
  if (bf16) return gate_bf16 ? launch_step_types<__nv_bfloat16, __nv_bfloat16>(p, st) : launch_step_types<__nv_bfloat16, float>(p, st);
  return gate_bf16 ? launch_step_types<float, __nv_bfloat16>(p, st) : launch_step_types<float, float>(p, st);
}

}  // namespace glr
}  // namespace kda
