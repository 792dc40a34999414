// glr.cu -- gated linear recurrence, per channel:  h_t = e^{g_t} h_{t-1} + x_t,  y_t = h_t,
// and its gradients:  lam_t = dy_t + mu_{t+1},  mu_t = e^{g_t} lam_t,  dx_t = lam_t,
// dg_t = mu_t h_{t-1}  (mu behind the last token: d_final; d_initial: mu of the first).
//
// Both are one scan  c -> e^{g_t} c + x_t  (backward, from the last token to the first:
// c -> e^{g_t} (c + dy_t)) over all tokens laid end to end, which starts anew at each sequence's
// first token from its initial value.  Bound by HBM: each input is read and each output
// written once, 8 bytes an element forward (bf16 with an fp32 gate), 14 backward.
//
// A CTA owns 32 channels and walks over the tokens in tiles of 128 (64 in the fp32 backward): 8
// threads a row with 4 channels each, 4 neighbouring tokens a thread.  Any stretch of tokens acts on
// what enters it as c -> A c + H; a thread's (A, H) join over the warp by shuffles, over the warps
// through shared memory.  Where there are fewer channel tiles than places for CTAs, a cluster takes
// its step's tiles side by side and each CTA writes its (A, H) into the others' shared memory: one
// cluster barrier a step, and it is waited for a step later, under the next tile's sums.  So a
// tile's inputs lie in a ring in shared memory from their load, one step ahead, until what enters
// them is known, and the recurrence itself never leaves the chip.  Every fold goes over the same
// terms in the same order on every call.
#include "layer_ops.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChannels = 32;             // of a tile: 4 a thread, 8 threads a row
constexpr int kRows = kThreads / 8;       // threads along the tokens, each with R neighbours
constexpr int kMaxCluster = 8;

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
};
template <>
struct Raw4<float> {
  float4 u;
  __device__ __forceinline__ float get(int j) const { return j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w; }
};

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

// 16 or 8 bytes to shared memory without passing through registers; the issuing thread alone reads
// them, so waiting for its own groups is all it needs.  Zeros where there is nothing to copy.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool there) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst)), bytes = there ? BYTES : 0;
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// 4 floats into the same place of another CTA of the cluster
__device__ __forceinline__ void store_remote(float* mine, uint32_t rank, const float (&v)[4]) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  uint32_t to;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}

// The sequence around a token: its number and tokens [begin, end); empty where the token is in none.
struct Span {
  int seq, begin, end;
};
__device__ __forceinline__ void locate(Span& s, const Params& p, int t) {
  if (p.cu == nullptr) {
    s.seq = t / p.T;
    s.begin = s.seq * p.T;
    s.end = s.begin + p.T;
    return;
  }
  int lo = 0, hi = p.num_seqs;               // the last one that starts at or before t, whatever cu holds
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  s.seq = lo;
  s.begin = p.cu[lo];
  s.end = p.cu[lo + 1];
  if (t < s.begin || t >= s.end) s.begin = s.end = -1;
}

// c -> A c + H; closed: the scan started anew on the way, nothing of c gets through
struct Map {
  float A[4], H[4];
  bool closed;
};
// first `before`, then `m`
__device__ __forceinline__ void after(Map& m, const Map& before) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!m.closed) m.H[j] = fmaf(m.A[j], before.H[j], m.H[j]);
    m.A[j] *= before.A[j];
  }
  m.closed |= before.closed;
}

// Tokens of a thread, and stages of the ring: what leaves room for two blocks an SM.
template <typename IO, bool BWD>
constexpr int tokens_each() { return BWD && sizeof(IO) == 4 ? 2 : 4; }
template <typename IO, bool BWD>
constexpr int stage_bytes() { return tokens_each<IO, BWD>() * kThreads * (16 + (BWD ? 2 : 1) * 4 * static_cast<int>(sizeof(IO))); }
template <typename IO, bool BWD>
constexpr int stages() { return 98304 / stage_bytes<IO, BWD>(); }

template <typename IO, typename G, bool BWD, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) glr_scan_kernel(const Params p, const int cluster) {
  constexpr int R = tokens_each<IO, BWD>(), S = stages<IO, BWD>(), TL = kRows * R, GAP = 8;
  using RawIO = decltype(Raw4<IO>::u);
  using RawG = decltype(Raw4<G>::u);
  static_assert(S >= 3, "a tile waits for what enters it, one is summed up, one is on its way");
  // the ring, every thread's own 4 channels of its tokens: [S][R][thread]
  extern __shared__ __align__(16) uint8_t dynamic[];
  float4* ring_g = reinterpret_cast<float4*>(dynamic);   // g as it lies in memory, then e^g (or what a sequence starts from)
  RawIO* ring_x = reinterpret_cast<RawIO*>(ring_g + S * R * kThreads);
  RawIO* ring_y = ring_x + S * R * kThreads;
  __shared__ __align__(16) float warp_a[2][kWarps][kChannels], warp_h[2][kWarps][kChannels];
  __shared__ bool warp_closed[2][kWarps];
  // what the cluster's tiles of a step do: written by each into all; three steps, as one may be a step
  // ahead of a CTA that still reads
  __shared__ __align__(16) float tile_a[3][kMaxCluster][kChannels], tile_h[3][kMaxCluster][kChannels];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane >> 3, cq = lane & 7;
  const int rank = blockIdx.x % cluster, ct = blockIdx.x / cluster;
  const int c0 = ct * kChannels + (VEC ? 4 * cq : cq), D = p.D;
  const int total = static_cast<int>(p.tokens);
  const int steps = static_cast<int>((p.tokens + static_cast<long>(cluster) * TL - 1) / (static_cast<long>(cluster) * TL));
  // in scan order, this thread's first token of a step
  auto first = [&](int n) { return (static_cast<long>(n) * cluster + rank) * TL + (warp * 4 + sub) * R; };
  auto token = [&](long pos) { return static_cast<int>(BWD ? total - 1 - pos : pos); };
  auto slot = [&](int n, int r) { return (n % S * R + r) * kThreads + tid; };
  const G* pg = static_cast<const G*>(p.g);
  const IO* px = static_cast<const IO*>(p.x);
  const IO* py = static_cast<const IO*>(p.y);

  auto fetch = [&](int n) {                   // a step's inputs on their way
    const long pos = first(n);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool there = n < steps && pos + r < total && c0 < D;
      const int t = token(pos + r);
      const size_t at = there ? static_cast<size_t>(t) * D + c0 : 0;
      copy_async<4 * sizeof(G)>(&ring_g[slot(n, r)], pg + at, there);
      copy_async<4 * sizeof(IO)>(&ring_x[slot(n, r)], px + at, there);
      if constexpr (BWD) copy_async<4 * sizeof(IO)>(&ring_y[slot(n, r)], py + (there && t > 0 ? at - D : 0), there && t > 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the same through registers, for rows that asynchronous copies cannot start at
  Raw4<G> held_g[VEC ? 1 : R];
  Raw4<IO> held_x[VEC ? 1 : R], held_y[VEC ? 1 : R];
  auto load = [&](int n) {
    const long pos = first(n);
#pragma unroll
    for (int r = 0; r < (VEC ? 0 : R); ++r) {
      const bool there = n < steps && pos + r < total;
      const int t = there ? token(pos + r) : 0;
      const size_t row = static_cast<size_t>(t) * D;
      held_g[r] = load4<false, GAP>(pg + row, c0, there ? D : 0);
      held_x[r] = load4<false, GAP>(px + row, c0, there ? D : 0);
      if constexpr (BWD) held_y[r] = load4<false, GAP>(py + (t > 0 ? row - D : 0), c0, there && t > 0 ? D : 0);
    }
  };
  auto put = [&](int n) {
#pragma unroll
    for (int r = 0; r < (VEC ? 0 : R); ++r) {
      *reinterpret_cast<RawG*>(&ring_g[slot(n, r)]) = held_g[r].u;
      ring_x[slot(n, r)] = held_x[r].u;
      if constexpr (BWD) ring_y[slot(n, r)] = held_y[r].u;
    }
  };

  // What a thread's tokens of step n, and those before them in the tile, do to what enters the tile; its
  // e^g go where g was.  The tile's own map goes to the cluster.
  Span ahead{0, -1, -1};
  auto sum_up = [&](int n, Map& m) {
    m = {{1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}, false};
    const long pos = first(n);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (pos + r >= total) break;
      const int t = token(pos + r);
      if (t < ahead.begin || t >= ahead.end) locate(ahead, p, t);
      if (ahead.end < 0) continue;            // (a token of no sequence leaves everything as it is)
      const Raw4<G> g{*reinterpret_cast<const RawG*>(&ring_g[slot(n, r)])};
      const Raw4<IO> x{ring_x[slot(n, r)]};
      const bool start = t == (BWD ? ahead.end - 1 : ahead.begin);
      float a[4], keep[4];
      if (start) {
        load_state<VEC, GAP>(m.H, p.init, ahead.seq, c0, D);
        m.closed = true;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = expf(g.get(j));
        keep[j] = start ? m.H[j] : a[j];      // (a final state may take the initial one's place: read it once)
        m.A[j] *= a[j];
        m.H[j] = BWD ? a[j] * (m.H[j] + x.get(j)) : fmaf(a[j], m.H[j], x.get(j));
      }
      ring_g[slot(n, r)] = make_float4(keep[0], keep[1], keep[2], keep[3]);
    }
    // over the warp's 4 threads of these channels
#pragma unroll
    for (int d = 8; d <= 16; d *= 2) {
      Map b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b.A[j] = __shfl_up_sync(0xFFFFFFFFu, m.A[j], d);
        b.H[j] = __shfl_up_sync(0xFFFFFFFFu, m.H[j], d);
      }
      b.closed = __shfl_up_sync(0xFFFFFFFFu, m.closed, d);
      if (lane >= d) after(m, b);
    }
    const int half = n & 1;
    if (sub == 3) {
      *reinterpret_cast<float4*>(&warp_a[half][warp][4 * cq]) = make_float4(m.A[0], m.A[1], m.A[2], m.A[3]);
      *reinterpret_cast<float4*>(&warp_h[half][warp][4 * cq]) = make_float4(m.H[0], m.H[1], m.H[2], m.H[3]);
      if (cq == 0) warp_closed[half][warp] = m.closed;
    }
    const Map whole = m;                       // (of the warp, where sub = 3)
    // the threads before this one: the subs of the warp, and the warps
    Map b{{1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}, false};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float A = __shfl_up_sync(0xFFFFFFFFu, m.A[j], 8), H = __shfl_up_sync(0xFFFFFFFFu, m.H[j], 8);
      if (sub > 0) b.A[j] = A, b.H[j] = H;
    }
    b.closed = __shfl_up_sync(0xFFFFFFFFu, m.closed, 8) && sub > 0;
    __syncthreads();
    Map w{{1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}, false};
    for (int i = 0; i < warp; ++i) {
      const float4 fa = *reinterpret_cast<const float4*>(&warp_a[half][i][4 * cq]),
                   fh = *reinterpret_cast<const float4*>(&warp_h[half][i][4 * cq]);
      Map next{{fa.x, fa.y, fa.z, fa.w}, {fh.x, fh.y, fh.z, fh.w}, warp_closed[half][i]};
      after(next, w);
      w = next;
    }
    m = b;
    after(m, w);
    return [whole, w]() { Map t = whole; after(t, w); return t; }();
  };
  auto publish = [&](int n, const Map& tile) {
    if (warp == kWarps - 1 && sub == 3) {
      // (where nothing gets through, an A of -1 says so: exponentials are never below 0)
      float A[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) A[j] = tile.closed ? -1.f : tile.A[j];
      for (int q = 0; q < cluster; ++q) {
        store_remote(&tile_a[n % 3][rank][4 * cq], q, A);
        store_remote(&tile_h[n % 3][rank][4 * cq], q, tile.H);
      }
    }
    cluster_arrive();
  };

  float carry[4] = {0.f, 0.f, 0.f, 0.f};       // what enters the step, the same in every CTA of the cluster
  Span here{0, -1, -1};
  Map cur, next;
  cluster_arrive();                            // (every CTA runs before another one writes into it)
  if constexpr (VEC) {
    for (int n = 0; n < S - 1; ++n) fetch(n);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
  } else {
    for (int n = 0; n < 2; ++n) {
      load(n);
      put(n);
    }
  }
  cluster_wait();
  if (steps > 0) publish(0, sum_up(0, cur));
  for (int n = 0; n < steps; ++n) {
    if constexpr (VEC) {
      fetch(n + S - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    } else {
      load(n + 2);
    }
    const bool more = n + 1 < steps;
    Map tile;
    if (more) tile = sum_up(n + 1, next);
    cluster_wait();                            // the step's maps are there
    if (more) publish(n + 1, tile);
    float c[4];
    for (int q = 0; q < cluster; ++q) {
      const float4 fa = *reinterpret_cast<const float4*>(&tile_a[n % 3][q][4 * cq]),
                   fh = *reinterpret_cast<const float4*>(&tile_h[n % 3][q][4 * cq]);
      const float A[4] = {fa.x, fa.y, fa.z, fa.w}, H[4] = {fh.x, fh.y, fh.z, fh.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (q == rank) c[j] = carry[j];
        carry[j] = A[j] == -1.f ? H[j] : fmaf(A[j], carry[j], H[j]);
      }
    }
    // the step's tokens again, from what enters them
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = cur.closed ? cur.H[j] : fmaf(cur.A[j], c[j], cur.H[j]);
    const long pos = first(n);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (pos + r >= total) break;
      const int t = token(pos + r);
      if (t < here.begin || t >= here.end) locate(here, p, t);
      if (here.end < 0) continue;
      const size_t row = static_cast<size_t>(t) * D;
      const float4 kept = ring_g[slot(n, r)];
      const Raw4<IO> x{ring_x[slot(n, r)]};
      float a[4] = {kept.x, kept.y, kept.z, kept.w}, out[4];
      if (t == (BWD ? here.end - 1 : here.begin)) {
        const Raw4<G> g = load4<VEC, GAP>(pg + row, c0, D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[j] = a[j];
          a[j] = expf(g.get(j));
        }
      }
      const bool end = t == (BWD ? here.begin : here.end - 1);
      if constexpr (BWD) {
        const Raw4<IO> y{ring_y[slot(n, r)]};
        float before[4], dg[4];
        if (end) load_state<VEC, GAP>(before, p.h0, here.seq, c0, D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!end) before[j] = y.get(j);
          out[j] = c[j] + x.get(j);
          c[j] = a[j] * out[j];
          dg[j] = c[j] * before[j];
        }
        store4<VEC, GAP>(static_cast<G*>(p.dg) + row, c0, D, dg);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = c[j] = fmaf(a[j], c[j], x.get(j));
      }
      store4<VEC, GAP>(static_cast<IO*>(p.out) + row, c0, D, out);
      if (end && p.fin) store_state<VEC, GAP>(p.fin, here.seq, c0, D, c);
    }
    if constexpr (!VEC) put(n + 2);
    cur = next;
  }

  // sequences without tokens keep their initial value; one block checks cu_seqlens and sets the status
  if constexpr (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");     // (zeros, past the last step)
  if (p.cu) {
    bool bad = false;
    for (int s0 = (rank * kWarps + warp) * 32; s0 < p.num_seqs; s0 += 32 * kWarps * cluster) {
      const int q = s0 + lane;
      const bool none = q < p.num_seqs && p.cu[q + 1] <= p.cu[q] && p.fin;
      const int c = ct * kChannels + lane;
      for (uint32_t m = __ballot_sync(0xFFFFFFFFu, none); m; m &= m - 1) {
        const size_t at = static_cast<size_t>(s0 + __ffs(m) - 1) * D + c;
        if (c < D) p.fin[at] = p.init ? p.init[at] : 0.f;
      }
    }
    if (blockIdx.x == 0) {
      for (int q = tid; q < p.num_seqs; q += kThreads) {
        const int b = p.cu[q], e = p.cu[q + 1];
        bad |= b < 0 || e < b || e > total || (q == 0 && b != 0) || (q == p.num_seqs - 1 && e != total);
      }
      bad = __syncthreads_or(bad);
      if (tid == 0) *p.status = bad ? kStatusBounds : 0u;
    }
  } else if (blockIdx.x == 0 && tid == 0) {
    *p.status = 0u;
  }
  cluster_arrive();                            // (nobody writes into a CTA that has ended)
  cluster_wait();
}

// The serving step: 4 channels a thread, the state in registers between its load and its store.
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

template <typename IO, typename G, bool BWD, bool VEC>
cudaError_t launch_scan(const Params& p, cudaStream_t st) {
  constexpr int ring = stages<IO, BWD>() * stage_bytes<IO, BWD>(), TL = kRows * tokens_each<IO, BWD>();
  const auto kernel = glr_scan_kernel<IO, G, BWD, VEC>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  static bool raised[64] = {};         // (a race raises it twice, to the same value)
  if (dev < 0 || dev >= 64 || !raised[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) raised[dev] = true;
  }
  // CTAs of a cluster share a channel tile's tokens: as many as there are places for, and tiles
  const long cts = (p.D + kChannels - 1) / kChannels, tiles = (p.tokens + TL - 1) / TL;
  int cluster = 1;
  while (cluster < kMaxCluster && cts * cluster * 2 <= 2 * sms && cluster * 2 <= tiles) cluster *= 2;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cts * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = ring;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, cluster);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename IO, typename G>
cudaError_t launch_types(const Params& p, bool backward, cudaStream_t st) {
  const bool vec = p.D % 4 == 0 && aligned(p.x, 4 * sizeof(IO)) && aligned(p.y, 4 * sizeof(IO)) && aligned(p.out, 4 * sizeof(IO)) &&
                   aligned(p.g, 4 * sizeof(G)) && aligned(p.dg, 4 * sizeof(G));
  if (backward) return vec ? launch_scan<IO, G, true, true>(p, st) : launch_scan<IO, G, true, false>(p, st);
  return vec ? launch_scan<IO, G, false, true>(p, st) : launch_scan<IO, G, false, false>(p, st);
}

template <typename IO, typename G>
cudaError_t launch_step_types(const StepParams& p, cudaStream_t st) {
  const bool vec = p.D % 4 == 0 && aligned(p.x, 4 * sizeof(IO)) && aligned(p.y, 4 * sizeof(IO)) && aligned(p.g, 4 * sizeof(G)) &&
                   aligned(p.state, 16);
  for (int b = 0; b < p.B; b += 65535) {        // (a grid's second dimension)
    StepParams q = p;
    const size_t row = static_cast<size_t>(b) * p.T * p.D;
    q.x = static_cast<const IO*>(p.x) + row;
    q.g = static_cast<const G*>(p.g) + row;
    q.y = static_cast<IO*>(p.y) + row;
    if (p.slots) q.slots = p.slots + b;
    else q.state = p.state + static_cast<size_t>(b) * p.D;
    q.B = p.B - b < 65535 ? p.B - b : 65535;
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
