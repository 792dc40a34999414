// glr.cu -- gated linear recurrence, per channel:  h_t = e^{g_t} h_{t-1} + x_t,  y_t = h_t,
// and its gradients:  lam_t = dy_t + mu_{t+1},  mu_t = e^{g_t} lam_t,  dx_t = lam_t,
// dg_t = mu_t h_{t-1}  (mu behind the last token: d_final; d_initial: mu of the first).
//
// Both are one scan  c -> e^{g_t} c + x_t  (backward, from the last token to the first:
// c -> e^{g_t} (c + dy_t)) over all tokens laid end to end, which starts anew at each sequence's
// first token from its initial value.  Bound by HBM: each input is read and each output
// written once, 8 bytes an element forward (bf16 with an fp32 gate), 14 backward.
//
// A block takes a tile of 128 channels and 64 tokens (32 in the fp32 backward), a warp 8 of the
// tokens with 4 channels a thread, all of them in registers from one burst of loads.  A warp's
// tokens act on what enters them as c -> A c + H; the warps' (A, H) join through shared memory, and the
// tiles of a channel through words in the workspace.  16 tiles make a group: a tile publishes its
// (A, H), reads those of its group's tiles before it and the value that enters the group, and
// folds forward over them; the group's last tile publishes what enters the next one.  So the serial
// part is one exchange through L2 for 1024 tokens, and every fold goes over the same terms in the
// same order on every call.  Tiles are taken in order by a counter, so whoever a tile waits for is
// already running; the waits are bounded all the same.
#include "layer_ops.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int kChannels = 128;  // of a tile: 4 a thread
constexpr int kWarps = 8;
constexpr int kGroup = 16;      // tiles joined without an exchange from one to the next

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

// A thread's channels: c0 .. c0 + 3 (VEC: D % 4 = 0 and aligned rows), else c0, c0 + 32, ...
template <bool VEC, typename T>
__device__ __forceinline__ Raw4<T> load4(const T* row, int c0, int D) {
  Raw4<T> r;
  if constexpr (VEC) {
    if (c0 < D) r.u = __ldcs(reinterpret_cast<const decltype(r.u)*>(row + c0));
    else r.u = {};
  } else if constexpr (sizeof(T) == 2) {
    uint16_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = c0 + 32 * j < D ? __ldcs(reinterpret_cast<const unsigned short*>(row) + c0 + 32 * j) : uint16_t(0);
    r.u = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
  } else {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = c0 + 32 * j < D ? __ldcs(row + c0 + 32 * j) : 0.f;
    r.u = make_float4(v[0], v[1], v[2], v[3]);
  }
  return r;
}

template <bool VEC, typename T>
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
      if (c0 + 32 * j < D) row[c0 + 32 * j] = from_f32<T>(v[j]);
  }
}

// A state row's 4 channels (fp32; zeros without one); through element loads, as states need 4-byte
// alignment only and a sequence has one.
template <bool VEC>
__device__ __forceinline__ void load_state(float (&v)[4], const float* states, int seq, int c0, int D) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = VEC ? c0 + j : c0 + 32 * j;
    v[j] = states && c < D ? states[static_cast<size_t>(seq) * D + c] : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store_state(float* states, int seq, int c0, int D, const float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = VEC ? c0 + j : c0 + 32 * j;
    if (c < D) states[static_cast<size_t>(seq) * D + c] = v[j];
  }
}

// A published word: (A, H) of a tile, or (kKnown, its outgoing value) where nothing that enters it
// gets through; kEmpty before.
constexpr uint64_t kEmpty = ~0ull;
constexpr float kKnown = -1.f;   // (an A is a product of exponentials, never below 0)

__device__ __forceinline__ uint64_t word(float a, float h) {
  if (a != a) a = __int_as_float(0x7FC00000);   // (no NaN looks like kEmpty)
  return static_cast<uint64_t>(__float_as_uint(h)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ float word_a(uint64_t w) { return __uint_as_float(static_cast<uint32_t>(w)); }
__device__ __forceinline__ float word_h(uint64_t w) { return __uint_as_float(static_cast<uint32_t>(w >> 32)); }
// Each word carries its own state, so no order between words is needed.
__device__ __forceinline__ void store_words(uint64_t* p, const uint64_t (&w)[4]) {
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(w[0]), "l"(w[1]) : "memory");
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p + 2), "l"(w[2]), "l"(w[3]) : "memory");
}
__device__ __forceinline__ void load_words(uint64_t (&w)[4], const uint64_t* p) {
  asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(w[0]), "=l"(w[1]) : "l"(p) : "memory");
  asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(w[2]), "=l"(w[3]) : "l"(p + 2) : "memory");
}

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// The last sequence that starts at or before token t (0 .. num_seqs - 1, whatever cu holds), by a whole
// warp: 32 probes at a time.
__device__ __forceinline__ int find_seq(const int32_t* cu, int num_seqs, int t, int lane) {
  int lo = 0, n = num_seqs;                // it is among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lo + lane * step;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, lane * step < n && cu[at] <= t);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Waits until a thread's 4 words are there; false where the wait gave up.
__device__ __forceinline__ bool wait_words(uint64_t (&w)[4], const uint64_t* p, unsigned long long limit_ns, uint32_t* status) {
  unsigned long long t0 = 0;
  for (;;) {
    load_words(w, p);
    if (__all_sync(0xFFFFFFFFu, w[0] != kEmpty && w[1] != kEmpty && w[2] != kEmpty && w[3] != kEmpty)) return true;
    const unsigned long long t = now_ns();
    if (t0 == 0) t0 = t;
    // (one clock for the warp: its lanes leave together)
    const bool late = t - t0 > limit_ns || (*reinterpret_cast<volatile uint32_t*>(status) & kStatusTimeout);
    if (__any_sync(0xFFFFFFFFu, late)) break;
  }
  if ((threadIdx.x & 31) == 0) atomicOr(status, kStatusTimeout);
  return false;
}

struct Scan {
  Params p;
  int tiles, channel_tiles;      // tiles along the tokens; tiles of channels
  uint64_t* words;               // [tiles][channel_tiles][128], or null for one tile along the tokens; what a
                                 // group's last tile writes is what enters the next group
  uint32_t* counter;
};

// Sets up the words, the counter and the status of a scan of several tiles.
__global__ void __launch_bounds__(256) glr_clear_kernel(ulonglong2* words, size_t pairs, uint32_t* counter, uint32_t* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (size_t i = blockIdx.x * 256ul + threadIdx.x; i < pairs; i += gridDim.x * 256ul) words[i] = make_ulonglong2(kEmpty, kEmpty);
  if (blockIdx.x == 0 && threadIdx.x == 0) *counter = *status = 0u;
}

template <typename IO, typename G, bool BWD, bool VEC, int R>
__global__ void __launch_bounds__(32 * kWarps, 2) glr_scan_kernel(const Scan s) {
  constexpr int TL = kWarps * R;
  __shared__ __align__(16) float sa[kWarps][kChannels], sh[kWarps][kChannels];
  __shared__ __align__(16) uint64_t win[kGroup][kChannels];
  __shared__ uint8_t known_in[kGroup];
  __shared__ uint32_t ticket;
  __shared__ uint8_t closed_by[kWarps];
  const Params& p = s.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t id = blockIdx.x;
  if (s.words) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) ticket = atomicAdd(s.counter, 1u);
    __syncthreads();
    id = ticket;
  }
  const int tile = id / s.channel_tiles, ct = id % s.channel_tiles;
  const int c0 = ct * kChannels + (VEC ? 4 * lane : lane);
  const int total = static_cast<int>(p.tokens), D = p.D;
  const long pos0 = static_cast<long>(tile) * TL + warp * R;          // of this warp's tokens, in scan order
  const int n = pos0 >= total ? 0 : total - pos0 < R ? static_cast<int>(total - pos0) : R;
  auto token = [&](int r) { return BWD ? total - 1 - static_cast<int>(pos0) - r : static_cast<int>(pos0) + r; };

  // every load of the tile's inputs on its way
  Raw4<IO> x[R], y[BWD ? R : 1];
  Raw4<G> gr[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r < n) {
      const size_t row = static_cast<size_t>(token(r)) * D;
      gr[r] = load4<VEC>(static_cast<const G*>(p.g) + row, c0, D);
      x[r] = load4<VEC>(static_cast<const IO*>(p.x) + row, c0, D);
      if constexpr (BWD) {
        if (token(r) > 0) y[r] = load4<VEC>(static_cast<const IO*>(p.y) + row - D, c0, D);
        else y[r].u = {};
      }
    } else {
      gr[r].u = {};
      x[r].u = {};
      if constexpr (BWD) y[r].u = {};
    }
  }

  // lane r < n: the sequence of the warp's token r, and whether the scan starts anew or ends there
  int seq = 0;
  bool starts = false, ends = false, live = false;
  if (p.cu && n > 0) seq = find_seq(p.cu, p.num_seqs, token(BWD ? n - 1 : 0), lane);
  if (lane < n) {
    const int t = token(lane);
    bool first, last;
    if (p.cu) {
      if (p.cu[seq + 1] <= t) {        // another one than that of the warp's earliest token
        int hi = p.num_seqs;
        while (hi - seq > 1) {
          const int mid = (seq + hi) >> 1;
          if (p.cu[mid] <= t) seq = mid;
          else hi = mid;
        }
      }
      const int a = p.cu[seq], b = p.cu[seq + 1];
      live = a <= t && t < b;
      first = t == a;
      last = t + 1 == b;
    } else {
      seq = t / p.T;
      live = true;
      first = t == seq * p.T;
      last = t + 1 == (seq + 1) * p.T;
    }
    starts = live && (BWD ? last : first);
    ends = live && (BWD ? first : last);
  }
  const uint32_t m_start = __ballot_sync(0xFFFFFFFFu, starts), m_end = __ballot_sync(0xFFFFFFFFu, ends),
                 m_live = __ballot_sync(0xFFFFFFFFu, live);

  // c -> A c + H over the warp's tokens (closed: the scan started anew among them, and A is 0)
  // (the last value that the scan started from is kept: where it goes on beyond this warp, its array may
  // hold the final state by the time the tokens are gone through again)
  float a[R][4], A[4] = {1.f, 1.f, 1.f, 1.f}, H[4] = {0.f, 0.f, 0.f, 0.f}, from[4] = {};
  bool closed = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (m_start >> r & 1) {
      load_state<VEC>(from, p.init, __shfl_sync(0xFFFFFFFFu, seq, r), c0, D);
#pragma unroll
      for (int j = 0; j < 4; ++j) H[j] = from[j];
      closed = true;
    }
    const bool on = m_live >> r & 1;        // (a token of no sequence leaves everything as it is)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[r][j] = on ? expf(gr[r].get(j)) : 1.f;
      const float in = on ? x[r].get(j) : 0.f;
      A[j] *= a[r][j];
      H[j] = BWD ? a[r][j] * (H[j] + in) : fmaf(a[r][j], H[j], in);
    }
  }
  *reinterpret_cast<float4*>(&sa[warp][4 * lane]) = make_float4(A[0], A[1], A[2], A[3]);
  *reinterpret_cast<float4*>(&sh[warp][4 * lane]) = make_float4(H[0], H[1], H[2], H[3]);
  if (lane == 0) closed_by[warp] = closed;
  __syncthreads();

  // what the warps before this one do to what enters the tile: PA c + PH
  float PA[4] = {1.f, 1.f, 1.f, 1.f}, PH[4] = {0.f, 0.f, 0.f, 0.f};
  bool pclosed = false;
  for (int w = 0; w < warp; ++w) {
    const float4 fa = *reinterpret_cast<const float4*>(&sa[w][4 * lane]), fh = *reinterpret_cast<const float4*>(&sh[w][4 * lane]);
    const bool cl = closed_by[w];
    const float ea[4] = {fa.x, fa.y, fa.z, fa.w}, eh[4] = {fh.x, fh.y, fh.z, fh.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      PH[j] = cl ? eh[j] : fmaf(ea[j], PH[j], eh[j]);
      PA[j] *= ea[j];
    }
    pclosed |= cl;
  }
  float C[4] = {0.f, 0.f, 0.f, 0.f};       // what enters the tile
  if (s.words) {
    const size_t row = static_cast<size_t>(s.channel_tiles) * kChannels;          // words of a tile
    uint64_t* mine = s.words + tile * row + ct * kChannels + 4 * lane;
    const int m = tile % kGroup;                                                  // tiles of the group before this one
    const bool last = m == kGroup - 1;
    // the whole tile's A c + H, in the last warp
    float TA[4], TH[4];
    const bool known = pclosed || closed || tile == 0;
    if (warp == kWarps - 1) {
      uint64_t w4[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        TA[j] = PA[j] * A[j];
        TH[j] = closed ? H[j] : fmaf(A[j], PH[j], H[j]);
        w4[j] = word(known ? kKnown : TA[j], TH[j]);
      }
      if (known || !last) store_words(mine, w4);
    }
    // (uniform over the block: the tile's first token says whether anything enters)
    if (tile > 0 && !__syncthreads_or(warp == 0 && (m_start & 1))) {
      // the group's tiles before this one, a warp each
      for (int k = warp; k < m; k += kWarps) {
        uint64_t w4[4];
        wait_words(w4, mine - (m - k) * row, p.wait_ns, p.status);
        *reinterpret_cast<ulonglong2*>(&win[k][4 * lane]) = make_ulonglong2(w4[0], w4[1]);
        *reinterpret_cast<ulonglong2*>(&win[k][4 * lane + 2]) = make_ulonglong2(w4[2], w4[3]);
        if (lane == 0) known_in[k] = word_a(w4[0]) == kKnown;                     // (the same in every channel)
      }
      __syncthreads();
      int k = m - 1;
      while (k >= 0 && !known_in[k]) --k;
      if (k >= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) C[j] = word_h(win[k][4 * lane + j]);
      } else if (tile >= kGroup) {
        uint64_t w4[4];
        wait_words(w4, mine - (m + 1) * row, p.wait_ns, p.status);
#pragma unroll
        for (int j = 0; j < 4; ++j) C[j] = word_h(w4[j]);
      }
      while (++k < m) {
#pragma unroll
        for (int j = 0; j < 4; ++j) C[j] = fmaf(word_a(win[k][4 * lane + j]), C[j], word_h(win[k][4 * lane + j]));
      }
    }
    if (warp == kWarps - 1 && last && !known) {
      uint64_t w4[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w4[j] = word(kKnown, fmaf(TA[j], C[j], TH[j]));
      store_words(mine, w4);
    }
  }

  // the warp's tokens again, from what enters them
  float c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = pclosed ? PH[j] : fmaf(PA[j], C[j], PH[j]);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (m_live >> r & 1) {
      const int sq = __shfl_sync(0xFFFFFFFFu, seq, r);
      if (m_start >> r & 1) {
        if (m_start >> r == 1u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] = from[j];
        } else {
          load_state<VEC>(c, p.init, sq, c0, D);
        }
      }
      const bool end = m_end >> r & 1;
      const size_t row = static_cast<size_t>(token(r)) * D;
      float out[4];
      if constexpr (BWD) {
        float before[4], dg[4];
        if (end) load_state<VEC>(before, p.h0, sq, c0, D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!end) before[j] = y[r].get(j);
          out[j] = c[j] + x[r].get(j);
          c[j] = a[r][j] * out[j];
          dg[j] = c[j] * before[j];
        }
        store4<VEC>(static_cast<G*>(p.dg) + row, c0, D, dg);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = c[j] = fmaf(a[r][j], c[j], x[r].get(j));
      }
      store4<VEC>(static_cast<IO*>(p.out) + row, c0, D, out);
      if (end && p.fin) store_state<VEC>(p.fin, sq, c0, D, c);
    }
  }

  // sequences without tokens keep their initial value; one block checks cu_seqlens
  if (tile == 0) {
    bool bad = false;
    if (p.cu)
      for (int s0 = warp * 32; s0 < p.num_seqs; s0 += 32 * kWarps) {
        const int q = s0 + lane;
        bool none = false;
        if (q < p.num_seqs) {
          const int b = p.cu[q], e = p.cu[q + 1];
          none = e <= b;
          bad |= b < 0 || e < b || e > total || (q == 0 && b != 0) || (q == p.num_seqs - 1 && e != total);
        }
        for (uint32_t m = __ballot_sync(0xFFFFFFFFu, none && p.fin); m; m &= m - 1) {
          float v[4];
          load_state<VEC>(v, p.init, s0 + __ffs(m) - 1, c0, D);
          store_state<VEC>(p.fin, s0 + __ffs(m) - 1, c0, D, v);
        }
      }
    if (ct == 0) {
      bad = __syncthreads_or(bad);
      if (tid == 0) {
        if (!s.words) *p.status = bad ? kStatusBounds : 0u;
        else if (bad) atomicOr(p.status, kStatusBounds);
      }
    }
  }
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
  Raw4<IO> xr = load4<VEC>(x, c0, D);
  Raw4<G> gr = load4<VEC>(g, c0, D);
  int slot = b;
  if (p.slots) {
    slot = p.slots[b];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot >= p.num_slots && p.status && threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
      const float zero[4] = {};
      for (int t = 0; t < p.T; ++t) store4<VEC>(y + static_cast<size_t>(t) * D, c0, D, zero);
      return;
    }
  }
  float* state = p.state + static_cast<size_t>(slot) * D;
  float h[4];
  if constexpr (VEC) {
    const float4 u = c0 < D ? *reinterpret_cast<const float4*>(state + c0) : make_float4(0.f, 0.f, 0.f, 0.f);
    h[0] = u.x; h[1] = u.y; h[2] = u.z; h[3] = u.w;
  } else {
    load_state<false>(h, state, 0, c0, D);
  }
  for (int t = 0; t < p.T; ++t) {
    const Raw4<IO> xt = xr;
    const Raw4<G> gt = gr;
    if (t + 1 < p.T) {
      xr = load4<VEC>(x + static_cast<size_t>(t + 1) * D, c0, D);
      gr = load4<VEC>(g + static_cast<size_t>(t + 1) * D, c0, D);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = fmaf(expf(gt.get(j)), h[j], xt.get(j));
    store4<VEC>(y + static_cast<size_t>(t) * D, c0, D, h);
  }
  if constexpr (VEC) {
    if (c0 < D) *reinterpret_cast<float4*>(state + c0) = make_float4(h[0], h[1], h[2], h[3]);
  } else {
    store_state<false>(state, 0, c0, D, h);
  }
}

// Tokens a warp takes: 8, and 4 where dy, y and g of 8 would fill a thread's registers.
constexpr int tokens_each(bool backward, bool bf16) { return backward && !bf16 ? 4 : 8; }

long tiles_of(long tokens, bool backward, bool bf16) {
  const long n = kWarps * tokens_each(backward, bf16);
  return tokens > n ? (tokens + n - 1) / n : 1;
}
long channel_tiles_of(int D) { return (D + kChannels - 1) / kChannels; }

template <typename IO, typename G, bool BWD, bool VEC>
cudaError_t launch_scan(const Params& p, cudaStream_t st) {
  constexpr int R = tokens_each(BWD, sizeof(IO) == 2);
  const long tiles = tiles_of(p.tokens, BWD, sizeof(IO) == 2), cts = channel_tiles_of(p.D);
  if (tiles * cts > INT32_MAX) return cudaErrorInvalidValue;
  Scan s{p, static_cast<int>(tiles), static_cast<int>(cts), nullptr, nullptr};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * cts));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cfg.attrs = &attr;
  if (tiles > 1) {
    s.counter = reinterpret_cast<uint32_t*>(p.work);
    s.words = reinterpret_cast<uint64_t*>(p.work + 256);
    const size_t pairs = static_cast<size_t>(tiles) * cts * kChannels / 2;
    const size_t blocks = (pairs + 1023) / 1024;
    glr_clear_kernel<<<static_cast<unsigned>(blocks < 608 ? blocks : 608), 256, 0, st>>>(reinterpret_cast<ulonglong2*>(s.words), pairs,
                                                                                        s.counter, p.status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;                 // starts under the kernel that clears, waits for its end
  }
  return cudaLaunchKernelEx(&cfg, glr_scan_kernel<IO, G, BWD, VEC, R>, s);
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

size_t workspace_bytes(long tokens, int D, bool backward, bool bf16) {
  const long tiles = tiles_of(tokens, backward, bf16);
  return tiles > 1 ? 256 + static_cast<size_t>(tiles) * channel_tiles_of(D) * kChannels * sizeof(uint64_t) : 0;
}

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
