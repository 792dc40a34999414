// gdr_chunk.cuh -- the chunk form of the gated delta rule with a scalar gate: layouts and
// helpers shared by its kernels (gdr_chunk.cu: forward; gdr_grad.cu: backward).
//
// Mathematics, per chunk of C = 64 tokens of one (sequence, value head).  With gc the
// running sum of g inside the chunk, D_ij = e^{gc_i - gc_j} (i >= j), G = e^{gc} and
// E = e^{gc_last - gc} per row, gamma = e^{gc_last}, S the state entering the chunk:
//     M  = strict_tril(beta_i (k_i . k_j) D_ij),   P = scale tril((q_i . k_j) D_ij)
//     T  = (I + M)^{-1},   R = P T
//     Y  = beta (v - G (k S)),   vn = T Y
//     o  = scale G (q S) + R Y,   S' = gamma S + k^T (E vn)
// (o's inner part is P vn = P T Y.)  The gate is a scalar per token, so it stays out of the
// products: k and q enter the tensor cores exactly as they lie in memory, in bf16, and
// every decay is a factor <= 1 on a row of an fp32 result; there is no range of g that the
// form cannot take.
//
// Precision: q, k, v and d_out are exact bf16 operands; states, gates and sums are fp32.  Every
// fp32 operand of a tensor-core product is taken as two bf16 parts, high + low (2^-18 of the
// value is lost), and the parts' products are summed in fp32; of two such operands the product
// of the low parts is left out (2^-18 too), but for [T; R] Y in the thin chains, where it comes
// for nothing.  That is S with k and q, Y with T and R, E vn with k, P with T; in the backward dS'
// with k, E (k dS') with T, R and scale G do with do and q, G beta z with k, z and vn (kept in
// memory as two parts) with do, with each other, with S and with dS' (three parts), A and B with
// q and k; the inverse's block products take two TF32 parts.  fp32 results come out 3e-6 to 5e-6
// off in the 2-norm, where the same formulas in fp32 are at 2e-7 to 5e-7.  Three parts (24 bits)
// would take half to twice as many products again and more TMEM and shared memory than there is
// (both are full).  Beside bf16 results, 1.7e-3 off by their own rounding, it does not count; a
// caller who wants the states to fp32 passes fp32 q, k and v, which run the token recurrence
// (the gradients: kda_backward's token recurrence, with g repeated over the key dims).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "gdr_common.cuh"
#include "pairs.cuh"
#include "sm103.cuh"

namespace kda {
namespace gdr {

constexpr int C = 64;                                  // tokens of a chunk
constexpr unsigned long long kDrainNs = 2000000000ull; // limit for work already issued

// Record of one (chunk, value head), written by the preparation and read by the chains:
// [T; R] as two K-major, 128-byte-swizzled bf16 tiles of 128 rows x 64 (high, then low
// parts), then per-row factors (fp32): G, E, beta, gamma, and a word that is not zero where
// the preparation ran out of time.  (The preparation is the call's first kernel and clears
// the status word, so it reports through the record; the kernels after it report directly.)
constexpr uint32_t kTileBytes = 128 * 128;
constexpr uint32_t kRecFactors = 2 * kTileBytes;
constexpr uint32_t kRecBytes = kRecFactors + 1024;
constexpr int kRecGamma = 192, kRecFailed = 193;       // indices among the factors

struct ChunkParams {
  Params p;
  uint8_t* rec;       // [slots, HV] records
  // backward: what the chains leave for the gradient kernel, per (slot, hv)
  float* states;      // S entering the chunk: [V / 64][K rows][16 chunks of 4, chunk ^= row & 7]
  float* dstates;     // dS' leaving it, likewise
  uint8_t* vn;        // vn as an operand image: [2 parts][V / 64][64 rows][64] bf16
  uint8_t* z;         // z, same layout
  const void* dout;   // [tokens, HV, V] bf16
  const float* dfin;  // [NS, HV, K, V] or null
  void* dq;           // [tokens, H, K] bf16, or with grouped heads fp32 shares [tokens, HV, K]
  void* dk;
  void* dv;           // [tokens, HV, V] bf16
  float* dg;          // [tokens, HV]
  float* dbeta;
  float* ds0;         // [NS, HV, K, V] or null
  unsigned long long wait_ns;
  int chunks;         // chunks of a sequence (fixed length) or slots in all (packed)
  int slots;
};

struct ChainMaps {
  CUtensorMap q, k;   // boxes of 64 dims x 64 tokens
  CUtensorMap v;      // forward: v, reverse: d_out; boxes of N columns x 64 tokens
  CUtensorMap o;      // forward: out, likewise; gradients without grouped heads: dq and (o2) dk, as q and k
  CUtensorMap o2;
};

// First slot of a sequence's chunks.  Packed sequences: floor(tok0 / 64) + seq leaves room
// for every sequence's partial chunk without reading the other lengths.
__device__ __forceinline__ int first_slot(const ChunkParams& a, int seq, long tok0) {
  return a.p.cu ? static_cast<int>(tok0 >> 6) + seq : seq * a.chunks;
}
__device__ __forceinline__ int num_chunks(int len) { return (len + C - 1) >> 6; }

// The sequence and chunk of a slot, by a whole warp; false where the slot holds no chunk
// (bounds out of order are reported by the chains).
__device__ __forceinline__ bool find_chunk(const ChunkParams& a, int slot, int& seq, long& tok, int& rows) {
  long tok0;
  int len, m;
  if (a.p.cu == nullptr) {
    seq = slot / a.chunks;
    m = slot - seq * a.chunks;
    tok0 = static_cast<long>(seq) * a.p.T;
    len = a.p.T;
  } else {
    // the last sequence whose first slot is <= slot: 32 probes at a time (by halves, each a
    // load that waits for the last, 16 sequences took the preparation 2000 of 14000 cycles)
    int lo = 0, hi = a.p.num_seqs;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5, s = lo + static_cast<int>(threadIdx.x & 31) * step;
      const bool at = s < hi && (a.p.cu[s] >> 6) + s <= slot;
      lo += max(__popc(__ballot_sync(0xFFFFFFFFu, at)) - 1, 0) * step;
      hi = min(hi, lo + step);
    }
    seq = lo;
    if (!seq_tokens(a.p.cu, a.p.T, a.p.num_seqs, nullptr, seq, tok0, len)) return false;
    m = slot - first_slot(a, seq, tok0);
  }
  if (m < 0 || m >= num_chunks(len)) return false;
  tok = tok0 + 64l * m;
  rows = min(C, len - C * m);
  return true;
}

// Two fp32 values as packed bf16 high parts and low parts.
__device__ __forceinline__ void split2(uint64_t x, uint32_t& hi, uint32_t& lo) {
  float a, b;
  unpack2f(x, a, b);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
  const uint64_t h = pack2f(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u));
  unpack2f(fma2(h, pack2f(-1.f, -1.f), x), a, b);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(b), "f"(a));
}
__device__ __forceinline__ void split8(const uint64_t* x, uint4& hi, uint4& lo) {
  split2(x[0], hi.x, lo.x);
  split2(x[1], hi.y, lo.y);
  split2(x[2], hi.z, lo.z);
  split2(x[3], hi.w, lo.w);
}
__device__ __forceinline__ void split8(const float* x, uint4& hi, uint4& lo) {
  split2(pack2f(x[0], x[1]), hi.x, lo.x);
  split2(pack2f(x[2], x[3]), hi.y, lo.y);
  split2(pack2f(x[4], x[5]), hi.z, lo.z);
  split2(pack2f(x[6], x[7]), hi.w, lo.w);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk `c` (0..7) of row r in a tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(uint32_t r, uint32_t c) {
  return (r >> 3) * 1024u + (r & 7) * 128u + ((c ^ (r & 7)) << 4);
}
// The same for 64-byte rows (4 chunks), 64-byte swizzle.
__device__ __forceinline__ uint32_t sw64(uint32_t r, uint32_t c) {
  return (r >> 3) * 512u + (r & 7) * 64u + ((c ^ ((r >> 1) & 3)) << 4);
}

// A real branch to one lane of a converged warp around all products of a step, where each
// product was predicated on its own: 124 -> 118 us for a forward of 4096 tokens and 32 heads.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// The warp's number, known to the compiler as the same for all its lanes.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0); }

// Four chained products D (+)= A B (16 of K each; AS and BS bytes from one to the next) of a
// converged warp: the first accumulates if `acc`, the others always.
template <uint32_t AS, uint32_t BS>
__device__ __forceinline__ void umma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (elect_one()) {
#pragma unroll
    for (int s = 0; s < 4; ++s) umma_f16(d, a + s * (AS >> 4), b + s * (BS >> 4), idesc, s ? 1u : acc);
  }
  __syncwarp();
}
// The same with A in tensor memory (8 columns are 16 of K).
template <uint32_t BS>
__device__ __forceinline__ void umma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (elect_one()) {
#pragma unroll
    for (int s = 0; s < 4; ++s) umma_f16_ts(d, a + 8 * s, b + s * (BS >> 4), idesc, s ? 1u : acc);
  }
  __syncwarp();
}

// A kernel of a call starts while the one before it still runs: before it touches what that
// one wrote it waits for its end, and it lets the next one start once all its blocks have
// started and taken their TMEM (a waiting block must not hold what a running one needs).
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// mbarrier.try_wait may suspend a thread until the phase completes, so a limit is only looked
// at where it returns without; a limit below this is kept by polling.
constexpr unsigned long long kPollNs = 20000ull;
// Wait for a barrier's phase, giving up after `limit_ns` or once *failed is set.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t* failed) {
  uint64_t t0 = 0;
#pragma unroll 1
  while (!(limit_ns < kPollNs ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit_ns || *failed != 0u) return false;
  }
  return true;
}

// The same by a whole warp of a CTA that reports its failure once.  What a wait needs after its
// first look is one function for all of them: written out at every wait, this code alone
// pushed the others out of the instruction cache.
static __device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t* failed,
                                         uint32_t* status) {
  if (__all_sync(0xFFFFFFFFu, wait_phase(bar, parity, limit_ns, failed))) return true;
  if ((threadIdx.x & 31) == 0 && *failed == 0u) {
    atomicOr(status, kStatusTimeout);
    *failed = 1u;
  }
  return false;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t* failed,
                                          uint32_t* status) {
  return __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)) || wait_longer(bar, parity, limit_ns, failed, status);
}

static __device__ __noinline__ bool wait_or_drain_longer(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (limit_ns >= kPollNs) {
    if (mbar_wait_sleep(bar, parity, limit_ns)) return true;
  } else {
    const uint64_t t0 = globaltimer_ns();
    do {
      if (mbar_test_wait(bar, parity)) return true;
    } while (globaltimer_ns() - t0 <= limit_ns);
  }
  mbar_wait_sleep(bar, parity, kDrainNs);
  return false;
}

// A wait for work that ends by itself: false if it took longer than the limit (it has ended all
// the same, or kDrainNs are over too).
__device__ __forceinline__ bool wait_or_drain(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return (limit_ns >= kPollNs && mbar_try_wait(bar, parity)) || wait_or_drain_longer(bar, parity, limit_ns);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A lane's two rows of g or beta; zero past the end.
__device__ __forceinline__ void load_gate(const float* x, const Params& p, long tok, int rows, int hv, int lane, float (&v)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) v[e] = 2 * lane + e < rows ? x[(tok + 2 * lane + e) * p.HV + hv] : 0.f;
}
// A sum kept as a float and what the float misses (the pair is good to about 2^-46).
__device__ __forceinline__ void add_pairs(float& h, float& l, float h2, float l2) {
  const float s = h + h2, b = s - h, e = ((h - (s - b)) + (h2 - b)) + (l + l2);
  h = s + e;
  l = e - (h - s);
}
// gc of a chunk's rows 2 lane, 2 lane + 1 (one warp), in log2 units, as such pairs: decays
// between neighbours stay exact after a steep drop.  g below -120 already is e^g = 0.
__device__ __forceinline__ void gate_scan(float g0, float g1, int lane, float (&hi)[2], float (&lo)[2]) {
  g0 = g0 < -120.f ? -120.f : g0;
  g1 = g1 < -120.f ? -120.f : g1;
  constexpr float kL = 1.44269502f, kLlow = 1.92596299e-8f;  // log2 e and its rest
  const float h0 = g0 * kL, l0 = fmaf(g0, kL, -h0) + g0 * kLlow, h1 = g1 * kL, l1 = fmaf(g1, kL, -h1) + g1 * kLlow;
  float h = h0, l = l0;
  add_pairs(h, l, h1, l1);                    // the lane's two rows
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const float uh = __shfl_up_sync(0xFFFFFFFFu, h, s), ul = __shfl_up_sync(0xFFFFFFFFu, l, s);
    if (lane >= s) add_pairs(h, l, uh, ul);
  }
  hi[1] = h;
  lo[1] = l;
  add_pairs(h, l, -h1, -l1);
  hi[0] = h;
  lo[0] = l;
}

// Processors of the current device.
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
  if (dev < 64 && (v = known[dev].load(std::memory_order_relaxed)) > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) return 152;
  if (dev < 64) known[dev].store(v, std::memory_order_relaxed);
  return v;
}

// Launch a kernel, as a dependent of the stream's previous one where `after` says so; its
// shared-memory limit is raised on its first launch on a device.
struct LaunchState {
  bool raised[64] = {};
};
template <class... P, class... A>
cudaError_t launch_kernel(LaunchState& state, void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, bool after,
                          cudaStream_t st, const A&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !state.raised[dev]) {  // (a race raises it twice, to the same value)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) state.raised[dev] = true;
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace gdr
}  // namespace kda
