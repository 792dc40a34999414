// gdr_chunk.cu -- the gated delta rule in chunk form on tcgen05: the preparation of the
// chunks (all in parallel) and the chain that carries the state through a sequence.
// The mathematics stands in gdr_chunk.cuh.
#include <cstring>

#include "gdr_chunk.cuh"

namespace kda {
namespace gdr {
namespace {

// ------------------------------------------------------------ preparation ---
// One CTA of 128 threads per (chunk, value head).  [k; q] k^T is one product of M = 128
// (rows 0-63: k, 64-127: q), read back a row a thread: M to shared memory in fp32, P as an
// operand in two bf16 parts.  T = (I + M)^-1 in blocks of 16: the diagonal ones by
// substitution (a row a thread), the others by
//     [A 0; B D]^-1 = [A^-1 0; -D^-1 B A^-1  D^-1],
// first within the 32-row halves, then between them: 16 block products of a depth of 6, on
// warp-level TF32 tensor instructions, each operand in two TF32 parts (2^-20).  R = P T is a
// product of tcgen05 again (P's and T's parts: high high, high low, low high; on blocks of 16
// it took 20 more block products).
// What bounds it is instruction fetch and issue: written out straight (the solves unrolled
// into registers), the code ran once per CTA at an instruction a cycle and SM, 47 us for 2048
// chunks and heads by plain substitution, 87 us with block products unrolled; so the block
// product is one small loop body and its operands stay in shared memory.  Now 31 us for those
// 2048 (K = 128), 275 us for 23424 of packed sequences: 1.9 instructions a cycle and SM, 6600 a
// chunk and head; it writes 33 KB each.
namespace prep {
constexpr int NT = 128;
constexpr uint32_t LDM = 68;                           // floats between rows of M and T: no bank conflicts
// [k; q] tiles at 0; over them, in 64-row tiles of an operand's high and low part, P, then R; and
// between these M, 32 rows each, then T.  So six CTAs share an SM (with M apart from the tiles, four).
constexpr uint32_t HALF_M = 32 * LDM * 4;
constexpr uint32_t OFF_T = 0, OFF_P = 9216, PART = 17408;  // low parts: PART on; rows 32-63 of M: likewise
constexpr uint32_t OFF_GC = 2 * PART;                  // -gc high parts, low parts (log2), beta, block factors; then the record's row factors
constexpr uint32_t OFF_BAR = OFF_GC + 1024;
constexpr uint32_t SMEM = OFF_BAR + 64 + 1024;
static_assert(OFF_GC >= 2 * kTileBytes && HALF_M <= OFF_P && OFF_P + 8192 <= PART && OFF_P >= 8192, "the tiles fit");
__device__ __forceinline__ float* row_of_m(uint8_t* sm, int r) {
  return reinterpret_cast<float*>(sm + (r >= 32 ? PART : 0)) + (r & 31) * LDM;
}

// Two TF32 parts by truncation (the low 13 bits cleared).
__device__ __forceinline__ void tf32_parts(float x, uint32_t& h, uint32_t& l) {
  h = __float_as_uint(x) & 0xFFFFE000u;
  l = __float_as_uint(x - __uint_as_float(h)) & 0xFFFFE000u;
}
// acc (16 x 16, two 8-column tiles) += A B, both 16 x 16 floats in shared memory.  K is
// taken in the order 0, 2, 4, 6, 1, 3, 5, 7 of an 8-column tile, for A's rows to be read in pairs.
__device__ __forceinline__ void block_mma(float (&acc)[2][4], const float* x, int ldx, const float* b, int ldb, int lane) {
  const int g = lane >> 2, t = lane & 3;
  float cross[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // apart: shorter chains
  uint32_t ah[2][4], al[2][4], bh[2][2][2], bl[2][2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float2 u = *reinterpret_cast<const float2*>(x + g * ldx + 8 * s + 2 * t);
    const float2 w = *reinterpret_cast<const float2*>(x + (g + 8) * ldx + 8 * s + 2 * t);
    tf32_parts(u.x, ah[s][0], al[s][0]);
    tf32_parts(w.x, ah[s][1], al[s][1]);
    tf32_parts(u.y, ah[s][2], al[s][2]);
    tf32_parts(w.y, ah[s][3], al[s][3]);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) tf32_parts(b[(8 * s + 2 * t + e) * ldb + 8 * n + g], bh[s][n][e], bl[s][n][e]);
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      mma_tf32_m16n8k8(acc[n], ah[s], bh[s][n][0], bh[s][n][1]);
      mma_tf32_m16n8k8(cross[n], ah[s], bl[s][n][0], bl[s][n][1]);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) mma_tf32_m16n8k8(cross[n], al[s], bh[s][n][0], bh[s][n][1]);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] += cross[n][e];
}
__device__ __forceinline__ void block_put(float* x, const float (&acc)[2][4], float f, int lane) {
  x += (lane >> 2) * LDM + 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    *reinterpret_cast<float2*>(x + 8 * n) = make_float2(f * acc[n][0], f * acc[n][1]);
    *reinterpret_cast<float2*>(x + 8 * n + 8 * LDM) = make_float2(f * acc[n][2], f * acc[n][3]);
  }
}
}  // namespace prep

template <int K>
__global__ void __launch_bounds__(prep::NT, 6) gdr_prep_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a) {
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  float* gh = reinterpret_cast<float*>(sm + prep::OFF_GC);   // -gc
  float* gl = gh + C;
  float* bs = gl + C;
  float* cf = bs + C;                             // e^{gc of the 16-block's last row - gc_j}
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + prep::OFF_BAR);  // [0]: tiles; [1], [2]: products
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 3);
  const Params& p = a.p;
  const int slot = blockIdx.x / p.HV, hv = blockIdx.x % p.HV, hk = hv / (p.HV / p.H);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  int seq, rows;
  long tok;
  if (blockIdx.x == 0 && tid == 0) *p.status = 0u;
  if (!find_chunk(a, slot, seq, tok, rows)) return;
  bool ok = true;                                // this thread's waits
  if (warp == 0) {
    if (lane == 0) {
      mbar_init(&bar[0], 1);
      mbar_init(&bar[1], 1);
      mbar_init(&bar[2], 1);
      fence_mbar_init();
      mbar_arrive_expect_tx_relaxed(&bar[0], (K / 64) * kTileBytes);
#pragma unroll
      for (int b = 0; b < K / 64; ++b) {
        tma_load_3d(sm + b * kTileBytes, &maps.k, &bar[0], 64 * b, hk, static_cast<int>(tok));
        tma_load_3d(sm + b * kTileBytes + 8192, &maps.q, &bar[0], 64 * b, hk, static_cast<int>(tok));
      }
    }
    __syncwarp();
    tmem_alloc(tslot, 64);
    tmem_relinquish();
  }
  if (warp == 1) {
    float g[2], h[2], l[2];
    load_gate(p.g, p, tok, rows, hv, lane, g);
    gate_scan(g[0], g[1], lane, h, l);
    gh[2 * lane] = -h[0];
    gh[2 * lane + 1] = -h[1];
    gl[2 * lane] = -l[0];
    gl[2 * lane + 1] = -l[1];
    const float eh = __shfl_sync(0xFFFFFFFFu, h[1], lane | 7), el = __shfl_sync(0xFFFFFFFFu, l[1], lane | 7);
    cf[2 * lane] = ex2((eh - h[0]) + (el - l[0]));
    cf[2 * lane + 1] = ex2((eh - h[1]) + (el - l[1]));
  } else if (warp == 2) {
    const int i0 = 2 * lane;
    bs[i0] = i0 < rows ? p.beta[(tok + i0) * p.HV + hv] : 0.f;
    bs[i0 + 1] = i0 + 1 < rows ? p.beta[(tok + i0 + 1) * p.HV + hv] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now: a block of the next kernel that shares this SM takes its TMEM after this one's
  let_next_kernel_start();
  const uint32_t tmem = *tslot;
  if (warp == 0) {
    ok = wait_or_drain(&bar[0], 0, a.wait_ns);
    __syncwarp();
    const uint64_t d = sdesc_sw128(smem_u32(sm));
#pragma unroll
    for (int b = 0; b < K / 64; ++b)
      umma4<32, 32>(tmem, d + (b * kTileBytes >> 4), d + (b * kTileBytes >> 4), idesc_f16kind(128, 64), b > 0);
    umma_commit_warp(&bar[1]);
  }
  // row i of D in log2: gc_i - gc_j; the factors of the row
  const int i = tid & 63;
  const bool isq = tid >= 64;
  const float hi = -gh[i], lo = -gl[i], be = bs[i], end_hi = -gh[63], end_lo = -gl[63];
  ok &= wait_or_drain(&bar[1], 0, a.wait_ns);
  tc_fence_after();
  // M and P.  D_ij = e^{gc_i - gc_j} directly in the last two 16-blocks of the warp's rows;
  // before them through the block's last row, as two factors <= 1, one per row and block, one
  // per column
  {
    const uint32_t t = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    const float f = i < rows ? (isq ? p.scale : be) : 0.f;   // rows past the sequence's end: M = P = 0
    const int last = isq ? i : i - 1;                        // columns 0 .. last of the row are not zero
    const int blocks = 2 + 2 * (warp & 1);                   // (rows 0-31 end in column 31)
#pragma unroll 1
    for (int b = 0; b < blocks; ++b) {
      float y[16];
      tmem_ld16(t + 16 * b, y);
      const uint64_t hh = pack2f(hi, hi), ll = pack2f(lo, lo);
      uint64_t d[8];
      if (b >= blocks - 2) {                                 // a block of some of the warp's rows
#pragma unroll
        for (int j = 0; j < 8; ++j) {                        // (gh, gl hold -gc)
          const uint64_t at = add2(add2(hh, *reinterpret_cast<const uint64_t*>(gh + 16 * b + 2 * j)),
                                   add2(ll, *reinterpret_cast<const uint64_t*>(gl + 16 * b + 2 * j)));
          float d0, d1;
          unpack2f(at, d0, d1);
          d[j] = pack2f(ex2(d0), ex2(d1));
        }
      } else {
        const float e = ex2((hi + gh[16 * b + 15]) + (lo + gl[16 * b + 15]));
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = mul2(pack2f(e, e), *reinterpret_cast<const uint64_t*>(cf + 16 * b + 2 * j));
      }
      tmem_ld_wait();
      const int end = i < rows ? last - 16 * b : -1;         // columns 0 .. end of the block are not zero
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float d0, d1;
        unpack2f(mul2(mul2(pack2f(f, f), d[j]), pack2f(y[2 * j], y[2 * j + 1])), d0, d1);
        y[2 * j] = 2 * j <= end ? d0 : 0.f;
        y[2 * j + 1] = 2 * j + 1 <= end ? d1 : 0.f;
      }
      if (isq) {                                             // P over the tiles, as an operand
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 h, l;
          split8(y + 8 * c, h, l);
          *reinterpret_cast<uint4*>(sm + prep::OFF_P + sw128(i, 2 * b + c)) = h;
          *reinterpret_cast<uint4*>(sm + prep::OFF_P + prep::PART + sw128(i, 2 * b + c)) = l;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(prep::row_of_m(sm, i) + 16 * b + 4 * j) =
              make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
      }
    }
    if (warp == 2) {                                         // (the rest of P's rows 0-31)
#pragma unroll
      for (int c = 4; c < 8; ++c) {
        *reinterpret_cast<uint4*>(sm + prep::OFF_P + sw128(i, c)) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(sm + prep::OFF_P + prep::PART + sw128(i, c)) = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if (warp < 2) {                                  // rows 32 warp ..: a half of I + M, of one warp alone
    __syncwarp();
    {                                              // row i of its diagonal block inverted, in the block's place
      const int rr = tid & 15;
      float* mb = prep::row_of_m(sm, tid & ~15) + (tid & ~15);
      float x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = j == rr ? 1.f : 0.f;
#pragma unroll
      for (int l = 15; l >= 1; --l)
#pragma unroll
        for (int j = 0; 4 * j < l; ++j) {
          const float4 r = *reinterpret_cast<const float4*>(mb + l * prep::LDM + 4 * j);
          x[4 * j] = fmaf(-x[l], r.x, x[4 * j]);
          if (4 * j + 1 < l) x[4 * j + 1] = fmaf(-x[l], r.y, x[4 * j + 1]);
          if (4 * j + 2 < l) x[4 * j + 2] = fmaf(-x[l], r.z, x[4 * j + 2]);
          if (4 * j + 3 < l) x[4 * j + 3] = fmaf(-x[l], r.w, x[4 * j + 3]);
        }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(mb + rr * prep::LDM + 4 * j) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      __syncwarp();
    }
    float* ha = prep::row_of_m(sm, 32 * warp) + 32 * warp;  // [A 0; B D] of 16-row blocks: B A^-1, then -D^-1 of it
    float* hb = ha + 16 * prep::LDM;
#pragma unroll 1
    for (int n = 0; n < 2; ++n) {
      float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      prep::block_mma(acc, n ? hb + 16 : hb, prep::LDM, n ? hb : ha, prep::LDM, lane);
      __syncwarp();
      prep::block_put(hb, acc, n ? -1.f : 1.f, lane);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();  // the halves are done, P is written, the accumulator is read
  {                 // the same between the halves, a block a warp; B A^-1 in the unused upper right
    const int I = warp >> 1, J = warp & 1;
    float* top = prep::row_of_m(sm, 0);
    float* low = prep::row_of_m(sm, 32);
#pragma unroll 1
    for (int n = 0; n < 2; ++n) {
      const float* x = low + 16 * I * prep::LDM + (n ? 32 : 0);
      const float* y = top + 16 * J + (n ? 32 : 0);
      const int from = n ? 0 : J, to = n ? I : 1;
      float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 1
      for (int l = from; l <= to; ++l) prep::block_mma(acc, x + 16 * l, prep::LDM, y + 16 * l * prep::LDM, prep::LDM, lane);
      prep::block_put((n ? low : top + 32) + 16 * I * prep::LDM + 16 * J, acc, n ? -1.f : 1.f, lane);
      __syncthreads();
    }
  }
  {                 // T as an operand over M, half a row a thread
    const int own = i >> 4, half = tid >> 6;       // columns past the row's own block are zero
    float y[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c4 = 8 * half + j;
      const float4 u = (c4 >> 2) <= own ? *reinterpret_cast<const float4*>(prep::row_of_m(sm, i) + 4 * c4)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
      y[4 * j] = u.x; y[4 * j + 1] = u.y; y[4 * j + 2] = u.z; y[4 * j + 3] = u.w;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint4 h, l;
      split8(y + 8 * c, h, l);
      *reinterpret_cast<uint4*>(sm + prep::OFF_T + sw128(i, 4 * half + c)) = h;
      *reinterpret_cast<uint4*>(sm + prep::OFF_T + prep::PART + sw128(i, 4 * half + c)) = l;
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) {  // R = P T in lanes 64-127 (0-63: of whatever lies before P, read by nobody)
    tc_fence_after();
    const uint64_t dp = sdesc_sw128(smem_u32(sm) + prep::OFF_P - 8192), dt = sdesc(smem_u32(sm) + prep::OFF_T, 8192, 1024, 2);
    constexpr uint32_t id = idesc_f16kind(128, 64) | IDESC_B_MN_MAJOR;
#pragma unroll 1
    for (int n = 0; n < 3; ++n)
      umma4<32, 2048>(tmem, dp + (n == 2 ? prep::PART >> 4 : 0u), dt + (n == 1 ? prep::PART >> 4 : 0u), id, n > 0);
    umma_commit_warp(&bar[2]);
  }
  float* fac = gh;
  if (!isq) {
    fac[i] = ex2(hi);
    fac[64 + i] = ex2((end_hi - hi) + (end_lo - lo));
    fac[128 + i] = be;
    if (i == 63) fac[kRecGamma] = ex2(hi);
  }
  ok &= wait_or_drain(&bar[2], 0, a.wait_ns);
  tc_fence_after();
  if (isq) {
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
      float y[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + 32 * b, y);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4 h, l;
        split8(y + 8 * c, h, l);
        *reinterpret_cast<uint4*>(sm + prep::OFF_P + sw128(i, 4 * b + c)) = h;
        *reinterpret_cast<uint4*>(sm + prep::OFF_P + prep::PART + sw128(i, 4 * b + c)) = l;
      }
    }
  }
  tc_fence_before();
  ok = __syncthreads_and(ok);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
  if (tid == 0) fac[kRecFailed] = ok ? 0.f : 1.f;
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    uint8_t* rec = a.rec + (static_cast<size_t>(slot) * p.HV + hv) * kRecBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bulk_store(rec + h * kTileBytes, sm + prep::OFF_T + h * prep::PART, 8192);
      bulk_store(rec + h * kTileBytes + 8192, sm + prep::OFF_P + h * prep::PART, 8192);
    }
    bulk_store(rec + kRecFactors, fac, 1024);
    bulk_commit();
    bulk_wait_read();
  }
}

// ------------------------------------------------------------------ chain ---
// For V = 64: one CTA per (sequence, value head).  16 warps hold the state in fp32 registers (warp w: key dims 32 (w % 4) + lane, columns
// 16 (w / 4) ..) and do everything between the products; of three more one issues the
// products, one loads the chunks two ahead (TMA tiles of k, q and v, the record by bulk
// copy), one stores results from their staging.  Per chunk:
//   1. D1 = [k; q] S      M = 128, K = key dims       lanes 0-63: k S, 64-127: q S
//   2. D2 = [T; R] Y      M = 128, K = 64             lanes 0-63: vn,  64-127: R Y
//   3. D3 = k^T (E vn)    M = 128 key dims, K = 64    S = gamma S + D3 in registers
// The lanes 0-63 carry the recurrence, the lanes 64-127 make the output meanwhile.  The high
// and low parts of S, Y and E vn lie side by side as 2 N columns of one operand (their
// products land in 2 N columns and are added when read), so that a product is one
// instruction per 16 of K: the chain is bound by the latency of these three steps, not by
// the tensor cores' rate.  (In all chains the code between the products has to stay small:
// it does not fit the first instruction caches, and every warp's wait, branch and product
// issue that was made shorter showed at once -- the products' issue behind one branch, for
// one, took 124 us of a forward to 118.)  4096 tokens, K = 128, 128 pairs: 247 us a forward;
// 4 packed sequences of 1 to 511, 8 heads, K = 64: 25 us for both chains of the backward.
//
// SAVE is the same recurrence for the backward: no output (the q and R rows are not
// loaded; what lies in their place only meets lanes that nobody reads); the state entering
// each chunk goes to memory in fp32, vn as an operand image in two bf16 parts.
//
// REVERSE carries the state's gradient from the last chunk to the first, with dS' the
// gradient leaving the chunk:
//   1. D1 = k dS'                               z = T^T (E k dS') + R^T do
//   2. D2 = T^T (E D1),  D2' = R^T do           dv = beta z
//   3. D3 = k^T (-G beta z) + q^T (scale G do)  dS = gamma dS' + D3
// with the transposed operands read from the same tiles (MN-major), so M is 128 where only
// 64 lanes are wanted: the other lanes' atom is some other tile and nobody reads them.
namespace chain {
constexpr int N = 64, NW = N / 4, THREADS = 32 * (NW + 3);   // NW warps hold the state; then products, loads, stores
enum Mode { FORWARD, SAVE, REVERSE };
template <int K, Mode MODE>
struct Lay {
  static constexpr bool BWD = MODE != FORWARD;
  static constexpr uint32_t YROWS = MODE == REVERSE ? 128 : C;    // REVERSE: rows 64-127 hold scale G do
  // a stage: [k; q] tiles at 0, then the record's row factors, v (or do), 64 rows x N; and
  // FORWARD [T; R] (the others keep one buffer of it: it is free from step 2 to the next)
  static constexpr uint32_t FAC = (K / 64) * kTileBytes;
  static constexpr uint32_t VS = FAC + 1024;
  static constexpr uint32_t TT = VS + C * N * 2;
  static constexpr uint32_t STAGE = BWD ? TT : TT + 2 * kTileBytes;
  static constexpr uint32_t TT1 = 2 * STAGE;
  static constexpr uint32_t S = TT1 + (BWD ? 2 * kTileBytes : 0); // S parts: K-rows of 2 N columns
  static constexpr uint32_t Y = S + 128 * 2 * N * 2;              // Y, then E vn
  // on the way to memory: o (64 rows x N bf16), or vn (z) in two parts and S in fp32
  static constexpr uint32_t OUT = Y + YROWS * 2 * N * 2;
  static constexpr uint32_t SF = OUT + (BWD ? 2 * C * 128 : C * N * 2);
  static constexpr uint32_t BAR = SF + (BWD ? K * 256 : 0);
  static constexpr uint32_t SLACK = 832;                          // for the base's alignment
  static constexpr uint32_t SMEM = BAR + 192 + SLACK;
  static constexpr uint32_t LBO_S = 128 * 128, LBO_Y = YROWS * 128;   // between 64-column atoms
  static constexpr uint32_t TX = (MODE == SAVE ? (K / 64) * 8192 : (K / 64) * kTileBytes) + 1024 + C * N * 2 +
                                 (BWD ? 0 : 2 * kTileBytes);
  static_assert(SMEM <= 232448, "shared memory");
};
enum { FULL0 = 0, FULL1, EMPTY0, EMPTY1, TFULL, TFREE, D1, D2, D3, SREADY, YREADY, VREADY, QREADY, SFREADY, OUTREADY, OUTFREE,
       DRAIN, NBAR };
}  // namespace chain

// 16 values of a row (in pairs) as the two parts of a 2 N-column operand (c0: first column; lbo:
// between its 64-column atoms).
template <int N>
__device__ __forceinline__ void put_parts(uint8_t* base, uint32_t lbo, int row, int c0, const uint64_t (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint4 h, l;
    split8(x + 4 * j, h, l);
    *reinterpret_cast<uint4*>(base + sw128(row, (c0 >> 3) + j)) = h;
    if constexpr (N == 32) *reinterpret_cast<uint4*>(base + sw128(row, 4 + (c0 >> 3) + j)) = l;   // both in one 128-byte row
    else *reinterpret_cast<uint4*>(base + lbo + sw128(row, (c0 >> 3) + j)) = l;
  }
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t x) {
  float a, b;
  unpack2f(x, a, b);
  return pack_bf16(a, b);
}
// 16 values of a row as bf16: to the staging tile (its TMA store takes whole chunks), or
// straight to memory.
__device__ __forceinline__ void put_tile(uint8_t* tile, int row, int c0, const uint64_t (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    *reinterpret_cast<uint4*>(tile + sw128(row, (c0 >> 3) + j)) =
        make_uint4(pack_pair(x[4 * j]), pack_pair(x[4 * j + 1]), pack_pair(x[4 * j + 2]), pack_pair(x[4 * j + 3]));
}
__device__ __forceinline__ void put_bf16(void* out, size_t at, const uint64_t (&x)[8]) {
  __nv_bfloat16* op = static_cast<__nv_bfloat16*>(out) + at;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    *reinterpret_cast<uint4*>(op + 8 * j) =
        make_uint4(pack_pair(x[4 * j]), pack_pair(x[4 * j + 1]), pack_pair(x[4 * j + 2]), pack_pair(x[4 * j + 3]));
}
// x = the sum of the two parts' products
template <int N>
__device__ __forceinline__ void tmem_ld_parts(uint32_t t, uint64_t (&x)[8]) {
  float a[16], b[16];
  tmem_ld16(t, a);
  tmem_ld16(t + N, b);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = add2(pack2f(a[2 * j], a[2 * j + 1]), pack2f(b[2 * j], b[2 * j + 1]));
}

// The sequence a chain takes: packed sequences start the longest first (by rank, ties by
// index), for the grid to end together (16 sequences of 1 to 8192 tokens, 32 heads, a forward
// of 1224 us in their own order took 1084).  Any lengths, valid or not, give every rank once.
constexpr int kRanked = 256;                              // more sequences than that come in their own order
__device__ __forceinline__ int ranked_sequence(const Params& p, int rank, volatile uint32_t* slot) {
  if (p.cu == nullptr || p.num_seqs == 1 || p.num_seqs > kRanked) return rank;
  for (int s = threadIdx.x; s < p.num_seqs; s += blockDim.x) {
    const unsigned len = static_cast<unsigned>(p.cu[s + 1]) - static_cast<unsigned>(p.cu[s]);
    unsigned last = p.cu[0];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < p.num_seqs; ++j) {
      const unsigned next = p.cu[j + 1], l = next - last;
      before += l > len || (l == len && j < s);
      last = next;
    }
    if (before == rank) *slot = s;
  }
  __syncthreads();
  return static_cast<int>(*slot);
}

template <int K, chain::Mode MODE>
__device__ __forceinline__ void chain_body(const ChainMaps& maps, const ChunkParams& a, int unit, uint8_t* raw) {
  using L = chain::Lay<K, MODE>;
  using namespace chain;
  constexpr int CPT = 16, H2 = CPT / 2, V = N;
  const uint32_t shift = (1024u - (smem_u32(raw) & 1023u)) & 1023u;  // 0: nothing lies before the dynamic part
  uint8_t* sm = raw + shift;
  if (shift > L::SLACK) {
    if (threadIdx.x == 0) atomicOr(a.p.status, kStatusTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + NBAR);
  volatile uint32_t* failed = tslot + 1;
  const Params& p = a.p;
  const int hv = unit % p.HV, hk = hv / (p.HV / p.H), seq = ranked_sequence(p, unit / p.HV, tslot + 2);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  long tok0;
  int len;
  const bool in_order = seq_tokens(p.cu, p.T, p.num_seqs, nullptr, seq, tok0, len);
  const int nch = num_chunks(len), slot0 = first_slot(a, seq, tok0);
  const auto chunk = [&](int n) { return MODE == REVERSE ? nch - 1 - n : n; };  // of step n
  if (tid == 0) {
    for (int b = 0; b < NBAR; ++b)
      mbar_init(&bars[b], b == SREADY || b == SFREADY ? NW : b == YREADY || b == VREADY || b == QREADY || b == OUTREADY ? NW / 2 : 1);
    *failed = 0u;
    fence_mbar_init();
  }
  constexpr uint32_t TD2 = 2 * N, TD3 = 4 * N, TD2R = 6 * N;
  if (warp == NW) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  wait_for_previous_kernel();  // the records, the cleared status
  let_next_kernel_start();
  if (!in_order && tid == 0) atomicOr(p.status, kStatusBounds);
  // waits of a whole warp; false once the CTA has failed
  auto wait = [&](int b, uint32_t parity) { return wait_warp(&bars[b], parity, a.wait_ns, failed, p.status); };
  // the loader's keep a short limit from the first look on
  auto wait_load = [&](int b, uint32_t parity) {
    return a.wait_ns < kPollNs ? wait_longer(&bars[b], parity, a.wait_ns, failed, p.status) : wait(b, parity);
  };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[b]);
  };

  if (warp == NW + 1) {
    // ---------------------------------------------------------------- loads ---
    auto record = [&](int n) { return a.rec + (static_cast<size_t>(slot0 + chunk(n)) * p.HV + hv) * kRecBytes; };
    auto load = [&](int n) {
      if (lane == 0) {
        uint8_t* st = sm + (n & 1) * L::STAGE;
        uint64_t* full = &bars[FULL0 + (n & 1)];
        const int tok = static_cast<int>(tok0 + C * static_cast<long>(chunk(n)));
        mbar_arrive_expect_tx_relaxed(full, L::TX);
#pragma unroll
        for (int b = 0; b < K / 64; ++b) {
          tma_load_3d(st + b * kTileBytes, &maps.k, full, 64 * b, hk, tok);
          if (MODE != SAVE) tma_load_3d(st + b * kTileBytes + 8192, &maps.q, full, 64 * b, hk, tok);
        }
        bulk_load(st + L::FAC, record(n) + kRecFactors, 1024, full);
        if (MODE == FORWARD) bulk_load(st + L::TT, record(n), 2 * kTileBytes, full);
        tma_load_3d(st + L::VS, &maps.v, full, 0, hv, tok);
      }
      __syncwarp();
    };
    auto load_t = [&](int n) {  // the one buffer of [T; R]: T alone for SAVE
      if (lane == 0) {
        mbar_arrive_expect_tx_relaxed(&bars[TFULL], MODE == SAVE ? 16384 : 2 * kTileBytes);
        bulk_load(sm + L::TT1, record(n), MODE == SAVE ? 8192 : 2 * kTileBytes, &bars[TFULL]);
        if (MODE == SAVE) bulk_load(sm + L::TT1 + kTileBytes, record(n) + kTileBytes, 8192, &bars[TFULL]);
      }
      __syncwarp();
    };
    int nf = 0, nt = 0;   // loads issued
    for (; nf < 2 && nf < nch; ++nf) load(nf);
    if (MODE != FORWARD && nch > 0) load_t(nt++);
    for (int n = 1; n < nch; ++n) {
      if (MODE != FORWARD) {                       // free once step 2 of the chunk before is done
        if (!wait_load(TFREE, (n - 1) & 1)) break;
        load_t(nt++);
      }
      if (nf < nch) {                              // a stage's readers are done once the next chunk's products start
        if (!wait_load(EMPTY0 + ((n - 1) & 1), ((n - 1) >> 1) & 1)) break;
        load(nf++);
      }
    }
    // what was issued lands before the CTA gives up its memory (the last may not have been
    // waited for by anybody if the chain failed)
    for (int m = nf < 2 ? 0 : nf - 2; m < nf; ++m) mbar_wait(&bars[FULL0 + (m & 1)], (m >> 1) & 1, kDrainNs);
    if (nt > 0) mbar_wait(&bars[TFULL], (nt - 1) & 1, kDrainNs);
  } else if (warp == NW) {
    // ------------------------------------------------------------- products ---
    const uint32_t sb = smem_u32(sm);
    constexpr uint32_t id2n = idesc_f16kind(128, 2 * N) | IDESC_B_MN_MAJOR;   // both parts of B
    constexpr uint32_t idn = idesc_f16kind(128, N) | IDESC_B_MN_MAJOR;        // the high part
    const uint64_t ds = sdesc(sb + L::S, L::LBO_S, 1024, 2), dy = sdesc(sb + L::Y, L::LBO_Y, 1024, 2);
    auto issue = [&](uint32_t d, uint64_t aa, uint64_t bb, uint32_t idesc, uint32_t acc, uint32_t as) {
      if (as == 32) umma4<32, 2048>(d, aa, bb, idesc, acc);
      else umma4<2048, 2048>(d, aa, bb, idesc, acc);
    };
    for (int n = 0; n < nch; ++n) {
      const uint32_t ph = n & 1, st = sb + ph * L::STAGE, tt = MODE == FORWARD ? st + L::TT : sb + L::TT1;
      const uint64_t dkq = sdesc_sw128(st), dkt = sdesc(st, kTileBytes, 1024, 2);
      const uint64_t dt = MODE == REVERSE ? sdesc(tt, kTileBytes, 1024, 2) : sdesc_sw128(tt);
      if (!wait(FULL0 + (n & 1), (n >> 1) & 1)) break;
      if (!wait(SREADY, ph)) break;
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < K / 64; ++b) issue(tmem, dkq + (b * kTileBytes >> 4), ds + (b * 8192 >> 4), id2n, b > 0, 32);
      umma_commit_warp(&bars[D1]);
      if (n > 0 && lane == 0) mbar_arrive(&bars[EMPTY0 + ((n - 1) & 1)]);
      __syncwarp();
      if (MODE != FORWARD && !wait(TFULL, ph)) break;
      if (MODE == REVERSE) {
        if (!wait(QREADY, ph)) break;
        tc_fence_after();
        const uint64_t dd = sdesc(st + L::VS, 8192, 1024, 2);
        constexpr uint32_t idr = idesc_f16kind(128, N) | IDESC_A_MN_MAJOR | IDESC_B_MN_MAJOR;
        // R^T do, the two parts of R (rows 64-127 of the record's tiles); q^T (scale G do)
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) issue(tmem + TD2R, dt + ((8192 + h * kTileBytes) >> 4), dd, idr, h, 2048);
        issue(tmem + TD3, dkt + (8192 >> 4), dy + (8192 >> 4), id2n | IDESC_A_MN_MAJOR, 0u, 2048);
      }
      if (!wait(YREADY, ph)) break;
      tc_fence_after();
      constexpr uint32_t am = MODE == REVERSE ? IDESC_A_MN_MAJOR : 0u;
      constexpr uint32_t as = MODE == REVERSE ? 2048 : 32;   // bytes of 16 of K in [T; R]
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) issue(tmem + TD2, dt + (h * kTileBytes >> 4), dy, (h ? idn : id2n) | am, h, as);
      umma_commit_warp(&bars[D2]);
      if (MODE != FORWARD) umma_commit_warp(&bars[TFREE]);
      if (!wait(VREADY, ph)) break;
      tc_fence_after();
      issue(tmem + TD3, dkt, dy, id2n | IDESC_A_MN_MAJOR, MODE == REVERSE, 2048);
      umma_commit_warp(&bars[D3]);
    }
    // what is in flight ends before the CTA gives up its memory
    umma_commit_warp(&bars[DRAIN]);
    mbar_wait(&bars[DRAIN], 0, kDrainNs);
  } else if (warp == NW + 2) {
    // --------------------------------------------------------------- stores ---
    for (int n = 0; n < nch; ++n) {
      const int c = chunk(n);
      const size_t cu = static_cast<size_t>(slot0 + c) * p.HV + hv;
      if (MODE != FORWARD) {
        if (!wait(SFREADY, n & 1)) break;
        if (lane == 0) {
          bulk_store((MODE == SAVE ? a.states : a.dstates) + cu * K * V, sm + L::SF, K * 256);
          bulk_commit();
        }
        __syncwarp();
      }
      if (!wait(OUTREADY, n & 1)) break;
      if (lane == 0) {
        if (MODE != FORWARD) {
          uint8_t* img = (MODE == SAVE ? a.vn : a.z) + cu * (4 * C * V);
          bulk_store(img, sm + L::OUT, 2 * 8192);
        } else if (C * c + C <= len) {
          tma_store_3d(&maps.o, sm + L::OUT, 0, hv, static_cast<int>(tok0 + C * static_cast<long>(c)));
        }
        bulk_commit();
        bulk_wait_read();
        mbar_arrive(&bars[OUTFREE]);
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_read();
  } else {
    // ------------------------------------------ state, Y, vn (z), output ---
    const int quad = warp & 3, c0 = (warp >> 2) * CPT;
    const int r = 32 * quad + lane;                  // TMEM lane: key dim of S, row of [k; q]
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16) + c0;
    const size_t soff = ((static_cast<size_t>(seq) * p.HV + hv) * K + r) * V + c0;
    const bool isk = quad < 2;                       // token rows of k; else rows r - 64 of q
    const int i = r & 63;
    const float* first = MODE == REVERSE ? a.dfin : p.s0;
    float* final = MODE == FORWARD ? p.sfin : MODE == REVERSE ? a.ds0 : nullptr;
    uint64_t s[H2];
#pragma unroll
    for (int j = 0; j < H2 / 2; ++j) {
      const float4 t = first && r < K ? *reinterpret_cast<const float4*>(first + soff + 4 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[2 * j] = pack2f(t.x, t.y);
      s[2 * j + 1] = pack2f(t.z, t.w);
    }
    put_parts<N>(sm + L::S, L::LBO_S, r, c0, s);
    fence_proxy_async_smem();
    arrive(SREADY);
    bool good = true;
    for (int n = 0; n < nch; ++n) {
      const uint32_t ph = n & 1;
      uint8_t* st = sm + ph * L::STAGE;
      const float* fac = reinterpret_cast<const float*>(st + L::FAC);
      const int c = chunk(n);
      const size_t tok = static_cast<size_t>(tok0 + C * static_cast<long>(c) + i);
      const bool live = C * c + i < len, whole = C * c + C <= len;  // this row; every row of the chunk
      if (!(good = wait(FULL0 + (n & 1), (n >> 1) & 1))) break;
      if (tid == 0 && fac[kRecFailed] != 0.f) atomicOr(p.status, kStatusTimeout);
      const float row = fac[i];
      const uint64_t gamma = pack2f(fac[kRecGamma], fac[kRecGamma]);
      const size_t orow = (tok * p.HV + hv) * V + c0;
      // rows past the sequence's end hold the next one's tokens, whatever they are: every
      // operand that meets them in a sum over tokens has them zeroed first
      auto clear_row = [&](uint8_t* tile) {
#pragma unroll 1
        for (int ch = 0; ch < 8 * (K / 64); ++ch)
          *reinterpret_cast<uint4*>(tile + (ch >> 3) * kTileBytes + sw128(i, ch & 7)) = make_uint4(0, 0, 0, 0);
      };
      auto put_state = [&]() {  // S (dS') in fp32 to its staging; rows of 16 chunks, swizzled
        if (n > 0 && !wait(OUTFREE, (n - 1) & 1)) return false;
        if (r < K) {
#pragma unroll
          for (int j = 0; j < CPT / 4; ++j) {
            float4 t;
            unpack2f(s[2 * j], t.x, t.y);
            unpack2f(s[2 * j + 1], t.z, t.w);
            *reinterpret_cast<float4*>(sm + L::SF + r * 256 + ((((c0 >> 2) + j) ^ (r & 7)) << 4)) = t;
          }
        }
        fence_proxy_async_smem();
        arrive(SFREADY);
        return true;
      };
      uint64_t x[H2], y[H2];
      auto load_v = [&](uint64_t (&out)[H2], float f) {  // f times this thread's values of v (do)
        const uint64_t ff = pack2f(f, f);
#pragma unroll
        for (int j = 0; j < CPT / 8; ++j) {
          const uint32_t ch = (c0 >> 3) + j;
          const uint4 u = *reinterpret_cast<const uint4*>(st + L::VS + sw128(i, ch));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            out[4 * j + e] = mul2(ff, pack2f(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)));
        }
      };
      if (isk) {
        const float be = fac[128 + i], tail = fac[64 + i];
        if (MODE != REVERSE) load_v(y, be);
        const float f1 = MODE == REVERSE ? tail : -be * row, f2 = MODE == REVERSE ? -row * be : tail;
        const uint64_t ff1 = pack2f(f1, f1), ff2 = pack2f(f2, f2);
        if (!(good = wait(D1, ph))) break;
        tc_fence_after();
        tmem_ld_parts<N>(tl, x);
#pragma unroll
        for (int j = 0; j < H2; ++j) x[j] = MODE == REVERSE ? mul2(ff1, x[j]) : fma2(ff1, x[j], y[j]);
        if (!whole && !live) {
#pragma unroll
          for (int j = 0; j < H2; ++j) x[j] = 0;
          if (warp < 4) clear_row(st);
        }
        put_parts<N>(sm + L::Y, L::LBO_Y, i, c0, x);
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(YREADY);
        if (!(good = wait(D2, ph))) break;
        tc_fence_after();
        tmem_ld_parts<N>(tl + TD2, x);
        if (MODE == REVERSE) {
          float t[CPT];
          tmem_ld16(tl + TD2R, t);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < H2; ++j) x[j] = add2(x[j], pack2f(t[2 * j], t[2 * j + 1]));
        }
#pragma unroll
        for (int j = 0; j < H2; ++j) {
          if (MODE == REVERSE && !live) x[j] = 0;   // (vn is zero there by itself: row i of T is e_i)
          y[j] = mul2(ff2, x[j]);
        }
        put_parts<N>(sm + L::Y, L::LBO_Y, i, c0, y);
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(VREADY);
        if (MODE != FORWARD) {  // while step 3 runs: S, and vn (z) as it is, in two parts
          if (!(good = put_state())) break;
#pragma unroll
          for (int j = 0; j < CPT / 8; ++j) {
            uint4 h, l;
            split8(x + 4 * j, h, l);
            *reinterpret_cast<uint4*>(sm + L::OUT + sw128(i, (c0 >> 3) + j)) = h;
            *reinterpret_cast<uint4*>(sm + L::OUT + 8192 + sw128(i, (c0 >> 3) + j)) = l;
          }
          fence_proxy_async_smem();
          arrive(OUTREADY);
        }
      } else if (MODE == FORWARD) {
        const uint64_t f = pack2f(p.scale * row, p.scale * row);
        if (!(good = wait(D1, ph))) break;
        tc_fence_after();
        tmem_ld_parts<N>(tl, x);
        if (!(good = wait(D2, ph))) break;
        tc_fence_after();
        tmem_ld_parts<N>(tl + TD2, y);
#pragma unroll
        for (int j = 0; j < H2; ++j) x[j] = fma2(f, x[j], y[j]);
        // through shared memory: a row a thread straight to memory, the stores would take the
        // load/store unit 500 to 1300 cycles a chunk from the warps on the way to step 3
        if (n > 0 && !(good = wait(OUTFREE, (n - 1) & 1))) break;
        if (whole) put_tile(sm + L::OUT, i, c0, x);
        else if (live) put_bf16(p.out, orow, x);
        fence_proxy_async_smem();
        arrive(OUTREADY);
      } else if (MODE == REVERSE) {
        load_v(x, p.scale * row);
        if (!whole && !live) {
#pragma unroll
          for (int j = 0; j < H2; ++j) x[j] = 0;
          if (warp < 4) clear_row(st + 8192);
#pragma unroll
          for (int j = 0; j < CPT / 8; ++j)
            *reinterpret_cast<uint4*>(st + L::VS + sw128(i, (c0 >> 3) + j)) = make_uint4(0, 0, 0, 0);
        }
        put_parts<N>(sm + L::Y, L::LBO_Y, 64 + i, c0, x);
        fence_proxy_async_smem();
        arrive(QREADY);
        if (!(good = put_state())) break;
      } else if (!(good = put_state())) {
        break;
      }
      if (!(good = wait(D3, ph))) break;
      tc_fence_after();
      tmem_ld_parts<N>(tl + TD3, x);
#pragma unroll
      for (int j = 0; j < H2; ++j) s[j] = fma2(gamma, s[j], x[j]);
      put_parts<N>(sm + L::S, L::LBO_S, r, c0, s);
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(SREADY);
    }
    if (good && final && r < K) {
#pragma unroll
      for (int j = 0; j < H2 / 2; ++j) {
        float4 t;
        unpack2f(s[2 * j], t.x, t.y);
        unpack2f(s[2 * j + 1], t.z, t.w);
        *reinterpret_cast<float4*>(final + soff + 4 * j) = t;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == NW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int K>
__global__ void __launch_bounds__(chain::THREADS, 1) gdr_chain_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a) {
  extern __shared__ __align__(16) uint8_t raw[];
  chain_body<K, chain::FORWARD>(maps, a, blockIdx.x, raw);
}

// ------------------------------------------------- chain, 32 columns thin ---
// The forward where one CTA per 32 value columns fits the SMs: few sequences, all latency.
// The same three steps as above, but the products over tokens are of M = 64, the rows that
// the recurrence waits for (k S, T Y) first and the output's (q S, R Y) behind them, in the
// shadow of what follows.  M = 64 puts 16 rows into each quadrant of TMEM, so the work
// between the products lies on all four parts of the SM, on one code path, in fragments of
// 8 x 8 tiles (v, Y, E vn and o move by tile accesses): a thread holds 8 values of a block.
// What the recurrence does not wait for is done where a warp waits for a product: a chunk's
// output while step 2 of the next runs, the next chunk's v and factors while step 3 runs
// (with two stages the loads came too late for that: a call of 158 us where three took 130;
// eight further warps for the output were no faster).
// 90 us for 4096 tokens, 32 heads of 128: 1.4 us a chunk, of it about 0.8 in the three
// products' latency, the rest in the hand-over between warps.  [k; q] S as one product of
// M = 128, the k rows on two of the four parts of the SM, took 110 us.
namespace thin {
constexpr int N = 32, NW = 8, THREADS = 32 * (NW + 3);
// TMEM columns: both parts' products, 2 x 32 each; q S and R Y twice, for chunks in turn
constexpr uint32_t TK = 0, TD3 = 0, TT = 64, TQ = 128, TR = 256, TURN = 64;
template <int K>
struct Lay {
  static constexpr uint32_t FAC = (K / 64) * kTileBytes;          // a stage of three: [k; q], row factors, v
  static constexpr uint32_t VS = FAC + 1024;
  static constexpr uint32_t STAGE = VS + C * N * 2;
  static constexpr uint32_t TT = 3 * STAGE;                       // [T; R], of two
  static constexpr uint32_t S = TT + 2 * 2 * kTileBytes;          // rows of 2 x 32 columns, high and low parts
  static constexpr uint32_t Y = S + 128 * 128;
  static constexpr uint32_t VN = Y + C * 128;                     // E vn
  static constexpr uint32_t OUT = VN + C * 128;
  static constexpr uint32_t BAR = OUT + C * N * 2;
  static constexpr uint32_t SLACK = 832;
  static constexpr uint32_t SMEM = BAR + 192 + SLACK;
  static_assert(SMEM <= 232448 && STAGE % 1024 == 0, "shared memory");
};
enum { FULL = 0, EMPTY = 3, TFULL = 6, TFREE = 8, D1 = 10, D2, D3, SREADY, YREADY, VREADY, OUTREADY, OUTFREE, DRAIN, NBAR };
// 16 rows x 16 columns of a result, the two parts' products added: pair 2 m + r is row
// lane / 4 + 8 r, columns 8 m + 2 (lane % 4) and one on
__device__ __forceinline__ void frag_ld(uint32_t t, uint64_t (&x)[4]) {
  uint32_t a[2][4], b[2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    tmem_ld_16x256b(t + 8 * m, a[m]);
    tmem_ld_16x256b(t + N + 8 * m, b[m]);
  }
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = add2(pack2f(__uint_as_float(a[j >> 1][2 * (j & 1)]), __uint_as_float(a[j >> 1][2 * (j & 1) + 1])),
                pack2f(__uint_as_float(b[j >> 1][2 * (j & 1)]), __uint_as_float(b[j >> 1][2 * (j & 1) + 1])));
}
}  // namespace thin

template <int K>
__global__ void __launch_bounds__(thin::THREADS, 1) gdr_thin_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a,
                                                                   int V) {
  extern __shared__ __align__(16) uint8_t raw[];
  using L = thin::Lay<K>;
  using namespace thin;
  const uint32_t shift = (1024u - (smem_u32(raw) & 1023u)) & 1023u;
  uint8_t* sm = raw + shift;
  if (shift > L::SLACK) {
    if (threadIdx.x == 0) atomicOr(a.p.status, kStatusTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + NBAR);
  volatile uint32_t* failed = tslot + 1;
  const Params& p = a.p;
  const int slices = V / N, unit = blockIdx.x / slices, v0 = (blockIdx.x % slices) * N;
  const int hv = unit % p.HV, hk = hv / (p.HV / p.H), seq = ranked_sequence(p, unit / p.HV, tslot + 2);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  long tok0;
  int len;
  const bool in_order = seq_tokens(p.cu, p.T, p.num_seqs, nullptr, seq, tok0, len);
  const int nch = num_chunks(len), slot0 = first_slot(a, seq, tok0);
  if (tid == 0) {
    for (int b = 0; b < NBAR; ++b) mbar_init(&bars[b], b >= SREADY && b <= OUTREADY ? NW : 1);
    *failed = 0u;
    fence_mbar_init();
  }
  if (warp == NW) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  wait_for_previous_kernel();  // the records, the cleared status
  let_next_kernel_start();
  if (!in_order && tid == 0) atomicOr(p.status, kStatusBounds);
  auto wait = [&](int b, uint32_t parity) { return wait_warp(&bars[b], parity, a.wait_ns, failed, p.status); };
  // the loader's keep a short limit from the first look on
  auto wait_load = [&](int b, uint32_t parity) {
    return a.wait_ns < kPollNs ? wait_longer(&bars[b], parity, a.wait_ns, failed, p.status) : wait(b, parity);
  };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[b]);
  };

  if (warp == NW + 1) {
    // ---------------------------------------------------------------- loads ---
    auto record = [&](int n) { return a.rec + (static_cast<size_t>(slot0 + n) * p.HV + hv) * kRecBytes; };
    auto load = [&](int n) {
      if (lane == 0) {
        uint8_t* st = sm + (n % 3) * L::STAGE;
        uint64_t* full = &bars[FULL + n % 3];
        const int tok = static_cast<int>(tok0 + C * static_cast<long>(n));
        mbar_arrive_expect_tx_relaxed(full, L::STAGE);
#pragma unroll
        for (int b = 0; b < K / 64; ++b) {
          tma_load_3d(st + b * kTileBytes, &maps.k, full, 64 * b, hk, tok);
          tma_load_3d(st + b * kTileBytes + 8192, &maps.q, full, 64 * b, hk, tok);
        }
        bulk_load(st + L::FAC, record(n) + kRecFactors, 1024, full);
        tma_load_3d(st + L::VS, &maps.v, full, v0, hv, tok);
      }
      __syncwarp();
    };
    auto load_t = [&](int n) {
      if (lane == 0) {
        mbar_arrive_expect_tx_relaxed(&bars[TFULL + (n & 1)], 2 * kTileBytes);
        bulk_load(sm + L::TT + (n & 1) * 2 * kTileBytes, record(n), 2 * kTileBytes, &bars[TFULL + (n & 1)]);
      }
      __syncwarp();
    };
    int nf = 0, nt = 0;
    for (; nf < 3 && nf < nch; ++nf) {
      load(nf);
      if (nf < 2) load_t(nt++);
    }
    for (int n = 1; n < nch; ++n) {
      if (nt < nch) {                              // free once step 2 of the chunk before is done
        if (!wait_load(TFREE + ((n - 1) & 1), ((n - 1) >> 1) & 1)) break;
        load_t(nt++);
      }
      if (nf < nch) {                              // a stage's readers are done once the next chunk's products start
        if (!wait_load(EMPTY + (n - 1) % 3, ((n - 1) / 3) & 1)) break;
        load(nf++);
      }
    }
    // what was issued lands before the CTA gives up its memory
    for (int m = nf < 3 ? 0 : nf - 3; m < nf; ++m) mbar_wait(&bars[FULL + m % 3], (m / 3) & 1, kDrainNs);
    for (int m = nt < 2 ? 0 : nt - 2; m < nt; ++m) mbar_wait(&bars[TFULL + (m & 1)], (m >> 1) & 1, kDrainNs);
  } else if (warp == NW) {
    // ------------------------------------------------------------- products ---
    const uint32_t sb = smem_u32(sm);
    constexpr uint32_t id64 = idesc_f16kind(64, 2 * N) | IDESC_B_MN_MAJOR;
    constexpr uint32_t idk = idesc_f16kind(128, 2 * N) | IDESC_A_MN_MAJOR | IDESC_B_MN_MAJOR;  // (K = 64: the other lanes' rows are some other tile)
    const uint64_t ds = sdesc(sb + L::S, 128 * 128, 1024, 2), dy = sdesc(sb + L::Y, C * 128, 1024, 2), dv = sdesc(sb + L::VN, C * 128, 1024, 2);
    auto times_s = [&](uint32_t d, uint64_t rows) {
#pragma unroll
      for (int b = 0; b < K / 64; ++b) umma4<32, 2048>(d, rows + (b * kTileBytes >> 4), ds + (b * 8192 >> 4), id64, b > 0);
    };
    auto times_y = [&](uint32_t d, uint64_t rows) {  // high and low parts of T or R
      umma4<32, 2048>(d, rows, dy, id64, 0u);
      umma4<32, 2048>(d, rows + (kTileBytes >> 4), dy, id64, 1u);
    };
    for (int n = 0; n < nch; ++n) {
      const uint32_t ph = n & 1, st = sb + (n % 3) * L::STAGE;
      const uint64_t dkq = sdesc_sw128(st), dkt = sdesc(st, kTileBytes, 1024, 2), dt = sdesc_sw128(sb + L::TT + ph * 2 * kTileBytes);
      if (!wait(FULL + n % 3, (n / 3) & 1)) break;
      if (!wait(SREADY, ph)) break;
      tc_fence_after();
      times_s(tmem + TK, dkq);
      umma_commit_warp(&bars[D1]);
      if (n > 0 && lane == 0) mbar_arrive(&bars[EMPTY + (n - 1) % 3]);
      __syncwarp();
      times_s(tmem + TQ + TURN * ph, dkq + (8192 >> 4));
      if (!wait(TFULL + ph, (n >> 1) & 1)) break;
      if (!wait(YREADY, ph)) break;
      tc_fence_after();
      times_y(tmem + thin::TT, dt);
      umma_commit_warp(&bars[D2]);
      times_y(tmem + TR + TURN * ph, dt + (8192 >> 4));
      umma_commit_warp(&bars[TFREE + ph]);
      if (!wait(VREADY, ph)) break;
      tc_fence_after();
      umma4<2048, 2048>(tmem + TD3, dkt, dv, idk, 0u);
      umma_commit_warp(&bars[D3]);
    }
    umma_commit_warp(&bars[DRAIN]);                // what is in flight ends before the CTA gives up its memory
    mbar_wait(&bars[DRAIN], 0, kDrainNs);
  } else if (warp == NW + 2) {
    // --------------------------------------------------------------- stores ---
    for (int n = 0; n < nch; ++n) {
      if (!wait(OUTREADY, n & 1)) break;
      if (lane == 0) {
        if (C * n + C <= len) {
          tma_store_3d(&maps.o, sm + L::OUT, v0, hv, static_cast<int>(tok0 + C * static_cast<long>(n)));
          bulk_commit();
        }
        bulk_wait_read();
        mbar_arrive(&bars[OUTFREE]);
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_read();
  } else {
    // ------------------------------------------ state, Y, vn, output ---
    const int quad = warp & 3, cg = warp >> 2, c0 = 16 * cg;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16) + c0;
    // S: a key dim a thread, 16 columns
    const int r = 32 * quad + lane;
    const size_t soff = ((static_cast<size_t>(seq) * p.HV + hv) * K + r) * V + v0 + c0;
    // tokens: rows i, i + 8; and the row of this thread's address in tile accesses
    const int i = 16 * quad + (lane >> 2), ir = 16 * quad + (lane & 15), ch = 2 * cg + (lane >> 4);
    const uint32_t in_v = sw64(ir, ch), in_y = sw128(ir, ch), in_ylow = sw128(ir, 4 + ch);
    uint64_t s[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t = p.s0 && r < K ? *reinterpret_cast<const float4*>(p.s0 + soff + 4 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[2 * j] = pack2f(t.x, t.y);
      s[2 * j + 1] = pack2f(t.z, t.w);
    }
    put_parts<N>(sm + L::S, 0, r, c0, s);
    fence_proxy_async_smem();
    arrive(SREADY);
    uint64_t x[4], y[4], bv[4], fe[2], fo[2], fy[2], gamma = 0;  // of the chunk: beta v, E, scale G, -beta G
    uint32_t w[4], wl[4];
    auto fetch = [&](int n) {                      // a chunk's v and factors
      if (!wait(FULL + n % 3, (n / 3) & 1)) return false;
      uint8_t* st = sm + (n % 3) * L::STAGE;
      const float* fac = reinterpret_cast<const float*>(st + L::FAC);
      if (tid == 0 && fac[kRecFailed] != 0.f) atomicOr(p.status, kStatusTimeout);
      ldmatrix_x4(smem_u32(st + L::VS + in_v), w);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float g = fac[i + 8 * e], tail = fac[64 + i + 8 * e], be = fac[128 + i + 8 * e];
        fe[e] = pack2f(tail, tail);
        fo[e] = pack2f(p.scale * g, p.scale * g);
        fy[e] = pack2f(-be * g, -be * g);
#pragma unroll
        for (int m = 0; m < 2; ++m)
          bv[2 * m + e] = mul2(pack2f(be, be), pack2f(__uint_as_float(w[2 * m + e] << 16), __uint_as_float(w[2 * m + e] & 0xFFFF0000u)));
      }
      gamma = pack2f(fac[kRecGamma], fac[kRecGamma]);
      // rows past the end hold the next sequence's tokens, whatever they are: zero wherever a
      // sum over tokens meets them
      if (tid < C && tid >= len - C * n) {
#pragma unroll 1
        for (int c = 0; c < 8 * (K / 64); ++c)
          *reinterpret_cast<uint4*>(st + (c >> 3) * kTileBytes + sw128(tid, c & 7)) = make_uint4(0, 0, 0, 0);
      }
      return true;
    };
    auto put_y = [&](uint8_t* tile) {              // y as an operand's two parts
#pragma unroll
      for (int j = 0; j < 4; ++j) split2(y[j], w[j], wl[j]);
      stmatrix_x4(smem_u32(tile + in_y), w);
      stmatrix_x4(smem_u32(tile + in_ylow), wl);
      fence_proxy_async_smem();
      tc_fence_before();
    };
    uint64_t fo_last[2];
    auto output = [&](int n) {                     // of a chunk whose step 3 is done, and so its products
      frag_ld(tl + TQ + TURN * (n & 1), y);
      frag_ld(tl + TR + TURN * (n & 1), x);
      if (n > 0 && !wait(OUTFREE, (n - 1) & 1)) return false;
      const int rows = len - C * n;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = pack_pair(fma2(fo_last[j & 1], y[j], x[j]));
        const int row = i + 8 * (j & 1);
        if (rows < C && row < rows)
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) +
                                       (static_cast<size_t>(tok0 + C * static_cast<long>(n) + row) * p.HV + hv) * V + v0 + c0 +
                                       8 * (j >> 1) + 2 * (lane & 3)) = w[j];
      }
      if (rows >= C) stmatrix_x4(smem_u32(sm + L::OUT + in_v), w);
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(OUTREADY);
      return true;
    };
    bool good = nch == 0 || fetch(0);
    for (int n = 0; n < nch && good; ++n) {
      const uint32_t ph = n & 1;
      const int rows = len - C * n;                // of the chunk, from the first; 64 and more: all
      if (!(good = wait(D1, ph))) break;
      tc_fence_after();
      frag_ld(tl + TK, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {                // beta (v - G k S)
        y[j] = fma2(fy[j & 1], x[j], bv[j]);
        if (i + 8 * (j & 1) >= rows) y[j] = 0;
      }
      put_y(sm + L::Y);
      arrive(YREADY);
      if (n > 0 && !(good = output(n - 1))) break;
      fo_last[0] = fo[0];
      fo_last[1] = fo[1];
      if (!(good = wait(D2, ph))) break;
      tc_fence_after();
      frag_ld(tl + thin::TT, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul2(fe[j & 1], x[j]);   // E vn
      put_y(sm + L::VN);
      arrive(VREADY);
      const uint64_t gm = gamma;
      if (n + 1 < nch && !(good = fetch(n + 1))) break;
      if (!(good = wait(D3, ph))) break;
      tc_fence_after();
      uint64_t z[8];
      tmem_ld_parts<N>(tl + TD3, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = fma2(gm, s[j], z[j]);
      put_parts<N>(sm + L::S, 0, r, c0, s);
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(SREADY);
    }
    if (good && nch > 0) good = output(nch - 1);
    if (good && p.sfin && r < K) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4 t;
        unpack2f(s[2 * j], t.x, t.y);
        unpack2f(s[2 * j + 1], t.z, t.w);
        *reinterpret_cast<float4*>(p.sfin + soff + 4 * j) = t;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == NW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------- chain, 128 columns wide ---
// The same recurrence turned over, for V = 128 where the slices of 32 columns do not fit the
// SMs at once, and in the backward: one CTA per pair, lane = value column, all transposed:
//   1. D1 = S^T [k; q]^T    M = 128 columns of S, N = 64 + 64 tokens, K = key dims
//   2. D2 = Y^T [T; R]^T    N = 64 + 64 tokens, K = 64 tokens
//   3. D3 = (E vn)^T k      N = key dims, K = 64
// S, Y and E vn are the A operands and lie in TMEM (two bf16 parts, each a product of its own
// that adds to the same accumulator), so a product reads only its B operand from shared
// memory, nothing is staged there in parts, and all 16 warps run one and the same code in
// all three steps (a warp: 32 columns, 16 tokens or K / 4 key dims) -- against the
// 64-column slices, whose two halves run different code.
//
// 370 us for 16 packed sequences (46402 tokens, 32 heads, 23424 chunks and heads), 2.4 us a
// chunk: the tensor pipes are active in 51 % of an SM's cycles, 1.2 us of it (each fp32 operand
// counts twice), the rest is the work between the products, one after the other.  64-column
// slices took 650.  Splitting the steps' operands in halves, products over the first while the
// second is made, did not help (687 us a call for 680).
//
// SAVE leaves out the q and R halves.  REVERSE:
//   1. D1 = dS'^T k^T
//   2. D2 = do^T R (do from shared memory as it is; it does not wait for step 1) + (E D1)^T T
//   3. D3 = (scale G do)^T q (issued with step 2's) - (G beta z)^T k
namespace wide {
constexpr int NW = 16, THREADS = 32 * (NW + 3);
using chain::Mode;
template <int K, Mode MODE>
struct Lay {
  static constexpr bool BWD = MODE != chain::FORWARD;
  // TMEM columns, all 512.  FORWARD: D1 has a q half, D3 lies over D1; REVERSE: z's operand over Y's
  static constexpr uint32_t TS = 0, TD1 = 128, TY = 256, TV = MODE == chain::REVERSE ? TY : 320, TW = 320,
                            TD2 = BWD ? 192 : 384, TD3 = BWD ? 384 : TD1;
  static constexpr uint32_t FAC = (K / 64) * kTileBytes;          // a stage: [k; q], row factors, v (two boxes), [T; R]
  static constexpr uint32_t VS = FAC + 1024;
  static constexpr uint32_t TT = VS + 2 * 8192;
  static constexpr uint32_t STAGE = BWD ? TT : TT + 2 * kTileBytes;  // (the others keep one buffer of [T; R])
  static constexpr uint32_t TT1 = 2 * STAGE;
  static constexpr uint32_t OUT = TT1 + (BWD ? 2 * kTileBytes : 0);  // o: two boxes of 64 rows x 64; or vn (z) in two parts
  static constexpr uint32_t SF = OUT + (BWD ? 4 : 2) * 8192;         // S (dS') in fp32
  static constexpr uint32_t BAR = SF + (BWD ? K * 512 : 0);
  static constexpr uint32_t SLACK = 832;
  static constexpr uint32_t SMEM = BAR + 192 + SLACK;
  static constexpr uint32_t TX = (MODE == chain::SAVE ? (K / 64) * 8192 : (K / 64) * kTileBytes) + 1024 + 2 * 8192 +
                                 (BWD ? 0 : 2 * kTileBytes);
  static_assert(SMEM <= 232448 && STAGE % 1024 == 0, "shared memory");
};
enum { FULL0 = 0, FULL1, EMPTY0, EMPTY1, TFULL, TFREE, D1, D1Q, D2, D2R, D3, SREADY, YREADY, VREADY, QREADY, SFREADY, OUTREADY,
       SFFREE, OUTFREE, DRAIN, NBAR };
static_assert(NBAR * 8 + 12 <= 192, "barriers, the TMEM address, the failure flag, the sequence");

// A thread's 16 values of a [32 columns, 16 tokens] block, in pairs of neighbouring tokens: pair
// 4 h + 2 m + r is column 16 h + 8 r + lane / 4, tokens 8 m + 2 (lane % 4) and one on -- the
// fragments of the 16-lane TMEM accesses and of transposed 8 x 8 tiles in shared memory.  With
// a column a thread instead, v and o took 16 16-bit accesses a thread and the row factors 8
// each (here 2).
__device__ __forceinline__ void block_ld(uint32_t t, uint64_t (&x)[8]) {
  float u[16];
  tmem_ld_16x256b_x2(t, u);
  tmem_ld_16x256b_x2(t + (16u << 16), u + 8);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = pack2f(u[2 * j], u[2 * j + 1]);
}
// ... as the two parts of an A operand, the low part's columns 32 on
__device__ __forceinline__ void block_parts(uint32_t t, const uint64_t (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split2(x[4 * h + j], a[j], b[j]);
    tmem_st_16x128b_x2(t + (static_cast<uint32_t>(16 * h) << 16), a[0], a[1], a[2], a[3]);
    tmem_st_16x128b_x2(t + (static_cast<uint32_t>(16 * h) << 16) + 32, b[0], b[1], b[2], b[3]);
  }
  tmem_st_wait();
}

// CNT values of a lane as the two parts of an A operand in TMEM (pairs: one column).
template <int CNT>
__device__ __forceinline__ void parts_to_tmem(uint32_t hi, uint32_t lo, const uint64_t (&x)[CNT / 2]) {
  uint32_t h[CNT / 2], l[CNT / 2];
#pragma unroll
  for (int j = 0; j < CNT / 2; ++j) split2(x[j], h[j], l[j]);
  if constexpr (CNT == 16) {
    tmem_st8u(hi, h);
    tmem_st8u(lo, l);
  } else {
    tmem_st16u(hi, h);
    tmem_st16u(lo, l);
  }
  tmem_st_wait();
}
}  // namespace wide

template <int K, chain::Mode MODE>
__device__ __forceinline__ void wide_body(const ChainMaps& maps, const ChunkParams& a, int unit, uint8_t* raw) {
  using L = wide::Lay<K, MODE>;
  using namespace wide;
  using namespace chain;
  constexpr int NW = wide::NW, V = 128, DPT = K / 4;   // DPT: key dims of a thread's share of S
  const uint32_t shift = (1024u - (smem_u32(raw) & 1023u)) & 1023u;
  uint8_t* sm = raw + shift;
  if (shift > L::SLACK) {
    if (threadIdx.x == 0) atomicOr(a.p.status, kStatusTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + wide::NBAR);
  volatile uint32_t* failed = tslot + 1;
  const Params& p = a.p;
  const int hv = unit % p.HV, hk = hv / (p.HV / p.H), seq = ranked_sequence(p, unit / p.HV, tslot + 2);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  long tok0;
  int len;
  const bool in_order = seq_tokens(p.cu, p.T, p.num_seqs, nullptr, seq, tok0, len);
  const int nch = num_chunks(len), slot0 = first_slot(a, seq, tok0);
  const auto chunk = [&](int n) { return MODE == REVERSE ? nch - 1 - n : n; };  // of step n
  if (tid == 0) {
    for (int b = 0; b < wide::NBAR; ++b) mbar_init(&bars[b], b >= wide::SREADY && b <= wide::OUTREADY ? NW : 1);
    *failed = 0u;
    fence_mbar_init();
  }
  if (warp == NW) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  wait_for_previous_kernel();  // the records, the cleared status
  let_next_kernel_start();
  if (!in_order && tid == 0) atomicOr(p.status, kStatusBounds);
  auto wait = [&](int b, uint32_t parity) { return wait_warp(&bars[b], parity, a.wait_ns, failed, p.status); };
  // the loader's keep a short limit from the first look on
  auto wait_load = [&](int b, uint32_t parity) {
    return a.wait_ns < kPollNs ? wait_longer(&bars[b], parity, a.wait_ns, failed, p.status) : wait(b, parity);
  };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[b]);
  };

  if (warp == NW + 1) {
    // ---------------------------------------------------------------- loads ---
    auto record = [&](int n) { return a.rec + (static_cast<size_t>(slot0 + chunk(n)) * p.HV + hv) * kRecBytes; };
    auto load = [&](int n) {
      if (lane == 0) {
        uint8_t* st = sm + (n & 1) * L::STAGE;
        uint64_t* full = &bars[wide::FULL0 + (n & 1)];
        const int tok = static_cast<int>(tok0 + C * static_cast<long>(chunk(n)));
        mbar_arrive_expect_tx_relaxed(full, L::TX);
#pragma unroll
        for (int b = 0; b < K / 64; ++b) {
          tma_load_3d(st + b * kTileBytes, &maps.k, full, 64 * b, hk, tok);
          if (MODE != SAVE) tma_load_3d(st + b * kTileBytes + 8192, &maps.q, full, 64 * b, hk, tok);
        }
        bulk_load(st + L::FAC, record(n) + kRecFactors, 1024, full);
        tma_load_3d(st + L::VS, &maps.v, full, 0, hv, tok);
        tma_load_3d(st + L::VS + 8192, &maps.v, full, 64, hv, tok);
        if (MODE == FORWARD) bulk_load(st + L::TT, record(n), 2 * kTileBytes, full);
      }
      __syncwarp();
    };
    auto load_t = [&](int n) {  // the one buffer of [T; R]: T alone for SAVE
      if (lane == 0) {
        mbar_arrive_expect_tx_relaxed(&bars[wide::TFULL], MODE == SAVE ? 16384 : 2 * kTileBytes);
        bulk_load(sm + L::TT1, record(n), MODE == SAVE ? 8192 : 2 * kTileBytes, &bars[wide::TFULL]);
        if (MODE == SAVE) bulk_load(sm + L::TT1 + kTileBytes, record(n) + kTileBytes, 8192, &bars[wide::TFULL]);
      }
      __syncwarp();
    };
    int nf = 0, nt = 0;   // loads issued
    for (; nf < 2 && nf < nch; ++nf) load(nf);
    if (MODE != FORWARD && nch > 0) load_t(nt++);
    for (int n = 1; n < nch; ++n) {
      if (MODE != FORWARD) {                       // free once step 2 of the chunk before is done
        if (!wait_load(wide::TFREE, (n - 1) & 1)) break;
        load_t(nt++);
      }
      if (nf < nch) {                              // a stage's readers are done once the next chunk's products start
        if (!wait_load(wide::EMPTY0 + ((n - 1) & 1), ((n - 1) >> 1) & 1)) break;
        load(nf++);
      }
    }
    // what was issued lands before the CTA gives up its memory
    for (int m = nf < 2 ? 0 : nf - 2; m < nf; ++m) mbar_wait(&bars[wide::FULL0 + (m & 1)], (m >> 1) & 1, kDrainNs);
    if (nt > 0) mbar_wait(&bars[wide::TFULL], (nt - 1) & 1, kDrainNs);
  } else if (warp == NW) {
    // ------------------------------------------------------------- products ---
    const uint32_t sb = smem_u32(sm);
    constexpr uint32_t id64 = idesc_f16kind(128, 64), idk = idesc_f16kind(128, K) | IDESC_B_MN_MAJOR;
    auto s_times = [&](uint32_t d, uint64_t b) {   // both parts of S^T times 64 rows of [k; q]
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int kb = 0; kb < K / 64; ++kb)
          umma_ts4<32>(d, tmem + L::TS + h * (K / 2) + 32 * kb, b + (kb * kTileBytes >> 4), id64, h + kb > 0);
    };
    auto y_times = [&](uint32_t d, uint64_t b) {   // Y^T times 64 rows of [T; R]: high high, high low, low high
      constexpr uint32_t id = MODE == REVERSE ? id64 | IDESC_B_MN_MAJOR : id64, acc = MODE == REVERSE, step = MODE == REVERSE ? 2048 : 32;
      umma_ts4<step>(d, tmem + L::TY, b, id, acc);
      umma_ts4<step>(d, tmem + L::TY, b + (kTileBytes >> 4), id, 1u);
      umma_ts4<step>(d, tmem + L::TY + 32, b, id, 1u);
    };
    auto into_state = [&](uint32_t at, uint64_t b, uint32_t acc) {  // both parts of a [columns, tokens] operand times rows of q or k
      umma_ts4<2048>(tmem + L::TD3, tmem + at, b, idk, acc);
      umma_ts4<2048>(tmem + L::TD3, tmem + at + 32, b, idk, 1u);
    };
    for (int n = 0; n < nch; ++n) {
      const uint32_t ph = n & 1, st = sb + ph * L::STAGE, tt = MODE == FORWARD ? st + L::TT : sb + L::TT1;
      const uint64_t dkq = sdesc_sw128(st), dkt = sdesc(st, kTileBytes, 1024, 2);
      const uint64_t dt = MODE == REVERSE ? sdesc(tt, kTileBytes, 1024, 2) : sdesc_sw128(tt);
      if (!wait(wide::FULL0 + (n & 1), (n >> 1) & 1)) break;
      if (!wait(wide::SREADY, ph)) break;
      tc_fence_after();
      s_times(tmem + L::TD1, dkq);
      umma_commit_warp(&bars[wide::D1]);
      if (n > 0 && lane == 0) mbar_arrive(&bars[wide::EMPTY0 + ((n - 1) & 1)]);
      __syncwarp();
      if (MODE == FORWARD) {
        s_times(tmem + L::TD1 + 64, dkq + (8192 >> 4));
        umma_commit_warp(&bars[wide::D1Q]);
      } else if (!wait(wide::TFULL, ph)) {
        break;
      }
      if (MODE == REVERSE) {
        if (!wait(wide::QREADY, ph)) break;
        tc_fence_after();
        const uint64_t dd = sdesc(st + L::VS, 8192, 1024, 2);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
          umma4<2048, 2048>(tmem + L::TD2, dd, dt + ((8192 + h * kTileBytes) >> 4), id64 | IDESC_A_MN_MAJOR | IDESC_B_MN_MAJOR, h);
        into_state(L::TW, dkt + (8192 >> 4), 0u);
      }
      if (!wait(wide::YREADY, ph)) break;
      tc_fence_after();
      y_times(tmem + L::TD2, dt);
      umma_commit_warp(&bars[wide::D2]);
      if (MODE == FORWARD) {
        y_times(tmem + L::TD2 + 64, dt + (8192 >> 4));
        umma_commit_warp(&bars[wide::D2R]);
      } else {
        umma_commit_warp(&bars[wide::TFREE]);
      }
      if (!wait(wide::VREADY, ph)) break;
      tc_fence_after();
      into_state(L::TV, dkt, MODE == REVERSE);
      umma_commit_warp(&bars[wide::D3]);
    }
    umma_commit_warp(&bars[wide::DRAIN]);          // what is in flight ends before the CTA gives up its memory
    mbar_wait(&bars[wide::DRAIN], 0, kDrainNs);
  } else if (warp == NW + 2) {
    // --------------------------------------------------------------- stores ---
    for (int n = 0; n < nch; ++n) {
      const int c = chunk(n);
      const size_t cu = static_cast<size_t>(slot0 + c) * p.HV + hv;
      if (MODE != FORWARD) {
        if (!wait(wide::SFREADY, n & 1)) break;
        if (lane == 0) {
          bulk_store((MODE == SAVE ? a.states : a.dstates) + cu * K * V, sm + L::SF, K * V * 4);
          bulk_commit();
          bulk_wait_read();
          mbar_arrive(&bars[wide::SFFREE]);
        }
        __syncwarp();
      }
      if (!wait(wide::OUTREADY, n & 1)) break;
      if (lane == 0) {
        if (MODE != FORWARD) {
          bulk_store((MODE == SAVE ? a.vn : a.z) + cu * (4 * C * V), sm + L::OUT, 4 * C * V);
        } else if (C * c + C <= len) {
          const int tok = static_cast<int>(tok0 + C * static_cast<long>(c));
          tma_store_3d(&maps.o, sm + L::OUT, 0, hv, tok);
          tma_store_3d(&maps.o, sm + L::OUT + 8192, 64, hv, tok);
        }
        bulk_commit();
        bulk_wait_read();
        mbar_arrive(&bars[wide::OUTFREE]);
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_read();
  } else {
    // ------------------------------------------ state, Y, vn (z), output ---
    const int quad = warp & 3, grp = warp >> 2, t0 = 16 * grp, d0 = DPT * grp;
    const int col = 32 * quad + lane;              // TMEM lane: value column
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    const uint32_t ts = tl + L::TS + d0 / 2;
    // this thread's row of the block's 8 x 8 tiles (its first 16 columns; the others: ^ 32)
    const uint32_t toff = (quad >> 1) * 8192 + (t0 / 8 + (lane >> 4)) * 1024 + (lane & 7) * 128 +
                          ((4 * (quad & 1) + ((lane >> 3) & 1)) ^ (lane & 7)) * 16;
    const int tk = t0 + 2 * (lane & 3);            // pair j: tokens tk + 8 ((j >> 1) & 1) and one on
    const size_t soff = ((static_cast<size_t>(seq) * p.HV + hv) * K + d0) * V + col;
    const float* first = MODE == REVERSE ? a.dfin : p.s0;
    float* final = MODE == FORWARD ? p.sfin : MODE == REVERSE ? a.ds0 : nullptr;
    uint64_t s[DPT / 2];
#pragma unroll
    for (int j = 0; j < DPT / 2; ++j)
      s[j] = first ? pack2f(first[soff + 2 * j * V], first[soff + (2 * j + 1) * V]) : 0ull;
    parts_to_tmem<DPT>(ts, ts + K / 2, s);
    tc_fence_before();
    arrive(wide::SREADY);
    const uint64_t scale = pack2f(p.scale, p.scale);
    bool good = true;
    for (int n = 0; n < nch; ++n) {
      const uint32_t ph = n & 1;
      uint8_t* st = sm + ph * L::STAGE;
      const float* fac = reinterpret_cast<const float*>(st + L::FAC);
      const int c = chunk(n), rows = len - C * c;  // rows of the chunk, from the first; 64 and more: all
      uint64_t x[8], y[8], o[8];
      // rows past the end hold the next sequence's tokens, whatever they are: zero wherever a
      // sum over tokens meets them
      auto zero_past_end = [&](uint64_t (&w)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v0, v1;
          unpack2f(w[j], v0, v1);
          const int t = tk + 8 * ((j >> 1) & 1);
          w[j] = pack2f(t < rows ? v0 : 0.f, t + 1 < rows ? v1 : 0.f);
        }
      };
      auto factors = [&](int at, uint64_t (&f)[2]) {  // of this thread's tokens
#pragma unroll
        for (int m = 0; m < 2; ++m) f[m] = *reinterpret_cast<const uint64_t*>(fac + at + tk + 8 * m);
      };
      auto put_block = [&](uint8_t* tile, const uint32_t (&w)[8]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          stmatrix_x4_trans(smem_u32(tile + (toff ^ (32 * h))), w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
      };
      uint64_t fg[2], fe[2], fb[2];                // G, E, beta
      if (!(good = wait(wide::FULL0 + (n & 1), (n >> 1) & 1))) break;
      if (tid == 0 && fac[kRecFailed] != 0.f) atomicOr(p.status, kStatusTimeout);
#pragma unroll
      for (int h = 0; h < 2; ++h) {                // v (do)
        uint32_t u[4];
        ldmatrix_x4_trans(smem_u32(st + L::VS + (toff ^ (32 * h))), u);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[4 * h + j] = pack2f(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xFFFF0000u));
      }
      factors(0, fg);
      factors(64, fe);
      factors(128, fb);
      if (rows < C) {
        if (tid < (MODE == REVERSE ? 3 * C : C) && (tid & 63) >= rows) {  // rows of k, of q, of do
          uint8_t* tile = tid < 2 * C ? st : st + L::VS;
          const uint32_t step = tid < 2 * C ? kTileBytes : 8192u;
          const int row = tid < 2 * C ? tid : tid - 2 * C, chunks = tid < 2 * C ? 8 * (K / 64) : 16;
#pragma unroll 1
          for (int ch = 0; ch < chunks; ++ch)
            *reinterpret_cast<uint4*>(tile + (ch >> 3) * step + sw128(row, ch & 7)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      if (MODE == REVERSE) {                       // scale G do
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = mul2(mul2(scale, fg[(j >> 1) & 1]), y[j]);
        if (rows < C) zero_past_end(y);
        block_parts(tl + L::TW + t0 / 2, y);
        tc_fence_before();
        arrive(wide::QREADY);
      }
      if (MODE != REVERSE) {                       // beta v, -beta G
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = mul2(fb[(j >> 1) & 1], y[j]);
#pragma unroll
        for (int m = 0; m < 2; ++m) fb[m] = mul2(pack2f(-1.f, -1.f), mul2(fb[m], fg[m]));
      }
      if (!(good = wait(wide::D1, ph))) break;
      tc_fence_after();
      block_ld(tl + L::TD1 + t0, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (MODE == REVERSE) {                     // E k dS'
          y[j] = mul2(fe[(j >> 1) & 1], x[j]);
        } else {                                   // beta v - (beta G) k S
          y[j] = fma2(fb[(j >> 1) & 1], x[j], y[j]);
        }
      }
      if (rows < C) zero_past_end(y);
      block_parts(tl + L::TY + t0 / 2, y);
      tc_fence_before();
      arrive(wide::YREADY);
      if (MODE == FORWARD) {                       // while step 2 runs: scale G q S
        if (!(good = wait(wide::D1Q, ph))) break;
        tc_fence_after();
        block_ld(tl + L::TD1 + 64 + t0, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = mul2(mul2(scale, fg[(j >> 1) & 1]), o[j]);
      } else {                                     // S (dS') in fp32 to its staging: rows of 16 chunks, swizzled
        if (n > 0 && !(good = wait(wide::SFFREE, (n - 1) & 1))) break;
        uint8_t* sf = sm + L::SF + (col >> 6) * (K * 256) + d0 * 256 + (col & 3) * 4;
        const uint32_t ch = ((col & 63) >> 2) << 4;
#pragma unroll
        for (int j = 0; j < DPT / 2; ++j) {
          float u, w;
          unpack2f(s[j], u, w);
          *reinterpret_cast<float*>(sf + 2 * j * 256 + (ch ^ (((2 * j) & 7) << 4))) = u;
          *reinterpret_cast<float*>(sf + (2 * j + 1) * 256 + (ch ^ (((2 * j + 1) & 7) << 4))) = w;
        }
        fence_proxy_async_smem();
        arrive(wide::SFREADY);
      }
      if (!(good = wait(wide::D2, ph))) break;
      tc_fence_after();
      block_ld(tl + L::TD2 + t0, x);
      if (MODE == REVERSE && rows < C) zero_past_end(x);  // (vn is zero there by itself: row i of T is e_i)
#pragma unroll
      for (int j = 0; j < 8; ++j)                  // E vn, or -G beta z
        y[j] = MODE == REVERSE ? mul2(mul2(pack2f(-1.f, -1.f), mul2(fg[(j >> 1) & 1], fb[(j >> 1) & 1])), x[j])
                               : mul2(fe[(j >> 1) & 1], x[j]);
      block_parts(tl + L::TV + t0 / 2, y);
      tc_fence_before();
      arrive(wide::VREADY);
      if (MODE == FORWARD) {                       // while step 3 runs: the output
        if (!(good = wait(wide::D2R, ph))) break;
        tc_fence_after();
        block_ld(tl + L::TD2 + 64 + t0, x);
      }
      if (n > 0 && !(good = wait(wide::OUTFREE, (n - 1) & 1))) break;
      uint32_t w[8], wl[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (MODE == FORWARD) w[j] = pack_pair(add2(o[j], x[j]));
        else split2(x[j], w[j], wl[j]);            // vn (z) as it is, in two parts
      }
      if (MODE != FORWARD) {
        put_block(sm + L::OUT, w);
        put_block(sm + L::OUT + 16384, wl);
      } else if (rows >= C) {
        put_block(sm + L::OUT, w);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = tk + 8 * ((j >> 1) & 1);
          uint16_t* op = static_cast<uint16_t*>(p.out) +
                         (static_cast<size_t>(tok0 + C * static_cast<long>(c) + t) * p.HV + hv) * V + 32 * quad + 16 * (j >> 2) +
                         8 * (j & 1) + (lane >> 2);
          if (t < rows) op[0] = static_cast<uint16_t>(w[j]);
          if (t + 1 < rows) op[static_cast<size_t>(p.HV) * V] = static_cast<uint16_t>(w[j] >> 16);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(wide::OUTREADY);
      const float gm = fac[kRecGamma];
      const uint64_t gamma = pack2f(gm, gm);
      if (!(good = wait(wide::D3, ph))) break;
      tc_fence_after();
      float z[DPT];
      if constexpr (DPT == 16) tmem_ld16(tl + L::TD3 + d0, z);
      else tmem_ld32(tl + L::TD3 + d0, z);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < DPT / 2; ++j) s[j] = fma2(gamma, s[j], pack2f(z[2 * j], z[2 * j + 1]));
      parts_to_tmem<DPT>(ts, ts + K / 2, s);
      tc_fence_before();
      arrive(wide::SREADY);
    }
    if (good && final) {
#pragma unroll
      for (int j = 0; j < DPT / 2; ++j) {
        float u, w;
        unpack2f(s[j], u, w);
        final[soff + 2 * j * V] = u;
        final[soff + (2 * j + 1) * V] = w;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == NW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int K>
__global__ void __launch_bounds__(wide::THREADS, 1) gdr_wide_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a) {
  extern __shared__ __align__(16) uint8_t raw[];
  wide_body<K, chain::FORWARD>(maps, a, blockIdx.x, raw);
}

template <int K>
__global__ void __launch_bounds__(wide::THREADS, 1) gdr_wide_chains_kernel(const __grid_constant__ ChainMaps maps,
                                                                          const __grid_constant__ ChainMaps maps_r,
                                                                          const ChunkParams a) {
  extern __shared__ __align__(16) uint8_t raw[];
  if (blockIdx.x & 1) wide_body<K, chain::REVERSE>(maps_r, a, blockIdx.x >> 1, raw);
  else wide_body<K, chain::SAVE>(maps, a, blockIdx.x >> 1, raw);
}

// The backward's two chains in one launch: even blocks SAVE (maps: v), odd blocks REVERSE
// (maps_r: d_out).  They share nothing but the records, so they run side by side.
template <int K>
__global__ void __launch_bounds__(chain::THREADS, 1) gdr_chains_kernel(const __grid_constant__ ChainMaps maps,
                                                                  const __grid_constant__ ChainMaps maps_r,
                                                                  const ChunkParams a) {
  extern __shared__ __align__(16) uint8_t raw[];
  if (blockIdx.x & 1) chain_body<K, chain::REVERSE>(maps_r, a, blockIdx.x >> 1, raw);
  else chain_body<K, chain::SAVE>(maps, a, blockIdx.x >> 1, raw);
}

// ------------------------------------------------------------------- host ---
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* ptr = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// 3-D map over a [tokens, heads, dim] bf16 tensor, boxes of `cols` dims x 64 tokens.
bool make_map(CUtensorMap* m, const void* base, int dim, int heads, long tokens, int cols) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(dim) * 2, static_cast<cuuint64_t>(heads) * dim * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(cols), 1, C};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int K>
cudaError_t launch_prep(const ChainMaps& maps, const ChunkParams& a, cudaStream_t st) {
  static LaunchState state;
  return launch_kernel(state, gdr_prep_kernel<K>, static_cast<unsigned>(a.slots) * a.p.HV, prep::NT, prep::SMEM, false, st,
                       maps, a);
}

template <int K>
cudaError_t launch_chain(const ChainMaps& maps, const ChunkParams& a, cudaStream_t st) {
  static LaunchState state;
  return launch_kernel(state, gdr_chain_kernel<K>, static_cast<unsigned>(a.p.num_seqs) * a.p.HV, chain::THREADS,
                       chain::Lay<K, chain::FORWARD>::SMEM, true, st, maps, a);
}

template <int K>
cudaError_t launch_thin(const ChainMaps& maps, const ChunkParams& a, int V, cudaStream_t st) {
  static LaunchState state;
  return launch_kernel(state, gdr_thin_kernel<K>, static_cast<unsigned>(a.p.num_seqs) * a.p.HV * (V / thin::N), thin::THREADS,
                       thin::Lay<K>::SMEM, true, st, maps, a, V);
}

template <int K>
cudaError_t launch_wide(const ChainMaps& maps, const ChunkParams& a, cudaStream_t st) {
  static LaunchState state;
  return launch_kernel(state, gdr_wide_kernel<K>, static_cast<unsigned>(a.p.num_seqs) * a.p.HV, wide::THREADS,
                       wide::Lay<K, chain::FORWARD>::SMEM, true, st, maps, a);
}
template <int K>
cudaError_t launch_wide_chains(const ChainMaps& maps, const ChainMaps& maps_r, const ChunkParams& a, cudaStream_t st) {
  constexpr uint32_t bytes = wide::Lay<K, chain::REVERSE>::SMEM;
  static_assert(bytes >= wide::Lay<K, chain::SAVE>::SMEM, "shared memory of the two chains");
  static LaunchState state;
  return launch_kernel(state, gdr_wide_chains_kernel<K>, 2u * static_cast<unsigned>(a.p.num_seqs) * a.p.HV, wide::THREADS, bytes,
                       true, st, maps, maps_r, a);
}

template <int K>
cudaError_t launch_chains(const ChainMaps& maps, const ChainMaps& maps_r, const ChunkParams& a, cudaStream_t st) {
  constexpr uint32_t bytes = chain::Lay<K, chain::REVERSE>::SMEM;   // the larger of the two
  static_assert(bytes >= chain::Lay<K, chain::SAVE>::SMEM, "shared memory of the two chains");
  static LaunchState state;
  return launch_kernel(state, gdr_chains_kernel<K>, 2u * static_cast<unsigned>(a.p.num_seqs) * a.p.HV,
                       chain::THREADS, bytes, true, st, maps, maps_r, a);
}

}  // namespace

// gdr_grad.cu
cudaError_t launch_grads(const ChainMaps& maps, const ChunkParams& a, int K, int V, cudaStream_t st);
cudaError_t launch_group_sum(const float* shares, void* dq, void* dk, size_t tokens, int H, int G, int K, cudaStream_t st);

// Slots of chunk records: every chunk (packed: floor(T / 64) and one more per sequence).
size_t chunk_slots(size_t tokens, size_t ns, bool packed, int T) {
  return packed ? tokens / C + ns : ns * ((static_cast<size_t>(T) + C - 1) / C);
}
size_t chunk_fwd_bytes(size_t slots, int HV) { return slots * HV * kRecBytes; }

cudaError_t launch_chunk_fwd(const Params& p, uint8_t* rec, unsigned long long wait_ns, int K, int V, cudaStream_t st) {
  const size_t tokens = p.cu ? static_cast<size_t>(p.T) : static_cast<size_t>(p.num_seqs) * p.T;
  ChunkParams a;
  std::memset(&a, 0, sizeof(a));
  a.p = p;
  a.rec = rec;
  a.wait_ns = wait_ns;
  a.chunks = (p.T + C - 1) / C;
  a.slots = static_cast<int>(chunk_slots(tokens, p.num_seqs, p.cu != nullptr, p.T));
  // Thin chains, 32 columns a CTA, while they fit the SMs at once: a step is latency, and more
  // CTAs are free (4096 tokens, V = 128, 32 pairs: 119 us, wide 180).  Beyond that a pair's
  // whole V in one CTA (64 pairs: wide 205, thin 226; 128 pairs: 256 and 432; V = 64, 128 pairs:
  // 247 and 272).
  const int N = static_cast<long>(p.num_seqs) * p.HV * (V / 32) <= sm_count() ? 32 : 64;
  ChainMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (!make_map(&maps.q, p.q, K, p.H, tokens, 64) || !make_map(&maps.k, p.k, K, p.H, tokens, 64) ||
      !make_map(&maps.v, p.v, V, p.HV, tokens, N) || !make_map(&maps.o, p.out, V, p.HV, tokens, N))
    return cudaErrorInvalidValue;
  cudaError_t e = K == 128 ? launch_prep<128>(maps, a, st) : launch_prep<64>(maps, a, st);
  if (e != cudaSuccess) return e;
  if (N == 64 && V == 128) return K == 128 ? launch_wide<128>(maps, a, st) : launch_wide<64>(maps, a, st);
  if (N == 32) return K == 128 ? launch_thin<128>(maps, a, V, st) : launch_thin<64>(maps, a, V, st);
  return K == 128 ? launch_chain<128>(maps, a, st) : launch_chain<64>(maps, a, st);
}

// Bytes of a backward's intermediates per (slot, value head): the record, S and dS', vn and z.
size_t chunk_bwd_bytes(size_t slots, int HV, int K, int V) {
  return slots * HV * (kRecBytes + 8 * static_cast<size_t>(K) * V + 8 * static_cast<size_t>(C) * V);
}

cudaError_t launch_chunk_bwd(const Params& p, const void* dout, const float* dfin, void* dq, void* dk, void* dv,
                             float* dg, float* dbeta, float* ds0, uint8_t* ws, float* shares,
                             unsigned long long wait_ns, int K, int V, cudaStream_t st) {
  const size_t tokens = p.cu ? static_cast<size_t>(p.T) : static_cast<size_t>(p.num_seqs) * p.T;
  ChunkParams a;
  std::memset(&a, 0, sizeof(a));
  a.p = p;
  a.wait_ns = wait_ns;
  a.chunks = (p.T + C - 1) / C;
  a.slots = static_cast<int>(chunk_slots(tokens, p.num_seqs, p.cu != nullptr, p.T));
  const size_t units = static_cast<size_t>(a.slots) * p.HV, kv = 4 * static_cast<size_t>(K) * V, cv = 4 * static_cast<size_t>(C) * V;
  a.rec = ws;
  a.states = reinterpret_cast<float*>(a.rec + units * kRecBytes);
  a.dstates = a.states + units * kv / 4;
  a.vn = a.rec + units * (kRecBytes + 2 * kv);
  a.z = a.vn + units * cv;
  a.dout = dout;
  a.dfin = dfin;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.ds0 = ds0;
  const bool grouped = p.HV != p.H;
  a.dq = grouped ? static_cast<void*>(shares) : dq;
  a.dk = grouped ? static_cast<void*>(shares + tokens * p.HV * K) : dk;
  ChainMaps maps, maps_r;
  std::memset(&maps, 0, sizeof(maps));
  if (!make_map(&maps.q, p.q, K, p.H, tokens, 64) || !make_map(&maps.k, p.k, K, p.H, tokens, 64) ||
      !make_map(&maps.v, p.v, V, p.HV, tokens, 64))
    return cudaErrorInvalidValue;
  maps_r = maps;
  if (!make_map(&maps_r.v, dout, V, p.HV, tokens, 64) || !make_map(&maps_r.o, dq, K, p.H, tokens, 64) ||
      !make_map(&maps_r.o2, dk, K, p.H, tokens, 64))
    return cudaErrorInvalidValue;
  cudaError_t e = K == 128 ? launch_prep<128>(maps, a, st) : launch_prep<64>(maps, a, st);
  if (e != cudaSuccess) return e;
  // (4096 tokens, 32 pairs: 439 us wide when 64-column slices, on twice the SMs, took 453)
  if (V == 128) e = K == 128 ? launch_wide_chains<128>(maps, maps_r, a, st) : launch_wide_chains<64>(maps, maps_r, a, st);
  else e = K == 128 ? launch_chains<128>(maps, maps_r, a, st) : launch_chains<64>(maps, maps_r, a, st);
  if (e != cudaSuccess) return e;
  if ((e = launch_grads(maps_r, a, K, V, st)) != cudaSuccess || !grouped) return e;
  return launch_group_sum(static_cast<const float*>(a.dq), dq, dk, tokens, p.H, p.HV / p.H, K, st);
}

}  // namespace gdr
}  // namespace kda
