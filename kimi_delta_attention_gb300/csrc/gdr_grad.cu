// gdr_grad.cu -- the gated delta rule's gradients of one chunk, all chunks in parallel,
// from what the two chains left (gdr_chunk.cu): S entering the chunk and dS' leaving it in
// fp32, vn and z = T^T (E k dS') + R^T do as operand images in two bf16 parts.
//
// With G, E, D, beta as in gdr_chunk.cuh, Z = z vn^T and dP = do vn^T (64 x 64):
//     dq    = scale G (do S^T) + A k,                        A  = scale dP D   (lower)
//     dk    = E (vn dS'^T) - G beta (z S^T) + A^T q + (B + B^T) k,
//                                                            B  = -beta Z D    (strictly lower)
//     dbeta = z . v - G k . (z S^T) + k . (B k) / beta
//     dgc   = scale G q . (do S^T) + q . (A k) + k . (B k) - k . (A^T q + B^T k)
//             - G beta k . (z S^T) - t,                      t  = E k . (vn dS'^T)
//     dgl   = sum t + gamma <S, dS'>   (of the chunk's last gc);  dg = suffix sums of dgc
// dv = beta z.  A row's decay gradient is what the row's
// products say: the gate multiplies whole rows, so every sum over D's entries is a dot of q
// or k with a product that dq or dk need anyway.  A's diagonal has D = 1 and would enter
// dgc twice with opposite signs; it stays out of the products and is added to dq and dk in
// fp32.  Where |beta| < 1e-20, B is taken with 1e-20 (an error of 1e-20), so that
// k . (B k) / beta = -sum_j G_ij D_ij Z_ij holds for beta = 0 too.  <S, dS'> is one number
// for 64 values of dg and cancels against the rows' terms, so it is taken from the fp32
// states (with their 16-bit parts it alone was off by 4e-6 of dg), and vn dS'^T, whose
// dots t every later dg sums up, takes dS' in three parts (dg off by 2.9e-6 in a model of
// the arithmetic, 4.3e-6 with two).  In calls of a few tokens and one head, whose few terms may
// cancel, dg is further off: 9.5e-6 the largest of some 570 drawn calls of all sizes.
//
// One CTA of 512 threads an SM, walking over the (chunk, value head) pairs.  Products on tcgen05 with M = 128: rows
// 0-63 belong to q's side (do; A), rows 64-127 to k's side (z, vn; B), stacked in shared
// memory so that one instruction serves both, and thread (lane r, quarter h) of the CTA owns
// row r and a quarter of the key dims throughout.
// 188 us for 2048 chunks and heads (K = V = 128), the tensor pipes active in 19 % of the cycles.  A unit takes 27000 cycles for 33000
// instructions: it is a chain of phases (loads, S and dS' into their parts, three groups of
// products, the rows of dq and dk) of which only the loads overlap with their neighbours, and
// these only where shared memory is free again (224 KB a unit: none to spare).  The loads are
// not the bound: started half a unit apart on half of the SMs, it took as long.
#include "gdr_chunk.cuh"

namespace kda {
namespace gdr {
namespace {

namespace grad {
constexpr int NT = 512;
// 64-row pieces of 8 KB in each 64-column block of V; neighbours make 128-row operands
// (do and z's high part later make room for the third part of dS', 128 rows at most)
enum { P_DO, P_ZH, P_ZERO, P_ZL, P_VL, P_VH, PIECES };
constexpr uint32_t BLOCK = PIECES * 8192;
template <int K, int V>
struct Lay {
  static constexpr uint32_t VB = V / 64;
  static constexpr uint32_t S = VB * BLOCK;               // S; later the A;B parts (low, high), then the halves' exchange
  static constexpr uint32_t CLO = S, CHI = S + kTileBytes;
  static constexpr uint32_t MAT = VB * K * 256;           // bytes of S or dS', fp32 or two parts
  static constexpr uint32_t QK = S + 2 * kTileBytes;      // [q; k], after A;B
  static constexpr uint32_t DS = S + 65536;               // dS'
  static constexpr uint32_t X = DS + MAT;                 // 2 x (gc high, low, beta), A's diagonal, z . v, warp sums
  static constexpr uint32_t BAR = X + (8 * C + 24) * 4;
  static constexpr uint32_t SLACK = 800;                  // for the base's alignment
  static constexpr uint32_t SMEM = BAR + 64 + SLACK;
};
static_assert(Lay<128, 128>::SMEM <= 232448 && Lay<64, 64>::DS >= Lay<64, 64>::QK + kTileBytes, "shared memory");
enum { LD_A = 0, LD_S, LD_D, LD_QK, M1, M2, M3, NBAR };
constexpr uint32_t E1 = 0, E2 = 128, E3 = 256, E4 = 320, E5A = 448, E5B = 256;  // TMEM columns

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A matrix from fp32 rows (256 bytes, 16-byte chunks swizzled by the row) into its two bf16
// parts in place: 8 rows are 2048 bytes of fp32, and one 1024-byte swizzle atom of each
// part.  A warp takes 8 rows at a time; lane: row lane / 4, columns 8 q and 8 (q + 4) with
// q = lane % 4.  `f(x, m)` sees the values and the 8-column chunk's number.
template <class F>
__device__ __forceinline__ void parts_in_place(uint8_t* mat, int groups, int warp, int lane, const F& f) {
  const int row = lane >> 2, q = lane & 3;
#pragma unroll 1
  for (int g = warp; g < groups; g += NT / 32) {
    uint8_t* at = mat + g * 2048;
    float x[2][8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = 2 * q + (e & 1) + 8 * (e >> 1);
      const float4 u = *reinterpret_cast<const float4*>(at + row * 256 + ((c ^ row) << 4));
      float* d = x[e >> 1] + 4 * (e & 1);
      d[0] = u.x; d[1] = u.y; d[2] = u.z; d[3] = u.w;
    }
    uint4 h[2], l[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      split8(x[e], h[e], l[e]);
      f(x[e], h[e], l[e], g, row, q + 4 * e);
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      *reinterpret_cast<uint4*>(at + row * 128 + (((q + 4 * e) ^ row) << 4)) = h[e];
      *reinterpret_cast<uint4*>(at + 1024 + row * 128 + (((q + 4 * e) ^ row) << 4)) = l[e];
    }
  }
}

struct Unit {
  int slot, hv, rows;
  long tok;
};
// (The helpers that run once a unit stay out of line.)  The next unit from `u` on that holds
// a chunk; `units` if there is none.
__device__ __noinline__ int next_unit(const ChunkParams& a, int u, int units, Unit& x) {
  for (; u < units; u += gridDim.x) {
    int seq;
    x.slot = u / a.p.HV;
    x.hv = u - x.slot * a.p.HV;
    if (find_chunk(a, x.slot, seq, x.tok, x.rows)) break;
  }
  return u;
}
// gc (high, low) and beta of a chunk's rows, by one warp.
__device__ __noinline__ void put_gates(float g0, float g1, float b0, float b1, float* to) {
  const int lane = threadIdx.x & 31;
  float h[2], l[2];
  gate_scan(g0, g1, lane, h, l);
  reinterpret_cast<float2*>(to)[lane] = make_float2(h[0], h[1]);
  reinterpret_cast<float2*>(to + C)[lane] = make_float2(l[0], l[1]);
  reinterpret_cast<float2*>(to + 2 * C)[lane] = make_float2(b0, b1);
}
// Wait for a phase that will come: the work waited for is this CTA's own copies and products.
// Running out of time is recorded; then it drains, for its memory may not go before them.
__device__ __noinline__ void wait_own(uint64_t* bar, uint32_t parity, uint64_t limit_ns, uint32_t* status,
                                      volatile uint32_t* never) {
  if (wait_phase(bar, parity, limit_ns, never)) return;
  atomicOr(status, kStatusTimeout);
  wait_phase(bar, parity, kDrainNs, never);
}
}  // namespace grad

// One CTA per SM walks over the units.  The next unit's loads start when the last products
// of this one are done and run under its epilogue (S after it), its gates are read under
// those products.  Everything is small loops: unrolled, the code was bound by instruction
// fetch (207 us for 2048 chunks and heads, a CTA each).
template <int K, int V>
__global__ void __launch_bounds__(grad::NT, 1) gdr_grad_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a,
                                                               int units) {
  using L = grad::Lay<K, V>;
  using namespace grad;
  constexpr int VB = V / 64, KB = K / 64, DPT = K / 4;
  extern __shared__ __align__(16) uint8_t raw[];
  const uint32_t shift = (1024u - (smem_u32(raw) & 1023u)) & 1023u;  // 0: nothing lies before the dynamic part
  uint8_t* sm = raw + shift;
  const Params& p = a.p;
  if (shift > L::SLACK) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  float* gates = reinterpret_cast<float*>(sm + L::X);
  float* diag = gates + 6 * C;
  float* zvs = diag + C;
  float* wsum = zvs + C;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + NBAR);
  volatile uint32_t* never = tslot + 1;   // (zero)
  struct Upcoming {
    Unit unit;
    int u;
  };
  Upcoming* upcoming = reinterpret_cast<Upcoming*>(wsum + 16);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;

  Unit cur;
  int u = next_unit(a, blockIdx.x, units, cur);
  if (u >= units) {
    wait_for_previous_kernel();   // this kernel does not end before the chains, whatever comes after it
    return;
  }
  auto load = [&](const Unit& x) {  // all but S; one thread
    const size_t unit = static_cast<size_t>(x.slot) * p.HV + x.hv;
    const uint8_t* z = a.z + unit * (4 * C * V);
    const uint8_t* vn = a.vn + unit * (4 * C * V);
    mbar_arrive_expect_tx_relaxed(&bars[LD_A], VB * 5 * 8192);
#pragma unroll 1
    for (int b = 0; b < VB; ++b) {
      uint8_t* blk = sm + b * BLOCK;
      tma_load_3d(blk + P_DO * 8192, &maps.v, &bars[LD_A], 64 * b, x.hv, static_cast<int>(x.tok));
      bulk_load(blk + P_ZH * 8192, z + b * 8192, 8192, &bars[LD_A]);
      bulk_load(blk + P_ZL * 8192, z + 2 * C * V + b * 8192, 8192, &bars[LD_A]);
      bulk_load(blk + P_VH * 8192, vn + b * 8192, 8192, &bars[LD_A]);
      bulk_load(blk + P_VL * 8192, vn + 2 * C * V + b * 8192, 8192, &bars[LD_A]);
    }
    mbar_arrive_expect_tx_relaxed(&bars[LD_D], L::MAT);
    bulk_load(sm + L::DS, a.dstates + unit * (K * V), L::MAT, &bars[LD_D]);
  };
  auto load_s = [&](const Unit& x) {
    mbar_arrive_expect_tx_relaxed(&bars[LD_S], L::MAT);
    bulk_load(sm + L::S, a.states + (static_cast<size_t>(x.slot) * p.HV + x.hv) * (K * V), L::MAT, &bars[LD_S]);
  };
  if (warp == 0) {
    if (lane == 0) {
      for (int b = 0; b < NBAR; ++b) mbar_init(&bars[b], 1);
      tslot[1] = 0u;
      fence_mbar_init();
      wait_for_previous_kernel();  // the chains' results; all other threads meet them behind this one's copies
      load(cur);
      load_s(cur);
    }
    __syncwarp();
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  } else if (warp == 1) {
    float g[2], b[2];
    load_gate(p.g, p, cur.tok, cur.rows, cur.hv, lane, g);
    load_gate(p.beta, p, cur.tok, cur.rows, cur.hv, lane, b);
    put_gates(g[0], g[1], b[0], b[1], gates);
  } else {
    for (int n = tid - 64; n < VB * 512; n += NT - 64)
      *reinterpret_cast<uint4*>(sm + (n >> 9) * BLOCK + P_ZERO * 8192 + (n & 511) * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot, sb = smem_u32(sm);
  const auto kmaj = [&](uint32_t off) { return sdesc_sw128(sb + off); };             // rows of 128 bytes
  const auto mat = [&](uint32_t off) { return sdesc_sw128(sb + off, 2048); };        // a part of S or dS'
  constexpr uint32_t id1 = idesc_f16kind(128, K), id3 = idesc_f16kind(128, 64);
  const int r = 32 * (warp & 3) + lane, part = warp >> 2, i = r & 63;
  const bool kside = r >= 64;
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);

#pragma unroll 1
  for (uint32_t it = 0; u < units; ++it) {
    auto wait = [&](int b) {
      wait_own(&bars[b], it & 1, a.wait_ns, p.status, never);
      __syncwarp();
    };
    const float* gh = gates + (it & 1) * 3 * C;
    const float* gl = gh + C;
    const float* bs = gl + C;
    const int rows = cur.rows, hv = cur.hv;
    const long tok0 = cur.tok;
    const bool live = i < rows;
    float ng[2] = {0.f, 0.f}, nb[2] = {0.f, 0.f};
    if (warp == 1) {       // the unit after this one, and its gates on their way
      Unit x;
      const int n = next_unit(a, u + gridDim.x, units, x);
      if (lane == 0) *upcoming = Upcoming{x, n};
      if (n < units) {
        load_gate(p.g, p, x.tok, x.rows, x.hv, lane, ng);
        load_gate(p.beta, p, x.tok, x.rows, x.hv, lane, nb);
      }
    }
    // v for z . v
    constexpr int CH = V / 8, NV = C * CH / NT;            // 16-byte chunks of a row, of a thread
    uint4 vv[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int rw = (tid + NT * n) / CH, ch = (tid + NT * n) % CH;
      vv[n] = rw < rows ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v) +
                                                          (static_cast<size_t>(tok0 + rw) * p.HV + hv) * V + 8 * ch)
                        : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();       // (the zeros are back)
    // ---- [do; z] vn^T
    wait(LD_A);
    if (warp == 0) {
      tc_fence_after();
#pragma unroll 1
      for (int n = 0; n < 3 * VB; ++n) {  // (high, high), (high, low), (low, high)
        const int b = n >= 3 ? 1 : 0, j = n - 3 * b;
        const uint64_t o = b * BLOCK >> 4;
        umma4<32, 32>(tmem + E3, kmaj((j == 2 ? P_ZERO : P_DO) * 8192) + o, kmaj((j == 1 ? P_VL : P_VH) * 8192) + o, id3, n > 0);
      }
      umma_commit_warp(&bars[M1]);
    }
    const float hi = gh[i], lo = gl[i], be = bs[i];
    const float bsafe = fabsf(be) < 1e-20f ? 1e-20f : be;
    const float row = ex2(hi), tail = ex2((gh[63] - hi) + (gl[63] - lo));
    // ---- A and B, strictly lower, as [A; B] operand parts; to shared memory once E1 has read S
    wait(M1);
    tc_fence_after();
    const int c0 = 16 * part;
    uint4 abh[2], abl[2];
    {
      const float f = kside ? -bsafe : p.scale;
      float x[16];
      tmem_ld16(tl + E3 + c0, x);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int c = c0 + j;
        if (!kside && c == i) diag[i] = live ? f * x[j] : 0.f;
        x[j] = (live && c < i) ? f * x[j] * ex2((hi - gh[c]) + (lo - gl[c])) : 0.f;
      }
      split8(x, abh[0], abl[0]);
      split8(x + 8, abh[1], abl[1]);
    }
    // ---- S into its parts; <S, dS'> on the way
    wait(LD_S);
    wait(LD_D);
    {
      float dot = 0.f;
      parts_in_place(sm + L::S, L::MAT / 2048, warp, lane, [&](const float (&x)[8], uint4, uint4, int g, int row, int m) {
        const uint8_t* at = sm + L::DS + g * 2048 + row * 256;
        const float4 s = *reinterpret_cast<const float4*>(at + (((2 * m) ^ row) << 4));
        const float4 w = *reinterpret_cast<const float4*>(at + (((2 * m + 1) ^ row) << 4));
        dot = fmaf(x[0], s.x, fmaf(x[1], s.y, fmaf(x[2], s.z, fmaf(x[3], s.w, dot))));
        dot = fmaf(x[4], w.x, fmaf(x[5], w.y, fmaf(x[6], w.z, fmaf(x[7], w.w, dot))));
      });
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, m);
      if (lane == 0) wsum[warp] = dot;
    }
    fence_proxy_async_smem();
    __syncthreads();
    // ---- [do; z] S^T
    if (warp == 0) {
#pragma unroll 1
      for (int n = 0; n < 3 * VB; ++n) {
        const int b = n >= 3 ? 1 : 0, j = n - 3 * b;
        const uint64_t o = b * BLOCK >> 4, os = (b * K * 256 + (j == 1 ? 1024 : 0)) >> 4;
        umma4<32, 32>(tmem + E1, kmaj((j == 2 ? P_ZERO : P_DO) * 8192) + o, mat(L::S) + os, id1, n > 0);
      }
      umma_commit_warp(&bars[M2]);
    }
    // ---- while it runs: z . v, and dv = beta z, a row's 16-byte chunks on neighbouring threads
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int rw = (tid + NT * n) / CH, ch = (tid + NT * n) % CH;
      const uint8_t* at = sm + (ch >> 3) * BLOCK + sw128(rw, ch & 7);
      const uint4 uh = *reinterpret_cast<const uint4*>(at + P_ZH * 8192), ul = *reinterpret_cast<const uint4*>(at + P_ZL * 8192);
      const uint32_t h[4] = {uh.x, uh.y, uh.z, uh.w}, l[4] = {ul.x, ul.y, ul.z, ul.w};
      const uint32_t w[4] = {vv[n].x, vv[n].y, vv[n].z, vv[n].w};
      const float b = bs[rw];
      uint32_t out[4];
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z0 = lo16(h[e]) + lo16(l[e]), z1 = hi16(h[e]) + hi16(l[e]);
        dot = fmaf(z0, lo16(w[e]), fmaf(z1, hi16(w[e]), dot));
        out[e] = pack_bf16(b * z0, b * z1);
      }
      if (rw < rows)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dv) + (static_cast<size_t>(tok0 + rw) * p.HV + hv) * V + 8 * ch) =
            make_uint4(out[0], out[1], out[2], out[3]);
#pragma unroll
      for (int m = CH / 2; m >= 1; m >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, m);
      if (ch == 0) zvs[rw] = dot;
    }
    wait(M2);            // S, do and z are no longer read by products
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      *reinterpret_cast<uint4*>(sm + L::CHI + sw128(r, (c0 >> 3) + j)) = abh[j];
      *reinterpret_cast<uint4*>(sm + L::CLO + sw128(r, (c0 >> 3) + j)) = abl[j];
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();     // z . v and dv have read z, A and B are written
    if (warp == 0) {     // [q; k]
      if (lane == 0) {
        mbar_arrive_expect_tx_relaxed(&bars[LD_QK], KB * kTileBytes);
        const int hk = hv / (p.HV / p.H);
#pragma unroll 1
        for (int b = 0; b < KB; ++b) {
          tma_load_3d(sm + L::QK + b * kTileBytes, &maps.q, &bars[LD_QK], 64 * b, hk, static_cast<int>(tok0));
          tma_load_3d(sm + L::QK + b * kTileBytes + 8192, &maps.k, &bars[LD_QK], 64 * b, hk, static_cast<int>(tok0));
        }
      }
      __syncwarp();
    }
    auto issue_qk = [&]() {  // [A; B] k; and [low; high]^T of [A; B] times [q; k]: lanes i and 64 + i together are row i
                             // of A^T q + B^T k
      constexpr uint32_t id4 = id1 | IDESC_B_MN_MAJOR, id5 = id3 | IDESC_A_MN_MAJOR | IDESC_B_MN_MAJOR;
      const uint64_t bk = sdesc(sb + L::QK + 8192, kTileBytes, 1024, 2), bq = sdesc(sb + L::QK, kTileBytes, 1024, 2);
      const uint64_t al = sdesc(sb + L::CLO, kTileBytes, 1024, 2);
      umma4<32, 2048>(tmem + E4, kmaj(L::CHI), bk, id4, 0u);
      umma4<32, 2048>(tmem + E4, kmaj(L::CLO), bk, id4, 1u);
#pragma unroll 1
      for (int n = 0; n < 2 * KB; ++n) {
        const int b = n >> 1, h = n & 1;
        umma4<2048, 2048>(tmem + (b ? E5B : E5A), al + (h * 8192 >> 4), bq + ((b * kTileBytes + h * 8192) >> 4), id5, h);
      }
    };
    // a whole chunk's [A; B] products run while dS' is converted
    if (warp == 0 && rows == C) {
      wait(LD_QK);
      tc_fence_after();
      issue_qk();
    }
    // ---- dS' into three parts, the third in place of do and z's high part
    parts_in_place(sm + L::DS, L::MAT / 2048, warp, lane, [&](const float (&x)[8], uint4 h, uint4 l, int g, int rw, int m) {
      const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
      uint32_t t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        t[e] = pack_bf16(x[2 * e] - lo16(hw[e]) - lo16(lw[e]), x[2 * e + 1] - hi16(hw[e]) - hi16(lw[e]));
      const int vb = g / (K / 8), dim = (g % (K / 8)) * 8 + rw;
      *reinterpret_cast<uint4*>(sm + vb * BLOCK + sw128(dim, m)) = make_uint4(t[0], t[1], t[2], t[3]);
    });
    wait(LD_QK);
    if (!live && part == 0) {  // rows past the sequence's end: other tokens, of any value
#pragma unroll 1
      for (int c = 0; c < 8 * KB; ++c)
        *reinterpret_cast<uint4*>(sm + L::QK + (c >> 3) * kTileBytes + sw128(r, c & 7)) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    const Unit nxt = upcoming->unit;
    const int next = upcoming->u;
    if (warp == 0) {
      tc_fence_after();
      if (rows != C) issue_qk();
#pragma unroll 1
      for (int n = 0; n < 3 * VB; ++n) {  // [low; high] of vn times the three parts of dS': lanes i and 64 + i again
        const int b = n >= 3 ? 1 : 0, j = n - 3 * b;
        const uint64_t o = (b * BLOCK + P_VL * 8192) >> 4;
        umma4<32, 32>(tmem + E2, kmaj(0) + o, j == 2 ? kmaj(b * BLOCK) : mat(L::DS + b * K * 256 + j * 1024), id1, n > 0);
      }
      umma_commit_warp(&bars[M3]);
    } else if (warp == 1 && next < units) {
      put_gates(ng[0], ng[1], nb[0], nb[1], gates + ((it + 1) & 1) * 3 * C);
    }
    wait(M3);
    tc_fence_after();
    if (tid == 0 && next < units) load(nxt);
    // ---- rows of dq and dk, and their dots.  First the q side hands over what its lanes hold of
    // the k side's rows: E (vn dS'^T) + A^T q + B^T k, low parts
    float dgc = 0.f, t = 0.f, db = 0.f;
    float a1 = 0.f, a2 = 0.f, a4 = 0.f, a5 = 0.f;
    float* ex = reinterpret_cast<float*>(sm + L::S) + i * K;   // rows of K / 4 chunks, swizzled by the row
    const auto unpack_row = [&](uint32_t rw, int d, float (&o)[16]) {  // 16 values of a row of [q; k]
      const uint8_t* tile = sm + L::QK + (d >> 6) * kTileBytes;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 q = *reinterpret_cast<const uint4*>(tile + sw128(rw, ((d & 63) >> 3) + c));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[8 * c + 2 * e] = lo16(w[e]);
          o[8 * c + 2 * e + 1] = hi16(w[e]);
        }
      }
    };
    if (!kside) {
#pragma unroll 1
      for (int d0 = 0; d0 < DPT; d0 += 16) {
        const int d = part * DPT + d0;
        float e2[16], e5[16], kk[16];
        tmem_ld16(tl + E2 + d, e2);
        tmem_ld16(tl + ((d >> 6) ? E5B : E5A) + (d & 63), e5);
        unpack_row(64 + i, d, kk);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          a2 = fmaf(kk[j], e2[j], a2);
          a5 = fmaf(kk[j], e5[j], a5);
          e5[j] = fmaf(tail, e2[j], e5[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(ex + (((d >> 2) + j) ^ (i & 7)) * 4) = make_float4(e5[4 * j], e5[4 * j + 1], e5[4 * j + 2], e5[4 * j + 3]);
      }
    }
    __syncthreads();
    {
      const float dg_ = diag[i], f1 = kside ? -row * be : p.scale * row;
      const size_t orow = static_cast<size_t>(tok0 + i);
      const bool grouped = p.HV != p.H;
      const int hk = hv / (p.HV / p.H);
      uint4 packed[DPT / 8];   // of dq or dk, until every row of [q; k] is read
#pragma unroll
      for (int n = 0; n < DPT / 16; ++n) {
        const int d = part * DPT + 16 * n;
        float e1[16], e4[16], out[16], own[16];
        tmem_ld16(tl + E1 + d, e1);
        tmem_ld16(tl + E4 + d, e4);
        unpack_row(r, d, own);
        unpack_row(r ^ 64, d, out);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          a1 = fmaf(own[j], e1[j], a1);
          a4 = fmaf(own[j], e4[j], a4);
          out[j] = fmaf(f1, e1[j], fmaf(dg_, out[j], e4[j]));
        }
        if (kside) {
          tmem_ld16(tl + E2 + d, e1);
          tmem_ld16(tl + ((d >> 6) ? E5B : E5A) + (d & 63), e4);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 x = *reinterpret_cast<const float4*>(ex + (((d >> 2) + j) ^ (i & 7)) * 4);
            out[4 * j] += x.x;
            out[4 * j + 1] += x.y;
            out[4 * j + 2] += x.z;
            out[4 * j + 3] += x.w;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            a2 = fmaf(own[j], e1[j], a2);
            a5 = fmaf(own[j], e4[j], a5);
            out[j] += fmaf(tail, e1[j], e4[j]);
          }
        }
        if (grouped) {
          if (live) {
            float* op = static_cast<float*>(kside ? a.dk : a.dq) + (orow * p.HV + hv) * K + d;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float4*>(op + 4 * j) = make_float4(out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            packed[2 * n + j] = make_uint4(pack_bf16(out[8 * j], out[8 * j + 1]), pack_bf16(out[8 * j + 2], out[8 * j + 3]),
                                           pack_bf16(out[8 * j + 4], out[8 * j + 5]), pack_bf16(out[8 * j + 6], out[8 * j + 7]));
        }
      }
      // dq and dk over [q; k] and out by TMA (a row a thread, the stores cost the epilogue 3000 of
      // its 7000 cycles); a sequence's last rows straight to memory
      if (!grouped) {
        __syncthreads();
        if (rows == C) {
#pragma unroll
          for (int n = 0; n < DPT / 8; ++n) {
            const int d = part * DPT + 8 * n;
            *reinterpret_cast<uint4*>(sm + L::QK + (d >> 6) * kTileBytes + sw128(r, (d & 63) >> 3)) = packed[n];
          }
        } else if (live) {
          __nv_bfloat16* op = static_cast<__nv_bfloat16*>(kside ? a.dk : a.dq) + (orow * p.H + hk) * K + part * DPT;
#pragma unroll
          for (int n = 0; n < DPT / 8; ++n) reinterpret_cast<uint4*>(op)[n] = packed[n];
        }
      }
      if (live) {
        t = tail * a2;
        dgc = f1 * a1 + a4 - a5 - t;
        if (kside) {
          db = a4 / bsafe - row * a1;
          if (part == 0) db += zvs[i];
        }
      }
    }
    // ---- the rows' shares of dg and dbeta, where block 0's zeros will be again
    float* sg = reinterpret_cast<float*>(sm + P_ZERO * 8192);  // [4 quarters][128] dgc, then t; [4][64] dbeta
    sg[part * 128 + r] = dgc;
    sg[512 + part * 128 + r] = t;
    if (kside) sg[1024 + part * 64 + i] = db;
    // every thread's use of the exchange rows and of [q; k] comes before the copies that follow:
    // the next unit's S over both, and dq and dk from [q; k]
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      if (p.HV == p.H && rows == C) {
#pragma unroll 1
        for (int b = 0; b < KB; ++b) {
          tma_store_3d(&maps.o, sm + L::QK + b * kTileBytes, 64 * b, hv, static_cast<int>(tok0));
          tma_store_3d(&maps.o2, sm + L::QK + b * kTileBytes + 8192, 64 * b, hv, static_cast<int>(tok0));
        }
        bulk_commit();
        bulk_wait_read();
      }
      if (next < units) load_s(nxt);
    }
    float sd = 0.f, st = 0.f, b0 = 0.f, b1 = 0.f, g0 = 0.f, g1 = 0.f;
    const int i0 = 2 * lane;
    if (warp == 1) {
      sd = lane < NT / 32 ? wsum[lane] : 0.f;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        g0 += sg[h * 128 + i0] + sg[h * 128 + 64 + i0];
        g1 += sg[h * 128 + i0 + 1] + sg[h * 128 + 64 + i0 + 1];
        st += (sg[512 + h * 128 + i0] + sg[512 + h * 128 + 64 + i0]) + (sg[512 + h * 128 + i0 + 1] + sg[512 + h * 128 + 65 + i0]);
        b0 += sg[1024 + h * 64 + i0];
        b1 += sg[1024 + h * 64 + i0 + 1];
      }
    }
    __syncthreads();
    if (tid < 320) {       // the zeros back (5 KB)
      reinterpret_cast<uint4*>(sg)[tid] = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
    }
    if (warp == 1) {
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) {
        sd += __shfl_xor_sync(0xFFFFFFFFu, sd, m);
        st += __shfl_xor_sync(0xFFFFFFFFu, st, m);
      }
      const float last = fmaf(ex2(gh[63]), sd, st);
      float run = g0 + g1;   // suffix sums over the pairs
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const float up = __shfl_down_sync(0xFFFFFFFFu, run, s);
        if (lane + s < 32) run += up;
      }
      const size_t o = static_cast<size_t>(tok0 + i0) * p.HV + hv;
      if (i0 < rows) {
        a.dg[o] = run + last;
        a.dbeta[o] = b0;
      }
      if (i0 + 1 < rows) {
        a.dg[o + p.HV] = run - g0 + last;
        a.dbeta[o + p.HV] = b1;
      }
    }
    u = next;
    cur = nxt;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dq and dk of a key head: its G value heads' shares, in their order.
__global__ void __launch_bounds__(256) group_sum_kernel(const float* dqs, const float* dks, __nv_bfloat16* dq,
                                                        __nv_bfloat16* dk, size_t quads, int G, int K) {
  const size_t n = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;  // 4 dims of one (token, key head)
  if (n >= quads) return;
  const float* src = blockIdx.y == 0 ? dqs : dks;
  __nv_bfloat16* dst = blockIdx.y == 0 ? dq : dk;
  const size_t q4 = K / 4, th = n / q4, d = (n % q4) * 4;
  const float* s = src + th * G * K + d;
  float4 x = *reinterpret_cast<const float4*>(s);
  for (int g = 1; g < G; ++g) {
    const float4 y = *reinterpret_cast<const float4*>(s + static_cast<size_t>(g) * K);
    x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
  }
  *reinterpret_cast<uint2*>(dst + th * K + d) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

template <int K, int V>
cudaError_t launch(const ChainMaps& maps, const ChunkParams& a, cudaStream_t st) {
  static LaunchState state;
  const int units = a.slots * a.p.HV, sms = sm_count();
  return launch_kernel(state, gdr_grad_kernel<K, V>, static_cast<unsigned>(units < sms ? units : sms), grad::NT,
                       grad::Lay<K, V>::SMEM, true, st, maps, a, units);
}

}  // namespace

cudaError_t launch_grads(const ChainMaps& maps, const ChunkParams& a, int K, int V, cudaStream_t st) {
  if (K == 128) return V == 128 ? launch<128, 128>(maps, a, st) : launch<128, 64>(maps, a, st);
  return V == 128 ? launch<64, 128>(maps, a, st) : launch<64, 64>(maps, a, st);
}

cudaError_t launch_group_sum(const float* shares, void* dq, void* dk, size_t tokens, int H, int G, int K, cudaStream_t st) {
  const size_t quads = tokens * H * (K / 4);
  group_sum_kernel<<<dim3(static_cast<unsigned>((quads + 255) / 256), 2), 256, 0, st>>>(
      shares, shares + tokens * H * G * K, static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk), quads, G, K);
  return cudaGetLastError();
}

}  // namespace gdr
}  // namespace kda
