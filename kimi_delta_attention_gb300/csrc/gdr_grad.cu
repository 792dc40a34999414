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
// the arithmetic, 4.3e-6 with two; the largest of small cases 5.7e-6 and 9.9e-6).
//
// One CTA of 256 threads per (chunk, value head).  Products on tcgen05 with M = 128: rows
// 0-63 belong to q's side (do; A), rows 64-127 to k's side (z, vn; B), stacked in shared
// memory so that one instruction serves both, and thread (lane r, quarter h) of the CTA owns
// row r and a quarter of the key dims throughout.
#include "gdr_chunk.cuh"

namespace kda {
namespace gdr {
namespace {

namespace grad {
constexpr int NT = 512;
// 64-row pieces of 8 KB in each 64-column block of V; neighbours make 128-row operands
// (the first four of block 0 later hold the third part of dS', 2 x 128 rows at most)
enum { P_DO, P_ZH, P_ZERO, P_ZL, P_VL, P_VH, PIECES };
constexpr uint32_t BLOCK = PIECES * 8192;
template <int K, int V>
struct Lay {
  static constexpr uint32_t VB = V / 64;
  static constexpr uint32_t S = VB * BLOCK;               // S; later the A;B parts (low, high) and [q; k]
  static constexpr uint32_t CLO = S, CHI = S + kTileBytes, QK = S + 2 * kTileBytes;
  static constexpr uint32_t MAT = VB * K * 256;           // bytes of S or dS', fp32 or two parts
  static constexpr uint32_t DS = S + 65536;               // dS'; later the partial sums
  static constexpr uint32_t X = DS + MAT;                 // gc high, low, beta, A's diagonal, z . v, warp sums
  static constexpr uint32_t BAR = X + (5 * C + 16) * 4;
  static constexpr uint32_t SMEM = BAR + 64 + 1024;
};
static_assert(Lay<128, 128>::SMEM <= 232448, "shared memory");
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
}  // namespace grad

// Code that runs once per CTA is bound by instruction fetch, so everything here is small
// loops: with the conversions, products and epilogue unrolled the same kernel took 207 us for
// 2048 chunks and heads.
template <int K, int V>
__global__ void __launch_bounds__(grad::NT, 1) gdr_grad_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a) {
  using L = grad::Lay<K, V>;
  using namespace grad;
  constexpr int VB = V / 64, KB = K / 64, DPT = K / 4;
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  float* gh = reinterpret_cast<float*>(sm + L::X);
  float* gl = gh + C;
  float* bs = gl + C;
  float* diag = bs + C;
  float* zvs = diag + C;
  float* wsum = zvs + C;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + NBAR);
  const Params& p = a.p;
  const int slot = blockIdx.x / p.HV, hv = blockIdx.x % p.HV, hk = hv / (p.HV / p.H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int seq, rows;
  long tok0;
  if (!find_chunk(a, nullptr, slot, seq, tok0, rows)) return;
  const size_t unit = static_cast<size_t>(slot) * p.HV + hv;
  if (warp == 0) {
    if (lane == 0) {
      for (int b = 0; b < NBAR; ++b) mbar_init(&bars[b], 1);
      tslot[1] = 0u;
      fence_mbar_init();
      wait_for_previous_kernel();  // the chains' results; all other threads meet them behind this one's copies
      const uint8_t* z = a.z + unit * (4 * C * V);
      const uint8_t* vn = a.vn + unit * (4 * C * V);
      mbar_arrive_expect_tx_relaxed(&bars[LD_A], VB * 5 * 8192);
      for (int b = 0; b < VB; ++b) {
        uint8_t* blk = sm + b * BLOCK;
        tma_load_3d(blk + P_DO * 8192, &maps.v, &bars[LD_A], 64 * b, hv, static_cast<int>(tok0));
        bulk_load(blk + P_ZH * 8192, z + b * 8192, 8192, &bars[LD_A]);
        bulk_load(blk + P_ZL * 8192, z + 2 * C * V + b * 8192, 8192, &bars[LD_A]);
        bulk_load(blk + P_VH * 8192, vn + b * 8192, 8192, &bars[LD_A]);
        bulk_load(blk + P_VL * 8192, vn + 2 * C * V + b * 8192, 8192, &bars[LD_A]);
      }
      mbar_arrive_expect_tx_relaxed(&bars[LD_S], L::MAT);
      bulk_load(sm + L::S, a.states + unit * (K * V), L::MAT, &bars[LD_S]);
      mbar_arrive_expect_tx_relaxed(&bars[LD_D], L::MAT);
      bulk_load(sm + L::DS, a.dstates + unit * (K * V), L::MAT, &bars[LD_D]);
    }
    __syncwarp();
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  } else if (warp == 1) {
    float h[2], l[2];
    gate_scan(p, tok0, rows, hv, lane, h, l);
    gh[2 * lane] = h[0];
    gh[2 * lane + 1] = h[1];
    gl[2 * lane] = l[0];
    gl[2 * lane + 1] = l[1];
  } else if (warp == 2) {
    for (int i = lane; i < C; i += 32) bs[i] = i < rows ? p.beta[(tok0 + i) * p.HV + hv] : 0.f;
  } else {
    for (int i = tid - 96; i < VB * 512; i += NT - 96)
      *reinterpret_cast<uint4*>(sm + (i >> 9) * BLOCK + P_ZERO * 8192 + (i & 511) * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot, sb = smem_u32(sm);
  volatile uint32_t* never = tslot + 1;   // (zero)
  // a wait that runs out records the timeout and then drains: the work waited for is this
  // CTA's own copies and products, and its memory may not go before they are done
  auto wait = [&](int b) {
#pragma unroll 1
    for (uint64_t limit = a.wait_ns; !wait_phase(&bars[b], 0, limit, never) && limit != ~0ull; limit = limit == kDrainNs ? ~0ull : kDrainNs)
      atomicOr(p.status, kStatusTimeout);
    __syncwarp();
  };
  const auto kmaj = [&](uint32_t off) { return sdesc_sw128(sb + off); };             // rows of 128 bytes
  const auto mat = [&](uint32_t off) { return sdesc_sw128(sb + off, 2048); };        // a part of S or dS'
  constexpr uint32_t id1 = idesc_f16kind(128, K), id3 = idesc_f16kind(128, 64);

  // ---- [do; z] vn^T
  wait(LD_A);
  if (warp == 0) {
#pragma unroll 1
    for (int b = 0; b < VB; ++b) {
      const uint64_t o = b * BLOCK >> 4;
      umma4<32, 32>(tmem + E3, kmaj(P_DO * 8192) + o, kmaj(P_VH * 8192) + o, id3, b > 0);
      umma4<32, 32>(tmem + E3, kmaj(P_DO * 8192) + o, kmaj(P_VL * 8192) + o, id3, 1u);
      umma4<32, 32>(tmem + E3, kmaj(P_ZERO * 8192) + o, kmaj(P_VH * 8192) + o, id3, 1u);
    }
    umma_commit_warp(&bars[M1]);
  }
  // ---- S into its parts; <S, dS'> on the way
  wait(LD_S);
  wait(LD_D);
  {
    float dot = 0.f;
    parts_in_place(sm + L::S, L::MAT / 2048, warp, lane, [&](const float (&x)[8], uint4, uint4, int g, int row, int m) {
      const uint8_t* at = sm + L::DS + g * 2048 + row * 256;
      const float4 u = *reinterpret_cast<const float4*>(at + (((2 * m) ^ row) << 4));
      const float4 w = *reinterpret_cast<const float4*>(at + (((2 * m + 1) ^ row) << 4));
      dot = fmaf(x[0], u.x, fmaf(x[1], u.y, fmaf(x[2], u.z, fmaf(x[3], u.w, dot))));
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
    for (int b = 0; b < VB; ++b) {
      const uint64_t o = b * BLOCK >> 4, os = b * K * 256 >> 4;
      umma4<32, 32>(tmem + E1, kmaj(P_DO * 8192) + o, mat(L::S) + os, id1, b > 0);
      umma4<32, 32>(tmem + E1, kmaj(P_DO * 8192) + o, mat(L::S + 1024) + os, id1, 1u);
      umma4<32, 32>(tmem + E1, kmaj(P_ZERO * 8192) + o, mat(L::S) + os, id1, 1u);
    }
    umma_commit_warp(&bars[M2]);
  }
  // ---- while it runs: z . v, and dv = beta z, a row's 16-byte chunks on neighbouring threads
  const int r = 32 * (warp & 3) + lane, part = warp >> 2, i = r & 63;
  const bool kside = r >= 64, live = i < rows;
  {
    constexpr int CH = V / 8;                              // 16-byte chunks of a row
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v);
    __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(a.dv);
#pragma unroll 1
    for (int n = tid; n < C * CH; n += NT) {
      const int rw = n / CH, ch = n % CH;
      const uint8_t* at = sm + (ch >> 3) * BLOCK + sw128(rw, ch & 7);
      const uint4 uh = *reinterpret_cast<const uint4*>(at + P_ZH * 8192), ul = *reinterpret_cast<const uint4*>(at + P_ZL * 8192);
      const size_t o = (static_cast<size_t>(tok0 + rw) * p.HV + hv) * V + 8 * ch;
      const uint4 uv = rw < rows ? *reinterpret_cast<const uint4*>(v + o) : make_uint4(0, 0, 0, 0);
      const uint32_t h[4] = {uh.x, uh.y, uh.z, uh.w}, l[4] = {ul.x, ul.y, ul.z, ul.w}, w[4] = {uv.x, uv.y, uv.z, uv.w};
      const float b = bs[rw];
      uint32_t out[4];
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z0 = lo16(h[e]) + lo16(l[e]), z1 = hi16(h[e]) + hi16(l[e]);
        dot = fmaf(z0, lo16(w[e]), fmaf(z1, hi16(w[e]), dot));
        out[e] = pack_bf16(b * z0, b * z1);
      }
      if (rw < rows) *reinterpret_cast<uint4*>(dv + o) = make_uint4(out[0], out[1], out[2], out[3]);
#pragma unroll
      for (int m = CH / 2; m >= 1; m >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, m);
      if (ch == 0) zvs[rw] = dot;
    }
  }
  const float hi = gh[i], lo = gl[i], be = bs[i];
  const float bsafe = fabsf(be) < 1e-20f ? 1e-20f : be;
  const float row = ex2(hi), tail = ex2((gh[63] - hi) + (gl[63] - lo));
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  wait(M1);
  wait(M2);          // S, do and z are no longer read by products
  tc_fence_after();
  if (tid == 0) {
    mbar_arrive_expect_tx_relaxed(&bars[LD_QK], KB * kTileBytes);
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      tma_load_3d(sm + L::QK + b * kTileBytes, &maps.q, &bars[LD_QK], 64 * b, hk, static_cast<int>(tok0));
      tma_load_3d(sm + L::QK + b * kTileBytes + 8192, &maps.k, &bars[LD_QK], 64 * b, hk, static_cast<int>(tok0));
    }
  }
  // ---- A and B, strictly lower, as [A; B] operand parts
  {
    const float f = kside ? -bsafe : p.scale;
    {
      const int c0 = 16 * part;
      float x[16];
      tmem_ld16(tl + E3 + c0, x);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int c = c0 + j;
        if (!kside && c == i) diag[i] = live ? f * x[j] : 0.f;
        x[j] = (live && c < i) ? f * x[j] * ex2((hi - gh[c]) + (lo - gl[c])) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint4 ph, pl;
        split8(x + 8 * j, ph, pl);
        *reinterpret_cast<uint4*>(sm + L::CHI + sw128(r, (c0 >> 3) + j)) = ph;
        *reinterpret_cast<uint4*>(sm + L::CLO + sw128(r, (c0 >> 3) + j)) = pl;
      }
    }
  }
  __syncthreads();   // z . v and dv have read z
  // ---- dS' into three parts, the third in place of do and z
  parts_in_place(sm + L::DS, L::MAT / 2048, warp, lane, [&](const float (&x)[8], uint4 h, uint4 l, int g, int rw, int m) {
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
    uint32_t t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      t[e] = pack_bf16(x[2 * e] - lo16(hw[e]) - lo16(lw[e]), x[2 * e + 1] - hi16(hw[e]) - hi16(lw[e]));
    const int vb = g / (K / 8), dim = (g % (K / 8)) * 8 + rw;
    *reinterpret_cast<uint4*>(sm + vb * (K * 128) + sw128(dim, m)) = make_uint4(t[0], t[1], t[2], t[3]);
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
  // ---- vn dS'^T, [A; B] k and A^T q + B^T k (the last in lanes 64-127: the first atom of M is
  // the neighbouring tile, whose lanes nobody reads)
  if (warp == 0) {
    tc_fence_after();
#pragma unroll 1
    for (int b = 0; b < VB; ++b) {
      const uint64_t o = b * BLOCK >> 4, os = b * K * 256 >> 4;
      umma4<32, 32>(tmem + E2, kmaj(P_VL * 8192) + o, mat(L::DS) + os, id1, b > 0);
      umma4<32, 32>(tmem + E2, kmaj(P_VL * 8192) + o, mat(L::DS + 1024) + os, id1, 1u);
      umma4<32, 32>(tmem + E2, kmaj(P_ZL * 8192) + o, mat(L::DS) + os, id1, 1u);
      umma4<32, 32>(tmem + E2, kmaj(P_ZL * 8192) + o, mat(L::DS + 1024) + os, id1, 1u);
      umma4<32, 32>(tmem + E2, kmaj(P_VL * 8192) + o, kmaj(b * K * 128), id1, 1u);
    }
    constexpr uint32_t id4 = id1 | IDESC_B_MN_MAJOR, id5 = id3 | IDESC_A_MN_MAJOR | IDESC_B_MN_MAJOR;
    const uint64_t bk = sdesc(sb + L::QK + 8192, kTileBytes, 1024, 2), bq = sdesc(sb + L::QK, kTileBytes, 1024, 2);
    umma4<32, 2048>(tmem + E4, kmaj(L::CHI), bk, id4, 0u);
    umma4<32, 2048>(tmem + E4, kmaj(L::CLO), bk, id4, 1u);
    const uint64_t ah = sdesc(sb + L::CLO, kTileBytes, 1024, 2), al = sdesc(sb + L::CLO - kTileBytes, kTileBytes, 1024, 2);
#pragma unroll 1
    for (int b = 0; b < KB; ++b)
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint64_t o = h * 8192 >> 4, ob = (b * kTileBytes + h * 8192) >> 4;
        umma4<2048, 2048>(tmem + (b ? E5B : E5A), ah + o, bq + ob, id5, h);
        umma4<2048, 2048>(tmem + (b ? E5B : E5A), al + o, bq + ob, id5, 1u);
      }
    umma_commit_warp(&bars[M3]);
  }
  wait(M3);
  tc_fence_after();
  // ---- rows of dq and dk, and their dots
  float dgc = 0.f, t = 0.f, db = 0.f;
  {
    const float dg_ = diag[i], f1 = kside ? -row * be : p.scale * row;
    float a1 = 0.f, a2 = 0.f, a4 = 0.f, a5 = 0.f;
    const size_t orow = static_cast<size_t>(tok0 + i);
    const bool grouped = p.HV != p.H;
#pragma unroll 1
    for (int d0 = 0; d0 < DPT; d0 += 16) {
      const int d = part * DPT + d0;
      float e1[16], e4[16], out[16], own[16];
      tmem_ld16(tl + E1 + d, e1);
      tmem_ld16(tl + E4 + d, e4);
      const uint8_t* tile = sm + L::QK + (d >> 6) * kTileBytes;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 uo = *reinterpret_cast<const uint4*>(tile + sw128(r, ((d & 63) >> 3) + c));
        const uint4 ut = *reinterpret_cast<const uint4*>(tile + sw128(r ^ 64, ((d & 63) >> 3) + c));
        const uint32_t wo[4] = {uo.x, uo.y, uo.z, uo.w}, wt[4] = {ut.x, ut.y, ut.z, ut.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          own[8 * c + 2 * e] = lo16(wo[e]);
          own[8 * c + 2 * e + 1] = hi16(wo[e]);
          out[8 * c + 2 * e] = dg_ * lo16(wt[e]);
          out[8 * c + 2 * e + 1] = dg_ * hi16(wt[e]);
        }
      }
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        a1 = fmaf(own[j], e1[j], a1);
        a4 = fmaf(own[j], e4[j], a4);
        out[j] = fmaf(f1, e1[j], out[j] + e4[j]);
      }
      if (kside) {
        tmem_ld16(tl + E2 + d, e1);
        tmem_ld16(tl + ((d >> 6) ? E5B : E5A) + (d & 63), e4);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          a2 = fmaf(own[j], e1[j], a2);
          a5 = fmaf(own[j], e4[j], a5);
          out[j] += fmaf(tail, e1[j], e4[j]);
        }
      }
      if (live) {
        void* dst = kside ? a.dk : a.dq;
        if (grouped) {
          float* op = static_cast<float*>(dst) + (orow * p.HV + hv) * K + d;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(op + 4 * j) = make_float4(out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
        } else {
          __nv_bfloat16* op = static_cast<__nv_bfloat16*>(dst) + (orow * p.H + hk) * K + d;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            *reinterpret_cast<uint4*>(op + 8 * j) =
                make_uint4(pack_bf16(out[8 * j], out[8 * j + 1]), pack_bf16(out[8 * j + 2], out[8 * j + 3]),
                           pack_bf16(out[8 * j + 4], out[8 * j + 5]), pack_bf16(out[8 * j + 6], out[8 * j + 7]));
        }
      }
    }
    if (live) {
      if (kside) {
        t = tail * a2;
        dgc = a4 - a5 + f1 * a1 - t;
        db = a4 / bsafe - row * a1;
        if (part == 0) db += zvs[i];
      } else {
        dgc = f1 * a1 + a4;
      }
    }
  }
  // ---- the rows' shares of dg and dbeta (over dS', whose products are done)
  float* sg = reinterpret_cast<float*>(sm + L::DS);  // [4 quarters][128] dgc, then t, then dbeta
  sg[part * 128 + r] = dgc;
  if (kside) {
    sg[512 + part * 64 + i] = t;
    sg[768 + part * 64 + i] = db;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (warp == 1) {
    float sd = lane < NT / 32 ? wsum[lane] : 0.f, st = 0.f, b0 = 0.f, b1 = 0.f;
    float g0 = 0.f, g1 = 0.f;
    const int i0 = 2 * lane;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      g0 += sg[h * 128 + i0] + sg[h * 128 + 64 + i0];
      g1 += sg[h * 128 + i0 + 1] + sg[h * 128 + 64 + i0 + 1];
      st += sg[512 + h * 64 + i0] + sg[512 + h * 64 + i0 + 1];
      b0 += sg[768 + h * 64 + i0];
      b1 += sg[768 + h * 64 + i0 + 1];
    }
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
  return launch_kernel(state, gdr_grad_kernel<K, V>, static_cast<unsigned>(a.slots) * a.p.HV, grad::NT, grad::Lay<K, V>::SMEM,
                       true, st, maps, a);
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
