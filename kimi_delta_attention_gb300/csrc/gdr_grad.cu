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
// (dv = beta z is written by the reverse chain.)  A row's decay gradient is what the row's
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
// memory so that one instruction serves both, and thread (lane r, half h) of the CTA owns
// row r and half of the key dims throughout.
#include "gdr_chunk.cuh"

namespace kda {
namespace gdr {
namespace {

namespace grad {
constexpr int NT = 256;
// 64-row pieces of 8 KB in each 64-column block of V; neighbours make 128-row operands
// (the first four of block 0 later hold the third part of dS', 2 x 128 rows at most)
enum { P_DO, P_ZH, P_ZERO, P_ZL, P_VL, P_VH, PIECES };
constexpr uint32_t BLOCK = PIECES * 8192;
template <int K, int V>
struct Lay {
  static constexpr uint32_t VB = V / 64;
  static constexpr uint32_t S = VB * BLOCK;               // S parts; later A;B low, high parts and [q; k]
  static constexpr uint32_t CLO = S, CHI = S + kTileBytes, QK = S + 2 * kTileBytes;
  static constexpr uint32_t PART = VB * K * 128;          // bytes of one part of S
  static constexpr uint32_t DS = S + 65536;               // dS' parts; later the partial sums
  static constexpr uint32_t X = DS + 2 * PART;            // gc high, low, beta, A's diagonal, warp sums
  static constexpr uint32_t BAR = X + (4 * C + 8) * 4;
  static constexpr uint32_t SMEM = BAR + 64 + 1024;
};
static_assert(Lay<128, 128>::SMEM <= 232448, "shared memory");
enum { LD_A = 0, LD_S, LD_D, LD_QK, M1, M2, M3, NBAR };
constexpr uint32_t E1 = 0, E2 = 128, E3 = 256, E4 = 320, E5A = 448, E5B = 256;  // TMEM columns
}  // namespace grad

template <int K, int V>
__global__ void __launch_bounds__(grad::NT, 1) gdr_grad_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a) {
  using L = grad::Lay<K, V>;
  using namespace grad;
  constexpr int VB = V / 64, KB = K / 64, DPT = K / 2;
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  float* gh = reinterpret_cast<float*>(sm + L::X);
  float* gl = gh + C;
  float* bs = gl + C;
  float* diag = bs + C;
  float* wsum = diag + C;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + NBAR);
  const Params& p = a.p;
  const int slot = blockIdx.x / p.HV, hv = blockIdx.x % p.HV, hk = hv / (p.HV / p.H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int seq, rows;
  long tok0;
  if (!find_chunk(a, slot, seq, tok0, rows)) return;
  const size_t unit = static_cast<size_t>(slot) * p.HV + hv;
  if (warp == 0) {
    if (lane == 0) {
      for (int b = 0; b < NBAR; ++b) mbar_init(&bars[b], 1);
      fence_mbar_init();
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
      mbar_arrive_expect_tx_relaxed(&bars[LD_S], 2 * L::PART);
      bulk_load(sm + L::S, a.states + unit * (K * V), 2 * L::PART, &bars[LD_S]);
      mbar_arrive_expect_tx_relaxed(&bars[LD_D], 2 * L::PART);
      bulk_load(sm + L::DS, a.dstates + unit * (K * V), 2 * L::PART, &bars[LD_D]);
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
  // a wait that runs out records the timeout and then drains: the work waited for is this
  // CTA's own copies and products, and its memory may not go before they are done
  auto wait = [&](int b) {
    if (!mbar_wait(&bars[b], 0, a.wait_ns)) {
      atomicOr(p.status, kStatusTimeout);
      mbar_wait(&bars[b], 0, kDrainNs);
    }
    __syncwarp();
  };
  const auto dk_ = [&](uint32_t off) { return sdesc_sw128(sb + off); };  // K-major operand

  // ---- the products that need no k or q
  wait(LD_A);
  if (warp == 0) {
    constexpr uint32_t id3 = idesc_f16kind(128, 64);
    uint32_t acc = 0;
#pragma unroll
    for (int b = 0; b < VB; ++b)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint64_t o = (b * BLOCK + s * 32) >> 4;
        umma_f16_warp(tmem + E3, dk_(P_DO * 8192) + o, dk_(P_VH * 8192) + o, id3, acc);
        umma_f16_warp(tmem + E3, dk_(P_DO * 8192) + o, dk_(P_VL * 8192) + o, id3, 1u);
        umma_f16_warp(tmem + E3, dk_(P_ZERO * 8192) + o, dk_(P_VH * 8192) + o, id3, 1u);
        acc = 1;
      }
    umma_commit_warp(&bars[M1]);
  }
  // ---- S and dS' from fp32 into operand parts, in place; <S, dS'> on the way
  constexpr int NU = K * V / 8 / NT;                       // 8-value chunks of a thread
  uint32_t d3[NU][4];
  {
    float s[NU][8], d[NU][8], dot = 0.f;
    // (d3: the third part of dS', put in place of do and z once their products are done)
    wait(LD_S);
    wait(LD_D);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const float4* ps = reinterpret_cast<const float4*>(sm + L::S + (tid + NT * u) * 32);
      const float4* pd = reinterpret_cast<const float4*>(sm + L::DS + (tid + NT * u) * 32);
      const float4 s0 = ps[0], s1 = ps[1], d0 = pd[0], d1 = pd[1];
      s[u][0] = s0.x; s[u][1] = s0.y; s[u][2] = s0.z; s[u][3] = s0.w;
      s[u][4] = s1.x; s[u][5] = s1.y; s[u][6] = s1.z; s[u][7] = s1.w;
      d[u][0] = d0.x; d[u][1] = d0.y; d[u][2] = d0.z; d[u][3] = d0.w;
      d[u][4] = d1.x; d[u][5] = d1.y; d[u][6] = d1.z; d[u][7] = d1.w;
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(s[u][e], d[u][e], dot);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, m);
    if (lane == 0) wsum[warp] = dot;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int c = tid + NT * u, dim = c / (V / 8), ch = c % (V / 8);
      const uint32_t o = (ch >> 3) * (K * 128) + sw128(dim, ch & 7);
      uint4 h, l;
      split8(s[u], h, l);
      *reinterpret_cast<uint4*>(sm + L::S + o) = h;
      *reinterpret_cast<uint4*>(sm + L::S + L::PART + o) = l;
      split8(d[u], h, l);
      *reinterpret_cast<uint4*>(sm + L::DS + o) = h;
      *reinterpret_cast<uint4*>(sm + L::DS + L::PART + o) = l;
      const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        d3[u][e] = pack_bf16(d[u][2 * e] - __uint_as_float(hw[e] << 16) - __uint_as_float(lw[e] << 16),
                             d[u][2 * e + 1] - __uint_as_float(hw[e] & 0xFFFF0000u) - __uint_as_float(lw[e] & 0xFFFF0000u));
    }
    fence_proxy_async_smem();
    __syncthreads();
  }
  if (warp == 0) {
    constexpr uint32_t id1 = idesc_f16kind(128, K);
    uint32_t acc = 0;
#pragma unroll
    for (int b = 0; b < VB; ++b)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint64_t o = (b * BLOCK + s * 32) >> 4, os = (b * K * 128 + s * 32) >> 4;
        umma_f16_warp(tmem + E1, dk_(P_DO * 8192) + o, dk_(L::S) + os, id1, acc);
        umma_f16_warp(tmem + E1, dk_(P_DO * 8192) + o, dk_(L::S + L::PART) + os, id1, 1u);
        umma_f16_warp(tmem + E1, dk_(P_ZERO * 8192) + o, dk_(L::S) + os, id1, 1u);
        acc = 1;
      }
    umma_commit_warp(&bars[M2]);
    acc = 0;
#pragma unroll
    for (int b = 0; b < VB; ++b)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint64_t o = (b * BLOCK + s * 32) >> 4, os = (b * K * 128 + s * 32) >> 4;
        umma_f16_warp(tmem + E2, dk_(P_VL * 8192) + o, dk_(L::DS) + os, id1, acc);
        umma_f16_warp(tmem + E2, dk_(P_VL * 8192) + o, dk_(L::DS + L::PART) + os, id1, 1u);
        umma_f16_warp(tmem + E2, dk_(P_ZL * 8192) + o, dk_(L::DS) + os, id1, 1u);
        umma_f16_warp(tmem + E2, dk_(P_ZL * 8192) + o, dk_(L::DS + L::PART) + os, id1, 1u);
        acc = 1;
      }
  }
  // ---- z . v, while they run
  const int r = 32 * (warp & 3) + lane, half = warp >> 2, i = r & 63;
  const bool kside = r >= 64, live = i < rows;
  const float hi = gh[i], lo = gl[i], be = bs[i];
  const float bsafe = fabsf(be) < 1e-20f ? 1e-20f : be;
  const float row = ex2(hi), tail = ex2((gh[63] - hi) + (gl[63] - lo));
  float zv = 0.f;
  if (kside && live) {
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + (static_cast<size_t>(tok0 + i) * p.HV + hv) * V;
#pragma unroll
    for (int c = 0; c < V / 16; ++c) {
      const int col = half * (V / 16) + c;                // 16-byte chunk of the row
      const uint8_t* blk = sm + (col >> 3) * BLOCK;
      const uint4 uh = *reinterpret_cast<const uint4*>(blk + P_ZH * 8192 + sw128(i, col & 7));
      const uint4 ul = *reinterpret_cast<const uint4*>(blk + P_ZL * 8192 + sw128(i, col & 7));
      const uint4 uv = *reinterpret_cast<const uint4*>(v + 8 * col);
      const uint32_t h[4] = {uh.x, uh.y, uh.z, uh.w}, l[4] = {ul.x, ul.y, ul.z, ul.w}, w[4] = {uv.x, uv.y, uv.z, uv.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        zv = fmaf(__uint_as_float(h[e] << 16) + __uint_as_float(l[e] << 16), __uint_as_float(w[e] << 16), zv);
        zv = fmaf(__uint_as_float(h[e] & 0xFFFF0000u) + __uint_as_float(l[e] & 0xFFFF0000u),
                  __uint_as_float(w[e] & 0xFFFF0000u), zv);
      }
    }
  }
  // ---- A and B, strictly lower, as [A; B] operand parts
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  wait(M1);
  tc_fence_after();
  float x[32];
  tmem_ld32(tl + E3 + 32 * half, x);
  tmem_ld_wait();
  {
    const float f = kside ? -bsafe : p.scale;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int c = 32 * half + j;
      if (!kside && c == i) diag[i] = live ? f * x[j] : 0.f;
      x[j] = (live && c < i) ? f * x[j] * ex2((hi - gh[c]) + (lo - gl[c])) : 0.f;
    }
  }
  wait(M2);          // S is no longer read by products
  __syncthreads();
  if (tid == 0) {
    mbar_arrive_expect_tx_relaxed(&bars[LD_QK], KB * kTileBytes);
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      tma_load_3d(sm + L::QK + b * kTileBytes, &maps.q, &bars[LD_QK], 64 * b, hk, static_cast<int>(tok0));
      tma_load_3d(sm + L::QK + b * kTileBytes + 8192, &maps.k, &bars[LD_QK], 64 * b, hk, static_cast<int>(tok0));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 h, l;
    split8(x + 8 * j, h, l);
    *reinterpret_cast<uint4*>(sm + L::CHI + sw128(r, 4 * half + j)) = h;
    *reinterpret_cast<uint4*>(sm + L::CLO + sw128(r, 4 * half + j)) = l;
  }
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = tid + NT * u, dim = c / (V / 8), ch = c % (V / 8);
    *reinterpret_cast<uint4*>(sm + (ch >> 3) * (K * 128) + sw128(dim, ch & 7)) = make_uint4(d3[u][0], d3[u][1], d3[u][2], d3[u][3]);
  }
  wait(LD_QK);
  if (!live && half == 0) {  // rows past the sequence's end: other tokens, of any value
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(sm + L::QK + b * kTileBytes + sw128(r, c)) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  // ---- [A; B] k and A^T q + B^T k (the latter in lanes 64-127: the first atom of M is the
  // neighbouring tile, whose lanes nobody reads)
  if (warp == 0) {
    tc_fence_after();
    constexpr uint32_t id4 = idesc_f16kind(128, K) | IDESC_B_MN_MAJOR;
    constexpr uint32_t id5 = idesc_f16kind(128, 64) | IDESC_A_MN_MAJOR | IDESC_B_MN_MAJOR;
#pragma unroll
    for (int b = 0; b < VB; ++b)
#pragma unroll
      for (int s = 0; s < 4; ++s)  // vn (third part of dS')^T
        umma_f16_warp(tmem + E2, dk_(P_VL * 8192) + ((b * BLOCK + s * 32) >> 4), dk_(0) + ((b * K * 128 + s * 32) >> 4),
                      idesc_f16kind(128, K), 1u);
    const uint64_t bk = sdesc(sb + L::QK + 8192, kTileBytes, 1024, 2), bq = sdesc(sb + L::QK, kTileBytes, 1024, 2);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      umma_f16_warp(tmem + E4, dk_(L::CHI) + (s * 32 >> 4), bk + (s * 2048 >> 4), id4, s > 0);
      umma_f16_warp(tmem + E4, dk_(L::CLO) + (s * 32 >> 4), bk + (s * 2048 >> 4), id4, 1u);
    }
    const uint64_t ah = sdesc(sb + L::CLO, kTileBytes, 1024, 2), al = sdesc(sb + L::CLO - kTileBytes, kTileBytes, 1024, 2);
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint64_t o = s * 2048 >> 4, ob = (b * kTileBytes + s * 2048) >> 4;
        umma_f16_warp(tmem + (b ? E5B : E5A), ah + o, bq + ob, id5, s > 0);
        umma_f16_warp(tmem + (b ? E5B : E5A), al + o, bq + ob, id5, 1u);
      }
    umma_commit_warp(&bars[M3]);
  }
  wait(M3);
  tc_fence_after();
  // ---- rows of dq and dk, and their dots
  float dgc = 0.f, t = 0.f, db = zv;
  {
    const float dg_ = diag[i], f1 = kside ? -row * be : p.scale * row;
    float a1 = 0.f, a2 = 0.f, a4 = 0.f, a5 = 0.f;
    const size_t orow = static_cast<size_t>(tok0 + i);
    const bool grouped = p.HV != p.H;
#pragma unroll
    for (int d0 = 0; d0 < DPT; d0 += 16) {
      const int d = half * DPT + d0;
      float e1[16], e4[16], out[16], own[16], oth[16];
      tmem_ld16(tl + E1 + d, e1);
      tmem_ld16(tl + E4 + d, e4);
      tmem_ld_wait();
      const uint8_t* tile = sm + L::QK + (d >> 6) * kTileBytes;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 uo = *reinterpret_cast<const uint4*>(tile + sw128(r, ((d & 63) >> 3) + c));
        const uint4 ut = *reinterpret_cast<const uint4*>(tile + sw128(r ^ 64, ((d & 63) >> 3) + c));
        const uint32_t wo[4] = {uo.x, uo.y, uo.z, uo.w}, wt[4] = {ut.x, ut.y, ut.z, ut.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          own[8 * c + 2 * e] = __uint_as_float(wo[e] << 16);
          own[8 * c + 2 * e + 1] = __uint_as_float(wo[e] & 0xFFFF0000u);
          oth[8 * c + 2 * e] = __uint_as_float(wt[e] << 16);
          oth[8 * c + 2 * e + 1] = __uint_as_float(wt[e] & 0xFFFF0000u);
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        a1 = fmaf(own[j], e1[j], a1);
        a4 = fmaf(own[j], e4[j], a4);
        out[j] = fmaf(f1, e1[j], fmaf(dg_, oth[j], e4[j]));
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
        db += a4 / bsafe - row * a1;
      } else {
        dgc = f1 * a1 + a4;
      }
    }
  }
  // ---- the rows' shares of dg and dbeta (over dS', whose products are done)
  float* sg = reinterpret_cast<float*>(sm + L::DS);  // [2 halves][128] dgc, then t, then dbeta
  sg[half * 128 + r] = dgc;
  if (kside) {
    sg[256 + half * 64 + i] = t;
    sg[384 + half * 64 + i] = db;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (warp == 1) {
    float sd = lane < 8 ? wsum[lane] : 0.f, st = 0.f;
    float g0 = 0.f, g1 = 0.f;
    const int i0 = 2 * lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      g0 += sg[h * 128 + i0] + sg[h * 128 + 64 + i0];
      g1 += sg[h * 128 + i0 + 1] + sg[h * 128 + 64 + i0 + 1];
      st += sg[256 + h * 64 + i0] + sg[256 + h * 64 + i0 + 1];
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
      a.dbeta[o] = sg[384 + i0] + sg[448 + i0];
    }
    if (i0 + 1 < rows) {
      a.dg[o + p.HV] = run - g0 + last;
      a.dbeta[o + p.HV] = sg[384 + i0 + 1] + sg[448 + i0 + 1];
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
  constexpr uint32_t bytes = grad::Lay<K, V>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(gdr_grad_kernel<K, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  gdr_grad_kernel<K, V><<<static_cast<unsigned>(a.slots) * a.p.HV, grad::NT, bytes, st>>>(maps, a);
  return cudaGetLastError();
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
