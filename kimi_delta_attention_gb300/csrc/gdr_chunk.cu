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
// (rows 0-63: k, 64-127: q), read back a row a thread.  Then thread i < 64 solves
// x (I + M) = e_i, thread 64 + i solves x (I + M) = P_i: row i of T and of R = P T by the
// same code, from the last column to the first, right-looking (once x_l is known it leaves
// every x_j, j < l, independently), in fp32 with two columns per instruction.
namespace prep {
constexpr int NT = 128;
constexpr uint32_t LDM = 68;                           // floats between rows of M (conflict-free rows)
// [k; q] tiles at 0, then the record's image over them
constexpr uint32_t OFF_M = 33792;
constexpr uint32_t OFF_GC = OFF_M + C * LDM * 4;       // gc high parts, low parts (log2), beta
constexpr uint32_t OFF_BAR = OFF_GC + 3 * C * 4;
constexpr uint32_t SMEM = OFF_BAR + 64 + 1024;
}  // namespace prep

__device__ __forceinline__ uint64_t pack2f(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2f(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// x_j -= x_l M_lj for l = HI .. LO and j < l; x holds columns in pairs.
template <int HI, int LO>
__device__ __forceinline__ void solve_columns(uint64_t (&x)[32], const float* m) {
#pragma unroll
  for (int l = HI; l >= LO; --l) {
    float a, b;
    unpack2f(x[l >> 1], a, b);
    const float xl = (l & 1) ? b : a;
    const uint64_t n = pack2f(-xl, -xl);
    const ulonglong2* row = reinterpret_cast<const ulonglong2*>(m + l * prep::LDM);
#pragma unroll
    for (int j = 0; 4 * j < l; ++j) {  // M_lj = 0 for j >= l: the last group may run past l
      const ulonglong2 r = row[j];
      x[2 * j] = fma2(n, r.x, x[2 * j]);
      if (4 * j + 2 < l) x[2 * j + 1] = fma2(n, r.y, x[2 * j + 1]);
    }
  }
}

template <int K>
__global__ void __launch_bounds__(prep::NT) gdr_prep_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a) {
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  float* ms = reinterpret_cast<float*>(sm + prep::OFF_M);
  float* gh = reinterpret_cast<float*>(sm + prep::OFF_GC);
  float* gl = gh + C;
  float* bs = gl + C;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + prep::OFF_BAR);  // [0]: tiles; [1]: product
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 2);
  const Params& p = a.p;
  const int slot = blockIdx.x / p.HV, hv = blockIdx.x % p.HV, hk = hv / (p.HV / p.H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int seq, rows;
  long tok;
  if (!find_chunk(a, slot, seq, tok, rows)) return;
  if (warp == 0) {
    if (lane == 0) {
      mbar_init(&bar[0], 1);
      mbar_init(&bar[1], 1);
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
    float h[2], l[2];
    gate_scan(p, tok, rows, hv, lane, h, l);
    gh[2 * lane] = h[0];
    gh[2 * lane + 1] = h[1];
    gl[2 * lane] = l[0];
    gl[2 * lane + 1] = l[1];
  } else if (warp == 2) {
    const int i0 = 2 * lane;
    bs[i0] = i0 < rows ? p.beta[(tok + i0) * p.HV + hv] : 0.f;
    bs[i0 + 1] = i0 + 1 < rows ? p.beta[(tok + i0 + 1) * p.HV + hv] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  bool ok = true;
  if (warp == 0) {
    ok = mbar_wait(&bar[0], 0, a.wait_ns);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      if (lane == 0) atomicOr(p.status, kStatusTimeout);
      mbar_wait(&bar[0], 0, kDrainNs);
    }
    const uint64_t d = sdesc_sw128(smem_u32(sm));
#pragma unroll
    for (int s = 0; s < K / 16; ++s) {
      const uint64_t o = ((s >> 2) * kTileBytes + (s & 3) * 32) >> 4;
      umma_f16_warp(tmem, d + o, d + o, idesc_f16kind(128, 64), s > 0 ? 1u : 0u);
    }
    umma_commit_warp(&bar[1]);
  }
  // row i of D in log2: gc_i - gc_j; the factors of the row
  const int i = tid & 63;
  const bool isq = tid >= 64;
  const float hi = gh[i], lo = gl[i], be = bs[i];
  if (!mbar_wait(&bar[1], 0, a.wait_ns)) {
    atomicOr(p.status, kStatusTimeout);
    mbar_wait(&bar[1], 0, kDrainNs);
  }
  tc_fence_after();
  uint64_t x[32];
  {
    const uint32_t t = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    const float f = isq ? p.scale : be;
    const int last = isq ? i : i - 1;            // columns 0 .. last of the row are not zero
    const bool have = i < rows;                  // rows past the sequence's end: M = P = 0
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[32];
      tmem_ld32(t + 32 * h, y);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const int c = 32 * h + j;
        y[j] = (have && c <= last) ? f * y[j] * ex2((hi - gh[c]) + (lo - gl[c])) : 0.f;
      }
      if (!isq) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(ms + i * prep::LDM + 32 * h + 4 * j) =
              make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int c = 32 * h + 2 * j;
        x[16 * h + j] = isq ? pack2f(y[2 * j], y[2 * j + 1]) : pack2f(c == i ? 1.f : 0.f, c + 1 == i ? 1.f : 0.f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();  // M is in shared memory, the accumulator is read
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
  if (i >= 32) solve_columns<63, 32>(x, ms);     // (warps of rows 0-31: x_l = 0 there)
  solve_columns<31, 1>(x, ms);
  // the record's image over the tiles (the product that read them is complete)
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) unpack2f(x[4 * c + e], y[2 * e], y[2 * e + 1]);
    uint4 h, l;
    split8(y, h, l);
    *reinterpret_cast<uint4*>(sm + sw128(tid, c)) = h;
    *reinterpret_cast<uint4*>(sm + kTileBytes + sw128(tid, c)) = l;
  }
  float* fac = reinterpret_cast<float*>(sm + kRecFactors);
  if (!isq) {
    fac[i] = ex2(hi);
    fac[64 + i] = ex2((gh[63] - hi) + (gl[63] - lo));
    fac[128 + i] = be;
    if (i == 63) fac[192] = ex2(hi);
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    bulk_store(a.rec + (static_cast<size_t>(slot) * p.HV + hv) * kRecBytes, sm, kRecBytes);
    bulk_commit();
    bulk_wait_read();
  }
}

// ------------------------------------------------------------------ chain ---
// One CTA per (sequence, value head, N value columns): the columns of S never meet.  Warps
// 0-7 hold the state in fp32 registers (warp w: key dims 32 (w % 4) + lane, half w / 4 of
// the columns) and do everything between the products; warp 8 loads the chunks two ahead
// (TMA tiles of k, q and v, the record by bulk copy) and issues the products.  Per chunk:
//   1. D1 = [k; q] S      M = 128, K = key dims       lanes 0-63: k S, 64-127: q S
//   2. D2 = [T; R] Y      M = 128, K = 64             lanes 0-63: vn,  64-127: R Y
//   3. D3 = k^T (E vn)    M = 128 key dims, K = 64    S = gamma S + D3 in registers
// The lanes 0-63 carry the recurrence, the lanes 64-127 make the output meanwhile.  The high
// and low parts of S, Y and E vn lie side by side as 2 N columns of one operand (their
// products land in 2 N columns and are added when read), so that a product is one
// instruction per 16 of K: the chain is bound by the latency of these three steps, not by
// the tensor cores' rate.
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
constexpr int NT = 288;
enum Mode { FORWARD, SAVE, REVERSE };
template <int K, int N, Mode MODE>
struct Lay {
  static constexpr uint32_t YROWS = MODE == REVERSE ? 128 : C;    // REVERSE: rows 64-127 hold scale G do
  // a stage: [k; q] tiles at 0, then
  static constexpr uint32_t REC = (K / 64) * kTileBytes;          // the record
  static constexpr uint32_t VS = REC + kRecBytes;                 // v (or do): 64 rows x N
  static constexpr uint32_t STAGE = VS + C * N * 2;
  static constexpr uint32_t S = 2 * STAGE;                        // S parts: K-rows of 2 N columns
  static constexpr uint32_t Y = S + 128 * 2 * N * 2;              // Y, then E vn
  static constexpr uint32_t BAR = Y + YROWS * 2 * N * 2;
  static constexpr uint32_t SMEM = BAR + 128 + 1024;
  static constexpr uint32_t LBO_S = 128 * 128, LBO_Y = YROWS * 128;   // between 64-column atoms
  static constexpr uint32_t TX = MODE == SAVE ? (K / 64) * 8192 + 2 * 8192 + 1024 + C * N * 2 : STAGE;
};
enum { FULL0 = 0, FULL1, D1, D2, D3, SREADY, YREADY, VREADY, QREADY, DRAIN, NBAR };
}  // namespace chain

// CPT values of a row as the two parts of a 2 N-column operand (c0: first column).
template <int N, int CPT>
__device__ __forceinline__ void put_parts(uint8_t* base, uint32_t lbo, int row, int c0, const float (&x)[CPT]) {
#pragma unroll
  for (int j = 0; j < CPT / 8; ++j) {
    uint4 h, l;
    split8(x + 8 * j, h, l);
    if constexpr (N == 32) {
      *reinterpret_cast<uint4*>(base + sw128(row, (c0 >> 3) + j)) = h;
      *reinterpret_cast<uint4*>(base + sw128(row, 4 + (c0 >> 3) + j)) = l;
    } else {
      *reinterpret_cast<uint4*>(base + sw128(row, (c0 >> 3) + j)) = h;
      *reinterpret_cast<uint4*>(base + lbo + sw128(row, (c0 >> 3) + j)) = l;
    }
  }
}
// The same as the two parts of a 64-row operand image in memory.
template <int CPT>
__device__ __forceinline__ void put_image(uint8_t* hi, uint8_t* lo, int row, int c0, const float (&x)[CPT]) {
#pragma unroll
  for (int j = 0; j < CPT / 8; ++j) {
    uint4 h, l;
    split8(x + 8 * j, h, l);
    *reinterpret_cast<uint4*>(hi + sw128(row, (c0 >> 3) + j)) = h;
    *reinterpret_cast<uint4*>(lo + sw128(row, (c0 >> 3) + j)) = l;
  }
}
template <int CPT>
__device__ __forceinline__ void put_bf16(void* out, size_t at, const float (&x)[CPT]) {
  __nv_bfloat16* op = static_cast<__nv_bfloat16*>(out) + at;
#pragma unroll
  for (int j = 0; j < CPT / 8; ++j)
    *reinterpret_cast<uint4*>(op + 8 * j) =
        make_uint4(pack_bf16(x[8 * j], x[8 * j + 1]), pack_bf16(x[8 * j + 2], x[8 * j + 3]),
                   pack_bf16(x[8 * j + 4], x[8 * j + 5]), pack_bf16(x[8 * j + 6], x[8 * j + 7]));
}
__device__ __forceinline__ void st_global_v8(float* p, const float* x) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}
template <int CPT>
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&x)[CPT]) {
  if constexpr (CPT == 16) tmem_ld16(t, x);
  else tmem_ld32(t, x);
}
// x = the sum of the two parts' products
template <int N, int CPT>
__device__ __forceinline__ void tmem_ld_parts(uint32_t t, float (&x)[CPT]) {
  float y[CPT];
  tmem_ld<CPT>(t, x);
  tmem_ld<CPT>(t + N, y);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < CPT; ++j) x[j] += y[j];
}

template <int K, int N, chain::Mode MODE>
__device__ __forceinline__ void chain_body(const ChainMaps& maps, const ChunkParams& a, int V, int block, uint8_t* raw) {
  using L = chain::Lay<K, N, MODE>;
  using namespace chain;
  constexpr int CPT = N / 2;
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + NBAR);
  volatile uint32_t* failed = tslot + 1;
  const Params& p = a.p;
  const int slices = V / N;
  const int unit = block / slices, v0 = (block % slices) * N;
  const int seq = unit / p.HV, hv = unit % p.HV, hk = hv / (p.HV / p.H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long tok0;
  int len;
  seq_tokens(p.cu, p.T, p.num_seqs, p.status, seq, tok0, len);
  const int nch = num_chunks(len), slot0 = first_slot(a, seq, tok0);
  const auto chunk = [&](int n) { return MODE == REVERSE ? nch - 1 - n : n; };  // of step n
  if (tid == 0) {
    for (int b = 0; b < NBAR; ++b)
      mbar_init(&bars[b], b == SREADY ? 8 : (b == YREADY || b == VREADY || b == QREADY) ? 4 : 1);
    *failed = 0u;
    fence_mbar_init();
  }
  constexpr uint32_t TCOLS = N == 32 ? 256 : 512;
  constexpr uint32_t TD2 = 2 * N, TD3 = 4 * N, TD2R = 6 * N;
  if (warp == 8) {
    tmem_alloc(tslot, TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  // waits of a whole warp; false once the CTA has failed
  auto wait = [&](int b, uint32_t parity) {
    bool ok = *failed == 0u && mbar_wait(&bars[b], parity, a.wait_ns);
    if (__all_sync(0xFFFFFFFFu, ok)) return true;
    if (lane == 0 && *failed == 0u) {
      atomicOr(p.status, kStatusTimeout);
      *failed = 1u;
    }
    return false;
  };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[b]);
  };

  if (warp == 8) {
    // ------------------------------------------------ loads and products ---
    const uint32_t sb = smem_u32(sm);
    auto load = [&](int n) {
      if (lane == 0) {
        uint8_t* st = sm + (n & 1) * L::STAGE;
        uint64_t* full = &bars[FULL0 + (n & 1)];
        const int tok = static_cast<int>(tok0 + C * static_cast<long>(chunk(n)));
        const uint8_t* rec = a.rec + (static_cast<size_t>(slot0 + chunk(n)) * p.HV + hv) * kRecBytes;
        mbar_arrive_expect_tx_relaxed(full, L::TX);
        if (MODE == SAVE) {
          bulk_load(st + L::REC, rec, 8192, full);
          bulk_load(st + L::REC + kTileBytes, rec + kTileBytes, 8192, full);
          bulk_load(st + L::REC + kRecFactors, rec + kRecFactors, 1024, full);
        } else {
          bulk_load(st + L::REC, rec, kRecBytes, full);
        }
#pragma unroll
        for (int b = 0; b < K / 64; ++b) {
          tma_load_3d(st + b * kTileBytes, &maps.k, full, 64 * b, hk, tok);
          if (MODE != SAVE) tma_load_3d(st + b * kTileBytes + 8192, &maps.q, full, 64 * b, hk, tok);
        }
        tma_load_3d(st + L::VS, &maps.v, full, v0, hv, tok);
      }
      __syncwarp();
    };
    int issued = 0, landed = 0;
    for (; issued < 2 && issued < nch; ++issued) load(issued);
    constexpr uint32_t id2n = idesc_f16kind(128, 2 * N) | IDESC_B_MN_MAJOR;   // both parts of B
    constexpr uint32_t idn = idesc_f16kind(128, N == 32 ? 2 * N : N) | IDESC_B_MN_MAJOR;  // the high part (N = 32: both)
    const uint64_t ds = sdesc(sb + L::S, L::LBO_S, 1024, 2), dy = sdesc(sb + L::Y, L::LBO_Y, 1024, 2);
    for (int n = 0; n < nch; ++n) {
      const uint32_t ph = n & 1, st = sb + ph * L::STAGE;
      const uint64_t dkq = sdesc_sw128(st), dkt = sdesc(st, kTileBytes, 1024, 2);
      const uint64_t dt = MODE == REVERSE ? sdesc(st + L::REC, kTileBytes, 1024, 2) : sdesc_sw128(st + L::REC);
      if (!wait(FULL0 + (n & 1), (n >> 1) & 1)) break;
      landed = n + 1;
      if (!wait(SREADY, ph)) break;
      tc_fence_after();
#pragma unroll
      for (int s = 0; s < K / 16; ++s)
        umma_f16_warp(tmem, dkq + (((s >> 2) * kTileBytes + (s & 3) * 32) >> 4), ds + (s * 2048 >> 4), id2n, s > 0);
      umma_commit_warp(&bars[D1]);
      // everything that read the other stage is done (SREADY): the next chunk into it
      if (n > 0 && issued < nch) {
        load(issued);
        ++issued;
      }
      if (MODE == REVERSE) {
        if (!wait(QREADY, ph)) break;
        tc_fence_after();
        const uint64_t dd = sdesc(st + L::VS, 8192, 1024, 2);
        constexpr uint32_t idr = idesc_f16kind(128, N) | IDESC_A_MN_MAJOR | IDESC_B_MN_MAJOR;
#pragma unroll
        for (int h = 0; h < 2; ++h)  // R^T do, the two parts of R (rows 64-127 of the record's tiles)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            umma_f16_warp(tmem + TD2R, dt + ((h * kTileBytes + 8192 + s * 2048) >> 4), dd + (s * 2048 >> 4), idr,
                          h + s > 0);
#pragma unroll
        for (int s = 4; s < 8; ++s)  // q^T (scale G do)
          umma_f16_warp(tmem + TD3, dkt + (s * 2048 >> 4), dy + (s * 2048 >> 4), id2n | IDESC_A_MN_MAJOR, s > 4);
      }
      if (!wait(YREADY, ph)) break;
      tc_fence_after();
      constexpr uint32_t am = MODE == REVERSE ? IDESC_A_MN_MAJOR : 0u;
      constexpr uint32_t as = MODE == REVERSE ? 2048 : 32;   // bytes of 16 of K in [T; R]
#pragma unroll
      for (int s = 0; s < 4; ++s) umma_f16_warp(tmem + TD2, dt + (s * as >> 4), dy + (s * 2048 >> 4), id2n | am, s > 0);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        umma_f16_warp(tmem + TD2, dt + ((kTileBytes + s * as) >> 4), dy + (s * 2048 >> 4), idn | am, 1u);
      umma_commit_warp(&bars[D2]);
      if (!wait(VREADY, ph)) break;
      tc_fence_after();
#pragma unroll
      for (int s = 0; s < 4; ++s)
        umma_f16_warp(tmem + TD3, dkt + (s * 2048 >> 4), dy + (s * 2048 >> 4), id2n | IDESC_A_MN_MAJOR,
                      MODE == REVERSE || s > 0);
      umma_commit_warp(&bars[D3]);
    }
    // what is in flight ends before the CTA gives up its memory
    for (int n = landed; n < issued; ++n) mbar_wait(&bars[FULL0 + (n & 1)], (n >> 1) & 1, kDrainNs);
    umma_commit_warp(&bars[DRAIN]);
    mbar_wait(&bars[DRAIN], 0, kDrainNs);
  } else {
    // ------------------------------------------ state, Y, vn (z), output ---
    const int quad = warp & 3, c0 = (warp >> 2) * CPT;
    const int r = 32 * quad + lane;                  // TMEM lane: key dim of S, row of [k; q]
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16) + c0;
    const size_t soff = ((static_cast<size_t>(seq) * p.HV + hv) * K + r) * V + v0 + c0;
    const bool isk = quad < 2;                       // token rows of k; else rows r - 64 of q
    const int i = r & 63;
    const float* first = MODE == REVERSE ? a.dfin : p.s0;
    float* final = MODE == FORWARD ? p.sfin : MODE == REVERSE ? a.ds0 : nullptr;
    float s[CPT];
    if (first && r < K) {
#pragma unroll
      for (int j = 0; j < CPT / 4; ++j) {
        const float4 t = *reinterpret_cast<const float4*>(first + soff + 4 * j);
        s[4 * j] = t.x; s[4 * j + 1] = t.y; s[4 * j + 2] = t.z; s[4 * j + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < CPT; ++j) s[j] = 0.f;
    }
    put_parts<N, CPT>(sm + L::S, L::LBO_S, r, c0, s);
    fence_proxy_async_smem();
    arrive(SREADY);
    bool good = true;
    for (int n = 0; n < nch; ++n) {
      const uint32_t ph = n & 1;
      uint8_t* st = sm + ph * L::STAGE;
      const float* fac = reinterpret_cast<const float*>(st + L::REC + kRecFactors);
      const int c = chunk(n);
      const size_t tok = static_cast<size_t>(tok0 + C * static_cast<long>(c) + i);
      const bool live = C * c + i < len;
      if (MODE != FORWARD && r < K) {
        float* img = (MODE == SAVE ? a.states : a.dstates) +
                     ((static_cast<size_t>(slot0 + c) * p.HV + hv) * K + r) * V + v0 + c0;
#pragma unroll
        for (int j = 0; j < CPT / 8; ++j) st_global_v8(img + 8 * j, s + 8 * j);
      }
      if (!(good = wait(FULL0 + (n & 1), (n >> 1) & 1))) break;
      const float row = fac[i], gamma = fac[192];
      const size_t orow = (tok * p.HV + hv) * V + v0 + c0;
      // rows past the sequence's end hold the next one's tokens, whatever they are: every
      // operand that meets them in a sum over tokens has them zeroed first
      auto clear_row = [&](uint8_t* tile) {
#pragma unroll
        for (int b = 0; b < K / 64; ++b)
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<uint4*>(tile + b * kTileBytes + sw128(i, ch)) = make_uint4(0, 0, 0, 0);
      };
      float x[CPT], y[CPT];
      auto load_v = [&](float (&o)[CPT]) {
#pragma unroll
        for (int j = 0; j < CPT / 8; ++j) {
          const uint32_t ch = (c0 >> 3) + j;
          const uint4 u = *reinterpret_cast<const uint4*>(st + L::VS + (N == 32 ? sw64(i, ch) : sw128(i, ch)));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[8 * j + 2 * e] = __uint_as_float(w[e] << 16);
            o[8 * j + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
          }
        }
      };
      if (isk) {
        const float be = fac[128 + i], tail = fac[64 + i];
        if (MODE != REVERSE) load_v(y);
        if (!(good = wait(D1, ph))) break;
        tc_fence_after();
        tmem_ld_parts<N, CPT>(tl, x);
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          const float t = MODE == REVERSE ? tail * x[j] : be * (y[j] - row * x[j]);
          x[j] = live ? t : 0.f;
        }
        if (!live && warp < 4) clear_row(st);
        put_parts<N, CPT>(sm + L::Y, L::LBO_Y, i, c0, x);
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(YREADY);
        if (!(good = wait(D2, ph))) break;
        tc_fence_after();
        tmem_ld_parts<N, CPT>(tl + TD2, x);
        if (MODE == REVERSE) {
          tmem_ld<CPT>(tl + TD2R, y);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < CPT; ++j) x[j] += y[j];
        }
        const float f = MODE == REVERSE ? -row * be : tail;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          x[j] = live ? x[j] : 0.f;
          y[j] = f * x[j];
        }
        put_parts<N, CPT>(sm + L::Y, L::LBO_Y, i, c0, y);
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(VREADY);
        if (MODE != FORWARD) {
          uint8_t* img = (MODE == SAVE ? a.vn : a.z) +
                         (static_cast<size_t>(slot0 + c) * p.HV + hv) * (4 * C * static_cast<size_t>(V)) + (v0 >> 6) * 8192;
          put_image<CPT>(img, img + 2 * C * static_cast<size_t>(V), i, c0, x);
        }
        if (MODE == REVERSE && live) {
#pragma unroll
          for (int j = 0; j < CPT; ++j) y[j] = be * x[j];
          put_bf16<CPT>(a.dv, orow, y);
        }
      } else if (MODE == FORWARD) {
        if (!(good = wait(D1, ph))) break;
        tc_fence_after();
        tmem_ld_parts<N, CPT>(tl, x);
        const float f = p.scale * row;
#pragma unroll
        for (int j = 0; j < CPT; ++j) x[j] *= f;
        if (!(good = wait(D2, ph))) break;
        tc_fence_after();
        tmem_ld_parts<N, CPT>(tl + TD2, y);
#pragma unroll
        for (int j = 0; j < CPT; ++j) x[j] += y[j];
        if (live) put_bf16<CPT>(p.out, orow, x);
      } else if (MODE == REVERSE) {
        load_v(x);
        const float f = p.scale * row;
#pragma unroll
        for (int j = 0; j < CPT; ++j) x[j] = live ? f * x[j] : 0.f;
        if (!live) {
          if (warp < 4) clear_row(st + 8192);
#pragma unroll
          for (int j = 0; j < CPT / 8; ++j)
            *reinterpret_cast<uint4*>(st + L::VS + sw128(i, (c0 >> 3) + j)) = make_uint4(0, 0, 0, 0);
        }
        put_parts<N, CPT>(sm + L::Y, L::LBO_Y, 64 + i, c0, x);
        fence_proxy_async_smem();
        arrive(QREADY);
      }
      if (!(good = wait(D3, ph))) break;
      tc_fence_after();
      tmem_ld_parts<N, CPT>(tl + TD3, x);
#pragma unroll
      for (int j = 0; j < CPT; ++j) s[j] = fmaf(gamma, s[j], x[j]);
      put_parts<N, CPT>(sm + L::S, L::LBO_S, r, c0, s);
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(SREADY);
    }
    if (good && final && r < K) {
#pragma unroll
      for (int j = 0; j < CPT / 4; ++j)
        *reinterpret_cast<float4*>(final + soff + 4 * j) = make_float4(s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, TCOLS);
  }
}

template <int K, int N>
__global__ void __launch_bounds__(chain::NT, 1) gdr_chain_kernel(const __grid_constant__ ChainMaps maps, const ChunkParams a,
                                                                 int V) {
  extern __shared__ __align__(16) uint8_t raw[];
  chain_body<K, N, chain::FORWARD>(maps, a, V, blockIdx.x, raw);
}

// The backward's two chains in one launch: even blocks SAVE (maps: v), odd blocks REVERSE
// (maps_r: d_out).  They share nothing but the records, so they run side by side.
template <int K>
__global__ void __launch_bounds__(chain::NT, 1) gdr_chains_kernel(const __grid_constant__ ChainMaps maps,
                                                                  const __grid_constant__ ChainMaps maps_r,
                                                                  const ChunkParams a, int V) {
  extern __shared__ __align__(16) uint8_t raw[];
  if (blockIdx.x & 1) chain_body<K, 64, chain::REVERSE>(maps_r, a, V, blockIdx.x >> 1, raw);
  else chain_body<K, 64, chain::SAVE>(maps, a, V, blockIdx.x >> 1, raw);
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

int sm_count() {
  static int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
      return 152;
    return v;
  }();
  return n;
}

template <int K>
cudaError_t launch_prep(const ChainMaps& maps, const ChunkParams& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(gdr_prep_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, prep::SMEM);
  if (e != cudaSuccess) return e;
  gdr_prep_kernel<K><<<static_cast<unsigned>(a.slots) * a.p.HV, prep::NT, prep::SMEM, st>>>(maps, a);
  return cudaGetLastError();
}

template <int K, int N>
cudaError_t launch_chain(const ChainMaps& maps, const ChunkParams& a, int V, cudaStream_t st) {
  constexpr uint32_t bytes = chain::Lay<K, N, chain::FORWARD>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(gdr_chain_kernel<K, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  gdr_chain_kernel<K, N><<<static_cast<unsigned>(a.p.num_seqs) * a.p.HV * (V / N), chain::NT, bytes, st>>>(maps, a, V);
  return cudaGetLastError();
}

template <int K>
cudaError_t launch_chains(const ChainMaps& maps, const ChainMaps& maps_r, const ChunkParams& a, int V, cudaStream_t st) {
  constexpr uint32_t bytes = chain::Lay<K, 64, chain::REVERSE>::SMEM;   // the larger of the two
  static_assert(bytes >= chain::Lay<K, 64, chain::SAVE>::SMEM, "shared memory of the two chains");
  cudaError_t e = cudaFuncSetAttribute(gdr_chains_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  gdr_chains_kernel<K><<<2u * static_cast<unsigned>(a.p.num_seqs) * a.p.HV * (V / 64), chain::NT, bytes, st>>>(maps, maps_r, a, V);
  return cudaGetLastError();
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
  // 32 columns a CTA while those CTAs fit the SMs at once (the chain's steps are latency, so
  // more CTAs are free); else 64.
  const int N = static_cast<long>(p.num_seqs) * p.HV * (V / 32) <= sm_count() ? 32 : 64;
  ChainMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (!make_map(&maps.q, p.q, K, p.H, tokens, 64) || !make_map(&maps.k, p.k, K, p.H, tokens, 64) ||
      !make_map(&maps.v, p.v, V, p.HV, tokens, N))
    return cudaErrorInvalidValue;
  cudaError_t e = K == 128 ? launch_prep<128>(maps, a, st) : launch_prep<64>(maps, a, st);
  if (e != cudaSuccess) return e;
  if (K == 128) return N == 32 ? launch_chain<128, 32>(maps, a, V, st) : launch_chain<128, 64>(maps, a, V, st);
  return N == 32 ? launch_chain<64, 32>(maps, a, V, st) : launch_chain<64, 64>(maps, a, V, st);
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
  if (!make_map(&maps_r.v, dout, V, p.HV, tokens, 64)) return cudaErrorInvalidValue;
  cudaError_t e = K == 128 ? launch_prep<128>(maps, a, st) : launch_prep<64>(maps, a, st);
  if (e != cudaSuccess) return e;
  e = K == 128 ? launch_chains<128>(maps, maps_r, a, V, st) : launch_chains<64>(maps, maps_r, a, V, st);
  if (e != cudaSuccess) return e;
  if ((e = launch_grads(maps_r, a, K, V, st)) != cudaSuccess || !grouped) return e;
  return launch_group_sum(static_cast<const float*>(a.dq), dq, dk, tokens, p.H, p.HV / p.H, K, st);
}

}  // namespace gdr
}  // namespace kda
