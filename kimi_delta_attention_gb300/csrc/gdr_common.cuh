// gdr_common.cuh -- launch parameters shared by the gated delta rule kernels (one scalar
// gate per token and value head).
#pragma once

#include <cstddef>
#include <cstdint>

#include "kda_common.cuh"

namespace kda {
namespace gdr {

struct Params {
  const void* q;        // [tokens, H, K]   io type
  const void* k;        // [tokens, H, K]
  const void* v;        // [tokens, HV, V]
  const float* g;       // [tokens, HV]     log decay (<= 0)
  const float* beta;    // [tokens, HV]
  const float* s0;      // [NS, HV, K, V] or null (zeros)
  const int32_t* cu;    // [NS + 1] or null
  void* out;            // [tokens, HV, V]  io type
  float* sfin;          // [NS, HV, K, V] or null
  uint32_t* status;     // device status word or null
  float scale;
  int T;                // tokens per sequence, or the packed total with cu
  int H, HV;
  int num_seqs;
};

// Token range [tok0, tok0 + len) of sequence `seq`; a malformed cu_seqlens entry sets
// kStatusBounds and gives an empty range.
__device__ __forceinline__ bool seq_tokens(const int32_t* cu, int T, int num_seqs, uint32_t* status, int seq,
                                           long& tok0, int& len) {
  if (cu == nullptr) {
    tok0 = static_cast<long>(seq) * T;
    len = T;
    return true;
  }
  const int a = cu[seq], b = cu[seq + 1];
  if (a < 0 || b < a || b > T || (seq == 0 && a != 0) || (seq == num_seqs - 1 && b != T)) {
    if (status) atomicOr(status, kStatusBounds);
    tok0 = 0;
    len = 0;
    return false;
  }
  tok0 = a;
  len = b - a;
  return true;
}

}  // namespace gdr
}  // namespace kda
