// layer_ops.cuh -- launch parameters of the gated linear recurrence, of group norm and of the
// AdamW step, between their C entries (layer_abi.cu) and their kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/kda.h"
#include "kda_common.cuh"

namespace kda {
namespace glr {

struct Params {
  const void* x;        // forward: x;  backward: d_out           [tokens, D] io type
  const void* g;        // [tokens, D] gate type
  const void* y;        // backward: the forward's y              [tokens, D] io type
  const float* h0;      // initial states [NS, D] or null (zeros)
  const float* init;    // what the scan starts from: h0, backward d_final_state; or null (zeros)
  const int32_t* cu;    // [NS + 1] or null
  void* out;            // forward: y;  backward: dx              [tokens, D] io type
  void* dg;             // backward: [tokens, D] gate type
  float* fin;           // forward: final states; backward: d_initial_state; [NS, D] or null
  uint32_t* status;     // device status word (null where nothing is reported)
  unsigned long long wait_ns;  // limit of a bounded wait for work (drains have their own)
  long tokens;          // in all
  int T, D, num_seqs;   // T: tokens of a sequence (without cu)
};

cudaError_t launch(const Params& p, bool backward, bool bf16, bool gate_bf16, cudaStream_t stream);

struct StepParams {
  const void* x;
  const void* g;
  float* state;
  const int32_t* slots;  // [B] or null
  void* y;
  uint32_t* status;
  int B, T, D, num_slots;
};
cudaError_t launch_step(const StepParams& p, bool bf16, bool gate_bf16, cudaStream_t stream);

}  // namespace glr

namespace gn {

struct Params {
  const void* x;
  const void* dy;      // backward
  const float* w;      // [C] or null (ones)
  const float* b;      // [C] or null (zeros)
  void* out;           // forward: y; backward: dx or null
  float* mean;         // [N, groups] forward: written or null; backward: read
  float* rstd;
  float* dw;           // backward: [C] or null
  float* db;
  uint8_t* work;
  long N, L;
  int C, groups;
  float eps;
  bool silu;
};

size_t fwd_workspace_bytes(long N, long L, int C, int groups);
size_t bwd_workspace_bytes(long N, long L, int C, int groups);
cudaError_t launch_fwd(const Params& p, bool bf16, cudaStream_t stream);
cudaError_t launch_bwd(const Params& p, bool bf16, cudaStream_t stream);

}  // namespace gn

namespace adamw {

cudaError_t launch(const kda_adamw_tensor* tensors, int count, const kda_adamw_config& config, cudaStream_t stream);

}  // namespace adamw
}  // namespace kda
