// Declarations shared by the translation units of nm_block.h beside the products (whose arguments are
// in nm_internal.h): the checked arguments of the norms and of the scores.
#pragma once

#include "nm_block.h"
#include "nm_internal.h"

namespace nm {

struct NormCall {
  const void* x;            // the stream (fp16 or fp32), or what is normalised
  const uint16_t* branch;   // NULL: y = norm(x)
  void* h;                  // NULL: not stored
  uint16_t* y;
  const uint16_t *post, *gate, *weight, *bias;
  int64_t x_stride, branch_stride, h_stride, y_stride, gate_stride;   // elements between tokens
  int64_t rows;             // tokens * heads
  int heads, width;
  int kind;
  float scale, offset, eps;
};

struct ScoreCall {
  const void* logits;
  const int32_t* tokens;    // NULL: no log probability of given tokens
  float *logprob, *entropy, *top_logprobs;
  int32_t* top_tokens;
  int64_t stride;
  int rows, vocab, top;
  float scale;
};

hipError_t launch_norm(const NormCall& c, bool fp32_stream, hipStream_t stream, const DeviceInfo& dev);
hipError_t launch_score(const ScoreCall& c, bool fp16, void* workspace, size_t workspace_bytes, hipStream_t stream,
                        const DeviceInfo& dev);
size_t score_workspace_bytes(int64_t rows, int64_t vocab, const DeviceInfo& dev);

}  // namespace nm
