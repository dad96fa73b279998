// C ABI of nm_block.h: argument checks (no HIP call before they pass) and dispatch to the kernels.
#include <cmath>

#include "nm_block_internal.h"
#include "nm_decode.h"

namespace nm {
namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool within(int64_t v, int64_t low, int64_t high) { return v >= low && v <= high; }

bool positive(float v) { return v > 0.0f && std::isfinite(v); }

int finish(hipError_t e) {
  if (e == hipSuccess) return NM_OK;
  set_last_hip_error(e);
  return NM_ERR_HIP;
}

// Sizes of the block products whose every launch stays within a grid's 2^32 threads: 64 a row in the
// single-vector kernels, 256 for 64 x 64 outputs of the prompt kernels. all: the rows of both matrices.
bool grid_fits(int64_t all, int64_t batch) { return all <= (int64_t(1) << 26) - 64 && batch <= (int64_t(1) << 35) / all; }

int norm_check(const NormCall& c, bool fp32, int64_t heads, int64_t width) {
  const uintptr_t wide = fp32 ? 4 : 2;
  if (!c.x || !c.y) return NM_ERR_NULL;
  if (!within(c.kind, NM_NORM_RMS, NM_NORM_LAYER)) return NM_ERR_FORMAT;
  // a row takes at most a thread for every four elements, 16 or more, and a grid 2^32
  if (c.rows < 1 || !within(width, 1, 32768) || c.rows > (int64_t(1) << 33) / (width < 128 ? 128 : width))
    return NM_ERR_SHAPE;
  const int64_t row = heads * width;
  if (!within(c.x_stride, row, kMaxStride) || !within(c.y_stride, row, kMaxStride)) return NM_ERR_SHAPE;
  if (c.branch && !within(c.branch_stride, row, kMaxStride)) return NM_ERR_SHAPE;
  if (c.h && !within(c.h_stride, row, kMaxStride)) return NM_ERR_SHAPE;
  if (c.gate && c.gate_stride != 0 && !within(c.gate_stride, row, kMaxStride)) return NM_ERR_SHAPE;
  if (!(c.eps >= 0.0f) || !std::isfinite(c.eps) || !std::isfinite(c.scale) || !std::isfinite(c.offset)) return NM_ERR_SHAPE;
  if (!aligned(c.x, wide) || !aligned(c.h, wide)) return NM_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(c.branch), static_cast<const void*>(c.y), static_cast<const void*>(c.post),
                        static_cast<const void*>(c.gate), static_cast<const void*>(c.weight), static_cast<const void*>(c.bias)})
    if (!aligned(p, 2)) return NM_ERR_ALIGN;
  return NM_OK;
}

int norm(const NormCall& c, bool fp32, void* stream) {
  DeviceInfo dev;
  const hipError_t e = current_device_info(&dev);
  if (e != hipSuccess) return finish(e);
  return finish(launch_norm(c, fp32, static_cast<hipStream_t>(stream), dev));
}

}  // namespace
}  // namespace nm

using nm::aligned;
using nm::within;

extern "C" {

int nm_linear(const uint16_t* values, const uint32_t* masks, const uint16_t* X, uint16_t* Y, int64_t rows, int64_t cols,
              int64_t batch, int N, int M, const uint16_t* bias, int activation, float scale, const uint16_t* residual,
              void* workspace, size_t workspace_bytes, void* stream) {
  const int st = nm::spmm_check(values, masks, X, Y, rows, cols, batch, N, M);
  if (st != NM_OK) return st;
  if (!nm::grid_fits(rows, batch)) return NM_ERR_SHAPE;
  if (!within(activation, NM_ACT_NONE, NM_ACT_GELU_TANH)) return NM_ERR_FORMAT;
  if (!aligned(bias, 2) || !aligned(residual, 2)) return NM_ERR_ALIGN;
  const nm::BlockArgs e{nullptr, nullptr, bias, nullptr, residual, scale, activation};
  return nm::spmm_dispatch(values, masks, X, Y, rows, cols, batch, N, M, stream, workspace, workspace_bytes, &e);
}

int nm_gated(const uint16_t* gate_values, const uint32_t* gate_masks, const uint16_t* up_values, const uint32_t* up_masks,
             const uint16_t* X, uint16_t* Y, int64_t rows, int64_t cols, int64_t batch, int N, int M,
             const uint16_t* gate_bias, const uint16_t* up_bias, int activation, void* workspace, size_t workspace_bytes,
             void* stream) {
  if (!up_values || !up_masks) return NM_ERR_NULL;
  int st = nm::spmm_check(gate_values, gate_masks, X, Y, rows, cols, batch, N, M);
  // the rows of both are what the launches go by
  if (st == NM_OK && rows > INT64_MAX / 2) st = NM_ERR_SHAPE;
  if (st == NM_OK) st = nm::spmm_check(up_values, up_masks, X, Y, 2 * rows, cols, batch, N, M);
  if (st != NM_OK) return st;
  if (!nm::grid_fits(2 * rows, batch)) return NM_ERR_SHAPE;
  if (!within(activation, NM_ACT_NONE, NM_ACT_GELU_TANH)) return NM_ERR_FORMAT;
  if (!aligned(gate_bias, 2) || !aligned(up_bias, 2)) return NM_ERR_ALIGN;
  const nm::BlockArgs e{up_values, up_masks, gate_bias, up_bias, nullptr, 1.0f, activation};
  return nm::spmm_dispatch(gate_values, gate_masks, X, Y, rows, cols, batch, N, M, stream, workspace, workspace_bytes, &e);
}

size_t nm_gated_workspace_bytes(int64_t rows, int64_t cols, int64_t batch, int N, int M) {
  if (nm_values_count(rows, cols, N, M) == 0 || nm_values_count(2 * rows, cols, N, M) == 0 || batch < 1) return 0;
  nm::DeviceInfo dev;
  if (nm::current_device_info(&dev) != hipSuccess) return 0;
  return nm::spmm_workspace_bytes(rows, cols, batch, N, M, dev, true);
}

int nm_norm(const void* x, uint16_t* y, const uint16_t* weight, const uint16_t* bias, int64_t tokens, int64_t heads,
            int64_t width, int64_t x_stride, int64_t y_stride, int fp32_input, int kind, float offset, float eps,
            void* stream) {
  if (tokens < 1 || !within(heads, 1, int64_t(1) << 24) || tokens > (int64_t(1) << 33) / heads) return NM_ERR_SHAPE;
  nm::NormCall c{};
  c.x = x;
  c.y = y;
  c.weight = weight;
  c.bias = bias;
  c.x_stride = x_stride;
  c.y_stride = y_stride;
  c.rows = tokens * heads;
  c.heads = int(heads);
  c.width = int(width < 32769 ? width : 32769);
  c.kind = kind;
  c.scale = 1.0f;
  c.offset = offset;
  c.eps = eps;
  const int st = nm::norm_check(c, fp32_input != 0, heads, width);
  return st != NM_OK ? st : nm::norm(c, fp32_input != 0, stream);
}

int nm_block_norm(const void* x, const uint16_t* branch, void* h, uint16_t* y, const uint16_t* post, const uint16_t* gate,
                  const uint16_t* weight, const uint16_t* bias, int64_t rows, int64_t width, int64_t x_stride,
                  int64_t branch_stride, int64_t h_stride, int64_t y_stride, int64_t gate_stride, int fp32_stream, int kind,
                  float scale, float offset, float eps, void* stream) {
  if (!branch) return NM_ERR_NULL;
  nm::NormCall c{};
  c.x = x;
  c.branch = branch;
  c.h = h;
  c.y = y;
  c.post = post;
  c.gate = gate;
  c.weight = weight;
  c.bias = bias;
  c.x_stride = x_stride;
  c.branch_stride = branch_stride;
  c.h_stride = h_stride;
  c.y_stride = y_stride;
  c.gate_stride = gate_stride;
  c.rows = rows;
  c.heads = 1;
  c.width = int(width < 32769 ? width : 32769);
  c.kind = kind;
  c.scale = scale;
  c.offset = offset;
  c.eps = eps;
  const int st = nm::norm_check(c, fp32_stream != 0, 1, width);
  return st != NM_OK ? st : nm::norm(c, fp32_stream != 0, stream);
}

int nm_logprobs(const void* logits, const int32_t* tokens, float* logprob, float* entropy, int32_t* top_tokens,
                float* top_logprobs, int64_t rows, int64_t vocab, int64_t stride, int64_t top, int fp16_logits, float scale,
                void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits || (tokens != nullptr) != (logprob != nullptr)) return NM_ERR_NULL;
  if (!within(rows, 1, int64_t(1) << 23) || !within(vocab, 1, int64_t(1) << 24) || !within(top, 0, NM_MAX_TOP) || top > vocab ||
      !within(stride, vocab, nm::kMaxStride) || !nm::positive(scale))
    return NM_ERR_SHAPE;
  if (top > 0 && (!top_tokens || !top_logprobs)) return NM_ERR_NULL;
  if (!aligned(logits, fp16_logits ? 2 : 4) || !aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
      !aligned(top_tokens, 4) || !aligned(top_logprobs, 4) || !aligned(workspace, 16))
    return NM_ERR_ALIGN;
  nm::DeviceInfo dev;
  const hipError_t e = nm::current_device_info(&dev);
  if (e != hipSuccess) return nm::finish(e);
  const nm::ScoreCall c{logits, tokens, logprob, entropy, top_logprobs, top_tokens, stride, int(rows), int(vocab), int(top), scale};
  return nm::finish(nm::launch_score(c, fp16_logits != 0, workspace, workspace_bytes, static_cast<hipStream_t>(stream), dev));
}

size_t nm_logprobs_workspace_bytes(int64_t rows, int64_t vocab) {
  if (!within(rows, 1, int64_t(1) << 23) || !within(vocab, 1, int64_t(1) << 24)) return 0;
  nm::DeviceInfo dev;
  if (nm::current_device_info(&dev) != hipSuccess) return 0;
  return nm::score_workspace_bytes(rows, vocab, dev);
}

}  // extern "C"
