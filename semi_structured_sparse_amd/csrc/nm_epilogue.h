// What the block products (nm_linear, nm_gated) do with their fp32 sums before the one rounding
// to fp16. Every product kernel calls these where it would round and store.
//
//   linear  y = scale * act(sum + bias) + residual
//   gated   y = act(sum_gate + bias_gate) * (sum_up + bias_up)
//
// The activation is chosen at run time by a uniform branch: one a workgroup or an output, beside the
// hundreds of products that made its sum, and a kernel for each would multiply the library.
#pragma once

#include "../../include/nm_block.h"   // by its place: programs that check a kernel header give csrc alone
#include "nm_internal.h"

namespace nm {

__device__ __forceinline__ float half_at(const uint16_t* p, size_t i) { return float(__builtin_bit_cast(_Float16, p[i])); }

// x * 1/(1 + exp(-t)). v_exp_f32 and v_rcp_f32 are good to about 1 ulp of fp32 (the exponent's
// product with log2 e to |t| 2^-24 more), far below the fp16 rounding that follows. exp(-t) past the
// largest float is infinite and its reciprocal 0, the limit.
__device__ __forceinline__ float logistic_times(float x, float t) {
  return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.4426950408889634f));
}

// x Phi(x) = max(x, 0) - |x| Q, Q = Phi(-|x|) = t P(t) exp(-x^2 / 2) with t = 1 / (1 + k |x|). P, of
// degree 7, was fitted to Q exp(x^2 / 2) by least squares, weighted until its ripples were even: 9.4e-8
// of it up to |x| = 14, past which |x| Q is below every float here. A rounding of x^2 / 2 moves exp by
// x^2 / 2 of its own size. Nothing cancels on the far negative side (1 + erf would lose its digits there).
__device__ __forceinline__ float gelu(float x) {
  const float w = fminf(fabsf(x), 14.0f);
  const float t = __builtin_amdgcn_rcpf(fmaf(w, 0.23334524f, 1.0f));
  float p = -6.767277420e-02f;
  p = fmaf(p, t, 2.301182747e-01f);
  p = fmaf(p, t, -1.755743772e-01f);
  p = fmaf(p, t, 2.042495608e-01f);
  p = fmaf(p, t, 2.361056022e-02f);
  p = fmaf(p, t, 1.006118730e-01f);
  p = fmaf(p, t, 9.147798270e-02f);
  p = fmaf(p, t, 9.317889810e-02f);
  const float q = w * t * p * __builtin_amdgcn_exp2f(w * w * -0.72134752044448170f);
  return (x < 0.0f ? 0.0f : x) - q;   // NaN stays
}

// (1 + tanh u) / 2 is the logistic function of 2 u; 2 sqrt(2 / pi) = 1.5957...
__device__ __forceinline__ float gelu_tanh(float x) {
  return logistic_times(x, 1.5957691216057308f * x * fmaf(0.044715f * x, x, 1.0f));
}

__device__ __forceinline__ float relu(float x) { return x < 0.0f ? 0.0f : x; }   // NaN stays

__device__ __forceinline__ float activate(float x, int activation) {
  switch (activation) {
    case NM_ACT_RELU: return relu(x);
    case NM_ACT_SILU: return logistic_times(x, x);
    case NM_ACT_GELU: return gelu(x);
    case NM_ACT_GELU_TANH: return gelu_tanh(x);
    default: return x;
  }
}

// Calls f with the activation as a function: one branch for many elements.
template <typename F>
__device__ __forceinline__ void with_activation(int activation, F f) {
  switch (activation) {
    case NM_ACT_RELU: f([](float x) { return relu(x); }); break;
    case NM_ACT_SILU: f([](float x) { return logistic_times(x, x); }); break;
    case NM_ACT_GELU: f([](float x) { return gelu(x); }); break;
    case NM_ACT_GELU_TANH: f([](float x) { return gelu_tanh(x); }); break;
    default: f([](float x) { return x; });
  }
}

__device__ __forceinline__ float linear_out(const BlockArgs& e, float sum, float bias, float residual) {
  return fmaf(e.scale, activate(sum + bias, e.activation), residual);
}

__device__ __forceinline__ float gated_out(const BlockArgs& e, float gate, float up, float gate_bias, float up_bias) {
  return activate(gate + gate_bias, e.activation) * (up + up_bias);
}

__device__ __forceinline__ uint16_t to_half(float x) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x)); }

// The fp16 output of one row and vector from its sum (gated: `up` the second matrix's).
template <int FORM>
__device__ __forceinline__ uint16_t finish(const BlockArgs& e, float sum, float up, unsigned row, size_t at) {
  if constexpr (FORM == kLinearForm) {
    return to_half(linear_out(e, sum, e.bias ? half_at(e.bias, row) : 0.0f, e.residual ? half_at(e.residual, at) : 0.0f));
  } else if constexpr (FORM == kGatedForm) {
    return to_half(gated_out(e, sum, up, e.bias ? half_at(e.bias, row) : 0.0f, e.up_bias ? half_at(e.up_bias, row) : 0.0f));
  } else {
    return to_half(sum);
  }
}

// Whether groups of 8 rows of one vector can be read and written in 16 bytes.
__device__ __forceinline__ bool wide_ok(const BlockArgs& e, const uint16_t* Y, int rows) {
  const uintptr_t any = reinterpret_cast<uintptr_t>(Y) | reinterpret_cast<uintptr_t>(e.bias) |
                        reinterpret_cast<uintptr_t>(e.up_bias) | reinterpret_cast<uintptr_t>(e.residual);
  return (rows & 7) == 0 && (any & 15) == 0;
}

// Elements i .. i+N-1 of an fp16 array of which `count` from i on exist; zeros for NULL.
template <int N>
__device__ __forceinline__ void load_halves(const uint16_t* p, size_t i, int count, bool wide, float (&f)[N]) {
  typedef _Float16 group __attribute__((ext_vector_type(N)));
#pragma unroll
  for (int k = 0; k < N; ++k) f[k] = 0.0f;
  if (p == nullptr) return;
  if (wide) {
    const group v = *reinterpret_cast<const group*>(p + i);
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = float(v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < count) f[k] = half_at(p, i + k);
  }
}

// The outputs of rows row .. row+N-1 (those below `rows`) of one vector from their sums, stored at
// Y[at ..]. wide: all N rows are there, and aligned to N halves.
template <int FORM, int N>
__device__ __forceinline__ void finish_rows(const BlockArgs& e, const float (&sum)[N], const float (&up)[N], int row, int rows,
                                            size_t at, bool wide, uint16_t* Y) {
  typedef _Float16 group __attribute__((ext_vector_type(N)));
  float b[N], c[N];
  load_halves<N>(e.bias, size_t(row), rows - row, wide, b);
  load_halves<N>(FORM == kGatedForm ? e.up_bias : e.residual, FORM == kGatedForm ? size_t(row) : at, rows - row, wide, c);
  group h;
#pragma unroll
  for (int k = 0; k < N; ++k)
    h[k] = static_cast<_Float16>(FORM == kGatedForm ? gated_out(e, sum[k], up[k], b[k], c[k]) : linear_out(e, sum[k], b[k], c[k]));
  if (wide) {
    *reinterpret_cast<group*>(Y + at) = h;
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (row + k < rows) Y[at + k] = to_half(float(h[k]));
  }
}

}  // namespace nm
