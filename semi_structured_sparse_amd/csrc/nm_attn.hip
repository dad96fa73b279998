// Attention of a step's nodes over the paged cache.
#include <cmath>

#include "nm_decode_internal.h"

namespace nm {
namespace {

constexpr int kThreads = 256;

template <int FMT>
__device__ __forceinline__ float decode(const char* row, int i) {
  if constexpr (FMT == NM_KV_FP16) return half_bits_to_float(reinterpret_cast<const uint16_t*>(row)[i]);
  if constexpr (FMT == NM_KV_INT8) return float(reinterpret_cast<const signed char*>(row)[i]);
  return __builtin_amdgcn_cvt_f32_fp8(int(uint8_t(row[i])), 0);
}

// One workgroup per query row; its four waves take every fourth key, a lane D/64 elements,
// with the running maximum and sum of the softmax.
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttnCall a) {
  constexpr int E = D / 64;
  constexpr int kBytes = FMT == NM_KV_FP16 ? 2 : 1;
  __shared__ float part[4][D + 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int head = blockIdx.x % a.heads, t = blockIdx.x / a.heads;
  const int64_t b = blockIdx.y;
  const int count = count_of(a.count, b, a.tokens);
  const int64_t most = int64_t(a.cache.table_width) << a.cache.page_shift;
  const int64_t ctx = a.context[b] < 0 ? 0 : a.context[b] > most ? most : a.context[b];
  const int64_t keys = ctx + count < most ? ctx + count : most;
  const uint64_t mask = a.mask != nullptr ? a.mask[b * a.tokens + t] : t >= 63 ? ~0ull : (2ull << t) - 1;
  uint16_t* out = a.out + ((b * a.tokens + t) * a.heads + head) * D;
  float q[E], o[E], m = -__builtin_inff(), l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = half_bits_to_float(a.q[(b * a.tokens + t) * a.q_stride + int64_t(head) * D + lane + 64 * e]) * a.scale;
    o[e] = 0.f;
  }
  for (int64_t j = wave; j < keys && t < count; j += 4) {
    if (j >= ctx && !((mask >> (j - ctx)) & 1)) continue;
    const int64_t row = cache_row(a.cache, b, j, head / a.group);
    if (row < 0) continue;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * decode<FMT>(a.cache.k + row * D * kBytes, lane + 64 * e);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) s += __shfl_xor(s, x);
    if constexpr (FMT != NM_KV_FP16) s *= a.cache.k_scale[row];
    const float top = fmaxf(m, s);
    const float old = m > -__builtin_inff() ? expf(m - top) : 0.f, p = s == -__builtin_inff() ? 0.f : expf(s - top);
    m = top;
    l = l * old + p;
    float w = p;
    if constexpr (FMT != NM_KV_FP16) w *= a.cache.v_scale[row];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * old + w * decode<FMT>(a.cache.v + row * D * kBytes, lane + 64 * e);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[wave][lane + 64 * e] = o[e];
  if (lane == 0) {
    part[wave][D] = m;
    part[wave][D + 1] = l;
  }
  __syncthreads();
  if (wave != 0) return;
  m = fmaxf(fmaxf(part[0][D], part[1][D]), fmaxf(part[2][D], part[3][D]));
  l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float f = part[w][D] > -__builtin_inff() ? expf(part[w][D] - m) : 0.f;
    l += part[w][D + 1] * f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += part[w][lane + 64 * e] * f;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 64 * e] = uint16_t(float_to_half_bits(l == 0.f ? 0.f : o[e] / l));
}

template <int D>
const void* of_format(int format) {
  return format == NM_KV_FP16   ? reinterpret_cast<const void*>(attention_kernel<D, NM_KV_FP16>)
         : format == NM_KV_INT8 ? reinterpret_cast<const void*>(attention_kernel<D, NM_KV_INT8>)
                                : reinterpret_cast<const void*>(attention_kernel<D, NM_KV_E4M3>);
}

}  // namespace

size_t attention_workspace_bytes(const AttnCall&, int, int, const DeviceInfo&) { return 0; }

hipError_t launch_attention(const AttnCall& c, int head_dim, int format, void*, size_t, hipStream_t stream,
                            const DeviceInfo& dev) {
  AttnCall a = c;
  void* args[] = {&a};
  const void* f = head_dim == 64 ? of_format<64>(format) : head_dim == 128 ? of_format<128>(format) : of_format<256>(format);
  return launch(f, dim3(uint32_t(c.heads) * uint32_t(c.tokens), uint32_t(c.batch)), dim3(kThreads), args, 0, stream, dev);
}

}  // namespace nm
