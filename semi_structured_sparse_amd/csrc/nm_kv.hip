// The paged key/value cache: appending (with or without rotary positions), reading back, and
// moving an accepted tree path's rows together.
#include "nm_decode_internal.h"

namespace nm {
namespace {

constexpr int kThreads = 256;

template <int FMT>
struct Codes {
  static constexpr int kBytes = FMT == NM_KV_FP16 ? 2 : 1;
  static constexpr float kLargest = FMT == NM_KV_INT8 ? 127.0f : 448.0f;
};

constexpr float kTiniest = 1e-30f;   // rows below it are held as zeros

// One wave per (token, head) row; lane l holds elements 2l, 2l+1 (+128 for 256).
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendCall a) {
  constexpr int P = D / 128 > 0 ? D / 128 : 1;
  const int lane = threadIdx.x & 63;
  const int heads = a.q_heads + 2 * a.cache.kv_heads;
  const int64_t row = int64_t(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= a.batch * a.tokens * heads) return;
  const int head = int(row % heads);
  const int64_t token = row / heads, b = token / a.tokens;
  const int t = int(token % a.tokens);
  const bool live = t < count_of(a.count, b, int(a.tokens));
  const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.cache.kv_heads;
  const int h = is_q ? head : is_v ? head - a.q_heads - a.cache.kv_heads : head - a.q_heads;
  const uint16_t* x = is_q ? a.q + token * a.q_stride : is_v ? a.v + token * a.v_stride : a.k + token * a.k_stride;
  x += int64_t(h) * D;
  float e[2 * P];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 128 * p + 2 * lane + j;
      float y = 0.f;
      if (i < D && live) {
        y = half_bits_to_float(x[i]);
        if (!is_v && a.rope.positions != nullptr && i < a.rope.rot_dim) {
          const int pairs = a.rope.rot_dim / 2;
          const bool half = a.rope.layout == NM_ROPE_HALF;
          const bool second = half ? i >= pairs : (i & 1);
          const int u = half ? (second ? i - pairs : i) : i / 2;
          const int other = half ? (second ? i - pairs : i + pairs) : i ^ 1;
          float c, s;
          rotation(a.rope.positions[token], a.rope.turns[u], a.rope.scale, c, s);
          const float z = half_bits_to_float(x[other]);
          y = second ? y * c + z * s : y * c - z * s;
        }
      }
      e[2 * p + j] = y;
    }
  if (is_q) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 128 * p + 2 * lane + j;
        if (i < D) a.q_out[token * a.q_out_stride + int64_t(h) * D + i] = uint16_t(float_to_half_bits(e[2 * p + j]));
      }
    return;
  }
  if (!live) return;
  const int64_t at = cache_row(a.cache, b, int64_t(a.start[b]) + t, h);
  if (at < 0) return;
  char* out = (is_v ? a.cache.v : a.cache.k) + at * D * Codes<FMT>::kBytes;
  float up = 0.f;
  if constexpr (FMT != NM_KV_FP16) {
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) {
      amax = fmaxf(amax, fabsf(e[j]));
      bad |= !(fabsf(e[j]) < __builtin_inff());
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    bad = __any(bad);
    const bool held = !bad && amax >= kTiniest;
    up = held ? Codes<FMT>::kLargest / amax : 0.f;
    if (lane == 0)
      (is_v ? a.cache.v_scale : a.cache.k_scale)[at] =
          bad ? __builtin_nanf("") : held ? amax / Codes<FMT>::kLargest : 0.f;
    if (bad)
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) e[j] = 0.f;
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 128 * p + 2 * lane + j;
      if (i >= D) continue;
      const float y = e[2 * p + j];
      if constexpr (FMT == NM_KV_FP16) {
        reinterpret_cast<uint16_t*>(out)[i] = uint16_t(float_to_half_bits(y));
      } else {
        const float z = fminf(fmaxf(y * up, -Codes<FMT>::kLargest), Codes<FMT>::kLargest);
        if constexpr (FMT == NM_KV_INT8)
          out[i] = char(int(rintf(z)));
        else
          out[i] = char(__builtin_amdgcn_cvt_pk_fp8_f32(z, z, 0, false) & 0xFF);
      }
    }
}

template <int FMT>
__device__ __forceinline__ float decode(const char* row, int i) {
  if constexpr (FMT == NM_KV_FP16) return half_bits_to_float(reinterpret_cast<const uint16_t*>(row)[i]);
  if constexpr (FMT == NM_KV_INT8) return float(reinterpret_cast<const signed char*>(row)[i]);
  return __builtin_amdgcn_cvt_f32_fp8(int(uint8_t(row[i])), 0);
}

// One element of k or v per thread.
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadCall a) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t all = a.batch * a.tokens * a.cache.kv_heads * D;
  if (i >= 2 * all) return;
  const bool is_v = i >= all;
  const int64_t j = is_v ? i - all : i;
  const int e = int(j % D), head = int(j / D % a.cache.kv_heads);
  const int64_t token = j / D / a.cache.kv_heads, b = token / a.tokens;
  const int t = int(token % a.tokens);
  float y = 0.f;
  if (t < count_of(a.count, b, int(a.tokens))) {
    const int64_t at = cache_row(a.cache, b, int64_t(a.start[b]) + t, head);
    if (at >= 0) {
      y = decode<FMT>((is_v ? a.cache.v : a.cache.k) + at * D * Codes<FMT>::kBytes, e);
      if constexpr (FMT != NM_KV_FP16) y *= (is_v ? a.cache.v_scale : a.cache.k_scale)[at];
    }
  }
  (is_v ? a.v_out : a.k_out)[j] = uint16_t(float_to_half_bits(y));
}

// One workgroup per sequence, head and side (k or v). Every row is in registers before any is
// written: destinations of some rows are sources of others.
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void compact_kernel(CompactCall a) {
  constexpr int kChunks = D * Codes<FMT>::kBytes / 16;           // 16-byte pieces of a row
  constexpr int kEach = (kMaxNodes * kChunks + kThreads - 1) / kThreads;
  const int head = blockIdx.x % a.cache.kv_heads;
  const bool is_v = blockIdx.x / a.cache.kv_heads;
  const int64_t b = blockIdx.y;
  char* base = is_v ? a.cache.v : a.cache.k;
  float* scales = is_v ? a.cache.v_scale : a.cache.k_scale;
  const int accepted = count_of(a.accepted, b, a.nodes - 1);
  const int64_t start = a.start[b];
  uint4 held[kEach];
  int64_t to[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int piece = threadIdx.x + kThreads * j, d = piece / kChunks + 1;
    to[j] = -1;
    if (d > accepted) continue;
    const int node = a.path[b * a.nodes + d];
    if (node < 0 || node >= a.nodes || node == d) continue;
    const int64_t from = cache_row(a.cache, b, start + node, head);
    const int64_t into = cache_row(a.cache, b, start + d, head);
    if (from < 0 || into < 0) continue;
    held[j] = reinterpret_cast<const uint4*>(base + from * D * Codes<FMT>::kBytes)[piece % kChunks];
    to[j] = into * kChunks + piece % kChunks;
  }
  float scale = 0.f;
  int64_t scale_to = -1;
  if (FMT != NM_KV_FP16 && threadIdx.x >= 1 && int(threadIdx.x) <= accepted) {
    const int node = a.path[b * a.nodes + threadIdx.x];
    if (node >= 0 && node < a.nodes) {
      const int64_t from = cache_row(a.cache, b, start + node, head);
      scale_to = cache_row(a.cache, b, start + threadIdx.x, head);
      if (from >= 0 && scale_to >= 0) scale = scales[from]; else scale_to = -1;
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // the loads have returned
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kEach; ++j)
    if (to[j] >= 0) reinterpret_cast<uint4*>(base)[to[j]] = held[j];
  if (scale_to >= 0) scales[scale_to] = scale;
}

template <template <int, int> class K, class Call>
hipError_t by_kind(const Call& c, int head_dim, int format, dim3 grid, hipStream_t stream, const DeviceInfo& dev) {
  Call a = c;
  void* args[] = {&a};
  const void* f = nullptr;
#define NM_KIND(D, F) \
  if (head_dim == D && format == F) f = K<D, F>::kernel();
  NM_KIND(64, 0) NM_KIND(64, 1) NM_KIND(64, 2)
  NM_KIND(128, 0) NM_KIND(128, 1) NM_KIND(128, 2)
  NM_KIND(256, 0) NM_KIND(256, 1) NM_KIND(256, 2)
#undef NM_KIND
  if (f == nullptr) return hipErrorInvalidValue;
  return launch(f, grid, dim3(kThreads), args, 0, stream, dev);
}

template <int D, int F>
struct AppendKernel { static const void* kernel() { return reinterpret_cast<const void*>(append_kernel<D, F>); } };
template <int D, int F>
struct ReadKernel { static const void* kernel() { return reinterpret_cast<const void*>(read_kernel<D, F>); } };
template <int D, int F>
struct CompactKernel { static const void* kernel() { return reinterpret_cast<const void*>(compact_kernel<D, F>); } };

}  // namespace

hipError_t launch_append(const AppendCall& c, int head_dim, int format, hipStream_t stream, const DeviceInfo& dev) {
  const int64_t rows = c.batch * c.tokens * (c.q_heads + 2 * c.cache.kv_heads);
  const int64_t grid = (rows + kThreads / 64 - 1) / (kThreads / 64);
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  return by_kind<AppendKernel>(c, head_dim, format, dim3(uint32_t(grid)), stream, dev);
}

hipError_t launch_read(const ReadCall& c, int head_dim, int format, hipStream_t stream, const DeviceInfo& dev) {
  const int64_t grid = (2 * c.batch * c.tokens * c.cache.kv_heads * head_dim + kThreads - 1) / kThreads;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  return by_kind<ReadKernel>(c, head_dim, format, dim3(uint32_t(grid)), stream, dev);
}

hipError_t launch_compact(const CompactCall& c, int head_dim, int format, hipStream_t stream, const DeviceInfo& dev) {
  return by_kind<CompactKernel>(c, head_dim, format, dim3(2 * c.cache.kv_heads, uint32_t(c.batch)), stream, dev);
}

}  // namespace nm
