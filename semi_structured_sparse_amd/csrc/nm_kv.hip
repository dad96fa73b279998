// The paged key/value cache: appending (with or without rotary positions), reading back, and
// moving an accepted tree path's rows together.
#include <type_traits>

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

// Lanes that hold a row of D elements, 16 each.
template <int D>
struct RowLanes {
  static constexpr int kLanes = D / 16;
  static constexpr int kRows = kThreads / kLanes;   // of a workgroup
};

// The largest of the row's lanes (4, 8 or 16 neighbours): within quads, then mirrored across
// them.
template <int LANES>
__device__ __forceinline__ float row_max(float x) {
  const auto dpp = [](float v, auto ctrl) {
    return __uint_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0xB1>{}));    // quad_perm 1,0,3,2
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x4E>{}));    // quad_perm 2,3,0,1
  if (LANES > 4) x = fmaxf(x, dpp(x, std::integral_constant<int, 0x141>{}));   // row_half_mirror
  if (LANES > 8) x = fmaxf(x, dpp(x, std::integral_constant<int, 0x140>{}));   // row_mirror
  return x;
}

// 8 codes of e * up, which is at most the largest code's value (and an fp32 rounding, which the
// rounding to a code takes off). An integer to nearest even is what 1.5 2^23 leaves room for: it
// ends up in the sum's low bits, in two's complement.
template <int FMT>
__device__ __forceinline__ u32x2 codes_of(const float (&e)[8], float up) {
#pragma clang fp contract(off)   // the product is rounded before it is made an integer
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = e[4 * h + i] * up;
    if constexpr (FMT == NM_KV_E4M3) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
      w[h] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], v, true));
    } else {
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(z[i] + 12582912.0f);
      w[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0C0C0400u),
                                   __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), 0x05040100u);
    }
  }
  return w;
}

// D / 16 lanes per (token, head) row; the token's rows are its q heads (turned only), its k
// heads and its v heads. Mathematics: nm_decode.h's rounding of a row to codes; the row's largest
// magnitude is a maximum over its lanes, its scale an exact division. What bounds it: the copy, 2
// bytes an element in, 1 or 2 out, and behind it about as long in instructions, two divisions, a
// maximum and a rounding for 16 elements a lane. 14337 of 16384 tokens, 8 + 8 heads of 128, to
// int8 (89 MB): 20.6 us, 4.3 TB/s (19.8 before the angles took registers of the eighth wave of
// a SIMD; held to eight, turned prompts take 3% longer; 24.0 before with clamped conversions to
// integers and a comparison an element for infinities, 1 of it by looking the page up only once the
// elements have come); one rotated token of 16 sequences 3.9 us.
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendCall a) {
  constexpr int kLanes = RowLanes<D>::kLanes;
  const uint32_t heads = uint32_t(a.q_heads + 2 * a.cache.kv_heads);
  const uint32_t row = blockIdx.x * RowLanes<D>::kRows + threadIdx.x / kLanes;
  const int unit = threadIdx.x % kLanes;
  if (row >= uint32_t(a.batch * a.tokens) * heads) return;
  const uint32_t token = row / heads, b = token / uint32_t(a.tokens);
  const int head = int(row - token * heads), t = int(token - b * uint32_t(a.tokens));
  const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.cache.kv_heads;
  const int h = is_q ? head : is_v ? head - a.q_heads - a.cache.kv_heads : head - a.q_heads;
  const uint16_t* x = is_q   ? a.q + int64_t(token) * a.q_stride
                      : is_v ? a.v + int64_t(token) * a.v_stride
                             : a.k + int64_t(token) * a.k_stride;
  x += int64_t(h) * D;
  // the row's place is looked up while its elements are on their way
  const int count = count_of(a.count, b, int(a.tokens));
  const int64_t start = a.start[b];
  const HeadUnit hu = head_unit(unit, is_v ? 0 : a.rope.rot_dim, D);
  u32x4 p = *reinterpret_cast<const u32x4*>(x + hu.first), q = *reinterpret_cast<const u32x4*>(x + hu.second);
  const bool live = t < count;
  const int64_t at = is_q ? -1 : cache_row(a.cache, b, start + t, h);
  float e[8], f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    e[i] = half_at(p, i);
    f[i] = half_at(q, i);
  }
  if (hu.turned) {
    turn_unit(unit_rotation(a.rope, unit, a.rope.positions[token]), a.rope.layout, e, f);
    if (is_q || FMT == NM_KV_FP16) {
      p = halves_of(e);
      q = halves_of(f);
    }
  }
  if (is_q) {
    if (!live) p = q = u32x4{0, 0, 0, 0};
    uint16_t* y = a.q_out + int64_t(token) * a.q_out_stride + int64_t(h) * D;
    *reinterpret_cast<u32x4*>(y + hu.first) = p;
    *reinterpret_cast<u32x4*>(y + hu.second) = q;
    return;
  }
  if (!live || at < 0) return;   // a row's lanes go together
  char* out = (is_v ? a.cache.v : a.cache.k) + at * D * Codes<FMT>::kBytes;
  if constexpr (FMT == NM_KV_FP16) {
    *reinterpret_cast<u32x4*>(out + 2 * hu.first) = p;
    *reinterpret_cast<u32x4*>(out + 2 * hu.second) = q;
  } else {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)   // NaN if one is
      amax = __builtin_elementwise_maximum(amax, __builtin_elementwise_maximum(fabsf(e[i]), fabsf(f[i])));
    amax = row_max<kLanes>(amax < __builtin_inff() ? amax : __builtin_inff());
    const bool bad = amax == __builtin_inff();
    const bool held = !bad && amax >= kTiniest;
    const float up = held ? Codes<FMT>::kLargest / amax : 0.f;
    if (unit == 0)
      (is_v ? a.cache.v_scale : a.cache.k_scale)[at] =
          bad ? __builtin_nanf("") : held ? amax / Codes<FMT>::kLargest : 0.f;
    u32x2 c = codes_of<FMT>(e, up), d = codes_of<FMT>(f, up);
    if (bad) c = d = u32x2{0, 0};
    *reinterpret_cast<u32x2*>(out + hu.first) = c;
    *reinterpret_cast<u32x2*>(out + hu.second) = d;
  }
}

// Four codes to fp32.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t codes, float (&y)[4]) {
  if constexpr (FMT == NM_KV_E4M3) {
    y[0] = __builtin_amdgcn_cvt_f32_fp8(int(codes), 0);
    y[1] = __builtin_amdgcn_cvt_f32_fp8(int(codes), 1);
    y[2] = __builtin_amdgcn_cvt_f32_fp8(int(codes), 2);
    y[3] = __builtin_amdgcn_cvt_f32_fp8(int(codes), 3);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = float(int(codes << (24 - 8 * i)) >> 24);
  }
}

// D / 16 lanes per (token, head) row of k, then of v; a copy, widened to fp16: 16 bytes of codes
// a lane in, 32 out. 14337 int8 tokens of 8 + 8 heads into 16384 (97 MB): 17.6 us, 5.5 TB/s.
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadCall a) {
  constexpr int kLanes = RowLanes<D>::kLanes;
  const uint32_t heads = uint32_t(a.cache.kv_heads), rows = uint32_t(a.batch * a.tokens) * heads;
  const uint32_t row = blockIdx.x * RowLanes<D>::kRows + threadIdx.x / kLanes;
  const int unit = threadIdx.x % kLanes;
  const bool is_v = blockIdx.y != 0;
  if (row >= rows) return;
  const uint32_t token = row / heads, b = token / uint32_t(a.tokens);
  const int head = int(row - token * heads), t = int(token - b * uint32_t(a.tokens));
  u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  if (t < count_of(a.count, b, int(a.tokens))) {
    const int64_t at = cache_row(a.cache, b, int64_t(a.start[b]) + t, head);
    if (at >= 0) {
      const char* in = (is_v ? a.cache.v : a.cache.k) + (at * D + 16 * unit) * Codes<FMT>::kBytes;
      if constexpr (FMT == NM_KV_FP16) {
        lo = reinterpret_cast<const u32x4*>(in)[0];
        hi = reinterpret_cast<const u32x4*>(in)[1];
      } else {
        const u32x4 c = *reinterpret_cast<const u32x4*>(in);
        const float scale = (is_v ? a.cache.v_scale : a.cache.k_scale)[at];
        float y[2][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float z[4];
          decode4<FMT>(c[i], z);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i >> 1][4 * (i & 1) + j] = z[j] * scale;
        }
        lo = halves_of(y[0]);
        hi = halves_of(y[1]);
      }
    }
  }
  u32x4* out = reinterpret_cast<u32x4*>((is_v ? a.v_out : a.k_out) + int64_t(row) * D + 16 * unit);
  out[0] = lo;
  out[1] = hi;
}

// One workgroup per sequence, head and side (k or v). The rows' places are looked up by a
// thread each; then every row is in registers before any is written: destinations of some rows
// are sources of others. Bound by its chain of dependent loads (path, page table, rows): 3.2
// us for 8 sequences of 8 heads, 12.3 with a wave that moved row after row.
template <int D, int FMT>
__global__ __launch_bounds__(kThreads) void compact_kernel(CompactCall a) {
  constexpr int kChunks = D * Codes<FMT>::kBytes / 16;           // 16-byte pieces of a row
  constexpr int kEach = (kMaxNodes * kChunks + kThreads - 1) / kThreads;
  __shared__ int64_t from[kMaxNodes], into[kMaxNodes];
  const int tid = threadIdx.x;
  const int head = blockIdx.x % a.cache.kv_heads;
  const bool is_v = int(blockIdx.x) >= a.cache.kv_heads;
  const int64_t b = blockIdx.y;
  u32x4* base = reinterpret_cast<u32x4*>(is_v ? a.cache.v : a.cache.k);
  float* scales = is_v ? a.cache.v_scale : a.cache.k_scale;
  float scale = 0.f;
  int64_t scale_into = -1;
  const int accepted = count_of(a.accepted, b, a.nodes - 1);
  if (tid < kMaxNodes) {
    int64_t f = -1, t = -1;
    if (tid < a.nodes) {
      const int node = a.path[b * a.nodes + tid];
      const int64_t start = a.start[b];
      if (tid >= 1 && tid <= accepted && node >= 0 && node < a.nodes && node != tid) {
        f = cache_row(a.cache, b, start + node, head);
        t = cache_row(a.cache, b, start + tid, head);
        if (f < 0) t = -1;
        if (FMT != NM_KV_FP16 && t >= 0) {
          scale = scales[f];
          scale_into = t;
        }
      }
    }
    from[tid] = f;
    into[tid] = t;
  }
  __syncthreads();
  u32x4 held[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int piece = tid + kThreads * j, d = piece / kChunks;
    if (d < kMaxNodes && into[d] >= 0) held[j] = base[from[d] * kChunks + piece % kChunks];
  }
  __builtin_amdgcn_s_waitcnt(0);   // the loads have returned
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int piece = tid + kThreads * j, d = piece / kChunks;
    if (d < kMaxNodes && into[d] >= 0) base[into[d] * kChunks + piece % kChunks] = held[j];
  }
  if (scale_into >= 0) scales[scale_into] = scale;
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
  const int64_t per = kThreads / (head_dim / 16);
  return by_kind<AppendKernel>(c, head_dim, format, dim3(uint32_t((rows + per - 1) / per)), stream, dev);
}

hipError_t launch_read(const ReadCall& c, int head_dim, int format, hipStream_t stream, const DeviceInfo& dev) {
  const int64_t rows = c.batch * c.tokens * c.cache.kv_heads;
  const int64_t per = kThreads / (head_dim / 16);
  return by_kind<ReadKernel>(c, head_dim, format, dim3(uint32_t((rows + per - 1) / per), 2), stream, dev);
}

hipError_t launch_compact(const CompactCall& c, int head_dim, int format, hipStream_t stream, const DeviceInfo& dev) {
  return by_kind<CompactKernel>(c, head_dim, format, dim3(2 * c.cache.kv_heads, uint32_t(c.batch)), stream, dev);
}

}  // namespace nm
