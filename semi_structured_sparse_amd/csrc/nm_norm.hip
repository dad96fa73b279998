// Norms of rows, alone or between two blocks: h = x + scale * gate * post(branch), y = norm(h).
//
// Mathematics. A row stays in the registers of G lanes, 8 neighbouring elements a unit, so that it
// is read once however many sums it takes: one for the root mean square, two for a layer norm (the
// mean, then the squares around it, which keeps the digits that mean(v^2) - mean(v)^2 loses), and as
// many before it for the norm after the branch. Sums are in fp32 in a fixed order.
//
// What bounds it: the bytes of the rows, once in and once out (8191 rows of 8192 in fp32 with a branch,
// 805 MB: 151 us, 5.3 TB/s; 81920 heads of 128: 8.7 us, 4.8); for few rows the trips to memory (8 rows of
// 4096: 3.9 us on the device, little more than an empty launch).
#include "nm_block_internal.h"
#include "nm_epilogue.h"

namespace nm {
namespace {

// Rows start at any element, so the loads and stores of 16 bytes are not aligned to them.
typedef _Float16 halves __attribute__((ext_vector_type(8), aligned(2)));
typedef float floats __attribute__((ext_vector_type(4), aligned(4)));

// Elements i .. i+7 of a row of `width` (zeros past its end).
__device__ __forceinline__ void load_unit(const uint16_t* p, int i, int width, float (&f)[8]) {
  if (i + 8 <= width) {
    const halves v = *reinterpret_cast<const halves*>(p + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = float(v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k < width ? half_at(p, size_t(i + k)) : 0.0f;
  }
}

__device__ __forceinline__ void load_unit(const float* p, int i, int width, float (&f)[8]) {
  if (i + 8 <= width) {
    const floats a = *reinterpret_cast<const floats*>(p + i), b = *reinterpret_cast<const floats*>(p + i + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = a[k];
      f[4 + k] = b[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k < width ? p[i + k] : 0.0f;
  }
}

__device__ __forceinline__ void store_unit(uint16_t* p, int i, int width, const float (&f)[8]) {
  if (i + 8 <= width) {
    halves v;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = static_cast<_Float16>(f[k]);
    *reinterpret_cast<halves*>(p + i) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < width) p[i + k] = to_half(f[k]);
  }
}

__device__ __forceinline__ void store_unit(float* p, int i, int width, const float (&f)[8]) {
  if (i + 8 <= width) {
    *reinterpret_cast<floats*>(p + i) = floats{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<floats*>(p + i + 4) = floats{f[4], f[5], f[6], f[7]};
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < width) p[i + k] = f[k];
  }
}

template <int CTRL>
__device__ __forceinline__ float lane_moved(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

constexpr int kMaxWaves = 16;

// The sum over the G lanes of a row, or (G = 0) over the workgroup's waves, in all of them. room: LDS of
// a float a wave, of this sum alone.
template <int G>
__device__ __forceinline__ float row_sum(float v, float* room) {
  v += lane_moved<0xB1>(v);    // quad_perm: neighbours, then pairs
  v += lane_moved<0x4E>(v);
  v += lane_moved<0x141>(v);   // row_half_mirror: the other quad of 8
  if constexpr (G == 0 || G >= 16) v += lane_moved<0x140>(v);   // row_mirror: the other 8 of 16
  if constexpr (G == 0 || G >= 32) v += __shfl_xor(v, 16);
  if constexpr (G == 0 || G >= 64) v += __shfl_xor(v, 32);
  if constexpr (G == 0) {
    if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
    __syncthreads();
    v = room[0];
    for (int w = 1; w < int(blockDim.x >> 6); ++w) v += room[w];
  }
  return v;
}

// Elements of a row as the norm leaves them without weight and bias: v - mean (layer) times 1 / its
// root mean square.
template <int G, int NU>
__device__ __forceinline__ void normalise(float (&v)[NU][8], int first, int width, int kind, float eps, float* room) {
  const int step = 8 * (G ? G : int(blockDim.x));
  const float each = 1.0f / float(width);
  if (kind == NM_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[j][k];
    const float mean = row_sum<G>(s, room) * each;
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = first + step * j + k < width ? v[j][k] - mean : 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < NU; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(v[j][k], v[j][k], s);
  const float square = row_sum<G>(s, room + kMaxWaves) * each + eps;
  // v_rsq_f32 is good to 1 ulp, but takes a subnormal for 0: a power of 4 brings it to it and back
  const float r = square < 0x1p-100f ? __builtin_amdgcn_rsqf(square * 0x1p100f) * 0x1p50f : __builtin_amdgcn_rsqf(square);
#pragma unroll
  for (int j = 0; j < NU; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] *= r;
}

__device__ __forceinline__ void weigh(float (&v)[8], const uint16_t* weight, float offset, int i, int width) {
  if (weight == nullptr) return;
  float w[8];
  load_unit(weight, i, width, w);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= offset + w[k];
}

// G lanes a row, or the workgroup's (G = 0), and NU units a lane (8 * NU of all of them >= width).
template <int G, int NU, typename Stream, bool BRANCH>
__global__ __launch_bounds__((G ? 256 : 64 * kMaxWaves)) void norm_kernel(NormCall a) {
  __shared__ float room[4 * kMaxWaves];
  const int tid = threadIdx.x, lanes = G ? G : int(blockDim.x), step = 8 * lanes;
  const int64_t row = G ? int64_t(blockIdx.x) * (256 / (G ? G : 1)) + tid / lanes : int64_t(blockIdx.x);
  if (row >= a.rows) return;   // whole rows of lanes; a workgroup that meets at barriers has one row
  const int first = 8 * (G ? tid % lanes : tid), width = a.width;
  int64_t token = row;
  int64_t in_token = 0;
  if (!BRANCH && a.heads > 1) {
    token = int64_t(uint32_t(row) / uint32_t(a.heads));
    in_token = (row - token * a.heads) * width;
  }
  const Stream* x = static_cast<const Stream*>(a.x) + token * a.x_stride + in_token;
  float v[NU][8];
#pragma unroll
  for (int j = 0; j < NU; ++j) load_unit(x, first + step * j, width, v[j]);
  if constexpr (BRANCH) {
    const uint16_t* branch = a.branch + token * a.branch_stride;
    float b[NU][8];
#pragma unroll
    for (int j = 0; j < NU; ++j) load_unit(branch, first + step * j, width, b[j]);
    if (a.post != nullptr) {
      normalise<G, NU>(b, first, width, a.kind, a.eps, room);
#pragma unroll
      for (int j = 0; j < NU; ++j) weigh(b[j], a.post, a.offset, first + step * j, width);
    }
    const uint16_t* gate = a.gate != nullptr ? a.gate + token * a.gate_stride : nullptr;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      weigh(b[j], gate, 0.0f, first + step * j, width);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = fmaf(a.scale, b[j][k], v[j][k]);
    }
    if (a.h != nullptr) {
      Stream* h = static_cast<Stream*>(a.h) + token * a.h_stride;
#pragma unroll
      for (int j = 0; j < NU; ++j) store_unit(h, first + step * j, width, v[j]);
    }
  }
  normalise<G, NU>(v, first, width, a.kind, a.eps, room + 2 * kMaxWaves);
  uint16_t* y = a.y + token * a.y_stride + in_token;
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    const int i = first + step * j;
    weigh(v[j], a.weight, a.offset, i, width);
    if (a.bias != nullptr) {
      float c[8];
      load_unit(a.bias, i, width, c);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] += c[k];
    }
    store_unit(y, i, width, v[j]);
  }
}

struct Shape {
  int lanes, units, threads;   // lanes 0: the workgroup's
};

// Lanes a row and units a lane: as few lanes as hold the row, since idle ones cost as much as others
// (8191 x 4100 with a branch in fp32 101 us with 512 lanes, 90 with 320; heads of 64 3.3 TB/s with 16
// lanes, 5.5 with 8). Several waves share a row from two units a lane on.
Shape shape_of(int width) {
  const int units = (width + 7) / 8;
  for (int lanes = 8; lanes <= 64; lanes *= 2)
    if (units <= lanes) return {lanes, 1, 256};
  if (units <= 128) return {64, 2, 256};
  const int each = units <= 256 ? 1 : units <= 2048 ? 2 : 4;
  return {0, each, 64 * ((units + 64 * each - 1) / (64 * each))};
}

template <typename Stream, bool BRANCH>
const void* kernel_of(const Shape& s) {
  switch (s.lanes) {
    case 8: return reinterpret_cast<const void*>(&norm_kernel<8, 1, Stream, BRANCH>);
    case 16: return reinterpret_cast<const void*>(&norm_kernel<16, 1, Stream, BRANCH>);
    case 32: return reinterpret_cast<const void*>(&norm_kernel<32, 1, Stream, BRANCH>);
    case 64: return s.units == 1 ? reinterpret_cast<const void*>(&norm_kernel<64, 1, Stream, BRANCH>)
                                 : reinterpret_cast<const void*>(&norm_kernel<64, 2, Stream, BRANCH>);
    default: return s.units == 1   ? reinterpret_cast<const void*>(&norm_kernel<0, 1, Stream, BRANCH>)
                    : s.units == 2 ? reinterpret_cast<const void*>(&norm_kernel<0, 2, Stream, BRANCH>)
                                   : reinterpret_cast<const void*>(&norm_kernel<0, 4, Stream, BRANCH>);
  }
}

}  // namespace

hipError_t launch_norm(const NormCall& c, bool fp32_stream, hipStream_t stream, const DeviceInfo& dev) {
  NormCall a = c;
  const Shape s = shape_of(a.width);
  const int each = s.lanes ? s.threads / s.lanes : 1;   // rows a workgroup
  const int64_t grid = (a.rows + each - 1) / each;
  const bool branch = a.branch != nullptr;
  const void* k = fp32_stream ? (branch ? kernel_of<float, true>(s) : kernel_of<float, false>(s))
                              : (branch ? kernel_of<uint16_t, true>(s) : kernel_of<uint16_t, false>(s));
  void* args[] = {&a};
  return launch(k, dim3(unsigned(grid)), dim3(unsigned(s.threads)), args, 0, stream, dev);
}

}  // namespace nm
