// Declarations shared by the translation units of the speculative-decoding operators: the
// checked arguments their kernels take, and the device helpers of the paged cache and the
// rotary positions. Not part of the public ABI (include/nm_decode.h is).
#pragma once

#include <hip/hip_fp16.h>

#include "nm_decode.h"
#include "nm_internal.h"

namespace nm {

constexpr int kMaxNodes = 64;   // nodes of one sequence's step (a mask word's bits)

// A paged cache and the page table of the sequences that a call works on.
struct PagedCache {
  char* k;
  char* v;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  int table_width;
  uint32_t blocks;
  int kv_heads;
  int page_shift;
};

struct RopeArgs {
  const int32_t* positions;
  const double* turns;
  int rot_dim;
  int layout;
  float scale;
};

struct RopeCall {
  const uint16_t* x;
  uint16_t* y;
  int64_t x_stride, y_stride;
  int64_t tokens;
  int heads, head_dim;
  RopeArgs rope;
};

struct AppendCall {
  PagedCache cache;
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_stride, q_out_stride, k_stride, v_stride;
  const int32_t *start, *count;
  int64_t batch, tokens;
  int q_heads;
  RopeArgs rope;   // positions NULL: no rotation
};

struct ReadCall {
  PagedCache cache;
  uint16_t *k_out, *v_out;
  const int32_t *start, *count;
  int64_t batch, tokens;
};

struct CompactCall {
  PagedCache cache;
  const int32_t *start, *path, *accepted;
  int64_t batch;
  int nodes;
};

struct AttnCall {
  PagedCache cache;
  const uint16_t* q;
  uint16_t* out;
  const int32_t *context, *count;
  const uint64_t* mask;
  int64_t q_stride;
  int batch, tokens, heads, group;
  float scale;
};

struct VerifyCall {
  const float *target, *draft, *uniforms;
  const int32_t *tokens, *parents, *count;
  int32_t *accepted, *out_tokens, *path;
  int batch, nodes, vocab;
};

hipError_t launch_rope(const RopeCall& c, hipStream_t stream, const DeviceInfo& dev);
hipError_t launch_append(const AppendCall& c, int head_dim, int format, hipStream_t stream, const DeviceInfo& dev);
hipError_t launch_read(const ReadCall& c, int head_dim, int format, hipStream_t stream, const DeviceInfo& dev);
hipError_t launch_compact(const CompactCall& c, int head_dim, int format, hipStream_t stream, const DeviceInfo& dev);
hipError_t launch_attention(const AttnCall& c, int head_dim, int format, void* workspace, size_t workspace_bytes,
                            hipStream_t stream, const DeviceInfo& dev);
size_t attention_workspace_bytes(const AttnCall& c, int head_dim, int format, const DeviceInfo& dev);
hipError_t launch_verify(const VerifyCall& c, void* workspace, size_t workspace_bytes, hipStream_t stream,
                         const DeviceInfo& dev);
size_t verify_workspace_bytes(int64_t batch, int64_t vocab, const DeviceInfo& dev);

// ------------------------------------------------------------------------ device helpers
// The cache row (token slot of one head) of position pos of sequence b, or -1 where the
// position or its table entry is out of range.
__device__ __forceinline__ int64_t cache_row(const PagedCache& c, int64_t b, int64_t pos, int head) {
  if (pos < 0 || (pos >> c.page_shift) >= c.table_width) return -1;
  const uint32_t block = uint32_t(c.table[b * c.table_width + (pos >> c.page_shift)]);
  if (block >= c.blocks) return -1;
  return (((int64_t(block) * c.kv_heads + head) << c.page_shift) + (pos & ((1 << c.page_shift) - 1)));
}

// count[b] clamped to 0 .. most (NULL: most).
__device__ __forceinline__ int count_of(const int32_t* count, int64_t b, int most) {
  if (count == nullptr) return most;
  const int n = count[b];
  return n < 0 ? 0 : n > most ? most : n;
}

__device__ __forceinline__ float half_bits_to_float(uint32_t bits) {
  return float(__builtin_bit_cast(_Float16, uint16_t(bits)));
}

__device__ __forceinline__ uint32_t float_to_half_bits(float x) {   // round to nearest even
  return __builtin_bit_cast(uint16_t, _Float16(x));
}

// Partial results cross workgroups on different XCDs, whose L2 caches are not coherent with
// each other: accesses with the SC1 cache-policy bit are, without a fence that writes back or
// invalidates a whole L2. `bytes` bounds the resource: accesses past it read zero or are dropped.
constexpr int kCoherent = 16;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t coherent_buffer(void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(p, 0, bytes, 0x00027000);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float half_at(u32x4 v, int i) {   // element i of 8 halves
  return half_bits_to_float((v[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
}

__device__ __forceinline__ u32x4 halves_of(const float (&e)[8]) {   // each to nearest even
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = float_to_half_bits(e[2 * i]) | float_to_half_bits(e[2 * i + 1]) << 16;
  return v;
}

// Cosine and sine of 2 pi * pos * turns, times scale. The product keeps its fraction in 64 bits
// (at a position of 10^6 and one turn in 6 a product in 32 would leave it off by 2^-7 of a turn).
// From it comes, exactly, the nearest quarter, whose number stands in the low bits of a sum with
// 1.5 2^52, and the rest, an eighth of a turn at most. The rest's Taylor series, whose last terms
// are 2^-25 of the result, give both to about 2^-24; the quarter swaps them and sets their signs.
// (The instructions for a turn's sine and cosine take an fp32 fraction of a whole turn, off by
// 2^-23 as an angle: of results that nearly cancel 31% were not the fp16 nearest to the exact one,
// 10% now, 12% in fp32 with rounded products. What that costs: the prompt of nm_rope.hip, whose
// heads share the angles, 54.5 us then and 55.2 now; 4 x 4096 tokens of 32 / 8 heads turned,
// appended and read back, where they do not, 99 and 108.)
__device__ __forceinline__ void rotation(int pos, double turns, float scale, float& c, float& s) {
  constexpr double w = 2.0 * 3.14159265358979323846, w2 = w * w;
  constexpr double s3 = -w * w2 / 6, s5 = -s3 * w2 / 20, s7 = -s5 * w2 / 42, s9 = -s7 * w2 / 72;
  constexpr double c2 = -w2 / 2, c4 = -c2 * w2 / 12, c6 = -c4 * w2 / 30, c8 = -c6 * w2 / 56, c10 = -c8 * w2 / 90;
  constexpr double whole = 0x1.8p52;
  const double f = __builtin_amdgcn_fract(double(pos) * turns);
  const double quarters = fma(4.0, f, whole);
  const float r = float(fma(-0.25, quarters - whole, f)), z = r * r;
  float p = fmaf(z, float(s9), float(s7));
  p = fmaf(z, p, float(s5));
  p = fmaf(z, p, float(s3));
  p = fmaf(z, p, float(w - double(float(w))));   // what fp32 leaves of 2 pi
  const float sine = fmaf(r, float(w), r * p);
  float g = fmaf(z, float(c10), float(c8));
  g = fmaf(z, g, float(c6));
  g = fmaf(z, g, float(c4));
  g = fmaf(z, g, float(c2));
  const float cosine = fmaf(z, g, 1.0f);
  const uint32_t q = uint32_t(__double_as_longlong(quarters));
  c = __uint_as_float(__float_as_uint(q & 1 ? sine : cosine) ^ ((q + 1) << 30 & 0x80000000u)) * scale;
  s = __uint_as_float(__float_as_uint(q & 1 ? cosine : sine) ^ (q << 30 & 0x80000000u)) * scale;
}

// A unit of a head: 16 elements, as two runs of 8 that lie half of the rotated part, or half of
// the rest, apart. So the pairs of NM_ROPE_HALF are the runs' elements (those of the other layout
// are neighbours in a run), and neighbouring threads' loads and stores are neighbours in memory:
// with runs that lie together 8191 tokens of 72 heads took 2.3 us longer, of 55.
struct HeadUnit {
  int first, second;   // where the runs start
  bool turned;
};

__device__ __forceinline__ HeadUnit head_unit(int unit, int rot_dim, int head_dim) {
  HeadUnit u;
  u.turned = 16 * unit < rot_dim;
  u.first = 8 * unit + (u.turned ? 0 : rot_dim / 2);
  u.second = u.first + (u.turned ? rot_dim : head_dim - rot_dim) / 2;
  return u;
}

struct UnitRotation {
  float c[8], s[8];
};

__device__ __forceinline__ UnitRotation unit_rotation(const RopeArgs& r, int unit, int pos) {
  UnitRotation t;
  // the pairs of the two runs: the same 8, or 4 of each
  const double* first = r.turns + (r.layout == NM_ROPE_HALF ? 8 : 4) * unit;
  const double* second = first + (r.layout == NM_ROPE_HALF ? 4 : r.rot_dim / 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    rotation(pos, first[i], r.scale, t.c[i], t.s[i]);
    rotation(pos, second[i], r.scale, t.c[4 + i], t.s[4 + i]);
  }
  return t;
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a * c - b * s;
  b = b * c + a * s;
  a = x;
}

__device__ __forceinline__ void turn_unit(const UnitRotation& t, int layout, float (&a)[8], float (&b)[8]) {
  if (layout == NM_ROPE_HALF) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(a[i], b[i], t.c[i], t.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn(a[2 * i], a[2 * i + 1], t.c[i], t.s[i]);
      turn(b[2 * i], b[2 * i + 1], t.c[4 + i], t.s[4 + i]);
    }
  }
}

}  // namespace nm
