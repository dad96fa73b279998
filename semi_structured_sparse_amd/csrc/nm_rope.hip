// Rotary positions (nm_rope) and the host table of their frequencies (nm_rope_turns).
//
// Mathematics: each pair of a head's rotated elements is turned by 2 pi pos turns_i. The product
// and its fraction of a turn are worked out in 64 bits, the cosine and sine of that fraction and
// the turn in fp32, rounded once (rotation() in nm_decode_internal.h). What bounds it: the copy, 4
// bytes an element; the angles are the costly part, five operations in 64 bits and some 25 in 32
// each.
#include <algorithm>
#include <cmath>

#include "nm_decode_internal.h"

namespace nm {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kGridThreads = int64_t(1) << 31;

// Any head size, stride and alignment: one pair (or, past the rotated part, two elements) per
// thread, which works out its angle: 184 us for the 8191 tokens of 72 heads below.
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeCall a) {
  const int units = (a.head_dim + 1) / 2, pairs = a.rope.rot_dim / 2;
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.tokens * a.heads * units) return;
  const int u = int(i % units);
  const int64_t head = i / units % a.heads, token = i / units / a.heads;
  const uint16_t* x = a.x + token * a.x_stride + head * a.head_dim;
  uint16_t* y = a.y + token * a.y_stride + head * a.head_dim;
  if (u >= pairs) {
    const int e = 2 * u;
    y[e] = x[e];
    if (e + 1 < a.head_dim) y[e + 1] = x[e + 1];
    return;
  }
  const bool half = a.rope.layout == NM_ROPE_HALF;
  const int e0 = half ? u : 2 * u, e1 = half ? u + pairs : 2 * u + 1;
  float c, s;
  rotation(a.rope.positions[token], a.rope.turns[u], a.rope.scale, c, s);
  const float p = half_bits_to_float(x[e0]), q = half_bits_to_float(x[e1]);
  y[e0] = uint16_t(float_to_half_bits(p * c - q * s));
  y[e1] = uint16_t(float_to_half_bits(q * c + p * s));
}

// Heads of whole 16-element units with 16-byte alignment. A thread keeps one unit's cosines and
// sines and turns that unit of every `step`-th head of its token, so that they are worked out
// once for several heads; what is left is a copy, two 16-byte loads and stores a unit. 8191
// tokens x 72 heads x 128 elements (302 MB read and written): 55.0 us, 5.5 TB/s, where a large
// copy reaches 4.8; 8 tokens x 40 heads 3.1 us, where an empty launch takes 2.6. Loads that bypass
// the caches made the large one 4 us longer, such stores too 11.
__global__ __launch_bounds__(kThreads) void rope_wide_kernel(RopeCall a, int units, int step, int each) {
  const int unit = threadIdx.x % units, h0 = blockIdx.y * each + threadIdx.x / units;
  const int64_t token = blockIdx.x;
  if (int(threadIdx.x) >= units * step) return;
  const int end = min(a.heads, (int(blockIdx.y) + 1) * each);
  const HeadUnit hu = head_unit(unit, a.rope.rot_dim, a.head_dim);
  const uint16_t* x = a.x + token * a.x_stride;
  uint16_t* y = a.y + token * a.y_stride;
  UnitRotation t;
  if (hu.turned) t = unit_rotation(a.rope, unit, a.rope.positions[token]);
#pragma unroll 2
  for (int h = h0; h < end; h += step) {
    const int64_t at = int64_t(h) * a.head_dim;
    u32x4 p = *reinterpret_cast<const u32x4*>(x + at + hu.first), q = *reinterpret_cast<const u32x4*>(x + at + hu.second);
    if (hu.turned) {
      float e[8], f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = half_at(p, i);
        f[i] = half_at(q, i);
      }
      turn_unit(t, a.rope.layout, e, f);
      p = halves_of(e);
      q = halves_of(f);
    }
    *reinterpret_cast<u32x4*>(y + at + hu.first) = p;
    *reinterpret_cast<u32x4*>(y + at + hu.second) = q;
  }
}

// Launches `most` tokens at a time: a grid has fewer than 2^32 threads across.
template <class F>
hipError_t by_tokens(RopeCall& a, int64_t most, F&& launch_some) {
  const RopeCall all = a;
  for (int64_t t = 0; t < all.tokens; t += most) {
    a.tokens = std::min(most, all.tokens - t);
    a.x = all.x + t * all.x_stride;
    a.y = all.y + t * all.y_stride;
    a.rope.positions = all.rope.positions + t;
    const hipError_t e = launch_some();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

hipError_t launch_rope(const RopeCall& c, hipStream_t stream, const DeviceInfo& dev) {
  RopeCall a = c;
  if (aligned16(c.x) && aligned16(c.y) && c.x_stride % 8 == 0 && c.y_stride % 8 == 0 && c.head_dim % 16 == 0 &&
      c.rope.rot_dim % 16 == 0) {
    int units = c.head_dim / 16, step = kThreads / units;
    // one head a thread where that is needed to fill the GPU, else up to kPasses
    constexpr int kPasses = 4;
    const int passes = (c.heads + step - 1) / step;
    const int64_t room = 8 * int64_t(dev.cu_count);
    int split = passes;
    if (c.tokens * passes > room) split = int((room + c.tokens - 1) / c.tokens);
    if (split < (passes + kPasses - 1) / kPasses) split = (passes + kPasses - 1) / kPasses;
    int each = (passes + split - 1) / split * step;
    void* args[] = {&a, &units, &step, &each};
    return by_tokens(a, kGridThreads / kThreads, [&] {
      return launch(reinterpret_cast<const void*>(rope_wide_kernel),
                    dim3(uint32_t(a.tokens), (c.heads + each - 1) / each), dim3(kThreads), args, 0, stream, dev);
    });
  }
  const int64_t per_token = c.heads * int64_t((c.head_dim + 1) / 2);
  void* args[] = {&a};
  return by_tokens(a, kGridThreads / per_token, [&] {
    return launch(reinterpret_cast<const void*>(rope_kernel), dim3(uint32_t((a.tokens * per_token + kThreads - 1) / kThreads)),
                  dim3(kThreads), args, 0, stream, dev);
  });
}

}  // namespace nm

int nm_rope_turns(double* turns, int rot_dim, int scaling, double base, double factor, double length, double low,
                  double high) {
  if (!turns) return NM_ERR_NULL;
  if (scaling < NM_ROPE_PLAIN || scaling > NM_ROPE_BANDS) return NM_ERR_FORMAT;
  const auto positive = [](double v) { return std::isfinite(v) && v > 0.0; };
  if (rot_dim < (scaling == NM_ROPE_BASE ? 4 : 2) || rot_dim > 1024 || rot_dim % 2 != 0) return NM_ERR_SHAPE;
  if (!positive(base) || (scaling != NM_ROPE_PLAIN && !positive(factor))) return NM_ERR_SHAPE;
  if (scaling == NM_ROPE_BANDS && !(positive(length) && std::isfinite(low) && low >= 0.0 && positive(high) && high > low))
    return NM_ERR_SHAPE;
  if (scaling == NM_ROPE_BASE) base *= std::pow(factor, double(rot_dim) / double(rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double t = std::pow(base, -2.0 * i / rot_dim) / (2.0 * 3.14159265358979323846);
    if (scaling == NM_ROPE_LINEAR) t /= factor;
    if (scaling == NM_ROPE_BANDS) {
      double w = (length * t - low) / (high - low);
      w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
      t = t * w + t / factor * (1.0 - w);
    }
    turns[i] = t;
  }
  return NM_OK;
}
