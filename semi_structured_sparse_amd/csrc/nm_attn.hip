// Launch of the attention kernel (nm_attn_impl.h): rows per workgroup, the split of the
// contexts over the GPU, and the workspace.
#include <algorithm>

#include "nm_attn_impl.h"

namespace nm {
namespace {

struct Plan {
  int nr;          // row tiles of 16 a workgroup takes
  int row_tiles;   // workgroups of rows
  int slots;       // chunks over all sequences; 0: one a sequence
  uint32_t part_bytes;
  float join;      // what a partial result costs in the join, in tiles
};

struct Kernel {
  const void* f;
  int waves;       // workgroups of a CU
  int lds;
};

template <int FMT, int D, int NR>
Kernel kernel_of() {
  using S = AttnShape<FMT, D, NR>;
  return {reinterpret_cast<const void*>(attention_kernel<FMT, D, NR>), S::kWaves, S::kLdsBytes};
}

// The most row tiles a workgroup takes: what its accumulators leave two waves a SIMD (one for
// heads of 256 elements).
int widest(int head_dim) { return head_dim > 128 ? 2 : head_dim > 64 ? 3 : 4; }

template <int FMT, int D>
Kernel kernel_of(int nr) {
  if constexpr (D <= 64)
    if (nr == 4) return kernel_of<FMT, D, 4>();
  if constexpr (D <= 128)
    if (nr == 3) return kernel_of<FMT, D, 3>();
  return nr == 2 ? kernel_of<FMT, D, 2>() : kernel_of<FMT, D, 1>();
}

template <int FMT>
Kernel kernel_of(int head_dim, int nr) {
  return head_dim == 64 ? kernel_of<FMT, 64>(nr) : head_dim == 128 ? kernel_of<FMT, 128>(nr) : kernel_of<FMT, 256>(nr);
}

Kernel kernel_of(int format, int head_dim, int nr) {
  return format == NM_KV_FP16   ? kernel_of<NM_KV_FP16>(head_dim, nr)
         : format == NM_KV_INT8 ? kernel_of<NM_KV_INT8>(head_dim, nr)
                                : kernel_of<NM_KV_E4M3>(head_dim, nr);
}

Plan plan_of(const AttnCall& c, int head_dim, int format, const DeviceInfo& dev) {
  Plan p;
  const int rows = c.tokens * c.group;
  // row tiles evenly over the fewest workgroups
  const int tiles = (rows + 15) / 16, most_tiles = widest(head_dim);
  p.row_tiles = (tiles + most_tiles - 1) / most_tiles;
  p.nr = (tiles + p.row_tiles - 1) / p.row_tiles;
  p.part_bytes = uint32_t(head_dim / 16 * p.nr * 1024 + p.nr * 128);
  const int live = std::min(rows, 16 * p.nr), code_bytes = format == NM_KV_FP16 ? 2 : 1;
  p.join = 2.0f * float(live * 4) / float(2 * kTileKeys * code_bytes);   // twice its bytes over a tile's
  const int64_t items = int64_t(c.batch) * c.cache.kv_heads * p.row_tiles;
  const int64_t most = int64_t(c.cache.table_width) << c.cache.page_shift;
  // Slots for as many workgroups as the GPU holds at once (once more for every two thirds of
  // them that the sequences themselves take), none for less than a round of the waves.
  const int64_t room = int64_t(dev.cu_count) * kernel_of(format, head_dim, p.nr).waves / (int64_t(c.cache.kv_heads) * p.row_tiles);
  const int64_t rounds = room > 0 ? (3 * int64_t(c.batch) + 2 * room - 1) / (2 * room) : 0;
  const int64_t shortest = kTileKeys * kMinChunkTiles;
  const int64_t slots = std::min(rounds * room, c.batch * ((most + shortest - 1) / shortest));
  p.slots = items > NM_DECODE_COUNTER_BYTES / 4 || slots <= c.batch ? 0 : int(slots);
  return p;
}

// A slot's partial results.
size_t slot_bytes(const AttnCall& c, const Plan& p) {
  return size_t(unsigned(c.cache.kv_heads)) * unsigned(p.row_tiles) * p.part_bytes;
}

size_t plan_bytes(const AttnCall& c, const Plan& p) {
  return p.slots == 0 ? 0 : NM_DECODE_COUNTER_BYTES + p.slots * slot_bytes(c, p);
}

}  // namespace

// The most that a step of as many nodes or fewer takes: fewer nodes may make for smaller row tiles,
// or fewer of them, and more slots (64 / 8 heads of 128 over 16384 tokens: 8 nodes 8.6 MB, 5 or 6
// 12.8).
size_t attention_workspace_bytes(const AttnCall& c, int head_dim, int format, const DeviceInfo& dev) {
  size_t most = 0;
  AttnCall a = c;
  for (a.tokens = 1; a.tokens <= c.tokens; ++a.tokens) most = std::max(most, plan_bytes(a, plan_of(a, head_dim, format, dev)));
  return most;
}

hipError_t launch_attention(const AttnCall& c, int head_dim, int format, void* workspace, size_t workspace_bytes,
                            hipStream_t stream, const DeviceInfo& dev) {
  AttnCall a = c;
  Plan p = plan_of(c, head_dim, format, dev);
  // fewer slots where the workspace holds no more; one a sequence needs none
  const size_t room = workspace == nullptr || workspace_bytes < NM_DECODE_COUNTER_BYTES
                          ? 0 : (workspace_bytes - NM_DECODE_COUNTER_BYTES) / slot_bytes(c, p);
  if (size_t(p.slots) > room) p.slots = room > size_t(c.batch) ? int(room) : 0;
  AttnSplit sp{p.slots, p.row_tiles, static_cast<uint32_t*>(workspace),
               p.slots ? static_cast<char*>(workspace) + NM_DECODE_COUNTER_BYTES : nullptr, p.part_bytes, p.join};
  void* args[] = {&a, &sp};
  // Row tiles of one chunk read the same keys: a grid width that is a multiple of the 8 XCDs
  // puts them on one XCD's L2.
  const int64_t wide = (int64_t(p.slots ? p.slots : c.batch) * c.cache.kv_heads + 7) / 8 * 8;
  const Kernel k = kernel_of(format, head_dim, p.nr);
  return launch(k.f, dim3(uint32_t(wide), uint32_t(p.row_tiles)), dim3(kAttnThreads), args, size_t(k.lds), stream, dev);
}

}  // namespace nm
