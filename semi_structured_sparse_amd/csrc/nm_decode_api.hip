// C ABI of the speculative-decoding operators: argument checks (no HIP call before they
// pass) and dispatch to the kernels.
#include <cmath>

#include "nm_decode_internal.h"
#include "nm_sparse.h"

namespace nm {
namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;
// Elements of a cache call, 16 a thread: a grid has fewer than 2^32 threads across.
constexpr int64_t kMaxElements = int64_t(1) << 35;
constexpr int64_t kMaxAttnHeads = int64_t(1) << 23;   // key heads of an attention call's sequences, likewise

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool within(int64_t v, int64_t low, int64_t high) { return v >= low && v <= high; }

// A token stride that holds `row` elements and keeps 16-byte loads aligned.
bool stride_ok(int64_t stride, int64_t row) { return within(stride, row, kMaxStride); }

int finish(hipError_t e) {
  if (e == hipSuccess) return NM_OK;
  set_last_hip_error(e);
  return NM_ERR_HIP;
}

int cache_check(const nm_kv_cache* c, const int32_t* table, int64_t table_width, int64_t batch, int64_t tokens) {
  if (!c || !c->k || !c->v || !table) return NM_ERR_NULL;
  if (!within(c->format, NM_KV_FP16, NM_KV_E4M3)) return NM_ERR_FORMAT;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NM_ERR_FORMAT;
  if (!within(c->page, 16, 1024) || (c->page & (c->page - 1)) != 0) return NM_ERR_FORMAT;
  if (c->format != NM_KV_FP16 && (!c->k_scale || !c->v_scale)) return NM_ERR_NULL;
  if (!within(c->blocks, 1, 0x7FFFFFFF) || !within(c->kv_heads, 1, 4096)) return NM_ERR_SHAPE;
  if (!within(table_width, 1, int64_t(1) << 24) || table_width * c->page > (int64_t(1) << 30)) return NM_ERR_SHAPE;
  if (!within(batch, 1, 65535) || !within(tokens, 1, int64_t(1) << 24) || batch * tokens > (int64_t(1) << 30))
    return NM_ERR_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(table, 4)) return NM_ERR_ALIGN;
  if (c->format != NM_KV_FP16 && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))) return NM_ERR_ALIGN;
  return NM_OK;
}

PagedCache paged(const nm_kv_cache* c, const int32_t* table, int64_t table_width) {
  PagedCache p;
  p.k = static_cast<char*>(c->k);
  p.v = static_cast<char*>(c->v);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.table = table;
  p.table_width = int(table_width);
  p.blocks = uint32_t(c->blocks);
  p.kv_heads = c->kv_heads;
  p.page_shift = __builtin_ctz(unsigned(c->page));
  return p;
}

int rope_check(int head_dim, int rot_dim, int layout, const int32_t* positions, const double* turns) {
  if (layout != NM_ROPE_HALF && layout != NM_ROPE_INTERLEAVED) return NM_ERR_FORMAT;
  if (!within(rot_dim, 2, head_dim) || rot_dim % 2 != 0) return NM_ERR_SHAPE;
  if (!aligned(positions, 4) || !aligned(turns, 8)) return NM_ERR_ALIGN;
  return NM_OK;
}

// nm_kv_append with (rope.positions set) or without the rotation of q and k.
int append(const nm_kv_cache* cache, const uint16_t* q, uint16_t* q_out, int64_t q_heads, int64_t q_stride,
           int64_t q_out_stride, const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
           const RopeArgs& rope, const int32_t* table, int64_t table_width, const int32_t* start,
           const int32_t* count, int64_t batch, int64_t tokens, void* stream) {
  if (!k || !v || !start) return NM_ERR_NULL;
  int st = cache_check(cache, table, table_width, batch, tokens);
  if (st != NM_OK) return st;
  const int64_t row = int64_t(cache->kv_heads) * cache->head_dim;
  if (!stride_ok(k_stride, row) || !stride_ok(v_stride, row)) return NM_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 != 0 || v_stride % 8 != 0) return NM_ERR_ALIGN;
  if (!aligned(start, 4) || !aligned(count, 4)) return NM_ERR_ALIGN;
  if (batch * tokens * (q_heads + 2 * cache->kv_heads) > kMaxElements / cache->head_dim) return NM_ERR_SHAPE;
  if (q_heads > 0) {
    if (!q || !q_out) return NM_ERR_NULL;
    if (!stride_ok(q_stride, q_heads * cache->head_dim) || !stride_ok(q_out_stride, q_heads * cache->head_dim))
      return NM_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(q_out, 16) || q_stride % 8 != 0 || q_out_stride % 8 != 0) return NM_ERR_ALIGN;
  }
  DeviceInfo dev;
  const hipError_t e = current_device_info(&dev);
  if (e != hipSuccess) return finish(e);
  AppendCall c{paged(cache, table, table_width), q, k, v, q_out, q_stride, q_out_stride, k_stride, v_stride, start,
               count, batch, tokens, int(q_heads), rope};
  return finish(launch_append(c, cache->head_dim, cache->format, static_cast<hipStream_t>(stream), dev));
}

int attention_check(const nm_kv_cache* cache, int64_t heads, const int32_t* table, int64_t table_width, int64_t batch,
                    int64_t tokens) {
  const int st = cache_check(cache, table, table_width, batch, tokens);
  if (st != NM_OK) return st;
  if (tokens > kMaxNodes || !within(heads, 1, 65536) || heads % cache->kv_heads != 0 || heads / cache->kv_heads > 16 ||
      batch * cache->kv_heads > kMaxAttnHeads)
    return NM_ERR_SHAPE;
  return NM_OK;
}

AttnCall attention_call(const nm_kv_cache* cache, int64_t heads, const int32_t* table, int64_t table_width,
                        int64_t batch, int64_t tokens) {
  AttnCall c{};
  c.cache = paged(cache, table, table_width);
  c.batch = int(batch);
  c.tokens = int(tokens);
  c.heads = int(heads);
  c.group = int(heads) / cache->kv_heads;
  return c;
}

int verify(const VerifyCall& given, int64_t batch, int64_t nodes, int64_t vocab, void* workspace,
           size_t workspace_bytes, void* stream) {
  VerifyCall c = given;
  if (!c.target || !c.tokens || !c.uniforms || !c.accepted || !c.out_tokens) return NM_ERR_NULL;
  if (!within(batch, 1, 65535) || !within(nodes, 1, kMaxNodes) || !within(vocab, 1, int64_t(1) << 24))
    return NM_ERR_SHAPE;
  for (const void* p : {static_cast<const void*>(c.target), static_cast<const void*>(c.draft),
                        static_cast<const void*>(c.uniforms), static_cast<const void*>(c.tokens),
                        static_cast<const void*>(c.parents), static_cast<const void*>(c.count),
                        static_cast<const void*>(c.accepted), static_cast<const void*>(c.out_tokens),
                        static_cast<const void*>(c.path)})
    if (!aligned(p, 4)) return NM_ERR_ALIGN;
  if (!aligned(workspace, 16)) return NM_ERR_ALIGN;
  c.batch = int(batch);
  c.nodes = int(nodes);
  c.vocab = int(vocab);
  DeviceInfo dev;
  const hipError_t e = current_device_info(&dev);
  if (e != hipSuccess) return finish(e);
  return finish(launch_verify(c, workspace, workspace_bytes, static_cast<hipStream_t>(stream), dev));
}

}  // namespace
}  // namespace nm

using namespace nm;

int nm_rope(const uint16_t* x, uint16_t* y, const int32_t* positions, const double* turns, int64_t tokens,
            int64_t heads, int head_dim, int rot_dim, int layout, float scale, int64_t x_stride, int64_t y_stride,
            void* stream) {
  if (!x || !y || !positions || !turns) return NM_ERR_NULL;
  if (!within(tokens, 1, int64_t(1) << 30) || !within(heads, 1, 65536) || !within(head_dim, 2, 1024))
    return NM_ERR_SHAPE;
  const int st = rope_check(head_dim, rot_dim, layout, positions, turns);
  if (st != NM_OK) return st;
  if (!stride_ok(x_stride, heads * head_dim) || !stride_ok(y_stride, heads * head_dim)) return NM_ERR_SHAPE;
  if (!aligned(x, 2) || !aligned(y, 2)) return NM_ERR_ALIGN;
  DeviceInfo dev;
  const hipError_t e = current_device_info(&dev);
  if (e != hipSuccess) return finish(e);
  RopeCall c{x, y, x_stride, y_stride, tokens, int(heads), head_dim, {positions, turns, rot_dim, layout, scale}};
  return finish(launch_rope(c, static_cast<hipStream_t>(stream), dev));
}

int nm_kv_append(const nm_kv_cache* cache, const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                 const int32_t* table, int64_t table_width, const int32_t* start, const int32_t* count, int64_t batch,
                 int64_t tokens, void* stream) {
  return append(cache, nullptr, nullptr, 0, 0, 0, k, v, k_stride, v_stride, RopeArgs{}, table, table_width, start,
                count, batch, tokens, stream);
}

int nm_rope_kv_append(const nm_kv_cache* cache, const uint16_t* q, uint16_t* q_out, int64_t q_heads, int64_t q_stride,
                      int64_t q_out_stride, const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                      const int32_t* positions, const double* turns, int rot_dim, int layout, float scale,
                      const int32_t* table, int64_t table_width, const int32_t* start, const int32_t* count,
                      int64_t batch, int64_t tokens, void* stream) {
  if (!positions || !turns) return NM_ERR_NULL;
  int st = cache_check(cache, table, table_width, batch, tokens);
  if (st != NM_OK) return st;
  if (!within(q_heads, 0, 65536)) return NM_ERR_SHAPE;
  st = rope_check(cache->head_dim, rot_dim, layout, positions, turns);
  if (st != NM_OK) return st;
  if (rot_dim % 16 != 0) return NM_ERR_SHAPE;
  return append(cache, q, q_out, q_heads, q_stride, q_out_stride, k, v, k_stride, v_stride,
                RopeArgs{positions, turns, rot_dim, layout, scale}, table, table_width, start, count, batch, tokens,
                stream);
}

int nm_kv_read(const nm_kv_cache* cache, uint16_t* k_out, uint16_t* v_out, const int32_t* table, int64_t table_width,
               const int32_t* start, const int32_t* count, int64_t batch, int64_t tokens, void* stream) {
  if (!k_out || !v_out || !start) return NM_ERR_NULL;
  const int st = cache_check(cache, table, table_width, batch, tokens);
  if (st != NM_OK) return st;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(start, 4) || !aligned(count, 4)) return NM_ERR_ALIGN;
  if (batch * tokens * cache->kv_heads > kMaxElements / cache->head_dim) return NM_ERR_SHAPE;
  DeviceInfo dev;
  const hipError_t e = current_device_info(&dev);
  if (e != hipSuccess) return finish(e);
  ReadCall c{paged(cache, table, table_width), k_out, v_out, start, count, batch, tokens};
  return finish(launch_read(c, cache->head_dim, cache->format, static_cast<hipStream_t>(stream), dev));
}

int nm_kv_compact(const nm_kv_cache* cache, const int32_t* table, int64_t table_width, const int32_t* start,
                  const int32_t* path, const int32_t* accepted, int64_t batch, int64_t nodes, void* stream) {
  if (!start || !path || !accepted) return NM_ERR_NULL;
  const int st = cache_check(cache, table, table_width, batch, nodes);
  if (st != NM_OK) return st;
  if (nodes > kMaxNodes) return NM_ERR_SHAPE;
  if (!aligned(start, 4) || !aligned(path, 4) || !aligned(accepted, 4)) return NM_ERR_ALIGN;
  DeviceInfo dev;
  const hipError_t e = current_device_info(&dev);
  if (e != hipSuccess) return finish(e);
  CompactCall c{paged(cache, table, table_width), start, path, accepted, batch, int(nodes)};
  return finish(launch_compact(c, cache->head_dim, cache->format, static_cast<hipStream_t>(stream), dev));
}

int nm_tree_attention(const nm_kv_cache* cache, const uint16_t* q, uint16_t* out, int64_t heads, int64_t q_stride,
                      const int32_t* table, int64_t table_width, const int32_t* context, const uint64_t* mask,
                      const int32_t* count, int64_t batch, int64_t tokens, float scale, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!q || !out || !context) return NM_ERR_NULL;
  const int st = attention_check(cache, heads, table, table_width, batch, tokens);
  if (st != NM_OK) return st;
  if (!stride_ok(q_stride, heads * cache->head_dim) || !std::isfinite(scale)) return NM_ERR_SHAPE;
  if (!aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 16) || !aligned(context, 4) || !aligned(count, 4) ||
      !aligned(mask, 8) || !aligned(workspace, 16))
    return NM_ERR_ALIGN;
  DeviceInfo dev;
  const hipError_t e = current_device_info(&dev);
  if (e != hipSuccess) return finish(e);
  AttnCall c = attention_call(cache, heads, table, table_width, batch, tokens);
  c.q = q;
  c.out = out;
  c.context = context;
  c.count = count;
  c.mask = mask;
  c.q_stride = q_stride;
  c.scale = scale;
  return finish(launch_attention(c, cache->head_dim, cache->format, workspace, workspace_bytes,
                                 static_cast<hipStream_t>(stream), dev));
}

size_t nm_tree_attention_workspace_bytes(const nm_kv_cache* cache, int64_t heads, int64_t table_width, int64_t batch,
                                         int64_t tokens) {
  static const int32_t no_table = 0;   // only its presence is checked
  if (attention_check(cache, heads, &no_table, table_width, batch, tokens) != NM_OK) return 0;
  DeviceInfo dev;
  if (current_device_info(&dev) != hipSuccess) return 0;
  return attention_workspace_bytes(attention_call(cache, heads, nullptr, table_width, batch, tokens), cache->head_dim,
                                   cache->format, dev);
}

int nm_verify_chain(const float* target, const float* draft, const int32_t* tokens, const float* uniforms,
                    const int32_t* count, int32_t* accepted, int32_t* out_tokens, int64_t batch, int64_t nodes,
                    int64_t vocab, void* workspace, size_t workspace_bytes, void* stream) {
  if (!draft && nodes > 1) return NM_ERR_NULL;
  VerifyCall c{};
  c.target = target;
  c.draft = draft;
  c.tokens = tokens;
  c.uniforms = uniforms;
  c.count = count;
  c.accepted = accepted;
  c.out_tokens = out_tokens;
  return verify(c, batch, nodes, vocab, workspace, workspace_bytes, stream);
}

int nm_verify_tree(const float* target, const int32_t* tokens, const int32_t* parents, const float* uniforms,
                   const int32_t* count, int32_t* accepted, int32_t* out_tokens, int32_t* path, int64_t batch,
                   int64_t nodes, int64_t vocab, void* workspace, size_t workspace_bytes, void* stream) {
  if (!parents || !path) return NM_ERR_NULL;
  VerifyCall c{};
  c.target = target;
  c.tokens = tokens;
  c.parents = parents;
  c.uniforms = uniforms;
  c.count = count;
  c.accepted = accepted;
  c.out_tokens = out_tokens;
  c.path = path;
  return verify(c, batch, nodes, vocab, workspace, workspace_bytes, stream);
}

size_t nm_verify_workspace_bytes(int64_t batch, int64_t vocab) {
  if (!within(batch, 1, 65535) || !within(vocab, 1, int64_t(1) << 24)) return 0;
  DeviceInfo dev;
  if (current_device_info(&dev) != hipSuccess) return 0;
  return verify_workspace_bytes(batch, vocab, dev);
}
