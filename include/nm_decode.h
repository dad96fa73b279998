/*
 * nm_decode.h -- C ABI of libnmsparse.so for what stands between the sparse products of a
 * speculative decoding step on AMD Instinct MI355X (gfx950): rotary positions, a paged
 * key/value cache, the attention of the drafted tokens over it, and the verification of the
 * drafts against the target's probabilities.
 *
 * A step: the products (nm_sparse.h) of the last accepted token and the drafted ones give q,
 * k and v; nm_rope_kv_append turns q and k and writes k and v into the cache;
 * nm_tree_attention reads it; after the last layer nm_verify_chain or nm_verify_tree says
 * how many drafts stand and draws the token after them; nm_kv_compact moves the rows of an
 * accepted tree path together.
 *
 * Conventions: those of nm_sparse.h (device pointers owned by the caller, work enqueued on
 * `stream`, arguments checked before any HIP call, status codes, no allocation, copy or
 * synchronisation in the library). fp16 is passed as its raw bit pattern (uint16_t). Strides
 * count elements between one token and the next; a token's heads are contiguous. Values that
 * lie in device memory (page tables, lengths, positions, masks, tokens) cannot be checked by
 * the call: bad ones give unspecified or skipped results as documented, but never an access
 * outside the caller's arrays.
 *
 * Nodes: the tokens of one sequence's step are nodes 0 .. n-1 (n <= 64 for attention and
 * verification): node 0 is the last accepted token, whose k and v are not in the cache yet,
 * the others are drafts, each after its parent. In a chain node i's parent is node i-1. Node
 * i's k and v go to cache position start + i, whatever its depth in the tree.
 */
#ifndef NM_DECODE_H
#define NM_DECODE_H

#include <stddef.h>
#include <stdint.h>

#include "nm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further status of these calls: an unknown cache format or rotary layout, or a head size
 * or page size that they do not take. */
#define NM_ERR_FORMAT 8

/* Cache formats. The 8-bit ones hold each head's row x of a token as codes and one fp32 scale:
 * scale = max|x| / L, code = round(x * (L / max|x|)) to nearest even, value = code * scale,
 * with L = 127 (int8) or 448 (e4m3, the OCP 8-bit float without infinities). Rows whose
 * max|x| is below 1e-30 are held as zeros (scale 0). A row with an infinity or NaN in it is
 * held as NaN (scale NaN, codes 0) in the 8-bit formats, and as it is in fp16. */
enum { NM_KV_FP16 = 0, NM_KV_INT8 = 1, NM_KV_E4M3 = 2 };

/* A paged cache: `blocks` pages of `page` tokens each. A sequence's position p lies in slot
 * p % page of block table[p / page] of its row of the page table.
 *   k, v              [blocks][kv_heads][page][head_dim] fp16, int8 or e4m3; 16-byte aligned
 *   k_scale, v_scale  [blocks][kv_heads][page] fp32, 16-byte aligned (8-bit formats; else NULL)
 *   page      a power of two, 16 .. 1024;   head_dim  64, 128 or 256
 * The structure is read during the call only. */
typedef struct nm_kv_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t blocks;
  int32_t kv_heads;
  int32_t page;
  int32_t head_dim;
  int32_t format;
} nm_kv_cache;

/* Rotary layouts: pair i of a head is (x[i], x[i + rot_dim/2]) or (x[2i], x[2i+1]). */
enum { NM_ROPE_HALF = 0, NM_ROPE_INTERLEAVED = 1 };
/* Frequency scalings for long contexts, see nm_rope_turns. */
enum { NM_ROPE_PLAIN = 0, NM_ROPE_LINEAR = 1, NM_ROPE_BASE = 2, NM_ROPE_BANDS = 3 };

/* Host function, no HIP call: turns[i] for i < rot_dim/2 (host memory), the turns (full
 * circles) that pair i makes per position, in 64 bits:
 *   PLAIN   t_i = base^(-2i/rot_dim) / (2 pi)
 *   LINEAR  t_i / factor (positions interpolated)
 *   BASE    t_i with base * factor^(rot_dim/(rot_dim-2)) (the slowest pair slowed by factor)
 *   BANDS   pairs that turn fewer than `low` times within `length` positions are slowed by
 *           factor, pairs that turn more than `high` times are left, linear in between:
 *           t_i * w + t_i / factor * (1 - w), w = clamp((length * t_i - low)/(high - low), 0, 1)
 * factor, length, low and high are read by the scalings that name them. NM_ERR_NULL;
 * NM_ERR_SHAPE: rot_dim odd or outside 2 .. 1024 (BASE: below 4), or a parameter that is not
 * positive and finite (low may be 0; high > low); NM_ERR_FORMAT: unknown scaling. */
int nm_rope_turns(double* turns, int rot_dim, int scaling, double base, double factor, double length,
                  double low, double high);

/* Rotary positions: each head's first rot_dim elements turned by its token's position, the
 * rest copied: y = (a c - b s, b c + a s) * scale for pair (a, b), with c and s the cosine and
 * sine of 2 pi * positions[t] * turns[i]; the product and its fraction in 64 bits, so that far
 * positions lose nothing, the rest in 32, one rounding to fp16. A negative position turns
 * back (with -positions this is the transposed map). `scale` multiplies the turned part only
 * (1, or the magnitude factor some long-context scalings use).
 *   x, y       fp16, token t's head h at [t * stride + h * head_dim]; y may be x (same
 *              stride) but not overlap it otherwise
 *   positions  int32 [tokens];  turns  fp64 [rot_dim/2], device copies
 * NM_ERR_SHAPE: tokens outside 1 .. 2^30, heads outside 1 .. 65536, head_dim outside 2 .. 1024,
 * rot_dim odd or outside 2 .. head_dim, a stride below heads * head_dim or above 2^40;
 * NM_ERR_FORMAT: unknown layout; NM_ERR_ALIGN: x, y not 2-byte, positions not 4-byte, turns
 * not 8-byte aligned. (16-byte aligned x and y with strides that are multiples of 8, and head_dim
 * and rot_dim multiples of 16, take wide loads.) */
int nm_rope(const uint16_t* x, uint16_t* y, const int32_t* positions, const double* turns, int64_t tokens,
            int64_t heads, int head_dim, int rot_dim, int layout, float scale, int64_t x_stride,
            int64_t y_stride, void* stream);

/* Writes k and v of tokens 0 .. count[b]-1 of each sequence b at positions start[b] + t.
 *   k, v    fp16, token (b, t)'s head h at [(b * tokens + t) * stride + h * head_dim]; 16-byte
 *           aligned, strides multiples of 8
 *   table   int32 [batch][table_width];  start  int32 [batch];  count  int32 [batch], or NULL
 *           (all `tokens`); counts outside 0 .. tokens are clamped
 * Tokens whose position is outside 0 .. table_width * page - 1 or whose table entry is outside
 * 0 .. blocks - 1 are skipped (an entry of -1 is the usual filler). Two tokens of one call must
 * not share a slot. NM_ERR_SHAPE: batch outside 1 .. 65535, tokens outside 1 .. 2^24, batch * tokens
 * above 2^30, the call's q, k and v together (k alone, where it reads) above 2^35 elements,
 * table_width outside 1 .. 2^24 or table_width * page above 2^30, kv_heads outside 1 .. 4096,
 * blocks outside 1 .. 2^31 - 1, a stride below the heads' size or above 2^40. */
int nm_kv_append(const nm_kv_cache* cache, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                 int64_t v_stride, const int32_t* table, int64_t table_width, const int32_t* start,
                 const int32_t* count, int64_t batch, int64_t tokens, void* stream);

/* nm_rope on q and k and nm_kv_append in one launch: q turned into q_out (zeros for tokens
 * at or past count), k turned in fp32 and rounded once into the cache, v appended.
 *   q, q_out   as x, y of nm_rope, tokens (b, t) in order (q_out may be q with the same
 *              stride); 16-byte aligned, strides multiples of 8; q_heads may be 0 (q, q_out unused)
 *   positions  int32 [batch][tokens] (in a tree: start + depth);  rot_dim a multiple of 16
 * Other arguments and errors as nm_rope and nm_kv_append. */
int nm_rope_kv_append(const nm_kv_cache* cache, const uint16_t* q, uint16_t* q_out, int64_t q_heads,
                      int64_t q_stride, int64_t q_out_stride, const uint16_t* k, const uint16_t* v,
                      int64_t k_stride, int64_t v_stride, const int32_t* positions, const double* turns,
                      int rot_dim, int layout, float scale, const int32_t* table, int64_t table_width,
                      const int32_t* start, const int32_t* count, int64_t batch, int64_t tokens, void* stream);

/* Reads positions start[b] .. start[b] + count[b] - 1 of each sequence into k_out and v_out,
 * fp16 [batch][tokens][kv_heads][head_dim] (16-byte aligned), code * scale rounded once; zeros
 * for tokens at or past count and for positions that nm_kv_append would skip. Arguments and
 * errors as nm_kv_append. */
int nm_kv_read(const nm_kv_cache* cache, uint16_t* k_out, uint16_t* v_out, const int32_t* table,
               int64_t table_width, const int32_t* start, const int32_t* count, int64_t batch, int64_t tokens,
               void* stream);

/* Moves an accepted tree path's rows together: for 1 <= d <= accepted[b], position
 * start[b] + d gets the k, v and scales of position start[b] + path[b][d], all read before
 * any is written. path  int32 [batch][nodes] and accepted  int32 [batch], as nm_verify_tree
 * gives them (accepted is clamped to 0 .. nodes - 1). Entries outside 0 .. nodes - 1 and
 * positions that nm_kv_append would skip are left alone. nodes 1 .. 64; other limits as
 * nm_kv_append. */
int nm_kv_compact(const nm_kv_cache* cache, const int32_t* table, int64_t table_width, const int32_t* start,
                  const int32_t* path, const int32_t* accepted, int64_t batch, int64_t nodes, void* stream);

/* Attention of the nodes of each sequence's step over its cache:
 *   out[b][t][h] = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q[b][t][h] . k_j - max)
 * over the keys j that node t sees: positions 0 .. context[b] - 1, and position context[b] + i
 * where bit i of mask[b][t] is set and i < count[b] (mask NULL: a chain, node t sees nodes
 * 0 .. t). Query head h reads key head h / (heads / kv_heads). A node that sees no key, and
 * nodes at or past count, get zeros. Keys that a node does not see do not touch its result,
 * whatever they hold (NaN and infinities too). A draft whose v row has an infinity or NaN in
 * it makes the results of the nodes that see it NaN. fp16 products of exact codes, fp32 sums;
 * the weights times v's scale are rounded to fp16 for the second product: relative 2^-11 down to
 * 2^-21 of the largest in the row, below that 2^-32 of the largest.
 * Bit-identical from run to run for the same arguments, lengths and size of workspace.
 *   q     fp16, token (b, t)'s head h at [(b * tokens + t) * q_stride + h * head_dim]; 16-byte
 *         aligned, q_stride a multiple of 8;  out  fp16 [batch][tokens][heads][head_dim], 16-byte
 *         aligned
 *   mask  uint64 [batch][tokens], 8-byte aligned, or NULL;  context, count  int32 [batch]
 * context and context + count are clamped to 0 .. table_width * page (nodes past that end are
 * seen by none, and see what lies before it); positions whose table entry is outside
 * 0 .. blocks - 1 have unspecified keys and values.
 * workspace: device memory for the split of long contexts over the GPU, 16-byte aligned, or
 * NULL (no split). Its first NM_DECODE_COUNTER_BYTES are counters that must be zero before
 * the first call on it; every call leaves them zero, so one workspace serves any sequence of
 * nm_tree_attention and nm_verify calls in stream order. Fewer bytes than
 * nm_tree_attention_workspace_bytes split as far as they go. Calls that overlap on one workspace
 * race. NM_ERR_SHAPE: tokens outside 1 .. 64, heads not a multiple of kv_heads or above 16
 * times kv_heads or 65536, batch outside 1 .. 65535, batch * kv_heads above 2^23, a scale that
 * is not finite, others as nm_kv_append. */
#define NM_DECODE_COUNTER_BYTES 65536u
int nm_tree_attention(const nm_kv_cache* cache, const uint16_t* q, uint16_t* out, int64_t heads,
                      int64_t q_stride, const int32_t* table, int64_t table_width, const int32_t* context,
                      const uint64_t* mask, const int32_t* count, int64_t batch, int64_t tokens, float scale,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace nm_tree_attention uses at most for these arguments, or for fewer tokens, on
 * the current device (0: it takes no split, or the arguments are invalid, or no device). So one
 * workspace, made for the most tokens, serves every step of these sequences. */
size_t nm_tree_attention_workspace_bytes(const nm_kv_cache* cache, int64_t heads, int64_t table_width,
                                         int64_t batch, int64_t tokens);

/* Verification of a drafted chain by rejection sampling. For sequence b with n = count[b]
 * nodes (clamped to 0 .. nodes; NULL: all), draft i = 1 .. n-1 with token x = tokens[b][i] stands
 * if the drafts before it do and
 *   uniforms[b][i] * draft[b][i-1][x] < target[b][i-1][x]
 * (the product in 64 bits); the first that does not ends the chain. With m drafts accepted the
 * next token is drawn from target[b][m] where m = n - 1, else from the positive part of
 * target[b][m] - draft[b][m]: the first index whose running sum of weights (64 bits) exceeds
 * uniforms[b][0] times their sum. Weights that are not positive and finite count as zero; if
 * none is left the draw is from target[b][m], and the token is -1 if that leaves none either.
 * The target's distribution is kept exactly.
 *   target  fp32 [batch][nodes][vocab], the target's probabilities after each node
 *   draft   fp32 [batch][nodes-1][vocab], the distribution draft i+1 was drawn from (NULL only
 *           if nodes is 1)
 *   tokens  int32 [batch][nodes] ([b][0] is not read);  uniforms  fp32 [batch][nodes] in [0, 1)
 *   accepted   int32 [batch]: m;  out_tokens  int32 [batch][nodes]: the accepted drafts'
 *              tokens, the drawn token, then -1 (all -1 and accepted 0 where count is 0)
 * A token outside 0 .. vocab - 1 is refused. workspace: as nm_tree_attention's, at least
 * nm_verify_workspace_bytes, or NULL (each sequence on one workgroup); the draw is the same
 * up to the order of 64-bit sums. NM_ERR_SHAPE: nodes outside 1 .. 64, batch outside
 * 1 .. 65535, vocab outside 1 .. 2^24. fp32 and int32 arrays 4-byte aligned, workspace 16. */
int nm_verify_chain(const float* target, const float* draft, const int32_t* tokens, const float* uniforms,
                    const int32_t* count, int32_t* accepted, int32_t* out_tokens, int64_t batch, int64_t nodes,
                    int64_t vocab, void* workspace, size_t workspace_bytes, void* stream);

/* Verification of a drafted tree whose tokens were chosen (not drawn), e.g. a draft head's
 * best candidates. From node 0 on, the children of the node reached are tried in node order:
 * child c with token x stands if
 *   uniforms[b][c] * (1 - sum of target[.][x'] over the siblings tried before) < target[.][x]
 * on the node's row of the target (in 64 bits; a token that an earlier sibling had counts as
 * zero); the first that stands is the next node. Where none does, the next token is drawn as
 * in nm_verify_chain from the row without the refused tokens. The target's distribution is
 * kept exactly.
 *   parents  int32 [batch][nodes]: the parent of each node, before it ([b][0] is not read);
 *            a node whose parent is outside 0 .. its own index - 1 is not reached
 *   path     int32 [batch][nodes]: the nodes reached, from node 0 on, then -1
 * Other arguments, outputs and errors as nm_verify_chain. */
int nm_verify_tree(const float* target, const int32_t* tokens, const int32_t* parents, const float* uniforms,
                   const int32_t* count, int32_t* accepted, int32_t* out_tokens, int32_t* path, int64_t batch,
                   int64_t nodes, int64_t vocab, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace the nm_verify calls use at most for these sizes, or for fewer sequences, on
 * the current device (0: none). */
size_t nm_verify_workspace_bytes(int64_t batch, int64_t vocab);

#ifdef __cplusplus
}
#endif

#endif /* NM_DECODE_H */
