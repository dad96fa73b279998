// Attention of a step's nodes over the paged cache, on the matrix instructions.
//
// Mathematics. For one sequence and key head the T nodes' queries of the G query heads that
// share it are R = T G rows; S^T = K Q^T gives keys down, rows across, the softmax runs over the
// keys with a running maximum, and O^T = V^T P^T adds up. A value's scale z_j goes into the
// exponent: with x_j = s_j + log2 z_j (scores in units of log2) the weight that the second
// product takes in fp16 is 2^(x_j - m), and l = sum 2^(x_j - m) / z_j is kept in fp32. Each row's
// reference m is the largest x_j so far, so the weights stay in fp16's range whatever the
// scales of v; it moves only when it would grow by more than 8 (weights up to 2^8 are as exact
// in fp16), which takes the maximum over lanes and the rescaling out of most tiles.
//
// Work split. A workgroup of 4 waves takes one key head's rows (16 NR of them) and a chunk of
// one sequence's keys; its waves take every fourth tile of 32 keys, so that no K or V passes
// through LDS: in the instruction v_mfma_f32_16x16x32_f16 (A: lane l holds row l % 16, K-slots
// 8 (l / 16) + 0..7; D: lane l holds column l % 16, rows 4 (l / 16) + 0..3) the K-slots may stand
// for any elements as long as A and B agree, which is used twice:
//   - S: a lane's 16-byte loads of a key row are its K-slots; Q is read in the same order.
//     Row m of tile h stands for key 8 (m / 4) + m % 4 + 4 h of the 32, so that the two tiles'
//     results leave lane (g, row) with keys 8 g + 0..7: its K-slots of the second product.
//   - O: a lane loads, of each of those 8 keys, the d's DM l%16 .. + DM - 1 (DM = D / 16), and
//     tile j's row m stands for d = DM m + j: bytes of the 8 key rows are paired in registers.
// 8-bit codes are exact in fp16 (integers up to 127; e4m3 is a subset), so the first product
// is exact up to its fp32 sums.
#pragma once

#include "nm_decode_internal.h"

namespace nm {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kTileKeys = 32;
constexpr int kMinChunkTiles = kAttnWaves;   // one tile a wave
constexpr float kLowest = -3e38f;            // the reference of a row that has seen nothing
// A value's scale counts as at least this (rows of zeros have scale 0, and codes 0): far below
// what fp16 results can show, and its reciprocal times any number of keys is finite.
constexpr float kLeastScale = 0x1p-100f;

// How the host cuts a call up: `slots` chunks over all sequences (0: one a sequence), row_tiles
// workgroups of rows, and where the chunks' partial results go.
struct AttnSplit {
  int slots;
  int row_tiles;
  uint32_t* counters;
  char* parts;
  uint32_t part_bytes;
};

template <int FMT, int D, int NR>
struct AttnShape {
  static constexpr int kCodeBytes = FMT == NM_KV_FP16 ? 2 : 1;
  static constexpr int kRowBytes = D * kCodeBytes;
  static constexpr int kSteps = D / 32;               // matrix steps of a score
  static constexpr int kLoadsK = kRowBytes / 64;      // 16-byte loads of a key row by its 4 lanes
  static constexpr int kWordsV = kRowBytes / 64;      // dwords of a value row by its 16 lanes
  static constexpr int kJ = D / 16;                   // d tiles
  static constexpr int kOwn = kJ / kAttnWaves;        // d tiles of each row tile a wave ends up with
  static constexpr int kPer = kOwn < 2 ? kOwn : 2;    // of them exchanged in a round
  static constexpr uint32_t kPartBytes = kJ * NR * 1024 + NR * 128;
};

// Waves a SIMD holds (its 512 registers a lane over the accumulators, Q and one tile), which is
// also the workgroups a CU holds.
constexpr int kPairRows = 2;
constexpr int attn_waves(int D, int NR) { return D > 128 ? (NR == 1 ? 2 : 1) : NR == 1 ? 3 : NR <= kPairRows ? 2 : 1; }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// max and sum over the 4 lanes that share l % 16
__device__ __forceinline__ float max4(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum4(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Two fp16 from bytes 0, 1 (hi: 2, 3) of a word of codes. int8 codes come with their sign bit
// flipped: 0x6400 + u is 1024 + u in fp16, and 1152 taken off is exact.
template <int FMT>
__device__ __forceinline__ uint32_t pair_of(uint32_t codes, bool hi) {
  if constexpr (FMT == NM_KV_E4M3) {
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(codes), 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(codes), 1.0f, false));
  } else {
    const uint32_t u = __builtin_amdgcn_perm(codes, 0x64646464u, hi ? 0x00070006u : 0x00050004u);
    const f16x2 c = {_Float16(1152.0f), _Float16(1152.0f)};
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, u) - c);
  }
}

template <int FMT>
__device__ __forceinline__ uint32_t flipped(uint32_t codes) {
  return FMT == NM_KV_INT8 ? codes ^ 0x80808080u : codes;
}

__device__ __forceinline__ f16x8 as_half8(const uint32_t (&w)[4]) {
  const u32x4 v = {w[0], w[1], w[2], w[3]};
  return __builtin_bit_cast(f16x8, v);
}

// Bits 15 and 31: whether the two fp16 of a word are infinite or NaN.
__device__ __forceinline__ uint32_t non_finite(uint32_t v) {
  return ((v & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}

// One tile of 32 keys in a lane's registers.
template <int FMT, int D>
struct AttnTile {
  using S = AttnShape<FMT, D, 1>;
  u32x4 k[2][S::kLoadsK];
  uint32_t v[8][S::kWordsV];
  float ks[8], vs[8];   // scales of keys 8 g + 0..7 (8-bit formats)
};

template <int FMT, int D, int NR>
struct AttnWave {
  using S = AttnShape<FMT, D, NR>;
  const PagedCache& cache;
  const int32_t* table;       // this sequence's page table
  int head, lane, li, g;
  uint32_t keys, context;     // all of the sequence's keys; those every node sees
  float scale;                // of the scores, times log2 e
  u32x4 q[NR][S::kSteps];
  uint64_t mask[NR];
  f32x4 o[S::kJ][NR];
  float m[NR], l[NR];

  // The pages of a tile: of this lane's K rows (8 (li / 4) + ..) and of its V rows (8 g + ..).
  struct Pages {
    uint32_t k, v;
  };
  __device__ __forceinline__ Pages pages(uint32_t tile) const {
    const uint32_t last = uint32_t(cache.table_width) - 1, base = tile * kTileKeys;
    Pages p;
    p.k = uint32_t(table[min((base + 8u * (li >> 2)) >> cache.page_shift, last)]);
    p.v = uint32_t(table[min((base + 8u * g) >> cache.page_shift, last)]);
    return p;
  }

  __device__ __forceinline__ int64_t row_of(uint32_t block, uint32_t pos) const {
    block = min(block, cache.blocks - 1u);   // a bad entry reads some page of the cache
    return ((int64_t(block) * cache.kv_heads + head) << cache.page_shift) +
           (pos & ((1u << cache.page_shift) - 1u));
  }

  // 8 fp32 scales of the keys from row on.
  static __device__ __forceinline__ void load_scales(float (&s)[8], const float* base, int64_t row) {
    const float4* p = reinterpret_cast<const float4*>(base + row);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 a = p[h];
      s[4 * h] = a.x;
      s[4 * h + 1] = a.y;
      s[4 * h + 2] = a.z;
      s[4 * h + 3] = a.w;
    }
  }

  __device__ __forceinline__ void load_keys(AttnTile<FMT, D>& t, uint32_t tile, const Pages& p) const {
    const uint32_t base = tile * kTileKeys;
    const char* kr = cache.k + row_of(p.k, base + 8u * (li >> 2) + (li & 3)) * S::kRowBytes + 16 * g;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < S::kLoadsK; ++j)
        t.k[h][j] = *reinterpret_cast<const u32x4*>(kr + h * 4 * S::kRowBytes + 64 * j);
    if constexpr (FMT != NM_KV_FP16) load_scales(t.ks, cache.k_scale, row_of(p.v, base + 8u * g));
  }

  __device__ __forceinline__ void load_values(AttnTile<FMT, D>& t, uint32_t tile, const Pages& p) const {
    const int64_t vrow = row_of(p.v, tile * kTileKeys + 8u * g);
    if constexpr (FMT != NM_KV_FP16) load_scales(t.vs, cache.v_scale, vrow);
    const char* vr = cache.v + vrow * S::kRowBytes + 4 * S::kWordsV * li;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const char* r = vr + e * S::kRowBytes;
      if constexpr (S::kWordsV == 1) {
        t.v[e][0] = *reinterpret_cast<const uint32_t*>(r);
      } else if constexpr (S::kWordsV == 2) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(r);
        t.v[e][0] = x[0];
        t.v[e][1] = x[1];
      } else {
#pragma unroll
        for (int c = 0; c < S::kWordsV / 4; ++c) {
          const u32x4 x = reinterpret_cast<const u32x4*>(r)[c];
#pragma unroll
          for (int i = 0; i < 4; ++i) t.v[e][4 * c + i] = x[i];
        }
      }
    }
  }

  // The A operand of d tile j: this lane's 8 keys at d = DM li + j.
  __device__ __forceinline__ void value_frags(const AttnTile<FMT, D>& t, int c, f16x8 (&f)[4 / S::kCodeBytes]) const {
    uint32_t w[4 / S::kCodeBytes][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if constexpr (FMT == NM_KV_FP16) {
        w[0][p] = __builtin_amdgcn_perm(t.v[2 * p + 1][c], t.v[2 * p][c], 0x05040100u);
        w[1][p] = __builtin_amdgcn_perm(t.v[2 * p + 1][c], t.v[2 * p][c], 0x07060302u);
      } else {
        const uint32_t a = flipped<FMT>(t.v[2 * p][c]), b = flipped<FMT>(t.v[2 * p + 1][c]);
        const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x05010400u), hi = __builtin_amdgcn_perm(b, a, 0x07030602u);
        w[0][p] = pair_of<FMT>(lo, false);
        w[1][p] = pair_of<FMT>(lo, true);
        w[2][p] = pair_of<FMT>(hi, false);
        w[3][p] = pair_of<FMT>(hi, true);
      }
    }
#pragma unroll
    for (int x = 0; x < 4 / S::kCodeBytes; ++x) f[x] = as_half8(w[x]);
  }

  // The scores of a tile in units of log2, without log2 z: x[n][e] is this lane's row n, key 8 g + e.
  __device__ __forceinline__ void scores(const AttnTile<FMT, D>& t, float (&x)[NR][8]) const {
    f32x4 s[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) s[n][0] = s[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) {
        f16x8 a;
        if constexpr (FMT == NM_KV_FP16) {
          a = __builtin_bit_cast(f16x8, t.k[h][st]);
        } else {
          const uint32_t c0 = flipped<FMT>(t.k[h][st / 2][2 * (st & 1)]), c1 = flipped<FMT>(t.k[h][st / 2][2 * (st & 1) + 1]);
          const uint32_t w[4] = {pair_of<FMT>(c0, false), pair_of<FMT>(c0, true), pair_of<FMT>(c1, false), pair_of<FMT>(c1, true)};
          a = as_half8(w);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
          s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(f16x8, q[n][st]), s[n][h], 0, 0, 0);
      }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = FMT == NM_KV_FP16 ? scale : t.ks[e] * scale;
#pragma unroll
      for (int n = 0; n < NR; ++n) x[n][e] = s[n][e >> 2][e & 3] * c;
    }
  }

  // Which of a tile's keys this lane's row n sees, a bit each.
  __device__ __forceinline__ uint32_t seen_of(int n, uint32_t key0) const {
    uint32_t seen = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t node = key0 + e - context;   // wraps to a large number in the context
      seen |= uint32_t(key0 + e < context || (node < 64u && ((mask[n] >> node) & 1))) << e;
    }
    return seen;
  }

  // The softmax's weights of a tile in fp16; the running reference and sum. edge: the tile holds
  // keys that not every node sees, or that are past the end.
  __device__ __forceinline__ void weights(AttnTile<FMT, D>& t, float (&x)[NR][8], f16x8 (&w)[NR], bool edge,
                                          uint32_t key0) {
    uint32_t bad = 0;   // keys of a draft whose scale is not a number: rows that see them are NaN
    if constexpr (FMT != NM_KV_FP16) {
      if (edge) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool b = !(t.vs[e] < __builtin_inff());
          bad |= uint32_t(b) << e;
          if (b) t.vs[e] = 1.0f;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t.vs[e] = t.vs[e] < kLeastScale ? kLeastScale : t.vs[e];   // NaN stays
        const float lz = __builtin_amdgcn_logf(t.vs[e]);
#pragma unroll
        for (int n = 0; n < NR; ++n) x[n][e] += lz;
      }
    }
    if (edge) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const uint32_t seen = seen_of(n, key0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if ((bad >> e) & 1) x[n][e] = __builtin_nanf("");
          if (!((seen >> e) & 1)) x[n][e] = -__builtin_inff();
        }
      }
    }
    float top[NR];
    bool grows = false;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      top[n] = fmaxf(fmaxf(fmaxf(x[n][0], x[n][1]), fmaxf(x[n][2], x[n][3])),
                     fmaxf(fmaxf(x[n][4], x[n][5]), fmaxf(x[n][6], x[n][7])));
      grows |= top[n] > m[n] + 8.0f;
    }
    if (__any(grows)) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float next = fmaxf(m[n], max4(top[n]));
        const float f = exp2_fast(m[n] - next);
        m[n] = next;
        l[n] *= f;
#pragma unroll
        for (int j = 0; j < S::kJ; ++j) o[j][n] *= f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float iz = FMT == NM_KV_FP16 ? 1.0f : __builtin_amdgcn_rcpf(t.vs[e]);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float y = exp2_fast(x[n][e] - m[n]);
        l[n] = FMT == NM_KV_FP16 ? l[n] + y : fmaf(y, iz, l[n]);
        w[n][e] = _Float16(y);   // to nearest even: 2^-11 of the weight
      }
    }
  }

  // O^T += V^T P^T.
  __device__ __forceinline__ void product(AttnTile<FMT, D>& t, const f16x8 (&w)[NR], bool edge, uint32_t key0) {
    if (edge) {
      uint32_t bad = 0;   // whether this lane holds a non-finite half of a draft
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t held = key0 + e < keys ? ~0u : 0u, draft = key0 + e < context ? 0u : ~0u;
#pragma unroll
        for (int c = 0; c < S::kWordsV; ++c) {
          t.v[e][c] &= held;   // past the end: never written, perhaps NaN, and 0 times that is not 0
          if (FMT == NM_KV_FP16) bad |= non_finite(t.v[e][c]) & draft;
        }
      }
      if (FMT == NM_KV_FP16 && __any(bad != 0)) {
        poisoned(t, w, key0);
        return;
      }
    }
#pragma unroll
    for (int c = 0; c < S::kWordsV; ++c) {
      constexpr int F = 4 / S::kCodeBytes;
      f16x8 f[F];
      value_frags(t, c, f);
#pragma unroll
      for (int x = 0; x < F; ++x)
#pragma unroll
        for (int n = 0; n < NR; ++n)
          o[F * c + x][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[x], w[n], o[F * c + x][n], 0, 0, 0);
    }
  }

  // The second product of a tile in which a draft's fp16 v holds infinities or NaN: they are
  // taken out of it, and a product of "is one" with "is seen" marks the results they reach.
  __device__ __forceinline__ void poisoned(AttnTile<FMT, D>& t, const f16x8 (&w)[NR], uint32_t key0) {
    f16x8 on[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const uint32_t seen = seen_of(n, key0);
#pragma unroll
      for (int e = 0; e < 8; ++e) on[n][e] = _Float16(float((seen >> e) & 1));
    }
#pragma unroll
    for (int c = 0; c < S::kWordsV; ++c) {
      AttnTile<FMT, D> ind;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t n = key0 + e < context ? 0u : non_finite(t.v[e][c]);
        const uint32_t halves = (n >> 15) * 0xFFFFu;
        ind.v[e][c] = halves & 0x3C003C00u;
        t.v[e][c] &= ~halves;
      }
      f16x8 f[4 / S::kCodeBytes], b[4 / S::kCodeBytes];
      value_frags(t, c, f);
      value_frags(ind, c, b);
#pragma unroll
      for (int x = 0; x < 4 / S::kCodeBytes; ++x)
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const int j = (4 / S::kCodeBytes) * c + x;
          o[j][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[x], w[n], o[j][n], 0, 0, 0);
          const f32x4 hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[x], on[n], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (hit[i] > 0.f) o[j][n][i] = __builtin_nanf("");
        }
    }
  }
};

// Which sequence and chunk of it a slot is: the chunk's size in tiles follows from the
// sequences' lengths, so that the slots' work is even however ragged they are.
struct AttnChunk {
  int b;            // -1: no work
  int first;        // the sequence's first slot
  int chunks;       // its number of slots
  uint32_t tiles;   // tiles a chunk
  uint32_t context, keys;
  int count;
};

__device__ __forceinline__ void attn_lengths(const AttnCall& a, int b, uint32_t& context, uint32_t& keys, int& count) {
  const int64_t most = int64_t(a.cache.table_width) << a.cache.page_shift;
  const int64_t c = a.context[b];
  count = count_of(a.count, b, a.tokens);
  context = uint32_t(c < 0 ? 0 : c > most ? most : c);
  keys = uint32_t(min(int64_t(context) + count, most));
}

__device__ __forceinline__ uint32_t chunks_of(uint32_t tiles, uint32_t per) {
  return tiles <= per ? 1u : (tiles + per - 1) / per;
}

// Every wave works this out for itself: 64 sequences a pass, one a lane.
__device__ __forceinline__ AttnChunk find_chunk(const AttnCall& a, int slots, int slot) {
  const int lane = threadIdx.x & 63;
  const auto tiles_of = [&](int b) {
    uint32_t context, keys = 0;
    int count;
    if (b < a.batch) attn_lengths(a, b, context, keys, count);
    return (keys + kTileKeys - 1) / kTileKeys;
  };
  uint32_t per = 0x7FFFFFFFu;
  if (slots > a.batch) {
    double total = 0.0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) total += double(tiles_of(b0 + lane));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) total += __shfl_xor(total, o);
    // The last chunk of a sequence is half empty on average: that many slots are set aside, and
    // one a sequence, which always fits, if they do not do. Whole rounds of the waves.
    const double half = ceil(total / ((double(slots) - 0.5 * a.batch) * kAttnWaves));
    per = half < 1.0 ? kAttnWaves : uint32_t(half) * kAttnWaves;
    uint32_t used = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) used += b0 + lane < a.batch ? chunks_of(tiles_of(b0 + lane), per) : 0u;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) used += __shfl_xor(used, o);
    if (used > uint32_t(slots)) per = uint32_t(ceil(total / (double(slots - a.batch) * kAttnWaves))) * kAttnWaves;
  }
  AttnChunk k;
  k.b = -1;
  int before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    uint32_t context = 0, keys = 0;
    int count = 0, n = 0;
    if (b0 + lane < a.batch) {
      attn_lengths(a, b0 + lane, context, keys, count);
      n = int(chunks_of((keys + kTileKeys - 1) / kTileKeys, per));
    }
    int upto = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(upto, o);
      if (lane >= o) upto += x;
    }
    const uint64_t past = __ballot(before + upto > slot);
    if (past != 0) {
      const int at = __builtin_ctzll(past);
      k.b = b0 + at;
      k.chunks = __shfl(n, at);
      k.first = before + __shfl(upto, at) - k.chunks;
      k.tiles = per;
      k.context = __shfl(context, at);
      k.keys = __shfl(keys, at);
      k.count = __shfl(count, at);
      return k;
    }
    before += __shfl(upto, 63);
  }
  return k;
}

template <int FMT, int D, int NR>
__global__ __launch_bounds__(kAttnThreads, attn_waves(D, NR)) void attention_kernel(AttnCall a, AttnSplit sp) {
  using S = AttnShape<FMT, D, NR>;
  __shared__ f32x4 xch[kAttnWaves][kAttnWaves * S::kPer][64];
  __shared__ float stat_m[kAttnWaves][16 * NR], stat_l[kAttnWaves][16 * NR];
  __shared__ uint32_t arrived;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = int(blockIdx.x) % a.cache.kv_heads, slot = int(blockIdx.x) / a.cache.kv_heads;
  const int rt = blockIdx.y;
  AttnChunk ck = find_chunk(a, sp.slots, slot);
  const int b = __builtin_amdgcn_readfirstlane(ck.b);
  if (b < 0) return;
  const int chunks = __builtin_amdgcn_readfirstlane(ck.chunks), first = __builtin_amdgcn_readfirstlane(ck.first);
  const int count = __builtin_amdgcn_readfirstlane(ck.count);
  const uint32_t per = __builtin_amdgcn_readfirstlane(ck.tiles);

  AttnWave<FMT, D, NR> w{a.cache, a.cache.table + int64_t(b) * a.cache.table_width};
  w.head = head;
  w.lane = tid & 63;
  w.li = w.lane & 15;
  w.g = w.lane >> 4;
  w.context = __builtin_amdgcn_readfirstlane(ck.context);
  w.keys = __builtin_amdgcn_readfirstlane(ck.keys);
  w.scale = a.scale * 1.44269504088896341f;
  const int rows = a.tokens * a.group;
  // the nodes' rows: t = r / group, query head head * group + r % group
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = (rt * NR + n) * 16 + w.li, t = r / a.group;
    const bool live = r < rows && t < count;
    const uint16_t* qr = a.q + (int64_t(b) * a.tokens + t) * a.q_stride + int64_t(head * a.group + r % a.group) * D;
    uint64_t mk = 0;
    if (live) mk = a.mask != nullptr ? a.mask[int64_t(b) * a.tokens + t] : t >= 63 ? ~0ull : (2ull << t) - 1;
    w.mask[n] = count >= 64 ? mk : mk & ((1ull << count) - 1);
#pragma unroll
    for (int st = 0; st < S::kSteps; ++st) {
      const int d = FMT == NM_KV_FP16 ? 32 * st + 8 * w.g : 64 * (st >> 1) + 16 * w.g + 8 * (st & 1);
      w.q[n][st] = live ? *reinterpret_cast<const u32x4*>(qr + d) : u32x4{0, 0, 0, 0};
    }
    w.m[n] = kLowest;
    w.l[n] = 0.f;
#pragma unroll
    for (int j = 0; j < S::kJ; ++j) w.o[j][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // this chunk's tiles, every fourth a wave's. A tile's registers are loaded again as soon as it
  // is done with them: the next keys after the scores, the next values after their product
  const uint32_t all = (w.keys + kTileKeys - 1) / kTileKeys;
  const uint32_t begin = uint32_t(slot - first) * per;
  const uint32_t end = min(all, begin + per);   // per <= 2^31 - 1, begin <= all
  uint32_t tile = begin + wave;
  if (tile < end) {
    using Wave = AttnWave<FMT, D, NR>;
    AttnTile<FMT, D> t;
    typename Wave::Pages p = w.pages(tile), next = w.pages(tile + kAttnWaves);
    w.load_keys(t, tile, p);
    w.load_values(t, tile, p);
    while (true) {
      const uint32_t after = tile + kAttnWaves, key0 = tile * kTileKeys + 8u * w.g;
      const bool edge = (tile + 1) * kTileKeys > w.context;
      p = next;
      next = w.pages(after + kAttnWaves);
      float x[NR][8];
      f16x8 y[NR];
      w.scores(t, x);
      if (after < end) w.load_keys(t, after, p);
      w.weights(t, x, y, edge, key0);
      w.product(t, y, edge, key0);
      if (after >= end) break;
      w.load_values(t, after, p);
      tile = after;
    }
  }

  // the waves' results together: each scaled to the common reference, then every wave adds up
  // its share of the (row tile, d tile) units over the waves in order
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    w.l[n] = sum4(w.l[n]);
    if (w.g == 0) {
      stat_m[wave][16 * n + w.li] = w.m[n];
      stat_l[wave][16 * n + w.li] = w.l[n];
    }
  }
  __syncthreads();
  float mm[NR], ll[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    mm[n] = kLowest;
    ll[n] = 0.f;
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) mm[n] = fmaxf(mm[n], stat_m[x][16 * n + w.li]);
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) ll[n] += stat_l[x][16 * n + w.li] * exp2_fast(stat_m[x][16 * n + w.li] - mm[n]);
    const float f = exp2_fast(w.m[n] - mm[n]);
#pragma unroll
    for (int j = 0; j < S::kJ; ++j) w.o[j][n] *= f;
  }
  f32x4 own[NR][S::kOwn];
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int r = 0; r < S::kOwn / S::kPer; ++r) {
      if (n + r) __syncthreads();
#pragma unroll
      for (int x = 0; x < kAttnWaves; ++x)
#pragma unroll
        for (int k = 0; k < S::kPer; ++k) xch[wave][x * S::kPer + k][w.lane] = w.o[x * S::kOwn + r * S::kPer + k][n];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < S::kPer; ++k) {
        f32x4 sum = xch[0][wave * S::kPer + k][w.lane];
#pragma unroll
        for (int x = 1; x < kAttnWaves; ++x) sum += xch[x][wave * S::kPer + k][w.lane];
        own[n][r * S::kPer + k] = sum;
      }
    }
  // d tiles wave * kOwn + k of every row tile are this wave's now
  int row[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) row[n] = (rt * NR + n) * 16 + w.li;

  if (chunks == 1) {
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      if (row[n] >= rows) continue;
      const int t = row[n] / a.group;
      const float inv = t < count && ll[n] != 0.f ? 1.0f / ll[n] : 0.f;
      uint16_t* out = a.out + ((int64_t(b) * a.tokens + t) * a.heads + head * a.group + row[n] % a.group) * D;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        typedef uint16_t run_t __attribute__((ext_vector_type(S::kOwn)));
        run_t y;
#pragma unroll
        for (int k = 0; k < S::kOwn; ++k) y[k] = uint16_t(float_to_half_bits(inv == 0.f ? 0.f : own[n][k][i] * inv));
        *reinterpret_cast<run_t*>(out + S::kJ * (4 * w.g + i) + wave * S::kOwn) = y;
      }
    }
    return;
  }

  // A chunk's partial: the rows' {m, l}, then 16 bytes (4 d's) for each (d tile, lane group, row),
  // rows fastest; `live` rows of this workgroup's are real.
  const int live = min(16 * NR, rows - rt * 16 * NR), units = live * (D / 4);
  const uint32_t stride = uint32_t(a.cache.kv_heads) * uint32_t(sp.row_tiles) * S::kPartBytes;
  char* p0 = sp.parts + ((uint64_t(first) * a.cache.kv_heads + head) * sp.row_tiles + rt) * S::kPartBytes;
  constexpr uint32_t kStats = 16 * NR * 8;
  __amdgpu_buffer_rsrc_t buf = coherent_buffer(p0, (chunks - 1) * stride + S::kPartBytes);
  const uint32_t mine = (slot - first) * stride;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    if (row[n] >= rows) continue;
    const int r = 16 * n + w.li;
#pragma unroll
    for (int k = 0; k < S::kOwn; ++k)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, own[n][k]), buf,
                                             mine + kStats + (((wave * S::kOwn + k) * 4 + w.g) * live + r) * 16, 0, kCoherent);
    if (wave == 0 && w.g == 0) {
      const u32x2 x = {__float_as_uint(mm[n]), __float_as_uint(ll[n])};
      __builtin_amdgcn_raw_buffer_store_b64(x, buf, mine + r * 8, 0, kCoherent);
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // the partial has reached the coherence point
  __syncthreads();
  uint32_t* counter = sp.counters + (int64_t(b) * a.cache.kv_heads + head) * sp.row_tiles + rt;
  if (tid == 0) arrived = atomicAdd(counter, 1u);
  __syncthreads();
  if (arrived != uint32_t(chunks - 1)) return;
  if (tid == 0) atomicExch(counter, 0u);
  // The last of the sequence's chunks: all partials are complete. A thread takes units of 16
  // bytes of every `groups`-th chunk, 8 chunks' loads in flight; the groups' sums, and then the
  // rows, come together in LDS. The order is fixed, so the result is the same each time.
  float* sum = reinterpret_cast<float*>(xch);                 // [row][d]
  const int groups = units < kAttnThreads ? kAttnThreads / units : 1;
  const int grp = groups > 1 ? tid / units : 0;
  constexpr int U = 8;
  // the rows' references and sums: up to 16 threads a row, then one
  const int threads = min(16, kAttnThreads / live);
  const int r0 = tid % live, s0 = tid / live;
  float2* stat = reinterpret_cast<float2*>(xch);
  if (s0 < threads) {
    float m1 = kLowest, l1 = 0.f;
    for (int c0 = s0; c0 < chunks; c0 += threads * U) {
      u32x2 x[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        x[k] = __builtin_amdgcn_raw_buffer_load_b64(buf, min(c0 + k * threads, chunks - 1) * stride + r0 * 8, 0, kCoherent);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (c0 + k * threads >= chunks) continue;
        const float m2 = __uint_as_float(x[k][0]), next = fmaxf(m1, m2);
        l1 = l1 * exp2_fast(m1 - next) + __uint_as_float(x[k][1]) * exp2_fast(m2 - next);
        m1 = next;
      }
    }
    stat[s0 * live + r0] = make_float2(m1, l1);
  }
  __syncthreads();
  if (tid < live) {
    float m1 = kLowest, l1 = 0.f;
    for (int x = 0; x < threads; ++x) m1 = fmaxf(m1, stat[x * live + tid].x);
    for (int x = 0; x < threads; ++x) l1 += stat[x * live + tid].y * exp2_fast(stat[x * live + tid].x - m1);
    stat_m[0][tid] = m1;
    stat_l[0][tid] = l1;
  }
  __syncthreads();
  for (int u0 = groups > 1 ? tid - grp * units : tid; u0 < units; u0 += kAttnThreads) {
    if (grp >= groups) break;
    const int r = u0 % live, jg = u0 / live, j = jg >> 2, g = jg & 3;
    const float top = stat_m[0][r];
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = grp; c0 < chunks; c0 += groups * U) {
      u32x4 y[U];
      uint32_t mc[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const uint32_t at = min(c0 + x * groups, chunks - 1) * stride;
        mc[x] = __builtin_amdgcn_raw_buffer_load_b32(buf, at + r * 8, 0, kCoherent);
        y[x] = __builtin_amdgcn_raw_buffer_load_b128(buf, at + kStats + u0 * 16, 0, kCoherent);
      }
#pragma unroll
      for (int x = 0; x < U; ++x) {
        if (c0 + x * groups >= chunks) continue;
        acc += __builtin_bit_cast(f32x4, y[x]) * exp2_fast(__uint_as_float(mc[x]) - top);
      }
    }
    float* at = sum + (grp * live + r) * D + S::kJ * 4 * g + j;
#pragma unroll
    for (int i = 0; i < 4; ++i) at[S::kJ * i] = acc[i];
  }
  __syncthreads();
  for (int u = tid; u < live * (D / 8); u += kAttnThreads) {
    const int r = u / (D / 8), d = u % (D / 8) * 8, node = (rt * NR * 16 + r) / a.group;
    const float l1 = stat_l[0][r], inv = node < count && l1 != 0.f ? 1.0f / l1 : 0.f;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = 0.f;
      for (int x = 0; x < groups; ++x) y[e] += sum[(x * live + r) * D + d + e];
      y[e] = inv == 0.f ? 0.f : y[e] * inv;
    }
    *reinterpret_cast<u32x4*>(a.out + ((int64_t(b) * a.tokens + node) * a.heads + head * a.group +
                                       (rt * NR * 16 + r) % a.group) * D + d) = halves_of(y);
  }
}

}  // namespace nm
