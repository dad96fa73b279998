// Attention of a step's nodes over the paged cache, on the matrix instructions.
//
// Mathematics. For one sequence and key head the T nodes' queries of the G query heads that
// share it are R = T G rows; S^T = K Q^T gives keys down, rows across, the softmax runs over the
// keys with a running maximum, and O^T = V^T P^T adds up. A value's scale z_j goes into the
// exponent: with x_j = s_j + log2 z_j (scores in units of log2) the weight that the second
// product takes in fp16 is 2^(x_j - m), and l = sum 2^(x_j - m) / z_j is kept in fp32. Each row's
// reference m is set 7 below the largest x_j so far, so the weights stay in fp16's range whatever
// the scales of v; it moves only when it would grow by more than 8, which takes the maximum over
// lanes and the rescaling out of most tiles. So the largest weight is 2^7 to 2^15, and fp16's
// normal numbers hold what is down to 2^-21 of it to 2^-11, smaller ones to 2^-32 of it. (Without
// the 7, 4096 keys 2^-22.5 below a leading one were off by 6%.)
//
// Work split. A workgroup of 4 waves takes one key head's rows (16 NR of them) and a chunk of
// one sequence's keys; its waves take every fourth tile of 32 keys. Each wave loads its own tiles
// of keys and values straight into its own part of LDS (16 bytes a lane, no registers, nothing
// shared, so no barriers) and loads a side again as soon as it has been read. In the instruction
// v_mfma_f32_16x16x32_f16 (A: lane l holds row l % 16, K-slots 8 (l / 16) + 0..7; D: lane l holds
// column l % 16, rows 4 (l / 16) + 0..3) the K-slots may stand for any elements as long as A and B
// agree, which is used twice:
//   - S: a lane's 16-byte pieces of a key row are its K-slots; Q is read in the same order.
//     Row m of tile h stands for key 8 (m / 4) + m % 4 + 4 h of the 32, so that the two tiles'
//     results leave lane (g, row) with keys 8 g + 0..7: its K-slots of the second product.
//   - O: a lane reads, of each of those 8 keys, the d's DM l%16 .. + DM - 1 (DM = D / 16), and
//     tile j's row m stands for d = DM m + j: bytes of the 8 key rows are paired in registers.
// 8-bit codes are exact in fp16 (integers up to 127; e4m3 is a subset), so the first product
// is exact up to its fp32 sums.
// The workgroup's waves add up through LDS, a sequence's chunks through the workspace: the last to
// arrive joins the partial results, in the chunks' order, so that a result is the same each time.
//
// What bounds it, with times on one GPU (a pure read of the same bytes reaches 7.0 TB/s, a large
// copy 4.8):
//   - few tokens over long contexts: reading the cache. 32 sequences of up to 8192 int8 tokens, 8
//     key heads of 128, one token each of 32 heads (353 MB): 69.1 us, 5.1 TB/s. Three workgroups a
//     CU hold 100 KB in flight there; the vector units are busy 30% of the time.
//   - many rows: a tile's vector work (codes to fp16, scales, softmax) and its waits on LDS, at two
//     workgroups a CU. 2 x 131071 int8 tokens, 8 nodes, 40 heads (450 MB, 33 GFLOP): 97 to 102 us; 4
//     x 64 nodes over up to 8192 int8 tokens, 64 heads: 125 us, 360 TFLOP/s.
//   - short work: the chain of dependent steps, lengths and page table 2, first tile 3, exchange
//     0.5, partial and count 2.5, join 2 us. One token over 777 fp16 tokens: 11 us.
#pragma once

#include <type_traits>

#include "nm_decode_internal.h"

namespace nm {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kTileKeys = 32;
constexpr int kMinChunkTiles = 2 * kAttnWaves;   // two tiles a wave: a chunk more costs the join as much
constexpr int kNonTemporal = 2;              // cache policy bit of a load
constexpr float kLowest = -3e38f;            // the reference of a row that has seen nothing
constexpr float kLift = 7.0f;                // from a row's reference, when it moves, to its largest score
constexpr float kLag = 8.0f;                 // the score's growth until it moves: 2^(kLift + kLag) fits fp16
// A value's scale counts as at least this (rows of zeros have scale 0, and codes 0): far below
// what fp16 results can show, its reciprocal times any number of keys is finite, and a key's term
// of the sum, 2^(x - m) before the reciprocal, stays in fp32's range down to 2^-60 of the largest
// beside values up to fp16's. (With 2^-100 it did not: 65535 rows of zeros 2^-18.5 below one of
// 61440 were left out: the result was 18% too large.)
constexpr float kLeastScale = 0x1p-60f;

// How the host cuts a call up: `slots` chunks over all sequences (0: one a sequence), row_tiles
// workgroups of rows, and where the chunks' partial results go.
struct AttnSplit {
  int slots;
  int row_tiles;
  uint32_t* counters;
  char* parts;
  uint32_t part_bytes;
  float join;      // what a partial result costs in the join, in tiles
};

// What a kernel variant holds: registers and LDS set the waves of a SIMD (the workgroups of a
// CU), the row bytes the loads of a tile, and what is left of the 160 KiB the tiles in flight.
template <int FMT, int D, int NR>
struct AttnShape {
  static constexpr int kCodeBytes = FMT == NM_KV_FP16 ? 2 : 1;
  static constexpr int kRowBytes = D * kCodeBytes;
  static constexpr int kSteps = D / 32;               // matrix steps of a score
  static constexpr int kLoadsK = kRowBytes / 64;      // 16-byte pieces of a key row for each of its 4 lanes
  static constexpr int kWordsV = kRowBytes / 64;      // dwords of a value row for each of its 16 lanes
  static constexpr int kJ = D / 16;                   // d tiles
  static constexpr int kOwn = kJ / kAttnWaves;        // d tiles of each row tile a wave ends up with
  static constexpr int kPer = kOwn < 2 ? kOwn : 2;    // of them exchanged in a round
  static constexpr uint32_t kPartBytes = kJ * NR * 1024 + NR * 128;

  static constexpr int kPieces = kRowBytes / 16;      // of a row
  static constexpr int kLoadRows = 64 / kPieces;      // rows one load of the wave brings
  static constexpr int kLoads = kTileKeys / kLoadRows;                   // of a tile's keys, or values
  static constexpr int kScaleLoads = FMT == NM_KV_FP16 ? 0 : 1;          // both scales, with the keys
  static constexpr int kTileLoads = 2 * kLoads + kScaleLoads;
  static constexpr int kSideBytes = kTileKeys * kRowBytes;
  static constexpr int kSlotBytes = 2 * kSideBytes + 384 * kScaleLoads;  // a tile

  // LDS: Q in operand order, {m, l} of each wave and row, a flag, and the waves' tiles (all of it
  // dynamic: a kernel's limit is raised for dynamic LDS alone). The exchange of results and the
  // join of partials take the tiles' LDS after them.
  static constexpr int kQBytes = NR * kSteps * 1024;
  static constexpr int kFixedBytes = kQBytes + 2 * kAttnWaves * 16 * NR * 4 + 16;
  static constexpr int kXchBytes = kAttnWaves * kAttnWaves * kPer * 1024;
  static constexpr int tiles_of(int waves) { return (160 * 1024 / waves - kFixedBytes) / kAttnWaves / kSlotBytes; }
  // Waves of a SIMD, which are also the workgroups of a CU: as the accumulators allow (beyond 256
  // registers the compiler moves them to and fro every tile), if a tile a wave fits in LDS.
  static constexpr int kByRows = D * NR <= 128 ? 3 : 2;
  static constexpr int kWaves = tiles_of(kByRows) >= 1 ? kByRows : tiles_of(2) >= 1 ? 2 : 1;
  static constexpr int kDepth = tiles_of(kWaves) > 4 ? 4 : tiles_of(kWaves);   // tiles in flight
  static constexpr int kWaveBytes = kDepth * kSlotBytes;
  static constexpr int kTilesAt = kQBytes;
  // chunks a sequence may have: 8 for each of the threads that take a row's {m, l} in the join
  static constexpr int kRowThreads = kAttnThreads / (16 * NR) < 16 ? kAttnThreads / (16 * NR) : 16;
  static constexpr int kMaxChunks = 8 * kRowThreads;
  static constexpr int kSumBytes = 16 * NR * D * 4, kFactorBytes = kMaxChunks * 16 * NR * 4;
  static constexpr int kAfterBytes = kXchBytes > kSumBytes + kFactorBytes ? kXchBytes : kSumBytes + kFactorBytes;
  static constexpr int kTilesBytes = kAttnWaves * kWaveBytes > kAfterBytes ? kAttnWaves * kWaveBytes : kAfterBytes;
  static constexpr int kStatAt = kTilesAt + kTilesBytes;
  static constexpr int kLdsBytes = kStatAt + kFixedBytes - kQBytes;
  static_assert(kDepth >= 1, "a tile fits");
};

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

// Two fp16 of a word of codes: bytes 0, 1 (hi: 2, 3) of e4m3. int8 codes come with their sign
// bit flipped, u = code + 128, and zero-extended to 16 bits they are the subnormals u 2^-24,
// exact in the matrix instruction. The scores' sums over a head's elements are corrected by 128
// times the sum of q. The values' run over the keys, and 128 times a long sum of weights would
// take the bits of a result that cancels: there the 128 comes off each pair of codes, exactly
// (131072 keys in one chunk, values that nearly cancel: off by 240 times the bound with the sums
// corrected; 32 sequences of one token 68.9 us then, 69.3 now, 2 of 8 nodes 100.8 and 100.7).
constexpr float kCodeUnit = 0x1p24f;    // int8: the products come out in 2^-24
constexpr float kCodeBias = 128.0f;

template <int FMT>
__device__ __forceinline__ uint32_t pair_of(uint32_t codes, bool hi) {
  if constexpr (FMT == NM_KV_E4M3)
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(codes), 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(codes), 1.0f, false));
  else
    return __builtin_amdgcn_perm(codes, codes, hi ? 0x0C030C02u : 0x0C010C00u);   // 0x0C: a zero byte
}

// Two flipped int8 codes, zero-extended, to code 2^-24.
__device__ __forceinline__ uint32_t unbiased(uint32_t pair) {
  const _Float16 bias = _Float16(-kCodeBias / kCodeUnit);
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, pair) + f16x2{bias, bias});
}

template <int FMT>
__device__ __forceinline__ uint32_t flipped(uint32_t codes) {
  return FMT == NM_KV_INT8 ? codes ^ 0x80808080u : codes;
}

__device__ __forceinline__ f16x8 as_half8(const uint32_t (&w)[4]) {
  const u32x4 v = {w[0], w[1], w[2], w[3]};
  return __builtin_bit_cast(f16x8, v);
}

// Nonzero where one of a word's two fp16 is infinite or NaN, or one of its four e4m3 codes is NaN
// (0x7F with either sign; there are no infinities). int8 codes are numbers.
template <int FMT>
__device__ __forceinline__ uint32_t non_finite(uint32_t v) {
  if constexpr (FMT == NM_KV_FP16) return ((v & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
  if constexpr (FMT == NM_KV_E4M3) return ((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return 0;
}

// The 16-byte pieces of a row in LDS are permuted by its number, so that the 8 lanes that read
// one piece of 8 different rows at a time find them in 8 different bank groups: piece p of row
// r lies at p ^ swizzle(r). (Rows of one read are 8 (li / 4) + li % 4 (+ 4), hence the bits.)
template <int ROW_BYTES>
constexpr __host__ __device__ int swizzle(int r) {
  return ROW_BYTES == 64 ? ((r >> 1) & 1) | ((r >> 3) & 1) << 1 : (r & 3) | ((r >> 3) & 1) << 2;
}

// Reads of LDS that direct loads have filled. The compiler would wait for every such load in
// flight before any read of LDS; the counted waits below are enough, so the reads are written
// out, each group with its own wait, and as few groups as may be: a wait costs some 200 cycles.

// N fragments of Q, 1 KiB apart.
template <int N>
__device__ __forceinline__ void lds_read_fragments(u32x4 (&d)[N], uint32_t at) {
  static_assert(N == 2 || N == 4 || N == 6, "");
  if constexpr (N == 2)
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:1024\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d[0]), "=&v"(d[1])
                 : "v"(at) : "memory");
  if constexpr (N == 4)
    asm volatile("ds_read_b128 %0, %4\n\t"
                 "ds_read_b128 %1, %4 offset:1024\n\t"
                 "ds_read_b128 %2, %4 offset:2048\n\t"
                 "ds_read_b128 %3, %4 offset:3072\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3])
                 : "v"(at) : "memory");
  if constexpr (N == 6)
    asm volatile("ds_read_b128 %0, %6\n\t"
                 "ds_read_b128 %1, %6 offset:1024\n\t"
                 "ds_read_b128 %2, %6 offset:2048\n\t"
                 "ds_read_b128 %3, %6 offset:3072\n\t"
                 "ds_read_b128 %4, %6 offset:4096\n\t"
                 "ds_read_b128 %5, %6 offset:5120\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(d[4]), "=&v"(d[5])
                 : "v"(at) : "memory");
}

// 8 pieces of 16, 8 or 4 bytes: 4 at a[0..3], and 4 OFFSET bytes further.
template <int OFFSET>
__device__ __forceinline__ void lds_read_rows(u32x4 (&d)[8], const uint32_t (&a)[4]) {
  asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %10\n\tds_read_b128 %3, %11\n\t"
               "ds_read_b128 %4, %8 offset:%12\n\tds_read_b128 %5, %9 offset:%12\n\t"
               "ds_read_b128 %6, %10 offset:%12\n\tds_read_b128 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(d[4]), "=&v"(d[5]), "=&v"(d[6]), "=&v"(d[7])
               : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(OFFSET) : "memory");
}
template <int OFFSET>
__device__ __forceinline__ void lds_read_rows(u32x2 (&d)[8], const uint32_t (&a)[4]) {
  asm volatile("ds_read_b64 %0, %8\n\tds_read_b64 %1, %9\n\tds_read_b64 %2, %10\n\tds_read_b64 %3, %11\n\t"
               "ds_read_b64 %4, %8 offset:%12\n\tds_read_b64 %5, %9 offset:%12\n\t"
               "ds_read_b64 %6, %10 offset:%12\n\tds_read_b64 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(d[4]), "=&v"(d[5]), "=&v"(d[6]), "=&v"(d[7])
               : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(OFFSET) : "memory");
}
template <int OFFSET>
__device__ __forceinline__ void lds_read_rows(uint32_t (&d)[8], const uint32_t (&a)[4]) {
  asm volatile("ds_read_b32 %0, %8\n\tds_read_b32 %1, %9\n\tds_read_b32 %2, %10\n\tds_read_b32 %3, %11\n\t"
               "ds_read_b32 %4, %8 offset:%12\n\tds_read_b32 %5, %9 offset:%12\n\t"
               "ds_read_b32 %6, %10 offset:%12\n\tds_read_b32 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(d[4]), "=&v"(d[5]), "=&v"(d[6]), "=&v"(d[7])
               : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(OFFSET) : "memory");
}

// A key row's pieces for both halves of a tile (rows 4 apart): L of each, from `a` on, and this
// lane's key's two scales at `s` (SCALES).
template <int L, int ROW_BYTES, bool SCALES>
__device__ __forceinline__ void lds_read_keys(u32x4 (&d)[2][L], float& ks, float& vs, uint32_t a, uint32_t s) {
  const uint32_t b = a ^ 64;   // the odd pieces of a row, every 128 bytes like the even ones
  if constexpr (L == 1)
    asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:%6\n\t"
                 "ds_read_b32 %2, %5\n\tds_read_b32 %3, %5 offset:128\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d[0][0]), "=&v"(d[1][0]), "=&v"(ks), "=&v"(vs) : "v"(a), "v"(s), "n"(4 * ROW_BYTES) : "memory");
  if constexpr (L == 2 && SCALES)
    asm volatile("ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\tds_read_b128 %2, %6 offset:%9\n\t"
                 "ds_read_b128 %3, %7 offset:%9\n\tds_read_b32 %4, %8\n\tds_read_b32 %5, %8 offset:128\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(d[0][0]), "=&v"(d[0][1]), "=&v"(d[1][0]), "=&v"(d[1][1]), "=&v"(ks), "=&v"(vs)
                 : "v"(a), "v"(b), "v"(s), "n"(4 * ROW_BYTES) : "memory");
  if constexpr (L == 2 && !SCALES)
    asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %4 offset:%6\n\t"
                 "ds_read_b128 %3, %5 offset:%6\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d[0][0]), "=&v"(d[0][1]), "=&v"(d[1][0]), "=&v"(d[1][1]) : "v"(a), "v"(b), "n"(4 * ROW_BYTES)
                 : "memory");
  if constexpr (L == 4 && SCALES)
    asm volatile("ds_read_b128 %0, %10\n\tds_read_b128 %1, %11\n\tds_read_b128 %2, %10 offset:128\n\t"
                 "ds_read_b128 %3, %11 offset:128\n\tds_read_b128 %4, %10 offset:%13\n\tds_read_b128 %5, %11 offset:%13\n\t"
                 "ds_read_b128 %6, %10 offset:%14\n\tds_read_b128 %7, %11 offset:%14\n\t"
                 "ds_read_b32 %8, %12\n\tds_read_b32 %9, %12 offset:128\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d[0][0]), "=&v"(d[0][1]), "=&v"(d[0][2]), "=&v"(d[0][3]), "=&v"(d[1][0]), "=&v"(d[1][1]),
                   "=&v"(d[1][2]), "=&v"(d[1][3]), "=&v"(ks), "=&v"(vs)
                 : "v"(a), "v"(b), "v"(s), "n"(4 * ROW_BYTES), "n"(4 * ROW_BYTES + 128) : "memory");
  if constexpr (L == 4 && !SCALES)
    asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %8 offset:128\n\t"
                 "ds_read_b128 %3, %9 offset:128\n\tds_read_b128 %4, %8 offset:%10\n\tds_read_b128 %5, %9 offset:%10\n\t"
                 "ds_read_b128 %6, %8 offset:%11\n\tds_read_b128 %7, %9 offset:%11\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d[0][0]), "=&v"(d[0][1]), "=&v"(d[0][2]), "=&v"(d[0][3]), "=&v"(d[1][0]), "=&v"(d[1][1]),
                   "=&v"(d[1][2]), "=&v"(d[1][3])
                 : "v"(a), "v"(b), "n"(4 * ROW_BYTES), "n"(4 * ROW_BYTES + 128) : "memory");
  if constexpr (L == 8)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %8 offset:128\n\t"
                   "ds_read_b128 %3, %9 offset:128\n\tds_read_b128 %4, %8 offset:256\n\tds_read_b128 %5, %9 offset:256\n\t"
                   "ds_read_b128 %6, %8 offset:384\n\tds_read_b128 %7, %9 offset:384\n\ts_waitcnt lgkmcnt(0)"
                   : "=&v"(d[h][0]), "=&v"(d[h][1]), "=&v"(d[h][2]), "=&v"(d[h][3]), "=&v"(d[h][4]), "=&v"(d[h][5]),
                     "=&v"(d[h][6]), "=&v"(d[h][7])
                   : "v"(a + h * 4 * ROW_BYTES), "v"(b + h * 4 * ROW_BYTES) : "memory");
}

// Hands three numbers of each key (by the lane of its number, at `to`) to the lanes that need
// them, 8 keys' from `from` on, and reads the first fragments of Q, 1 KiB apart from `qa` on.
__device__ __forceinline__ void lds_share(u32x4 (&d)[6], u32x4 (&q)[2], uint32_t to, float x, float y, float z,
                                          uint32_t from, uint32_t qa) {
  asm volatile("ds_write_b32 %8, %9\n\tds_write_b32 %8, %10 offset:128\n\tds_write_b32 %8, %11 offset:256\n\t"
               "ds_read_b128 %6, %13\n\tds_read_b128 %7, %13 offset:1024\n\t"
               "ds_read_b128 %0, %12\n\tds_read_b128 %1, %12 offset:16\n\tds_read_b128 %2, %12 offset:128\n\t"
               "ds_read_b128 %3, %12 offset:144\n\tds_read_b128 %4, %12 offset:256\n\tds_read_b128 %5, %12 offset:272\n\t"
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(d[4]), "=&v"(d[5]),
                 "=&v"(q[0]), "=&v"(q[1])
               : "v"(to), "v"(x), "v"(y), "v"(z), "v"(from), "v"(qa) : "memory");
}
__device__ __forceinline__ void lds_share(u32x4 (&d)[6], u32x4 (&q)[4], uint32_t to, float x, float y, float z,
                                          uint32_t from, uint32_t qa) {
  asm volatile("ds_write_b32 %10, %11\n\tds_write_b32 %10, %12 offset:128\n\tds_write_b32 %10, %13 offset:256\n\t"
               "ds_read_b128 %6, %15\n\tds_read_b128 %7, %15 offset:1024\n\tds_read_b128 %8, %15 offset:2048\n\tds_read_b128 %9, %15 offset:3072\n\t"
               "ds_read_b128 %0, %14\n\tds_read_b128 %1, %14 offset:16\n\tds_read_b128 %2, %14 offset:128\n\t"
               "ds_read_b128 %3, %14 offset:144\n\tds_read_b128 %4, %14 offset:256\n\tds_read_b128 %5, %14 offset:272\n\t"
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(d[4]), "=&v"(d[5]),
                 "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3])
               : "v"(to), "v"(x), "v"(y), "v"(z), "v"(from), "v"(qa) : "memory");
}
__device__ __forceinline__ void lds_share(u32x4 (&d)[6], u32x4 (&q)[6], uint32_t to, float x, float y, float z,
                                          uint32_t from, uint32_t qa) {
  asm volatile("ds_write_b32 %12, %13\n\tds_write_b32 %12, %14 offset:128\n\tds_write_b32 %12, %15 offset:256\n\t"
               "ds_read_b128 %6, %17\n\tds_read_b128 %7, %17 offset:1024\n\tds_read_b128 %8, %17 offset:2048\n\tds_read_b128 %9, %17 offset:3072\n\tds_read_b128 %10, %17 offset:4096\n\tds_read_b128 %11, %17 offset:5120\n\t"
               "ds_read_b128 %0, %16\n\tds_read_b128 %1, %16 offset:16\n\tds_read_b128 %2, %16 offset:128\n\t"
               "ds_read_b128 %3, %16 offset:144\n\tds_read_b128 %4, %16 offset:256\n\tds_read_b128 %5, %16 offset:272\n\t"
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(d[4]), "=&v"(d[5]),
                 "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3]), "=&v"(q[4]), "=&v"(q[5])
               : "v"(to), "v"(x), "v"(y), "v"(z), "v"(from), "v"(qa) : "memory");
}

// Waits until at most N loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "");
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// A lane's share of a tile, as read from LDS.
template <int FMT, int D>
struct AttnTile {
  using S = AttnShape<FMT, D, 1>;
  u32x4 k[2][S::kLoadsK];
  uint32_t v[8][S::kWordsV];
  // of keys 8 g + 0..7 in the 8-bit formats: the key's scale times the softmax's, log2 of the
  // value's scale and its reciprocal
  float kc[8], lz[8], iz[8];
};

template <int FMT, int D, int NR>
struct AttnWave {
  using S = AttnShape<FMT, D, NR>;
  const PagedCache& cache;
  const int32_t* table;       // this sequence's page table
  int head, lane, li, g;
  uint32_t keys, context;     // all of the sequence's keys; those every node sees
  float scale;                // of the scores, times log2 e
  bool once;                  // one workgroup of rows: keys and values are read by it alone
  uint64_t mask[NR];
  f32x4 o[S::kJ][NR];
  float m[NR], l[NR];
  float qs[NR];           // int8: -128 sum(q), for the codes' bias
  uint32_t tile0, step, tiles;   // this wave's tiles: tile0 + i * step, i < tiles
  char* ring;                    // its LDS: kDepth slots of {keys, values, scales}
  uint32_t ring_at, q_at;        // LDS addresses of the same, and of this lane's piece of Q
  uint32_t page;                 // pages of 32 tiles ahead: lane 2 i + h has half h of tile i's
  uint32_t fetch;                // byte offset of this lane's piece in a load's rows
  uint32_t read_k, read_v[4];    // LDS offsets of this lane's first pieces in a slot

  static __device__ __forceinline__ uint32_t lds_address(const char* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(p)));
  }

  __device__ __forceinline__ void begin(uint32_t first, uint32_t end, uint32_t every, const char* q, char* slots) {
    tile0 = first;
    step = every;
    tiles = first < end ? (end - first + every - 1) / every : 0;
    ring = slots;
    ring_at = lds_address(slots);
    q_at = lds_address(q) + 16u * lane;
    const int r = lane / S::kPieces;
    fetch = uint32_t(r * S::kRowBytes + ((lane % S::kPieces) ^ swizzle<S::kRowBytes>(r)) * 16);
    const int rk = 8 * (li >> 2) + (li & 3);
    read_k = uint32_t(rk * S::kRowBytes + (g ^ swizzle<S::kRowBytes>(rk)) * 16);
    constexpr int kBytes = 4 * S::kWordsV;   // of a value row a lane takes
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int rv = 8 * g + x;
      read_v[x] = uint32_t(rv * S::kRowBytes + ((li * kBytes / 16) ^ swizzle<S::kRowBytes>(rv)) * 16 + li * kBytes % 16);
    }
  }

  __device__ __forceinline__ void load_pages(uint32_t i) {
    const uint32_t last = uint32_t(cache.table_width) - 1;
    const uint32_t key = (tile0 + (i + (uint32_t(lane) >> 1)) * step) * kTileKeys + 16u * (lane & 1);
    page = uint32_t(table[min(key >> cache.page_shift, last)]);
  }

  // The cache row where half h of tile i starts (a tile's halves may be in two pages).
  __device__ __forceinline__ int64_t half_row(uint32_t i, int h) const {
    uint32_t block = __builtin_amdgcn_readlane(page, int(2 * (i & 31)) + h);
    block = min(block, cache.blocks - 1u);   // a bad entry reads some page of the cache
    const uint32_t key = (tile0 + i * step) * kTileKeys + 16u * h;
    return ((int64_t(block) * cache.kv_heads + head) << cache.page_shift) + (key & ((1u << cache.page_shift) - 1u));
  }

  typedef __attribute__((address_space(3))) void lds_void;
  typedef __attribute__((address_space(1))) const void global_void;

  // 16 bytes of each lane's own address to 1 KiB of LDS, in lane order.
  static __device__ __forceinline__ void start_piece(const void* from, void* to) {
    __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)to, 16, 0, 0);
  }

  // The J-th and later loads of a half's rows, 1024 bytes each.
  template <int J, int POLICY>
  __device__ __forceinline__ void start_rows(const char* from, char* to, int h) const {
    if constexpr (J < S::kLoads / 2) {
      const uint32_t piece = fetch ^ uint32_t(swizzle<S::kRowBytes>(16 * h + J * S::kLoadRows) * 16);
      __builtin_amdgcn_global_load_lds((global_void*)(from + J / 4 * 4096 + piece), (lds_void*)(to + J / 4 * 4096), 16,
                                       J % 4 * 1024, POLICY);
      start_rows<J + 1, POLICY>(from, to, h);
    }
  }

  // Starts the loads of a tile's keys (with both scales) or values into its slot.
  template <bool KEYS>
  __device__ __forceinline__ void start(uint32_t i, uint32_t slot) {
    if (KEYS && (i & 31) == 0 && i > 0) load_pages(i);
    const int64_t row[2] = {half_row(i, 0), half_row(i, 1)};
    char* to = ring + slot * S::kSlotBytes + (KEYS ? 0 : S::kSideBytes);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // a half's rows follow each other in memory as in LDS: one base and an offset of both
      const char* from = (KEYS ? cache.k : cache.v) + row[h] * S::kRowBytes;
      // Read once, they need not stay in the caches: 2 x 131071 int8 tokens 120 -> 110 us. With
      // several workgroups of rows they are read again, from L2.
      if (once)
        start_rows<0, kNonTemporal>(from, to + h * 16 * S::kRowBytes, h);
      else
        start_rows<0, 0>(from, to + h * 16 * S::kRowBytes, h);
    }
    if constexpr (KEYS && FMT != NM_KV_FP16) {
      const float* s = lane < 32 ? cache.k_scale : cache.v_scale;
      const float* from = s + ((lane & 16) ? row[1] : row[0]) + (lane & 15);
      __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)(ring + slot * S::kSlotBytes + 2 * S::kSideBytes), 4, 0, 0);
    }
  }

  // Waits for a tile's keys (values): all loads started after them may still be in flight,
  // those of min(kDepth, left) tiles in all, the last of which may lack its values.
  template <int N>
  static __device__ __forceinline__ void wait_keys(uint32_t left) {
    if constexpr (N > 1) {
      if (left < N) return wait_keys<N - 1>(left);
    }
    wait_loads<N * S::kTileLoads - S::kLoads - S::kScaleLoads>();
  }
  template <int N>
  static __device__ __forceinline__ void wait_values(uint32_t after) {
    if constexpr (N > 0) {
      if (after < N) return wait_values<N - 1>(after);
    }
    wait_loads<N * S::kTileLoads - (N == S::kDepth && N > 0 ? S::kLoads : 0)>();
  }

  static constexpr int kGroup = NR == 1 ? (S::kSteps < 4 ? S::kSteps : 4) : NR < 4 ? 2 : 1;   // steps of Q read at a time

  // A tile's keys, the first group of Q, and what the scores need of the scales, worked out once
  // a key and handed round through LDS in place of the scales. Returns the keys, a bit each of
  // this lane's 8, whose value's scale is not a number (edge tiles; elsewhere it makes NaN by
  // itself).
  __device__ __forceinline__ uint32_t read_keys(AttnTile<FMT, D>& t, u32x4 (&q)[NR * kGroup], uint32_t slot, bool edge) const {
    const uint32_t base = ring_at + slot * S::kSlotBytes, shared = base + 2 * S::kSideBytes, mine = shared + 4 * (lane & 31);
    float ks = 0.f, vs = 0.f;
    lds_read_keys<S::kLoadsK, S::kRowBytes, FMT != NM_KV_FP16>(t.k, ks, vs, base + read_k, mine);
    if constexpr (FMT == NM_KV_FP16) {
      lds_read_fragments(q, q_at);
      return 0;
    } else {
      uint32_t bad = 0;
      if (edge) {
        const bool b = !(vs < __builtin_inff());
        bad = uint32_t(__ballot(b)) >> (8 * g) & 0xFFu;
        if (b) vs = 1.0f;
      }
      vs = vs < kLeastScale ? kLeastScale : vs;   // NaN stays
      u32x4 d[6];
      lds_share(d, q, mine, ks * scale, __builtin_amdgcn_logf(vs), __builtin_amdgcn_rcpf(vs), shared + 32 * g, q_at);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t.kc[e] = __uint_as_float(d[e >> 2][e & 3]);
        t.lz[e] = __uint_as_float(d[2 + (e >> 2)][e & 3]);
        t.iz[e] = __uint_as_float(d[4 + (e >> 2)][e & 3]);
      }
      return bad;
    }
  }

  __device__ __forceinline__ void read_values(AttnTile<FMT, D>& t, uint32_t slot) const {
    const uint32_t base = ring_at + slot * S::kSlotBytes + S::kSideBytes;
    uint32_t at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) at[x] = base + read_v[x];
    if constexpr (S::kWordsV == 1) {
      uint32_t d[8];
      lds_read_rows<4 * S::kRowBytes>(d, at);
#pragma unroll
      for (int e = 0; e < 8; ++e) t.v[e][0] = d[e];
    } else if constexpr (S::kWordsV == 2) {
      u32x2 d[8];
      lds_read_rows<4 * S::kRowBytes>(d, at);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t.v[e][0] = d[e][0];
        t.v[e][1] = d[e][1];
      }
    } else {
#pragma unroll
      for (int c = 0; c < S::kWordsV / 4; ++c) {
        u32x4 d[8];
        lds_read_rows<4 * S::kRowBytes>(d, at);
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) t.v[e][4 * c + i] = d[e][i];
#pragma unroll
        for (int x = 0; x < 4; ++x) at[x] ^= 16;   // the other half of a 32-byte run
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
        if constexpr (FMT == NM_KV_INT8) {
          w[0][p] = unbiased(__builtin_amdgcn_perm(b, a, 0x0C040C00u));
          w[1][p] = unbiased(__builtin_amdgcn_perm(b, a, 0x0C050C01u));
          w[2][p] = unbiased(__builtin_amdgcn_perm(b, a, 0x0C060C02u));
          w[3][p] = unbiased(__builtin_amdgcn_perm(b, a, 0x0C070C03u));
        } else {
          const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x05010400u), hi = __builtin_amdgcn_perm(b, a, 0x07030602u);
          w[0][p] = pair_of<FMT>(lo, false);
          w[1][p] = pair_of<FMT>(lo, true);
          w[2][p] = pair_of<FMT>(hi, false);
          w[3][p] = pair_of<FMT>(hi, true);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 4 / S::kCodeBytes; ++x) f[x] = as_half8(w[x]);
  }

  // The scores of a tile in units of log2, with log2 z: x[n][e] is this lane's row n, key 8 g + e.
  __device__ __forceinline__ void scores(const AttnTile<FMT, D>& t, u32x4 (&q)[NR * kGroup], float (&x)[NR][8]) const {
    f32x4 s[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) s[n][0] = s[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s0 = 0; s0 < S::kSteps; s0 += kGroup) {
      if (s0 > 0) lds_read_fragments(q, q_at + s0 * NR * 1024);
#pragma unroll
      for (int u = 0; u < kGroup; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int st = s0 + u;
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
            s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(f16x8, q[u * NR + n]), s[n][h], 0, 0, 0);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float y = FMT == NM_KV_INT8 ? s[n][e >> 2][e & 3] + qs[n] : s[n][e >> 2][e & 3];
        x[n][e] = FMT == NM_KV_FP16 ? y * scale : fmaf(y, t.kc[e], t.lz[e]);
      }
  }

  // -128 times each row's sum of q, in the products' unit (a product with ones gives every lane
  // its row's sum).
  __device__ __forceinline__ void sum_queries() {
    if constexpr (FMT != NM_KV_INT8) return;
    f16x8 ones;
#pragma unroll
    for (int e = 0; e < 8; ++e) ones[e] = _Float16(1.0f);
    f32x4 sum[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) sum[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s0 = 0; s0 < S::kSteps; s0 += kGroup) {
      u32x4 q[NR * kGroup];
      lds_read_fragments(q, q_at + s0 * NR * 1024);
#pragma unroll
      for (int x = 0; x < NR * kGroup; ++x)
        sum[x % NR] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, __builtin_bit_cast(f16x8, q[x]), sum[x % NR], 0, 0, 0);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) qs[n] = sum[n][0] * (-kCodeBias / kCodeUnit);
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
  // keys that not every node sees, or that are past the end; bad: keys, a bit each, that make the
  // rows that see them NaN (a scale that is not a number does too).
  __device__ __forceinline__ void weights(const AttnTile<FMT, D>& t, float (&x)[NR][8], f16x8 (&w)[NR], bool edge,
                                          uint32_t bad, uint32_t key0) {
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
      grows |= top[n] > m[n] + (kLift + kLag);
    }
    if (__any(grows)) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float next = fmaxf(m[n], max4(top[n]) - kLift);
        const float f = exp2_fast(m[n] - next);
        m[n] = next;
        l[n] *= f;
#pragma unroll
        for (int j = 0; j < S::kJ; ++j) o[j][n] *= f;
      }
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = exp2_fast(x[n][e] - m[n]);
        // fp16: the sum is of the weights as rounded, so that a weighted mean of equal values is
        // exact; with 8-bit codes, whose own rounding is coarser, that took 4% longer at 64 nodes
        if constexpr (FMT != NM_KV_FP16) l[n] = fmaf(y, t.iz[e], l[n]);
        w[n][e] = _Float16(y);   // to nearest even: 2^-11 of the weight
        if constexpr (FMT == NM_KV_FP16) l[n] += float(w[n][e]);
      }
    }
  }

  // Values of an edge tile: those past the end, which were never written and may be NaN, become
  // 0, since 0 times them is not; so does a draft's row with an infinity or NaN in it (an fp16, or
  // an e4m3 code, which no append writes but a caller's own tensor may hold), whose key is returned
  // as a bit: the rows that see it are NaN, the others must not be.
  __device__ __forceinline__ uint32_t edge_values(AttnTile<FMT, D>& t, uint32_t key0) const {
    uint32_t bad = 0;
    if constexpr (FMT != NM_KV_INT8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t any = 0;
#pragma unroll
        for (int c = 0; c < S::kWordsV; ++c) any |= non_finite<FMT>(t.v[e][c]);
        bad |= uint32_t(any != 0 && key0 + e >= context) << e;
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) bad |= __shfl_xor(bad, o);   // over the row's lanes
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t held = key0 + e < keys && !((bad >> e) & 1) ? ~0u : 0u;
#pragma unroll
      for (int c = 0; c < S::kWordsV; ++c) t.v[e][c] &= held;
    }
    return bad;
  }

  // O^T += V^T P^T.
  __device__ __forceinline__ void product(const AttnTile<FMT, D>& t, const f16x8 (&w)[NR]) {
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
  keys = uint32_t(c + count < 0 ? 0 : c + count > most ? most : c + count);
}

// Tiles of a sequence's chunk: `per`, more where that would make more than `most` chunks, or where
// the last of c chunks would spend longer on the partial results (c of them) than on its tiles (a
// c-th of the sequence's): join is what a partial costs in tiles. (us without, with join at half,
// once, twice a partial's bytes over a tile's, and at 4 times: 4 x 4 nodes over 16384 e4m3 tokens
// of 256 40.8, 37.9, 38.1, 33.0, 34.2; 2 x 5 over 16384 int8 tokens of 64 26.8, 23.3, 23.0, 22.6,
// 26.1; 2 x 8 over 131071 int8 tokens 104, 104, 104, 103 to 105, 120. It is set at twice.)
__device__ __forceinline__ uint32_t chunk_tiles(uint32_t tiles, uint32_t per, uint32_t most, float join) {
  const uint32_t least = (tiles + most * kAttnWaves - 1) / (most * kAttnWaves) * kAttnWaves;
  const uint32_t even = uint32_t(__builtin_amdgcn_sqrtf(float(tiles) * join) * (1.0f / kAttnWaves) + 0.999f) * kAttnWaves;
  const uint32_t size = max(max(per, least), even);
  // two chunks of that are not worth their join: 5 trees of 34 nodes over up to 569 int8 tokens, 32
  // heads, 21.8 us whole and 26.9 cut; 3 of 26 over 248 14.9 and 19.4
  return tiles <= 2 * even ? max(tiles, size) : size;
}
__device__ __forceinline__ uint32_t chunks_of(uint32_t tiles, uint32_t per) {
  return tiles <= per ? 1u : (tiles + per - 1) / per;
}

// Inclusive sums over the wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // the row before's last, rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // the first half's last, rows 2 and 3
  return x;
}

// Every wave works this out for itself: 64 sequences a pass, one a lane; the first 64 stay in
// registers.
__device__ __forceinline__ AttnChunk find_chunk(const AttnCall& a, int slots, int slot, uint32_t most, float join) {
  const int lane = threadIdx.x & 63;
  struct Lengths {
    uint32_t context, keys, tiles;   // tiles: at most 2^25
    int count;
  };
  const auto load = [&](int b) {
    Lengths x{0, 0, 0, 0};
    if (b < a.batch) {
      attn_lengths(a, b, x.context, x.keys, x.count);
      x.tiles = (x.keys + kTileKeys - 1) / kTileKeys;
    }
    return x;
  };
  const Lengths front = load(lane);
  const auto at_group = [&](int b0) { return b0 == 0 ? front : load(b0 + lane); };
  uint32_t per = 0x7FFFFFFFu;
  if (slots > a.batch) {
    uint64_t total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64)
      total += uint32_t(__builtin_amdgcn_readlane(wave_scan(at_group(b0).tiles), 63));
    // The smallest chunk, in whole rounds of the waves, whose number fits the slots: steps of a
    // 32nd up from an even split, and from there to one slot a sequence set aside, which always
    // fits. (The sums are below 2^41, exact in 64-bit floats.)
    const double round = 1.0 / kAttnWaves;
    per = max(uint32_t(ceil(double(total) / slots * round)) * kAttnWaves, uint32_t(kMinChunkTiles));
    for (int tries = 0;; ++tries) {
      uint32_t used = 0;
      for (int b0 = 0; b0 < a.batch; b0 += 64)
        used += uint32_t(__builtin_amdgcn_readlane(
            wave_scan(b0 + lane < a.batch ? chunks_of(at_group(b0).tiles, per) : 0u), 63));
      if (used <= uint32_t(slots)) break;
      if (tries == 8) {
        per = uint32_t(ceil(double(total) / (slots - a.batch) * round)) * kAttnWaves;
        break;
      }
      per += (per / 32 + kAttnWaves) / kAttnWaves * kAttnWaves;
    }
  }
  AttnChunk k;
  k.b = -1;
  int before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const Lengths x = at_group(b0);
    uint32_t mine = per;
    int n = 0;
    if (b0 + lane < a.batch) {
      if (slots > a.batch) {   // as many chunks as `per` asks for, of even size
        n = int(chunks_of(x.tiles, chunk_tiles(x.tiles, per, most, join)));
        mine = max((x.tiles + n * kAttnWaves - 1) / (n * kAttnWaves), 1u) * kAttnWaves;
      }
      n = int(chunks_of(x.tiles, mine));
    }
    const uint32_t upto = wave_scan(uint32_t(n));
    const uint64_t past = __ballot(before + int(upto) > slot);
    if (past != 0) {
      const int at = __builtin_ctzll(past);
      k.b = b0 + at;
      k.chunks = __builtin_amdgcn_readlane(n, at);
      k.first = before + int(__builtin_amdgcn_readlane(upto, at)) - k.chunks;
      k.tiles = __builtin_amdgcn_readlane(mine, at);
      k.context = __builtin_amdgcn_readlane(x.context, at);
      k.keys = __builtin_amdgcn_readlane(x.keys, at);
      k.count = __builtin_amdgcn_readlane(x.count, at);
      return k;
    }
    before += int(__builtin_amdgcn_readlane(upto, 63));
  }
  return k;
}

template <int FMT, int D, int NR>
__global__ __launch_bounds__(kAttnThreads, (AttnShape<FMT, D, NR>::kWaves)) void attention_kernel(AttnCall a, AttnSplit sp) {
  using S = AttnShape<FMT, D, NR>;
  extern __shared__ __align__(16) char lds[];
  f32x4(*xch)[kAttnWaves * S::kPer][64] = reinterpret_cast<f32x4(*)[kAttnWaves * S::kPer][64]>(lds + S::kTilesAt);
  float(*stat_m)[16 * NR] = reinterpret_cast<float(*)[16 * NR]>(lds + S::kStatAt);
  float(*stat_l)[16 * NR] = stat_m + kAttnWaves;
  uint32_t* arrived = reinterpret_cast<uint32_t*>(stat_l + kAttnWaves);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = int(blockIdx.x) % a.cache.kv_heads, slot = int(blockIdx.x) / a.cache.kv_heads;
  const int rt = blockIdx.y;
  AttnChunk ck = find_chunk(a, sp.slots, slot, S::kMaxChunks, sp.join);
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
  w.once = sp.row_tiles == 1;
  w.scale = a.scale * 1.44269504088896341f * (FMT == NM_KV_INT8 ? kCodeUnit : 1.0f);
  const int rows = a.tokens * a.group;
  // the nodes' rows: t = r / group, query head head * group + r % group
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = (rt * NR + n) * 16 + w.li, t = r / a.group;
    const bool live = r < rows && t < count;
    uint64_t mk = 0;
    if (live) mk = a.mask != nullptr ? a.mask[int64_t(b) * a.tokens + t] : t >= 63 ? ~0ull : (2ull << t) - 1;
    // nodes past the page table's end are not there: their tile may reach further than the keys
    const uint32_t held = w.keys - w.context;
    w.mask[n] = held >= 64 ? mk : mk & ((1ull << held) - 1);
    w.m[n] = kLowest;
    w.l[n] = 0.f;
#pragma unroll
    for (int j = 0; j < S::kJ; ++j) w.o[j][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // this chunk's tiles, every fourth a wave's; kDepth of them in flight into the wave's own part
  // of LDS, whose keys and values are fetched again as soon as they are read
  const uint32_t all = (w.keys + kTileKeys - 1) / kTileKeys;
  const uint32_t begin = uint32_t(slot - first) * per;   // per <= 2^31 - 1, begin <= all
  w.begin(begin + wave, min(all, begin + per), kAttnWaves, lds, lds + S::kTilesAt + wave * S::kWaveBytes);
  // Q, in operand order: every wave loads its share of the (row tile, step) fragments. Rows past
  // the last node's repeat row 0: nothing of theirs is stored.
#pragma unroll
  for (int f = 0; f < (NR * S::kSteps + kAttnWaves - 1) / kAttnWaves; ++f) {
    const int x = f * kAttnWaves + wave, fn = x % NR, st = x / NR;
    if (x >= NR * S::kSteps) break;
    int r = (rt * NR + fn) * 16 + w.li;
    r = r < rows ? r : 0;
    const int d = FMT == NM_KV_FP16 ? 32 * st + 8 * w.g : 64 * (st >> 1) + 16 * w.g + 8 * (st & 1);
    const uint16_t* from = a.q + (int64_t(b) * a.tokens + r / a.group) * a.q_stride +
                           int64_t(head * a.group + r % a.group) * D + d;
    w.start_piece(from, lds + x * 1024);
  }
  if (w.tiles > 0) w.load_pages(0);
  for (uint32_t i = 0; i < uint32_t(S::kDepth) && i < w.tiles; ++i) {
    w.template start<true>(i, i);
    w.template start<false>(i, i);
  }
  if (w.tiles >= uint32_t(S::kDepth))
    wait_loads<S::kDepth * S::kTileLoads>();
  else
    wait_loads<0>();
  __builtin_amdgcn_s_barrier();   // all of Q has arrived
  if (w.tiles > 0) {
    w.sum_queries();
    uint32_t slot_i = 0;
    for (uint32_t i = 0; i < w.tiles; ++i) {
      const uint32_t tile = w.tile0 + i * w.step, key0 = tile * kTileKeys + 8u * w.g, left = w.tiles - i;
      const bool edge = (tile + 1) * kTileKeys > w.context;
      AttnTile<FMT, D> t;
      float x[NR][8];
      f16x8 y[NR];
      w.template wait_keys<S::kDepth>(left);
      u32x4 q[NR * AttnWave<FMT, D, NR>::kGroup];
      uint32_t bad = w.read_keys(t, q, slot_i, edge);
      if (left > uint32_t(S::kDepth)) w.template start<true>(i + S::kDepth, slot_i);
      w.scores(t, q, x);
      if (edge) {
        w.template wait_values<S::kDepth>(left - 1);
        w.read_values(t, slot_i);
        bad |= w.edge_values(t, key0);
      }
      w.weights(t, x, y, edge, bad, key0);
      if (!edge) {
        w.template wait_values<S::kDepth>(left - 1);
        w.read_values(t, slot_i);
      }
      if (left > uint32_t(S::kDepth)) w.template start<false>(i + S::kDepth, slot_i);
      w.product(t, y);
      slot_i = slot_i + 1 == uint32_t(S::kDepth) ? 0 : slot_i + 1;
    }
  }
  __syncthreads();   // the waves' tiles are done with: the exchange takes their LDS

  // the waves' results together: each scaled to the common reference, then every wave adds up
  // its share of the (row tile, d tile) units over the waves in order
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    w.l[n] = sum4(w.l[n]);
    if constexpr (FMT == NM_KV_INT8) {   // O in its own unit
#pragma unroll
      for (int j = 0; j < S::kJ; ++j) w.o[j][n] *= kCodeUnit;
    }
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
  if (tid == 0) *arrived = atomicAdd(counter, 1u);
  __syncthreads();
  if (*arrived != uint32_t(chunks - 1)) return;
  if (tid == 0) atomicExch(counter, 0u);
  // The last of the sequence's chunks: all partials are complete. First the rows' common
  // references and sums, and what each chunk's partial is worth against them.
  float* sum = reinterpret_cast<float*>(lds + S::kTilesAt);                        // [group][row][d]
  float* factor = reinterpret_cast<float*>(lds + S::kTilesAt + S::kSumBytes);      // [chunk][row]
  const int r0 = tid % live, s0 = tid / live;
  if (s0 < S::kRowThreads) {
    float m1 = kLowest, l1 = 0.f;
    u32x2 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k * S::kRowThreads < chunks)
        x[k] = __builtin_amdgcn_raw_buffer_load_b64(buf, (s0 + k * S::kRowThreads) * stride + r0 * 8, 0, kCoherent);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k * S::kRowThreads < chunks) m1 = fmaxf(m1, __uint_as_float(x[k][0]));
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k * S::kRowThreads < chunks) {
        const float f = exp2_fast(__uint_as_float(x[k][0]) - m1);
        l1 += __uint_as_float(x[k][1]) * f;
        factor[(s0 + k * S::kRowThreads) * live + r0] = f;
      }
    reinterpret_cast<float2*>(sum)[s0 * live + r0] = make_float2(m1, l1);
  }
  __syncthreads();
  float f0 = 0.f;   // of this thread's chunks, from its own reference to the row's
  if (s0 < S::kRowThreads) {
    const float2* part = reinterpret_cast<const float2*>(sum);
    float m1 = kLowest, l1 = 0.f;
#pragma unroll
    for (int x = 0; x < S::kRowThreads; ++x) m1 = fmaxf(m1, part[x * live + r0].x);
#pragma unroll
    for (int x = 0; x < S::kRowThreads; ++x) l1 += part[x * live + r0].y * exp2_fast(part[x * live + r0].x - m1);
    f0 = exp2_fast(part[s0 * live + r0].x - m1);
    if (s0 == 0) stat_l[0][r0] = l1;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k * S::kRowThreads < chunks) factor[(s0 + k * S::kRowThreads) * live + r0] *= f0;
  }
  __syncthreads();
  // Then the partials, 16 bytes a unit: a thread takes units of every `groups`-th chunk, as many
  // loads in flight as it has registers for; the groups' sums and the rows come together in LDS.
  // The order is fixed, so the result is the same each time.
  const int groups = units < kAttnThreads ? kAttnThreads / units : 1, grp = groups > 1 ? tid / units : 0;
  const auto join = [&](auto units_at_once, auto chunks_at_once) {
    constexpr int UU = decltype(units_at_once)::value, CC = decltype(chunks_at_once)::value;
    for (int u0 = groups > 1 ? tid - grp * units : tid; u0 < units && grp < groups; u0 += kAttnThreads * UU) {
      f32x4 acc[UU];
#pragma unroll
      for (int v = 0; v < UU; ++v) acc[v] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int c0 = grp; c0 < chunks; c0 += groups * CC) {
        u32x4 y[UU][CC];
#pragma unroll
        for (int x = 0; x < CC; ++x)
          if (c0 + x * groups < chunks)
#pragma unroll
            for (int v = 0; v < UU; ++v)
              if (v == 0 || u0 + v * kAttnThreads < units)
                y[v][x] = __builtin_amdgcn_raw_buffer_load_b128(
                    buf, (c0 + x * groups) * stride + kStats + (u0 + v * kAttnThreads) * 16, 0, kCoherent);
#pragma unroll
        for (int x = 0; x < CC; ++x)
          if (c0 + x * groups < chunks)
#pragma unroll
            for (int v = 0; v < UU; ++v)
              acc[v] += __builtin_bit_cast(f32x4, y[v][x]) * factor[(c0 + x * groups) * live + (u0 + v * kAttnThreads) % live];
      }
#pragma unroll
      for (int v = 0; v < UU; ++v) {
        const int u = u0 + v * kAttnThreads;
        if (u >= units) break;
        const int r = u % live, jg = u / live;
        float* at = sum + (grp * live + r) * D + S::kJ * 4 * (jg & 3) + (jg >> 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) at[S::kJ * i] = acc[v][i];
      }
    }
  };
  // (What fits the registers. us with 1 x 16, 4 x 4 and all of a thread's units, 24 loads: 20 rows
  // of 64, 2 x 16384 tokens 27.7, 30.7 and -; 40 rows of 128, 2 x 131071 tokens -, 109 and 103.5; 16
  // rows of 256, 4 x 16384 tokens 44.9, 40.5 and 41.0.)
  constexpr int kUnits = D > 128 ? 4 : NR * D / 64 > 1 ? NR * D / 64 : 2;   // of a thread, if all rows are live
  if (units <= 2 * kAttnThreads)
    join(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
  else
    join(std::integral_constant<int, kUnits>{}, std::integral_constant<int, (D > 128 ? 16 : 24) / kUnits>{});
  __syncthreads();
  for (int u = tid; u < live * (D / 8); u += kAttnThreads) {
    const int r = u / (D / 8), d = u % (D / 8) * 8, at = rt * NR * 16 + r, node = at / a.group;
    const float l1 = stat_l[0][r], inv = node < count && l1 != 0.f ? 1.0f / l1 : 0.f;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = 0.f;
      for (int x = 0; x < groups; ++x) y[e] += sum[(x * live + r) * D + d + e];
      y[e] = inv == 0.f ? 0.f : y[e] * inv;
    }
    *reinterpret_cast<u32x4*>(a.out + ((int64_t(b) * a.tokens + node) * a.heads + head * a.group + at % a.group) * D + d) =
        halves_of(y);
  }
}

}  // namespace nm
