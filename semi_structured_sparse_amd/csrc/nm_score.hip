// Log probabilities of given tokens, the entropy and the most likely tokens of rows of logits.
//
// Mathematics. With the row's maximum M, c = scale * log2 e and d = (M - x) c >= 0,
//   S = sum 2^-d over all but one element at M,   T = sum 2^-d d,
//   log p(x) = scale (x - M) - log1p(S),   entropy = ln2 (log2(1 + S) + T / (1 + S)),
// in one pass with a running M: where it grows by g, S becomes (S + 1) 2^-g (the old maximum joins the
// others) and T becomes 2^-g (T + g (S + 1)). Nothing cancels, and the maximum's own term never
// stands beside the small ones, so log p of a token that is nearly certain keeps its digits. M is a
// wave's, not a lane's, so that it grows a few times a row and the rare tile where it does takes a
// longer way.
//
// The best tokens: each lane keeps the largest value that it saw. The top-th largest of a workgroup's
// 256 is exceeded or met by at least `top` elements and by few more, and only the lanes whose largest
// meets it look at their elements again, which the caches still have. What they find is put in
// order by counting, for each, how many go before it.
//
// What bounds it: reading the logits once. A row goes to several workgroups where there are few rows;
// the last to arrive joins their sums and lists.
#include "nm_block_internal.h"
#include "nm_decode_internal.h"
#include "nm_epilogue.h"

namespace nm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kLoads = 4;                  // 16-byte loads of a tile a lane
constexpr int kMaxChunks = 32;             // workgroups of a row
constexpr int kMinChunk = 2048;            // elements
constexpr int kRoom = 2048;                // candidates for the best tokens
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kNone = -__builtin_inff();

typedef _Float16 halves __attribute__((ext_vector_type(8), aligned(2)));   // rows start at any element
typedef float floats __attribute__((ext_vector_type(4), aligned(4)));

template <bool HALF>
constexpr int kElements = HALF ? 8 : 4;    // of a load

// Where a row's workgroups leave their sums and lists, and each row's counter.
struct ScoreSplit {
  int chunks;
  int counter_step;
  uint32_t* counters;
  char* parts;             // kPartBytes a chunk
};
constexpr uint32_t kPartBytes = 16 + NM_MAX_TOP * 8;

struct Sums {
  float m, s, t;
};

// The order of the best: the larger value (-0 as 0), then the lower index; 0 is below them all.
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return uint64_t(b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u)) << 32 | uint32_t(~index);
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t b = uint32_t(key >> 32);
  return __uint_as_float(b >> 31 ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ int index_of(uint64_t key) { return int(~uint32_t(key)); }

// The sums of two sets; without a maximum (kNone) one holds nothing, or NaN.
__device__ __forceinline__ Sums joined(const Sums& a, const Sums& b, float c) {
  const bool first = a.m >= b.m;
  const Sums &hi = first ? a : b, &lo = first ? b : a;
  Sums r = hi;
  if (lo.m == kNone) {
    r.s += lo.s;
  } else {
    const float g = fminf((hi.m - lo.m) * c, 200.0f), f = __builtin_amdgcn_exp2f(-g);   // 2^-200 is 0
    r.s += f * (lo.s + 1.0f);
    r.t += f * fmaf(g, lo.s + 1.0f, lo.t);
  }
  return r;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// A lane's elements of a tile of kThreads * kLoads * kElements from `at` on: load u at
// at + (u * kThreads + tid) * kElements; kNone past `hi`.
template <bool HALF>
struct Part {
  static constexpr int E = kElements<HALF>;
  float x[kLoads * E];

  static __device__ __forceinline__ int index(int at, int u) { return at + (u * kThreads + int(threadIdx.x)) * E; }

  __device__ __forceinline__ void load(const void* row, int at, int hi) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = index(at, u);
      if constexpr (HALF) {
        const uint16_t* p = static_cast<const uint16_t*>(row);
        if (i + E <= hi) {
          const halves v = *reinterpret_cast<const halves*>(p + i);
#pragma unroll
          for (int e = 0; e < E; ++e) x[u * E + e] = float(v[e]);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) x[u * E + e] = i + e < hi ? half_at(p, size_t(i + e)) : kNone;
        }
      } else {
        const float* p = static_cast<const float*>(row);
        if (i + E <= hi) {
          const floats v = *reinterpret_cast<const floats*>(p + i);
#pragma unroll
          for (int e = 0; e < E; ++e) x[u * E + e] = v[e];
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) x[u * E + e] = i + e < hi ? p[i + e] : kNone;
        }
      }
    }
  }
  __device__ __forceinline__ float largest() const {
    float m = x[0];
#pragma unroll
    for (int e = 1; e < kLoads * E; ++e) m = fmaxf(m, x[e]);   // NaN aside: the sums find it
    return m;
  }
  // Adds the terms, relative to m; skip: the lane's first element at m is left out.
  template <bool SKIP>
  __device__ __forceinline__ void add(float m, float c, bool skip, float& s, float& t) const {
#pragma unroll
    for (int e = 0; e < kLoads * E; ++e) {
      const float d = (x[e] - m) * c;
      float f = __builtin_amdgcn_exp2f(d);
      if constexpr (SKIP) {
        if (skip && x[e] == m) {
          f = 0.0f;
          skip = false;
        }
      }
      s += f;
      t = fmaf(f, -fmaxf(d, -200.0f), t);   // 2^-200 is 0, and stays that beside an infinite d
    }
  }
};

struct Shared {
  uint64_t keys[kRoom];
  float largest[kThreads];
  Sums sums[kWaves];
  uint64_t best[kWaves];
  int counts[kWaves];
  uint32_t found;
  float limit;
  uint32_t arrived;
};

// Puts the `top` first of the n keys in sh.keys (all different) in order and calls put(rank, key).
template <typename Put>
__device__ __forceinline__ void in_order(const Shared& sh, int n, int top, Put put) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t mine = sh.keys[i];
    int before = 0;
    for (int j = 0; j < n; ++j) before += sh.keys[j] > mine ? 1 : 0;
    if (before < top) put(before, mine);
  }
}

// Where too many elements meet the limit (long runs of equal logits, or the largest ones in few
// lanes): the keys one after the other, each the largest below the one before.
template <bool HALF>
__device__ __forceinline__ int one_by_one(const void* row, int lo, int hi, int top, Shared& sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint64_t last = ~uint64_t(0);
  int n = 0;
  for (; n < top; ++n) {
    uint64_t best = 0;
    for (int i = lo + int(threadIdx.x); i < hi; i += kThreads) {
      const float x = HALF ? half_at(static_cast<const uint16_t*>(row), size_t(i)) : static_cast<const float*>(row)[i];
      if (x > kNone) {
        const uint64_t k = key_of(x, i);
        if (k < last && k > best) best = k;
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t other = uint64_t(__shfl_xor((unsigned long long)best, d));
      best = other > best ? other : best;
    }
    __syncthreads();   // the round before has read sh.best
    if (lane == 0) sh.best[wave] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) best = sh.best[w] > best ? sh.best[w] : best;
    if (best == 0) break;
    if (threadIdx.x == 0) sh.keys[n] = best;
    last = best;
  }
  __syncthreads();
  return n;
}

// Leaves the keys of at least the `top` best elements of the run in sh.keys; returns their number.
template <bool HALF>
__device__ __forceinline__ int candidates(const void* row, int lo, int hi, int top, float largest, Shared& sh) {
  constexpr int E = kElements<HALF>;
  const int tid = threadIdx.x;
  sh.largest[tid] = largest;
  if (tid == 0) {
    sh.found = 0;
    sh.limit = kNone;
  }
  __syncthreads();
  int before = 0;
  for (int j = 0; j < kThreads; ++j) {
    const float other = sh.largest[j];
    before += other > largest || (other == largest && j < tid) ? 1 : 0;
  }
  if (before == top - 1) sh.limit = largest;
  __syncthreads();
  const float limit = sh.limit;
  if (largest >= limit && largest > kNone) {
    for (int at = lo; at < hi; at += kThreads * kLoads * E) {
      Part<HALF> p;
      p.load(row, at, hi);
#pragma unroll
      for (int e = 0; e < kLoads * E; ++e) {
        if (p.x[e] >= limit && p.x[e] > kNone) {
          const uint32_t n = atomicAdd(&sh.found, 1u);
          if (n < kRoom) sh.keys[n] = key_of(p.x[e], Part<HALF>::index(at, e / E) + e % E);
        }
      }
    }
  }
  __syncthreads();
  const uint32_t n = sh.found;
  __syncthreads();
  return n <= kRoom ? int(n) : one_by_one<HALF>(row, lo, hi, top, sh);
}

template <bool HALF, bool TOP>
__global__ __launch_bounds__(kThreads) void score_kernel(ScoreCall a, ScoreSplit sp) {
  constexpr int E = kElements<HALF>, kTile = kThreads * kLoads * E;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r = int64_t(blockIdx.x) / sp.chunks;
  const int chunk = int(int64_t(blockIdx.x) - r * sp.chunks);
  const void* row = static_cast<const char*>(a.logits) + r * a.stride * (HALF ? 2 : 4);
  const int each = (a.vocab + sp.chunks - 1) / sp.chunks;
  const int lo = min(a.vocab, chunk * each), hi = min(a.vocab, lo + each);
  const float c = a.scale * kLog2e;

  // the wave's maximum, the lane's share of its sums, the lane's own maximum
  float m = kNone, s = 0.0f, t = 0.0f, largest = kNone;
  for (int at = lo; at < hi; at += kTile) {
    Part<HALF> p;
    p.load(row, at, hi);
    const float mine = p.largest();
    if (TOP) largest = fmaxf(largest, mine);
    if (__ballot(mine > m) != 0) {
      const float top = wave_max(mine);
      if (m > kNone) {
        const float g = fminf((top - m) * c, 200.0f), f = __builtin_amdgcn_exp2f(-g);
        if (lane == 0) s += 1.0f;
        t = f * fmaf(g, s, t);
        s *= f;
      }
      m = top;
      const bool skip = lane == __builtin_ctzll(__ballot(mine == m));
      p.template add<true>(m, c, skip, s, t);
    } else {
      p.template add<false>(m > kNone ? m : 0.0f, c, false, s, t);
    }
  }
  Sums all{m, wave_sum(s), wave_sum(t)};
  if (lane == 0) sh.sums[wave] = all;
  __syncthreads();
  all = sh.sums[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) all = joined(all, sh.sums[w], c);

  int n = 0;
  if constexpr (TOP) n = candidates<HALF>(row, lo, hi, a.top, largest, sh);

  if (sp.chunks > 1) {
    char* parts = sp.parts + r * sp.chunks * int64_t(kPartBytes);
    const __amdgpu_buffer_rsrc_t buf = coherent_buffer(parts, uint32_t(sp.chunks) * kPartBytes);
    const uint32_t at = uint32_t(chunk) * kPartBytes;
    if (tid == 0)
      __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(all.m), __float_as_uint(all.s), __float_as_uint(all.t), 0u},
                                             buf, at, 0, kCoherent);
    if constexpr (TOP) {
      auto put = [&](int i, uint64_t key) {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{uint32_t(key), uint32_t(key >> 32)}, buf, at + 16u + 8u * uint32_t(i), 0,
                                              kCoherent);
      };
      in_order(sh, n, a.top, put);
      if (tid >= n && tid < a.top) put(tid, 0);
    }
    __builtin_amdgcn_s_waitcnt(0);   // the part has reached the coherence point
    __syncthreads();
    uint32_t* counter = sp.counters + r * sp.counter_step;
    if (tid == 0) sh.arrived = atomicAdd(counter, 1u);
    __syncthreads();
    if (sh.arrived != uint32_t(sp.chunks - 1)) return;
    if (tid == 0) atomicExch(counter, 0u);
    all = Sums{kNone, 0.0f, 0.0f};
    for (int k = 0; k < sp.chunks; ++k) {   // in the chunks' order
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(buf, uint32_t(k) * kPartBytes, 0, kCoherent);
      all = joined(all, Sums{__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2])}, c);
    }
    if constexpr (TOP) {
      // of the lists' first `ahead` keys, at least `top` in all, the top-th is met by all that matter
      auto listed = [&](int k, int j) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(buf, uint32_t(k) * kPartBytes + 16u + 8u * uint32_t(j), 0, kCoherent);
        return uint64_t(v[1]) << 32 | v[0];
      };
      const int ahead = min(a.top, (2 * a.top + sp.chunks - 1) / sp.chunks), few = sp.chunks * ahead;
      static_assert(2 * NM_MAX_TOP + kMaxChunks <= kThreads && kMaxChunks * NM_MAX_TOP <= kRoom, "room for the lists");
      const uint64_t mine = tid < few ? listed(tid / ahead, tid % ahead) : 0;
      sh.keys[tid] = mine;
      if (tid == 0) sh.found = 0;
      __syncthreads();
      int before = 0;
      for (int j = 0; j < few; ++j) before += sh.keys[j] > mine || (sh.keys[j] == mine && j < tid) ? 1 : 0;
      if (tid < few && before == a.top - 1) sh.best[0] = mine;
      __syncthreads();
      const uint64_t limit = sh.best[0];
      for (int i = tid; i < sp.chunks * a.top; i += kThreads) {
        const uint64_t key = listed(i / a.top, i % a.top);
        if (key != 0 && key >= limit) sh.keys[atomicAdd(&sh.found, 1u)] = key;
      }
      __syncthreads();
      n = int(sh.found);
    }
  }

  // a NaN is in the sums; +infinity is the maximum
  const bool bad = !(all.s == all.s) || all.m == __builtin_inff();
  const float nan = __builtin_nanf("");
  const float log_all = log1pf(all.s);
  if (tid == 0) {
    if (a.tokens != nullptr) {
      const int token = a.tokens[r];
      float lp = 0.0f;
      if (token >= a.vocab || (token >= 0 && bad)) {
        lp = nan;
      } else if (token >= 0) {
        const float x = HALF ? half_at(static_cast<const uint16_t*>(row), size_t(token)) : static_cast<const float*>(row)[token];
        lp = x == kNone ? kNone : fmaf(a.scale, x - all.m, -log_all);
      }
      a.logprob[r] = lp;
    }
    if (a.entropy != nullptr)
      a.entropy[r] = bad ? nan : all.m == kNone ? 0.0f : log_all + kLn2 * all.t / (1.0f + all.s);
  }
  if constexpr (TOP) {
    int32_t* tokens = a.top_tokens + r * a.top;
    float* logprobs = a.top_logprobs + r * a.top;
    if (bad) {
      if (tid < a.top) {
        tokens[tid] = -1;
        logprobs[tid] = nan;
      }
      return;
    }
    in_order(sh, n, a.top, [&](int i, uint64_t key) {
      tokens[i] = index_of(key);
      logprobs[i] = fmaf(a.scale, value_of(key) - all.m, -log_all);
    });
    if (tid >= n && tid < a.top) {
      tokens[tid] = -1;
      logprobs[tid] = kNone;
    }
  }
}

// Workgroups of a row: four a CU in all, of kMinChunk elements or more.
int chunks_of(int64_t rows, int64_t vocab, const DeviceInfo& dev) {
  if (rows > NM_DECODE_COUNTER_BYTES / 4) return 1;
  int64_t c = 4 * int64_t(dev.cu_count) / rows;
  if (c > kMaxChunks) c = kMaxChunks;
  if (c > vocab / kMinChunk) c = vocab / kMinChunk;
  return c < 1 ? 1 : int(c);
}

size_t split_bytes(int64_t rows, int64_t vocab, const DeviceInfo& dev) {
  const int c = chunks_of(rows, vocab, dev);
  return c > 1 ? NM_DECODE_COUNTER_BYTES + size_t(rows) * size_t(c) * kPartBytes : 0;
}

}  // namespace

// The most that as many rows or fewer take: rows * chunks is at most four workgroups a CU.
size_t score_workspace_bytes(int64_t rows, int64_t vocab, const DeviceInfo& dev) {
  size_t most = 0;
  for (int64_t r = rows < 2 * int64_t(dev.cu_count) ? rows : 2 * int64_t(dev.cu_count); r > 0; --r) {
    const size_t n = split_bytes(r, vocab, dev);
    if (n > most) most = n;
  }
  return most;
}

hipError_t launch_score(const ScoreCall& c, bool fp16, void* workspace, size_t workspace_bytes, hipStream_t stream,
                        const DeviceInfo& dev) {
  ScoreCall a = c;
  ScoreSplit sp{1, 0, nullptr, nullptr};
  const size_t need = split_bytes(c.rows, c.vocab, dev);
  if (need > 0 && workspace != nullptr && workspace_bytes >= need) {
    sp.chunks = chunks_of(c.rows, c.vocab, dev);
    // a counter a line where they are few: additions to one line wait for each other
    const int64_t room = NM_DECODE_COUNTER_BYTES / 4 / c.rows;
    sp.counter_step = room > 32 ? 32 : int(room);
    sp.counters = static_cast<uint32_t*>(workspace);
    sp.parts = static_cast<char*>(workspace) + NM_DECODE_COUNTER_BYTES;
  }
  const bool top = c.top > 0;
  const void* k = fp16 ? (top ? reinterpret_cast<const void*>(&score_kernel<true, true>)
                              : reinterpret_cast<const void*>(&score_kernel<true, false>))
                       : (top ? reinterpret_cast<const void*>(&score_kernel<false, true>)
                              : reinterpret_cast<const void*>(&score_kernel<false, false>));
  void* args[] = {&a, &sp};
  return launch(k, dim3(unsigned(int64_t(c.rows) * sp.chunks)), dim3(kThreads), args, 0, stream, dev);
}

}  // namespace nm
