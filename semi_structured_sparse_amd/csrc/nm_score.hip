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
// The best tokens: each lane keeps the largest value that it saw, its tile, and the largest of its other
// tiles. A limit that `top` of a workgroup's 256 largest meet is met by few elements more, and they
// are looked for in the tiles of those lanes alone, 16 or 32 elements of one lane and tile at a time, by
// as many threads (each lane through its own elements instead, in its registers or read again, most of it
// instructions that find nothing: 256 rows of 151936 46 us against 41); of a lane with a second such tile, in
// all of its tiles. What is found is put in order by counting, for each, how many go before it.
//
// What bounds it: reading the logits once, with an exponential an element close behind (2047 rows of
// 128256 fp16, 525 MB: 5.2 TB/s; 1024 in fp32 5.2). A row goes to several workgroups where there are few
// rows; the last to arrive joins their sums and lists. There it is a chain of trips to memory (8 rows
// of 128256 fp32 10.7 us: 7 without alternatives, finding them 2, joining their lists 2).
#include <algorithm>
#include <type_traits>

#include "nm_block_internal.h"
#include "nm_decode_internal.h"
#include "nm_epilogue.h"

namespace nm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxChunks = 32;             // workgroups of a row
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
  int each;                // elements of a chunk
  int loads;               // of a lane's tile
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

// scale * log2 e, and (a - b) times it by halves, in an order in which neither the difference nor the factor
// has to be a float where the result is one: a and b of both ends of the type, scales past 2.3e38.
struct Factor {
  float scale, c;
  __device__ __forceinline__ explicit Factor(float scale_) : scale(scale_), c(scale_ * kLog2e) {}
  __device__ __forceinline__ float of(float a, float b) const { return (0.5f * a - 0.5f * b) * scale * (2.0f * kLog2e); }
};

// The sums of two sets; without a maximum (kNone) one holds nothing, or NaN.
__device__ __forceinline__ Sums joined(const Sums& a, const Sums& b, const Factor& c) {
  const bool first = a.m >= b.m;
  const Sums &hi = first ? a : b, &lo = first ? b : a;
  Sums r = hi;
  if (lo.m == kNone) {
    r.s += lo.s;
  } else {
    const float g = fminf(c.of(hi.m, lo.m), 200.0f), f = __builtin_amdgcn_exp2f(-g);   // 2^-200 is 0
    r.s += f * (lo.s + 1.0f);
    r.t += f * fmaf(g, lo.s + 1.0f, lo.t);
  }
  return r;
}

// log p of a logit of x. In 64 bits, few as they are: x - m or its product alone may be past the largest float.
__device__ __forceinline__ float log_p(float x, float m, float scale, float log_all) {
  return float(double(scale) * (double(x) - double(m)) - double(log_all));
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

// What a wave's terms are relative to: 2^(x c - mc), mc the rounded m c, so that a term's exponent is
// one instruction from fp16 (its conversion in it); what the rounding of mc left, half a step of it, goes into
// the sums when they are closed. From 2^24 on that is more than 1 and soon past what an exponent holds: there,
// and where m c is no number, the exponent is that of (x - m), and nothing is left.
struct Reference {
  Factor f;
  float m, mc;
  bool direct;
  __device__ __forceinline__ Reference(float m_, const Factor& f_)
      : f(f_), m(m_), mc(m_ * f_.c), direct(!(fabsf(m_ * f_.c) < 16777216.0f)) {}
  __device__ __forceinline__ float rest() const { return direct ? 0.0f : fmaf(m, f.c, -mc); }
  template <bool DIRECT>
  __device__ __forceinline__ float exponent(float x) const {
    return DIRECT ? f.of(x, m) : fmaf(x, f.c, -mc);
  }
};

// A lane's elements of a tile of kThreads * LOADS * kElements from `at` on: load u at
// at + (u * kThreads + tid) * kElements; kNone past `hi`.
template <bool HALF, int LOADS>
struct Part {
  static constexpr int E = kElements<HALF>;
  typedef _Float16 half_group __attribute__((ext_vector_type(8)));
  typedef float float_group __attribute__((ext_vector_type(4)));
  typedef std::conditional_t<HALF, half_group, float_group> Group;
  typedef std::conditional_t<HALF, halves, floats> Anywhere;
  typedef std::conditional_t<HALF, _Float16, float> Element;
  Group v[LOADS];

  static __device__ __forceinline__ int index(int at, int u) { return at + (u * kThreads + int(threadIdx.x)) * E; }

  __device__ __forceinline__ void load(const void* row, int at, int hi) {
    const Element* p = static_cast<const Element*>(row);
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int i = index(at, u);
      if (i + E <= hi) {
        v[u] = *reinterpret_cast<const Anywhere*>(p + i);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = i + e < hi ? p[i + e] : Element(kNone);
      }
    }
  }
  __device__ __forceinline__ float at(int u, int e) const { return float(v[u][e]); }
  __device__ __forceinline__ float largest() const {   // NaN aside: the sums find it
    Group m = v[0];
#pragma unroll
    for (int u = 1; u < LOADS; ++u) m = __builtin_elementwise_max(m, v[u]);
    Element r = m[0];
#pragma unroll
    for (int e = 1; e < E; ++e) r = __builtin_elementwise_max(r, m[e]);
    return float(r);
  }
  // Adds the terms; skip: the lane's first element at the maximum is left out.
  template <bool DIRECT, bool SKIP>
  __device__ __forceinline__ void add(const Reference& r, bool skip, float& s, float& t) const {
#pragma unroll
    for (int u = 0; u < LOADS; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = r.exponent<DIRECT>(at(u, e));
        float f = __builtin_amdgcn_exp2f(d);
        if constexpr (SKIP) {
          if (skip && at(u, e) == r.m) {
            f = 0.0f;
            skip = false;
          }
        }
        s += f;
        t = fmaf(f, fmaxf(d, -200.0f), t);   // 2^-200 is 0, and stays that beside an infinite d
      }
  }
};

// A wave's sums as they grow: s and t (of 2^d d, so negative) are a lane's, m the wave's.
struct Running {
  float m = kNone, s = 0.0f, t = 0.0f;
  // s and t as sums of 2^((x - m) c) and of that times (m - x) c
  __device__ __forceinline__ Sums closed(const Factor& c) const {
    if (!(m > kNone)) return Sums{m, s, 0.0f};
    const float rest = Reference(m, c).rest(), f = __builtin_amdgcn_exp2f(-rest);
    return Sums{m, s * f, f * fmaf(rest, s, -t)};   // the rest is in each term's exponent, and so in t beside s
  }
  __device__ __forceinline__ void open(float m_, const Factor& c, float s_, float t_) {   // the same, backwards
    const float rest = Reference(m_, c).rest(), f = __builtin_amdgcn_exp2f(rest);
    m = m_;
    s = s_ * f;
    t = f * fmaf(rest, s_, -t_);
  }
};


struct Shared {
  uint64_t keys[kRoom];
  int places[kThreads];     // where to look: a lane's first element in its tile,
  int lanes[kThreads];      // or in every tile
  Sums sums[kWaves];
  uint64_t best[kWaves];
  int counts[kWaves];
  uint32_t found, tiles, everywhere;
  float limits[kWaves];
  uint64_t limit;
  uint32_t arrived;
};

// Puts the `top` first of the n keys in sh.keys (all different) in order and calls put(rank, key).
template <typename Put>
__device__ __forceinline__ void in_order(const Shared& sh, int n, int top, Put put) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t mine = sh.keys[i];
    int before = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) before += sh.keys[j] > mine ? 1 : 0;
    if (before < top) put(before, mine);
  }
}

// Where too many elements meet the limit: the keys one after the other, each the largest below the one
// before, a reading of the run each. That is what long runs of equal logits take, and finite masks that leave a
// workgroup's run fewer tokens than alternatives: 64 rows of 151936 fp16 with 20 and four tokens above -1e4 296 us,
// 2047 of 128256 8.2 ms, against 19 and 135 of ordinary rows and 14 and 115 of rows masked with -infinity.
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

// A value that at least `count` of a wave's lanes' values meet, and few more: halvings between the
// least and the largest until `count` meet it (twelve at most, then what they came to).
__device__ __forceinline__ float met_by(float mine, float most, int count) {
  float low = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) low = fminf(low, __shfl_xor(low, d));
  float high = most;
  for (int i = 0; i < 12 && low > kNone; ++i) {   // without -infinity there, all halves are finite
    const float half = 0.5f * low + 0.5f * high;
    const int met = __builtin_popcountll(__ballot(mine >= half));
    if (met >= count) low = half;
    else high = half;
    if (met == count) break;
  }
  if (low > kNone) return low;
  // lanes without a value: the count-th largest, one after the other
  float best = __builtin_inff();
  for (int n = 0; n < count && best > kNone;) {
    best = wave_max(mine < best ? mine : kNone);
    n += __builtin_popcountll(__ballot(mine == best));
  }
  return best;
}

// What a lane keeps of the values that it saw.
struct Largest {
  float value = kNone, other = kNone;   // the largest; the largest of its other tiles
  int at = 0;                           // its tile
  __device__ __forceinline__ void see(float v, int tile) {
    const bool more = v > value;
    other = fmaxf(other, more ? value : v);
    at = more ? tile : at;
    value = fmaxf(value, v);
  }
};

// Fewer of the n > kThreads keys in sh.keys, the `top` best among them; returns their number. A limit once
// more, now on the keys themselves, spread over all the threads: each wave's count-th largest of its lanes' largest.
__device__ __forceinline__ int fewer(int n, int top, Shared& sh) {
  constexpr int kEach = kRoom / kThreads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint64_t mine[kEach], most = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = int(threadIdx.x) + k * kThreads;
    mine[k] = i < n ? sh.keys[i] : 0;
    most = mine[k] > most ? mine[k] : most;
  }
  uint64_t limit = ~uint64_t(0);
  for (int i = 0; i < (top + kWaves - 1) / kWaves; ++i) {   // at most 16: each lane has one
    uint64_t next = most < limit ? most : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t other = uint64_t(__shfl_xor((unsigned long long)next, d));
      next = other > next ? other : next;
    }
    limit = next;
  }
  if (lane == 0) sh.best[wave] = limit;
  if (threadIdx.x == 0) sh.found = 0;
  __syncthreads();   // every key is read, too
#pragma unroll
  for (int w = 0; w < kWaves; ++w) limit = sh.best[w] < limit ? sh.best[w] : limit;
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (mine[k] != 0 && mine[k] >= limit) sh.keys[atomicAdd(&sh.found, 1u)] = mine[k];
  __syncthreads();
  return int(sh.found);
}

// Leaves the keys of at least the `top` best elements of the run in sh.keys; returns their number.
// Each wave finds a value that a quarter of `top` of its lanes' largest meet; the least of the four
// values is met by `top` elements at least. Where a wave has too few lanes with values (the run ends before its
// places, or masks leave it nothing), everything meets it: many keys are cut down once more before they are put
// in order, which takes a step for each beside each 256 (8 rows of 50257 fp16, five alternatives, whose last run
// is short: 87 us, 13 so; 2000 of 1500 with 20: 548 and 37).
template <bool HALF, int LOADS>
__device__ __forceinline__ int candidates(const void* row, int lo, int hi, int top, const Largest& mine, float most,
                                          Shared& sh) {
  constexpr int E = kElements<HALF>, kTile = kThreads * LOADS * E, kGroup = LOADS * E, kAtOnce = 4;
  const int tid = threadIdx.x;
  const float own = met_by(mine.value, most, (top + kWaves - 1) / kWaves);
  if ((tid & 63) == 0) sh.limits[tid >> 6] = own;
  if (tid == 0) sh.found = sh.tiles = sh.everywhere = 0;
  __syncthreads();
  float limit = sh.limits[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) limit = fminf(limit, sh.limits[w]);
  limit = fmaxf(limit, HALF ? -65504.0f : -3.402823466e38f);   // -infinity meets no limit
  if (mine.value >= limit) {
    if (mine.other >= limit) sh.lanes[atomicAdd(&sh.everywhere, 1u)] = lo + tid * E;
    else sh.places[atomicAdd(&sh.tiles, 1u)] = mine.at + tid * E;
  }
  __syncthreads();
  const int tiles = (hi - lo + kTile - 1) / kTile, lanes = int(sh.everywhere), some = int(sh.tiles);
  const int places = some + lanes * tiles;
  const int j = tid % kGroup, offset = (j / E) * (kThreads * E) + j % E;
  for (int i = tid / kGroup; i < places; i += kAtOnce * (kThreads / kGroup)) {
    float x[kAtOnce];
    int at[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int place = i + k * (kThreads / kGroup);
      at[k] = hi;
      if (place < some) {
        at[k] = sh.places[place] + offset;
      } else if (place < places) {
        const int tile = int(unsigned(place - some) / unsigned(lanes));
        at[k] = sh.lanes[place - some - tile * lanes] + tile * kTile + offset;
      }
      x[k] = kNone;
      if (at[k] < hi) x[k] = float(static_cast<const typename Part<HALF, LOADS>::Element*>(row)[at[k]]);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (x[k] >= limit) {
        const uint32_t n = atomicAdd(&sh.found, 1u);
        if (n < kRoom) sh.keys[n] = key_of(x[k], at[k]);
      }
  }
  __syncthreads();
  const uint32_t n = sh.found;
  __syncthreads();
  if (n > kRoom) return one_by_one<HALF>(row, lo, hi, top, sh);
  return n <= kThreads ? int(n) : fewer(int(n), top, sh);
}

// Four waves a SIMD: with the 131 registers that the compiler takes otherwise only three fit (2047 rows
// of 128256 fp16 with 20 alternatives 135 us, 120 so; five, and the loads no longer overlap: 270).
template <bool HALF, bool TOP, int LOADS>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4))) void score_kernel(ScoreCall a, ScoreSplit sp) {
  constexpr int kTile = kThreads * LOADS * kElements<HALF>;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r = int64_t(blockIdx.x) / sp.chunks;
  const int chunk = int(int64_t(blockIdx.x) - r * sp.chunks);
  const void* row = static_cast<const char*>(a.logits) + r * a.stride * (HALF ? 2 : 4);
  const int lo = int(min(int64_t(a.vocab), int64_t(chunk) * sp.each)), hi = int(min(int64_t(a.vocab), int64_t(lo) + sp.each));
  const Factor c(a.scale);

  Running run;
  Largest largest;   // the lane's own
  Part<HALF, LOADS> p, next;
  const int token = a.tokens != nullptr ? a.tokens[r] : -1;
  p.load(row, lo, hi);
  // the token's logit, asked for now: two trips at the end otherwise (64 rows of 151936 with 20 alternatives
  // 18.8 us, 18.3 so)
  float of_token = kNone;
  if (tid == 0 && token >= 0 && token < a.vocab)
    of_token = float(static_cast<const typename Part<HALF, LOADS>::Element*>(row)[token]);
  for (int at = lo; at < hi; at += kTile) {
    const bool more = at + kTile < hi;
    if (more) next.load(row, at + kTile, hi);   // in flight while this tile's terms are added
    const float mine = p.largest();
    if (TOP) largest.see(mine, at);
    bool skip = false;
    const bool grows = __ballot(mine > run.m) != 0;
    if (grows) {
      const float top = wave_max(mine);
      if (run.m > kNone) {
        const Sums old = run.closed(c);
        const float g = fminf(c.of(top, run.m), 200.0f), f = __builtin_amdgcn_exp2f(-g);
        const float s = lane == 0 ? old.s + 1.0f : old.s;   // the old maximum joins the others
        run.open(top, c, f * s, f * fmaf(g, s, old.t));
      }
      run.m = top;
      skip = lane == __builtin_ctzll(__ballot(mine == top));
    }
    const Reference ref(run.m > kNone ? run.m : 0.0f, c);
    if (ref.direct)
      p.template add<true, true>(ref, skip, run.s, run.t);
    else if (grows)
      p.template add<false, true>(ref, skip, run.s, run.t);
    else
      p.template add<false, false>(ref, false, run.s, run.t);
    if (more) p = next;
  }
  Sums all = run.closed(c);
  all = Sums{all.m, wave_sum(all.s), wave_sum(all.t)};
  if (lane == 0) sh.sums[wave] = all;
  __syncthreads();
  all = sh.sums[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) all = joined(all, sh.sums[w], c);

  int n = 0;
  if constexpr (TOP) n = candidates<HALF, LOADS>(row, lo, hi, a.top, largest, run.m, sh);

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
    // every part at once: the sums a lane each, the lists' keys a few a thread
    auto listed = [&](int k, int j) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(buf, uint32_t(k) * kPartBytes + 16u + 8u * uint32_t(j), 0, kCoherent);
      return uint64_t(v[1]) << 32 | v[0];
    };
    constexpr int kKeys = kMaxChunks * NM_MAX_TOP / kThreads;
    static_assert(kMaxChunks <= 32 && kMaxChunks * NM_MAX_TOP <= kRoom, "a lane for each part, room for the lists");
    Sums part{kNone, 0.0f, 0.0f};
    if (lane < sp.chunks) {
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(buf, uint32_t(lane) * kPartBytes, 0, kCoherent);
      part = Sums{__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2])};
    }
    // of the lists' first `ahead` keys, `top` or more in all, the top-th is met by all that matter
    const int total = sp.chunks * a.top, ahead = min(a.top, (2 * a.top + sp.chunks - 1) / sp.chunks);
    uint64_t keys[kKeys] = {};
    bool first[kKeys];
    if constexpr (TOP) {
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        if (kThreads * i >= total) break;
        const int at_key = tid + kThreads * i;
        const int k = int(unsigned(at_key) / unsigned(a.top)), j = at_key - k * a.top;
        if (at_key < total) keys[i] = listed(k, j);
        first[i] = j < ahead;
      }
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {   // neighbours first, the lower one on the left: one order
      const Sums other{__shfl_xor(part.m, d), __shfl_xor(part.s, d), __shfl_xor(part.t, d)};
      part = (lane & d) ? joined(other, part, c) : joined(part, other, c);
    }
    all = Sums{__shfl(part.m, 0), __shfl(part.s, 0), __shfl(part.t, 0)};
    if constexpr (TOP) {
      if (tid == 0) {
        sh.found = 0;
        sh.limit = 0;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kKeys; ++i)
        if (kThreads * i < total && keys[i] != 0 && first[i]) sh.keys[atomicAdd(&sh.found, 1u)] = keys[i];
      __syncthreads();
      const int few = int(sh.found);
      for (int i = tid; i < few; i += kThreads) {
        const uint64_t mine = sh.keys[i];
        int before = 0;
        for (int j = 0; j < few; ++j) before += sh.keys[j] > mine ? 1 : 0;
        if (before == a.top - 1) sh.limit = mine;   // no one: fewer than `top` keys there, all are taken
      }
      __syncthreads();
      const uint64_t limit = sh.limit;
      if (tid == 0) sh.found = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kKeys; ++i)
        if (kThreads * i < total && keys[i] != 0 && keys[i] >= limit) sh.keys[atomicAdd(&sh.found, 1u)] = keys[i];
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
      float lp = 0.0f;
      if (token >= a.vocab || (token >= 0 && bad))
        lp = nan;
      else if (token >= 0)
        lp = of_token == kNone ? kNone : log_p(of_token, all.m, a.scale, log_all);
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
      logprobs[i] = log_p(value_of(key), all.m, a.scale, log_all);
    });
    if (tid >= n && tid < a.top) {
      tokens[tid] = -1;
      logprobs[tid] = kNone;
    }
  }
}

// The tiles of a row's workgroups: whole ones, for about three workgroups a CU in all. Measured with four: 64
// rows of 151936 20.7 us, 512 of 32000 20.8, against 18.6 with three and 18.4 with two, which take 36.2 for 256
// of 151936 against 33.8.
//
// Loads of a lane's tile: two, with which kAtOnce workgroups fit a CU (fp16 by its registers, fp32 by LDS; four loads
// leave room for four and five) and little of a row's last tile is empty. Measured (us, two / four loads): fp16 700
// rows of 50257 23.5 / 28.3, 1500 of 151936 98 / 109, 64 in 10 parts with 20 alternatives 19.1 / 21.0; fp32 1500
// 183 / 188, 64 in parts 19.2 / 21.2. Four in two places:
// - a part of two tiles becomes one of a wait less: 8 rows of 128256 fp32 11.5 / 11.1, 1 of 151936 fp16 11.5 / 11.2;
// - rows a little past what fits at once, most of whose second round of workgroups would be empty (128256, fp16:
//   1700 rows 91 / 95, 1800 108 / 100, 2047 128 / 114, 2200 130 / 126, 2500 139 / 137, 2800 152 / 149; fp32: 2047
//   206 / 212, 2049 227 / 213, 2300 243 / 234, 2500 255 / 252, 2800 278 / 280), but for short ones, whose last tile
//   is much of them (fp16 2047 of 50257 56 / 60).
template <bool HALF>
constexpr int kAtOnce = HALF ? 7 : 8;
constexpr int kLongTiles = 8;

template <bool HALF>
ScoreSplit split_of(int64_t rows, int64_t vocab, const DeviceInfo& dev) {
  constexpr int64_t kTile = kThreads * 2 * kElements<HALF>;
  ScoreSplit sp{1, int(vocab), 2, 0, nullptr, nullptr};
  const int64_t tiles = (vocab + kTile - 1) / kTile;
  int64_t want = 3 * int64_t(dev.cu_count) / rows;
  if (want > kMaxChunks) want = kMaxChunks;
  if (want < 2 || rows > NM_DECODE_COUNTER_BYTES / 4) return sp;
  const int64_t each = (tiles + want - 1) / want;
  sp.chunks = int((tiles + each - 1) / each);
  if (sp.chunks > 1) sp.each = int(each * kTile);
  if (sp.chunks > 1 && each == 2) sp.loads = 4;
  return sp;
}

ScoreSplit split_of(int64_t rows, int64_t vocab, bool fp16, const DeviceInfo& dev) {
  return fp16 ? split_of<true>(rows, vocab, dev) : split_of<false>(rows, vocab, dev);
}

template <bool HALF>
ScoreSplit whole_rows(int64_t rows, int64_t vocab, const DeviceInfo& dev) {
  const int64_t fit = int64_t(kAtOnce<HALF>) * dev.cu_count, tile = kThreads * 4 * kElements<HALF>;
  const bool past = rows > fit && 4 * rows <= 5 * fit && vocab >= kLongTiles * tile;
  return {1, int(vocab), past ? 4 : 2, 0, nullptr, nullptr};
}

size_t split_bytes(int64_t rows, int64_t vocab, bool fp16, const DeviceInfo& dev) {
  const int c = split_of(rows, vocab, fp16, dev).chunks;
  return c > 1 ? NM_DECODE_COUNTER_BYTES + size_t(rows) * size_t(c) * kPartBytes : 0;
}

template <bool HALF, bool TOP>
const void* kernel_of(int loads) {
  return loads == 4 ? reinterpret_cast<const void*>(&score_kernel<HALF, TOP, 4>)
                    : reinterpret_cast<const void*>(&score_kernel<HALF, TOP, 2>);
}

}  // namespace

// The most that as many rows or fewer take: rows * chunks is at most three workgroups a CU.
size_t score_workspace_bytes(int64_t rows, int64_t vocab, const DeviceInfo& dev) {
  size_t most = 0;
  for (int64_t r = rows < 2 * int64_t(dev.cu_count) ? rows : 2 * int64_t(dev.cu_count); r > 0; --r) {
    const size_t n = std::max(split_bytes(r, vocab, true, dev), split_bytes(r, vocab, false, dev));
    if (n > most) most = n;
  }
  return most;
}

hipError_t launch_score(const ScoreCall& c, bool fp16, void* workspace, size_t workspace_bytes, hipStream_t stream,
                        const DeviceInfo& dev) {
  ScoreCall a = c;
  ScoreSplit sp = fp16 ? whole_rows<true>(c.rows, c.vocab, dev) : whole_rows<false>(c.rows, c.vocab, dev);
  const size_t need = split_bytes(c.rows, c.vocab, fp16, dev);
  if (need > 0 && workspace != nullptr && workspace_bytes >= need) {
    sp = split_of(c.rows, c.vocab, fp16, dev);
    // a counter a line where they are few: additions to one line wait for each other
    const int64_t room = NM_DECODE_COUNTER_BYTES / 4 / c.rows;
    sp.counter_step = room > 32 ? 32 : int(room);
    sp.counters = static_cast<uint32_t*>(workspace);
    sp.parts = static_cast<char*>(workspace) + NM_DECODE_COUNTER_BYTES;
  }
  const bool top = c.top > 0;
  const void* k = fp16 ? (top ? kernel_of<true, true>(sp.loads) : kernel_of<true, false>(sp.loads))
                       : (top ? kernel_of<false, true>(sp.loads) : kernel_of<false, false>(sp.loads));
  void* args[] = {&a, &sp};
  return launch(k, dim3(unsigned(int64_t(c.rows) * sp.chunks)), dim3(kThreads), args, 0, stream, dev);
}

}  // namespace nm
