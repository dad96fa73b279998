// Verification of drafted chains and trees against the target's probabilities.
//
// Mathematics. A chain's drafts i are accepted while u_i q(x_i) < p(x_i); the tests of all
// drafts are independent, so one wave makes them at once and the first failure ends the chain.
// A tree's child c stands if u_c (1 - mass of its earlier siblings) < p(x_c), which also depends
// on its own row and siblings only: every node is decided at once, and the walk from the root
// follows the first child that stands. The next token is the first index whose running sum of
// the last row's weights exceeds u_0 times their sum, in 64 bits, so that the order of the sums
// moves a border by about 2^-50.
//
// What bounds it: one row of the target (and of the draft) a sequence is read for the draw,
// e.g. 64 x 128256 x 8 bytes. A single workgroup reads a row at the rate of one CU, so a row
// goes to several: each sums a chunk, the last to arrive finds the chunk the threshold falls
// in and walks that one alone. The decisions cost a chain of dependent loads (count, tokens,
// probabilities), so every workgroup makes them for itself rather than wait for another.
#include "nm_decode_internal.h"

namespace nm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxChunks = 64;                     // workgroups of a row
constexpr int kMaxParts = kMaxChunks * kWaves;     // its waves' runs: four a lane of the joining wave
constexpr int kMinChunk = 2048;                    // elements: shorter rows are not worth the hand-over

// Where a row's waves leave the sums of their runs: {with the draft (or the refused tokens)
// taken off, the target alone} for every sequence and run.
struct VerifySplit {
  int chunks;
  uint32_t* counters;
  double* sums;
};

struct Row {               // the row the next token is drawn from
  const float* target;
  const float* draft;      // NULL: none subtracted
  const int* refused;      // LDS, tokens of weight zero
  int refusals;
};

typedef float quad __attribute__((ext_vector_type(4), aligned(4)));   // rows start at any element

// Positive and finite, else zero.
__device__ __forceinline__ double kept(double x) { return x > 0.0 && x < __builtin_inf() ? x : 0.0; }

struct Pair {
  double rest, whole;      // weights with what is taken off, and of the target alone
};

// The weights of element i, exact (or rounded once) in 64 bits.
template <bool DRAFT>
__device__ __forceinline__ Pair weigh(const Row& w, int i, float p, float q) {
  Pair x;
  x.whole = kept(double(p));
  x.rest = DRAFT ? kept(double(p) - double(q)) : x.whole;
  if (!DRAFT)
    for (int k = 0; k < w.refusals; ++k)
      if (w.refused[k] == i) x.rest = 0.0;
  return x;
}

// Sums of the weights from lo + first on, `step` apart in groups of four neighbours.
template <bool DRAFT>
__device__ __forceinline__ Pair sum_run(const Row& w, int lo, int hi, int first, int step) {
  Pair s{0.0, 0.0};
  int i = lo + first;
  constexpr int U = 4;     // groups in flight
  for (; i + (U - 1) * step + 4 <= hi; i += U * step) {
    quad p[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      p[u] = *reinterpret_cast<const quad*>(w.target + i + u * step);
      if (DRAFT) q[u] = *reinterpret_cast<const quad*>(w.draft + i + u * step);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const Pair x = weigh<DRAFT>(w, i + u * step + e, p[u][e], DRAFT ? q[u][e] : 0.f);
        s.rest += x.rest;
        s.whole += x.whole;
      }
  }
  for (; i < hi; i += step)
    for (int e = 0; e < 4 && i + e < hi; ++e) {
      const Pair x = weigh<DRAFT>(w, i + e, w.target[i + e], DRAFT ? w.draft[i + e] : 0.f);
      s.rest += x.rest;
      s.whole += x.whole;
    }
  return s;
}

__device__ __forceinline__ double lane_value(double x, int lane) {   // lane: the same in all lanes
  const uint64_t v = uint64_t(__double_as_longlong(x));
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(v), lane), hi = __builtin_amdgcn_readlane(uint32_t(v >> 32), lane);
  return __longlong_as_double((long long)(uint64_t(hi) << 32 | lo));
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
  return x;
}

__device__ __forceinline__ double wave_scan(double x) {   // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}

struct Decision {
  int accepted;       // drafts that stand
  int row;            // node whose row the next token is drawn from
  bool stopped;       // a draft was refused
};

// A chain, by one wave: lane i tests draft i + 1.
__device__ __forceinline__ Decision decide_chain(const VerifyCall& a, int64_t b, int& n) {
  const int lane = threadIdx.x & 63;
  int x = -1;
  double u = 0.0;
  if (lane + 1 < a.nodes) {
    x = a.tokens[b * a.nodes + lane + 1];
    u = a.uniforms[b * a.nodes + lane + 1];
  }
  n = count_of(a.count, b, a.nodes);
  bool stands = false;
  if (lane + 1 < n && x >= 0 && x < a.vocab) {
    const double q = a.draft[(b * (a.nodes - 1) + lane) * a.vocab + x];
    stands = u * q < double(a.target[(b * a.nodes + lane) * a.vocab + x]);
  }
  Decision d;
  d.accepted = __builtin_ctzll(~__ballot(stands));   // lane 63 never stands
  d.row = d.accepted;
  d.stopped = d.accepted < n - 1;
  return d;
}

// A tree, by one wave: lane c decides node c. refused and path are LDS arrays.
__device__ __forceinline__ Decision decide_tree(const VerifyCall& a, int64_t b, int& n, int* refused, int* path,
                                                int* refusals) {
  const int lane = threadIdx.x & 63;
  int parent = -1, token = -1;
  double mass = 0.0, u = 0.0;
  if (lane > 0 && lane < a.nodes) {
    parent = a.parents[b * a.nodes + lane];
    token = a.tokens[b * a.nodes + lane];
    u = a.uniforms[b * a.nodes + lane];
  }
  n = count_of(a.count, b, a.nodes);
  if (lane >= n || parent < 0 || parent >= lane || token < 0 || token >= a.vocab) parent = -1;
  if (parent >= 0) mass = kept(double(a.target[(b * a.nodes + parent) * a.vocab + token]));
  // siblings in node order: lane s is final when its turn comes
  double left = 1.0;
  bool again = false, taken = false;
  for (int s = 1; s < n; ++s) {
    const int ps = __builtin_amdgcn_readlane(parent, s), ts = __builtin_amdgcn_readlane(token, s);
    const bool stood = (__ballot(!again && u * left < mass) >> s) & 1;
    const double ms = lane_value(again ? 0.0 : mass, s);
    if (ps >= 0 && ps == parent && lane > s) {
      again |= ts == token;
      left -= ms;
      taken |= stood;
    }
  }
  const bool chosen = parent >= 0 && !again && !taken && u * left < mass;
  Decision d{0, 0, false};
  if (lane == 0) path[0] = 0;
  while (true) {
    const uint64_t next = __ballot(chosen && parent == d.row);   // parents are before their children
    if (next == 0) break;
    d.row = __builtin_ctzll(next);
    ++d.accepted;
    if (lane == 0) path[d.accepted] = d.row;
  }
  const uint64_t tried = __ballot(parent == d.row);   // all refused
  if (parent == d.row) refused[__builtin_popcountll(tried & ((1ull << lane) - 1))] = token;
  if (lane == 0) *refusals = __builtin_popcountll(tried);
  d.stopped = tried != 0;
  return d;
}

// The part of a row where the running sum passes u times the sum, found by a wave from the
// runs' sums, four a lane.
struct Target {
  int part;
  bool plain;                 // nothing is left but the target itself
  double before, threshold;   // the running sum before the part; what the draw's has to exceed
};

__device__ __forceinline__ Target find_part(const Pair (&x)[4], double u) {
  const int lane = threadIdx.x & 63;
  double r[4], run[4];
  double sum = wave_sum((x[0].rest + x[1].rest) + (x[2].rest + x[3].rest));
  Target t;
  t.plain = !(sum > 0.0);
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = t.plain ? x[j].whole : x[j].rest;
  const double mine = (r[0] + r[1]) + (r[2] + r[3]);
  const double scan = wave_scan(mine);
  run[0] = (scan - mine) + r[0];
#pragma unroll
  for (int j = 1; j < 4; ++j) run[j] = run[j - 1] + r[j];
  t.threshold = u * lane_value(scan, 63);
  uint64_t past[4], any[4];
  int first = 4 * 64, top = -1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    past[j] = __ballot(r[j] > 0.0 && run[j] > t.threshold);
    any[j] = __ballot(r[j] > 0.0);
    if (past[j] != 0) first = min(first, 4 * __builtin_ctzll(past[j]) + j);
    if (any[j] != 0) top = max(top, 4 * (63 - __builtin_clzll(any[j])) + j);
  }
  // rounding may leave no part past the threshold: then the last that has any weight
  t.part = first < 4 * 64 ? first : max(top, 0);
  const int at = t.part >> 2, j = t.part & 3;
  const double upto = j == 0 ? run[0] - r[0] : j == 1 ? run[0] : j == 2 ? run[1] : run[2];
  t.before = lane_value(upto, at);
  return t;
}

// The first index of the part whose running sum passes the threshold, by the workgroup: a
// thread sums a few neighbours, and those that reach past it walk theirs.
template <bool DRAFT>
__device__ __forceinline__ void walk(const Row& w, const Target& t, int lo, int hi, double* parts, int* found, int* last) {
  const int tid = threadIdx.x, wave = tid >> 6;
  const int each = ((hi - lo + kThreads - 1) / kThreads + 3) & ~3;   // a thread's neighbours
  const int i0 = min(hi, lo + tid * each), i1 = min(hi, i0 + each);
  const Pair s = sum_run<DRAFT>(w, i0, i1, 0, 4);
  const double mine = t.plain ? s.whole : s.rest;
  const double scan = wave_scan(mine);
  if ((tid & 63) == 63) parts[wave] = scan;
  __syncthreads();
  double before = t.before;
  for (int x = 0; x < wave; ++x) before += parts[x];
  if (mine > 0.0 && before + scan > t.threshold) {
    double run = before + (scan - mine);
    for (int i = i0; i < i1; ++i) {
      const Pair x = weigh<DRAFT>(w, i, w.target[i], DRAFT ? w.draft[i] : 0.f);
      const double v = t.plain ? x.whole : x.rest;
      run += v;
      if (v > 0.0 && run > t.threshold) {
        atomicMin(found, i);
        break;
      }
    }
  }
  __syncthreads();
  if (*found != 0x7FFFFFFF || !(mine > 0.0)) return;
  // rounding took the threshold past the last sum: the last index with any weight
  for (int i = i1 - 1; i >= i0; --i) {
    const Pair x = weigh<DRAFT>(w, i, w.target[i], DRAFT ? w.draft[i] : 0.f);
    if ((t.plain ? x.whole : x.rest) > 0.0) {
      atomicMax(last, i);
      break;
    }
  }
}

__global__ __launch_bounds__(kThreads) void verify_kernel(VerifyCall a, VerifySplit sp) {
  __shared__ double parts[2][kWaves];
  __shared__ int refused[kMaxNodes], path[kMaxNodes];
  __shared__ int refusals, found, last;
  __shared__ uint32_t arrived;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b = blockIdx.y;
  if (tid == 0) {
    found = 0x7FFFFFFF;
    last = -1;
  }
  const double u0 = a.uniforms[b * a.nodes];
  int n;
  Decision d;
  if (a.parents == nullptr) {
    d = decide_chain(a, b, n);
  } else {
    d = decide_tree(a, b, n, refused, path, &refusals);   // every wave writes the same
    __syncthreads();
  }
  Row w{a.target + (b * a.nodes + d.row) * a.vocab, nullptr, refused, 0};
  if (a.parents != nullptr)
    w.refusals = refusals;
  else if (d.stopped)
    w.draft = a.draft + (b * (a.nodes - 1) + d.row) * a.vocab;

  // this wave's run of the row
  const int each = ((a.vocab + sp.chunks * kWaves - 1) / (sp.chunks * kWaves) + 3) & ~3;
  const int64_t lo64 = int64_t(int(blockIdx.x) * kWaves + wave) * each;
  int lo = int(lo64 < a.vocab ? lo64 : a.vocab), hi = min(a.vocab, lo + each);
  Pair s = w.draft != nullptr ? sum_run<true>(w, lo, hi, 4 * lane, 256) : sum_run<false>(w, lo, hi, 4 * lane, 256);
  s.rest = wave_sum(s.rest);
  s.whole = wave_sum(s.whole);
  Pair x[4] = {};
  if (sp.chunks > 1) {
    __amdgpu_buffer_rsrc_t buf = coherent_buffer(sp.sums + b * kMaxParts * 2, kMaxParts * 16);
    if (lane == 0) {
      const uint64_t r = uint64_t(__double_as_longlong(s.rest)), t = uint64_t(__double_as_longlong(s.whole));
      const u32x4 v = {uint32_t(r), uint32_t(r >> 32), uint32_t(t), uint32_t(t >> 32)};
      __builtin_amdgcn_raw_buffer_store_b128(v, buf, (blockIdx.x * kWaves + wave) * 16, 0, kCoherent);
    }
    __builtin_amdgcn_s_waitcnt(0);   // the sums have reached the coherence point
    __syncthreads();
    if (tid == 0) arrived = atomicAdd(sp.counters + b, 1u);
    __syncthreads();
    if (arrived != uint32_t(sp.chunks - 1)) return;
    if (tid == 0) atomicExch(sp.counters + b, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * lane + j < sp.chunks * kWaves) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(buf, (4 * lane + j) * 16, 0, kCoherent);
        x[j].rest = __longlong_as_double((long long)(uint64_t(v[1]) << 32 | v[0]));
        x[j].whole = __longlong_as_double((long long)(uint64_t(v[3]) << 32 | v[2]));
      }
  } else {
    if (lane == 0) {
      parts[0][wave] = s.rest;
      parts[1][wave] = s.whole;
    }
    __syncthreads();
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = Pair{parts[0][j], parts[1][j]};
    __syncthreads();
  }
  const Target t = find_part(x, u0);
  lo = int(min(int64_t(a.vocab), int64_t(t.part) * each));
  hi = min(a.vocab, lo + each);
  if (w.draft != nullptr)
    walk<true>(w, t, lo, hi, parts[0], &found, &last);
  else
    walk<false>(w, t, lo, hi, parts[0], &found, &last);
  __syncthreads();
  const int token = found != 0x7FFFFFFF ? found : last;
  if (tid == 0) a.accepted[b] = d.accepted;
  if (tid < a.nodes) {
    int32_t* out = a.out_tokens + b * a.nodes;
    const int next = tid < d.accepted ? (a.parents == nullptr ? tid + 1 : path[tid + 1]) : 0;
    out[tid] = n == 0 ? -1 : tid < d.accepted ? a.tokens[b * a.nodes + next] : tid == d.accepted ? token : -1;
    if (a.path != nullptr) a.path[b * a.nodes + tid] = n > 0 && tid <= d.accepted ? path[tid] : -1;
  }
}

// Chunks of a row: enough workgroups to fill the GPU twice over.
int chunks_of(int64_t batch, int64_t vocab, const DeviceInfo& dev) {
  if (batch > NM_DECODE_COUNTER_BYTES / 4) return 1;
  int64_t c = 2 * int64_t(dev.cu_count) / batch;
  if (c > kMaxChunks) c = kMaxChunks;
  if (c > vocab / kMinChunk) c = vocab / kMinChunk;
  return c < 1 ? 1 : int(c);
}

}  // namespace

size_t verify_workspace_bytes(int64_t batch, int64_t vocab, const DeviceInfo& dev) {
  return chunks_of(batch, vocab, dev) > 1 ? NM_DECODE_COUNTER_BYTES + size_t(batch) * kMaxParts * 16 : 0;
}

hipError_t launch_verify(const VerifyCall& c, void* workspace, size_t workspace_bytes, hipStream_t stream,
                         const DeviceInfo& dev) {
  VerifyCall a = c;
  VerifySplit sp{1, nullptr, nullptr};
  const size_t need = verify_workspace_bytes(c.batch, c.vocab, dev);
  if (need > 0 && workspace != nullptr && workspace_bytes >= need) {
    sp.chunks = chunks_of(c.batch, c.vocab, dev);
    sp.counters = static_cast<uint32_t*>(workspace);
    sp.sums = reinterpret_cast<double*>(static_cast<char*>(workspace) + NM_DECODE_COUNTER_BYTES);
  }
  void* args[] = {&a, &sp};
  return launch(reinterpret_cast<const void*>(verify_kernel), dim3(sp.chunks, uint32_t(c.batch)), dim3(kThreads), args, 0,
                stream, dev);
}

}  // namespace nm
