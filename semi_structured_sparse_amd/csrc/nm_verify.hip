// Verification of drafted chains and trees against the target's probabilities.
//
// Mathematics. A chain's drafts i are accepted while u_i q(x_i) < p(x_i); the tests of all
// drafts are independent, so one wave makes them at once and the first failure ends the chain.
// A tree's child c stands if u_c (1 - mass of its earlier siblings) < p(x_c): the nodes' p are
// gathered at once, and the walk from the root tests the children of the nodes it reaches. The
// next token is the first index whose running sum of the last row's weights exceeds u_0 times
// their sum, in 64 bits, so that the order of the sums moves a border by about 2^-50.
//
// What bounds it: one row of the target (and of the draft) a sequence is read for the draw,
// e.g. 64 x 128256 x 8 bytes. A single workgroup reads a row at the rate of one CU, so a row
// goes to several: each sums a chunk, the last to arrive finds the run of it that the threshold
// falls in and walks that one alone. The decisions cost a chain of dependent loads (tokens,
// probabilities), so every workgroup makes them for itself rather than wait for another. Measured:
// 64 chains of 8, vocabulary 128256 (66 MB) 16.1 us, 4.1 TB/s; 16 trees of 32, 151936 9.1 us; 8
// chains of 5, 32000 6.8 us, most of it the chain of loads (decisions about 2, a run 1.5, the sums'
// hand-off 2, the walk 1).
#include "nm_decode_internal.h"

namespace nm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxChunks = 64;                     // workgroups of a row
constexpr int kMaxParts = kMaxChunks * kWaves;     // its waves' runs: four a lane of the joining wave
constexpr int kMinChunk = 1024;                    // elements: one load of 16 bytes a lane

// Where a row's waves leave the sums of their runs, and each sequence's counter: apart, since
// additions to one line wait for each other.
struct VerifySplit {
  int chunks;
  int counter_step;
  uint32_t* counters;
  double* sums;
};

struct Row {               // the row the next token is drawn from
  const float* target;
  const float* draft;      // NULL: none subtracted
  int refused;             // lane k < refusals: a token of weight zero
  int refusals;
};

typedef float quad __attribute__((ext_vector_type(4), aligned(4)));   // rows start at any element

// Positive and finite, else zero.
__device__ __forceinline__ double kept(double x) { return x > 0.0 && x < __builtin_inf() ? x : 0.0; }

// The refused tokens (lanes, a bit each) in [lo, hi): mostly none.
__device__ __forceinline__ uint64_t refused_in(const Row& w, int lo, int hi) {
  return __ballot(int(threadIdx.x & 63) < w.refusals && w.refused >= lo && w.refused < hi);
}

// The weights of N elements in groups of four from i on, `step` apart, exact (or rounded once) in
// 64 bits. some: refused tokens to look for.
template <bool DRAFT, int N>
__device__ __forceinline__ void weigh(const Row& w, uint64_t some, int i, int step, const float (&p)[N], const float (&q)[N],
                                      double (&v)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = kept(DRAFT ? double(p[e]) - double(q[e]) : double(p[e]));
  for (uint64_t m = some; m != 0; m &= m - 1) {
    const int x = __builtin_amdgcn_readlane(w.refused, __builtin_ctzll(m)) - i;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (x == e / 4 * step + e % 4) v[e] = 0.0;
  }
}

// N elements from i on (zeros at and past hi) in groups of four, `step` apart.
template <bool DRAFT, int N>
__device__ __forceinline__ void load_run(const Row& w, int i, int step, int hi, float (&p)[N], float (&q)[N]) {
#pragma unroll
  for (int u = 0; u < N / 4; ++u) {
    const int at = i + u * step;
    quad a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
    if (at + 4 <= hi) {
      a = *reinterpret_cast<const quad*>(w.target + at);
      if (DRAFT) b = *reinterpret_cast<const quad*>(w.draft + at);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at + e < hi) {
          a[e] = w.target[at + e];
          if (DRAFT) b[e] = w.draft[at + e];
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[4 * u + e] = a[e];
      q[4 * u + e] = b[e];
    }
  }
}

__device__ __forceinline__ double lane_value(double x, int lane) {   // lane: the same in all lanes
  const uint64_t v = uint64_t(__double_as_longlong(x));
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(v), lane), hi = __builtin_amdgcn_readlane(uint32_t(v >> 32), lane);
  return __longlong_as_double((long long)(uint64_t(hi) << 32 | lo));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double x) {   // zero where there is no lane to take from
  const uint64_t v = uint64_t(__double_as_longlong(x));
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, uint32_t(v), CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, uint32_t(v >> 32), CTRL, ROWS, 0xF, false);
  return __longlong_as_double((long long)(uint64_t(hi) << 32 | lo));
}

__device__ __forceinline__ double wave_scan(double x) {   // inclusive
  x += shifted<0x111, 0xF>(x);   // row_shr 1, 2, 4, 8
  x += shifted<0x112, 0xF>(x);
  x += shifted<0x114, 0xF>(x);
  x += shifted<0x118, 0xF>(x);
  x += shifted<0x142, 0xA>(x);   // the row before's last, rows 1 and 3
  x += shifted<0x143, 0xC>(x);   // the first half's last, rows 2 and 3
  return x;
}

// The sum of a wave's run [lo, hi). Weights that are infinite, and refused tokens, are looked for
// only where the plain sum is not finite, and where a token is in the run.
template <bool DRAFT>
__device__ __forceinline__ double sum_run(const Row& w, int lo, int hi) {
  const uint64_t some = refused_in(w, lo, hi);
  const int first = lo + 4 * int(threadIdx.x & 63);
  constexpr int N = 16;   // elements in flight a lane: 32 or non-temporal loads gained nothing
  double s = 0.0;
  if (some == 0) {
    for (int i = first; i < hi; i += 64 * N) {
      float p[N], q[N];
      load_run<DRAFT>(w, i, 256, hi, p, q);
#pragma unroll
      for (int e = 0; e < N; ++e) s += fmax(DRAFT ? double(p[e]) - double(q[e]) : double(p[e]), 0.0);
    }
    s = lane_value(wave_scan(s), 63);
    if (s < __builtin_inf()) return s;
  }
  s = 0.0;
  for (int i = first; i < hi; i += 64 * N) {
    float p[N], q[N];
    double v[N];
    load_run<DRAFT>(w, i, 256, hi, p, q);
    weigh<DRAFT>(w, some, i, 256, p, q, v);
#pragma unroll
    for (int e = 0; e < N; ++e) s += v[e];
  }
  return lane_value(wave_scan(s), 63);
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

// A tree, by one wave: lane c holds node c. path is an LDS array; the tokens refused at the last
// node go to the row.
__device__ __forceinline__ Decision decide_tree(const VerifyCall& a, int64_t b, int& n, int* path, Row& w) {
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
  Decision d{0, 0, false};
  if (lane == 0) path[0] = 0;
  while (true) {
    uint64_t children = __ballot(parent == d.row);   // after their parent: the walk ends
    double left = 1.0;
    bool stands = false;
    w.refusals = 0;
    for (; children != 0; children &= children - 1) {
      const int c = __builtin_ctzll(children), x = __builtin_amdgcn_readlane(token, c);
      const bool again = __ballot(lane < w.refusals && w.refused == x) != 0;
      const double p = again ? 0.0 : lane_value(mass, c);
      stands = lane_value(u, c) * left < p;
      if (stands) {
        d.row = c;
        ++d.accepted;
        if (lane == 0) path[d.accepted] = c;
        break;
      }
      left -= p;
      if (lane == w.refusals) w.refused = x;
      ++w.refusals;
    }
    if (!stands) break;
  }
  d.stopped = w.refusals > 0;
  return d;
}

// The part of a row where the running sum passes u times the sum, found by a wave from the
// runs' sums, four a lane.
struct Target {
  int part;
  bool any;                   // the row has a weight
  double before, threshold;   // the running sum before the part; what the draw's has to exceed
};

__device__ __forceinline__ Target find_part(const double (&x)[4], double u) {
  const double mine = (x[0] + x[1]) + (x[2] + x[3]), scan = wave_scan(mine), sum = lane_value(scan, 63);
  double run[4];
  run[0] = (scan - mine) + x[0];
#pragma unroll
  for (int j = 1; j < 4; ++j) run[j] = run[j - 1] + x[j];
  Target t;
  t.any = sum > 0.0;
  t.threshold = u * sum;
  int first = 4 * 64, top = -1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t past = __ballot(x[j] > 0.0 && run[j] > t.threshold), any = __ballot(x[j] > 0.0);
    if (past != 0) first = min(first, 4 * __builtin_ctzll(past) + j);
    if (any != 0) top = max(top, 4 * (63 - __builtin_clzll(any)) + j);
  }
  // rounding may leave no part past the threshold: then the last that has any weight
  t.part = first < 4 * 64 ? first : max(top, 0);
  const int at = t.part >> 2, j = t.part & 3;
  const double upto = j == 0 ? scan - mine : j == 1 ? run[0] : j == 2 ? run[1] : run[2];
  t.before = lane_value(upto, at);
  return t;
}

// What a workgroup's waves tell each other.
struct Shared {
  double sum[kWaves];
  int hit[kWaves], top[kWaves];
  uint32_t arrived;
  int path[kMaxNodes];
};

constexpr int kNone = 0x7FFFFFFF;

// The first index of the part whose running sum passes the threshold, by the workgroup, 16
// neighbours a thread at a time; else (rounding took the threshold past the last sum) the last
// index with any weight; -1 if none has.
template <bool DRAFT>
__device__ __forceinline__ int walk(const Row& w, const Target& t, int lo, int hi, Shared& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint64_t some = refused_in(w, lo, hi);
  double before = t.before;
  int last = -1;
  for (int block = lo; block < hi; block += 16 * kThreads) {
    const int i0 = block + 16 * tid;
    float p[16], q[16];
    load_run<DRAFT>(w, i0, 4, hi, p, q);
    double v[16], mine = 0.0;
    weigh<DRAFT>(w, some, i0, 4, p, q, v);
    int top = -1;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      mine += v[e];
      if (v[e] > 0.0) top = i0 + e;
    }
    const double scan = wave_scan(mine);
    if (lane == 63) sh.sum[wave] = scan;
    __syncthreads();
    double run = before, all = 0.0;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
      if (x < wave) run += sh.sum[x];
      all += sh.sum[x];
    }
    // the wave's first thread whose neighbours take the sum past the threshold looks for the one
    const uint64_t past = __ballot(top >= 0 && run + scan > t.threshold), any = __ballot(top >= 0);
    if (lane == (past != 0 ? __builtin_ctzll(past) : 0)) {
      int hit = past != 0 ? top : kNone;
      run += scan - mine;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        run += v[e];
        if (v[e] > 0.0 && run > t.threshold) hit = min(hit, i0 + e);
      }
      sh.hit[wave] = hit;
    }
    if (lane == (any != 0 ? 63 - __builtin_clzll(any) : 0)) sh.top[wave] = top;
    __syncthreads();
    int found = kNone;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
      found = min(found, sh.hit[x]);
      last = max(last, sh.top[x]);
    }
    if (found != kNone) return found;
    before += all;
  }
  return last;
}

// A row's elements for each of `runs` waves, in whole quads.
__device__ __forceinline__ int run_length(int vocab, int runs) { return ((vocab + runs - 1) / runs + 3) & ~3; }

__global__ __launch_bounds__(kThreads) void verify_kernel(VerifyCall a, VerifySplit sp) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b = blockIdx.y;
  const double u0 = a.uniforms[b * a.nodes];
  int n;
  Decision d;
  Row w{nullptr, nullptr, -1, 0};
  if (a.parents == nullptr) {
    d = decide_chain(a, b, n);
    if (d.stopped) w.draft = a.draft + (b * (a.nodes - 1) + d.row) * a.vocab;
  } else {
    d = decide_tree(a, b, n, sh.path, w);   // every wave writes the same path
  }
  w.target = a.target + (b * a.nodes + d.row) * a.vocab;

  // this wave's run of the row
  int each = run_length(a.vocab, sp.chunks * kWaves);
  const int64_t lo64 = int64_t(int(blockIdx.x) * kWaves + wave) * each;
  int lo = int(lo64 < a.vocab ? lo64 : a.vocab), hi = min(a.vocab, lo + each);
  double s = w.draft != nullptr ? sum_run<true>(w, lo, hi) : sum_run<false>(w, lo, hi);
  double x[4] = {0.0, 0.0, 0.0, 0.0};
  if (sp.chunks > 1) {
    __amdgpu_buffer_rsrc_t buf = coherent_buffer(sp.sums + b * kMaxParts, kMaxParts * 8);
    if (lane == 0)
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, s), buf, (blockIdx.x * kWaves + wave) * 8, 0, kCoherent);
    __builtin_amdgcn_s_waitcnt(0);   // the sums have reached the coherence point
    __syncthreads();
    uint32_t* counter = sp.counters + b * sp.counter_step;
    if (tid == 0) sh.arrived = atomicAdd(counter, 1u);
    __syncthreads();
    if (sh.arrived != uint32_t(sp.chunks - 1)) return;
    if (tid == 0) atomicExch(counter, 0u);
    if (lane < sp.chunks) {   // a chunk's waves a lane
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(buf, lane * 32, 0, kCoherent);
      const u32x4 z = __builtin_amdgcn_raw_buffer_load_b128(buf, lane * 32 + 16, 0, kCoherent);
      x[0] = __builtin_bit_cast(double, u32x2{v[0], v[1]});
      x[1] = __builtin_bit_cast(double, u32x2{v[2], v[3]});
      x[2] = __builtin_bit_cast(double, u32x2{z[0], z[1]});
      x[3] = __builtin_bit_cast(double, u32x2{z[2], z[3]});
    }
  }
  Target t;
  bool alone = sp.chunks == 1;
  while (true) {
    if (alone) {
      if (lane == 0) sh.sum[wave] = s;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kWaves; ++j) x[j] = lane == 0 ? sh.sum[j] : 0.0;
      __syncthreads();
    }
    t = find_part(x, u0);
    if (t.any || (w.draft == nullptr && w.refusals == 0)) break;
    // nothing is left but the target itself, whose sum this workgroup takes alone
    w.draft = nullptr;
    w.refusals = 0;
    alone = true;
    each = run_length(a.vocab, kWaves);
    lo = min(a.vocab, wave * each);
    s = sum_run<false>(w, lo, min(a.vocab, lo + each));
  }
  lo = int(min(int64_t(a.vocab), int64_t(t.part) * each));
  hi = min(a.vocab, lo + each);
  const int token = w.draft != nullptr ? walk<true>(w, t, lo, hi, sh) : walk<false>(w, t, lo, hi, sh);
  if (tid == 0) a.accepted[b] = d.accepted;
  if (tid < a.nodes) {
    int32_t* out = a.out_tokens + b * a.nodes;
    const int next = tid < d.accepted ? (a.parents == nullptr ? tid + 1 : sh.path[tid + 1]) : 0;
    out[tid] = n == 0 ? -1 : tid < d.accepted ? a.tokens[b * a.nodes + next] : tid == d.accepted ? token : -1;
    if (a.path != nullptr) a.path[b * a.nodes + tid] = n > 0 && tid <= d.accepted ? sh.path[tid] : -1;
  }
}

// Chunks of a row: four workgroups a CU. (us at 1, 2, 4, 8 a CU: 64 rows of 128256 with their
// drafts 17.9, 16.0, 16.1, 17.5; 16 rows of 151936 11.1, 9.6, 9.1, 9.0: each makes the decisions
// for itself.)
int chunks_of(int64_t batch, int64_t vocab, const DeviceInfo& dev) {
  if (batch > NM_DECODE_COUNTER_BYTES / 4) return 1;
  int64_t c = 4 * int64_t(dev.cu_count) / batch;
  if (c > kMaxChunks) c = kMaxChunks;
  if (c > vocab / kMinChunk) c = vocab / kMinChunk;
  return c < 1 ? 1 : int(c);
}

// From one sequence's counter to the next: a line where they are few (8 chains as above 6.7 us,
// 8.9 with neighbouring counters; 16 trees 9.6 and 13.1).
int counter_step(int64_t batch) {
  const int64_t room = NM_DECODE_COUNTER_BYTES / 4 / batch;
  return room > 32 ? 32 : int(room);
}

size_t split_bytes(int64_t batch, int64_t vocab, const DeviceInfo& dev) {
  return chunks_of(batch, vocab, dev) > 1 ? NM_DECODE_COUNTER_BYTES + size_t(batch) * kMaxParts * sizeof(double) : 0;
}

}  // namespace

// The most that as many sequences or fewer take: more than two a CU have a workgroup each, unsplit.
size_t verify_workspace_bytes(int64_t batch, int64_t vocab, const DeviceInfo& dev) {
  return split_bytes(batch < 2 * int64_t(dev.cu_count) ? batch : 2 * int64_t(dev.cu_count), vocab, dev);
}

hipError_t launch_verify(const VerifyCall& c, void* workspace, size_t workspace_bytes, hipStream_t stream,
                         const DeviceInfo& dev) {
  VerifyCall a = c;
  VerifySplit sp{1, 0, nullptr, nullptr};
  const size_t need = split_bytes(c.batch, c.vocab, dev);
  if (need > 0 && workspace != nullptr && workspace_bytes >= need) {
    sp.chunks = chunks_of(c.batch, c.vocab, dev);
    sp.counter_step = counter_step(c.batch);
    sp.counters = static_cast<uint32_t*>(workspace);
    sp.sums = reinterpret_cast<double*>(static_cast<char*>(workspace) + NM_DECODE_COUNTER_BYTES);
  }
  void* args[] = {&a, &sp};
  return launch(reinterpret_cast<const void*>(verify_kernel), dim3(sp.chunks, uint32_t(c.batch)), dim3(kThreads), args, 0,
                stream, dev);
}

}  // namespace nm
