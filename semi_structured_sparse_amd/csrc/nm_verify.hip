// Verification of drafted chains and trees against the target's probabilities.
#include "nm_decode_internal.h"

namespace nm {
namespace {

constexpr int kThreads = 256;

struct Weights {           // the row the next token is drawn from
  const float* target;
  const float* draft;      // NULL: none subtracted
  const int* refused;      // LDS, tokens of weight zero
  int refusals;
};

// A token's weight: positive and finite, else zero; exact (or rounded once) in 64 bits.
__device__ __forceinline__ double weight(const Weights& w, int i) {
  const double x = w.draft != nullptr ? double(w.target[i]) - double(w.draft[i]) : double(w.target[i]);
  for (int k = 0; k < w.refusals; ++k)
    if (w.refused[k] == i) return 0.0;
  return x > 0.0 && x < __builtin_inf() ? x : 0.0;
}

// The first index whose running sum exceeds u times the sum, by the whole workgroup: thread t
// sums an interval of the row, and the thread whose interval the threshold falls in walks it.
// -1 where no weight is left.
__device__ int pick(const Weights& w, int vocab, double u, double* sums, int* found) {
  const int each = (vocab + kThreads - 1) / kThreads;
  const int lo = min(vocab, int(threadIdx.x) * each), hi = min(vocab, lo + each);
  double s = 0.0;
  int last = -1;
  for (int i = lo; i < hi; ++i) {
    const double x = weight(w, i);
    s += x;
    if (x > 0.0) last = i;
  }
  sums[threadIdx.x] = s;
  if (threadIdx.x == 0) *found = 0x7FFFFFFF;
  __syncthreads();
  double before = 0.0, all = 0.0;
  for (int t = 0; t < kThreads; ++t) {
    if (t < int(threadIdx.x)) before += sums[t];
    all += sums[t];
  }
  const double threshold = u * all;
  for (int i = lo; i < hi; ++i) {
    before += weight(w, i);
    if (before > threshold) {
      atomicMin(found, i);
      break;
    }
  }
  __syncthreads();
  int got = *found;
  __syncthreads();
  if (got == 0x7FFFFFFF) {          // rounding took the threshold past the last sum
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    if (last >= 0) atomicMax(found, last);
    __syncthreads();
    got = *found;
    __syncthreads();
  }
  return got;
}

__global__ __launch_bounds__(kThreads) void verify_kernel(VerifyCall a) {
  __shared__ double sums[kThreads];
  __shared__ int refused[kMaxNodes], path[kMaxNodes];
  __shared__ int found, refusals, accepted;
  const int64_t b = blockIdx.x;
  const int n = count_of(a.count, b, a.nodes);
  const int32_t* tokens = a.tokens + b * a.nodes;
  const float* uniforms = a.uniforms + b * a.nodes;
  const int64_t row0 = b * a.nodes;
  int32_t* out = a.out_tokens + b * a.nodes;
  if (threadIdx.x == 0) {
    refusals = 0;
    int m = 0, at = 0;
    path[0] = 0;
    if (a.parents == nullptr) {
      for (; m < n - 1; ++m) {
        const int x = tokens[m + 1];
        if (x < 0 || x >= a.vocab) break;
        if (!(double(uniforms[m + 1]) * double(a.draft[(b * (a.nodes - 1) + m) * a.vocab + x]) <
              double(a.target[(row0 + m) * a.vocab + x])))
          break;
      }
    } else {
      const int32_t* parents = a.parents + b * a.nodes;
      double left = 1.0;
      for (int c = 1; c < n; ++c) {
        if (parents[c] != at) continue;
        const int x = tokens[c];
        if (x < 0 || x >= a.vocab) continue;
        bool again = false;
        for (int k = 0; k < refusals; ++k) again |= refused[k] == x;
        const double p = again ? 0.0 : double(a.target[(row0 + at) * a.vocab + x]);
        if (double(uniforms[c]) * left < p) {
          at = c;
          path[++m] = c;
          refusals = 0;
          left = 1.0;
        } else {
          left -= p;
          refused[refusals++] = x;
        }
      }
    }
    accepted = m;
  }
  __syncthreads();
  const int m = accepted;
  const int row = a.parents == nullptr ? m : path[m];
  const float* target = a.target + (row0 + row) * a.vocab;
  const bool stopped = a.parents == nullptr && m < n - 1;
  int token = -1;
  if (n > 0) {
    Weights w{target, stopped ? a.draft + (b * (a.nodes - 1) + m) * a.vocab : nullptr, refused, refusals};
    token = pick(w, a.vocab, double(uniforms[0]), sums, &found);
    if (token < 0 && (stopped || refusals > 0)) {
      w = Weights{target, nullptr, refused, 0};
      token = pick(w, a.vocab, double(uniforms[0]), sums, &found);
    }
  }
  if (threadIdx.x == 0) a.accepted[b] = m;
  if (int(threadIdx.x) < a.nodes) {
    const int d = threadIdx.x;
    const int next = d < m ? (a.parents == nullptr ? d + 1 : path[d + 1]) : 0;
    out[d] = n == 0 ? -1 : d < m ? tokens[next] : d == m ? token : -1;
    if (a.path != nullptr) a.path[b * a.nodes + d] = n > 0 && d <= m ? path[d] : -1;
  }
}

}  // namespace

size_t verify_workspace_bytes(int64_t, int64_t, const DeviceInfo&) { return 0; }

hipError_t launch_verify(const VerifyCall& c, void*, size_t, hipStream_t stream, const DeviceInfo& dev) {
  VerifyCall a = c;
  void* args[] = {&a};
  return launch(reinterpret_cast<const void*>(verify_kernel), dim3(uint32_t(c.batch)), dim3(kThreads), args, 0, stream, dev);
}

}  // namespace nm
