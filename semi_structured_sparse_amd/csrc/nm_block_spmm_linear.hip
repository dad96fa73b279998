// nm_linear's small-batch kernels (nm_spmm_impl.h), by the choices of nm_spmm.hip.
#include "nm_spmm_impl.h"

namespace nm {

using namespace spmm_detail;

namespace {

template <int N, int B, int CI>
const void* kernel() { return reinterpret_cast<const void*>(&block_spmm_kernel<N, B, N == 16 ? kBitWalk : kByteLut, CI, kLinearForm>); }

template <int N, int B>
const void* of_ci(int ci) { return ci == 4 ? kernel<N, B, 4>() : ci == 2 ? kernel<N, B, 2>() : kernel<N, B, 1>(); }

template <int N>
const void* of_batch(int batch, int ci) {
  switch (batch) {
    case 1: return of_ci<N, 1>(ci);
    case 2: return of_ci<N, 2>(ci);
    case 3: return of_ci<N, 3>(ci);
    case 4: return of_ci<N, 4>(ci);
    case 5: return of_ci<N, 5>(ci);
    case 6: return of_ci<N, 6>(ci);
    case 7: return of_ci<N, 7>(ci);
    default: return of_ci<N, 8>(ci);
  }
}

}  // namespace

const void* block_spmm_linear_kernel_for(int N, int batch, int ci) {
  switch (N) {
    case 2: return of_batch<2>(batch, ci);
    case 4: return of_batch<4>(batch, ci);
    case 8: return of_batch<8>(batch, ci);
    default: return of_batch<16>(batch, ci);
  }
}

}  // namespace nm
