// nm_gated's small-batch kernels (nm_spmm_impl.h), by the choices of nm_spmm.hip.
#include "nm_spmm_impl.h"

namespace nm {

using namespace spmm_detail;

namespace {

template <int N, int B, int CI>
const void* kernel() { return reinterpret_cast<const void*>(&block_spmm_kernel<N, B, N == 16 ? kBitWalk : kByteLut, CI, kGatedForm>); }

template <int N>
const void* of_batch(int batch) {
  switch (batch) {
    case 1: return kernel<N, 1, 1>();
    case 2: return kernel<N, 2, 1>();
    case 3: return kernel<N, 3, 1>();
    case 4: return kernel<N, 4, 1>();
    case 5: return kernel<N, 5, 1>();
    case 6: return kernel<N, 6, 1>();
    case 7: return kernel<N, 7, 1>();
    default: return kernel<N, 8, 1>();
  }
}

}  // namespace

const void* block_spmm_gated_kernel_for(int N, int batch) {
  switch (N) {
    case 2: return of_batch<2>(batch);
    case 4: return of_batch<4>(batch);
    case 8: return of_batch<8>(batch);
    default: return of_batch<16>(batch);
  }
}

}  // namespace nm
