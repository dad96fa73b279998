// The block products' single-vector kernels (nm_spmv_impl.h), by the choices of nm_spmv.hip.
#include "nm_spmv_impl.h"

namespace nm {

using namespace spmv_detail;

namespace {

constexpr int kBatch = 4;   // as nm_spmv.hip

template <int N, int DEC, int CI, int FORM>
const void* kernel() { return reinterpret_cast<const void*>(&block_spmv_kernel<N, kBatch, true, DEC, CI, FORM>); }

template <int FORM>
const void* of_form(int N, int dec, int ci) {
  if constexpr (FORM == kLinearForm) {
    if (N == 16 && dec == kRevWalk && ci > 1)
      return ci == 2 ? kernel<16, kRevWalk, 2, FORM>() : ci == 4 ? kernel<16, kRevWalk, 4, FORM>() : kernel<16, kRevWalk, 8, FORM>();
  }
  const bool walk = dec == kBitWalk;
  switch (N) {
    case 2: return walk ? kernel<2, kBitWalk, 1, FORM>() : kernel<2, kPairTable, 1, FORM>();
    case 4: return walk ? kernel<4, kBitWalk, 1, FORM>() : kernel<4, kByteLut, 1, FORM>();
    case 8: return walk ? kernel<8, kBitWalk, 1, FORM>() : kernel<8, kByteLut, 1, FORM>();
    default: return walk ? kernel<16, kBitWalk, 1, FORM>() : kernel<16, kRevWalk, 1, FORM>();
  }
}

}  // namespace

const void* block_spmv_kernel_for(int form, int N, int dec, int ci) {
  return form == kGatedForm ? of_form<kGatedForm>(N, dec, ci) : of_form<kLinearForm>(N, dec, ci);
}

const void* block_spmv_quarter_kernel_for(int form) {
  return form == kGatedForm ? reinterpret_cast<const void*>(&block_spmv_quarter_kernel<kBatch, true, kGatedForm>)
                            : reinterpret_cast<const void*>(&block_spmv_quarter_kernel<kBatch, true, kLinearForm>);
}

}  // namespace nm
