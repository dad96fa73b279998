// nm_linear's matrix-core kernels (nm_prefill_impl.h) for the tiles that nm_prefill.hip
// chooses.
#include "nm_internal.h"
#include "nm_prefill_impl.h"

namespace nm {

using namespace prefill_detail;

namespace {

template <int TR, int TT, int MODE>
const void* whole() { return reinterpret_cast<const void*>(&block_prefill_kernel<TR, TT, 64, 2, MODE, kLinearForm>); }
template <int TR, int TT, int MODE>
const void* split() { return reinterpret_cast<const void*>(&block_colsplit_kernel<TR, TT, 64, 2, MODE, kLinearForm>); }

template <int MODE>
const void* of_mode(int tr, int tt, bool colsplit) {
  if (colsplit) {
    if (tr == 1) return tt == 2 ? split<1, 2, MODE>() : split<1, 4, MODE>();
    if constexpr (MODE == kPfDirect)
      if (tr == 4) return split<4, 8, MODE>();
    return split<2, 8, MODE>();
  }
  if (tr == 1) {
    if constexpr (MODE == kPfExpand)
      if (tt == 16) return whole<1, 16, MODE>();
    return tt == 4 ? whole<1, 4, MODE>() : whole<1, 8, MODE>();
  }
  if constexpr (MODE != kPfDirect)
    if (tr == 2 && tt == 16) return whole<2, 16, MODE>();
  if constexpr (MODE != kPfExpand)
    if (tr == 4) return tt == 8 ? whole<4, 8, MODE>() : whole<4, 16, MODE>();
  return tt == 4 ? whole<2, 4, MODE>() : whole<2, 8, MODE>();
}

}  // namespace

const void* block_prefill_linear_kernel_for(int mode, int tr, int tt, bool colsplit) {
  return mode == kPfDirect  ? of_mode<kPfDirect>(tr, tt, colsplit)
         : mode == kPfSplit ? of_mode<kPfSplit>(tr, tt, colsplit)
                            : of_mode<kPfExpand>(tr, tt, colsplit);
}

}  // namespace nm
