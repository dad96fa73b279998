// The block products' kernels of up to 16 vectors on the matrix instructions (nm_skinny_impl.h), by
// the choices of nm_skinny.hip.
#include "nm_skinny_impl.h"

namespace nm {

using namespace skinny_detail;

namespace {

template <int FORM>
const void* of_mode(int mode) {
  return mode == kModeDirect  ? reinterpret_cast<const void*>(&block_skinny_kernel<kModeDirect, FORM>)
         : mode == kModeSplit ? reinterpret_cast<const void*>(&block_skinny_kernel<kModeSplit, FORM>)
                              : reinterpret_cast<const void*>(&block_skinny_kernel<kModeExpand, FORM>);
}

template <int FORM>
const void* wide_of_mode(int mode) {
  return mode == kModeDirect  ? reinterpret_cast<const void*>(&block_skinny_wide_kernel<kModeDirect, FORM>)
         : mode == kModeSplit ? reinterpret_cast<const void*>(&block_skinny_wide_kernel<kModeSplit, FORM>)
                              : reinterpret_cast<const void*>(&block_skinny_wide_kernel<kModeExpand, FORM>);
}

}  // namespace

const void* block_skinny_kernel_for(int form, int mode) {
  return form == kGatedForm ? of_mode<kGatedForm>(mode) : of_mode<kLinearForm>(mode);
}

const void* block_skinny_wide_kernel_for(int form, int mode) {
  return form == kGatedForm ? wide_of_mode<kGatedForm>(mode) : wide_of_mode<kLinearForm>(mode);
}

const void* block_skinny_colsplit_kernel_for(int mode) {
  return mode == kModeSplit ? reinterpret_cast<const void*>(&block_skinny_colsplit_kernel<kModeSplit>)
                            : reinterpret_cast<const void*>(&block_skinny_colsplit_kernel<kModeDirect>);
}

}  // namespace nm
