// The matrix products of packed rows in f16.
#include "linear_kernels.h"

namespace spconv {
hipError_t launch_product_f16(const ProductArgs& a, ProductForm form, ProductShape shape, hipStream_t stream) {
  return lin::launch_typed<_Float16>(a, form, shape, stream);
}
}  // namespace spconv
