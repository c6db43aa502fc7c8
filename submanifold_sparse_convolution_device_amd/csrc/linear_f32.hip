// The matrix products of packed rows in f32.
#include "linear_kernels.h"

namespace spconv {
hipError_t launch_product_f32(const ProductArgs& a, ProductForm form, ProductShape shape, hipStream_t stream) {
  return lin::launch_typed<float>(a, form, shape, stream);
}
}  // namespace spconv
