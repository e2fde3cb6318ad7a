// C = P^T Q, both operands in k-row form: gradients with respect to weights.
#include "product_tile.h"

namespace muon {

hipError_t launch_tn(int shape, const ProductArgs& a, int cus, hipStream_t stream) {
  if (a.f32 && shape == SHAPE_LARGE) return launch_shape<LargeF32, FORM_TN, EPI_STORE>(a, cus, stream);
  if (a.f32) return launch_shape<MediumF32, FORM_TN, EPI_STORE>(a, cus, stream);
  if (shape == SHAPE_NARROW) return launch_shape<Narrow, FORM_TN, EPI_STORE>(a, cus, stream);
  if (shape == SHAPE_MEDIUM) return launch_shape<MediumTn, FORM_TN, EPI_STORE>(a, cus, stream);
  return launch_shape<Large, FORM_TN, EPI_STORE>(a, cus, stream);
}

}  // namespace muon
