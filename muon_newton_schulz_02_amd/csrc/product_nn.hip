// C = P Q, P in row form, Q in k-row form: gradients with respect to inputs.
#include "product_tile.h"

namespace muon {

hipError_t launch_nn(int shape, const ProductArgs& a, int cus, hipStream_t stream) {
  if (a.f32 && shape == SHAPE_LARGE) return launch_shape<LargeF32, FORM_NN, EPI_STORE>(a, cus, stream);
  if (a.f32)
    return shape == SHAPE_SMALL ? launch_shape<SmallF32, FORM_NN, EPI_STORE>(a, cus, stream)
                                : launch_shape<MediumF32, FORM_NN, EPI_STORE>(a, cus, stream);
  if (shape == SHAPE_SMALL) return launch_shape<Small, FORM_NN, EPI_STORE>(a, cus, stream);
  if (shape == SHAPE_NARROW) return launch_shape<Narrow, FORM_NN, EPI_STORE>(a, cus, stream);
  if (shape == SHAPE_MEDIUM) return launch_shape<Medium, FORM_NN, EPI_STORE>(a, cus, stream);
  return launch_shape<Large, FORM_NN, EPI_STORE>(a, cus, stream);
}

}  // namespace muon
