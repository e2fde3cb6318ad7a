// C = P Q, P in row form, Q in k-row form: gradients with respect to inputs.
#include "product_tile.h"

namespace muon {

hipError_t launch_nn(int shape, int epi, const ProductArgs& a, int cus, hipStream_t stream) {
  if (a.f32 && shape == SHAPE_LARGE) return launch_shape<LargeF32, FORM_NN, EPI_STORE>(a, cus, stream);
  if (a.f32)
    return shape == SHAPE_SMALL ? launch_shape<SmallF32, FORM_NN, EPI_STORE>(a, cus, stream)
                                : launch_shape<MediumF32, FORM_NN, EPI_STORE>(a, cus, stream);
  auto with = [&](auto s) {
    using S = decltype(s);
    return epi == EPI_STORE_TARGET ? launch_shape<S, FORM_NN, EPI_STORE_TARGET>(a, cus, stream)
                                   : launch_shape<S, FORM_NN, EPI_STORE>(a, cus, stream);
  };
  if (shape == SHAPE_SMALL) return with(Small{});
  if (shape == SHAPE_NARROW) return with(Narrow{});
  return shape == SHAPE_MEDIUM ? with(Medium{}) : with(Large{});
}

}  // namespace muon
