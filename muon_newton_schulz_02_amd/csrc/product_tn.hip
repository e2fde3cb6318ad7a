// C = P^T Q, both operands in k-row form: gradients with respect to weights.
#include "product_tile.h"

namespace muon {

hipError_t launch_tn(int shape, int epi, const ProductArgs& a, int cus, hipStream_t stream) {
  if (a.f32 && shape == SHAPE_LARGE) return launch_shape<LargeF32, FORM_TN, EPI_STORE>(a, cus, stream);
  if (a.f32) return launch_shape<MediumF32, FORM_TN, EPI_STORE>(a, cus, stream);
  auto with = [&](auto s) {
    using S = decltype(s);
    return epi == EPI_STORE_TARGET ? launch_shape<S, FORM_TN, EPI_STORE_TARGET>(a, cus, stream)
                                   : launch_shape<S, FORM_TN, EPI_STORE>(a, cus, stream);
  };
  return shape == SHAPE_NARROW ? with(Narrow{}) : shape == SHAPE_MEDIUM ? with(MediumTn{}) : with(Large{});
}

}  // namespace muon
