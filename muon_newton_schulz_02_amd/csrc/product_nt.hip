// C = P Q^T, both operands in row form: products of the experts, and the head's logits.
#include "product_tile.h"

namespace muon {

hipError_t launch_nt(int shape, int epi, const ProductArgs& a, int cus, hipStream_t stream) {
  auto with = [&](auto s) -> hipError_t {
    using S = decltype(s);
    switch (epi) {
      case EPI_LSE: return launch_shape<S, FORM_NT, EPI_LSE>(a, cus, stream);
      case EPI_LSE_CAP: return launch_shape<S, FORM_NT, EPI_LSE_CAP>(a, cus, stream);
      case EPI_DZ: return launch_shape<S, FORM_NT, EPI_DZ>(a, cus, stream);
      case EPI_DZ_CAP: return launch_shape<S, FORM_NT, EPI_DZ_CAP>(a, cus, stream);
      case EPI_LSE_LARGE_CAP:
        if constexpr (!S::F32) return launch_shape<S, FORM_NT, EPI_LSE_LARGE_CAP>(a, cus, stream);
        return hipErrorInvalidValue;
      case EPI_DZ_LARGE_CAP:
        if constexpr (!S::F32) return launch_shape<S, FORM_NT, EPI_DZ_LARGE_CAP>(a, cus, stream);
        return hipErrorInvalidValue;
      default: return launch_shape<S, FORM_NT, EPI_STORE>(a, cus, stream);
    }
  };
  if (shape == SHAPE_NARROW) return launch_shape<Narrow, FORM_NT, EPI_STORE>(a, cus, stream);
  if (a.f32) return shape == SHAPE_SMALL ? with(SmallF32{}) : shape == SHAPE_MEDIUM ? with(MediumF32{}) : with(LargeF32{});
  return shape == SHAPE_SMALL ? with(Small{}) : shape == SHAPE_MEDIUM ? with(Medium{}) : with(Large{});
}

}  // namespace muon
