// The tensor-core products of sla_product.cuh for float data.
#include "sla_product.cuh"

namespace sla {

template <>
cudaError_t launch_product<float>(int epi, int shape, int blocks, const CUtensorMap &a, const CUtensorMap &b,
                               const ProductArgs &p, cudaStream_t st) {
  switch (epi) {
    case kStore: return launch_product_shape<float, kStore>(shape, blocks, a, b, p, st);
    case kGate: return launch_product_shape<float, kGate>(shape, blocks, a, b, p, st);
    case kGateBack: return launch_product_shape<float, kGateBack>(shape, blocks, a, b, p, st);
    default: return launch_product_shape<float, kPartial>(shape, blocks, a, b, p, st);
  }
}

}  // namespace sla
