// The tensor-core products of sla_product.cuh and sla_few.cuh for float data.
#include "sla_few.cuh"
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

template <>
cudaError_t launch_few<float>(Epilogue epi, const FewArgs &p, cudaStream_t st) {
  return epi == kGate ? launch_few_gate<float, true>(p, st) : launch_few_gate<float, false>(p, st);
}

}  // namespace sla
