// The kernels of sla_product.cuh and sla_few.cuh for float data.
#include "sla_few.cuh"
#include "sla_product.cuh"

namespace sla {

template <>
cudaError_t launch_product<float>(int epi, int shape, int blocks, const ProductLaunch &l, bool early, cudaStream_t st) {
  switch (epi) {
    case kStore: return launch_product_shape<float, kStore>(shape, blocks, l, early, st);
    case kGate: return launch_product_shape<float, kGate>(shape, blocks, l, early, st);
    default: return launch_product_shape<float, kGateBack>(shape, blocks, l, early, st);
  }
}

template <>
cudaError_t launch_few<float>(Epilogue epi, const FewArgs &p, cudaStream_t st) {
  return epi == kGate ? launch_few_gate<float, true>(p, st) : launch_few_gate<float, false>(p, st);
}

}  // namespace sla
