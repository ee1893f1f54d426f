// The kernels of sla_product.cuh, sla_few.cuh and sla_narrow.cuh for bf16 data.
#include "sla_few.cuh"
#include "sla_narrow.cuh"
#include "sla_product.cuh"

namespace sla {

template <>
cudaError_t launch_product<bf16>(int epi, int shape, int blocks, const ProductLaunch &l, bool early, cudaStream_t st) {
  switch (epi) {
    case kStore: return launch_product_shape<bf16, kStore>(shape, blocks, l, early, st);
    case kGate: return launch_product_shape<bf16, kGate>(shape, blocks, l, early, st);
    case kLinear: return launch_product_shape<bf16, kLinear>(shape, blocks, l, early, st);
    case kAdd: return launch_product_shape<bf16, kAdd>(shape, blocks, l, early, st);
    default: return launch_product_shape<bf16, kGateBack>(shape, blocks, l, early, st);
  }
}

template <>
cudaError_t launch_few<bf16>(Epilogue epi, const FewArgs &p, cudaStream_t st) {
  return epi == kGate     ? launch_few_as<bf16, kGate>(p, st)
         : epi == kLinear ? launch_few_as<bf16, kLinear>(p, st)
                          : launch_few_as<bf16, kStore>(p, st);
}

template <>
cudaError_t launch_narrow<bf16>(const NarrowArgs &p, int blocks, bool early, cudaStream_t st) {
  return launch_narrow_as<bf16>(p, blocks, early, st);
}

}  // namespace sla
