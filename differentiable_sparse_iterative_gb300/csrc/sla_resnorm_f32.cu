// The kernels of sla_resnorm.cuh for float data.
#include "sla_resnorm.cuh"

namespace sla {

template <>
cudaError_t resnorm_forward<float, float>(ResNormArgs p, bool vec, cudaStream_t st) {
  return resnorm_forward_as<float, float>(p, vec, st);
}

template <>
cudaError_t resnorm_backward<float, float>(ResNormArgs p, bool vec, int grid, cudaStream_t st) {
  return resnorm_backward_as<float, float>(p, vec, grid, st);
}

}  // namespace sla
