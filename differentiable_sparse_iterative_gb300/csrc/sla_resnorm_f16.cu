// The kernels of sla_resnorm.cuh for f16 data.
#include "sla_resnorm.cuh"

namespace sla {

template <>
cudaError_t resnorm_forward<f16, f16>(ResNormArgs p, bool vec, cudaStream_t st) {
  return resnorm_forward_as<f16, f16>(p, vec, st);
}

template <>
cudaError_t resnorm_backward<f16, f16>(ResNormArgs p, bool vec, int grid, cudaStream_t st) {
  return resnorm_backward_as<f16, f16>(p, vec, grid, st);
}

template <>
cudaError_t resnorm_forward<f16, float>(ResNormArgs p, bool vec, cudaStream_t st) {
  return resnorm_forward_as<f16, float>(p, vec, st);
}

template <>
cudaError_t resnorm_backward<f16, float>(ResNormArgs p, bool vec, int grid, cudaStream_t st) {
  return resnorm_backward_as<f16, float>(p, vec, grid, st);
}

}  // namespace sla
