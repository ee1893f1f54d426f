// The kernels of sla_resnorm.cuh for bf16 data.
#include "sla_resnorm.cuh"

namespace sla {

template <>
cudaError_t resnorm_forward<bf16, bf16>(ResNormArgs p, bool vec, cudaStream_t st) {
  return resnorm_forward_as<bf16, bf16>(p, vec, st);
}

template <>
cudaError_t resnorm_backward<bf16, bf16>(ResNormArgs p, bool vec, int grid, cudaStream_t st) {
  return resnorm_backward_as<bf16, bf16>(p, vec, grid, st);
}

template <>
cudaError_t resnorm_forward<bf16, float>(ResNormArgs p, bool vec, cudaStream_t st) {
  return resnorm_forward_as<bf16, float>(p, vec, st);
}

template <>
cudaError_t resnorm_backward<bf16, float>(ResNormArgs p, bool vec, int grid, cudaStream_t st) {
  return resnorm_backward_as<bf16, float>(p, vec, grid, st);
}

}  // namespace sla
