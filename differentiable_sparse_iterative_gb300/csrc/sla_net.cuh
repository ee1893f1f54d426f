// Element types and vector loads of the dense operators (layer norm, gated feed-forward block).
//
// Data is bfloat16, float16 or float32; everything is computed in float32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sla.h"

namespace sla {

using bf16 = __nv_bfloat16;
using f16 = __half;

template <typename T>
struct NetType;
template <>
struct NetType<float> {
  static constexpr int dtype = SLA_F32;
};
template <>
struct NetType<f16> {
  static constexpr int dtype = SLA_F16;
};
template <>
struct NetType<bf16> {
  static constexpr int dtype = SLA_BF16;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(f16 v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }

// Rounded to nearest even; float16 overflows to infinity beyond 65504.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ f16 from_f32<f16>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) {
  return __float2bfloat16_rn(v);
}

// N consecutive elements moved in the widest pieces their size allows (p aligned to them).
template <typename T, int N>
struct alignas(sizeof(T) * N >= 16 ? 16 : sizeof(T) * N) Pack {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ void load_f32(const T *p, float (&out)[N]) {
  const Pack<T, N> q = *reinterpret_cast<const Pack<T, N> *>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = to_f32(q.v[i]);
}

template <typename T, int N>
__device__ __forceinline__ void store_f32(T *p, const float (&in)[N]) {
  Pack<T, N> q;
#pragma unroll
  for (int i = 0; i < N; ++i) q.v[i] = from_f32<T>(in[i]);
  *reinterpret_cast<Pack<T, N> *>(p) = q;
}

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 f2(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// A word of two 16-bit values, or one float32, to and from float32.
__device__ __forceinline__ uint32_t pair16(float a, float b, f16) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pair16(float a, float b, bf16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpair16(uint32_t w, f16) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 unpair16(uint32_t w, bf16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Programmatic dependent launch: a kernel of a chain may start while the one before it still runs; it
// waits here before it touches memory that others write, and lets the next one start in turn.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

// A launch's attributes.  early: it may start before its predecessor in the stream has ended (which then
// has to be a kernel of the same call: others' results are waited for in the ordinary way).
struct LaunchConfig {
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute at[2];
  LaunchConfig(dim3 grid, int block, size_t smem, cudaStream_t st, bool early, int cluster = 1) {
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = at;
    if (cluster > 1) {
      at[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
      at[c.numAttrs].val.clusterDim.x = cluster;
      at[c.numAttrs].val.clusterDim.y = at[c.numAttrs].val.clusterDim.z = 1;
      ++c.numAttrs;
    }
    if (early) {
      at[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[c.numAttrs].val.programmaticStreamSerializationAllowed = 1;
      ++c.numAttrs;
    }
  }
};

inline bool net_dtype(int32_t d) { return d == SLA_F32 || d == SLA_F16 || d == SLA_BF16; }
inline size_t net_size(int32_t d) { return d == SLA_F32 ? 4 : 2; }

// Streaming multiprocessors of the current device (152 on GB300), asked once per device.
int sm_count();

}  // namespace sla
