// Bounded waits that have expired, counted by the kernels and reported to the host.
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

#include "sla_host.h"
#include "sla_tc.cuh"

namespace sla {
namespace {

constexpr int kDevices = 64;

std::mutex expired_mutex;
std::atomic<uint32_t *> expired_count[kDevices];
thread_local bool expired_met[kDevices];  // this thread has been here
thread_local uint32_t expired_told[kDevices];

uint32_t read_count(const Expired &x) { return *(const volatile uint32_t *)x.count; }

// A wait that nothing ends, of a quarter of a millisecond, counted as the products' kernels count theirs.
__global__ void __launch_bounds__(32) expire_wait(uint32_t *timeouts) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) mbar_init(&bar, 1);
  __syncwarp();
  if (!mbar_wait_clocks(&bar, 0, 500000) && threadIdx.x == 0) atomicAdd_system(timeouts, 1u);
}

}  // namespace

Expired expired() {
  Expired x;
  x.err = cudaGetDevice(&x.dev);
  if (x.err == cudaSuccess && x.dev >= kDevices) x.err = cudaErrorInvalidDevice;
  if (x.err != cudaSuccess) return x;
  x.count = expired_count[x.dev].load();
  if (!x.count) {
    std::lock_guard<std::mutex> lock(expired_mutex);
    x.count = expired_count[x.dev].load();
    if (!x.count) {
      cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // another thread's capture has nothing to do with this
      cudaThreadExchangeStreamCaptureMode(&mode);
      x.err = cudaHostAlloc((void **)&x.count, sizeof(uint32_t), cudaHostAllocPortable | cudaHostAllocMapped);
      cudaThreadExchangeStreamCaptureMode(&mode);
      if (x.err != cudaSuccess) return x;
      *x.count = 0;
      expired_count[x.dev].store(x.count);
    }
  }
  if (!expired_met[x.dev]) {
    expired_met[x.dev] = true;
    expired_told[x.dev] = read_count(x);
  }
  return x;
}

sla_status report_expired(const Expired &x) {
  const uint32_t n = read_count(x);
  if (n == expired_told[x.dev]) return SLA_OK;
  expired_told[x.dev] = n;
  return SLA_TIMEOUT;
}

}  // namespace sla

using namespace sla;

extern "C" {

SLA_API sla_status sla_gated_ffn_check(void *stream) {
  const Expired x = expired();
  if (x.err != cudaSuccess) return fail(x.err);
  const cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  return e == cudaSuccess ? report_expired(x) : fail(e);
}

SLA_API sla_status sla_test_expire_wait(void *stream) {
  const Expired x = expired();
  if (x.err != cudaSuccess) return fail(x.err);
  expire_wait<<<1, 32, 0, (cudaStream_t)stream>>>(x.count);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

}  // extern "C"
