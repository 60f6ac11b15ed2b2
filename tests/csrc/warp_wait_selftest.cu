// GPU self-test of the warp's bounded wait (sm100.cuh, mbar_wait_warp), which the
// channel recurrence uses: on a phase that never completes it gives up after its
// limit, alike in all lanes, and awaits nothing from then on.
//   out[0] lanes that were late on a barrier nobody arrives on
//   out[1] lanes that were late on one whose phase is complete
//   out[2] nanoseconds of the first wait,  out[3] of a second one after it
#include <cstdint>
#include <cuda_runtime.h>

#include "sm100.cuh"

using namespace gdn::sm100;

__global__ void warp_wait_kernel(unsigned long long limit_ns, unsigned long long* out) {
  __shared__ __align__(8) uint64_t never, done;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&never), 1);
    mbar_init(smem_u32(&done), 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_arrive(smem_u32(&done));
  __syncwarp();
  bool late = false, other = false;
  const unsigned long long t0 = globaltimer_ns();
  mbar_wait_warp(smem_u32(&never), 0, &late, limit_ns);
  const unsigned long long t1 = globaltimer_ns();
  mbar_wait_warp(smem_u32(&never), 0, &late, limit_ns);
  const unsigned long long t2 = globaltimer_ns();
  mbar_wait_warp(smem_u32(&done), 0, &other, limit_ns);
  atomicAdd(out, late);
  atomicAdd(out + 1, other);
  if (threadIdx.x == 0) {
    out[2] = t1 - t0;
    out[3] = t2 - t1;
  }
}

extern "C" int warp_wait_selftest(unsigned long long limit_ns, unsigned long long* out,
                                  void* stream) {
  warp_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(limit_ns, out);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}
