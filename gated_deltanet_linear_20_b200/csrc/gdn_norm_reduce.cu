// The second launch of the norms' gradients: the CTAs' partial sums of the weight
// gradients are added in a fixed order.
#include "gdn_norm.cuh"

namespace gdn {
namespace {

// 32 columns a CTA; warp i adds the parts i, i + 32, ..., then the warps are added.
// The launch may start before the parts are complete: it waits for the launch
// before it first.
constexpr int kReduceWarps = 32;
__global__ void __launch_bounds__(32 * kReduceWarps)
    reduce_parts_kernel(const float* part, int n, int cols, float* d0, float* d1, float* d2, int D) {
  __shared__ float sum[kReduceWarps][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 10
    for (int p = w; p < n; p += kReduceWarps) s += part[size_t(p) * cols + c];
  }
  sum[w][lane] = s;
  __syncthreads();
  // warp w adds column w: lane i has the sum of warp i
  s = sum[lane][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + w;
  if (lane == 0 && col < cols) (col < D ? d0 : col < 2 * D ? d1 : d2)[col % D] = s;
}

}  // namespace

int launch_reduce_parts(const float* part, int n, int cols, float* const* dst, int D,
                        cudaStream_t stream) {
  const int weights = cols / D;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((cols + 31) / 32);
  cfg.blockDim = dim3(32 * kReduceWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at{};  // its start overlaps the end of the launch before it
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, &reduce_parts_kernel, part, n, cols, dst[0],
                            weights > 1 ? dst[1] : static_cast<float*>(nullptr),
                            weights > 2 ? dst[2] : static_cast<float*>(nullptr), D) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_LAUNCH;
}

}  // namespace gdn
