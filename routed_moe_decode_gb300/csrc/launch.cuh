// Host-side parts of the kernels around the layer (grouped router, 4-bit K/V cache).  They are not in
// moe_kernels.cuh, so that the expert kernels' sources, by which the committed DRAM captures are recognised,
// change with the expert kernels only.
#pragma once

#include <atomic>

#include "moe_kernels.cuh"

namespace moe {

// launch_pdl for a kernel whose attributes do not change between calls: they are set at its first
// launch on a device (two driver calls of ~1 us each are as long as a small kernel).
template <auto Kernel, typename... Args>
cudaError_t launch_ready(dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args&&... args) {
  static std::atomic<unsigned long long> ready{0};  // bit d: done on device d
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((ready.load(std::memory_order_acquire) >> dev) & 1ull)) {
    if (smem > 48 * 1024)  // such a kernel always asks for the same amount
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               static_cast<int>(cudaSharedmemCarveoutMaxShared));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, Kernel, static_cast<Args&&>(args)...);
}

// Grouped router (route_grouped.cu); vec: rows can be read 16 bytes at a time.
struct RouteGroupedArgs {
  const void* logits;
  int64_t row_stride;
  const float* bias;
  int32_t* ids;
  float* weights;
  int T, E, k, groups, keep_groups, dtype;
  bool softmax, top2, renormalise;
  bool vec, vec_bias;  // 16-byte loads of the logits, of the bias
  float scale;
};
cudaError_t launch_route_grouped(const RouteGroupedArgs& a, cudaStream_t stream);

void set_last_cuda_error(const char* where, cudaError_t e);
// SMs of the current device (MOE_OK or a status).
int device_sms(int* sms);

}  // namespace moe
