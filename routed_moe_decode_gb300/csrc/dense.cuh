// Kernels of the dense path around the layer (include/moe_dense.h): norm and quantised rows, block-scaled
// products in 8 bits, log probabilities.
#pragma once

#include <cuda.h>

#include "../../include/moe_dense.h"
#include "launch.cuh"

namespace moe {
namespace dense {

constexpr int kBlock = 128;  // channels of a scale, rows and channels of a weight's scale

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery's round-up method).
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {d, static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
}
__device__ __forceinline__ uint32_t div(const FastDiv& f, uint32_t n) { return (__umulhi(f.mul, n) + n) >> f.shift; }

// Rows of norm_rows.cu; dtype and weight_dtype: MOE_DENSE_*; row r of x and of normed lies at
// (r / inner) * outer stride + (r % inner) * inner stride.
struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* residual_out;
  void* normed;
  uint8_t* codes;
  float* scales;
  int64_t x_outer, x_inner, n_outer, n_inner, r_stride, ro_stride, code_stride, scale_row, scale_block;
  FastDiv inner;
  uint32_t rows;
  int d, dtype, weight_dtype;
  float eps, inv_d, add;  // inv_d: 1 / d; add: 1 where the norm multiplies by 1 + weight
  bool vec;        // every row can be read and written 16 bytes (weights: 8 elements) at a time
  bool vec_codes;  // codes can be written 8 bytes at a time
};
cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t stream);

struct QuantArgs {
  const void* x;
  uint8_t* codes;
  float* scales;
  int64_t x_stride, code_stride, scale_row, scale_block;
  FastDiv nblocks;  // blocks of a row
  uint32_t rows, rows_step;
  int d, dtype;
  bool gated, vec, vec_codes;
};
cudaError_t launch_quantize(const QuantArgs& a, int sms, cudaStream_t stream);

// Block-scaled products.
constexpr uint32_t kWaitCycles = 1u << 31;  // ~1 s: a copy takes microseconds
constexpr int kMaxGroups = 1024;
struct MatmulArgs {
  const uint8_t* x;
  const uint8_t* w;
  const float* xs;
  const float* ws;
  const int* offsets;  // null: one group of all rows
  void* out;
  uint32_t* status;
  int64_t x_stride, scale_row, scale_block, out_stride;
  int rows, n, k, groups, out_dtype;
  uint32_t wait_cycles;
  int copy_arrivals;  // arrivals that a stage's barrier waits for beside its bytes
};
// Rows of a group on average, rounded up.
inline int64_t rows_of_a_group(const MatmulArgs& a) { return (static_cast<int64_t>(a.rows) + a.groups - 1) / a.groups; }
cudaError_t launch_fp8_stream(const MatmulArgs& a, int sms, int split, cudaStream_t stream);
// Parts of k for that kernel, 1 where the rows' tiles keep the SMs busy as they are.
int fp8_stream_split(const MatmulArgs& a, int sms);
// Rows of x in a tile of that kernel, at most, for so many rows (of a group, on average).
constexpr int kFewRows = 32, kSomeRows = 128;
cudaError_t launch_fp8_wide(const MatmulArgs& a, int sms, cudaStream_t stream);
// Map of a matrix of size-byte elements, copied in boxes of 128 bytes x box_rows rows with the 128-byte swizzle; stride in bytes.
int encode_rows_map(CUtensorMap* map, const void* base, int size, uint64_t cols, uint64_t rows, uint64_t stride,
                    uint32_t box_cols, uint32_t box_rows);
inline int encode_fp8_map(CUtensorMap* map, const void* base, uint64_t k, uint64_t rows, uint64_t stride, uint32_t box_rows) {
  return encode_rows_map(map, base, 1, k, rows, stride, 128, box_rows);
}

// Log probabilities.
struct LogprobArgs {
  const void* logits;
  const int* tokens;
  float* logprobs;
  float* lse;
  float* entropy;
  int* top_ids;
  float* top_logprobs;
  int64_t row_stride, token_stride;
  float scale, exp_scale;  // exp_scale: scale * log2(e)
  int rows, vocab, n_tokens, top, dtype;
};
cudaError_t launch_logprobs(const LogprobArgs& a, int sms, cudaStream_t stream);

// Bounded wait of a whole warp for a phase of a barrier.  *limit: cycles that a wait may take, 0 once one of the CTA
// gave up.  False: give up too.
__device__ __forceinline__ uint32_t cycles() {
  uint32_t c;
  asm volatile("mov.u32 %0, %%clock;" : "=r"(c));
  return c;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* limit, uint32_t* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint32_t t0 = cycles();
    while (!(ok = mbar_try_wait(bar, parity))) {
      const uint32_t most = *limit;
      if (cycles() - t0 >= most) {
        if (most) {
          *limit = 0;
          atomicOr(status, MOE_DENSE_TIMEOUT);
        }
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// D[tmem] (+)= A[smem] B[smem]^T of E4M3 codes, FP32 sums.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of it: FP32 sums (bits 4-5 = 1), E4M3 (bits 7-9, 10-12 = 0), both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
        "l"(reinterpret_cast<const unsigned long long&>(c)));
  return d;
}

// The same, where what is multiplied comes from tensor memory: not moved before the wait for it.
__device__ __forceinline__ float2 fma2_in_order(float2 a, float2 b, float2 c) {
  float2 d;
  asm volatile("fma.rn.f32x2 %0, %1, %2, %3;"
               : "=l"(reinterpret_cast<unsigned long long&>(d))
               : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
                 "l"(reinterpret_cast<const unsigned long long&>(c)));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return d;
}

// Clusters.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The two halves of a wait for the cluster's CTAs to have started.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address that `local`, an address of this CTA's shared memory, has in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t mapa(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Clusters of `cluster` CTAs of a kernel that are resident together on the current device (0: it cannot be said).
template <auto Kernel>
int resident_clusters(int cluster, dim3 block, size_t smem) {
  constexpr int kMost = 8;
  static std::atomic<int> known[64][kMost + 1];  // 1 + the number
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64 || cluster > kMost) return 0;
  int n = known[dev][cluster].load(std::memory_order_relaxed);
  if (n == 0) {
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
      return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int most = 0;
    if (cudaOccupancyMaxActiveClusters(&most, Kernel, &cfg) != cudaSuccess) most = 0;
    known[dev][cluster].store(n = 1 + most, std::memory_order_relaxed);
  }
  return n - 1;
}

// launch_ready for clusters of `cluster` CTAs along x (and the SM's memory divided as by default: loads under way need L1).
template <auto Kernel, typename... Args>
cudaError_t launch_cluster(int cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args&&... args) {
  static std::atomic<unsigned long long> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((ready.load(std::memory_order_acquire) >> dev) & 1ull)) {
    if (smem > 48 * 1024)
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, Kernel, static_cast<Args&&>(args)...);
}

}  // namespace dense
}  // namespace moe
