// Grouped routing of one token by one warp.
//
//   s_e   = sigmoid(l_e), or the softmax of the row
//   key_e = s_e + bias_e  (softmax without a bias: l_e itself, whose order is that of s_e)
//   a group's score is its largest key, or the sum of its two largest; the keep_groups groups of
//   the largest scores stay; the k largest keys among their experts are selected, larger first;
//   equal scores and equal keys go to the lower index
//   w_j = scale * s_j / sum_selected s, or scale * s_j
// All in FP32, each operation rounded once as written (no contraction), so that a selection can
// be reproduced bit by bit by the same operations elsewhere.
//
// A NaN logit counts as -infinity and a logit above the largest float as that; a NaN key as
// -infinity.  Experts outside the groups that stay are never selected (their key is below that of
// -infinity); w is 0 where the selected scores sum to 0.
//
// Bound by latency for a step of a few tokens and by instruction issue for thousands (each score
// costs an exponential and a division, ~16 of each a lane at E = 512): lane l holds the experts
// [NPL l, NPL l + NPL) in registers and keeps its best four keys in a sorted list, a selection is
// one warp maximum and one warp minimum, as in the ungrouped router.  Only the groups' scores go
// through shared memory, where the lanes are dealt out evenly over the groups (32 / groups lanes
// each, whatever the group size), so that any group size costs the same.
#include "moe_kernels.cuh"
#include "route_select.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;
constexpr float kInf = INFINITY;

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float(float v) { return v; }
template <>
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }

__device__ __forceinline__ float clean(float l) { return l != l ? -kInf : fminf(l, FLT_MAX); }
__device__ __forceinline__ float sigmoid(float l) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l))); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ void top2(float& a, float& b, float x) {  // a >= b
  b = fmaxf(b, fminf(a, x));
  a = fmaxf(a, x);
}

template <int NPL, typename T>
__global__ void __launch_bounds__(32 * kWarps) route_grouped_kernel(RouteGroupedArgs a) {
  constexpr int C = NPL < 4 ? NPL : 4;
  extern __shared__ float s_keys[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  const int E = a.E, k = a.k, base = NPL * lane;
  const int nvalid = max(0, min(NPL, E - base));
  const T* row = static_cast<const T*>(a.logits) + static_cast<int64_t>(t) * a.row_stride;
  const bool by_logit = a.softmax && a.bias == nullptr;

  float v[NPL];
  constexpr int kVec = 16 / sizeof(T);
  if (NPL % kVec == 0 && a.vec && nvalid == NPL) {
#pragma unroll
    for (int j = 0; j < NPL / kVec; ++j) {
      const uint4 w = reinterpret_cast<const uint4*>(row + base)[j];
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[kVec * j + i] = clean(as_float<T>(e[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = i < nvalid ? clean(as_float<T>(row[base + i])) : -kInf;
  }
  float mx = 0.f, sum = 1.f;  // of the softmax
  if (a.softmax) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) top = max(top, float_key(v[i]));
    mx = key_float(__reduce_max_sync(kFull, top));
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) sum += v[i] == -kInf ? 0.f : expf(v[i] - mx);
    sum = warp_sum(sum);
  }
  auto score_of = [&](float l) {
    if (!a.softmax) return sigmoid(l);
    return l == -kInf ? 0.f : __fdiv_rn(expf(l - mx), sum);
  };
  if (!by_logit) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      if (i >= nvalid) continue;
      float x = score_of(v[i]);
      if (a.bias != nullptr) x = __fadd_rn(x, a.bias[base + i]);
      v[i] = x != x ? -kInf : x;
    }
  }

  uint32_t stay = 0xffffffffu;  // bit g: group g stays
  if (a.keep_groups < a.groups) {
    float* keys = s_keys + warp * E;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (i < nvalid) keys[base + i] = v[i];
    __syncwarp();
    const int sub = 32 / a.groups, grp = lane / sub, part = lane - grp * sub, size = E / a.groups;
    float x = -kInf, y = -kInf;
    if (grp < a.groups) {
      // elements part, part + sub, ... of the group, starting at a place that differs from group to
      // group, since groups a multiple of 32 apart share their banks
      const int n = (size - part + sub - 1) / sub;
      int i = n > 0 ? grp % n : 0;
      for (int c = 0; c < n; ++c) {
        top2(x, y, keys[grp * size + part + i * sub]);
        if (++i == n) i = 0;
      }
    }
    float gx = x, gy = y;  // of the group's lanes together, at its first lane
    for (int o = 1; o < sub; ++o) {
      const float ox = __shfl_down_sync(kFull, x, o), oy = __shfl_down_sync(kFull, y, o);
      top2(gx, gy, ox);
      top2(gx, gy, oy);
    }
    float score = a.top2 && size > 1 ? __fadd_rn(gx, gy) : gx;
    if (score != score) score = -kInf;
    const uint32_t mine = float_key(score);
    int better = 0;
    for (int o = 0; o < a.groups; ++o) {
      const uint32_t other = __shfl_sync(kFull, mine, o * sub);
      better += other > mine || (other == mine && o < grp) ? 1 : 0;
    }
    const uint32_t leads = __ballot_sync(kFull, grp < a.groups && part == 0 && better < a.keep_groups);
    stay = 0;
    for (int o = 0; o < a.groups; ++o) stay |= ((leads >> (o * sub)) & 1u) << o;
  }

  uint32_t key[NPL];
  {
    const int size = E / a.groups;
    int g = base / size, left = size - (base - g * size);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      key[i] = i < nvalid && ((stay >> g) & 1u) ? float_key(v[i]) : 0u;  // 0: below the key of -infinity
      if (--left == 0) {
        ++g;
        left = size;
      }
    }
  }
  uint32_t ck[C];
  int cs[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    ck[c] = 0u;
    cs[c] = 0;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) cache_insert<C>(ck, cs, key[i], i);
  int nused = 0, my_id = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t kmax = __reduce_max_sync(kFull, ck[0]);
    const uint32_t cand = ck[0] == kmax ? static_cast<uint32_t>(base + cs[0]) : 0xffffffffu;
    const uint32_t idx = __reduce_min_sync(kFull, cand);
    if (lane == j) my_id = static_cast<int>(idx);
    const bool own = static_cast<int>(idx / NPL) == lane;
    nused += own ? 1 : 0;
#pragma unroll
    for (int c = 0; c + 1 < C; ++c) {
      ck[c] = own ? ck[c + 1] : ck[c];
      cs[c] = own ? cs[c + 1] : cs[c];
    }
    ck[C - 1] = own ? 0u : ck[C - 1];
  }
  if constexpr (NPL > C) {
    uint32_t unused = 0;
    if (__any_sync(kFull, nused >= C && nvalid > C)) select_scan<NPL>(key, k, unused, my_id);
  }
  float w = lane < k ? score_of(clean(as_float<T>(row[my_id]))) : 0.f;
  if (a.renormalise) {
    const float all = warp_sum(w);
    w = all > 0.f ? __fdiv_rn(__fmul_rn(a.scale, w), all) : 0.f;
  } else {
    w *= a.scale;
  }
  if (lane < k) {
    a.ids[static_cast<int64_t>(t) * k + lane] = my_id;
    a.weights[static_cast<int64_t>(t) * k + lane] = w;
  }
}

template <typename T>
cudaError_t launch(const RouteGroupedArgs& a, cudaStream_t stream) {
  const dim3 grid((a.T + kWarps - 1) / kWarps), block(32 * kWarps);
  const size_t smem = a.keep_groups < a.groups ? size_t(kWarps) * a.E * 4 : 0;
  auto kernel = a.E <= 32    ? route_grouped_kernel<1, T>
                : a.E <= 64  ? route_grouped_kernel<2, T>
                : a.E <= 128 ? route_grouped_kernel<4, T>
                : a.E <= 256 ? route_grouped_kernel<8, T>
                : a.E <= 512 ? route_grouped_kernel<16, T>
                             : route_grouped_kernel<32, T>;
  return launch_pdl(kernel, grid, block, smem, stream, a);
}

}  // namespace

cudaError_t launch_route_grouped(const RouteGroupedArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch<__nv_bfloat16>(a, stream);
    case MOE_DTYPE_FP16: return launch<__half>(a, stream);
    default: return launch<float>(a, stream);
  }
}

}  // namespace moe
