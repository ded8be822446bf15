// Grouped routing of one token by one warp.
//
//   s_e   = sigmoid(l_e), or the softmax of the row
//   key_e = s_e + bias_e  (softmax without a bias: l_e itself, whose order is that of s_e; not where
//           groups are ranked by sums of two keys, since sums of logits have another order)
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
// Bound by latency for a step of a few tokens and by instruction issue for thousands.  Lane l holds
// the experts [NPL l, NPL l + NPL) in registers.  Its best four keys come from a max / min network over
// the keys alone (76 instructions for 16 keys; insertion into a list of (key, index) pairs took 330),
// a selection is one warp maximum and one vote, and the indices of what a lane gave away are found at
// the end by comparing its keys with those.  A group's score is found in registers where the groups
// are made of whole lanes; otherwise the keys go through shared memory, 32 / groups lanes a group.
// Measured: 8192 tokens of 512 scores 18.5 us (~1600 instructions a token; 17.4 MB would take 2.6), with softmax 16.8,
// with softmax and groups ranked by two scores 21.6; 4 tokens 5.2 us, the call's own time.
#include "launch.cuh"
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
__device__ __forceinline__ float sigmoid(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ void top2(float& a, float& b, float x) {  // a >= b
  b = fmaxf(b, fminf(a, x));
  a = fmaxf(a, x);
}

// a >= b after it
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}

// The C largest of N keys, descending (C = min(N, 4)).
template <int N, int C>
__device__ __forceinline__ void best_of(const uint32_t* key, uint32_t (&best)[C]) {
  if constexpr (N == 1) {
    best[0] = key[0];
  } else if constexpr (N == 2) {
    best[0] = key[0];
    best[1] = key[1];
    order(best[0], best[1]);
  } else if constexpr (N == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) best[i] = key[i];
    order(best[0], best[1]);
    order(best[2], best[3]);
    order(best[0], best[2]);
    order(best[1], best[3]);
    order(best[1], best[2]);
  } else {
    uint32_t x[4], y[4];
    best_of<N / 2, 4>(key, x);
    best_of<N / 2, 4>(key + N / 2, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) best[i] = max(x[i], y[3 - i]);  // the four largest, bitonic
    order(best[0], best[2]);
    order(best[1], best[3]);
    order(best[0], best[1]);
    order(best[2], best[3]);
  }
}

template <int NPL, typename T>
__global__ void __launch_bounds__(32 * kWarps) route_grouped_kernel(RouteGroupedArgs a) {
  constexpr int C = NPL < 4 ? NPL : 4;
  extern __shared__ float s_keys[];
  __shared__ int s_ids[kWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  const int E = a.E, k = a.k, base = NPL * lane;
  const int nvalid = max(0, min(NPL, E - base));
  const T* row = static_cast<const T*>(a.logits) + static_cast<int64_t>(t) * a.row_stride;
  const bool sums = a.top2 && a.keep_groups < a.groups && a.groups < E;  // groups are ranked by sums of two keys
  const bool by_logit = a.softmax && a.bias == nullptr && !sums;

  float v[NPL];
  constexpr int kVec = 16 / sizeof(T);
  if (NPL % kVec == 0 && a.vec && nvalid == NPL) {
#pragma unroll
    for (int j = 0; j < NPL / kVec; ++j) {
      const uint4 w = reinterpret_cast<const uint4*>(row + base)[j];
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[kVec * j + i] = as_float<T>(e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = i < nvalid ? as_float<T>(row[base + i]) : -kInf;
  }
  float bias[NPL];
  if (a.bias != nullptr) {
    if (NPL % 4 == 0 && a.vec_bias && nvalid == NPL) {
#pragma unroll
      for (int j = 0; j < NPL / 4; ++j) {
        const float4 w = reinterpret_cast<const float4*>(a.bias + base)[j];
        bias[4 * j] = w.x;
        bias[4 * j + 1] = w.y;
        bias[4 * j + 2] = w.z;
        bias[4 * j + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i) bias[i] = i < nvalid ? a.bias[base + i] : 0.f;
    }
  }
  float mx = 0.f, sum = 1.f;  // of the softmax
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = clean(v[i]);
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
    if (!a.softmax) return sigmoid(fmaxf(l, -kInf));  // of a NaN: 0
    return l == -kInf ? 0.f : __fdiv_rn(expf(l - mx), sum);
  };
  if (!by_logit) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      float x = score_of(v[i]);
      if (a.bias != nullptr) x = __fadd_rn(x, bias[i]);
      v[i] = i < nvalid && x == x ? x : -kInf;
    }
  }

  bool in_whole = true;         // this lane's experts are all in a group that stays (groups of whole lanes)
  uint32_t stay = 0xffffffffu;  // bit g: group g stays
  const int size = E / a.groups;
  const bool whole = size % NPL == 0;
  if (a.keep_groups < a.groups) {
    // the lanes of a group: lead .. lead + lanes - 1
    int lanes, grp, lead;
    float x = -kInf, y = -kInf;  // this lane's two largest keys of its group
    if (whole) {
      lanes = size / NPL;
      grp = lane / lanes;
      lead = grp * lanes;
#pragma unroll
      for (int i = 0; i < NPL; ++i) top2(x, y, v[i]);
    } else {
      float* keys = s_keys + warp * E;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i < nvalid) keys[base + i] = v[i];
      __syncwarp();
      lanes = 32 / a.groups;
      grp = lane / lanes;
      lead = grp * lanes;
      if (grp < a.groups) {
        // elements part, part + lanes, ... of the group, starting at a place that differs from group to
        // group, since groups a multiple of 32 apart share their banks
        const int part = lane - lead, n = (size - part + lanes - 1) / lanes;
        int i = n > 0 ? grp % n : 0;
        for (int c = 0; c < n; ++c) {
          top2(x, y, keys[grp * size + part + i * lanes]);
          if (++i == n) i = 0;
        }
      }
    }
    float gx = x, gy = y;  // of the group's lanes together, at its first lane
    for (int o = 1; o < lanes; ++o) {
      const float ox = __shfl_down_sync(kFull, x, o), oy = __shfl_down_sync(kFull, y, o);
      top2(gx, gy, ox);
      top2(gx, gy, oy);
    }
    float score = a.top2 && size > 1 ? __fadd_rn(gx, gy) : gx;
    if (score != score) score = -kInf;
    const uint32_t mine = float_key(score);
    int better = 0;
    for (int o = 0; o < a.groups; ++o) {
      const uint32_t other = __shfl_sync(kFull, mine, o * lanes);
      better += other > mine || (other == mine && o < grp) ? 1 : 0;
    }
    const uint32_t leads = __ballot_sync(kFull, grp < a.groups && lane == lead && better < a.keep_groups);
    if (whole) {
      in_whole = grp < a.groups && ((leads >> lead) & 1u);
    } else {
      stay = 0;
      for (int o = 0; o < a.groups; ++o) stay |= ((leads >> (o * lanes)) & 1u) << o;
    }
  }

  uint32_t key[NPL];  // 0: below the key of -infinity
  if (whole || a.keep_groups == a.groups) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = i < nvalid && in_whole ? float_key(v[i]) : 0u;
  } else {
    int g = base / size, left = size - (base - g * size);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      key[i] = i < nvalid && ((stay >> g) & 1u) ? float_key(v[i]) : 0u;
      if (--left == 0) {
        ++g;
        left = size;
      }
    }
  }
  uint32_t best[C];
  best_of<NPL, C>(key, best);
  int given = 0;          // how many of its keys this lane gave away,
  uint32_t given_to = 0;  // in which rounds (a byte each),
  uint32_t gave[C];       // and which
#pragma unroll
  for (int c = 0; c < C; ++c) gave[c] = best[c];
  bool over = false;
  for (int j = 0; j < k; ++j) {
    const uint32_t kmax = __reduce_max_sync(kFull, best[0]);
    // the lowest lane that holds it: its experts have the lowest indices
    if (lane == __ffs(__ballot_sync(kFull, best[0] == kmax)) - 1) {
      over |= given >= C;
      given_to |= static_cast<uint32_t>(j) << (8 * (given & 3));
      ++given;
#pragma unroll
      for (int c = 0; c + 1 < C; ++c) best[c] = best[c + 1];
      best[C - 1] = 0u;
    }
  }
  int my_id = 0;
  if (__any_sync(kFull, over || (given >= C && nvalid > C))) {
    uint32_t unused = 0;
    select_scan<NPL>(key, k, unused, my_id);
  } else {
    uint32_t used = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!__any_sync(kFull, c < given)) break;
      uint32_t at = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) at |= key[i] == gave[c] ? 1u << i : 0u;
      at &= ~used;
      at &= 0u - at;  // equal keys: the lower index first
      used |= at;
      if (c < given) s_ids[warp][(given_to >> (8 * c)) & 0xffu] = base + __ffs(at) - 1;
    }
    __syncwarp();
    if (lane < k) my_id = s_ids[warp][lane];
  }
  float w = lane < k ? score_of(a.softmax ? clean(as_float<T>(row[my_id])) : as_float<T>(row[my_id])) : 0.f;
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

template <int NPL, typename T>
cudaError_t launch(const RouteGroupedArgs& a, cudaStream_t stream) {
  const dim3 grid((a.T + kWarps - 1) / kWarps), block(32 * kWarps);
  const bool shared = a.keep_groups < a.groups && (a.E / a.groups) % NPL != 0;
  return launch_ready<route_grouped_kernel<NPL, T>>(grid, block, shared ? size_t(kWarps) * a.E * 4 : 0, stream, a);
}

template <typename T>
cudaError_t launch_for(const RouteGroupedArgs& a, cudaStream_t stream) {
  return a.E <= 32    ? launch<1, T>(a, stream)
         : a.E <= 64  ? launch<2, T>(a, stream)
         : a.E <= 128 ? launch<4, T>(a, stream)
         : a.E <= 256 ? launch<8, T>(a, stream)
         : a.E <= 512 ? launch<16, T>(a, stream)
                      : launch<32, T>(a, stream);
}

}  // namespace

cudaError_t launch_route_grouped(const RouteGroupedArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch_for<__nv_bfloat16>(a, stream);
    case MOE_DTYPE_FP16: return launch_for<__half>(a, stream);
    default: return launch_for<float>(a, stream);
  }
}

}  // namespace moe
