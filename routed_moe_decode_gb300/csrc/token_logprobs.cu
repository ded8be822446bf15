// Log probabilities of given tokens, log-sum-exp, entropy and the best alternatives of rows of logits
// (include/moe_dense.h), in one pass over them.
//
// A thread keeps a running maximum m of x = scale * logit, s = sum exp(x - m) and u = sum exp(x - m) (x - m), each
// rescaled when m rises; joined over a row, lse = m + log s and entropy = log s - u / s.
//
// Alternatives are keys: the logit's order-preserving bits above the complement of its id, so that equal logits are in
// the order of their ids and no two keys are equal.  The pass keeps only the largest logit of every thread's step (or of a
// few), which the sums need anyway, in shared memory.  At its end each warp shows its threads' four largest logits; the
// top-th of these 32 is a threshold that at least `top` logits reach.  Only the steps whose largest reaches it, about `top`
// of them, are read again, and what reaches it there is put into lists that the warps keep sorted over their lanes.  (With lists
// kept during the pass, 20 alternatives cost 53 us beside 96 without any for 2048 rows of 131072, and 13 beside 11 for 127 of 100003.)
// Where very many reach the threshold (nothing but masks, equal logits) the row is read again as a whole.
//
// A row is one CTA's, or a cluster's of up to eight where there are few rows; the parts join through distributed shared
// memory in a fixed order.
#include <cfloat>
#include <type_traits>

#include "dense.cuh"

namespace moe {
namespace dense {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kVecs = 4;  // 16-byte vectors of a thread's step
constexpr int kShown = 32 / kWarps;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896340736f;
typedef unsigned long long Key;

__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ Key key_of(float logit, int id) {
  const float v = logit == logit ? logit : -INFINITY;
  return (static_cast<Key>(float_key(v)) << 32) | static_cast<uint32_t>(~id);
}
__device__ __forceinline__ float logit_of(Key k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ Key shfl_xor(Key k, int o) { return __shfl_xor_sync(kAll, k, o); }

struct Sums {
  float m, s, u;
};
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  if (b.m > a.m) { const Sums t = a; a = b; b = t; }
  const float d = fmaxf(b.m - a.m, -1e30f), f = exp2_of(d * kLog2e);
  if (b.s != 0.f && f != 0.f) {
    a.u += (b.u + b.s * d) * f;
    a.s += b.s * f;
  } else if (b.s != b.s) {
    a.s = b.s;
  }
  return a;
}

// Sorted descending over the lanes: the 32 best of two such lists.
__device__ __forceinline__ Key merge(Key a, Key b, int lane) {
  const Key other = __shfl_sync(kAll, b, 31 - lane);
  Key k = a > other ? a : other;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Key p = shfl_xor(k, o);
    k = ((lane & o) == 0) == (k > p) ? k : p;
  }
  return k;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

// A 16-byte vector: its values in pairs, and the largest value of a step's.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kLowest = 0xff800000u;
  static __device__ __forceinline__ void get(uint4 r, float2* v) {
    v[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
    v[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  static __device__ __forceinline__ float most(const uint4 (&)[kVecs], const float2 (&v)[kVecs * N / 2]) {
    float m = fmaxf(v[0].x, v[0].y);
#pragma unroll
    for (int i = 1; i < kVecs * N / 2; ++i) m = fmaxf(m, fmaxf(v[i].x, v[i].y));
    return m;
  }
};
template <typename P>
__device__ __forceinline__ P most_pair(const uint4 (&r)[kVecs]) {
  P m = *reinterpret_cast<const P*>(&r[0].x);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    if (j) m = __hmax2(m, *reinterpret_cast<const P*>(&r[j].x));
    m = __hmax2(m, *reinterpret_cast<const P*>(&r[j].y));
    m = __hmax2(m, *reinterpret_cast<const P*>(&r[j].z));
    m = __hmax2(m, *reinterpret_cast<const P*>(&r[j].w));
  }
  return m;
}
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kLowest = 0xff80ff80u;
  static __device__ __forceinline__ void get(uint4 r, float2* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ float most(const uint4 (&r)[kVecs], const float2 (&)[kVecs * N / 2]) {
    const float2 m = __bfloat1622float2(most_pair<__nv_bfloat162>(r));
    return fmaxf(m.x, m.y);
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static constexpr uint32_t kLowest = 0xfc00fc00u;
  static __device__ __forceinline__ void get(uint4 r, float2* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
  }
  static __device__ __forceinline__ float most(const uint4 (&r)[kVecs], const float2 (&)[kVecs * N / 2]) {
    const float2 m = __half22float2(most_pair<__half2>(r));
    return fmaxf(m.x, m.y);
  }
};

constexpr int kGroups = 8, kPairs = 1024;  // steps, or groups of them, whose largest logits are kept; of those read again

struct Sorted {
  float largest[kGroups][kThreads];
  uint16_t pairs[kPairs];  // thread, group << 8
  int npairs;
  Key lists[kWarps][32];
  uint32_t shown[kWarps * kShown];  // logits of each warp, as float_key has them
  Key part_list[32];                // a cluster's parts read this
};
struct None {};
template <bool TOP>
struct Shared : std::conditional_t<TOP, Sorted, None> {
  Sums sums[kWarps];
  Sums part_sums;  // a cluster's parts read this
};

__device__ __forceinline__ float value_of(uint32_t key) { return logit_of(static_cast<Key>(key) << 32); }

// Lanes' keys into a warp's list (0: none).
__device__ __noinline__ Key insert(Key list, Key k, int top, int lane) {
  k = k > __shfl_sync(kAll, list, top - 1) ? k : 0;
  uint32_t want = __ballot_sync(kAll, k != 0);
  if (__popc(want) > 6) {  // as costly as a sort: bitonic, descending over the lanes
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
      for (int o = size >> 1; o > 0; o >>= 1) {
        const Key p = shfl_xor(k, o);
        const bool larger = ((lane & o) == 0) == ((lane & size) == 0);
        k = larger == (k > p) ? k : p;
      }
    return merge(list, k, lane);
  }
  while (want) {
    const Key c = __shfl_sync(kAll, k, __ffs(want) - 1);
    want &= want - 1;
    const int at = __popc(__ballot_sync(kAll, list > c));
    const Key up = __shfl_up_sync(kAll, list, 1);
    list = lane < at ? list : lane == at ? c : up;
  }
  return list;
}

// The top-th largest of the lanes' keys.
__device__ __forceinline__ uint32_t nth(uint32_t k, int top, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint32_t p = __shfl_xor_sync(kAll, k, o);
      k = ((lane & o) == 0) == ((lane & size) == 0) ? max(k, p) : min(k, p);
    }
  return __shfl_sync(kAll, k, top - 1);
}

// The warp's lists into the first warp's.
template <bool TOP>
__device__ __forceinline__ Key best_of_warps(Shared<TOP>& sh, Key list, int warp, int lane) {
  if constexpr (TOP) {
    for (int n = kWarps / 2; n > 0; n >>= 1) {
      if (warp >= n && warp < 2 * n) sh.lists[warp][lane] = list;
      __syncthreads();
      if (warp < n) list = merge(list, sh.lists[warp + n][lane], lane);
    }
  } else {
    __syncthreads();
  }
  return list;
}
// With the sums of the lane `o` away, in the same order on both sides.
__device__ __forceinline__ Sums joined(Sums a, int o, int lane) {
  const Sums b{__shfl_xor_sync(kAll, a.m, o), __shfl_xor_sync(kAll, a.s, o), __shfl_xor_sync(kAll, a.u, o)};
  return (lane & o) ? join(b, a) : join(a, b);
}

constexpr int kCtas = 4;  // of an SM

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, kCtas) logprobs_kernel(const LogprobArgs a) {
  typedef Vec<T> V;
  constexpr int N = kVecs * V::N;
  __shared__ Shared<TOP> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = static_cast<int>(cluster_size()), part = static_cast<int>(cluster_rank());
  if constexpr (TOP) {
    if (tid == 0) sh.npairs = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x / parts;
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  // elements before the first 16-byte boundary, whole vectors, the rest
  const int head = min(a.vocab, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)));
  const int vecs = (a.vocab - head) / V::N, rest = a.vocab - head - vecs * V::N;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  const int v0 = static_cast<int>(static_cast<int64_t>(vecs) * part / parts);
  const int v1 = static_cast<int>(static_cast<int64_t>(vecs) * (part + 1) / parts);

  Sums mine{-FLT_MAX, 0.f, 0.f};
  Key list = 0;
  float best = -INFINITY, group_best = -INFINITY;  // of this thread; of its steps in the group at hand
  // steps, in groups of 2^shift
  const int steps = (v1 - v0 + kVecs * kThreads - 1) / (kVecs * kThreads);
  int shift = 0;
  while (((steps - 1) >> shift) >= kGroups) ++shift;
  const float2 scale = make_float2(a.scale, a.scale), log2e = make_float2(kLog2e, kLog2e);

  auto load = [&](uint4 (&raw)[kVecs], int at) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = at + j * kThreads + tid;
      raw[j] = i < v1 ? __ldcs(xv + i) : make_uint4(V::kLowest, V::kLowest, V::kLowest, V::kLowest);
    }
  };
  auto add = [&](const float2 (&v)[N / 2], float most) {
    const float m = fmaxf(mine.m, most * a.scale);
    if (m > mine.m) {
      const float d = fmaxf(mine.m - m, -1e30f), f = exp2_of(d * kLog2e);
      mine.u = (mine.u + mine.s * d) * f;
      mine.s *= f;
      mine.m = m;
    }
    const float2 down = make_float2(-m, -m);
    float2 s[2], u[2];
    s[0] = s[1] = u[0] = u[1] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 d = fma2(v[i], scale, down), t = mul2(d, log2e);
      const float2 e = make_float2(exp2_of(t.x), exp2_of(t.y));
      s[i & 1] = add2(s[i & 1], e);
      u[i & 1] = fma2(e, make_float2(fmaxf(d.x, -FLT_MAX), fmaxf(d.y, -FLT_MAX)), u[i & 1]);
    }
    mine.s += (s[0].x + s[0].y) + (s[1].x + s[1].y);
    mine.u += (u[0].x + u[0].y) + (u[1].x + u[1].y);
  };

  uint4 raw[kVecs];
  if (v0 < v1) load(raw, v0);
  for (int at = v0; at < v1; at += kVecs * kThreads) {
    uint4 next[kVecs];
    const bool more = at + kVecs * kThreads < v1;
    if (more) load(next, at + kVecs * kThreads);
    float2 v[N / 2];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) V::get(raw[j], v + j * (V::N / 2));
    const float most = V::most(raw, v);
    add(v, most);
    if constexpr (TOP) {
      group_best = fmaxf(group_best, most);
      const int step = (at - v0) / (kVecs * kThreads);
      if (!more || ((step + 1) & ((1 << shift) - 1)) == 0) {
        sh.largest[step >> shift][tid] = group_best;
        best = fmaxf(best, group_best);
        group_best = -INFINITY;
      }
    }
    if (more) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) raw[j] = next[j];
    }
  }
  if (part == 0 && head + rest > 0 && warp == 0) {  // at most 14 elements
    const int id = lane < head ? lane : a.vocab - rest + lane - head;
    const bool there = lane < head + rest;
    float2 v[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = make_float2(-INFINITY, -INFINITY);
    if (there) v[0].x = to_float(x[id]);
    add(v, v[0].x);
    if constexpr (TOP) list = insert(list, there ? key_of(v[0].x, id) : 0, a.top, lane);
  }

  if constexpr (TOP) {
    uint32_t k = float_key(best);
#pragma unroll
    for (int p = 0; p < kShown; ++p) {
      const uint32_t w = __reduce_max_sync(kAll, k);
      if (lane == p) sh.shown[warp * kShown + p] = w;
      if (lane == __ffs(__ballot_sync(kAll, k == w)) - 1) k = 0;
    }
    __syncthreads();
    const float bar = value_of(nth(sh.shown[lane], a.top, lane));
    // a NaN ranks as -infinity: a group of nothing else has that as its largest
    for (int g = 0; g <= (steps - 1) >> shift && steps; ++g) {
      if (!(sh.largest[g][tid] < bar)) {
        const int at = atomicAdd(&sh.npairs, 1);
        if (at < kPairs) sh.pairs[at] = static_cast<uint16_t>(tid | g << 8);
      }
    }
    __syncthreads();
    // vector i, or none: its values into the list
    auto look = [&](int i, bool there) {
      const uint4 r = there ? __ldcg(xv + i) : make_uint4(0, 0, 0, 0);
      float2 v[V::N / 2];
      V::get(r, v);
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        const float l = e & 1 ? v[e / 2].y : v[e / 2].x;
        const bool good = there && !(l < bar);
        if (__any_sync(kAll, good)) list = insert(list, good ? key_of(l, head + i * V::N + e) : 0, a.top, lane);
      }
    };
    const int pairs = sh.npairs;
    if (pairs <= kPairs) {
      const int per = kVecs << shift, log = 31 - __clz(per);
      for (int n0 = warp * 32; n0 < pairs << log; n0 += kThreads) {
        const int n = n0 + lane, pair = n < pairs << log ? sh.pairs[n >> log] : 0, sub = n & (per - 1);
        const int step = ((pair >> 8) << shift) + sub / kVecs;
        const int i = v0 + (step * kVecs + sub % kVecs) * kThreads + (pair & 255);
        look(i, n < pairs << log && i < v1);
      }
    } else {
      for (int i0 = v0 + warp * 32; i0 < v1; i0 += kThreads) look(i0 + lane, i0 + lane < v1);
    }
  }

  // the CTA's sums and lists
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine = joined(mine, o, lane);
  if (lane == 0) sh.sums[warp] = mine;
  list = best_of_warps<TOP>(sh, list, warp, lane);
  if (warp == 0) {
    mine = sh.sums[lane & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) mine = joined(mine, o, lane);
  }
  if (parts > 1) {
    if (warp == 0) {
      if constexpr (TOP) sh.part_list[lane] = list;
      if (lane == 0) sh.part_sums = mine;
    }
    __syncwarp();
    cluster_sync();
    if (part == 0) {  // a warp has a part's list, a lane a part's sums
      if constexpr (TOP) {
        list = warp < parts ? ld_cluster_u64(mapa(smem_addr(&sh.part_list[lane]), warp)) : 0;
        list = best_of_warps<TOP>(sh, list, warp, lane);
      }
      if (warp == 0) {
        const uint32_t at = mapa(smem_addr(&sh.part_sums), lane & (parts - 1));
        mine = Sums{ld_cluster(at), ld_cluster(at + 4), ld_cluster(at + 8)};
        for (int o = parts / 2; o > 0; o >>= 1) mine = joined(mine, o, lane);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  if (part != 0 || warp != 0) return;
  if (!(mine.m < INFINITY)) mine.s = __int_as_float(0x7fc00000);  // scale * logit is +infinity, of a finite logit too
  const bool none = mine.s == 0.f;
  const float logs = logf(mine.s);
  if (lane == 0) {
    if (a.lse) a.lse[row] = none ? -INFINITY : mine.m + logs;
    if (a.entropy) a.entropy[row] = none ? 0.f : logs - mine.u / mine.s;
  }
  auto logprob = [&](float l) { return none ? -INFINITY : fmaf(l, a.scale, -mine.m) - logs; };
  if (a.logprobs) {
    for (int j = lane; j < a.n_tokens; j += 32) {
      const int t = a.tokens[row * a.token_stride + j];
      a.logprobs[row * a.n_tokens + j] = logprob(t >= 0 && t < a.vocab ? to_float(x[t]) : -INFINITY);
    }
  }
  if (TOP && lane < a.top) {
    const int id = static_cast<int>(~static_cast<uint32_t>(list));
    if (a.top_ids) a.top_ids[row * a.top + lane] = id;
    if (a.top_logprobs) a.top_logprobs[row * a.top + lane] = logprob(logit_of(list));
  }
}

template <typename T>
cudaError_t run(const LogprobArgs& a, int sms, cudaStream_t stream) {
  // parts of a row: while all CTAs are resident together, and a part is worth a CTA
  int parts = 1;
  const int64_t most = static_cast<int64_t>(kCtas) * sms;
  while (parts < 8 && static_cast<int64_t>(a.rows) * parts * 2 <= most && a.vocab / (parts * 2) >= 2048) parts *= 2;
  const dim3 grid(static_cast<unsigned>(a.rows) * parts), block(kThreads);
  return a.top > 0 ? launch_cluster<logprobs_kernel<T, true>>(parts, grid, block, 0, stream, a)
                   : launch_cluster<logprobs_kernel<T, false>>(parts, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int sms, cudaStream_t stream) {
  if (a.dtype == MOE_DENSE_FP32) return run<float>(a, sms, stream);
  if (a.dtype == MOE_DENSE_BF16) return run<__nv_bfloat16>(a, sms, stream);
  return run<__half>(a, sms, stream);
}

}  // namespace dense
}  // namespace moe
