// Log probabilities of given tokens, log-sum-exp, entropy and the best alternatives of rows of logits
// (include/moe_dense.h), in one pass over them.
//
// A thread keeps a running maximum m of x = scale * logit, s = sum exp(x - m) and u = sum exp(x - m) (x - m), each
// rescaled when m rises; joined over a row, lse = m + log s and entropy = log s - u / s.
//
// Alternatives are keys: the logit's order-preserving bits above the complement of its id, so that equal logits are in
// the order of their ids and no two keys are equal.  A warp keeps its best 32 sorted over its lanes.  What cannot be
// among the best is told from the maximum of a thread's values, which the sums need anyway, against a threshold: the
// warp's own last place, or the smallest of all warps' ceil(top / 8)-th places (together they have `top` better ones).
//
// A row is one CTA's, or a cluster's of up to eight where there are few rows; the parts join through distributed shared
// memory in a fixed order.
#include <cfloat>

#include "dense.cuh"

namespace moe {
namespace dense {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kVecs = 4;  // 16-byte vectors of a thread's step
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

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(uint4 r, float* v) {
    v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y); v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return __ldcg(p); }
  static constexpr uint32_t kLowest = 0xff800000u;
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 r, float* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static constexpr uint32_t kLowest = 0xff80ff80u;
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 r, float* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = p.x;
      v[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ float one(const __half* p) { return __half2float(*p); }
  static constexpr uint32_t kLowest = 0xfc00fc00u;
};

struct Shared {
  Key lists[kWarps][32];
  Sums sums[kWarps];
  float level[kWarps];  // a warp's ceil(top / 8)-th best logit, -infinity before it has as many
  // a cluster's parts, at its first CTA
  Key part_lists[8][32];
  Sums part_sums[8];
};

// A warp's best keys.
struct Best {
  Key list;     // lane i: the i-th best, 0 where there is none
  float floor;  // the warp's `top`-th best logit
};
template <int N>
__device__ __forceinline__ void offer(Best& b, const float (&v)[N], const int (&id0)[kVecs], const int (&valid)[kVecs],
                                      int top, int place, float bar, volatile float* level, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    constexpr int PER = N / kVecs;
    const float l = v[i];
    Key k = 0;
    if (i % PER < valid[i / PER] && !(l < bar)) k = key_of(l, id0[i / PER] + i % PER);
    const Key last = __shfl_sync(kAll, b.list, top - 1);
    uint32_t want = __ballot_sync(kAll, k > last);
    while (want) {
      const int src = __ffs(want) - 1;
      want &= want - 1;
      const Key c = __shfl_sync(kAll, k, src);
      const int at = __popc(__ballot_sync(kAll, b.list > c));
      const Key up = __shfl_up_sync(kAll, b.list, 1);
      if (lane == at) b.list = c;
      else if (lane > at) b.list = up;
    }
  }
  const Key last = __shfl_sync(kAll, b.list, top - 1), at = __shfl_sync(kAll, b.list, place - 1);
  b.floor = last ? logit_of(last) : -INFINITY;
  if (lane == 0) *level = at ? logit_of(at) : -INFINITY;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
  typedef Vec<T> V;
  constexpr int N = kVecs * V::N;
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = static_cast<int>(cluster_size()), part = static_cast<int>(cluster_rank());
  if (TOP && lane == 0) sh.level[warp] = -INFINITY;
  __syncthreads();
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
  Best best{0, -INFINITY};
  const int place = (a.top + kWarps - 1) / kWarps;

  auto take = [&](const float (&v)[N], const int (&id0)[kVecs], const int (&valid)[kVecs]) {
    float most = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) most = fmaxf(most, v[i]);
    const float m = fmaxf(mine.m, most * a.scale);
    if (m > mine.m) {
      const float d = fmaxf(mine.m - m, -1e30f), f = exp2_of(d * kLog2e);
      mine.u = (mine.u + mine.s * d) * f;
      mine.s *= f;
      mine.m = m;
    }
    float2 s = make_float2(0.f, 0.f), u = s;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float d0 = fmaf(v[i], a.scale, -m), d1 = fmaf(v[i + 1], a.scale, -m);
      const float e0 = exp2_of(d0 * kLog2e), e1 = exp2_of(d1 * kLog2e);
      s.x += e0; s.y += e1;
      u = fma2(make_float2(e0, e1), make_float2(fmaxf(d0, -FLT_MAX), fmaxf(d1, -FLT_MAX)), u);
    }
    mine.s += s.x + s.y;
    mine.u += u.x + u.y;
    if constexpr (TOP) {
      float bar = *const_cast<volatile float*>(&sh.level[0]);
#pragma unroll
      for (int w = 1; w < kWarps; ++w) bar = fminf(bar, *const_cast<volatile float*>(&sh.level[w]));
      bar = fmaxf(bar, best.floor);
      // a NaN ranks as -infinity, and so does a maximum of NaNs alone
      if (__any_sync(kAll, !(most < bar))) offer<N>(best, v, id0, valid, a.top, place, bar, &sh.level[warp], lane);
    }
  };

  for (int at = v0; at < v1; at += kVecs * kThreads) {
    uint4 raw[kVecs];
    int id0[kVecs], valid[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = at + j * kThreads + tid;
      raw[j] = i < v1 ? __ldcs(xv + i) : make_uint4(V::kLowest, V::kLowest, V::kLowest, V::kLowest);
      id0[j] = head + i * V::N;
      valid[j] = i < v1 ? V::N : 0;
    }
    float v[N];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) V::get(raw[j], v + j * V::N);
    take(v, id0, valid);
  }
  if (part == 0 && head + rest > 0 && warp == 0) {  // at most 14 elements
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = -INFINITY;
    const int id = lane < head ? lane : a.vocab - rest + lane - head;
    const bool there = lane < head + rest;
    if (there) v[0] = V::one(x + id);
    const int id0[kVecs] = {id, 0, 0, 0}, valid[kVecs] = {there ? 1 : 0, 0, 0, 0};
    take(v, id0, valid);
  }

  // the CTA's sums and lists
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.m = __shfl_xor_sync(kAll, mine.m, o);
    b.s = __shfl_xor_sync(kAll, mine.s, o);
    b.u = __shfl_xor_sync(kAll, mine.u, o);
    // the same order on both sides
    mine = (lane & o) ? join(b, mine) : join(mine, b);
  }
  if (lane == 0) sh.sums[warp] = mine;
  if constexpr (TOP) {
    for (int n = kWarps / 2; n > 0; n >>= 1) {
      sh.lists[warp][lane] = best.list;
      __syncthreads();
      if (warp < n) best.list = merge(best.list, sh.lists[warp + n][lane], lane);
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  if (warp == 0) {
    mine = sh.sums[0];
    for (int w = 1; w < kWarps; ++w) mine = join(mine, sh.sums[w]);
  }
  if (parts > 1) {
    if (warp == 0) {
      if (TOP) sh.part_lists[0][lane] = best.list;
      if (lane == 0) sh.part_sums[0] = mine;
    }
    __syncwarp();
    cluster_sync();
    if (part == 0 && warp == 0) {
      for (int p = 1; p < parts; ++p) {
        const uint32_t at = mapa(smem_addr(&sh.part_sums[0]), p);
        mine = join(mine, Sums{ld_cluster(at), ld_cluster(at + 4), ld_cluster(at + 8)});
        if (TOP) best.list = merge(best.list, ld_cluster_u64(mapa(smem_addr(&sh.part_lists[0][lane]), p)), lane);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  if (part != 0 || warp != 0) return;
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
      a.logprobs[row * a.n_tokens + j] = logprob(t >= 0 && t < a.vocab ? V::one(x + t) : -INFINITY);
    }
  }
  if (TOP && lane < a.top) {
    const int id = static_cast<int>(~static_cast<uint32_t>(best.list));
    if (a.top_ids) a.top_ids[row * a.top + lane] = id;
    if (a.top_logprobs) a.top_logprobs[row * a.top + lane] = logprob(logit_of(best.list));
  }
}

template <typename T>
cudaError_t run(const LogprobArgs& a, int sms, cudaStream_t stream) {
  // parts of a row: while all CTAs are resident together, and a part is worth a CTA
  int parts = 1;
  while (parts < 8 && static_cast<int64_t>(a.rows) * parts * 2 <= 4 * sms && a.vocab / (parts * 2) >= 2048) parts *= 2;
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
