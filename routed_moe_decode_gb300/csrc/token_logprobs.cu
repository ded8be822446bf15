// Log probabilities of given tokens, log-sum-exp, entropy and the best alternatives of rows of logits
// (include/moe_dense.h), in one pass over them.
//
// A thread keeps a running maximum m of the logits l, s = sum exp(scale (l - m)) and u = sum exp(scale (l - m)) (l - m), each
// rescaled when m rises; joined over a row, lse = scale m + log s and entropy = log s - scale u / s.  The difference comes
// before the scale, so that the largest logit's own term is exactly 1: next to a rounded scale * m, what the rounding left of a
// large logit (half a unit of 1e10 is 512) would be its exponent.
//
// Where one token has more than half of the probability, that 1 would take the digits of all else in s: next to a rest of 1e-6,
// 1 + rest keeps it to 6 %.  So the joins keep the sum of the thread that holds the largest logit apart from the rest, and at
// the end a warp reads that thread's logits again (1 / 256 of the row) and adds them up without the largest; the logarithm is
// log1p of the sum of all others.  (Left out during the pass, it would cost a comparison and a selection for every term.)
// The second reading takes ~1 us at the end of such a row: nothing beside that of the alternatives; without any 13.1 -> 14.0 us
// for 127 rows of 100003 in FP32, 5.5 -> 6.3 for 4 of 131072, 41 -> 54 for 8192 of 8000 in BF16.
//
// Alternatives are keys: the logit's order-preserving bits above the complement of its id, so that equal logits are in
// the order of their ids and no two keys are equal.  The pass keeps only the largest logit of every thread's step (or of a
// few), which the sums need anyway, in shared memory.  At its end the largest logits of groups of threads, as many groups as
// alternatives or more, give a threshold that at least `top` logits reach: the smallest of eight warps', or the top-th of 32
// groups of eight threads.  Only the steps whose largest reaches it are read again, and what reaches it there, some 20
// logits, is sorted by counting.  (With lists kept during the pass, 20 alternatives cost 53 us beside 96 without any for 2048 rows of
// 131072.)  Where very many reach the threshold (nothing but masks, equal logits) each warp keeps a list sorted over its
// lanes, and the row is read again as a whole if need be.
//
// A row is one CTA's, or a cluster's of up to eight where there are few rows; the parts join through distributed shared
// memory in a fixed order.
//
// Measured (graph replays; in brackets where the model is sure of every row's token or of most): 2048 rows of 131072 BF16 logits
// with 5 alternatives 100 us [101] (5.4 TB/s), without any 101 [103]; the same in FP32 181 [186] and 172 [170] (6.2 TB/s); 127 rows of
// 100003 in FP32 with 20 alternatives 17.5 [17.5], without 13.1 [14.0]; 4 rows of 131072 with 8, 8.6 [8.5], without 5.5 [6.3];
// inputs from memory, as many in turn as are larger than L2.  Where masks leave fewer logits than there are groups to give the threshold,
// every logit reaches it and the lists below work for 4 rows of 131072 with 8 alternatives 50 us, for 127 of 100003 with 20, 64.
// The end of a row is a chain of trips through shared memory and back to the logits, 3 to 4 us that other CTAs hide where
// there are more rows than CTAs fit.  The pass is close to the limit of its registers (64 of a thread; see kCtas): how the
// second reading is written moved 2048 rows from 96 to 113 us by what it left for the pass.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "dense.cuh"

namespace moe {
namespace dense {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kVecs = 4;  // 16-byte vectors of a thread's step
constexpr int kParts = 8;  // of a row, at most
constexpr uint32_t kAll = 0xffffffffu;
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

struct Sums {  // of a thread
  float m, s, u;
};
// Of several: m, the largest logit; s, the sum of the terms of thread `at`, which holds it; rest, that of all others; u of all.
// at < 0: s is the largest logit's own term, 1, and nothing else.
struct Joined {
  float m, s, rest, u;
  int at;
};
// Differences of a rescaled sum: no further down, so that s times one is finite; exp of the smallest scale times this is 0.
constexpr float kFarDown = -1e28f;

// Sorted descending over the lanes: the 32 best of two such lists.
__device__ __forceinline__ Key merge(Key a, Key b, int lane) {
  const Key other = __shfl_sync(kAll, b, 31 - lane);
  Key k = a > other ? a : other;
#pragma unroll 1
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
  static __device__ __forceinline__ float first(uint4& r) {  // and the others move up
    const float v = __uint_as_float(r.x);
    r = make_uint4(r.y, r.z, r.w, 0);
    return v;
  }
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
  static __device__ __forceinline__ float first(uint4& r) {
    const float v = __uint_as_float(r.x << 16);
    r = make_uint4(__funnelshift_r(r.x, r.y, 16), __funnelshift_r(r.y, r.z, 16), __funnelshift_r(r.z, r.w, 16), r.w >> 16);
    return v;
  }
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
  static __device__ __forceinline__ float first(uint4& r) {
    const float v = __half2float(__ushort_as_half(static_cast<unsigned short>(r.x & 0xffffu)));
    r = make_uint4(__funnelshift_r(r.x, r.y, 16), __funnelshift_r(r.y, r.z, 16), __funnelshift_r(r.z, r.w, 16), r.w >> 16);
    return v;
  }
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
constexpr int kFound = 256;                // logits that reach the threshold, sorted by one warp

struct Sorted {
  float largest[kGroups][kThreads];
  uint16_t pairs[kPairs];  // thread, group << 8
  int npairs[2], nfound[2];  // of even and odd rows
  union {
    Key found[kFound];
    Key lists[kWarps][32];  // where more than that reach it
  };
  Key result[32];
  Key incoming[kParts][32];               // the best of a cluster's parts
  alignas(16) uint32_t shown[32];         // the largest logit of eight threads, as float_key has it
  uint32_t bar;                           // the top-th of them
};
struct None {};
template <bool TOP>
struct Shared : std::conditional_t<TOP, Sorted, None> {
  Joined sums[2][kWarps];  // of even and odd rows: the first warp may still read one row's when another has the next's
  Joined whole, incoming_sums[kParts];
};

__device__ __forceinline__ float value_of(uint32_t key) { return logit_of(static_cast<Key>(key) << 32); }

// Lanes' keys into a warp's list (0: none).
__device__ __noinline__ Key insert(Key list, Key k, int top, int lane) {
  k = k > __shfl_sync(kAll, list, top - 1) ? k : 0;
  uint32_t want = __ballot_sync(kAll, k != 0);
  if (__popc(want) > 6) {  // as costly as a sort: bitonic, descending over the lanes
#pragma unroll 1
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll 1
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

// How many of 32 keys are before the CTA's key number tid / 8, equal ones by their places: four are compared by each of eight
// threads.
__device__ __forceinline__ int before(const uint32_t (&keys)[32], int tid) {
  const int at = tid >> 3, first = 4 * (tid & 7);
  const uint32_t k = keys[at];
  int n = 0;
#pragma unroll
  for (int i = first; i < first + 4; ++i) n += keys[i] > k - (i < at);  // no key is 0
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) n += __shfl_xor_sync(kAll, n, o);
  return n;
}

// The lists of the first `lists` warps into the first one's.
__device__ __forceinline__ Key best_of_warps(Sorted& sh, Key list, int lists, int warp, int lane) {
  for (int n = lists / 2; n > 0; n >>= 1) {
    if (warp >= n && warp < 2 * n) sh.lists[warp][lane] = list;
    __syncthreads();
    if (warp < n) list = merge(list, sh.lists[warp + n][lane], lane);
  }
  return list;
}
// The lanes' sums into shared memory, in an order that does not change.  (Results and what a rare call needs go through memory: the
// registers belong to the pass.  As a function of its own, with the steps in a loop, it took 8192 rows of 8000 from 41 to 48 us.)
__device__ __forceinline__ void join(float m, float s, float rest, float u, int at, float exp_scale, Joined* to) {
  const float most = value_of(__reduce_max_sync(kAll, float_key(m)));
  const int lane = threadIdx.x & 31, holder = __ffs(__ballot_sync(kAll, m == most)) - 1;
  const float d = fmaxf(m - most, kFarDown), f = exp2_of(d * exp_scale);
  const float all = s + rest;
  u = all != 0.f && f != 0.f ? (u + all * d) * f : 0.f;
  if (lane != holder) rest = all;
  rest = f != 0.f || rest != rest ? rest * f : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    rest += __shfl_xor_sync(kAll, rest, o);
    u += __shfl_xor_sync(kAll, u, o);
  }
  if (lane == holder) *to = {most, s, rest, u, at};
}
__device__ __forceinline__ void join(const Joined* of, int n, float exp_scale, Joined* to) {
  const int lane = threadIdx.x & 31;
  const Joined j = lane < n ? of[lane] : Joined{-FLT_MAX, 0.f, 0.f, 0.f, 0};
  join(j.m, j.s, j.rest, j.u, j.at, exp_scale, to);
}

// Of a row: elements before the first 16-byte boundary, whole vectors (a part's from v0 to v1), the rest.
template <typename T>
struct Row {
  const T* x;
  int head, rest, v0, v1;
  __device__ __forceinline__ Row(const LogprobArgs& a, uint32_t row, int part, int log_parts) {
    x = static_cast<const T*>(a.logits) + row * a.row_stride;
    head = min(a.vocab, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)));
    const int vecs = (a.vocab - head) / Vec<T>::N;
    rest = a.vocab - head - vecs * Vec<T>::N;
    v0 = static_cast<int>(static_cast<uint32_t>(vecs) * part >> log_parts);  // below 2^29 * 8
    v1 = static_cast<int>(static_cast<uint32_t>(vecs) * (part + 1u) >> log_parts);
  }
};

// Whether one logit has most of a sum (it is then the only one of its size).
__device__ __forceinline__ bool one_has_most(const Joined& j) {
  const float all = j.s + j.rest;
  return all > 0.5f && all < 1.9f;
}
// By a warp: the sum of the thread that holds that logit again, without it.
template <typename T>
__device__ __noinline__ void largest_apart(const LogprobArgs& a, uint32_t row, int part, int log_parts, Joined* j) {
  typedef Vec<T> V;
  const float m = j->m, exp_scale = a.exp_scale;
  const int lane = threadIdx.x & 31, at = j->at;
  const Row<T> r(a, row, part, log_parts);
  const uint4* const xv = reinterpret_cast<const uint4*>(r.x + r.head);
  float s = 0.f;
  bool found = false;
  auto add = [&](float l) {
    if (l == m) found = true;
    else s += exp2_of((l - m) * exp_scale);
  };
  const bool alone = lane == 0 && part == 0 && at < r.head + r.rest;  // the thread's logit that is in no vector
  const float single = alone ? to_float(r.x[at < r.head ? at : a.vocab - r.rest + at - r.head]) : -INFINITY;
  constexpr int kAhead = 4;
  for (int i0 = r.v0 + at; i0 < r.v1; i0 += kAhead * 32 * kThreads) {
    uint4 raw[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int i = i0 + (n * 32 + lane) * kThreads;
      raw[n] = i < r.v1 ? __ldcg(xv + i) : make_uint4(V::kLowest, V::kLowest, V::kLowest, V::kLowest);
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      float2 v[V::N / 2];
      V::get(raw[n], v);
#pragma unroll
      for (int e = 0; e < V::N / 2; ++e) {
        add(v[e].x);
        add(v[e].y);
      }
    }
  }
  add(single);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if (__any_sync(kAll, found) && lane == 0) {
    j->s = 1.f;
    j->rest += s;
    j->at = -1;
  }
}

constexpr int kCtas = 4;  // of an SM: 3, with more registers, take 112 us for 2048 rows of 131072 with 5 alternatives (104 at that time)

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, kCtas) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  typedef Vec<T> V;
  constexpr int N = kVecs * V::N;
  __shared__ Shared<TOP> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = static_cast<int>(cluster_size()), log_parts = 31 - __clz(parts), part = static_cast<int>(cluster_rank());
  if constexpr (TOP) {
    if (tid < 2) sh.npairs[tid] = sh.nfound[tid] = 0;
  }
  if (parts > 1) cluster_arrive();
  pdl_wait();
  pdl_launch_dependents();
  const T* x;
  const uint4* xv;
  int head, rest, v0, v1;
  auto go_to = [&](uint32_t row) {
    const Row<T> r(a, row, part, log_parts);
    x = r.x;
    head = r.head;
    rest = r.rest;
    v0 = r.v0;
    v1 = r.v1;
    xv = reinterpret_cast<const uint4*>(x + head);
  };
  const Sums kNoSums{-FLT_MAX, 0.f, 0.f};
  Sums mine;
  const float2 exp_scale = make_float2(a.exp_scale, a.exp_scale);

  auto load = [&](uint4 (&raw)[kVecs], int at) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = at + j * kThreads + tid;
      raw[j] = i < v1 ? __ldcs(xv + i) : make_uint4(V::kLowest, V::kLowest, V::kLowest, V::kLowest);
    }
  };
  auto add = [&](const float2 (&v)[N / 2], float most) {
    const float m = fmaxf(mine.m, most);
    if (m > mine.m) {
      const float d = fmaxf(mine.m - m, kFarDown), f = exp2_of(d * a.exp_scale);
      mine.u = (mine.u + mine.s * d) * f;
      mine.s *= f;
      mine.m = m;
    }
    const float2 down = make_float2(-m, -m);
    float2 s[2], u[2];
    s[0] = s[1] = u[0] = u[1] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 d = add2(v[i], down), t = mul2(d, exp_scale);
      const float2 e = make_float2(exp2_of(t.x), exp2_of(t.y));
      s[i & 1] = add2(s[i & 1], e);
      u[i & 1] = fma2(e, make_float2(fmaxf(d.x, -FLT_MAX), fmaxf(d.y, -FLT_MAX)), u[i & 1]);
    }
    mine.s += (s[0].x + s[0].y) + (s[1].x + s[1].y);
    mine.u += (u[0].x + u[0].y) + (u[1].x + u[1].y);
  };

  uint4 raw[kVecs];
  const uint32_t rows = a.rows, row_step = gridDim.x >> log_parts;
  uint32_t row = blockIdx.x >> log_parts;
  int buffer = 0;
  go_to(row);
  load(raw, v0);
  for (;; buffer ^= 1) {
    mine = kNoSums;
    Key list = 0;
    float best = -INFINITY, group_best = -INFINITY;  // of this thread; of its steps in the group at hand
    // steps, in groups of 2^shift
    const int steps = (v1 - v0 + kVecs * kThreads - 1) / (kVecs * kThreads);
    int shift = 0;
    while (((steps - 1) >> shift) >= kGroups) ++shift;
    const bool finishes = part == 0 && warp == 0;
    int token = -1;
    if (finishes && a.logprobs && lane < a.n_tokens) token = a.tokens[row * a.token_stride + lane];
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
    const float token_logit = token >= 0 && token < a.vocab ? to_float(x[token]) : -INFINITY;
    // elements that are in no vector, 14 at most
    const bool there = finishes && lane < head + rest;
    const int id = lane < head ? lane : a.vocab - rest + lane - head;
    const float single = there ? to_float(x[id]) : -INFINITY;
    if (finishes && head + rest > 0) {
      float2 v[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) v[i] = make_float2(-INFINITY, -INFINITY);
      v[0].x = single;
      add(v, single);
    }
    // what the end of the row needs, before the next row's loads
    const uint4* const row_xv = xv;
    const int row_head = head, row_v0 = v0, row_v1 = v1;
    const uint32_t next_row = row + row_step;
    if (next_row < rows) {
      go_to(next_row);
      load(raw, v0);
    }

    join(mine.m, mine.s, 0.f, mine.u, tid, a.exp_scale, &sh.sums[buffer][warp]);
    if constexpr (TOP) {
    float most = best;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
      if (a.top > kWarps) {
        if ((lane & 7) == 0) sh.shown[tid >> 3] = float_key(most);
      } else {
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
        if (lane == 0) sh.shown[warp] = float_key(most);
      }
      __syncthreads();
      uint32_t bar_key;
      if (a.top > kWarps) {
        if (before(sh.shown, tid) == a.top - 1) sh.bar = sh.shown[tid >> 3];
        __syncthreads();
        bar_key = sh.bar;
      } else {
        bar_key = sh.shown[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) bar_key = min(bar_key, sh.shown[i]);
      }
      if (warp == kWarps - 1) {
        join(sh.sums[buffer], kWarps, a.exp_scale, &sh.whole);
      }
      const float bar = value_of(bar_key);
      // a NaN ranks as -infinity: a group of nothing else has that as its largest
      uint32_t reach = 0;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) reach |= (sh.largest[g][tid] < bar ? 0u : 1u) << g;
      reach &= (1u << ((steps + (1 << shift) - 1) >> shift)) - 1;
      for (; reach; reach &= reach - 1) {
        const int at = atomicAdd(&sh.npairs[buffer], 1);
        if (at < kPairs) sh.pairs[at] = static_cast<uint16_t>(tid | (__ffs(reach) - 1) << 8);
      }
      __syncthreads();
      if (warp == 0) sh.result[lane] = 0;
      const int pairs = sh.npairs[buffer];
      if (tid == 0) sh.npairs[buffer ^ 1] = sh.nfound[buffer ^ 1] = 0;
      if (warp == kWarps - 1 && one_has_most(sh.whole)) largest_apart<T>(a, row, part, log_parts, &sh.whole);
      // the values of vector i, or of none
      auto look = [&](int i, bool there, auto&& take) {
        uint4 r = there ? __ldcg(row_xv + i) : make_uint4(0, 0, 0, 0);
        const int id = row_head + i * V::N;
#pragma unroll 1
        for (int e = 0; e < V::N; ++e) {
          const float l = V::first(r);
          const bool good = there && !(l < bar);
          if (__any_sync(kAll, good)) take(l, id + e, good);
        }
      };
      auto look_at_pairs = [&](auto&& take) {
        const int per = kVecs << shift, log = 31 - __clz(per);
        for (int n0 = warp * 32; n0 < pairs << log; n0 += kThreads) {
          const int n = n0 + lane, pair = n < pairs << log ? sh.pairs[n >> log] : 0, sub = n & (per - 1);
          const int step = ((pair >> 8) << shift) + sub / kVecs;
          const int i = row_v0 + (step * kVecs + sub % kVecs) * kThreads + (pair & 255);
          look(i, n < pairs << log && i < row_v1, take);
        }
      };
      auto find = [&](float l, int id, bool good) {
        if (!good) return;
        const int at = atomicAdd(&sh.nfound[buffer], 1);
        if (at < kFound) sh.found[at] = key_of(l, id);
      };
      if (pairs <= kPairs) {
        look_at_pairs(find);
        find(single, id, there && !(single < bar));
      } else if (tid == 0) {
        sh.nfound[buffer] = kFound + 1;
      }
      __syncthreads();
      const int found = sh.nfound[buffer];
      if (found <= kFound) {
        for (int n0 = 0; n0 < found; n0 += kThreads / 8) {  // a key's place is the number of larger ones: eight threads count
          const int n = n0 + (tid >> 3);
          const Key k = sh.found[min(n, kFound - 1)];
          int at = 0;
          for (int i = tid & 7; i < found; i += 8) at += sh.found[i] > k;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) at += __shfl_xor_sync(kAll, at, o);
          if (n < found && at < 32) sh.result[at] = k;
        }
        __syncthreads();
        if (warp == 0) list = sh.result[lane];
      } else {
        auto keep = [&](float l, int id, bool good) {
          list = insert(list, good ? key_of(l, id) : 0, a.top, lane);
        };
        if (warp == 0) keep(single, id, there);
        if (pairs <= kPairs) look_at_pairs(keep);
        else
          for (int i0 = row_v0 + warp * 32; i0 < row_v1; i0 += kThreads) look(i0 + lane, i0 + lane < row_v1, keep);
        list = best_of_warps(sh, list, kWarps, warp, lane);
      }
    } else {
      __syncthreads();
    }
    if (!TOP && warp == 0) {
      join(sh.sums[buffer], kWarps, a.exp_scale, &sh.whole);
      __syncwarp();
      if (one_has_most(sh.whole)) largest_apart<T>(a, row, part, log_parts, &sh.whole);
      __syncwarp();
    }
    if (parts > 1) {  // of one row: see the launch
      __syncwarp();
      cluster_wait();  // all of them have started
      if (warp == 0) {
        if constexpr (TOP) {
          st_cluster(mapa(smem_addr(&sh.incoming[part][lane]), 0), list);
        }
        if (lane < sizeof(Joined) / 4)
          st_cluster(mapa(smem_addr(&sh.incoming_sums[part]), 0) + 4 * lane, reinterpret_cast<const float*>(&sh.whole)[lane]);
      }
      __syncwarp();
      cluster_sync();
      if (part != 0) return;
      if (warp == (TOP ? kWarps - 1 : 0)) join(sh.incoming_sums, parts, a.exp_scale, &sh.whole);
      if constexpr (TOP) list = best_of_warps(sh, warp < parts ? sh.incoming[warp][lane] : 0, parts, warp, lane);
      else __syncwarp();
    }
    if (finishes) {
      Joined all = sh.whole;
      const float most = all.m * a.scale;
      if (!(most < INFINITY)) all.rest = __int_as_float(0x7fc00000);  // scale * logit is +infinity, of a finite logit too
      const float sum = all.s + all.rest;
      const bool none = sum == 0.f || (most == -INFINITY && sum == sum);  // a NaN beside what has no probability is one
      const float logs = all.at < 0 ? log1pf(all.rest) : logf(sum);
      if (lane == 0) {
        if (a.lse) a.lse[row] = none ? -INFINITY : fmaf(all.m, a.scale, logs);
        if (a.entropy) a.entropy[row] = none ? 0.f : logs - a.scale * (all.u / sum);
      }
      auto logprob = [&](float l) {
        const float d = l - all.m;  // -infinity also where two finite logits are too far apart for their difference
        return none ? -INFINITY : d >= -FLT_MAX ? fmaf(d, a.scale, -logs) : fmaf(l, a.scale, -most) - logs;
      };
      if (a.logprobs) {
        float* const to = a.logprobs + static_cast<int64_t>(row) * a.n_tokens;
        if (lane < a.n_tokens) to[lane] = logprob(token_logit);
        for (int j = lane + 32; j < a.n_tokens; j += 32) {
          const int t = a.tokens[row * a.token_stride + j];
          to[j] = logprob(t >= 0 && t < a.vocab ? to_float((static_cast<const T*>(a.logits) + row * a.row_stride)[t]) : -INFINITY);
        }
      }
      if (TOP && lane < a.top) {
        const int64_t at = static_cast<int64_t>(row) * a.top + lane;
        if (a.top_ids) a.top_ids[at] = static_cast<int>(~static_cast<uint32_t>(list));
        if (a.top_logprobs) a.top_logprobs[at] = logprob(logit_of(list));
      }
    }
    if (next_row >= rows) return;
    row = next_row;
  }
}

template <typename T>
cudaError_t run(const LogprobArgs& a, int sms, cudaStream_t stream) {
  // parts of a row: while all CTAs are resident together, and a part is worth a CTA
  int parts = 1;
  const int64_t most = static_cast<int64_t>(kCtas) * sms;
  while (parts < kParts && static_cast<int64_t>(a.rows) * parts * 2 <= most && a.vocab / (parts * 2) >= 2048) parts *= 2;
  // CTAs of short rows go on from row to row, with the next row's first loads under way at the end of one: 8192 rows of 8000
  // BF16 logits take 41 us, with a CTA for each row 55.  Of rows of more steps the hardware's own order is better: 2048 of 131072
  // 96 us, with CTAs that go on 102.
  const bool keep = a.vocab <= 8 * kVecs * kThreads * Vec<T>::N;
  const int64_t ctas = static_cast<int64_t>(a.rows) * parts;
  const dim3 grid(static_cast<unsigned>(keep ? std::min(ctas, most) : ctas)), block(kThreads);
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
