// What the two attention kernels of the 4-bit cache share: the items of the work and a place in
// them, the end of a row, and the kernel that joins the items that were cut.
#pragma once

#include "kv4_common.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
// A row's reference m moves only when a score exceeds it by more than this (in powers of two): p
// stays below 2^8, far inside FP16, and the sums are rescaled a few times instead of at every tile.
constexpr float kSlack = 8.0f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr float kLowest = -3.0e38f;  // a row's reference before it has seen a token
constexpr int kStatusTimeout = static_cast<int>(MOE_KV4_TIMEOUT);
constexpr long long kWaitCycles = 1ll << 32;   // ~2 s: a copy takes microseconds
constexpr long long kDrainCycles = 1ll << 24;

// A sequence's items.
struct Item {
  int s;         // sequence
  int row0, n;   // its rows
  int len;       // its tokens
  int first;     // position of its first row
  int lo, units; // first unit and number of units of each of its items
  int blocks;    // row blocks
  int items;     // heads * blocks (0: no rows)
};

constexpr long long kMaxTokens = 1ll << 30;

// The step's rows and the lengths: of up to kSeqCache sequences they are kept in shared memory, so
// that the step from one item to the next costs no trip to memory.
constexpr int kSeqCache = 256;
struct Steps {
  const AttendArgs& a;
  const int* cu;    // shared: [seqs + 1], [seqs]; nullptr past kSeqCache
  const int* lens;
  __device__ __forceinline__ int row(int s) const { return min(max(cu != nullptr ? cu[s] : ld(a.cu + s), 0), a.rows); }
  __device__ __forceinline__ int len(int s) const { return max(lens != nullptr ? lens[s] : ld(a.c.lens + s), 0); }
};

// a / b, a >= 0: nearly always of 32 bits, whose division is far shorter.
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a <= 0x7fffffffll ? static_cast<long long>(static_cast<unsigned>(a) / static_cast<unsigned>(b)) : a / b;
}

template <int ROWS, int UNIT_TOKENS>
__device__ __forceinline__ Item item_of(const Steps& st, int s) {
  const AttendArgs& a = st.a;
  Item it;
  it.s = s;
  it.row0 = st.row(s);
  it.n = max(st.row(s + 1) - it.row0, 0);
  it.items = 0;
  it.units = 1;
  if (it.n == 0) return it;
  const long long room = min(static_cast<long long>(a.c.max_pages) * a.c.page_size, kMaxTokens);
  it.len = static_cast<int>(min(static_cast<long long>(st.len(s)), room));
  it.first = it.len - it.n;
  const int from = a.window > 0 ? max(it.first - a.window + 1, 0) : 0;
  it.lo = min(from, max(it.len - 1, 0)) / UNIT_TOKENS;
  it.units = max((it.len + UNIT_TOKENS - 1) / UNIT_TOKENS - it.lo, 1);
  it.blocks = static_cast<int>((static_cast<long long>(it.n) * a.group + ROWS - 1) / ROWS);
  it.items = a.c.heads * it.blocks;
  return it;
}
__device__ __forceinline__ long long work_of(const Item& it) { return static_cast<long long>(it.items) * it.units; }

// t / tiles_per_page = umulhi(t, magic): exact for t below 2^26 (2^30 tokens) and up to 64 tiles a page
inline uint32_t page_magic(const Cache& c) {
  return static_cast<uint32_t>(((1ull << 32) + c.tiles_per_page - 1) / c.tiles_per_page);
}

// A place in the work: an item and the part of it that lies in a chunk.
struct Walk {
  Item it;
  int idx, off, count;  // item of the sequence, first unit of the item, units
  int more;             // 0: past the chunk
  long long pos;
};

// The next item's part of a chunk that ends at `end`; more is 0 past it.
template <int ROWS, int UNIT_TOKENS>
__device__ __forceinline__ void advance(const Steps& steps, const Walk& cur, Walk& nxt, long long end) {
  nxt = cur;
  nxt.pos += cur.count;
  nxt.more = nxt.pos < end;
  if (!nxt.more) return;
  nxt.off = 0;  // the chunk goes on past this item
  if (++nxt.idx == nxt.it.items) {
    nxt.idx = 0;
    int s = nxt.it.s;
    do nxt.it = item_of<ROWS, UNIT_TOKENS>(steps, ++s); while (nxt.it.items == 0);
  }
  nxt.count = static_cast<int>(min(end - nxt.pos, static_cast<long long>(nxt.it.units)));
}

// The place of position `begin` of the work in a chunk that ends at `end`: in w.it, a sequence's items,
// which begin at `at`.
__device__ __forceinline__ void settle_in(long long at, long long begin, long long end, Walk& w) {
  w.pos = begin;
  w.idx = static_cast<int>(quotient(begin - at, w.it.units));
  w.off = static_cast<int>(begin - at - static_cast<long long>(w.idx) * w.it.units);
  w.count = static_cast<int>(min(end - begin, static_cast<long long>(w.it.units - w.off)));
  w.more = 1;
}

// The same from the sequences s, s + 1, ..., of which the first begins at `at`.
template <int ROWS, int UNIT_TOKENS>
__device__ __forceinline__ void settle(const Steps& steps, int s, long long at, long long begin, long long end, Walk& w) {
  for (;; ++s) {
    w.it = item_of<ROWS, UNIT_TOKENS>(steps, s);
    const long long n = work_of(w.it);
    if (begin < at + n) break;
    at += n;
  }
  settle_in(at, begin, end, w);
}

// A chunk of the work and its first part, found by a warp alone, for up to 32 sequences (a lane a sequence):
// the sums over a block take longer (one short sequence 12.1 against 11.3 us, long documents 116 against 114).  Fills cu and
// lens (every warp of a CTA with the same values).  False: there is nothing in the chunk.
struct Chunk {
  long long per, begin, end;
};
template <int ROWS, int UNIT_TOKENS>
__device__ __forceinline__ bool settle_warp(const AttendArgs& a, int* cu, int* lens, int chunk, Chunk& c, Walk* w) {
  const int lane = threadIdx.x & 31, n = a.c.seqs;
  if (lane < n) {
    cu[lane] = ld(a.cu + lane);
    lens[lane] = ld(a.c.lens + lane);
    if (lane == n - 1) cu[n] = ld(a.cu + n);
  }
  __syncwarp();
  Item it;
  it.items = 0;
  it.units = 1;
  if (lane < n) it = item_of<ROWS, UNIT_TOKENS>(Steps{a, cu, lens}, lane);
  const long long mine = work_of(it);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const long long total = __shfl_sync(0xffffffffu, upto, 31);
  c.per = quotient(total + a.chunks - 1, a.chunks);
  c.begin = c.per * chunk;
  c.end = min(c.begin + c.per, total);
  if (c.begin >= c.end) return false;
  if (w != nullptr && c.begin >= upto - mine && c.begin < upto) {
    w->it = it;
    settle_in(upto - mine, c.begin, c.end, *w);
  }
  __syncwarp();
  return true;
}

// Exclusive prefix sum of one value per thread over the block, and the block's sum.
template <int W>
__device__ __forceinline__ long long block_prefix(long long v, long long* sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long before = 0;
  total = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  return before + x - v;
}

// Channels c, c + 1 of row r (step row r / group, query head r % group of K/V head h) of the step that
// begins at row0: from the sums, their reference m and the sum l.
template <int D>
__device__ __forceinline__ void finish(const AttendArgs& a, int row0, int h, int r, int c, float v0, float v1, float m, float l) {
  const int step_row = r / a.group, hq = h * a.group + r - step_row * a.group;
  const int64_t at = static_cast<int64_t>(row0 + step_row) * (a.c.heads * a.group) + hq;
  const bool seen = l > 0.f || l != l;
  const float f = seen ? a.v_ts / l : 0.f;
  *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + 2 * (at * D + c)) = pack2(v0 * f, v1 * f, a.fp16);
  if (c == 0 && a.lse != nullptr) a.lse[at] = seen ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Joins the parts of the items that were cut.  CTA (b, n): n-tile n of the items that begin in the
// chunks [b kJoinChunks, + kJoinChunks) and go on past them.  A warp takes one m-tile of the output
// and every GROUPS-th part of the item.  It is all latency, so the sums of a batch of parts are under
// way before their m and l are here: two trips to memory for up to 16 GROUPS parts.
constexpr int kJoinThreads = 512, kJoinChunks = 8;
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttendArgs a) {
  constexpr int ROWS = 8 * NT, KS = D / 16, PART = ROWS * D + 2 * ROWS, GROUPS = kJoinThreads / 32 / KS;
  constexpr int DEEP = 16, BATCH = DEEP * GROUPS;
  __shared__ float s_w[BATCH][8], s_l[BATCH][8];  // m of a batch of parts, then their weights; their l
  __shared__ float s_top[8], s_total[8], s_worth[8];  // of the batches so far
  __shared__ float4 s_sum[kJoinThreads];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, k = warp % KS, group = warp / KS, n = blockIdx.y;
  const int q = lane & 3;
  // lane l of every warp looks at the CTA's chunk l
  int4 px = make_int4(0, 0, 0, 0), py = px;
  if (lane < kJoinChunks && blockIdx.x * kJoinChunks + lane < a.chunks) {
    const int4* pp = reinterpret_cast<const int4*>(a.pieces + blockIdx.x * kJoinChunks + lane);
    px = __ldcg(pp);
    py = __ldcg(pp + 1);
  }
  uint32_t on = __ballot_sync(0xffffffffu, px.x != 0 && 8 * n < py.x);
  for (; on != 0; on &= on - 1) {
    const int src = __ffs(on) - 1, c0 = blockIdx.x * kJoinChunks + src;
    const int parts = __shfl_sync(0xffffffffu, px.y, src) - c0 + 1, row0 = __shfl_sync(0xffffffffu, px.z, src);
    const int r0 = __shfl_sync(0xffffffffu, px.w, src), nrows = __shfl_sync(0xffffffffu, py.x, src);
    const int h = __shfl_sync(0xffffffffu, py.y, src);
    // of the chunk c0 + c: the first chunk's part starts at the item's first unit
    auto part_of = [&](int c) { return a.part + (2 * static_cast<size_t>(c0 + c) + (c == 0 ? 1 : 0)) * PART; };
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tid < 8) {
      s_top[tid] = kLowest;
      s_total[tid] = 0.f;
    }
    for (int cb = 0; cb < parts; cb += BATCH) {
      const int nb = min(BATCH, parts - cb);
      for (int i = tid; i < 8 * nb; i += kJoinThreads) {
        const float* p = part_of(cb + (i >> 3)) + ROWS * D + 8 * n + (i & 7);
        s_w[i >> 3][i & 7] = __ldcg(p);
        s_l[i >> 3][i & 7] = __ldcg(p + ROWS);
      }
      float4 z[DEEP];
#pragma unroll
      for (int j = 0; j < DEEP; ++j)
        if (group + j * GROUPS < nb)
          z[j] = __ldcg(reinterpret_cast<const float4*>(part_of(cb + group + j * GROUPS)) + (n * KS + k) * 32 + lane);
      __syncthreads();
      if (warp < 8) {  // a warp a row
        const float old = s_top[warp];
        float top = old, l = 0.f;
        for (int c = lane; c < nb; c += 32) top = fmaxf(top, s_w[c][warp]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (int c = lane; c < nb; c += 32) {
          const float w = exp2_approx(s_w[c][warp] - top);
          s_w[c][warp] = w;
          l += w * s_l[c][warp];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
          const float f = exp2_approx(old - top);
          s_top[warp] = top;
          s_total[warp] = s_total[warp] * f + l;
          s_worth[warp] = f;
        }
      }
      __syncthreads();
      const float f0 = s_worth[2 * q], f1 = s_worth[2 * q + 1];
      v.x *= f0; v.y *= f1; v.z *= f0; v.w *= f1;
#pragma unroll
      for (int j = 0; j < DEEP; ++j)
        if (group + j * GROUPS < nb) {
          const float w0 = s_w[group + j * GROUPS][2 * q], w1 = s_w[group + j * GROUPS][2 * q + 1];
          v.x += w0 * z[j].x; v.y += w1 * z[j].y; v.z += w0 * z[j].z; v.w += w1 * z[j].w;
        }
      __syncthreads();  // the weights have been used
    }
    if constexpr (GROUPS > 1) {
      s_sum[tid] = v;
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int j = 1; j < GROUPS; ++j) {
          const float4 y = s_sum[tid + j * KS * 32];
          v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
      }
    }
    if (group == 0) {
      const int c = (lane >> 2) * (D / 8) + 2 * k, r = 8 * n + 2 * q;
      if (r < nrows) finish<D>(a, row0, h, r0 + r, c, v.x, v.z, s_top[2 * q], s_total[2 * q]);
      if (r + 1 < nrows) finish<D>(a, row0, h, r0 + r + 1, c, v.y, v.w, s_top[2 * q + 1], s_total[2 * q + 1]);
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace kv4
}  // namespace moe
