// What the two attention kernels of the 4-bit cache share: the items of the work and a place in them.
#pragma once

#include "kv4_common.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
// A row's reference m is set kBelow under its largest score (all in powers of two) and moves only when a score
// exceeds it by more than kSlack: p stays below 2^15, inside FP16, and the sums are rescaled a few times instead
// of at every tile.  The row's largest p is then at least 2^7, and what FP16 cannot hold of a small p (2^-25)
// is below 2^-32 of the largest: with m at the largest score itself it was 2^-25, and the many small p of a long
// row beside one large score were in l but not in the output.
constexpr float kSlack = 15.0f, kBelow = 7.0f;

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
constexpr uint32_t kDrainCycles = 1u << 24;  // ~8 ms, for what is in flight after a wait gave up

// Cycles, of which differences below 2^32 count: every wait has its own copy of the comparison.
__device__ __forceinline__ uint32_t cycles() { return static_cast<uint32_t>(clock()); }

// Whether a barrier's phase is complete.
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

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
  __device__ __forceinline__ int len(int s) const { return max(lens != nullptr ? lens[s] : step_len(a.c, s), 0); }
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
    lens[lane] = step_len(a.c, lane);
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

}  // namespace
}  // namespace kv4
}  // namespace moe
