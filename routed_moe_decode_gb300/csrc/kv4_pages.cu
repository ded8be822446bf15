// Pages of the 4-bit cache: reserve (allocate, copy on write), fork, trim and compact.
//
// The tables, lengths and reference counts live on the device, so a serving step allocates and
// frees without a host wait.  The bookkeeping is a few integers per sequence and page and is
// bound by latency: fork and trim take a CTA or a warp per sequence; the allocation is one CTA,
// because the free pages have to be handed out in one fixed order (lowest number to the first
// sequence that needs one), and reads the counts 4096 pages a round until it has enough.  The
// data moves (copy on write, compaction) are separate grids over every layer and are bound by
// the bytes they read and write.
//
// Measured: forking 16 prompts into 128 branches and reserving for them on 48 layers (906 MB copied, the 16 sources
// from L2) 127 us; one prompt into 4 on 12 layers 11 us, bound by three launches; compaction of 64 steps on 48 layers with the calls
// around it (23 MB in 16-byte pieces) 25 us.
#include "kv4_common.cuh"

namespace moe {
namespace kv4 {

namespace {

constexpr int kAllocThreads = 1024;
constexpr int kNeedShared = 2048;  // sequences whose needs and lengths are kept in shared memory

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return tokens / page_size + (tokens % page_size != 0);
}

// Exclusive prefix sum over the block of (need, copies) packed as need << 32 | copies; returns
// the sum over the block in `total`.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* warp_sums,
                                                         unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warp_sums is free
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned long long s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[31];
  return x - v + (warp ? warp_sums[warp - 1] : 0ull);
}

// One sequence's entry of the allocation: pages needed before it (bits 32 up), pages copied
// before it (bits 2 to 31), whether its last page is copied (bit 0) and whether its table has no
// room (bit 1).
typedef unsigned long long Entry;
__device__ __forceinline__ int entry_start(Entry e) { return static_cast<int>(e >> 32); }
__device__ __forceinline__ int entry_rank(Entry e) { return static_cast<int>((e >> 2) & 0x3fffffffu); }
constexpr Entry kCopy = 1, kRefused = 2;

__device__ __forceinline__ int first_free(const Cache& c, int p0, unsigned& free) {
  free = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (p0 + i < c.pages && ld(c.refs + p0 + i) == 0) free |= 1u << i;
  return __popc(free);
}

// One CTA.  1: what every sequence needs and the running sums; 2: the free pages are counted, as
// far as they are needed; 3: the i-th free page goes to the sequence whose needs cover i, if all
// its needs are met; 4: lengths, refusals, and the counts of the pages that were replaced by a copy.  Pages
// given up by a copy are counted down only in 4, so that none is handed out here while the copy
// still has to read it.
__global__ void __launch_bounds__(kAllocThreads) reserve_kernel(PageArgs a) {
  __shared__ unsigned long long warp_sums[32];
  __shared__ Entry s_entry[kNeedShared + 1];
  __shared__ int s_len[kNeedShared], s_grow[kNeedShared];
  __shared__ int s_copies;
  pdl_wait();
  pdl_launch_dependents();
  const Cache& c = a.c;
  const int tid = threadIdx.x;
  const bool kept = c.seqs <= kNeedShared;
  Entry* entry = kept ? s_entry : a.need;  // [seqs + 1]
  unsigned free0;  // of the first 4096 pages, which mostly are enough: under way with the lengths
  const int n0 = first_free(c, 4 * tid, free0);
  if (tid == 0) s_copies = 0;
  const int per = (c.seqs + kAllocThreads - 1) / kAllocThreads;
  const int s0 = min(tid * per, c.seqs), s1 = min(s0 + per, c.seqs);
  Entry mine = 0;  // needs << 32 | copies << 2
  for (int s = s0; s < s1; ++s) {
    const int len = max(ld(c.lens + s), 0), grow = max(ld(a.a + s), 0);
    if (kept) {
      s_len[s] = len;
      s_grow[s] = grow;
    }
    Entry flags = 0;
    int need = 0;
    if (grow > 0) {
      const long long end = static_cast<long long>(len) + grow;
      const long long want = (end + c.page_size - 1) / c.page_size;
      const int have = pages_of(len, c.page_size);
      if (want > c.max_pages || end > 0x7fffffffll) {
        flags = kRefused;
      } else {
        if (len % c.page_size != 0) {
          const int last = ld(c.table + static_cast<size_t>(s) * c.max_pages + have - 1);
          if (last >= 0 && last < c.pages && ld(c.refs + last) > 1) flags = kCopy;
        }
        need = static_cast<int>(want) - have + static_cast<int>(flags & kCopy);
      }
    }
    entry[s] = (static_cast<Entry>(need) << 32) | flags;
    mine += (static_cast<Entry>(need) << 32) | ((flags & kCopy) << 2);
  }
  Entry total;
  Entry at = block_scan(mine, warp_sums, total);
  for (int s = s0; s < s1; ++s) {
    const Entry e = entry[s];
    entry[s] = at | (e & 3u);
    at += (e >> 32 << 32) | ((e & kCopy) << 2);
  }
  const int all = entry_start(total);
  if (tid == 0) entry[c.seqs] = total;
  __syncthreads();

  unsigned free;
  int found = 0, rank0 = 0, first_round = 0;
  for (int base = 0; base < c.pages && found < all; base += 4 * kAllocThreads) {
    unsigned long long round;
    const int n = base == 0 ? n0 : first_free(c, base + 4 * tid, free);
    const int before_me = found + static_cast<int>(block_scan(static_cast<unsigned>(n), warp_sums, round));
    if (base == 0) {
      rank0 = before_me;
      first_round = static_cast<int>(round);
    }
    found += static_cast<int>(round);
  }
  const int got = min(found, all);
  int seen = 0;
  for (int base = 0; base < c.pages && seen < got; base += 4 * kAllocThreads) {
    int rank = rank0;
    if (base == 0) {
      free = free0;
      seen = first_round;
    } else {
      unsigned long long round;
      const int n = first_free(c, base + 4 * tid, free);
      rank = seen + static_cast<int>(block_scan(static_cast<unsigned>(n), warp_sums, round));
      seen += static_cast<int>(round);
    }
    for (; free != 0 && rank < got; free &= free - 1, ++rank) {
      const int page = base + 4 * tid + __ffs(free) - 1;
      int lo = 0, hi = c.seqs - 1;  // the last sequence that starts at or before `rank`: it needs the page
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (entry_start(entry[mid]) <= rank) lo = mid; else hi = mid - 1;
      }
      const Entry e = entry[lo];
      if (entry_start(entry[lo + 1]) > got) continue;  // not all its needs are met
      const int slot = rank - entry_start(e), copy = static_cast<int>(e & kCopy);
      int* row = c.table + static_cast<size_t>(lo) * c.max_pages;
      const int have = pages_of(kept ? s_len[lo] : max(ld(c.lens + lo), 0), c.page_size);
      if (copy && slot == 0) {
        a.copies[1 + 2 * entry_rank(e)] = ld(row + have - 1);
        a.copies[2 + 2 * entry_rank(e)] = page;
      }
      row[have + slot - copy] = page;
      c.refs[page] = 1;
    }
  }
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int grow = kept ? s_grow[s] : max(ld(a.a + s), 0);
    if (grow == 0) continue;
    const Entry e = entry[s];
    const int end = entry_start(entry[s + 1]);
    if ((e & kRefused) || (end > got && end > entry_start(e))) {
      atomicOr(c.status, static_cast<int>(MOE_KV4_NO_PAGE));
      c.refused[s] = 1;
      continue;
    }
    c.refused[s] = 0;
    c.lens[s] = (kept ? s_len[s] : max(ld(c.lens + s), 0)) + grow;
    if (e & kCopy) {
      atomicSub(c.refs + a.copies[1 + 2 * entry_rank(e)], 1);
      atomicAdd(&s_copies, 1);
    }
  }
  __syncthreads();
  if (tid == 0) a.copies[0] = s_copies;  // the sequences that were refused pages are the last that need some
}

// The pages that reserve_kernel replaced, on every layer, kCopyBytes at a time: one copy and layer's
// pieces go to the CTAs that come next, so that the last of them end together whatever a page's size.
constexpr int kCopyThreads = 256, kCopyLoads = 4;
constexpr int kCopyBytes = 32 * kCopyThreads * kCopyLoads;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(PageArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const Cache& c = a.c;
  const long long pieces = (static_cast<long long>(c.page_bytes) + kCopyBytes - 1) / kCopyBytes;
  const long long units = static_cast<long long>(ld(a.copies)) * c.layers * pieces;
  const size_t layer_bytes = static_cast<size_t>(c.pages) * c.page_bytes;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long il = u / pieces;
    const int i = static_cast<int>(il / c.layers), layer = static_cast<int>(il - static_cast<long long>(i) * c.layers);
    const long long first = (u - il * pieces) * kCopyBytes + 32 * threadIdx.x;
    uint8_t* base = c.pool + layer * layer_bytes + first;
    const uint8_t* src = base + static_cast<size_t>(ld(a.copies + 1 + 2 * i)) * c.page_bytes;
    uint8_t* dst = base + static_cast<size_t>(ld(a.copies + 2 + 2 * i)) * c.page_bytes;
    Line v[kCopyLoads];
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (first + 32 * kCopyThreads * j < static_cast<long long>(c.page_bytes)) v[j] = load_line(src + 32 * kCopyThreads * j);
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (first + 32 * kCopyThreads * j < static_cast<long long>(c.page_bytes)) store_line(dst + 32 * kCopyThreads * j, v[j]);
  }
}

// Table entry j of a sequence from `from` on leaves it: its page has one reference less.
__device__ __forceinline__ void drop_entry(const Cache& c, int* entry) {
  const int page = ld(entry);
  if (page >= 0 && page < c.pages) atomicSub(c.refs + page, 1);
  *entry = -1;
}

__global__ void __launch_bounds__(128) fork_kernel(PageArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const Cache& c = a.c;
  const int s = ld(a.a + blockIdx.x), d = ld(a.b + blockIdx.x);
  if (s < 0 || s >= c.seqs || d < 0 || d >= c.seqs || s == d) {
    if (threadIdx.x == 0) atomicOr(c.status, static_cast<int>(MOE_KV4_BAD_SEQ));
    return;
  }
  const int len = max(ld(c.lens + s), 0);
  const int n = min(pages_of(len, c.page_size), c.max_pages);
  const int* from = c.table + static_cast<size_t>(s) * c.max_pages;
  int* to = c.table + static_cast<size_t>(d) * c.max_pages;
  for (int j = threadIdx.x; j < c.max_pages; j += blockDim.x) {
    const int old = ld(to + j), page = j < n ? ld(from + j) : -1;
    if (old >= 0 && old < c.pages) atomicSub(c.refs + old, 1);
    if (page >= 0 && page < c.pages) atomicAdd(c.refs + page, 1);
    if (old != page) to[j] = page;
  }
  if (threadIdx.x == 0) {
    c.lens[d] = len;
    c.refused[d] = 0;
  }
}

// Sequence s keeps `to` tokens: a warp takes its further pages out of the table.
__device__ __forceinline__ void cut(const Cache& c, int s, int len, int to) {
  const int lane = threadIdx.x & 31;
  const int keep = pages_of(to, c.page_size), have = min(pages_of(len, c.page_size), c.max_pages);
  int* row = c.table + static_cast<size_t>(s) * c.max_pages;
  for (int j = keep + lane; j < have; j += 32) drop_entry(c, row + j);
  if (lane == 0 && to != len) c.lens[s] = to;
}

constexpr int kTrimWarps = 4;
__global__ void __launch_bounds__(32 * kTrimWarps) trim_kernel(PageArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int s = blockIdx.x * kTrimWarps + (threadIdx.x >> 5);
  if (s >= a.c.seqs) return;
  const int len = max(ld(a.c.lens + s), 0);
  const int to = min(max(ld(a.a + s), 0), len);
  cut(a.c, s, len, to);
  if (to != len && (threadIdx.x & 31) == 0) a.c.refused[s] = 0;
}

// The kept rows of sequence s's step, as bits: row i of the first 64.
__device__ __forceinline__ unsigned long long kept_rows(const PageArgs& a, const StepRows& st) {
  const int lane = threadIdx.x & 31, n = min(st.n, kStepRows);
  const unsigned lo = __ballot_sync(0xffffffffu, lane < n && ld(a.keep + st.first + lane) != 0);
  const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < n && ld(a.keep + st.first + lane + 32) != 0);
  return (static_cast<unsigned long long>(hi) << 32) | lo;
}

// grid (units of one sequence / kMoveThreads, sequences).  A unit is one piece of a token's bytes on one
// layer and head: D / 32 pieces of 16 bytes of K codes, as many of V codes, one of D / 16 bytes of
// K scales and one of V scales.  Its thread moves that piece of every kept row, in order; a row
// only ever moves to an earlier place, which by then has been read, so no other thread has to be
// waited for.  Eight rows are read before the first of them is written.  The sequence's last CTA to
// have looked at its length and table cuts it to what it keeps (the moves need neither again).
constexpr int kMoveThreads = 128;  // 64 steps on 48 layers: 25.3 us with the calls around it, 256 threads 28.8, 64 26.0
template <int D>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(PageArgs a) {
  __shared__ int s_page_from[kStepRows], s_page_to[kStepRows], s_from[kStepRows], s_to[kStepRows];
  __shared__ int s_moves, s_kept;
  pdl_wait();
  pdl_launch_dependents();
  const Cache& c = a.c;
  const int s = blockIdx.y;
  const int refused = ld(c.refused + s);
  const StepRows st = step_rows(a.cu, s, a.rows);
  if (st.n == 0 || refused != 0) return;
  if (threadIdx.x < 32) {
    const unsigned long long kept = kept_rows(a, st);
    const int first = ld(c.lens + s) - st.n;
    // rows that stay where they are: the kept ones before the first gap
    const int stay = __ffsll(~kept) == 0 ? kStepRows : __ffsll(~kept) - 1;
    const int moves = __popcll(kept) - stay;
    bool bad = false;
    for (int i = threadIdx.x; i < kStepRows; i += 32) {
      if (!((kept >> i) & 1ull) || i < stay) continue;
      const int rank = __popcll(kept & ((1ull << i) - 1ull)), m = rank - stay;
      const int pf = first + i, pt = first + rank;
      int page_f = -1, page_t = -1;
      if (pt >= 0 && pf / c.page_size < c.max_pages) {
        page_f = ld(c.table + static_cast<size_t>(s) * c.max_pages + pf / c.page_size);
        page_t = ld(c.table + static_cast<size_t>(s) * c.max_pages + pt / c.page_size);
      }
      if (page_f < 0 || page_f >= c.pages || page_t < 0 || page_t >= c.pages) {
        bad = true;
        page_f = -1;
      }
      s_page_from[m] = page_f;
      s_page_to[m] = page_t;
      s_from[m] = max(pf, 0) % c.page_size;
      s_to[m] = max(pt, 0) % c.page_size;
    }
    if (bad) atomicOr(c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
    if (threadIdx.x == 0) {
      s_moves = moves;
      s_kept = __popcll(kept);
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int last = 0;
    if (threadIdx.x == 0) last = atom_add_acqrel_u32(a.arrivals + s, 1u) == gridDim.x - 1;
    if (__shfl_sync(0xffffffffu, last, 0)) {
      if (threadIdx.x == 0) a.arrivals[s] = 0;  // for the next call
      const int len = max(ld(c.lens + s), 0);
      cut(c, s, len, min(max(len - st.n, 0) + s_kept, len));
    }
  }
  const int moves = s_moves;
  if (moves == 0) return;
  constexpr int kCodes = D / 32, kPieces = 2 * kCodes + 2;
  const long long u = static_cast<long long>(blockIdx.x) * kMoveThreads + threadIdx.x;
  const long long lh = u / kPieces;
  const int piece = static_cast<int>(u - lh * kPieces);
  if (lh >= static_cast<long long>(c.layers) * c.heads) return;
  const int layer = static_cast<int>(lh / c.heads), h = static_cast<int>(lh - static_cast<long long>(layer) * c.heads);
  uint8_t* base = c.pool + static_cast<size_t>(layer) * c.pages * c.page_bytes +
                  static_cast<size_t>(h) * c.tiles_per_page * (18 * D);
  // offset of the piece in a tile and the stride from slot to slot
  int off, stride;
  const bool codes = piece < 2 * kCodes;
  if (piece < kCodes) { off = piece * 256; stride = 16; }
  else if (codes) { off = 8 * D + (piece - kCodes) * 16; stride = D / 2; }
  else { off = 16 * D + (piece - 2 * kCodes) * D; stride = D / 16; }
  auto place = [&](int page, int slot) {
    return base + static_cast<size_t>(page) * c.page_bytes + (slot / kTile) * (18 * D) + off + (slot % kTile) * stride;
  };
  auto move = [&](auto sample) {
    typedef decltype(sample) V;
    for (int m0 = 0; m0 < moves; m0 += 8) {
      V v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (m0 + j < moves && s_page_from[m0 + j] >= 0)
          v[j] = *reinterpret_cast<const V*>(place(s_page_from[m0 + j], s_from[m0 + j]));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (m0 + j < moves && s_page_from[m0 + j] >= 0)
          *reinterpret_cast<V*>(place(s_page_to[m0 + j], s_to[m0 + j])) = v[j];
    }
  };
  if (codes || D == 256) move(uint4());
  else if (D == 128) move(uint2());
  else move(uint32_t());
}

}  // namespace

cudaError_t launch_reserve(const PageArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_ready<reserve_kernel>(dim3(1), dim3(kAllocThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  // as many CTAs as an SM holds: 127 us for 128 branches (906 MB); 4 an SM 136 (at the time).  With 10 an SM 124, but
  // 12.3 us instead of 11.0 for the forks of one prompt, whose few copies wait for CTAs that find none
  return launch_ready<copy_kernel>(dim3(num_sms * 5), dim3(kCopyThreads), 0, stream, a);
}
cudaError_t launch_fork(const PageArgs& a, cudaStream_t stream) {
  return launch_ready<fork_kernel>(dim3(a.n), dim3(128), 0, stream, a);
}
cudaError_t launch_trim(const PageArgs& a, cudaStream_t stream) {
  return launch_ready<trim_kernel>(dim3((a.c.seqs + kTrimWarps - 1) / kTrimWarps), dim3(32 * kTrimWarps), 0, stream, a);
}
cudaError_t launch_compact(const PageArgs& a, cudaStream_t stream) {
  const Cache& c = a.c;
  const long long units = static_cast<long long>(c.layers) * c.heads * (c.dim / 16 + 2);
  const dim3 grid(static_cast<unsigned>((units + kMoveThreads - 1) / kMoveThreads), c.seqs), block(kMoveThreads);
  return c.dim == 64    ? launch_ready<compact_kernel<64>>(grid, block, 0, stream, a)
         : c.dim == 128 ? launch_ready<compact_kernel<128>>(grid, block, 0, stream, a)
                        : launch_ready<compact_kernel<256>>(grid, block, 0, stream, a);
}

}  // namespace kv4
}  // namespace moe
