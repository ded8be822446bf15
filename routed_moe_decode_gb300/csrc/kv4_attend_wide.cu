// Attention over the 4-bit paged cache for blocks of up to 128 query rows (a step's rows times query
// heads per K/V head): chunks of a prompt, and draft trees of many heads.
//
// The mathematics is that of the warp-MMA kernel (one pass, running reference m, FP32 sums, p
// rounded to FP16); the products of 64 tokens at a time, a step, are
//   S [128 rows x 64 tokens] = Q [128 x D] K^T       Q, K: shared memory
//   O [128 rows x D]        += P [128 x 64] V        P: tensor memory; V: shared memory
// with S (two buffers) and O in tensor memory, at head size 128 p over its scores.  A query row is a lane
// of tensor memory and a thread: its maximum, its sum and its masks need no other thread.  The cache is
// dequantised once for 128 rows.
//
// Every role has warps of its own, and only barriers in shared memory between them:
//   a loader copies the tiles of up to S steps ahead into a ring and says what they hold;
//   four warps dequantise keys and values into the operands' swizzled lines;
//   an issuer starts the next step's first product before this step's second, so that the scores of
//   a step are there when the last one's p have been written;
//   four warps turn scores into p.
// A row's m moves only when a score exceeds it by more than kSlack; then the output in tensor memory is rescaled.
//
// A block reads no step that none of its rows sees; blocks are walked from both ends of the rows inwards,
// so that neighbouring items of a causal chunk are about equally long together.
//
// A step takes a CTA 0.95 us at head size 64 and 1.20 at 128, two CTAs an SM (from the slope between 12001 and 24001
// tokens of 24 sequences).  At 128 the operands' traffic through shared memory (105 KB a step, of which the query
// rows are 32) comes to two thirds of that; otherwise what the warps share is the issue and fetching of four roles' code
// (17.8 M instructions for the trees below, issue slots ~40 % busy).  17 to 20 us of a call do not depend on
// the tokens: ~4 until the first products, the end of an item and the start of the next, joining, CTAs that have more to do.
// Measured: 24 sequences of up to 6001 tokens, 112 rows, 4 K/V heads of 64: 40 us (78 with the warp-MMA kernel); a chunk of
// 2048 rows with 4 query heads a K/V head over 4096 tokens, 8 heads of 128: 143 us (657), 0.7 PFLOP/s of unmasked
// products; 64 rows of 16 sequences of 4096 to 8192 tokens, 8 heads of 128: 64 us (105).  More warps were slower:
// two threads a row 51 and 175, two groups of them on alternate steps 47 and 167, eight warps that dequantise the
// chunk 160 (against 42 and 151 at the time).  One word for the waits' limit and the flag that ends them: 143 against 147.
#include "kv4_attend.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kRows = 128, kTokens = 64, kTiles = kTokens / kTile;
constexpr int kSoft = 4, kDeq = 4;                   // warps [0, kSoft), [kSoft, kSoft + kDeq)
constexpr int kLoader = kSoft + kDeq, kIssuer = kLoader + 1, kWarps = kIssuer + 1, kThreads = 32 * kWarps;
constexpr uint32_t kBIsMn = 1u << 16;  // instruction descriptor: B's rows are consecutive in memory
// what the loader says of a step: tiles without a page, tokens of the sequence, and
constexpr uint32_t kFirst = 1u << 16, kEnd = 1u << 17;  // the first of an item; no step, the end of the work
constexpr int kInfos = 16;

// D[tmem] (+)= A[smem] B[smem]^T, FP16 inputs, FP32 sums.
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of an operand whose rows (the M or N index) are consecutive in memory: 128-byte lines of 64
// rows for one k, swizzled like smem_desc_sw128, 1024 bytes from 8 k to the next 8, `next` bytes
// from 64 rows to the next 64.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t next) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | uint64_t((next >> 4) & 0x3FFFu) << 16 | uint64_t(1024u >> 4) << 32 |
         uint64_t(1u) << 46 | uint64_t(2u) << 61;
}

// 32 lanes x 32 bits, 8 or 16 consecutive columns, written.
__device__ __forceinline__ void tmem_store(uint32_t t, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t t, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Two FP32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
        "l"(reinterpret_cast<const unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return d;
}

// Offsets in dynamic shared memory (from a 1024-byte boundary), tensor-memory columns, and the floats
// of a partial result: [D / 4][128 rows][4] sums, so that a warp's 32 rows are consecutive, then m and l.
// VB: buffers of values, S: steps in the ring.
template <int D, int VB, int S>
struct WideShape {
  static constexpr int kOperand = kTokens * D * 2;
  static constexpr int kQ = 0;                          // [D / 64][128 rows][64] FP16, swizzled lines
  static constexpr int kK = kQ + kRows * D * 2;         // [2][D / 64][64 tokens][64]
  static constexpr int kV = kK + 2 * kOperand;          // [VB][D / 64][64 tokens][64]
  static constexpr int kRing = kV + VB * kOperand;      // [S][4 tiles]
  static constexpr int kBars = kRing + S * kTiles * 18 * D;
  static constexpr int kNumBars = 2 * S + 2 + VB + 2 + 2 + 2 + 2;
  static constexpr int kSeqs = kBars + 8 * kNumBars;    // cu [kSeqCache + 1], lens [kSeqCache]
  static constexpr int kTotal = kSeqs + (2 * kSeqCache + 1) * 4 + 1024;
  static constexpr int kPart = kRows * D + 2 * kRows;
  static constexpr int kColO = 2 * kTokens;
  static constexpr int kCols = kColO + D <= 256 ? 256 : 512;
  // p in columns of its own, where there are some left: scores are then read once, and again only where the
  // reference rises (16 sequences, 64 rows of 64: 51.2 us, and 53.0 with a pass for the maximum first, at the time; now 50.4)
  static constexpr bool kApart = kColO + D + kTokens <= kCols;
  static constexpr int kColP = kApart ? kColO + D : 0, kStepP = kApart ? kTokens / 2 : kTokens;
};

// The block of rows of an item, and the steps of a part that some of its rows see.
struct Block {
  int h, r0, nrows;
  int unit, steps;  // first step of the part that is taken, and their number
};
__device__ __forceinline__ Block block_of(const AttendArgs& a, const Walk& w) {
  const Item& it = w.it;
  Block b;
  b.h = w.idx / it.blocks;
  const int j = w.idx - b.h * it.blocks;
  b.r0 = (j & 1 ? it.blocks - 1 - (j >> 1) : j >> 1) * kRows;
  b.nrows = min(kRows, it.n * a.group - b.r0);
  const int last = it.first + (b.r0 + b.nrows - 1) / a.group;
  const int hi = a.tree != nullptr ? it.len : min(it.len, last + 1);
  const int lo = a.window > 0 ? max(it.first + b.r0 / a.group - a.window + 1, 0) : 0;
  const int from = it.lo + w.off;
  b.unit = max(from, lo / kTokens);
  b.steps = max(min(from + w.count, (max(hi, 0) + kTokens - 1) / kTokens) - b.unit, 0);
  return b;
}

__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// Eight codes a word, 32 channels of a token, as FP16 into the token's line: chunks c0 .. c0 + 3 of 16 bytes.
__device__ __forceinline__ void expand(const uint4& codes, uint32_t scales, uint8_t* line, int c0, int tok) {
  const uint32_t s = e4m3x2_to_f16x2(scales), lo = bcast_lo_half(s), hi = bcast_hi_half(s);
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t x[4];
    e2m1x8_to_f16x2x4(w[k], x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = hmul2_bits(x[e], k < 2 ? lo : hi);
    *reinterpret_cast<uint4*>(line + (((c0 + k) ^ (tok & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
  }
}

template <int D, int VB, int S, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) attend_wide_kernel(AttendArgs a) {
  typedef WideShape<D, VB, S> L;
  constexpr int TILE = 18 * D, PIECES = D / 32;
  static_assert(S + VB + 4 <= kInfos, "steps whose description is alive");
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long s_scan[kWarps];
  __shared__ Walk s_walk[kSoft + 1][2];  // of the warps that walk the items: this part, the next
  __shared__ uint32_t s_info[kInfos], s_tmem;
  __shared__ uint32_t s_limit;  // of a wait, in cycles; 0 once one gave up
  __shared__ uint32_t s_landed, s_issued;  // steps whose copies the loader knows to have landed, has started
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_addr(smem);
  int* s_cu = reinterpret_cast<int*>(smem + L::kSeqs);
  int* s_len = s_cu + kSeqCache + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // barriers: the ring's stages filled and taken; keys and values written; scores there; p written;
  // second product done; query rows written; the end
  const uint32_t full = base + L::kBars, taken = full + 8 * S, k_full = taken + 8 * S, v_full = k_full + 16,
                 s_full = v_full + 8 * VB, p_full = s_full + 16, o_done = p_full + 16, q_full = o_done + 16,
                 drain = q_full + 8;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + 8 * i, a.copy_arrivals);
      mbar_init(taken + 8 * i, kDeq);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, kDeq);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, kSoft);
      mbar_init(o_done + 8 * i, 1);
    }
    for (int i = 0; i < VB; ++i) mbar_init(v_full + 8 * i, kDeq);
    mbar_init(q_full, kSoft);
    mbar_init(drain, 1);
    s_limit = a.wait_cycles;
  }
  fence_barrier_init();
  pdl_wait();
  pdl_launch_dependents();

  // the work, cut into one chunk of `per` steps per CTA: this one's is [begin, end)
  const bool cached = a.c.seqs <= kSeqCache;
  const Steps steps{a, cached ? s_cu : nullptr, cached ? s_len : nullptr};
  const int chunk = blockIdx.x;
  if (tid == 0) a.pieces[chunk].on = 0;
  Chunk c;
  if (a.c.seqs <= 32) {
    Walk* own = warp < kSoft ? &s_walk[warp][0] : warp == kLoader ? &s_walk[kSoft][0] : nullptr;
    if (!settle_warp<kRows, kTokens>(a, s_cu, s_len, chunk, c, own)) return;
  } else {
    if (cached) {
      for (int s = tid; s <= a.c.seqs; s += kThreads) {
        s_cu[s] = ld(a.cu + s);
        if (s < a.c.seqs) s_len[s] = step_len(a.c, s);
      }
      __syncthreads();
    }
    const int per_thread = (a.c.seqs + kThreads - 1) / kThreads;
    const int sa = min(tid * per_thread, a.c.seqs), sb = min(sa + per_thread, a.c.seqs);
    long long mine = 0;
    for (int s = sa; s < sb; ++s) mine += work_of(item_of<kRows, kTokens>(steps, s));
    long long total;
    const long long before = block_prefix<kWarps>(mine, s_scan, total);
    c.per = quotient(total + a.chunks - 1, a.chunks);
    c.begin = c.per * chunk;
    c.end = min(c.begin + c.per, total);
    if (c.begin >= c.end) return;
    if (c.begin >= before && c.begin < before + mine) {
      Walk w;
      settle<kRows, kTokens>(steps, sa, before, c.begin, c.end, w);
      for (int i = 0; i <= kSoft; ++i) s_walk[i][0] = w;
    }
    __syncwarp();
  }
  const long long end = c.end;
  if (warp == 0) {
    tmem_alloc(smem_addr(&s_tmem), L::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // A wait of a whole warp, with a limit: false where it gave up or another warp did; the roles then
  // leave their work and meet at the end of the kernel.
  auto wait = [&](uint32_t bar, uint32_t parity) {
    bool ok = phase_done(bar, parity & 1u);
    if (!__all_sync(0xffffffffu, ok)) {
      const uint32_t t0 = cycles();
      while (!ok && cycles() - t0 < *reinterpret_cast<volatile uint32_t*>(&s_limit)) ok = mbar_try_wait(bar, parity & 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) {
        *reinterpret_cast<volatile uint32_t*>(&s_limit) = 0;
        atomicOr(a.c.status, kStatusTimeout);
      }
    }
    return ok;
  };
  auto arrive = [&](uint32_t bar) {  // of a whole warp, once
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto info_of = [&](uint32_t n) { return *reinterpret_cast<volatile uint32_t*>(&s_info[n % kInfos]); };

  if (warp == kLoader) {
    // lane l holds the place of tile 32 b + l of the part (8 steps), issues its copy, and has the page
    // number of the tile 32 further on
    auto page_slot = [&](int t) {
      return a.c.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(static_cast<uint32_t>(t), a.page_magic));
    };
    uint32_t n = 0;  // steps of the chunk
    bool ok = true;
    for (int turn = 0; ok; turn ^= 1) {
      const Walk& w = s_walk[kSoft][turn];
      const Block b = block_of(a, w);
      const int tile0 = kTiles * b.unit, tiles = kTiles * b.steps, len = w.it.len;
      const int head = b.h * a.c.tiles_per_page;
      const int* table = a.c.table + static_cast<size_t>(w.it.s) * a.c.max_pages;
      auto load_page = [&](int i) {  // of the part's i-th tile
        if (i >= tiles || (tile0 + i) * kTile >= len) return -1;
        const int page = ld(table + page_slot(tile0 + i));
        if (page < 0 || page >= a.c.pages) {
          atomicOr(a.c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
          return -1;
        }
        return page;
      };
      int page = load_page(lane), page_next = load_page(32 + lane);
      for (int i = 0; i < b.steps; ++i, ++n) {
        constexpr int kAtOnce = 32 / kTiles;
        const int j = i % kAtOnce, st = static_cast<int>(n % S);
        if (j == 0 && i > 0) {
          page = page_next;
          page_next = load_page(kTiles * i + 32 + lane);
        }
        const uint32_t good = __ballot_sync(0xffffffffu, page >= 0) >> (kTiles * j) & ((1u << kTiles) - 1u);
        if (n >= S) ok = wait(taken + 8 * st, n / S - 1);
        if (!ok) break;
        if (lane == 0) {
          const int valid = min(max(len - (tile0 + kTiles * i) * kTile, 0), kTokens);
          *reinterpret_cast<volatile uint32_t*>(&s_info[n % kInfos]) =
              (~good & ((1u << kTiles) - 1u)) | (static_cast<uint32_t>(valid) << 8) | (i == 0 ? kFirst : 0u);
          if (good == 0) mbar_arrive(full + 8 * st);
          else mbar_arrive_expect_tx(full + 8 * st, __popc(good) * TILE);
        }
        __syncwarp();
        if (lane / kTiles == j && page >= 0) {
          const int t = tile0 + kTiles * (i - j) + lane;
          const uint8_t* src = a.c.pool + static_cast<size_t>(page) * a.c.page_bytes +
                               static_cast<size_t>(head + t - page_slot(t) * a.c.tiles_per_page) * TILE;
          bulk_copy_g2s(base + L::kRing + (st * kTiles + lane % kTiles) * TILE, src, TILE, full + 8 * st);
        }
      }
      if (!ok) break;
      if (lane == 0) advance<kRows, kTokens>(steps, w, s_walk[kSoft][turn ^ 1], end);
      __syncwarp();
      if (!s_walk[kSoft][turn ^ 1].more) break;
    }
    uint32_t landed = n > S ? n - S : 0;
    if (ok) {
      const uint32_t st = n % S;
      if (n < S || wait(taken + 8 * st, n / S - 1)) {
        if (lane == 0) {
          *reinterpret_cast<volatile uint32_t*>(&s_info[n % kInfos]) = kEnd;
          mbar_arrive(full + 8 * st);
        }
        if (n >= S) landed = n - S + 1;  // step n - S has been taken, and its stage's barrier says the end
      }
    }
    if (lane == 0) {
      s_landed = landed;
      s_issued = n;
    }
  } else if (warp == kIssuer) {
    // the products, by one lane of a converged warp
    const uint64_t q_desc = smem_desc_sw128(base + L::kQ, 1024);
    bool first = false;  // of the step before
    uint32_t items = 0;
    auto second = [&](uint32_t m) {  // the second product of step m
      if (!wait(p_full + 8 * (m & 1u), m >> 1) || !wait(v_full + 8 * (m % VB), m / VB)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t v_desc = desc_mn_sw128(base + L::kV + (m % VB) * L::kOperand, kTokens * 128);
#pragma unroll
        for (int k = 0; k < kTokens / 16; ++k)
          tc_mma_f16_ts(tmem + L::kColO, tmem + L::kColP + (m & 1u) * L::kStepP + 8 * k, v_desc + (k * 2048 >> 4),
                        idesc_f16_f32(kRows, D) | kBIsMn, !first || k > 0);
        tc_commit(o_done + 8 * (m & 1u));
      }
      __syncwarp();
      return true;
    };
    for (uint32_t n = 0;; ++n) {
      if (!wait(k_full + 8 * (n & 1u), n >> 1)) break;
      const uint32_t info = info_of(n);
      const bool begins = (info & (kFirst | kEnd)) != 0;
      if (begins && n > 0 && !second(n - 1)) break;  // the item before ends: its rows make room
      if (info & kEnd) break;
      if (begins && !wait(q_full, items++)) break;
      // the scores of two steps ago have become p, and those have been used
      if (n >= 2 && !wait(o_done + 8 * (n & 1u), (n >> 1) - 1)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t k_desc = smem_desc_sw128(base + L::kK + (n & 1u) * L::kOperand, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_f16_ss(tmem + (n & 1u) * kTokens, q_desc + (((k >> 2) * (kRows * 128) + (k & 3) * 32) >> 4),
                     k_desc + (((k >> 2) * (kTokens * 128) + (k & 3) * 32) >> 4), idesc_f16_f32(kRows, kTokens), k > 0);
        tc_commit(s_full + 8 * (n & 1u));
      }
      __syncwarp();
      if (!begins && !second(n - 1)) break;
      first = begins;
    }
  } else if (warp >= kSoft) {
    // a lane takes 32 channels of one token of the keys, then of the values; the values' pieces are
    // dealt so that eight lanes read all 32 banks, although a token's line is D / 2 bytes long
    const int dt = tid - 32 * kSoft;
    auto stage_of = [&](uint32_t n) { return smem + L::kRing + static_cast<int>(n % S) * kTiles * TILE; };
    bool ok = true, more = true;
    auto keys = [&](uint32_t n) {  // of step n; or the end of the work is passed on
      ok = wait(full + 8 * (n % S), n / S) && (n < 2 || wait(s_full + 8 * (n & 1u), (n >> 1) - 1));
      if (!ok) return;
      more = (info_of(n) & kEnd) == 0;
      if (more) {
        uint8_t* dst = smem + L::kK + (n & 1u) * L::kOperand;
#pragma unroll
        for (int r = 0; r < D / 64; ++r) {
          const int x = (dt >> 4) + 8 * r, piece = x % PIECES, slot = dt & 15, tok = (x / PIECES) * kTile + slot;
          const uint8_t* tile = stage_of(n) + (x / PIECES) * TILE;
          expand(*reinterpret_cast<const uint4*>(tile + piece * 256 + slot * 16),
                 *reinterpret_cast<const uint16_t*>(tile + 16 * D + slot * (D / 16) + 2 * piece),
                 dst + (piece >> 1) * (kTokens * 128) + tok * 128, (piece & 1) * 4, tok);
        }
        fence_proxy_async_smem();
      }
      arrive(k_full + 8 * (n & 1u));
    };
    keys(0);
    for (uint32_t n = 0; ok && more; ++n) {  // the keys are a step ahead
      keys(n + 1);
      if (!ok) break;
      if (n >= VB && !wait(o_done + 8 * ((n - VB) & 1u), (n - VB) >> 1)) break;
      const uint32_t info = info_of(n);
      uint8_t* values = smem + L::kV + (n % VB) * L::kOperand;
      const int tok = dt & (kTokens - 1), slot = tok & 15;
      const uint8_t* tile = stage_of(n) + (tok >> 4) * TILE;
      // a token that is none of the sequence's is 0, so that 0 * p is 0
      const bool real = tok < static_cast<int>(info >> 8 & 0xffu) && !((info >> (tok >> 4)) & 1u);
#pragma unroll
      for (int r = 0; r < D / 64; ++r) {
        const int piece = (tok / (8 / PIECES) + (dt >> 6) * (PIECES / 2) + r) % PIECES;
        const uint32_t scales = *reinterpret_cast<const uint16_t*>(tile + 17 * D + slot * (D / 16) + 2 * piece);
        expand(*reinterpret_cast<const uint4*>(tile + 8 * D + slot * (D / 2) + piece * 16), real ? scales : 0u,
               values + (piece >> 1) * (kTokens * 128) + tok * 128, (piece & 1) * 4, tok);
      }
      fence_proxy_async_smem();
      arrive(v_full + 8 * (n % VB));
      arrive(taken + 8 * (n % S));
    }
  } else {
    const int r = tid;  // this thread's row of the block, and its lane of tensor memory
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    uint32_t n = 0;
    bool ok = true;
    for (int turn = 0; ok; turn ^= 1) {
      const Walk& cur = s_walk[warp][turn];
      const Block b = block_of(a, cur);
      const int len = cur.it.len, first = cur.it.first;
      const bool mine_ok = r < b.nrows, warp_on = 32 * warp < b.nrows;
      const int x = b.r0 + min(r, b.nrows - 1), step_row = x / a.group, hq = b.h * a.group + x - step_row * a.group;
      const int pos = first + step_row;
      float factor = 1.f;
      unsigned long long tree = 0;
      if (b.steps > 0) {
        // the query row as FP16, brought near 2^10 by a power of two that z's factor takes back; the
        // sign of the scale goes to the row, so that a larger product is a larger score
        if (warp_on) {
          const char* src = static_cast<const char*>(a.q) + 2 * ((cur.it.row0 + step_row) * a.q_row + hq * a.q_head);
          if (a.tree != nullptr) tree = a.tree[cur.it.row0 + step_row];
          constexpr int PASS = D > 128 ? 2 : 1, HELD = D / 8 / PASS;  // 16-byte words held at a time
          uint4 v[HELD];
          float top = 0.f;
          auto load = [&](int p) {
#pragma unroll
            for (int j = 0; j < HELD; ++j)
              v[j] = mine_ok ? *reinterpret_cast<const uint4*>(src + 16 * (p * HELD + j)) : make_uint4(0, 0, 0, 0);
          };
#pragma unroll
          for (int p = 0; p < PASS; ++p) {
            load(p);
#pragma unroll
            for (int j = 0; j < HELD; ++j) {
              const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2(w[e], a.fp16);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            }
          }
          const int e = static_cast<int>(__float_as_uint(top) >> 23);
          const int shift = e == 0 || e == 255 ? 0 : min(max(137 - e, -100), 100);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23) * (a.scale2 < 0.f ? -1.f : 1.f);
          // above 0, so that a masked score stays -infinity
          factor = fmaxf(__uint_as_float(static_cast<uint32_t>(127 - shift) << 23) * fabsf(a.scale2), 1.2e-38f);
#pragma unroll
          for (int p = PASS - 1; p >= 0; --p) {
            if (p < PASS - 1) load(p);
#pragma unroll
            for (int j = 0; j < HELD; ++j) {
              const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
              uint32_t o[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2(w[i], a.fp16);
                o[i] = half2_bits(f.x * up, f.y * up);
              }
              const int c = p * HELD + j;
              *reinterpret_cast<uint4*>(smem + L::kQ + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        fence_proxy_async_smem();
        arrive(q_full);
      }
      float m = kLowest, l = 0.f;
      // tokens that every row of the block sees without a look at the masks: from `open_lo`, before `open_hi`
      const int open_hi = a.tree != nullptr ? first : min(first + b.r0 / a.group + 1, len);
      const int open_lo = a.window > 0 ? max(first + (b.r0 + b.nrows - 1) / a.group - a.window + 1, 0) : 0;
      int tok0 = b.unit * kTokens;
      for (int i = 0; i < b.steps; ++i, ++n, tok0 += kTokens) {
        ok = wait(s_full + 8 * (n & 1u), n >> 1);
        if (!ok) break;
        tc_fence_after();
        if (warp_on) {
          const uint32_t cols = lanes + (n & 1u) * kTokens;
          const uint32_t bad = info_of(n) & ((1u << kTiles) - 1u);
          const bool open = tok0 >= open_lo && tok0 + kTokens <= open_hi && bad == 0;
          unsigned long long see = ~0ull;  // of the step's tokens
          if (!open) {
            see = low_bits(len - tok0);
#pragma unroll
            for (int u = 0; u < kTiles; ++u)
              if ((bad >> u) & 1u) see &= ~(0xffffull << (kTile * u));
            if (a.tree != nullptr) {
              const int d = tok0 - first;  // of the step's first token
              if (d > -64) see &= d <= 0 ? low_bits(-d) | (tree << -d) : d < 64 ? tree >> d : 0ull;
            } else {
              see &= low_bits(pos + 1 - tok0);
              if (a.window > 0 && pos >= a.window) see &= ~low_bits(pos + 1 - a.window - tok0);
            }
          }
          // 16 scores at a time, in short loops: the warps of an SM sub-partition run the code of four roles and
          // fetch it through one small cache (64 at a time in registers, unrolled: 5 to 7 % slower)
          constexpr int CH = 16;
          auto scores = [&](int c0, uint32_t (&v)[CH]) {
            tmem_ld_x16(cols + c0, v);
            tc_wait_ld();
            if (!open) {
              const uint32_t bits = static_cast<uint32_t>(see >> c0);
#pragma unroll
              for (int c = 0; c < CH; ++c) v[c] = (bits >> c) & 1u ? v[c] : 0xff800000u;
            }
          };
          auto largest = [&]() {
            float top = -INFINITY;
#pragma unroll 1
            for (int c0 = 0; c0 < kTokens; c0 += CH) {
              uint32_t v[CH];
              scores(c0, v);
#pragma unroll
              for (int c = 0; c < CH; ++c) top = fmaxf(top, __uint_as_float(v[c]));
            }
            return top;
          };
          auto raise = [&](float top) {  // the reference, for that product; false: a wait gave up
            // of the rows that need it alone: a row's result does not depend on the block's others
            const float higher = fmaf(top, factor, -m) > kSlack ? top * factor - kBelow : m;
            const float worth = exp2_approx(m - higher);
            m = higher;
            l *= worth;
            if (i == 0) return true;
            if (!wait(o_done + 8 * ((n - 1) & 1u), (n - 1) >> 1)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld_x16(lanes + L::kColO + c0, o);
              tc_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * worth);
              tmem_store(lanes + L::kColO + c0, o);
            }
            return true;
          };
          const uint32_t cols_p = lanes + L::kColP + (n & 1u) * L::kStepP;
          float2 sum;
          auto powers = [&]() {  // p and their sum; returns the largest exponent
            sum = make_float2(0.f, 0.f);
            float most = -INFINITY;
            const float2 factor2 = make_float2(factor, factor), minus_m = make_float2(-m, -m);
#pragma unroll 1
            for (int c0 = 0; c0 < kTokens; c0 += CH) {
              uint32_t v[CH], p[CH / 2];
              scores(c0, v);
#pragma unroll
              for (int c = 0; c < CH; c += 2) {
                const float2 z = fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), factor2, minus_m);
                const float2 e = make_float2(exp2_approx(z.x), exp2_approx(z.y));
                if (L::kApart) most = fmaxf(most, fmaxf(z.x, z.y));
                sum = add2(sum, e);
                p[c / 2] = half2_bits(e.x, e.y);
              }
              tmem_store(cols_p + c0 / 2, p);  // kApart false: over scores that have been read
            }
            return most;
          };
          if constexpr (L::kApart) {
            // against the reference as it is, and once more where that was too low
            for (int again = 0; ok; ++again) {
              const float most = powers();
              if (again > 0 || !__any_sync(0xffffffffu, most > kSlack)) break;
              ok = raise(largest());
            }
          } else {
            const float top = largest();
            if (__any_sync(0xffffffffu, fmaf(top, factor, -m) > kSlack)) ok = raise(top);
            if (ok) powers();
          }
          if (!ok) break;
          l += sum.x + sum.y;
          tc_wait_st();
        }
        tc_fence_before();
        arrive(p_full + 8 * (n & 1u));
      }
      if (!ok) break;
      if (lane == 0) advance<kRows, kTokens>(steps, cur, s_walk[warp][turn ^ 1], end);
      __syncwarp();
      if (b.steps > 0) {
        ok = wait(o_done + 8 * ((n - 1) & 1u), (n - 1) >> 1);
        if (!ok) break;
        tc_fence_after();
      }
      const bool whole = cur.count == cur.it.units;
      if (warp_on) {
        float* part = a.part + (2 * static_cast<size_t>(chunk) + (cur.off == 0 ? 1 : 0)) * L::kPart;
        const int64_t at = static_cast<int64_t>(cur.it.row0 + step_row) * (a.c.heads * a.group) + hq;
        const bool seen = l > 0.f || l != l;
        const float f = seen ? a.v_ts / l : 0.f;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          if (b.steps > 0) {
            tmem_ld_x32(lanes + L::kColO + c0, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0u;
          }
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(a.out) + 2 * (at * D + c0));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = seen ? pack2(__uint_as_float(o[8 * j + 2 * e]) * f, __uint_as_float(o[8 * j + 2 * e + 1]) * f, a.fp16) : 0u;
              if (mine_ok) dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              reinterpret_cast<float4*>(part)[(c0 / 4 + j) * kRows + r] =
                  make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]), __uint_as_float(o[4 * j + 2]),
                              __uint_as_float(o[4 * j + 3]));
          }
        }
        if (!whole) {
          part[kRows * D + r] = m;
          part[kRows * D + kRows + r] = l;
        } else if (mine_ok && a.lse != nullptr) {
          a.lse[at] = seen ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
      }
      if (tid == 0 && !whole && cur.off == 0) {  // the item goes on in the chunks up to that of its last unit
        Piece p;
        p.on = 1;
        p.last = static_cast<int>((cur.pos + cur.it.units - 1) / c.per);
        p.row0 = cur.it.row0; p.r0 = b.r0; p.nrows = b.nrows; p.h = b.h;
        a.pieces[chunk] = p;
      }
      if (!s_walk[warp][turn ^ 1].more) break;
    }
    tc_wait_st();  // of a step that was left
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s_limit == 0) {  // whichever role gave up: what is in flight ends before the memory is given up
    const uint32_t t0 = cycles();
    if (warp == kIssuer) {
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      while (!phase_done(drain, 0) && cycles() - t0 < kDrainCycles) {
      }
    } else if (warp == kLoader) {
      for (uint32_t r = s_landed; r < s_issued; ++r)
        while (!phase_done(full + 8 * (r % S), (r / S) & 1u) && cycles() - t0 < kDrainCycles) {
        }
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, L::kCols);
}

// Joins the parts of the items that were cut.  CTA (c, g, y): the item that begins in chunk c and goes on
// past it, 32 of its rows, a lane a row, and 64 channels, 8 a warp; kBatch parts' trips to memory at a time.
constexpr int kBatch = 4;
template <int D>
__global__ void __launch_bounds__(256) join_wide_kernel(AttendArgs a) {
  constexpr int PART = kRows * D + 2 * kRows;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = 32 * blockIdx.y + lane;
  const int4* pp = reinterpret_cast<const int4*>(a.pieces + blockIdx.x);
  const int4 px = __ldcg(pp), py = __ldcg(pp + 1);
  if (px.x == 0 || 32 * static_cast<int>(blockIdx.y) >= py.x) return;
  const int c0 = blockIdx.x, parts = px.y - c0 + 1, quad = blockIdx.z * 16 + 2 * warp;
  // of the chunk c0 + c: the first chunk's part starts at the item's first unit
  auto part_of = [&](int c) { return a.part + (2 * static_cast<size_t>(c0 + c) + (c == 0 ? 1 : 0)) * PART; };
  float m = kLowest, l = 0.f, v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
  for (int cb = 0; cb < parts; cb += kBatch) {
    float pm[kBatch], pl[kBatch];
    float4 z[kBatch][2];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      pm[j] = kLowest;
      pl[j] = 0.f;
      z[j][0] = z[j][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (cb + j < parts) {
        const float* part = part_of(cb + j);
        pm[j] = __ldcg(part + kRows * D + r);
        pl[j] = __ldcg(part + kRows * D + kRows + r);
#pragma unroll
        for (int i = 0; i < 2; ++i) z[j][i] = __ldcg(reinterpret_cast<const float4*>(part) + (quad + i) * kRows + r);
      }
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) top = fmaxf(top, pm[j]);
    const float f = exp2_approx(m - top);
    m = top;
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float w = exp2_approx(pm[j] - top);
      l += w * pl[j];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[4 * i] += w * z[j][i].x;
        v[4 * i + 1] += w * z[j][i].y;
        v[4 * i + 2] += w * z[j][i].z;
        v[4 * i + 3] += w * z[j][i].w;
      }
    }
  }
  if (r >= py.x) return;
  const int x = px.w + r, step_row = x / a.group, hq = py.y * a.group + x - step_row * a.group;
  const int64_t at = static_cast<int64_t>(px.z + step_row) * (a.c.heads * a.group) + hq;
  const bool seen = l > 0.f || l != l;
  const float f = seen ? a.v_ts / l : 0.f;
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = seen ? pack2(v[2 * e] * f, v[2 * e + 1] * f, a.fp16) : 0u;
  *reinterpret_cast<uint4*>(static_cast<char*>(a.out) + 2 * (at * D + 4 * quad)) = make_uint4(w[0], w[1], w[2], w[3]);
  if (quad == 0 && a.lse != nullptr) a.lse[at] = seen ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <int D, int VB, int S, int CTAS>
cudaError_t launch(AttendArgs a, int num_sms, cudaStream_t stream) {
  typedef WideShape<D, VB, S> L;
  constexpr int smem = L::kTotal;
  static_assert(smem <= 227 * 1024 / CTAS - 3072 && CTAS * L::kCols <= 512, "shared memory and tensor memory of an SM");
  a.page_magic = page_magic(a.c);
  const int grid = max(1, min(CTAS * num_sms, min(kMaxChunks, static_cast<int>(kPartFloats / 2 / L::kPart))));
  a.chunks = grid;
  const cudaError_t e = launch_ready<attend_wide_kernel<D, VB, S, CTAS>>(dim3(grid), dim3(kThreads), smem, stream, a);
  if (e != cudaSuccess) return e;
  return launch_ready<join_wide_kernel<D>>(dim3(grid, kRows / 32, D / 64), dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_attend_wide(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  return a.c.dim == 64    ? launch<64, 2, 4, 2>(a, num_sms, stream)
         : a.c.dim == 128 ? launch<128, 1, 3, 2>(a, num_sms, stream)
                          : launch<256, 1, 3, 1>(a, num_sms, stream);
}

}  // namespace kv4
}  // namespace moe
