// Attention over the 4-bit paged cache for blocks of many query rows (steps whose rows times query
// heads per K/V head exceed 8), on the fifth-generation tensor cores.
//
// The mathematics is that of the warp-MMA kernel (one pass, running reference m, FP32 sums, p
// rounded to FP16); the products of 128 tokens at a time are
//   S^T [128 tokens x N rows] = K [128 x D] Q^T       K: tensor memory, a lane a token
//   O^T [D x N rows]         += V^T [D x 128] P^T     V, P: shared memory
// with both accumulators in tensor memory.  With 16 rows and more the warp-MMA kernel is bound by
// its MMAs (a quarter of tcgen05's rate per SM) and by doing the dequantisation again for every
// 16 or 32 rows; here the cache is dequantised once for up to 128 rows, and the tensor cores need a
// tenth of the time of the exponentials, which bound blocks of 64 rows and more.
//
// One CTA of G groups of four warps.  For every 128 tokens, a round:
//   group 0 dequantises the next round's keys into one of two tensor-memory buffers, a thread a token;
//   the other groups dequantise this round's values into shared memory, channels consecutive (the
//   transposed operand is read by the tensor core, not made);
//   every thread takes its token's scores against N / G rows, and leaves p transposed in shared
//   memory;
//   one thread issues this round's second product and the next round's first, and the copies of the
//   round that will take this one's place in the ring.
// Two CTAs share an SM where they fit, so that one's dequantisation fills the other's waits.
// A row's m moves only when a score exceeds it by kSlack; then the accumulators in tensor memory are
// rescaled, which after an item's first round is rare.
#include "kv4_attend.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kTokens = 128;                // of a round
constexpr int kTiles = kTokens / kTile;

// D[tmem] (+)= A[smem] B[smem]^T, FP16 inputs, FP32 sums.
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of an operand whose rows (the M index) are consecutive in memory: 128-byte lines of 64
// rows for one k, swizzled like smem_desc_sw128, 1024 bytes from 8 k to the next 8, `next` bytes
// from 64 rows to the next 64.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t next) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | uint64_t((next >> 4) & 0x3FFFu) << 16 | uint64_t(1024u >> 4) << 32 |
         uint64_t(1u) << 46 | uint64_t(2u) << 61;
}
constexpr uint32_t kAIsMn = 1u << 15;  // instruction descriptor: A is such an operand

// 32 lanes x 32 bits, C consecutive columns.
template <int C>
__device__ __forceinline__ void tmem_load(uint32_t t, uint32_t (&v)[C]) {
  if constexpr (C == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(t)
                 : "memory");
  } else if constexpr (C == 16) {
    tmem_ld_x16(t, v);
  } else {
    tmem_ld_x32(t, v);
  }
}
template <int C>
__device__ __forceinline__ void tmem_store(uint32_t t, const uint32_t (&v)[C]) {
  if constexpr (C == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
  }
}

// Offsets in dynamic shared memory (from a 1024-byte boundary), tensor-memory columns, and the floats
// of a partial result, which lies as the warp-MMA kernel's does: [N / 8][D / 16][32][4] sums, m, l.
template <int D, int N, int G, int S>
struct TcShape {
  static constexpr int kV = 0;                                  // [D / 64][128 tokens][64] FP16, swizzled lines
  static constexpr int kQ = kV + D * kTokens * 2;               // [D / 64][N][64] FP16, swizzled lines
  static constexpr int kP = kQ + N * D * 2;                     // [2][N][64 tokens] FP16, swizzled lines
  static constexpr int kRing = kP + N * kTokens * 2;            // [S][8 tiles]
  static constexpr int kFactor = kRing + S * kTiles * 18 * D;   // [N] float: a row's scale,
  static constexpr int kM = kFactor + N * 4;                    // [N] float: reference,
  static constexpr int kTree = kM + N * 4;                      // [N] uint64: tree bits,
  static constexpr int kPos = kTree + N * 8;                    // [N] int: position
  static constexpr int kMax = kPos + N * 4;                     // [4][N] floats
  static constexpr int kBars = kMax + 4 * N * 4;                // [S] ring, scores, sums
  static constexpr int kSeqs = kBars + (S + 2) * 8;             // cu [kSeqCache + 1], lens [kSeqCache]
  static constexpr int kTotal = kSeqs + (2 * kSeqCache + 1) * 4 + 1024;
  static constexpr int kPart = N * D + 2 * N;
  static constexpr int kColS = D, kColO = D + N;                // after two key buffers of D / 2 columns
  static constexpr int kCols = D + 2 * N <= 128 ? 128 : D + 2 * N <= 256 ? 256 : 512;
};

template <int D, int N, int G, int S, int CTAS>
__global__ void __launch_bounds__(128 * G, CTAS) attend_tc_kernel(AttendArgs a) {
  typedef TcShape<D, N, G, S> L;
  constexpr int kThreads = 128 * G, WARPS = 4 * G;
  constexpr int NC = N / G;  // rows of a thread
  constexpr int KS = D / 16, TILE = 18 * D;
  static_assert(NC == 8 || NC == 16 || NC == 32, "columns of a tensor-memory load");
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long s_scan[WARPS];
  __shared__ Walk s_walk[2];  // this part, the next
  __shared__ uint32_t s_bad[8], s_tmem;  // s_bad[u & 7]: tiles of the CTA's round u without a page
  __shared__ int s_abort;
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_addr(smem);
  float* s_f = reinterpret_cast<float*>(smem + L::kFactor);
  float* s_m = reinterpret_cast<float*>(smem + L::kM);
  unsigned long long* s_tree = reinterpret_cast<unsigned long long*>(smem + L::kTree);
  int* s_pos = reinterpret_cast<int*>(smem + L::kPos);
  float* s_max = reinterpret_cast<float*>(smem + L::kMax);
  int* s_cu = reinterpret_cast<int*>(smem + L::kSeqs);
  int* s_len = s_cu + kSeqCache + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3, group = warp >> 2;
  const int c0 = group * NC;                 // this thread's rows
  const int me = 32 * quarter + lane;        // its token of a round; its channel of the output
  const uint32_t bars = base + L::kBars, bar_s = bars + 8 * S, bar_o = bar_s + 8;
  if (tid < S + 2) mbar_init(bars + 8 * tid, 1);
  if (tid == 0) s_abort = 0;
  fence_barrier_init();
  pdl_wait();
  pdl_launch_dependents();

  // the work, cut into one chunk of `per` rounds per CTA: this one's is [begin, end)
  const bool cached = a.c.seqs <= kSeqCache;
  if (cached) {
    for (int s = tid; s <= a.c.seqs; s += kThreads) {
      s_cu[s] = ld(a.cu + s);
      if (s < a.c.seqs) s_len[s] = ld(a.c.lens + s);
    }
    __syncthreads();
  }
  const Steps steps{a, cached ? s_cu : nullptr, cached ? s_len : nullptr};
  const int per_thread = (a.c.seqs + kThreads - 1) / kThreads;
  const int sa = min(tid * per_thread, a.c.seqs), sb = min(sa + per_thread, a.c.seqs);
  long long mine = 0;
  for (int s = sa; s < sb; ++s) mine += work_of(item_of<N, kTokens>(steps, s));
  long long total;
  const long long before = block_prefix<WARPS>(mine, s_scan, total);
  const int chunk = blockIdx.x;
  const long long per = (total + a.chunks - 1) / a.chunks;
  const long long begin = per * chunk, end = min(begin + per, total);
  if (tid == 0) a.pieces[chunk].on = 0;
  if (begin >= end) return;
  if (begin >= before && begin < before + mine) settle<N, kTokens>(steps, sa, before, begin, end, s_walk[0]);
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(smem_addr(&s_tmem), L::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem, lanes = static_cast<uint32_t>(32 * quarter) << 16;

  // ---- waits, with a limit: a thread that gives up tells the others, and the CTA leaves its work
  // together at the next barrier ----
  bool gone = false;
  auto wait = [&](uint32_t bar, uint32_t parity, long long limit) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
      const long long t0 = clock64();
      while (!ok && clock64() - t0 < limit && *reinterpret_cast<volatile int*>(&s_abort) == 0) ok = mbar_try_wait(bar, parity);
    }
    return ok;
  };
  auto must = [&](uint32_t bar, uint32_t parity) {
    if (gone || wait(bar, parity, kWaitCycles)) return;
    gone = true;
    *reinterpret_cast<volatile int*>(&s_abort) = 1;
    atomicOr(a.c.status, kStatusTimeout);
  };

  // ---- the ring, filled by warp 0: lane l holds the place of tile 32 b + l of the part (4 rounds),
  // issues its copy, and has the page number of the tile 32 further on ----
  int stage = 0;          // of the part's next round to be consumed
  uint32_t ring_par = 0;  // bit st: of stage st's phase (every thread waits once for every phase)
  uint32_t par_s = 0, par_o = 0;
  long long place = 0;
  uint32_t there = 0;
  int page_next = -1;
  auto page_slot = [&](int t) {
    return a.c.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(static_cast<uint32_t>(t), a.page_magic));
  };
  auto load_page = [&](const Walk& w, int i) {  // of the part's i-th tile
    const int t = kTiles * (w.it.lo + w.off) + i;
    if (i >= kTiles * w.count || t * kTile >= w.it.len) return -1;
    const int page = ld(a.c.table + static_cast<size_t>(w.it.s) * a.c.max_pages + page_slot(t));
    if (page < 0 || page >= a.c.pages) {
      atomicOr(a.c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
      return -1;
    }
    return page;
  };
  auto set_places = [&](const Walk& w, int i, int page) {
    const int t = kTiles * (w.it.lo + w.off) + i, h = w.idx / w.it.blocks;
    place = static_cast<long long>(page) * static_cast<long long>(a.c.page_bytes) +
            static_cast<long long>(h * a.c.tiles_per_page + t - page_slot(t) * a.c.tiles_per_page) * TILE;
    there = __ballot_sync(0xffffffffu, page >= 0);
  };
  // warp 0, a barrier before anyone looks: what the part's round i, the CTA's round u, lacks
  auto prepare = [&](const Walk& w, int i, uint32_t u) {
    if ((i & 3) == 0 && i > 0) {
      set_places(w, kTiles * i + lane, page_next);
      page_next = load_page(w, kTiles * i + 32 + lane);
    }
    if (lane == 0) s_bad[u & 7] = ~(there >> (kTiles * (i & 3))) & 0xffu;
  };
  // warp 0: the copies of the part's round i into stage st, after `prepare`
  auto issue = [&](int i, int st) {
    const int j = i & 3;
    const uint32_t good = there >> (kTiles * j) & 0xffu;
    if (lane >> 3 == j && ((there >> lane) & 1u)) {
      // one lane announces all copies; another's may land before, which the barrier allows
      if ((lane & 7) == __ffs(good) - 1) mbar_arrive_expect_tx(bars + 8 * st, __popc(good) * TILE);
      bulk_copy_g2s(base + L::kRing + (st * kTiles + (lane & 7)) * TILE, a.c.pool + place, TILE, bars + 8 * st);
    }
  };
  auto start = [&](const Walk& w, uint32_t u) {  // warp 0: the first rounds of a part
    const int page = load_page(w, lane);
    page_next = w.count > 4 ? load_page(w, 32 + lane) : -1;
    set_places(w, lane, page);
    int st = stage;
    for (int i = 0; i < S && i < w.count; ++i) {
      prepare(w, i, u + i);
      issue(i, st);
      if (++st == S) st = 0;
    }
  };
  auto arrived = [&](int st, uint32_t u) {  // every thread, once for every round
    if (s_bad[u & 7] == 0xffu) return;
    must(bars + 8 * st, ring_par >> st & 1u);
    ring_par ^= 1u << st;
  };

  // group 0: the keys of a round into a tensor-memory buffer, a thread its token
  auto keys = [&](int st, int buf) {
    const uint8_t* tile = smem + L::kRing + (st * kTiles + (me >> 4)) * TILE;
    const int slot = me & 15;
    uint32_t sc[D / 32];  // scales of the channels 32 j, 32 j + 16
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + 16 * D + slot * (D / 16) + 4 * j);
      sc[2 * j] = e4m3x2_to_f16x2(w);
      sc[2 * j + 1] = e4m3x2_to_f16x2(w >> 16);
    }
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
      uint32_t v[32];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 c = *reinterpret_cast<const uint4*>(tile + (2 * half + j) * 256 + slot * 16);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        const uint32_t s = sc[2 * half + j], lo = bcast_lo_half(s), hi = bcast_hi_half(s);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t x[4];
          e2m1x8_to_f16x2x4(w[k], x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[16 * j + 4 * k + e] = hmul2_bits(x[e], k < 2 ? lo : hi);
        }
      }
      tmem_store<32>(tmem + lanes + buf * (D / 2) + 32 * half, v);
    }
    tc_wait_st();
  };
  // the other groups: the values of a round into shared memory, a thread 32 channels of a token at a
  // time; a token that is none of the sequence's is zeroed
  auto values = [&](int st, int tok0, int len, uint32_t bad) {
    constexpr int PIECES = D / 32;
    for (int u = tid - 128; u < kTokens * PIECES; u += kThreads - 128) {
      const int t = (u & 7) + 8 * (u / (8 * PIECES)), piece = (u >> 3) % PIECES;
      const uint8_t* tile = smem + L::kRing + (st * kTiles + (t >> 4)) * TILE;
      const uint4 c = *reinterpret_cast<const uint4*>(tile + 8 * D + (t & 15) * (D / 2) + piece * 16);
      uint32_t s = *reinterpret_cast<const uint16_t*>(tile + 17 * D + (t & 15) * (D / 16) + 2 * piece);
      if (tok0 + t >= len || ((bad >> (t >> 4)) & 1u)) s = 0;
      s = e4m3x2_to_f16x2(s);
      const uint32_t lo = bcast_lo_half(s), hi = bcast_hi_half(s);
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      uint8_t* line = smem + L::kV + (piece >> 1) * (kTokens * 128) + t * 128;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t x[4];
        e2m1x8_to_f16x2x4(w[k], x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = hmul2_bits(x[e], k < 2 ? lo : hi);
        *reinterpret_cast<uint4*>(line + ((((piece & 1) * 4 + k) ^ (t & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  };
  auto first_product = [&](int buf) {  // one thread
#pragma unroll
    for (int k = 0; k < KS; ++k)
      tc_mma_f16_ts(tmem + L::kColS, tmem + buf * (D / 2) + 8 * k,
                    smem_desc_sw128(base + L::kQ + (k >> 2) * (N * 128) + (k & 3) * 32, 1024), idesc_f16_f32(128, N), k > 0);
    tc_commit(bar_s);
  };
  auto second_product = [&](bool add) {  // one thread; D = 64: the upper 64 lanes repeat the lower
#pragma unroll
    for (int k = 0; k < kTokens / 16; ++k)
      mma_f16_ss(tmem + L::kColO, desc_mn_sw128(base + L::kV + k * 2048, D == 128 ? kTokens * 128 : 0),
                 smem_desc_sw128(base + L::kP + (k >> 2) * (N * 128) + (k & 3) * 32, 1024), idesc_f16_f32(128, N) | kAIsMn,
                 add || k > 0);
    tc_commit(bar_o);
  };

  static_assert(S <= 4, "rounds whose lack of pages is known at a time");
  uint32_t round = 0;  // of the CTA
  if (warp == 0) start(s_walk[0], 0);
  bool left = false;  // the CTA has left its work after a wait that gave up
  for (int turn = 0;; turn ^= 1) {
    const Walk& cur = s_walk[turn];
    const int count = cur.count, len = cur.it.len, first = cur.it.first;
    const int h = cur.idx / cur.it.blocks;
    const int r0 = (cur.idx - h * cur.it.blocks) * N;  // first of the block's rows: row r is (step row r / group, query head r % group)
    const int nrows = min(N, cur.it.n * a.group - r0);

    // the query rows as FP16, a warp a row, brought near 2^10 by a power of two that z's factor takes
    // back; the sign of the scale goes to the rows, so that a larger product is a larger score
    for (int r = warp; r < N; r += WARPS) {
      const int x = r0 + min(r, nrows - 1), step_row = x / a.group, hq = h * a.group + x - step_row * a.group;
      const char* src = static_cast<const char*>(a.q) + 2 * ((cur.it.row0 + step_row) * a.q_row + hq * a.q_head);
      uint32_t w[D / 64];
      if constexpr (D == 128) {
        const uint2 v = *reinterpret_cast<const uint2*>(src + 8 * lane);
        w[0] = v.x; w[1] = v.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(src + 4 * lane);
      }
      float2 f[D / 64];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        f[i] = unpack2(r < nrows ? w[i] : 0u, a.fp16);
        top = fmaxf(top, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = static_cast<int>(__float_as_uint(top) >> 23);
      const int shift = e == 0 || e == 255 ? 0 : min(max(137 - e, -100), 100);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23) * (a.scale2 < 0.f ? -1.f : 1.f);
      const int ch = lane * (D / 32);
      uint8_t* dst = smem + L::kQ + (ch >> 6) * (N * 128) + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4) + (ch & 7) * 2;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) reinterpret_cast<uint32_t*>(dst)[i] = half2_bits(f[i].x * up, f[i].y * up);
      if (lane == 0) {
        // above 0, so that a masked score stays -infinity
        s_f[r] = fmaxf(__uint_as_float(static_cast<uint32_t>(127 - shift) << 23) * fabsf(a.scale2), 1.2e-38f);
        s_m[r] = kLowest;
        s_pos[r] = first + step_row;
        s_tree[r] = a.tree != nullptr ? a.tree[cur.it.row0 + step_row] : 0ull;
      }
    }
    float l[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) l[c] = 0.f;
    // tokens that every row of the block sees without a look at the masks: from `open_lo`, before `open_hi`
    const int open_hi = a.tree != nullptr ? first : min(first + r0 / a.group + 1, len);
    const int open_lo = a.window > 0 ? max(first + (r0 + nrows - 1) / a.group - a.window + 1, 0) : 0;
    fence_proxy_async_smem();
    __syncthreads();  // the rows, and what the ring's first stages hold, are known to all
    if (group == 0) {
      arrived(stage, round);
      keys(stage, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      first_product(0);
    }

    int tok0 = (cur.it.lo + cur.off) * kTokens;
    for (int i = 0; i < count; ++i, ++round, tok0 += kTokens) {
      const int next = stage + 1 == S ? 0 : stage + 1;
      const uint32_t bad = s_bad[round & 7];
      if (group == 0) {
        if (i + 1 < count) {
          arrived(next, round + 1);
          keys(next, (i + 1) & 1);
        }
        if (i > 0) must(bar_o, par_o);  // the last round's p have been used
      } else {
        arrived(stage, round);
        if (i > 0) must(bar_o, par_o);  // and its values
        values(stage, tok0, len, bad);
      }
      if (i > 0) par_o ^= 1u;
      must(bar_s, par_s);
      par_s ^= 1u;
      tc_fence_after();
      uint32_t sv[NC];
      tmem_load<NC>(tmem + lanes + L::kColS + c0, sv);
      tc_wait_ld();
      if (!(tok0 >= open_lo && tok0 + kTokens <= open_hi && bad == 0)) {
        const int tok = tok0 + me, d = tok - first;
        const bool real = tok < len && !((bad >> (me >> 4)) & 1u);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          bool see = real;
          if (a.tree != nullptr) see = see && (d < 0 || (d < 64 && ((s_tree[c0 + c] >> d) & 1ull)));
          else see = see && tok <= s_pos[c0 + c] && (a.window <= 0 || tok > s_pos[c0 + c] - a.window);
          if (!see) sv[c] = 0xff800000u;
        }
      }
      float z[NC];
      float most = -INFINITY;
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        const float4 f = *reinterpret_cast<const float4*>(s_f + c0 + c), m = *reinterpret_cast<const float4*>(s_m + c0 + c);
        z[c] = fmaf(__uint_as_float(sv[c]), f.x, -m.x);
        z[c + 1] = fmaf(__uint_as_float(sv[c + 1]), f.y, -m.y);
        z[c + 2] = fmaf(__uint_as_float(sv[c + 2]), f.z, -m.z);
        z[c + 3] = fmaf(__uint_as_float(sv[c + 3]), f.w, -m.w);
        most = fmaxf(most, fmaxf(fmaxf(z[c], z[c + 1]), fmaxf(z[c + 2], z[c + 3])));
      }
      if (__syncthreads_or(most > kSlack)) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const uint32_t k = __reduce_max_sync(0xffffffffu, float_key(__uint_as_float(sv[c]) * s_f[c0 + c]));
          if (lane == 0) s_max[quarter * N + c0 + c] = __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
        }
        __syncthreads();
        auto raised = [&](int r) {
          return fmaxf(s_m[r], fmaxf(fmaxf(s_max[r], s_max[N + r]), fmaxf(s_max[2 * N + r], s_max[3 * N + r])));
        };
        uint32_t o[NC];
        if (i > 0) {
          tmem_load<NC>(tmem + lanes + L::kColO + c0, o);
          tc_wait_ld();
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float m = raised(c0 + c), w = exp2_approx(s_m[c0 + c] - m);
          l[c] *= w;
          if (i > 0) o[c] = __float_as_uint(__uint_as_float(o[c]) * w);
          z[c] = fmaf(__uint_as_float(sv[c]), s_f[c0 + c], -m);
        }
        if (i > 0) {
          tmem_store<NC>(tmem + lanes + L::kColO + c0, o);
          tc_wait_st();
        }
        float m = 0.f;
        if (tid < N) m = raised(tid);
        __syncthreads();
        if (tid < N) s_m[tid] = m;
      }
      // p, transposed: row c0 + c, 64 tokens to a line
      uint8_t* line = smem + L::kP + (me >> 6) * (N * 128) + c0 * 128 + (me & 7) * 2;
      const int chunk16 = (me & 63) >> 3;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float p = exp2_approx(z[c]);
        l[c] += p;
        *reinterpret_cast<__half*>(line + c * 128 + ((chunk16 ^ (c & 7)) << 4)) = __float2half_rn(p);
      }
      if (warp == 0 && i + S < count) prepare(cur, i + S, round + S);
      tc_fence_before();
      fence_proxy_async_smem();
      if (__syncthreads_or(gone)) {
        left = true;
        break;
      }
      if (tid == 0) {
        tc_fence_after();
        second_product(i > 0);
        if (i + 1 < count) first_product((i + 1) & 1);
      }
      if (warp == 0 && i + S < count) issue(i + S, stage);
      stage = next;
    }
    if (left) break;
    if (tid == 0) advance<N, kTokens>(steps, cur, s_walk[turn ^ 1], end);
    must(bar_o, par_o);
    par_o ^= 1u;
    tc_fence_after();
    // a row's l over its tokens
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
      if (lane == 0) s_max[quarter * N + c0 + c] = l[c];
    }
    if (__syncthreads_or(gone)) {
      left = true;
      break;
    }
    const bool more = s_walk[turn ^ 1].more;
    if (more && warp == 0) start(s_walk[turn ^ 1], round);
    const bool whole = cur.count == cur.it.units;
    float* part = a.part + (2 * static_cast<size_t>(chunk) + (cur.off == 0 ? 1 : 0)) * L::kPart;
    auto sum_of = [&](int r) { return (s_max[r] + s_max[N + r]) + (s_max[2 * N + r] + s_max[3 * N + r]); };
    uint32_t o[NC];
    tmem_load<NC>(tmem + lanes + L::kColO + c0, o);
    tc_wait_ld();
    if (me < D) {  // this thread's channel
      if (whole) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int x = r0 + c0 + c, step_row = x / a.group, hq = h * a.group + x - step_row * a.group;
          if (c0 + c >= nrows) break;
          const int64_t at = static_cast<int64_t>(cur.it.row0 + step_row) * (a.c.heads * a.group) + hq;
          const float sum = sum_of(c0 + c);
          const bool seen = sum > 0.f || sum != sum;
          const uint32_t v = pack2(seen ? __uint_as_float(o[c]) * (a.v_ts / sum) : 0.f, 0.f, a.fp16);
          static_cast<uint16_t*>(a.out)[at * D + me] = static_cast<uint16_t>(v);
          if (me == 0 && a.lse != nullptr) a.lse[at] = seen ? (s_m[c0 + c] + log2f(sum)) * kLn2 : -INFINITY;
        }
      } else {
        const int gg = me / (D / 8), k = me % (D / 8) / 2, e = me & 1;
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          const int n = (c0 + c) >> 3, q = ((c0 + c) & 7) >> 1;
          *reinterpret_cast<float2*>(part + ((n * KS + k) * 32 + gg * 4 + q) * 4 + 2 * e) =
              make_float2(__uint_as_float(o[c]), __uint_as_float(o[c + 1]));
        }
      }
    }
    if (!whole && tid < N) {
      part[N * D + tid] = s_m[tid];
      part[N * D + N + tid] = sum_of(tid);
    }
    if (tid == 0 && !whole && cur.off == 0) {  // the item goes on in the chunks up to that of its last unit
      Piece p;
      p.on = 1;
      p.last = static_cast<int>((cur.pos + cur.it.units - 1) / per);
      p.row0 = cur.it.row0; p.r0 = r0; p.nrows = nrows; p.h = h;
      a.pieces[chunk] = p;
    }
    tc_fence_before();
    __syncthreads();  // the output has been read, the rows' places are free
    tc_fence_after();
    if (!more) break;
  }
  if (left && tid == 0) {  // let what is still in flight land before the memory is given up
    *reinterpret_cast<volatile int*>(&s_abort) = 0;
    for (int st = 0; st < S; ++st) wait(bars + 8 * st, ring_par >> st & 1u, kDrainCycles);
    wait(bar_s, par_s, kDrainCycles);
    wait(bar_o, par_o, kDrainCycles);
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

template <int D, int N, int G, int S, int CTAS>
cudaError_t launch(AttendArgs a, int num_sms, cudaStream_t stream) {
  typedef TcShape<D, N, G, S> L;
  constexpr int smem = L::kTotal;
  static_assert(smem <= 227 * 1024 / CTAS - 2048 && CTAS * L::kCols <= 512, "shared memory and tensor memory of an SM");
  a.page_magic = page_magic(a.c);
  const int grid = max(1, min(CTAS * num_sms, min(kMaxChunks, static_cast<int>(kPartFloats / 2 / L::kPart))));
  a.chunks = grid;
  const cudaError_t e = launch_ready<attend_tc_kernel<D, N, G, S, CTAS>>(dim3(grid), dim3(128 * G), smem, stream, a);
  if (e != cudaSuccess) return e;
  return launch_ready<join_kernel<D, N / 8>>(dim3((a.chunks + kJoinChunks - 1) / kJoinChunks, N / 8), dim3(kJoinThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_attend_tc(const AttendArgs& a, int block_rows, int num_sms, cudaStream_t stream) {
  if (a.c.dim == 64)
    return block_rows <= 16   ? launch<64, 16, 2, 4, 2>(a, num_sms, stream)
           : block_rows <= 32 ? launch<64, 32, 2, 4, 2>(a, num_sms, stream)
           : block_rows <= 64 ? launch<64, 64, 2, 3, 2>(a, num_sms, stream)
                              : launch<64, 128, 4, 4, 1>(a, num_sms, stream);
  return block_rows <= 16   ? launch<128, 16, 2, 3, 2>(a, num_sms, stream)
         : block_rows <= 32 ? launch<128, 32, 2, 3, 2>(a, num_sms, stream)
         : block_rows <= 64 ? launch<128, 64, 2, 2, 2>(a, num_sms, stream)
                            : launch<128, 128, 4, 3, 1>(a, num_sms, stream);
}

}  // namespace kv4
}  // namespace moe
