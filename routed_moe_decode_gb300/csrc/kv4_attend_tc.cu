// Attention over the 4-bit paged cache for head size 128 and blocks of more than 16 query rows (a
// step's rows times query heads per K/V head), on the fifth-generation tensor cores.
//
// The mathematics is that of the warp-MMA kernel (one pass, running reference m, FP32 sums, p
// rounded to FP16); the products of 128 tokens at a time, a round, are
//   S^T [128 tokens x N rows] = K [128 x D] Q^T       K: tensor memory, a lane a token
//   O^T [D x N rows]         += V^T [D x 128] P^T     V, P: shared memory
// with both accumulators in tensor memory.  The cache is dequantised once for up to 64 rows (the
// warp-MMA kernel does it again for every 32), and the products leave the warps free.
//
// One CTA of G groups of four warps and a loader.  In a round
//   the loader copies the tiles of a round up to S rounds ahead into a ring, over the whole chunk;
//   group 0 dequantises the next round's keys into one of two tensor-memory buffers, a thread a token;
//   two groups dequantise this round's values into shared memory, channels consecutive (the
//   transposed operand is read by the tensor core, not made), once the last round's product is done;
//   every thread takes its token's scores against N / G rows, and leaves p transposed in shared
//   memory;
//   two warps issue this round's second product and the next round's first.
// A row's m moves only when a score exceeds it by kSlack; then the accumulators in tensor memory are
// rescaled, which after an item's first round is rare.
//
// A round takes ~2500 cycles, of which the products need ~500: it is bound by the chain values ->
// scores -> p -> product, which two CTAs an SM (N = 32) or sixteen warps (N = 64) hide only in part.
// Measured against the warp-MMA kernel with blocks of 32 rows, on 32 sequences of 4096 to 8192 tokens and 8 heads of
// 128: 32 rows 117 against 123 us; 16 such sequences, 64 rows: 107 against 110; a chunk of 2048 rows
// with 4 query heads a K/V head over 4096 tokens: 499 against 692.  At head size 64 (99 against 82 us
// for 32 rows) and with 16 rows (100 against 73) the warp-MMA kernel is faster and is taken.
#include "kv4_attend.cuh"
#include "kv4_tc.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int D = 128;
constexpr int kTokens = 128;                // of a round
constexpr int kTiles = kTokens / kTile;

constexpr uint32_t kAIsMn = 1u << 15;  // instruction descriptor: A is such an operand

// Column c of v over the warp's 32 lanes, to the lanes that equal c modulo 16: the lanes exchange
// half of what they still hold at every step (31 exchanges instead of 80).
template <typename Op>
__device__ __forceinline__ float over_lanes(const float (&v)[16], int lane, Op op) {
  float x[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) x[c] = op(v[c], __shfl_xor_sync(0xffffffffu, v[c], 16));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool upper = (lane & o) != 0;  // keeps the upper o columns
#pragma unroll
    for (int c = 0; c < o; ++c) {
      const float keep = upper ? x[c + o] : x[c], give = upper ? x[c] : x[c + o];
      x[c] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  return x[0];
}

// Offsets in dynamic shared memory (from a 1024-byte boundary), tensor-memory columns, and the floats
// of a partial result, which lies as the warp-MMA kernel's does: [N / 8][D / 16][32][4] sums, m, l.
template <int N, int G, int S>
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
  static constexpr int kBars = kMax + 4 * N * 4;                // [S] arrived, [S] taken, scores, sums
  static constexpr int kSeqs = kBars + (2 * S + 2) * 8;             // cu [kSeqCache + 1], lens [kSeqCache]
  static constexpr int kTotal = kSeqs + (2 * kSeqCache + 1) * 4 + 1024;
  static constexpr int kPart = N * D + 2 * N;
  static constexpr int kColS = D, kColO = D + N;                // after two key buffers of D / 2 columns
  static constexpr int kCols = 256;
  static_assert(D + 2 * N <= kCols, "tensor-memory columns");
};

template <int N, int G, int S, int CTAS>
__global__ void __launch_bounds__(128 * G + 32, CTAS) attend_tc_kernel(AttendArgs a) {
  typedef TcShape<N, G, S> L;
  constexpr int kThreads = 128 * G, WARPS = 4 * G;  // that compute; one more warp loads
  constexpr int NC = N / G;  // rows of a thread
  constexpr int KS = D / 16, TILE = 18 * D;
  // warps that issue the products (an instruction takes ~45 cycles to issue, and there are up to 8 of each)
  constexpr int kFirst = 5, kSecond = 4;
  static_assert(NC == 16, "columns of a tensor-memory load");
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long s_scan[WARPS + 1];
  __shared__ Walk s_walk[2];  // this part, the next
  __shared__ Walk s_load[2];  // the loader's
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
  const uint32_t bars = base + L::kBars, taken = bars + 8 * S, bar_s = taken + 8 * S, bar_o = bar_s + 8;
  if (tid < 2 * S + 2) mbar_init(bars + 8 * tid, 1);
  if (tid == 0) s_abort = 0;
  fence_barrier_init();
  pdl_wait();
  pdl_launch_dependents();

  // the work, cut into one chunk of `per` rounds per CTA: this one's is [begin, end)
  const bool cached = a.c.seqs <= kSeqCache;
  if (cached) {
    for (int s = tid; s <= a.c.seqs; s += kThreads + 32) {
      s_cu[s] = ld(a.cu + s);
      if (s < a.c.seqs) s_len[s] = ld(a.c.lens + s);
    }
    __syncthreads();
  }
  const Steps steps{a, cached ? s_cu : nullptr, cached ? s_len : nullptr};
  constexpr int kAll = kThreads + 32;
  const int per_thread = (a.c.seqs + kAll - 1) / kAll;
  const int sa = min(tid * per_thread, a.c.seqs), sb = min(sa + per_thread, a.c.seqs);
  long long mine = 0;
  for (int s = sa; s < sb; ++s) mine += work_of(item_of<N, kTokens>(steps, s));
  long long total;
  const long long before = block_prefix<WARPS + 1>(mine, s_scan, total);
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
    bool ok = phase_done(bar, parity);
    if (!ok) {
      const long long t0 = clock64();
      while (!ok && clock64() - t0 < limit && *reinterpret_cast<volatile int*>(&s_abort) == 0) ok = phase_done(bar, parity);
    }
    return ok;
  };
  auto must = [&](uint32_t bar, uint32_t parity) {
    if (gone || wait(bar, parity, kWaitCycles)) return;
    gone = true;
    *reinterpret_cast<volatile int*>(&s_abort) = 1;
    atomicOr(a.c.status, kStatusTimeout);
  };

  // ---- the loader: a warp of its own, ahead of the others by up to S rounds, over the whole chunk.
  // Lane l holds the place of tile 32 b + l of the part (4 rounds), issues its copy, and has the page
  // number of the tile 32 further on ----
  if (warp == WARPS) {
    auto page_slot = [&](int t) {
      return a.c.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(static_cast<uint32_t>(t), a.page_magic));
    };
    if (lane == 0) s_load[0] = s_walk[0];
    __syncwarp();
    uint32_t round = 0;
    bool ok = true;
    for (int turn = 0; ok; turn ^= 1) {
      const Walk& w = s_load[turn];
      const int tile0 = kTiles * (w.it.lo + w.off), tiles = kTiles * w.count, len = w.it.len;
      const int head = w.idx / w.it.blocks * a.c.tiles_per_page;
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
      int page = load_page(lane);
      for (int i = 0; i < w.count && ok; ++i, ++round) {
        const int j = i & 3, st = static_cast<int>(round % S);
        if (j == 0 && i > 0) page = load_page(kTiles * i + lane);
        const uint32_t good = __ballot_sync(0xffffffffu, page >= 0) >> (kTiles * j) & 0xffu;
        if (round >= S) {
          must(taken + 8 * st, (round / S - 1) & 1u);
          ok = __all_sync(0xffffffffu, !gone);
          if (!ok) break;
        }
        if (lane == 0) {
          s_bad[round & 7] = ~good & 0xffu;
          if (good == 0) mbar_arrive(bars + 8 * st);
          else mbar_arrive_expect_tx(bars + 8 * st, __popc(good) * TILE);
        }
        __syncwarp();
        if (lane >> 3 == j && page >= 0) {
          const int t = tile0 + kTiles * (i - j) + lane;
          const uint8_t* src = a.c.pool + static_cast<size_t>(page) * a.c.page_bytes +
                               static_cast<size_t>(head + t - page_slot(t) * a.c.tiles_per_page) * TILE;
          bulk_copy_g2s(base + L::kRing + (st * kTiles + (lane & 7)) * TILE, src, TILE, bars + 8 * st);
        }
      }
      if (!ok) break;
      if (lane == 0) advance<N, kTokens>(steps, w, s_load[turn ^ 1], end);
      __syncwarp();
      if (!s_load[turn ^ 1].more) break;
    }
    if (!ok) {  // let what is still in flight land before the memory is given up
      const long long t0 = clock64();
      for (uint32_t r = round > S ? round - S : 0; r < round; ++r)
        while (!phase_done(bars + 8 * (r % S), (r / S) & 1u) && clock64() - t0 < kDrainCycles) {
        }
    }
    return;
  }
  auto sync = [&]() { named_bar_sync(1, kThreads); };
  auto any = [&](bool x) { return !named_bar_and(1, kThreads, !x); };
  uint32_t par_s = 0, par_o = 0;
  uint32_t round = 0;  // of the CTA
  auto arrived = [&](uint32_t u) { must(bars + 8 * (u % S), (u / S) & 1u); };

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
      tmem_store(tmem + lanes + buf * (D / 2) + 32 * half, v);
    }
    tc_wait_st();
  };
  // every group: the values of a round into shared memory, a thread 32 channels of a token at a time;
  // a token that is none of the sequence's is zeroed
  constexpr int PIECES = D / 32;
  constexpr int VT = 256;            // threads that do: groups 0 and 1, or 1 and 2 where there are four
  constexpr int STEP = VT / PIECES;  // tokens that they cover at a time
  const int v_tid = tid - (G == 2 ? 0 : 128);
  static_assert(STEP % kTile == 0 && kTokens % STEP == 0, "a thread keeps its slot of the tiles");
  const int v_tok = (tid & 7) + 8 * (max(v_tid, 0) / (8 * PIECES));
  const int v_piece = (tid >> 3) % PIECES;
  const uint8_t* v_src = smem + L::kRing + (v_tok >> 4) * TILE + 8 * D + (v_tok & 15) * (D / 2) + v_piece * 16;
  const uint8_t* v_scale = smem + L::kRing + (v_tok >> 4) * TILE + 17 * D + (v_tok & 15) * (D / 16) + 2 * v_piece;
  uint8_t* v_dst = smem + L::kV + (v_piece >> 1) * (kTokens * 128) + v_tok * 128;
  auto values = [&](int st, int tok0, int len, uint32_t bad) {
    if (v_tid < 0 || v_tid >= VT) return;
    const int at = st * kTiles * TILE;
    const bool all = bad == 0 && tok0 + kTokens <= len;
#pragma unroll
    for (int n = 0; n < kTokens / STEP; ++n) {
      const uint4 c = *reinterpret_cast<const uint4*>(v_src + at + n * (STEP / kTile) * TILE);
      uint32_t s = *reinterpret_cast<const uint16_t*>(v_scale + at + n * (STEP / kTile) * TILE);
      if (!all) {
        const int t = v_tok + n * STEP;
        if (tok0 + t >= len || ((bad >> (t >> 4)) & 1u)) s = 0;
      }
      s = e4m3x2_to_f16x2(s);
      const uint32_t lo = bcast_lo_half(s), hi = bcast_hi_half(s);
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t x[4];
        e2m1x8_to_f16x2x4(w[k], x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = hmul2_bits(x[e], k < 2 ? lo : hi);
        *reinterpret_cast<uint4*>(v_dst + n * STEP * 128 + ((((v_piece & 1) * 4 + k) ^ (v_tok & 7)) << 4)) =
            make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  };
  const uint64_t q_desc = smem_desc_sw128(base + L::kQ, 1024), p_desc = smem_desc_sw128(base + L::kP, 1024);
  const uint64_t v_desc = desc_mn_sw128(base + L::kV, kTokens * 128);
  // the products, by one lane of a converged warp: in divergent code every instruction's descriptors
  // are moved to uniform registers one by one, which took 2000 cycles a round
  auto first_product = [&](int buf) {
#pragma unroll
    for (int k = 0; k < KS; ++k)
      tc_mma_f16_ts(tmem + L::kColS, tmem + buf * (D / 2) + 8 * k, q_desc + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4),
                    idesc_f16_f32(128, N), k > 0);
    tc_commit(bar_s);
  };
  auto second_product = [&](bool add) {
#pragma unroll
    for (int k = 0; k < kTokens / 16; ++k)
      mma_f16_ss(tmem + L::kColO, v_desc + (k * 2048 >> 4), p_desc + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4),
                 idesc_f16_f32(128, N) | kAIsMn, add || k > 0);
    tc_commit(bar_o);
  };

  static_assert(S <= 4, "rounds whose lack of pages is known at a time");
  bool left = false;  // the CTA has left its work after a wait that gave up
  for (int turn = 0;; turn ^= 1) {
    const Walk& cur = s_walk[turn];
    const int count = cur.count, len = cur.it.len, first = cur.it.first;
    const int h = cur.idx / cur.it.blocks;
    const int r0 = (cur.idx - h * cur.it.blocks) * N;  // first of the block's rows: row r is (step row r / group, query head r % group)
    const int nrows = min(N, cur.it.n * a.group - r0);

    // the query rows as FP16, a warp a row, brought near 2^10 by a power of two that z's factor takes
    // back; the sign of the scale goes to the rows, so that a larger product is a larger score
    constexpr int OWN = N / WARPS;
    uint32_t w[OWN][D / 64];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {  // all of the warp's rows under way at once
      const int x = r0 + min(warp + i * WARPS, nrows - 1), step_row = x / a.group, hq = h * a.group + x - step_row * a.group;
      const char* src = static_cast<const char*>(a.q) + 2 * ((cur.it.row0 + step_row) * a.q_row + hq * a.q_head);
      const uint2 v = *reinterpret_cast<const uint2*>(src + 8 * lane);
      w[i][0] = v.x;
      w[i][1] = v.y;
    }
    if (tid < N) {
      const int step_row = (r0 + min(tid, nrows - 1)) / a.group;
      s_m[tid] = kLowest;
      s_pos[tid] = first + step_row;
      s_tree[tid] = a.tree != nullptr ? a.tree[cur.it.row0 + step_row] : 0ull;
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int r = warp + i * WARPS;
      float2 f[D / 64];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        f[j] = unpack2(r < nrows ? w[i][j] : 0u, a.fp16);
        top = fmaxf(top, fmaxf(fabsf(f[j].x), fabsf(f[j].y)));
      }
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // magnitudes compare as their bits
      const int e = static_cast<int>(__float_as_uint(top) >> 23);
      const int shift = e == 0 || e == 255 ? 0 : min(max(137 - e, -100), 100);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23) * (a.scale2 < 0.f ? -1.f : 1.f);
      const int ch = lane * (D / 32);
      uint8_t* dst = smem + L::kQ + (ch >> 6) * (N * 128) + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4) + (ch & 7) * 2;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) reinterpret_cast<uint32_t*>(dst)[j] = half2_bits(f[j].x * up, f[j].y * up);
      // above 0, so that a masked score stays -infinity
      if (lane == 0) s_f[r] = fmaxf(__uint_as_float(static_cast<uint32_t>(127 - shift) << 23) * fabsf(a.scale2), 1.2e-38f);
    }
    float l[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) l[c] = 0.f;
    // tokens that every row of the block sees without a look at the masks: from `open_lo`, before `open_hi`
    const int open_hi = a.tree != nullptr ? first : min(first + r0 / a.group + 1, len);
    const int open_lo = a.window > 0 ? max(first + (r0 + nrows - 1) / a.group - a.window + 1, 0) : 0;
    fence_proxy_async_smem();
    sync();  // the rows, and what the ring's first stages hold, are known to all
    if (group == 0) {
      arrived(round);
      keys(round % S, 0);
    }
    tc_fence_before();
    sync();
    if (warp == kFirst) {
      tc_fence_after();
      if (elect_one()) first_product(0);
    }

    int tok0 = (cur.it.lo + cur.off) * kTokens;
    for (int i = 0; i < count; ++i, ++round, tok0 += kTokens) {
      if (group == 0) {
        if (i + 1 < count) {
          arrived(round + 1);
          keys((round + 1) % S, (i + 1) & 1);
        }
      } else {
        arrived(round);
      }
      const uint32_t bad = s_bad[round & 7];
      if (i > 0) must(bar_o, par_o);  // the last round's p and values have been used
      values(round % S, tok0, len, bad);
      if (i > 0) par_o ^= 1u;
      must(bar_s, par_s);
      par_s ^= 1u;
      tc_fence_after();
      auto scores = [&](uint32_t (&sv)[NC]) {
        tmem_ld_x16(tmem + lanes + L::kColS + c0, sv);
        tc_wait_ld();
        if (tok0 >= open_lo && tok0 + kTokens <= open_hi && bad == 0) return;
        const int tok = tok0 + me, d = tok - first;
        const bool real = tok < len && !((bad >> (me >> 4)) & 1u);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          bool see = real;
          if (a.tree != nullptr) see = see && (d < 0 || (d < 64 && ((s_tree[c0 + c] >> d) & 1ull)));
          else see = see && tok <= s_pos[c0 + c] && (a.window <= 0 || tok > s_pos[c0 + c] - a.window);
          if (!see) sv[c] = 0xff800000u;
        }
      };
      float z[NC];
      float most = -INFINITY;
      {
        uint32_t sv[NC];
        scores(sv);
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s_f + c0 + c), m = *reinterpret_cast<const float4*>(s_m + c0 + c);
          z[c] = fmaf(__uint_as_float(sv[c]), f.x, -m.x);
          z[c + 1] = fmaf(__uint_as_float(sv[c + 1]), f.y, -m.y);
          z[c + 2] = fmaf(__uint_as_float(sv[c + 2]), f.z, -m.z);
          z[c + 3] = fmaf(__uint_as_float(sv[c + 3]), f.w, -m.w);
          most = fmaxf(most, fmaxf(fmaxf(z[c], z[c + 1]), fmaxf(z[c + 2], z[c + 3])));
        }
      }
      if (any(most > kSlack)) {
        uint32_t sv[NC];
        scores(sv);
#pragma unroll
        for (int c = 0; c < NC; ++c) z[c] = __uint_as_float(sv[c]) * s_f[c0 + c];
        const float top = over_lanes(z, lane, [](float x, float y) { return fmaxf(x, y); });
        if (lane < NC) s_max[quarter * N + c0 + lane] = top;
        sync();
        auto raised = [&](int r) {
          return fmaxf(s_m[r], fmaxf(fmaxf(s_max[r], s_max[N + r]), fmaxf(s_max[2 * N + r], s_max[3 * N + r])));
        };
        float worth[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float m = raised(c0 + c);
          worth[c] = exp2_approx(s_m[c0 + c] - m);
          z[c] -= m;
          l[c] *= worth[c];
        }
        if (i > 0) {
          uint32_t o[NC];
          tmem_ld_x16(tmem + lanes + L::kColO + c0, o);
          tc_wait_ld();
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * worth[c]);
          tmem_store(tmem + lanes + L::kColO + c0, o);
          tc_wait_st();
        }
        float m = 0.f;
        if (tid < N) m = raised(tid);
        sync();
        if (tid < N) s_m[tid] = m;
      }
      // p, transposed: row c0 + c, 64 tokens to a line
      uint8_t* line = smem + L::kP + (me >> 6) * (N * 128) + c0 * 128 + (me & 7) * 2;
      const int chunk16 = (me & 63) >> 3;
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        const float p0 = exp2_approx(z[c]), p1 = exp2_approx(z[c + 1]);
        l[c] += p0;
        l[c + 1] += p1;
        const uint32_t both = half2_bits(p0, p1);
        *reinterpret_cast<uint16_t*>(line + c * 128 + ((chunk16 ^ (c & 7)) << 4)) = static_cast<uint16_t>(both);
        *reinterpret_cast<uint16_t*>(line + (c + 1) * 128 + ((chunk16 ^ ((c + 1) & 7)) << 4)) = static_cast<uint16_t>(both >> 16);
      }
      tc_fence_before();
      fence_proxy_async_smem();
      if (any(gone)) {
        left = true;
        break;
      }
      if (warp == kSecond) {
        tc_fence_after();
        if (elect_one()) second_product(i > 0);
        __syncwarp();
      } else if (warp == kFirst && i + 1 < count) {
        tc_fence_after();
        if (elect_one()) first_product((i + 1) & 1);
        __syncwarp();
      }
      if (tid == 0) mbar_arrive(taken + 8 * (round % S));
    }
    if (left) break;
    if (tid == 0) advance<N, kTokens>(steps, cur, s_walk[turn ^ 1], end);
    must(bar_o, par_o);
    par_o ^= 1u;
    tc_fence_after();
    {  // a row's l over its tokens
      const float sum = over_lanes(l, lane, [](float x, float y) { return x + y; });
      if (lane < NC) s_max[quarter * N + c0 + lane] = sum;
    }
    if (any(gone)) {
      left = true;
      break;
    }
    const bool more = s_walk[turn ^ 1].more;
    const bool whole = cur.count == cur.it.units;
    float* part = a.part + (2 * static_cast<size_t>(chunk) + (cur.off == 0 ? 1 : 0)) * L::kPart;
    auto sum_of = [&](int r) { return (s_max[r] + s_max[N + r]) + (s_max[2 * N + r] + s_max[3 * N + r]); };
    uint32_t o[NC];
    tmem_ld_x16(tmem + lanes + L::kColO + c0, o);
    tc_wait_ld();
    // this thread's channel
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
    sync();  // the output has been read, the rows' places are free
    tc_fence_after();
    if (!more) break;
  }
  if (left && tid == 0) {  // let the products in flight end before the memory is given up
    const long long t0 = clock64();
    while (!(phase_done(bar_s, par_s) && phase_done(bar_o, par_o)) && clock64() - t0 < kDrainCycles) {
    }
  }
  sync();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

template <int N, int G, int S, int CTAS>
cudaError_t launch(AttendArgs a, int num_sms, cudaStream_t stream) {
  typedef TcShape<N, G, S> L;
  constexpr int smem = L::kTotal;
  static_assert(smem <= 227 * 1024 / CTAS - 2048 && CTAS * L::kCols <= 512, "shared memory and tensor memory of an SM");
  a.page_magic = page_magic(a.c);
  const int grid = max(1, min(CTAS * num_sms, min(kMaxChunks, static_cast<int>(kPartFloats / 2 / L::kPart))));
  a.chunks = grid;
  const cudaError_t e = launch_ready<attend_tc_kernel<N, G, S, CTAS>>(dim3(grid), dim3(128 * G + 32), smem, stream, a);
  if (e != cudaSuccess) return e;
  return launch_ready<join_kernel<D, N / 8>>(dim3((a.chunks + kJoinChunks - 1) / kJoinChunks, N / 8), dim3(kJoinThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_attend_tc(const AttendArgs& a, int block_rows, int num_sms, cudaStream_t stream) {
  return block_rows <= 32 ? launch<32, 2, 3, 2>(a, num_sms, stream) : launch<64, 4, 4, 1>(a, num_sms, stream);
}

}  // namespace kv4
}  // namespace moe
