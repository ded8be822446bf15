// Attention of a step's query rows over the 4-bit paged cache.
//
// out = sum_t p_t v_t / sum_t p_t with p_t = exp2(z_t - m), z = scale log2(e) q.k: one pass over
// the tokens with a running reference m, FP32 sums, and the products on warp-level tensor-core
// MMAs (m16n8k16, FP16 operands, FP32 accumulators).  E2M1 x E4M3 has at most 6 significant bits
// and is exact in FP16, and a query row is brought by a power of two into FP16's range, so the
// scores are exact products summed in FP32; the one rounding inside is that of p to FP16 (11
// bits; p below 2^-21 of a row's largest have fewer, and those below 2^-32 none).
//
// Both products take the cache as the 16-row operand and the query rows as the 8-column one:
//   S^T [16 tokens x 8 rows]   = K [16 x D]  Q^T         O^T [D x 8 rows] += V^T [D x 16] P^T
// A lane's registers of S^T, packed to FP16 and transposed by movmatrix, are its operand of the
// second product.  The order of the channels within a sum and of the tokens within a tile is free,
// and is chosen so that the shared-memory reads are of whole words and (nearly) free of bank
// conflicts: lane (g = lane / 4, q = lane % 4) dequantises of K the tokens pi(g) and pi(g) + 8,
// pi(g) = g / 2 + 4 (g % 2), channels 32 j + 8 q .. + 7 (one word of every piece j), and of V the
// tokens q, q + 4, q + 8, q + 12, channels [g D/8, (g + 1) D/8).
//
// Memory.  Every warp streams its own tiles (18 D bytes, contiguous) through its own ring in shared
// memory by bulk copies, so that the bytes in flight do not cost registers: with loads to registers
// one tile ahead the same products ran at 45 % of the copy bandwidth, waiting for memory.
//
// Work split.  The (sequence, K/V head, block of 8 NT rows) items are laid end to end, each as long
// as the units of 32 tokens it has to read, and cut into one equal chunk per warp of the grid, so that
// any mix of lengths keeps every SM busy and no warp ever waits for another: joining the warps of a CTA
// at the end of every item cost a quarter of a batch of 32 ragged sequences.  An item that is cut
// leaves partial results (FP32 sums, m and l) in the workspace, and a second small kernel joins them
// in the order of the chunks, so results do not depend on timing.  The chunks are found on the device
// from the lengths: no host wait, no plan.
//
// Measured: four sequences of 131072 tokens, 8 K/V heads of 128 with 8 query heads each (604 MB) 112 us, 0.79 of the
// copy bandwidth; 32 sequences of 4096 to 8192 tokens, 16 rows (228 MB) 71 us, of which joining is ~8.  Bound by
// the conversions, multiplies and MMAs of an SM sub-partition, which add up instead of overlapping (at 8
// rows the ALU pipe is 51 % busy, at 16 rows 42 % and the MMA pipe 37 %; 8 warps run as fast as 12).
#include "kv4_attend.cuh"
#include "mma_parts.cuh"

namespace moe {
namespace kv4 {

namespace {

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Wait for a phase of a barrier by the whole warp, with a limit.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t limit) {
  bool ok = phase_done(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    const uint32_t t0 = cycles();
    while (!ok && cycles() - t0 < limit) ok = mbar_try_wait(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}

__device__ __forceinline__ uint32_t scale2_lo(uint32_t x, uint32_t s) {  // both halves of x by the low half of s
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&x), __low2half2(*reinterpret_cast<__half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t scale2_hi(uint32_t x, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&x), __high2half2(*reinterpret_cast<__half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The scales of the channels 32 j + 8 q of a token (byte 2 j + q / 2 of its D / 16), as FP16 pairs
// (j, j + 1).
template <int D>
__device__ __forceinline__ void key_scales(const uint8_t* p, int q, uint32_t (&o)[D / 64]) {
  const uint32_t sel = (q & 2) ? 0x7531u : 0x6420u;
  if constexpr (D == 64) {
    o[0] = e4m3x2_to_f16x2(__byte_perm(*reinterpret_cast<const uint32_t*>(p), 0u, sel));
  } else {
    uint32_t w[D / 64];
    if constexpr (D == 128) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const uint32_t four = __byte_perm(w[2 * i], w[2 * i + 1], sel);
      o[2 * i] = e4m3x2_to_f16x2(four);
      o[2 * i + 1] = e4m3x2_to_f16x2(four >> 16);
    }
  }
}

template <int N>
struct Words {
  uint32_t w[N];
};
template <int N>
__device__ __forceinline__ Words<N> shared_words(const uint8_t* p) {
  Words<N> o;
  if constexpr (N == 1) {
    o.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    o.w[0] = v.x; o.w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    o.w[0] = v.x; o.w[1] = v.y; o.w[2] = v.z; o.w[3] = v.w;
  }
  return o;
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

// The work is counted in units of two tiles (32 tokens), each of which a warp takes as one step: two
// independent chains of products, and one look at the masks and at the reference m for both.  (One
// tile a step leaves registers for more warps, and measured 0 to 30 % slower at every size.)
constexpr int U = 2;

// W warps, blocks of 8 NT rows, rings of S units; QS: the query rows' operands are read from shared
// memory for every unit instead of being kept in registers.  The offsets in dynamic shared memory,
// and the floats of a partial result: [NT][D / 16][32 lanes][4] sums as the accumulators lie in the
// warp's registers, then [2][8 NT] m and l.
template <int D, int NT, int W, int S, bool QS>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRing = 0;                               // [W][S] units
  static constexpr int kQuery = kRing + W * S * U * 18 * D;         // QS: [W][NT][D / 32][32] uint4
  static constexpr int kBars = kQuery + (QS ? W * kRows * D * 2 : 0);
  static constexpr int kSeqs = kBars + W * S * 8;               // cu [kSeqCache + 1], lens [kSeqCache]
  static constexpr int kTotal = kSeqs + (2 * kSeqCache + 1) * 4;
  static constexpr int kPart = kRows * D + 2 * kRows;
};

template <int D, int NT, int W, int S, int CTAS, bool QS>
__global__ void __launch_bounds__(32 * W, CTAS) attend_kernel(AttendArgs a) {
  typedef Shape<D, NT, W, S, QS> L;
  constexpr int ROWS = 8 * NT;
  constexpr int KS = D / 16;   // k16 steps of a score, and m16 tiles of the output
  constexpr int TILE = 18 * D;
  constexpr int UNIT = U * TILE;
  constexpr int kUnit = U * kTile;  // tokens
  constexpr int kThreads = 32 * W;
  extern __shared__ __align__(128) uint8_t smem[];
  int* s_cu = reinterpret_cast<int*>(smem + L::kSeqs);
  int* s_len = s_cu + kSeqCache + 1;
  __shared__ long long s_scan[W];
  __shared__ long long s_before[kThreads];
  __shared__ Walk s_walk[W][2];  // this part, the next
  __shared__ Chunk s_chunk[W];   // of the warp: lane 0's, out of the registers
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const uint8_t* ring = smem + L::kRing + warp * S * UNIT;
  uint4* queries = reinterpret_cast<uint4*>(smem + L::kQuery) + warp * (QS ? NT * (D / 32) * 32 : 0);
  const uint32_t ring_addr = smem_addr(ring), bar0 = smem_addr(smem + L::kBars + warp * S * 8);
  if (lane < S) mbar_init(bar0 + 8 * lane, a.copy_arrivals);
  fence_barrier_init();
  pdl_wait();
  pdl_launch_dependents();

  // the work, cut into one chunk of `per` units per warp of the grid: this one's is [begin, end).
  // Neighbouring chunks go to different SMs, so that a few units keep as many SMs busy.
  const bool cached = a.c.seqs <= kSeqCache;
  const Steps steps{a, cached ? s_cu : nullptr, cached ? s_len : nullptr};
  const int chunk = warp * gridDim.x + blockIdx.x;
  if (lane == 0) a.pieces[chunk].on = 0;
  Chunk c;
  if (a.c.seqs <= 32) {
    if (!settle_warp<ROWS, kUnit>(a, s_cu, s_len, chunk, c, &s_walk[warp][0])) return;
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
    for (int s = sa; s < sb; ++s) mine += work_of(item_of<ROWS, kUnit>(steps, s));
    long long total;
    s_before[tid] = block_prefix<W>(mine, s_scan, total);
    c.per = quotient(total + a.chunks - 1, a.chunks);
    c.begin = c.per * chunk;
    c.end = min(c.begin + c.per, total);
    __syncthreads();
    if (c.begin >= c.end) return;
    if (lane == 0) {
      int lo = 0, hi = kThreads - 1;  // the last thread whose sequences begin at or before the chunk
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_before[mid] <= c.begin) lo = mid; else hi = mid - 1;
      }
      settle<ROWS, kUnit>(steps, lo * per_thread, s_before[lo], c.begin, c.end, s_walk[warp][0]);
    }
    __syncwarp();
  }
  if (lane == 0) s_chunk[warp] = c;

  // ---- this warp's ring ----
  int stage = 0;            // next stage to be consumed; all stages are empty between items
  uint32_t parity = 0;      // bit st: of stage st's phase
  uint32_t invalid = 0;     // bits U st ..: the unit's tile has no page
  // the places of the warp's tiles in the cache, 32 at a time (32 / U units): lane l holds that of tile
  // 32 b + l, issues its copy, and has the page number of the tile 32 further on
  long long place = 0;
  uint32_t there = 0;       // lanes whose tile has a page
  int page_next = -1;
  auto page_slot = [&](int t) {
    return a.c.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(static_cast<uint32_t>(t), a.page_magic));
  };
  auto tile_at = [&](const Walk& w, int i) { return U * (w.it.lo + w.off) + i; };
  auto load_page = [&](const Walk& w, int i) {  // of the warp's i-th tile of the part
    const int t = tile_at(w, i);
    if (i >= U * w.count || t * kTile >= w.it.len) return -1;
    const int page = ld(a.c.table + static_cast<size_t>(w.it.s) * a.c.max_pages + page_slot(t));
    if (page < 0 || page >= a.c.pages) {
      atomicOr(a.c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
      return -1;
    }
    return page;
  };
  auto set_places = [&](const Walk& w, int i, int page) {
    const int t = tile_at(w, i), h = w.idx / w.it.blocks;
    place = static_cast<long long>(page) * static_cast<long long>(a.c.page_bytes) +
            static_cast<long long>(h * a.c.tiles_per_page + t - page_slot(t) * a.c.tiles_per_page) * TILE;
    there = __ballot_sync(0xffffffffu, page >= 0);
  };
  // start the copies of the part's unit i into stage st
  auto issue = [&](const Walk& w, int i, int st) {
    const int j = i % (32 / U);
    if (j == 0 && i > 0) {
      set_places(w, U * i + lane, page_next);
      page_next = load_page(w, U * i + 32 + lane);
    }
    constexpr uint32_t kAll = (1u << U) - 1u;
    const uint32_t bad = ~(there >> (U * j)) & kAll;
    invalid = (invalid & ~(kAll << (U * st))) | (bad << (U * st));
    if (lane / U == j && ((there >> lane) & 1u)) {
      const uint32_t bar = bar0 + 8 * st;
      // one lane announces the copies of both; the other's may land before, which the barrier allows
      if (lane % U == 0 || bad == 1u) mbar_arrive_expect_tx(bar, bad == 0 ? UNIT : TILE);
      bulk_copy_g2s(ring_addr + st * UNIT + lane % U * TILE, a.c.pool + place, TILE, bar);
    }
  };
  // the first units of a part
  auto start = [&](const Walk& w) {
    const int page = load_page(w, lane);
    page_next = w.count > 32 / U ? load_page(w, 32 + lane) : -1;
    set_places(w, lane, page);
    int st = stage;
    for (int i = 0; i < S && i < w.count; ++i) {
      issue(w, i, st);
      if (++st == S) st = 0;
    }
  };
  start(s_walk[warp][0]);

  for (int turn = 0;; turn ^= 1) {
    const Walk& cur = s_walk[warp][turn];
    const int h = cur.idx / cur.it.blocks;
    const int r0 = (cur.idx - h * cur.it.blocks) * ROWS;  // first of the block's rows: row r is (step row r / group, query head r % group)
    const int nrows = min(ROWS, cur.it.n * a.group - r0);

    // the query rows as FP16, brought near 2^10 by a power of two that z's factor takes back; the
    // sign of the scale goes to the rows, so that a larger product is a larger score
    uint32_t qf[QS ? 1 : NT][QS ? 1 : 2 * KS];
    float factor[NT][2];  // of the rows 2q and 2q + 1 of each n-tile
    {
      const float sign = a.scale2 < 0.f ? -1.f : 1.f, size = fabsf(a.scale2);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int x = r0 + 8 * t + g;
        const bool ok = 8 * t + g < nrows;
        const int step_row = x / a.group, hq = h * a.group + x - step_row * a.group;
        const char* src = static_cast<const char*>(a.q) +
                          2 * ((cur.it.row0 + (ok ? step_row : 0)) * a.q_row + (ok ? hq : 0) * a.q_head + 8 * q);
        uint32_t raw[D / 8];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {  // channels 32 i + 8 q ..
          const uint4 v = ok ? *reinterpret_cast<const uint4*>(src + 64 * i) : make_uint4(0, 0, 0, 0);
          raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 f = unpack2(raw[i], a.fp16);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^shift: the exponent field of top, brought to that of 2^10
        const int e = static_cast<int>(__float_as_uint(top) >> 23);
        const int shift = e == 0 || e == 255 ? 0 : min(max(137 - e, -100), 100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23) * sign;
        // above 0, so that a masked score stays -infinity
        const float down = fmaxf(__uint_as_float(static_cast<uint32_t>(127 - shift) << 23) * size, 1.2e-38f);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 f = unpack2(raw[i], a.fp16);
          raw[i] = half2_bits(f.x * up, f.y * up);
          if constexpr (!QS) qf[t][i] = raw[i];
        }
        if constexpr (QS) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            queries[(t * (D / 32) + i) * 32 + lane] = make_uint4(raw[4 * i], raw[4 * i + 1], raw[4 * i + 2], raw[4 * i + 3]);
        }
        factor[t][0] = __shfl_sync(0xffffffffu, down, 8 * q);      // lane of row 2q: g = 2q
        factor[t][1] = __shfl_sync(0xffffffffu, down, 8 * q + 4);
      }
    }

    float acc[NT][KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = kLowest;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
    }
    // tokens that every row of the block sees without a look at the masks: from `open_lo`, before `open_hi`
    const int first = cur.it.first, len = cur.it.len;
    const int open_hi = a.tree != nullptr ? first : min(first + r0 / a.group + 1, len);
    const int open_lo = a.window > 0 ? max(first + (r0 + nrows - 1) / a.group - a.window + 1, 0) : 0;

    const int n_units = cur.count;
    int tok0 = (cur.it.lo + cur.off) * kUnit;
    for (int i = 0; i < n_units; ++i, tok0 += kUnit) {
      const uint32_t bad = invalid >> (U * stage) & ((1u << U) - 1u);
      if (bad != (1u << U) - 1u) {
        if (!warp_wait(bar0 + 8 * stage, parity >> stage & 1u, a.wait_cycles)) {
          if (lane == 0) atomicOr(a.c.status, kStatusTimeout);
          for (int j = i; j < min(i + S, n_units); ++j) {  // what is in flight lands before the memory is given up
            if ((invalid >> (U * stage) & ((1u << U) - 1u)) != (1u << U) - 1u)
              warp_wait(bar0 + 8 * stage, parity >> stage & 1u, kDrainCycles);
            if (++stage == S) stage = 0;
          }
          return;
        }
        parity ^= 1u << stage;
        const uint8_t* unit = ring + stage * UNIT;
        const int tok_g = (g >> 1) + 4 * (g & 1);
        // ---- S^T = K Q^T, one word (8 channels, half a scale block) of each token at a time ----
        float sc[U][NT][4];
        uint32_t ks[2 * U][D / 64];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int n = 0; n < NT; ++n) sc[u][n][0] = sc[u][n][1] = sc[u][n][2] = sc[u][n][3] = 0.f;
          key_scales<D>(unit + u * TILE + 16 * D + tok_g * (D / 16), q, ks[2 * u]);
          key_scales<D>(unit + u * TILE + 16 * D + (tok_g + 8) * (D / 16), q, ks[2 * u + 1]);
        }
        const uint8_t* kp = unit + tok_g * 16 + q * 4;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t x[U][4], y[U][4];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint8_t* p = kp + u * TILE + w * 256;
            e2m1x8_to_f16x2x4(*reinterpret_cast<const uint32_t*>(p), x[u][0], x[u][1], x[u][2], x[u][3]);
            e2m1x8_to_f16x2x4(*reinterpret_cast<const uint32_t*>(p + 128), y[u][0], y[u][1], y[u][2], y[u][3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[u][j] = w & 1 ? scale2_hi(x[u][j], ks[2 * u][w / 2]) : scale2_lo(x[u][j], ks[2 * u][w / 2]);
              y[u][j] = w & 1 ? scale2_hi(y[u][j], ks[2 * u + 1][w / 2]) : scale2_lo(y[u][j], ks[2 * u + 1][w / 2]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint4 b;
            if constexpr (QS) b = queries[(n * (D / 32) + w) * 32 + lane];
            else b = make_uint4(qf[n][4 * w], qf[n][4 * w + 1], qf[n][4 * w + 2], qf[n][4 * w + 3]);
#pragma unroll
            for (int u = 0; u < U; ++u) mk::mma_16816(sc[u][n], x[u][0], y[u][0], x[u][1], y[u][1], b.x, b.y);
#pragma unroll
            for (int u = 0; u < U; ++u) mk::mma_16816(sc[u][n], x[u][2], y[u][2], x[u][3], y[u][3], b.z, b.w);
          }
        }
        // ---- masks, running reference, p ----
        const bool open = tok0 >= open_lo && tok0 + kUnit <= open_hi && bad == 0;
        if (!open) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int tok = tok0 + kTile * u + tok_g + 8 * (j >> 1), r = 8 * n + 2 * q + (j & 1);
                const int row = (r0 + min(r, nrows - 1)) / a.group, x = first + row;
                bool see = tok < len && !((bad >> u) & 1u);
                if (a.tree != nullptr) {
                  const int d = tok - first;
                  see = see && (d < 0 || (d < 64 && ((a.tree[cur.it.row0 + row] >> d) & 1ull)));
                } else {
                  see = see && tok <= x && (a.window <= 0 || tok > x - a.window);
                }
                if (!see) sc[u][n][j] = -INFINITY;
              }
        }
        float hi[NT][2];  // the largest product; compared as its p's exponent is formed, so that no p is above 2^kSlack
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(sc[0][n][j], sc[0][n][2 + j]);
            top = fmaxf(top, fmaxf(sc[1][n][j], sc[1][n][2 + j]));
            hi[n][j] = top;
            rise |= fmaf(top, factor[n][j], -m[n][j]) > kSlack;
          }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top = hi[n][j];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              // of the rows that need it alone: a row's result does not depend on the block's others
              const float v = fmaf(top, factor[n][j], -m[n][j]) > kSlack ? top * factor[n][j] - kBelow : m[n][j];
              const float c = exp2_approx(m[n][j] - v);
              m[n][j] = v;
              l[n][j] *= c;
#pragma unroll
              for (int k = 0; k < KS; ++k) { acc[n][k][j] *= c; acc[n][k][2 + j] *= c; }
            }
        }
        uint32_t pf[U][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f0 = factor[n][0], f1 = factor[n][1];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float p0 = exp2_approx(fmaf(sc[u][n][0], f0, -m[n][0])), p1 = exp2_approx(fmaf(sc[u][n][1], f1, -m[n][1]));
            const float p2 = exp2_approx(fmaf(sc[u][n][2], f0, -m[n][0])), p3 = exp2_approx(fmaf(sc[u][n][3], f1, -m[n][1]));
            l[n][0] += p0 + p2;
            l[n][1] += p1 + p3;
            pf[u][n][0] = movmatrix(half2_bits(p0, p1));
            pf[u][n][1] = movmatrix(half2_bits(p2, p3));
          }
        }
        // ---- O^T += V^T P^T ----
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint8_t* tile = unit + u * TILE;
          uint32_t vs[4];  // D = 256: two bytes, else one
          const uint8_t* sp = tile + 17 * D + q * (D / 16) + (D == 64 ? g >> 1 : D == 128 ? g : 2 * g);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            vs[j] = D == 256 ? *reinterpret_cast<const uint16_t*>(sp + j * (D / 4)) : sp[j * (D / 4)];
          if (tok0 + kUnit > len || bad != 0) {  // scales that are no token's of the sequence: 0, so that 0 * p is 0
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (tok0 + kTile * u + 4 * j + q >= len || ((bad >> u) & 1u)) vs[j] = 0;
          }
          Words<D / 64> vc[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) vc[j] = shared_words<D / 64>(tile + 8 * D + (4 * j + q) * (D / 2) + g * (D / 16));
          uint32_t vscale[2][D == 256 ? 2 : 1];  // tokens (q, q + 4), (q + 8, q + 12)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t x = vs[2 * j], y = vs[2 * j + 1];
            if constexpr (D == 256) {
              const uint32_t four = __byte_perm(x, y, 0x5140);  // x0 y0 x1 y1
              vscale[j][0] = e4m3x2_to_f16x2(four);
              vscale[j][1] = e4m3x2_to_f16x2(four >> 16);
            } else {
              vscale[j][0] = e4m3x2_to_f16x2(x | (y << 8));
            }
          }
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {  // words: 8 channels, 4 m-tiles
            uint32_t e[2][4], o[2][4];        // even and odd channels of each token pair
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t x = vc[2 * j].w[w], y = vc[2 * j + 1].w[w];
              const uint32_t we = (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
              const uint32_t wo = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
              e2m1x8_to_f16x2x4(we, e[j][0], e[j][1], e[j][2], e[j][3]);
              e2m1x8_to_f16x2x4(wo, o[j][0], o[j][1], o[j][2], o[j][3]);
              const uint32_t s = vscale[j][D == 256 ? w / 2 : 0];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                e[j][k] = hmul2_bits(e[j][k], s);
                o[j][k] = hmul2_bits(o[j][k], s);
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mk::mma_16816(acc[n][4 * w + k], e[0][k], o[0][k], e[1][k], o[1][k], pf[u][n][0], pf[u][n][1]);
          }
        }
        __syncwarp();  // every lane has read the stage
      }
      if (i + S < n_units) issue(cur, i + S, stage);
      if (++stage == S) stage = 0;
    }
    // the next part of the chunk: its first units are in flight while this one's results leave
    if (lane == 0) advance<ROWS, kUnit>(steps, cur, s_walk[warp][turn ^ 1], s_chunk[warp].end);
    __syncwarp();
    const bool more = s_walk[warp][turn ^ 1].more;
    if (more) start(s_walk[warp][turn ^ 1]);

    const bool whole = cur.count == cur.it.units;
    float* part = a.part + (2 * static_cast<size_t>(chunk) + (cur.off == 0 ? 1 : 0)) * L::kPart;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], o);
      }
      // accumulator 2 e + i of m-tile k: channel g D/8 + 2k + e, row 2q + i
      if (whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * n + 2 * q + i;
          if (r < nrows) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
              finish<D>(a, cur.it.row0, h, r0 + r, g * (D / 8) + 2 * k, acc[n][k][i], acc[n][k][2 + i], m[n][i], l[n][i]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k)
          reinterpret_cast<float4*>(part)[(n * KS + k) * 32 + lane] =
              make_float4(acc[n][k][0], acc[n][k][1], acc[n][k][2], acc[n][k][3]);
        if (g == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            part[ROWS * D + 8 * n + 2 * q + i] = m[n][i];
            part[ROWS * D + ROWS + 8 * n + 2 * q + i] = l[n][i];
          }
        }
      }
    }
    if (lane == 0 && !whole && cur.off == 0) {  // the item goes on in the chunks up to that of its last unit
      Piece p;
      p.on = 1;
      p.last = static_cast<int>((cur.pos + cur.it.units - 1) / s_chunk[warp].per);
      p.row0 = cur.it.row0; p.r0 = r0; p.nrows = nrows; p.h = h;
      a.pieces[chunk] = p;
    }
    if (!more) break;
  }
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

template <int D, int NT, int W, int S, int CTAS, bool QS>
cudaError_t launch(AttendArgs a, int num_sms, cudaStream_t stream) {
  typedef Shape<D, NT, W, S, QS> L;
  constexpr int smem = L::kTotal;
  static_assert(smem <= 227 * 1024 / CTAS - 2048, "shared memory");
  a.page_magic = page_magic(a.c);
  constexpr int stride = L::kPart;  // floats of a partial result
  const int grid = max(1, min(CTAS * num_sms, min(kMaxChunks / W, static_cast<int>(kPartFloats / 2 / stride / W))));
  a.chunks = grid * W;
  const cudaError_t e = launch_ready<attend_kernel<D, NT, W, S, CTAS, QS>>(dim3(grid), dim3(32 * W), smem, stream, a);
  if (e != cudaSuccess) return e;
  return launch_ready<join_kernel<D, NT>>(dim3((a.chunks + kJoinChunks - 1) / kJoinChunks, NT), dim3(kJoinThreads), 0, stream, a);
}

}  // namespace

// Blocks of up to 128 rows from 17 rows on at head size 128, and from 33 on at 64 and 256; measured on 32 sequences
// of 4096 to 8192 tokens and 8 (at 256: 2) K/V heads, wide against warp-MMA, in us:
//   128: 16 rows 110 and 71, 32 rows 110 and 124, 64 rows 115 and 230
//    64: 16 rows 84 and 55, 32 rows 84 and 83, 64 rows 88 and 147
//   256: 16 rows 70 and 45, 32 rows 71 and 67, 64 rows 73 and 114
// The wide kernel's time goes by tokens and hardly by rows.  The warp-MMA kernel's goes by blocks: of 32 rows at 64, of 16 at
// 128 and 256, so that 17 to 32 rows read the cache twice there and take what 32 take.  One kernel takes a whole call: a long
// step among short ones takes them all to the wide one.
cudaError_t launch_attend(const AttendArgs& a, int row_tile, int num_sms, cudaStream_t stream) {
  if (row_tile > (a.c.dim == 128 ? 16 : 32)) return launch_attend_wide(a, num_sms, stream);
  switch (a.c.dim) {
    case 64:
      return row_tile <= 8    ? launch<64, 1, 8, 4, 2, false>(a, num_sms, stream)
             : row_tile <= 16 ? launch<64, 2, 8, 4, 2, false>(a, num_sms, stream)  // 28 bytes spilled for two CTAs an SM
                              : launch<64, 4, 8, 4, 1, false>(a, num_sms, stream);
    case 128:
      return row_tile <= 8 ? launch<128, 1, 16, 2, 1, false>(a, num_sms, stream) : launch<128, 2, 12, 3, 1, true>(a, num_sms, stream);
    default:
      return row_tile <= 8 ? launch<256, 1, 8, 2, 1, false>(a, num_sms, stream) : launch<256, 2, 8, 2, 1, true>(a, num_sms, stream);
  }
}

}  // namespace kv4
}  // namespace moe
