// Attention of a step's query rows over the 4-bit paged cache.
//
// out = sum_t p_t v_t / sum_t p_t with p_t = exp2(z_t - m), z = scale log2(e) q.k: one pass over
// the tokens with a running reference m, FP32 sums, and the products on warp-level tensor-core
// MMAs (m16n8k16, FP16 operands, FP32 accumulators).  E2M1 x E4M3 has at most 6 significant bits
// and is exact in FP16, and a query row is brought by a power of two into FP16's range, so the
// scores are exact products summed in FP32; the one rounding inside is that of p to FP16 (11
// bits, relative to a row's largest about 1).
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
// memory, one bulk copy a tile, kStages tiles ahead, so that no warp waits for another and the bytes
// in flight do not cost registers: with loads to registers one tile ahead the same products ran at
// 45 % of the copy bandwidth, waiting for memory.  The first tiles of the next item are in flight
// while the warps' results of this one are joined.
//
// Work split.  The (sequence, K/V head, block of 8 NT rows) items are laid end to end, each as
// long as the tiles of 16 tokens it has to read, and cut into one equal range per CTA, so that any
// mix of lengths keeps every SM busy.  A CTA joins its warps' results per item in shared memory; an
// item cut over several CTAs leaves partial results (FP32 sums, m and l) in the workspace, and the
// last of its CTAs to arrive joins them in the order of the CTAs, so results do not depend on
// timing.  The ranges are found on the device from the lengths: no host wait, no plan.
#include "kv4_common.cuh"
#include "mma_parts.cuh"

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
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr float kLowest = -3.0e38f;  // a row's reference before it has seen a token
constexpr int kStatusTimeout = static_cast<int>(MOE_KV4_TIMEOUT);
constexpr long long kWaitCycles = 1ll << 32;   // ~2 s: a copy takes microseconds
constexpr long long kDrainCycles = 1ll << 24;

// Wait for a phase of a barrier by the whole warp, with a limit.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, long long limit) {
  bool ok = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    const long long t0 = clock64();
    while (!ok && clock64() - t0 < limit) ok = mbar_try_wait(bar, parity);
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

// The item that a position of the work lies in.
struct Item {
  int s;         // sequence
  int row0, n;   // its rows
  int len;       // its tokens
  int first;     // position of its first row
  int lo, tiles; // first tile and number of tiles of each of its items
  int blocks;    // row blocks
  int items;     // heads * blocks (0: no rows)
};

constexpr long long kMaxTokens = 1ll << 30;

template <int ROWS>
__device__ __forceinline__ Item item_of(const AttendArgs& a, int s) {
  Item it;
  const StepRows st = step_rows(a.cu, s, a.rows);
  it.s = s;
  it.row0 = st.first;
  it.n = st.n;
  it.items = 0;
  it.tiles = 1;
  if (st.n == 0) return it;
  const long long room = min(static_cast<long long>(a.c.max_pages) * a.c.page_size, kMaxTokens);
  const int len = max(ld(a.c.lens + s), 0);
  it.len = static_cast<int>(min(static_cast<long long>(len), room));
  it.first = len - st.n;
  const int from = a.window > 0 ? max(it.first - a.window + 1, 0) : 0;
  it.lo = min(from, max(it.len - 1, 0)) / kTile;
  it.tiles = max((it.len + kTile - 1) / kTile - it.lo, 1);
  it.blocks = static_cast<int>((static_cast<long long>(st.n) * a.group + ROWS - 1) / ROWS);
  it.items = a.c.heads * it.blocks;
  return it;
}
__device__ __forceinline__ long long work_of(const Item& it) { return static_cast<long long>(it.items) * it.tiles; }

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

// W warps, blocks of 8 NT rows, rings of S tiles; QS: the query rows' operands are kept in shared
// memory (one copy for all warps) instead of registers.
template <int D, int NT, int W, int S, bool QS>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kJoin = W / 2;  // warps whose sums lie in shared memory at a time
  static constexpr int kRingBytes = W * S * 18 * D;
  static constexpr int kSumBytes = kJoin * kRows * (D + 4) * 4;  // rows padded by 4 floats
  static constexpr int kStatBytes = W * kRows * 2 * 4;           // the warps' m and l
  static constexpr int kQBytes = QS ? kRows * D * 2 : 0;
  static constexpr int kSmem = kRingBytes + kSumBytes + kStatBytes + kRows * 2 * 4 + kQBytes + W * S * 8;
};

// A CTA's place in the work: an item and the part of it that lies in the CTA's range.
struct Walk {
  Item it;
  int idx, off, count;  // item of the sequence, first tile of the item, tiles
  long long pos;
};
template <int ROWS>
__device__ __forceinline__ bool advance(const AttendArgs& a, Walk& w, long long end) {
  w.pos += w.count;
  if (w.pos >= end) return false;
  w.off = 0;  // the range goes on past this item
  if (++w.idx == w.it.items) {
    w.idx = 0;
    int s = w.it.s;
    do w.it = item_of<ROWS>(a, ++s); while (w.it.items == 0);
  }
  w.count = static_cast<int>(min(end - w.pos, static_cast<long long>(w.it.tiles)));
  return true;
}

template <int D, int NT, int W, int S, int CTAS, bool QS>
__global__ void __launch_bounds__(32 * W, CTAS) attend_kernel(AttendArgs a) {
  constexpr int ROWS = 8 * NT;
  constexpr int KS = D / 16;   // k16 steps of a score, and m16 tiles of the output
  constexpr int PITCH = D + 4;
  constexpr int TILE = 18 * D;
  constexpr int kThreads = 32 * W;
  constexpr int JOIN = W / 2;
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_sum = reinterpret_cast<float*>(smem + W * S * TILE);        // [JOIN][rows][PITCH]
  uint4* s_q = reinterpret_cast<uint4*>(s_sum + JOIN * ROWS * PITCH);  // QS: [n-tile][word][lane]
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(s_q + (QS ? ROWS * D / 8 : 0));  // [warps][S]
  float* s_m = reinterpret_cast<float*>(s_bar + W * S);                // [warps][rows]
  float* s_l = s_m + W * ROWS;                                         // [warps][rows]
  float* s_mt = s_l + W * ROWS;                                        // [rows] joined m
  float* s_lt = s_mt + ROWS;                                           // [rows] joined l
  __shared__ long long s_scan[W];
  __shared__ long long s_off;
  __shared__ int s_seq, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const uint8_t* ring = smem + warp * S * TILE;
  const uint32_t ring_addr = smem_addr(ring), bar0 = smem_addr(s_bar + warp * S);
  if (lane < S) mbar_init(bar0 + 8 * lane, 1);
  fence_barrier_init();
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();

  // this CTA's range [pos, end) of the work
  const int per_thread = (a.c.seqs + kThreads - 1) / kThreads;
  const int sa = min(tid * per_thread, a.c.seqs), sb = min(sa + per_thread, a.c.seqs);
  long long mine = 0;
  for (int s = sa; s < sb; ++s) mine += work_of(item_of<ROWS>(a, s));
  long long total;
  const long long before = block_prefix<W>(mine, s_scan, total);
  const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(W));
  Walk cur;
  cur.pos = per * blockIdx.x;
  const long long end = min(cur.pos + per, total);
  if (cur.pos >= end) return;
  if (cur.pos >= before && cur.pos < before + mine) {
    long long at = before;
    for (int s = sa; s < sb; ++s) {
      const long long w = work_of(item_of<ROWS>(a, s));
      if (cur.pos < at + w) {
        s_seq = s;
        s_off = cur.pos - at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  cur.it = item_of<ROWS>(a, s_seq);
  cur.idx = static_cast<int>(s_off / cur.it.tiles);
  cur.off = static_cast<int>(s_off - static_cast<long long>(cur.idx) * cur.it.tiles);
  cur.count = static_cast<int>(min(end - cur.pos, static_cast<long long>(cur.it.tiles - cur.off)));

  // ---- this warp's ring.  Its i-th tile of an item's part is tile `warp + i W` of the part ----
  int stage = 0;            // next stage to be consumed; all stages are empty between items
  uint32_t parity = 0;      // of that stage's phase
  uint32_t invalid = 0;     // stages whose tile has no page
  bool dead = false;        // a copy did not arrive
  int pids = 0, pids_next = 0;  // this lane's page numbers: of tiles 32 b + lane and the batch after
  auto load_pids = [&](const Walk& w, int i) {
    const int n = i * W + warp;  // tile of the part
    const int t = w.it.lo + w.off + n;
    if (n >= w.count || t * kTile >= w.it.len) return -1;
    const int pi = a.c.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(static_cast<uint32_t>(t), a.page_magic));
    const int page = ld(a.c.table + static_cast<size_t>(w.it.s) * a.c.max_pages + pi);
    if (page < 0 || page >= a.c.pages) {
      atomicOr(a.c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
      return -1;
    }
    return page;
  };
  // start the copy of the part's tile i (this warp's count) into stage st
  auto issue = [&](const Walk& w, int i, int st, int h) {
    if (i > 0 && (i & 31) == 0) {
      pids = pids_next;
      pids_next = load_pids(w, i + 32 + lane);
    }
    const int page = __shfl_sync(0xffffffffu, pids, i & 31);
    if (page < 0) {
      invalid |= 1u << st;
      return;
    }
    invalid &= ~(1u << st);
    if (lane == 0) {
      const int t = w.it.lo + w.off + i * W + warp;
      const int pi = a.c.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(static_cast<uint32_t>(t), a.page_magic));
      const uint8_t* src = a.c.pool + static_cast<size_t>(page) * a.c.page_bytes +
                           static_cast<size_t>(h * a.c.tiles_per_page + (t - pi * a.c.tiles_per_page)) * TILE;
      mbar_arrive_expect_tx(bar0 + 8 * st, TILE);
      bulk_copy_g2s(ring_addr + st * TILE, src, TILE, bar0 + 8 * st);
    }
  };
  auto tiles_of = [&](const Walk& w) { return w.count > warp ? (w.count - warp + W - 1) / W : 0; };
  auto start = [&](const Walk& w) {  // the first tiles of a part
    if (dead) return;
    const int n = tiles_of(w), h = w.idx / w.it.blocks;
    pids = load_pids(w, lane);
    pids_next = n > 32 ? load_pids(w, 32 + lane) : -1;
    int st = stage;
    for (int i = 0; i < S && i < n; ++i) {
      issue(w, i, st, h);
      if (++st == S) st = 0;
    }
  };
  start(cur);

  while (true) {
    const Item& it = cur.it;
    const int h = cur.idx / it.blocks, blk = cur.idx - h * it.blocks, off = cur.off, count = cur.count;
    const int r0 = blk * ROWS;  // first of the block's rows: row r is (step row r / group, query head r % group)
    const int nrows = min(ROWS, it.n * a.group - r0);

    // the query rows as FP16, brought near 2^10 by a power of two that z's factor takes back; the
    // sign of the scale goes to the rows, so that a larger product is a larger score
    uint32_t qf[QS ? 1 : NT][QS ? 1 : 2 * KS];
    float factor[NT][2];  // of the rows 2q and 2q + 1 of each n-tile
    {
      const float sign = a.scale2 < 0.f ? -1.f : 1.f, size = fabsf(a.scale2);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = 8 * t + g;
        const bool ok = r < nrows;
        const int step_row = (r0 + r) / a.group, hq = h * a.group + (r0 + r) - step_row * a.group;
        const char* src = static_cast<const char*>(a.q) +
                          2 * ((it.row0 + (ok ? step_row : 0)) * a.q_row + (ok ? hq : 0) * a.q_head + 8 * q);
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
        const float down = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23) * size;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 f = unpack2(raw[i], a.fp16);
          raw[i] = half2_bits(f.x * up, f.y * up);
          if constexpr (!QS) qf[t][i] = raw[i];
        }
        if constexpr (QS) {
          if (t % W == warp) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              s_q[(t * (D / 32) + i) * 32 + lane] = make_uint4(raw[4 * i], raw[4 * i + 1], raw[4 * i + 2], raw[4 * i + 3]);
          }
        }
        factor[t][0] = __shfl_sync(0xffffffffu, down, 8 * q);      // lane of row 2q: g = 2q
        factor[t][1] = __shfl_sync(0xffffffffu, down, 8 * q + 4);
      }
    }
    if constexpr (QS) __syncthreads();

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
    const int open_hi = a.tree != nullptr ? it.first : min(it.first + r0 / a.group + 1, it.len);
    const int open_lo = a.window > 0 ? max(it.first + (r0 + nrows - 1) / a.group - a.window + 1, 0) : 0;

    const int n_tiles = dead ? 0 : tiles_of(cur);
    int tok0 = (it.lo + off + warp) * kTile;
    for (int i = 0; i < n_tiles; ++i, tok0 += W * kTile) {
      if (!((invalid >> stage) & 1u)) {
        if (!warp_wait(bar0 + 8 * stage, parity >> stage & 1u, kWaitCycles)) {
          if (lane == 0) atomicOr(a.c.status, kStatusTimeout);
          dead = true;
          break;
        }
        parity ^= 1u << stage;
        const uint8_t* tile = ring + stage * TILE;
        const int tok_g = (g >> 1) + 4 * (g & 1);
        // ---- S^T = K Q^T, one word (8 channels, half a scale block) of each token at a time ----
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        uint32_t ks0[D / 64], ks1[D / 64];
        key_scales<D>(tile + 16 * D + tok_g * (D / 16), q, ks0);
        key_scales<D>(tile + 16 * D + (tok_g + 8) * (D / 16), q, ks1);
        const uint8_t* kp = tile + tok_g * 16 + q * 4;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t x[4], y[4];
          e2m1x8_to_f16x2x4(*reinterpret_cast<const uint32_t*>(kp + w * 256), x[0], x[1], x[2], x[3]);
          e2m1x8_to_f16x2x4(*reinterpret_cast<const uint32_t*>(kp + w * 256 + 128), y[0], y[1], y[2], y[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = w & 1 ? scale2_hi(x[j], ks0[w / 2]) : scale2_lo(x[j], ks0[w / 2]);
            y[j] = w & 1 ? scale2_hi(y[j], ks1[w / 2]) : scale2_lo(y[j], ks1[w / 2]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint4 b;
            if constexpr (QS) b = s_q[(n * (D / 32) + w) * 32 + lane];
            else b = make_uint4(qf[n][4 * w], qf[n][4 * w + 1], qf[n][4 * w + 2], qf[n][4 * w + 3]);
            mk::mma_16816(sc[n], x[0], y[0], x[1], y[1], b.x, b.y);
            mk::mma_16816(sc[n], x[2], y[2], x[3], y[3], b.z, b.w);
          }
        }
        // ---- masks, running reference, p ----
        const bool open = tok0 >= open_lo && tok0 + kTile <= open_hi;
        if (!open) {  // products become scores here; their factors are 1 below
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int tok = tok0 + tok_g + 8 * (j >> 1), r = 8 * n + 2 * q + (j & 1);
              const int row = (r0 + min(r, nrows - 1)) / a.group, x = it.first + row;
              bool see = tok < it.len;
              if (a.tree != nullptr) {
                const int d = tok - it.first;
                see = see && (d < 0 || (d < 64 && ((a.tree[it.row0 + row] >> d) & 1ull)));
              } else {
                see = see && tok <= x && (a.window <= 0 || tok > x - a.window);
              }
              sc[n][j] = see ? sc[n][j] * factor[n][j & 1] : -INFINITY;
            }
        }
        float hi[NT][2];
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float top = fmaxf(sc[n][j], sc[n][2 + j]);
            hi[n][j] = open ? top * factor[n][j] : top;
            rise |= hi[n][j] > m[n][j] + kSlack;
          }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float v = fmaxf(hi[n][j], m[n][j]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
              const float c = exp2_approx(m[n][j] - v);
              m[n][j] = v;
              l[n][j] *= c;
#pragma unroll
              for (int k = 0; k < KS; ++k) { acc[n][k][j] *= c; acc[n][k][2 + j] *= c; }
            }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f0 = open ? factor[n][0] : 1.f, f1 = open ? factor[n][1] : 1.f;
          const float p0 = exp2_approx(fmaf(sc[n][0], f0, -m[n][0])), p1 = exp2_approx(fmaf(sc[n][1], f1, -m[n][1]));
          const float p2 = exp2_approx(fmaf(sc[n][2], f0, -m[n][0])), p3 = exp2_approx(fmaf(sc[n][3], f1, -m[n][1]));
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          pf[n][0] = movmatrix(half2_bits(p0, p1));
          pf[n][1] = movmatrix(half2_bits(p2, p3));
        }
        // ---- O^T += V^T P^T ----
        uint32_t vs[4];  // D = 256: two bytes, else one
        {
          const uint8_t* sp = tile + 17 * D + q * (D / 16) + (D == 64 ? g >> 1 : D == 128 ? g : 2 * g);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            vs[j] = D == 256 ? *reinterpret_cast<const uint16_t*>(sp + j * (D / 4)) : sp[j * (D / 4)];
          if (tok0 + kTile > it.len) {  // scales past the end are not the sequence's: 0, so that 0 * p is 0
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (tok0 + 4 * j + q >= it.len) vs[j] = 0;
          }
        }
        Words<D / 64> vc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) vc[j] = shared_words<D / 64>(tile + 8 * D + (4 * j + q) * (D / 2) + g * (D / 16));
        uint32_t vscale[2][D == 256 ? 2 : 1];  // tokens (q, q + 4), (q + 8, q + 12)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t u = vs[2 * j], v = vs[2 * j + 1];
          if constexpr (D == 256) {
            const uint32_t four = __byte_perm(u, v, 0x5140);  // u0 v0 u1 v1
            vscale[j][0] = e4m3x2_to_f16x2(four);
            vscale[j][1] = e4m3x2_to_f16x2(four >> 16);
          } else {
            vscale[j][0] = e4m3x2_to_f16x2(u | (v << 8));
          }
        }
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {  // words: 8 channels, 4 m-tiles
          uint32_t e[2][4], o[2][4];        // even and odd channels of each token pair
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t u = vc[2 * j].w[w], v = vc[2 * j + 1].w[w];
            const uint32_t we = (u & 0x0f0f0f0fu) | ((v << 4) & 0xf0f0f0f0u);
            const uint32_t wo = ((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u);
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
              mk::mma_16816(acc[n][4 * w + k], e[0][k], o[0][k], e[1][k], o[1][k], pf[n][0], pf[n][1]);
        }
        __syncwarp();  // every lane has read the stage
      }
      if (i + S < n_tiles) issue(cur, i + S, stage, h);
      if (++stage == S) stage = 0;
    }
    if (dead) {  // let what is still in flight land before the memory is given up
      for (int st = 0; st < S; ++st)
        if (!((invalid >> st) & 1u)) warp_wait(bar0 + 8 * st, parity >> st & 1u, kDrainCycles);
    }
    Walk nxt = cur;
    const bool more = advance<ROWS>(a, nxt, end);
    if (more) start(nxt);

    // ---- join the warps: the second half's sums go to the first half's registers through shared
    // memory, the first half's to all threads ----
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], o);
        l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], o);
      }
      if (g == 0) {
        const int r = 8 * n + 2 * q;
        s_m[warp * ROWS + r] = m[n][0];
        s_m[warp * ROWS + r + 1] = m[n][1];
        s_l[warp * ROWS + r] = l[n][0];
        s_l[warp * ROWS + r + 1] = l[n][1];
      }
    }
    __syncthreads();
    if (tid < ROWS) {
      float mt = kLowest, lt = 0.f;
      for (int w = 0; w < W; ++w) mt = fmaxf(mt, s_m[w * ROWS + tid]);
      for (int w = 0; w < W; ++w) {
        const float c = exp2_approx(s_m[w * ROWS + tid] - mt);
        lt += c * s_l[w * ROWS + tid];
        s_m[w * ROWS + tid] = c;  // the warp's factor
      }
      s_mt[tid] = mt;
      s_lt[tid] = lt;
    }
    __syncthreads();
    // accumulator i of m-tile k: channel g D/8 + 2k + (i >> 1), row 2q + (i & 1)
    const int slot = warp % JOIN;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float c = s_m[warp * ROWS + 8 * n + 2 * q + i];
#pragma unroll
        for (int k = 0; k < KS; ++k) { acc[n][k][i] *= c; acc[n][k][2 + i] *= c; }
      }
    auto spot = [&](int n, int i, int k) {
      return reinterpret_cast<float2*>(s_sum + (slot * ROWS + 8 * n + 2 * q + i) * PITCH + g * (D / 8) + 2 * k);
    };
    if (warp >= JOIN) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < KS; ++k) *spot(n, i, k) = make_float2(acc[n][k][i], acc[n][k][2 + i]);
    }
    __syncthreads();
    if (warp < JOIN) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            float2* p = spot(n, i, k);
            const float2 x = *p;
            *p = make_float2(acc[n][k][i] + x.x, acc[n][k][2 + i] + x.y);
          }
    }
    __syncthreads();

    auto finish = [&](int r, int d4, float4 v, float mt, float lt) {  // channels 4 d4 .. of row r
      const int step_row = it.row0 + (r0 + r) / a.group, hq = h * a.group + (r0 + r) % a.group;
      const int64_t at = static_cast<int64_t>(step_row) * (a.c.heads * a.group) + hq;
      const float f = lt > 0.f || lt != lt ? a.v_ts / lt : 0.f;
      uint2 o;
      o.x = pack2(v.x * f, v.y * f, a.fp16);
      o.y = pack2(v.z * f, v.w * f, a.fp16);
      *reinterpret_cast<uint2*>(static_cast<char*>(a.out) + 2 * (at * D + 4 * d4)) = o;
      if (d4 == 0 && a.lse != nullptr)
        a.lse[at] = lt > 0.f || lt != lt ? (mt + log2f(lt)) * kLn2 : -INFINITY;
    };
    const bool whole = count == it.tiles;
    float* part = a.part + (2 * static_cast<size_t>(blockIdx.x) + (off == 0 ? 1 : 0)) * a.part_floats;
    for (int i = tid; i < ROWS * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d4 = i - r * (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < JOIN; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(s_sum + (w * ROWS + r) * PITCH + 4 * d4);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      if (whole) {
        if (r < nrows) finish(r, d4, v, s_mt[r], s_lt[r]);
      } else {
        *reinterpret_cast<float4*>(part + 4 * i) = v;
        if (d4 == 0) {
          part[kPartSums + r] = s_mt[r];
          part[kPartSums + kPartRows + r] = s_lt[r];
        }
      }
    }
    if (!whole) {
      // the CTAs that hold parts of this item: those whose ranges its tiles [b, b + tiles) meet
      const long long b = cur.pos - off;
      const int c0 = static_cast<int>(b / per), c1 = static_cast<int>((b + it.tiles - 1) / per);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t old = atom_add_acqrel_u32(a.counters + c0, 1u);
        s_last = old == static_cast<uint32_t>(c1 - c0);
        if (s_last) a.counters[c0] = 0;  // for the next call
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        auto part_of = [&](int c) {  // the first CTA's part starts at the item's first tile
          return a.part + (2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0)) * a.part_floats;
        };
        if (tid < ROWS) {
          float mt = kLowest, lt = 0.f;
          for (int c = c0; c <= c1; ++c) mt = fmaxf(mt, ld(part_of(c) + kPartSums + tid));
          for (int c = c0; c <= c1; ++c)
            lt += exp2_approx(ld(part_of(c) + kPartSums + tid) - mt) * ld(part_of(c) + kPartSums + kPartRows + tid);
          s_mt[tid] = mt;
          s_lt[tid] = lt;
        }
        __syncthreads();
        for (int i = tid; i < nrows * (D / 4); i += kThreads) {
          const int r = i / (D / 4), d4 = i - r * (D / 4);
          const float mt = s_mt[r];
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c = c0; c <= c1; ++c) {
            const float* p = part_of(c);
            const float f = exp2_approx(ld(p + kPartSums + r) - mt);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(p + 4 * i));
            v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
          }
          finish(r, d4, v, mt, s_lt[r]);
        }
      }
    }
    __syncthreads();  // the shared arrays are free for the next item

    if (!more) break;
    cur = nxt;
  }
}

template <int D, int NT, int W, int S, int CTAS, bool QS>
cudaError_t launch(AttendArgs a, int num_sms, cudaStream_t stream) {
  constexpr int smem = Shape<D, NT, W, S, QS>::kSmem;
  static_assert(8 * NT * D <= kPartSums && 8 * NT <= kPartRows, "a partial result holds a block");
  auto kernel = attend_kernel<D, NT, W, S, CTAS, QS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // t / tiles_per_page = umulhi(t, magic): exact for t below 2^26 (2^30 tokens) and up to 64 tiles a page
  a.page_magic = static_cast<uint32_t>(((1ull << 32) + a.c.tiles_per_page - 1) / a.c.tiles_per_page);
  const int grid = min(CTAS * num_sms, kMaxGrid);
  return launch_pdl(kernel, dim3(grid), dim3(32 * W), smem, stream, a);
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& a, int row_tile, int num_sms, cudaStream_t stream) {
  switch (a.c.dim) {
    case 64:
      return row_tile <= 8    ? launch<64, 1, 8, 6, 2, false>(a, num_sms, stream)
             : row_tile <= 16 ? launch<64, 2, 8, 6, 2, false>(a, num_sms, stream)
                              : launch<64, 4, 12, 6, 1, false>(a, num_sms, stream);
    case 128:
      return row_tile <= 8    ? launch<128, 1, 8, 4, 2, false>(a, num_sms, stream)
             : row_tile <= 16 ? launch<128, 2, 12, 4, 1, false>(a, num_sms, stream)
                              : launch<128, 4, 8, 4, 1, true>(a, num_sms, stream);
    default:
      return row_tile <= 8 ? launch<256, 1, 12, 3, 1, false>(a, num_sms, stream) : launch<256, 2, 8, 4, 1, true>(a, num_sms, stream);
  }
}

}  // namespace kv4
}  // namespace moe
