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
// second product.  A lane (g = lane / 4, q = lane % 4) dequantises the channels
// [q D/4, (q + 1) D/4) of the tokens g and g + 8 of K, and the channels [g D/8, (g + 1) D/8) of
// the tokens 2q, 2q + 1, 2q + 8, 2q + 9 of V: the order of the channels within a sum is free, so
// each is one or a few wide loads of consecutive bytes.
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

template <int BYTES>
struct Bytes {
  uint32_t w[BYTES / 4];
};
// Streamed load of BYTES consecutive bytes (4, 8 or a multiple of 16).
template <int BYTES>
__device__ __forceinline__ void load_bytes(const uint8_t* p, Bytes<BYTES>& o) {
  if constexpr (BYTES == 4) {
    asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(o.w[0]) : "l"(p));
  } else if constexpr (BYTES == 8) {
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(o.w[0]), "=r"(o.w[1]) : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(o.w[4 * i]), "=r"(o.w[4 * i + 1]), "=r"(o.w[4 * i + 2]), "=r"(o.w[4 * i + 3])
                   : "l"(p + 16 * i));
  }
}

// N scale bytes (1, 2 or 4) in the low bytes of a word.
template <int N>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p) {
  if constexpr (N == 4) {
    uint32_t v;
    asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
  } else if constexpr (N == 2) {
    uint16_t v;
    asm volatile("ld.global.L1::no_allocate.b16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
  } else {
    uint32_t v;
    asm volatile("ld.global.L1::no_allocate.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
  }
}

// A lane's share of the keys of one tile as they lie in memory: tokens g and g + 8, channels
// [q D/4, +D/4) and their D / 64 scales; and of the values: tokens 2q, 2q + 1, 2q + 8, 2q + 9,
// channels [g D/8, +D/8) and their scale (D = 256: two).
template <int D>
struct KeyData {
  Bytes<D / 8> c[2];
  uint32_t s[2];
};
template <int D>
struct ValueData {
  Bytes<D / 16> c[4];
  uint32_t s[4];
};

template <int D>
__device__ __forceinline__ void load_keys(const uint8_t* tile, int lane, KeyData<D>& t) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tok = g + 8 * i;
    if constexpr (D == 64) {
      load_bytes<8>(tile + (q >> 1) * 256 + tok * 16 + (q & 1) * 8, t.c[i]);
      t.s[i] = load_scales<1>(tile + 16 * D + tok * (D / 16) + q);
    } else if constexpr (D == 128) {
      load_bytes<16>(tile + q * 256 + tok * 16, t.c[i]);
      t.s[i] = load_scales<2>(tile + 16 * D + tok * (D / 16) + 2 * q);
    } else {
      Bytes<16> a, b;
      load_bytes<16>(tile + (2 * q) * 256 + tok * 16, a);
      load_bytes<16>(tile + (2 * q + 1) * 256 + tok * 16, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) { t.c[i].w[j] = a.w[j]; t.c[i].w[4 + j] = b.w[j]; }
      t.s[i] = load_scales<4>(tile + 16 * D + tok * (D / 16) + 4 * q);
    }
  }
}
template <int D>
__device__ __forceinline__ void load_values(const uint8_t* tile, int lane, ValueData<D>& t) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = 2 * q + (i & 1) + 8 * (i >> 1);
    load_bytes<D / 16>(tile + 8 * D + tok * (D / 2) + g * (D / 16), t.c[i]);
    const uint8_t* sp = tile + 17 * D + tok * (D / 16);
    t.s[i] = D == 64 ? load_scales<1>(sp + (g >> 1)) : D == 128 ? load_scales<1>(sp + g) : load_scales<2>(sp + 2 * g);
  }
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

// W warps, blocks of 8 NT rows; QS: the query rows' operands are kept in shared memory (one copy for
// all warps) instead of registers.
template <int D, int NT, int W, bool QS>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kJoin = W / 2;  // warps whose sums lie in shared memory at a time
  static constexpr int kSumBytes = kJoin * kRows * (D + 4) * 4;  // rows padded by 4 floats
  static constexpr int kStatBytes = W * kRows * 2 * 4;           // the warps' m and l
  static constexpr int kQBytes = QS ? kRows * D * 2 : 0;
  static constexpr int kSmem = kSumBytes + kStatBytes + kRows * 2 * 4 + kQBytes;
};

template <int D, int NT, int W, int CTAS, bool QS>
__global__ void __launch_bounds__(32 * W, CTAS) attend_kernel(AttendArgs a) {
  constexpr int ROWS = 8 * NT;
  constexpr int KS = D / 16;   // k16 steps of a score, and m16 tiles of the output
  constexpr int PITCH = D + 4;
  constexpr int kThreads = 32 * W;
  constexpr int JOIN = W / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  float* s_sum = reinterpret_cast<float*>(smem);                       // [JOIN][rows][PITCH]
  float* s_m = s_sum + JOIN * ROWS * PITCH;                            // [warps][rows]
  float* s_l = s_m + W * ROWS;                                         // [warps][rows]
  float* s_mt = s_l + W * ROWS;                                        // [rows] joined m
  float* s_lt = s_mt + ROWS;                                           // [rows] joined l
  uint4* s_q = reinterpret_cast<uint4*>(s_lt + ROWS);                  // QS: [n-tile][word][lane]
  __shared__ long long s_scan[W];
  __shared__ long long s_off;
  __shared__ int s_seq, s_last;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;

  // this CTA's range [pos, end) of the work
  const int per_thread = (a.c.seqs + kThreads - 1) / kThreads;
  const int sa = min(tid * per_thread, a.c.seqs), sb = min(sa + per_thread, a.c.seqs);
  long long mine = 0;
  for (int s = sa; s < sb; ++s) mine += work_of(item_of<ROWS>(a, s));
  long long total;
  const long long before = block_prefix<W>(mine, s_scan, total);
  const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(W));
  long long pos = per * blockIdx.x;
  const long long end = min(pos + per, total);
  if (pos >= end) return;
  if (pos >= before && pos < before + mine) {
    long long at = before;
    for (int s = sa; s < sb; ++s) {
      const long long w = work_of(item_of<ROWS>(a, s));
      if (pos < at + w) {
        s_seq = s;
        s_off = pos - at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  Item it = item_of<ROWS>(a, s_seq);
  int idx = static_cast<int>(s_off / it.tiles);                  // item of the sequence
  int off = static_cast<int>(s_off - static_cast<long long>(idx) * it.tiles);  // tile of the item

  while (pos < end) {
    const int h = idx / it.blocks, blk = idx - h * it.blocks;
    const int count = static_cast<int>(min(end - pos, static_cast<long long>(it.tiles - off)));
    const int r0 = blk * ROWS;  // first of the block's rows: row r is (step row r / group, query head r % group)
    const int nrows = min(ROWS, it.n * a.group - r0);

    // the query rows as FP16, brought near 2^10 by a power of two that z's factor takes back; the
    // sign of the scale goes to the rows, so that a larger product is a larger score
    uint32_t qf[QS ? 1 : NT][QS ? 1 : 2 * KS];
    float factor[NT][2];  // of the rows 2q and 2q + 1 of each n-tile
    const float sign = a.scale2 < 0.f ? -1.f : 1.f, size = fabsf(a.scale2);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + g;
      const bool ok = r < nrows;
      const int step_row = (r0 + r) / a.group, hq = h * a.group + (r0 + r) % a.group;
      const char* src = static_cast<const char*>(a.q) +
                        2 * ((it.row0 + (ok ? step_row : 0)) * a.q_row + (ok ? hq : 0) * a.q_head + q * (D / 4));
      uint32_t raw[D / 8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = ok ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0, 0, 0, 0);
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
    if constexpr (QS) __syncthreads();

    float acc[NT][KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
    }
    // tokens that every row of the block sees without a look at the masks: from `open_lo`, before `open_hi`
    const int last_row = (r0 + nrows - 1) / a.group;
    const int open_hi = a.tree != nullptr ? it.first : min(it.first + r0 / a.group + 1, it.len);
    const int open_lo = a.window > 0 ? max(it.first + last_row - a.window + 1, 0) : 0;

    const int t0 = it.lo + off, t1 = t0 + count;
    const int* table = a.c.table + static_cast<size_t>(it.s) * a.c.max_pages;
    auto tile_ptr = [&](int t) -> const uint8_t* {  // nullptr: no token of it may be read
      if (t * kTile >= it.len) return nullptr;
      const int pi = a.c.tiles_per_page == 1 ? t : static_cast<int>(__umulhi(static_cast<uint32_t>(t), a.page_magic));
      const int page = ld(table + pi);
      if (page < 0 || page >= a.c.pages) {
        if (lane == 0) atomicOr(a.c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
        return nullptr;
      }
      return a.c.pool + static_cast<size_t>(page) * a.c.page_bytes +
             (static_cast<size_t>(h) * a.c.tiles_per_page + (t - pi * a.c.tiles_per_page)) * a.c.tile_bytes;
    };
    KeyData<D> kd;
    ValueData<D> vd;
    int t = t0 + warp;
    const uint8_t* p_cur = t < t1 ? tile_ptr(t) : nullptr;
    if (p_cur) {
      load_keys<D>(p_cur, lane, kd);
      load_values<D>(p_cur, lane, vd);
    }
    const uint8_t* p_nxt = t + W < t1 ? tile_ptr(t + W) : nullptr;
    for (; t < t1; t += W) {
      const uint8_t* p_nxt2 = t + 2 * W < t1 ? tile_ptr(t + 2 * W) : nullptr;
      const int tok0 = t * kTile;
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
      if (p_cur) {
        // ---- S^T = K Q^T, one word (8 channels, half a scale block) of each token at a time ----
        uint32_t kscale[2][D / 64];  // broadcast pairs
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t s2 = e4m3x2_to_f16x2(kd.s[i]);
          kscale[i][0] = bcast_lo_half(s2);
          if constexpr (D >= 128) kscale[i][1] = bcast_hi_half(s2);
          if constexpr (D == 256) {
            const uint32_t s3 = e4m3x2_to_f16x2(kd.s[i] >> 16);
            kscale[i][2] = bcast_lo_half(s3);
            kscale[i][3] = bcast_hi_half(s3);
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t x[4], y[4];
          e2m1x8_to_f16x2x4(kd.c[0].w[w], x[0], x[1], x[2], x[3]);
          e2m1x8_to_f16x2x4(kd.c[1].w[w], y[0], y[1], y[2], y[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = hmul2_bits(x[i], kscale[0][w / 2]);
            y[i] = hmul2_bits(y[i], kscale[1][w / 2]);
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
      }
      if (p_nxt) load_keys<D>(p_nxt, lane, kd);  // the next tile's, in flight until it comes round
      if (p_cur) {
        // ---- masks, running reference, p ----
        const bool open = tok0 >= open_lo && tok0 + kTile <= open_hi;
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = sc[n][i] * factor[n][i & 1];
            if (!open) {
              const int tok = tok0 + g + 8 * (i >> 1), r = 8 * n + 2 * q + (i & 1);
              const int row = (r0 + min(r, nrows - 1)) / a.group, x = it.first + row;
              bool see = tok < it.len;
              if (a.tree != nullptr) {
                const int j = tok - it.first;
                see = see && (j < 0 || (j < 64 && ((a.tree[it.row0 + row] >> j) & 1ull)));
              } else {
                see = see && tok <= x && (a.window <= 0 || tok > x - a.window);
              }
              if (!see) z[i] = -INFINITY;
            }
          }
          const float hi0 = fmaxf(z[0], z[2]), hi1 = fmaxf(z[1], z[3]);
          if (__any_sync(0xffffffffu, hi0 > m[n][0] + kSlack || hi1 > m[n][1] + kSlack)) {
            float n0 = fmaxf(hi0, m[n][0]), n1 = fmaxf(hi1, m[n][1]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
              n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
            }
            const float c0 = n0 == -INFINITY ? 1.f : exp2_approx(m[n][0] - n0);
            const float c1 = n1 == -INFINITY ? 1.f : exp2_approx(m[n][1] - n1);
            m[n][0] = n0;
            m[n][1] = n1;
            l[n][0] *= c0;
            l[n][1] *= c1;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              acc[n][i][0] *= c0; acc[n][i][1] *= c1; acc[n][i][2] *= c0; acc[n][i][3] *= c1;
            }
          }
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
          const float p0 = exp2_approx(z[0] - m0), p1 = exp2_approx(z[1] - m1);
          const float p2 = exp2_approx(z[2] - m0), p3 = exp2_approx(z[3] - m1);
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          pf[n][0] = movmatrix(half2_bits(p0, p1));
          pf[n][1] = movmatrix(half2_bits(p2, p3));
        }
        // ---- O^T += V^T P^T ----
        if (tok0 + kTile > it.len) {  // scales past the end are not the sequence's: 0, so that 0 * p is 0
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (tok0 + 2 * q + (i & 1) + 8 * (i >> 1) >= it.len) vd.s[i] = 0;
        }
        uint32_t vscale[2][D == 256 ? 2 : 1];  // (token 2q, 2q + 1), (2q + 8, 2q + 9)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t u = vd.s[2 * i], v = vd.s[2 * i + 1];
          vscale[i][0] = e4m3x2_to_f16x2((u & 0xffu) | ((v & 0xffu) << 8));
          if constexpr (D == 256) vscale[i][1] = e4m3x2_to_f16x2((u >> 8) | (v & 0xff00u));
        }
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {  // words: 8 channels, 4 m-tiles
          uint32_t e[2][4], o[2][4];        // even and odd channels, (2q, 2q + 1) and (2q + 8, 2q + 9)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t u = vd.c[2 * i].w[w], v = vd.c[2 * i + 1].w[w];
            const uint32_t we = (u & 0x0f0f0f0fu) | ((v << 4) & 0xf0f0f0f0u);
            const uint32_t wo = ((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u);
            e2m1x8_to_f16x2x4(we, e[i][0], e[i][1], e[i][2], e[i][3]);
            e2m1x8_to_f16x2x4(wo, o[i][0], o[i][1], o[i][2], o[i][3]);
            const uint32_t s = vscale[i][D == 256 ? w / 2 : 0];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              e[i][j] = hmul2_bits(e[i][j], s);
              o[i][j] = hmul2_bits(o[i][j], s);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mk::mma_16816(acc[n][4 * w + j], e[0][j], o[0][j], e[1][j], o[1][j], pf[n][0], pf[n][1]);
        }
      }
      if (p_nxt) load_values<D>(p_nxt, lane, vd);
      p_cur = p_nxt;
      p_nxt = p_nxt2;
    }

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
      float mt = -INFINITY, lt = 0.f;
      for (int w = 0; w < W; ++w) mt = fmaxf(mt, s_m[w * ROWS + tid]);
      for (int w = 0; w < W; ++w) {
        const float c = s_m[w * ROWS + tid] == -INFINITY ? 0.f : exp2_approx(s_m[w * ROWS + tid] - mt);
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
      const long long b = pos - off;
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
          float mt = -INFINITY, lt = 0.f;
          for (int c = c0; c <= c1; ++c) mt = fmaxf(mt, __ldcg(part_of(c) + kPartSums + tid));
          for (int c = c0; c <= c1; ++c) {
            const float mc = __ldcg(part_of(c) + kPartSums + tid);
            if (mc != -INFINITY) lt += exp2_approx(mc - mt) * __ldcg(part_of(c) + kPartSums + kPartRows + tid);
          }
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
            const float mc = __ldcg(p + kPartSums + r);
            const float f = mc == -INFINITY ? 0.f : exp2_approx(mc - mt);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(p + 4 * i));
            v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
          }
          finish(r, d4, v, mt, s_lt[r]);
        }
      }
    }
    __syncthreads();  // the shared arrays are free for the next item

    pos += count;
    off += count;
    if (off == it.tiles && pos < end) {
      off = 0;
      if (++idx == it.items) {
        idx = 0;
        int s = it.s;
        do it = item_of<ROWS>(a, ++s); while (it.items == 0);
      }
    }
  }
}

template <int D, int NT, int W, int CTAS, bool QS>
cudaError_t launch(AttendArgs a, int num_sms, cudaStream_t stream) {
  constexpr int smem = Shape<D, NT, W, QS>::kSmem;
  static_assert(8 * NT * D <= kPartSums && 8 * NT <= kPartRows, "a partial result holds a block");
  auto kernel = attend_kernel<D, NT, W, CTAS, QS>;
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
      return row_tile <= 8    ? launch<64, 1, 8, 2, false>(a, num_sms, stream)
             : row_tile <= 16 ? launch<64, 2, 8, 2, false>(a, num_sms, stream)
                              : launch<64, 4, 12, 1, false>(a, num_sms, stream);
    case 128:
      return row_tile <= 8    ? launch<128, 1, 8, 2, false>(a, num_sms, stream)
             : row_tile <= 16 ? launch<128, 2, 12, 1, false>(a, num_sms, stream)
                              : launch<128, 4, 8, 1, true>(a, num_sms, stream);
    default:
      return row_tile <= 8 ? launch<256, 1, 12, 1, false>(a, num_sms, stream) : launch<256, 2, 8, 1, true>(a, num_sms, stream);
  }
}

}  // namespace kv4
}  // namespace moe
