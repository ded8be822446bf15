// A step's K and V rows into the pages of the 4-bit cache (append), and the values that the
// pages hold back out of them (read).
//
// One thread owns two blocks of 16 channels of one row and head: 64 bytes of BF16 or FP16 on one
// side, 16 bytes of codes (one piece of K) and two scale bytes on the other, so no thread needs
// another's data (the largest magnitude of a block is found in registers) and consecutive threads
// touch consecutive bytes of the row.  Both kernels are bound by those bytes, 2 * 2 D H +
// 2 * 0.5625 D H per row, once there are enough of them; a short step is bound by the chain of lookups
// (row -> sequence -> page -> bytes), which a CTA does once for a few rows, a warp a row, in two trips
// to memory, with the inputs of its first units already under way.
//
// Scale and codes are those of exact divisions: inputs have 8 or 11 significant bits and scales 4,
// so ties are frequent, and a multiplication by a rounded reciprocal alone would move some of them
// to the wrong neighbour.  The quotients by the scale are the rounded product with the reciprocal,
// corrected once by the remainder, which one FMA gives exactly (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): 3 instructions instead of the
// ~10 of a division, of which there were 16 a thread.
//
// Measured: append and read of 6144 rows of 8 heads of 128 (65 MB in all) 25.7 us together, 0.37 of the copy
// bandwidth; with 16 bytes an access instead of a sector's 32, 29 us at the time; a step of 128 rows is bound by its two calls.
#include "kv4_common.cuh"

namespace moe {
namespace kv4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRowsPerCta = 32;
constexpr int kAppendCtas = 4, kReadCtas = 6;  // of an SM

// Where a row's bytes lie: the tile of head 0 that holds it, and its slot; tile nullptr: no page;
// slot < 0: the row is no sequence's.
struct RowPlace {
  uint8_t* tile;
  int slot;
};

// The place of a row, by a warp.  Its sequence is the last s with cu[s] <= row (empty sequences share
// a start and are passed over), found with 32 probes a step; at the last step, of up to 32
// sequences, the lanes have the ends and the lengths in hand.
__device__ __forceinline__ RowPlace find_row(const RowArgs& a, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = a.c.seqs;  // the answer lies in [lo, lo + span)
  while (span > 32) {
    const int step = (span + 31) >> 5;
    const unsigned m = __ballot_sync(0xffffffffu, lane * step < span && ld(a.cu + lo + lane * step) <= row);
    const int l = m ? 31 - __clz(m) : 0;
    const int nlo = lo + l * step;
    span = min(step, lo + span - nlo);
    lo = nlo;
  }
  int begin = 0x7fffffff, end = 0, len = 0, refused = 0;
  if (lane < span) {
    begin = ld(a.cu + lo + lane);
    end = ld(a.cu + lo + lane + 1);
    len = ld(a.c.lens + lo + lane);
    refused = ld(a.c.refused + lo + lane);
  }
  const unsigned m = __ballot_sync(0xffffffffu, lane < span && begin <= row);
  const int l = m ? 31 - __clz(m) : 0;
  begin = min(max(__shfl_sync(0xffffffffu, begin, l), 0), a.rows);
  end = min(max(__shfl_sync(0xffffffffu, end, l), begin), a.rows);
  len = __shfl_sync(0xffffffffu, len, l);
  refused = __shfl_sync(0xffffffffu, refused, l);
  RowPlace p{nullptr, -1};
  if (row >= begin && row < end) {
    const int pos = len - (end - row);
    if (refused == 0) p.tile = tile_of(a.c, lo + l, pos, 0);
    p.slot = pos & (kTile - 1);
    if (refused == 0 && p.tile == nullptr && lane == 0) atomicOr(a.c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
  }
  return p;
}

// The places of the CTA's rows, a warp a row.
__device__ __forceinline__ void find_rows(const RowArgs& a, int row0, int n, RowPlace* s_place) {
  for (int i = threadIdx.x >> 5; i < n; i += kThreads / 32) {
    const RowPlace p = find_row(a, row0 + i);
    if ((threadIdx.x & 31) == 0) s_place[i] = p;
  }
  __syncthreads();
}

// Unit j of the CTA's rows: a row's are K then V, heads, pieces of 32 channels.
template <int D>
struct Unit {
  int row, head, piece;  // row: of the CTA's
  bool is_v;
  __device__ __forceinline__ Unit(const Cache& c, unsigned j) {
    const unsigned half = c.heads * (D / 32);
    row = static_cast<int>(j / (2 * half));
    unsigned i = j - row * (2 * half);
    is_v = i >= half;
    if (is_v) i -= half;
    head = static_cast<int>(i / (D / 32));
    piece = static_cast<int>(i % (D / 32));
  }
  __device__ __forceinline__ uint8_t* tile(const Cache& c, const RowPlace& p) const {
    return p.tile + static_cast<size_t>(head) * c.tiles_per_page * (18 * D);
  }
  __device__ __forceinline__ uint4* codes(uint8_t* tile, int slot) const {
    return reinterpret_cast<uint4*>(is_v ? tile + 8 * D + slot * (D / 2) + piece * 16 : tile + piece * 256 + slot * 16);
  }
  __device__ __forceinline__ uint16_t* scales(uint8_t* tile, int slot) const {
    return reinterpret_cast<uint16_t*>(tile + 16 * D + (is_v ? D : 0) + slot * (D / 16) + 2 * piece);
  }
};

__device__ __forceinline__ uint32_t e4m3_byte(float x) {
  uint16_t o;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(o) : "f"(0.f), "f"(x));
  return o & 0xffu;
}
__device__ __forceinline__ float e4m3_float(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(byte) & 0xffffu)));
}
// Eight values to a word of E2M1 codes, value i in nibble i.
__device__ __forceinline__ uint32_t e2m1x8(const float* y) {
  uint32_t o;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(o)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return o;
}

// The codes and the scale byte of 16 values.
__device__ __forceinline__ uint2 quantise(const uint32_t (&w)[8], bool fp16, float ts, uint32_t& scale, int* status) {
  // magnitudes compare as their bits
  uint32_t most = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) most = __vmaxu2(most, w[k] & 0x7fff7fffu);
  most = max(most & 0xffffu, most >> 16);
  const bool finite = most < (fp16 ? 0x7c00u : 0x7f80u);
  float x[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = unpack2(w[k], fp16);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
  float top = unpack2(most, fp16).x;
  if (!finite) {  // infinities stay the largest, a NaN is held as 0
    atomicOr(status, static_cast<int>(MOE_KV4_NONFINITE));
    top = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (x[k] != x[k]) x[k] = 0.f;
      top = fmaxf(top, fabsf(x[k]));
    }
  }
  scale = e4m3_byte(fminf(__fdiv_rn(top, 6.0f * ts), 448.0f));
  const float d = e4m3_float(scale) * ts;
  float y[16];
  const float r = __frcp_rn(d);
  // where no quotient and no product with d leaves FP32's range (a block far above 448 * 6 * ts has quotients
  // that do, and their remainders are no numbers)
  if (d >= 0x1p-60f && d <= 0x1p60f && top * r <= 0x1p60f && finite) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float y0 = x[k] * r;
      y[k] = fmaf(fmaf(-y0, d, x[k]), r, y0);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] = d > 0.f ? __fdiv_rn(x[k], d) : 0.f;
  }
  return make_uint2(e2m1x8(y), e2m1x8(y + 8));
}

struct Piece32 {
  Line v[2];  // two blocks
};

template <int D>
__global__ void __launch_bounds__(kThreads, kAppendCtas) append_kernel(RowArgs a) {
  __shared__ RowPlace s_place[kMaxRowsPerCta];
  pdl_wait();
  pdl_launch_dependents();
  const int row0 = blockIdx.x * a.rows_per_cta, n = min(a.rows_per_cta, a.rows - row0);
  const unsigned total = n * 2u * a.c.heads * (D / 32);
  auto load = [&](unsigned j, Piece32& x) {
    const Unit<D> u(a.c, j);
    const int64_t row = row0 + u.row;
    const int64_t off = u.is_v ? row * a.v_row + u.head * a.v_head : row * a.k_row + u.head * a.k_head;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(u.is_v ? a.v : a.k) + 2 * (off + u.piece * 32));
    if (a.wide) {
#pragma unroll
      for (int k = 0; k < 2; ++k) x.v[k] = load_line(reinterpret_cast<const uint8_t*>(src) + 32 * k);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(x.v)[k] = src[k];
    }
  };
  Piece32 x, next;
  unsigned j = threadIdx.x;
  if (j < total) load(j, x);
  find_rows(a, row0, n, s_place);
  for (; j < total; j += kThreads) {
    if (j + kThreads < total) load(j + kThreads, next);
    const Unit<D> u(a.c, j);
    const RowPlace p = s_place[u.row];
    if (p.tile != nullptr) {
      const float ts = u.is_v ? a.v_ts : a.k_ts;
      uint32_t s0, s1;
      const uint2 c0 = quantise(x.v[0].w, a.fp16, ts, s0, a.c.status), c1 = quantise(x.v[1].w, a.fp16, ts, s1, a.c.status);
      uint8_t* tile = u.tile(a.c, p);
      *u.codes(tile, p.slot) = make_uint4(c0.x, c0.y, c1.x, c1.y);
      *u.scales(tile, p.slot) = static_cast<uint16_t>(s0 | (s1 << 8));
    }
    x = next;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, kReadCtas) read_kernel(RowArgs a) {
  __shared__ RowPlace s_place[kMaxRowsPerCta];
  pdl_wait();
  pdl_launch_dependents();
  const int row0 = blockIdx.x * a.rows_per_cta, n = min(a.rows_per_cta, a.rows - row0);
  find_rows(a, row0, n, s_place);
  const unsigned total = n * 2u * a.c.heads * (D / 32);
#pragma unroll 2
  for (unsigned j = threadIdx.x; j < total; j += kThreads) {
    const Unit<D> u(a.c, j);
    const RowPlace p = s_place[u.row];
    char* dst = static_cast<char*>(u.is_v ? a.v_out : a.k_out);
    if (p.slot < 0 || dst == nullptr) continue;
    uint4 codes = make_uint4(0u, 0u, 0u, 0u);
    uint32_t sb = 0;
    if (p.tile != nullptr) {
      uint8_t* tile = u.tile(a.c, p);
      codes = *u.codes(tile, p.slot);
      sb = *u.scales(tile, p.slot);
    }
    const float ts = u.is_v ? a.v_ts : a.k_ts;
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
    const int64_t row = row0 + u.row;
    uint8_t* q = reinterpret_cast<uint8_t*>(dst) + 2 * ((row * a.c.heads + u.head) * D + u.piece * 32);
#pragma unroll
    for (int block = 0; block < 2; ++block) {
      const float f = e4m3_float(block == 0 ? sb & 0xffu : sb >> 8) * ts;
      Line o;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h[4];
        e2m1x8_to_f16x2x4(c[2 * block + k], h[0], h[1], h[2], h[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = unpack2(h[i], true);
          o.w[4 * k + i] = pack2(v.x * f, v.y * f, a.fp16);
        }
      }
      if (a.wide) {
        store_line(q + 32 * block, o);
      } else {
        reinterpret_cast<uint4*>(q)[2 * block] = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
        reinterpret_cast<uint4*>(q)[2 * block + 1] = make_uint4(o.w[4], o.w[5], o.w[6], o.w[7]);
      }
    }
  }
}

// As many rows a CTA as let the SMs hold all CTAs at once (one row each, for a short step): a second,
// partly filled wave would cost as much as the first.
RowArgs split(RowArgs a, int ctas) {
  a.rows_per_cta = max(1, min(kMaxRowsPerCta, (a.rows + ctas - 1) / ctas));
  return a;
}
dim3 grid_of(const RowArgs& a) { return dim3((a.rows + a.rows_per_cta - 1) / a.rows_per_cta); }

}  // namespace

cudaError_t launch_append(const RowArgs& args, int num_sms, cudaStream_t stream) {
  const RowArgs a = split(args, kAppendCtas * num_sms);
  return a.c.dim == 64    ? launch_ready<append_kernel<64>>(grid_of(a), dim3(kThreads), 0, stream, a)
         : a.c.dim == 128 ? launch_ready<append_kernel<128>>(grid_of(a), dim3(kThreads), 0, stream, a)
                          : launch_ready<append_kernel<256>>(grid_of(a), dim3(kThreads), 0, stream, a);
}
cudaError_t launch_read(const RowArgs& args, int num_sms, cudaStream_t stream) {
  const RowArgs a = split(args, kReadCtas * num_sms);
  return a.c.dim == 64    ? launch_ready<read_kernel<64>>(grid_of(a), dim3(kThreads), 0, stream, a)
         : a.c.dim == 128 ? launch_ready<read_kernel<128>>(grid_of(a), dim3(kThreads), 0, stream, a)
                          : launch_ready<read_kernel<256>>(grid_of(a), dim3(kThreads), 0, stream, a);
}

}  // namespace kv4
}  // namespace moe
