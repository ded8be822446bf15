// A step's K and V rows into the pages of the 4-bit cache (append), and the values that the
// pages hold back out of them (read).
//
// One thread owns one block of 16 channels of one row and head: 32 bytes of BF16 or FP16 on one
// side, 8 bytes of codes and one scale byte on the other, so no thread needs another's data
// (the largest magnitude of a block is found in registers) and consecutive threads touch
// consecutive bytes of the row.  Both kernels are bound by those bytes: 2 * 2 D H + 2 * 0.5625 D H
// per row.  A warp's units are of one row, so that the row's sequence is found once per warp.
//
// Scale and codes are formed with IEEE divisions, in the order of the definition: inputs have
// 8 or 11 significant bits and scales 4, so ties are frequent and a multiplication by a rounded
// reciprocal would move some of them to the wrong neighbour.
#include "kv4_common.cuh"

namespace moe {
namespace kv4 {

namespace {

constexpr int kThreads = 256;

// seq_of_row by a warp: 32 probes a step.
__device__ __forceinline__ int warp_seq_of_row(const int* cu, int seqs, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = seqs;  // the answer lies in [lo, lo + span)
  while (span > 1) {
    const int step = (span + 31) >> 5;
    const int at = lo + lane * step;
    const bool le = lane * step < span && ld(cu + at) <= r;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int l = m ? 31 - __clz(m) : 0;
    const int nlo = lo + l * step;
    span = min(step, lo + span - nlo);
    lo = nlo;
  }
  return lo;
}

// Units of a row: K then V, heads, blocks of 16 channels.  Sets the unit's row, whether it is V,
// its head and block; false past the end.
struct Unit {
  int row, head, block;
  bool is_v, ok;
  uint8_t* tile;
  int slot;
};
__device__ __forceinline__ Unit unit_of(const RowArgs& a) {
  const int nb = a.c.dim / 16, per_row = 2 * a.c.heads * nb;
  const int warps_per_row = (per_row + 31) / 32;
  const long long w = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  Unit u{};
  const long long row = w / warps_per_row;
  if (row >= a.rows) return u;  // the whole warp
  u.row = static_cast<int>(row);
  const int s = warp_seq_of_row(a.cu, a.c.seqs, u.row);
  const StepRows st = step_rows(a.cu, s, a.rows);
  const int i = static_cast<int>(w - row * warps_per_row) * 32 + (threadIdx.x & 31);
  if (i >= per_row || u.row < st.first || u.row >= st.first + st.n) return u;  // a row of no sequence
  const int kv = i / (per_row / 2), rest = i - kv * (per_row / 2);
  u.is_v = kv != 0;
  u.head = rest / nb;
  u.block = rest - u.head * nb;
  const int pos = ld(a.c.lens + s) - st.n + (u.row - st.first);
  u.tile = tile_of(a.c, s, pos, u.head);
  u.slot = pos & (kTile - 1);
  u.ok = true;
  return u;
}

__device__ __forceinline__ uint8_t* codes_at(const Unit& u, int dim) {
  return u.is_v ? u.tile + 8 * dim + u.slot * (dim / 2) + u.block * 8
                : u.tile + (u.block >> 1) * 256 + u.slot * 16 + (u.block & 1) * 8;
}
__device__ __forceinline__ uint8_t* scale_at(const Unit& u, int dim) {
  return u.tile + 16 * dim + (u.is_v ? dim : 0) + u.slot * (dim / 16) + u.block;
}

__device__ __forceinline__ uint32_t e4m3_byte(float x) {
  uint16_t o;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(o) : "f"(0.f), "f"(x));
  return o & 0xffu;
}
// Eight values to a word of E2M1 codes, value i in nibble i.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8]) {
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

__global__ void __launch_bounds__(kThreads) append_kernel(RowArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const Unit u = unit_of(a);
  if (!u.ok) return;
  if (u.tile == nullptr) {
    atomicOr(a.c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
    return;
  }
  const char* src = static_cast<const char*>(u.is_v ? a.v : a.k);
  const int64_t off = u.is_v ? u.row * a.v_row + u.head * a.v_head : u.row * a.k_row + u.head * a.k_head;
  const uint4* p = reinterpret_cast<const uint4*>(src + 2 * (off + u.block * 16));
  const uint4 lo = p[0], hi = p[1];
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack2(w[i], a.fp16);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  float top = 0.f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float m = fabsf(x[i]);
    odd |= !(m <= 3.402823466e38f);
    if (m != m) x[i] = 0.f;  // a NaN is held as 0
    top = fmaxf(top, fabsf(x[i]));
  }
  if (odd) atomicOr(a.c.status, static_cast<int>(MOE_KV4_NONFINITE));
  const float ts = u.is_v ? a.v_ts : a.k_ts;
  const uint32_t sb = e4m3_byte(fminf(__fdiv_rn(top, 6.0f * ts), 448.0f));
  const float d = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(sb) & 0xffffu))) * ts;
  float y[8];
  uint2 codes;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = d > 0.f ? __fdiv_rn(x[i], d) : 0.f;
  codes.x = e2m1x8(y);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = d > 0.f ? __fdiv_rn(x[8 + i], d) : 0.f;
  codes.y = e2m1x8(y);
  *reinterpret_cast<uint2*>(codes_at(u, a.c.dim)) = codes;
  *scale_at(u, a.c.dim) = static_cast<uint8_t>(sb);
}

__global__ void __launch_bounds__(kThreads) read_kernel(RowArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const Unit u = unit_of(a);
  if (!u.ok) return;
  char* dst = static_cast<char*>(u.is_v ? a.v_out : a.k_out);
  if (dst == nullptr) return;
  uint2 codes = make_uint2(0u, 0u);
  uint32_t sb = 0;
  if (u.tile == nullptr) {
    atomicOr(a.c.status, static_cast<int>(MOE_KV4_BAD_PAGE));
  } else {
    codes = *reinterpret_cast<const uint2*>(codes_at(u, a.c.dim));
    sb = *scale_at(u, a.c.dim);
  }
  const float f = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(sb) & 0xffffu))) *
                  (u.is_v ? a.v_ts : a.k_ts);
  uint32_t h[8], o[8];
  e2m1x8_to_f16x2x4(codes.x, h[0], h[1], h[2], h[3]);
  e2m1x8_to_f16x2x4(codes.y, h[4], h[5], h[6], h[7]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = unpack2(h[i], true);
    o[i] = pack2(v.x * f, v.y * f, a.fp16);
  }
  uint4* p = reinterpret_cast<uint4*>(
      dst + 2 * ((static_cast<int64_t>(u.row) * a.c.heads + u.head) * a.c.dim + u.block * 16));
  __stcs(p, make_uint4(o[0], o[1], o[2], o[3]));
  __stcs(p + 1, make_uint4(o[4], o[5], o[6], o[7]));
}

unsigned grid_of(const RowArgs& a) {
  const long long per_row = 2ll * a.c.heads * (a.c.dim / 16), warps = (per_row + 31) / 32 * a.rows;
  return static_cast<unsigned>((warps * 32 + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_append(const RowArgs& a, cudaStream_t stream) {
  return launch_pdl(append_kernel, dim3(grid_of(a)), dim3(kThreads), 0, stream, a);
}
cudaError_t launch_read(const RowArgs& a, cudaStream_t stream) {
  return launch_pdl(read_kernel, dim3(grid_of(a)), dim3(kThreads), 0, stream, a);
}

}  // namespace kv4
}  // namespace moe
