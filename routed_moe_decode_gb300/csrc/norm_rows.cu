// Root-mean-square norm with the residual's addition, and rows in 8 bits with a scale for each 128 channels.
//
//   h = round(x + r);  n = h / sqrt(mean(h^2) + eps) * (w or 1 + w)
//   s = max|v| / 448 over a block of 128 values v (n, x, or silu(gate) * up);  code = E4M3(v / s)
//
// Both kernels read every input and write every output once; memory bounds them from some hundred rows on, and below that
// the launch and one trip to memory (4 rows of 2048 channels: 2 us).  A thread has 8 consecutive values (16 bytes of
// a 16-bit type), so 16 neighbouring lanes have a block, whose maximum takes four shuffles.
//
// Measured: 8192 rows of 2048 BF16 channels with a residual, normed and in 8 bits, 29 to 30 us (5.1 TB/s of what has to move); 8192
// gated rows of 4096, 36.3 us (4.7 TB/s; 38.5 where each call has an output of its own), where the exponentials, quotients and conversions take as many instruction
// slots as memory leaves.  Norm rows that a persistent grid fetches ahead, 64 channels a lane with a warp to a row (66 us), or
// other numbers of CTAs (28.9 to 29.6 us) are no faster.
#include <algorithm>
#include <cfloat>

#include "dense.cuh"

namespace moe {
namespace dense {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float2 pair(uint32_t bits, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&bits)); }
__device__ __forceinline__ float2 pair(uint32_t bits, __nv_bfloat16) {
  return make_float2(__uint_as_float(bits << 16), __uint_as_float(bits & 0xffff0000u));
}
__device__ __forceinline__ uint32_t packed(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t packed(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight consecutive values from channel c on (zeros past the row's end), 16-byte accesses where VEC.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c, int d, float (&v)[8]) {
  if constexpr (VEC && sizeof(T) == 4) {
    const float4 a = __ldcg(reinterpret_cast<const float4*>(row + c)), b = __ldcg(reinterpret_cast<const float4*>(row + c) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else if constexpr (VEC) {
    const uint4 a = __ldcg(reinterpret_cast<const uint4*>(row + c));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = pair(w[i], T());
      v[2 * i] = p.x; v[2 * i + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < d ? to_float<T>(row[c + i]) : 0.f;
  }
}
// The same, converted when they are needed.
template <typename T, bool VEC>
struct Raw8 {
  uint4 r[VEC ? sizeof(T) / 2 : 1];
  float f[VEC ? 1 : 8];
  __device__ __forceinline__ void load(const T* row, int c, int d) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
        r[i] = c < d ? __ldcs(reinterpret_cast<const uint4*>(row + c) + i) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = c + i < d ? to_float<T>(row[c + i]) : 0.f;
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 4) {
            v[4 * i + j] = __uint_as_float(w[j]);
          } else {
            const float2 p = pair(w[j], T());
            v[2 * j] = p.x;
            v[2 * j + 1] = p.y;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = f[i];
    }
  }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int c, int d, const float (&v)[8]) {
  if constexpr (VEC && sizeof(T) == 4) {
    reinterpret_cast<float4*>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else if constexpr (VEC) {
    *reinterpret_cast<uint4*>(row + c) =
        make_uint4(packed(v[0], v[1], T()), packed(v[2], v[3], T()), packed(v[4], v[5], T()), packed(v[6], v[7], T()));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < d) row[c + i] = from_float<T>(v[i]);
  }
}

// Four values as E4M3 codes, to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// Halfway between two neighbouring codes' magnitudes.
__device__ __forceinline__ float e4m3_border(uint32_t a, uint32_t b) {
  const uint32_t two = e4m3x2_to_f16x2((a & 0x7fu) | (b & 0x7fu) << 8);
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&two));
  return 0.5f * (v.x + v.y);
}

// The quotients' errors are below 2^-22 (an approximate reciprocal and two rounded products), so codes of quotients 2^-21
// smaller and larger are the same unless a border between two codes lies next to the quotient.  There the exact
// quotient decides: |v| against border * scale, by the sign of one fused multiply-add; on the border the even code.
// (Rows of 16-bit types meet borders often: v / s is then a fraction of small numbers.  A rounded division costs 87 cycles
// of a quarter of the SM's warp slots, as much as all else of eight values.)
__device__ __noinline__ uint32_t settle(uint32_t less, uint32_t more, float v0, float v1, float v2, float v3, float s) {
  uint32_t apart = less ^ more;
  while (apart) {  // one value, seldom more
    const uint32_t at = (__ffs(apart) - 1) & ~7u, a = (less >> at) & 0xffu, b = (more >> at) & 0xffu;
    const float v = at & 16 ? (at & 8 ? v3 : v2) : (at & 8 ? v1 : v0);
    const float over = fmaf(-e4m3_border(a, b), s, fabsf(v));
    const bool up = over > 0.f || (over == 0.f && (a & 1u));
    if (up) less ^= (a ^ b) << at;
    apart &= ~(0xffu << at);
  }
  return less;
}

// The largest magnitude of three; a NaN stays one.
__device__ __forceinline__ float most_of(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Codes of a thread's 8 values; 16 neighbouring lanes have a block.  All lanes of the warp take part.
// MINUS: of the values' negatives.
template <bool MINUS = false>
__device__ __forceinline__ uint2 quantize8(float (&v)[8], float* scale) {
  float most = most_of(most_of(v[0], v[1], v[2]), most_of(v[3], v[4], v[5]), most_of(v[6], v[7], v[7]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float m = __shfl_xor_sync(kAll, most, o);
    most = most_of(most, m, m);
  }
  // most / 448, rounded: a product and one correction by its residual (Markstein), exact steps above 2^-80
  float s = most * (1.f / 448.f);
  s = fmaf(fmaf(-s, 448.f, most), 1.f / 448.f, s);
  if (!(most >= 0x1p-80f && most < INFINITY)) {
    if (!(most < INFINITY)) {  // an infinity or a NaN
      *scale = __uint_as_float(0x7fc00000u);
      return make_uint2(0, 0);
    }
    s = __fdiv_rn(most, 448.f);
    *scale = s;
    if (s == 0.f) return make_uint2(0, 0);
    // the same quotients, with a reciprocal and border products inside FP32's range
    s *= 0x1p64f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= 0x1p64f;
  } else {
    *scale = s;
  }
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(MINUS ? -s : s));
  const float down = inv * (1.f - 0x1p-21f), up = inv * (1.f + 0x1p-21f);
  uint32_t less[2], more[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 a = make_float2(v[4 * h], v[4 * h + 1]), b = make_float2(v[4 * h + 2], v[4 * h + 3]);
    less[h] = e4m3x4(mul2(a, make_float2(down, down)), mul2(b, make_float2(down, down)));
    more[h] = e4m3x4(mul2(a, make_float2(up, up)), mul2(b, make_float2(up, up)));
    if (less[h] != more[h]) less[h] = settle(less[h], more[h], v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3], s);
  }
  return make_uint2(less[0], less[1]);
}

__device__ __forceinline__ void store_codes(uint8_t* row, int c, int d, uint2 codes, bool vec) {
  if (vec && c + 8 <= d) {
    *reinterpret_cast<uint2*>(row + c) = codes;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < d) row[c + i] = static_cast<uint8_t>((i < 4 ? codes.x >> (8 * i) : codes.y >> (8 * (i - 4))) & 0xffu);
}

// Sum over the TPR threads of a row; CTA-wide through red[] where TPR is over a warp.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < TPR / 32 ? red[(warp & ~(TPR / 32 - 1)) + lane] : 0.f;
#pragma unroll
    for (int o = TPR / 64; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    v = __shfl_sync(kAll, v, 0);
  }
  return v;
}

template <typename T>
struct RowPtrs {
  const T* x;
  const T* r;
  T* ro;
  T* n;
  uint8_t* codes;
  float* scales;
};
template <typename T>
__device__ __forceinline__ RowPtrs<T> row_of(const NormArgs& a, uint32_t row) {
  const uint32_t o = div(a.inner, row), i = row - o * a.inner.d;
  RowPtrs<T> p;
  p.x = static_cast<const T*>(a.x) + o * a.x_outer + i * a.x_inner;
  p.n = a.normed ? static_cast<T*>(a.normed) + o * a.n_outer + i * a.n_inner : nullptr;
  p.r = a.residual ? static_cast<const T*>(a.residual) + row * a.r_stride : nullptr;
  p.ro = a.residual_out ? static_cast<T*>(a.residual_out) + row * a.ro_stride : nullptr;
  p.codes = a.codes ? a.codes + row * a.code_stride : nullptr;
  p.scales = a.codes ? a.scales + row * a.scale_row : nullptr;
  return p;
}

template <bool VEC>
__device__ __forceinline__ void load_weight(const NormArgs& a, int c, float (&w)[8]) {
  if (a.weight_dtype == MOE_DENSE_FP32) load8<float, VEC>(static_cast<const float*>(a.weight), c, a.d, w);
  else if (a.weight_dtype == MOE_DENSE_BF16) load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(a.weight), c, a.d, w);
  else load8<__half, VEC>(static_cast<const __half*>(a.weight), c, a.d, w);
}

// h of eight channels: x + r rounded to T.
template <typename T, bool VEC>
__device__ __forceinline__ void load_h(const NormArgs& a, const RowPtrs<T>& p, int c, float (&h)[8]) {
  load8<T, VEC>(p.x, c, a.d, h);
  if (p.r) {
    float r[8];
    load8<T, VEC>(p.r, c, a.d, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = to_float<T>(from_float<T>(h[i] + r[i]));
  }
}

// The normed values of eight channels and what is written of them.  The weight comes first: h * w of 16-bit values is
// exact, so that n has one rounding after the factor's.
template <typename T, bool VEC>
__device__ __forceinline__ void finish(const NormArgs& a, const RowPtrs<T>& p, int c, bool in, float (&h)[8], float factor) {
  float w[8];
  if (in) {
    load_weight<VEC>(a, c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = h[i] * (a.add + w[i]) * factor;
    if (p.n) store8<T, VEC>(p.n, c, a.d, h);
  }
  if (p.codes) {  // the same for the whole warp
    float scale;
    const uint2 codes = quantize8(h, &scale);
    if (in) {
      store_codes(p.codes, c, a.d, codes, a.vec_codes);
      if ((threadIdx.x & 15) == 0) p.scales[(c / kBlock) * a.scale_block] = scale;
    }
  }
}

// 1 / sqrt(m): the approximate root's reciprocal (2 units) and a step of Newton's iteration.
__device__ __forceinline__ float root(float m) {
  const float f = rsqrtf(m);
  return fmaf(0.5f * f, fmaf(-m * f, f, 1.f), f);
}

// Rows whose mean square (with eps) is beyond FP32 or below its normal values, where squares lose their digits: their squares are
// added up again of h * far_scale.  Large ones (an element is 2^52 or more; scaled, at most 2^48, so 2^24 squares are finite) and
// small ones (elements at most 2^-51; the smallest, 2^-149, has a normal square, and one in 2^24 a normal mean).
__device__ __forceinline__ bool is_far(float m) { return !(m >= 0x1p-126f && m <= FLT_MAX); }
__device__ __forceinline__ float far_scale(float m) { return m < 1.f ? 0x1p100f : 0x1p-80f; }
// n = h * before * after * w * factor.  A large row's h meets the factor before the scale: its small elements stay normal, and the
// product is at most 2^92.
struct Far {
  float before, after, factor;
};
__device__ __forceinline__ Far far_row(float squares, float scale, const NormArgs& a) {
  const float m = fmaf(squares, a.inv_d, a.eps * scale * scale);
  const float f = m <= FLT_MAX || m != m ? root(m) : 0.f;  // an infinite element: finite ones become 0
  return scale < 1.f ? Far{f, scale, 1.f} : Far{scale, 1.f, f};
}

// A row's channels in the registers of TPR threads, VPT times 8 each.
template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(256, VPT == 1 ? 8 : VPT == 2 ? (sizeof(T) == 4 ? 4 : 6) : sizeof(T) == 4 ? 3 : 4) norm_kernel(const NormArgs a) {
  __shared__ float red[8];
  pdl_wait();
  const uint32_t row0 = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  const bool live = row0 < a.rows;
  const RowPtrs<T> p = row_of<T>(a, live ? row0 : a.rows - 1);
  const int t = threadIdx.x % TPR;
  Raw8<T, true> x[VPT], r[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = 8 * (t + j * TPR);
    x[j].load(p.x, c, a.d);
    if (p.r) r[j].load(p.r, c, a.d);
  }
  pdl_launch_dependents();
  float h[VPT][8];
  float squares = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    x[j].get(h[j]);
    if (p.r) {
      float v[8];
      r[j].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = to_float<T>(from_float<T>(h[j][i] + v[i]));
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(h[j][i], h[j][i], s);
    squares += s;
    const int c = 8 * (t + j * TPR);
    if (p.ro && live && c < a.d) store8<T, true>(p.ro, c, a.d, h[j]);
  }
  const float m = fmaf(row_sum<TPR>(squares, red), a.inv_d, a.eps);
  float factor = root(m);
  if (__any_sync(kAll, is_far(m))) {  // all threads of a row, and of a warp
    if constexpr (TPR > 32) __syncthreads();
    const float scale = far_scale(m);
    squares = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) squares = fmaf(h[j][i] * scale, h[j][i] * scale, squares);
    const Far far = far_row(row_sum<TPR>(squares, red), scale, a);
    if (is_far(m)) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * far.before * far.after;
      factor = far.factor;
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = 8 * (t + j * TPR);
    finish<T, true>(a, p, c, live && c < a.d, h[j], factor);
  }
}

// Any length and alignment: the row is read twice (h again from residual_out, where it is written: x or the residual may
// be the same memory; each thread reads back what it wrote itself).
template <typename T, int TPR, bool VEC>
__global__ void __launch_bounds__(256) norm_long_kernel(const NormArgs a) {
  __shared__ float red[8];
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t row0 = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  const bool live = row0 < a.rows;
  const RowPtrs<T> p = row_of<T>(a, live ? row0 : a.rows - 1);
  const int t = threadIdx.x % TPR;
  const int steps = (a.d + 8 * TPR - 1) / (8 * TPR);
  float squares = 0.f;
  for (int j = 0; j < steps; ++j) {
    const int c = 8 * (t + j * TPR);
    if (!live || c >= a.d) continue;
    float h[8], s = 0.f;
    load_h<T, VEC>(a, p, c, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(h[i], h[i], s);
    squares += s;
    if (p.ro) store8<T, VEC>(p.ro, c, a.d, h);
  }
  auto again = [&](int c, float (&h)[8]) {
    if (p.ro) load8<T, VEC>(p.ro, c, a.d, h);
    else load_h<T, VEC>(a, p, c, h);
  };
  const float m = fmaf(row_sum<TPR>(squares, red), a.inv_d, a.eps);
  Far far = {1.f, 1.f, root(m)};
  if (__any_sync(kAll, is_far(m))) {  // all threads of a row, and of a warp
    if constexpr (TPR > 32) __syncthreads();
    const float scale = far_scale(m);
    squares = 0.f;
    for (int j = 0; j < steps; ++j) {
      const int c = 8 * (t + j * TPR);
      if (!live || c >= a.d) continue;
      float h[8];
      again(c, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) squares = fmaf(h[i] * scale, h[i] * scale, squares);
    }
    const Far f = far_row(row_sum<TPR>(squares, red), scale, a);
    if (is_far(m)) far = f;
  }
  const float factor = far.factor;
  for (int j = 0; j < steps; ++j) {
    const int c = 8 * (t + j * TPR);
    const bool in = live && c < a.d;
    float h[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
      again(c, h);
      if (is_far(m)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = h[i] * far.before * far.after;
      }
    }
    finish<T, VEC>(a, p, c, in, h, factor);
  }
}

template <typename T, int TPR, int VPT>
cudaError_t run_norm(const NormArgs& a, cudaStream_t stream) {
  const uint32_t per = 256 / TPR;
  return launch_ready<norm_kernel<T, TPR, VPT>>(dim3((a.rows + per - 1) / per), dim3(256), 0, stream, a);
}
template <typename T, int TPR, bool VEC>
cudaError_t run_norm_long(const NormArgs& a, cudaStream_t stream) {
  const uint32_t per = 256 / TPR;
  return launch_ready<norm_long_kernel<T, TPR, VEC>>(dim3((a.rows + per - 1) / per), dim3(256), 0, stream, a);
}

template <typename T>
cudaError_t norm_of(const NormArgs& a, cudaStream_t stream) {
  // Threads of a row: 256 from 1025 channels on, below a warp.  Measured with a residual, normed and in 8 bits: 8192 rows of 2048
  // 28.6 us (with 128 threads to a row 30.5, 64: 31.8), 4 rows 1.9 (2.9, 4.1).  Rows of more channels: 2 or 4 times 8 a thread,
  // 6 and 4 CTAs an SM: 4096 of 4096 29.3 us (4 CTAs 30.8), 2048 of 8192 31.2 (3 CTAs 33.5).
  if (!a.vec) return a.d <= 1024 ? run_norm_long<T, 32, false>(a, stream) : run_norm_long<T, 256, false>(a, stream);
  if (a.d <= 128) return run_norm<T, 16, 1>(a, stream);
  if (a.d <= 256) return run_norm<T, 32, 1>(a, stream);
  if (a.d <= 512) return run_norm<T, 32, 2>(a, stream);
  if (a.d <= 1024) return run_norm<T, 32, 4>(a, stream);
  if (a.d <= 2048) return run_norm<T, 256, 1>(a, stream);
  if (a.d <= 4096) return run_norm<T, 256, 2>(a, stream);
  if (a.d <= 8192) return run_norm<T, 256, 4>(a, stream);
  return run_norm_long<T, 256, true>(a, stream);
}

// -g / (1 + exp(-g)) * u (its sign is turned when it is quantised), with e = exp(-|g|) (0 below 2^-126) so that nothing
// overflows: the larger of g and g e, over 1 + e.  The exponential's argument is a product and its rounding error (Dekker's
// exact product, by a fused multiply-add), the quotient a product corrected once by its residual (Markstein): errors
// of a unit or two, as with expf and a rounded division, which took a gated chunk 47 us.
__device__ __forceinline__ float2 gated_pair(float2 g, float2 u) {
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925962991e-08f, kLn2 = 0.693147180559945f;  // log2(e) = kHi + kLo
  const float2 one = make_float2(1.f, 1.f);
  const float2 a = make_float2(fmaxf(-fabsf(g.x), -200.f), fmaxf(-fabsf(g.y), -200.f));  // below: 0 all the same
  const float2 minus_t = mul2(a, make_float2(-kHi, -kHi));
  const float2 low = fma2(a, make_float2(kLo, kLo), fma2(a, make_float2(kHi, kHi), minus_t));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(-minus_t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(-minus_t.y));
  e = fma2(e, mul2(low, make_float2(kLn2, kLn2)), e);
  const float2 den = add2(one, e), less = mul2(g, e);
  const float2 num = make_float2(fmaxf(g.x, less.x), fmaxf(g.y, less.y));
  float both;  // one reciprocal for two: both denominators are within [1, 2]
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(both) : "f"(-(den.x * den.y)));
  const float2 r = mul2(make_float2(both, both), make_float2(den.y, den.x));  // -1 / den
  const float2 q = mul2(num, r);
  return mul2(fma2(fma2(q, den, num), r, q), u);
}

// A group of 16 lanes has one block of the rows, every a.rows_step-th of them; the next row's loads are under way meanwhile.
// CTAs of an SM.  6 leave too few registers and 4 too few loads under way: 8192 gated rows of 4096 take 36.7 us (39.9 with 6,
// 36.3 with 4), without a gate 23.4 (25.3, 23.4), twice as long 45.1 (46.2, 48.5).
constexpr int kQuantCtas = 5;

template <typename T, bool GATED, bool VEC>
__global__ void __launch_bounds__(256, kQuantCtas) quantize_kernel(const QuantArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 15;
  const uint32_t group = blockIdx.x * 16 + threadIdx.x / 16, row0 = div(a.nblocks, group), b = group - row0 * a.nblocks.d;
  const bool mine = row0 < a.rows_step;  // the last groups may have no row
  uint32_t left = mine && row0 < a.rows ? (a.rows - row0 + a.rows_step - 1) / a.rows_step : 0;
  // a warp's two groups go on together: they share the shuffles
  uint32_t turns = max(left, __shfl_xor_sync(kAll, left, 16));
  const int c = static_cast<int>(b) * kBlock + 8 * lane;
  const T* x = static_cast<const T*>(a.x) + row0 * a.x_stride;
  uint8_t* codes = a.codes + row0 * a.code_stride;
  float* scales = a.scales + row0 * a.scale_row + b * a.scale_block;
  const int64_t x_step = a.rows_step * a.x_stride, code_step = a.rows_step * a.code_stride, scale_step = a.rows_step * a.scale_row;
  Raw8<T, VEC> next, next_up;
  auto load = [&] {
    const int d = left ? a.d : 0;
    next.load(x, c, d);
    if constexpr (GATED) next_up.load(x + a.d, c, d);
    x += x_step;
  };
  load();
  for (; turns; --turns) {
    float v[8];
    next.get(v);
    const bool live = left != 0;
    if (live) --left;
    if constexpr (GATED) {
      float u[8];
      next_up.get(u);
      load();
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 p = gated_pair(make_float2(v[i], v[i + 1]), make_float2(u[i], u[i + 1]));
        v[i] = p.x;
        v[i + 1] = p.y;
      }
    } else {
      load();
    }
    float scale;
    const uint2 eight = quantize8<GATED>(v, &scale);
    if (live) {
      if (c < a.d) store_codes(codes, c, a.d, eight, a.vec_codes);
      if (lane == 0) *scales = scale;
      codes += code_step;
      scales += scale_step;
    }
  }
}

template <typename T>
cudaError_t quantize_of(QuantArgs a, int sms, cudaStream_t stream) {
  // a multiple of a row's blocks, as far as there are rows for them
  const uint32_t nb = a.nblocks.d, groups = std::max(nb, static_cast<uint32_t>(sms) * kQuantCtas * 16);
  a.rows_step = std::min(groups / nb, a.rows);
  const dim3 grid((a.rows_step * nb + 15) / 16), block(256);
  if (a.gated)
    return a.vec ? launch_ready<quantize_kernel<T, true, true>>(grid, block, 0, stream, a)
                 : launch_ready<quantize_kernel<T, true, false>>(grid, block, 0, stream, a);
  return a.vec ? launch_ready<quantize_kernel<T, false, true>>(grid, block, 0, stream, a)
               : launch_ready<quantize_kernel<T, false, false>>(grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t stream) {
  if (a.dtype == MOE_DENSE_FP32) return norm_of<float>(a, stream);
  if (a.dtype == MOE_DENSE_BF16) return norm_of<__nv_bfloat16>(a, stream);
  return norm_of<__half>(a, stream);
}

cudaError_t launch_quantize(const QuantArgs& a, int sms, cudaStream_t stream) {
  if (a.dtype == MOE_DENSE_FP32) return quantize_of<float>(a, sms, stream);
  if (a.dtype == MOE_DENSE_BF16) return quantize_of<__nv_bfloat16>(a, sms, stream);
  return quantize_of<__half>(a, sms, stream);
}

}  // namespace dense
}  // namespace moe
