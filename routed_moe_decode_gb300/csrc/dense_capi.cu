// Host entry points of the dense path in 8 bits (include/moe_dense.h).
#include <cmath>
#include <cstdio>
#include <mutex>

#include "../../include/moe_selftest.h"
#include "dense.cuh"

namespace moe {
namespace dense {

int encode_rows_map(CUtensorMap* map, const void* base, int size, uint64_t cols, uint64_t rows, uint64_t stride,
                    uint32_t box_cols, uint32_t box_rows) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Encode encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<Encode>(p);
  });
  if (!encode) {
    set_last_error_message("no cuTensorMapEncodeTiled");
    return MOE_ERR_CUDA;
  }
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride};
  const cuuint32_t box[2] = {box_cols, box_rows}, steps[2] = {1, 1};
  const CUresult r = encode(map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : size == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    char text[64];
    snprintf(text, sizeof text, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    set_last_error_message(text);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace dense
}  // namespace moe

namespace {

using moe::dense::MatmulArgs;

__global__ void take_status(uint32_t* status, uint32_t* bits) { *bits = atomicExch(status, 0u); }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int d) { return d == MOE_DENSE_FP32 || d == MOE_DENSE_BF16 || d == MOE_DENSE_FP16; }
int size_of(int dtype) { return dtype == MOE_DENSE_FP32 ? 4 : 2; }
int64_t blocks(int64_t n) { return (n + 127) / 128; }

int done(const char* where, cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  moe::set_last_cuda_error(where, e);
  return MOE_ERR_CUDA;
}

// Rows of `size`-byte elements that can be accessed 16 bytes at a time.
bool rows_vec(const void* p, int64_t s0, int64_t s1, int size) {
  const int64_t per = 16 / size;
  return !p || (aligned(p, 16) && s0 % per == 0 && s1 % per == 0);
}

// Whether outer x inner pieces of `size` elements, so far apart, lie apart.
bool apart(int64_t outer, int64_t outer_stride, int64_t inner, int64_t inner_stride, int64_t size) {
  if (outer <= 1) return inner <= 1 || inner_stride >= size;
  if (inner <= 1) return outer_stride >= size;
  if (outer_stride < size || inner_stride < size) return false;
  return outer_stride >= inner_stride ? (outer_stride - size) / (inner - 1) >= inner_stride
                                      : (inner_stride - size) / (outer - 1) >= outer_stride;
}

// Whether CTA pairs (256 rows x 256 channels a tile) take the product, rather than the kernel with up to 128 rows x 128
// channels a tile and k in parts.  Estimates of both in us, fitted to measured products (us, pairs / the others): a block of 128 k
// takes a pair 0.375 and a CTA 0.28 + n / 800 for n rows of x.
//   rows 256: 5120 x 2048 11.0 / 11.6, 2048 x 8192 29.5 / 14.9, 8192 x 8192 30.1 / 29.2, 16384 x 4096 18.5 / 31.9
//   rows 512: 5120 x 2048 11.6 / 19.9, 2048 x 8192 29.7 / 22.8, 8192 x 8192 31.0 / 54.9
// Groups: by their rows on average, as the numbers of each are on the device.  256 weights of 1024 x 2048 (us, pairs / the others):
// 48 rows each 110.0 / 93.6, 64: 114.8 / 110.2, 96: 117.2 / 116.0, 128: 122.3 / 188.3, 256: 169.7 / 309.0.  Between 64 and 96 they are
// alike; groups are never equal in practice, and those above 128 cost the others twice.
bool wide(const MatmulArgs& a, int sms, int split) {
  if (a.offsets) return moe::dense::rows_of_a_group(a) > 64;
  if (a.rows <= moe::dense::kSomeRows) return false;
  const double kblocks = static_cast<double>(blocks(a.k));
  const int64_t row_tiles = (a.rows + 127) / 128;
  const double rows = static_cast<double>(a.rows) / row_tiles;
  const int64_t pair_turns = ((a.rows + 255) / 256 * ((a.n + 255) / 256) + sms / 2 - 1) / (sms / 2);
  const int64_t turns = (row_tiles * blocks(a.n) * split + sms - 1) / sms;
  const double pairs_us = 4.5 + pair_turns * (1.8 + kblocks * 0.375);
  const double others_us = 4.0 + (split > 1 ? 2.0 : 0.0) + turns * std::ceil(kblocks / split) * (0.28 + rows / 800);
  return pairs_us < others_us;
}

int matmul(int rows, int n, int k, int groups, const uint8_t* codes, int64_t code_stride, const float* scales,
           int64_t scale_row, int64_t scale_block, const uint8_t* w_codes, const float* w_scales, const int32_t* offsets,
           void* out, int64_t out_stride, int out_dtype, uint32_t* status, uint32_t wait_cycles, int copy_arrivals,
           moe_stream_t stream) {
  if (rows < 0 || n <= 0 || k <= 0 || groups < 0 || !dtype_ok(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (k % 16 || groups > moe::dense::kMaxGroups) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !w_codes || !w_scales || !out || !status || (groups > 0) != (offsets != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(w_codes, 16) || !aligned(scales, 4) || !aligned(w_scales, 4) ||
      !aligned(offsets, 4) || !aligned(out, size_of(out_dtype)) || !aligned(status, 4))
    return MOE_ERR_INVALID_ARG;
  if (rows > 1 && (code_stride < k || code_stride % 16 || out_stride < n)) return MOE_ERR_INVALID_ARG;  // one row has no stride
  const int64_t wrows = static_cast<int64_t>(groups ? groups : 1) * n;
  // row tiles times channel tiles, and rows of the weights, are ints
  if (wrows > 0x7fffff00ll || (blocks(rows) * 4 + groups) * blocks(n) > 0x7fffffffll || rows > 0x7fffff00) return MOE_ERR_UNSUPPORTED;
  if (rows > 1 && code_stride >= (1ll << 40)) return MOE_ERR_UNSUPPORTED;
  int sms = 0;
  const int rc = moe::device_sms(&sms);
  if (rc != MOE_OK) return rc;
  MatmulArgs a{};
  a.x = codes; a.w = w_codes; a.xs = scales; a.ws = w_scales; a.offsets = offsets; a.out = out; a.status = status;
  a.x_stride = rows > 1 ? code_stride : (k + 15) / 16 * 16; a.scale_row = scale_row; a.scale_block = scale_block; a.out_stride = out_stride;
  a.rows = rows; a.n = n; a.k = k; a.groups = groups ? groups : 1; a.out_dtype = out_dtype;
  a.wait_cycles = wait_cycles; a.copy_arrivals = copy_arrivals;
  const int split = moe::dense::fp8_stream_split(a, sms);
  return done("product launch", wide(a, sms, split) ? moe::dense::launch_fp8_wide(a, sms, stream)
                                                    : moe::dense::launch_fp8_stream(a, sms, split, stream));
}

}  // namespace

extern "C" {

int moe_rms_norm(int outer, int inner, int d, int dtype, const void* x, int64_t x_outer, int64_t x_inner,
                 const void* residual, int64_t residual_stride, const void* weight, int weight_dtype, int one_plus,
                 float eps, void* residual_out, int64_t residual_out_stride, void* normed, int64_t normed_outer,
                 int64_t normed_inner, uint8_t* codes, int64_t code_stride, float* scales, int64_t scale_row,
                 int64_t scale_block, moe_stream_t stream) {
  if (outer < 0 || inner < 0 || d <= 0 || !dtype_ok(dtype) || !dtype_ok(weight_dtype) || !(eps >= 0.f) || !std::isfinite(eps))
    return MOE_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(outer) * inner;
  if (rows == 0) return MOE_OK;
  if (rows > 0x7fffffffll || d > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (!x || !weight || (!residual_out && !normed && !codes) || (residual_out && !residual) ||
      (codes == nullptr) != (scales == nullptr))
    return MOE_ERR_INVALID_ARG;
  const int size = size_of(dtype), wsize = size_of(weight_dtype);
  if (!aligned(x, size) || !aligned(residual, size) || !aligned(residual_out, size) || !aligned(normed, size) ||
      !aligned(weight, wsize) || !aligned(scales, 4))
    return MOE_ERR_INVALID_ARG;
  if (normed && normed == residual_out) return MOE_ERR_INVALID_ARG;
  if (residual_out && !apart(rows, residual_out_stride, 1, 0, d)) return MOE_ERR_INVALID_ARG;
  if (normed && !apart(outer, normed_outer, inner, normed_inner, d)) return MOE_ERR_INVALID_ARG;
  if (codes && (!apart(rows, code_stride, 1, 0, d) || !apart(rows, scale_row, blocks(d), scale_block, 1)))
    return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = moe::device_sms(&sms);
  if (rc != MOE_OK) return rc;
  moe::dense::NormArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.residual_out = residual_out; a.normed = normed; a.codes = codes;
  a.scales = scales;
  a.x_outer = x_outer; a.x_inner = x_inner; a.n_outer = normed_outer; a.n_inner = normed_inner;
  a.r_stride = residual_stride; a.ro_stride = residual_out_stride; a.code_stride = code_stride;
  a.scale_row = scale_row; a.scale_block = scale_block;
  a.inner = moe::dense::fast_div(static_cast<uint32_t>(inner));
  a.rows = static_cast<uint32_t>(rows); a.d = d; a.dtype = dtype; a.weight_dtype = weight_dtype; a.eps = eps; a.inv_d = 1.f / static_cast<float>(d);
  a.add = one_plus ? 1.f : 0.f;
  a.vec = d % 8 == 0 && rows_vec(x, x_outer, x_inner, size) && rows_vec(residual, residual_stride, 0, size) &&
          rows_vec(residual_out, residual_out_stride, 0, size) && rows_vec(normed, normed_outer, normed_inner, size) &&
          aligned(weight, 16);
  a.vec_codes = aligned(codes, 8) && code_stride % 8 == 0;
  return done("norm launch", moe::dense::launch_norm(a, sms, stream));
}

int moe_quantize_rows(int rows, int d, int gated, int dtype, const void* x, int64_t x_stride, uint8_t* codes,
                      int64_t code_stride, float* scales, int64_t scale_row, int64_t scale_block, moe_stream_t stream) {
  if (rows < 0 || d <= 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const int64_t all = static_cast<int64_t>(rows) * blocks(d);
  if (all > 0x7fffffffll || d > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  const int size = size_of(dtype);
  if (!x || !codes || !scales || !aligned(x, size) || !aligned(scales, 4) || !apart(rows, code_stride, 1, 0, d) ||
      !apart(rows, scale_row, blocks(d), scale_block, 1))
    return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = moe::device_sms(&sms);
  if (rc != MOE_OK) return rc;
  moe::dense::QuantArgs a{};
  a.x = x; a.codes = codes; a.scales = scales; a.x_stride = x_stride; a.code_stride = code_stride;
  a.scale_row = scale_row; a.scale_block = scale_block;
  a.nblocks = moe::dense::fast_div(static_cast<uint32_t>(blocks(d)));
  a.rows = static_cast<uint32_t>(rows); a.d = d; a.dtype = dtype; a.gated = gated != 0;
  a.vec = d % 8 == 0 && rows_vec(x, x_stride, 0, size);
  a.vec_codes = aligned(codes, 8) && code_stride % 8 == 0;
  return done("quantize launch", moe::dense::launch_quantize(a, sms, stream));
}

int moe_fp8_matmul(int rows, int n, int k, int groups, const uint8_t* codes, int64_t code_stride, const float* scales,
                   int64_t scale_row, int64_t scale_block, const uint8_t* w_codes, const float* w_scales,
                   const int32_t* offsets, void* out, int64_t out_stride, int out_dtype, uint32_t* status,
                   moe_stream_t stream) {
  return matmul(rows, n, k, groups, codes, code_stride, scales, scale_row, scale_block, w_codes, w_scales, offsets, out,
                out_stride, out_dtype, status, moe::dense::kWaitCycles, 1, stream);
}

int moe_token_logprobs(int rows, int vocab, int dtype, const void* logits, int64_t row_stride, float scale,
                       const int32_t* tokens, int n_tokens, int64_t token_stride, int top, float* logprobs, float* lse,
                       float* entropy, int32_t* top_ids, float* top_logprobs, moe_stream_t stream) {
  if (rows < 0 || vocab <= 0 || !dtype_ok(dtype) || !(scale > 0.f) || !std::isfinite(scale) || n_tokens < 0 || top < 0 ||
      top > vocab)
    return MOE_ERR_INVALID_ARG;
  if (top > 32 || n_tokens > 1024 || vocab > (1 << 30) || rows > (1 << 28) || scale < 0x1p-80f || scale > 0x1p80f) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!logits || !aligned(logits, size_of(dtype)) || !aligned(tokens, 4) || !aligned(logprobs, 4) || !aligned(lse, 4) ||
      !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
    return MOE_ERR_INVALID_ARG;
  if ((logprobs && n_tokens && !tokens) || (top == 0 && (top_ids || top_logprobs))) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = moe::device_sms(&sms);
  if (rc != MOE_OK) return rc;
  moe::dense::LogprobArgs a{};
  a.logits = logits; a.tokens = tokens; a.logprobs = logprobs; a.lse = lse; a.entropy = entropy; a.top_ids = top_ids;
  a.top_logprobs = top_logprobs; a.row_stride = row_stride; a.token_stride = token_stride; a.scale = scale;
  a.exp_scale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.rows = rows; a.vocab = vocab; a.n_tokens = n_tokens; a.top = top; a.dtype = dtype;
  return done("log probabilities launch", moe::dense::launch_logprobs(a, sms, stream));
}

int moe_dense_read_status(uint32_t* status, int clear, uint32_t* status_bits, moe_stream_t stream) {
  if (!status || !aligned(status, 4) || !status_bits) return MOE_ERR_INVALID_ARG;
  // Cleared by the exchange that reads it: a product of another stream may set a bit at any time, which this read or a later one has.
  uint32_t bits = 0, *taken = nullptr;
  cudaError_t e = cudaSuccess;
  if (clear) {
    e = cudaMallocAsync(reinterpret_cast<void**>(&taken), sizeof bits, stream);
    if (e != cudaSuccess) return done("status", e);
    take_status<<<1, 1, 0, stream>>>(status, taken);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpyAsync(&bits, clear ? taken : status, sizeof bits, cudaMemcpyDeviceToHost, stream);
  if (taken) {
    const cudaError_t freed = cudaFreeAsync(taken, stream);
    if (e == cudaSuccess) e = freed;
  }
  const cudaError_t waited = cudaStreamSynchronize(stream);  // `bits` is written until then
  if (e == cudaSuccess) e = waited;
  if (e != cudaSuccess) return done("status", e);
  *status_bits = bits;
  return bits ? MOE_ERR_DEVICE : MOE_OK;
}

int moe_selftest_fp8_matmul(int rows, int n, int k, int groups, const uint8_t* codes, int64_t code_stride,
                            const float* scales, int64_t scale_row, int64_t scale_block, const uint8_t* w_codes,
                            const float* w_scales, const int32_t* offsets, void* out, int64_t out_stride, int out_dtype,
                            uint32_t* status, int stuck, long long wait_limit_cycles, moe_stream_t stream) {
  if (stuck < 0 || stuck > 1 || wait_limit_cycles < 0) return MOE_ERR_INVALID_ARG;
  // 0 would say that a wait has given up already
  const uint32_t limit = static_cast<uint32_t>(wait_limit_cycles < 1 ? 1 : wait_limit_cycles < 0xffffffffll ? wait_limit_cycles : 0xffffffffll);
  return matmul(rows, n, k, groups, codes, code_stride, scales, scale_row, scale_block, w_codes, w_scales, offsets, out,
                out_stride, out_dtype, status, limit, 1 + stuck, stream);
}

}  // extern "C"
