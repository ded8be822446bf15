// Host entry points of the 4-bit K/V cache (include/moe_kv4.h).
#include <cmath>

#include "../../include/moe_selftest.h"
#include "kv4_common.cuh"

namespace {

using moe::kv4::Cache;
using moe::kv4::WsLayout;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t page_bytes(const moe_kv4_cache& c) {
  return static_cast<size_t>(c.kv_heads) * (c.page_size / moe::kv4::kTile) * (18 * c.head_dim);
}

int check_sizes(const moe_kv4_cache* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->layers <= 0 || c->pages <= 0 || c->kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0 || c->seqs <= 0 ||
      c->max_pages <= 0)
    return MOE_ERR_INVALID_ARG;
  if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || !std::isfinite(c->k_scale) || !std::isfinite(c->v_scale))
    return MOE_ERR_INVALID_ARG;
  if (c->k_scale > 0x1p119f || c->v_scale > 0x1p119f) return MOE_ERR_UNSUPPORTED;  // 448 * scale is a float
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
  if (c->page_size % moe::kv4::kTile || c->page_size > 1024 || c->kv_heads > 1024 || c->seqs > 65535 ||
      c->pages > (1 << 30) || c->layers > 65536 || c->max_pages > (1 << 27))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Sizes, pointers and workspace of a cache; fills the kernels' view of it (pool at `layer`).
int view(const moe_kv4_cache* c, int layer, Cache* v, WsLayout* L) {
  const int rc = check_sizes(c);
  if (rc != MOE_OK) return rc;
  if (layer < 0 || layer >= c->layers) return MOE_ERR_INVALID_ARG;
  if (!c->pool || !c->table || !c->lens || !c->refs || !aligned(c->pool, 256) || !aligned(c->table, 4) ||
      !aligned(c->lens, 4) || !aligned(c->refs, 4))
    return MOE_ERR_INVALID_ARG;
  *L = moe::kv4::ws_layout(*c);
  if (!c->workspace || !aligned(c->workspace, 256) || c->workspace_bytes < L->total) return MOE_ERR_WORKSPACE;
  v->layers = c->layers; v->pages = c->pages; v->heads = c->kv_heads; v->dim = c->head_dim;
  v->page_size = c->page_size; v->seqs = c->seqs; v->max_pages = c->max_pages;
  v->tile_bytes = 18 * c->head_dim;
  v->tiles_per_page = c->page_size / moe::kv4::kTile;
  v->page_bytes = page_bytes(*c);
  v->pool = static_cast<uint8_t*>(c->pool) + static_cast<size_t>(layer) * c->pages * v->page_bytes;
  v->table = c->table; v->lens = c->lens; v->refs = c->refs;
  v->refused = reinterpret_cast<int*>(static_cast<char*>(c->workspace) + L->refused);
  v->status = reinterpret_cast<int*>(static_cast<char*>(c->workspace) + L->status);
  return MOE_OK;
}

template <typename T>
T* at(const moe_kv4_cache* c, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(c->workspace) + off);
}

int done(const char* where, cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  moe::set_last_cuda_error(where, e);
  return MOE_ERR_CUDA;
}

bool dtype_ok(int d) { return d == MOE_KV4_BF16 || d == MOE_KV4_FP16; }
// A row tensor of 2-byte elements read 16 bytes at a time.
bool rows_ok(const void* p, int64_t row_stride, int64_t head_stride) {
  return p && aligned(p, 16) && row_stride % 8 == 0 && head_stride % 8 == 0;
}

int attend(const moe_kv4_cache* c, int layer, const void* q, int64_t q_row_stride, int64_t q_head_stride, int q_heads,
           int dtype, const int32_t* cu_rows, int rows, int max_rows, float scale, int window, const uint64_t* tree,
           void* out, float* lse, uint32_t wait_cycles, int copy_arrivals, moe_stream_t stream) {
  moe::kv4::AttendArgs a{};
  WsLayout L;
  int rc = view(c, layer, &a.c, &L);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || max_rows < 0 || window < 0 || q_heads <= 0 || q_heads % c->kv_heads || !dtype_ok(dtype) ||
      !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (tree && (window > 0 || max_rows > moe::kv4::kStepRows)) return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(rows) * q_heads > 0x7fffffffll / 2) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!rows_ok(q, q_row_stride, q_head_stride) || !cu_rows || !aligned(cu_rows, 4) || !out || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(tree, 8))
    return MOE_ERR_INVALID_ARG;
  a.scale2 = scale * c->k_scale * 1.44269504088896340736f;
  if (!std::isfinite(a.scale2)) return MOE_ERR_UNSUPPORTED;
  int sms = 0;
  rc = moe::device_sms(&sms);
  if (rc != MOE_OK) return rc;
  a.q = q; a.q_row = q_row_stride; a.q_head = q_head_stride;
  a.group = q_heads / c->kv_heads;
  a.cu = cu_rows; a.rows = rows; a.fp16 = dtype == MOE_KV4_FP16;
  a.v_ts = c->v_scale;
  a.window = window < (1 << 30) ? window : 1 << 30;  // as many tokens as there can be; first - window stays an int
  a.tree = reinterpret_cast<const unsigned long long*>(tree);
  a.out = out; a.lse = lse;
  a.part = at<float>(c, L.part);
  a.pieces = at<moe::kv4::Piece>(c, L.pieces);
  a.wait_cycles = wait_cycles; a.copy_arrivals = copy_arrivals;
  const int64_t block = static_cast<int64_t>(max_rows < 1 ? 1 : max_rows) * a.group;
  return done("attend launch", moe::kv4::launch_attend(a, static_cast<int>(block > 1024 ? 1024 : block), sms, stream));
}

}  // namespace

extern "C" {

size_t moe_kv4_page_bytes(const moe_kv4_cache* c) { return check_sizes(c) == MOE_OK ? page_bytes(*c) : 0; }

size_t moe_kv4_workspace_bytes(const moe_kv4_cache* c) {
  return check_sizes(c) == MOE_OK ? moe::kv4::ws_layout(*c).total : 0;
}

int moe_kv4_check(const moe_kv4_cache* c) { return check_sizes(c); }

int moe_kv4_workspace_init(const moe_kv4_cache* c, moe_stream_t stream) {
  const int rc = check_sizes(c);
  if (rc != MOE_OK) return rc;
  const WsLayout L = moe::kv4::ws_layout(*c);
  if (!c->workspace || !aligned(c->workspace, 256) || c->workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  return done("workspace init", cudaMemsetAsync(c->workspace, 0, L.pieces, stream));  // the status word, the arrivals, the refusals
}

int moe_kv4_append(const moe_kv4_cache* c, int layer, const void* k, int64_t k_row_stride, int64_t k_head_stride,
                   const void* v, int64_t v_row_stride, int64_t v_head_stride, int dtype, const int32_t* cu_rows,
                   int rows, moe_stream_t stream) {
  moe::kv4::RowArgs a{};
  WsLayout L;
  const int rc = view(c, layer, &a.c, &L);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!rows_ok(k, k_row_stride, k_head_stride) || !rows_ok(v, v_row_stride, v_head_stride) || !cu_rows ||
      !aligned(cu_rows, 4))
    return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(rows) * c->kv_heads * c->head_dim > (1ll << 36)) return MOE_ERR_UNSUPPORTED;
  a.k = k; a.v = v; a.k_row = k_row_stride; a.k_head = k_head_stride; a.v_row = v_row_stride; a.v_head = v_head_stride;
  a.cu = cu_rows; a.rows = rows; a.fp16 = dtype == MOE_KV4_FP16; a.k_ts = c->k_scale; a.v_ts = c->v_scale;
  a.wide = aligned(k, 32) && aligned(v, 32) && (k_row_stride | k_head_stride | v_row_stride | v_head_stride) % 16 == 0;
  int sms = 0;
  const int src = moe::device_sms(&sms);
  if (src != MOE_OK) return src;
  return done("append launch", moe::kv4::launch_append(a, sms, stream));
}

int moe_kv4_read(const moe_kv4_cache* c, int layer, void* k, void* v, int dtype, const int32_t* cu_rows, int rows,
                 moe_stream_t stream) {
  moe::kv4::RowArgs a{};
  WsLayout L;
  const int rc = view(c, layer, &a.c, &L);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (rows == 0 || (!k && !v)) return MOE_OK;
  if (!aligned(k, 16) || !aligned(v, 16) || !cu_rows || !aligned(cu_rows, 4)) return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(rows) * c->kv_heads * c->head_dim > (1ll << 36)) return MOE_ERR_UNSUPPORTED;
  a.k_out = k; a.v_out = v;
  a.cu = cu_rows; a.rows = rows; a.fp16 = dtype == MOE_KV4_FP16; a.k_ts = c->k_scale; a.v_ts = c->v_scale;
  a.wide = aligned(k, 32) && aligned(v, 32);
  int sms = 0;
  const int src = moe::device_sms(&sms);
  if (src != MOE_OK) return src;
  return done("read launch", moe::kv4::launch_read(a, sms, stream));
}

int moe_kv4_attend(const moe_kv4_cache* c, int layer, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                   int q_heads, int dtype, const int32_t* cu_rows, int rows, int max_rows, float scale, int window,
                   const uint64_t* tree, void* out, float* lse, moe_stream_t stream) {
  return attend(c, layer, q, q_row_stride, q_head_stride, q_heads, dtype, cu_rows, rows, max_rows, scale, window, tree, out,
                lse, moe::kv4::kWaitCycles, 1, stream);
}

int moe_selftest_kv4_attend(const moe_kv4_cache* c, int layer, const void* q, int64_t q_row_stride,
                            int64_t q_head_stride, int q_heads, int dtype, const int32_t* cu_rows, int rows,
                            int max_rows, float scale, void* out, int stuck, long long wait_limit_cycles,
                            moe_stream_t stream) {
  if (stuck < 0 || stuck > 1 || wait_limit_cycles < 0) return MOE_ERR_INVALID_ARG;
  const uint32_t limit = static_cast<uint32_t>(wait_limit_cycles < 0xffffffffll ? wait_limit_cycles : 0xffffffffll);
  return attend(c, layer, q, q_row_stride, q_head_stride, q_heads, dtype, cu_rows, rows, max_rows, scale, 0, nullptr, out,
                nullptr, limit, 1 + stuck, stream);
}

int moe_kv4_reserve(const moe_kv4_cache* c, const int32_t* new_tokens, moe_stream_t stream) {
  moe::kv4::PageArgs a{};
  WsLayout L;
  int rc = view(c, 0, &a.c, &L);
  if (rc != MOE_OK) return rc;
  if (!new_tokens || !aligned(new_tokens, 4)) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  rc = moe::device_sms(&sms);
  if (rc != MOE_OK) return rc;
  a.a = new_tokens;
  a.copies = at<int>(c, L.copies);
  a.need = at<unsigned long long>(c, L.need);
  return done("reserve launch", moe::kv4::launch_reserve(a, sms, stream));
}

int moe_kv4_fork(const moe_kv4_cache* c, const int32_t* src, const int32_t* dst, int n, moe_stream_t stream) {
  moe::kv4::PageArgs a{};
  WsLayout L;
  const int rc = view(c, 0, &a.c, &L);
  if (rc != MOE_OK) return rc;
  if (n < 0 || n > c->seqs) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return MOE_ERR_INVALID_ARG;
  a.a = src; a.b = dst; a.n = n;
  return done("fork launch", moe::kv4::launch_fork(a, stream));
}

int moe_kv4_trim(const moe_kv4_cache* c, const int32_t* to_tokens, moe_stream_t stream) {
  moe::kv4::PageArgs a{};
  WsLayout L;
  const int rc = view(c, 0, &a.c, &L);
  if (rc != MOE_OK) return rc;
  if (!to_tokens || !aligned(to_tokens, 4)) return MOE_ERR_INVALID_ARG;
  a.a = to_tokens;
  return done("trim launch", moe::kv4::launch_trim(a, stream));
}

int moe_kv4_compact(const moe_kv4_cache* c, const uint8_t* keep, const int32_t* cu_rows, int rows, int max_rows,
                    moe_stream_t stream) {
  moe::kv4::PageArgs a{};
  WsLayout L;
  const int rc = view(c, 0, &a.c, &L);
  if (rc != MOE_OK) return rc;
  if (rows < 0 || max_rows < 0) return MOE_ERR_INVALID_ARG;
  if (max_rows > moe::kv4::kStepRows) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!keep || !cu_rows || !aligned(cu_rows, 4)) return MOE_ERR_INVALID_ARG;
  a.keep = keep; a.cu = cu_rows; a.rows = rows;
  a.arrivals = at<uint32_t>(c, L.arrivals);
  return done("compact launch", moe::kv4::launch_compact(a, stream));
}

int moe_kv4_read_status(const moe_kv4_cache* c, int clear, uint32_t* status_bits, moe_stream_t stream) {
  if (!status_bits) return MOE_ERR_INVALID_ARG;
  Cache v;
  WsLayout L;
  const int rc = view(c, 0, &v, &L);
  if (rc != MOE_OK) return rc;
  uint32_t bits = 0;
  cudaError_t e = cudaMemcpyAsync(&bits, v.status, sizeof bits, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess && clear) e = cudaMemsetAsync(v.status, 0, sizeof bits, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return done("status", e);
  *status_bits = bits;
  return bits ? MOE_ERR_DEVICE : MOE_OK;
}

}  // extern "C"
