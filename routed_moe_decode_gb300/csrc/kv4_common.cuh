// Shared definitions of the 4-bit K/V cache kernels: the page format, the workspace and the
// lookup of a step's rows.
#pragma once

#include "../../include/moe_kv4.h"
#include "launch.cuh"

namespace moe {
namespace kv4 {

constexpr int kTile = 16;       // tokens of a tile
constexpr int kMaxChunks = 2560;              // warps of an attention launch at most, each with one chunk of the work
// floats of the partial results, two per chunk (43 MB): 163 CTAs of the wide kernel at head size 256, more of any other
constexpr size_t kPartFloats = 2 * 1280 * 4224;
constexpr int kStepRows = 64;   // rows of a sequence's step with a tree or in a compaction

// A cache as the kernels see it.
struct Cache {
  uint8_t* pool;  // of the layer (append, read, attend) or of layer 0 (pages)
  int* table;
  int* lens;
  int* refs;
  int* refused;  // [seqs] 1: the sequence's last reservation was refused
  int* status;
  int layers, pages, heads, dim, page_size, seqs, max_pages;
  int tile_bytes;       // 18 * dim
  int tiles_per_page;   // page_size / 16
  size_t page_bytes;    // heads * tiles_per_page * tile_bytes
};

constexpr uint32_t kWaitCycles = 1u << 31;  // ~1 s: a copy takes microseconds

// An item of the attention's work that its first chunk does not end (on: there is one).
struct alignas(16) Piece {
  int on, last;  // the item's last chunk
  int row0, r0, nrows, h;
};  // 32 bytes, read as two of 16

struct WsLayout {
  size_t status, arrivals, refused, pieces, copies, need, part, total;
};

inline WsLayout ws_layout(const moe_kv4_cache& c) {
  WsLayout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  L.status = take(64);
  L.arrivals = take(size_t(c.seqs) * 4);  // moe_kv4_compact: CTAs of each sequence
  L.refused = take(size_t(c.seqs) * 4);
  L.pieces = take(size_t(kMaxChunks) * sizeof(Piece));
  // moe_kv4_reserve: copies [1 + 2 * seqs] (their number, then page pairs), need [seqs + 1]
  L.copies = take((1 + 2 * size_t(c.seqs)) * 4);
  L.need = take((1 + size_t(c.seqs)) * 8);
  L.part = take(kPartFloats * 4);
  L.total = o;
  return L;
}

// A load of what an earlier kernel wrote (lengths, tables, counts): volatile, so that it stays
// behind the wait for that kernel.
template <typename T>
MOE_DEVICE T ld(const T* p) {
  return *reinterpret_cast<const volatile T*>(p);
}

// Rows [first, first + n) of the step and sequence s, cut to the `rows` that exist.
struct StepRows {
  int first, n;
};
MOE_DEVICE StepRows step_rows(const int* __restrict__ cu, int s, int rows) {
  const int a = min(max(ld(cu + s), 0), rows);
  const int b = min(max(ld(cu + s + 1), a), rows);
  return {a, b - a};
}

// The tokens of sequence s for the calls of a step: none where its reservation was refused, since the step's rows
// then have no place and its last tokens are older ones.
MOE_DEVICE int step_len(const Cache& c, int s) {
  const int len = ld(c.lens + s), refused = ld(c.refused + s);
  return refused != 0 ? 0 : len;
}

// The tile that holds token `pos` of sequence s and head h, or nullptr where it has no page.
MOE_DEVICE uint8_t* tile_of(const Cache& c, int s, int pos, int h) {
  if (pos < 0) return nullptr;
  const int pi = pos / c.page_size;
  if (pi >= c.max_pages) return nullptr;
  const int page = ld(c.table + static_cast<size_t>(s) * c.max_pages + pi);
  if (page < 0 || page >= c.pages) return nullptr;
  return c.pool + static_cast<size_t>(page) * c.page_bytes +
         (static_cast<size_t>(h) * c.tiles_per_page + (pos - pi * c.page_size) / kTile) * c.tile_bytes;
}

// Two BF16 or FP16 values of one word as floats.
MOE_DEVICE float2 unpack2(uint32_t w, bool fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
MOE_DEVICE uint32_t pack2(float a, float b, bool fp16) {
  uint32_t o;
  if (fp16) {
    const __half2 h = __floats2half2_rn(a, b);
    o = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    o = *reinterpret_cast<const uint32_t*>(&h);
  }
  return o;
}

// 32 bytes in one access (a whole sector).
struct alignas(32) Line {
  uint32_t w[8];
};
MOE_DEVICE Line load_line(const uint8_t* p) {
  Line l;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(l.w[0]), "=r"(l.w[1]), "=r"(l.w[2]), "=r"(l.w[3]), "=r"(l.w[4]), "=r"(l.w[5]), "=r"(l.w[6]), "=r"(l.w[7])
               : "l"(p));
  return l;
}
MOE_DEVICE void store_line(uint8_t* p, const Line& l) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(l.w[0]), "r"(l.w[1]), "r"(l.w[2]),
               "r"(l.w[3]), "r"(l.w[4]), "r"(l.w[5]), "r"(l.w[6]), "r"(l.w[7])
               : "memory");
}

struct RowArgs {
  Cache c;
  const void* k;
  const void* v;
  int64_t k_row, k_head, v_row, v_head;  // strides in elements
  void* k_out;
  void* v_out;
  const int* cu;
  int rows;
  int rows_per_cta;  // set by the launcher
  bool fp16;
  bool wide;  // the rows' 32-byte pieces are aligned to 32 bytes
  float k_ts, v_ts;
};

struct AttendArgs {
  Cache c;
  const void* q;
  int64_t q_row, q_head;
  int group;   // query heads per K/V head
  const int* cu;
  int rows;
  bool fp16;
  float scale2;  // scale * k tensor scale * log2(e)
  float v_ts;
  int window;
  const unsigned long long* tree;
  void* out;
  float* lse;
  uint32_t page_magic;  // set by the launcher, as is
  int chunks;           // the number of chunks
  float* part;
  Piece* pieces;
  uint32_t wait_cycles;  // limit of every wait
  int copy_arrivals;      // arrivals that complete a stage's barrier: 1; 2, which none has, in the self-test
};

struct PageArgs {
  Cache c;
  const int* a;  // new_tokens / to_tokens / src
  const int* b;  // dst
  const uint8_t* keep;
  const int* cu;
  int n, rows;
  uint32_t* arrivals;
  int* copies;
  unsigned long long* need;
};

cudaError_t launch_append(const RowArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_read(const RowArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_attend(const AttendArgs& a, int row_tile, int num_sms, cudaStream_t stream);
cudaError_t launch_attend_wide(const AttendArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_reserve(const PageArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_fork(const PageArgs& a, cudaStream_t stream);
cudaError_t launch_trim(const PageArgs& a, cudaStream_t stream);
cudaError_t launch_compact(const PageArgs& a, cudaStream_t stream);

}  // namespace kv4
}  // namespace moe
