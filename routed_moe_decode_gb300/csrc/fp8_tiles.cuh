// What the kernels of the block-scaled products share: groups of rows, tiles, outputs.
#pragma once

#include "dense.cuh"

namespace moe {
namespace dense {

// Rows, first rows and row tiles of the groups, in shared memory.
struct Groups {
  int first[kMaxGroups], rows[kMaxGroups], before[kMaxGroups + 1];
};

// Behind offsets that decrease a group begins where those before it have ended, so that every row has one writer and there are no
// more row tiles than the host has allowed for.  (A function of its own: in place it cost calls without groups 0.2 us.)
static __device__ __noinline__ void part_groups(Groups& gs, int groups) {
  int end = 0;
#pragma unroll 1
  for (int g = 0; g < groups; ++g) {
    const int b = gs.first[g], e = b + gs.rows[g], from = max(b, end);
    gs.first[g] = from;
    gs.rows[g] = max(e - from, 0);
    end = max(end, gs.rows[g] > 0 ? e : 0);
  }
}

// By all WARPS warps of the CTA; tiles of ROWS rows.  scan: WARPS ints.
template <int WARPS, int ROWS>
__device__ __forceinline__ void make_groups(const MatmulArgs& a, Groups& gs, int* scan) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.groups + 32 * WARPS - 1) / (32 * WARPS);
  const int g0 = min(tid * per, a.groups), g1 = min(g0 + per, a.groups);
  int mine = 0;
  bool back = false;
  for (int g = g0; g < g1; ++g) {
    int b = 0, e = a.rows;
    if (a.offsets) {
      const int rb = __ldcg(a.offsets + g), re = __ldcg(a.offsets + g + 1);
      b = min(max(rb, 0), a.rows);
      e = min(max(re, 0), a.rows);
      if (blockIdx.x == 0 && (b != rb || e != re || re < rb)) atomicOr(a.status, MOE_DENSE_BAD_OFFSETS);
      back |= re < rb;
    }
    gs.first[g] = b;
    gs.rows[g] = max(e - b, 0);
    mine += (gs.rows[g] + ROWS - 1) / ROWS;
  }
  if (a.offsets && __syncthreads_or(back)) {
    if (tid == 0) part_groups(gs, a.groups);
    __syncthreads();
    mine = 0;
    for (int g = g0; g < g1; ++g) mine += (gs.rows[g] + ROWS - 1) / ROWS;
  }
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) scan[warp] = sum;
  __syncthreads();
  int at = sum - mine;
  for (int i = 0; i < warp; ++i) at += scan[i];
  for (int g = g0; g < g1; ++g) {
    gs.before[g] = at;
    at += (gs.rows[g] + ROWS - 1) / ROWS;
  }
  if (tid == 32 * WARPS - 1) gs.before[a.groups] = at;
}

struct Tile {
  int64_t w_row;    // row of the weights' matrix at which it begins
  const float* ws;  // scales of its first 128 channels [blocks of k], those of the next 128 kblocks further
  int c0, row0, rows;
};

// Tile `id` of ctiles channel tiles (of CH channels) times the groups' row tiles; a channel tile's row tiles follow each other.
// EVEN: a group's tiles have about as many rows each, in steps of 16.
template <int ROWS, int CH, bool EVEN>
__device__ __forceinline__ Tile tile_of(const MatmulArgs& a, int id, int ctiles, int kblocks, const Groups& gs) {
  // the last group with before[g] <= id / ctiles: that one's tiles end behind it, so it has rows
  int g = 0;
  if (a.groups > 1) {
    const int at = id / ctiles;
    for (int left = a.groups; left > 1;) {  // groups from g on that are left
      const int step = left >> 1;
      if (gs.before[g + step] <= at) { g += step; left -= step; }
      else left = step;
    }
  }
  const int local = id - gs.before[g] * ctiles, tts = gs.before[g + 1] - gs.before[g];
  const int ct = local / tts, tt = local - ct * tts;
  const int per = EVEN ? ((gs.rows[g] + tts - 1) / tts + 15) & ~15 : ROWS;
  Tile t;
  t.c0 = ct * CH;
  t.w_row = static_cast<int64_t>(g) * a.n + t.c0;
  t.ws = a.ws + (static_cast<int64_t>(g) * ((a.n + 127) / 128) + ct * (CH / 128)) * kblocks;
  t.row0 = gs.first[g] + tt * per;
  t.rows = min(per, gs.rows[g] - tt * per);
  return t;
}

// Four bytes, or zeros, asynchronously into shared memory.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

template <typename T>
__device__ __forceinline__ uint32_t two(float lo, float hi) {  // of a 16-bit type
  if constexpr (sizeof(T) == 2) {
    const T v[2] = {rounded<T>(lo), rounded<T>(hi)};
    return *reinterpret_cast<const uint32_t*>(v);
  } else {
    return 0;
  }
}

}  // namespace dense
}  // namespace moe
