// Block-scaled products with the weights as the 128-row operand (include/moe_dense.h): few rows, and groups of rows.
//
//   out[t][c] = sum_b xs[t][b] ws[c / 128][b] * (sum over block b of x[t][k] w[c][k])
//
// A tile is 128 channels of a weight, which is one row of its scales, times up to NT rows of x.  Each block of 128 k
// is one product of its own in tensor memory (four tcgen05 MMAs of 32 k, weights 128 x rows n); it is multiplied by its
// scales on the way into FP32 registers, so nothing is rounded between the blocks.  Weights are read once for all rows of a tile: with
// few rows the weights' bytes bound the product, with many rows the tensor cores and the sums.
//
// Roles: warps 0-7 add up (a lane of tensor memory is a channel; two groups of four warps take half of the rows
// each), a warp copies tiles into a ring, a warp issues the MMAs, two warps bring a block's scales into shared memory.
// CTAs take tiles statically, one after the other; the ring runs on across tiles.  Where one row of x tiles would leave
// SMs idle, a cluster's CTAs take a part of k each and add up through distributed shared memory, in order.
//
// Measured: 16 rows x 131072 x 2048 into FP32 47 us (5.9 TB/s of what has to move, 0.87 of the measured copy); 256 weights of
// 1024 x 2048 with 8 rows each 88 us (6.2 TB/s); 4 rows x 5120 x 2048 6.1 us, of which ~2 are the launch and the first trip to
// memory and ~1.5 the parts' join.  What bounds the long ones is memory and the start: the tensor cores are 4 % busy, the issue
// slots 26 %.  Scales come by asynchronous copies, far ahead: loaded into registers they held 256 weights at 113 us.
#include "fp8_tiles.cuh"

namespace moe {
namespace dense {
namespace {

constexpr int kSumWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kScaleWarps = 2, kScaleWarp = 10, kThreads = 32 * 12;
constexpr uint32_t kDrainCycles = 1u << 24;
constexpr int kMostParts = 8;  // of k, the CTAs of a cluster
constexpr int kSlab = 16;      // rows of x whose sums are staged for writing at a time

template <int NT>
struct Shape {
  static constexpr int kStage = (128 + NT) * 128;
  static constexpr int kStages = NT == 128 ? 6 : 9;
  static constexpr int kBufs = NT == 128 ? 4 : 8;  // products in tensor memory
  static constexpr int kCols = NT * kBufs;
  static constexpr int kSlots = NT == 128 ? 8 : 32, kSlot = NT + 4;  // blocks' scales: of the rows, the weight's
  static constexpr int kScales = kStage * kStages;                   // [kSlots][kSlot] floats
  static constexpr int kStaged = kScales + 4 * kSlots * kSlot;       // [2][kSlab][128] floats
  static constexpr int kBars = kStaged + 4 * 2 * kSlab * 128;
  static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 2 * kSlots + 1;
  static constexpr int kGroups = kBars + 8 * kNumBars;
  static constexpr int kTotal = kGroups + static_cast<int>(sizeof(Groups)) + 1024;
  static_assert(kTotal <= 227 * 1024);
};

struct Maps {
  CUtensorMap w, x16, x64;
};

__device__ __forceinline__ void store_one(const MatmulArgs& a, int64_t row, int c, float v) {
  if (a.out_dtype == MOE_DENSE_FP32) static_cast<float*>(a.out)[row * a.out_stride + c] = v;
  else if (a.out_dtype == MOE_DENSE_BF16) static_cast<__nv_bfloat16*>(a.out)[row * a.out_stride + c] = __float2bfloat16_rn(v);
  else static_cast<__half*>(a.out)[row * a.out_stride + c] = __float2half_rn(v);
}

// Four channels from c on; vec: rows can be written four at a time.
__device__ __forceinline__ void store4(const MatmulArgs& a, int64_t row, int c, float4 v, bool vec) {
  if (vec && c + 4 <= a.n) {
    const int64_t at = row * a.out_stride + c;
    if (a.out_dtype == MOE_DENSE_FP32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
    else if (a.out_dtype == MOE_DENSE_BF16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = make_uint2(two<__nv_bfloat16>(v.x, v.y), two<__nv_bfloat16>(v.z, v.w));
    else *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at) = make_uint2(two<__half>(v.x, v.y), two<__half>(v.z, v.w));
    return;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < a.n) store_one(a, row, c + i, f[i]);
}

template <int N>
__device__ __forceinline__ void load_scales(float2 (&f)[N], const float* s, float ws) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 v = *reinterpret_cast<const float4*>(s + 2 * i);
    f[i] = mul2(make_float2(v.x, v.y), make_float2(ws, ws));
    f[i + 1] = mul2(make_float2(v.z, v.w), make_float2(ws, ws));
  }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_stream_kernel(const __grid_constant__ Maps maps, const __grid_constant__ MatmulArgs a) {
  typedef Shape<NT> L;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem, s_limit;
  __shared__ int s_scan[12];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_addr(smem);
  Groups& gs = *reinterpret_cast<Groups*>(smem + L::kGroups);
  const uint32_t full = base + L::kBars, empty = full + 8 * L::kStages, done = empty + 8 * L::kStages,
                 freed = done + 8 * L::kBufs, scaled = freed + 8 * L::kBufs, used = scaled + 8 * L::kSlots, end = used + 8 * L::kSlots;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(full + 8 * i, a.copy_arrivals);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < L::kBufs; ++i) {
      mbar_init(done + 8 * i, 1);
      mbar_init(freed + 8 * i, kSumWarps);
    }
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(scaled + 8 * i, 32 * kScaleWarps);
      mbar_init(used + 8 * i, kSumWarps);
    }
    mbar_init(end, 1);
    s_limit = a.wait_cycles;
  }
  fence_barrier_init();
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&s_tmem), L::kCols);
    tmem_relinquish();
  }
  if (warp == kCopyWarp && lane == 0) {
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.x16);
    prefetch_tmap(&maps.x64);
  }
  pdl_wait();
  pdl_launch_dependents();

  make_groups<kThreads / 32, NT>(a, gs, s_scan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile uint32_t* limit = &s_limit;

  const int split = static_cast<int>(cluster_size()), part = static_cast<int>(cluster_rank());
  const int ctiles = (a.n + 127) / 128, kblocks = (a.k + 127) / 128;
  const int k0 = kblocks * part / split, k1 = kblocks * (part + 1) / split;
  const int tiles = gs.before[a.groups] * ctiles, stride = gridDim.x / split;

  if (warp == kCopyWarp) {
    uint32_t it = 0;
    bool ok = true;
    for (int id = blockIdx.x / split; ok && id < tiles; id += stride) {
      const Tile t = tile_of<NT, 128, true>(a, id, ctiles, kblocks, gs);
      const int n16 = (t.rows + 15) >> 4;
      const uint32_t bytes = 128 * 128 + n16 * 16 * 128;
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const uint32_t s = it % L::kStages;
        if (!(ok = warp_wait(empty + 8 * s, ((it / L::kStages) & 1) ^ 1, limit, a.status))) break;
        if (elect_one()) {
          const uint32_t at = base + s * L::kStage, bar = full + 8 * s;
          mbar_arrive_expect_tx(bar, bytes);
          tma_load_2d_plain(at, &maps.w, kb * 128, static_cast<int>(t.w_row), bar);
          int i = 0;
          if constexpr (NT > 32)
            for (; i + 4 <= n16; i += 4) tma_load_2d_plain(at + 16384 + i * 2048, &maps.x64, kb * 128, t.row0 + i * 16, bar);
          for (; i < n16; ++i) tma_load_2d_plain(at + 16384 + i * 2048, &maps.x16, kb * 128, t.row0 + i * 16, bar);
        }
        __syncwarp();
      }
    }
    // copies in flight land before the CTA leaves
    __shared__ uint32_t s_drain;
    if (lane == 0) s_drain = kDrainCycles;
    __syncwarp();
    for (uint32_t i = it > L::kStages ? it - L::kStages : 0; i < it; ++i)
      warp_wait(full + 8 * (i % L::kStages), (i / L::kStages) & 1, &s_drain, a.status);
  } else if (warp == kMmaWarp) {
    uint32_t it = 0;
    bool ok = true;
    for (int id = blockIdx.x / split; ok && id < tiles; id += stride) {
      const Tile t = tile_of<NT, 128, true>(a, id, ctiles, kblocks, gs);
      const uint32_t idesc = idesc_e4m3(128, max(16, (t.rows + 15) & ~15));
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const uint32_t s = it % L::kStages, b = it % L::kBufs;
        ok = warp_wait(freed + 8 * b, ((it / L::kBufs) & 1) ^ 1, limit, a.status) &&
             warp_wait(full + 8 * s, (it / L::kStages) & 1, limit, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t da = smem_desc_sw128(base + s * L::kStage, 1024);
        const uint64_t db = smem_desc_sw128(base + s * L::kStage + 16384, 1024);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_e4m3(tmem + b * NT, da + 2 * k, db + 2 * k, idesc, k > 0);
          tc_commit(empty + 8 * s);
          tc_commit(done + 8 * b);
        }
        __syncwarp();
      }
    }
    // products in flight end before their memory is given back
    if (elect_one()) tc_commit(end);
    __syncwarp();
    __shared__ uint32_t s_drain_mma;
    if (lane == 0) s_drain_mma = kDrainCycles;
    __syncwarp();
    warp_wait(end, 0, &s_drain_mma, a.status);
  } else if (warp >= kScaleWarp) {
    // scales of rows r0 and r0 + 64, and of the weight, kSlots blocks ahead, across tiles (four blocks ahead in
    // registers, 256 groups of 8 rows took 113 us instead of the 89 of this)
    const int r0 = (warp - kScaleWarp) * 32 + lane;
    const uint32_t out = base + L::kScales;
    uint32_t it = 0;
    bool ok = true;
    for (int id = blockIdx.x / split; ok && id < tiles; id += stride) {
      const Tile t = tile_of<NT, 128, true>(a, id, ctiles, kblocks, gs);
      const float* xs = a.xs + static_cast<int64_t>(t.row0 + r0) * a.scale_row;
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const uint32_t slot = it % L::kSlots, to = out + slot * (L::kSlot * 4);
        if (!(ok = warp_wait(used + 8 * slot, ((it / L::kSlots) & 1) ^ 1, limit, a.status))) break;
#pragma unroll
        for (int r = r0; r < NT; r += 64)
          copy4(to + 4 * r, r < t.rows ? xs + (r - r0) * a.scale_row + kb * a.scale_block : a.xs, r < t.rows);
        if (r0 == 0) copy4(to + 4 * NT, t.ws + kb, true);
        cp_async_arrive_noinc(scaled + 8 * slot);
      }
    }
    cp_async_wait_all();
  } else {
    constexpr int H = NT / 2;
    const int half = warp >> 2, quarter = warp & 3;
    const float* scales = reinterpret_cast<const float*>(smem + L::kScales);
    const int size = a.out_dtype == MOE_DENSE_FP32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(a.out) % (4 * size) == 0 && a.out_stride % 4 == 0;
    uint32_t it = 0;
    bool ok = true;
    for (int id = blockIdx.x / split; ok && id < tiles; id += stride) {
      const Tile t = tile_of<NT, 128, true>(a, id, ctiles, kblocks, gs);
      const int n = (t.rows + 15) & ~15, cut = ((n / 2) + 15) & ~15;  // rows [0, cut) and [cut, n)
      const int first = half ? cut : 0, mine = half ? n - cut : cut;
      float2 acc[H / 2];
#pragma unroll
      for (int i = 0; i < H / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const uint32_t b = it % L::kBufs, phase = (it / L::kBufs) & 1;
        // a step's scales are in registers before its products are there (or are read from tensor memory)
        constexpr int STEP = H < 32 ? H : 32;
        float2 f[STEP / 2];
        const uint32_t slot = it % L::kSlots;
        const float* s = scales + slot * L::kSlot + first;
        ok = warp_wait(scaled + 8 * slot, (it / L::kSlots) & 1, limit, a.status);
        const float ws = scales[slot * L::kSlot + NT];
        load_scales(f, s, ws);
        ok = ok && warp_wait(done + 8 * b, phase, limit, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = tmem + b * NT + first + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
        for (int c = 0; c < H; c += STEP) {
          if (c >= mine) break;  // (columns past `mine` in its last step are added up and not used)
          uint32_t v[STEP];
          if constexpr (STEP == 32) tmem_ld_x32(from + c, v);
          else tmem_ld_x16(from + c, v);
          if (c) load_scales(f, s + c, ws);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < STEP; i += 2)
            acc[(c + i) / 2] = fma2_in_order(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), f[i / 2],
                                             acc[(c + i) / 2]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(freed + 8 * b);
          mbar_arrive(used + 8 * slot);
        }
      }
      // the four warps of a half write together, so they go on or give up together
      ok = named_bar_and(1 + half, 128, ok);
      if (!ok) break;
      const int ch = quarter * 32 + lane;
      if (split == 1) {
        float* staged = reinterpret_cast<float*>(smem + L::kStaged) + half * kSlab * 128;
#pragma unroll
        for (int c = 0; c < H; c += kSlab) {
          if (c >= mine) break;
#pragma unroll
          for (int i = 0; i < kSlab; i += 2) {
            staged[i * 128 + ch] = acc[(c + i) / 2].x;
            staged[(i + 1) * 128 + ch] = acc[(c + i) / 2].y;
          }
          named_bar_sync(1 + half, 128);
          for (int i = ch; i < kSlab * 32; i += 128) {
            const int r = first + c + (i >> 5), at = (i & 31) * 4;
            if (r < t.rows) store4(a, t.row0 + r, t.c0 + at, *reinterpret_cast<const float4*>(staged + 4 * i), vec);
          }
          named_bar_sync(1 + half, 128);
        }
      } else {
        // the only tile of this cluster: its copies have landed and its products have read them, so the ring is free
        float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < H / 2; ++i) {
          if (2 * i < mine) {
            sums[(first + 2 * i) * 128 + ch] = acc[i].x;
            sums[(first + 2 * i + 1) * 128 + ch] = acc[i].y;
          }
        }
      }
    }
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync();
    const int id = blockIdx.x / split;
    if (id < tiles && s_limit) {
      const Tile t = tile_of<NT, 128, true>(a, id, ctiles, kblocks, gs);
      // a warp takes a row, a lane four channels of it; the parts' loads are under way together and added in order
      const int size = a.out_dtype == MOE_DENSE_FP32 ? 4 : 2;
      const bool vec = reinterpret_cast<uintptr_t>(a.out) % (4 * size) == 0 && a.out_stride % 4 == 0;
      for (int r = part + split * warp; r < t.rows; r += split * (kThreads / 32)) {
        float4 v[kMostParts];
#pragma unroll
        for (int p = 0; p < kMostParts; ++p)
          if (p < split) v[p] = ld_cluster4(mapa(base + (r * 128 + lane * 4) * 4, p));
#pragma unroll
        for (int p = 1; p < kMostParts; ++p)
          if (p < split) v[0] = make_float4(v[0].x + v[p].x, v[0].y + v[p].y, v[0].z + v[p].z, v[0].w + v[p].w);
        store4(a, t.row0 + r, t.c0 + lane * 4, v[0], vec);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

template <int NT>
cudaError_t run(const Maps& maps, const MatmulArgs& a, int split, int grid, cudaStream_t stream) {
  return launch_cluster<fp8_stream_kernel<NT>>(split, dim3(grid), dim3(kThreads), Shape<NT>::kTotal, stream, maps, a);
}

// Few rows: 32 at most in a tile (groups: 16 on average), else 128.  256 weights of 1024 x 2048 (us, tiles of 32 / 128 rows): 16 rows
// each 89.8 / 89.6, 32 (some above) 116.2 / 92.5; 16 weights of 4096 x 4096: 8 rows each 49.9 / 51.4, 32: 62.6 / 53.2.
bool few_rows(const MatmulArgs& a) {
  return a.offsets ? rows_of_a_group(a) <= 16 : a.rows <= kFewRows;
}

}  // namespace

int fp8_stream_split(const MatmulArgs& a, int sms) {
  if (a.offsets) return 1;
  const bool few = few_rows(a);
  const int nt = few ? kFewRows : kSomeRows, kblocks = (a.k + 127) / 128;
  const int64_t tiles = static_cast<int64_t>((a.n + 127) / 128) * ((a.rows + nt - 1) / nt);
  // clusters that would not all be resident take twice the time (16 of 8 CTAs: 12.2 us, of 6: 7.7, 8192 k x 2048 channels)
  for (int split = kMostParts; split > 1; --split) {
    if (split > kblocks || tiles * split > sms) continue;
    const int most = few ? resident_clusters<fp8_stream_kernel<kFewRows>>(split, dim3(kThreads), Shape<kFewRows>::kTotal)
                         : resident_clusters<fp8_stream_kernel<kSomeRows>>(split, dim3(kThreads), Shape<kSomeRows>::kTotal);
    if (tiles <= most) return split;
  }
  return 1;
}

cudaError_t launch_fp8_stream(const MatmulArgs& a, int sms, int split, cudaStream_t stream) {
  Maps maps;
  const int64_t groups = a.offsets ? a.groups : 1;
  if (encode_fp8_map(&maps.w, a.w, a.k, groups * a.n, a.k, 128) != MOE_OK ||
      encode_fp8_map(&maps.x16, a.x, a.k, a.rows, a.x_stride, 16) != MOE_OK ||
      encode_fp8_map(&maps.x64, a.x, a.k, a.rows, a.x_stride, 64) != MOE_OK)
    return cudaErrorInvalidValue;
  const bool few = few_rows(a);
  int grid = sms;
  if (!a.offsets) {
    const int nt = few ? kFewRows : kSomeRows;
    const int64_t tiles = static_cast<int64_t>((a.n + 127) / 128) * ((a.rows + nt - 1) / nt);
    if (tiles * split < sms || split > 1) grid = static_cast<int>(tiles) * split;
  }
  return few ? run<kFewRows>(maps, a, split, grid, stream) : run<kSomeRows>(maps, a, split, grid, stream);
}

}  // namespace dense
}  // namespace moe
