// Block-scaled products of many rows (include/moe_dense.h): pairs of CTAs, 256 rows of x times 256 channels a tile.
//
// As in fp8_stream.cu each block of 128 k is a product of its own in tensor memory, which is multiplied by its scales on the
// way into FP32 registers.  Here a lane of tensor memory is a row of x, so that a thread has one scale a block: that of
// its row times that of its 128 channels.  One tcgen05.mma (cta_group::2) multiplies 256 x 32 by 32 x 256 codes: each CTA holds
// 128 rows of x and 128 channels of the weight, so a block costs a CTA 32 KB of copies for 512 cycles of the tensor
// core; with a CTA on its own (128 x 256) it would be 48 KB, more than an SM gets from L2 in that time.
//
// Roles in each CTA: eight warps add up (a thread has 128 sums; sixteen with 64 each were no faster), a warp copies,
// two bring the scales of a block's rows into shared memory (loaded by the warps that add up, they cost a
// third of the time); the first CTA's issuing warp starts the MMAs of both.  Two products alternate in tensor memory.
// Whole slices of 32 rows leave as bulk tensor stores of boxes of 128 bytes a row, while the next tile is under way; written
// by their threads they held up the warps 5000 cycles a tile.
//
// What bounds it: the warps that add up.  A block takes ~765 cycles against 512 of the MMAs and ~560 of its copies (57 bytes a
// cycle and SM from L2): 256 x 128 multiply-adds of an SM are 256 cycles of its FP32 lanes, and the reads of tensor memory
// overlap with them only in part.  8192 x 8192 x 4096 takes 196 us, with the sums and reads left out (and their waits kept) 134,
// without the multiply-adds 167, without the reads 174, with buffers given back before they are read 201.  Reads of 8 columns,
// or ahead of the multiply-adds, 207 to 211; of 32 columns in two sets of registers, with more of them for these warps, 202.
// A tile's outputs cost another ~1400 cycles.  Measured in graph replays, codes of normal values, clocks left alone, on several machines:
// 8192 x 8192 x 4096 194 to 206 us, 2.7 to 2.84 PFLOP/s (1.4 to 1.48 of the measured bf16 rate; the tensor cores are busy
// 60 % of the time); 512 weights of 1024 x 2048 with 160 rows each, unequal, 229 to 236 us (185 us of bytes).  Single calls one after
// the other, with a new output each, take 215 to 224 and 256 to 262.
#include "fp8_tiles.cuh"

namespace moe {
namespace dense {
namespace {

constexpr int kSumWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kScaleWarps = 2, kWarps = 12, kThreads = 32 * kWarps;
constexpr int kTileRows = 256, kTileCh = 256, kCols = 1024 / kSumWarps;  // kCols: sums of a thread
constexpr uint32_t kDrainCycles = 1u << 24, kLandCycles = 1u << 20;
constexpr int kStages = 4, kStage = 2 * 128 * 128, kBufs = 2;
constexpr int kBatch = 4, kSlot = 132;  // blocks whose scales come together; floats of one: 128 rows', the weight's two, two of the tile's
constexpr int kBox = 32 * 128;  // bytes of a box of outputs: 32 rows of 128 bytes, in swizzled lines

struct Layout {
  static constexpr int kStaged = kStages * kStage;  // [8 warps][2 boxes]
  static constexpr int kScales = kStaged + kSumWarps * 2 * kBox;  // [2][kBatch][kSlot]
  static constexpr int kBars = kScales + 2 * kBatch * kSlot * 4;
  static constexpr int kGroups = kBars + 8 * (2 * kStages + 2 * kBufs + 4 + 2);
  static constexpr int kTotal = kGroups + static_cast<int>(sizeof(Groups)) + 1024;
  static_assert(kTotal <= 227 * 1024);
};

struct Maps {
  CUtensorMap w, x, out;  // boxes of 128, 64 and 32 rows
  bool store;             // outputs can be written through `out`
};

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives at `bar` of both CTAs once the MMAs issued so far have completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
      : "memory");
}
// Of the pair's first CTA.  The sums are in registers and tcgen05.fence orders the reads of tensor memory; a release of
// cluster scope would wait for the thread's accesses to global memory too (a block then took 2700 cycles).
__device__ __forceinline__ void arrive_lead(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 16 bytes of a row's outputs: sums i, i + 1, ...
template <typename T>
__device__ __forceinline__ uint4 sixteen(const float2* v) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  else
    return make_uint4(two<T>(v[0].x, v[0].y), two<T>(v[1].x, v[1].y), two<T>(v[2].x, v[2].y), two<T>(v[3].x, v[3].y));
}
__device__ __forceinline__ void add_up(float2* acc, const uint32_t (&v)[16], float s) {
#pragma unroll
  for (int i = 0; i < 16; i += 2)
    acc[i / 2] = fma2_in_order(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), make_float2(s, s), acc[i / 2]);
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_wide_kernel(const __grid_constant__ Maps maps, const __grid_constant__ MatmulArgs a) {
  typedef Layout L;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem, s_limit, s_drain;
  __shared__ int s_scan[kWarps];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_addr(smem);
  Groups& gs = *reinterpret_cast<Groups*>(smem + L::kGroups);
  // barriers; full and freed are the first CTA's, waited for by its issuing warp
  const uint32_t full = base + L::kBars, empty = full + 8 * kStages, done = empty + 8 * kStages, freed = done + 8 * kBufs,
                 scaled = freed + 8 * kBufs, used = scaled + 16, end = used + 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + 8 * i, a.copy_arrivals);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(done + 8 * i, 1);
      mbar_init(freed + 8 * i, 2 * kSumWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(scaled + 8 * i, kScaleWarps);
      mbar_init(used + 8 * i, kSumWarps);
    }
    mbar_init(end, 1);
    s_limit = a.wait_cycles;
    s_drain = kDrainCycles;
  }
  fence_barrier_init();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == kCopyWarp && lane == 0) {
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.x);
  }
  pdl_wait();
  pdl_launch_dependents();
  make_groups<kWarps, kTileRows>(a, gs, s_scan);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile uint32_t* limit = &s_limit;

  const int ctiles = (a.n + kTileCh - 1) / kTileCh, kblocks = (a.k + 127) / 128;
  const int tiles = gs.before[a.groups] * ctiles, stride = gridDim.x / 2;

  // of the launch's 384 x 168 registers, the 256 threads that add up take 208 each and the others keep 88
  if (warp >= kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kCopyWarp) {
      const uint32_t lead = mapa(full, 0);
      uint32_t it = 0;
      bool ok = true;
      for (int id = blockIdx.x / 2; ok && id < tiles; id += stride) {
        const Tile t = tile_of<kTileRows, kTileCh, false>(a, id, ctiles, kblocks, gs);
        // 64 rows at a time, as far as there are rows
        const int boxes0 = min(2, (t.rows + 63) / 64), boxes1 = max(0, (t.rows - 128 + 63) / 64);
        const int boxes = rank ? boxes1 : boxes0;
        const uint32_t bytes = 2 * 128 * 128 + (boxes0 + boxes1) * 64 * 128;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const uint32_t s = it % kStages;
          if (!(ok = warp_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1, limit, a.status))) break;
          if (elect_one()) {
            const uint32_t at = base + s * kStage, bar = lead + 8 * s;
            if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
            for (int i = 0; i < boxes; ++i)
              tma_load_pair(at + i * 64 * 128, &maps.x, kb * 128, t.row0 + static_cast<int>(rank) * 128 + i * 64, bar);
            tma_load_pair(at + 16384, &maps.w, kb * 128, static_cast<int>(t.w_row) + static_cast<int>(rank) * 128, bar);
          }
          __syncwarp();
        }
      }
      // copies in flight land before the CTAs leave: the first CTA's barriers count both CTAs' bytes
      // (and so does what the products' end says to both)
      for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) {
        if (rank == 0) warp_wait(full + 8 * (i % kStages), (i / kStages) & 1, &s_drain, a.status);
        warp_wait(empty + 8 * (i % kStages), (i / kStages) & 1, &s_drain, a.status);
      }
      if (*limit == 0)
        for (const uint32_t t0 = cycles(); cycles() - t0 < kLandCycles;) {}
    } else if (warp == kMmaWarp) {
      if (rank == 0) {
        uint32_t it = 0;
        bool ok = true;
        constexpr uint32_t idesc = idesc_e4m3(256, 256);
        for (int id = blockIdx.x / 2; ok && id < tiles; id += stride) {
          for (int kb = 0; kb < kblocks; ++kb, ++it) {
            const uint32_t s = it % kStages, b = it % kBufs;
            const uint64_t da = smem_desc_sw128(base + s * kStage, 1024);
            const uint64_t db = smem_desc_sw128(base + s * kStage + 16384, 1024);
            // the copies first: they are mostly there long before the sums have left the buffer
            ok = warp_wait(full + 8 * s, (it / kStages) & 1, limit, a.status) &&
                 warp_wait(freed + 8 * b, ((it / kBufs) & 1) ^ 1, limit, a.status);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
  #pragma unroll
              for (int k = 0; k < 4; ++k) mma_pair(tmem + b * 256, da + 2 * k, db + 2 * k, idesc, k > 0);
              commit_pair(done + 8 * b);
              commit_pair(empty + 8 * s);
            }
            __syncwarp();
          }
        }
        if (elect_one()) commit_pair(end);
        __syncwarp();
      }
    } else {
      // rows r and r + 64 of this CTA's 128, and a half's weight scales
      const int second = warp - kScaleWarp, r = second * 32 + lane;
      float* out = reinterpret_cast<float*>(smem + L::kScales);
      uint32_t bt = 0;
      bool ok = true;
      for (int id = blockIdx.x / 2; ok && id < tiles; id += stride) {
        const Tile t = tile_of<kTileRows, kTileCh, false>(a, id, ctiles, kblocks, gs);
        const int row = static_cast<int>(rank) * 128 + r;
        const bool low = row < t.rows, high = row + 64 < t.rows, wide = lane < kBatch && t.c0 + second * 128 < a.n;
        const float* xs = a.xs + static_cast<int64_t>(t.row0 + row) * a.scale_row;
        const float* ws = t.ws + second * kblocks + lane;
        const int64_t next = 64 * a.scale_row;
        for (int kb0 = 0; ok && kb0 < kblocks; kb0 += kBatch, ++bt) {
          float x0[kBatch], x1[kBatch];
  #pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const bool there = kb0 + j < kblocks;
            x0[j] = there && low ? __ldcg(xs + (kb0 + j) * a.scale_block) : 0.f;
            x1[j] = there && high ? __ldcg(xs + next + (kb0 + j) * a.scale_block) : 0.f;
          }
          const float w = wide && kb0 + lane < kblocks ? __ldcg(ws + kb0) : 0.f;  // lane j: block j's
          ok = warp_wait(used + 8 * (bt & 1), ((bt >> 1) & 1) ^ 1, limit, a.status);
          if (!ok) break;
          float* to = out + (bt & 1) * (kBatch * kSlot);
  #pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            to[j * kSlot + r] = x0[j];
            to[j * kSlot + r + 64] = x1[j];
          }
          if (lane < kBatch) to[lane * kSlot + 128 + second] = w;
          if (kb0 == 0 && second == 0 && lane == 0) {  // the tile, for the warps that add up
            to[130] = __int_as_float(t.row0);
            to[131] = __int_as_float(t.c0);
            to[kSlot + 130] = __int_as_float(t.rows);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(scaled + 8 * (bt & 1));
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int half = warp >> 2, quarter = warp & 3;
    const uint32_t lead = mapa(freed, 0);
    const int slice = static_cast<int>(rank) * 128 + quarter * 32;  // rows of the tile that are this warp's
    uint8_t* staged = smem + L::kStaged + warp * 2 * kBox;
    const float* scales = reinterpret_cast<const float*>(smem + L::kScales);
    uint32_t it = 0, bt = 0;
    bool ok = true;
    for (int id = blockIdx.x / 2; ok && id < tiles; id += stride) {
      ok = warp_wait(scaled + 8 * (bt & 1), (bt >> 1) & 1, limit, a.status);
      const float* tile = scales + (bt & 1) * (kBatch * kSlot);
      const int row0 = __float_as_int(tile[130]) + slice, ch = __float_as_int(tile[131]) + half * kCols;
      const int live = min(32, __float_as_int(tile[kSlot + 130]) - slice);
      const bool work = live > 0 && ch < a.n;
      const uint32_t mine = tmem + half * kCols + (static_cast<uint32_t>(quarter * 32) << 16);
      float2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = 0; kb < kblocks; ++kb, ++it) {
        const uint32_t b = it % kBufs, from = mine + b * 256;
        const bool turn = kb % kBatch == kBatch - 1 || kb == kblocks - 1;  // of the scales' buffer
        if (kb % kBatch == 0 && kb) ok = warp_wait(scaled + 8 * (bt & 1), (bt >> 1) & 1, limit, a.status);
        const float* slot = scales + ((bt & 1) * kBatch + kb % kBatch) * kSlot;
        const float s = slot[quarter * 32 + lane] * slot[128 + half];
        ok = ok && warp_wait(done + 8 * b, (it / kBufs) & 1, limit, a.status);
        if (!ok) break;
        if (work) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            uint32_t v[16];
            tmem_ld_x16(from + c, v);
            tc_wait_ld();
            if (c == kCols - 16) {  // the block's place is given back with the last sums still to come
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_lead(lead + 8 * b);
            }
            add_up(acc + c / 2, v, s);
          }
        } else {
          __syncwarp();
          if (lane == 0) arrive_lead(lead + 8 * b);
        }
        if (turn) {
          if (lane == 0) mbar_arrive(used + 8 * (bt & 1));
          ++bt;
        }
      }
      if (!ok) break;
      if (!work) continue;
      constexpr int PER = 128 / sizeof(T), EL = 16 / sizeof(T);  // channels of a box, of 16 bytes
      T* out = static_cast<T*>(a.out) + static_cast<int64_t>(row0) * a.out_stride + ch;
#pragma unroll
      for (int c = 0; c < kCols; c += PER) {
        const int left = a.n - ch - c;
        if (left <= 0) break;
        uint8_t* box = staged + (c / PER % 2) * kBox;
        if (c / PER % 2 == 0) {  // what was written from here has been read
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) = sixteen<T>(acc + (c + j * EL) / 2);
        if (maps.store && live == 32) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&maps.out),
                         "r"(ch + c), "r"(row0), "r"(smem_addr(box))
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else {  // rows behind these are not to be written, or addresses that bulk copies do not take
          __syncwarp();
          if (maps.store && left >= PER) {
            for (int r = lane >> 3; r < live; r += 4)
              *reinterpret_cast<uint4*>(out + r * a.out_stride + c + (lane & 7) * EL) =
                  *reinterpret_cast<const uint4*>(box + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          } else {
            for (int i = lane; i < PER && i < left; i += 32)
              for (int r = 0; r < live; ++r)
                out[r * a.out_stride + c + i] =
                    *reinterpret_cast<const T*>(box + r * 128 + (((i / EL) ^ (r & 7)) << 4) + (i % EL) * sizeof(T));
          }
          __syncwarp();
        }
      }
    }
    tc_wait_ld();
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  if (warp == kMmaWarp) warp_wait(end, 0, &s_drain, a.status);  // products in flight end before their memory is given back
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace

cudaError_t launch_fp8_wide(const MatmulArgs& a, int sms, cudaStream_t stream) {
  Maps maps;
  const int64_t groups = a.offsets ? a.groups : 1;
  if (encode_fp8_map(&maps.w, a.w, a.k, groups * a.n, a.k, 128) != MOE_OK ||
      encode_fp8_map(&maps.x, a.x, a.k, a.rows, a.x_stride, 64) != MOE_OK)
    return cudaErrorInvalidValue;
  const int size = a.out_dtype == MOE_DENSE_FP32 ? 4 : 2;
  maps.store = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_stride * size % 16 == 0;
  if (maps.store && encode_rows_map(&maps.out, a.out, size, a.n, a.rows, a.out_stride * size, 128 / size, 32) != MOE_OK)
    return cudaErrorInvalidValue;
  int64_t pairs = sms / 2;
  if (!a.offsets) {
    const int64_t tiles = static_cast<int64_t>((a.n + kTileCh - 1) / kTileCh) * ((a.rows + kTileRows - 1) / kTileRows);
    if (tiles < pairs) pairs = tiles;
  }
  const dim3 grid(static_cast<unsigned>(2 * pairs)), block(kThreads);
  if (a.out_dtype == MOE_DENSE_FP32)
    return launch_ready<fp8_wide_kernel<float>>(grid, block, Layout::kTotal, stream, maps, a);
  if (a.out_dtype == MOE_DENSE_BF16)
    return launch_ready<fp8_wide_kernel<__nv_bfloat16>>(grid, block, Layout::kTotal, stream, maps, a);
  return launch_ready<fp8_wide_kernel<__half>>(grid, block, Layout::kTotal, stream, maps, a);
}

}  // namespace dense
}  // namespace moe
