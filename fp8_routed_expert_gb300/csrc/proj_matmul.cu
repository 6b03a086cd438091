// Product of e4m3 rows with e4m3 weights, a f32 scale for each 1 x 128 of the rows
// and each 128 x 128 of the weights (moe_proj_matmul of the C ABI):
//   out[m, n] = bf16( sum over K blocks b of a_scale[m, b] * w_scale[n / 128, b] *
//                     sum over k in b of a[m, k] * w[n, k] )
//
// Tile: 128 rows x Columns columns, K in steps of one block.  TMA brings 128-byte
// rows of both operands (zeros outside the matrices, so any M, N and K), the
// 128-byte swizzle is what tcgen05.mma kind::f8f6f4 reads, and the sums of one or two
// blocks (kTurn) land in one of two TMEM buffers.  The other warps take them from there
// and add them, times the product of the two scales, to f32 registers while the other
// buffer fills: lane = row, so a thread's scale is one number per block (and 128 columns).
//
// What bounds it.  Few rows: launch, one chain of loads, products, sums and, where tiles
// are split, the exchange: 1 x 6144 x 2048 takes 7.0 to 7.4 us where the weights alone take
// 1.9 at the copy rate, 64 x 8192 x 4096 10.5 of 5.1.  Many: 4096 x 8192 x 6144 takes
// 165 to 168 us in bursts of a few milliseconds, 2480 TFLOP/s, and 172 to 177 back to back,
// where the clocks come down: a block of 128 x 256 in about 880 cycles, of which its
// products take 520.  A summing warp waits 140 of them and adds up for 650 (its packed FMAs
// alone take 290 of a sub-partition's issue); between tiles go 2500.  16 summing warps
// (200 to 217 us) were no faster.
//
// Outputs of tiles of 256 columns leave by TMA from boxes in shared memory, which takes
// one block in flight of the ring: a row per lane stored 32 bytes at a time, the tile's end
// took 8000 cycles, in which the products run two blocks ahead at most (173 us, so 169;
// 4000 x 8000 x 208 27.3, so 22.2).  The narrower tiles' rows are short: through shared
// memory 512 x 4096 x 4096 took 14.8 instead of 13.7.
//
// A tile's K blocks may be split over the CTAs of a cluster (few tiles): each CTA
// owns as many rows, and each pushes its sums of the others' rows into their
// shared memory, and behind one cluster barrier a CTA adds its rows over all of them, in
// rank order.  (Sums left in place and read by the others took two barriers and reads
// that wait: 333 x 1000 x 2880 in six parts 15000 cycles.)  Nothing is added in order of
// arrival, and no call needs a workspace.
//
// Warps: 0 issues TMA, 1 allocates TMEM and issues the products, 2 copies the scales, 4..
// add up.
#include "common.cuh"
#include "kernels.h"
#include "proj.h"
#include "tcgen05_ops.cuh"

namespace fp8moe {
using namespace sm100;
namespace {

constexpr int kRows = 128, kBlock = 128;
constexpr uint64_t kWaitNs = 2000000000ull;

// A block's scales are copied when its operands are; kHeld blocks on, the block of that
// place has long been added up: at most kMostStages and the two TMEM buffers' four lie
// between.
constexpr int kHeld = 16, kScales = kRows + 2;
constexpr int kMostStages = 8;
constexpr int kOutBytes = 32 * 128 * 2;  // a summing warp's outputs of a tile of 256 columns

// Quarters: of a tile's 128 rows (TMEM's lanes by warp) that are of use.  With one or two,
// which a warp each adds up, two CTAs of 64 columns fit on an SM (a sub-partition then has
// four of their warps, of 128 registers each); else two warps share a quarter.
template <int Columns, int Quarters>
struct Ring {
  static constexpr bool kFew = Quarters < 4;
  // blocks that are handed over at a time: what a summing warp waits, reads and answers
  // per turn takes as long as its sums of a block (shared memory is busy with the
  // products' operands); tiles of 256 columns fill TMEM with two blocks
  static constexpr int kTurn = Columns == 256 ? 1 : 2;
  static constexpr uint32_t kTmem = 2 * kTurn * Columns;
  static constexpr int kGroups = kFew ? 1 : 2, kSumWarps = Quarters * kGroups, kThreads = 128 + 32 * kSumWarps;
};

// Tiles of 256 columns: 384 threads start with 168 registers each, of which the summing
// warps, with 128 sums each, take more: 128 * 80 + 256 * 208 <= 384 * 168 (checked against
// the build in ready_one).  Each branch asks for itself, which is where the compiler looks.
constexpr int kFewRegs = 80, kManyRegs = 208;

struct Item {
  int m0, n0;
  int b0, b1;  // K blocks
};

template <int Columns>
__device__ __forceinline__ Item item_of(const MatmulArgs &p, int64_t tile, int rank) {
  const int64_t m_tiles = (p.M + kRows - 1) / kRows;
  Item it;
  it.m0 = (int)(tile % m_tiles * kRows);
  it.n0 = (int)(tile / m_tiles * Columns);
  it.b0 = Columns == 256 ? 0 : (int)((int64_t)p.blocks * rank / p.splits);
  it.b1 = Columns == 256 ? p.blocks : (int)((int64_t)p.blocks * (rank + 1) / p.splits);
  return it;
}

__device__ __forceinline__ void give_up(volatile int *stop, int *err) {
  *stop = 1;
  set_error(err, DEV_ERR_TIMEOUT);
}

// Eight neighbouring columns of a row, as far as the matrix goes.
__device__ __forceinline__ void store8(const MatmulArgs &p, int64_t row, int64_t col, const float (&v)[8]) {
  __nv_bfloat16 *o = p.out + row * p.out_stride + col;
  if (col + 8 <= p.N) {
    *reinterpret_cast<uint4 *>(o) =
        make_uint4(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]), bf16x2_of(v[4], v[5]), bf16x2_of(v[6], v[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < p.N) o[j] = __float2bfloat16_rn(v[j]);
  }
}

template <int Columns, int Quarters>
__global__ void __launch_bounds__(Quarters < 4 ? 256 : Ring<Columns, Quarters>::kThreads, Quarters < 4 ? 2 : 1) matmul_kernel(const __grid_constant__ CUtensorMap ta,
                                                             const __grid_constant__ CUtensorMap tw,
                                                             const __grid_constant__ CUtensorMap to, const MatmulArgs p) {
  using R = Ring<Columns, Quarters>;
  constexpr int kMine = Columns / R::kGroups;  // columns of a summing warp
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMostStages], empty[kMostStages], sum_full[2], sum_empty[2];
  __shared__ uint32_t tmem_sh;
  __shared__ volatile int stop;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // stages, what a product of the last one may read behind it, a cluster's sums, and the
  // scales of kHeld blocks: 128 of rows, two of weights
  const int a_bytes = R::kFew ? p.a_bytes : kRows * kBlock, stage_bytes = a_bytes + Columns * kBlock;
  const float4 *sums = reinterpret_cast<const float4 *>(smem + p.sums_at);
  float *scales = reinterpret_cast<float *>(smem + p.scales_at);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1 + 32), mbar_init(&empty[s], 2);
    for (int b = 0; b < 2; ++b) mbar_init(&sum_full[b], 2), mbar_init(&sum_empty[b], R::kSumWarps);
    stop = 0;
    fence_mbar_init();
    prefetch_tmap(&ta);
    prefetch_tmap(&tw);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_sh, R::kTmem);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_wait();
  pdl_trigger();
  const int splits = Columns == 256 ? 1 : p.splits;  // (tiles of 256 columns are many)
  const int rank = splits > 1 ? (int)cluster_rank() : 0;
  if (splits > 1) cluster_started();  // nothing is pushed to a CTA that does not run yet
  const int64_t first = blockIdx.x / splits, step = gridDim.x / splits;

  const auto few_registers = [] {
    if constexpr (Columns == 256) fewer_registers<kFewRegs>();
  };
  if (warp == 0) {
    few_registers();
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int64_t tile = first; tile < p.tiles && !stop; tile += step) {
        const Item it = item_of<Columns>(p, tile, rank);
        for (int b = it.b0; b < it.b1; ++b) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, &stop, kWaitNs)) {
            give_up(&stop, p.err);
            break;
          }
          uint8_t *s = smem + (size_t)stage * stage_bytes;
          mbar_arrive_expect_tx(&full[stage], (uint32_t)(p.a_rows + Columns) * kBlock);
          tma_load_2d(s, &ta, b * kBlock, it.m0, &full[stage]);
          tma_load_2d(s + a_bytes, &tw, b * kBlock, it.n0, &full[stage]);
          if (++stage == stages) stage = 0, phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    few_registers();
    // the whole warp in step, one lane issues (see mma_e4m3_ss)
    constexpr uint32_t idesc = idesc_e4m3_f32(kRows, Columns);
    const uint32_t leader = elect_lane();
    const uint64_t desc = sw128_kmajor_desc(smem_u32(smem));
    int stage = 0, buf = 0;
    uint32_t phase = 0, bphase = 0;
    bool ok = true;
    const auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, &stop, kWaitNs));
      if (!ok) give_up(&stop, p.err);
      return ok;
    };
    for (int64_t tile = first; ok && tile < p.tiles; tile += step) {
      const Item it = item_of<Columns>(p, tile, rank);
      for (int b = it.b0; ok && b < it.b1; b += R::kTurn) {
        if (!wait(&sum_empty[buf], bphase ^ 1u)) break;
#pragma unroll
        for (int u = 0; u < R::kTurn; ++u) {
          if (b + u >= it.b1 || !wait(&full[stage], phase)) break;
          tc_fence_after();
          const uint64_t a = desc + (uint64_t)(stage * (stage_bytes / 16)), w = a + (uint64_t)(a_bytes / 16);
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k)
            mma_e4m3_ss(leader, tmem + (uint32_t)((buf * R::kTurn + u) * Columns), a + k * 2, w + k * 2, idesc, k > 0 ? 1u : 0u);
          mma_commit_by(leader, &empty[stage]);
          if (lane == 0) mbar_arrive(&empty[stage]);
          if (++stage == stages) stage = 0, phase ^= 1u;
        }
        mma_commit_by(leader, &sum_full[buf]);
        // The scales, which other warps copy and read, pass through this one: commits tell of
        // products alone, a thread's own arrival hands on what it has waited for.
        if (lane == 0) mbar_arrive(&sum_full[buf]);
        buf ^= 1;
        if (buf == 0) bphase ^= 1u;
      }
    }
  } else if (warp == 2) {
    few_registers();
    const int n_blocks = (int)((p.N + 127) / 128);
    int stage = 0;
    uint32_t phase = 0, count = 0;
    bool ok = true;
    for (int64_t tile = first; ok && tile < p.tiles; tile += step) {
      const Item it = item_of<Columns>(p, tile, rank);
      const float *sa[4], *sw = p.w_scale + (int64_t)min((int)(it.n0 / 128) + (lane & 1), n_blocks - 1) * p.blocks;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = it.m0 + 32 * i + lane;
        sa[i] = p.a_scale + (row < p.M ? row : p.M - 1) * p.a_row;
      }
      for (int b = it.b0; b < it.b1; ++b, ++count) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, &stop, kWaitNs));
        if (!ok) {
          give_up(&stop, p.err);
          break;
        }
        float *to = scales + (count & (kHeld - 1)) * kScales;
#pragma unroll
        for (int i = 0; i < Quarters; ++i) copy4(to + 32 * i + lane, sa[i] + b * p.a_block);
        if (lane < 2) copy4(to + kRows + lane, sw + b);
        copies_arrive(&full[stage]);
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
    }
  } else if (warp == 3) {
    few_registers();
  } else {
    if constexpr (Columns == 256) more_registers<kManyRegs>();
    const int quarter = warp & 3, group = (warp - 4) >> 2;  // TMEM lanes and columns of this warp
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(group * kMine);
    uint32_t count = 0;
    int buf = 0;
    uint32_t bphase = 0;
    bool ok = true;
    for (int64_t tile = first; ok && tile < p.tiles; tile += step) {
      const Item it = item_of<Columns>(p, tile, rank);
      const bool any = it.m0 + quarter * 32 < p.M && it.n0 + group * kMine < p.N;  // of the warp
      uint64_t acc[kMine / 2];
#pragma unroll
      for (int j = 0; j < kMine / 2; ++j) acc[j] = 0;
      for (int b = it.b0; b < it.b1; b += R::kTurn) {
        // (to the vote: a warp that was split would not get through its collective instructions)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sum_full[buf], bphase, &stop, kWaitNs)))) {
          give_up(&stop, p.err);
          break;
        }
        tc_fence_after();
        const int here = min(R::kTurn, it.b1 - b);
        const auto give_back = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sum_empty[buf]);
        };
        if (any) {
          float c[R::kTurn];  // (the products were of operands that came with these scales)
#pragma unroll
          for (int u = 0; u < R::kTurn; ++u) {
            const float *sc = scales + (count + u & (kHeld - 1)) * kScales;
            c[u] = sc[quarter * 32 + lane] * sc[kRows + group * kMine / 128];
          }
          const uint32_t from = t_lane + (uint32_t)(buf * R::kTurn * Columns);
          if constexpr (Columns == 256) {
            // the next 16 columns on their way while these are added, and the buffer given
            // back before the last are (4096 x 8192 x 6144: 169 us, so 164; the narrow
            // tiles' warps take turns by themselves: 512 x 4096 x 4096 13.6, so 14.6)
            const uint64_t cc = pack_f32x2(c[0], c[0]);
            uint32_t v[2][16];
            tmem_ld16(from, v[0]);
            tmem_wait_ld16(v[0]);
#pragma unroll
            for (int l = 0; l < kMine; l += 16) {
              uint32_t(&x)[16] = v[l / 16 & 1], (&next)[16] = v[l / 16 & 1 ^ 1];
              if (l + 16 < kMine) tmem_ld16(from + l + 16, next);
              if (l + 16 == kMine) give_back();
#pragma unroll
              for (int j = 0; j < 16; j += 2)
                acc[(l + j) / 2] = fma_f32x2_in_order(pack_f32x2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), cc, acc[(l + j) / 2]);
              if (l + 16 < kMine) tmem_wait_ld16(next);
            }
          } else {
#pragma unroll
            for (int u = 0; u < R::kTurn; ++u) {
              if (u >= here) break;
              const uint64_t cc = pack_f32x2(c[u], c[u]);
#pragma unroll
              for (int l = 0; l < kMine; l += 16) {
                uint32_t v[16];
                tmem_ld16(from + u * Columns + l, v);
                tmem_wait_ld16(v);
#pragma unroll
                for (int j = 0; j < 16; j += 2)
                  acc[(l + j) / 2] = fma_f32x2(pack_f32x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), cc, acc[(l + j) / 2]);
              }
            }
          }
        }
        count += (uint32_t)here;
        if (Columns < 256 || !any) give_back();
        buf ^= 1;
        if (buf == 0) bphase ^= 1u;
      }
      if (splits > 1) cluster_wait_started();  // (a cluster has one tile)
      // the coordinates again, rather than held in registers through the blocks
      int64_t again = tile;
      asm volatile("" : "+l"(again));
      const Item at = item_of<Columns>(p, again, rank);
      const int64_t row = at.m0 + quarter * 32 + lane, col = at.n0 + group * kMine;
      if constexpr (Columns == 256) {
        // 64 columns at a time into the warp's boxes, which leave by themselves, but for up to
        // seven last columns: a box is cut off at 16 bytes, which would reach behind the row
        if (!ok || !any) continue;
        if (lane == 0) bulk_wait_read<0>();  // the tile before
        __syncwarp();
        uint8_t *box = smem + p.sums_at + (warp - 4) * kOutBytes;
#pragma unroll
        for (int j = 0; j < kMine; j += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_f32x2(acc[j / 2 + i]);
            w[i] = bf16x2_of(f.x, f.y);
          }
          *reinterpret_cast<uint4 *>(box + j / 64 * 4096 + lane * 128 + ((j / 8 & 7) ^ (lane & 7)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const int rest = (int)(p.N & 7), j = (int)(p.N - rest - col);
        if (rest != 0 && j >= 0 && j < kMine && row < p.M) {
          const uint16_t *last = reinterpret_cast<const uint16_t *>(box + j / 64 * 4096 + lane * 128 + ((j / 8 & 7) ^ (lane & 7)) * 16);
          for (int i = 0; i < rest; ++i) p.out[row * p.out_stride + col + j + i] = __ushort_as_bfloat16(last[i]);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < kMine; j += 64)
            if (col + j < (p.N & ~INT64_C(7))) tma_store_2d(&to, box + j / 64 * 4096, (int)col + j, at.m0 + quarter * 32);
          bulk_commit();
        }
        continue;
      }
      if (!ok || !any || row >= p.M) continue;
      if (splits == 1) {
        __nv_bfloat16 *out = p.out + row * p.out_stride + col;
        // 32 bytes at a time where they lie in one line: half as many line accesses
        if (p.whole_lines && col + kMine <= p.N) {
#pragma unroll
          for (int j = 0; j < kMine; j += 16) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 f = unpack_f32x2(acc[j / 2 + i]);
              w[i] = bf16x2_of(f.x, f.y);
            }
            st_global32(out + j, w);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kMine; j += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = unpack_f32x2(acc[j / 2 + i]);
              v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
            if (col + j < p.N) store8(p, row, col + j, v);
          }
        }
      } else {
        // to the row's CTA: [rank][row % held][Columns] f32, the 16-byte pieces of a
        // row exchanged by its number so that a warp's rows do not meet in one bank
        const int r = quarter * 32 + lane, owner = r / p.held, place = r - owner * p.held;
        const uint32_t mine = map_to_rank(smem_u32(sums + (rank * p.held + place) * (Columns / 4)), (uint32_t)owner);
#pragma unroll
        for (int j = 0; j < kMine; j += 4) {
          const float2 f = unpack_f32x2(acc[j / 2]), g = unpack_f32x2(acc[j / 2 + 1]);
          const int piece = (group * kMine + j) / 4 ^ (place & (Columns / 4 - 1));
          st_cluster16(mine + 16 * piece, f.x, f.y, g.x, g.y);
        }
      }
    }
    if (Columns == 256 && lane == 0) bulk_wait<0>();
  }
  __syncwarp();
  if (splits > 1) {
    if (warp < 4) cluster_wait_started();
    cluster_sync_all();
    // a lane adds 8 columns of a row of this CTA's
    const Item it = item_of<Columns>(p, first, rank);
    const int rows = (int)(p.M - it.m0 < kRows ? p.M - it.m0 : kRows);
    for (int u = threadIdx.x; u < p.held * (Columns / 8); u += R::kThreads) {
      const int at = u / (Columns / 8), c = u % (Columns / 8) * 2, r = rank * p.held + at;
      if (r >= rows || it.n0 + 4 * c >= p.N) continue;
      const int swap = at & (Columns / 4 - 1);
      float v[8] = {};
#pragma unroll 2
      for (int q = 0; q < splits; ++q) {
        const float4 *row = sums + (q * p.held + at) * (Columns / 4);
        const float4 f = row[c ^ swap], g = row[c + 1 ^ swap];
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w, v[4] += g.x, v[5] += g.y, v[6] += g.z, v[7] += g.w;
      }
      store8(p, it.m0 + r, it.n0 + 4 * c, v);
    }
  }
  __syncthreads();
  if (stop) {
    // copies and products in flight land before the memory goes away
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 50000ull) {
    }
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, R::kTmem);
  }
}

template <int Columns, int Quarters>
cudaError_t launch_one(const CUtensorMap &a, const CUtensorMap &w, const CUtensorMap &o, const MatmulArgs &m, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)m.grid);
  cfg.blockDim = dim3(Ring<Columns, Quarters>::kThreads);
  cfg.dynamicSmemBytes = (size_t)m.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)m.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = m.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, matmul_kernel<Columns, Quarters>, a, w, o, m);
}

// Shared memory of a CTA where one or two of them have an SM.
constexpr int kOnePerSm = 226 * 1024, kTwoPerSm = 112 * 1024, kAround = kHeld * kScales * 4 + 1024;

// Stands in for a kernel in the question how many clusters are resident: the answer for
// one that allocates TMEM is always one CTA per SM, however little it takes.
__global__ void __launch_bounds__(256, 2) place_kernel() {}

template <int Columns, int Quarters>
cudaError_t ready_one(int (&fit)[kMostSplits + 1]) {
  constexpr int kSmem = Quarters < 4 ? kTwoPerSm : kOnePerSm;
  cudaError_t e = cudaFuncSetAttribute(matmul_kernel<Columns, Quarters>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  cudaFuncAttributes at;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, matmul_kernel<Columns, Quarters>);
  // the summing warps would wait forever for registers that the launch does not have
  if (e == cudaSuccess && Columns == 256 && at.numRegs * 3 < kFewRegs + 2 * kManyRegs) e = cudaErrorInvalidKernelImage;
  const auto kernel = place_kernel;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  for (int c = 1; e == cudaSuccess && c <= kMostSplits; ++c) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&fit[c], kernel, &cfg);
  }
  return e;
}

}  // namespace

cudaError_t ready_matmul(MatmulFit *fit) {
  for (cudaError_t e : {ready_one<64, 1>(fit->few), ready_one<64, 2>(fit->few), ready_one<64, 4>(fit->many[0]), ready_one<128, 4>(fit->many[1]),
                        ready_one<256, 4>(fit->many[2])})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

// How a product is split.  A tile's K blocks go over as many CTAs as are resident
// together: clusters that come in a second round double the time.  The time is
// about, in cycles: a block 420, 560 and 880 for 64, 128 and 256 columns (260 with few
// rows), a tile's start and end 2000, 2600 and 2500, a cluster's exchange 150 for each CTA
// and what a CTA pushes at 12 bytes.  Against the best of all splits (us):
//   64 x 2048 x 2048      5.5: 64 columns, 4 CTAs; 3 CTAs 5.9, 8 CTAs 6.5, 2 CTAs 6.4
//   16 x 4096 x 4096      6.6: 64, 4; 3 CTAs 7.4, 2 CTAs 8.1, alone 11.1
//   333 x 1000 x 2880     8.2: 64, 2; 128 columns, 4 CTAs 9.1; 64 alone 9.3
//   512 x 4096 x 4096     14.2: 128, alone; 256 columns 18.9
//   700 x 512 x 7008      11.4: 128, 5; 64, 2 CTAs 12.3; 128, 2 CTAs 14.4
//   800 x 7000 x 400      10.9: 256, alone; 128 columns 11.9
//   2048 x 2048 x 4096    19.8: 256, alone; 128 columns 25.2
//   1 x 6144 x 2048       7.0: 64, 3, where 2 CTAs take 6.3 and one 7.2: the largest miss
// of these, the others are the best.
void plan_matmul(const MatmulFit &fit, int sms, int limit, MatmulArgs *m) {
  const bool few = m->M <= 64;
  const int64_t rows = (m->M + kRows - 1) / kRows;
  double best = 0.0;
  m->columns = 0;
  for (int i = 0; i < (few ? 1 : 3); ++i) {
    const int columns = 64 << i;
    const int64_t tiles = rows * ((m->N + columns - 1) / columns);
    const int *places = few ? fit.few : fit.many[i];
    for (int splits = 1; splits <= kMostSplits && splits <= m->blocks; ++splits) {
      // (with a limit a CTA per SM: two would go to an SM each while others are idle)
      const int64_t most = (limit > 0 ? limit : (int64_t)sms * (few ? 2 : 1)) / splits, resident = places[splits] < most ? places[splits] : most;
      if (splits > 1 && (tiles > resident || columns == 256)) continue;
      const double rounds = (double)((tiles + resident - 1) / (resident > 0 ? resident : 1));
      const double block = few ? 260.0 : columns == 64 ? 420.0 : columns == 128 ? 560.0 : 880.0;
      const double around = columns == 64 ? 2000.0 : columns == 128 ? 2600.0 : 2500.0;
      double t = rounds * ((double)((m->blocks + splits - 1) / splits) * block + around);
      if (splits > 1) t += 150.0 * splits + (double)(m->M < kRows ? m->M : kRows) * columns * 4 * (splits - 1) / splits / 12.0;
      if (m->columns == 0 || t < best) {
        best = t;
        m->columns = columns;
        m->splits = splits;
        m->tiles = tiles;
        m->grid = splits > 1 ? tiles * splits : tiles < resident ? tiles : resident;
      }
    }
  }
  m->few = few;
  m->a_rows = m->M < kRows ? (int)((m->M + 7) / 8 * 8) : kRows;
  m->a_bytes = few ? m->a_rows * kBlock : kRows * kBlock;  // whole 8-row atoms of 1024 bytes
  const int sum_rows = m->M < kRows ? (int)m->M : kRows;
  m->held = (sum_rows + m->splits - 1) / m->splits;
  const int sums = m->columns == 256 ? 8 * kOutBytes : m->splits > 1 ? m->held * m->splits * m->columns * 4 : 0;
  const int stage = m->a_bytes + m->columns * kBlock;
  // a product reads 128 rows of either operand: those behind the last stage's few rows are
  // of no use, but have to be there
  const int behind = stage < kRows * kBlock ? kRows * kBlock - stage : 0;
  const int room = (few ? kTwoPerSm : kOnePerSm) - kAround - sums - behind;
  m->stages = room / stage < kMostStages ? room / stage : kMostStages;
  m->sums_at = m->stages * stage + behind;
  m->scales_at = m->sums_at + sums;
  m->smem = m->scales_at + kAround;
}

cudaError_t launch_matmul(const CUtensorMap &a, const CUtensorMap &w, const CUtensorMap &o, const MatmulArgs &m, cudaStream_t s) {
  if (m.few) return m.M <= 32 ? launch_one<64, 1>(a, w, o, m, s) : launch_one<64, 2>(a, w, o, m, s);
  switch (m.columns) {
    case 64: return launch_one<64, 4>(a, w, o, m, s);
    case 128: return launch_one<128, 4>(a, w, o, m, s);
    default: return launch_one<256, 4>(a, w, o, m, s);
  }
}

}  // namespace fp8moe
