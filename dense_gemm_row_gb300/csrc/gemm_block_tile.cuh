// gemm_block_tile.cuh -- e4m3 products with a scale for each block of 128 along k, on
// 256-row tiles:
//
//   Z_ij = alpha sum_b sa[i][b] sb[j / 128][b] sum_{k in b} A_ik B_jk + bias_j,  D = act(Z) + R
//   gated   D = act(G) U, where G and U are Z for two matrices B
//
// A block of 128 is one 128-byte row of a stage, so the accumulator is restarted for
// every stage (4 MMAs) and its 256 x kN sums are added, scaled, into fp32 registers:
// 128 per thread at kN = 256. The scales of a thread are one value per row and one per
// 128 columns, which a warp's columns never cross. The accumulators alternate, so that
// the MMAs of the next k-block run meanwhile.
//
// What bounds it (8192^3 with a residual: 396 us in short runs, 438 or 2.5 PFLOP/s
// repeated at the power limit; e4m3 with row scales 302 and 345): the
// epilogue's chain of loads from tensor memory, each about 100 cycles, 8 per k-block
// whose MMAs take 512. In short runs of a form that took 388: without the multiply-adds
// 336 us, without all but one of the loads 362, without either 309. Multiply-adds on
// packed pairs cost moves (441 us); loads of 32 columns or of 8 were slower (419, 397),
// and so were accumulators of 128 columns, four under way, emptied by all eight warps
// (463) or by half of them (383, but gated 245 against 225).
//
// Warps as in gemm_epi_tile.cuh, whose producer this kernel shares; the final epilogue
// works on the registers. Each warp has two staging buffers: R of both of its blocks
// of 64 columns is requested before the main loop, and D takes its place.
#pragma once

#include "block_scales.cuh"
#include "gemm_epi_tile.cuh"

namespace dgr {
namespace {

struct BlockScales {
  const float *a, *b, *b2;  // b2: a gated layer's second B
  int64_t lda, ldb, ldb2;
  int KB;
};

// Three warpgroups: producer, MMAs and two idle warps; the epilogue's eight. They are
// launched with 168 registers a thread, of which the first group keeps 40 and the
// others take 232: 40 + 2 * 232 = 3 * 168.
constexpr int kBlockThreads = 384, kBlockFirst = 4;  // the first epilogue warp

template <int kN>
constexpr int kBlockBufs = 512 / kN;  // accumulators in tensor memory

template <int kN>
using BlockSmem = EpiSmem<kN, 2>;

// The leader's MMA loop: one accumulator per k-block.
template <int kN>
__device__ __forceinline__ void block_multiply(const EpiArgs &p, BlockSmem<kN> &sm,
                                               uint32_t tmem_base, int unit, int units) {
  using Cf = EpiCfg<kN, 2>;
  constexpr int kBufs = kBlockBufs<kN>;
  volatile int *abort = &sm.abort;
  const int KB = (p.K - 1) / 128 + 1;
  const uint64_t adesc0 = smem_desc(smem_u32(sm.a[0]), 16, kAtomBytes, 2u);
  const uint64_t bdesc0 = smem_desc(smem_u32(sm.b[0]), 16, kAtomBytes, 2u);
  uint32_t stage = 0, phase = 0, buf = 0, use = 0;
  bool ok = true, any = false;
  for (int t = unit; ok && t < p.tiles; t += units) {
    for (int kb = 0; kb < KB; ++kb) {
      // (Cluster scope: both CTAs' warps give the accumulator back. Their relaxed arrivals
      // hand over nothing but their loads from it, which the fence below orders.)
      if (!mbar_wait_lazy<true>(smem_u32(&sm.tmem_empty[buf]), use ^ 1u, abort, p.err_word,
                                kWaitTmemEmpty) ||
          !mbar_wait_lazy(smem_u32(&sm.full[stage]), phase, abort, p.err_word, kWaitFull)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint64_t ad = adesc0 + stage * (Cf::kABytes >> 4);
      const uint64_t bd = bdesc0 + stage * (Cf::kBBytes >> 4);
      const uint32_t d_tmem = tmem_base + buf * kN;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_f8_pair(d_tmem, ad + kk * 2, bd + kk * 2, p.idesc, kk > 0 ? 1u : 0u);
        tc_commit_pair_mc(smem_u32(&sm.empty[stage]), 0x3);
        tc_commit_pair_mc(smem_u32(&sm.tmem_full[buf]), 0x3);
      }
      __syncwarp();
      any = true;
      if (++stage == Cf::kStages) {
        stage = 0;
        phase ^= 1u;
      }
      if (++buf == kBufs) {
        buf = 0;
        use ^= 1u;
      }
    }
  }
  // Never leave with an MMA still reading shared memory or writing TMEM. (The
  // same lane is elected each time, so its commit covers them all.)
  if (any) {
    if (elect_one()) tc_commit_pair_mc(smem_u32(&sm.drain), 0x1);
    __syncwarp();
    drain_wait(smem_u32(&sm.drain), 0, p.err_word);
  }
}

// Gives an accumulator back to the MMAs. Relaxed: the loads from it are complete
// (tcgen05.wait::ld), and nothing else is handed over. An arrive that releases waits
// for the thread's other accesses too, 1 us per k-block: 8192^3 took 916 us with one
// and 433 with this one.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr)
               : "memory");
}

// The bias of a warp's columns, two values per lane and 64 columns (packed), and z =
// alpha sum + bias: each pair comes from its lane.
__device__ __forceinline__ uint32_t load_bias(const uint16_t *bias, int col, int N) {
  if (bias == nullptr) return 0;
  const uint32_t lo = col < N ? bias[col] : 0, hi = col + 1 < N ? bias[col + 1] : 0;
  return lo | (hi << 16);
}
template <bool kBf16>
__device__ __forceinline__ void add_bias(float (&sum)[64], float alpha, bool have,
                                         uint32_t bias) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    float lo, hi;
    unpack16<kBf16>(have ? __shfl_sync(0xffffffffu, bias, j) : 0, lo, hi);
    sum[2 * j] = fmaf(sum[2 * j], alpha, lo);
    sum[2 * j + 1] = fmaf(sum[2 * j + 1], alpha, hi);
  }
}

// The final epilogue of a warp's 64 kCount columns, block of 64 columns by block.
template <bool kBf16, int kCount>
__device__ __forceinline__ void block_finish(const CUtensorMap &tmD, const CUtensorMap &tmZ,
                                             const EpiArgs &p, const uint32_t (&bias)[2],
                                             float (&sum)[kCount][64],
                                             const uint32_t (&stage)[2], int row0, int col0,
                                             bool early_r, uint32_t rbar, uint32_t &rphase,
                                             const CUtensorMap &tmR, int lane) {
  const bool have_r = p.c.R != nullptr;
#pragma unroll
  for (int c = 0; c < kCount; ++c)
    add_bias<kBf16>(sum[c], p.c.alpha, p.c.bias != nullptr, bias[c]);
  if (have_r && early_r && p.r_tma) {
    wait_copy(rbar, rphase, p.err_word);
    rphase ^= 1u;
  }
#pragma unroll
  for (int c = 0; c < kCount; ++c) {
    const int col = col0 + 64 * c;
    if (p.c.Z != nullptr) {
      stage_free(lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack16<kBf16>(sum[c][32 * h + 2 * j], sum[c][32 * h + 2 * j + 1]);
        stage_half(stage[c], lane, h, w);
      }
      store_block(&tmZ, p.z_tma, p.c.Z, p.c.ldz, row0, col, p.M, p.N, stage[c], lane);
    }
    if (have_r && !early_r) {
      stage_free(lane);
      if (p.r_tma) {
        // The buffer's last accesses were ordinary ones where no TMA store followed them.
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(rbar, kStageCBytes);
          tma_load_3d(stage[c], &tmR, rbar, col, row0, 0);
        }
        wait_copy(rbar, rphase, p.err_word);
        rphase ^= 1u;
      } else {
        stage_block(p.c.R, p.c.ldr, row0, col, p.M, p.N, stage[c], lane);
      }
    } else if (!have_r) {
      stage_free(lane);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r[16];
      F2 v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = f2(sum[c][32 * h + 2 * j], sum[c][32 * h + 2 * j + 1]);
      if (p.c.act != kActNone)
        with_act(p.c.act, [&](auto a) { act_values<decltype(a)::value>(v); });
      if (have_r) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ld_shared_v4(stage_unit(stage[c], lane, 4 * h + j), r[4 * j], r[4 * j + 1], r[4 * j + 2],
                       r[4 * j + 3]);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = add2(v[j], unpack2<kBf16>(r[j]));
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) r[j] = pack2<kBf16>(v[j]);
      stage_half(stage[c], lane, h, r);
    }
    store_block(&tmD, p.d_tma, p.c.D, p.c.ldd, row0, col, p.M, p.N, stage[c], lane);
  }
}

// The same for the gated layer: sum holds 64 columns of G, then the same ones of U.
template <bool kBf16>
__device__ __forceinline__ void block_finish_gated(const CUtensorMap &tmD, const CUtensorMap &tmG,
                                                   const CUtensorMap &tmU, const EpiArgs &p,
                                                   const uint32_t (&bias)[2], float (&sum)[2][64],
                                                   const uint32_t (&stage)[2], int row0, int col,
                                                   int lane) {
  add_bias<kBf16>(sum[0], p.c.alpha, p.c.bias != nullptr, bias[0]);
  add_bias<kBf16>(sum[1], p.c.alpha, p.c.bias2 != nullptr, bias[1]);
  stage_free(lane);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint16_t *out = which ? p.c.Z2 : p.c.Z;
    if (out == nullptr) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) 
        w[j] = pack16<kBf16>(sum[which][32 * h + 2 * j], sum[which][32 * h + 2 * j + 1]);
      stage_half(stage[which], lane, h, w);
    }
    store_block(which ? &tmU : &tmG, which ? p.r_tma : p.z_tma, out, which ? p.c.ldz2 : p.c.ldz,
                row0, col, p.M, p.N, stage[which], lane);
  }
  if (p.c.Z != nullptr) stage_free(lane);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[16];
    F2 g[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) g[j] = f2(sum[0][32 * h + 2 * j], sum[0][32 * h + 2 * j + 1]);
    with_act(p.c.act, [&](auto a) { act_values<decltype(a)::value>(g); });
#pragma unroll
    for (int j = 0; j < 16; ++j) 
      w[j] = pack2<kBf16>(mul2(g[j], f2(sum[1][32 * h + 2 * j], sum[1][32 * h + 2 * j + 1])));
    stage_half(stage[0], lane, h, w);
  }
  store_block(&tmD, p.d_tma, p.c.D, p.c.ldd, row0, col, p.M, p.N, stage[0], lane);
}

// Maps as gemm_epi_tile_kernel's.
template <int kN, bool kGated>
__global__ void __launch_bounds__(kBlockThreads, 1)
    gemm_block_tile_kernel(const __grid_constant__ CUtensorMap tmA,
                           const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmD,
                           const __grid_constant__ CUtensorMap tmZ,
                           const __grid_constant__ CUtensorMap tmR,
                           const __grid_constant__ std::conditional_t<kGated, CUtensorMap, NoMap> tmS,
                           const __grid_constant__ EpiArgs p,
                           const __grid_constant__ BlockScales sc) {
  static_assert(!kGated || kN == 256, "a warp has one block of 64 columns of D");
  constexpr int kBufs = kBlockBufs<kN>;
  constexpr int kTileCols = kGated ? kN / 2 : kN;  // of D
  constexpr int kCols = kN / 2;                    // accumulator columns of a warp
  constexpr int kChunks = kCols / 16;
  extern __shared__ uint8_t smem_raw[];
  // Same offset in both CTAs of the pair, as the pair MMA needs.
  BlockSmem<kN> &sm = *reinterpret_cast<BlockSmem<kN> *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < EpiCfg<kN, 2>::kStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_u32(&sm.tmem_full[i]), 1);
      mbar_init(smem_u32(&sm.tmem_empty[i]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&sm.drain), 1);
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(smem_u32(&sm.arrived[i]), 1);
    sm.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    if (p.d_tma) prefetch_tmap(&tmD);
    if (p.r_tma) prefetch_tmap(&tmR);
    if constexpr (kGated) prefetch_tmap(&tmS);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync();  // the leader's barriers exist before the peer signals them
  tc_fence_after_sync();
  const uint32_t tmem_base = sm.tmem_base;
  // Launched as a programmatic dependent, as gemm_epi_tile_kernel.
  grid_launch_dependents();

  if (warp < kBlockFirst) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
    if (warp == 0) {
      const CUtensorMap *b = &tmB;
      if constexpr (kGated) b = rank == 0 ? &tmB : &tmS;
      epi_produce<true, kN, false, true, 2, kGated>(tmA, *b, p, sm, rank, unit, units);
    } else if (warp == 1 && rank == 0) {
      block_multiply<kN>(p, sm, tmem_base, unit, units);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n");
    grid_dependency_wait();
    const int e = warp - kBlockFirst, quarter = warp & 3, half = e >> 2;
    const uint32_t stage[2] = {smem_u32(sm.stage[2 * e]), smem_u32(sm.stage[2 * e + 1])};
    const uint32_t rbar = smem_u32(&sm.arrived[e]);
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const bool have_r = !kGated && p.c.R != nullptr, early_r = have_r && p.c.Z == nullptr;
    const bool vec_a = scales_whole(sc.a, sc.lda), vec_b = scales_whole(sc.b, sc.ldb);
    const bool vec_b2 = kGated && scales_whole(sc.b2, sc.ldb2);
    // The warp's part of a tile: its place, the rows of its scales and the first of them.
    struct Part {
      int row0, col0;
      const float *sa, *sb, *sb2;
      float4 a, b, b2;
    };
    auto begin = [&](int t) {
      Part w;
      int tm = 0, tn = 0;
      const bool is = t < p.tiles;
      if (is) tile_coords<kEpiGroupM>(t, p.tiles_m, p.tiles_n, tm, tn);
      w.row0 = tm * 256 + static_cast<int>(rank) * kBM + quarter * 32;
      w.col0 = tn * kTileCols + half * (kTileCols / 2);
      const int64_t row = w.row0 + lane, jb = w.col0 / 128;
      w.sa = is && row < p.M ? sc.a + row * sc.lda : nullptr;
      w.sb = is && w.col0 < p.N ? sc.b + jb * sc.ldb : nullptr;
      w.sb2 = kGated && is && w.col0 < p.N ? sc.b2 + jb * sc.ldb2 : nullptr;
      w.a = load_scales(w.sa, 0, sc.KB, vec_a);
      w.b = load_scales(w.sb, 0, sc.KB, vec_b);
      w.b2 = load_scales(w.sb2, 0, sc.KB, vec_b2);
      return w;
    };
    uint32_t rphase = 0, buf = 0, use = 0;
    bool ok = true;
    Part next = begin(unit);
    for (int t = unit; t < p.tiles; t += units) {
      // (The warp reads the flag as one: its lanes must take the same branch.)
      if (__any_sync(0xffffffffu, !ok || *static_cast<volatile int *>(&sm.abort))) break;
      const Part w = next;
      // The products of four k-blocks' scales. (The factors, kept beside the next four's,
      // left the gated form too few registers: 4096 x 8192 x 4096 245 us against 224.)
      float4 s4 = scale_products(w.a, w.b), u4 = scale_products(w.a, w.b2);
      const uint32_t bias[2] = {
          load_bias(p.c.bias, w.col0 + 2 * lane, p.N),
          kGated ? load_bias(p.c.bias2, w.col0 + 2 * lane, p.N)
                 : kCols > 64 ? load_bias(p.c.bias, w.col0 + 64 + 2 * lane, p.N) : 0u};
      if (early_r) {
        stage_free(lane);
        if (p.r_tma) {
          // The buffers' last accesses were ordinary ones where no TMA store followed.
          if (!p.d_tma) {
            fence_proxy_async_shared();
            __syncwarp();
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(rbar, kCols / 64 * kStageCBytes);
#pragma unroll
            for (int c = 0; c < kCols / 64; ++c)
              tma_load_3d(stage[c], &tmR, rbar, w.col0 + 64 * c, w.row0, 0);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols / 64; ++c)
            stage_block(p.c.R, p.c.ldr, w.row0, w.col0 + 64 * c, p.M, p.N, stage[c], lane);
        }
      }
      float sum[kCols / 64][64];
#pragma unroll
      for (int j = 0; j < kCols; ++j) sum[j / 64][j % 64] = 0.f;
      for (int kb0 = 0; ok && kb0 < sc.KB; kb0 += 4) {
        const float4 an = load_scales(w.sa, kb0 + 4, sc.KB, vec_a);
        const float4 bn = load_scales(w.sb, kb0 + 4, sc.KB, vec_b);
        const float4 un = load_scales(w.sb2, kb0 + 4, sc.KB, vec_b2);
        const int left = min(sc.KB - kb0, 4);
#pragma unroll 1
        for (int i = 0; i < left; ++i) {
          const float s = pick(s4, i), s2 = kGated ? pick(u4, i) : s;
          const uint32_t full = smem_u32(&sm.tmem_full[buf]);
          if (!__all_sync(0xffffffffu, mbar_try_wait(full, use)) &&
              !mbar_wait_lazy(full, use, &sm.abort, p.err_word, kWaitTmemFull)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t taddr =
              tmem_base + lane_addr + buf * kN + half * (kTileCols / 2);
          // The next 16 columns are on their way while these are added.
          uint32_t r[2][16];
          auto column = [&](int c) {  // gated: 64 of G's columns, then 64 of U's
            return kGated && c >= kChunks / 2 ? kTileCols + 16 * (c - kChunks / 2) : 16 * c;
          };
          tmem_ld_x16(taddr + column(0), r[0]);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tmem_ld_wait();
            if (c + 1 < kChunks) {
              tmem_ld_x16(taddr + column(c + 1), r[(c + 1) & 1]);
            } else {  // all in registers: the MMAs may have it
              tc_fence_before_sync();
              __syncwarp();
              if (lane == 0) arrive_relaxed(mapa_shared(smem_u32(&sm.tmem_empty[buf]), 0));
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float &to = sum[c / 4][16 * (c % 4) + j];
              to = fmaf(__uint_as_float(r[c & 1][j]), kGated && c >= kChunks / 2 ? s2 : s, to);
            }
          }
          if (++buf == kBufs) {
            buf = 0;
            use ^= 1u;
          }
        }
        s4 = scale_products(an, bn), u4 = scale_products(an, un);
      }
      if (!ok) {
        // Never leave with a copy of R still writing into shared memory.
        if (early_r && p.r_tma) wait_copy(rbar, rphase, p.err_word);
        break;
      }
      next = begin(t + units);  // its first scales arrive during the final epilogue
      if constexpr (kGated) {
        if (p.c.bf16) {
          block_finish_gated<true>(tmD, tmZ, tmR, p, bias, sum, stage, w.row0, w.col0, lane);
        } else {
          block_finish_gated<false>(tmD, tmZ, tmR, p, bias, sum, stage, w.row0, w.col0, lane);
        }
      } else if (p.c.bf16) {
        block_finish<true, kCols / 64>(tmD, tmZ, p, bias, sum, stage, w.row0, w.col0, early_r, rbar,
                                       rphase, tmR, lane);
      } else {
        block_finish<false, kCols / 64>(tmD, tmZ, p, bias, sum, stage, w.row0, w.col0, early_r,
                                        rbar, rphase, tmR, lane);
      }
    }
    // Never leave with a TMA store still reading the staging buffers (its writes
    // are complete when the grid is).
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
  }

  tc_fence_before_sync();
  cluster_sync();  // both CTAs done: no MMA, copy or arrival targets either
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int kN, bool kGated>
cudaError_t launch_block_form(const DeviceInfo &dev, int M, int N, int K, const void *A,
                              int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                              cudaStream_t stream) {
  using Cf = EpiCfg<kN, 2>;
  constexpr int kTileCols = kGated ? kN / 2 : kN;
  static_assert(sizeof(BlockSmem<kN>) + 1024 <= 232448, "shared memory");
  const size_t smem = sizeof(BlockSmem<kN>) + 1024;
  auto kern = gemm_block_tile_kernel<kN, kGated>;
  const int pairs = pair_capacity(dev, reinterpret_cast<const void *>(kern), smem, kBlockThreads);
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  constexpr CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap tmA, tmB, tmD, tmZ, tmR;
  std::conditional_t<kGated, CUtensorMap, NoMap> tmS;
  std::memset(&tmD, 0, sizeof tmD);
  std::memset(&tmZ, 0, sizeof tmZ);
  std::memset(&tmR, 0, sizeof tmR);
  std::memset(&tmS, 0, sizeof tmS);
  if (!make_tmap(&tmA, dt, 1, A, M, K, lda, 1, 0, kBM, 128) ||
      !make_tmap(&tmB, dt, 1, B, N, K, ldb, 1, 0, Cf::kBNLoad, 128))
    return cudaErrorInvalidValue;
  EpiArgs p;
  p.M = M, p.N = N, p.K = K;
  p.tiles_m = (M - 1) / Cf::kTileM + 1;  // sizes up to 2^31 - 1
  p.tiles_n = (N - 1) / kTileCols + 1;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > 0x7fffffffLL - pairs) return cudaErrorInvalidValue;
  p.tiles = static_cast<int>(tiles);
  p.a_t = false, p.b_t = true;
  p.d_tma = out_tmap(&tmD, epi.bf16, epi.D, epi.ldd, M, N);
  p.z_tma = out_tmap(&tmZ, epi.bf16, epi.Z, epi.ldz, M, N);
  if constexpr (kGated) {
    if (!make_tmap(&tmS, dt, 1, epi.B2, N, K, epi.ldb2, 1, 0, Cf::kBNLoad, 128))
      return cudaErrorInvalidValue;
    p.r_tma = out_tmap(&tmR, epi.bf16, epi.Z2, epi.ldz2, M, N);
  } else {
    p.r_tma = block_tmap(&tmR, epi.bf16, epi.R, epi.ldr, M, N);
  }
  p.s_tma = false;
  p.idesc = idesc_mma(0u, false, false, Cf::kTileM, kN);
  p.err_word = dev.err_word;
  p.part = nullptr, p.part_apart = 0;
  p.loop_ns = kWaitLimitNs;  // (not used: every k-block has an accumulator of its own)
  p.c = epi;
  const BlockScales sc{epi.block_a, epi.block_b,  epi.block_b2,     epi.ldsa,
                       epi.ldsb,    epi.ldsb2, (K - 1) / 128 + 1};
  const int units = static_cast<int>(tiles < pairs ? tiles : pairs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(units), 1, 1);
  cfg.blockDim = dim3(kBlockThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmA, tmB, tmD, tmZ, tmR, tmS, p, sc);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace
}  // namespace dgr
