// gemm_epi_tile.cuh -- the tensor-core product with a fused epilogue on
// 256-row tiles, shared by the translation units that instantiate it:
//
//   forward   Z = alpha op(A) op(B) scale_a_i scale_b_j + bias_j,  D = act(Z) + R
//   gradient  D = alpha op(A) op(B) act'(Zin), column sums of D
//
// 16-bit operands (kind::f16) or e4m3 (kind::f8f6f4: twice the k per MMA, the
// same bytes per stage), fp32 accumulation in tensor memory, 16-bit results.
//
// A CTA pair (cta_group::2) owns a 256 x kBN tile; persistent, ten warps per CTA:
//   warp 0      TMA producer: 128 rows of A and kBN / 2 columns of B per CTA and
//               stage, 128 bytes of k (64 16-bit or 128 8-bit values)
//   warp 1      the leader's issues the pair's MMAs into one of two
//               accumulators, so a tile's epilogue overlaps the next main loop
//   warps 2..9  epilogue: each owns 32 rows x kBN / 2 columns, in units of 64
//               columns (one 128-byte row of 16-bit output per lane)
//
// The operand forms differ in the producer's boxes and the MMA's descriptors
// only, so both loops are compiled for each form inside one kernel (a branch per
// kernel, none per k-block) and the epilogue, most of the code, is shared.
//
// Epilogue data: the tile's bias and column scales are put in shared memory once
// per tile (read back as broadcasts); R or Zin comes by TMA into the warp's 4 KiB
// buffer, requested before the accumulator is waited for; results are packed and
// staged in the same buffer in the layout of a 128-byte swizzle and stored by
// TMA. (R read straight from global memory, a row per lane, cost 2.3 us per unit
// in L1 lookups, which showed for short k. Blocks of 32 columns with two half
// buffers, R a block ahead, were slower: twice the fences and stores.) Matrices that TMA cannot address (rows not
// in whole 16-byte units) go through the same buffer with coalesced 2-byte
// accesses, a row of 64 columns per two warp instructions: a lane per row would
// touch 32 rows per instruction.
//
// Column sums (gradient): a lane holds one row of 32 columns; five halving
// exchanges (16 + 8 + 4 + 2 + 1 shuffles) leave the sum over the warp's 32 rows
// of column l in lane l, which goes to partial row (row / 32); col_sums adds the
// partial rows. No atomics: the same bits on every call.
#pragma once

#include "epi.cuh"
#include "gemm_tc_kernel.cuh"
#include "tc_issue.cuh"

namespace dgr {
namespace {

__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int kN>
struct EpiCfg {
  static constexpr int kTileM = 256;
  static constexpr int kBNLoad = kN / 2;             // B columns staged per CTA
  static constexpr int kStages = kN == 256 ? 6 : 8;  // 192 KiB
  static constexpr uint32_t kABytes = kBM * kRowBytes;
  static constexpr uint32_t kBBytes = kBNLoad * kRowBytes;
  static constexpr uint32_t kTxBytes = 2 * (kABytes + kBBytes);  // both CTAs, one phase
  static constexpr uint32_t kTmem = 2 * kN;                      // two accumulators
};

template <int kN>
struct __align__(1024) EpiSmem {
  uint8_t a[EpiCfg<kN>::kStages][EpiCfg<kN>::kABytes];
  uint8_t b[EpiCfg<kN>::kStages][EpiCfg<kN>::kBBytes];
  uint8_t stage[kEpiWarps][kStageCBytes];
  uint16_t bias[kN];  // the tile's bias (as stored) and column scales
  float scale[kN];
  uint64_t full[EpiCfg<kN>::kStages];
  uint64_t empty[EpiCfg<kN>::kStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t arrived[kEpiWarps];  // R is in a warp's buffer
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

struct EpiArgs {
  int M, N, K;
  int tiles_m, tiles_n, tiles;
  bool a_t, b_t;
  bool d_tma, z_tma;  // D / Z written through their tensor maps
  bool r_tma;         // R (Zin) read through its tensor map
  uint32_t idesc;
  uint32_t *err_word;
  float *part;        // gradient: partial column sums [ceil(M / 32)][N], or null
  EpiCall c;
};

// Shared-memory address of 16-byte unit u of row `lane` in a staging buffer.
__device__ __forceinline__ uint32_t stage_unit(uint32_t stage, int row, int u) {
  return stage + static_cast<uint32_t>(row) * 128u + (static_cast<uint32_t>(u ^ (row & 7)) << 4);
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c,
                                             uint32_t &d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
// The 16-bit value at column j (0..63) of a staged row.
__device__ __forceinline__ uint32_t stage_elem(uint32_t stage, int row, int j) {
  return stage_unit(stage, row, j >> 3) + static_cast<uint32_t>(j & 7) * 2u;
}

// The lane's row of a staged block, packed.
__device__ __forceinline__ void read_staged(uint32_t stage, int lane, uint32_t (&w)[32]) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    ld_shared_v4(stage_unit(stage, lane, u), w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
}
// Stages 32 rows x 64 columns of a matrix that TMA cannot read, row by row,
// coalesced; zeros outside it.
__device__ __forceinline__ void stage_block(const uint16_t *p, int64_t ld, int row0, int col,
                                            int M, int N, uint32_t stage, int lane) {
  // 16 rows' loads (two per lane) are in flight together.
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 16) {
    uint16_t v[16][2];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint16_t *q = p + (row0 + r0 + i) * ld + col + lane;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[i][h] = row0 + r0 + i < M && col + lane + 32 * h < N ? q[32 * h] : 0;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(stage_elem(stage, r0 + i, lane + 32 * h)),
                     "h"(v[i][h])
                     : "memory");
  }
  __syncwarp();
}

// Waits (bounded) for a copy of R that is in flight, whatever else has failed.
__device__ __forceinline__ void wait_copy(uint32_t bar, uint32_t parity, uint32_t *err_word) {
  volatile int never = 0;
  mbar_wait_lazy(bar, parity, &never, err_word, kWaitDrain);
}

// The staging buffer's three steps: wait until the last store has left it, put
// 32 columns of the lane's row (half h of 64) into it, and write the block of 32
// rows x 64 columns, by TMA or by coalesced 2-byte stores.
__device__ __forceinline__ void stage_free(int lane) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
}
__device__ __forceinline__ void stage_half(uint32_t stage, int lane, int h,
                                           const uint32_t (&w)[16]) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    st_shared_v4(stage_unit(stage, lane, 4 * h + u), w[4 * u], w[4 * u + 1], w[4 * u + 2],
                 w[4 * u + 3]);
}
__device__ __forceinline__ void store_block(const void *tm, bool tma, uint16_t *p, int64_t ld,
                                            int row0, int col, int M, int N, uint32_t stage,
                                            int lane) {
  if (tma) {
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0 && col < N && row0 < M) {
      tma_store_3d(tm, col, row0, 0, stage);
      bulk_commit();
    }
    __syncwarp();  // the next accumulator load needs the warp converged
  } else {
    __syncwarp();
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      uint16_t *q = p + (row0 + r) * ld + col + lane;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(stage_elem(stage, r, lane + 32 * h))
                     : "memory");
        if (row0 + r < M && col + lane + 32 * h < N) q[32 * h] = v;
      }
    }
    __syncwarp();
  }
}

// Sums v[0..31] over the warp's lanes: lane l returns the sum of v[l].
__device__ __forceinline__ float warp_column_sums(float (&v)[32], int lane) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float give = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, s);
    }
  }
  return v[0];
}

// z of 32 columns of one row from the accumulator (forward), in pairs.
template <bool kE4m3, bool kBf16>
__device__ __forceinline__ void epi_preact(const uint16_t *bias, const float *scale,
                                           float row_scale, const uint32_t (&acc)[32],
                                           F2 (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    const uint4 q = *reinterpret_cast<const uint4 *>(bias + 2 * j);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      F2 s = f2(row_scale);
      if constexpr (kE4m3) {
        const float2 c = *reinterpret_cast<const float2 *>(scale + 2 * (j + h));
        s = mul2(s, f2(c.x, c.y));
      }
      v[j + h] = fma2(f2(__uint_as_float(acc[2 * (j + h)]), __uint_as_float(acc[2 * (j + h) + 1])),
                      s, unpack2<kBf16>(w[h]));
    }
  }
}

// Tile rows per raster group. Sustained loops at 4096 x 16384 x 4096, 8192^3 e4m3
// and 8192 x 8192 x 4096 (gradient): 4 rows 354 / 368 / 370 us, 8 rows 341 / 358 /
// 356 us, 16 rows 337 / 357 / 350 us.
constexpr int kEpiGroupM = 16;

// The producer's loop for one operand form.
template <bool kE4m3, int kN, bool kAT, bool kBT>
__device__ __forceinline__ void epi_produce(const CUtensorMap &tmA, const CUtensorMap &tmB,
                                            const EpiArgs &p, EpiSmem<kN> &sm, uint32_t rank,
                                            int unit, int units) {
  using Cf = EpiCfg<kN>;
  constexpr int kBK = kE4m3 ? 128 : 64;
  constexpr uint32_t kMNBoxBytes = kRowBytes * 64;  // 64 rows of k x 64 16-bit values
  volatile int *abort = &sm.abort;
  const uint64_t keep = l2_policy_evict_last();
  const int KB = (p.K - 1) / kBK + 1;
  uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
  bool ok = true;
  for (int t = unit; ok && t < p.tiles; t += units) {
    int tm, tn;
    tile_coords<kEpiGroupM>(t, p.tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * Cf::kTileM + static_cast<int>(rank) * kBM;
    const int n0 = tn * kN + static_cast<int>(rank) * Cf::kBNLoad;
    for (int kb = 0; kb < KB; ++kb) {
      if (!mbar_wait_lazy(smem_u32(&sm.empty[stage]), phase ^ 1u, abort, p.err_word,
                          kWaitEmpty)) {
        ok = false;
        break;
      }
      if (issued == 0) grid_dependency_wait();
      if (elect_one()) {
        const uint32_t full_bar = smem_u32(&sm.full[stage]);
        if (rank == 0) mbar_arrive_expect_tx(full_bar, Cf::kTxBytes);
        const uint32_t bar = mapa_shared(full_bar, 0);
        const int k0 = kb * kBK;
        if constexpr (!kAT) {
          tma_load_3d_pair_hint(smem_u32(sm.a[stage]), &tmA, bar, k0, m0, 0, keep);
        } else {
#pragma unroll
          for (int j = 0; j < kBM / 64; ++j)
            tma_load_3d_pair_hint(smem_u32(sm.a[stage] + j * kMNBoxBytes), &tmA, bar, m0 + 64 * j,
                                  k0, 0, keep);
        }
        if constexpr (!kBT) {
#pragma unroll
          for (int j = 0; j < Cf::kBNLoad / 64; ++j)
            tma_load_3d_pair(smem_u32(sm.b[stage] + j * kMNBoxBytes), &tmB, bar, n0 + 64 * j, k0,
                             0);
        } else {
          tma_load_3d_pair(smem_u32(sm.b[stage]), &tmB, bar, k0, n0, 0);
        }
      }
      __syncwarp();
      issued |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == Cf::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  // Never leave with a copy still writing into shared memory (the leader's full
  // barriers count both CTAs' bytes; the peer is held at the last cluster barrier).
  if (rank == 0)
    for (int s = 0; s < Cf::kStages; ++s)
      if (issued & (1u << s))
        drain_wait(smem_u32(&sm.full[s]), (issued_parity >> s) & 1u, p.err_word);
}

// The leader's MMA loop for one operand form.
template <bool kE4m3, int kN, bool kAT, bool kBT>
__device__ __forceinline__ void epi_multiply(const EpiArgs &p, EpiSmem<kN> &sm,
                                             uint32_t tmem_base, int unit, int units) {
  using Cf = EpiCfg<kN>;
  constexpr int kBK = kE4m3 ? 128 : 64;
  constexpr uint32_t kMNBoxBytes = kRowBytes * 64;
  constexpr uint32_t kMNStep = kRowBytes * 16;  // 16 rows of k
  volatile int *abort = &sm.abort;
  const int KB = (p.K - 1) / kBK + 1;
  // K-major: SBO = one 8-row swizzle atom, the next MMA 32 bytes along the row.
  // MN-major (16-bit only): LBO = one 64-value box, the next MMA 16 k-rows on.
  const uint64_t adesc0 =
      smem_desc(smem_u32(sm.a[0]), kAT ? kMNBoxBytes : 16, kAtomBytes, 2u);
  const uint64_t bdesc0 =
      smem_desc(smem_u32(sm.b[0]), kBT ? 16 : kMNBoxBytes, kAtomBytes, 2u);
  constexpr uint32_t kAStage = Cf::kABytes >> 4, kBStage = Cf::kBBytes >> 4;
  constexpr uint32_t kAStep = (kAT ? kMNStep : 32u) >> 4, kBStep = (kBT ? 32u : kMNStep) >> 4;
  uint32_t stage = 0, phase = 0, n = 0;
  bool ok = true, any = false;
  for (int t = unit; ok && t < p.tiles; t += units, ++n) {
    const uint32_t buf = n & 1u, use = (n >> 1) & 1u;
    if (!mbar_wait_lazy<true>(smem_u32(&sm.tmem_empty[buf]), use ^ 1u, abort, p.err_word,
                              kWaitTmemEmpty))
      break;
    tc_fence_after_sync();
    const uint32_t d_tmem = tmem_base + buf * kN;
    for (int kb = 0; kb < KB; ++kb) {
      if (!mbar_wait_lazy(smem_u32(&sm.full[stage]), phase, abort, p.err_word, kWaitFull)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint64_t ad = adesc0 + stage * kAStage, bd = bdesc0 + stage * kBStage;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t acc = kk > 0 || kb > 0 ? 1u : 0u;
          if constexpr (kE4m3) {
            tc_mma_f8_pair(d_tmem, ad + kk * kAStep, bd + kk * kBStep, p.idesc, acc);
          } else {
            tc_mma_f16_pair(d_tmem, ad + kk * kAStep, bd + kk * kBStep, p.idesc, acc);
          }
        }
        tc_commit_pair_mc(smem_u32(&sm.empty[stage]), 0x3);
        if (kb == KB - 1) tc_commit_pair_mc(smem_u32(&sm.tmem_full[buf]), 0x3);
      }
      __syncwarp();
      any = true;
      if (++stage == Cf::kStages) {
        stage = 0;
        phase ^= 1u;
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

// One tile's epilogue by one warp (32 rows x kN / 2 columns).
template <bool kE4m3, bool kGrad, bool kBf16, int kN>
__device__ __forceinline__ void epi_tile(const CUtensorMap &tmD, const CUtensorMap &tmZ,
                                         const CUtensorMap &tmR, const EpiArgs &p,
                                         EpiSmem<kN> &sm, uint32_t tmem_base, uint32_t n, int tm,
                                         int tn, uint32_t rank, int warp, int lane,
                                         uint32_t &rphase, bool &ok) {
  const int e = warp - 2, quarter = warp & 3, half = e >> 2;
  const uint32_t stage = smem_u32(sm.stage[e]);
  const uint32_t buf = n & 1u, use = (n >> 1) & 1u;
  volatile int *abort = &sm.abort;
  const int row0 = tm * EpiCfg<kN>::kTileM + static_cast<int>(rank) * kBM + quarter * 32;
  const int row = row0 + lane;
  const int local0 = half * (kN / 2), col0 = tn * kN + local0;
  if constexpr (!kGrad) {
    epilogue_sync();  // every warp has read the previous tile's
    for (int i = threadIdx.x - 64; i < kN; i += 32 * kEpiWarps) {
      const int col = tn * kN + i;
      sm.bias[i] = p.c.bias && col < p.N ? p.c.bias[col] : 0;
      if constexpr (kE4m3) sm.scale[i] = p.c.scale_b && col < p.N ? p.c.scale_b[col] : 1.f;
    }
    epilogue_sync();
  }
  float row_scale = p.c.alpha;
  if (kE4m3 && p.c.scale_a && row < p.M) row_scale *= p.c.scale_a[row];
  uint32_t r[32];
  const bool have_r = p.c.R != nullptr;
  // Requests the unit's R into the staging buffer, and takes it from there.
  const uint32_t rbar = smem_u32(&sm.arrived[e]);
  auto request_r = [&](int col) {
    stage_free(lane);
    if (p.r_tma) {
      // The buffer's last accesses were ordinary ones where no TMA store followed them.
      if (!p.d_tma) {
        fence_proxy_async_shared();
        __syncwarp();
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(rbar, kStageCBytes);
        tma_load_3d(stage, &tmR, rbar, col, row0, 0);
      }
    } else {
      stage_block(p.c.R, p.c.ldr, row0, col, p.M, p.N, stage, lane);
    }
  };
  auto take_r = [&] {
    if (p.r_tma) {
      wait_copy(rbar, rphase, p.err_word);
      rphase ^= 1u;
    }
    read_staged(stage, lane, r);
    __syncwarp();
  };
  if (have_r) request_r(col0);
  const bool got = mbar_wait_lazy(smem_u32(&sm.tmem_full[buf]), use, abort, p.err_word,
                                  kWaitTmemFull);
  if (have_r) take_r();
  if (!got) {
    ok = false;
    return;
  }
  tc_fence_after_sync();
  const uint32_t taddr =
      tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kN + local0;
#pragma unroll 1
  for (int c = 0; c < kN / 2; c += 64) {
    if (!kGrad && p.c.Z != nullptr) {
      stage_free(lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t acc[32], w[16];
        F2 v[16];
        tmem_ld_32x32b_x32(taddr + c + 32 * h, acc);
        tmem_ld_wait();
        epi_preact<kE4m3, kBf16>(&sm.bias[local0 + c + 32 * h], &sm.scale[local0 + c + 32 * h],
                                 row_scale, acc, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack2<kBf16>(v[j]);
        stage_half(stage, lane, h, w);
      }
      store_block(&tmZ, p.z_tma, p.c.Z, p.c.ldz, row0, col0 + c, p.M, p.N, stage, lane);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t acc[32], w[16];
      F2 v[16];
      tmem_ld_32x32b_x32(taddr + c + 32 * h, acc);
      tmem_ld_wait();
      if (c + 32 * h + 32 == kN / 2) {  // all in registers: the next tile may have it
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sm.tmem_empty[buf]), 0));
      }
      if constexpr (!kGrad) {
        epi_preact<kE4m3, kBf16>(&sm.bias[local0 + c + 32 * h], &sm.scale[local0 + c + 32 * h],
                                 row_scale, acc, v);
        with_act(p.c.act, [&](auto a) { act_values<decltype(a)::value>(v); });
        if (have_r) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = add2(v[j], unpack2<kBf16>(r[16 * h + j]));
        }
      } else {
        with_act(p.c.act, [&](auto a) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float lo = 0.f, hi = 0.f;
            if constexpr (decltype(a)::value != kActNone) unpack16<kBf16>(r[16 * h + j], lo, hi);
            const F2 d = mul2(f2(__uint_as_float(acc[2 * j]), __uint_as_float(acc[2 * j + 1])),
                              f2(row_scale));
            v[j] = mul2(d, act_slope2<decltype(a)::value>(lo, hi));
          }
        });
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = pack2<kBf16>(v[j]);
      if (h == 0) stage_free(lane);
      stage_half(stage, lane, h, w);
      if constexpr (kGrad) {
        // Rows beyond M are left out: they hold 0 * B, NaN where B is not finite.
        if (p.part != nullptr && row0 < p.M) {
          float u[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) split(v[j], u[2 * j], u[2 * j + 1]);
          if (row >= p.M) {
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = 0.f;
          }
          const float s = warp_column_sums(u, lane);
          const int col = col0 + c + 32 * h + lane;
          if (col < p.N) p.part[static_cast<int64_t>(row0 / 32) * p.N + col] = s;
        }
      }
    }
    store_block(&tmD, p.d_tma, p.c.D, p.c.ldd, row0, col0 + c, p.M, p.N, stage, lane);
    if (have_r && c + 64 < kN / 2) {
      request_r(col0 + c + 64);
      take_r();
    }
  }
}

template <bool kE4m3, int kN, bool kGrad>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_epi_tile_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmD,
                         const __grid_constant__ CUtensorMap tmZ,
                         const __grid_constant__ CUtensorMap tmR,
                         const __grid_constant__ EpiArgs p) {
  using Cf = EpiCfg<kN>;
  extern __shared__ uint8_t smem_raw[];
  // Same offset in both CTAs of the pair, as the pair MMA needs.
  EpiSmem<kN> &sm = *reinterpret_cast<EpiSmem<kN> *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cf::kStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
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
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sm.tmem_base), Cf::kTmem);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync();  // the leader's barriers exist before the peer signals them
  tc_fence_after_sync();
  const uint32_t tmem_base = sm.tmem_base;
  // Launched as a programmatic dependent: the set-up overlaps the previous
  // kernel's tail. Each role that touches global memory waits for that kernel
  // just before it does, with its loop's code already fetched.
  grid_launch_dependents();

  if (warp == 0) {
    if constexpr (kE4m3) {
      epi_produce<true, kN, false, true>(tmA, tmB, p, sm, rank, unit, units);
    } else if (p.a_t) {
      if (p.b_t) {
        epi_produce<false, kN, true, true>(tmA, tmB, p, sm, rank, unit, units);
      } else {
        epi_produce<false, kN, true, false>(tmA, tmB, p, sm, rank, unit, units);
      }
    } else if (p.b_t) {
      epi_produce<false, kN, false, true>(tmA, tmB, p, sm, rank, unit, units);
    } else {
      epi_produce<false, kN, false, false>(tmA, tmB, p, sm, rank, unit, units);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      if constexpr (kE4m3) {
        epi_multiply<true, kN, false, true>(p, sm, tmem_base, unit, units);
      } else if (p.a_t) {
        if (p.b_t) {
          epi_multiply<false, kN, true, true>(p, sm, tmem_base, unit, units);
        } else {
          epi_multiply<false, kN, true, false>(p, sm, tmem_base, unit, units);
        }
      } else if (p.b_t) {
        epi_multiply<false, kN, false, true>(p, sm, tmem_base, unit, units);
      } else {
        epi_multiply<false, kN, false, false>(p, sm, tmem_base, unit, units);
      }
    }
    __syncwarp();
  } else {
    // Every epilogue warp walks the same tiles and meets the same named
    // barriers; after a wait that gave up it skips the work, not the barriers.
    grid_dependency_wait();
    bool ok = true;
    uint32_t n = 0, rphase = 0;
    for (int t = unit; t < p.tiles; t += units, ++n) {
      int tm, tn;
      tile_coords<kEpiGroupM>(t, p.tiles_m, p.tiles_n, tm, tn);
      // (The warp reads the flag as one: its lanes must take the same branch.)
      if (__any_sync(0xffffffffu, !ok || *static_cast<volatile int *>(&sm.abort))) {
        ok = false;
        if constexpr (!kGrad) {
          epilogue_sync();
          epilogue_sync();
        }
        continue;
      }
      if (p.c.bf16) {
        epi_tile<kE4m3, kGrad, true, kN>(tmD, tmZ, tmR, p, sm, tmem_base, n, tm, tn, rank, warp,
                                          lane, rphase, ok);
      } else {
        epi_tile<kE4m3, kGrad, false, kN>(tmD, tmZ, tmR, p, sm, tmem_base, n, tm, tn, rank, warp,
                                          lane, rphase, ok);
      }
    }
    // Never leave with a TMA store still reading the staging buffer (its writes
    // are complete when the grid is).
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
  }

  tc_fence_before_sync();
  cluster_sync();  // both CTAs done: no MMA, copy or arrival targets either
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, Cf::kTmem);
  }
}

// A 16-bit matrix as a tensor map of 32 x 64 blocks, where TMA can address it
// (16-byte aligned rows). An output's rows also have to be whole 16-byte units
// long: a store box is clipped at the right edge in such units only.
inline bool block_tmap(CUtensorMap *tm, bool bf16, const uint16_t *p, int64_t ld, int M, int N) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 &&
         make_tmap(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                   p, M, N, ld, 1, 0, 32, 64, false);
}
inline bool out_tmap(CUtensorMap *tm, bool bf16, const uint16_t *p, int64_t ld, int M, int N) {
  return N % 8 == 0 && block_tmap(tm, bf16, p, ld, M, N);
}

template <bool kE4m3, int kN, bool kGrad>
cudaError_t launch_epi_tile(const DeviceInfo &dev, bool a_t, bool b_t, int M, int N, int K,
                            const void *A, int64_t lda, const void *B, int64_t ldb,
                            const EpiCall &epi, float *part, cudaStream_t stream) {
  using Cf = EpiCfg<kN>;
  constexpr int kEs = kE4m3 ? 1 : 2, kBK = kE4m3 ? 128 : 64;
  static_assert(sizeof(EpiSmem<kN>) + 1024 <= 232448, "shared memory");
  const size_t smem = sizeof(EpiSmem<kN>) + 1024;
  auto kern = gemm_epi_tile_kernel<kE4m3, kN, kGrad>;
  const int pairs = pair_capacity(dev, reinterpret_cast<const void *>(kern), smem);
  if (pairs < 1) return cudaErrorInvalidConfiguration;

  const CUtensorMapDataType dt = kE4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : epi.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap tmA, tmB, tmD, tmZ, tmR;
  std::memset(&tmD, 0, sizeof tmD);
  std::memset(&tmZ, 0, sizeof tmZ);
  std::memset(&tmR, 0, sizeof tmR);
  if (!(a_t ? make_tmap(&tmA, dt, kEs, A, K, M, lda, 1, 0, 64, 64)
            : make_tmap(&tmA, dt, kEs, A, M, K, lda, 1, 0, kBM, kBK)) ||
      !(b_t ? make_tmap(&tmB, dt, kEs, B, N, K, ldb, 1, 0, Cf::kBNLoad, kBK)
            : make_tmap(&tmB, dt, kEs, B, K, N, ldb, 1, 0, 64, 64)))
    return cudaErrorInvalidValue;
  EpiArgs p;
  p.M = M, p.N = N, p.K = K;
  p.tiles_m = (M - 1) / Cf::kTileM + 1;  // sizes up to 2^31 - 1
  p.tiles_n = (N - 1) / kN + 1;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > 0x7fffffffLL - pairs) return cudaErrorInvalidValue;
  p.tiles = static_cast<int>(tiles);
  p.a_t = a_t, p.b_t = b_t;
  p.d_tma = out_tmap(&tmD, epi.bf16, epi.D, epi.ldd, M, N);
  p.z_tma = out_tmap(&tmZ, epi.bf16, epi.Z, epi.ldz, M, N);
  p.r_tma = block_tmap(&tmR, epi.bf16, epi.R, epi.ldr, M, N);
  p.idesc = idesc_mma(kE4m3 || !epi.bf16 ? 0u : kFmtBF16, a_t, !b_t, Cf::kTileM, kN);
  p.err_word = dev.err_word;
  p.part = part;
  p.c = epi;
  const int units = static_cast<int>(tiles < pairs ? tiles : pairs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(units), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmA, tmB, tmD, tmZ, tmR, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace
}  // namespace dgr
