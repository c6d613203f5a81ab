// gemm_epi_split.cuh -- the product with a fused epilogue for few rows: problems
// whose 256-row tiles would not fill the GPU, down to one token.
//
// Such a product is bound by reading the weights B once, so every SM has to
// stream its share of them. The transposed product D^T = op(B)^T A^T is formed:
// 128 columns of D fill the MMA's rows and up to kMP rows of D (tokens) its N,
// and the k range of a 128 x kMP tile is cut into `cl` parts, one per CTA of a
// thread-block cluster. Each CTA streams its part (a TMA warp, a ring of
// 128-byte-k stages, one MMA thread, the accumulator in tensor memory), writes
// its fp32 partial sums to its own shared memory, and after a cluster barrier
// CTA r adds the cl partials of 128 / cl columns in CTA order through
// distributed shared memory and applies the epilogue. One launch, no workspace,
// no atomics, the same bits on every call. Two CTAs share an SM, so one's
// stream covers the other's start and tail.
//
// Operands: A (tokens) as stored M x K; B stored N x K (K-major) or K x N
// (N-major, 16-bit only); 16-bit or e4m3.
#pragma once

#include "epi.cuh"
#include "gemm_tc_kernel.cuh"
#include "tc_issue.cuh"

namespace dgr {
namespace {

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

constexpr int kSplitThreads = 192;  // TMA warp, MMA warp, four warps that drain TMEM
constexpr int kSplitFinish = 128;  // threads that add and finish: those four warps
constexpr int kSplitN = 128;        // columns of D per tile (the MMA's M)
constexpr int kSplitMaxCl = 8;      // portable cluster size
constexpr int kSplitCtasPerSm = 2;

template <int kMP>
struct SplitCfg {
  static constexpr uint32_t kBBytes = kSplitN * kRowBytes;
  static constexpr uint32_t kABytes = kMP * kRowBytes;
  static constexpr int kStages = kMP == 16 ? 6 : kMP == 32 ? 5 : kMP == 64 ? 4 : 3;
  static constexpr uint32_t kTmem = kMP < 32 ? 32 : kMP;
};

template <int kMP>
struct __align__(1024) SplitSmem {
  uint8_t b[SplitCfg<kMP>::kStages][SplitCfg<kMP>::kBBytes];  // also the partial sums
  uint8_t a[SplitCfg<kMP>::kStages][SplitCfg<kMP>::kABytes];
  uint64_t full[SplitCfg<kMP>::kStages];
  uint64_t empty[SplitCfg<kMP>::kStages];
  uint64_t done;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

struct SplitArgs {
  int M, N, K;
  int mp;       // rows of a token tile: min(M, kMP) rounded up to 16 (the MMA's N)
  int tiles_m;
  int cl;
  bool b_t;     // B stored N x K
  bool r_vec, d_vec, z_vec;  // rows of R / D / Z in whole 8-byte units
  uint32_t idesc;
  uint32_t *err_word;
  float *part;  // gradient, several token tiles: column sums of each [tiles_m][N]
  EpiCall c;
};

// Four consecutive 16-bit values, packed; n is how many of them exist.
__device__ __forceinline__ uint2 load4(const uint16_t *p, bool vec, int n) {
  if (vec && n >= 4) return *reinterpret_cast<const uint2 *>(p);
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = e < n ? p[e] : 0;
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
__device__ __forceinline__ void store4(uint16_t *p, bool vec, int n, uint2 v) {
  if (vec && n >= 4) {
    *reinterpret_cast<uint2 *>(p) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = static_cast<uint16_t>((e < 2 ? v.x : v.y) >> (16 * (e & 1)));
  }
}

// What one finishing thread needs besides the sums: its four columns' bias and
// scales and one row's R and scale, as stored. Loaded before the accumulator is
// waited for, so the loads' latency is off the tail.
struct SplitCols {
  uint32_t bias[4];
  float scale[4];
};
struct SplitRow {
  uint2 r;
  float scale;
};
template <bool kGrad>
__device__ __forceinline__ void split_load_cols(const SplitArgs &p, int col, SplitCols &k) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    k.bias[e] = !kGrad && p.c.bias && col + e < p.N ? p.c.bias[col + e] : 0;
    k.scale[e] = !kGrad && p.c.scale_b && col + e < p.N ? p.c.scale_b[col + e] : 1.f;
  }
}
template <bool kGrad>
__device__ __forceinline__ void split_load_row(const SplitArgs &p, int64_t row, int col,
                                               SplitRow &k) {
  k.r = make_uint2(0, 0);
  k.scale = 1.f;
  if (row >= p.M || col >= p.N) return;
  if (p.c.R) k.r = load4(p.c.R + row * p.c.ldr + col, p.r_vec, p.N - col);
  if (!kGrad && p.c.scale_a) k.scale = p.c.scale_a[row];
}

// Adds the partial sums of this CTA's columns over the cluster and writes them.
// Thread t of kSplitFinish owns four columns and rows t / wq, + kSplitFinish / wq ...
template <bool kGrad, bool kBf16, int kAct>
__device__ __forceinline__ void split_finish(const SplitArgs &p, uint32_t red, int t, int lc,
                                             int m0, int col, const SplitCols &cols,
                                             SplitRow next, float (&sum)[4]) {
  const int wq = kSplitN / p.cl / 4, step = kSplitFinish / wq;
  const int rows = min(p.M - m0, p.mp), left = p.N - col;
  if (left <= 0) return;
  for (int m = t / wq; m < rows; m += step) {
    const int64_t row = m0 + m;
    const SplitRow now = next;
    const uint32_t off = red + static_cast<uint32_t>((m * kSplitN + lc) * 4);
    float4 s[kSplitMaxCl];
#pragma unroll
    for (int q = 0; q < kSplitMaxCl; ++q)
      if (q < p.cl) s[q] = ld_dsmem_f4(mapa_shared(off, static_cast<uint32_t>(q)));
    if (m + step < rows) split_load_row<kGrad>(p, row + step, col, next);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < kSplitMaxCl; ++q)  // CTA order: one fixed order per element
      if (q < p.cl) v[0] += s[q].x, v[1] += s[q].y, v[2] += s[q].z, v[3] += s[q].w;
    float r[4];
    unpack16<kBf16>(now.r.x, r[0], r[1]);
    unpack16<kBf16>(now.r.y, r[2], r[3]);
    const float sa = p.c.alpha * now.scale;
    if constexpr (!kGrad) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = fmaf(v[e] * sa, cols.scale[e], from16<kBf16>(cols.bias[e]));
      if (p.c.Z)
        store4(p.c.Z + row * p.c.ldz + col, p.z_vec, left,
               make_uint2(pack16<kBf16>(v[0], v[1]), pack16<kBf16>(v[2], v[3])));
#pragma unroll
      for (int e = 0; e < 4; e += 2) split(act_value2<kAct>(f2(v[e], v[e + 1])), v[e], v[e + 1]);
      if (p.c.R) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += r[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; e += 2)
        split(mul2(mul2(f2(v[e], v[e + 1]), f2(sa)), act_slope2<kAct>(r[e], r[e + 1])), v[e],
              v[e + 1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += v[e];
    }
    store4(p.c.D + row * p.c.ldd + col, p.d_vec, left,
           make_uint2(pack16<kBf16>(v[0], v[1]), pack16<kBf16>(v[2], v[3])));
  }
}

template <bool kE4m3, int kMP, bool kGrad>
__global__ void __launch_bounds__(kSplitThreads, kSplitCtasPerSm)
    gemm_epi_split_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ SplitArgs p) {
  using Cf = SplitCfg<kMP>;
  constexpr int kBK = kE4m3 ? 128 : 64;
  extern __shared__ uint8_t smem_raw[];
  SplitSmem<kMP> &sm = *reinterpret_cast<SplitSmem<kMP> *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  volatile int *abort = &sm.abort;
  const int cl = p.cl;
  const int rank = cl > 1 ? static_cast<int>(cluster_ctarank()) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cf::kStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    mbar_init(smem_u32(&sm.done), 1);
    mbar_init(smem_u32(&sm.drain), 1);
    sm.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), Cf::kTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = sm.tmem_base;
  // Launched as a programmatic dependent: the set-up overlaps the previous
  // kernel's tail. Each role that touches global memory waits for that kernel
  // just before it does, with its loop's code already fetched.
  grid_launch_dependents();

  // Token tiles of one column block are neighbours, so its weights are read
  // from memory once and found in L2 by the others.
  const int tile = static_cast<int>(blockIdx.x) / cl;
  const int n0 = tile / p.tiles_m * kSplitN, m0 = tile % p.tiles_m * kMP;
  const int KB = (p.K - 1) / kBK + 1;
  const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * KB / cl);
  const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * KB / cl);

  // Finishing threads: t owns columns lc .. lc + 3 of the tile (wq divides the
  // thread count, so they stay the same from row to row).
  const int W = kSplitN / cl, wq = W / 4;
  const int t = static_cast<int>(threadIdx.x) - 64;
  const int lc = rank * W + (t & (wq - 1)) * 4, col = n0 + lc;
  SplitCols cols;
  SplitRow first;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t bytes = Cf::kBBytes + static_cast<uint32_t>(p.mp) * kRowBytes;
    uint32_t stage = 0, phase = 0, issued = 0, issued_parity = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_lazy(smem_u32(&sm.empty[stage]), phase ^ 1u, abort, p.err_word, kWaitEmpty))
        break;
      if (kb == kb0) grid_dependency_wait();
      if (elect_one()) {
        const uint32_t bar = smem_u32(&sm.full[stage]);
        mbar_arrive_expect_tx(bar, bytes);
        const int k0 = kb * kBK;
        if (kE4m3 || p.b_t) {
          tma_load_3d(smem_u32(sm.b[stage]), &tmB, bar, k0, n0, 0);
        } else {
          tma_load_3d(smem_u32(sm.b[stage]), &tmB, bar, n0, k0, 0);
          tma_load_3d(smem_u32(sm.b[stage]) + kRowBytes * 64, &tmB, bar, n0 + 64, k0, 0);
        }
        tma_load_3d(smem_u32(sm.a[stage]), &tmA, bar, k0, m0, 0);
      }
      __syncwarp();
      issued |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == Cf::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // Never leave with a copy still writing into shared memory.
    for (int s = 0; s < Cf::kStages; ++s)
      if (issued & (1u << s))
        drain_wait(smem_u32(&sm.full[s]), (issued_parity >> s) & 1u, p.err_word);
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    const bool kmajor = kE4m3 || p.b_t;
    // The MMA's A operand is the weights' tile: K-major rows of n, or N-major
    // rows of k (LBO = one 64-column box, 16 k-rows per MMA).
    const uint64_t wdesc = kmajor ? smem_desc(smem_u32(sm.b[0]), 16, kAtomBytes, 2u)
                                  : smem_desc(smem_u32(sm.b[0]), kRowBytes * 64, kAtomBytes, 2u);
    const uint64_t xdesc = smem_desc(smem_u32(sm.a[0]), 16, kAtomBytes, 2u);
    const uint32_t wstep = (kmajor ? 32u : kRowBytes * 16) >> 4;
    uint32_t stage = 0, phase = 0;
    bool ok = true, any = false;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_lazy(smem_u32(&sm.full[stage]), phase, abort, p.err_word, kWaitFull)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint64_t wd = wdesc + stage * (Cf::kBBytes >> 4);
      const uint64_t xd = xdesc + stage * (Cf::kABytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t acc = kk > 0 || kb > kb0 ? 1u : 0u;
          if constexpr (kE4m3) {
            tc_mma_f8(tmem_base, wd + kk * wstep, xd + kk * 2, p.idesc, acc);
          } else {
            tc_mma_f16(tmem_base, wd + kk * wstep, xd + kk * 2, p.idesc, acc);
          }
        }
        tc_commit(smem_u32(&sm.empty[stage]));
      }
      __syncwarp();
      any = true;
      if (++stage == Cf::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // A commit covers the MMAs of the lane that issues it: the same lane is
    // elected each time (the lowest of a full warp).
    if (elect_one()) {
      if (ok) tc_commit(smem_u32(&sm.done));
      if (any) tc_commit(smem_u32(&sm.drain));
    }
    __syncwarp();
    // Never leave with an MMA still reading shared memory or writing TMEM.
    if (any) drain_wait(smem_u32(&sm.drain), 0, p.err_word);
    __syncwarp();
  } else {
    // ------------------------------------------- accumulator -> partial sums
    const int quarter = warp & 3;
    grid_dependency_wait();
    split_load_cols<kGrad>(p, col, cols);
    split_load_row<kGrad>(p, m0 + t / wq, col, first);
    int got = 0;
    if (lane == 0)
      got = mbar_wait_bounded(smem_u32(&sm.done), 0, abort, p.err_word, kWaitTmemFull);
    got = __shfl_sync(0xffffffffu, got, 0);
    // Every MMA has completed and every copy was consumed by one, so the stages
    // are free: partial sums [row][column], lanes on columns. A CTA whose wait
    // gave up (recorded in the error word, which is what counts) has NaN for sums,
    // except where a late copy still lands on them.
    tc_fence_after_sync();
    float *red = reinterpret_cast<float *>(sm.b[0]) + quarter * 32 + lane;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
    for (int c = 0; c < kMP; c += 16) {
      if (c < p.mp) {
        uint32_t r[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
            "%10, %11, %12, %13, %14, %15}, [%16];\n"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
              "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr + c)
            : "memory");
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          red[(c + j) * kSplitN] = got ? __uint_as_float(r[j]) : __uint_as_float(0x7fffffffu);
      }
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  if (cl > 1) {
    cluster_sync();  // every CTA's partial sums are in its shared memory
  } else {
    __syncthreads();
  }

  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (warp >= 2) {
    const uint32_t red = smem_u32(sm.b[0]);
    with_act(p.c.act, [&](auto a) {
      constexpr int kAct = decltype(a)::value;
      if (p.c.bf16) {
        split_finish<kGrad, true, kAct>(p, red, t, lc, m0, col, cols, first, sum);
      } else {
        split_finish<kGrad, false, kAct>(p, red, t, lc, m0, col, cols, first, sum);
      }
    });
  }
  // Lanes leave the finishing loop after different numbers of rows; the barrier
  // below is one the whole warp has to execute together.
  __syncwarp();
  if (cl > 1) {
    // No CTA leaves while another reads its sums. That is all the barrier is for:
    // every value read has been used by the additions before it, and no CTA writes
    // where a peer reads once the sums are exchanged, so it orders no memory. (A
    // releasing arrive, here, before the results' stores, or per warp on an mbarrier,
    // takes 0.7 to 2.5 us: 1 x 4096 x 4096 8.5 -> 9.3, 256 x 4096 x 4096 16.1 -> 18.5.)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n"
                 "barrier.cluster.wait.aligned;\n" ::: "memory");
  } else {
    __syncthreads();
  }

  if constexpr (kGrad) {
    if (p.c.dbias != nullptr) {
      // Column sums of this CTA's columns: the threads of a column in row order, in a
      // part of the stages that holds no partial sums (other CTAs read those).
      constexpr uint32_t kSums = kMP * kSplitN * 4, kB = Cf::kStages * Cf::kBBytes;
      constexpr uint32_t kSlots = kSums > kB ? kSums - kB : 0;  // offset into the stages of A
      static_assert(kSlots + kSplitFinish * 16 <= Cf::kStages * Cf::kABytes, "room for the sums");
      float4 *slots = reinterpret_cast<float4 *>(&sm.a[0][0] + kSlots);
      if (warp >= 2) slots[t] = make_float4(sum[0], sum[1], sum[2], sum[3]);
      __syncthreads();
      const int at = n0 + rank * W + t;
      if (warp >= 2 && t < W && at < p.N) {
        float s = 0.f;
        for (int i = t / 4; i < kSplitFinish; i += wq)
          s += reinterpret_cast<const float *>(slots + i)[t & 3];
        // All rows in one token tile: the sum is complete.
        if (p.part != nullptr) {
          p.part[static_cast<int64_t>(tile % p.tiles_m) * p.N + at] = s;
        } else {
          p.c.dbias[at] = p.c.bf16 ? to16<true>(s) : to16<false>(s);
        }
      }
    }
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, Cf::kTmem);
  }
}

// Whether clusters of cl CTAs of a kernel can be resident (queried once).
inline bool split_clusters_fit(const DeviceInfo &dev, const void *kern, size_t smem, int cl) {
  static std::mutex mu;
  static std::map<std::pair<const void *, int>, int> cache;  // (kernel, device * 16 + cl)
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_pair(kern, dev.device * 16 + cl);
  auto it = cache.find(key);
  if (it != cache.end()) return it->second > 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cl), 1, 1);
  cfg.blockDim = dim3(kSplitThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cl);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
  cudaGetLastError();
  cache[key] = n;
  return n > 0;
}

template <bool kE4m3, int kMP, bool kGrad>
cudaError_t launch_split_form(const DeviceInfo &dev, bool b_t, int M, int N, int K, const void *A,
                              int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                              float *part, cudaStream_t stream) {
  using Cf = SplitCfg<kMP>;
  constexpr int kEs = kE4m3 ? 1 : 2, kBK = kE4m3 ? 128 : 64;
  // 228 KiB of shared memory per SM, 1 KiB of it reserved per CTA.
  static_assert(kSplitCtasPerSm * (sizeof(SplitSmem<kMP>) + 2048) <= 228 * 1024, "shared memory");
  static_assert(Cf::kStages * Cf::kBBytes >= kMP * kSplitN * 4 ||
                    Cf::kStages * (Cf::kBBytes + Cf::kABytes) >= kMP * kSplitN * 4,
                "partial sums fit in the stages");
  const size_t smem = sizeof(SplitSmem<kMP>) + 1024;
  auto kern = gemm_epi_split_kernel<kE4m3, kMP, kGrad>;
  const void *kp = reinterpret_cast<const void *>(kern);
  cudaError_t e = set_max_dynamic_smem(kp, static_cast<int>(smem), dev.device);
  if (e != cudaSuccess) return e;

  SplitArgs p;
  p.M = M, p.N = N, p.K = K;
  p.mp = (std::min(M, kMP) + 15) / 16 * 16;
  p.tiles_m = (M - 1) / kMP + 1;
  p.b_t = b_t;
  auto vec = [](const uint16_t *q, int64_t ld) {
    return reinterpret_cast<uintptr_t>(q) % 8 == 0 && ld % 4 == 0;
  };
  p.r_vec = vec(epi.R, epi.ldr), p.d_vec = vec(epi.D, epi.ldd), p.z_vec = vec(epi.Z, epi.ldz);
  p.idesc = idesc_mma(kE4m3 || !epi.bf16 ? 0u : kFmtBF16, !b_t, false, kSplitN, p.mp);
  p.err_word = dev.err_word;
  p.part = part;
  p.c = epi;
  const CUtensorMapDataType dt = kE4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : epi.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap tmA, tmB;
  if (!make_tmap(&tmA, dt, kEs, A, M, K, lda, 1, 0, static_cast<uint32_t>(p.mp), kBK) ||
      !(b_t ? make_tmap(&tmB, dt, kEs, B, N, K, ldb, 1, 0, kSplitN, kBK)
            : make_tmap(&tmB, dt, kEs, B, K, N, ldb, 1, 0, 64, 64)))
    return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>((N - 1) / kSplitN + 1) * p.tiles_m;
  if (tiles > 0x7fffffffLL / kSplitMaxCl) return cudaErrorInvalidValue;
  const int KB = (K - 1) / kBK + 1;
  // As many parts of k as fill the SMs twice, at least one k-block each.
  int cl = 1;
  while (cl < kSplitMaxCl && tiles * cl * 2 <= static_cast<int64_t>(kSplitCtasPerSm) * dev.sm_count &&
         cl * 2 <= KB)
    cl *= 2;
  while (cl > 1 && !split_clusters_fit(dev, kp, smem, cl)) cl /= 2;
  p.cl = cl;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * cl), 1, 1);
  cfg.blockDim = dim3(kSplitThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cl);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, tmA, tmB, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <bool kE4m3, bool kGrad>
cudaError_t launch_split(const DeviceInfo &dev, int mp, bool b_t, int M, int N, int K,
                         const void *A, int64_t lda, const void *B, int64_t ldb,
                         const EpiCall &epi, float *part, cudaStream_t stream) {
  switch (mp) {
    case 16: return launch_split_form<kE4m3, 16, kGrad>(dev, b_t, M, N, K, A, lda, B, ldb, epi, part, stream);
    case 32: return launch_split_form<kE4m3, 32, kGrad>(dev, b_t, M, N, K, A, lda, B, ldb, epi, part, stream);
    case 64: return launch_split_form<kE4m3, 64, kGrad>(dev, b_t, M, N, K, A, lda, B, ldb, epi, part, stream);
    default: return launch_split_form<kE4m3, 128, kGrad>(dev, b_t, M, N, K, A, lda, B, ldb, epi, part, stream);
  }
}

}  // namespace
}  // namespace dgr
