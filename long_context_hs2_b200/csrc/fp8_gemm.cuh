// E4M3 matrix product with fp32 scales per block of 128.
//
//   C[m][n] = sum_kb sa[m][kb] * sb[n / 128][kb] * sum_{k in block kb} A[m][k] * B[n][k]
//
// A [M][K], B [N][K] E4M3 (both K-major), sa [M][ceil(K/128)], sb
// [ceil(N/128)][ceil(K/128)] fp32, C bf16 [M][N].  The tensor cores sum one
// block of 128 (four tcgen05.mma kind::f8f6f4 of K = 32) into a fresh
// accumulator in tensor memory; the scaled sum over the blocks is kept in fp32
// registers, C = sum_kb s * T_kb, so each block costs one tensor-memory read and
// one FMA per element next to its MMAs.
//
// Two kernels, by the number of rows M:
// * fp8_gemm_kernel (many rows): persistent, tiles of 128 rows x BN columns.
//   Warp 0 TMA producer (one 128-byte-swizzled stage per block: A 128 x 128
//   bytes, B BN x 128 bytes), warps 1 and 2 MMA issuers, warps 4.. consumers: warp w
//   owns TMEM lanes 32 (w % 4) .. (its rows) and a share of the columns.  Tensor
//   memory holds 512 / BN accumulators, so the MMAs of the next blocks run while one
//   is scaled and added.  What bounds it: an accumulator's way to the registers and
//   back (115 us for 18,944 x 1536 x 4096, where MMAs and copies alone take 77; 835 us,
//   1.97 PFLOP/s, for 131,072 rows).
// * fp8_gemm_small_kernel (few rows): the product transposed (TMEM lane =
//   column n, MMA N = rows), the contraction split over a cluster of CTAs and
//   joined through distributed shared memory in rank order: bound by reading B
//   once, so the whole machine streams it (8 x 1536 x 4096: 5.5 us).
#pragma once

#include "paged_common.cuh"

namespace hs2 {

constexpr int kFgBK = 128;             // one scale block per stage

struct Fp8GemmParams {
  const float* sa;
  const float* sb;
  __nv_bfloat16* c;
  int M, N, K, kb;                     // kb = ceil(K / 128)
  int m_tiles, n_tiles;
};

// kind::f8f6f4, A = B = E4M3, fp32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t tc_idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ------------------------------------------------------------- many rows --
// CW: consumer warps; each owns 32 rows and BN / (CW / 4) columns.
template <int BN, int CW>
struct FgSmem {
  static constexpr int kABytes = 128 * kFgBK, kBBytes = BN * kFgBK;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kFit = (200 * 1024) / kStage;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kBytes = kBarOff + 256 + 1024;
  static constexpr int kCols = BN / (CW / 4);            // columns of a consumer warp
  static constexpr int kThreads = 32 * (4 + CW);
  static constexpr int kAcc = 512 / BN < 8 ? 512 / BN : 8;   // accumulators in tensor memory
  static constexpr int kTmem = kAcc * BN;
};

// A row's `left` next columns of C (at most COLS) as bf16, in the widest pieces that
// rows of N columns allow; rows of an odd length start on 2 or on 4 bytes by turns,
// so every other one puts its first column out alone (63,704 x 197 x 2352: 188 us with
// 2-byte stores, 114 so).
template <int COLS>
__device__ __forceinline__ void fg_store(__nv_bfloat16* out, const float* v, int left, int N) {
  if (left >= COLS && (N & 7) == 0) {
#pragma unroll
    for (int c = 0; c < COLS; c += 8)
      *reinterpret_cast<uint4*>(out + c) =
          make_uint4(pack_bf16(v[c], v[c + 1]), pack_bf16(v[c + 2], v[c + 3]),
                     pack_bf16(v[c + 4], v[c + 5]), pack_bf16(v[c + 6], v[c + 7]));
  } else if (((uintptr_t)out & 3u) == 0) {
#pragma unroll
    for (int c = 0; c < COLS; c += 2) {
      if (c + 1 < left) *reinterpret_cast<uint32_t*>(out + c) = pack_bf16(v[c], v[c + 1]);
      else if (c < left) out[c] = __float2bfloat16_rn(v[c]);
    }
  } else {
    if (left > 0) out[0] = __float2bfloat16_rn(v[0]);
#pragma unroll
    for (int c = 1; c < COLS; c += 2) {
      if (c + 1 < COLS && c + 1 < left)
        *reinterpret_cast<uint32_t*>(out + c) = pack_bf16(v[c], v[c + 1 < COLS ? c + 1 : c]);
      else if (c < left) out[c] = __float2bfloat16_rn(v[c]);
    }
  }
}

// An accumulator that the CW consumer warps have read goes back to its MMA issuer
// (one warp) by a named barrier: the mbarrier way back, an arrival and a wait
// through shared memory that the MMAs' operands keep busy, was some 500 cycles of
// the 1,200 that a 256-column accumulator waited between two uses (18,944 x 1536 x
// 4096: 128 -> 115 us).
template <int CW>
__device__ __forceinline__ void fg_acc_arrive(int acc) {
  asm volatile("bar.arrive %0, %1;" ::"r"(1 + acc), "n"(32 * (CW + 1)) : "memory");
}
template <int CW>
__device__ __forceinline__ void fg_acc_sync(int acc) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + acc), "n"(32 * (CW + 1)) : "memory");
}

template <int BN, int CW>
__global__ void __launch_bounds__(32 * (4 + CW), 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap amap,
                    const __grid_constant__ CUtensorMap bmap, const Fp8GemmParams p) {
  using SM = FgSmem<BN, CW>;
  constexpr int COLS = SM::kCols, A = SM::kAcc;
  static_assert(SM::kBytes <= 232448 && SM::kStages >= 3, "shared memory per CTA");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBarOff);
  uint64_t* empty = full + SM::kStages;
  uint64_t* acc_full = empty + SM::kStages;    // [A]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + A);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = p.m_tiles * p.n_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SM::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < A; ++a) mbar_init(&acc_full[a], 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, SM::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr bool kMove = COLS >= 128;   // 128 sums a thread do not fit 168 registers
  static_assert(!kMove || CW == 8, "128 * 40 + 256 * 232 = 384 * 168, what the block is given");

  if (warp < 4) {
    if (kMove) regs_give_up<40>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA producer
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
      const uint64_t pol = policy_evict_normal();
      uint32_t it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const int m0 = tile / p.n_tiles * 128, n0 = tile % p.n_tiles * BN;
        for (int kb = 0; kb < p.kb; ++kb, ++it) {
          const int s = it % SM::kStages;
          if (!mbar_wait(&empty[s], ((it / SM::kStages) & 1) ^ 1)) { ok = false; break; }
          uint8_t* a = smem + s * SM::kStage;
          mbar_arrive_expect_tx(&full[s], SM::kStage);
          tma_load_2d(a, &amap, &full[s], kb * kFgBK, m0, pol);
          tma_load_2d(a + SM::kABytes, &bmap, &full[s], kb * kFgBK, n0, pol);
        }
      }
    } else if (warp == 1 || warp == 2) {
      // ----------------------------------------------------- MMA issuers
      // Two take the blocks in turn: one's waits and commits, a few hundred cycles
      // next to a block's MMAs, pass while the other's MMAs run.
      const uint32_t total =
          (uint32_t)((tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x) * p.kb;
      constexpr uint32_t idesc = tc_idesc_e4m3(128, BN);
      bool ok = true;
      for (uint32_t it = warp - 1; it < total; it += 2) {
        const uint32_t s = it % SM::kStages, acc = it % A;
        // (after a wait that gave up, reported, the barriers are still met)
        if (ok) ok = mbar_wait_warp(&full[s], (it / SM::kStages) & 1);
        if (it >= (uint32_t)A) fg_acc_sync<CW>(acc);
        if (ok && lane == 0) {
          tc_fence_after();
          const uint32_t addr = smem_u32(smem + s * SM::kStage);
          const uint64_t ad = sw128_kmajor_desc(addr), bd = sw128_kmajor_desc(addr + SM::kABytes);
#pragma unroll
          for (int k = 0; k < kFgBK / 32; ++k)   // +32 bytes along K per step
            tc_mma_f8(tmem + acc * BN, ad + 2 * k, bd + 2 * k, idesc, k != 0);
          tc_commit(&acc_full[acc]);
          tc_commit(&empty[s]);
        }
        __syncwarp();
      }
      // the accumulators are read before tensor memory is given back
      for (uint32_t i = total >= A ? total - A : 0; i < total; ++i)
        if ((i & 1) == (uint32_t)(warp - 1)) fg_acc_sync<CW>(i % A);
      asm volatile("bar.sync 15, 64;" ::: "memory");
      if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, SM::kTmem);
      }
    }
  } else {
    // --------------------------------------------------------- consumers
    if (kMove) regs_take<232>();
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + part * COLS;
    constexpr int CH = COLS / 32;
    static_assert(CH % 2 == 0, "a block's chunks alternate between two register sets");
    const uint32_t total =
        (uint32_t)((tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x) * p.kb;
    // Chunks of 32 columns, one after another through blocks and tiles: each is read
    // while the one before it is added, so neither the barrier of a block nor the
    // tensor memory's latency is waited for where the MMAs are ahead.
    float v[2][32];
    bool ok = mbar_wait_warp(&acc_full[0], 0);
    tc_fence_after();
    tmem_ld32(taddr, v[0]);
    uint32_t it = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const int m = tile / p.n_tiles * 128 + quarter * 32 + lane;
      const int n0 = tile % p.n_tiles * BN + part * COLS;
      const float* sa = p.sa + (size_t)min(m, p.M - 1) * p.kb;
      const float* sb = p.sb + (size_t)min(n0 / 128, (p.N - 1) / 128) * p.kb;
      float acc[COLS];
#pragma unroll
      for (int i = 0; i < COLS; ++i) acc[i] = 0.f;
      // scales are loaded a block ahead and multiplied where they are used, so that
      // no load is waited for where it is issued
      float sa_next = sa[0], sb_next = sb[0];
      for (int kb = 0; kb < p.kb; ++kb, ++it) {
        const float s = sa_next * sb_next;
        if (kb + 1 < p.kb) sa_next = sa[kb + 1], sb_next = sb[kb + 1];
        const uint32_t a = it % A, an = (it + 1) % A;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          tmem_ld_wait();
          if (c + 1 < CH) {
            tmem_ld32(taddr + a * BN + (c + 1) * 32, v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            if (ok) fg_acc_arrive<CW>(a);
            else fg_acc_sync<CW>(a);   // (in step with the issuer, which the wait was for)
            if (it + 1 < total) {
              // (after a wait that gave up, reported, the barriers are still met)
              if (ok) ok = mbar_wait_warp(&acc_full[an], ((it + 1) / A) & 1);
              tc_fence_after();
              tmem_ld32(taddr + an * BN, v[0]);
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c * 32 + i] = fmaf(v[c & 1][i], s, acc[c * 32 + i]);
        }
      }
      if (ok && m < p.M) fg_store<COLS>(p.c + (size_t)m * p.N + n0, acc, p.N - n0, p.N);
    }
    tmem_ld_wait();
  }
}

// -------------------------------------------------------------- few rows --
// NP: rows of the tile (the MMA's N).  Cluster of `cs` CTAs along x per
// (128 columns of C, NP rows).
constexpr int kFsMaxCluster = 8;
constexpr int kFsThreads = 192;

template <int NP>
struct FsSmem {
  static constexpr int kWBytes = 128 * kFgBK, kXBytes = NP * kFgBK;
  static constexpr int kStage = kWBytes + kXBytes;
  static constexpr int kRedBytes = NP * 128 * 4;          // [source][row][column]
  static constexpr int kFit = (200 * 1024 - kRedBytes) / kStage;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kRedOff = kStages * kStage;
  static constexpr int kBarOff = kRedOff + kRedBytes;
  static constexpr int kBytes = kBarOff + 256 + 1024;
  static constexpr int kTmem = 2 * NP < 32 ? 32 : 2 * NP;
};

template <int NP>
__global__ void __launch_bounds__(kFsThreads, 1)
    fp8_gemm_small_kernel(const __grid_constant__ CUtensorMap amap,
                          const __grid_constant__ CUtensorMap bmap, const Fp8GemmParams p,
                          const int cs) {
  using SM = FsSmem<NP>;
  static_assert(SM::kBytes <= 232448 && SM::kStages >= 3, "shared memory per CTA");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBarOff);
  uint64_t* empty = full + SM::kStages;
  uint64_t* acc_full = empty + SM::kStages;    // [2]
  uint64_t* acc_empty = acc_full + 2;          // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  float* red = reinterpret_cast<float*>(smem + SM::kRedOff);

  cluster_arrive_relaxed();   // first phase: this CTA runs
  const int rank = (int)cluster_ctarank();
  const int seg = blockIdx.x / cs, n0 = seg % p.n_tiles * 128, m0 = seg / p.n_tiles * NP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's blocks of the contraction (none, for a short one)
  const int kb0 = (int)((long long)p.kb * rank / cs), kb1 = (int)((long long)p.kb * (rank + 1) / cs);
  const int n_kb = kb1 - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SM::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 4);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, SM::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  float acc[NP];
#pragma unroll
  for (int t = 0; t < NP; ++t) acc[t] = 0.f;
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
      const uint64_t pol = policy_evict_normal();
      for (int i = 0; i < n_kb; ++i) {
        const int s = i % SM::kStages;
        if (!mbar_wait(&empty[s], ((i / SM::kStages) & 1) ^ 1)) break;
        uint8_t* st = smem + s * SM::kStage;
        mbar_arrive_expect_tx(&full[s], SM::kStage);
        tma_load_2d(st, &bmap, &full[s], (kb0 + i) * kFgBK, n0, pol);
        tma_load_2d(st + SM::kWBytes, &amap, &full[s], (kb0 + i) * kFgBK, m0, pol);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = tc_idesc_e4m3(128, NP);
      for (int i = 0; i < n_kb; ++i) {
        const int s = i % SM::kStages, a = i & 1;
        if (!mbar_wait(&acc_empty[a], ((i >> 1) & 1) ^ 1) ||
            !mbar_wait(&full[s], (i / SM::kStages) & 1))
          break;
        tc_fence_after();
        const uint32_t addr = smem_u32(smem + s * SM::kStage);
        const uint64_t wd = sw128_kmajor_desc(addr), xd = sw128_kmajor_desc(addr + SM::kWBytes);
#pragma unroll
        for (int k = 0; k < kFgBK / 32; ++k)
          tc_mma_f8(tmem + a * NP, wd + 2 * k, xd + 2 * k, idesc, k != 0);
        tc_commit(&empty[s]);
        tc_commit(&acc_full[a]);
      }
    }
  } else {
    const uint32_t taddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float* sb = p.sb + (size_t)(n0 / 128) * p.kb;
    for (int i = 0; i < n_kb; ++i) {
      const int a = i & 1;
      // the rows' scales of this block, one per lane and 32 rows, times B's
      float sc[(NP + 31) / 32];
#pragma unroll
      for (int q = 0; q < (NP + 31) / 32; ++q)
        sc[q] = p.sa[(size_t)min(m0 + q * 32 + lane, p.M - 1) * p.kb + kb0 + i] * sb[kb0 + i];
      if (!mbar_wait_warp(&acc_full[a], (i >> 1) & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < NP; c += 16) {
        float v[16];
        tmem_ld16(taddr + a * NP + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < 16; ++t)
          acc[c + t] =
              fmaf(v[t], __shfl_sync(0xffffffffu, sc[(c + t) / 32], (c + t) & 31), acc[c + t]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[a]);
    }
  }
  __syncwarp();             // (warps 0 and 1: from the one lane that had work)
  cluster_wait_acquire();   // every CTA of the cluster runs
  const int col = (warp & 3) * 32 + lane;
  const int per = (NP + cs - 1) / cs;           // rows that a CTA finishes
  if (warp >= 2) {
    const uint32_t at = smem_u32(red);
#pragma unroll
    for (int t = 0; t < NP; ++t)
      if (m0 + t < p.M) {
        const int owner = t / per, slot = (rank * per + t % per) * 128 + col;
        st_dsmem_f32(mapa_shared(at + slot * 4, owner), acc[t]);
      }
  }
  cluster_arrive_release();
  cluster_wait_acquire();   // every push has landed
  if (warp >= 2 && n0 + col < p.N) {
    for (int tl = 0; tl < per; ++tl) {
      const int t = rank * per + tl;
      if (t >= NP || m0 + t >= p.M) break;
      float v = 0.f;
      for (int src = 0; src < cs; ++src) v += red[(src * per + tl) * 128 + col];
      p.c[(size_t)(m0 + t) * p.N + n0 + col] = __float2bfloat16_rn(v);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, SM::kTmem);
  }
}

}  // namespace hs2
