// Paged decode attention on the 5th-generation tensor cores (tcgen05), for
// head_dim 128 and pages of at least 8 positions.  Same definition, work shares
// and workspace as paged_attn.cuh.
//
// Tiles are computed transposed, 128 positions each:
//   S^T[128 positions][rows]  = K_tile . Q^T      (M = 128 positions)
//   O^T[128 d][rows]         += V_tile^T . P^T    (M = 128 d, V read MN-major)
// with NR = 16 or 32 rows (the G heads of one K/V head) as the MMAs' N.  TMEM
// lane = position in S^T, so a softmax thread owns one position and 8 rows: the
// mask is a predicate of the thread, E4M3 scales are two scalars of the thread,
// and the exponentials need no exchange.  Row references are registers, the same
// in all threads of a group of 8 rows; they are raised (O and the sums rescaled)
// only when a logit passes one by 2^8, agreed on by a barrier with an OR.
//
// E4M3.  K's codes go to the tensor cores as they are (kind::f8f6f4); the queries
// are split into two E4M3 terms instead, extra rows of the MMA's N: scaled by a
// power of two per row to |q| < 256, q = q1 + q2 / 16, exact for bf16 values down
// to 2^-13 of the row's largest, else off by 2^-14 of 128.  V becomes f16 (exact)
// by four converter warps, P is f16.  v_scale is a factor of p, put into the
// exponent: P = 2^(x + log2 v_scale - ref), and the row sum takes P / v_scale; so
// P stays in f16's range whatever the scales are.
//
// Warp roles: 0 TMA producer, 1 MMA issuer, 2-3 queries, then the softmax warps
// (warp w: TMEM lanes 32 (w % 4) .., rows of group (w - 4) / 4), then E4M3's
// converters.
#pragma once

#include "fp8_gemm.cuh"
#include "paged_attn.cuh"

namespace hs2 {

constexpr float kPtMinScale = 1e-30f;   // least |v_scale| in the exponent
constexpr int kPtRows = 8;              // rows of a softmax thread

template <int NR, bool FP8>
struct PtSmem {
  static constexpr int kGroups = NR / kPtRows;                   // row groups of 4 softmax warps
  static constexpr int kSoftmax = 4 * kGroups;                   // softmax warps
  static constexpr int kThreads = 32 * (4 + kSoftmax + (FP8 ? 4 : 0));
  static constexpr int kTile = 128 * 128 * (FP8 ? 1 : 2);
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = FP8 ? 4 : 3;
  static constexpr int kQTerms = FP8 ? 2 : 1;
  static constexpr int kV16Off = kStages * kStage;               // E4M3: two f16 V tiles
  static constexpr int kQOff = kV16Off + (FP8 ? 2 * 32768 : 0);
  static constexpr int kQBytes = NR * 256;                       // bf16, or two terms of codes
  static constexpr int kPOff = kQOff + kQBytes;
  static constexpr int kPBytes = NR * 256;
  static constexpr int kMetaOff = kPOff + 2 * kPBytes;           // per stage: scales, mask
  static constexpr int kMetaBytes = (FP8 ? 1024 : 0) + 64;
  static constexpr int kRsOff = kMetaOff + kStages * kMetaBytes; // float [4][NR]: queries' scales
  static constexpr int kRedOff = kRsOff + 4 * NR * 4;            // float [4][NR]
  static constexpr int kBarOff = kRedOff + 4 * NR * 4;
  static constexpr int kBars = 3 * kStages + 18;
  static constexpr int kSlotOff = kBarOff + kBars * 8;
  static constexpr int kWorkOff = (kSlotOff + 16 + 15) / 16 * 16;   // int4
  static constexpr int kBytes = kWorkOff + 64 + 1024;
  // TMEM columns
  static constexpr int kSCols = kQTerms * NR, kOCol = 2 * kSCols;
  static constexpr int kTmem = kOCol + NR <= 64 ? 64 : kOCol + NR <= 128 ? 128 : 256;
};

// 8 consecutive fp32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
// Barrier, and barrier with OR, of a row group (128 threads, named 1 + group).
__device__ __forceinline__ void pt_group_sync(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}
__device__ __forceinline__ bool pt_group_any(int group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + group), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The producer warp: tile t of an item into stage st (K, scales and mask on
// kfull, V on vfull).  ids[0]: the page of the lane's run, as in pa_fetch.
template <int NR, bool FP8, bool KONLY>
__device__ __forceinline__ void pt_fetch(const PagedCache& c, const CUtensorMap* km,
                                         const CUtensorMap* vm, uint8_t* kt, uint8_t* meta,
                                         uint64_t* kfull, uint64_t* vfull, int id, int t, int len,
                                         int head, int* slots, uint64_t kpol, uint64_t vpol) {
  using SM = PtSmem<NR, FP8>;
  const int lane = threadIdx.x & 31;
  const int shift = min(c.page_shift, 7), runs = kPaTile >> shift, rows = 1 << shift;
  const int page_mask = (1 << c.page_shift) - 1, j0 = t * kPaTile;
  unsigned live[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = i * 32 + lane;
    const int page = __shfl_sync(0xffffffffu, id, key >> shift);
    const bool ok = j0 + key < len && page >= 0;
    live[i] = __ballot_sync(0xffffffffu, ok);
    const int slot = (int)(((long long)page << c.page_shift) + ((j0 + key) & page_mask));
    if (KONLY) slots[key] = slot;
    if (FP8 && ok) {
      const size_t at = (size_t)slot * c.heads + head;
      cp_async4(smem_u32(meta) + key * 4, c.k_scale + at);
      if (!KONLY) cp_async4(smem_u32(meta) + 512 + key * 4, c.v_scale + at);
    }
  }
  unsigned* mask = reinterpret_cast<unsigned*>(meta + (FP8 ? 1024 : 0));
  if (lane < 4)
    mask[lane] = lane == 0 ? live[0] : lane == 1 ? live[1] : lane == 2 ? live[2] : live[3];
  __syncwarp();
  const bool ok = lane < runs && j0 + lane * rows < len && id >= 0;
  const unsigned bytes = __popc(__ballot_sync(0xffffffffu, ok)) * rows * (SM::kTile / 128);
  if (lane == 0) {
    mbar_arrive_expect_tx(kfull, bytes);
    if (!KONLY) mbar_arrive_expect_tx(vfull, bytes);
  }
  __syncwarp();
  if (ok) {
    const int z = (int)(((long long)id << c.page_shift) + ((j0 + lane * rows) & page_mask));
    const uint32_t dst = smem_u32(kt) + lane * rows * 128;
    tma_load_3d(dst, km, kfull, 0, head, z, kpol);
    if (!FP8) tma_load_3d(dst + 16384, km, kfull, 64, head, z, kpol);
    if (!KONLY) {
      tma_load_3d(dst + SM::kTile, vm, vfull, 0, head, z, vpol);
      if (!FP8) tma_load_3d(dst + SM::kTile + 16384, vm, vfull, 64, head, z, vpol);
    }
  }
  if (FP8) cp_async_arrive(kfull);
}

// The producer's view of a sequence's page list: 32 entries a load, the next 32
// on their way.  Pages of at least 8 positions: a tile has at most 16 of them,
// and they lie in one window.
struct PtPages {
  const int* list;
  int base, n, cur, next;   // entry of lane 0; entries the sequence has
  __device__ __forceinline__ int load(const PagedCache& c, int at) const {
    const int i = at + (threadIdx.x & 31);
    if (i >= n) return -1;
    const int id = list[i];
    if ((unsigned)id < (unsigned)c.n_pages) return id;
    raise_status(kStatusBadIndex);
    return -1;
  }
  __device__ __forceinline__ void start(const PagedCache& c, int b, int t, int len) {
    list = c.page_table + (size_t)b * c.max_pages;
    n = (len + (1 << c.page_shift) - 1) >> c.page_shift;
    base = (int)(((long long)t * kPaTile) >> c.page_shift) & ~31;
    cur = load(c, base);
    next = load(c, base + 32);
  }
  // the page of the lane's run of tile t (tiles in ascending order)
  __device__ __forceinline__ int at(const PagedCache& c, int t) {
    const int first = (int)(((long long)t * kPaTile) >> c.page_shift);
    if (first - base >= 32) {
      base += 32;
      cur = next;
      next = load(c, base + 32);
    }
    return __shfl_sync(0xffffffffu, cur, (first - base + (threadIdx.x & 31)) & 31);
  }
};

// The query warps (64 threads): an item's rows from global memory ...
template <int NR>
__device__ __forceinline__ void pt_read_q(const __nv_bfloat16* q, int G, int tid, uint4* w) {
#pragma unroll
  for (int i = 0; i < NR / 4; ++i) {
    const int r = i * 4 + (tid >> 4), ch = tid & 15;
    w[i] = r < G ? *reinterpret_cast<const uint4*>(q + (size_t)r * 128 + ch * 8)
                 : make_uint4(0, 0, 0, 0);
  }
}
// ... and into shared memory as the MMA's B operand.
template <int NR, bool FP8>
__device__ __forceinline__ void pt_write_q(uint8_t* qs, float* row_scale, int tid, const uint4* w) {
  const int ch = tid & 15;
#pragma unroll
  for (int i = 0; i < NR / 4; ++i) {
    const int r = i * 4 + (tid >> 4);
    if (!FP8) {
      *reinterpret_cast<uint4*>(qs + sw128_offset(r, ch * 16, NR)) = w[i];
    } else {
      const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      float f[8], amax = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = bf16x2_to_float2(ww[k]);
        f[2 * k] = v.x;
        f[2 * k + 1] = v.y;
        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = amax > 0.f ? max(-110, (int)(__float_as_uint(amax) >> 23) - 127) : 0;
      const float down = __uint_as_float((uint32_t)(134 - e) << 23);   // 2^(7 - e)
      if (ch == 0) row_scale[r] = __uint_as_float((uint32_t)(120 + e) << 23);
      uint32_t t1[2] = {0, 0}, t2[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = f[2 * k] * down, b = f[2 * k + 1] * down;
        const uint32_t c1 = float2_to_e4m3x2(a, b);
        const float2 back = e4m3x2_to_float2(c1);
        const uint32_t c2 = float2_to_e4m3x2((a - back.x) * 16.f, (b - back.y) * 16.f);
        t1[k >> 1] |= c1 << ((k & 1) * 16);
        t2[k >> 1] |= c2 << ((k & 1) * 16);
      }
      const uint32_t at = r * 128 + (((ch >> 1) ^ (r & 7)) << 4) + (ch & 1) * 8;
      *reinterpret_cast<uint2*>(qs + at) = make_uint2(t1[0], t1[1]);
      *reinterpret_cast<uint2*>(qs + NR * 128 + at) = make_uint2(t2[0], t2[1]);
    }
  }
}

// S^T of one tile into TMEM columns d.
template <int NR, bool FP8>
__device__ __forceinline__ void pt_issue_qk(uint32_t d, uint32_t k, uint32_t q) {
  if (FP8) {
    const uint64_t ad = sw128_kmajor_desc(k), bd = sw128_kmajor_desc(q);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      tc_mma_f8(d, ad + 2 * ks, bd + 2 * ks, tc_idesc_e4m3(128, 2 * NR), ks > 0);
  } else {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint32_t half = ks >> 2, off = (ks & 3) * 32;
      tc_mma_f16(d, sw128_kmajor_desc(k + half * 16384 + off),
                 sw128_kmajor_desc(q + half * (NR * 128) + off),
                 tc_idesc_f16(128, NR, kTcBF16, false, false), ks > 0);
    }
  }
}
// O^T (+)= V^T P^T.
template <int NR, bool FP8>
__device__ __forceinline__ void pt_issue_pv(uint32_t d, uint32_t v, uint32_t pt, bool accumulate) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint32_t half = ks >> 2, off = (ks & 3) * 32;
    tc_mma_f16(d, sw128_mnmajor_desc(v + ks * 2048, 16384),
               sw128_kmajor_desc(pt + half * (NR * 128) + off),
               tc_idesc_f16(128, NR, FP8 ? kTcF16 : kTcBF16, true, false), accumulate || ks > 0);
  }
}

template <int NR, bool FP8>
__global__ void __launch_bounds__(PtSmem<NR, FP8>::kThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap km,
                         const __grid_constant__ CUtensorMap vm, const PagedAttnParams p) {
  using SM = PtSmem<NR, FP8>;
  constexpr int NC = kPtRows, S = SM::kStages, NW = SM::kSoftmax;
  static_assert(SM::kBytes <= 232448, "shared memory per CTA");
  static_assert(SM::kWorkOff % 16 == 0 && SM::kBarOff % 8 == 0 && SM::kMetaOff % 16 == 0 &&
                    SM::kMetaBytes % 16 == 0, "alignment of shared words");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + SM::kBarOff);
  uint64_t* vfull = kfull + S;
  uint64_t* empty = vfull + S;
  uint64_t* s_full = empty + S;      // [2]
  uint64_t* s_empty = s_full + 2;    // [2]
  uint64_t* p_full = s_empty + 2;    // [2]
  uint64_t* pv_done = p_full + 2;    // [2]
  uint64_t* v16_full = pv_done + 2;  // [2] E4M3: a V tile is f16
  uint64_t* q_full = v16_full + 2;
  uint64_t* q_free = q_full + 1;
  // Row scales of item i of the share are in buffer i % 4: the queries of item i
  // are written after the last S^T of item i - 1, so after the softmax warps read
  // the S^T two tiles before that one: they are at most three items behind, which
  // neither a buffer's reuse nor a barrier's phase can outrun.
  uint64_t* rs_full = q_free + 1;    // [4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kSlotOff);
  int4* work = reinterpret_cast<int4*>(smem + SM::kWorkOff);
  float* row_scale = reinterpret_cast<float*>(smem + SM::kRsOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&kfull[i], pa_full_count(FP8, false));
      mbar_init(&vfull[i], 1);
      // bf16: O^T is done with the stage; E4M3: S^T is done with K, V is
      // converted, the softmax warps have read the scales
      mbar_init(&empty[i], FP8 ? 1 + 4 + NW : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], NW);
      mbar_init(&p_full[i], NW);
      mbar_init(&pv_done[i], 1);
      mbar_init(&v16_full[i], 4);
    }
    mbar_init(q_full, 2);
    mbar_init(q_free, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&rs_full[i], 2);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, SM::kTmem);
    tmem_relinquish();
  } else if (warp == 0) {
    const int4 mine = pa_share(p.c, p.c.heads, p.grid);
    if (lane == 0) *work = mine;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool any = work->x < work->y;
  PaWalk w;
  if (any) w.start(p.c, *work);

  if (any && warp == 0) {
    // ----------------------------------------------------------- producer
    const uint64_t kpol = policy_evict_normal(), vpol = policy_evict_first();
    uint32_t it = 0;
    bool ok = true;
    do {
      PtPages pages;
      pages.start(p.c, w.b, w.t0, w.len);
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int st = it % S;
        if (it >= (uint32_t)S) ok = mbar_wait(&empty[st], ((it / S) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        pt_fetch<NR, FP8, false>(p.c, &km, &vm, smem + st * SM::kStage,
                                 smem + SM::kMetaOff + st * SM::kMetaBytes, &kfull[st], &vfull[st],
                                 pages.at(p.c, t), t, w.len, w.head, nullptr, kpol, vpol);
      }
    } while (ok && w.next(p.c, p.c.heads));
  } else if (any && warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t q_addr = smem_u32(smem + SM::kQOff), p_addr = smem_u32(smem + SM::kPOff);
      uint32_t it = 0, seg = 0;
      bool ok = true, pending = false, pending_first = false;
      auto pv = [&](uint32_t i, bool first) {
        const int st = i % S, bb = i & 1;
        if (!mbar_wait(&p_full[bb], (i >> 1) & 1) ||
            !(FP8 ? mbar_wait(&v16_full[bb], (i >> 1) & 1) : mbar_wait(&vfull[st], (i / S) & 1)))
          return false;
        tc_fence_after();
        pt_issue_pv<NR, FP8>(tmem + SM::kOCol,
                             smem_u32(FP8 ? smem + SM::kV16Off + bb * 32768
                                          : smem + st * SM::kStage + SM::kTile),
                             p_addr + bb * SM::kPBytes, !first);
        tc_commit(&pv_done[bb]);
        if (!FP8) tc_commit(&empty[st]);
        return true;
      };
      do {
        ok = mbar_wait(q_full, seg & 1);
        for (int t = w.t0; t < w.t1 && ok; ++t, ++it) {
          const int st = it % S, bb = it & 1;
          if (!mbar_wait(&kfull[st], (it / S) & 1) ||
              (it >= 2 && !mbar_wait(&s_empty[bb], ((it - 2) >> 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          pt_issue_qk<NR, FP8>(tmem + bb * SM::kSCols, smem_u32(smem + st * SM::kStage), q_addr);
          tc_commit(&s_full[bb]);
          if (FP8) tc_commit(&empty[st]);
          if (t + 1 == w.t1) tc_commit(q_free);
          if (pending) ok = pv(it - 1, pending_first);
          pending = true;
          pending_first = t == w.t0;
        }
        ++seg;
      } while (ok && w.next(p.c, p.c.heads));
      if (ok && pending) pv(it - 1, pending_first);
    }
  } else if (any && warp < 4) {
    // -------------------------------------------------------------- queries
    const int tid = threadIdx.x - 64;
    uint32_t seg = 0;
    bool dead = false;
    do {
      uint4 qw[NR / 4];
      pt_read_q<NR>(p.q + ((size_t)w.b * p.H + (size_t)w.head * p.G) * 128, p.G, tid, qw);
      if (seg > 0 && !dead) dead = !mbar_wait(q_free, (seg - 1) & 1);
      pt_write_q<NR, FP8>(smem + SM::kQOff, row_scale + (seg & 3) * NR, tid, qw);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(q_full);
        mbar_arrive(&rs_full[seg & 3]);
      }
      ++seg;
    } while (w.next(p.c, p.c.heads));
  } else if (FP8 && any && warp >= 4 + NW) {
    // ------------------------------------------------------- V to f16 tiles
    const int row = threadIdx.x - 32 * (4 + NW);
    uint32_t it = 0;
    bool dead = false;
    do {
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int st = it % S, bb = it & 1;
        if (!dead) dead = !mbar_wait(&kfull[st], (it / S) & 1);    // the mask
        if (!dead) dead = !mbar_wait(&vfull[st], (it / S) & 1);
        const unsigned word = reinterpret_cast<const unsigned*>(
            smem + SM::kMetaOff + st * SM::kMetaBytes + 1024)[row >> 5];
        const bool live = word >> lane & 1u;
        const uint8_t* src = smem + st * SM::kStage + SM::kTile + row * 128;
        uint4 c[8];
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
          c[ch] = *reinterpret_cast<const uint4*>(src + ((ch ^ (row & 7)) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (it >= 2 && !dead) dead = !mbar_wait(&pv_done[bb], ((it - 2) >> 1) & 1);
        uint8_t* dst = smem + SM::kV16Off + bb * 32768;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          // rows that are not positions become zeros, whatever they hold
          const uint32_t cw[4] = {c[ch].x, c[ch].y, c[ch].z, c[ch].w};
          uint32_t h[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            h[2 * q] = live ? e4m3x2_to_f16x2(cw[q] & 0xffffu) : 0u;
            h[2 * q + 1] = live ? e4m3x2_to_f16x2(cw[q] >> 16) : 0u;
          }
          *reinterpret_cast<uint4*>(dst + sw128_offset(row, ch * 32, 128)) =
              make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + sw128_offset(row, ch * 32 + 16, 128)) =
              make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v16_full[bb]);
      }
    } while (w.next(p.c, p.c.heads));
  } else if (any) {
    // -------------------------------------------------------------- softmax
    const int wq = warp & 3, group = (warp - 4) >> 2, c0 = group * NC;
    const int key = wq * 32 + lane;                 // position in the tile; d of O^T
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    float* red = reinterpret_cast<float*>(smem + SM::kRedOff);
    // where this lane's two positions of rows c0 + (lane & 1), + 2, .. go in P^T
    uint8_t* const p_row = smem + SM::kPOff + (key >> 6) * (NR * 128) + (c0 + (lane & 1)) * 128 +
                           (key & 6) * 2;
    const int p_chunk = (key & 63) >> 3;
    uint32_t it = 0, seg = 0;
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      // after a wait that gave up (reported), no more waits: every barrier is still met
      if (!dead) dead = !mbar_wait(bar, parity);
    };
    do {
      float mref[NC], l[NC], f[NC];
      if (FP8) wait(&rs_full[seg & 3], (seg >> 2) & 1);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        mref[i] = 0.f;
        l[i] = 0.f;
        f[i] = FP8 ? row_scale[(seg & 3) * NR + c0 + i] * p.scale_log2 : p.scale_log2;
      }
      bool fresh = true;                            // no position met yet: no references
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int st = it % S, bb = it & 1;
        const uint8_t* meta = smem + SM::kMetaOff + st * SM::kMetaBytes;
        wait(&kfull[st], (it / S) & 1);             // scales and mask
        const unsigned word =
            reinterpret_cast<const unsigned*>(meta + (FP8 ? 1024 : 0))[wq];
        const bool live = word >> lane & 1u;
        float ks = 1.f, lv = 0.f, inv = 1.f;
        uint32_t flip = 0;
        if (FP8) {
          ks = reinterpret_cast<const float*>(meta)[key];
          const float vs = reinterpret_cast<const float*>(meta + 512)[key];
          const float a = fmaxf(fabsf(vs), kPtMinScale);
          flip = vs < 0.f ? 0x80008000u : 0u;
          lv = __log2f(a);
          inv = fast_rcp(a);
        }
        wait(&s_full[bb], (it >> 1) & 1);
        tc_fence_after();
        float d[NC];                                // log2 of p, relative to the references
        tmem_ld8(lanes + bb * SM::kSCols + c0, d);
        if (FP8) {
          float d2[NC];
          tmem_ld8(lanes + bb * SM::kSCols + NR + c0, d2);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < NC; ++i)
            d[i] = fmaf(fmaf(d2[i], 0.0625f, d[i]) * f[i], ks, lv - mref[i]);
        } else {
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < NC; ++i) d[i] = fmaf(d[i], f[i], -mref[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s_empty[bb]);
          if (FP8) mbar_arrive(&empty[st]);
        }
        if (word != 0xffffffffu && !live) {         // replaced, not computed with
          inv = 1.f;
#pragma unroll
          for (int i = 0; i < NC; ++i) d[i] = -INFINITY;
        }
        float top = d[0];
#pragma unroll
        for (int i = 1; i < NC; ++i) top = fmaxf(top, d[i]);
        if (pt_group_any(group, fresh ? top > -INFINITY : top > kPaSlack)) {
          // references to the tile's maxima; O and the sums follow
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            float m = d[i];
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == i) red[wq * NR + c0 + i] = m;
          }
          pt_group_sync(group);
          float a[NC];
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            float m = fmaxf(fmaxf(red[c0 + i], red[NR + c0 + i]),
                            fmaxf(red[2 * NR + c0 + i], red[3 * NR + c0 + i]));
            if (!fresh) m = fmaxf(m, 0.f);
            if (m == -INFINITY) m = 0.f;
            a[i] = fast_exp2(-m);
            mref[i] += m;
            d[i] -= m;
            l[i] *= fresh ? 0.f : a[i];
          }
          if (!fresh) {
            wait(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
            tc_fence_after();
            float o[NC];
            tmem_ld8(lanes + SM::kOCol + c0, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < NC; ++i) o[i] *= a[i];
            tmem_st8(lanes + SM::kOCol + c0, o);
            tmem_st_wait();
            tc_fence_before();
          }
          fresh = false;
        }
        // P
        float e[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          e[i] = fast_exp2(d[i]);
          l[i] = fmaf(e[i], inv, l[i]);
        }
        if (it >= 2) wait(&pv_done[bb], ((it - 2) >> 1) & 1);   // P's buffer is free
#pragma unroll
        for (int i = 0; i < NC; i += 2) {
          // two rows of one position -> two positions of one row, over 2 lanes
          const uint32_t v = FP8 ? pack_f16(e[i], e[i + 1]) ^ flip : pack_bf16(e[i], e[i + 1]);
          const uint32_t other = __shfl_xor_sync(0xffffffffu, v, 1);
          *reinterpret_cast<uint32_t*>(p_row + bb * SM::kPBytes + i * 128 +
                                       ((p_chunk ^ (i + (lane & 1))) << 4)) =
              lane & 1 ? __byte_perm(other, v, 0x7632) : __byte_perm(v, other, 0x5410);
        }
        if (!FP8 && word != 0xffffffffu) {
          // rows that are not positions: zeros, whatever they held, before the product
          wait(&vfull[st], (it / S) & 1);
          if (!live) {
            constexpr int kShare = 256 / SM::kGroups;   // bytes of the row
            const int at = group * kShare;
            uint8_t* v = smem + st * SM::kStage + SM::kTile + (at >> 7) * 16384 + key * 128 +
                         (at & 127);
#pragma unroll
            for (int q = 0; q < kShare / 16; ++q)
              *reinterpret_cast<uint4*>(v + q * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[bb]);
      }

      // ---- the item's (or the part's) output
      // row sums over the warp: halves of the rows go each way until one is left
#pragma unroll
      for (int h = NC / 2, bit = 16; h; h >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < h; ++i) {
          const float send = up ? l[i] : l[i + h];
          l[i] = (up ? l[i + h] : l[i]) + __shfl_xor_sync(0xffffffffu, send, bit);
        }
      }
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], 2);
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
      pt_group_sync(group);                          // `red` is free
      if ((lane & 3) == 0) red[wq * NR + c0 + (lane >> 2)] = l[0];
      pt_group_sync(group);
      const uint32_t last = it - 1;
      wait(&pv_done[last & 1], (last >> 1) & 1);
      tc_fence_after();
      float o[NC];
      tmem_ld8(lanes + SM::kOCol + c0, o);
      tmem_ld_wait();
      tc_fence_before();
      const bool whole = w.t0 == 0 && w.t1 == w.nt;
      const int part = blockIdx.x * 2 + (w.t0 > 0 ? 0 : 1);
      const size_t row0 = (size_t)w.b * p.H + (size_t)w.head * p.G;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int r = c0 + i;
        if (r < p.G) {
          const float sum = (red[r] + red[NR + r]) + (red[2 * NR + r] + red[3 * NR + r]);
          if (whole) {
            p.o[(row0 + r) * 128 + key] = __float2bfloat16_rn(sum == 0.f ? 0.f : o[i] / sum);
            if (key == 0) {
              const float v = (mref[i] + log2f(sum)) * kPaLn2;
              p.lse[row0 + r] = v;
              if (p.lse_out) p.lse_out[row0 + r] = v;
            }
          } else {
            p.part_o[((size_t)part * p.G + r) * 128 + key] = o[i];
            if (key == 0)
              p.part_ml[(size_t)part * p.G + r] = make_float2(fresh ? -INFINITY : mref[i], sum);
          }
        }
      }
      ++seg;
    } while (w.next(p.c, p.c.heads));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, SM::kTmem);
  }
}

}  // namespace hs2
