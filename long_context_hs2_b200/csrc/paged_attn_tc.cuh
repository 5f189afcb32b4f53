// Paged decode attention on the 5th-generation tensor cores (tcgen05), for
// head_dim 128 and pages of at least 8 positions.  Same definition, work shares
// and workspace as paged_attn.cuh.
//
// Bound by HBM (K and V once) where a tile's work keeps up: 8 x up to 32K bf16
// streams at the copy rate between a start and an end of 4 and 2 us; 4 x 256K E4M3
// takes 1.4 us a tile and SM against 0.76 us of HBM time, 86 us in all (77 without V's
// conversion, 84 with one term of P).
//
// Tiles are computed transposed, 128 positions each:
//   S^T[128 positions][rows]  = K_tile . Q^T      (M = 128 positions)
//   O^T[128 d][rows]         += V_tile^T . P^T    (M = 128 d, V read MN-major)
// with NR = 16 or 32 rows (the G heads of one K/V head) as the MMAs' N.  TMEM
// lane = position in S^T, so a softmax thread owns one position and half of the
// rows: the mask is a predicate of the thread, E4M3 scales are two scalars of the
// thread, and the exponentials need no exchange.  Row references are registers,
// the same in all threads of a row half; they are raised (O and the sums rescaled)
// only when a logit passes one by 2^8, agreed on by a barrier with an OR.
// A tile's chain (S^T, softmax, P, O^T) is latency, so two run at once: even and odd
// tiles of a share belong to two sets of softmax warps with references, sums and an
// O^T of their own, joined when an item ends.
//
// E4M3.  K's codes go to the tensor cores as they are (kind::f8f6f4); the queries
// are split into two E4M3 terms instead, extra rows of the MMA's N: scaled by a
// power of two per row to |q| < 256, q = q1 + q2 / 16, exact for bf16 values down
// to 2^-13 of the row's largest, else off by 2^-14 of 128.  V becomes bf16 (exact)
// by four converter warps.  P = p * v_scale is split into two bf16 terms as well,
// 2^-16 of P at any size: scales have fp32's range, a position of little probability
// may hold all there is of a column, and f16 would lose it beside a row of a larger
// scale (a row of zeros has the scale 1).
//
// Warp roles: 0 TMA producer, 1 S^T and 3 O^T issuer, 2 queries, 4-11 and 12-19 the two
// softmax sets (warp w: TMEM lanes 32 (w % 4) .., row half (w - 4) / 4 % 2), 20-23
// E4M3's converters.
#pragma once

#include "fp8_gemm.cuh"
#include "paged_attn.cuh"

namespace hs2 {

constexpr int kPtSet = 8;               // softmax warps of a set

template <int NR, bool FP8>
struct PtSmem {
  static constexpr int kThreads = 32 * (4 + 2 * kPtSet + (FP8 ? 4 : 0));
  // rings: K tiles (with the tile's scales and mask), V tiles, E4M3's bf16 V tiles
  static constexpr int kTile = 128 * 128 * (FP8 ? 1 : 2);
  static constexpr int kK = FP8 ? 4 : 3, kV = 3, kH = FP8 ? 2 : 0;
  static constexpr int kQTerms = FP8 ? 2 : 1;
  static constexpr int kVOff = kK * kTile;
  static constexpr int kHOff = kVOff + kV * kTile;
  static constexpr int kQOff = kHOff + kH * 32768;
  static constexpr int kQBytes = NR * 256;                       // bf16, or two terms of codes
  static constexpr int kPOff = kQOff + kQBytes;
  // P^T of a set.  bf16: NR rows of 128 positions (K-major).  E4M3: 128 positions of 64
  // rows, one 128-byte swizzle row each (MN-major: a thread has all rows of its position
  // and writes them as they are): the first terms' NR, then the second terms'; with NR =
  // 16 the rest is not written, and its columns of O^T are not read.
  static constexpr int kPRows = FP8 ? 64 : NR;
  static constexpr int kPBytes = kPRows * 256;
  static constexpr int kMetaOff = kPOff + 2 * kPBytes;
  static constexpr int kMetaBytes = FP8 ? 1024 : 0;              // a K slot's scales
  // masks of live positions, of 8 tiles: a tile's K is fetched after its softmax set
  // gave back the K slot kK tiles before, and after the V of the tile before was
  // fetched, so the tile kV before that one converted: every reader is within 8
  static constexpr int kMaskOff = kMetaOff + kK * kMetaBytes;
  static constexpr int kRsOff = kMaskOff + 8 * 16;               // float [2][NR]: queries' scales
  static constexpr int kRedOff = kRsOff + 2 * NR * 4;            // float [2 sets][4][NR]
  static constexpr int kRefOff = kRedOff + 8 * NR * 4;           // float [2 sets][NR]
  static constexpr int kBarOff = kRefOff + 2 * NR * 4;
  static constexpr int kBars = 2 * kK + 2 * kV + 2 * kH + 18;
  static constexpr int kSlotOff = kBarOff + kBars * 8;
  static constexpr int kWorkOff = (kSlotOff + 16 + 15) / 16 * 16;   // int4
  static constexpr int kBytes = kWorkOff + 64 + 1024;
  // TMEM columns: S^T of four tiles, O^T of the two sets
  static constexpr int kSCols = kQTerms * NR, kOCol = 4 * kSCols;
  static constexpr int kNeed = kOCol + 2 * kPRows;
  static constexpr int kTmem = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  // registers: of the launch's kRegs a thread, warps 0-3 and the converters give
  // some to the softmax warps
  static constexpr int kRegs = FP8 ? 80 : 96, kFew = FP8 ? 56 : 64, kConv = 40,
                       kMany = FP8 ? 96 : 104;
  static_assert(128 * kFew + 512 * kMany + (FP8 ? 128 * kConv : 0) <= kThreads * kRegs,
                "shares of the registers");
  static_assert(2 * kPBytes >= NR * 128 * 4, "a set's O^T fits the two P^T buffers");
  static_assert(kNeed <= 512, "tensor memory");
};

// NC (8 or 16) consecutive columns.
template <int NC>
__device__ __forceinline__ void tmem_ldc(uint32_t taddr, float* v);
template <int NC>
__device__ __forceinline__ void tmem_stc(uint32_t taddr, const float* v);

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
template <>
__device__ __forceinline__ void tmem_ldc<8>(uint32_t taddr, float* v) { tmem_ld8(taddr, v); }
template <>
__device__ __forceinline__ void tmem_ldc<16>(uint32_t taddr, float* v) { tmem_ld16(taddr, v); }
template <>
__device__ __forceinline__ void tmem_stc<8>(uint32_t taddr, const float* v) { tmem_st8(taddr, v); }
template <>
__device__ __forceinline__ void tmem_stc<16>(uint32_t taddr, const float* v) { tmem_st16(taddr, v); }

// Barrier, and barrier with OR, of a row half of a set (128 threads, named 1-4),
// and a barrier of both sets.
__device__ __forceinline__ void pt_half_sync(int id) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + id) : "memory");
}
__device__ __forceinline__ bool pt_half_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + id), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void pt_sets_sync() {
  asm volatile("bar.sync 5, %0;" ::"n"(64 * kPtSet) : "memory");
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Maximum over the warp (NaN is left out).
__device__ __forceinline__ float warp_max_f32(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// One lane's run of a tile: its page's rows [j0 + lane * rows, + rows), if any.
struct PtRun {
  int slot;        // of its first row
  bool ok;
};
// The producer warp: tile t's K rows, scales and mask into a K slot.  id: the page
// of the lane's run.  KONLY: the weights' pass, which wants the runs' slots and no
// v_scale.  A tile that is all positions takes the short way (the warp's time for a
// tile bounds E4M3: position by position it was 1,300 cycles, and the 4 x 256K pass
// 83 us): scales four at a time where they lie together, a mask of ones.
template <bool FP8, bool KONLY>
__device__ __forceinline__ PtRun pt_fetch_k(const PagedCache& c, const CUtensorMap* km,
                                            uint8_t* kt, uint8_t* meta, unsigned* mask,
                                            uint64_t* full, int id, int t, int len, int head,
                                            int* slots, uint64_t pol) {
  const int lane = threadIdx.x & 31;
  const int shift = min(c.page_shift, 7), rows = 1 << shift;
  const int page_mask = (1 << c.page_shift) - 1, j0 = t * kPaTile;
  const bool mine = lane < (kPaTile >> shift);
  PtRun r;
  r.ok = mine && j0 + lane * rows < len && id >= 0;
  r.slot = (int)(((long long)id << c.page_shift) + ((j0 + lane * rows) & page_mask));
  if (KONLY && mine) slots[lane] = r.slot;
  const unsigned runs = __ballot_sync(0xffffffffu, r.ok);
  const bool whole = j0 + kPaTile <= len && runs == __ballot_sync(0xffffffffu, mine);
  if (whole) {
    if (lane < 4) mask[lane] = 0xffffffffu;
    if (FP8 && c.scale_vec) {
      const int slot = __shfl_sync(0xffffffffu, r.slot, lane * 4 >> shift) + (lane * 4 & (rows - 1));
      cp_async16(smem_u32(meta) + lane * 16, c.k_scale + slot, 16);
      if (!KONLY) cp_async16(smem_u32(meta) + 512 + lane * 16, c.v_scale + slot, 16);
    }
  }
  if (!whole || (FP8 && !c.scale_vec)) {
    unsigned live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = i * 32 + lane, run = key >> shift;
      const int slot = __shfl_sync(0xffffffffu, r.slot, run) + (key & (rows - 1));
      const bool ok = j0 + key < len && (runs >> run & 1u);
      live[i] = __ballot_sync(0xffffffffu, ok);
      if (FP8 && ok) {
        const size_t at = (size_t)slot * c.heads + head;
        cp_async4(smem_u32(meta) + key * 4, c.k_scale + at);
        if (!KONLY) cp_async4(smem_u32(meta) + 512 + key * 4, c.v_scale + at);
      }
    }
    if (lane < 4)
      mask[lane] = lane == 0 ? live[0] : lane == 1 ? live[1] : lane == 2 ? live[2] : live[3];
  }
  __syncwarp();
  if (lane == 0) mbar_arrive_expect_tx(full, __popc(runs) * rows * (FP8 ? 128 : 256));
  __syncwarp();
  if (r.ok) {
    const uint32_t dst = smem_u32(kt) + lane * rows * 128;
    tma_load_3d(dst, km, full, 0, head, r.slot, pol);
    if (!FP8) tma_load_3d(dst + 16384, km, full, 64, head, r.slot, pol);
  }
  if (FP8) cp_async_arrive(full);
  return r;
}
// The same tile's V rows into a V slot.
template <bool FP8>
__device__ __forceinline__ void pt_fetch_v(const PagedCache& c, const CUtensorMap* vm, uint8_t* vt,
                                           uint64_t* full, const PtRun& r, int head, uint64_t pol) {
  const int lane = threadIdx.x & 31, rows = 1 << min(c.page_shift, 7);
  const unsigned n = __popc(__ballot_sync(0xffffffffu, r.ok));
  if (lane == 0) mbar_arrive_expect_tx(full, n * rows * (FP8 ? 128 : 256));
  __syncwarp();
  if (r.ok) {
    const uint32_t dst = smem_u32(vt) + lane * rows * 128;
    tma_load_3d(dst, vm, full, 0, head, r.slot, pol);
    if (!FP8) tma_load_3d(dst + 16384, vm, full, 64, head, r.slot, pol);
  }
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

// The query warp: an item's rows from global memory into shared memory as the
// MMA's B operand; E4M3: as two terms, the rows' scales beside them.  (Rolled: it
// runs once an item, and long code that runs once is paid for in instruction
// fetches.)
template <int NR, bool FP8>
__device__ __forceinline__ void pt_stage_q(const __nv_bfloat16* q, int G, uint8_t* qs,
                                           float* row_scale) {
  const int lane = threadIdx.x & 31, ch = lane & 15;
#pragma unroll 1
  for (int i0 = 0; i0 < NR / 2; i0 += 4) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (i0 + i) * 2 + (lane >> 4);
      w[i] = r < G ? *reinterpret_cast<const uint4*>(q + (size_t)r * 128 + ch * 8)
                   : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (i0 + i) * 2 + (lane >> 4);
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
        // 2^(7 - e), + 0 * amax: NaN for a row with an infinity, which the saturating
        // conversion would make 448 of (its logits are infinite or NaN, its probabilities NaN)
        const float down = fmaf(amax, 0.f, __uint_as_float((uint32_t)(134 - e) << 23));
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
// O^T (+)= V^T P^T, PR rows; MN: P^T is MN-major.
template <int PR, bool MN>
__device__ __forceinline__ void pt_issue_pv(uint32_t d, uint32_t v, uint32_t pt, bool accumulate) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint32_t half = ks >> 2, off = (ks & 3) * 32;
    tc_mma_f16(d, sw128_mnmajor_desc(v + ks * 2048, 16384),
               MN ? sw128_mnmajor_desc(pt + ks * 2048, 16384)
                  : sw128_kmajor_desc(pt + half * (PR * 128) + off),
               tc_idesc_f16(128, PR, kTcBF16, true, MN), accumulate || ks > 0);
  }
}

template <int NR, bool FP8>
__global__ void __launch_bounds__(PtSmem<NR, FP8>::kThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap km,
                         const __grid_constant__ CUtensorMap vm, const PagedAttnParams p) {
  using SM = PtSmem<NR, FP8>;
  constexpr int NC = NR / 2, PR = SM::kPRows, KN = SM::kK, VN = SM::kV, HN = FP8 ? SM::kH : 1;
  static_assert(SM::kBytes <= 232448, "shared memory per CTA");
  static_assert(SM::kWorkOff % 16 == 0 && SM::kBarOff % 8 == 0 && SM::kMetaOff % 16 == 0 &&
                    SM::kMetaBytes % 16 == 0 && SM::kPOff % 1024 == 0 && SM::kPBytes % 1024 == 0,
                "alignment of shared words and operands");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + SM::kBarOff);
  uint64_t* kempty = kfull + KN;
  uint64_t* vfull = kempty + KN;
  uint64_t* vempty = vfull + VN;
  uint64_t* h_full = vempty + VN;    // E4M3: a V tile is bf16
  uint64_t* h_empty = h_full + SM::kH;
  uint64_t* s_full = h_empty + SM::kH;   // [4]
  uint64_t* s_empty = s_full + 4;    // [4]
  uint64_t* p_full = s_empty + 4;    // [2 sets]
  uint64_t* pv_done = p_full + 2;    // [2 sets]
  uint64_t* q_full = pv_done + 2;
  uint64_t* q_free = q_full + 1;
  // E4M3: the queries' row scales of item i of the share, in buffer i % 2
  uint64_t* rs_full = q_free + 1;    // [2]
  uint64_t* rs_free = rs_full + 2;   // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kSlotOff);
  int4* work = reinterpret_cast<int4*>(smem + SM::kWorkOff);
  float* row_scale = reinterpret_cast<float*>(smem + SM::kRsOff);
  unsigned* masks = reinterpret_cast<unsigned*>(smem + SM::kMaskOff);   // [8][4]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&km);
    tma_prefetch_desc(&vm);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < KN; ++i) {
      mbar_init(&kfull[i], pa_full_count(FP8, false));
      // S^T is done with K, and its softmax set has waited on the slot's arrival
      mbar_init(&kempty[i], 1 + kPtSet);
    }
    for (int i = 0; i < VN; ++i) {
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], FP8 ? 4 : 1);   // converted, or O^T is done with V
    }
    for (int i = 0; i < SM::kH; ++i) {
      mbar_init(&h_full[i], 4);
      mbar_init(&h_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kPtSet);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_full[i], kPtSet);
      mbar_init(&pv_done[i], 1);
      mbar_init(&rs_full[i], 1);
      mbar_init(&rs_free[i], 2 * kPtSet);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
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

  if (warp < 4) {
    regs_give_up<SM::kFew>();
    if (any && warp == 0) {
      // --------------------------------------------------------- producer
      const uint64_t kpol = policy_evict_normal(), vpol = policy_evict_first();
      uint32_t it = 0;
      bool ok = true;
      do {
        PtPages pages;
        pages.start(p.c, w.b, w.t0, w.len);
        for (int t = w.t0; t < w.t1; ++t, ++it) {
          const int ks = it % KN, vs = it % VN;
          if (it >= (uint32_t)KN) ok = mbar_wait(&kempty[ks], ((it / KN) - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const PtRun r = pt_fetch_k<FP8, false>(
              p.c, &km, smem + ks * SM::kTile, smem + SM::kMetaOff + ks * SM::kMetaBytes,
              masks + (it & 7) * 4, &kfull[ks], pages.at(p.c, t), t, w.len, w.head, nullptr, kpol);
          if (it >= (uint32_t)VN) ok = mbar_wait(&vempty[vs], ((it / VN) - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          pt_fetch_v<FP8>(p.c, &vm, smem + SM::kVOff + vs * SM::kTile, &vfull[vs], r, w.head, vpol);
        }
      } while (ok && w.next(p.c, p.c.heads));
    } else if (any && warp == 1) {
      // ------------------------------------------- S^T: up to four tiles ahead
      if (lane == 0) {
        const uint32_t q_addr = smem_u32(smem + SM::kQOff);
        uint32_t it = 0, seg = 0;
        bool ok = true;
        do {
          ok = mbar_wait(q_full, seg & 1);
          for (int t = w.t0; t < w.t1 && ok; ++t, ++it) {
            const uint32_t ks = it % KN, sb = it & 3;
            ok = mbar_wait(&kfull[ks], (it / KN) & 1) &&
                 (it < 4 || mbar_wait(&s_empty[sb], ((it >> 2) & 1) ^ 1));
            if (!ok) break;
            tc_fence_after();
            pt_issue_qk<NR, FP8>(tmem + sb * SM::kSCols, smem_u32(smem + ks * SM::kTile), q_addr);
            tc_commit(&s_full[sb]);
            tc_commit(&kempty[ks]);
          }
          tc_commit(q_free);
          ++seg;
        } while (ok && w.next(p.c, p.c.heads));
      }
    } else if (any && warp == 3) {
      // ------------------------------------------------------------- O^T
      if (lane == 0) {
        const uint32_t p_addr = smem_u32(smem + SM::kPOff);
        uint32_t it = 0;
        bool ok = true;
        do {
          for (int t = w.t0; t < w.t1 && ok; ++t, ++it) {
            const uint32_t vs = it % VN, hs = it % HN, set = it & 1;
            ok = (FP8 ? mbar_wait(&h_full[hs], (it / HN) & 1)
                      : mbar_wait(&vfull[vs], (it / VN) & 1)) &&
                 mbar_wait(&p_full[set], (it >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            pt_issue_pv<PR, FP8>(tmem + SM::kOCol + set * PR,
                                 smem_u32(FP8 ? smem + SM::kHOff + hs * 32768
                                              : smem + SM::kVOff + vs * SM::kTile),
                                 p_addr + set * SM::kPBytes, t - w.t0 >= 2);
            tc_commit(&pv_done[set]);
            tc_commit(FP8 ? &h_empty[hs] : &vempty[vs]);
          }
        } while (ok && w.next(p.c, p.c.heads));
      }
    } else if (any) {
      // ------------------------------------------------------------ queries
      uint32_t seg = 0;
      bool dead = false;
      do {
        if (seg > 0 && !dead) dead = !mbar_wait(q_free, (seg - 1) & 1);
        if (FP8 && seg > 1 && !dead) dead = !mbar_wait(&rs_free[seg & 1], ((seg >> 1) - 1) & 1);
        pt_stage_q<NR, FP8>(p.q + ((size_t)w.b * p.H + (size_t)w.head * p.G) * 128, p.G,
                            smem + SM::kQOff, row_scale + (seg & 1) * NR);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(q_full);
          if (FP8) mbar_arrive(&rs_full[seg & 1]);
        }
        ++seg;
      } while (w.next(p.c, p.c.heads));
    }
  } else if (FP8 && warp >= 4 + 2 * kPtSet) {
    // ------------------------------------------------------ V to bf16 tiles
    regs_give_up<SM::kConv>();
    const int row = threadIdx.x - 32 * (4 + 2 * kPtSet);
    const uint32_t total = (uint32_t)(work->y - work->x);
    bool dead = false;
    for (uint32_t it = 0; any && it < total; ++it) {
      const int vs = it % VN, hs = it % HN;
      if (!dead) dead = !mbar_wait(&vfull[vs], (it / VN) & 1);   // after the mask was written
      const unsigned word = masks[(it & 7) * 4 + (row >> 5)];
      const uint32_t r7 = (uint32_t)(row & 7) << 4;
      const uint32_t from = smem_u32(smem + SM::kVOff + vs * SM::kTile) + row * 128 + r7;
      const uint32_t to = smem_u32(smem + SM::kHOff + hs * 32768) + row * 128 + r7;
      // half a row at a time: the first is read before the bf16 slot is waited for
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t cw[4][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) ld_shared_v4(from ^ (half * 64 + c * 16), cw[c]);
        if (half == 0 && it >= (uint32_t)HN && !dead)
          dead = !mbar_wait(&h_empty[hs], ((it / HN) - 1) & 1);
        if (word != 0xffffffffu) {
          // rows that are not positions become zeros, whatever they hold
          const bool live = word >> lane & 1u;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) cw[c][q] = live ? cw[c][q] : 0u;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t h[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            h[2 * q] = e4m3x2_to_bf16x2((uint16_t)cw[c][q]);
            h[2 * q + 1] = e4m3x2_to_bf16x2((uint16_t)(cw[c][q] >> 16));
          }
          st_shared_v4((to ^ (c * 32)) + half * 16384, h[0], h[1], h[2], h[3]);
          st_shared_v4((to ^ (c * 32 + 16)) + half * 16384, h[4], h[5], h[6], h[7]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&vempty[vs]);
        mbar_arrive(&h_full[hs]);
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    regs_take<SM::kMany>();
    const int wq = warp & 3, set = (warp - 4) >> 3, half = (warp - 4) >> 2 & 1, c0 = half * NC;
    const int id = set * 2 + half;                  // named barrier
    const int key = wq * 32 + lane;                 // position in the tile; d of O^T
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    float* red = reinterpret_cast<float*>(smem + SM::kRedOff) + set * 4 * NR;
    float* ref = reinterpret_cast<float*>(smem + SM::kRefOff);        // [set][row]
    // where this lane's P goes in P^T.  bf16: two positions of rows c0 + (lane & 1), + 2, ..;
    // E4M3: its position's rows
    uint8_t* const p_row = smem + SM::kPOff + set * SM::kPBytes +
                           (FP8 ? key * 128 : (key >> 6) * (NR * 128) + (c0 + (lane & 1)) * 128 +
                                                  (key & 6) * 2);
    const int p_chunk = FP8 ? key & 7 : (key & 63) >> 3;
    uint32_t it0 = 0, seg = 0;                      // the item's first tile, counted over the share
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      // after a wait that gave up (reported), no more waits: every barrier is still met
      if (!dead) dead = !mbar_wait(bar, parity);
    };
    if (any) do {
      float mref[NC], l[NC];
      if (FP8) wait(&rs_full[seg & 1], (seg >> 1) & 1);
      const float* f = row_scale + (seg & 1) * NR + c0;
#pragma unroll
      for (int i = 0; i < NC; ++i) mref[i] = l[i] = 0.f;
      // rows with a reference: those that met a logit above -inf (the same in all threads of
      // the half; the others' mref is 0)
      constexpr uint32_t kAll = (1u << NC) - 1u;
      uint32_t have = 0;
      const int n = w.t1 - w.t0, skip = (it0 & 1) ^ set;
      for (uint32_t it = it0 + skip; it < it0 + n; it += 2) {
        const int st = it % KN, sb = it & 3;
        const uint32_t ph = (it >> 1) & 1;
        const uint8_t* meta = smem + SM::kMetaOff + st * SM::kMetaBytes;
        wait(&s_full[sb], (it >> 2) & 1);
        tc_fence_after();
        float d[NC];                                // log2 of p, relative to the references
        float d2[FP8 ? NC : 1];
        const uint32_t s_at = lanes + sb * SM::kSCols + c0;
        tmem_ldc<NC>(s_at, d);
        if (FP8) tmem_ldc<NC>(s_at + NR, d2);
        wait(&kfull[st], (it / KN) & 1);            // scales and mask
        const unsigned word = masks[(it & 7) * 4 + wq];
        const bool live = word >> lane & 1u;
        float ks = 1.f, vscale = 1.f;
        if (FP8) {
          ks = reinterpret_cast<const float*>(meta)[key] * p.scale_log2;
          vscale = reinterpret_cast<const float*>(meta + 512)[key];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&kempty[st]);
        tmem_ld_wait();
        if (FP8) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
            d[i] = fmaf(fmaf(d2[i], 0.0625f, d[i]) * f[i], ks, -mref[i]);
        } else {
#pragma unroll
          for (int i = 0; i < NC; ++i) d[i] = fmaf(d[i], p.scale_log2, -mref[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[sb]);
        if (word != 0xffffffffu && !live) {         // replaced, not computed with
          vscale = 0.f;
#pragma unroll
          for (int i = 0; i < NC; ++i) d[i] = -INFINITY;
        }
        float top = d[0];
#pragma unroll
        for (int i = 1; i < NC; ++i) top = fmaxf(top, d[i]);
        bool over = top > (have ? kPaSlack : -INFINITY);
        if (have && have != kAll) {
#pragma unroll
          for (int i = 0; i < NC; ++i) over |= !(have >> i & 1u) && d[i] > -INFINITY;
        }
        const bool raise = pt_half_any(id, over);
        // the set's tile before is done with O^T and P^T
        if (it >= 2) wait(&pv_done[set], ph ^ 1);
        if (raise) {
          // references to the tile's maxima; O and the sums follow.  Runs a few
          // times an item, so it is kept short in code: lane i works out row i
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const float x = warp_max_f32(d[i]);
            m = lane == i ? x : m;
          }
          float* at = red + c0 + (lane & (NC - 1));
          if (lane < NC) at[wq * NR] = m;
          pt_half_sync(id);
          m = fmaxf(fmaxf(at[0], at[NR]), fmaxf(at[2 * NR], at[3 * NR]));
          const bool had = have >> (lane & (NC - 1)) & 1u;
          const uint32_t now = __ballot_sync(0xffffffffu, had || m > -INFINITY) & kAll;
          if (had) m = fmaxf(m, 0.f);
          if (m == -INFINITY) m = 0.f;
          const float shrink = had ? fast_exp2(-m) : 1.f;
          float a[NC];
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const float mi = __shfl_sync(0xffffffffu, m, i);
            a[i] = __shfl_sync(0xffffffffu, shrink, i);
            mref[i] += mi;
            d[i] -= mi;
            l[i] *= a[i];
          }
          if (have) {
            tc_fence_after();
#pragma unroll
            for (int term = 0; term < (FP8 ? 2 * NR : NR); term += NR) {
              float o[NC];
              tmem_ldc<NC>(lanes + SM::kOCol + set * PR + term + c0, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < NC; ++i) o[i] *= a[i];
              tmem_stc<NC>(lanes + SM::kOCol + set * PR + term + c0, o);
            }
            tmem_st_wait();
            tc_fence_before();
          }
          have = now;
        }
        // P
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          d[i] = fast_exp2(d[i]);
          l[i] += d[i];
          if (FP8) d[i] *= vscale;
        }
        if (FP8) {
          // 8 rows at a time: the terms, and what the first term's rounding left
#pragma unroll
          for (int i = 0; i < NC; i += 8) {
            uint32_t v[4], r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float x = d[i + 2 * k], y = d[i + 2 * k + 1];
              v[k] = pack_bf16(x, y);
              const float2 back = bf16x2_to_float2(v[k]);
              r[k] = pack_bf16(x - back.x, y - back.y);
            }
            const int ch = (c0 + i) >> 3;
            *reinterpret_cast<uint4*>(p_row + ((ch ^ p_chunk) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(p_row + (((NR / 8 + ch) ^ p_chunk) << 4)) =
                make_uint4(r[0], r[1], r[2], r[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NC; i += 2) {
            // two rows of one position -> two positions of one row, over 2 lanes
            const uint32_t v = pack_bf16(d[i], d[i + 1]);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, v, 1);
            *reinterpret_cast<uint32_t*>(p_row + i * 128 +
                                         ((p_chunk ^ ((i + (lane & 1)) & 7)) << 4)) =
                lane & 1 ? __byte_perm(other, v, 0x7632) : __byte_perm(v, other, 0x5410);
          }
        }
        if (!FP8 && word != 0xffffffffu) {
          // rows that are not positions: zeros, whatever they held, before the product
          const int vs = it % VN;
          wait(&vfull[vs], (it / VN) & 1);
          if (!live) {
            uint8_t* v = smem + SM::kVOff + vs * SM::kTile + half * 16384 + key * 128;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(v + q * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[set]);
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
      if (NC == 8) l[0] += __shfl_xor_sync(0xffffffffu, l[0], 2);
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
      __syncwarp();
      if (FP8 && lane == 0) mbar_arrive(&rs_free[seg & 1]);
      pt_half_sync(id);                              // `red` is free
      if ((lane & (32 / NC - 1)) == 0) red[wq * NR + c0 + lane / (32 / NC)] = l[0];
      {
        float m = mref[0];
#pragma unroll
        for (int i = 1; i < NC; ++i) m = lane == i ? mref[i] : m;
        if (wq == 0 && lane < NC) ref[set * NR + c0 + lane] = have >> lane & 1u ? m : -INFINITY;
      }
      float o[NC];
      if (n > skip) {                                // the set had a tile
        const uint32_t last = it0 + skip + ((n - skip - 1) & ~1);
        wait(&pv_done[set], (last >> 1) & 1);
        tc_fence_after();
        tmem_ldc<NC>(lanes + SM::kOCol + set * PR + c0, o);
        tmem_ld_wait();
        if (FP8) {
          float o2[NC];
          tmem_ldc<NC>(lanes + SM::kOCol + set * PR + NR + c0, o2);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < NC; ++i) o[i] += o2[i];
        }
        tc_fence_before();
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) o[i] = 0.f;
      }
      pt_sets_sync();                                // statistics are there, P^T is free
      float* other_o = reinterpret_cast<float*>(smem + SM::kPOff);    // [row][d]
      const bool whole = w.t0 == 0 && w.t1 == w.nt;
      const int part = blockIdx.x * 2 + (w.t0 > 0 ? 0 : 1);
      const size_t row0 = (size_t)w.b * p.H + (size_t)w.head * p.G;
      if (set == 1) {
#pragma unroll
        for (int i = 0; i < NC; ++i) other_o[(c0 + i) * 128 + key] = o[i];
      } else if (warp == 4 && lane < NR) {           // row `lane`: the sets' factors, the statistics
        const float m0 = ref[lane], m1 = ref[NR + lane], m = fmaxf(m0, m1);
        float a0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - m);
        float a1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - m);
        const float* r0 = reinterpret_cast<const float*>(smem + SM::kRedOff) + lane;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) s0 += r0[q * NR], s1 += r0[(4 + q) * NR];
        const float sum = s0 * a0 + s1 * a1;
        if (lane < p.G) {
          if (whole) {
            const float lse = (m + log2f(sum)) * kPaLn2;
            p.lse[row0 + lane] = lse;
            if (p.lse_out) p.lse_out[row0 + lane] = lse;
          } else {
            p.part_ml[(size_t)part * p.G + lane] = make_float2(m, sum);
          }
        }
        if (whole) {
          const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
          a0 *= inv;
          a1 *= inv;
        }
        ref[lane] = a0;
        ref[NR + lane] = a1;
      }
      pt_sets_sync();
      if (set == 0) {
        __nv_bfloat16* ob = p.o + (row0 + c0) * 128 + key;
        float* op = p.part_o + ((size_t)part * p.G + c0) * 128 + key;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const float v = o[i] * ref[c0 + i] + other_o[(c0 + i) * 128 + key] * ref[NR + c0 + i];
          if (c0 + i < p.G) {
            if (whole) ob[i * 128] = __float2bfloat16_rn(v);
            else op[i * 128] = v;
          }
        }
      }
      pt_sets_sync();                                // P^T and the statistics are free again
      it0 += n;
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

// ----------------------------------------------------------------- weights --
// Second pass when weights are kept: S^T of every tile again (K, mostly still in
// L2), probabilities under the final normaliser, summed over the rows and the K/V
// heads in the thread that owns the position: one addition per position and call.
// The queries of all heads stay in shared memory (up to kPwRows rows); tiles go in
// pairs, one for each softmax set, all heads of a pair before the next.  Four more
// warps join the cut items' outputs meanwhile, as the combine kernel does when no
// weights are kept.
constexpr int kPwRows = 256;   // rows (K/V heads x NR) whose queries are resident

template <int NR, bool FP8>
struct PwSmem {
  static constexpr int kThreads = 32 * (4 + 2 * kPtSet + 4);
  static constexpr int kTile = 128 * 128 * (FP8 ? 1 : 2);
  static constexpr int kK = FP8 ? 8 : 4;
  static constexpr int kQTerms = FP8 ? 2 : 1;
  static constexpr int kQOff = kK * kTile;
  static constexpr int kQBytes = NR * 256;                       // of one head
  static constexpr int kMask = FP8 ? 1024 : 0, kSlots = kMask + 16;
  static constexpr int kMetaOff = kQOff + kPwRows * 256;
  static constexpr int kMetaBytes = kSlots + 64;                 // scales, mask, runs' slots
  static constexpr int kRsOff = kMetaOff + kK * kMetaBytes;      // float [rows]: queries' scales
  static constexpr int kNlOff = kRsOff + kPwRows * 4;            // float [rows]: -lse (log2)
  static constexpr int kSumOff = kNlOff + kPwRows * 4;           // float [2 sets][2][128]
  static constexpr int kJoinOff = kSumOff + 4 * 128 * 4;         // PaJoin
  static constexpr int kBarOff = kJoinOff + (int)sizeof(PaJoin);
  static constexpr int kBars = 2 * kK + 11;
  static constexpr int kSlotOff = (kBarOff + kBars * 8 + 15) / 16 * 16;
  static constexpr int kWorkOff = kSlotOff + 16;
  static constexpr int kBytes = kWorkOff + 64 + 1024;
  static constexpr int kSCols = kQTerms * NR;
  static constexpr int kTmem = 4 * kSCols < 64 ? 64 : 4 * kSCols;
};

__device__ __forceinline__ void pw_set_sync(int set) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + set), "n"(32 * kPtSet) : "memory");
}

template <int NR, bool FP8>
__global__ void __launch_bounds__(PwSmem<NR, FP8>::kThreads, 1)
    paged_weight_tc_kernel(const __grid_constant__ CUtensorMap km, const PagedAttnParams p) {
  using SM = PwSmem<NR, FP8>;
  constexpr int NC = NR / 2, KN = SM::kK;
  static_assert(SM::kBytes <= 232448, "shared memory per CTA");
  static_assert(SM::kWorkOff % 16 == 0 && SM::kBarOff % 8 == 0 && SM::kMetaOff % 16 == 0 &&
                    SM::kMetaBytes % 16 == 0, "alignment of shared words");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + SM::kBarOff);
  uint64_t* kempty = kfull + KN;
  uint64_t* s_full = kempty + KN;    // [4]
  uint64_t* s_empty = s_full + 4;    // [4]
  uint64_t* q_full = s_empty + 4;    // a sequence's queries: for the MMAs,
  uint64_t* rs_full = q_full + 1;    // and their scales and normalisers
  uint64_t* rs_free = rs_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kSlotOff);
  int4* work = reinterpret_cast<int4*>(smem + SM::kWorkOff);
  float* row_scale = reinterpret_cast<float*>(smem + SM::kRsOff);
  float* neg_lse = reinterpret_cast<float*>(smem + SM::kNlOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 32) tma_prefetch_desc(&km);
  if (threadIdx.x == 0) {
    for (int i = 0; i < KN; ++i) {
      mbar_init(&kfull[i], pa_full_count(FP8, false));
      mbar_init(&kempty[i], 1 + kPtSet);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kPtSet);
    }
    mbar_init(q_full, 2);
    mbar_init(rs_full, 2);
    mbar_init(rs_free, 2 * kPtSet);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, SM::kTmem);
    tmem_relinquish();
  } else if (warp == 0) {
    const int4 mine = pa_share(p.c, 1, p.grid);
    if (lane == 0) *work = mine;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool any = work->x < work->y;
  PaWalk w;
  if (any) w.start(p.c, *work);
  // Only the normalisers and the parts to join come from the attention kernel: the
  // query and the joining warps wait for it, K and the queries are fetched before.

  if (any && warp == 0) {
    // ------------------------------------------------------------- producer
    const uint64_t kpol = policy_evict_first();
    uint32_t it = 0;
    bool ok = true;
    do {
      PtPages pages;
      pages.start(p.c, w.b, w.t0, w.len);
      for (int t = w.t0; t < w.t1 && ok; t += 2) {
        const int id0 = pages.at(p.c, t), id1 = t + 1 < w.t1 ? pages.at(p.c, t + 1) : -1;
        for (int u = 0; u < 2 * p.c.heads; ++u) {
          if ((u & 1) && t + 1 >= w.t1) continue;
          const int ks = it % KN;
          if (it >= (uint32_t)KN) ok = mbar_wait(&kempty[ks], ((it / KN) - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* meta = smem + SM::kMetaOff + ks * SM::kMetaBytes;
          pt_fetch_k<FP8, true>(p.c, &km, smem + ks * SM::kTile, meta,
                                reinterpret_cast<unsigned*>(meta + SM::kMask), &kfull[ks],
                                u & 1 ? id1 : id0, t + (u & 1), w.len, u >> 1,
                                reinterpret_cast<int*>(meta + SM::kSlots), kpol);
          ++it;
        }
      }
    } while (ok && w.next(p.c, 1));
  } else if (any && warp == 1) {
    // ------------------------------------------------------------------ S^T
    if (lane == 0) {
      const uint32_t q_addr = smem_u32(smem + SM::kQOff);
      uint32_t it = 0, seg = 0;
      bool ok = true;
      do {
        ok = mbar_wait(q_full, seg & 1);
        for (int t = w.t0; t < w.t1 && ok; t += 2)
          for (int u = 0; u < 2 * p.c.heads; ++u) {
            if ((u & 1) && t + 1 >= w.t1) continue;
            const uint32_t ks = it % KN, sb = it & 3;
            ok = mbar_wait(&kfull[ks], (it / KN) & 1) &&
                 (it < 4 || mbar_wait(&s_empty[sb], ((it >> 2) & 1) ^ 1));
            if (!ok) break;
            tc_fence_after();
            pt_issue_qk<NR, FP8>(tmem + sb * SM::kSCols, smem_u32(smem + ks * SM::kTile),
                                 q_addr + (u >> 1) * SM::kQBytes);
            tc_commit(&s_full[sb]);
            tc_commit(&kempty[ks]);
            ++it;
          }
        ++seg;
      } while (ok && w.next(p.c, 1));
    }
  } else if (any && warp < 4) {
    // -------------------------------------------------------------- queries
    uint32_t seg = 0;
    bool dead = false;
    do {
      // both sets have ended the sequence before: its queries were used
      if (seg > 0 && !dead) dead = !mbar_wait(rs_free, (seg - 1) & 1);
      for (int head = warp - 2; head < p.c.heads; head += 2)
        pt_stage_q<NR, FP8>(p.q + ((size_t)w.b * p.H + (size_t)head * p.G) * 128, p.G,
                            smem + SM::kQOff + head * SM::kQBytes, row_scale + head * NR);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      if (seg == 0) pdl_wait();
      for (int head = warp - 2; head < p.c.heads; head += 2) {
        const float lse = pa_item_lse(p, w.b, head, lane);
        if (lane < NR) neg_lse[head * NR + lane] = lane < p.G ? -lse : -INFINITY;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(rs_full);
      ++seg;
    } while (w.next(p.c, 1));
  } else if (warp >= 4 + 2 * kPtSet) {
    // ------------------------------------------- the cut items' outputs
    const int tid = threadIdx.x - 32 * (4 + 2 * kPtSet);
    PaJoin& join = *reinterpret_cast<PaJoin*>(smem + SM::kJoinOff);
    pdl_wait();
    for (int row = blockIdx.x; row < p.c.B * p.H; row += gridDim.x)
      pa_join_row<128>(p, row, tid, join, false);
  } else if (any && warp >= 4) {
    // -------------------------------------------------------- probabilities
    const int wq = warp & 3, set = (warp - 4) >> 3, half = (warp - 4) >> 2 & 1, c0 = half * NC;
    const int key = wq * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    float* sums = reinterpret_cast<float*>(smem + SM::kSumOff) + set * 256;   // [2][128]
    const int run_shift = min(p.c.page_shift, 7);   // of a page's rows in a tile
    uint32_t it0 = 0, seg = 0, turn = 0;            // it0: tiles met before the pair
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!dead) dead = !mbar_wait(bar, parity);
    };
    do {
      wait(rs_full, seg & 1);
      for (int t = w.t0; t < w.t1; t += 2) {
        const int pair = min(2, w.t1 - t);
        if (set < pair) {
          float sum = 0.f;
          bool live = false;
          int slot = 0;
          for (int head = 0; head < p.c.heads; ++head) {
            const uint32_t it = it0 + head * pair + set;
            const int st = it % KN, sb = it & 3;
            const uint8_t* meta = smem + SM::kMetaOff + st * SM::kMetaBytes;
            wait(&s_full[sb], (it >> 2) & 1);
            tc_fence_after();
            float d[NC];
            float d2[FP8 ? NC : 1];
            const uint32_t s_at = lanes + sb * SM::kSCols + c0;
            tmem_ldc<NC>(s_at, d);
            if (FP8) tmem_ldc<NC>(s_at + NR, d2);
            wait(&kfull[st], (it / KN) & 1);
            const unsigned word = reinterpret_cast<const unsigned*>(meta + SM::kMask)[wq];
            live = word >> lane & 1u;
            slot = reinterpret_cast<const int*>(meta + SM::kSlots)[key >> run_shift] +
                   (key & ((1 << run_shift) - 1));
            const float ks = FP8 ? reinterpret_cast<const float*>(meta)[key] * p.scale_log2
                                 : p.scale_log2;
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&s_empty[sb]);
              mbar_arrive(&kempty[st]);
            }
            const float* f = row_scale + head * NR + c0;
            const float* nl = neg_lse + head * NR + c0;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float x = FP8 ? fmaf(d2[c], 0.0625f, d[c]) * f[c] : d[c];
              sum += fast_exp2(fmaf(x, ks, nl[c]));
            }
          }
          float* buf = sums + (turn++ & 1) * 128;
          if (half == 1) buf[key] = sum;
          pw_set_sync(set);
          if (half == 0 && live) atomicAdd(p.c.weight + slot, sum + buf[key]);
        }
        it0 += pair * p.c.heads;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(rs_free);
      ++seg;
    } while (w.next(p.c, 1));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, SM::kTmem);
  }
}

}  // namespace hs2
