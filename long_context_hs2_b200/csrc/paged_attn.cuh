// Attention of one new token per sequence over a paged cache, split over the
// cache's length and joined; optionally every position's head-summed
// probability is added to its accumulated weight.  This file: the shares of the
// work, the join, and the kernels on warp MMAs, which serve head_dim 64 and pages
// under 8 positions (777 positions, 8 heads x 64: 7.7 us with the join).  Larger
// pages of head_dim 128: paged_attn_tc.cuh (4 x 256K E4M3: 122 us with these
// kernels, bound by the warp MMAs and the codes' conversion, 86 there).
//
//   s_hj = scale <q_h, k_j>,  O_h = sum_j p_hj v_j,  p_hj = exp(s_hj - lse_h),
//   lse_h = log sum_j exp(s_hj),  weight_j += sum_h p_hj        (j < seq_len)
//
// The G = H / kv_heads query heads of one K/V head are the rows of the tiles
// (MT tiles of 16 rows), so each K and V row is read once for all of them.
//
// Work.  The unit is a tile of 128 positions of one (sequence, K/V head); all
// tiles of the call, in order, are dealt to the CTAs in equal contiguous
// shares, found on the device from the lengths (a scan by one warp): ragged
// batches, one long sequence and many short ones keep every SM equally busy,
// and a launch does not depend on host knowledge of the lengths.  A share cuts
// at most two (sequence, head) items; cut items leave partial sums (fp32, with
// the row maximum and sum) in the workspace, joined by the combine kernel in
// ascending order, so results do not depend on timing.
//
// Pipeline per CTA (one per SM): a producer warp brings K and V tiles through a
// ring (TMA boxes of a page's rows with the 128- or 64-byte swizzle; pages
// under 8 rows by cp.async), 8 consumer warps each own 16 positions of every
// tile: S = Q K^T and O += P V as warp MMAs, softmax statistics in fp32
// registers, one pass, no exchange between warps until the item ends.  A row's
// reference is raised only when a logit exceeds it by 2^8 (`kPaSlack`).
//
// Positions past the end and pages outside the pool are masked: logits are
// replaced (never computed with), V rows are zeroed in shared memory, so what
// stale pages hold -- infinities, NaN -- reaches no sum.
//
// E4M3: codes become f16 (K) or bf16 (V) in registers, exactly.  The queries are
// scaled by a power of two per row into f16's range, k_scale multiplies the logits,
// and v_scale the probabilities, whose product is split into two bf16 terms (2^-16
// of it at any size: f16 has not the range for scales that differ, and a row of
// zeros has the scale 1 whatever its neighbours have).  Over a bf16 cache P is one
// bf16: 2^-8 of each term, as the bf16 output's own rounding.
#pragma once

#include "paged_cache.cuh"
#include "tc_common.cuh"

namespace hs2 {

constexpr int kPaTile = 128;                 // positions per tile
constexpr int kPaWarps = 8;                  // consumer warps, 16 positions each
constexpr int kPaThreads = 32 * (kPaWarps + 1);
// 32 rows x 128 columns of O per warp are 128 registers a thread: the producer's
// warpgroup is made whole and gives its registers to the consumers
// (128 * 40 + 256 * 232 = 384 * 168, all that the block was launched with).
template <int MT, int D>
constexpr bool kPaMove = MT == 2 && D == 128;
template <int MT, int D>
constexpr int kPaAttnThreads = kPaMove<MT, D> ? 32 * (kPaWarps + 4) : kPaThreads;
constexpr float kPaSlack = 8.f;              // log2 a logit may exceed its reference by
constexpr float kPaLog2e = 1.4426950408889634f;
constexpr float kPaLn2 = 0.6931471805599453f;

struct PagedAttnParams {
  PagedCache c;
  const __nv_bfloat16* q;   // [B][H][D]
  __nv_bfloat16* o;         // [B][H][D]
  float* lse_out;           // [B][H] or nullptr
  float* lse;               // workspace [B][H]
  float* part_o;            // [CTA][2][G][D]
  float2* part_ml;          // [CTA][2][G]: row maximum (log2), sum
  int H, G, grid;
  float scale_log2;
};

// Shares of `total` tiles: CTA c has tiles [c * chunk, (c + 1) * chunk) of them.
struct PaShare {
  int total, chunk;
  __device__ __forceinline__ PaShare(int total_, int grid)
      : total(total_), chunk(max(1, (total_ + grid - 1) / grid)) {}
  __device__ __forceinline__ int begin(int c) const {
    return (int)min((long long)total, (long long)c * chunk);
  }
  __device__ __forceinline__ int owner(int g) const { return g / chunk; }
};
__device__ __forceinline__ int pa_tiles(int len) { return (len + kPaTile - 1) / kPaTile; }

// One warp: all tiles of the call, `mult` items per sequence.
__device__ __forceinline__ int pa_total(const PagedCache& c, int mult) {
  int n = 0;
  for (int b = threadIdx.x & 31; b < c.B; b += 32) n += pa_tiles(paged_len(c, b));
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * mult;
}
// One warp: the sequence that holds tile g, and the first tile of that sequence.
__device__ __forceinline__ void pa_find(const PagedCache& c, int mult, int g, int& b_out,
                                        int& first) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int b = b0 + lane;
    const int mine = b < c.B ? pa_tiles(paged_len(c, b)) * mult : 0;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, g < base + inc);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b_out = b0 + src;
      first = base + __shfl_sync(0xffffffffu, inc - mine, src);
      return;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  b_out = c.B;
  first = base;
}

// One warp: the CTA's share, for PaWalk::start (empty: x == y).
__device__ __forceinline__ int4 pa_share(const PagedCache& c, int mult, int grid) {
  const PaShare sh(pa_total(c, mult), grid);
  int4 w = make_int4(sh.begin(blockIdx.x), sh.begin(blockIdx.x + 1), 0, 0);
  if (w.x < w.y) pa_find(c, mult, w.x, w.w, w.z);
  return w;
}

// Walks a CTA's share item by item.
struct PaWalk {
  int b, head, len, nt, t0, t1;   // the current segment: tiles [t0, t1) of nt
  int g, end;                     // next tile of the share, and its end
  // the CTA's share: {first tile, end, first tile of the first sequence, that sequence}
  __device__ __forceinline__ void start(const PagedCache& c, const int4 work) {
    const int g0 = work.x, g1 = work.y, first = work.z, b0 = work.w;
    b = b0;
    g = g0;
    end = g1;
    len = paged_len(c, b);
    nt = pa_tiles(len);
    head = (g0 - first) / nt;
    t0 = (g0 - first) - head * nt;
    t1 = min(nt, t0 + (end - g));
  }
  // to the next segment; false at the share's end
  __device__ __forceinline__ bool next(const PagedCache& c, int mult) {
    g += t1 - t0;
    if (g >= end) return false;
    t0 = 0;
    if (++head == mult) {
      head = 0;
      do {
        ++b;
        len = paged_len(c, b);
        nt = pa_tiles(len);
      } while (nt == 0);
    }
    t1 = min(nt, end - g);
    return true;
  }
};

// Shared memory: a ring of stages (K tile, V tile, E4M3 scales, mask of live
// positions, their slots), the queries, per-warp statistics, barriers.
template <int MT, int D, bool FP8, bool WEIGHT>
struct PaSmem {
  static constexpr int kRow = D * (FP8 ? 1 : 2);             // bytes of a K or V row
  static constexpr int kTileBytes = kPaTile * kRow;
  static constexpr int kKvBytes = (WEIGHT ? 1 : 2) * kTileBytes;
  static constexpr int kMetaBytes = 2 * kPaTile * 4 + kPaTile * 4 + 64;
  static constexpr int kStage = kKvBytes;
  static constexpr int kFit = (196 * 1024) / (kKvBytes + kMetaBytes);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kMetaOff = kStages * kStage;
  static constexpr int kQOff = kMetaOff + (kStages * kMetaBytes + 1023) / 1024 * 1024;
  static constexpr int kQBytes = MT * 16 * D * 2;
  static constexpr int kMlOff = kQOff + kQBytes;             // float2 [warps][MT * 16]
  static constexpr int kRowOff = kMlOff + kPaWarps * MT * 16 * 8;   // float [MT * 16]
  static constexpr int kBarOff = kRowOff + MT * 16 * 4;
  static constexpr int kWorkOff = kBarOff + 2 * 8 * 8;       // int4
  static constexpr int kBytes = kWorkOff + 64 + 1024;
  // columns of the output joined at a time in a stage's bytes
  static constexpr int kJoin0 = kKvBytes / (kPaWarps * MT * 16 * 4);
  static constexpr int kJoin = kJoin0 < D ? kJoin0 : D;
};

// Byte offset of 16-byte chunk c of row r in a K or V tile.
template <int D, bool FP8>
__device__ __forceinline__ uint32_t pa_tile_at(int r, int c) {
  if (FP8 && D == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  return (c >> 3) * (kPaTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
// Byte offset of chunk c of row r of the queries.
template <int MT, int D>
__device__ __forceinline__ uint32_t pa_q_at(int r, int c) {
  return (c >> 3) * (MT * 16 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void mma_f16_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// S += Q K^T: E4M3's codes as f16.
template <bool FP8>
__device__ __forceinline__ void pa_mma_qk(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (FP8) mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  else mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}
// O += P V, the terms of P one after the other.
template <int TERMS>
__device__ __forceinline__ void pa_mma_pv(float* d, const uint32_t (&a)[TERMS][4], uint32_t b0,
                                          uint32_t b1) {
#pragma unroll
  for (int t = 0; t < TERMS; ++t) mma_bf16_16816(d, a[t][0], a[t][1], a[t][2], a[t][3], b0, b1);
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(uint16_t)two, __NV_E4M3);
  return *reinterpret_cast<uint32_t*>(&h);
}
// 3D tiled TMA load: columns x.., head y, slots z..
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on `bar` (counted in its initial count) once this thread's
// earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void pa_consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kPaWarps) : "memory");
}

// Arrivals of a full barrier: the producer's, and (E4M3 scales or small pages)
// one per lane when its copies have landed.
__device__ __forceinline__ uint32_t pa_full_count(bool fp8, bool small) {
  return (fp8 || small) ? 33u : 1u;
}

// The producer warp: one tile into stage `st`.  ids: the page of run i at
// ids[i / 32] of lane i % 32, a run being the rows of one page in the tile.
template <int MT, int D, bool FP8, bool WEIGHT>
__device__ __forceinline__ void pa_fetch(const PagedCache& c, const CUtensorMap* km,
                                         const CUtensorMap* vm, uint8_t* smem, int st,
                                         uint64_t* full, const int* ids, int t, int len, int head,
                                         uint64_t kpol, uint64_t vpol) {
  using SM = PaSmem<MT, D, FP8, WEIGHT>;
  const int lane = threadIdx.x & 31;
  const int shift = min(c.page_shift, 7);        // log2 of a run's rows
  const int runs = kPaTile >> shift, rows = 1 << shift;
  const int page_mask = (1 << c.page_shift) - 1;
  const int j0 = t * kPaTile;
  uint8_t* kt = smem + st * SM::kStage;
  uint8_t* meta = smem + SM::kMetaOff + st * SM::kMetaBytes;
  // live positions, and their slots
  unsigned live[4];
  int slot[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = i * 32 + lane, run = key >> shift;
    const int mine = (run >> 5) == 0 ? ids[0] : (run >> 5) == 1 ? ids[1]
                                              : (run >> 5) == 2 ? ids[2] : ids[3];
    const int page = __shfl_sync(0xffffffffu, mine, run & 31);
    const bool ok = j0 + key < len && page >= 0;
    live[i] = __ballot_sync(0xffffffffu, ok);
    slot[i] = ok ? (int)(((long long)page << c.page_shift) + ((j0 + key) & page_mask)) : -1;
    if (WEIGHT) reinterpret_cast<int*>(meta + 2 * kPaTile * 4)[key] = slot[i];
  }
  unsigned* mask = reinterpret_cast<unsigned*>(meta + 3 * kPaTile * 4);
  if (lane < 4)
    mask[lane] = lane == 0 ? live[0] : lane == 1 ? live[1] : lane == 2 ? live[2] : live[3];
  __syncwarp();
  if (rows >= 8) {   // at most 16 runs: one per lane
    const bool ok = lane < runs && j0 + lane * rows < len && ids[0] >= 0;
    const unsigned n = __popc(__ballot_sync(0xffffffffu, ok));
    if (lane == 0) mbar_arrive_expect_tx(&full[st], n * rows * SM::kRow * (WEIGHT ? 1 : 2));
    __syncwarp();
    if (ok) {
      const int z = (int)(((long long)ids[0] << c.page_shift) + ((j0 + lane * rows) & page_mask));
      constexpr int kParts = SM::kRow > 128 ? SM::kRow / 128 : 1;
      constexpr int kPitch = SM::kRow > 128 ? 128 : SM::kRow;
      const uint32_t dst = smem_u32(kt) + lane * rows * kPitch;
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        tma_load_3d(dst + h * kPaTile * 128, km, &full[st], h * 64, head, z, kpol);
        if (!WEIGHT)
          tma_load_3d(dst + SM::kTileBytes + h * kPaTile * 128, vm, &full[st], h * 64, head, z,
                      vpol);
      }
    }
  } else {           // pages of 1, 2 or 4 rows: every lane copies whole rows
    constexpr int kChunks = SM::kRow / 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (slot[i] < 0) continue;
      const int key = i * 32 + lane;
      const size_t at = ((size_t)slot[i] * c.heads + head) * SM::kRow;
      for (int ch = 0; ch < kChunks; ++ch) {
        const uint32_t off = smem_u32(kt) + pa_tile_at<D, FP8>(key, ch);
        cp_async16(off, c.k + at + ch * 16, 16);
        if (!WEIGHT) cp_async16(off + SM::kTileBytes, c.v + at + ch * 16, 16);
      }
    }
    if (lane == 0) mbar_arrive(&full[st]);
  }
  if (FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (slot[i] < 0) continue;
      const int key = i * 32 + lane;
      const size_t at = (size_t)slot[i] * c.heads + head;
      cp_async4(smem_u32(meta) + key * 4, c.k_scale + at);
      if (!WEIGHT) cp_async4(smem_u32(meta) + (kPaTile + key) * 4, c.v_scale + at);
    }
  }
  if (FP8 || rows < 8) cp_async_arrive(&full[st]);
}

// The pages of tile t's runs (-1: past the end, or reported as outside the pool).
__device__ __forceinline__ void pa_pages(const PagedCache& c, int b, int t, int len, int* ids) {
  const int lane = threadIdx.x & 31;
  const int shift = min(c.page_shift, 7);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int run = q * 32 + lane;
    const long long j = (long long)t * kPaTile + ((long long)run << shift);
    int id = -1;
    if (run < (kPaTile >> shift) && j < len) {
      id = c.page_table[(size_t)b * c.max_pages + (j >> c.page_shift)];
      if ((unsigned)id >= (unsigned)c.n_pages) {
        raise_status(kStatusBadIndex);
        id = -1;
      }
    }
    ids[q] = id;
  }
}

// All consumer threads: the queries of one item into shared memory.  bf16: as
// they are.  E4M3: as f16, scaled by a power of two per row (row_scale holds
// its inverse), and within every 16 columns in the order in which a thread's
// four consecutive K codes meet the MMA's contraction index.
template <int MT, int D, bool FP8>
__device__ __forceinline__ void pa_load_q(const __nv_bfloat16* q, int G, uint8_t* qs,
                                          float* row_scale) {
  constexpr int kLanes = D / 8;
  for (int u = threadIdx.x; u < MT * 16 * kLanes; u += 32 * kPaWarps) {
    const int r = u / kLanes, ch = u % kLanes;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (r < G) w = *reinterpret_cast<const uint4*>(q + r * D + ch * 8);
    if (!FP8) {
      *reinterpret_cast<uint4*>(qs + pa_q_at<MT, D>(r, ch)) = w;
    } else {
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      float f[8], amax = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = bf16x2_to_float2(ww[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      // 2^e <= amax < 2^(e+1); rows of zeros keep 1.  A row with an infinity becomes NaN
      // (its logits are infinite or NaN, its probabilities NaN)
      const int e = amax > 0.f ? max(-126, min(126, (int)(__float_as_uint(amax) >> 23) - 127)) : 0;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      const float down = fmaf(amax, 0.f, __uint_as_float((uint32_t)(127 - e) << 23));
      if (ch == 0) row_scale[r] = up;
      // column c of 16 goes to place: c = 4 t + i, place = 2 t + (i & 1) + 8 (i >> 1)
#pragma unroll
      for (int half = 0; half < 2; ++half) {       // two groups of 4 columns
        const int t = (ch & 1) * 2 + half;
        uint8_t* row0 = qs + pa_q_at<MT, D>(r, ch & ~1);
        uint8_t* row1 = qs + pa_q_at<MT, D>(r, ch | 1);
        *reinterpret_cast<uint32_t*>(row0 + t * 4) =
            pack_f16(f[4 * half] * down, f[4 * half + 1] * down);
        *reinterpret_cast<uint32_t*>(row1 + t * 4) =
            pack_f16(f[4 * half + 2] * down, f[4 * half + 3] * down);
      }
    }
  }
}

// One consumer warp: s[mt][n] = Q K^T for its 16 positions (rows key0 .. of the tile).
template <int MT, int D, bool FP8>
__device__ __forceinline__ void pa_scores(uint32_t qs, uint32_t kt, int key0,
                                          float (&s)[MT][2][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[m][n][i] = 0.f;
  const int krow = key0 + ((lane >> 3) & 1) * 8 + (lane & 7), kc = lane >> 4;
  const int qrow = (lane & 7) + ((lane >> 3) & 1) * 8, qc = lane >> 4;
  // one 16-byte chunk of codes is a whole step of 16, so a load serves two steps
  constexpr int kSteps = FP8 ? 2 : 1;
#pragma unroll
  for (int k0 = 0; k0 < D / 16; k0 += kSteps) {
    uint32_t r[4];
    ldsm_x4(kt + pa_tile_at<D, FP8>(krow, (FP8 ? k0 : 2 * k0) + kc), r[0], r[1], r[2], r[3]);
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      uint32_t lo[2], hi[2];   // per 8 positions: contraction 0-7 and 8-15
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (FP8) {
          lo[n] = e4m3x2_to_f16x2(r[2 * q + n] & 0xffffu);
          hi[n] = e4m3x2_to_f16x2(r[2 * q + n] >> 16);
        } else {
          lo[n] = r[n];
          hi[n] = r[2 + n];
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t a[4];
        ldsm_x4(qs + pa_q_at<MT, D>(m * 16 + qrow, 2 * (k0 + q) + qc), a[0], a[1], a[2], a[3]);
        pa_mma_qk<FP8>(s[m][0], a, lo[0], hi[0]);
        pa_mma_qk<FP8>(s[m][1], a, lo[1], hi[1]);
      }
    }
  }
}

template <int MT, int D, bool FP8>
__global__ void __launch_bounds__(kPaAttnThreads<MT, D>, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                      const PagedAttnParams p) {
  using SM = PaSmem<MT, D, FP8, false>;
  static_assert(SM::kBytes <= 232448 && SM::kStages >= 2, "shared memory per CTA");
  static_assert(SM::kWorkOff % 16 == 0 && SM::kBarOff % 8 == 0 && SM::kMetaBytes % 16 == 0,
                "alignment of shared words");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBarOff);
  uint64_t* empty = full + 8;
  int4* work = reinterpret_cast<int4*>(smem + SM::kWorkOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool small = p.c.page_shift < 3;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < SM::kStages; ++i) {
      mbar_init(&full[i], pa_full_count(FP8, small));
      mbar_init(&empty[i], kPaWarps);
    }
    fence_mbar_init();
  }
  if (warp == kPaWarps) {
    const int4 mine = pa_share(p.c, p.c.heads, p.grid);
    if (lane == 0) *work = mine;
  }
  __syncthreads();
  if (work->x == work->y) return;
  PaWalk w;
  w.start(p.c, *work);

  if (warp >= kPaWarps) {
    // ---------------------------------------------------------- producer
    if (kPaMove<MT, D>) {
      regs_give_up<40>();
      if (warp > kPaWarps) return;
    }
    const uint64_t kpol = policy_evict_normal(), vpol = policy_evict_first();
    uint32_t it = 0;
    bool ok = true;
    int ids[4];
    pa_pages(p.c, w.b, w.t0, w.len, ids);
    do {
      for (int t = w.t0; t < w.t1 && ok; ++t, ++it) {
        const int st = it % SM::kStages;
        if (it >= (uint32_t)SM::kStages)
          ok = mbar_wait(&empty[st], ((it / SM::kStages) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        int nxt[4] = {-1, -1, -1, -1};
        if (t + 1 < w.t1) pa_pages(p.c, w.b, t + 1, w.len, nxt);
        pa_fetch<MT, D, FP8, false>(p.c, &km, &vm, smem, st, full, ids, t, w.len, w.head, kpol,
                                    vpol);
#pragma unroll
        for (int q = 0; q < 4; ++q) ids[q] = nxt[q];
      }
      if (!ok || !w.next(p.c, p.c.heads)) break;
      pa_pages(p.c, w.b, w.t0, w.len, ids);
    } while (true);
    return;
  }

  // ------------------------------------------------------------ consumers
  if (kPaMove<MT, D>) regs_take<232>();
  uint8_t* qs = smem + SM::kQOff;
  float2* ml = reinterpret_cast<float2*>(smem + SM::kMlOff);
  float* row_scale = reinterpret_cast<float*>(smem + SM::kRowOff);
  const int key0 = warp * 16, t4 = lane & 3, g8 = lane >> 2;
  uint32_t it = 0;
  bool dead = false;
  do {
    pa_load_q<MT, D, FP8>(p.q + ((size_t)w.b * p.H + (size_t)w.head * p.G) * D, p.G, qs,
                          row_scale);
    pa_consumers_sync();
    float o[MT][D / 8][4], mref[MT][2], l[MT][2], f[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mref[m][h] = -INFINITY;
        l[m][h] = 0.f;
        f[m][h] = p.scale_log2 * (FP8 ? row_scale[m * 16 + h * 8 + g8] : 1.f);
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
    }
    int st = 0;
    for (int t = w.t0; t < w.t1; ++t, ++it) {
      st = it % SM::kStages;
      // after a wait that gave up (reported), no more waits: every barrier is still met
      if (!dead) dead = !mbar_wait(&full[st], (it / SM::kStages) & 1);
      const uint8_t* meta = smem + SM::kMetaOff + st * SM::kMetaBytes;
      const unsigned mask =
          reinterpret_cast<const unsigned*>(meta + 3 * kPaTile * 4)[warp >> 1] >>
              ((warp & 1) * 16) & 0xffffu;
      uint8_t* vt = smem + st * SM::kStage + SM::kTileBytes;
      if (mask) {
        float s[MT][2][4];
        pa_scores<MT, D, FP8>(smem_u32(qs), smem_u32(smem + st * SM::kStage), key0, s);
        float vs[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float2 ks2 = make_float2(1.f, 1.f), vs2 = ks2;
          if (FP8) {
            ks2 = *reinterpret_cast<const float2*>(meta + (key0 + n * 8 + t4 * 2) * 4);
            vs2 = *reinterpret_cast<const float2*>(meta + (kPaTile + key0 + n * 8 + t4 * 2) * 4);
          }
          vs[n][0] = vs2.x;
          vs[n][1] = vs2.y;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[m][n][i] *= f[m][i >> 1] * (FP8 ? ((i & 1) ? ks2.y : ks2.x) : 1.f);
        }
        if (mask != 0xffffu) {
          // nothing that masked rows hold may be computed with
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (!(mask >> (n * 8 + t4 * 2 + c) & 1u)) {
                vs[n][c] = 0.f;
#pragma unroll
                for (int m = 0; m < MT; ++m) s[m][n][c] = s[m][n][c + 2] = -INFINITY;
              }
          for (int u = lane; u < 16 * (SM::kRow / 16); u += 32) {
            const int r = u / (SM::kRow / 16), ch = u % (SM::kRow / 16);
            if (!(mask >> r & 1u))
              *reinterpret_cast<uint4*>(vt + pa_tile_at<D, FP8>(key0 + r, ch)) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();   // the next TMA write of this stage comes after these
          __syncwarp();
        }
        // references: raised when a logit passes one by 2^kPaSlack
        float top[MT][2];
        bool raise = false;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            top[m][h] = fmaxf(fmaxf(s[m][0][2 * h], s[m][0][2 * h + 1]),
                              fmaxf(s[m][1][2 * h], s[m][1][2 * h + 1]));
            raise |= top[m][h] > mref[m][h] + kPaSlack;
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float a[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x = top[m][h];
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
              a[h] = 1.f;
              if (x > mref[m][h]) {
                a[h] = fast_exp2(mref[m][h] - x);
                mref[m][h] = x;
              }
              l[m][h] *= a[h];
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[m][n][i] *= a[i >> 1];
          }
        }
        // P, in the MMA's A layout
        constexpr int kTerms = FP8 ? 2 : 1;
        uint32_t pa[MT][kTerms][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[i] = s[m][n][i] == -INFINITY ? 0.f : fast_exp2(s[m][n][i] - mref[m][i >> 1]);
              l[m][i >> 1] += e[i];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = FP8 ? e[2 * h] * vs[n][0] : e[2 * h];
              const float y = FP8 ? e[2 * h + 1] * vs[n][1] : e[2 * h + 1];
              pa[m][0][2 * n + h] = pack_bf16(x, y);
              if (FP8) {
                const float2 r = bf16x2_to_float2(pa[m][0][2 * n + h]);
                pa[m][kTerms - 1][2 * n + h] = pack_bf16(x - r.x, y - r.y);
              }
            }
          }
        const int vrow = key0 + ((lane >> 3) & 1) * 8 + (lane & 7), vc = lane >> 4;
        if (FP8) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];
            ldsm_x4_t(smem_u32(vt) + pa_tile_at<D, true>(vrow, c + vc), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              // even columns of the 16, then odd ones
              const uint32_t ev = __byte_perm(r[2 * q], r[2 * q + 1], 0x6420);
              const uint32_t od = __byte_perm(r[2 * q], r[2 * q + 1], 0x7531);
              const uint32_t e0 = e4m3x2_to_bf16x2((uint16_t)ev);
              const uint32_t e1 = e4m3x2_to_bf16x2((uint16_t)(ev >> 16));
              const uint32_t o0 = e4m3x2_to_bf16x2((uint16_t)od);
              const uint32_t o1 = e4m3x2_to_bf16x2((uint16_t)(od >> 16));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                pa_mma_pv(o[m][2 * (c + q)], pa[m], e0, e1);
                pa_mma_pv(o[m][2 * (c + q) + 1], pa[m], o0, o1);
              }
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t r[4];
            ldsm_x4_t(smem_u32(vt) + pa_tile_at<D, false>(vrow, 2 * c + vc), r[0], r[1], r[2],
                      r[3]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              pa_mma_pv(o[m][2 * c], pa[m], r[0], r[1]);
              pa_mma_pv(o[m][2 * c + 1], pa[m], r[2], r[3]);
            }
          }
        }
      }
      __syncwarp();
      if (t + 1 < w.t1 && lane == 0) mbar_arrive(&empty[st]);   // the last one is kept for the join
    }

    // ---- join the warps' parts of the item in the last tile's stage
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[m][h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (t4 == 0) ml[warp * (MT * 16) + m * 16 + h * 8 + g8] = make_float2(mref[m][h], x);
      }
    pa_consumers_sync();   // statistics visible; every warp is done with the stage
    const bool whole = w.t0 == 0 && w.t1 == w.nt;
    const int part = blockIdx.x * 2 + (w.t0 > 0 ? 0 : 1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < kPaWarps; ++q)
          top = fmaxf(top, ml[q * (MT * 16) + m * 16 + h * 8 + g8].x);
        f[m][h] = mref[m][h] == -INFINITY ? 0.f : fast_exp2(mref[m][h] - top);
      }
    float* buf = reinterpret_cast<float*>(smem + st * SM::kStage);   // [warp][row][kJoin]
    constexpr int C = SM::kJoin;
    for (int c0 = 0; c0 < D; c0 += C) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        if (FP8 && (n & 1)) continue;
        const int col = FP8 ? (n >> 1) * 16 + t4 * 4 : n * 8 + t4 * 2;
        if (col < c0 || col >= c0 + C) continue;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = m * 16 + h * 8 + g8;
            float* at = buf + (size_t)(warp * (MT * 16) + r) * C;
            if (FP8) {
              const int x = (col - c0) ^ (C >= 32 ? (r & 1) << 4 : 0);
              *reinterpret_cast<float4*>(at + x) =
                  make_float4(o[m][n][2 * h] * f[m][h], o[m][n + 1][2 * h] * f[m][h],
                              o[m][n][2 * h + 1] * f[m][h], o[m][n + 1][2 * h + 1] * f[m][h]);
            } else {
              const int x = (col - c0) ^ ((r & 3) << 3);
              *reinterpret_cast<float2*>(at + x) =
                  make_float2(o[m][n][2 * h] * f[m][h], o[m][n][2 * h + 1] * f[m][h]);
            }
          }
      }
      pa_consumers_sync();
      for (int u = threadIdx.x; u < MT * 16 * (C / 4); u += 32 * kPaWarps) {
        const int r = u / (C / 4), col = (u % (C / 4)) * 4;
        if (r < p.G) {
          const int x = FP8 ? col ^ (C >= 32 ? (r & 1) << 4 : 0) : col ^ ((r & 3) << 3);
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int q = 0; q < kPaWarps; ++q) {
            const float4 v =
                *reinterpret_cast<const float4*>(buf + (size_t)(q * (MT * 16) + r) * C + x);
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
            top = fmaxf(top, ml[q * (MT * 16) + r].x);
          }
#pragma unroll
          for (int q = 0; q < kPaWarps; ++q) {
            // a part without positions has the sum 0; one whose logits are all NaN has no
            // reference either, and its sum is NaN
            const float2 v = ml[q * (MT * 16) + r];
            if (v.y != 0.f) sum += v.y * fast_exp2(v.x == -INFINITY ? 0.f : v.x - top);
          }
          if (whole) {
            const size_t row = (size_t)w.b * p.H + (size_t)w.head * p.G + r;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint2*>(p.o + row * D + c0 + col) =
                make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
            if (c0 + col == 0) {
              const float v = (top + log2f(sum)) * kPaLn2;
              p.lse[row] = v;
              if (p.lse_out) p.lse_out[row] = v;
            }
          } else {
            *reinterpret_cast<float4*>(p.part_o + ((size_t)part * p.G + r) * D + c0 + col) = a;
            if (c0 + col == 0) p.part_ml[(size_t)part * p.G + r] = make_float2(top, sum);
          }
        }
      }
      fence_proxy_async_smem();
      pa_consumers_sync();
    }
    if (lane == 0) mbar_arrive(&empty[st]);
  } while (w.next(p.c, p.c.heads));
}

// ----------------------------------------------------------------- combine --
constexpr int kPaMaxParts = 512;   // grid CTAs at most

// Shared memory of joining a row.
struct PaJoin {
  float wgt[kPaMaxParts];
  float top, sum;
  int first, last, tiles, pad;
};

// One warp: which CTAs have a part of item (b, head), {first, last, tiles}: the
// first one's share ends inside the item (its part 1), the others' begin inside
// it (their part 0).
__device__ __forceinline__ int3 pa_item_parts(const PagedAttnParams& p, int b, int head) {
  int before = 0, total = 0, mine = 0;
  for (int i = threadIdx.x & 31; i < p.c.B; i += 32) {
    const int n = pa_tiles(paged_len(p.c, i));
    total += n;
    if (i < b) before += n;
    if (i == b) mine = n;
  }
  total = __reduce_add_sync(0xffffffffu, total);
  before = __reduce_add_sync(0xffffffffu, before);
  const int nt = __reduce_add_sync(0xffffffffu, mine), g = before * p.c.heads + head * nt;
  const PaShare sh(total * p.c.heads, p.grid);
  return nt ? make_int3(sh.owner(g), sh.owner(g + nt - 1), nt) : make_int3(0, 0, 0);
}

// One warp, after the attention kernel: log2-domain lse of the item's row `lane`
// (lanes past G: unspecified).
__device__ __forceinline__ float pa_item_lse(const PagedAttnParams& p, int b, int head,
                                             int lane) {
  const int3 parts = pa_item_parts(p, b, head);
  if (lane >= p.G) return 0.f;
  if (parts.x == parts.y)
    return p.lse[(size_t)b * p.H + (size_t)head * p.G + lane] * kPaLog2e;
  float top = -INFINITY, sum = 0.f;
#pragma unroll 8
  for (int c = parts.x; c <= parts.y; ++c) {
    const float2 v = p.part_ml[(size_t)(c * 2 + (c == parts.x)) * p.G + lane];
    const float m = fmaxf(top, v.x);
    const float s = sum * fast_exp2(top - m) + v.y * fast_exp2(v.x - m);   // (NaN stays)
    sum = v.y == 0.f ? sum : s;   // no positions (selected, not jumped over: loads in one go)
    top = m;
  }
  return top + log2f(sum);
}

// D threads: joins the parts of row (sequence, query head) in ascending order;
// empty sequences get O = 0, lse = -inf; an item that one CTA had is finished.
template <int D>
__device__ __forceinline__ void pa_join_sync() {
  asm volatile("bar.sync 6, %0;" ::"n"(D) : "memory");
}
template <int D>
__device__ __forceinline__ void pa_join_row(const PagedAttnParams& p, int row, int tid,
                                            PaJoin& s, bool wait) {
  const int b = row / p.H, h = row % p.H, head = h / p.G, r = h % p.G;
  if (tid < 32) {
    const int3 parts = pa_item_parts(p, b, head);
    if (tid == 0) {
      s.first = parts.x;
      s.last = parts.y;
      s.tiles = parts.z;
    }
    __syncwarp();
    if (wait) pdl_wait();   // (each thread that reads or writes results waits)
    const int n = parts.y - parts.x + 1;
    if (n > 1) {
      float top = -INFINITY, sum = 0.f;
      for (int i = tid; i < n; i += 32)
        top = fmaxf(top, p.part_ml[(size_t)((parts.x + i) * 2 + (i == 0)) * p.G + r].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      for (int i = tid; i < n; i += 32) {
        const float2 v = p.part_ml[(size_t)((parts.x + i) * 2 + (i == 0)) * p.G + r];
        const float e = v.x == -INFINITY ? 0.f : fast_exp2(v.x - top);
        s.wgt[i] = e;
        sum += v.y * e;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (tid == 0) {
        s.top = top;
        s.sum = sum;
      }
    }
  } else if (wait) {
    pdl_wait();
  }
  pa_join_sync<D>();
  const int c0 = s.first, n = s.last - s.first + 1;
  __nv_bfloat16* out = p.o + (size_t)row * D + tid;
  if (s.tiles == 0) {
    *out = __float2bfloat16_rn(0.f);
    if (tid == 0) {
      p.lse[row] = -INFINITY;
      if (p.lse_out) p.lse_out[row] = -INFINITY;
    }
  } else if (n > 1) {
    float a = 0.f;
#pragma unroll 8
    for (int i = 0; i < n; ++i)
      a += s.wgt[i] * p.part_o[((size_t)((c0 + i) * 2 + (i == 0)) * p.G + r) * D + tid];
    const float sum = s.sum;
    *out = __float2bfloat16_rn(sum == 0.f ? 0.f : a / sum);
    if (tid == 0) {
      const float v = (s.top + log2f(sum)) * kPaLn2;
      p.lse[row] = v;
      if (p.lse_out) p.lse_out[row] = v;
    }
  }
  pa_join_sync<D>();   // `s` is free
}

// One CTA of D threads per (sequence, head).
template <int D>
__global__ void __launch_bounds__(D) paged_attn_combine_kernel(const PagedAttnParams p) {
  __shared__ PaJoin s;
  pdl_launch_dependents();
  pa_join_row<D>(p, blockIdx.x, threadIdx.x, s, true);
}

// ----------------------------------------------------------------- weights --
// Second pass when weights are kept: the logits again (K, mostly still in L2)
// under the final normaliser, summed over all heads, added to each position's
// weight.  One addition per position and call, so its order does not matter.
template <int MT, int D, bool FP8>
__global__ void __launch_bounds__(kPaThreads, 1)
    paged_weight_kernel(const __grid_constant__ CUtensorMap km, const PagedAttnParams p) {
  using SM = PaSmem<MT, D, FP8, true>;
  static_assert(SM::kBytes <= 232448 && SM::kStages >= 2, "shared memory per CTA");
  static_assert(SM::kWorkOff % 16 == 0 && SM::kBarOff % 8 == 0 && SM::kMetaBytes % 16 == 0,
                "alignment of shared words");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBarOff);
  uint64_t* empty = full + 8;
  int4* work = reinterpret_cast<int4*>(smem + SM::kWorkOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool small = p.c.page_shift < 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < SM::kStages; ++i) {
      mbar_init(&full[i], pa_full_count(FP8, small));
      mbar_init(&empty[i], kPaWarps);
    }
    fence_mbar_init();
  }
  if (warp == kPaWarps) {
    const int4 mine = pa_share(p.c, 1, p.grid);
    if (lane == 0) *work = mine;
  }
  __syncthreads();
  pdl_wait();
  if (work->x == work->y) return;
  // a segment's tiles are walked once per K/V head inside each tile
  PaWalk w;
  w.start(p.c, *work);

  if (warp == kPaWarps) {
    const uint64_t kpol = policy_evict_normal();
    uint32_t it = 0;
    bool ok = true;
    do {
      for (int t = w.t0; t < w.t1 && ok; ++t) {
        int ids[4];
        pa_pages(p.c, w.b, t, w.len, ids);
        for (int head = 0; head < p.c.heads && ok; ++head, ++it) {
          const int st = it % SM::kStages;
          if (it >= (uint32_t)SM::kStages)
            ok = mbar_wait(&empty[st], ((it / SM::kStages) - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          pa_fetch<MT, D, FP8, true>(p.c, &km, &km, smem, st, full, ids, t, w.len, head, kpol,
                                     kpol);
        }
      }
    } while (ok && w.next(p.c, 1));
    return;
  }
  uint8_t* qs = smem + SM::kQOff;
  float* row_scale = reinterpret_cast<float*>(smem + SM::kRowOff);
  const int key0 = warp * 16, t4 = lane & 3, g8 = lane >> 2;
  uint32_t it = 0;
  bool dead = false;
  int q_b = -1, q_head = -1;   // whose queries are in shared memory
  float f[MT][2], nl[MT][2];
  do {
    for (int t = w.t0; t < w.t1; ++t) {
      float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      for (int head = 0; head < p.c.heads; ++head, ++it) {
        if (q_b != w.b || q_head != head) {
          pa_consumers_sync();
          const size_t row = (size_t)w.b * p.H + (size_t)head * p.G;
          pa_load_q<MT, D, FP8>(p.q + row * D, p.G, qs, row_scale);
          pa_consumers_sync();
          q_b = w.b;
          q_head = head;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = m * 16 + h * 8 + g8;
              f[m][h] = p.scale_log2 * (FP8 ? row_scale[r] : 1.f);
              nl[m][h] = r < p.G ? -p.lse[row + r] * kPaLog2e : -INFINITY;
            }
        }
        const int st = it % SM::kStages;
        if (!dead) dead = !mbar_wait(&full[st], (it / SM::kStages) & 1);
        const uint8_t* meta = smem + SM::kMetaOff + st * SM::kMetaBytes;
        const unsigned mask =
            reinterpret_cast<const unsigned*>(meta + 3 * kPaTile * 4)[warp >> 1] >>
                ((warp & 1) * 16) & 0xffffu;
        if (mask) {
          float s[MT][2][4];
          pa_scores<MT, D, FP8>(smem_u32(qs), smem_u32(smem + st * SM::kStage), key0, s);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float2 ks2 = make_float2(1.f, 1.f);
            if (FP8) ks2 = *reinterpret_cast<const float2*>(meta + (key0 + n * 8 + t4 * 2) * 4);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x = s[m][n][i] * (f[m][i >> 1] * (FP8 ? ((i & 1) ? ks2.y : ks2.x) : 1.f));
                sum[n][i & 1] += fast_exp2(x + nl[m][i >> 1]);
              }
          }
        }
        if (head + 1 == p.c.heads && mask) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float x = sum[n][c];
              x += __shfl_xor_sync(0xffffffffu, x, 4);
              x += __shfl_xor_sync(0xffffffffu, x, 8);
              x += __shfl_xor_sync(0xffffffffu, x, 16);
              const int key = n * 8 + t4 * 2 + c;
              if (g8 == 0 && (mask >> key & 1u))
                atomicAdd(p.c.weight + reinterpret_cast<const int*>(meta + 2 * kPaTile * 4)[key0 + key],
                          x);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
    }
  } while (w.next(p.c, 1));
}

}  // namespace hs2
