// Eviction from a paged cache by accumulated attention weight.
//
// Sequence b of length n keeps its `window` most recent positions and, of the
// candidates j < n - window, the min(topk, .) of largest weight (ties to the
// lower position; NaN below every number).  The survivors, in ascending order,
// become positions 0, 1, ... of the sequence: row r <- row kept[r].
//
// One launch, one cluster per sequence.  The threshold is found by a radix
// search over the weights' 32-bit order (digits of 11, 11 and 10 bits): every
// CTA counts its part of the candidates in shared memory, and after a cluster
// barrier every CTA sums all parts' counts through distributed shared memory
// and finds the digit for itself -- one barrier per digit.  Counts are whole
// numbers, so the result does not depend on the order of the atomics.
// Survivors are then written in order from ballots: each warp owns a contiguous
// run of candidates, counts it, learns what comes before it, and writes it.
//
// The move.  Into other pages (dst_table) it is a plain copy, rows spread over
// the cluster.  In place, row r overwrites a row that an earlier move has to
// have read (kept[r] >= r); so a CTA takes a column of every row -- kEvCol
// bytes of K or of V, or one array of scales or weights -- and walks the rows
// in ascending chunks: all reads of a chunk, a block barrier, its writes.
// Reads of later chunks lie above every row written so far, and no two CTAs
// share a column, so one barrier per chunk is enough.
#pragma once

#include "paged_cache.cuh"

namespace hs2 {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;
constexpr int kEvCache = 24 * 1024;   // weights of a CTA's part kept in shared memory (96 KB)
constexpr int kEvMaxCluster = 8;
constexpr int kEvCol = 64;            // bytes of a row that one CTA moves in place
constexpr int kEvBatch = 4;           // rows per thread and chunk, in place

struct EvictParams {
  PagedCache c;
  const int* dst_table;    // nullptr: in place
  int* kept;               // [B][topk + window]
  int* new_len;            // [B]
  int dst_max_pages, topk, window, cs, row_bytes, cache_keys;
};

struct EvSmem {
  unsigned hist[2][kEvBins];
  unsigned warp_gt[kEvWarps], warp_eq[kEvWarps];
  unsigned cnt[2 * kEvMaxCluster];   // pushed by every CTA: candidates above / at the threshold
  unsigned scan[kEvWarps];
  unsigned found[2];
};

// Order-preserving 32-bit key of a weight: -0 equals +0, NaN is lowest.
__device__ __forceinline__ unsigned weight_key(float w) {
  if (isnan(w)) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Ordered with the cluster barriers around it.
__device__ __forceinline__ unsigned ld_dsmem_u32_ordered(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ unsigned evict_key(const EvictParams& p, int b, int j) {
  const long long slot = paged_slot(p.c, p.c.page_table, b, p.c.max_pages, j);
  return slot < 0 ? 0u : weight_key(p.c.weight[slot]);
}

// Finds, from the counts of the cluster's CTAs, the largest bin whose suffix
// count reaches k: found[0] = bin, found[1] = how many of it are still wanted.
// Ends with a block barrier.
__device__ __forceinline__ void evict_find_bin(EvSmem& s, const unsigned* hist, int bins, int cs,
                                               unsigned k) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = bins / kEvThreads;   // 2 or 1, highest bins first
  const uint32_t at = smem_u32(hist);
  unsigned n[2] = {0, 0};
  for (int i = 0; i < per; ++i) {
    const int bin = bins - 1 - (threadIdx.x * per + i);
    unsigned v[kEvMaxCluster];
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r)
      v[r] = r < cs ? ld_dsmem_u32_ordered(mapa_shared(at + bin * 4, r)) : 0u;
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r) n[i] += v[r];
  }
  unsigned sum = n[0] + n[1], inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s.scan[warp] = inc;
  __syncthreads();
  unsigned before = 0;
  for (int w = 0; w < warp; ++w) before += s.scan[w];
  before += inc - sum;
  for (int i = 0; i < per; ++i) {
    if (before < k && before + n[i] >= k) {   // exactly one thread and bin
      s.found[0] = bins - 1 - (threadIdx.x * per + i);
      s.found[1] = k - before;
    }
    before += n[i];
  }
  __syncthreads();
}

// 16 (or 4) bytes of row `src` to row `dst` of one array, for the out-of-place copy.
template <typename V>
__device__ __forceinline__ void evict_copy(uint8_t* base, size_t row_bytes, long long dst,
                                           long long src, int at) {
  *reinterpret_cast<V*>(base + dst * row_bytes + at) =
      *reinterpret_cast<const V*>(base + src * row_bytes + at);
}

// In place: column [off, off + n_vec * sizeof(V)) of every row of one array.
// n_vec is a power of two that divides the block.
template <typename V>
__device__ __forceinline__ void evict_column(const EvictParams& p, int b, const int* kept, int r0,
                                             int count, uint8_t* base, size_t row_bytes, int off,
                                             int n_vec) {
  const int rows = kEvThreads / n_vec;          // rows per step of a chunk
  const int mine = threadIdx.x / n_vec, at = off + (threadIdx.x % n_vec) * (int)sizeof(V);
  for (int c0 = r0; c0 < count; c0 += rows * kEvBatch) {
    V v[kEvBatch];
#pragma unroll
    for (int i = 0; i < kEvBatch; ++i) {
      const int r = c0 + i * rows + mine;
      if (r < count) {
        const long long src = paged_slot(p.c, p.c.page_table, b, p.c.max_pages, kept[r]);
        if (src >= 0) v[i] = *reinterpret_cast<const V*>(base + src * row_bytes + at);
      }
    }
    __syncthreads();   // every row of the chunk is read
#pragma unroll
    for (int i = 0; i < kEvBatch; ++i) {
      const int r = c0 + i * rows + mine;
      if (r < count) {
        const long long src = paged_slot(p.c, p.c.page_table, b, p.c.max_pages, kept[r]);
        const long long dst = paged_slot(p.c, p.c.page_table, b, p.c.max_pages, r);
        if (src >= 0 && dst >= 0) *reinterpret_cast<V*>(base + dst * row_bytes + at) = v[i];
      }
    }
  }
}

// FP8: the cache has scales.
template <bool FP8>
__global__ void __launch_bounds__(kEvThreads, 1) paged_evict_kernel(const EvictParams p) {
  extern __shared__ uint8_t smem_raw[];
  EvSmem& s = *reinterpret_cast<EvSmem*>(smem_raw);
  unsigned* cache = reinterpret_cast<unsigned*>(smem_raw + sizeof(EvSmem));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cs = p.cs, rank = (int)cluster_ctarank();
  const int b = blockIdx.x / cs;
  const int len = paged_len(p.c, b);
  const int win = min(p.window, len), nc = len - win;
  const int k = min(p.topk, nc), count = k + win, slots = p.topk + p.window;
  int* kept = p.kept + (size_t)b * slots;

  if (k == nc || k == 0) {   // every candidate stays, or none
    for (int j = rank * kEvThreads + threadIdx.x; j < k; j += cs * kEvThreads) kept[j] = j;
  } else {
    // this CTA's candidates, in whole warps' runs
    const int run = ((nc + cs * kEvWarps - 1) / (cs * kEvWarps) + 31) & ~31;
    const int lo = min(nc, rank * kEvWarps * run), hi = min(nc, lo + kEvWarps * run);
    const bool cached = hi - lo <= p.cache_keys;
    for (int i = threadIdx.x; i < 2 * kEvBins; i += kEvThreads) (&s.hist[0][0])[i] = 0;
    __syncthreads();
    for (int j = lo + threadIdx.x; j < hi; j += kEvThreads) {
      const unsigned key = evict_key(p, b, j);
      if (cached) cache[j - lo] = key;
      atomicAdd(&s.hist[0][key >> 21], 1u);
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    evict_find_bin(s, s.hist[0], 2048, cs, (unsigned)k);
    unsigned prefix = s.found[0], want = s.found[1];
    for (int j = lo + threadIdx.x; j < hi; j += kEvThreads) {
      const unsigned key = cached ? cache[j - lo] : evict_key(p, b, j);
      if ((key >> 21) == prefix) atomicAdd(&s.hist[1][(key >> 10) & 2047u], 1u);
    }
    cluster_arrive_release();
    cluster_wait_acquire();   // every CTA has read the first counts
    for (int i = threadIdx.x; i < 1024; i += kEvThreads) s.hist[0][i] = 0;
    evict_find_bin(s, s.hist[1], 2048, cs, want);
    prefix = (prefix << 11) | s.found[0];
    want = s.found[1];
    for (int j = lo + threadIdx.x; j < hi; j += kEvThreads) {
      const unsigned key = cached ? cache[j - lo] : evict_key(p, b, j);
      if ((key >> 10) == prefix) atomicAdd(&s.hist[0][key & 1023u], 1u);
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    evict_find_bin(s, s.hist[0], 1024, cs, want);
    const unsigned tau = (prefix << 10) | s.found[0];
    want = s.found[1];        // candidates equal to tau that stay, lowest positions first

    // what each warp's run holds
    const int w0 = min(hi, lo + warp * run), w1 = min(hi, w0 + run);
    unsigned gt = 0, eq = 0;
    for (int j0 = w0; j0 < w1; j0 += 32) {
      const int j = j0 + lane;
      const unsigned key = j < w1 ? (cached ? cache[j - lo] : evict_key(p, b, j)) : 0u;
      gt += __popc(__ballot_sync(0xffffffffu, j < w1 && key > tau));
      eq += __popc(__ballot_sync(0xffffffffu, j < w1 && key == tau));
    }
    if (lane == 0) {
      s.warp_gt[warp] = gt;
      s.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
      const unsigned a = __reduce_add_sync(0xffffffffu, s.warp_gt[lane]);
      const unsigned e = __reduce_add_sync(0xffffffffu, s.warp_eq[lane]);
      if (lane < cs) {
        st_dsmem_u32(mapa_shared(smem_u32(&s.cnt[rank]), lane), a);
        st_dsmem_u32(mapa_shared(smem_u32(&s.cnt[kEvMaxCluster + rank]), lane), e);
      }
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    unsigned gt0 = 0, eq0 = 0;
    for (int r = 0; r < rank; ++r) gt0 += s.cnt[r], eq0 += s.cnt[kEvMaxCluster + r];
    for (int w = 0; w < warp; ++w) gt0 += s.warp_gt[w], eq0 += s.warp_eq[w];
    for (int j0 = w0; j0 < w1; j0 += 32) {
      const int j = j0 + lane;
      const unsigned key = j < w1 ? (cached ? cache[j - lo] : evict_key(p, b, j)) : 0u;
      const unsigned mg = __ballot_sync(0xffffffffu, j < w1 && key > tau);
      const unsigned me = __ballot_sync(0xffffffffu, j < w1 && key == tau);
      const unsigned below = (1u << lane) - 1u;
      const unsigned eqb = eq0 + __popc(me & below);
      const bool take = (mg >> lane & 1u) || ((me >> lane & 1u) && eqb < want);
      if (take) kept[gt0 + __popc(mg & below) + min(eqb, want)] = j;
      gt0 += __popc(mg);
      eq0 += __popc(me);
    }
  }
  for (int i = rank * kEvThreads + threadIdx.x; i < slots - k; i += cs * kEvThreads)
    kept[k + i] = i < win ? nc + i : -1;
  // the list is complete, and no CTA reads another's shared memory or its
  // length (new_len may be the lengths' own array) after this barrier
  cluster_arrive_release();
  cluster_wait_acquire();
  if (rank == 0 && threadIdx.x == 0) p.new_len[b] = count;

  const int heads = p.c.heads;
  if (p.dst_table) {
    const int vecs = p.row_bytes / 16;
    const long long total = (long long)count * (2 * vecs + (FP8 ? 2 * heads : 0) + 1);
    const int per_row = 2 * vecs + (FP8 ? 2 * heads : 0) + 1;
    for (long long u = rank * kEvThreads + threadIdx.x; u < total; u += cs * kEvThreads) {
      const int r = (int)(u / per_row), i = (int)(u - (long long)r * per_row);
      const long long src = paged_slot(p.c, p.c.page_table, b, p.c.max_pages, kept[r]);
      const long long dst = paged_slot(p.c, p.dst_table, b, p.dst_max_pages, r);
      if (src < 0 || dst < 0) continue;
      if (i < vecs) evict_copy<uint4>(p.c.k, p.row_bytes, dst, src, i * 16);
      else if (i < 2 * vecs) evict_copy<uint4>(p.c.v, p.row_bytes, dst, src, (i - vecs) * 16);
      else if (i == per_row - 1) p.c.weight[dst] = p.c.weight[src];
      else {
        const int h = i - 2 * vecs;
        float* sc = h < heads ? p.c.k_scale : p.c.v_scale;
        const int hh = h < heads ? h : h - heads;
        sc[dst * heads + hh] = sc[src * heads + hh];
      }
    }
  } else if (count < len) {
    const int cols = p.row_bytes / kEvCol;
    const int jobs = 2 * cols + 1 + (FP8 ? 2 * heads : 0);
    for (int job = rank; job < jobs; job += cs) {
      __syncthreads();
      if (job < 2 * cols)
        evict_column<uint4>(p, b, kept, 0, count, job < cols ? p.c.k : p.c.v, p.row_bytes,
                            (job % cols) * kEvCol, kEvCol / 16);
      else if (job == 2 * cols)
        evict_column<float>(p, b, kept, 0, count, reinterpret_cast<uint8_t*>(p.c.weight), 4, 0, 1);
      else {
        const int h = job - 2 * cols - 1;
        evict_column<float>(p, b, kept, 0, count,
                            reinterpret_cast<uint8_t*>(h < heads ? p.c.k_scale : p.c.v_scale),
                            (size_t)heads * 4, (h < heads ? h : h - heads) * 4, 1);
      }
    }
  }
}

}  // namespace hs2
