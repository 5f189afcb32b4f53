// Eviction from a paged cache by accumulated attention weight.
//
// Sequence b of length n keeps its `window` most recent positions and, of the
// candidates j < n - window, the min(topk, .) of largest weight (ties to the
// lower position; NaN below every number).  The survivors, in ascending order,
// become positions 0, 1, ... of the sequence: row r <- row kept[r].
//
// One launch, one cluster per sequence.  The threshold is found by a radix
// search over the weights' 32-bit order (digits of 11, 11 and 10 bits).  Up to
// kEvSolo candidates every CTA of the cluster searches all of them for itself, from
// keys it keeps in shared memory: no exchange, and the cluster only shares the
// move.  More are split over the cluster: each CTA counts its part, sums its share
// of the bins over all parts through distributed shared memory and hands the sums
// to all, two barriers a digit.  (8 sequences of 32K: 19 us split, 37 us each for
// itself; of 1216: 23 us and 11 us.)  Counts
// are whole numbers, so the result does not depend on the order of the atomics.
// Survivors are then written in order from ballots: each warp owns a contiguous
// run of candidates, counts it, learns what comes before it, and writes it.
//
// The move.  Into other pages (dst_table) it is a plain copy, a few rows for every
// warp of the cluster.  In place, row r overwrites a row that an earlier move has to
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
constexpr int kEvSolo = 8 * 1024;     // keys a CTA keeps (32 KB): so many it searches alone
constexpr int kEvMaxCluster = 8;
constexpr int kEvCol = 64;            // bytes of a row that one CTA moves in place
constexpr int kEvBatch = 4;           // rows per thread and chunk, in place

struct EvictParams {
  PagedCache c;
  const int* dst_table;    // nullptr: in place
  int* kept;               // [B][topk + window]
  int* new_len;            // [B]
  int dst_max_pages, topk, window, cs, row_bytes;
  int solo;                // keys a CTA keeps: up to so many candidates it searches alone
};

struct EvSmem {
  unsigned hist[2][kEvBins];
  unsigned total[kEvBins];           // the cluster's counts
  unsigned warp_gt[kEvWarps], warp_eq[kEvWarps];
  unsigned cnt[2 * kEvMaxCluster];   // pushed by every CTA: candidates above / at the threshold
  unsigned scan[kEvWarps];   // what the warps' bins hold, then what comes before them
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

// The counts of the `cs` CTAs of a search into `total` of each: CTA r sums its
// share of the bins and hands it to all.  Begins and ends with their barrier.
__device__ __forceinline__ void evict_sum(const unsigned* hist, unsigned* total, int bins, int cs,
                                          int rank) {
  cluster_arrive_release();
  cluster_wait_acquire();
  const int share = bins / cs;
  const uint32_t from = smem_u32(hist), to = smem_u32(total);
  for (int bin = rank * share + threadIdx.x; bin < (rank + 1) * share; bin += kEvThreads) {
    unsigned v[kEvMaxCluster], n = 0;
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r)
      v[r] = r < cs ? ld_dsmem_u32_ordered(mapa_shared(from + bin * 4, r)) : 0u;
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r) n += v[r];
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r)
      if (r < cs) st_dsmem_u32(mapa_shared(to + bin * 4, r), n);
  }
  cluster_arrive_release();
  cluster_wait_acquire();
}

// Finds the largest bin whose suffix count reaches k: found[0] = bin, found[1] =
// how many of it are still wanted.  Ends with a block barrier.
__device__ __forceinline__ void evict_find_bin(EvSmem& s, const unsigned* hist, int bins,
                                               unsigned k) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = bins / kEvThreads;   // 2 or 1, highest bins first
  unsigned n[2] = {0, 0};
  for (int i = 0; i < per; ++i) n[i] = hist[bins - 1 - (threadIdx.x * per + i)];
  const unsigned sum = n[0] + n[1];
  unsigned inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s.scan[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const unsigned mine = s.scan[lane];
    unsigned up = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    s.scan[lane] = up - mine;
  }
  __syncthreads();
  unsigned before = s.scan[warp] + inc - sum;
  for (int i = 0; i < per; ++i) {
    if (before < k && before + n[i] >= k) {   // exactly one thread and bin
      s.found[0] = bins - 1 - (threadIdx.x * per + i);
      s.found[1] = k - before;
    }
    before += n[i];
  }
  __syncthreads();
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

  // the CTAs that search together, and this one's place among them
  const int scs = nc <= p.solo ? 1 : cs, srank = scs == 1 ? 0 : rank;
  if (k == nc || k == 0) {   // every candidate stays, or none
    for (int j = threadIdx.x; j < k; j += kEvThreads) kept[j] = j;
  } else {
    // this CTA's candidates, in whole warps' runs
    const int run = ((nc + scs * kEvWarps - 1) / (scs * kEvWarps) + 31) & ~31;
    const int lo = min(nc, srank * kEvWarps * run), hi = min(nc, lo + kEvWarps * run);
    const bool cached = hi - lo <= p.solo;   // (always, when it searches alone)
    for (int i = threadIdx.x; i < 2 * kEvBins; i += kEvThreads) (&s.hist[0][0])[i] = 0;
    __syncthreads();
    for (int j0 = lo + threadIdx.x; j0 < hi; j0 += 4 * kEvThreads) {
      unsigned key[4];   // four dependent pairs of loads in flight
#pragma unroll
      for (int i = 0; i < 4; ++i)
        key[i] = j0 + i * kEvThreads < hi ? evict_key(p, b, j0 + i * kEvThreads) : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j0 + i * kEvThreads < hi) {
          if (cached) cache[j0 + i * kEvThreads - lo] = key[i];
          atomicAdd(&s.hist[0][key[i] >> 21], 1u);
        }
    }
    // a digit's counts: this CTA's, or the cluster's
    auto counts = [&](const unsigned* hist, int bins) -> const unsigned* {
      if (scs == 1) {
        __syncthreads();
        return hist;
      }
      evict_sum(hist, s.total, bins, scs, rank);
      return s.total;
    };
    evict_find_bin(s, counts(s.hist[0], 2048), 2048, (unsigned)k);
    unsigned prefix = s.found[0], want = s.found[1];
    for (int j = lo + threadIdx.x; j < hi; j += kEvThreads) {
      const unsigned key = cached ? cache[j - lo] : evict_key(p, b, j);
      if ((key >> 21) == prefix) atomicAdd(&s.hist[1][(key >> 10) & 2047u], 1u);
    }
    const unsigned* second = counts(s.hist[1], 2048);   // the first counts were all read
    for (int i = threadIdx.x; i < 1024; i += kEvThreads) s.hist[0][i] = 0;
    evict_find_bin(s, second, 2048, want);
    prefix = (prefix << 11) | s.found[0];
    want = s.found[1];
    for (int j = lo + threadIdx.x; j < hi; j += kEvThreads) {
      const unsigned key = cached ? cache[j - lo] : evict_key(p, b, j);
      if ((key >> 10) == prefix) atomicAdd(&s.hist[0][key & 1023u], 1u);
    }
    evict_find_bin(s, counts(s.hist[0], 1024), 1024, want);
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
      if (scs == 1) {
        if (lane == 0) s.cnt[0] = a, s.cnt[kEvMaxCluster] = e;
      } else if (lane < cs) {
        st_dsmem_u32(mapa_shared(smem_u32(&s.cnt[rank]), lane), a);
        st_dsmem_u32(mapa_shared(smem_u32(&s.cnt[kEvMaxCluster + rank]), lane), e);
      }
    }
    if (scs == 1) {
      __syncthreads();
    } else {
      cluster_arrive_release();
      cluster_wait_acquire();
    }
    unsigned gt0 = 0, eq0 = 0;
    for (int r = 0; r < srank; ++r) gt0 += s.cnt[r], eq0 += s.cnt[kEvMaxCluster + r];
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
  for (int i = threadIdx.x; i < slots - k; i += kEvThreads) kept[k + i] = i < win ? nc + i : -1;
  // (CTAs that searched for themselves have all written the same list)
  // After this barrier the list is complete, and no CTA reads a weight, another's
  // shared memory or its length (new_len may be the lengths' own array)
  cluster_arrive_release();
  cluster_wait_acquire();
  if (rank == 0 && threadIdx.x == 0) p.new_len[b] = count;

  const int heads = p.c.heads;
  if (p.dst_table) {
    // `each` rows for every warp of the cluster; lane i finds row i's slots and
    // moves its weight and scales, then the warp moves the rows
    const int vecs = p.row_bytes / 16, warps = cs * kEvWarps;
    const int each = min(32, (count + warps - 1) / warps);
    for (int r0 = (rank * kEvWarps + warp) * each; r0 < count; r0 += warps * each) {
      const int mine = r0 + lane, n = min(each, count - r0);
      long long src = -1, dst = -1;
      if (lane < n) {
        src = paged_slot(p.c, p.c.page_table, b, p.c.max_pages, kept[mine]);
        dst = paged_slot(p.c, p.dst_table, b, p.dst_max_pages, mine);
        if (src < 0 || dst < 0) src = dst = -1;
        if (src >= 0) {
          p.c.weight[dst] = p.c.weight[src];
          if (FP8)
            for (int h = 0; h < heads; ++h) {
              p.c.k_scale[dst * heads + h] = p.c.k_scale[src * heads + h];
              p.c.v_scale[dst * heads + h] = p.c.v_scale[src * heads + h];
            }
        }
      }
      for (int i0 = 0; i0 < n * 2 * vecs; i0 += 4 * 32) {
        uint4 v[4];
        uint8_t* to[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int i = i0 + q * 32 + lane, r = min(n - 1, i / (2 * vecs)), at = i % (2 * vecs);
          const long long rs = __shfl_sync(0xffffffffu, src, r), rd = __shfl_sync(0xffffffffu, dst, r);
          uint8_t* base = at < vecs ? p.c.k : p.c.v;
          const size_t off = (size_t)(at < vecs ? at : at - vecs) * 16;
          to[q] = i < n * 2 * vecs && rs >= 0 ? base + rd * p.row_bytes + off : nullptr;
          if (to[q]) v[q] = *reinterpret_cast<const uint4*>(base + rs * p.row_bytes + off);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (to[q]) *reinterpret_cast<uint4*>(to[q]) = v[q];
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
