// The paged K/V cache, and the append of new tokens' rows to it.
//
// A pool holds n_pages pages of page_size positions (a power of two); position
// j of sequence b lives in page page_table[b][j / page_size], at place
// j % page_size.  A position's "slot" is page * page_size + place; its K and V
// rows are [kv_heads][D] at slot * kv_heads * D of the pools, its E4M3 scales
// fp32 [kv_heads], its accumulated weight one fp32.
#pragma once

#include "add_rmsnorm.cuh"

namespace hs2 {

struct PagedCache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  float* weight;
  const int* page_table;   // [B][max_pages]
  const int* seq_len;      // [B]
  int n_pages, max_pages, page_shift, B, heads;
  int scale_vec;           // one head, scales on 16 bytes: four positions' scales a load
};

// Length of sequence b's cache, held to what its page table can name (a longer
// one is reported).
__device__ __forceinline__ int paged_len(const PagedCache& c, int b) {
  const int n = c.seq_len[b];
  const long long most = (long long)c.max_pages << c.page_shift;
  if (n >= 0 && n <= most) return n;
  raise_status(kStatusBadIndex);
  return n < 0 ? 0 : (int)most;
}

// Slot of position j of sequence b; -1 (reported) when the page is not one of
// the pool's.  j is within the table's reach.
__device__ __forceinline__ long long paged_slot(const PagedCache& c, const int* table, int b,
                                                int max_pages, int j) {
  const int page = table[(size_t)b * max_pages + (j >> c.page_shift)];
  if ((unsigned)page >= (unsigned)c.n_pages) {
    raise_status(kStatusBadIndex);
    return -1;
  }
  return ((long long)page << c.page_shift) + (j & ((1 << c.page_shift) - 1));
}

// ------------------------------------------------------------------ append --
struct AppendParams {
  PagedCache c;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long ld;            // elements between two rows of k, and of v
  const int* row_start;    // [B + 1], or nullptr: row r is sequence r's one new token
  long long n_rows;
  int rows;                // tokens of a CTA
  unsigned magic;          // ceil(2^32 / lanes of a token): a division by it, exact below
                           // 2^32 / lanes (at most 2^15 lanes, or 2^10 of several tokens)
};

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 64;     // rows of a CTA at most

// A CTA takes p.rows tokens, about four units a thread: a unit is 8 elements of
// one head's K or V row of one token (a 16-byte load; a 16- or 8-byte store), D / 8
// lanes a row, the row's maximum taken by shuffles.  While the first loads are on
// their way a thread per token finds its slot (bisecting row_start, then its page:
// a chain of dependent loads, once per token).  Bound by HBM for prompts (65,536 tokens of
// D = 128 to E4M3: 14.8 us, 3.5 TB/s; the bounds of the tokens' rows, two loads before
// the first row's, are 0.6 us of it, the quotients' remainders 0.5) and by one launch's latency for a
// decode step.
template <int D, bool FP8>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8, kBatch = 4;
  __shared__ long long slots[kAppendRows];
  const int heads = p.c.heads;
  const long long row0 = (long long)blockIdx.x * p.rows;
  const int rows = (int)min((long long)p.rows, p.n_rows - row0);
  const int per_row = 2 * heads * kLanes, total = rows * per_row;
  // rows before the first sequence's and behind the last one's are not read: n_rows may be
  // an upper bound, with no memory behind the tokens
  int first = 0, last = rows;
  if (p.row_start) {
    first = (int)max(0ll, min((long long)rows, p.row_start[0] - row0));
    last = (int)max(0ll, min((long long)rows, p.row_start[p.c.B] - row0));
  }
  const int live0 = first * per_row, live1 = last * per_row;
  uint4 w[kBatch];
  auto load = [&](int u0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = u0 + i * kAppendThreads;
      w[i] = make_uint4(0, 0, 0, 0);
      if (u >= live0 && u < live1) {
        const int row = __umulhi(u, p.magic), rest = u - row * per_row, hk = rest / kLanes;
        const bool is_v = hk >= heads;               // K heads, then V heads
        w[i] = *reinterpret_cast<const uint4*>((is_v ? p.v : p.k) + (row0 + row) * p.ld +
                                               (is_v ? hk - heads : hk) * D + rest % kLanes * 8);
      }
    }
  };
  load(threadIdx.x);
  if ((int)threadIdx.x < rows) {
    const long long row = row0 + threadIdx.x;
    long long slot = -1;
    int b = (int)row, pos = 0;
    if (p.row_start) {
      int lo = 0, hi = p.c.B;    // the last b with row_start[b] <= row
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.row_start[mid + 1] <= row) lo = mid + 1;
        else hi = mid;
      }
      // rows before the first sequence's or behind the last one's are no token's
      b = lo < p.c.B && row >= p.row_start[lo] ? lo : -1;
      if (b >= 0) pos = paged_len(p.c, b) - p.row_start[b + 1] + (int)row;
    } else {
      pos = paged_len(p.c, b) - 1;
    }
    if (b >= 0) {
      if (pos >= 0) slot = paged_slot(p.c, p.c.page_table, b, p.c.max_pages, pos);
      else raise_status(kStatusBadIndex);   // more new tokens than the cache has positions
    }
    slots[threadIdx.x] = slot;
    // a new position starts with no accumulated weight
    if (p.c.weight && slot >= 0) p.c.weight[slot] = 0.f;
  }
  __syncthreads();
  // (whole warps go round, for the shuffles)
  for (int u0 = threadIdx.x; u0 < (total + 31) / 32 * 32; u0 += kBatch * kAppendThreads) {
    if (u0 != (int)threadIdx.x) load(u0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = u0 + i * kAppendThreads;
      const int row = min(rows - 1, (int)__umulhi(u, p.magic)), rest = u - row * per_row;
      const int hk = rest / kLanes, part = rest % kLanes;
      const bool is_v = hk >= heads;
      const int head = is_v ? hk - heads : hk;
      const long long slot = u < total ? slots[row] : -1;
      const size_t at = ((size_t)slot * heads + head) * D + part * 8;
      uint8_t* to = (is_v ? p.c.v : p.c.k) + at * (FP8 ? 1 : 2);
      if (!FP8) {
        if (slot >= 0) *reinterpret_cast<uint4*>(to) = w[i];
      } else {
        float x[8];
        const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        float amax = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = bf16x2_to_float2(ww[q]);
          x[2 * q] = f.x;
          x[2 * q + 1] = f.y;
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (slot >= 0) {
          float inv;
          bool far;
          const float s = e4m3_scale(amax, inv, far);
          uint32_t c[2];
          e4m3_codes<8>(x, s, inv, far, c);
          *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
          if (part == 0) (is_v ? p.c.v_scale : p.c.k_scale)[slot * heads + head] = s;
        }
      }
    }
  }
}

}  // namespace hs2
