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
  long long n_units;       // rows * 2 * heads
};

constexpr int kAppendThreads = 256;

// One unit is one head's K or V row of one token: D / 8 lanes with 8 elements
// each (a 16-byte load; a 16- or 8-byte store), the row's maximum taken by
// shuffles.  Bound by HBM for prompts and by one launch's latency for a
// decode step; a sequence is found by bisecting row_start.
template <int D, bool FP8>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;
  const long long tid = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
  const long long unit = tid / kLanes;
  const int part = (int)(tid % kLanes);
  const int heads = p.c.heads;
  const bool live = unit < p.n_units;
  const long long row = live ? unit / (2 * heads) : 0;
  const int hk = (int)(unit - row * 2 * heads);     // K heads, then V heads
  const bool is_v = hk >= heads;
  const int head = is_v ? hk - heads : hk;

  long long slot = -1;
  uint4 w = make_uint4(0, 0, 0, 0);
  if (live) {
    w = *reinterpret_cast<const uint4*>((is_v ? p.v : p.k) + row * p.ld + head * D + part * 8);
    int b = (int)row, pos;
    if (p.row_start) {
      int lo = 0, hi = p.c.B;    // the last b with row_start[b] <= row
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.row_start[mid + 1] <= row) lo = mid + 1;
        else hi = mid;
      }
      b = lo;
      // rows before the first sequence's or behind the last one's are no token's
      if (b < p.c.B && row >= p.row_start[b])
        pos = paged_len(p.c, b) - p.row_start[b + 1] + (int)row;
      else
        b = -1, pos = 0;
    } else {
      pos = paged_len(p.c, b) - 1;
    }
    if (b >= 0) {
      if (pos >= 0) slot = paged_slot(p.c, p.c.page_table, b, p.c.max_pages, pos);
      else raise_status(kStatusBadIndex);   // more new tokens than the cache has positions
    }
  }
  const size_t at = slot < 0 ? 0 : ((size_t)slot * heads + head) * D + part * 8;
  uint8_t* pool = is_v ? p.c.v : p.c.k;
  if (!FP8) {
    if (slot >= 0) *reinterpret_cast<uint4*>(pool + at * 2) = w;
  } else {
    float x[8];
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_float2(ww[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (slot >= 0) {
      float inv;
      bool tiny;
      const float s = e4m3_scale(amax, inv, tiny);
      uint32_t c[2];
      e4m3_codes<8>(x, s, inv, tiny, c);
      *reinterpret_cast<uint2*>(pool + at) = make_uint2(c[0], c[1]);
      if (part == 0) (is_v ? p.c.v_scale : p.c.k_scale)[slot * heads + head] = s;
    }
  }
  // a new position starts with no accumulated weight
  if (p.c.weight && slot >= 0 && hk == 0 && part == 0) p.c.weight[slot] = 0.f;
}

}  // namespace hs2
