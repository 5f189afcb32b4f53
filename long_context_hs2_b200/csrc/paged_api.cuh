// Host side of the paged decode path's entry points (see include/hs2.h):
// argument checks, launch plans, launches.  Included by hs2_lib.cu after
// hs2_api.cu, whose helpers it uses.
#pragma once

#include "add_rmsnorm.cuh"
#include "fp8_gemm.cuh"
#include "paged_attn.cuh"
#include "paged_attn_tc.cuh"
#include "paged_cache.cuh"
#include "paged_evict.cuh"

namespace {

// --------------------------------------------------------- argument checks --
// The pool and its table: pointers, alignment, the page size, and that every
// position and slot is a 31-bit number.
hs2_status check_paged(const hs2_paged_cache* c, int B, int heads, int D, hs2_kv_dtype dt) {
  if (!c || !c->kv.k || !c->kv.v || !c->page_table || !c->seq_len) return HS2_ERR_INVALID_ARG;
  if (!aligned16(c->kv.k) || !aligned16(c->kv.v) || !aligned4(c->page_table) ||
      !aligned4(c->seq_len) || (c->weight && !aligned4(c->weight)))
    return HS2_ERR_INVALID_ARG;
  if (B < 1 || heads < 1 || D < 1 || c->n_pages < 1 || c->page_size < 1 || c->max_pages < 1)
    return HS2_ERR_INVALID_ARG;
  if (dt != HS2_KV_BF16 && dt != HS2_KV_FP8_E4M3) return HS2_ERR_INVALID_ARG;
  if (dt == HS2_KV_FP8_E4M3 && (!c->kv.k_scale || !c->kv.v_scale || !aligned4(c->kv.k_scale) ||
                                !aligned4(c->kv.v_scale)))
    return HS2_ERR_INVALID_ARG;
  if (!(D == 64 || D == 128) || heads > 1024 || B > 65535 ||
      (c->page_size & (c->page_size - 1)) != 0)
    return HS2_ERR_UNSUPPORTED;
  if ((int64_t)c->n_pages * c->page_size > INT32_MAX ||
      (int64_t)c->max_pages * c->page_size > (1 << 30))
    return HS2_ERR_UNSUPPORTED;
  return HS2_OK;
}

PagedCache paged_params(const hs2_paged_cache* c, int B, int heads, hs2_kv_dtype dt) {
  PagedCache p;
  p.k = static_cast<uint8_t*>(c->kv.k);
  p.v = static_cast<uint8_t*>(c->kv.v);
  p.k_scale = dt == HS2_KV_FP8_E4M3 ? c->kv.k_scale : nullptr;
  p.v_scale = dt == HS2_KV_FP8_E4M3 ? c->kv.v_scale : nullptr;
  p.weight = c->weight;
  p.page_table = c->page_table;
  p.seq_len = c->seq_len;
  p.n_pages = c->n_pages;
  p.max_pages = c->max_pages;
  p.page_shift = __builtin_ctz((unsigned)c->page_size);
  p.B = B;
  p.heads = heads;
  p.scale_vec = heads == 1 && aligned16(p.k_scale) && aligned16(p.v_scale);
  return p;
}

// A K or V pool as [slots][heads][D], boxes of `rows` slots of one head.
bool make_map_pool(CUtensorMap* map, const void* base, uint64_t slots, int heads, int D, int elem,
                   uint32_t rows) {
  const cuuint64_t row = (cuuint64_t)D * elem;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, slots};
  cuuint64_t strides[2] = {row, row * heads};
  const uint32_t cols = (uint32_t)std::min(D, 128 / elem);
  cuuint32_t box[3] = {cols, 1, rows};
  return encode_tiled(
      map, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base,
      dims, strides, box,
      cols * elem == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// ----------------------------------------------------------- attention plan --
struct PagedPlan {
  int grid;
  size_t off_lse, off_ml, off_o, total;
};

bool check_heads(int H, int heads) { return heads >= 1 && H >= 1 && H % heads == 0; }

PagedPlan paged_plan(int B, int H, int heads, int D) {
  PagedPlan pl;
  pl.grid = std::min(sm_count(), kPaMaxParts);
  const size_t G = (size_t)(H / heads);
  pl.off_lse = 0;
  pl.off_ml = align_up((size_t)B * H * 4, 256);
  pl.off_o = align_up(pl.off_ml + (size_t)pl.grid * 2 * G * 8, 256);
  pl.total = align_up(pl.off_o + (size_t)pl.grid * 2 * G * D * 4, 256);
  return pl;
}

template <int MT, int D, bool FP8>
hs2_status run_paged_attn(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnParams& p,
                          bool weight, cudaStream_t s) {
  using SM = PaSmem<MT, D, FP8, false>;
  using SW = PaSmem<MT, D, FP8, true>;
  auto kw = paged_weight_kernel<MT, D, FP8>;
  hs2_status st;
  // tcgen05 for head_dim 128 where a page's rows are a TMA box of whole swizzle atoms (4 x
  // 256K E4M3: 86 us against 122 with warp MMAs; 8 x up to 32K bf16: 18 against 30)
  if (D == 128 && p.c.page_shift >= 3) {
    using ST = PtSmem<16 * MT, FP8>;
    auto k = paged_attn_tc_kernel<16 * MT, FP8>;
    if (!set_smem(k, ST::kBytes)) return HS2_ERR_CUDA;
    st = launch(k, dim3(p.grid), dim3(ST::kThreads), ST::kBytes, s, 1, km, vm, p);
  } else {
    auto k = paged_attn_kernel<MT, D, FP8>;
    if (!set_smem(k, SM::kBytes)) return HS2_ERR_CUDA;
    st = launch(k, dim3(p.grid), dim3(kPaAttnThreads<MT, D>), SM::kBytes, s, 1, km, vm, p);
  }
  if (st != HS2_OK) return st;
  if (weight && D == 128 && p.c.page_shift >= 3 && p.c.heads * 16 * MT <= kPwRows) {
    // joins the parts as well
    using SP = PwSmem<16 * MT, FP8>;
    auto k = paged_weight_tc_kernel<16 * MT, FP8>;
    if (!set_smem(k, SP::kBytes)) return HS2_ERR_CUDA;
    return launch_ex(k, dim3(p.grid), dim3(SP::kThreads), SP::kBytes, s, 1, false, true, km, p);
  }
  st = launch_ex(paged_attn_combine_kernel<D>, dim3((unsigned)(p.c.B * p.H)), dim3(D), 0, s, 1,
                 false, true, p);
  if (st != HS2_OK || !weight) return st;
  if (!set_smem(kw, SW::kBytes)) return HS2_ERR_CUDA;
  return launch_ex(kw, dim3(p.grid), dim3(kPaThreads), SW::kBytes, s, 1, false, true, km, p);
}

// ------------------------------------------------------------- E4M3 product --
template <int BN, int CW>
hs2_status run_fp8_gemm(const void* A, const void* B, Fp8GemmParams p, cudaStream_t s) {
  using SM = FgSmem<BN, CW>;
  CUtensorMap am, bm;
  if (!make_map_2d(&am, A, (uint64_t)p.M, (uint64_t)p.K, 1, kFgBK, 128) ||
      !make_map_2d(&bm, B, (uint64_t)p.N, (uint64_t)p.K, 1, kFgBK, BN))
    return HS2_ERR_CUDA;
  p.m_tiles = (p.M + 127) / 128;
  p.n_tiles = (p.N + BN - 1) / BN;
  auto k = fp8_gemm_kernel<BN, CW>;
  if (!set_smem(k, SM::kBytes)) return HS2_ERR_CUDA;
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
  if (tiles > INT32_MAX) return HS2_ERR_UNSUPPORTED;
  return launch(k, dim3((unsigned)std::min<int64_t>(tiles, sm_count())), dim3(SM::kThreads),
                SM::kBytes, s, 1, am, bm, p);
}

template <int NP>
hs2_status run_fp8_gemm_small(const void* A, const void* B, Fp8GemmParams p, cudaStream_t s) {
  using SM = FsSmem<NP>;
  CUtensorMap am, bm;
  if (!make_map_2d(&am, A, (uint64_t)p.M, (uint64_t)p.K, 1, kFgBK, NP) ||
      !make_map_2d(&bm, B, (uint64_t)p.N, (uint64_t)p.K, 1, kFgBK, 128))
    return HS2_ERR_CUDA;
  p.m_tiles = (p.M + NP - 1) / NP;
  p.n_tiles = (p.N + 127) / 128;
  const int64_t segs = (int64_t)p.m_tiles * p.n_tiles;
  int cs = kFsMaxCluster;
  while (cs > 1 && (segs * cs > sm_count() || cs > p.kb)) cs /= 2;
  auto k = fp8_gemm_small_kernel<NP>;
  if (!set_smem(k, SM::kBytes)) return HS2_ERR_CUDA;
  if (segs * cs > INT32_MAX) return HS2_ERR_UNSUPPORTED;
  return launch(k, dim3((unsigned)(segs * cs)), dim3(kFsThreads), SM::kBytes, s, cs, am, bm, p,
                cs);
}

}  // namespace

extern "C" {

hs2_status hs2_fp8_gemm(const void* A, const float* A_scale, int64_t M, const void* B,
                        const float* B_scale, int N, int K, void* C, hs2_stream_t stream) {
  if (!A || !A_scale || !B || !B_scale || !C || M < 1 || N < 1 || K < 1) return HS2_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(B) || !aligned16(C) || !aligned4(A_scale) || !aligned4(B_scale))
    return HS2_ERR_INVALID_ARG;
  if (K % 16 != 0 || M > INT32_MAX - 128 || N > INT32_MAX - 256 || K > INT32_MAX - 128)
    return HS2_ERR_UNSUPPORTED;
  Fp8GemmParams p;
  p.sa = A_scale;
  p.sb = B_scale;
  p.c = static_cast<__nv_bfloat16*>(C);
  p.M = (int)M;
  p.N = N;
  p.K = K;
  p.kb = (K + kFgBK - 1) / kFgBK;
  cudaStream_t s = (cudaStream_t)stream;
  // Few rows: the whole machine streams B (8 rows x 1536 x 4096: 5.5 us against 12.0 with
  // the tiles of many rows; 64 rows: 12.3 us against 10.9, so not from there on).
  if (M <= 16) return run_fp8_gemm_small<16>(A, B, p, s);
  if (M <= 32) return run_fp8_gemm_small<32>(A, B, p, s);
  // Many rows: the tile width whose waves cost least.  A wave of K = 4096 takes 11.0, 14.5
  // and 23.5 us with 64, 128 and 256 columns (1003 x 1536: 21.5, 15.3, 24.2 us; 100 x 1536:
  // 11.2, 13.9, 22.3; 2048 x 6144: 101, 76, 66).
  const int64_t mt = (M + 127) / 128, sms = sm_count();
  auto cost = [&](int64_t bn, int64_t wave) {
    return (mt * ((N + bn - 1) / bn) + sms - 1) / sms * wave;
  };
  const int64_t c64 = cost(64, 110), c128 = cost(128, 145), c256 = cost(256, 235);
  if (c256 <= c128 && c256 <= c64) return run_fp8_gemm<256, 8>(A, B, p, s);
  if (c128 <= c64) return run_fp8_gemm<128, 8>(A, B, p, s);
  return run_fp8_gemm<64, 4>(A, B, p, s);
}

hs2_status hs2_add_rmsnorm(const void* X, const void* R, const void* gamma, int64_t T, int hidden,
                           float eps, void* sum, void* Y, void* Yq, float* Yq_scale,
                           hs2_stream_t stream) {
  if (!X || !gamma || (!sum && !Y && !Yq) || T < 1 || hidden < 1 || !(eps >= 0.f) ||
      !std::isfinite(eps))
    return HS2_ERR_INVALID_ARG;
  if (!aligned16(X) || (R && !aligned16(R)) || !aligned16(gamma) || (sum && !aligned16(sum)) ||
      (Y && !aligned16(Y)) || (Yq && !aligned16(Yq)))
    return HS2_ERR_INVALID_ARG;
  if ((Yq == nullptr) != (Yq_scale == nullptr) || (Yq_scale && !aligned4(Yq_scale)))
    return HS2_ERR_INVALID_ARG;
  if (hidden % kNormChunk != 0 || hidden > kNormMaxHidden || T > INT32_MAX)
    return HS2_ERR_UNSUPPORTED;
  NormParams p;
  p.x = static_cast<const __nv_bfloat16*>(X);
  p.r = static_cast<const __nv_bfloat16*>(R);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma);
  p.sum = static_cast<__nv_bfloat16*>(sum);
  p.y = static_cast<__nv_bfloat16*>(Y);
  p.codes = static_cast<uint8_t*>(Yq);
  p.scale = Yq_scale;
  p.T = T;
  p.hidden = hidden;
  p.n_chunks = hidden / kNormChunk;
  p.n_blocks = (hidden + kNormBlock - 1) / kNormBlock;
  p.eps = eps;
  cudaStream_t s = (cudaStream_t)stream;
  p.lanes = 32;
  if (p.n_chunks <= 32) {   // several rows to a warp, four warps to a CTA
    while (p.lanes / 2 >= p.n_chunks) p.lanes /= 2;
    const int64_t rows = 128 / p.lanes;
    return launch(add_rmsnorm_kernel<1, true>, dim3((unsigned)((T + rows - 1) / rows)), dim3(128),
                  0, s, 1, p);
  }
  const int nc = (p.n_chunks + kNormMaxThreads - 1) / kNormMaxThreads;
  const int threads = ((p.n_chunks + nc - 1) / nc + 31) / 32 * 32;
  auto k = nc == 1 ? add_rmsnorm_kernel<1, false>
                   : nc == 2 ? add_rmsnorm_kernel<2, false> : add_rmsnorm_kernel<4, false>;
  return launch(k, dim3((unsigned)T), dim3(threads), 0, s, 1, p);
}

hs2_status hs2_paged_append(const void* K, const void* V, int64_t ld, int64_t n_rows,
                            const int32_t* row_start, const hs2_paged_cache* cache, int B,
                            int kv_heads, int D, hs2_kv_dtype dt, hs2_stream_t stream) {
  if (!K || !V || !aligned16(K) || !aligned16(V) || n_rows < 1 ||
      (row_start && !aligned4(row_start)))
    return HS2_ERR_INVALID_ARG;
  const hs2_status st = check_paged(cache, B, kv_heads, D, dt);
  if (st != HS2_OK) return st;
  if (ld < (int64_t)kv_heads * D || ld % 8 != 0 || (!row_start && n_rows != B))
    return HS2_ERR_INVALID_ARG;
  if (n_rows > INT32_MAX - kAppendRows) return HS2_ERR_UNSUPPORTED;
  AppendParams p;
  p.c = paged_params(cache, B, kv_heads, dt);
  p.k = static_cast<const __nv_bfloat16*>(K);
  p.v = static_cast<const __nv_bfloat16*>(V);
  p.ld = ld;
  p.row_start = row_start;
  p.n_rows = n_rows;
  // four units a thread, unless that leaves SMs without a CTA
  const int lanes = 2 * kv_heads * (D / 8);
  p.magic = (unsigned)(((1ull << 32) + lanes - 1) / lanes);
  const int64_t four = 4 * kAppendThreads / lanes;
  p.rows = (int)std::max<int64_t>(
      1, std::min<int64_t>(std::min<int64_t>(kAppendRows, four), n_rows / sm_count()));
  const bool fp8 = dt == HS2_KV_FP8_E4M3;
  auto k = D == 128 ? (fp8 ? paged_append_kernel<128, true> : paged_append_kernel<128, false>)
                    : (fp8 ? paged_append_kernel<64, true> : paged_append_kernel<64, false>);
  return launch(k, dim3((unsigned)((n_rows + p.rows - 1) / p.rows)), dim3(kAppendThreads), 0,
                (cudaStream_t)stream, 1, p);
}

size_t hs2_paged_attn_workspace(int B, int H, int kv_heads, int D) {
  if (B < 1 || B > 65535 || !check_heads(H, kv_heads) || H / kv_heads > 32 || kv_heads > 1024 ||
      !(D == 64 || D == 128) || (int64_t)B * H > INT32_MAX)
    return 0;
  return paged_plan(B, H, kv_heads, D).total;
}

hs2_status hs2_paged_attn(const void* Q, const hs2_paged_cache* cache, int B, int H, int kv_heads,
                          int D, float scale, hs2_kv_dtype dt, void* O, float* lse,
                          int accumulate, void* workspace, size_t workspace_bytes,
                          hs2_stream_t stream) {
  if (!Q || !O || !aligned16(Q) || !aligned16(O) || (lse && !aligned4(lse)) ||
      !std::isfinite(scale))
    return HS2_ERR_INVALID_ARG;
  hs2_status st = check_paged(cache, B, kv_heads, D, dt);
  if (st != HS2_OK) return st;
  if (!check_heads(H, kv_heads) || (accumulate && !cache->weight)) return HS2_ERR_INVALID_ARG;
  // tiles and shares are counted in 31 bits
  const int64_t tiles = ((int64_t)cache->max_pages * cache->page_size + kPaTile - 1) / kPaTile;
  if (H / kv_heads > 32 || (int64_t)B * H > INT32_MAX || tiles * B * kv_heads > INT32_MAX - 1024)
    return HS2_ERR_UNSUPPORTED;
  const PagedPlan pl = paged_plan(B, H, kv_heads, D);
  if (!workspace || !aligned16(workspace) || workspace_bytes < pl.total)
    return HS2_ERR_WORKSPACE;
  const bool fp8 = dt == HS2_KV_FP8_E4M3;
  // a page's rows in a tile are one box; pages under 8 rows are not copied by
  // TMA, and the maps then only have to be valid
  const uint32_t rows = (uint32_t)std::min(128, std::max(8, cache->page_size));
  const uint64_t slots = (uint64_t)cache->n_pages * cache->page_size;
  CUtensorMap km, vm;
  if (!make_map_pool(&km, cache->kv.k, slots, kv_heads, D, fp8 ? 1 : 2, rows) ||
      !make_map_pool(&vm, cache->kv.v, slots, kv_heads, D, fp8 ? 1 : 2, rows))
    return HS2_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PagedAttnParams p;
  p.c = paged_params(cache, B, kv_heads, dt);
  p.q = static_cast<const __nv_bfloat16*>(Q);
  p.o = static_cast<__nv_bfloat16*>(O);
  p.lse_out = lse;
  p.lse = reinterpret_cast<float*>(ws + pl.off_lse);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.off_ml);
  p.part_o = reinterpret_cast<float*>(ws + pl.off_o);
  p.H = H;
  p.G = H / kv_heads;
  p.grid = pl.grid;
  p.scale_log2 = scale * kPaLog2e;
  cudaStream_t s = (cudaStream_t)stream;
  const bool w = accumulate != 0;
  if (p.G > 16) {
    if (D == 128) return fp8 ? run_paged_attn<2, 128, true>(km, vm, p, w, s)
                             : run_paged_attn<2, 128, false>(km, vm, p, w, s);
    return fp8 ? run_paged_attn<2, 64, true>(km, vm, p, w, s)
               : run_paged_attn<2, 64, false>(km, vm, p, w, s);
  }
  if (D == 128) return fp8 ? run_paged_attn<1, 128, true>(km, vm, p, w, s)
                           : run_paged_attn<1, 128, false>(km, vm, p, w, s);
  return fp8 ? run_paged_attn<1, 64, true>(km, vm, p, w, s)
             : run_paged_attn<1, 64, false>(km, vm, p, w, s);
}

hs2_status hs2_paged_evict(const hs2_paged_cache* cache, int B, int kv_heads, int D,
                           hs2_kv_dtype dt, int topk, int window, const int32_t* dst_table,
                           int dst_max_pages, int32_t* kept, int32_t* new_len,
                           hs2_stream_t stream) {
  if (!kept || !new_len || !aligned4(kept) || !aligned4(new_len) ||
      (dst_table && !aligned4(dst_table)) || topk < 0 || window < 1)
    return HS2_ERR_INVALID_ARG;
  const hs2_status st = check_paged(cache, B, kv_heads, D, dt);
  if (st != HS2_OK) return st;
  if (!cache->weight) return HS2_ERR_INVALID_ARG;
  const int64_t reach = (int64_t)cache->max_pages * cache->page_size;
  const int64_t most = std::min<int64_t>((int64_t)topk + window, reach);
  if (dst_table && (dst_max_pages < 1 || (int64_t)dst_max_pages * cache->page_size < most))
    return HS2_ERR_INVALID_ARG;
  if ((int64_t)topk + window > (1 << 24)) return HS2_ERR_UNSUPPORTED;
  EvictParams p;
  const bool fp8 = dt == HS2_KV_FP8_E4M3;
  p.c = paged_params(cache, B, kv_heads, dt);
  p.dst_table = dst_table == cache->page_table ? nullptr : dst_table;
  p.kept = kept;
  p.new_len = new_len;
  p.dst_max_pages = dst_max_pages;
  p.topk = topk;
  p.window = window;
  p.row_bytes = kv_heads * D * (fp8 ? 1 : 2);
  // the largest clusters that are all resident at once, with one CTA per SM, as if five
  // sixths of the SMs took them: on 148 SMs 15 of 8 fit and 16 do not (1,216 positions: 14 us
  // in clusters of 4, 23 of 8), 31 of 4 would and 34 do not (31 sequences: 18 us in clusters of
  // 2, 15 of 4, 57 and 25 of 32K; 34 sequences: 18 and 26)
  int cs = kEvMaxCluster;
  while (cs > 1 && B * cs > sm_count() * 5 / 6) cs /= 2;
  p.cs = cs;
  // shared memory for the keys that a CTA keeps
  p.solo = (int)std::min<int64_t>(kEvSolo, std::max<int64_t>(1, reach - window));
  const size_t bytes = sizeof(EvSmem) + (size_t)p.solo * 4;
  auto k = fp8 ? paged_evict_kernel<true> : paged_evict_kernel<false>;
  if (!set_smem(k, (int)sizeof(EvSmem) + kEvSolo * 4)) return HS2_ERR_CUDA;
  return launch(k, dim3((unsigned)(B * cs)), dim3(kEvThreads), bytes, (cudaStream_t)stream, cs, p);
}

}  // extern "C"
