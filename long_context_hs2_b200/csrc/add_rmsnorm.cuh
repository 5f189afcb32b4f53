// RMS norm with the residual's addition, and its output in bf16 or in E4M3
// with one scale per 128 columns.
//
//   h = X + R,  y = h * gamma / sqrt(mean(h^2) + eps),
//   per block of 128 columns: s = max|y| / 448 (1 where that is 0), code = E4M3(y / s)
//
// One pass: a row's values stay in registers between the sum of squares and
// the output, so every input is read once and every output written once, and
// HBM bounds it (131,072 x 4096 with residual to E4M3: 534 us in a replayed graph, 7.1 TB/s
// with the tail of the writes in L2; 8 rows: 2.4 us, a launch).  A thread owns chunks of 16 columns (two 16-byte loads of X
// and of R, one 16-byte store of codes); a block of 128 columns is then 8
// neighbouring lanes, and its maximum three shuffles.  h is kept in fp32 for
// the norm: the sum's rounding to bf16 goes to the residual stream only.
#pragma once

#include "paged_common.cuh"

namespace hs2 {

constexpr int kNormChunk = 16;        // columns of one thread's chunk
constexpr int kNormBlock = 128;       // columns that share an E4M3 scale
constexpr int kNormMaxThreads = 512;  // threads per row at most
constexpr int kNormMaxHidden = kNormMaxThreads * kNormChunk * 4;

struct NormParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* r;       // nullptr: no residual
  const __nv_bfloat16* gamma;
  __nv_bfloat16* sum;           // nullptr: h is not written
  __nv_bfloat16* y;             // nullptr: no bf16 output
  uint8_t* codes;               // nullptr: no E4M3 output
  float* scale;
  long long T;
  int hidden, n_chunks, n_blocks;
  int lanes;                    // of a row, where a warp has several
  float eps;
};

// The scale of values whose largest magnitude is amax, and an approximate 1 / s for their
// quotients.  Scales so small or so large that a quotient's remainder or 1 / s is not a
// normal number (infinite ones among them) are flagged (`far`), and their values divided.
__device__ __forceinline__ float e4m3_scale(float amax, float& inv, bool& far) {
  const float q = __fdiv_rn(amax, 448.f);
  const float s = q > 0.f ? q : 1.f;
  far = !(s >= 0x1p-80f && s <= 0x1p100f);
  inv = fast_rcp(s);
  return s;
}
// a b + c and a b of two values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// Two v / s: the product with 1 / s, corrected by its remainder, which is exact (Markstein,
// IBM J. Res. Dev. 34, 1990).  bf16 values often lie half-way between two codes, where the
// product alone went either way.
__device__ __forceinline__ float2 e4m3_quotients(float a, float b, float s, float inv) {
  const float2 v = make_float2(a, b), q = mul2(v, make_float2(inv, inv));
  const float2 rest = fma2(q, make_float2(s, s), make_float2(-a, -b));
  return fma2(rest, make_float2(-inv, -inv), q);   // (in these signs a -0 stays one)
}
// Four values as E4M3 codes (round to nearest even, saturating), first one lowest.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo =
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi =
      __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// v / s as codes, N values into N / 4 words.
template <int N>
__device__ __forceinline__ void e4m3_codes(const float* v, float s, float inv, bool far,
                                           uint32_t* w) {
  if (!far) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float2 a = e4m3_quotients(v[i], v[i + 1], s, inv);
      const float2 b = e4m3_quotients(v[i + 2], v[i + 3], s, inv);
      w[i / 4] = e4m3_pack4(a.x, a.y, b.x, b.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      w[i / 4] = e4m3_pack4(__fdiv_rn(v[i], s), __fdiv_rn(v[i + 1], s), __fdiv_rn(v[i + 2], s),
                            __fdiv_rn(v[i + 3], s));
  }
}

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void load_bf16x16(const __nv_bfloat16* p, uint32_t* w) {
  const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}
__device__ __forceinline__ void store_bf16x16(__nv_bfloat16* p, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// NC chunks per thread.  kWarpRow: rows of at most 32 chunks, each on p.lanes lanes
// (the power of two that holds its chunks), several to a warp (76,217 x 80: 8.9 us,
// 24.6 with a warp per row); else one row per CTA.
template <int NC, bool kWarpRow>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_kernel(const NormParams p) {
  __shared__ float part[kNormMaxThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = kWarpRow ? p.lanes : 32;
  const long long row =
      kWarpRow ? ((long long)blockIdx.x * blockDim.x + threadIdx.x) / lanes : (long long)blockIdx.x;
  const bool here = !kWarpRow || row < p.T;
  const int stride = kWarpRow ? 32 : blockDim.x;
  const int first = kWarpRow ? (lane & (lanes - 1)) : threadIdx.x;
  const size_t base = (size_t)row * p.hidden;

  float h[NC][kNormChunk];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = first + i * stride;
    if (here && c < p.n_chunks) {
      const size_t at = base + (size_t)c * kNormChunk;
      uint32_t xw[8];
      load_bf16x16(p.x + at, xw);
      if (p.r) {
        uint32_t rw[8];
        load_bf16x16(p.r + at, rw);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 a = bf16x2_to_float2(xw[q]), b = bf16x2_to_float2(rw[q]);
          h[i][2 * q] = a.x + b.x;
          h[i][2 * q + 1] = a.y + b.y;
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 a = bf16x2_to_float2(xw[q]);
          h[i][2 * q] = a.x;
          h[i][2 * q + 1] = a.y;
        }
      }
#pragma unroll
      for (int q = 0; q < kNormChunk; ++q) ss = fmaf(h[i][q], h[i][q], ss);
      if (p.sum) store_bf16x16(p.sum + at, h[i]);
    } else {
#pragma unroll
      for (int q = 0; q < kNormChunk; ++q) h[i][q] = 0.f;
    }
  }
  for (int o = lanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (!kWarpRow) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) ss += part[w];
  }
  const float f = 1.f / sqrtf(ss / (float)p.hidden + p.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = first + i * stride;
    const bool live = here && c < p.n_chunks;
    const size_t at = base + (size_t)c * kNormChunk;
    if (live) {
      uint32_t gw[8];
      load_bf16x16(p.gamma + (size_t)c * kNormChunk, gw);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 g = bf16x2_to_float2(gw[q]);
        h[i][2 * q] = h[i][2 * q] * f * g.x;
        h[i][2 * q + 1] = h[i][2 * q + 1] * f * g.y;
      }
      if (p.y) store_bf16x16(p.y + at, h[i]);
    }
    if (p.codes) {   // every lane takes part in the shuffles
      float amax = 0.f;
#pragma unroll
      for (int q = 0; q < kNormChunk; ++q) amax = fmaxf(amax, fabsf(h[i][q]));
      for (int o = min(8, lanes) / 2; o; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (live) {
        float inv;
        bool far;
        const float s = e4m3_scale(amax, inv, far);
        uint32_t w[4];
        e4m3_codes<kNormChunk>(h[i], s, inv, far, w);
        *reinterpret_cast<uint4*>(p.codes + at) = make_uint4(w[0], w[1], w[2], w[3]);
        if ((c & 7) == 0) p.scale[(size_t)row * p.n_blocks + (c >> 3)] = s;
      }
    }
  }
}

}  // namespace hs2
