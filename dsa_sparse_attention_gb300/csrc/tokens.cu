// tokens.cu — new tokens' records into the pages of the cache (dsa_write_tokens), and the
// values of cached positions out of them (dsa_read_tokens).
//
// Both are bound by the bytes they move: 1,408 bytes of bf16 values a token on one side and
// 708 (FP8) or 420 (FP4) of records on the other.  A thread takes 16 values, 32 bytes of bf16,
// whatever the format: 8 threads a key, 36 a latent, so that neighbouring threads touch
// neighbouring bytes on both sides.
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/dsa.h"
#include "prompt.cuh"
#include "ptx_prompt.cuh"

namespace dsa {

namespace {

constexpr int kKeyUnits = kIdxDim / 16;    // 8
constexpr int kLatUnits = kLatDim / 16;    // 36
constexpr int kTokThreads = 256;
constexpr int kWriteToks = 64;             // tokens of a CTA at most
constexpr int kReadRows = 32;              // rows of a CTA at most

// Where a token's records lie.
struct Place {
  int64_t row;   // row of the pool, -1: none
  int slot;
};

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// e2m1 codes of 16 values, packed two a byte.
__device__ __forceinline__ uint2 to_e2m1x16(const float* v) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t byte = __nv_cvt_float2_to_fp4x2(make_float2(v[2 * j], v[2 * j + 1]), __NV_E2M1, cudaRoundNearest);
    w[j >> 2] |= (byte & 0xFFu) << (8 * (j & 3));
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void load16(const __nv_bfloat16* src, float* v) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(src)), b = __ldg(reinterpret_cast<const uint4*>(src) + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// As whole sectors where the destination is 32-byte aligned.
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float* v, bool aligned32) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (aligned32) {
    st_global_v8(dst, w);
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ float abs_max16(const float* v) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(v[j]));
  return m;
}

// Row and slot of position `pos` of request `req`, both in range.
__device__ __forceinline__ Place place_of(const BatchView& b, const PoolView& pool, int req, int pos, uint32_t* status) {
  const int64_t blk = pos >> pool.log2_bs;
  const int64_t row = __ldg(b.bt + static_cast<int64_t>(req) * b.bt_stride + blk);
  if (row < 0 || row >= pool.num_rows) {
    atomicOr(status, DEV_BAD_BLOCK);
    return {-1, 0};
  }
  return {row, pos & (pool.bs - 1)};
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// 16 values of e4m3 codes.
__device__ __forceinline__ void from_e4m3x16(uint4 c, float* v) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// 16 values of packed e2m1 codes.
__device__ __forceinline__ void from_e2m1x16(uint2 c, float* v) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(w[j >> 2] >> (8 * (j & 3))), __NV_E2M1);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

}  // namespace

__global__ void __launch_bounds__(kTokThreads) write_tokens_kernel(WriteTokensParams p) {
  __shared__ Place place[kWriteToks];
  grid_dep_launch();
  grid_dep_wait();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.cta_toks;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.cta_toks), p.b.T - t0));
  if (threadIdx.x < nt) {
    const int t = static_cast<int>(t0) + threadIdx.x;
    const int req = __ldg(p.b.q_req + t), pos = __ldg(p.b.q_pos + t);
    Place pl = {-1, 0};
    if (req >= 0) {   // negative: padding
      bool bad = req >= p.b.B;
      if (!bad) {
        const int len = __ldg(p.b.ctx_lens + req);
        bad = len > p.b.max_ctx || pos < 0 || pos >= len;
      }
      if (bad) atomicOr(p.status, DEV_BAD_BATCH);
      else pl = place_of(p.b, p.pool, req, pos, p.status);
    }
    place[threadIdx.x] = pl;
  }
  __syncthreads();
  const bool mx = p.pool.idx_fmt == DSA_IDX_MXFP4, nv = p.pool.lat_fmt == DSA_LAT_NVFP4;
  float v[16];
  // ---- keys: the 8 threads of a token are neighbours in a warp
  for (int x = threadIdx.x; p.k_new && x < (nt * kKeyUnits + 31) / 32 * 32; x += kTokThreads) {
    const int i = x / kKeyUnits, u = x % kKeyUnits;
    const Place pl = i < nt ? place[i] : Place{-1, 0};
    float m = 0.f;
    if (pl.row >= 0) {
      load16(p.k_new + (t0 + i) * kIdxDim + 16 * u, v);
      m = abs_max16(v);
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (!mx) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
    }
    if (pl.row >= 0) {
      uint8_t* page = p.pool_w + pl.row * p.pool.row_stride + p.pool.idx_off;
      if (!mx) {
        const float s = m > 0.f ? m / 448.0f : 1.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = v[j] / s;
        *reinterpret_cast<uint4*>(page + pl.slot * kIdxDim + 16 * u) =
            make_uint4(to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7]),
                       to_e4m3x4(v[8], v[9], v[10], v[11]), to_e4m3x4(v[12], v[13], v[14], v[15]));
        if (u == 0) *reinterpret_cast<float*>(page + static_cast<int64_t>(p.pool.bs) * kIdxDim + pl.slot * 4) = s;
      } else {
        // E = floor(log2 m) - 2 + 127, at least 0; a bf16's exponent field is its float's, 254 at most
        const int e = max(static_cast<int>(__float_as_uint(m) >> 23) - 2, 0);
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);   // 2^(127 - E)
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= inv;
        *reinterpret_cast<uint2*>(page + pl.slot * (kIdxDim / 2) + 8 * u) = to_e2m1x16(v);
        if ((u & 1) == 0) page[static_cast<int64_t>(p.pool.bs) * (kIdxDim / 2) + pl.slot * 4 + (u >> 1)] = static_cast<uint8_t>(e);
      }
    }
  }
  if (!p.latent) return;
  for (int x = threadIdx.x; x < nt * kLatUnits; x += kTokThreads) {
    const int i = x / kLatUnits, u = x % kLatUnits;
    const Place pl = place[i];
    if (pl.row < 0) continue;
    load16(p.latent + (t0 + i) * kLatDim + 16 * u, v);
    uint8_t* page = p.pool_w + pl.row * p.pool.row_stride + p.pool.lat_off;
    if (!nv) {
      *reinterpret_cast<uint4*>(page + static_cast<int64_t>(pl.slot) * kLatDim + 16 * u) =
          make_uint4(to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7]),
                     to_e4m3x4(v[8], v[9], v[10], v[11]), to_e4m3x4(v[12], v[13], v[14], v[15]));
      continue;
    }
    const uint32_t code = __nv_cvt_float_to_fp8(abs_max16(v) / 6.0f, __NV_SATFINITE, __NV_E4M3);
    // x / s by the reciprocal and one correction (Markstein's): the residual is exact, so a quotient that
    // fp32 holds, as every midpoint between two e2m1 values is, comes out as itself; and bf16 over e4m3
    // comes no nearer to a midpoint, without being it, than 2^-12 of it: the codes are those of the
    // fp32 quotient. (Divisions: 66 us for 131,072 tokens, not 52.)
    const float s = e4m3_value(code), y = s > 0.f ? 1.0f / s : 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float q = v[j] * y;
      v[j] = s > 0.f ? copysignf(fmaf(fmaf(-q, s, v[j]), y, q), v[j]) : 0.f;   // a zero keeps its sign
    }
    uint8_t* rec = page + static_cast<int64_t>(pl.slot) * 352;
    *reinterpret_cast<uint2*>(rec + 8 * u) = to_e2m1x16(v);
    rec[288 + u] = static_cast<uint8_t>(code);
    if (u < 7) *reinterpret_cast<uint32_t*>(rec + 324 + 4 * u) = 0u;
  }
}

// Request of row n: the last r with cu[r] <= n, found by a warp, 32 of the remaining at a time.
// Rows outside cu[0] .. cu[B] have none (-1).
__device__ __forceinline__ int find_span(const int32_t* cu, int B, int64_t n) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;   // cu[lo] <= n < cu[hi]
  if (n < __ldg(cu) || n >= __ldg(cu + B)) return -1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && __ldg(cu + at) <= n);
    const int k = le ? 31 - __clz(le) : 0;
    hi = min(hi, lo + (k + 1) * step);
    lo = lo + k * step;
  }
  return lo;
}

__global__ void __launch_bounds__(kTokThreads) read_tokens_kernel(ReadTokensParams p) {
  __shared__ Place place[kReadRows];
  grid_dep_launch();
  grid_dep_wait();
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * p.cta_rows;
  const int nr = static_cast<int>(min(static_cast<int64_t>(p.cta_rows), p.rows - n0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    // the first row's request by a search, the others' by walking on from it
    const int64_t n = n0 + lane;
    int r = -1;
    const int64_t last = __ldg(p.cu + p.b.B), first = __ldg(p.cu);
    r = find_span(p.cu, p.b.B, n0 < first ? first : n0);
    Place pl = {-1, 0};
    if (lane < nr && r >= 0 && n >= first && n < last) {
      while (r + 1 < p.b.B && __ldg(p.cu + r + 1) <= n) ++r;
      const int c0 = __ldg(p.cu + r), c1 = __ldg(p.cu + r + 1);
      const int64_t pos = (p.start ? __ldg(p.start + r) : 0) + (n - c0);
      const int len = __ldg(p.b.ctx_lens + r);
      if (n < c0 || n >= c1 || pos < 0 || pos >= len || len > p.b.max_ctx) atomicOr(p.status, DEV_BAD_BATCH);
      else pl = place_of(p.b, p.pool, r, static_cast<int>(pos), p.status);
    }
    if (lane < nr) place[lane] = pl;
  }
  __syncthreads();
  const bool mx = p.pool.idx_fmt == DSA_IDX_MXFP4, nv = p.pool.lat_fmt == DSA_LAT_NVFP4;
  float v[16];
  if (p.lat_out) {
#pragma unroll 2
    for (int x = threadIdx.x; x < nr * kLatUnits; x += kTokThreads) {
      const int i = x / kLatUnits, u = x % kLatUnits;
      const Place pl = place[i];
      if (pl.row < 0) continue;
      const uint8_t* page = p.pool.pool + pl.row * p.pool.row_stride + p.pool.lat_off;
      if (!nv) {
        from_e4m3x16(*reinterpret_cast<const uint4*>(page + static_cast<int64_t>(pl.slot) * kLatDim + 16 * u), v);
      } else {
        const uint8_t* rec = page + static_cast<int64_t>(pl.slot) * 352;
        const uint32_t sc = rec[288 + u];
        from_e2m1x16(*reinterpret_cast<const uint2*>(rec + 8 * u), v);
        const float s = e4m3_value(sc);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= s;
      }
      store16(p.lat_out + (n0 + i) * kLatDim + 16 * u, v, p.lat_aligned32);
    }
  }
  if (p.k_out) {
    for (int x = threadIdx.x; x < nr * kKeyUnits; x += kTokThreads) {
      const int i = x / kKeyUnits, u = x % kKeyUnits;
      const Place pl = place[i];
      if (pl.row < 0) continue;
      const uint8_t* page = p.pool.pool + pl.row * p.pool.row_stride + p.pool.idx_off;
      float s;
      if (!mx) {
        s = *reinterpret_cast<const float*>(page + static_cast<int64_t>(p.pool.bs) * kIdxDim + pl.slot * 4);
        from_e4m3x16(*reinterpret_cast<const uint4*>(page + pl.slot * kIdxDim + 16 * u), v);
      } else {
        const uint32_t e = page[static_cast<int64_t>(p.pool.bs) * (kIdxDim / 2) + pl.slot * 4 + (u >> 1)];
        // 2^(E - 127); E = 0 is the subnormal 2^-127, E = 255 is not a number
        s = e == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(e ? e << 23 : 0x00400000u);
        from_e2m1x16(*reinterpret_cast<const uint2*>(page + pl.slot * (kIdxDim / 2) + 8 * u), v);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] *= s;
      store16(p.k_out + (n0 + i) * kIdxDim + 16 * u, v, p.k_aligned32);
    }
  }
}

cudaError_t launch_write_tokens(const WriteTokensParams& args, int num_sms, cudaStream_t st) {
  WriteTokensParams p = args;
  // The fewest tokens (4 to 64) with which 4 CTAs an SM take them all.
  p.cta_toks = 4;
  while (p.cta_toks < kWriteToks && cdiv(p.b.T, p.cta_toks) > 4 * num_sms) p.cta_toks *= 2;
  return launch_ex(write_tokens_kernel, dim3(static_cast<unsigned>(cdiv(p.b.T, p.cta_toks))), dim3(kTokThreads), 0, st, true, 0u,
                   p);
}

cudaError_t launch_read_tokens(const ReadTokensParams& args, int num_sms, cudaStream_t st) {
  ReadTokensParams p = args;
  // The fewest rows (4, 8, 16, 32) with which all CTAs run at a time, 8 an SM: 8,192 rows take 5.3, 4.3,
  // 5.3 and 5.5 us with each, 777 rows 2.6, 2.9, 3.1 and 4.0, 131,072 rows 59, 50, 46 and 45.
  p.cta_rows = 4;
  while (p.cta_rows < kReadRows && cdiv(p.rows, p.cta_rows) > 8 * num_sms) p.cta_rows *= 2;
  return launch_ex(read_tokens_kernel, dim3(static_cast<unsigned>(cdiv(p.rows, p.cta_rows))), dim3(kTokThreads), 0, st, true, 0u,
                   p);
}

}  // namespace dsa
