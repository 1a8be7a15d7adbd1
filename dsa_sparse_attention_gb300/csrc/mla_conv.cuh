// mla_conv.cuh — latents as 16-bit tensor-core operands: the conversions and small
// helpers shared by the attention kernels that convert on the fly (mla.cu, tree_mla.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dsa {

// 16 e4m3 bytes -> 16 bf16 values (exact), packed as 8 x bf16x2.
__device__ __forceinline__ void e4m3x16_to_bf16(const uint4 in, uint32_t (&o)[8]) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] & 0xFFFFu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> 16), __NV_E4M3);
    const float2 flo = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 fhi = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    const __nv_bfloat162 blo = __floats2bfloat162_rn(flo.x, flo.y);
    const __nv_bfloat162 bhi = __floats2bfloat162_rn(fhi.x, fhi.y);
    o[2 * i] = *reinterpret_cast<const uint32_t*>(&blo);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&bhi);
  }
}

// 16 e4m3 bytes -> 16 fp16 values (exact), packed as 8 x f16x2.
__device__ __forceinline__ void e4m3x16_to_f16(const uint4 in, uint32_t (&o)[8]) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] & 0xFFFFu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> 16), __NV_E4M3);
    o[2 * i] = static_cast<uint32_t>(lo.x) | (static_cast<uint32_t>(lo.y) << 16);
    o[2 * i + 1] = static_cast<uint32_t>(hi.x) | (static_cast<uint32_t>(hi.y) << 16);
  }
}

// 16 NVFP4 values (8 packed bytes, element 2i in the low nibble of byte i) with
// their e4m3 block scale -> 16 fp16 values.  e2m1 x e4m3 has at most 6
// significant bits and lies in [2^-10, 2688]: exact in fp16 (and in bf16).
__device__ __forceinline__ void nvfp4x16_to_f16(const uint2 in, uint32_t scale_code, uint32_t (&o)[8]) {
  const __half sc = __half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(scale_code), __NV_E4M3));
  const __half2 sc2 = __half2(sc, sc);
  const uint32_t w[2] = {in.x, in.y};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>((w[i >> 2] >> (8 * (i & 3))) & 0xFFu),
                                                     __NV_E2M1);
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&r), sc2);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

__device__ __forceinline__ void nvfp4x16_to_bf16(const uint2 in, uint32_t scale_code, uint32_t (&o)[8]) {
  nvfp4x16_to_f16(in, scale_code, o);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    o[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// 2^x on the multi-function unit (relative error about 2^-22; subnormal results flush to 0).
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One 64-dim chunk of a converter thread's half row: dims [64 kc + 32 hf, +32).
// FP8: 32 bytes in a, b.  NVFP4: 16 bytes of packed values in a, the two e4m3
// block scales in the low bytes of s.  An absent row reads as zeros.
struct LatPiece {
  uint4 a, b;
  uint32_t s;
};

template <bool NV>
__device__ __forceinline__ LatPiece load_piece(const uint8_t* src, int kc, int hf) {
  LatPiece r;
  r.a = r.b = make_uint4(0, 0, 0, 0);
  r.s = 0;
  if (src) {
    if (NV) {
      r.a = __ldg(reinterpret_cast<const uint4*>(src + 32 * kc + 16 * hf));
      r.s = __ldg(reinterpret_cast<const uint16_t*>(src + 288 + 4 * kc + 2 * hf));
    } else {
      r.a = __ldg(reinterpret_cast<const uint4*>(src + 64 * kc + 32 * hf));
      r.b = __ldg(reinterpret_cast<const uint4*>(src + 64 * kc + 32 * hf + 16));
    }
  }
  return r;
}

// 16 values (piece q2 of the chunk) -> 8 packed bf16x2 / f16x2 words.
template <bool NV>
__device__ __forceinline__ void piece_to_bf16(const LatPiece& c, int q2, uint32_t (&o)[8]) {
  if (NV)
    nvfp4x16_to_bf16(q2 ? make_uint2(c.a.z, c.a.w) : make_uint2(c.a.x, c.a.y), (c.s >> (8 * q2)) & 0xFFu, o);
  else
    e4m3x16_to_bf16(q2 ? c.b : c.a, o);
}
template <bool NV>
__device__ __forceinline__ void piece_to_f16(const LatPiece& c, int q2, uint32_t (&o)[8]) {
  if (NV)
    nvfp4x16_to_f16(q2 ? make_uint2(c.a.z, c.a.w) : make_uint2(c.a.x, c.a.y), (c.s >> (8 * q2)) & 0xFFu, o);
  else
    e4m3x16_to_f16(q2 ? c.b : c.a, o);
}

// 32 consecutive floats of shared memory (16-byte aligned) through 8 vector loads.
__device__ __forceinline__ void lds_f32x32(const float* src, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 x = reinterpret_cast<const float4*>(src)[i];
    v[4 * i] = x.x;
    v[4 * i + 1] = x.y;
    v[4 * i + 2] = x.z;
    v[4 * i + 3] = x.w;
  }
}

__device__ __forceinline__ void sts128(uint8_t* p, const uint32_t* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}

}  // namespace dsa
