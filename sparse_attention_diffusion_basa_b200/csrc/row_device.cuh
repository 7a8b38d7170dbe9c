// Device helpers shared by the kernels that walk token rows (basa_rope.cu,
// basa_gnorm.cu): eight consecutive elements of a row as one unit of loading,
// widening, narrowing and storing, sums over a warp, and the column sums that
// end a weight's gradient.  Everything here has internal linkage.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "basa_internal.h"

namespace basa {
namespace {

struct e4m3_t {
  uint8_t bits;
};

// Eight consecutive elements as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> { uint4 a; };
template <> struct Raw8<float> { uint4 a, b; };

__device__ __forceinline__ void load8(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* p) {
  r.a = __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void load8(Raw8<float>& r, const float* p) {
  r.a = __ldcs(reinterpret_cast<const uint4*>(p));
  r.b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
}
__device__ __forceinline__ void zero8(Raw8<__nv_bfloat16>& r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero8(Raw8<float>& r) { r.a = r.b = make_uint4(0, 0, 0, 0); }

// Exact: a bf16 value is the upper half of the fp32 value it stands for.
__device__ __forceinline__ void widen8(const Raw8<__nv_bfloat16>& r, float (&f)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&f)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}

// Rounds to nearest even, once, on the way out.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  uint4 r;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = r;
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  float4* o = reinterpret_cast<float4*>(p);
  o[0] = make_float4(f[0], f[1], f[2], f[3]);
  o[1] = make_float4(f[4], f[5], f[6], f[7]);
}
// e4m3: values beyond the type's largest, 448, become 448; NaN stays NaN.
__device__ __forceinline__ void store8(e4m3_t* p, const float (&f)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// Eight parameters (norm weights, modulations) of type bf16 or fp32 from
// column `col`, a multiple of 8; `fill` where there are none.
__device__ __forceinline__ void param8(const void* p, bool bf16, long long col, float fill,
                                       float (&f)[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fill;
  } else if (bf16) {
    Raw8<__nv_bfloat16> r;
    r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + col));
    widen8(r, f);
  } else {
    Raw8<float> r;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + col);
    r.a = __ldg(q);
    r.b = __ldg(q + 1);
    widen8(r, f);
  }
}
// Eight gradients of parameters, in the parameters' type.
__device__ __forceinline__ void store_param8(void* p, bool bf16, long long col,
                                             const float (&f)[8]) {
  if (bf16)
    store8(static_cast<__nv_bfloat16*>(p) + col, f);
  else
    store8(static_cast<float*>(p) + col, f);
}
__device__ __forceinline__ void store_param(void* p, bool bf16, long long col, float f) {
  if (bf16)
    static_cast<__nv_bfloat16*>(p)[col] = __float2bfloat16_rn(f);
  else
    static_cast<float*>(p)[col] = f;
}

template <int kLanes>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace
}  // namespace basa
