// Eight columns of a row at a time: 16-byte loads and stores where the row allows them, single values
// at its ragged end or where its address does not; bf16 and e4m3 packing.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sm103_ptx.cuh"

namespace mla {

__device__ __forceinline__ void bf16x8_unpack(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 bf16x8_pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
// nearest e4m3, saturating at 448; NaN stays NaN
__device__ __forceinline__ uint32_t e4m3x4_pack(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ uint2 e4m3x8_pack(const float (&f)[8]) {
  return make_uint2(e4m3x4_pack(f[0], f[1], f[2], f[3]), e4m3x4_pack(f[4], f[5], f[6], f[7]));
}

// a / b from r, 1 / b to an ulp or two: the product's remainder is exact in one fma and puts it right
// (Markstein's correction step), so that a value next to a border between two e4m3 values falls on its own side
// of it.  Finite a and b; an infinite quotient becomes NaN.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}
// 1 / sqrt(x), the approximation after one Newton step
__device__ __forceinline__ float rsqrt_newton(float x) {
  const float y = rsqrtf(x), z = fmaf(0.5f * y, fmaf(-(x * y), y, 1.f), y);
  return x > 0.f && x < __int_as_float(0x7f800000) ? z : y;
}

// Eight columns, two to an instruction.
__device__ __forceinline__ void quotient8(float (&f)[8], float b, float r) {
  const uint64_t rr = f32x2(r, r), nb = f32x2(-b, -b);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t a = f32x2(f[i], f[i + 1]), q = mul_f32x2(a, rr);
    f32x2_split(fma_f32x2(fma_f32x2(q, nb, a), rr, q), f[i], f[i + 1]);
  }
}
__device__ __forceinline__ void add8(float (&f)[8], const float (&g)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) f32x2_split(add_f32x2(f32x2(f[i], f[i + 1]), f32x2(g[i], g[i + 1])), f[i], f[i + 1]);
}
__device__ __forceinline__ void scale8(float (&f)[8], float s) {
  const uint64_t ss = f32x2(s, s);
#pragma unroll
  for (int i = 0; i < 8; i += 2) f32x2_split(mul_f32x2(f32x2(f[i], f[i + 1]), ss), f[i], f[i + 1]);
}
__device__ __forceinline__ void norm8(float (&f)[8], float inv, const float (&w)[8]) {   // (f * inv) * w
  const uint64_t ii = f32x2(inv, inv);
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    f32x2_split(mul_f32x2(mul_f32x2(f32x2(f[i], f[i + 1]), ii), f32x2(w[i], w[i + 1])), f[i], f[i + 1]);
}
// The same times `back`, of a row whose inv was found at `back` of its size: last, so that what is small next to the row
// but not to its weight stays, or before the weight where the product passes fp32 without it.
__device__ __forceinline__ void norm8_back(float (&f)[8], float inv, const float (&w)[8], float back) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = f[i] * inv, t = y * w[i];
    f[i] = fabsf(t) < __int_as_float(0x7f800000) ? t * back : y * back * w[i];
  }
}
__device__ __forceinline__ float square_sum8(const float (&f)[8]) {   // pairwise: a row's error is that of a few roundings
  const uint64_t a = f32x2(f[0], f[1]), b = f32x2(f[2], f[3]), c = f32x2(f[4], f[5]), d = f32x2(f[6], f[7]);
  float lo, hi;
  f32x2_split(add_f32x2(fma_f32x2(a, a, mul_f32x2(b, b)), fma_f32x2(c, c, mul_f32x2(d, d))), lo, hi);
  return lo + hi;
}

// n (1..8) bf16 values at src one by one; the rest are 0
__device__ __forceinline__ uint4 load_row8_narrow(const __nv_bfloat16* src, int n) {
  const uint16_t* b = reinterpret_cast<const uint16_t*>(src);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (2 * i < n ? b[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)b[2 * i + 1] << 16 : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_row8(__nv_bfloat16* dst, int n, bool wide, const float (&f)[8]) {
  if (wide && n == 8) {
    *reinterpret_cast<uint4*>(dst) = bf16x8_pack(f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) dst[i] = __float2bfloat16_rn(f[i]);
  }
}
// as e4m3; `wide`: dst is 8-byte aligned
__device__ __forceinline__ void store_row8_e4m3(uint8_t* dst, int n, bool wide, const float (&f)[8]) {
  const uint2 v = e4m3x8_pack(f);
  if (wide && n == 8) {
    *reinterpret_cast<uint2*>(dst) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) dst[i] = (uint8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
  }
}

}  // namespace mla
