// Rows of a paged cache and the values of 4-bit ones.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "mla_cache.h"
#include "row_vec.cuh"

namespace mla {

// an int32 of a table or list (guarded build: 0 outside it)
__device__ __forceinline__ int32_t guarded_int(uint32_t* err, const int32_t* base, int64_t i, int64_t n) {
  return guard_span(err, G_STEP_IN, base + i, 4, base, (uint64_t)n * 4) ? base[i] : 0;
}

// length of request b, cut to `cap`; `report`: one thread of the call records a length outside it
__device__ __forceinline__ int paged_len(const PagedRows& kv, uint32_t* err, int b, int64_t cap, bool report) {
  int64_t n = guarded_int(err, kv.lens, b, kv.B);
  if (n < 0 || n > cap) {
    if (report) record_error(err, DEV_RANGE_BASE | Y_LEN);
    n = n < 0 ? 0 : cap;
  }
  return (int)n;
}

// eight codes (a word, lowest four bits first) times a scale, in f16: exact, a product has at most six bits
__device__ __forceinline__ uint4 fp4x8_to_f16(uint32_t w, uint32_t scale2) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 c0, c1, c2, c3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 c0, b0;\n\tcvt.rn.f16x2.e2m1x2 c1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 c2, b2;\n\tcvt.rn.f16x2.e2m1x2 c3, b3;\n\t"
      "mul.rn.f16x2 %0, c0, %5;\n\tmul.rn.f16x2 %1, c1, %5;\n\tmul.rn.f16x2 %2, c2, %5;\n\tmul.rn.f16x2 %3, c3, %5;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w), "r"(scale2));
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// two scales (e4m3, low byte first) as f16, each in both halves of a word
__device__ __forceinline__ uint2 fp4_scales2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2((uint16_t)two);
  return make_uint2(__byte_perm(h, h, 0x1010), __byte_perm(h, h, 0x3232));
}
// the same with `cap`, in both halves, in the place of a NaN: the largest scale, or a NaN again
constexpr uint32_t kScaleNan = 0x7fff7fffu, kScale448 = 0x5f005f00u;
__device__ __forceinline__ uint2 fp4_scales2(uint32_t two, uint32_t cap) {
  uint32_t h = e4m3x2_to_f16x2((uint16_t)two);
  asm("min.f16x2 %0, %0, %1;" : "+r"(h) : "r"(cap));          // of a number and a NaN the number
  return make_uint2(__byte_perm(h, h, 0x1010), __byte_perm(h, h, 0x3232));
}
// eight e4m3 values as f16
__device__ __forceinline__ uint4 e4m3x8_to_f16(uint32_t a, uint32_t b) {
  return make_uint4(e4m3x2_to_f16x2((uint16_t)a), e4m3x2_to_f16x2((uint16_t)(a >> 16)), e4m3x2_to_f16x2((uint16_t)b),
                    e4m3x2_to_f16x2((uint16_t)(b >> 16)));
}
__device__ __forceinline__ uint4 bf16x8_to_f16(const uint4& v) {
  return make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

}  // namespace mla
