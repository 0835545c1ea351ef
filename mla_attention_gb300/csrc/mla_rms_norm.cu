// Root-mean-square norm of rows with the residual's addition, out in bf16 or in e4m3 with scales.
//
//   h = x (+ residual)      y = h / sqrt(mean(h^2) + eps) * w
//   out = bf16(y), or with one scale s = max(max|y| / 448, 2^-126) per group of columns: out = e4m3(y / s)
//
// HBM-bound: 2 bytes a column in, 2 more for the residual and 2 for its sum, 1 or 2 out.  A row is read
// once and kept in registers as h in fp32, eight columns (16 bytes) a vector: one warp a row up to 1024
// columns (no barrier), one CTA a row above.  The weight's vectors are asked for together with the row's
// where registers allow; x and the residual pass by L1, which keeps the weight, and are asked for in L2 a
// little before their CTA starts: what is on its way between HBM and L2 takes no registers.  bf16 rows written off the
// vector boundaries (an odd width) go value by value instead, neighbouring columns in neighbouring lanes.
// 16384 x 5120 with residual to e4m3: 90 us, 97 % of the copy's bandwidth; 8000 x 8192 with residual to bf16 78.8 us, 98 %;
// one row of 8192 2.3 to 2.5 us.  To e4m3 without a residual the arithmetic bounds it: 4000 x 16384 54.6 us, 53 %.
//
// max|y| and the sum keep a NaN (a row that holds one is NaN throughout).
#include "mla_step.h"
#include "row_vec.cuh"

namespace mla {
namespace {

constexpr float kMinScale = 0x1p-126f, kE4m3Max = 448.f;

#ifdef MLA_GUARD
__device__ uint32_t guard_status;   // the call has no workspace
#endif

__device__ __forceinline__ uint4 load_once(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// `bytes` at p, both multiples of 16
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// the larger one; NaN if either is
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// the largest magnitude of three; NaN if any is
__device__ __forceinline__ float nan_max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <bool kMax>
__device__ __forceinline__ float join(float a, float b) { return kMax ? nan_max(a, b) : a + b; }

template <bool kMax>
__device__ __forceinline__ float warp_reduce(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = join<kMax>(v, __shfl_xor_sync(~0u, v, d));
  return v;
}

// over the row's threads: its warp, or with kBlock its CTA, which gives each reduction a buffer of its own
template <bool kBlock, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float (&red)[32]) {
  v = warp_reduce<kMax>(v);
  if constexpr (kBlock) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (lane == 0) red[wid] = v;
    __syncthreads();
    v = warp_reduce<kMax>(lane < warps ? red[lane] : 0.f);
  }
  return v;
}

enum : int { kWideX = 1, kWideR = 2, kWideRo = 4, kWideW = 8, kWideOut = 16 };  // rows on vector boundaries

template <int NV, bool kBlock, bool kE4m3, bool kStrided>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) rms_norm_kernel(const __grid_constant__ RmsNormParams p, int wide, int ahead) {
  __shared__ float red[3][32];
  const int per_row = kBlock ? blockDim.x : 32, sub = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int64_t t = kBlock ? blockIdx.x : (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  if (!kBlock && t >= p.T) return;
  // a row that comes up in about a microsecond, from HBM into L2
  if (sub == 0 && p.D >= 8 && t + ahead < p.T) {
    if (wide & kWideX) prefetch_l2(p.x + (t + ahead) * p.x_stride, p.D / 8 * 16);
    if (p.residual && (wide & kWideR)) prefetch_l2(p.residual + (t + ahead) * p.residual_stride, p.D / 8 * 16);
  }
  // Vector k of this thread: columns c .. c + n - 1, or with kStrided every per_row-th from sub + 8 k per_row on.
  auto load = [&](const __nv_bfloat16* base, int64_t stride, int64_t row, bool on_vec, int k) {
    const uint64_t ext = ((uint64_t)(row ? p.T - 1 : 0) * stride + p.D) * 2;
    if constexpr (kStrided) {
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (8 * k + i) * per_row + sub;
        const __nv_bfloat16* src = base + row * stride + sub + (8 * k + i) * per_row;
        b[i] = c < p.D && guard_span(p.err, G_STEP_IN, src, 2, base, ext) ? *reinterpret_cast<const uint16_t*>(src) : 0u;
      }
      return make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
    }
    const int c = 8 * (sub + k * per_row), n = min(8, p.D - c);
    const __nv_bfloat16* src = base + row * stride + c;
    if (n <= 0 || !guard_span(p.err, G_STEP_IN, src, 2 * n, base, ext)) return make_uint4(0, 0, 0, 0);
    if (!on_vec || n < 8) return load_row8_narrow(src, n);
    return base == p.weight ? *reinterpret_cast<const uint4*>(src) : load_once(src);
  };
  auto store = [&](__nv_bfloat16* base, int64_t stride, bool on_vec, int k, const float(&f)[8]) {
    const uint64_t ext = ((uint64_t)(p.T - 1) * stride + p.D) * 2;
    if constexpr (kStrided) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (8 * k + i) * per_row + sub;
        __nv_bfloat16* dst = base + t * stride + c;
        if (c < p.D && guard_span(p.err, G_STEP_OUT, dst, 2, base, ext)) *dst = __float2bfloat16_rn(f[i]);
      }
    } else {
      const int c = 8 * (sub + k * per_row), n = min(8, p.D - c);
      __nv_bfloat16* dst = base + t * stride + c;
      if (n > 0 && guard_span(p.err, G_STEP_OUT, dst, 2 * n, base, ext)) store_row8(dst, n, on_vec, f);
    }
  };
  constexpr bool kWeightFirst = NV <= 2;   // more vectors leave no registers for it
  uint4 xv[NV], wv[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) xv[k] = load(p.x, p.x_stride, t, wide & kWideX, k);
  float h[NV][8];
  if (p.residual) {
    uint4 rv[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) rv[k] = load(p.residual, p.residual_stride, t, wide & kWideR, k);
    if constexpr (kWeightFirst)
#pragma unroll
      for (int k = 0; k < NV; ++k) wv[k] = load(p.weight, 0, 0, wide & kWideW, k);
    // the sum goes out before the norm: residual_out may be the residual or x, read by this thread alone
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float f[8];
      bf16x8_unpack(xv[k], h[k]);
      bf16x8_unpack(rv[k], f);
      add8(h[k], f);
      store(p.residual_out, p.residual_out_stride, wide & kWideRo, k, h[k]);
    }
  } else {
    if constexpr (kWeightFirst)
#pragma unroll
      for (int k = 0; k < NV; ++k) wv[k] = load(p.weight, 0, 0, wide & kWideW, k);
#pragma unroll
    for (int k = 0; k < NV; ++k) bf16x8_unpack(xv[k], h[k]);
  }

  float sum = 0.f, back = 1.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) sum += square_sum8(h[k]);
  float mean = row_reduce<kBlock, false>(sum, red[0]) / (float)p.D + p.eps;
  if (__builtin_expect(!(mean >= 0x1p-100f && mean <= 3e38f), 0)) {
    // The squares leave fp32's range (or the row holds a NaN): once more at 2^-96 of the row's size, where the largest values'
    // squares still add up and the smallest that count still have one, or at 2^96 of it, where every value's square
    // is a normal number.  A small row goes on at that size, a huge one as it is: 2^-96 of it would lose its small values.
    const bool tiny = mean < 0x1p-100f;
    const float up = tiny ? 0x1p96f : 0x1p-96f;
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = h[k][i] * up;
        sum = fmaf(f, f, sum);
        if (tiny) h[k][i] = f;
      }
    mean = row_reduce<kBlock, false>(sum, red[1]) / (float)p.D + p.eps * up * up;
    if (!tiny) back = up;
  }
  const float inv = rsqrt_newton(mean);
  auto weigh = [&](auto&& norm) {   // y; behind the row's end 0
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (!kWeightFirst) wv[k] = load(p.weight, 0, 0, wide & kWideW, k);
      float w[8];
      bf16x8_unpack(wv[k], w);
      norm(h[k], w);
    }
  };
  if (__builtin_expect(back == 1.f, 1)) weigh([&](float(&f)[8], const float(&w)[8]) { norm8(f, inv, w); });
  else weigh([&](float(&f)[8], const float(&w)[8]) { norm8_back(f, inv, w, back); });

  if constexpr (!kE4m3) {
#pragma unroll
    for (int k = 0; k < NV; ++k) store(reinterpret_cast<__nv_bfloat16*>(p.out), p.out_stride, wide & kWideOut, k, h[k]);
  } else {
    uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + t * p.out_stride;
    float m[NV], all = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      m[k] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i += 2) m[k] = nan_max_abs(m[k], h[k][i], h[k][i + 1]);
      all = nan_max(all, m[k]);
    }
    const bool whole = p.group == p.D;
    const int group_log2 = 31 - __clz(p.group);   // used where p.group is a power of two
    const int64_t groups = whole ? 1 : p.D >> group_log2;
    if (whole) {
      all = row_reduce<kBlock, true>(all, red[2]);
#pragma unroll
      for (int k = 0; k < NV; ++k) m[k] = all;
    } else {   // a group is 4, 8 or 16 vectors, held by as many lanes of one warp
#pragma unroll
      for (int d = 1; d < 16; d <<= 1)
        if (8 * d < p.group)
#pragma unroll
          for (int k = 0; k < NV; ++k) m[k] = nan_max(m[k], __shfl_xor_sync(~0u, m[k], d));
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (sub + k * per_row), n = min(8, p.D - c);
      // (max / 448; an infinite one is kept, leaves 0 of finite values and NaN of infinite ones)
      const bool fin = m[k] < __int_as_float(0x7f800000);
      const float s = nan_max(kMinScale, fin ? quotient(m[k], kE4m3Max, 1.f / kE4m3Max) : m[k]), s_or_0 = fin ? s : 0.f;
      float inv_s;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv_s) : "f"(s));
      quotient8(h[k], s_or_0, inv_s);
      float* sc = p.scales + t * groups + (whole ? 0 : c >> group_log2);
      const bool writes = whole ? sub == 0 && k == 0 : n > 0 && (c & (p.group - 1)) == 0;
      if (writes && guard_span(p.err, G_STEP_OUT, sc, 4, p.scales, (uint64_t)p.T * groups * 4)) *sc = s;
      const uint64_t ext = (uint64_t)(p.T - 1) * p.out_stride + p.D;
      if constexpr (kStrided) {
        const uint2 q = e4m3x8_pack(h[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int ci = (8 * k + i) * per_row + sub;
          if (ci < p.D && guard_span(p.err, G_STEP_OUT, out + ci, 1, p.out, ext)) out[ci] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
        }
      } else if (n > 0 && guard_span(p.err, G_STEP_OUT, out + c, n, p.out, ext)) {
        store_row8_e4m3(out + c, n, wide & kWideOut, h[k]);
      }
    }
  }
}

template <int NV, bool kBlock, bool kStrided = false>
cudaError_t launch(const RmsNormParams& p, int wide, int threads, cudaStream_t stream) {
  // Two rows an SM: 16384 x 5120 to e4m3 94.0 -> 89.4 us, 10678 x 2744 24.2 -> 21.7, 16384 x 1536 19.9 -> 18.3 (half an SM's, one
  // and six rows: 91.3, 90.4, 90.5 and 22.4, 22.1, 21.7 and 19.1, 18.9, 17.6).
  const int ahead = 2 * device_sm_count();
  const unsigned grid = kBlock ? (unsigned)p.T : (unsigned)(((int64_t)p.T * 32 + threads - 1) / threads);
  if (p.scales) rms_norm_kernel<NV, kBlock, true, kStrided><<<grid, threads, 0, stream>>>(p, wide, ahead);
  else rms_norm_kernel<NV, kBlock, false, kStrided><<<grid, threads, 0, stream>>>(p, wide, ahead);
  return cudaGetLastError();
}

bool on(const void* p, int64_t stride, int T, int bytes, int elem) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (T == 1 || stride * elem % bytes == 0);
}

}  // namespace

uint32_t* guard_word() {
  void* at = nullptr;
#ifdef MLA_GUARD
  if (cudaGetSymbolAddress(&at, guard_status) != cudaSuccess) return nullptr;
#endif
  return reinterpret_cast<uint32_t*>(at);
}

cudaError_t launch_rms_norm(const RmsNormParams& p, cudaStream_t stream) {
  int wide = 0;
  if (on(p.x, p.x_stride, p.T, 16, 2)) wide |= kWideX;
  if (on(p.residual, p.residual_stride, p.T, 16, 2)) wide |= kWideR;
  if (on(p.residual_out, p.residual_out_stride, p.T, 16, 2)) wide |= kWideRo;
  if (on(p.weight, 0, 1, 16, 2)) wide |= kWideW;
  if (p.scales ? on(p.out, p.out_stride, p.T, 8, 1) : on(p.out, p.out_stride, p.T, 16, 2)) wide |= kWideOut;
  const int vecs = (p.D + 7) / 8;
  auto threads = [&](int nv) { return (vecs + 32 * nv - 1) / (32 * nv) * 32; };
  // bf16 rows that are written off the vector boundaries: every eight values of a lane would be eight writes
  // with 16 bytes between the lanes, so neighbouring columns go to neighbouring lanes (30000 x 1279: 97 us and
  // 52; 3 x 8191 with residual: 6.9 and 3.6).  Rows that are only read off them, and bytes written so, stay with
  // vectors (10000 x 2047 to e4m3: 28.6 us, so 41; 32000 x 1024 with x alone off: 48 and 70).  Not with scales of
  // groups, whose columns lie in one warp only with eight to a lane, nor above 8192 columns, where eight
  // values a thread are too few.
  const bool narrow_out = (p.residual && !(wide & kWideRo)) || (!p.scales && !(wide & kWideOut));
  if (narrow_out && (!p.scales || p.group == p.D) && vecs <= 1024) {
    if (vecs <= 32) return launch<1, false, true>(p, wide, 128, stream);
    if (vecs <= 64) return launch<2, false, true>(p, wide, 128, stream);
    return launch<1, true, true>(p, wide, threads(1), stream);
  }
  if (vecs <= 32) return launch<1, false>(p, wide, 128, stream);
  if (vecs <= 64) return launch<2, false>(p, wide, 128, stream);
  if (vecs <= 128) return launch<4, false>(p, wide, 128, stream);
  // A CTA a row.  Two vectors a thread are the shorter way through one row (8192 columns when it was chosen: 2.6 us, four 3.4);
  // four put more rows on an SM, which pays for wide ones once the SMs are full (8000 x 8192 with residual:
  // 84.6 us and 80.2; 16384 x 5120 to e4m3: 100.4 and 98.2; 4000 x 16384 to e4m3: 78.8 and 61.4; but
  // 2048 x 4096: 12.9 and 13.9).
  const int sms = device_sm_count();
  if (vecs > (p.T >= 32 * sms ? 319 : p.T >= 2 * sms ? 1023 : 2048)) return launch<4, true>(p, wide, threads(4), stream);
  return launch<2, true>(p, wide, threads(2), stream);
}

}  // namespace mla
