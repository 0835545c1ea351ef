// Root-mean-square norm of rows with the residual's addition, out in bf16 or in e4m3 with scales.
//
//   h = x (+ residual)      y = h / sqrt(mean(h^2) + eps) * w
//   out = bf16(y), or with one scale s = max(max|y| / 448, 2^-126) per group of columns: out = e4m3(y / s)
//
// HBM-bound: 2 bytes a column in, 2 more for the residual and 2 for its sum, 1 or 2 out.  A row is read
// once and kept in registers as h in fp32, eight columns (16 bytes) a vector: one warp a row up to 1024
// columns (no barrier), one CTA a row above, as many threads as give each two vectors (four above 16384
// columns).  Short CTAs beat long ones here: six rows of 5120 columns share an SM, so that one's
// reduction is another's load.  The weight's vectors are asked for together with the row's; x and
// the residual pass by L1, which keeps the weight.
//
// max|y| and the sum keep a NaN (a row that holds one is NaN throughout).
#include "mla_step.h"
#include "row_vec.cuh"

namespace mla {
namespace {

constexpr float kMinScale = 0x1p-126f, kE4m3Max = 448.f;

__device__ __forceinline__ uint4 load_once(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// the larger one; NaN if either is
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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

// over the row's threads: its warp, or with kBlock its CTA
template <bool kBlock, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* red) {
  v = warp_reduce<kMax>(v);
  if constexpr (kBlock) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) red[wid] = v;
    __syncthreads();
    v = warp_reduce<kMax>(lane < warps ? red[lane] : 0.f);
  }
  return v;
}

enum : int { kWideX = 1, kWideR = 2, kWideRo = 4, kWideW = 8, kWideOut = 16 };  // rows on vector boundaries

template <int NV, bool kBlock, bool kE4m3>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) rms_norm_kernel(const __grid_constant__ RmsNormParams p, int wide) {
  __shared__ float red[32];
  const int per_row = kBlock ? blockDim.x : 32, sub = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int64_t t = kBlock ? blockIdx.x : (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  if (!kBlock && t >= p.T) return;
  // vector k of this thread: columns c .. c + n - 1
  auto load = [&](const __nv_bfloat16* base, int64_t stride, int64_t row, bool on_vec, int k) {
    const int c = 8 * (sub + k * per_row), n = min(8, p.D - c);
    const __nv_bfloat16* src = base + row * stride + c;
    if (n <= 0 || !guard_span(nullptr, G_STEP_IN, src, 2 * n, base, ((uint64_t)(row ? p.T - 1 : 0) * stride + p.D) * 2))
      return make_uint4(0, 0, 0, 0);
    if (!on_vec || n < 8) return load_row8_narrow(src, n);
    return base == p.weight ? *reinterpret_cast<const uint4*>(src) : load_once(src);
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
    __nv_bfloat16* ro = p.residual_out + t * p.residual_out_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (sub + k * per_row), n = min(8, p.D - c);
      float f[8];
      bf16x8_unpack(xv[k], h[k]);
      bf16x8_unpack(rv[k], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] += f[i];
      if (n > 0 && guard_span(nullptr, G_STEP_OUT, ro + c, 2 * n, p.residual_out, ((uint64_t)(p.T - 1) * p.residual_out_stride + p.D) * 2))
        store_row8(ro + c, n, wide & kWideRo, h[k]);
    }
  } else {
    if constexpr (kWeightFirst)
#pragma unroll
      for (int k = 0; k < NV; ++k) wv[k] = load(p.weight, 0, 0, wide & kWideW, k);
#pragma unroll
    for (int k = 0; k < NV; ++k) bf16x8_unpack(xv[k], h[k]);
  }

  auto sum_squares = [&] {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) sum += square_sum8(h[k]);
    return row_reduce<kBlock, false>(sum, red);
  };
  float sum = sum_squares(), eps = p.eps;
  if (sum > 3e38f) {
    // The squares leave fp32's range: the row once more at 2^-96 of its size, where the largest
    // values' squares still add up and the smallest that count still have one.
    eps *= 0x1p-96f;
    eps *= 0x1p-96f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] *= 0x1p-96f;
    sum = sum_squares();
  }
  const float inv = rsqrt_newton(sum / (float)p.D + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if constexpr (!kWeightFirst) wv[k] = load(p.weight, 0, 0, wide & kWideW, k);
    float w[8];
    bf16x8_unpack(wv[k], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * inv * w[i];   // y; behind the row's end 0
  }

  if constexpr (!kE4m3) {
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + t * p.out_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (sub + k * per_row), n = min(8, p.D - c);
      if (n > 0 && guard_span(nullptr, G_STEP_OUT, out + c, 2 * n, p.out, ((uint64_t)(p.T - 1) * p.out_stride + p.D) * 2))
        store_row8(out + c, n, wide & kWideOut, h[k]);
    }
  } else {
    uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + t * p.out_stride;
    float m[NV], all = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      m[k] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[k] = nan_max(m[k], fabsf(h[k][i]));
      all = nan_max(all, m[k]);
    }
    const bool whole = p.group == p.D;
    const int group_log2 = 31 - __clz(p.group);   // used where p.group is a power of two
    const int64_t groups = whole ? 1 : p.D >> group_log2;
    if (whole) {
      all = row_reduce<kBlock, true>(all, red);
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
      const int v = sub + k * per_row, c = 8 * v, n = min(8, p.D - c);
      // (max / 448; an infinite one is kept, leaves 0 of finite values and NaN of infinite ones)
      const bool fin = m[k] < __int_as_float(0x7f800000);
      const float s = nan_max(kMinScale, fin ? quotient(m[k], kE4m3Max, 1.f / kE4m3Max) : m[k]), s_or_0 = fin ? s : 0.f;
      float inv_s;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv_s) : "f"(s));
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = quotient(h[k][i], s_or_0, inv_s);
      if (n > 0) {
        if (guard_span(nullptr, G_STEP_OUT, out + c, n, p.out, (uint64_t)(p.T - 1) * p.out_stride + p.D))
          store_row8_e4m3(out + c, n, wide & kWideOut, h[k]);
        float* sc = p.scales + t * groups + (whole ? 0 : c >> group_log2);
        if ((whole ? v == 0 : (c & (p.group - 1)) == 0) && guard_span(nullptr, G_STEP_OUT, sc, 4, p.scales, (uint64_t)p.T * groups * 4)) *sc = s;
      }
    }
  }
}

template <int NV, bool kBlock>
cudaError_t launch(const RmsNormParams& p, int wide, int threads, cudaStream_t stream) {
  const unsigned grid = kBlock ? (unsigned)p.T : (unsigned)(((int64_t)p.T * 32 + threads - 1) / threads);
  if (p.scales) rms_norm_kernel<NV, kBlock, true><<<grid, threads, 0, stream>>>(p, wide);
  else rms_norm_kernel<NV, kBlock, false><<<grid, threads, 0, stream>>>(p, wide);
  return cudaGetLastError();
}

bool on(const void* p, int64_t stride, int T, int bytes, int elem) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (T == 1 || stride * elem % bytes == 0);
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormParams& p, cudaStream_t stream) {
  int wide = 0;
  if (on(p.x, p.x_stride, p.T, 16, 2)) wide |= kWideX;
  if (on(p.residual, p.residual_stride, p.T, 16, 2)) wide |= kWideR;
  if (on(p.residual_out, p.residual_out_stride, p.T, 16, 2)) wide |= kWideRo;
  if (on(p.weight, 0, 1, 16, 2)) wide |= kWideW;
  if (p.scales ? on(p.out, p.out_stride, p.T, 8, 1) : on(p.out, p.out_stride, p.T, 16, 2)) wide |= kWideOut;
  const int vecs = (p.D + 7) / 8;
  auto threads = [&](int nv) { return (vecs + 32 * nv - 1) / (32 * nv) * 32; };
  if (vecs <= 32) return launch<1, false>(p, wide, 128, stream);
  if (vecs <= 64) return launch<2, false>(p, wide, 128, stream);
  if (vecs <= 128) return launch<4, false>(p, wide, 128, stream);
  if (vecs <= 2048) return launch<2, true>(p, wide, threads(2), stream);
  return launch<4, true>(p, wide, threads(4), stream);
}

}  // namespace mla
