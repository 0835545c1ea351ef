// Root-mean-square norm of rows with the residual's addition, out in bf16 or in e4m3 with scales.
//
//   h = x (+ residual)      y = h / sqrt(mean(h^2) + eps) * w
//   out = bf16(y), or with one scale s = max(max|y| / 448, 2^-126) per group of columns: out = e4m3(y / s)
#include "mla_step.h"
#include "row_vec.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;

// the larger one; NaN if either is
__device__ __forceinline__ float nan_max(float a, float b) { return b > a || b != b ? b : a; }

__device__ __forceinline__ float block_reduce(float v, float* red, bool max) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float u = __shfl_xor_sync(~0u, v, d);
    v = max ? nan_max(v, u) : v + u;
  }
  __syncthreads();
  if (lane == 0) red[wid] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < kThreads / 32; ++i) v = max ? nan_max(v, red[i]) : v + red[i];
  return v;
}

// one CTA a row, three passes over it
__global__ void __launch_bounds__(kThreads) rms_norm_kernel(const __grid_constant__ RmsNormParams p) {
  __shared__ float red[kThreads / 32];
  const int64_t t = blockIdx.x;
  const __nv_bfloat16* x = p.x + t * p.x_stride;
  const __nv_bfloat16* r = p.residual ? p.residual + t * p.residual_stride : nullptr;
  auto h = [&](int i) { return __bfloat162float(x[i]) + (r ? __bfloat162float(r[i]) : 0.f); };
  float sum = 0.f;
  for (int i = threadIdx.x; i < p.D; i += kThreads) sum += h(i) * h(i);
  sum = block_reduce(sum, red, false);
  // Squares past fp32's range: the row is summed again at 2^-96 of its size (an infinite or NaN
  // value stays one).
  float pre = 1.f, eps = p.eps;
  if (sum > 3e38f) {
    pre = 0x1p-96f;
    eps = eps * pre * pre;
    sum = 0.f;
    for (int i = threadIdx.x; i < p.D; i += kThreads) sum += (h(i) * pre) * (h(i) * pre);
    sum = block_reduce(sum, red, false);
  }
  const float inv = rsqrtf(sum / (float)p.D + eps);
  auto y = [&](int i) { return h(i) * pre * inv * __bfloat162float(p.weight[i]); };
  if (!p.scales) {
    for (int i = threadIdx.x; i < p.D; i += kThreads) {
      const float v = y(i), hv = h(i);
      reinterpret_cast<__nv_bfloat16*>(p.out)[t * p.out_stride + i] = __float2bfloat16_rn(v);
      if (r) p.residual_out[t * p.residual_out_stride + i] = __float2bfloat16_rn(hv);
    }
    return;
  }
  const int groups = p.D / p.group;
  for (int g = 0; g < groups; ++g) {
    float m = 0.f;
    for (int i = g * p.group + threadIdx.x; i < (g + 1) * p.group; i += kThreads) {
      m = nan_max(m, fabsf(y(i)));
    }
    const float s = nan_max(1.17549435e-38f, block_reduce(m, red, true) / 448.f);
    if (threadIdx.x == 0) p.scales[t * groups + g] = s;
    for (int i = g * p.group + threadIdx.x; i < (g + 1) * p.group; i += kThreads) {
      const float hv = h(i);
      reinterpret_cast<uint8_t*>(p.out)[t * p.out_stride + i] = (uint8_t)e4m3x4_pack(y(i) / s, 0.f, 0.f, 0.f);
      if (r) p.residual_out[t * p.residual_out_stride + i] = __float2bfloat16_rn(hv);
    }
  }
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormParams& p, cudaStream_t stream) {
  rms_norm_kernel<<<p.T, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
