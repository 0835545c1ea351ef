// Products of a few rows with 4-bit weights and group scales, per head:
//   out[t, h, n] = sum_g scale[h, n, g] sum_{k in g} x[t, h, k] (code[h, n, k] - 8)
// One warp per output column (h, n), eight tokens at a time.
#include "mla_step.h"
#include "row_vec.cuh"

namespace mla {
namespace {

constexpr int kTok = 8;

__global__ void __launch_bounds__(256) bmm_w4_kernel(const __grid_constant__ BmmW4Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t col = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  if (col >= (int64_t)p.H * p.N) return;
  const int h = (int)(col / p.N), n = (int)(col - (int64_t)h * p.N);
  const int t0 = blockIdx.y * kTok;
  const uint8_t* w = p.w4 + col * (p.K / 2);
  const int groups = p.K / p.group;
  float acc[kTok] = {};
  for (int i = lane; i < p.K / 2; i += 32) {
    const int code = w[i];
    const int64_t si = col * groups + 2 * i / p.group;
    const float s = p.scales_f32 ? reinterpret_cast<const float*>(p.scales)[si]
                                 : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.scales)[si]);
    const float w0 = (float)((code & 15) - 8) * s, w1 = (float)((code >> 4) - 8) * s;
    for (int t = 0; t < kTok; ++t) {
      if (t0 + t >= p.T) break;
      const __nv_bfloat16* x = p.x + (t0 + t) * p.x_stride_t + h * p.x_stride_h + 2 * i;
      acc[t] += __bfloat162float(x[0]) * w0 + __bfloat162float(x[1]) * w1;
    }
  }
  for (int t = 0; t < kTok; ++t) {
    const float v = warp_sum(acc[t]);
    if (lane == 0 && t0 + t < p.T) p.out[(t0 + t) * p.out_stride_t + h * p.out_stride_h + n] = __float2bfloat16_rn(v);
  }
}

}  // namespace

cudaError_t launch_bmm_w4(const BmmW4Params& p, cudaStream_t stream) {
  const int64_t cols = (int64_t)p.H * p.N;
  bmm_w4_kernel<<<dim3((unsigned)((cols + 7) / 8), (p.T + kTok - 1) / kTok), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
