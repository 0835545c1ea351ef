// Decode over a 4-bit latent cache, plain form: a CTA of four warps per (query token, head), each warp every fourth key.
//   S = scale k . q,  P = softmax(S),  O = P V with V the key's latent columns; the sink is one more key with no value.
#include <math_constants.h>

#include "fp4_rows.cuh"

namespace mla {
namespace {

// lane l: latent columns 16 l .. 16 l + 15 (one scale) and RoPE columns 2 l, 2 l + 1
__global__ void __launch_bounds__(128) decode_fp4_kernel(const __grid_constant__ DecodeFp4Params p) {
  __shared__ float red_o[4][kLatent];
  __shared__ float red_m[4], red_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = blockIdx.x;
  const int h = (int)(item % p.H);
  const int64_t g = item / p.H;
  const int b = (int)(g / p.s), tok = (int)(g - (int64_t)b * p.s);
  const int len = paged_len(p.kv, p.err, b, (int64_t)p.kv.max_pages * p.kv.page_size, threadIdx.x == 0);
  const int seen = max(0, len - p.s + 1 + tok);
  float q[18], o[16], m = -CUDART_INF_F, l = 0.f;
  const __nv_bfloat16* qrow = p.q + item * kDk;
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = __bfloat162float(qrow[16 * lane + i]), o[i] = 0.f;
  q[16] = __bfloat162float(qrow[kLatent + 2 * lane]);
  q[17] = __bfloat162float(qrow[kLatent + 2 * lane + 1]);
  for (int j = warp; j < seen; j += 4) {
    const uint8_t* row = paged_row(p.kv, p.err, b, j);
    float k[18];
    if (row) {
      const uint2 w = *reinterpret_cast<const uint2*>(row + 8 * lane);
      const float s = e4m3_to_f32(row[kFp4Codes + lane]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v = e2m1x2_to_f16x2(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 255u);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
        k[2 * i] = f.x * s;
        k[2 * i + 1] = f.y * s;
      }
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(row + kFp4Pe + 4 * lane));
      k[16] = f.x, k[17] = f.y;
    } else {
#pragma unroll
      for (int i = 0; i < 18; ++i) k[i] = 0.f;
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 18; ++i) dot = fmaf(q[i], k[i], dot);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
    dot *= p.scale;
    const float mn = fmaxf(m, dot), a = expf(m - mn), e = expf(dot - mn);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = fmaf(e, k[i], o[i] * a);
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) red_o[warp][16 * lane + i] = o[i];
  if (lane == 0) red_m[warp] = m, red_l[warp] = l;
  __syncthreads();
  const float sink = p.sinks ? p.sinks[h] : -CUDART_INF_F;
  float top = sink;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, red_m[w]);
  const float ref = top == -CUDART_INF_F ? 0.f : top;
  float total = expf(sink - ref), f[4];
  for (int w = 0; w < 4; ++w) f[w] = expf(red_m[w] - ref), total += red_l[w] * f[w];
  const float inv = total == 0.f ? 0.f : p.kv_scale / total;    // a NaN shows
  for (int c = threadIdx.x; c < kLatent; c += 128) {
    float v = 0.f;
    for (int w = 0; w < 4; ++w) v += red_o[w][c] * f[w];
    p.out[item * kLatent + c] = __float2bfloat16_rn(v * inv);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[item] = total == 0.f ? -CUDART_INF_F : ref + logf(total);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeFp4Params& p, cudaStream_t stream) {
  decode_fp4_kernel<<<(unsigned)((int64_t)p.kv.B * p.s * p.H), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
