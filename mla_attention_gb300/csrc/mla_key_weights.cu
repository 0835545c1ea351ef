// The attention that each cached key got, plain form: a warp per key, its row in registers, over all query rows.
//   weights[b, j] = decay weights[b, j] + sum_{i, h} exp(scale q_{b,i,h} . k_j - lse_{b,i,h})
#include <math_constants.h>

#include "fp4_rows.cuh"

namespace mla {
namespace {

// lane l: columns 16 l .. 16 l + 15 and 512 + 2 l, 512 + 2 l + 1
__device__ __forceinline__ void load_key(const KeyWeightsParams& p, const uint8_t* row, int lane, float (&k)[18]) {
  if (!row) {
#pragma unroll
    for (int i = 0; i < 18; ++i) k[i] = 0.f;
  } else if (p.format == 0) {
    const __nv_bfloat16* r = reinterpret_cast<const __nv_bfloat16*>(row);
#pragma unroll
    for (int i = 0; i < 16; ++i) k[i] = __bfloat162float(r[16 * lane + i]);
    k[16] = __bfloat162float(r[kLatent + 2 * lane]), k[17] = __bfloat162float(r[kLatent + 2 * lane + 1]);
  } else if (p.format == 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) k[i] = e4m3_to_f32(row[16 * lane + i]);
    k[16] = e4m3_to_f32(row[kLatent + 2 * lane]), k[17] = e4m3_to_f32(row[kLatent + 2 * lane + 1]);
  } else {
    const float s = e4m3_to_f32(row[kFp4Codes + lane]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t v = e2m1x2_to_f16x2(row[8 * lane + i]);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
      k[2 * i] = f.x * s, k[2 * i + 1] = f.y * s;
    }
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(row + kFp4Pe + 4 * lane));
    k[16] = f.x, k[17] = f.y;
  }
}

__global__ void __launch_bounds__(256) key_weights_kernel(const __grid_constant__ KeyWeightsParams p) {
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const int64_t table = (int64_t)p.kv.max_pages * p.kv.page_size, cap = table < p.width ? table : p.width;
  const int len = paged_len(p.kv, p.err, b, cap, threadIdx.x == 0);
  for (int64_t j = blockIdx.x * 8 + (threadIdx.x >> 5); j < len; j += (int64_t)gridDim.x * 8) {
    float k[18], sum = 0.f;
    load_key(p, paged_row(p.kv, p.err, b, (int)j), lane, k);
    const int first = (int)max((int64_t)0, j - (len - p.s));      // the first token that sees the key
    for (int64_t r = (int64_t)first * p.H; r < (int64_t)p.s * p.H; ++r) {
      const int64_t at = (int64_t)b * p.s * p.H + r;
      const __nv_bfloat16* q = p.q + at * kDk;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) dot = fmaf(k[i], __bfloat162float(q[16 * lane + i]), dot);
      dot = fmaf(k[16], __bfloat162float(q[kLatent + 2 * lane]), dot);
      dot = fmaf(k[17], __bfloat162float(q[kLatent + 2 * lane + 1]), dot);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
      const float lse = p.lse[at];
      if (lse != -CUDART_INF_F) sum += expf(dot * p.scale - lse);
    }
    if (lane == 0) {
      float* w = p.weights + b * p.stride + j;
      *w = p.decay == 0.f ? sum : fmaf(p.decay, *w, sum);
    }
  }
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream) {
  const int64_t table = (int64_t)p.kv.max_pages * p.kv.page_size, cap = table < p.width ? table : p.width;
  const int64_t blocks = (cap + 7) / 8;
  key_weights_kernel<<<dim3((unsigned)(blocks < 1 ? 1 : blocks > 4096 ? 4096 : blocks), p.kv.B), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
