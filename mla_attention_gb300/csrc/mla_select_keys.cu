// Which rows of each request stay: the last, the first and the heaviest, in ascending order.
//
// The m heaviest of the rows between the first and the last ones are those above the m-th largest weight, and of the rows that
// have it the lowest indices.  A weight is a 32-bit key that orders as it does; the m-th largest key is found eight bits a
// pass, from the top: a histogram of the next byte among the keys that match the bytes found so far.  Then each warp
// counts and, after one prefix sum over the warps, writes what it keeps of its own range of rows.
#include "fp4_rows.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

// larger weights have larger keys; -0 is 0, a NaN of either sign the largest
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

__global__ void __launch_bounds__(kThreads) select_keys_kernel(const __grid_constant__ SelectParams p) {
  __shared__ int hist[256];
  __shared__ int warp_gt[kWarps], warp_eq[kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = guarded_int(p.err, p.lens, b, p.B), keep = guarded_int(p.err, p.keep, b, p.B);
  const int n = min(len, keep);
  int32_t* idx = p.idx + (int64_t)b * p.K;
  const bool ok = len >= 0 && len <= p.width && keep >= 0 && n <= p.K;
  if (tid == 0) {
    if (!ok) record_error(p.err, DEV_RANGE_BASE | Y_SELECT);
    if (guard_span(p.err, G_STEP_OUT, p.count + b, 4, p.count, (uint64_t)p.B * 4)) p.count[b] = ok ? n : 0;
    if (guard_span(p.err, G_STEP_OUT, p.dropped + b, 4, p.dropped, (uint64_t)p.B * 4)) p.dropped[b] = ok ? n - len : 0;
  }
  auto put = [&](int64_t i, int v) {
    if (guard_span(p.err, G_STEP_OUT, idx + i, 4, p.idx, (uint64_t)p.B * p.K * 4)) idx[i] = v;
  };
  for (int64_t i = (ok ? n : 0) + tid; i < p.K; i += kThreads) put(i, -1);
  if (!ok) return;
  if (n == len) {
    for (int i = tid; i < n; i += kThreads) put(i, i);
    return;
  }
  const int recent = min(p.recent, n), first = min(p.first, n - recent), m = n - recent - first;
  const int lo = first, hi = len - recent;          // the m heaviest of rows lo .. hi - 1
  for (int i = tid; i < first; i += kThreads) put(i, i);
  for (int i = tid; i < recent; i += kThreads) put(n - recent + i, hi + i);
  if (m == 0) return;
  const float* w = p.weights + b * p.stride;
  auto key_at = [&](int i) {
    return guard_span(p.err, G_STEP_IN, w + i, 4, p.weights, ((uint64_t)(p.B - 1) * p.stride + p.width) * 4) ? order_key(w[i]) : 0u;
  };
  uint32_t prefix = 0;
  int need = m;                                     // of the keys that match `prefix` so far, the largest `need` stay
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kThreads) {
      const uint32_t k = key_at(i);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {                                // lane l: bins 255 - 8 l .. 248 - 8 l, from the top
      int part[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) part[i] = hist[255 - 8 * lane - i], sum += part[i];
      int above = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(~0u, above, d);
        if (lane >= d) above += v;
      }
      above -= sum;                                 // keys in the bins of the lanes before
      if (above < need && need <= above + sum) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < need && need <= above + part[i]) {
            s_prefix = prefix | (uint32_t)(255 - 8 * lane - i) << shift;
            s_need = need - above;
          }
          above += part[i];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // `need` rows of key `prefix` stay, the lowest; all above it do
  const int span = ((hi - lo + kWarps - 1) / kWarps + 31) / 32 * 32, w0 = lo + warp * span, w1 = min(hi, w0 + span);
  int gt = 0, eq = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key_at(i);
    gt += k > prefix, eq += k == prefix;
  }
  gt = warp_sum(gt), eq = warp_sum(eq);
  if (lane == 0) warp_gt[warp] = gt, warp_eq[warp] = eq;
  __syncthreads();
  int at = first, eqs = 0;                          // rows kept and equal ones met before this warp's range
  for (int i = 0; i < warp; ++i) at += warp_gt[i], eqs += warp_eq[i];
  at += min(eqs, need);
  for (int i = w0; i < w1; i += 32) {
    const uint32_t k = i + lane < w1 ? key_at(i + lane) : 0u;
    const bool in = i + lane < w1, same = in && k == prefix;
    const uint32_t same_bits = __ballot_sync(~0u, same), below = (1u << lane) - 1u;
    const bool stay = in && (k > prefix || (same && eqs + __popc(same_bits & below) < need));
    const uint32_t bits = __ballot_sync(~0u, stay);
    if (stay) put(at + __popc(bits & below), i + lane);
    at += __popc(bits), eqs += __popc(same_bits);
  }
}

}  // namespace

cudaError_t launch_select_keys(const SelectParams& p, cudaStream_t stream) {
  select_keys_kernel<<<p.B, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
