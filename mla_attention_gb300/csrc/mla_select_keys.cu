// Which rows of each request stay: the last, the first and the heaviest, in ascending order.
//
// The m heaviest of the rows between the first and the last ones are those above the m-th largest weight, and of the rows that
// have it the lowest indices.  A weight is a 32-bit key that orders as it does; the m-th largest key is found eight bits a
// pass, from the top: a histogram of the next byte among the keys that match the bytes found so far.
//
// A cluster of CTAs has the rows of a request, each a range of them whose keys it holds in shared memory (what does not fit is
// read again).  A pass is a histogram of a CTA's own keys, one cluster barrier, and the sum of the CTAs' histograms, which each
// of them reads for itself.  Then each warp counts and, after a sum over the warps and CTAs before, writes what it keeps.
//
// Latency-bound: eight steps that wait for one another.  32767 rows of one request 12 us, 64 requests of 4096 to 32768 rows 18
// us (a CTA a request, the keys read from L2 in each pass: 24 and 24 us).  512 threads: with 256 13 and 22 us, with 1024 13
// and 20.  Plain shared-memory atomics: with the lanes of a common top byte added up first 16 and 24 us, with eight copies of
// the histogram 16 and 20.
#include "fp4_rows.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kParts = kThreads / 256, kMaxRanks = 16;
constexpr int kHeld = 24576;                          // keys in shared memory
constexpr int kSmem = kHeld * 4;

__device__ __forceinline__ int peer_int(const int* own, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(own), rank)) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  cluster_sync();
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

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

__global__ void __launch_bounds__(kThreads, 2) select_keys_kernel(const __grid_constant__ SelectParams p, int ranks) {
  extern __shared__ uint32_t held[];
  __shared__ int hist[4][256], part[kParts][256];
  __shared__ int warp_gt[kWarps], warp_eq[kWarps], total[2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int b = blockIdx.x / ranks, rank = blockIdx.x - b * ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t step = (int64_t)ranks * kThreads, own = (int64_t)rank * kThreads + tid;
  const int len = guarded_int(p.err, p.lens, b, p.B), keep = guarded_int(p.err, p.keep, b, p.B);
  const int n = min(len, keep);
  int32_t* idx = p.idx + (int64_t)b * p.K;
  const bool ok = len >= 0 && len <= p.width && keep >= 0 && n <= p.K;
  cluster_arrive();                                 // this thread has the length and the budget
  auto put = [&](int64_t i, int v) {
    if (guard_span(p.err, G_STEP_OUT, idx + i, 4, p.idx, (uint64_t)p.B * p.K * 4)) idx[i] = v;
  };
  for (int64_t i = (ok ? n : 0) + own; i < p.K; i += step) put(i, -1);
  cluster_wait();                                   // all have: count or dropped may be the same memory
  if (own == 0) {
    if (!ok) record_error(p.err, DEV_RANGE_BASE | Y_SELECT);
    if (guard_span(p.err, G_STEP_OUT, p.count + b, 4, p.count, (uint64_t)p.B * 4)) p.count[b] = ok ? n : 0;
    if (guard_span(p.err, G_STEP_OUT, p.dropped + b, 4, p.dropped, (uint64_t)p.B * 4)) p.dropped[b] = ok ? n - len : 0;
  }
  if (!ok) return;
  if (n == len) {
    for (int64_t i = own; i < n; i += step) put(i, (int)i);
    return;
  }
  const int recent = min(p.recent, n), first = min(p.first, n - recent), m = n - recent - first;
  for (int64_t i = own; i < first; i += step) put(i, (int)i);
  for (int64_t i = own; i < recent; i += step) put(n - recent + i, len - recent + (int)i);
  if (m == 0) return;

  // the m heaviest of rows first .. len - recent - 1; this CTA's: `rows` of them from `lo`
  const int among = len - recent - first, share = (among + ranks - 1) / ranks;
  const int lo = first + (int)min((int64_t)among, (int64_t)rank * share), rows = min(share, first + among - lo);
  const float* w = p.weights + b * p.stride + lo;
  auto read = [&](int i) {
    return guard_span(p.err, G_STEP_IN, w + i, 4, p.weights, ((uint64_t)(p.B - 1) * p.stride + p.width) * 4) ? order_key(w[i]) : 0u;
  };
  auto key = [&](int i) { return i < kHeld ? held[i] : read(i); };
  const int held_rows = min(rows, kHeld);
#pragma unroll 4
  for (int i = tid; i < held_rows; i += kThreads) held[i] = read(i);
  for (int i = tid; i < 1024; i += kThreads) hist[i >> 8][i & 255] = 0;
  __syncthreads();

  uint32_t prefix = 0;
  int need = m;                                     // of the keys that match `prefix` so far, the largest `need` stay
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* const own_hist = hist[pass];
#pragma unroll 4
    for (int i = tid; i < rows; i += kThreads) {
      const uint32_t k = key(i);
      if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&own_hist[(k >> shift) & 255u], 1);
    }
    cluster_barrier();
    int sum = 0, of[kMaxRanks / kParts];
#pragma unroll
    for (int i = 0; i < kMaxRanks / kParts; ++i) {
      const int r = (tid >> 8) + i * kParts;
      of[i] = r < ranks ? peer_int(&own_hist[tid & 255], r) : 0;
    }
#pragma unroll
    for (int i = 0; i < kMaxRanks / kParts; ++i) sum += of[i];
    part[tid >> 8][tid & 255] = sum;
    __syncthreads();
    if (warp == 0) {                                // lane l: bins 255 - 8 l .. 248 - 8 l, from the top
      int bins[8], sum8 = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bins[i] = 0;
#pragma unroll
        for (int g = 0; g < kParts; ++g) bins[i] += part[g][255 - 8 * lane - i];
        sum8 += bins[i];
      }
      int above = sum8;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(~0u, above, d);
        if (lane >= d) above += v;
      }
      above -= sum8;                                // keys in the bins of the lanes before
      if (above < need && need <= above + sum8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < need && need <= above + bins[i]) {
            s_prefix = prefix | (uint32_t)(255 - 8 * lane - i) << shift;
            s_need = need - above;
          }
          above += bins[i];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // `need` rows of key `prefix` stay, the lowest; all above it do
  const int span = ((rows + kWarps - 1) / kWarps + 31) / 32 * 32, w0 = min(rows, warp * span), w1 = min(rows, w0 + span);
  int gt = 0, eq = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key(i);
    gt += k > prefix, eq += k == prefix;
  }
  gt = warp_sum(gt), eq = warp_sum(eq);
  if (lane == 0) warp_gt[warp] = gt, warp_eq[warp] = eq;
  __syncthreads();
  if (warp == 0) {
    const int g = warp_sum(lane < kWarps ? warp_gt[lane] : 0), e = warp_sum(lane < kWarps ? warp_eq[lane] : 0);
    if (lane == 0) total[0] = g, total[1] = e;
  }
  cluster_barrier();
  // rows kept and equal ones met before this warp's range
  int at = lane < rank ? peer_int(&total[0], lane) : 0, eqs = lane < rank ? peer_int(&total[1], lane) : 0;
  if (lane < warp) at += warp_gt[lane], eqs += warp_eq[lane];
  at = first + warp_sum(at), eqs = warp_sum(eqs);
  at += min(eqs, need);
  for (int i = w0; i < w1; i += 32) {
    const uint32_t k = i + lane < w1 ? key(i + lane) : 0u;
    const bool in = i + lane < w1, same = in && k == prefix;
    const uint32_t same_bits = __ballot_sync(~0u, same), below = (1u << lane) - 1u;
    const bool stay = in && (k > prefix || (same && eqs + __popc(same_bits & below) < need));
    const uint32_t bits = __ballot_sync(~0u, stay);
    if (stay) put(at + __popc(bits & below), lo + i + lane);
    at += __popc(bits), eqs += __popc(same_bits);
  }
  cluster_barrier();                                // no CTA ends while another one reads its sums
}

}  // namespace

cudaError_t launch_select_keys(const SelectParams& p, cudaStream_t stream) {
  static PerDeviceOnce attrs;
  const cudaError_t e = attrs.run([] {
    const cudaError_t r = cudaFuncSetAttribute((const void*)select_keys_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return r == cudaSuccess ? cudaFuncSetAttribute((const void*)select_keys_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) : r;
  });
  if (e != cudaSuccess) return e;
  // clusters so large that all run at once (one request with four CTAs: 24 us for 12)
  int ranks = kMaxRanks;
  while (ranks > 1 && (int64_t)ranks * p.B > 2 * device_sm_count()) ranks /= 2;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3((unsigned)(p.B * ranks));
  config.blockDim = dim3(kThreads);
  config.dynamicSmemBytes = kSmem;
  config.stream = stream;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = (unsigned)ranks, cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  config.attrs = &cluster;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, select_keys_kernel, p, ranks);
}

}  // namespace mla
