// The kept rows moved to the front of their request, in place: row i <- row idx[i], idx ascending.
//
// A CTA moves a few 16-byte columns of all of a request's rows, so no CTA writes what another one reads.  It goes through the rows
// in order, a chunk at a time: all of a chunk is read before any of it is written (row i's source lies at or behind i, so a
// write meets no later chunk's source).
#include "fp4_rows.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256, kPer = 4, kUnits = 2;   // 16-byte loads in flight a thread; 16-byte columns a CTA

// the source of entry i, or -1 where it is refused
__device__ __forceinline__ int source(const CompactParams& p, int b, int i, int64_t limit) {
  const int64_t base = (int64_t)b * p.K, all = (int64_t)p.kv.B * p.K;
  const int src = guarded_int(p.err, p.idx, base + i, all), before = i > 0 ? guarded_int(p.err, p.idx, base + i - 1, all) : -1;
  if (src < i || src <= before || src >= limit) {
    record_error(p.err, DEV_RANGE_BASE | Y_COMPACT);
    return -1;
  }
  return src;
}

__device__ __forceinline__ uint8_t* row_at(const CompactParams& p, int b, int j) {
  const int pg = j / p.kv.page_size;
  const int page = guarded_int(p.err, p.kv.block_table, (int64_t)b * p.kv.max_pages + pg, (int64_t)p.kv.B * p.kv.max_pages);
  if (page < 0 || page >= p.kv.num_pages) {
    record_error(p.err, DEV_RANGE_BASE | Y_COMPACT);
    return nullptr;
  }
  return const_cast<uint8_t*>(p.kv.cache) + ((int64_t)page * p.kv.page_size + (j - pg * p.kv.page_size)) * p.kv.row_bytes;
}

__global__ void __launch_bounds__(kThreads) compact_rows_kernel(const __grid_constant__ CompactParams p) {
  const int b = blockIdx.y, units = p.kv.row_bytes / 16, slices = (units + kUnits - 1) / kUnits;
  int count = guarded_int(p.err, p.count, b, p.kv.B);
  if (count < 0 || count > p.K) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(p.err, DEV_RANGE_BASE | Y_COMPACT);
    return;
  }
  const int64_t table = (int64_t)p.kv.max_pages * p.kv.page_size;
  const int64_t limit = p.weights && p.width < table ? p.width : table;
  if ((int)blockIdx.x == slices) {                    // the weights
    float* w = p.weights + b * p.stride;
    const uint64_t ext = ((uint64_t)(p.kv.B - 1) * p.stride + p.width) * 4;
    for (int64_t i0 = 0; i0 < count; i0 += kThreads * kPer) {
      float v[kPer];
      int to[kPer];
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int64_t i = i0 + u * kThreads + threadIdx.x;
        const int src = i < count ? source(p, b, (int)i, limit) : -1;
        to[u] = src >= 0 && src != i && guard_span(p.err, G_STEP_IN, w + src, 4, p.weights, ext) ? (int)i : -1;
        if (to[u] >= 0) v[u] = w[src];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kPer; ++u)
        if (to[u] >= 0 && guard_span(p.err, G_STEP_OUT, w + to[u], 4, p.weights, ext)) w[to[u]] = v[u];
      __syncthreads();
    }
    return;
  }
  const int col = blockIdx.x * kUnits, have = min(kUnits, units - col);
  const uint64_t ext = (uint64_t)p.kv.num_pages * p.kv.page_size * p.kv.row_bytes;
  for (int64_t i0 = 0; i0 < count; i0 += kThreads / kUnits * kPer) {
    uint4 v[kPer];
    uint8_t* to[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t i = i0 + u * (kThreads / kUnits) + threadIdx.x / kUnits;
      const int unit = threadIdx.x % kUnits;
      const int src = i < count && unit < have ? source(p, b, (int)i, limit) : -1;
      to[u] = nullptr;
      if (src >= 0 && src != i) {
        const uint8_t* from = row_at(p, b, src);
        to[u] = row_at(p, b, (int)i);
        if (!from || !to[u]) to[u] = nullptr;
        if (to[u]) {
          to[u] += 16 * (col + unit), from += 16 * (col + unit);
          if (!guard_span(p.err, G_STEP_IN, from, 16, p.kv.cache, ext) || !guard_span(p.err, G_STEP_OUT, to[u], 16, p.kv.cache, ext)) to[u] = nullptr;
          if (to[u]) v[u] = *reinterpret_cast<const uint4*>(from);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = v[u];
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_compact_rows(const CompactParams& p, cudaStream_t stream) {
  const int slices = (p.kv.row_bytes / 16 + kUnits - 1) / kUnits + (p.weights ? 1 : 0);
  compact_rows_kernel<<<dim3(slices, p.kv.B), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
