// The kept rows moved to the front of their request, in place: row i <- row idx[i], idx ascending.
//
// Row i's source lies at or behind i, so with the rows taken in order, a chunk at a time, it is enough that all of a chunk is
// read before any of it is written: what is written meets no later chunk's source, and later chunks' loads may be on their
// way already.  A cluster of CTAs takes a request's rows (or some columns of them), and a CTA its share of each chunk:
//   warps 0-11   ask for two chunks ahead into shared memory, and write a chunk once all CTAs have theirs of it: each thread
//                the pieces that it asked for itself
//   warp 12      says to the cluster's CTAs that this one's pieces of a chunk are there.  It has no load or store of its own
//                on its way, which a release to the cluster would wait for
//   warps 13-15  look up where rows come from and go to, up to six chunks ahead
// Weights have a cluster of their own, and move where their rows do.
//
// Bound by the bytes on their way (up to 90 KB a CTA, two CTAs a SM) and at many requests by the longest of them: 64 of 4096
// to 16384 kept 4-bit rows take 0.118 ms, 4.3 TB/s; 21845 bf16 rows of one request 17 us, 2.9 TB/s.  Measured instead: a CTA
// for some columns of all of a request's rows, no cluster, 0.169 ms and 67 us; a cluster's barrier between reading and writing
// 0.176 ms (its release waits for the loads on their way); chunks of 24 KB, four in memory, 0.134; of 42 KB, two, 0.131.
#include "fp4_rows.cuh"
#include "tile_waits.cuh"

namespace mla {
namespace {

constexpr int kMoverWarps = 12, kMovers = 32 * kMoverWarps, kLookWarps = 3, kThreads = kMovers + 32 + 32 * kLookWarps;
constexpr int kPer = 5, kStages = 3;           // 16-byte pieces a thread and chunk; chunks in shared memory
constexpr int kRing = 2 * kLookWarps, kMaxRows = 192;    // chunks whose rows are known; rows a chunk and CTA at most
constexpr int kSmem = kStages * kPer * kMovers * 16;
enum : uint32_t { C_LANDED = 0x1E0, C_READ, C_KNOWN, C_FREE, C_STALL };

struct Bars {
  uint64_t landed[kStages];      // this CTA's pieces of the chunk are in shared memory
  uint64_t read[kStages];        // all CTAs' are
  uint64_t known[kRing], free[kRing], stall;
  uint32_t abort;
};

// entry i and the one before it 
__device__ __forceinline__ int2 entry(const CompactParams& p, int b, int64_t i, int count) {
  const int64_t base = (int64_t)b * p.K, all = (int64_t)p.kv.B * p.K;
  if (i >= count) return make_int2(-1, -1);
  return make_int2(i > 0 ? guarded_int(p.err, p.idx, base + i - 1, all) : -1, guarded_int(p.err, p.idx, base + i, all));
}
// is it one that moves?  Those that are refused are recorded and stay.
__device__ __forceinline__ bool moving(const CompactParams& p, int64_t i, int count, int2 en, int64_t limit, bool report) {
  if (i >= count) return false;
  if (en.y >= i && en.y > en.x && en.y < limit) return en.y > i;
  if (report) record_error(p.err, DEV_RANGE_BASE | Y_COMPACT);
  return false;
}
// cache row of row j of request b, -1 where its page is none
__device__ __forceinline__ int row_at(const CompactParams& p, int b, int j, bool report) {
  const int pg = j / p.kv.page_size;
  const int page = guarded_int(p.err, p.kv.block_table, (int64_t)b * p.kv.max_pages + pg, (int64_t)p.kv.B * p.kv.max_pages);
  if (page < 0 || page >= p.kv.num_pages) {
    if (report) record_error(p.err, DEV_RANGE_BASE | Y_COMPACT);
    return -1;
  }
  return page * p.kv.page_size + (j - pg * p.kv.page_size);
}

__device__ __forceinline__ void move_weights(const CompactParams& p, int b, int rank, int ranks, int count, int64_t limit) {
  constexpr int kMany = 8;
  float* w = p.weights + b * p.stride;
  const uint64_t ext = ((uint64_t)(p.kv.B - 1) * p.stride + p.width) * 4;
  for (int64_t i0 = 0; i0 < count; i0 += (int64_t)ranks * kThreads * kMany) {
    float v[kMany];
    int to[kMany];
#pragma unroll
    for (int u = 0; u < kMany; ++u) {
      const int64_t i = i0 + ((int64_t)rank * kMany + u) * kThreads + threadIdx.x;
      const int2 en = entry(p, b, i, count);
      // with its row: where that has no page, or its place has none, neither moves
      const bool moves = moving(p, i, count, en, limit, false) && row_at(p, b, en.y, false) >= 0 && row_at(p, b, (int)i, false) >= 0;
      to[u] = moves && guard_span(p.err, G_STEP_IN, w + en.y, 4, p.weights, ext) ? (int)i : -1;
      if (to[u] >= 0) v[u] = __ldcg(w + en.y);
    }
    __syncwarp();
    cluster_sync();
#pragma unroll
    for (int u = 0; u < kMany; ++u)
      if (to[u] >= 0 && guard_span(p.err, G_STEP_OUT, w + to[u], 4, p.weights, ext)) w[to[u]] = v[u];
  }
}

// A cluster: request and slice, `units` 16-byte columns of its rows (the slice behind the last one: the weights).
__global__ void __launch_bounds__(kThreads, 2) compact_rows_kernel(const __grid_constant__ CompactParams p, int units, int slices, int ranks) {
  extern __shared__ __align__(16) uint4 pieces[];     // [stage][piece of a thread][mover]
  __shared__ int2 moves[kRing][kMaxRows];        // cache rows (from, to), from < 0: stays
  __shared__ Bars bars;
  const int group = blockIdx.x / ranks, rank = blockIdx.x - group * ranks, all_slices = slices + (p.weights ? 1 : 0);
  const int b = group / all_slices, slice = group - b * all_slices, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int count = guarded_int(p.err, p.count, b, p.kv.B);
  const bool report = slice == 0;
  if (count < 0 || count > p.K) {
    if (report && rank == 0 && tid == 0) record_error(p.err, DEV_RANGE_BASE | Y_COMPACT);
    return;
  }
  const int64_t table = (int64_t)p.kv.max_pages * p.kv.page_size, limit = p.weights && p.width < table ? p.width : table;
  if (slice == slices) return move_weights(p, b, rank, ranks, count, limit);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars.landed[i], kMovers), mbar_init(&bars.read[i], ranks);
    for (int i = 0; i < kRing; ++i) mbar_init(&bars.known[i], 1), mbar_init(&bars.free[i], kMoverWarps);
    mbar_init(&bars.stall, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  cluster_sync();
  const TileWaits wait{&bars.abort, p.err, p.spin_limit};
  const int col = slice * units, have = min(units, p.kv.row_bytes / 16 - col), rows = min(kMaxRows, kMovers * kPer / have);
  const int chunks = (int)(((int64_t)count + (int64_t)ranks * rows - 1) / ((int64_t)ranks * rows));

  if (warp > kMoverWarps) {
    // ---------------- where the rows lie ----------------
    constexpr int kLooks = kMaxRows / 32;
    int2 en[kLooks];
    auto place = [&](int c, int k) { return ((int64_t)c * ranks + rank) * rows + k * 32 + lane; };
    auto ask = [&](int c) {
#pragma unroll
      for (int k = 0; k < kLooks; ++k)
        en[k] = c < chunks && k * 32 + lane < rows ? entry(p, b, place(c, k), count) : make_int2(-1, -1);
    };
    ask(warp - kMoverWarps - 1);
    for (int c = warp - kMoverWarps - 1; c < chunks; c += kLookWarps) {
      const int slot = c % kRing;
      if (!wait.warp(&bars.free[slot], ((c / kRing) & 1) ^ 1, C_FREE)) break;
#pragma unroll
      for (int k = 0; k < kLooks; ++k) {
        if (k * 32 + lane >= rows) continue;
        const int64_t i = place(c, k);
        int2 m = make_int2(-1, -1);
        if (moving(p, i, count, en[k], limit, report)) {
          m = make_int2(row_at(p, b, en[k].y, report), row_at(p, b, (int)i, report));
          if (m.y < 0) m.x = -1;
        }
        moves[slot][k * 32 + lane] = m;
      }
      warp_arrive(&bars.known[slot]);
      ask(c + kLookWarps);
    }
  } else if (warp == kMoverWarps) {
    // ---------------- this CTA's pieces are there ----------------
    bool live = !p.debug_stall || wait.warp(&bars.stall, 0, C_STALL);
    for (int c = 0; live && c < chunks; ++c) {
      if (!wait.warp(&bars.landed[c % kStages], (c / kStages) & 1, C_LANDED)) break;
      if (lane < ranks) mbar_arrive_remote(map_to_rank(smem_u32(&bars.read[c % kStages]), lane));
      __syncwarp();
    }
  } else {
    // ---------------- rows ----------------
    int at[kPer], off[kPer];                          // this thread's pieces: row of the CTA's share, byte of the row
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int item = tid + k * kMovers;
      at[k] = item / have, off[k] = 16 * (col + item - at[k] * have);
      if (at[k] >= rows) at[k] = -1;
    }
    const uint64_t ext = (uint64_t)p.kv.num_pages * p.kv.page_size * p.kv.row_bytes;
    uint8_t* const cache = const_cast<uint8_t*>(p.kv.cache);
    auto load = [&](int c) {
      if (c >= chunks) return true;
      if (!wait.warp(&bars.known[c % kRing], (c / kRing) & 1, C_KNOWN)) return false;
      const uint32_t stage = smem_u32(pieces + (c % kStages) * kPer * kMovers + tid);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int from = at[k] >= 0 ? moves[c % kRing][at[k]].x : -1;
        const uint8_t* s = cache + (int64_t)from * p.kv.row_bytes + off[k];
        if (from >= 0 && guard_span(p.err, G_STEP_IN, s, 16, p.kv.cache, ext)) cp_async16_zfill(stage + k * kMovers * 16, s, 16);
      }
      cp_async_arrive_noinc(&bars.landed[c % kStages]);
      return true;
    };
    bool live = true;
    for (int c = 0; live && c < kStages - 1; ++c) live = load(c);
    for (int c = 0; live && c < chunks; ++c) {
      if (!load(c + kStages - 1)) break;              // over the pieces written from in the step before
      if (!wait.warp(&bars.read[c % kStages], (c / kStages) & 1, C_READ, true)) break;
      const uint4* stage = pieces + (c % kStages) * kPer * kMovers + tid;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int2 m = at[k] >= 0 ? moves[c % kRing][at[k]] : make_int2(-1, -1);
        uint8_t* d = cache + (int64_t)m.y * p.kv.row_bytes + off[k];
        if (m.x >= 0 && guard_span(p.err, G_STEP_OUT, d, 16, p.kv.cache, ext)) *reinterpret_cast<uint4*>(d) = stage[k * kMovers];
      }
      warp_arrive(&bars.free[c % kRing]);
    }
    cp_async_wait_all();
  }
  __syncwarp();
  cluster_sync();                                     // no arrival is on its way to a CTA that has ended
}

}  // namespace

cudaError_t launch_compact_rows(const CompactParams& p, cudaStream_t stream) {
  static PerDeviceOnce attrs;
  const cudaError_t e = attrs.run([] {
    const cudaError_t r = cudaFuncSetAttribute((const void*)compact_rows_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return r == cudaSuccess ? cudaFuncSetAttribute((const void*)compact_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) : r;
  });
  if (e != cudaSuccess) return e;
  // No more CTAs than run at once: a request's rows to a cluster of up to sixteen, then their columns, in no more slices than
  // leave a chunk full with kMaxRows rows (one request: 96 CTAs for bf16 rows, 48 for e4m3, 32 for 4-bit ones, and 16 for the
  // weights, of 304).  (One request in clusters of eight: 28 us for 17.)
  const int columns = p.kv.row_bytes / 16, room = 2 * device_sm_count();
  int ranks = 16;
  while (ranks > 1 && (int64_t)ranks * p.kv.B > room) ranks /= 2;
  int slices = (int)(room / ((int64_t)ranks * p.kv.B));
  if (slices > columns * kMaxRows / (kMovers * kPer)) slices = columns * kMaxRows / (kMovers * kPer);
  if (slices < 1) slices = 1;
  int units = (columns + slices - 1) / slices;
  if (slices > 1 && units % 2) ++units;               // whole 32-byte sectors
  if (units > kMovers * kPer) units = kMovers * kPer;
  slices = (columns + units - 1) / units;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3((unsigned)(p.kv.B * (slices + (p.weights ? 1 : 0)) * ranks));
  config.blockDim = dim3(kThreads);
  config.dynamicSmemBytes = kSmem;
  config.stream = stream;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = (unsigned)ranks, cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  config.attrs = &cluster;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, compact_rows_kernel, p, units, slices, ranks);
}

}  // namespace mla
