// Block tables, positions and slots of one step's tokens, built on the GPU from request lengths.
//
// Request b holds lens[b] tokens and gains (n > 0) or drops (n < 0) n = new_tokens[b] of them:
//   len' = max(0, len + n), have = ceil(len / page_size), need = ceil(len' / page_size).
// A grown request takes need - have pages from the head of the ring of free pages into its table
// entries have .. need - 1; a shrunk one gives its entries need .. have - 1 back behind the ring's
// tail.  Which ring entry belongs to which request is a prefix sum over the requests, and so is the
// first token of each: token i of request b sits at position len + i, in slot
// page(position / page_size) * page_size + position % page_size.
//
// The call is a few KB to a few hundred KB of integers, so what bounds it is the latency of one
// launch and of one scan.  One cluster does all of it: every CTA scans the lengths (a chunk of
// kThreads requests at a time, 64-bit sums), and the tokens and the moved pages of the chunk are
// dealt over all threads of the cluster, so that one long prompt among many single tokens costs no
// more than the same tokens spread evenly.  A thread takes four tokens in a row: it finds the first
// one's request by bisection in shared memory and walks on from there, and looks a page up where the
// position enters it.
// lens_out and pool_state_out may be the buffers that are read: the cluster's barrier stands between
// the last read and the first write.
#include "mla_step.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {


struct Sums {
  long long tok, pop, put;
};
__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) {
  return {a.tok + b.tok, a.pop + b.pop, a.put + b.put};
}
__device__ __forceinline__ Sums shfl_up(const Sums& a, int d) {
  return {__shfl_up_sync(~0u, a.tok, d), __shfl_up_sync(~0u, a.pop, d), __shfl_up_sync(~0u, a.put, d)};
}

template <int kThreads>
struct Shared {
  Sums warp[32];
  long long total[3];
  // per request of the chunk: first token / popped / returned page, relative to the chunk's first
  int tok[kThreads + 1], pop[kThreads + 1], put[kThreads + 1];
  int len[kThreads], have[kThreads], need[kThreads];
  uint8_t ok[kThreads];
  long long popped, returned;  // ends of the last request whose pages were moved
};

// last index i in [0, n) with first[i] <= v
__device__ __forceinline__ int owner(const int* first, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) slot_map_kernel(const __grid_constant__ SlotMapParams p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ Shared<kThreads> s;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = blockIdx.x, step = gridDim.x * kThreads, mine = rank * kThreads + tid;
  const int64_t P = p.num_pages;
  const int64_t cap = min((int64_t)p.max_pages * p.page_size, (int64_t)INT32_MAX);
  const uint64_t ext_table = (uint64_t)p.B * p.max_pages * 4;
  auto load = [&](const int32_t* base, int64_t i, int64_t n) {
    return guard_span(p.err, G_STEP_IN, base + i, 4, base, (uint64_t)n * 4) ? base[i] : 0;
  };
  auto store = [&](int32_t* base, int64_t i, int64_t n, int32_t v) {
    if (guard_span(p.err, G_STEP_OUT, base + i, 4, base, (uint64_t)n * 4)) base[i] = v;
  };
  int64_t head = load(p.pool_state, 0, 2), count = load(p.pool_state, 1, 2);
  const int head_in = (int)head, count_in = (int)count;
  const bool pool_ok = head >= 0 && (head < P || (head == 0 && P == 0)) && count >= 0 && count <= P;
  if (!pool_ok) {
    head = count = 0;
    if (rank == 0 && tid == 0) record_error(p.err, DEV_RANGE_BASE | 0x74);
  }
  auto ring = [&](int64_t i) { return i >= P ? i - P : i; };  // i < 2 P
  const bool vec = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
  if (tid == 0) s.popped = s.returned = 0;
  Sums carry = {0, 0, 0};

  for (int64_t b0 = 0; b0 < p.B; b0 += kThreads) {
    const int nb = (int)min((int64_t)kThreads, p.B - b0);
    // ---- the chunk's requests ----
    int len = 0, n = 0;
    if (tid < nb) {
      len = load(p.lens, b0 + tid, p.B);
      n = load(p.new_tokens, b0 + tid, p.B);
    }
    const int64_t grown = max((int64_t)len + n, (int64_t)0);
    bool ok = len >= 0 && len <= cap && grown <= cap;
    uint32_t why = ok ? 0 : 0x70;
    const int now = ok ? (int)grown : len;
    const int have = ok ? (int)(((int64_t)len + p.page_size - 1) / p.page_size) : 0;
    const int need = ok ? (int)(((int64_t)now + p.page_size - 1) / p.page_size) : 0;
    Sums v = {max(n, 0), max(need - have, 0), max(have - need, 0)};
    const Sums own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums u = shfl_up(v, d);
      if (lane >= d) v = add(v, u);
    }
    if (lane == 31) s.warp[wid] = v;
    __syncthreads();
    if (wid == 0) {
      Sums w = lane < kWarps ? s.warp[lane] : Sums{0, 0, 0};
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Sums u = shfl_up(w, d);
        if (lane >= d) w = add(w, u);
      }
      s.warp[lane] = w;
    }
    __syncthreads();
    if (wid > 0) v = add(v, s.warp[wid - 1]);
    const Sums end = add(carry, v);                                               // through this request
    const Sums first = {end.tok - own.tok, end.pop - own.pop, end.put - own.put};  // before it
    const Sums chunk = s.warp[kWarps - 1];
    // A request that does not fit (its tokens in N, its pages in the pool or the ring) stays as it is.
    // The sums count it all the same, so every later request in need of the same thing stays too.
    if (ok && own.tok > 0 && end.tok > p.N) why = 0x72;
    if (ok && own.pop > 0 && end.pop > count) why = 0x71;
    if (ok && own.put > 0 && (!pool_ok || count + end.put > P)) why = 0x73;
    ok = ok && !why;
    if (tid < nb) {
      if (why && rank == 0) record_error(p.err, DEV_RANGE_BASE | why);
      // tokens past N have no owner: the bisection runs over offsets cut at N
      s.tok[tid] = (int)(min(first.tok, (long long)p.N) - min(carry.tok, (long long)p.N));
      s.pop[tid] = (int)(min(first.pop, (long long)count) - min(carry.pop, (long long)count));
      s.put[tid] = (int)(min(first.put, (long long)(P - count)) - min(carry.put, (long long)(P - count)));
      s.len[tid] = len;
      s.have[tid] = have;
      s.need[tid] = need;
      s.ok[tid] = ok;
      if (ok && own.pop > 0) atomicMax(&s.popped, end.pop);
      if (ok && own.put > 0) atomicMax(&s.returned, end.put);
    }
    const long long tok0 = min(carry.tok, (long long)p.N), pop0 = min(carry.pop, (long long)count),
                    put0 = min(carry.put, (long long)(P - count));
    const int ntok = (int)(min(carry.tok + chunk.tok, (long long)p.N) - tok0);
    const int npop = (int)(min(carry.pop + chunk.pop, (long long)count) - pop0);
    const int nput = (int)(min(carry.put + chunk.put, (long long)(P - count)) - put0);
    cluster_sync();  // every CTA has read the chunk's lens
    if (rank == 0 && tid < nb) {
      store(p.cu_tokens, b0 + tid, (int64_t)p.B + 1, (int32_t)min(first.tok, (long long)p.N));
      store(p.lens_out, b0 + tid, p.B, ok ? now : len);
    }
    // ---- pages taken from the ring ----
    for (int j = mine; j < npop; j += step) {
      const int r = owner(s.pop, nb, j);
      if (!s.ok[r]) continue;
      const int32_t pg = load(p.pool, ring(head + pop0 + j), P);
      const bool good = pg >= 0 && pg < P;
      if (!good) record_error(p.err, DEV_RANGE_BASE | 0x75);
      store(p.block_table, (b0 + r) * p.max_pages + s.have[r] + (j - s.pop[r]), (int64_t)(ext_table / 4), good ? pg : -1);
    }
    // ---- pages given back ----
    for (int j = mine; j < nput; j += step) {
      const int r = owner(s.put, nb, j);
      if (!s.ok[r]) continue;
      const int32_t pg = load(p.block_table, (b0 + r) * p.max_pages + s.need[r] + (j - s.put[r]), (int64_t)(ext_table / 4));
      const bool good = pg >= 0 && pg < P;
      if (!good) record_error(p.err, DEV_RANGE_BASE | 0x75);
      store(p.pool, ring(ring(head + count) + put0 + j), P, good ? pg : -1);
    }
    // ---- tokens ----
    for (int j0 = 4 * mine; j0 < ntok; j0 += 4 * step) {
      int r = owner(s.tok, nb, j0), e = -1, left = 0;   // left: tokens until the next page
      int32_t row = -1;                                 // the page's first slot, or -1
      int pos[4], slot[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i;
        pos[i] = slot[i] = -1;
        if (j >= ntok) continue;
        while (r + 1 < nb && s.tok[r + 1] <= j) ++r, e = -1;
        if (!s.ok[r]) continue;
        const int in = j - s.tok[r];
        pos[i] = s.len[r] + in;
        if (e < 0 || left == 0) {   // another page: of those held, or of those just taken
          e = pos[i] / p.page_size;
          left = (e + 1) * p.page_size - pos[i];
          const int32_t pg = e < s.have[r]
                                 ? load(p.block_table, (b0 + r) * p.max_pages + e, (int64_t)(ext_table / 4))
                                 : load(p.pool, ring(head + pop0 + s.pop[r] + (e - s.have[r])), P);
          row = pg >= 0 && pg < P ? pg * p.page_size : -1;
          if (row < 0) record_error(p.err, DEV_RANGE_BASE | 0x75);
        }
        if (row >= 0) slot[i] = row + p.page_size - left;
        --left;
      }
      const int64_t at = tok0 + j0;
      if (vec && j0 + 4 <= ntok && (at & 3) == 0) {
        if (guard_span(p.err, G_STEP_OUT, p.positions + at, 16, p.positions, (uint64_t)p.N * 4))
          *reinterpret_cast<int4*>(p.positions + at) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        if (guard_span(p.err, G_STEP_OUT, p.slots + at, 16, p.slots, (uint64_t)p.N * 4))
          *reinterpret_cast<int4*>(p.slots + at) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + i < ntok) {
            store(p.positions, at + i, p.N, pos[i]);
            store(p.slots, at + i, p.N, slot[i]);
          }
      }
    }
    carry = add(carry, chunk);
    __syncthreads();  // the chunk's tables are read
  }
  // ---- behind the last token, and the state ----
  const int64_t total = min(carry.tok, (long long)p.N);
  for (int64_t j = total + mine; j < p.N; j += step) {
    store(p.positions, j, p.N, -1);
    store(p.slots, j, p.N, -1);
  }
  cluster_sync();  // every CTA has read pool_state
  if (rank == 0 && tid == 0) {
    store(p.cu_tokens, p.B, (int64_t)p.B + 1, (int32_t)total);
    store(p.pool_state_out, 0, 2, pool_ok ? (int32_t)(P ? ring(head + s.popped) : 0) : head_in);
    store(p.pool_state_out, 1, 2, pool_ok ? (int32_t)(count - s.popped + s.returned) : count_in);
  }
}

template <int kThreads>
cudaError_t launch(const SlotMapParams& p, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, slot_map_kernel<kThreads>, p);
}

}  // namespace

cudaError_t launch_slot_map(const SlotMapParams& p, cudaStream_t stream) {
  // A decode batch fits one small CTA, whose scan and barriers are the shorter ones; a larger one gets
  // a full CTA, and eight (the portable cluster size) where those have four tokens a thread.
  if (p.B <= 128 && p.N <= 512) return launch<128>(p, 1, stream);
  return launch<1024>(p, p.N + (int64_t)p.B <= 4096 ? 1 : 8, stream);
}

}  // namespace mla
