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
// dealt over all threads of the cluster, so that one long prompt among many single tokens costs no more
// than the same tokens spread evenly; a thread finds its request by bisection in shared memory.
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
  // per request of the chunk: first token / popped / returned page, relative to the chunk's first
  int tok[kThreads + 1], pop[kThreads + 1], put[kThreads + 1];
  int len[kThreads], have[kThreads], need[kThreads];
  uint8_t ok[kThreads];
  long long popped, returned;  // ends of the last request whose pages were moved
};

// last index i in [lo, n) with first[i] <= v
__device__ __forceinline__ int owner(const int* first, int n, int v, int lo = 0) {
  int hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// kRun: neighbouring tokens of a thread
template <int kThreads, int kRun>
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
  const int head_in = load(p.pool_state, 0, 2), count_in = load(p.pool_state, 1, 2);
  const bool pool_ok = head_in >= 0 && (head_in < P || (head_in == 0 && P == 0)) && count_in >= 0 && count_in <= P;
  const int64_t head = pool_ok ? head_in : 0, count = pool_ok ? count_in : 0;
  if (!pool_ok && rank == 0 && tid == 0) record_error(p.err, DEV_RANGE_BASE | 0x74);
  // (32-bit quotients, a shift where the page size allows: the divisions are most of a thread's instructions)
  auto page_of = [&](int pos) { return p.page_log2 >= 0 ? pos >> p.page_log2 : pos / p.page_size; };
  auto pages_of = [&](int tokens) { return tokens > 0 ? page_of(tokens - 1) + 1 : 0; };
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
    const int have = ok ? pages_of(len) : 0, need = ok ? pages_of(now) : 0;
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
    // ---- tokens, pages taken from the ring, pages given back behind its tail.  A pass of the loop does kRun
    // neighbouring tokens and kPages of each kind of page, and asks for everything it reads before it
    // waits for any.  Tokens start with the first warps, pages with the last and the middle ones: where there
    // are few of each, no warp has the instructions of all three. ----
    constexpr int kPages = kThreads == 256 ? 1 : 2;   // (one CTA: fewer instructions to fetch, 64 requests 3.97 us -> 3.91)
    const int64_t table = (int64_t)(ext_table / 4);
    const int pop_first = step - 1 - mine, put_first = mine < step / 2 ? mine + step / 2 : mine - step / 2;
    // (unsigned: a pass beyond 2^31 - 1 still compares as beyond)
    for (uint32_t j0 = kRun * mine, jpop = pop_first, jput = put_first; j0 < (uint32_t)ntok || jpop < (uint32_t)npop || jput < (uint32_t)nput;
         j0 += kRun * step, jpop += kPages * step, jput += kPages * step) {
      auto checked = [&](int32_t pg) {
        if (pg >= 0 && pg < P) return pg;
        record_error(p.err, DEV_RANGE_BASE | 0x75);
        return -1;
      };
      // tokens j0 .. : their requests, on from the first one's, and their pages
      int pos[kRun], entry[kRun];
      int32_t page[kRun];
      if (j0 < (uint32_t)ntok) {
        int r = owner(s.tok, nb, (int)j0), before = -1;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
          const int jt = (int)(j0 + i);
          pos[i] = -1;
          entry[i] = 0;
          page[i] = 0;
          if (j0 + i >= (uint32_t)ntok) continue;
          if (r + 1 < nb && s.tok[r + 1] <= jt) {   // mostly the next one; one behind requests without tokens else
            ++r;
            if (r + 1 < nb && s.tok[r + 1] <= jt) r = owner(s.tok, nb, jt, r);
          }
          if (!s.ok[r]) continue;
          pos[i] = s.len[r] + (jt - s.tok[r]);
          const int e = page_of(pos[i]);
          entry[i] = e * p.page_size;
          if (i > 0 && before == r && entry[i] == entry[i - 1]) {   // the same page, held or just taken
            page[i] = page[i - 1];
          } else {
            page[i] = e < s.have[r] ? load(p.block_table, (b0 + r) * p.max_pages + e, table)
                                    : load(p.pool, ring(head + pop0 + s.pop[r] + (e - s.have[r])), P);
          }
          before = r;
        }
      }
      int64_t pop_to[kPages], put_from[kPages];   // the table entries that get and hold the pages
      int32_t pop_page[kPages], put_page[kPages];
#pragma unroll
      for (int i = 0; i < kPages; ++i) {
        pop_to[i] = put_from[i] = -1;
        if (const uint32_t j = jpop + i * step; j < (uint32_t)npop) {
          const int r = owner(s.pop, nb, (int)j);
          if (s.ok[r]) {
            pop_to[i] = (b0 + r) * p.max_pages + s.have[r] + ((int)j - s.pop[r]);
            pop_page[i] = load(p.pool, ring(head + pop0 + j), P);
          }
        }
        if (const uint32_t j = jput + i * step; j < (uint32_t)nput) {
          const int r = owner(s.put, nb, (int)j);
          if (s.ok[r]) {
            put_from[i] = (b0 + r) * p.max_pages + s.need[r] + ((int)j - s.put[r]);
            put_page[i] = load(p.block_table, put_from[i], table);
          }
        }
      }
      if (j0 < (uint32_t)ntok) {
        int slot[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
          slot[i] = -1;
          if (pos[i] < 0) continue;
          const int32_t pg = checked(page[i]);
          if (pg >= 0) slot[i] = pg * p.page_size + (pos[i] - entry[i]);
        }
        const int64_t at = tok0 + j0;
        if (kRun == 4 && vec && j0 + 4 <= (uint32_t)ntok && (at & 3) == 0) {
          if (guard_span(p.err, G_STEP_OUT, p.positions + at, 16, p.positions, (uint64_t)p.N * 4))
            *reinterpret_cast<int4*>(p.positions + at) = make_int4(pos[0], pos[1 % kRun], pos[2 % kRun], pos[3 % kRun]);
          if (guard_span(p.err, G_STEP_OUT, p.slots + at, 16, p.slots, (uint64_t)p.N * 4))
            *reinterpret_cast<int4*>(p.slots + at) = make_int4(slot[0], slot[1 % kRun], slot[2 % kRun], slot[3 % kRun]);
        } else {
#pragma unroll
          for (int i = 0; i < kRun; ++i)
            if (j0 + i < (uint32_t)ntok) {
              store(p.positions, at + i, p.N, pos[i]);
              store(p.slots, at + i, p.N, slot[i]);
            }
        }
      }
#pragma unroll
      for (int i = 0; i < kPages; ++i) {
        if (pop_to[i] >= 0) store(p.block_table, pop_to[i], table, checked(pop_page[i]));
        if (put_from[i] >= 0) store(p.pool, ring(ring(head + count) + put0 + jput + i * step), P, checked(put_page[i]));
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

template <int kThreads, int kRun>
cudaError_t launch(const SlotMapParams& p, int ctas, cudaStream_t stream) {
  if (ctas > 8) {   // more than the portable size has to be asked for
    static PerDeviceOnce once;
    cudaError_t e = once.run([] { return cudaFuncSetAttribute(slot_map_kernel<kThreads, kRun>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
    if (e != cudaSuccess) return e;
  }
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
  return cudaLaunchKernelEx(&cfg, slot_map_kernel<kThreads, kRun>, p);
}

}  // namespace

cudaError_t launch_slot_map(const SlotMapParams& p, cudaStream_t stream) {
  // What a small step takes is the length of one thread's instructions, so tokens go one to a thread while two
  // passes of a cluster's threads cover them, and a decode batch runs in one small CTA, whose scan and
  // barriers are the shorter ones.  Measured, one CTA of 256 / eight of 512 / sixteen of 1024 with four
  // tokens a thread: 1 request 3.1 / 4.5 / 5.6 us; 64 requests of 0-4 tokens 3.8 / 4.9 / 7; 512 requests of one
  // token in 16-token pages 23 / 6.4 / 8.5; 8192 tokens of 32 requests 29 / 5.6 / 7.0; 16384 of 64
  // 59 / 7.5 / 7.3; 65536 of 512 252 / 21 / 8.5 (eight of 1024: 10.9).
  if (p.B <= 64 && p.N <= 256) return launch<256, 1>(p, 1, stream);
  if (p.N <= 2 * 8 * 512) return launch<512, 1>(p, 8, stream);
  return launch<1024, 4>(p, 16, stream);
}

}  // namespace mla
