// The attention that each cached key got, added up over query tokens and heads.
//   weights[b, j] = decay weights[b, j] + sum_{i, h} exp(scale q_{b,i,h} . k_j - lse_{b,i,h})
//
// Scores are taken the other way round, S^T = K Q^T with 128 keys as the rows of a tile and up to 128 query rows (token, head) as
// its columns (a pair of SMs: 256 of either): a key is then a lane of tensor memory and its sum over the query rows stays in one thread, with neither
// shuffles nor atomics.  The query rows of a request stay in shared memory while its keys stream past.  More than 128 of
// them are taken a chunk after the other over a few tiles at a time (kSub), so that the keys come from L2 again; a CTA's
// part of such a range's sums goes to the workspace, and key_weights_sum_kernel adds the parts up in their order.
//
// More than 128 query rows go to clusters of two CTAs: MMAs of the pair (cta_group::2, M = N = 256), each CTA
// with 128 keys and half of the query rows, so that a key made f16 meets twice as many of them.
//
// A CTA (or pair) per SM takes an equal share of all tiles.  16 warps:
//   0-3   a key a thread: S from tensor memory, exponentials, the weight's update
//   4     MMAs (one thread, of the first CTA): nine 64-column boxes of K against those of Q
//   5     rows of the next tiles through the block table, and the chunk's log-sum-exps
//   6-15  producers, two for each stage of the ring, 64 rows each: bf16 rows by cp.async; e4m3 and 4-bit rows through
//         registers into f16 (exact), with q in f16 too, the next box's loads out before the last one's are converted; the RoPE
//         columns of 4-bit rows stay bf16.  A stage has producers of its own, as a parity tells no more than the last phase.
//
// One new token of 128 heads and request over bf16 rows is HBM-bound: 64 requests of 4096 to 32768 keys 0.224 to 0.229 ms, 6.0 to 6.2 TB/s.  The
// first-level cache (rows, their f16 form, the MMAs' operands) bounds the others: 32 such requests 0.110 ms with e4m3 rows, 0.128 with
// 4-bit ones; 4096 query rows over 32768 4-bit keys 0.119 ms, 1.30 PFLOP/s (without pairs 0.211).
#include <math_constants.h>

#include "fp4_rows.cuh"
#include "tile_waits.cuh"

namespace mla {
namespace {

constexpr int kTile = 128;                       // a CTA's keys of a tile, and its query rows of a chunk
constexpr int kBoxes = kDk / 64;
constexpr int kBoxBytes = kTile * 128;
constexpr int kStages = 5;                       // K boxes on their way
constexpr int kRowSlots = 3;                     // tiles whose rows are known
constexpr int kSub = 8;                          // tiles before the next chunk of query rows
constexpr int kThreads = 512, kProducers = 2 * kStages, kFirstProducer = 6;

constexpr int kOffQ = 0;
constexpr int kOffK = kBoxes * kBoxBytes;
constexpr int kOffRows = kOffK + kStages * kBoxBytes;
constexpr int kOffLse = kOffRows + kRowSlots * kTile * 4;
constexpr int kOffBars = kOffLse + 2 * kTile * 4;

struct Bars {
  uint64_t kfull[kStages], kempty[kStages];
  uint64_t qfull[kBoxes], qempty[kBoxes];
  uint64_t sfull[2], sfree[2];
  uint64_t rfull[kRowSlots], rfree[kRowSlots];
  uint64_t lfull[2], lfree[2];
  uint64_t drain, stall;
  uint32_t tmem_base, abort;
  uint32_t skips[2];             // a chunk of query rows has some that add nothing
  int32_t start_b, start_t, start_o;
  int64_t share, start_range;
};
constexpr int kSmem = kOffBars + 512;
static_assert(sizeof(Bars) <= 512, "barrier block too large");
static_assert(kSmem <= 232448, "shared memory over the sm_103a limit");

enum : uint32_t { W_KFULL = 0x180, W_KEMPTY, W_QFULL, W_QEMPTY, W_SFULL, W_SFREE, W_RFULL, W_RFREE, W_LFULL, W_LFREE, W_STALL, W_ALIGN };

// Work of one load of query rows: chunk c of request b against tiles t0 + i0 .. t0 + i1 - 1.
struct Segment {
  int b, len, t0, nt, c, i0, i1;
  int64_t range;           // with several chunks: the index of the range of nt tiles at t0
  int from;                // and the first unit (c * nt + tile) of it that this CTA has
};

template <int kCtas>
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile * kCtas - 1) / (kTile * kCtas); }

// This CTA's share of the units (tile, chunk): request by request, kSub tiles at a time, a chunk of query rows after the other
// over them.  With one chunk a segment is all of a request that the share has.
template <int kCtas>
struct Shares {
  const KeyWeightsParams* p;
  int64_t cap, left, range;
  int b, t0, o, from, chunks;
  __device__ Shares(const KeyWeightsParams& prm, int64_t cap_, const Bars& bars, int chunks_)
      : p(&prm), cap(cap_), left(bars.share), range(bars.start_range), b(bars.start_b), t0(bars.start_t), o(bars.start_o), from(bars.start_o),
        chunks(chunks_) {}
  __device__ __noinline__ bool next(Segment& s) {       // one copy for all roles: the loops should stay in the instruction cache
    while (left > 0 && b < p->kv.B) {
      const int len = paged_len(p->kv, p->err, b, cap, false), all = tiles_of<kCtas>(len) - t0;
      if (all <= 0) {
        ++b, t0 = 0;
        continue;
      }
      const int nt = chunks > 1 ? min(all, kSub) : all;
      s.b = b, s.len = len, s.t0 = t0, s.nt = nt, s.range = range, s.from = from;
      s.c = o / nt, s.i0 = o - s.c * nt;
      s.i1 = (int)min((int64_t)nt, s.i0 + left);
      o += s.i1 - s.i0, left -= s.i1 - s.i0;
      if (o == nt * chunks) t0 += nt, o = 0, from = 0, ++range;
      return true;
    }
    return false;
  }
};

// Where this CTA's share starts; by all threads.  With several chunks the first CTA puts down the tiles and ranges before each
// request.
template <int kCtas>
__device__ __noinline__ void find_share(const KeyWeightsParams& p, int64_t cap, int chunks, Bars& bars, int32_t* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.kv.B + kThreads - 1) / kThreads, b0 = min(tid * per, p.kv.B), b1 = min(b0 + per, p.kv.B);
  int64_t tiles = 0, ranges = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = tiles_of<kCtas>(paged_len(p.kv, p.err, b, cap, blockIdx.x == 0));
    tiles += n, ranges += (n + kSub - 1) / kSub;
  }
  int64_t t_upto = tiles, r_upto = ranges;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t v = __shfl_up_sync(~0u, t_upto, d), r = __shfl_up_sync(~0u, r_upto, d);
    if (lane >= d) t_upto += v, r_upto += r;
  }
  if (lane == 31) sums[2 * warp] = (int32_t)t_upto, sums[2 * warp + 1] = (int32_t)r_upto;   // below 2^31 / 128 rows
  __syncthreads();
  int64_t t_at = t_upto - tiles, r_at = r_upto - ranges, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) t_at += sums[2 * w], r_at += sums[2 * w + 1];
    total += sums[2 * w];
  }
  total *= chunks;
  const int64_t share = blockIdx.x / kCtas, all = gridDim.x / kCtas, lo = total * share / all, hi = total * (share + 1) / all;
  if (tid == 0) bars.share = hi - lo;
  const bool tell = chunks > 1 && blockIdx.x == 0, here = lo < hi && t_at * chunks <= lo && lo < (t_at + tiles) * chunks;
  if (tell || here) {
    for (int b = b0; b < b1; ++b) {
      const int n = tiles_of<kCtas>(paged_len(p.kv, p.err, b, cap, false));
      if (tell) {
        p.before[2 * b] = (int32_t)t_at, p.before[2 * b + 1] = (int32_t)r_at;
        if (b == p.kv.B - 1) p.before[2 * b + 2] = (int32_t)(t_at + n);
      }
      if (lo < hi && t_at * chunks <= lo && lo < (t_at + n) * chunks) {
        const int64_t off = lo - t_at * chunks;           // in units
        bars.start_b = b;
        if (chunks == 1) {
          bars.start_t = (int)off, bars.start_o = 0, bars.start_range = r_at;
        } else {
          const int64_t k = off / (kSub * chunks);
          bars.start_t = (int)(k * kSub), bars.start_o = (int)(off - k * kSub * chunks), bars.start_range = r_at + k;
        }
      }
      t_at += n, r_at += (n + kSub - 1) / kSub;
    }
  }
}

__device__ __forceinline__ uint32_t box_unit(uint32_t box, int row, int unit) {   // 16 bytes of a swizzled 128-byte row
  return box + row * 128 + ((unit ^ (row & 7)) << 4);
}
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Sums of exp2(score c2 + addend) over 32 query rows of this lane's key, without those that `none` tells.
template <class None>
__device__ __forceinline__ void key_sums32(uint32_t from, uint64_t c22, const float* addends, uint64_t (&sum2)[2], None none) {
  uint32_t s[32];
  tmem_ld32(from, s);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(addends + i);
    float x0, x1, x2, x3;
    f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c22, f32x2(l.x, l.y)), x0, x1);
    f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), c22, f32x2(l.z, l.w)), x2, x3);
    x0 = ex2_approx(x0), x1 = ex2_approx(x1), x2 = ex2_approx(x2), x3 = ex2_approx(x3);
    x0 = none(i, l.x) ? 0.f : x0, x1 = none(i + 1, l.y) ? 0.f : x1, x2 = none(i + 2, l.z) ? 0.f : x2, x3 = none(i + 3, l.w) ? 0.f : x3;
    sum2[0] = add_f32x2(sum2[0], f32x2(x0, x1));
    sum2[1] = add_f32x2(sum2[1], f32x2(x2, x3));
  }
}
__device__ __forceinline__ float sum_of(const uint64_t (&sum2)[2]) {
  float a, b;
  f32x2_split(add_f32x2(sum2[0], sum2[1]), a, b);
  return a + b;
}
// n query rows, of which the last 32 may be less
__device__ __forceinline__ float key_sum(uint32_t from, int n, uint64_t c22, const float* addends) {
  uint64_t sum2[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
  int n0 = 0;
  for (; n0 + 32 <= n; n0 += 32) key_sums32(from + n0, c22, addends + n0, sum2, [](int, float) { return false; });
  if (n0 < n) key_sums32(from + n0, c22, addends + n0, sum2, [=](int i, float) { return n0 + i >= n; });
  return sum_of(sum2);
}
// The same without the rows below `hidden` and those whose addend is -inf, whatever their score is (an infinite one, or a NaN, is
// not made nothing by the addend).  Out of line, for the tiles that need it: the loop stays in the instruction cache.
__device__ __noinline__ float key_sum_of_some(uint32_t from, int n, uint64_t c22, const float* addends, int hidden) {
  uint64_t sum2[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
  for (int n0 = 0; n0 < n; n0 += 32)
    key_sums32(from + n0, c22, addends + n0, sum2, [=](int i, float l) { return n0 + i < hidden || l == -CUDART_INF_F; });
  return sum_of(sum2);
}

constexpr int kNoRow = -1;                       // no key there, or its page is none
// kCtas 2: a cluster of two CTAs, MMAs of the pair
template <int kFmt, int kCtas>
__global__ void __launch_bounds__(kThreads, 1) key_weights_kernel(const __grid_constant__ KeyWeightsParams p) {
  constexpr int kChunk = kCtas * kTile, kLseSlots = 2 / kCtas;      // query rows a chunk
  constexpr uint32_t kTmemCols = 2 * kChunk;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + kOffBars);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t table = (int64_t)p.kv.max_pages * p.kv.page_size, cap = table < p.width ? table : p.width;
  const int rows = p.s * p.H, chunks = (rows + kChunk - 1) / kChunk;
  const int cta = kCtas == 1 ? 0 : (int)cluster_ctarank(), share = blockIdx.x / kCtas;
  const uint64_t cache_bytes = (uint64_t)p.kv.num_pages * p.kv.page_size * p.kv.row_bytes;
  // bf16: every lane of both producers arrives when its copies have landed, in its own CTA; warp 4 of the second CTA hands that on
  const uint32_t arrivals = kFmt == kCacheBf16 ? (kCtas == 2 && cta == 0 ? 65 : 64) : 2 * kCtas;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars.kfull[i], arrivals), mbar_init(&bars.kempty[i], 1);
    for (int i = 0; i < kBoxes; ++i) mbar_init(&bars.qfull[i], arrivals), mbar_init(&bars.qempty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bars.sfull[i], 1), mbar_init(&bars.sfree[i], 4 * kCtas);
    for (int i = 0; i < kRowSlots; ++i) mbar_init(&bars.rfull[i], 1), mbar_init(&bars.rfree[i], kProducers);
    for (int i = 0; i < 2; ++i) mbar_init(&bars.lfull[i], 1), mbar_init(&bars.lfree[i], 4);
    mbar_init(&bars.drain, 1);
    mbar_init(&bars.stall, 1);
    bars.abort = 0;
    if (smem_u32(smem) & 1023u) bars.abort = DEV_TIMEOUT_BASE | W_ALIGN, record_error(p.err, bars.abort);
    fence_mbar_init();
  }
  if (warp == 4) {
    if constexpr (kCtas == 1) {
      tmem_alloc(&bars.tmem_base, kTmemCols);
      tmem_relinquish();
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem_base)), "n"(kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  find_share<kCtas>(p, cap, chunks, bars, reinterpret_cast<int32_t*>(smem + kOffRows));   // no row is there yet
  tc_fence_before();
  __syncthreads();
  if constexpr (kCtas == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tbase = bars.tmem_base;
  const TileWaits wait{&bars.abort, p.err, p.spin_limit};
  int32_t* row_slots = reinterpret_cast<int32_t*>(smem + kOffRows);
  float* lse_slots = reinterpret_cast<float*>(smem + kOffLse);
  Shares<kCtas> shares(p, cap, bars, chunks);
  Segment it;
  uint32_t u = 0, c_all = 0;                     // units and segments gone through
  bool live = bars.abort == 0;
  // what the MMAs of the pair wait for, in the first CTA
  auto tell = [&](uint64_t* bar) {
    if constexpr (kCtas == 1) warp_arrive(bar);
    else first_cta_arrive<true>(bar, cta);
  };

  if (warp < 4) {
    // ---------------- a key a thread ----------------
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const float c2 = p.scale * 1.4426950408889634f;
    const uint64_t c22 = f32x2(c2, c2);
    while (live && shares.next(it)) {
      const uint32_t lslot = c_all % kLseSlots;
      const float* minus_lse = lse_slots + lslot * kChunk;
      if (!wait.warp(&bars.lfull[lslot], (c_all / kLseSlots) & 1, W_LFULL)) break;
      const bool skips = bars.skips[lslot] != 0;
      const int n = min(rows - it.c * kChunk, kChunk);
      for (int i = it.i0; i < it.i1; ++i, ++u) {
        const int j = ((it.t0 + i) * kCtas + cta) * kTile + tid, buf = u & 1;
        bool mine = j < it.len, first;
        float* w;
        if (chunks == 1) {
          w = p.weights + it.b * p.stride + j, first = p.decay == 0.f;
          mine = mine && guard_span(p.err, G_STEP_OUT, w, 4, p.weights, ((uint64_t)(p.kv.B - 1) * p.stride + p.width) * 4);
        } else {       // this CTA's part of the range's sums
          w = p.part + ((it.range + share) * kSub + i) * kChunk + cta * kTile + tid, first = it.c * it.nt + i - it.nt < it.from;
          mine = mine && guard_span(p.err, G_PART_O, w, 4, p.part, p.part_bytes);
        }
        const float old = mine && !first ? *w : 0.f;
        // query rows below `hidden` do not see the key
        const int hidden = (int)max((int64_t)0, (int64_t)(j - (it.len - p.s)) * p.H - it.c * kChunk);
        const bool choose = __any_sync(~0u, j < it.len && hidden > 0) || skips;
        if (!wait.warp(&bars.sfull[buf], (u >> 1) & 1, W_SFULL)) { live = false; break; }
        tc_fence_after();
        const uint32_t from = tbase + lanes + buf * kChunk;
        const float sum = choose ? key_sum_of_some(from, n, c22, minus_lse, hidden) : key_sum(from, n, c22, minus_lse);
        tc_fence_before();
        if constexpr (kCtas == 1) warp_arrive(&bars.sfree[buf]);
        else first_cta_arrive<false>(&bars.sfree[buf], cta);
        if (mine) *w = first ? sum : chunks == 1 ? fmaf(p.decay, old, sum) : old + sum;
      }
      if (live) warp_arrive(&bars.lfree[lslot]);
      ++c_all;
    }
  } else if (warp == 4) {
    // ---------------- MMAs (the whole warp waits, one lane issues) ----------------
    // (not unrolled: nine copies pass the instruction cache, without pairs 284 against 211 us for 4096 query rows and 32768 keys in 4 bits)
    if (p.debug_stall) live = live && wait.warp(&bars.stall, 0, W_STALL);
    if (cta == 0) {
      const uint64_t kdesc = sdesc_sw128(smem_u32(smem + kOffK), 16, 1024), qdesc = sdesc_sw128(smem_u32(smem + kOffQ), 16, 1024);
      uint32_t slot = 0, phase = 0;
      for (; live && shares.next(it); ++c_all) {
        const uint32_t n = (uint32_t)(min(rows - it.c * kChunk, kChunk) + 31) & ~31u;
        const uint32_t id_f16 = idesc_f16_f32(kChunk, n, false, false), id_bf16 = idesc_bf16_f32(kChunk, n, false, false);
        for (int i = it.i0; i < it.i1 && live; ++i, ++u) {
          const int buf = u & 1;
          const uint32_t d = tbase + buf * kChunk;
          const bool first = i == it.i0, last = i == it.i1 - 1;
          if (!wait.warp(&bars.sfree[buf], ((u >> 1) & 1) ^ 1, W_SFREE, kCtas == 2)) { live = false; break; }
#pragma unroll 1
          for (int k = 0; k < kBoxes; ++k) {
            if (first && !wait.warp(&bars.qfull[k], c_all & 1, W_QFULL, kCtas == 2)) { live = false; break; }
            if (!wait.warp(&bars.kfull[slot], phase, W_KFULL, kCtas == 2)) { live = false; break; }
            tc_fence_after();
            if constexpr (kFmt == kCacheBf16) fence_proxy_async_smem();    // copies that other threads issued
            if (elect_one()) {
              const bool bf = kFmt == kCacheBf16 || (kFmt == kCacheFp4 && k == kBoxes - 1);
              mma_box64<kCtas>(d, kdesc + slot * (kBoxBytes / 16), qdesc + k * (kBoxBytes / 16), bf ? id_bf16 : id_f16, k > 0 ? 1u : 0u);
              commit<kCtas>(&bars.kempty[slot]);
              if (last) commit<kCtas>(&bars.qempty[k]);
              if (k == kBoxes - 1) commit<kCtas>(&bars.sfull[buf]);
            }
            __syncwarp();
            if (++slot == kStages) slot = 0, phase ^= 1;
          }
        }
      }
      if (elect_one()) commit<kCtas>(&bars.drain);    // what was issued is done before tensor memory is given back
      mbar_drain(&bars.drain, 0);
      __syncwarp();
    } else if constexpr (kFmt == kCacheBf16) {
      uint32_t slot = 0, phase = 0;
      for (; live && shares.next(it); ++c_all)
        for (int i = it.i0; i < it.i1 && live; ++i)
          for (int k = 0; k < kBoxes; ++k) {
            if (i == it.i0) {
              if (!wait.warp(&bars.qfull[k], c_all & 1, W_QFULL)) { live = false; break; }
              fence_proxy_async_smem();
              first_cta_arrive<true>(&bars.qfull[k], cta);
            }
            if (!wait.warp(&bars.kfull[slot], phase, W_KFULL)) { live = false; break; }
            fence_proxy_async_smem();
            first_cta_arrive<true>(&bars.kfull[slot], cta);
            if (++slot == kStages) slot = 0, phase ^= 1;
          }
    }
  } else if (warp == 5) {
    // ---------------- rows of the tiles to come ----------------
    for (; live && shares.next(it); ++c_all) {
      const uint32_t lslot = c_all % kLseSlots;
      float l[kChunk / 32];
#pragma unroll
      for (int i = 0; i < kChunk / 32; ++i) {
        const int r = it.c * kChunk + 32 * i + lane;
        const float* src = p.lse + (int64_t)it.b * rows + r;
        l[i] = -CUDART_INF_F;
        if (r < rows && guard_span(p.err, G_STEP_IN, src, 4, p.lse, (uint64_t)p.kv.B * rows * 4)) l[i] = *src;
      }
      for (int i = it.i0; i < it.i1; ++i, ++u) {
        const int slot = u % kRowSlots;
        int32_t at[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = ((it.t0 + i) * kCtas + cta) * kTile + 32 * r + lane;
          at[r] = kNoRow;
          if (j < it.len) {
            const int pg = j / p.kv.page_size;
            const int page = guarded_int(p.err, p.kv.block_table, (int64_t)it.b * p.kv.max_pages + pg, (int64_t)p.kv.B * p.kv.max_pages);
            if (page >= 0 && page < p.kv.num_pages) at[r] = page * p.kv.page_size + (j - pg * p.kv.page_size);
            else record_error(p.err, DEV_RANGE_BASE | Y_PAGE);
          }
        }
        // the lines of narrow rows asked for in L2, by the first chunk that meets them (32 requests of 4096 to 32768 e4m3 rows
        // 0.134 -> 0.111 ms, 4-bit ones 0.147 -> 0.128; bf16 rows, which the copies ask for in time, 0.22 -> 0.37)
        if (kFmt != kCacheBf16 && it.c == 0) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (at[r] >= 0) {
              const uint8_t* row = p.kv.cache + (int64_t)at[r] * p.kv.row_bytes;
              for (int o = 0; o < p.kv.row_bytes; o += 128) prefetch_l2(row + o);
              prefetch_l2(row + p.kv.row_bytes - 1);
            }
        }
        if (!wait.warp(&bars.rfree[slot], ((u / kRowSlots) & 1) ^ 1, W_RFREE)) { live = false; break; }
#pragma unroll
        for (int r = 0; r < 4; ++r) row_slots[slot * kTile + 32 * r + lane] = at[r];
        warp_arrive(&bars.rfull[slot]);
        // the rows of two tiles go ahead of the log-sum-exps, whose place may be in use still
        if (i == min(it.i0 + 1, it.i1 - 1)) {
          if (!wait.warp(&bars.lfree[lslot], ((c_all / kLseSlots) & 1) ^ 1, W_LFREE)) { live = false; break; }
          bool none = false;
#pragma unroll
          for (int i = 0; i < kChunk / 32; ++i) {
            const float minus = l[i] == -CUDART_INF_F ? -CUDART_INF_F : -l[i] * 1.4426950408889634f;
            lse_slots[lslot * kChunk + 32 * i + lane] = minus;
            none |= minus == -CUDART_INF_F && it.c * kChunk + 32 * i + lane < rows;
          }
          none = __any_sync(~0u, none);
          if (lane == 0) bars.skips[lslot] = none;
          warp_arrive(&bars.lfull[lslot]);
        }
      }
    }
  } else {
    // ---------------- producers ----------------
    const uint32_t me = (warp - kFirstProducer) % kStages;
    const int r0 = (warp - kFirstProducer) / kStages * 64;     // this warp's rows of a box
    uint64_t* const kempty = &bars.kempty[me];
    uint64_t* const kfull = &bars.kfull[me];
    const uint32_t kslot = smem_u32(smem + kOffK + me * kBoxBytes);
    uint32_t made = 0;                            // boxes of this stage so far
    // a box whose loads are out: 4-bit rows two lanes a row, 32 columns each; e4m3 four lanes a row, 16 columns each
    constexpr int kVec = kFmt == kCacheFp4 ? 4 : 8;
    uint4 v[2][kVec];
    uint32_t sc[2][4];
    int held = -1;                                // which of the two holds a box
    auto convert = [&](const uint4 (&ready)[kVec], const uint32_t (&ready_sc)[4]) -> bool {
      held = -1;
      if (!wait.warp(kempty, (made & 1) ^ 1, W_KEMPTY)) return false;
      ++made;
      if constexpr (kFmt == kCacheFp4) {
        const int half = lane & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + 16 * i + (lane >> 1);
          const uint2 s = fp4_scales2(ready_sc[i]);
          st_shared16(box_unit(kslot, r, 4 * half), fp4x8_to_f16(ready[i].x, s.x));
          st_shared16(box_unit(kslot, r, 4 * half + 1), fp4x8_to_f16(ready[i].y, s.x));
          st_shared16(box_unit(kslot, r, 4 * half + 2), fp4x8_to_f16(ready[i].z, s.y));
          st_shared16(box_unit(kslot, r, 4 * half + 3), fp4x8_to_f16(ready[i].w, s.y));
        }
      } else {
        const int quarter = lane & 3;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int r = r0 + 8 * i + (lane >> 2);
          st_shared16(box_unit(kslot, r, 2 * quarter), e4m3x8_to_f16(ready[i].x, ready[i].y));
          st_shared16(box_unit(kslot, r, 2 * quarter + 1), e4m3x8_to_f16(ready[i].z, ready[i].w));
        }
      }
      fence_proxy_async_smem();
      tell(kfull);
      return true;
    };
    // (two copies of the code: a register that a load is on its way to is not moved without waiting for it)
    auto flush = [&]() -> bool { return held < 0 || (held == 0 ? convert(v[0], sc[0]) : convert(v[1], sc[1])); };
    int k0 = me;                                   // this stage's first box of the unit
    for (; live && shares.next(it); ++c_all) {
      const int n = min(rows - it.c * kChunk, kChunk), own = ((n + 31) & ~31) / kCtas;    // this CTA's query rows
      const __nv_bfloat16* qsrc = p.q + ((int64_t)it.b * rows + it.c * kChunk + cta * own) * kDk;
      const uint64_t q_bytes = (uint64_t)p.kv.B * rows * kDk * 2;
      const int unit = lane & 7;
      // the query rows' boxes me and me + 5, in the first unit each before the keys' box of its column
      int kq = me;
      auto query_box = [&](int k) -> bool {
        const uint32_t box = smem_u32(smem + kOffQ + k * kBoxBytes);
        if (!flush() || !wait.warp(&bars.qempty[k], (c_all & 1) ^ 1, W_QEMPTY)) return false;
        for (int r = r0 + (lane >> 3); r < min(own, r0 + 64); r += 4) {
          const __nv_bfloat16* src = qsrc + (int64_t)r * kDk + 64 * k + 8 * unit;
          const bool in = cta * own + r < n && guard_span(p.err, G_STEP_IN, src, 16, p.q, q_bytes);
          cp_async16_zfill(box_unit(box, r, unit), in ? src : p.q, in ? 16u : 0u);
        }
        if constexpr (kFmt == kCacheBf16) {
          cp_async_arrive_noinc(&bars.qfull[k]);
        } else {                                   // each lane puts its own copies into f16 where they lie
          cp_async_wait_all();
          if (kFmt == kCacheE4m3 || k < kBoxes - 1)
            for (int r = r0 + (lane >> 3); r < min(own, r0 + 64); r += 4) {
              const uint32_t at = box_unit(box, r, unit);
              st_shared16(at, bf16x8_to_f16(ld_shared16(at)));
            }
          fence_proxy_async_smem();
          tell(&bars.qfull[k]);
        }
        return true;
      };
      for (int t = it.i0; t < it.i1 && live; ++t, ++u) {
        const int rslot = u % kRowSlots;
        if (!wait.warp(&bars.rfull[rslot], (u / kRowSlots) & 1, W_RFULL)) { live = false; break; }
        const int32_t* at = row_slots + rslot * kTile + r0;
        int k = k0;
        for (; k < kBoxes; k += kStages) {
          for (; kq <= k && live; kq += kStages) live = query_box(kq);
          if (!live) break;
          if (kFmt == kCacheBf16 || (kFmt == kCacheFp4 && k == kBoxes - 1)) {
            int32_t a[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) a[i] = at[(lane >> 3) + 4 * i];
            if (!flush() || !wait.warp(kempty, (made & 1) ^ 1, W_KEMPTY)) { live = false; break; }
            ++made;
            const uint32_t off = (kFmt == kCacheBf16 ? 128 * k : kFp4Pe) + 16 * unit;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint8_t* src = p.kv.cache + (int64_t)a[i] * p.kv.row_bytes + off;
              const bool in = a[i] >= 0 && guard_span(p.err, G_STEP_IN, src, 16, p.kv.cache, cache_bytes);
              // (a row of zeros where there is none)
              cp_async16_zfill256(box_unit(kslot, r0 + (lane >> 3) + 4 * i, unit), in ? src : (const uint8_t*)p.q, in ? 16u : 0u);
            }
            if constexpr (kFmt == kCacheBf16) {
              cp_async_arrive_noinc(kfull);
            } else {
              cp_async_wait_all();
              fence_proxy_async_smem();
              tell(kfull);
            }
            continue;
          }
          auto load = [&](uint4 (&x)[kVec], uint32_t (&xs)[4]) {
            if constexpr (kFmt == kCacheFp4) {
              const int half = lane & 1;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int a = at[16 * i + (lane >> 1)];
                const uint8_t* r = p.kv.cache + (int64_t)a * kFp4Row;
                x[i] = make_uint4(0, 0, 0, 0), xs[i] = 0;
                if (a >= 0 && guard_span(p.err, G_STEP_IN, r, kFp4Row, p.kv.cache, cache_bytes)) {
                  x[i] = *reinterpret_cast<const uint4*>(r + 32 * k + 16 * half);
                  xs[i] = *reinterpret_cast<const uint16_t*>(r + kFp4Codes + 4 * k + 2 * half);
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < kVec; ++i) {
                const int a = at[8 * i + (lane >> 2)];
                const uint8_t* src = p.kv.cache + (int64_t)a * kDk + 64 * k + 16 * (lane & 3);
                x[i] = a >= 0 && guard_span(p.err, G_STEP_IN, src, 16, p.kv.cache, cache_bytes) ? *reinterpret_cast<const uint4*>(src)
                                                                                               : make_uint4(0, 0, 0, 0);
              }
            }
          };
          if constexpr (kFmt != kCacheBf16) {
            const int into = held == 0 ? 1 : 0;
            if (into == 0) load(v[0], sc[0]);
            else load(v[1], sc[1]);
            if (!flush()) { live = false; break; }
            held = into;
          }
        }
        for (; kq < kBoxes && live; kq += kStages) live = query_box(kq);
        k0 = k - kBoxes;                           // the ring goes on with the next unit's first box
        if (live) warp_arrive(&bars.rfree[rslot]);
      }
    }
    if (live) flush();
    cp_async_wait_all();                         // no copy into this CTA outlives it
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kCtas == 1) {
    if (warp == 4) tmem_dealloc(tbase, kTmemCols);
  } else {
    if (warp == 4) mbar_drain(&bars.drain, 0);   // the last arrival in either CTA
    __syncwarp();
    cluster_sync();                              // no MMA of the pair is left, no arrival on its way
    if (warp == 4) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "n"(kTmemCols) : "memory");
  }
}

// Several chunks of query rows: a range's sums are those of the CTAs that had units of it, in their order.  A CTA per tile.
template <int kCtas>
__global__ void __launch_bounds__(kTile * kCtas) key_weights_sum_kernel(const __grid_constant__ KeyWeightsParams p, int shares, int per_request) {
  const int64_t table = (int64_t)p.kv.max_pages * p.kv.page_size, cap = table < p.width ? table : p.width;
  constexpr int kChunk = kTile * kCtas;
  const int chunks = (p.s * p.H + kChunk - 1) / kChunk;
  const int at = blockIdx.x / kSub, i = blockIdx.x - at * kSub, b = at / per_request, r = at - b * per_request;
  const int len = paged_len(p.kv, p.err, b, cap, false), t0 = r * kSub, nt = min(tiles_of<kCtas>(len) - t0, kSub);
  if (i >= nt) return;
  const int64_t total = (int64_t)p.before[2 * p.kv.B] * chunks, u0 = ((int64_t)p.before[2 * b] + t0) * chunks, range = p.before[2 * b + 1] + r;
  const int j = (t0 + i) * kChunk + threadIdx.x;
  if (j >= len) return;
  float sum = 0.f;
  int s = (int)(((u0 + 1) * shares - 1) / total);         // the share that has unit u0
  int64_t lo, hi = total * s / shares - u0;
  for (; s < shares; ++s) {
    lo = hi, hi = total * (s + 1) / shares - u0;
    if (lo >= (int64_t)nt * chunks) break;
    const int64_t c = lo <= i ? 0 : (lo - i + nt - 1) / nt;  // its first chunk of this tile
    if (c >= chunks || c * nt + i >= hi) continue;
    const float* part = p.part + ((range + s) * kSub + i) * kChunk + threadIdx.x;
    if (guard_span(p.err, G_PART_O, part, 4, p.part, p.part_bytes)) sum += *part;
  }
  float* w = p.weights + b * p.stride + j;
  if (guard_span(p.err, G_STEP_OUT, w, 4, p.weights, ((uint64_t)(p.kv.B - 1) * p.stride + p.width) * 4))
    *w = p.decay == 0.f ? sum : fmaf(p.decay, *w, sum);
}

}  // namespace

// the most ranges of kSub tiles that requests of `width` keys have
static int64_t most_ranges(int B, int64_t width, int ctas) {
  const int64_t keys = (int64_t)kSub * kTile * ctas;
  return B * ((width + keys - 1) / keys);
}

size_t key_weights_scratch(int B, int64_t rows, int64_t width, size_t* before) {
  *before = 0;
  if (rows <= kTile || B <= 0 || width <= 0) return 0;
  *before = ((size_t)2 * B + 2) * sizeof(int32_t);
  const int sms = device_sm_count();             // of CTAs alone and of pairs
  const size_t one = (size_t)(most_ranges(B, width, 1) + sms), two = 2 * (size_t)(most_ranges(B, width, 2) + sms / 2);
  return (one > two ? one : two) * kSub * kTile * sizeof(float);
}

namespace {
template <int kFmt, int kCtas>
cudaError_t launch(const KeyWeightsParams& p, int64_t cap, cudaStream_t stream) {
  static PerDeviceOnce attrs;
  const void* fn = (const void*)key_weights_kernel<kFmt, kCtas>;
  cudaError_t e = attrs.run([fn] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (e != cudaSuccess) return e;
  // no more shares than tiles there can be, once for each chunk (1280 query rows over 464 4-bit keys: 41 us
  // with two shares, 23 with ten)
  const int64_t chunks = ((int64_t)p.s * p.H + kTile * kCtas - 1) / (kTile * kCtas);
  const int64_t most = p.kv.B * ((cap + kTile * kCtas - 1) / (kTile * kCtas)) * chunks, room = device_sm_count() / kCtas;
  const int shares = (int)(most < room ? most : room);
  cudaLaunchConfig_t config{};
  config.gridDim = dim3((unsigned)(shares * kCtas));
  config.blockDim = dim3(kThreads);
  config.dynamicSmemBytes = kSmem;
  config.stream = stream;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = kCtas, cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  config.attrs = &cluster;
  config.numAttrs = 1;
  e = cudaLaunchKernelEx(&config, key_weights_kernel<kFmt, kCtas>, p);
  if (e != cudaSuccess || (int64_t)p.s * p.H <= kTile * kCtas) return e;
  const int64_t ranges = most_ranges(p.kv.B, cap, kCtas);
  key_weights_sum_kernel<kCtas><<<(unsigned)(ranges * kSub), kTile * kCtas, 0, stream>>>(p, shares, (int)(ranges / p.kv.B));
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream) {
  const int64_t table = (int64_t)p.kv.max_pages * p.kv.page_size, cap = table < p.width ? table : p.width;
  if (p.kv.B == 0 || cap == 0) return cudaSuccess;
    // (of up to 128 query rows a pair gains 2 % over 4-bit rows and loses 1 % over e4m3 ones)
  const bool pair = (int64_t)p.s * p.H > kTile && device_sm_count() > 1;
  if (p.format == kCacheBf16) return pair ? launch<kCacheBf16, 2>(p, cap, stream) : launch<kCacheBf16, 1>(p, cap, stream);
  if (p.format == kCacheE4m3) return pair ? launch<kCacheE4m3, 2>(p, cap, stream) : launch<kCacheE4m3, 1>(p, cap, stream);
  return pair ? launch<kCacheFp4, 2>(p, cap, stream) : launch<kCacheFp4, 1>(p, cap, stream);
}

}  // namespace mla
