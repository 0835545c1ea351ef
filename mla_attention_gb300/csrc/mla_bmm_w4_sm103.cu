// Products of a few rows with 4-bit weights and group scales, per head:
//   out[t, h, n] = sum_g scale[h, n, g] sum_{k in g} x[t, h, k] (code[h, n, k] - 8)
//
// Bound by reading the weights (half a byte each) while the tokens are few, and next to that by the
// instructions that take a word of eight codes apart.  The weights are the M operand of m16n8k16
// products (16 columns n of the output x 16 k), the tokens the N operand, eight at a time, with fp32 sums;
// the scale multiplies a group's sum where it lies, in the thread's accumulators.
//
// A code c in the low bits of a bf16 word is the subnormal number c 2^-133, and one four bits higher
// is 16 c 2^-133.  So w & 0x000f000f, w & 0x00f000f0 and the same of w >> 8 hold the codes of (k0, k4),
// (k1, k5), (k2, k6), (k3, k7) of a word, and one exact fma a pair, times 2^127 or 2^123 and less 2^-3, makes them the
// weights (c - 8) 2^-6: nine instructions for eight weights.  x is put in the same order of k as it is, and
// the scale brings 2^6 back.  The weights have their sign before they meet x: a sum of c x less 8 sum x would
// be five instructions, but it rounds at the size of 8 x also where the weight is 0, so that one large x under a
// code of 8 takes the other terms with it.
// A sum that is not finite is done over in plain fp32, scale by scale, by the thread that stores it.
//
// A CTA's eight warps hold 16 columns each of one head and walk the CTA's slice of k together, 128
// k a step.  Every warp brings its own weights through a ring of kStages cp.async stages (no barrier for
// them): 1 KB per 16 columns and step, the 16-byte pieces of a row swizzled by its number so that the
// word reads hit 32 banks; lane (g, t) holds columns g and g + 8 and takes word t of each 32 k, so that
// the four words of a product lie in one group whatever the group's size.  Four more warps put the tokens'
// k (in the order in which a lane reads them) and the weights' scales down in shared
// memory, a chunk of kChunk steps ahead of the others: the same work between the products kept
// every warp waiting for loads and for the slowest.
// Few columns with a long k are cut over a cluster's CTAs, whose sums are joined in shared memory in
// a fixed order.
// 8192 columns, k of 16384, groups of 128, 4 tokens: 19.6 us, 52 % of the copy's bandwidth, at half of the
// issue slots.  128 heads of 512 columns, k of 128, one token 5.3 us, of 128 columns, k of 512, 17 tokens
// 5.8 (inputs from HBM): a launch, the first chunk's way in and the sums' way out.  Instructions are kept few as well: each is
// fetched once a launch (the helpers' loads in three places instead of one cost 0.2 us).  Two times side by side below are
// of two forms of one build, some of them before the weights had their sign.
#include <algorithm>
#include <type_traits>

#include "mla_step.h"
#include "row_vec.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8, kHelpers = 4, kThreads = 32 * (kWarps + kHelpers);
constexpr int kStages = 4;
constexpr int kStep = 128;          // k per step
constexpr int kCols = 16;           // columns n of a warp
constexpr int kTileBytes = kCols * kStep / 2;
constexpr int kPitch = kCols + 4;   // a token's sums: 16-byte reads, and the writes of a warp hit 32 banks
constexpr uint32_t kCode = 0x7f007f00u, kCode4 = 0x7d007d00u;   // bf16 2^127 and 2^123, twice: a code and one four bits higher to c 2^-6
constexpr uint32_t kEight = 0xbe00be00u;                        // -8 2^-6, twice
constexpr float kWeight = 64.f;                                 // what the scales take back

enum : uint32_t { W_CHUNK_FULL = 0x90, W_CHUNK_FREE };

template <int NT>
constexpr int kChunk = NT == 1 ? 4 : 2;   // steps of x put in place at a time

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// 16 bytes at constant offsets, where `at` is below `end`
template <int kDst, int kSrc>
__device__ __forceinline__ void cp_async16_below(uint32_t dst, const void* src, int at, int end) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %2, %3;\n\t"
      "@p cp.async.cg.shared.global [%0 + %4], [%1 + %5], 16;\n\t}" ::"r"(dst), "l"(src), "r"(at), "r"(end), "n"(kDst), "n"(kSrc)
      : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// (volatile: made where they are used, the weights keep fewer registers: 9 tokens of 128 heads, k of 128, groups of 32 5.8 -> 5.5 us)
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm volatile("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float scale_at(const BmmW4Params& p, const uint8_t* s) {
  const int bytes = p.scales_f32 ? 4 : 2;
  if (!guard_span(p.err, G_STEP_IN, s, bytes, p.scales, (uint64_t)p.H * p.N * (p.K / p.group) * bytes)) return 0.f;
  return p.scales_f32 ? *reinterpret_cast<const float*>(s) : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(s));
}

// One value in plain fp32: where a partial sum left fp32's range (its scale may bring it back).
__device__ __noinline__ float plain_value(const BmmW4Params& p, int tok, int h, int n) {
  const int64_t row = (int64_t)h * p.N + n;
  const uint8_t* w = p.w4 + row * (p.K / 2);
  const __nv_bfloat16* x = p.x + tok * p.x_stride_t + h * p.x_stride_h;
  const int groups = p.K / p.group;
  if (!guard_span(p.err, G_STEP_IN, w, p.K / 2, p.w4, (uint64_t)p.H * p.N * (p.K / 2)) ||
      !guard_span(p.err, G_STEP_IN, x, p.K * 2, p.x, ((uint64_t)(p.T - 1) * p.x_stride_t + (uint64_t)(p.H - 1) * p.x_stride_h + p.K) * 2))
    return 0.f;
  float v = 0.f;
  for (int q = 0; q < groups && v == v; ++q) {   // a NaN stays one
    const float s = scale_at(p, reinterpret_cast<const uint8_t*>(p.scales) + (row * groups + q) * (p.scales_f32 ? 4 : 2));
    for (int k = q * p.group; k < (q + 1) * p.group; ++k)
      v += __bfloat162float(x[k]) * ((float)((w[k / 2] >> (4 * (k & 1)) & 15) - 8) * s);
  }
  return v;
}

// kVec scales: fp32 to a word each, bf16 two to a word (the first kVec / 2 words)
template <int kVec>
__device__ __forceinline__ void load_scales(uint32_t* w, const uint8_t* f, bool f32) {
  if constexpr (kVec == 4) {
    if (f32) {
      const uint4 v = *reinterpret_cast<const uint4*>(f);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(f);
      w[0] = v.x, w[1] = v.y;
    }
  } else if constexpr (kVec == 2) {
    if (f32) {
      const uint2 v = *reinterpret_cast<const uint2*>(f);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(f);
    }
  }
}

// GL: 2^GL pieces of 32 k are a group
template <int NT, int GL>
struct W4Smem {
  uint8_t w[kWarps][kStages][kTileBytes];
  uint4 x[2 * kChunk<NT>][4][NT][32];         // [step][32 k][8 tokens][lane], two chunks
  float scale[2 * kChunk<NT>][4 >> GL][kWarps][8][2];   // times kWeight, of columns (g, g + 8)
  float sums[kWarps][8 * NT][kPitch];         // of a warp's columns, [token][column]
  uint64_t full[2], free[2];                  // a chunk's x and scales are in place / read
};

// NT: tokens by the eight.  (Two CTAs an SM up to 16 tokens.)
template <int NT, int GL>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1) bmm_w4_kernel(const __grid_constant__ BmmW4Params p, const W4Plan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kTok = 8 * NT, KC = kChunk<NT>;
  W4Smem<NT, GL>& s = *reinterpret_cast<W4Smem<NT, GL>*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int rank = plan.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int wide = plan.rounds * kWarps * kCols, blocks_h = plan.blocks_h;   // columns of a CTA, CTAs of a head
  const int block = plan.cluster > 1 ? blockIdx.x / plan.cluster : blockIdx.x;
  const int h = block / blocks_h, first = (block - h * blocks_h) * wide;
  const int rounds = min(plan.rounds, (p.N - 1 - first) / (kWarps * kCols) + 1);
  const int tok0 = blockIdx.y * kTok;
  const int steps = (p.K + kStep - 1) / kStep;
  const int u0 = plan.cluster > 1 ? (int)((int64_t)steps * rank / plan.cluster) : 0;
  const int u1 = plan.cluster > 1 ? (int)((int64_t)steps * (rank + 1) / plan.cluster) : steps;
  const int row_bytes = p.K / 2, groups = (p.K / 32) >> GL, scale_bytes = p.scales_f32 ? 4 : 2;
  constexpr int kPer = 4 >> GL, kLast = (1 << GL) - 1;   // groups of a step; piece i ends one where (i & kLast) == kLast

  const int count = u1 - u0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.full[i], kHelpers);
      mbar_init(&s.free[i], kWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  // Warp-uniform and bounded.  The status word is written where a wait runs out, but not heeded: another
  // call's report in the same workspace is no reason to stop.
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    const bool there = __all_sync(~0u, mbar_wait(bar, parity, nullptr, site, p.spin_limit)) != 0;
    if (!there && lane == 0) record_error(p.err, DEV_TIMEOUT_BASE | site);
    return there;
  };

  if (warp >= kWarps) {
    // ---- the helpers put a chunk's x and scales in place while the others compute on the one before ----
    const int helper = warp - kWarps;
    constexpr int kUnits = (KC * NT + kHelpers - 1) / kHelpers;     // (step, eight tokens) of a helper
    constexpr int kRow = KC * kPer, kScales = kCols * kRow / 32;    // a lane has kScales neighbours of one column
    constexpr int kTiles = kWarps / kHelpers;                       // warps whose scales a helper brings
    // Scales come one by one, or kVec in a load (8192 columns, k of 16384: groups of 32 28.4 -> 24.8 us, of 128 20.1 ->
    // 19.4; groups of 64 would spill: 128 heads, k of 128, 8 tokens 5.8 -> 6.4).
    constexpr int kVec = NT > 1 || GL == 1 ? 1 : GL == 0 ? 4 : 2;
    const bool vec_s = kVec > 1 && plan.vec_s && groups % kVec == 0 && u0 * kPer % kVec == 0, pairs = vec_s && !p.scales_f32;
    const uint64_t ext_x = ((uint64_t)(p.T - 1) * p.x_stride_t + (uint64_t)(p.H - 1) * p.x_stride_h + p.K) * 2;
    const uint64_t ext_s = (uint64_t)p.H * p.N * groups * scale_bytes;
    const __nv_bfloat16* xh = p.x + h * p.x_stride_h + tok0 * p.x_stride_t + 8 * t;   // lane (g, t): token g, k 8t ..
    const int col = lane % kCols, q0 = lane / kCols * kScales, to_f32 = p.scales_f32 ? 0 : 16;
    const uint8_t* scale[kTiles];
    auto to_round = [&](int r) {
#pragma unroll
      for (int w = 0; w < kTiles; ++w)
        scale[w] = reinterpret_cast<const uint8_t*>(p.scales) +
                   (((int64_t)h * p.N + min(first + (r * kWarps + helper + w * kHelpers) * kCols + col, p.N - 1)) * groups + u0 * kPer + q0) *
                       scale_bytes;
    };
    uint4 xv[kUnits][4];
    uint32_t sv[kTiles][kScales] = {};
    auto load_x = [&](int chunk) {   // past T and past K: zeros
#pragma unroll
      for (int n = 0; n < kUnits; ++n) {
        const int unit = helper + n * kHelpers, st = unit / NT, tok = tok0 + unit % NT * 8 + g;
        const __nv_bfloat16* from = xh + (int64_t)(unit % NT * 8 + g) * p.x_stride_t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = (u0 + chunk * KC + st) * kStep + 32 * i;
          xv[n][i] = make_uint4(0, 0, 0, 0);
          if (unit < KC * NT && chunk * KC + st < count && tok < p.T && k < p.K && guard_span(p.err, G_STEP_IN, from + k, 16, p.x, ext_x))
            xv[n][i] = plan.vec_x ? *reinterpret_cast<const uint4*>(from + k) : load_row8_narrow(from + k, 8);
        }
      }
    };
    auto load_s = [&](int chunk) {   // past K: what was there before, for weights that are not
      if constexpr (kVec > 1)
        if (vec_s) {
          if (chunk * KC < count)
#pragma unroll
            for (int w = 0; w < kTiles; ++w)
#pragma unroll
              for (int r = 0; r < kScales; r += kVec) {
                const int q = chunk * kRow + r;
                const uint8_t* f = scale[w] + q * scale_bytes;
                if (u0 * kPer + q0 + q < groups && guard_span(p.err, G_STEP_IN, f, kVec * scale_bytes, p.scales, ext_s))
                  load_scales<kVec>(&sv[w][r], f, p.scales_f32);
              }
          return;
        }
#pragma unroll
      for (int w = 0; w < kTiles; ++w)
#pragma unroll
        for (int r = 0; r < kScales; ++r) {
          const int q = chunk * kRow + r;
          const uint8_t* f = scale[w] + q * scale_bytes;
          if (u0 * kPer + q0 + q < groups && chunk * KC < count && guard_span(p.err, G_STEP_IN, f, scale_bytes, p.scales, ext_s)) {
            if (p.scales_f32) sv[w][r] = *reinterpret_cast<const uint32_t*>(f);
            else sv[w][r] = *reinterpret_cast<const uint16_t*>(f);
          }
        }
    };
    auto place_x = [&](int b) {
#pragma unroll
      for (int n = 0; n < kUnits; ++n) {
        const int unit = helper + n * kHelpers, st = unit / NT, nt = unit % NT;
        if (unit >= KC * NT) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = xv[n][i];
          s.x[b * KC + st][i][nt][lane] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                                     __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
      }
    };
    auto place_s = [&](int b) {
#pragma unroll
      for (int w = 0; w < kTiles; ++w)
#pragma unroll
        for (int r = 0; r < kScales; ++r) {
          uint32_t v = sv[w][r] << to_f32;
          if (kVec > 1 && pairs) {   // two to a word, in the first words of a load's
            v = sv[w][r / kVec * kVec + r % kVec / 2];
            v = r & 1 ? v & 0xffff0000u : v << 16;
          }
          s.scale[b * KC + (q0 + r) / kPer][(q0 + r) % kPer][helper + w * kHelpers][col & 7][col >> 3] = __uint_as_float(v) * kWeight;
        }
    };
    // one place in the code for each: a launch waits for its instructions
    for (int r = 0, chunk = 0, turn = 0;; ++turn) {
      if (turn > 0) {
        const int b = chunk & 1, use = r + (chunk >> 1);   // of the chunk's buffer
        if (use > 0 && !wait(&s.free[b], (use - 1) & 1, W_CHUNK_FREE)) break;
        if (r == 0) place_x(b);
        place_s(b);
        warp_arrive(&s.full[b]);
        if (++chunk * KC >= count) {
          chunk = 0;
          if (++r == rounds) break;
        }
      }
      if (chunk == 0) to_round(r);
      if (r == 0) load_x(chunk);
      load_s(chunk);
    }
    if (plan.cluster > 1) {
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // ---- weights: this lane copies piece t of a step of columns g and g + 8 of each 16 (columns past N: any
  // column of the head, nothing of theirs is stored) ----
  const uint8_t* src[2];
  int n0 = 0;
  auto to_round = [&](int r) {
    n0 = first + (r * kWarps + warp) * kCols;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      src[e] = p.w4 + ((int64_t)h * p.N + min(n0 + 8 * e + g, p.N - 1)) * row_bytes + u0 * (kStep / 2) + 16 * t;
  };
  const int swz = (g >> 1) & 3;
  const uint32_t put = smem_u32(s.w[warp]) + g * 64 + ((t ^ swz) << 4);
  const int left = min(row_bytes, u1 * (kStep / 2)) - u0 * (kStep / 2) - 16 * t;   // > 64 s: step u0 + s has this piece
  // step u0 + base + kAt into stage kAt % kStages; src stands at step u0 + base
  // Past K and past the slice nothing is copied: whatever lies there is codes too, and x is 0 for them.
  auto fetch = [&](auto at, int base) {
    constexpr int kAt = decltype(at)::value, kTo = kAt % kStages * kTileBytes, kFrom = kAt * (kStep / 2);
    const int k = (base + kAt) * (kStep / 2);
    auto ok = [&](const uint8_t* a) {
      return !kGuarded || k >= left || guard_span(p.err, G_STEP_IN, a + kFrom, 16, p.w4, (uint64_t)p.H * p.N * row_bytes);
    };
    if (ok(src[0])) cp_async16_below<kTo, kFrom>(put, src[0], k, left);
    if (ok(src[1])) cp_async16_below<kTo + 512, kFrom>(put, src[1], k, left);
    cp_commit();
  };
  auto fetch_first = [&] {
    fetch(std::integral_constant<int, 0>{}, 0);
    fetch(std::integral_constant<int, 1>{}, 0);
    fetch(std::integral_constant<int, 2>{}, 0);
  };
  to_round(0);
  fetch_first();
  float acc[NT][4], part[NT][4];
  const uint8_t* take[4];   // word t of piece i of column g
#pragma unroll
  for (int i = 0; i < 4; ++i) take[i] = s.w[warp][0] + g * 64 + ((i ^ swz) << 4) + 4 * t;
  bool live = true;

  auto step = [&](auto at, int base, int r) {
    constexpr int kAt = decltype(at)::value;
    const int j = base + kAt;
    const int chunk = j / KC;
    if (kAt % KC == 0 && live) live = wait(&s.full[chunk & 1], (r + (chunk >> 1)) & 1, W_CHUNK_FULL);
    cp_wait<kStages - 2>();
    __syncwarp();          // every lane's copies of step j have landed, and step j - 1 is read
    fetch(std::integral_constant<int, kAt + kStages - 1>{}, base);
    const int slot = (base & (2 * KC - 1)) + kAt % (2 * KC);   // of the two chunks
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // 32 k each
      const uint32_t* from = reinterpret_cast<const uint32_t*>(take[i] + kAt * kTileBytes);
      const uint32_t w0 = from[0], w1 = from[128], v0 = w0 >> 8, v1 = w1 >> 8;
      const uint32_t lo[4] = {fma_bf16x2(w0 & 0x000f000fu, kCode, kEight), fma_bf16x2(w1 & 0x000f000fu, kCode, kEight),
                              fma_bf16x2(w0 & 0x00f000f0u, kCode4, kEight), fma_bf16x2(w1 & 0x00f000f0u, kCode4, kEight)};
      const uint32_t hi[4] = {fma_bf16x2(v0 & 0x000f000fu, kCode, kEight), fma_bf16x2(v1 & 0x000f000fu, kCode, kEight),
                              fma_bf16x2(v0 & 0x00f000f0u, kCode4, kEight), fma_bf16x2(v1 & 0x00f000f0u, kCode4, kEight)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 b = s.x[slot][i][nt][lane];
        if ((i & kLast) == 0) part[nt][0] = part[nt][1] = part[nt][2] = part[nt][3] = 0.f;   // a group's sums start
        mma16816(part[nt], lo, b.x, b.y);
        mma16816(part[nt], hi, b.z, b.w);
      }
      if ((i & kLast) == kLast) {   // the end of a group
        const float2 sc = *reinterpret_cast<const float2*>(s.scale[slot][i >> GL][warp][g]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][e] += (e < 2 ? sc.x : sc.y) * part[nt][e];
      }
    }
    if (kAt % KC == KC - 1) warp_arrive(&s.free[chunk & 1]);
  };
  const uint64_t ext_out = ((uint64_t)(p.T - 1) * p.out_stride_t + (uint64_t)(p.H - 1) * p.out_stride_h + p.N) * 2;
  const int tokens = min(kTok, p.T - tok0);
  // ---- a warp's sums in shared memory, out along n, dealt over the cluster's CTAs ----
  auto total = [&](int tok, int c) {
    if (plan.cluster == 1) return s.sums[warp][tok][c];
    float v = 0.f;
    for (int q = 0; q < plan.cluster; ++q) v += ld_cluster_f32(map_to_rank(smem_u32(&s.sums[warp][tok][c]), q));
    return v;
  };
  auto put_value = [&](int tok, int c, int at) {   // one value, of column `at`
    float v = total(tok, c);
    if (!(fabsf(v) < __int_as_float(0x7f800000))) v = plain_value(p, tok0 + tok, h, at);
    __nv_bfloat16* o = p.out + (tok0 + tok) * p.out_stride_t + h * p.out_stride_h + at;
    if (guard_span(p.err, G_STEP_OUT, o, 2, p.out, ext_out)) *o = __float2bfloat16_rn(v);
  };
  auto epilogue = [&](int at) {   // columns from `at` on
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) s.sums[warp][8 * nt + 2 * t + (j & 1)][8 * (j >> 1) + g] = acc[nt][j];
    if (plan.cluster > 1) cluster_sync();
    else __syncwarp();
    if (NT > 1 && plan.cluster == 1) {
      // Eight columns a lane.  Where a cluster deals the tokens out, single columns keep more lanes at its
      // loads (2746 columns, k of 4608, 20 tokens: 10.4 us, eight at a time 14.7).
      for (int i = lane; i < 2 * tokens; i += 32) {
        const int c = 8 * (i & 1), tok = i >> 1, n = at + c;
        if (n >= p.N) continue;
        float f[8];
        *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(&s.sums[warp][tok][c]);
        *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(&s.sums[warp][tok][c + 4]);
        bool plain = plan.vec_out && p.N - n >= 8;   // (n + 8 can pass 2^31 - 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) plain = plain && fabsf(f[j]) < __int_as_float(0x7f800000);
        __nv_bfloat16* o = p.out + (tok0 + tok) * p.out_stride_t + h * p.out_stride_h + n;
        if (plain) {
          if (guard_span(p.err, G_STEP_OUT, o, 16, p.out, ext_out)) *reinterpret_cast<uint4*>(o) = bf16x8_pack(f);
        } else {
#pragma unroll 1
          for (int j = 0; j < min(8, p.N - n); ++j) put_value(tok, c + j, n + j);
        }
      }
    } else {
      for (int i = rank * 32 + lane; i < tokens * kCols; i += plan.cluster * 32)
        if (at + i % kCols < p.N) put_value(i / kCols, i % kCols, at + i % kCols);
    }
    __syncwarp();
  };

  for (int r = 0; r < rounds; ++r) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[nt][j] = 0.f;
    for (int base = 0; base < count; base += kStages) {
      const int n = count - base;
      step(std::integral_constant<int, 0>{}, base, r);
      if (n > 1) step(std::integral_constant<int, 1>{}, base, r);
      if (n > 2) step(std::integral_constant<int, 2>{}, base, r);
      if (n > 3) step(std::integral_constant<int, 3>{}, base, r);
      src[0] += kStages * (kStep / 2), src[1] += kStages * (kStep / 2);
    }
    const int at = n0;
    if (r + 1 < rounds) {   // the next round's weights come while this one's sums go out
      __syncwarp();
      if (count % KC) warp_arrive(&s.free[count / KC & 1]);
      to_round(r + 1);
      fetch_first();
    }
    epilogue(at);
  }
  cp_wait<0>();
  if (plan.cluster > 1) cluster_sync();   // the others may still read this CTA's sums
}

// What one launch of a kernel has running at once.
struct AtOnce {
  int clusters[4];   // of 1, 2, 4 and 8 CTAs
};
template <int NT, int GL>
void configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& attr, int cluster, unsigned ctas, unsigned rows) {
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas, rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(W4Smem<NT, GL>);
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
}
template <int NT, int GL>
cudaError_t prepare(AtOnce& n) {
  const auto kernel = bmm_w4_kernel<NT, GL>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(W4Smem<NT, GL>));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n.clusters[0], kernel, kThreads, sizeof(W4Smem<NT, GL>));
  n.clusters[0] *= device_sm_count();
  for (int i = 1; i < 4 && e == cudaSuccess; ++i) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    configure<NT, GL>(cfg, attr, 1 << i, n.clusters[0] << i, 1);
    e = cudaOccupancyMaxActiveClusters(&n.clusters[i], kernel, &cfg);
  }
  return e;
}

template <int NT, int GL>
cudaError_t launch(const BmmW4Params& p, W4Plan plan, cudaStream_t stream) {
  static PerDeviceOnce once;
  static AtOnce cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = once.run([dev] { return prepare<NT, GL>(cached[dev]); });
  if (e != cudaSuccess) return e;
  const AtOnce& at_once = cached[dev];
  // k is cut over a cluster's CTAs, two ways at a time, while all of them still run at once (8192 columns, k of
  // 16384, 4 tokens, cut 1, 2, 4, 8 ways: 40, 24, 19.3, 24.5 us; 2102 columns, k of 6400: 8 ways 7.9 us, 2 ways 11.4).
  // How many do depends on how clusters fit a part of the GPU: 4 tokens, k of 4096, 36 clusters of eight 5.8 us, 37 9.1.
  const int steps = (p.K - 1) / kStep + 1, blocks_h = (p.N - 1) / (kWarps * kCols) + 1;
  const int64_t rows = (int64_t)p.H * ((p.T + 8 * NT - 1) / (8 * NT));
  int log2 = 0;
  while (log2 < 3 && 2 << log2 <= steps && rows * blocks_h <= at_once.clusters[log2 + 1]) ++log2;
  plan.cluster = 1 << log2;
  // Where two chunks hold all of k, a CTA keeps x and goes on to the next columns of its head, so that all CTAs
  // run at once (128 heads of 512 columns, k of 128, 1, 32, 64 tokens: 5.4, 16.7, 28.4 us with a CTA for every
  // 128 columns and single columns a lane, 4.6, 7.4, 11.4 so).
  plan.rounds = 1;
  if (plan.cluster == 1 && steps <= 2 * kChunk<NT>) {
    const int of_a_head = (int)std::min<int64_t>(blocks_h, std::max<int64_t>(1, at_once.clusters[0] / rows));
    plan.rounds = (blocks_h - 1) / of_a_head + 1;
  }
  plan.blocks_h = (blocks_h - 1) / plan.rounds + 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  configure<NT, GL>(cfg, attr, plan.cluster, (unsigned)p.H * plan.blocks_h * plan.cluster, (unsigned)((p.T + 8 * NT - 1) / (8 * NT)));
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, bmm_w4_kernel<NT, GL>, p, plan);
}
template <int NT>
cudaError_t launch(const BmmW4Params& p, const W4Plan& plan, cudaStream_t stream) {
  if (p.group == 32) return launch<NT, 0>(p, plan, stream);
  if (p.group == 64) return launch<NT, 1>(p, plan, stream);
  return launch<NT, 2>(p, plan, stream);
}

}  // namespace

cudaError_t launch_bmm_w4(const BmmW4Params& p, cudaStream_t stream) {
  W4Plan plan;
  plan.vec_x = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.x_stride_t % 8 == 0 && p.x_stride_h % 8 == 0;
  plan.vec_out = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.out_stride_t % 8 == 0 && p.out_stride_h % 8 == 0;
  plan.vec_s = reinterpret_cast<uintptr_t>(p.scales) % (p.scales_f32 ? 16 : 8) == 0;
  if (p.T <= 8) return launch<1>(p, plan, stream);
  if (p.T <= 16) return launch<2>(p, plan, stream);
  // (24 and 48 as well as 32 and 64: 17 tokens of 128 heads, k of 512, 5.5 -> 5.05 us, 48 with k of 128 12.9 -> 9.6)
  if (p.T <= 24) return launch<3>(p, plan, stream);
  if (p.T <= 32) return launch<4>(p, plan, stream);
  if (p.T <= 48) return launch<6>(p, plan, stream);
  return launch<8>(p, plan, stream);
}

}  // namespace mla
