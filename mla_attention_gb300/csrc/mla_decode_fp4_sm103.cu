// Decode over a 4-bit latent cache (sm_103a: tcgen05 on pairs of SMs, TMEM).
//   S = scale k . q,  P = softmax(S),  O = P V with V the key's latent columns; a sink is one more key with no value.
//
// A cluster of two CTAs works on 128 query rows (token, head) of one request, 64 in each CTA, and goes through the request's keys
// 128 at a time.  Both products are MMAs of the pair (cta_group::2, M = 128): each CTA holds the scores, P and O of its own
// rows - 128 lanes of tensor memory with half of the columns each - so that P never crosses to the other SM, O of 512
// columns takes half of a tensor memory and two buffers of scores fit beside it; and each CTA brings half of either B
// operand, so that a key's row is taken apart once for the scores and once for the values.  CTA c has the tile's keys
// 64 c .. 64 c + 63 for the scores and the latent columns 128 c .. and 256 + 128 c .. of all its keys for the values.
//
// A code times its scale has at most six bits and is exact in f16; q and P are f16 too (P a weight of at most 2^8, times 2^7), the RoPE
// columns stay bf16 as their MMA's operands, sums are fp32.  28 warps a CTA:
//   0-7    rows: lanes L and L + 64 of tensor memory hold the same row's scores of 64 keys each, 32 of them a warp; maximum
//          through shared memory, lazy rescale of O (by more than 2^8), exponentials, P
//   8, 9   MMAs, in the first CTA alone (one lane issues for both): scores; values, once all row warps have scaled O and stored P
//   10     the tiles' rows through the block table, up to three tiles ahead, and their lines asked for in L2
//   11     the RoPE columns
//   12-27  4-bit rows into f16, 16 keys and 256 columns each: of K and of V
// 64 requests of 4096 to 32768 keys with 128 heads: 0.344 ms, 0.96 PFLOP/s.  No pipe is full: of 5000 cycles a tile the tensor
// pipe has 2200 (37 % with 32 requests), the issue slots 38 %, the first-level cache's data pipe 65 %, DRAM 19 %, and without any one
// of the parts it takes some 5 % less; what is left is the chain rows, conversion, scores, exponentials, values of two tiles at a
// time.  A second set of row registers a converting warp: 0.362.  One request of 4097 keys: 25 us, of which 5.5 join the partials and 18
// are one chain of loads through the lengths, the table and the rows, the products and the partials' way out.
// The tiles of all requests are dealt to the pairs in equal shares; fp32 partials of a request that several pairs share
// are merged by decode_fp4_reduce_kernel.
#include <math_constants.h>

#include "fp4_rows.cuh"
#include "softmax_rows.cuh"
#include "tile_waits.cuh"

namespace mla {
namespace {

constexpr int kTile = 128, kHalf = 64;                // keys a tile, and the part that one CTA brings for the scores
constexpr int kThreads = 896, kMmaS = 8, kMmaV = 9, kTableWarp = 10, kFirstK = 12, kFirstV = 20;
constexpr int kBox = 64 * 128;                        // 64 rows of 128 bytes
constexpr int kRowSlots = 3;
constexpr uint32_t kTmemO = 0, kTmemS = 256;          // O: 256 columns; S: two buffers of 64
constexpr float kRescale = 8.f;                       // a weight passes 1 by 2^8 at most
constexpr float kLift = 7.f;                          // P and O are held times 2^7: P is below f16's 2^16, its last bit 2^-31 of the largest

constexpr int kOffQ = 0;                              // 9 boxes
constexpr int kOffK = 9 * kBox;                       // 9 boxes
constexpr int kOffV = 18 * kBox;                      // 2 halves of 4 boxes
constexpr int kOffP = 26 * kBox;                      // 2 boxes
constexpr int kOffRows = 28 * kBox;
constexpr int kOffMax = kOffRows + kRowSlots * kTile * 4;   // [3][64]
constexpr int kOffBars = kOffMax + 3 * 64 * 4;

struct Bars {
  // in the first CTA, with arrivals of both CTAs' warps
  uint64_t kfull[2], vfull[2], qfull, pfull, sfree[2], ofree;
  // in each CTA, by commits to both
  uint64_t kempty[2], vempty[2], qempty, sfull[2], pvdone;
  // in each CTA
  uint64_t rfull[kRowSlots], rfree[kRowSlots];
  uint64_t same[2];                                   // the four warps that hold the same rows
  uint64_t drain[2], stall;
  uint32_t tmem_base, abort;
  int64_t share;
  int32_t start_g, start_t;
};
constexpr int kSmem = kOffBars + 512;
static_assert(sizeof(Bars) <= 512, "barrier block too large");
static_assert(kSmem <= 232448, "shared memory over the sm_103a limit");

enum : uint32_t { D_KFULL = 0x1C0, D_VFULL, D_QFULL, D_PFULL, D_SFREE, D_OFREE, D_KEMPTY, D_VEMPTY, D_QEMPTY, D_SFULL, D_PVDONE, D_RFULL,
                  D_RFREE, D_PAIR, D_STALL, D_ALIGN };

// ---- query groups: up to 128 (token, head) rows of a request ----
struct Group {
  int b, row0, rows;       // request, first row among the request's s * H, rows
  int len;                 // keys of the request
  int keys;                // keys that its last token sees
};
__device__ __forceinline__ Group group_of(const DecodeFp4Params& p, int g, bool report) {
  Group r;
  r.b = p.row_tiles == 1 ? g : g / p.row_tiles;
  r.row0 = (g - r.b * p.row_tiles) * kRows;
  r.rows = min(p.s * p.H - r.row0, kRows);
  r.len = paged_len(p.kv, p.err, r.b, (int64_t)p.kv.max_pages * p.kv.page_size, report);
  r.keys = p.s == 1 ? r.len : max(0, r.len - p.s + 1 + (r.row0 + r.rows - 1) / p.H);
  return r;
}

// A pair's part of one group: tiles t0 .. t1 - 1.
struct Part {
  Group g;
  int id, t0, t1;
};
struct Shares {
  const DecodeFp4Params* p;
  int g, t;
  int64_t left;
  __device__ Shares(const DecodeFp4Params& prm, const Bars& bars) : p(&prm), g(bars.start_g), t(bars.start_t), left(bars.share) {}
  __device__ __noinline__ bool next(Part& it) {
    while (left > 0 && g < p->groups) {
      it.g = group_of(*p, g, false);
      const int n = (it.g.keys + kTile - 1) / kTile - t;
      if (n <= 0) {
        ++g, t = 0;
        continue;
      }
      it.id = g, it.t0 = t, it.t1 = (int)(t + min((int64_t)n, left));
      left -= it.t1 - it.t0, t = it.t1;
      return true;
    }
    return false;
  }
};

// Tiles before share i of n: total * i / n (a 64-bit quotient takes hundreds of cycles, and the kernel waits for it).
__device__ __forceinline__ int64_t share_start(int64_t total, int64_t i, int64_t n) {
  if (i >= n) return total;
  if (total >= 1ll << 31) return total * i / n;
  const uint32_t t = (uint32_t)total, m = (uint32_t)n, q = t / m, r = t - q * m;
  return (int64_t)((uint64_t)q * (uint32_t)i + (uint32_t)(r * (uint32_t)i) / m);    // r i < n^2 <= 2^32
}

// Where this pair's share starts, and (first CTA of all) the tiles before each group; by all threads.
__device__ __noinline__ void find_share(const DecodeFp4Params& p, Bars& bars, int64_t* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.groups + kThreads - 1) / kThreads, g0 = min(tid * per, p.groups), g1 = min(g0 + per, p.groups);
  int64_t mine = 0;
  for (int g = g0; g < g1; ++g) mine += (group_of(p, g, blockIdx.x == 0).keys + kTile - 1) / kTile;
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t v = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int64_t at = upto - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) at += sums[w];
    total += sums[w];
  }
  // no more shares than tiles: none is empty but those of the pairs behind them
  const int64_t pair = blockIdx.x / 2, pairs = min((int64_t)(gridDim.x / 2), total);
  const int64_t lo = share_start(total, pair, pairs), hi = share_start(total, pair + 1, pairs);
  if (tid == 0) bars.share = hi - lo;
  const bool tell = blockIdx.x == 0, here = lo < hi && at <= lo && lo < at + mine;
  auto put = [&](int64_t g, int64_t v) {
    if (guard_span(p.err, G_TILE_PREFIX, p.before + g, 8, p.before, (uint64_t)(p.groups + 1) * 8)) p.before[g] = v;
  };
  if (tell && tid == 0) put(p.groups, total);
  if (tell || here) {
    for (int g = g0; g < g1; ++g) {
      const int n = (group_of(p, g, false).keys + kTile - 1) / kTile;
      if (tell) put(g, at);
      if (lo < hi && at <= lo && lo < at + n) bars.start_g = g, bars.start_t = (int)(lo - at);
      at += n;
    }
  }
}

__device__ __forceinline__ uint32_t box_unit(uint32_t box, int row, int unit) {   // 16 bytes of a swizzled 128-byte row
  return box + row * 128 + ((unit ^ (row & 7)) << 4);
}
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ---- MMAs of the pair ----
#define MLA_MMA2(D, X, Y, ID, P) "tcgen05.mma.cta_group::2.kind::f16 [" D "], " X ", " Y ", " ID ", " P ";\n\t"
#define MLA_STEP2(P, ID) MLA_MMA2("%0", "x", "y", ID, P) "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
#define MLA_BOX2(P, ID) MLA_STEP2(P, ID) MLA_STEP2("t", ID) MLA_STEP2("t", ID) MLA_MMA2("%0", "x", "y", ID, "t") \
  "add.s64 x, x, 506;\n\tadd.s64 y, y, 506;\n\t"
// S = Q K^T over four boxes of 64 columns, 64 rows each in either CTA
__device__ __forceinline__ void mma2_scores4(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred f, t;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.u32 f, %3, %3;\n\tsetp.eq.u32 t, %3, %3;\n\tmov.b64 x, %1;\n\tmov.b64 y, %2;\n\t"
      MLA_BOX2("f", "%3") MLA_BOX2("t", "%3") MLA_BOX2("t", "%3") MLA_BOX2("t", "%3") "}" ::"r"(d),
      "l"(a), "l"(b), "r"(id)
      : "memory");
}
// S += over the other four and the RoPE columns, whose operands are bf16
__device__ __forceinline__ void mma2_scores5(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t id_pe) {
  asm volatile(
      "{\n\t.reg .pred t;\n\t.reg .b64 x, y;\n\t"
      "setp.eq.u32 t, %3, %3;\n\tmov.b64 x, %1;\n\tmov.b64 y, %2;\n\t"
      MLA_BOX2("t", "%3") MLA_BOX2("t", "%3") MLA_BOX2("t", "%3") MLA_BOX2("t", "%3") MLA_BOX2("t", "%4") "}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(id_pe)
      : "memory");
}
#define MLA_PV2(P) MLA_MMA2("%0", "x", "y", "%4", P) MLA_MMA2("%5", "x", "z", "%4", P) \
  "add.s64 x, x, 2;\n\tadd.s64 y, y, 128;\n\tadd.s64 z, z, 128;\n\t"
// O (+)= P V over 64 keys: two MMAs of 256 columns (128 from either CTA) for each 16 keys
__device__ __forceinline__ void mma2_values(uint32_t d0, uint32_t d1, uint64_t a, uint64_t b0, uint64_t b1, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 x, y, z;\n\t"
      "setp.ne.b32 p, %6, 0;\n\tsetp.eq.u32 t, %4, %4;\n\tmov.b64 x, %1;\n\tmov.b64 y, %2;\n\tmov.b64 z, %3;\n\t"
      MLA_PV2("p") MLA_PV2("t") MLA_PV2("t") MLA_PV2("t") "}" ::"r"(d0),
      "l"(a), "l"(b0), "l"(b1), "r"(id), "r"(d1), "r"(accumulate)
      : "memory");
}
#undef MLA_MMA2
#undef MLA_STEP2
#undef MLA_BOX2
#undef MLA_PV2

// 16 rows of 256 columns as they lie: eight lanes a row, 32 columns each, and their two scales (four lanes a row ask the
// first-level cache for twice as many lines; 0.350 ms for 0.349)
struct Raw {
  uint4 v[4];
  uint32_t sc[4];
};
__device__ __forceinline__ void load_raw(const DecodeFp4Params& p, Raw& x, const int32_t* at, int col, int lane, uint64_t cache_bytes) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = at[4 * i + (lane >> 3)];
    const uint8_t* r = p.kv.cache + (int64_t)a * kFp4Row;
    x.v[i] = make_uint4(0, 0, 0, 0), x.sc[i] = 0;
    if (a >= 0 && guard_span(p.err, G_STEP_IN, r, kFp4Row, p.kv.cache, cache_bytes)) {
      x.v[i] = *reinterpret_cast<const uint4*>(r + col / 2);
      x.sc[i] = *reinterpret_cast<const uint16_t*>(r + kFp4Codes + col / 16);
    }
  }
}
// into four boxes of 64 columns, rows r0 .. r0 + 15.  A lane stores its four 16-byte pieces from its box's number on, so that
// the eight lanes of a row meet eight banks.  Of values a NaN scale becomes a finite one: the key's score is a NaN already, and so is the
// result of each row that sees it; a row from which the key is hidden (weight 0) has nothing of it.
__device__ __forceinline__ void convert_raw(const Raw& x, uint32_t boxes, int r0, int lane, uint32_t cap) {
  const int b = (lane >> 1) & 3, half = lane & 1;
  const bool odd = b & 1, high = b & 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * i + (lane >> 3);
    const uint32_t row = boxes + b * kBox + r * 128;
    const uint2 s = fp4_scales2(x.sc[i], cap);
    uint4 v = x.v[i];
    if (odd) v = make_uint4(v.y, v.z, v.w, v.x);
    if (high) v = make_uint4(v.z, v.w, v.x, v.y);
    // pieces b, b + 1, b + 2, b + 3 (mod 4); 0 and 1 have the first scale
    const uint32_t s0 = high ? s.y : s.x, s1 = odd != high ? s.y : s.x, s2 = high ? s.x : s.y, s3 = odd != high ? s.x : s.y;
    st_shared16(row + (((4 * half + b) ^ (r & 7)) << 4), fp4x8_to_f16(v.x, s0));
    st_shared16(row + (((4 * half + ((b + 1) & 3)) ^ (r & 7)) << 4), fp4x8_to_f16(v.y, s1));
    st_shared16(row + (((4 * half + (b ^ 2)) ^ (r & 7)) << 4), fp4x8_to_f16(v.z, s2));
    st_shared16(row + (((4 * half + ((b + 3) & 3)) ^ (r & 7)) << 4), fp4x8_to_f16(v.w, s3));
  }
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// Box k of this CTA's 64 query rows; rows behind the group's are zeros.  The copies go out ...
__device__ __forceinline__ void ask_query_box(const DecodeFp4Params& p, const Group& g, int first, uint32_t box, int k, int lane) {
  const uint64_t q_bytes = (uint64_t)p.kv.B * p.s * p.H * kDk * 2;
  const int unit = lane & 7;
  const __nv_bfloat16* q = p.q + ((int64_t)g.b * p.s * p.H + g.row0 + first) * kDk + 64 * k + 8 * unit;
#pragma unroll 4
  for (int r = lane >> 3; r < kHalf; r += 4) {
    const __nv_bfloat16* src = q + (int64_t)r * kDk;
    const bool in = first + r < g.rows && guard_span(p.err, G_Q, src, 16, p.q, q_bytes);
    cp_async16_zfill(box_unit(box, r, unit), in ? src : p.q, in ? 16u : 0u);
  }
}
// ... and each lane puts its own into f16 where they lie (the RoPE columns stay)
__device__ __forceinline__ void take_query_box(uint32_t box, int k, int lane) {
  const int unit = lane & 7;
  cp_async_wait_all();
  if (k < 8)
#pragma unroll 4
    for (int r = lane >> 3; r < kHalf; r += 4) st_shared16(box_unit(box, r, unit), bf16x8_to_f16(ld_shared16(box_unit(box, r, unit))));
  fence_proxy_async_smem();
}

// 128 columns of O of this lane's row times a
__device__ __noinline__ void rescale_o(uint32_t to, float a) {
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    uint32_t o[32];
    tmem_ld32(to + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
    tmem_st32(to + c, o);
  }
  tmem_wait_st();
}
// 128 columns of this warp's 32 rows as they are (weights relative to the row's maximum), 16 at a time through 2 KB of
// shared memory so that a store brings whole sectors
__device__ __noinline__ void store_part(const DecodeFp4Params& p, uint32_t to, int64_t slot_row0, int rows, int col, uint32_t stage, int lane) {
  if (rows <= 0) return;                              // (17 requests of 32 query rows 53.3 -> 51.3 us)
#pragma unroll 1
  for (int c = 0; c < 128; c += 16) {
    uint32_t o[16];
    tmem_ld16(to + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      st_shared16(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), unit = lane & 3;
      float* dst = p.part_o + (slot_row0 + r) * kLatent + col + c + 4 * unit;
      const uint4 v = ld_shared16(stage + r * 64 + ((unit ^ ((r >> 1) & 3)) << 4));
      if (r < rows && guard_span(p.err, G_PART_O, dst, 16, p.part_o, p.part_o_bytes)) *reinterpret_cast<uint4*>(dst) = v;
    }
    __syncwarp();
  }
}
// a float's order as an integer's
__device__ __forceinline__ int32_t ordered(float f) {
  const int32_t i = __float_as_int(f);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int32_t i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

template <bool kUp>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) decode_fp4_kernel(const __grid_constant__ DecodeFp4Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + kOffBars);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t cta = cluster_ctarank();
  const uint64_t cache_bytes = (uint64_t)p.kv.num_pages * p.kv.page_size * kFp4Row;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&bars.kfull[i], 2 * (4 + i)), mbar_init(&bars.kempty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.vfull[i], 8), mbar_init(&bars.vempty[i], 1);
      mbar_init(&bars.sfull[i], 1), mbar_init(&bars.sfree[i], 16);
      mbar_init(&bars.same[i], 4), mbar_init(&bars.drain[i], 1);
    }
    mbar_init(&bars.qfull, 18), mbar_init(&bars.qempty, 1);
    mbar_init(&bars.pfull, 16), mbar_init(&bars.pvdone, 1), mbar_init(&bars.ofree, 16);
    for (int i = 0; i < kRowSlots; ++i) mbar_init(&bars.rfull[i], 1), mbar_init(&bars.rfree[i], 17);
    mbar_init(&bars.stall, 1);
    bars.abort = 0;
    if (smem_u32(smem) & 1023u) bars.abort = DEV_TIMEOUT_BASE | D_ALIGN, record_error(p.err, bars.abort);
    fence_mbar_init();
  }
  if (tid < 192) reinterpret_cast<int32_t*>(smem + kOffMax)[tid] = INT32_MIN;
  if (warp == kMmaS) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bars.tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  find_share(p, bars, reinterpret_cast<int64_t*>(smem + kOffRows));    // no row is there yet
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tbase = bars.tmem_base;
  const TileWaits wait{&bars.abort, p.err, p.spin_limit};
  int32_t* row_slots = reinterpret_cast<int32_t*>(smem + kOffRows);
  Shares shares(p, bars);
  Part it;
  uint32_t u = 0, n = 0;                              // tiles and parts gone through
  bool live = bars.abort == 0;

  if (warp < kMmaS) {
    // ---------------- rows ----------------
    // key half hh, 32 of its keys (cc), row r of this CTA; the lanes' 128 columns cc of O
    const int hh = (warp >> 1) & 1, cc = warp >> 2, r = (warp & 1) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float c = p.scale * 1.4426950408889634f, c2 = c == 0.f ? 1e-30f : c;    // see mask_piece
    // Maxima are those of the scores as they come (their minimum, negated, where the scale is negative), and exponents are
    // (score - maximum) c: that difference is exact next to the maximum, where score c - maximum c is off by half a step of a large score.
    const uint64_t c22 = f32x2(c2, c2), lift2 = f32x2(kLift, kLift);
    const float size = fabsf(c2);
    int32_t* const tile_max = reinterpret_cast<int32_t*>(smem + kOffMax) + r;
    const uint32_t prow = smem_u32(smem + kOffP + hh * kBox);
    uint32_t into = 0;                                // tile_max's next third
    for (; live && shares.next(it); ++n) {
      const int row = (int)cta * kHalf + r;            // of the group
      const int seen = row < it.g.rows ? max(0, it.g.len - p.s + 1 + (it.g.row0 + row) / p.H) : 0;
      float m = -CUDART_INF_F, l = 0.f;
      for (int t = it.t0; t < it.t1; ++t, ++u) {
        const int buf = u & 1;
        if (!wait.warp(&bars.sfull[buf], (u >> 1) & 1, D_SFULL)) { live = false; break; }
        tc_fence_after();
        uint32_t s[32];
        tmem_ld32(tbase + lanes + kTmemS + buf * 64 + 32 * cc, s);
        tmem_wait_ld();
        tc_fence_before();
        first_cta_arrive<false>(&bars.sfree[buf], cta);
        const int visible = seen - t * kTile - hh * kHalf - 32 * cc;
        mask_piece<kUp>(s, visible);
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = kUp ? -CUDART_INF_F : CUDART_INF_F;
        row_extreme<kUp>(s, e);
        float mt = visible <= 0 ? -CUDART_INF_F : kUp ? extreme4<kUp>(e) : -extreme4<kUp>(e);
        // the largest of the four warps' (the third that comes next was read by all before they came here)
        const uint32_t next = into == 2 ? 0 : into + 1;
        atomicMax(tile_max + 64 * into, ordered(mt));
        if (hh == 0 && cc == 0) tile_max[64 * next] = INT32_MIN;
        warp_arrive(&bars.same[warp & 1]);
        if (!wait.warp(&bars.same[warp & 1], u & 1, D_PAIR)) { live = false; break; }
        mt = unordered(*reinterpret_cast<volatile int32_t*>(tile_max + 64 * into));
        into = next;
        float a = 1.f;
        if ((mt - m) * size > kRescale || m == -CUDART_INF_F) {
          a = m == -CUDART_INF_F ? 0.f : ex2_approx((m - mt) * size);
          m = mt;
        }
        const float ref = m == -CUDART_INF_F ? 0.f : kUp ? -m : m;
        const uint64_t ref2 = f32x2(ref, ref);
        uint64_t sum[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 16; ++i) {                 // packed into the first sixteen words
          float x0, x1;
          f32x2_split(fma_f32x2(add_f32x2(f32x2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), ref2), c22, lift2), x0, x1);
          x0 = ex2_approx(x0), x1 = ex2_approx(x1);
          sum[i & 1] = add_f32x2(sum[i & 1], f32x2(x0, x1));
          s[i] = pack_f16x2(x0, x1);
        }
        float l0, l1;
        f32x2_split(add_f32x2(sum[0], sum[1]), l0, l1);
        l = l * a + (l0 + l1);
        // the last tile's P V of this key half is done: P of the half may be written over (and O be scaled when all of it is)
        if (u > 0 && !wait.warp(&bars.vempty[hh], (u - 1) & 1, D_VEMPTY)) { live = false; break; }
        if (t > it.t0 && __any_sync(~0u, a != 1.f)) {
          if (!wait.warp(&bars.pvdone, (u - 1) & 1, D_PVDONE)) { live = false; break; }
          tc_fence_after();
          rescale_o(tbase + lanes + kTmemO + 128 * cc, a);
          tc_fence_before();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) st_shared16(box_unit(prow, r, 4 * cc + i), make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]));
        fence_proxy_async_smem();
        first_cta_arrive<true>(&bars.pfull, cta);
      }
      if (!live) break;
      if (!wait.warp(&bars.pvdone, (u - 1) & 1, D_PVDONE)) break;
      tc_fence_after();
      const int64_t slot_row = (int64_t)(it.id + (int)(blockIdx.x / 2)) * p.part_rows + row;
      // the place of P of these 32 rows and keys: free until the same four warps, all done with it, meet over the next tile's maximum
      store_part(p, tbase + lanes + kTmemO + 128 * cc, slot_row - lane, it.g.rows - (row - lane), 256 * cc + 128 * hh,
                 smem_u32(smem + kOffP + hh * kBox + (warp & 1) * 4096 + cc * 2048), lane);
      float* stat = p.part_stat + slot_row * 8;       // the maximum and the four sums
      if (row < it.g.rows && guard_span(p.err, G_PART_LSE, stat, 32, p.part_stat, p.part_stat_bytes)) {
        stat[1 + 2 * hh + cc] = l * 0x1p-7f;
        if (hh == 0 && cc == 0) stat[0] = m * size;
      }
      tc_fence_before();
      first_cta_arrive<false>(&bars.ofree, cta);
    }
  } else if (warp == kMmaS) {
    // ---------------- scores ----------------
    if (cta == 0) {
      if (p.debug_stall) live = live && wait.warp(&bars.stall, 0, D_STALL);
      const uint64_t qdesc = sdesc_sw128(smem_u32(smem + kOffQ), 16, 1024), kdesc = sdesc_sw128(smem_u32(smem + kOffK), 16, 1024);
      const uint32_t id = idesc_f16_f32(kRows, kTile, false, false), id_pe = idesc_bf16_f32(kRows, kTile, false, false);
      for (; live && shares.next(it); ++n) {
        if (!wait.warp(&bars.qfull, n & 1, D_QFULL, true)) break;
        for (int t = it.t0; t < it.t1; ++t, ++u) {
          const int buf = u & 1;
          if (!wait.warp(&bars.sfree[buf], ((u >> 1) & 1) ^ 1, D_SFREE, true)) { live = false; break; }
          if (!wait.warp(&bars.kfull[0], u & 1, D_KFULL, true)) { live = false; break; }
          tc_fence_after();
          if (elect_one()) {
            mma2_scores4(tbase + kTmemS + buf * 64, qdesc, kdesc, id);
            commit<2>(&bars.kempty[0]);
          }
          __syncwarp();
          if (!wait.warp(&bars.kfull[1], u & 1, D_KFULL, true)) { live = false; break; }
          tc_fence_after();
          if (elect_one()) {
            mma2_scores5(tbase + kTmemS + buf * 64, qdesc + 4 * kBox / 16, kdesc + 4 * kBox / 16, id, id_pe);
            commit<2>(&bars.kempty[1]);
            commit<2>(&bars.sfull[buf]);
            if (t == it.t1 - 1) commit<2>(&bars.qempty);
          }
          __syncwarp();
        }
      }
      if (elect_one()) commit<2>(&bars.drain[0]);       // what was issued is done before anything is given back
      mbar_drain(&bars.drain[0], 0);
      __syncwarp();
    }
  } else if (warp == kMmaV) {
    // ---------------- values ----------------
    if (cta == 0) {
      const uint32_t pst = smem_u32(smem + kOffP), vst = smem_u32(smem + kOffV);
      const uint32_t id = idesc_f16_f32(kRows, 256, false, true);
      for (; live && shares.next(it); ++n) {
        if (n > 0 && !wait.warp(&bars.ofree, (n - 1) & 1, D_OFREE, true)) break;
        for (int t = it.t0; t < it.t1; ++t, ++u) {
          // All row warps have scaled O ahead of either half: the MMAs over one half of the keys add to every lane of O, also
          // to those of the warps that bring P of the other half.
          if (!wait.warp(&bars.pfull, u & 1, D_PFULL, true)) { live = false; break; }
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (!wait.warp(&bars.vfull[h], u & 1, D_VFULL, true)) { live = false; break; }
            tc_fence_after();
            if (elect_one()) {
              mma2_values(tbase + kTmemO, tbase + kTmemO + 128, sdesc_sw128(pst + h * kBox, 16, 1024), sdesc_sw128(vst + h * 4 * kBox, kBox, 1024),
                          sdesc_sw128(vst + h * 4 * kBox + 2 * kBox, kBox, 1024), id, t > it.t0 || h > 0 ? 1u : 0u);
              commit<2>(&bars.vempty[h]);
              if (h == 1) commit<2>(&bars.pvdone);
            }
            __syncwarp();
          }
          if (!live) break;
        }
      }
      if (elect_one()) commit<2>(&bars.drain[1]);
      mbar_drain(&bars.drain[1], 0);
      __syncwarp();
    }
  } else if (warp >= kFirstK) {
    // ---------------- 4-bit rows into f16 ----------------
    const bool is_k = warp < kFirstV;
    // 16 rows w % 4: of K this CTA's keys and columns 256 (w / 4) ..; of V key half w / 4 and the CTA's columns
    const int w = (warp - kFirstK) & 7, part = w >> 2, r0 = (w & 3) * 16, chunk = lane & 7;
    const int col = is_k ? 256 * part + 32 * chunk : 256 * (chunk >> 2) + 128 * (int)cta + 32 * (chunk & 3);
    const int first = (is_k ? (int)cta : part) * kHalf + r0;       // of the tile's keys
    const uint32_t boxes = smem_u32(smem + (is_k ? kOffK : kOffV) + 4 * part * kBox);
    uint64_t* const empty = is_k ? &bars.kempty[part] : &bars.vempty[part];
    uint64_t* const full = is_k ? &bars.kfull[part] : &bars.vfull[part];
    uint32_t slot = 0, turn = 0;                      // of the next tile's rows
    Raw x;
    auto load = [&]() -> bool {
      if (!wait.warp(&bars.rfull[slot], turn, D_RFULL)) return false;
      load_raw(p, x, row_slots + slot * kTile + first, col, lane, cache_bytes);
      warp_arrive(&bars.rfree[slot]);
      if (++slot == kRowSlots) slot = 0, turn ^= 1;
      return true;
    };
    for (; live && shares.next(it); ++n) {
      const uint32_t qbox = smem_u32(smem + kOffQ + w * kBox);
      if (is_k) {
        if (!wait.warp(&bars.qempty, (n & 1) ^ 1, D_QEMPTY)) break;
        ask_query_box(p, it.g, (int)cta * kHalf, qbox, w, lane);
      }
      if (!load()) break;
      if (is_k) {
        take_query_box(qbox, w, lane);
        first_cta_arrive<true>(&bars.qfull, cta);
      }
      for (int t = it.t0; t < it.t1; ++t, ++u) {
        if (!wait.warp(empty, (u & 1) ^ 1, D_KEMPTY)) { live = false; break; }
        convert_raw(x, boxes, r0, lane, is_k ? kScaleNan : kScale448);
        fence_proxy_async_smem();
        first_cta_arrive<true>(full, cta);
        // the next tile's loads go out while its place is not free yet
        if (t + 1 < it.t1 && !load()) { live = false; break; }
      }
    }
  } else if (warp == kTableWarp) {
    // ---------------- rows through the block table ----------------
    for (; live && shares.next(it); ++n) {
      for (int t = it.t0; t < it.t1; ++t, ++u) {
        int32_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = t * kTile + 32 * i + lane;
          at[i] = -1;
          if (j < it.g.keys) {
            const int pg = j / p.kv.page_size;
            const int page = guarded_int(p.err, p.kv.block_table, (int64_t)it.g.b * p.kv.max_pages + pg, (int64_t)p.kv.B * p.kv.max_pages);
            if (page >= 0 && page < p.kv.num_pages) at[i] = page * p.kv.page_size + (j - pg * p.kv.page_size);
            else record_error(p.err, DEV_RANGE_BASE | Y_PAGE);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {                  // either CTA asks for the keys of its scores
          const int a = cta == 0 ? at[i] : at[2 + i];
          if (a >= 0) {
            const uint8_t* row = p.kv.cache + (int64_t)a * kFp4Row;
            for (int o = 0; o < kFp4Row; o += 128) prefetch_l2(row + o);
            prefetch_l2(row + kFp4Row - 1);
          }
        }
        const uint32_t slot = u % kRowSlots;
        if (!wait.warp(&bars.rfree[slot], ((u / kRowSlots) & 1) ^ 1, D_RFREE)) { live = false; break; }
#pragma unroll
        for (int i = 0; i < 4; ++i) row_slots[slot * kTile + 32 * i + lane] = at[i];
        warp_arrive(&bars.rfull[slot]);
      }
    }
  } else {
    // ---------------- RoPE columns of this CTA's keys ----------------
    const uint32_t box = smem_u32(smem + kOffK + 8 * kBox), qbox = smem_u32(smem + kOffQ + 8 * kBox);
    const int unit = lane & 7;
    for (; live && shares.next(it); ++n) {
      if (!wait.warp(&bars.qempty, (n & 1) ^ 1, D_QEMPTY)) break;
      ask_query_box(p, it.g, (int)cta * kHalf, qbox, 8, lane);
      take_query_box(qbox, 8, lane);
      first_cta_arrive<true>(&bars.qfull, cta);
      for (int t = it.t0; t < it.t1; ++t, ++u) {
        const uint32_t slot = u % kRowSlots;
        if (!wait.warp(&bars.rfull[slot], (u / kRowSlots) & 1, D_RFULL) || !wait.warp(&bars.kempty[1], (u & 1) ^ 1, D_KEMPTY)) { live = false; break; }
        const int32_t* at = row_slots + slot * kTile + cta * kHalf + (lane >> 3);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int a = at[4 * i];
          const uint8_t* src = p.kv.cache + (int64_t)a * kFp4Row + kFp4Pe + 16 * unit;
          const bool in = a >= 0 && guard_span(p.err, G_STEP_IN, src, 16, p.kv.cache, cache_bytes);
          cp_async16_zfill(box_unit(box, (lane >> 3) + 4 * i, unit), in ? src : (const uint8_t*)p.q, in ? 16u : 0u);
        }
        warp_arrive(&bars.rfree[slot]);
        cp_async_wait_all();
        fence_proxy_async_smem();
        first_cta_arrive<true>(&bars.kfull[1], cta);
      }
    }
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaS) mbar_drain(&bars.drain[0], 0), mbar_drain(&bars.drain[1], 0);    // the last arrivals in either CTA
  __syncwarp();
  cluster_sync();                                     // no MMA of the pair is left, no arrival on its way
  if (warp == kMmaS) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tbase) : "memory");
}

// A CTA a row, four columns a thread: the partials of the pairs that had tiles of its group, by their log-sum-exp, and the
// sink.  A thread a pair finds the weights (a pass over kPairs of them), eight partials' loads go out together: a warp that
// took the partials one after the other spent 63 us on one request's 33.  Up to kFew partials, as among many requests, need no
// pass of their own for the weights (8192 rows 20 -> 14 us; eight in registers 22).
constexpr int kPairs = 128, kFew = 4;
__global__ void __launch_bounds__(kPairs) decode_fp4_reduce_kernel(const __grid_constant__ DecodeFp4Params p, int pairs) {
  __shared__ float weight[kPairs], sums[kPairs], red[8];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t rows = (int64_t)p.kv.B * p.s * p.H, item = blockIdx.x;
  const int64_t b = item / (p.s * p.H);
  const int row = (int)(item - b * (p.s * p.H));
  const int g = (int)(b * p.row_tiles + row / kRows);
  auto before = [&](int64_t i) -> int64_t {
    return guard_span(p.err, G_TILE_PREFIX, p.before + i, 8, p.before, (uint64_t)(p.groups + 1) * 8) ? p.before[i] : 0;
  };
  const int64_t total = before(p.groups), t0 = before(g), t1 = before(g + 1);
  const float sink = p.sinks && guard_span(p.err, G_SINKS, p.sinks + row % p.H, 4, p.sinks, (uint64_t)p.H * 4) ? p.sinks[row % p.H] : -CUDART_INF_F;
  // pairs whose share meets tiles t0 .. t1 - 1
  const int64_t shares = min((int64_t)pairs, total);
  const int p0 = t1 > t0 ? (int)(((t0 + 1) * shares - 1) / total) : 0, p1 = t1 > t0 ? (int)((t1 * shares - 1) / total) : -1;
  // maximum (of scores in powers of two) and sum of pair q's weights
  auto stat_of = [&](int q, float& sum) -> float {
    sum = 0.f;
    const float* s = p.part_stat + ((int64_t)(g + q) * p.part_rows + (row & (kRows - 1))) * 8;
    if (q > p1 || !guard_span(p.err, G_PART_LSE, s, 32, p.part_stat, p.part_stat_bytes)) return -CUDART_INF_F;
    const float4 a = *reinterpret_cast<const float4*>(s);
    sum = (a.y + a.z) + (a.w + s[4]);
    return a.x;
  };
  const float sink2 = sink * 1.4426950408889634f;
  float m = -CUDART_INF_F, keys_m = -CUDART_INF_F;      // -inf: the row sees no key
  float wsum;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  bool nan = false;
  auto part_at = [&](int q) { return p.part_o + ((int64_t)(g + q) * p.part_rows + (row & (kRows - 1))) * kLatent + 4 * tid; };
  if (p1 - p0 < kFew) {
    // few partials: each thread takes them all, statistics and columns asked for together
    float of_m[kFew], of_sum[kFew];
    float4 v[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      of_m[i] = stat_of(p0 + i, of_sum[i]);
      const float* src = part_at(p0 + i);
      const bool in = p0 + i <= p1 && guard_span(p.err, G_PART_O, src, 16, p.part_o, p.part_o_bytes);
      v[i] = in ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kFew; ++i) keys_m = fmaxf(keys_m, of_m[i]), nan |= of_sum[i] != of_sum[i];
    m = fmaxf(keys_m, sink2);
    wsum = sink == -CUDART_INF_F ? 0.f : exp2f(sink2 - m);
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      if (of_m[i] == -CUDART_INF_F) continue;
      const float w = exp2f(of_m[i] - m);
      wsum += w * of_sum[i];
      if (w != 0.f) acc.x += w * v[i].x, acc.y += w * v[i].y, acc.z += w * v[i].z, acc.w += w * v[i].w;
    }
  } else {
    for (int q = p0 + tid; q <= p1; q += kPairs) {
      float l;
      m = fmaxf(m, stat_of(q, l));
      nan |= l != l;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    if (lane == 0) red[tid >> 5] = m;
    nan = __syncthreads_or(nan);
    keys_m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    m = fmaxf(keys_m, sink2);
    wsum = sink == -CUDART_INF_F ? 0.f : exp2f(sink2 - m);
    for (int q0 = p0; q0 <= p1; q0 += kPairs) {
      __syncthreads();
      float l;
      const float mq = stat_of(q0 + tid, l);
      weight[tid] = mq == -CUDART_INF_F ? 0.f : exp2f(mq - m);
      sums[tid] = l;
      __syncthreads();
      const int n = min(kPairs, p1 - q0 + 1);
      for (int i0 = 0; i0 < n; i0 += 8) {
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float* src = part_at(q0 + i0 + i);
          const bool in = i0 + i < n && weight[i0 + i] != 0.f && guard_span(p.err, G_PART_O, src, 16, p.part_o, p.part_o_bytes);
          v[i] = in ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = i0 + i < n ? weight[i0 + i] : 0.f;
          wsum += i0 + i < n ? w * sums[i0 + i] : 0.f;
          acc.x += w * v[i].x, acc.y += w * v[i].y, acc.z += w * v[i].z, acc.w += w * v[i].w;
        }
      }
    }
  }
  const float inv = nan ? CUDART_NAN_F : wsum > 0.f ? p.kv_scale * 0x1p-7f / wsum : 0.f;    // O has P's 2^7
  __nv_bfloat16* out = p.out + item * kLatent + 4 * tid;
  if (guard_span(p.err, G_OUT, out, 8, p.out, (uint64_t)rows * kLatent * 2))
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (tid == 0 && p.lse && guard_span(p.err, G_LSE, p.lse + item, 4, p.lse, (uint64_t)rows * 4))
    p.lse[item] = nan ? CUDART_NAN_F : keys_m == -CUDART_INF_F ? sink : wsum > 0.f ? fmaf(m, 0.6931471805599453f, logf(wsum)) : -CUDART_INF_F;
}

}  // namespace

DecodeFp4Scratch decode_fp4_scratch(int B, int s, int H, int num_splits) {
  DecodeFp4Scratch r;
  const int sms = device_sm_count();
  r.pairs = num_splits > 0 ? num_splits : sms / 2 > 1 ? sms / 2 : 1;
  const int64_t rows = (int64_t)s * H;
  r.row_tiles = (int)((rows + kRows - 1) / kRows);
  r.part_rows = rows < kRows ? (int)rows : kRows;
  r.groups = B * r.row_tiles;
  const size_t slots = (size_t)(r.groups + r.pairs) * r.part_rows;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  r.before = up((size_t)(r.groups + 1) * 8);
  r.part_stat = up(slots * 32);
  r.part_o = up(slots * kLatent * 4);
  return r;
}

cudaError_t launch_decode_fp4(const DecodeFp4Params& p, int pairs, cudaStream_t stream) {
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.run([] {
    cudaError_t r = cudaFuncSetAttribute((const void*)decode_fp4_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return r == cudaSuccess ? cudaFuncSetAttribute((const void*)decode_fp4_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) : r;
  });
  if (e != cudaSuccess) return e;
  if (p.scale >= 0.f) decode_fp4_kernel<true><<<2 * pairs, kThreads, kSmem, stream>>>(p);
  else decode_fp4_kernel<false><<<2 * pairs, kThreads, kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  decode_fp4_reduce_kernel<<<(unsigned)((int64_t)p.kv.B * p.s * p.H), kPairs, 0, stream>>>(p, pairs);
  return cudaGetLastError();
}

}  // namespace mla
