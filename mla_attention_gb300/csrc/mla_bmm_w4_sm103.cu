// Products of a few rows with 4-bit weights and group scales, per head:
//   out[t, h, n] = sum_g scale[h, n, g] sum_{k in g} x[t, h, k] (code[h, n, k] - 8)
//
// Bound by reading the weights (half a byte each) while the tokens are few, and next to that by the integer
// instructions that take a word of eight codes apart.  The weights are the M operand of m16n8k16
// products (16 columns n of the output x 16 k), the tokens the N operand, eight at a time, with fp32 sums;
// the scale multiplies a group's sum where it lies, in the thread's accumulators.  (With accumulators
// in TMEM that would be a read-back for every 32 to 128 k, and eight tokens are a sixteenth of a
// 128-row tile.)
//
// A code c in the low bits of a bf16 word is the subnormal number c 2^-133, and one four bits higher
// is 16 c 2^-133: numbers that the products take exactly.  So w & 0x000f000f, w & 0x00f000f0 and the same
// of w >> 8 are the bf16 pairs (k0, k4), (k1, k5), (k2, k6), (k3, k7) of a word, five
// instructions for eight weights and no conversion.  x is put in the same order of k, times 2^80, or 2^76
// where the code stands four bits higher; one more product with a constant 8 in every place gives
// 8 sum x, which is taken off, and the scale brings 2^53 back.  All of that is exact for |x| from 2^-73 to
// 2^48; larger and infinite values make the sum infinite or NaN, and a sum that is neither
// finite is done over in plain fp32 by the thread that stores it.
//
// Lane (g, t) of a warp holds columns g and g + 8 and takes word t of each 32 k: the four words of
// a product lie in one group whatever the group's size.  A warp owns 16 MT columns and a slice of k, and
// walks it 128 k at a time through a ring of kStages cp.async stages of its own (no barrier in the loop):
// 1 KB per 16 columns and step, the 16-byte pieces of a row swizzled by its number so that the word
// reads hit 32 banks.  The loop is unrolled over the ring, which makes every shared address a constant
// offset.  The slices of a CTA's warps (and of a cluster's CTAs, when there are few columns and a long k)
// are summed in shared memory in a fixed order, and go out along n.
#include <type_traits>

#include "mla_step.h"
#include "row_vec.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 4;
constexpr int kStep = 128;          // k per step
constexpr int kTileBytes = 16 * kStep / 2;

struct Plan {
  int wk_log2;    // 2^this warps of a CTA along k (the others along n)
  int cluster;    // CTAs along k
  int group_log2; // of a group in 32 k
  int vec_x;      // x rows on 16-byte boundaries
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// 16 bytes, or zeros with n = 0, at constant offsets
template <int kDst, int kSrc>
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(kDst), "n"(kSrc) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr uint32_t kUp = 0x67806780u, kUp4 = 0x65806580u;   // 2^80 and 2^76, twice
constexpr float kDown = 0x1p53f;                            // 2^(133 - 80)

// One value in plain fp32: where the products' range does not reach.
template <bool kF32>
__device__ __noinline__ float plain_value(const BmmW4Params& p, int tok, int h, int n) {
  const int64_t row = (int64_t)h * p.N + n;
  const uint8_t* w = p.w4 + row * (p.K / 2);
  const __nv_bfloat16* x = p.x + tok * p.x_stride_t + h * p.x_stride_h;
  const int groups = p.K / p.group;
  float v = 0.f;
  for (int q = 0; q < groups && v == v; ++q) {   // a NaN stays one
    const float s = kF32 ? reinterpret_cast<const float*>(p.scales)[row * groups + q]
                         : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.scales)[row * groups + q]);
    for (int k = q * p.group; k < (q + 1) * p.group; ++k)
      v += __bfloat162float(x[k]) * ((float)((w[k / 2] >> (4 * (k & 1)) & 15) - 8) * s);
  }
  return v;
}

template <int MT, int NT, bool kVec, bool kF32>
__global__ void __launch_bounds__(kThreads) bmm_w4_kernel(const __grid_constant__ BmmW4Params p, const Plan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kCols = 16 * MT, kTok = 8 * NT, kStage = MT * kTileBytes, kRing = kStages * kStage, kScaleBytes = kF32 ? 4 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int wks = 1 << plan.wk_log2, wk = warp & (wks - 1), wn = warp >> plan.wk_log2, wns = kWarps >> plan.wk_log2;
  const int rank = plan.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int tiles_h = (p.N + kCols - 1) / kCols, tiles = p.H * tiles_h;
  const int tile = (plan.cluster > 1 ? blockIdx.x / plan.cluster : blockIdx.x) * wns + wn;
  const int h = min(tile, tiles - 1) / tiles_h, n0 = (min(tile, tiles - 1) - h * tiles_h) * kCols;
  const int tok0 = blockIdx.y * kTok;
  const int steps = (p.K + kStep - 1) / kStep, slices = plan.cluster << plan.wk_log2, slice = (rank << plan.wk_log2) + wk;
  const int u0 = slices > 1 ? (int)((int64_t)steps * slice / slices) : 0;
  const int u1 = slices > 1 ? (int)((int64_t)steps * (slice + 1) / slices) : steps;
  const int row_bytes = p.K / 2, groups = (p.K / 32) >> plan.group_log2;
  const int last = (1 << plan.group_log2) - 1;   // piece i of a step ends a group where (i & last) == last
  const int64_t row0 = (int64_t)h * p.N;

  // ---- weights and scales of this lane's columns g and g + 8 of each 16 (columns past N: any column
  // of the head, nothing of theirs is stored): it copies piece t of a step's weights and holds
  // the scale of k piece t of a step's four ----
  uint8_t* ring = smem + warp * kRing;
  const uint8_t *src[MT][2], *scale[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t row = row0 + min(n0 + 16 * m + 8 * e + g, p.N - 1);
      src[m][e] = p.w4 + row * row_bytes + u0 * (kStep / 2) + 16 * t;
      scale[m][e] = reinterpret_cast<const uint8_t*>(p.scales) + row * groups * kScaleBytes;
    }
  const int swz = (g >> 1) & 3;
  const uint32_t put = smem_u32(ring) + g * 64 + ((t ^ swz) << 4);
  const int left = min(row_bytes, u1 * (kStep / 2)) - u0 * (kStep / 2) - 16 * t;   // > 64 s: step u0 + s has this piece
  // step u0 + base + kAt into stage kAt % kStages; src stands at step u0 + base
  auto fetch = [&](auto at, int base) {   // past K and past the slice: zeros
    constexpr int kAt = decltype(at)::value, kTo = kAt % kStages * kStage;
    const uint32_t n = (base + kAt) * (kStep / 2) < left ? 16u : 0u;
    auto copy = [&](auto mm) {
      constexpr int m = decltype(mm)::value;
      auto ok = [&](const uint8_t* s) {
        return !kGuarded || n == 0 || guard_span(nullptr, G_STEP_IN, s + kAt * (kStep / 2), 16, p.w4, (uint64_t)p.H * p.N * row_bytes);
      };
      if (ok(src[m][0])) cp_async16_at<kTo + m * kTileBytes, kAt * (kStep / 2)>(put, src[m][0], n);
      if (ok(src[m][1])) cp_async16_at<kTo + m * kTileBytes + 512, kAt * (kStep / 2)>(put, src[m][1], n);
    };
    copy(std::integral_constant<int, 0>{});
    if constexpr (MT > 1) copy(std::integral_constant<int, 1>{});
    cp_commit();
  };
  auto load_scales = [&](int u, float (&s)[MT][2]) {   // past K: the last group's, for weights that are not there
    const int i = min((4 * u + t) >> plan.group_log2, groups - 1) * kScaleBytes;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint8_t* f = scale[m][e] + i;
        s[m][e] = 0.f;
        if (guard_span(nullptr, G_STEP_IN, f, kScaleBytes, p.scales, (uint64_t)p.H * p.N * groups * kScaleBytes))
          s[m][e] = (kF32 ? *reinterpret_cast<const float*>(f) : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(f))) * kDown;
      }
  };
  // ---- x: eight k of token g of each eight (tokens past T: the last one's, whose sums are not stored) ----
  const uint64_t ext_x = ((uint64_t)(p.T - 1) * p.x_stride_t + (uint64_t)(p.H - 1) * p.x_stride_h + p.K) * 2;
  const __nv_bfloat16* xt[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xt[nt] = p.x + h * p.x_stride_h + (int64_t)min(tok0 + 8 * nt + g, p.T - 1) * p.x_stride_t + 8 * t;
  auto load_x = [&](int nt, int k, bool inside) {   // from k on; past K: zeros
    uint4 v = make_uint4(0, 0, 0, 0);
    if (inside || k < p.K) {
      const __nv_bfloat16* s = xt[nt] + k;
      if (!guard_span(nullptr, G_STEP_IN, s, 16, p.x, ext_x)) return v;
      v = kVec ? *reinterpret_cast<const uint4*>(s) : load_row8_narrow(s, 8);
    }
    return v;
  };

  // x is asked for ahead by kAhead pieces: a whole step, or one piece where more tokens take the registers
  constexpr int kAhead = NT <= 2 ? 4 : 1;
  const uint32_t eights[4] = {0x00080008u, 0x00080008u, 0x00800080u, 0x00800080u};
  float acc[MT][NT][4] = {}, part[MT][NT][4] = {}, off[NT][4] = {};
  float sc[MT][2];
  uint4 xv[kAhead][NT];
  fetch(std::integral_constant<int, 0>{}, 0);
  fetch(std::integral_constant<int, 1>{}, 0);
  fetch(std::integral_constant<int, 2>{}, 0);
  load_scales(u0, sc);
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xv[i][nt] = load_x(nt, u0 * kStep + 32 * i, false);
  const uint8_t* take[4];   // word t of piece i of column g
#pragma unroll
  for (int i = 0; i < 4; ++i) take[i] = ring + g * 64 + ((i ^ swz) << 4) + 4 * t;

  auto step = [&](auto at, int base) {
    constexpr int kAt = decltype(at)::value;
    const int u = u0 + base + kAt;
    const bool inside = (u + 2) * kStep <= p.K;   // this step and the next one end before K
    float sc_next[MT][2];
    load_scales(u + 1, sc_next);
    cp_wait<kStages - 2>();
    __syncwarp();       // every lane's copies of step u have landed, and step u - 1 is read
    fetch(std::integral_constant<int, kAt + kStages - 1>{}, base);
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // 32 k each
      uint4 xn[NT];                 // this piece, and in its place the one kAhead on
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        xn[nt] = xv[i % kAhead][nt];
        xv[i % kAhead][nt] = load_x(nt, u * kStep + 32 * (i + kAhead), inside);
      }
      uint32_t a[MT][2][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(take[i] + kAt * kStage + m * kTileBytes);
        const uint32_t w0 = from[0], w1 = from[128], v0 = w0 >> 8, v1 = w1 >> 8;
        a[m][0][0] = w0 & 0x000f000fu, a[m][0][1] = w1 & 0x000f000fu, a[m][0][2] = w0 & 0x00f000f0u, a[m][0][3] = w1 & 0x00f000f0u;
        a[m][1][0] = v0 & 0x000f000fu, a[m][1][1] = v1 & 0x000f000fu, a[m][1][2] = v0 & 0x00f000f0u, a[m][1][3] = v1 & 0x00f000f0u;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 v = xn[nt];
        const uint32_t b0 = mul_bf16x2(__byte_perm(v.x, v.z, 0x5410), kUp), b1 = mul_bf16x2(__byte_perm(v.x, v.z, 0x7632), kUp4);
        const uint32_t b2 = mul_bf16x2(__byte_perm(v.y, v.w, 0x5410), kUp), b3 = mul_bf16x2(__byte_perm(v.y, v.w, 0x7632), kUp4);
        mma16816(off[nt], eights, b0, b1);
        mma16816(off[nt], eights, b2, b3);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816(part[m][nt], a[m][0], b0, b1);
          mma16816(part[m][nt], a[m][1], b2, b3);
        }
      }
      if ((i & last) == last) {   // the end of a group
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float s0 = __shfl_sync(~0u, sc[m][0], i, 4), s1 = __shfl_sync(~0u, sc[m][1], i, 4);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[m][nt][j] += (j < 2 ? s0 : s1) * (part[m][nt][j] - off[nt][j]);
              part[m][nt][j] = 0.f;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) off[nt][0] = off[nt][1] = off[nt][2] = off[nt][3] = 0.f;
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) sc[m][0] = sc_next[m][0], sc[m][1] = sc_next[m][1];
  };
  for (int base = 0; base < u1 - u0; base += kStages) {
    const int n = u1 - u0 - base;
    step(std::integral_constant<int, 0>{}, base);
    if (n > 1) step(std::integral_constant<int, 1>{}, base);
    if (n > 2) step(std::integral_constant<int, 2>{}, base);
    if (n > 3) step(std::integral_constant<int, 3>{}, base);
#pragma unroll
    for (int m = 0; m < MT; ++m) src[m][0] += kStages * (kStep / 2), src[m][1] += kStages * (kStep / 2);
  }
  cp_wait<0>();

  // ---- the slices' sums: [warp][token][column] in shared memory, joined in order, out along n ----
  constexpr int kPitch = kCols + 1;
  float* sums = reinterpret_cast<float*>(smem);
  // a warp's sums lie in its own ring while it has them to itself, else anywhere once all rings are done
  constexpr int kOwn = kRing / 4 >= kTok * kPitch ? kRing / 4 : kTok * kPitch;
  if (slices > 1 || kOwn == kTok * kPitch) __syncthreads();
  else __syncwarp();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sums[warp * kOwn + (8 * nt + 2 * t + (j & 1)) * kPitch + 16 * m + 8 * (j >> 1) + g] = acc[m][nt][j];
  if (plan.cluster > 1) cluster_sync();
  else if (slices > 1) __syncthreads();
  else __syncwarp();
  if (tile < tiles) {
    const uint64_t ext_out = ((uint64_t)(p.T - 1) * p.out_stride_t + (uint64_t)(p.H - 1) * p.out_stride_h + p.N) * 2;
    const int items = min(kTok, p.T - tok0) * kCols;
    for (int i = slice * 32 + lane; i < items; i += slices * 32) {   // dealt over the tile's warps
      const int c = i % kCols, tok = i / kCols, n = n0 + c;
      if (n >= p.N) continue;
      const int at = (warp - wk) * kOwn + tok * kPitch + c;
      float v = 0.f;
      if (plan.cluster == 1) {
        for (int s = 0; s < wks; ++s) v += sums[at + s * kOwn];
      } else {
        for (int r = 0; r < plan.cluster; ++r) {
          const uint32_t base = map_to_rank(smem_u32(sums), r);
          for (int s = 0; s < wks; ++s) v += ld_cluster_f32(base + 4 * (at + s * kOwn));
        }
      }
      if (!(fabsf(v) < __int_as_float(0x7f800000))) v = plain_value<kF32>(p, tok0 + tok, h, n);
      __nv_bfloat16* o = p.out + (tok0 + tok) * p.out_stride_t + h * p.out_stride_h + n;
      if (guard_span(nullptr, G_STEP_OUT, o, 2, p.out, ext_out)) *o = __float2bfloat16_rn(v);
    }
  }
  if (plan.cluster > 1) cluster_sync();   // the others may still read this CTA's sums
}

template <int MT, int NT, bool kVec, bool kF32>
cudaError_t launch(const BmmW4Params& p, const Plan& plan, cudaStream_t stream) {
  constexpr size_t kRing = (size_t)kWarps * kStages * MT * kTileBytes;
  constexpr size_t kSums = (size_t)kWarps * 8 * NT * (16 * MT + 1) * 4;
  constexpr size_t kSmem = kRing > kSums ? kRing : kSums;
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    const auto f = bmm_w4_kernel<MT, NT, kVec, kF32>;
    cudaError_t r = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    return r != cudaSuccess ? r : cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  });
  if (e != cudaSuccess) return e;
  const int tiles = p.H * ((p.N + 16 * MT - 1) / (16 * MT)), wns = kWarps >> plan.wk_log2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = plan.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((tiles + wns - 1) / wns * plan.cluster), (unsigned)((p.T + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = plan.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, bmm_w4_kernel<MT, NT, kVec, kF32>, p, plan);
}

template <int MT, int NT, bool kVec>
cudaError_t launch(const BmmW4Params& p, const Plan& plan, cudaStream_t stream) {
  return p.scales_f32 ? launch<MT, NT, kVec, true>(p, plan, stream) : launch<MT, NT, kVec, false>(p, plan, stream);
}
template <int NT>
cudaError_t launch(const BmmW4Params& p, const Plan& plan, int mt, cudaStream_t stream) {
  if (!plan.vec_x) return launch<1, NT, false>(p, plan, stream);
  if constexpr (NT <= 4)
    if (mt == 2) return launch<2, NT, true>(p, plan, stream);
  return launch<1, NT, true>(p, plan, stream);
}

}  // namespace

cudaError_t launch_bmm_w4(const BmmW4Params& p, cudaStream_t stream) {
  const int steps = (p.K + kStep - 1) / kStep;
  const int64_t sms = device_sm_count(), warps = 12 * sms;   // warps that keep every SM's copies in flight
  Plan plan;
  plan.vec_x = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.x_stride_t % 8 == 0 && p.x_stride_h % 8 == 0;
  const int nt = p.T <= 8 ? 1 : p.T <= 16 ? 2 : p.T <= 32 ? 4 : 8;
  // Two tiles of 16 columns a warp (they share the reads of x) where that still leaves every SM its warps.
  int mt = !plan.vec_x || nt == 8 ? 1 : 2;
  while (mt > 1 && (int64_t)p.H * ((p.N + 16 * mt - 1) / (16 * mt)) * steps < warps) mt /= 2;
  // k is cut while there are too few warps and a slice keeps two steps: first over the CTA's warps
  // (each cut only moves warps from n to k), then over CTAs.
  const int64_t tiles = (int64_t)p.H * ((p.N + 16 * mt - 1) / (16 * mt));
  int wk = 1;
  plan.wk_log2 = 0;
  plan.cluster = 1;
  while (wk < kWarps && steps / (2 * wk) >= 2 && tiles * wk < warps) wk *= 2, ++plan.wk_log2;
  while (wk == kWarps && plan.cluster < 8 && steps / (2 * wk * plan.cluster) >= 2 && tiles * wk * plan.cluster < warps) plan.cluster *= 2;
  plan.group_log2 = p.group == 32 ? 0 : p.group == 64 ? 1 : 2;
  if (nt == 1) return launch<1>(p, plan, mt, stream);
  if (nt == 2) return launch<2>(p, plan, mt, stream);
  if (nt == 4) return launch<4>(p, plan, mt, stream);
  return launch<8>(p, plan, mt, stream);
}

}  // namespace mla
