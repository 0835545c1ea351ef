// Cache rows by slot: the latent's RMS norm, RoPE and the write of [latent | rotated k_pe] into the
// paged cache in bf16, e4m3 or 4 bits, and the rotated q_pe into the fused query.
//
//   row = [c_kv / sqrt(mean(c_kv^2) + eps) * w | turn(k_pe)]       cache[slot] = bf16(row) or e4m3(row / kv_scale)
// A pair (a, b) of a RoPE vector turns by its angle: (a cos - b sin, a sin + b cos); pair i is
// (x[2i], x[2i+1]) or, with is_neox, (x[i], x[i+32]).  Everything is computed in fp32 and rounded once.
// 4-bit rows (append_latents_fp4): two lanes hold the 16 columns of a scale.  Scale and codes are those of the exact
// quotients: each is rounded from its fp32 value a little below and a little above (2^-20, over the 13 roundings behind it); where
// the two differ, once or twice in 512 rows, the row is done again with its norm in fp64 and each such value is compared
// with the border itself.
//
// HBM-bound: per token 1152 bytes in, 576 or 1152 out and 256 per head of q.  Half a warp per latent, four
// lanes per row's RoPE columns and a warp per 16 heads of a token's q (eight: 55 us for the prefill below),
// all independent: no shared memory, no barrier.  What a warp reads goes
// out before it looks at its token's position and slot: a chain of three loads would leave most of the
// bandwidth idle; and two latents a warp, each lane with four 16-byte vectors, keep twice as many bytes on
// the way as one.  In both pairings a lane's two 16-byte vectors at columns 8u and 32 + 8u (u = 0..3)
// hold whole pairs, so four lanes serve a RoPE vector, read its angles once and use them for all of
// the warp's heads.
// Prefill of 8192 tokens with 128 heads and the rows written too 47.4 us, 93 % of the copy's bandwidth (the cache
// stays partly in L2); 32768 rows to e4m3 without heads 14.1 to 14.8 us, 65 to 68 %, bound by issue and load latency; a decode
// step of 64 tokens with 128 heads 2.4 to 2.6 us.  To 4 bits the prefill takes 54 us, 81 % (two roundings of each code), the
// decode step 3.3.
#include "fp4_rows.cuh"
#include "mla_step.h"
#include "row_vec.cuh"

namespace mla {
namespace {

constexpr int kR = 64, kPairs = 32;
constexpr int kHeadsPerWarp = 16;   // 2 steps of 8 heads, the loads of both in flight at once
constexpr int kSteps = kHeadsPerWarp / 8;

struct Angles {
  float c[8], s[8];
};

// the angles of lane u's eight pairs
__device__ __forceinline__ Angles load_angles(const KvAppendParams& p, int pos, int u, bool neox) {
  Angles a = {};
  const float* cs = p.cos_sin + (int64_t)pos * kR;
  if (!guard_span(p.err, G_STEP_IN, cs, kR * 4, p.cos_sin, (uint64_t)p.max_pos * kR * 4)) return a;
  const int i0 = neox ? 8 * u : 4 * u, i1 = neox ? 8 * u + 4 : 16 + 4 * u;
  const float4 c0 = *reinterpret_cast<const float4*>(cs + i0), c1 = *reinterpret_cast<const float4*>(cs + i1);
  const float4 s0 = *reinterpret_cast<const float4*>(cs + kPairs + i0);
  const float4 s1 = *reinterpret_cast<const float4*>(cs + kPairs + i1);
  a.c[0] = c0.x, a.c[1] = c0.y, a.c[2] = c0.z, a.c[3] = c0.w, a.c[4] = c1.x, a.c[5] = c1.y, a.c[6] = c1.z, a.c[7] = c1.w;
  a.s[0] = s0.x, a.s[1] = s0.y, a.s[2] = s0.z, a.s[3] = s0.w, a.s[4] = s1.x, a.s[5] = s1.y, a.s[6] = s1.z, a.s[7] = s1.w;
  return a;
}

// lo: columns 8u .. 8u + 7, hi: columns 32 + 8u ..
__device__ __forceinline__ void turn(float (&lo)[8], float (&hi)[8], const Angles& g, bool neox) {
  if (neox) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = lo[i], b = hi[i];
      lo[i] = a * g.c[i] - b * g.s[i];
      hi[i] = a * g.s[i] + b * g.c[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = lo[2 * i], b = lo[2 * i + 1];
      lo[2 * i] = a * g.c[i] - b * g.s[i];
      lo[2 * i + 1] = a * g.s[i] + b * g.c[i];
      a = hi[2 * i], b = hi[2 * i + 1];
      hi[2 * i] = a * g.c[4 + i] - b * g.s[4 + i];
      hi[2 * i + 1] = a * g.s[4 + i] + b * g.c[4 + i];
    }
  }
}

// eight values of row `row` of the cache from column `col`
__device__ __forceinline__ void store_cache8(const KvAppendParams& p, int64_t row, int col, const float (&f)[8]) {
  const uint64_t ext = (uint64_t)p.cache_rows * kDk * (p.e4m3 ? 1 : 2);
  if (p.e4m3) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = f[i];
    quotient8(q, p.kv_scale, p.inv_kv_scale);
    uint2 v = e4m3x8_pack(q);
    if ((((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u) {   // a NaN code
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (q[i] != q[i]) q[i] = f[i] * p.inv_kv_scale;   // of an infinite value or quotient saturates, of a NaN stays
      v = e4m3x8_pack(q);
    }
    uint8_t* dst = reinterpret_cast<uint8_t*>(p.cache) + row * kDk + col;
    if (guard_span(p.err, G_STEP_OUT, dst, 8, p.cache, ext)) *reinterpret_cast<uint2*>(dst) = v;
  } else {
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.cache) + row * kDk + col;
    if (guard_span(p.err, G_STEP_OUT, dst, 16, p.cache, ext)) *reinterpret_cast<uint4*>(dst) = bf16x8_pack(f);
  }
}

// eight RoPE columns of row `row` of a 4-bit cache
__device__ __forceinline__ void store_pe8_fp4(const KvAppendParams& p, int64_t row, int col, const float (&f)[8]) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = f[i];
  if (p.kv_scale != 1.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = f[i] / p.kv_scale;
  }
  uint8_t* dst = reinterpret_cast<uint8_t*>(p.cache) + row * kFp4Row + kFp4Pe + 2 * col;
  if (guard_span(p.err, G_STEP_OUT, dst, 16, p.cache, (uint64_t)p.cache_rows * kFp4Row)) *reinterpret_cast<uint4*>(dst) = bf16x8_pack(q);
}

__device__ __forceinline__ uint4 load16(const KvAppendParams& p, const __nv_bfloat16* src, const __nv_bfloat16* base, int64_t extent) {
  return guard_span(p.err, G_STEP_IN, src, 16, base, (uint64_t)extent * 2) ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void store16(const KvAppendParams& p, __nv_bfloat16* dst, const __nv_bfloat16* base, int64_t extent, const float (&f)[8]) {
  if (guard_span(p.err, G_STEP_OUT, dst, 16, base, (uint64_t)extent * 2)) *reinterpret_cast<uint4*>(dst) = bf16x8_pack(f);
}

__device__ __forceinline__ int token_int(const KvAppendParams& p, const int32_t* base, int t) {
  return guard_span(p.err, G_STEP_IN, base + t, 4, base, (uint64_t)p.T * 4) ? base[t] : -1;
}

// ---- 16 heads of a token: four lanes a head, eight heads a step ----
__device__ __forceinline__ void turn_heads(const KvAppendParams& p, int t, int first, int lane) {
  const bool neox = p.is_neox != 0;
  const int u = lane & 3, h0 = first + (lane >> 2), pos = token_int(p, p.positions, t);
  const int64_t ext_q = (p.T - 1) * p.q_pe_stride_t + (p.H - 1) * p.q_pe_stride_h + kR;
  const int64_t ext_o = (p.T - 1) * p.q_out_stride_t + (p.H - 1) * p.q_out_stride_h + kDk;
  uint4 lo[kSteps], hi[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int h = h0 + 8 * k;
    if (h < p.H) {
      const __nv_bfloat16* src = p.q_pe + t * p.q_pe_stride_t + h * p.q_pe_stride_h + 8 * u;
      lo[k] = load16(p, src, p.q_pe, ext_q);
      hi[k] = load16(p, src + 32, p.q_pe, ext_q);
    }
  }
  if (pos < 0 || pos >= p.max_pos) return;   // the token's row reports it
  const Angles g = load_angles(p, pos, u, neox);
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int h = h0 + 8 * k;
    if (h < p.H) {
      float a[8], b[8];
      bf16x8_unpack(lo[k], a);
      bf16x8_unpack(hi[k], b);
      turn(a, b, g, neox);
      __nv_bfloat16* dst = p.q_out + t * p.q_out_stride_t + h * p.q_out_stride_h + kLatent + 8 * u;
      store16(p, dst, p.q_out, ext_o, a);
      store16(p, dst + 32, p.q_out, ext_o, b);
    }
  }
}

// Where token t's row goes.  A position or slot outside its range but -1 is reported by the caller that
// asks for it.
struct Target {
  int pos;            // -1: nothing is written
  int64_t slot;       // -1: no cache row
};
__device__ __forceinline__ Target row_target(const KvAppendParams& p, int pos, int64_t slot, bool report) {
  if (pos < 0 || pos >= p.max_pos) {
    if (pos != -1 && report) record_error(p.err, DEV_RANGE_BASE | 0x78);
    return {-1, -1};
  }
  if (slot < 0 || slot >= p.cache_rows) {
    if (slot != -1 && report) record_error(p.err, DEV_RANGE_BASE | 0x79);
    slot = -1;
  }
  return {slot >= 0 || p.kv_out ? pos : -1, slot};
}
// columns col .. col + 7 of token t's row (kFp4: RoPE columns, kept in bf16)
template <bool kFp4 = false>
__device__ __forceinline__ void put_row8(const KvAppendParams& p, int t, int64_t slot, int col, const float (&f)[8]) {
  if (slot >= 0) {
    if constexpr (kFp4) store_pe8_fp4(p, slot, col - kLatent, f);
    else store_cache8(p, slot, col, f);
  }
  if (p.kv_out) store16(p, p.kv_out + t * p.kv_out_stride + col, p.kv_out, (p.T - 1) * p.kv_out_stride + kDk, f);
}

// ---- the RoPE columns of eight rows, four lanes a row ----
template <bool kFp4>
__device__ __forceinline__ void append_pe(const KvAppendParams& p, int t, int lane) {
  if (t >= p.T) return;
  const bool neox = p.is_neox != 0;
  const int u = lane & 3, pos = token_int(p, p.positions, t);
  const int64_t slot = token_int(p, p.slots, t), ext = (p.T - 1) * p.k_pe_stride + kR;
  const __nv_bfloat16* src = p.k_pe + t * p.k_pe_stride + 8 * u;
  const uint4 lo = load16(p, src, p.k_pe, ext), hi = load16(p, src + 32, p.k_pe, ext);
  const Target to = row_target(p, pos, slot, false);
  if (to.pos < 0) return;
  const Angles g = load_angles(p, to.pos, u, neox);
  float a[8], b[8];
  bf16x8_unpack(lo, a);
  bf16x8_unpack(hi, b);
  turn(a, b, g, neox);
  put_row8<kFp4>(p, t, to.slot, kLatent + 8 * u, a);
  put_row8<kFp4>(p, t, to.slot, kLatent + 32 + 8 * u, b);
}

__device__ __forceinline__ float row_sum16(float v) {   // over a row's 16 lanes
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// Two rows one or both of whose squares leave fp32's range at either end: the sum of squares at `up` of the row's size, a
// power of two.  A small row goes on at that size; of a huge one, whose small values that would lose, it goes back behind
// the weight.  Out of line: between the other instructions it cost 0.1 us a launch.
__device__ __noinline__ void append_far_latents(const KvAppendParams& p, int t, Target to, int lane, float up) {
  const int l = lane & 15;
  auto load = [&](int k, float(&f)[8]) {
    bf16x8_unpack(load16(p, p.c_kv + t * p.c_kv_stride + 128 * k + 8 * l, p.c_kv, (p.T - 1) * p.c_kv_stride + kLatent), f);
  };
  float sum = 0.f;
  if (to.pos >= 0)
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      float f[8];
      load(k, f);
      scale8(f, up);
      sum += square_sum8(f);
    }
  const float inv = rsqrt_newton(row_sum16(sum) * (1.f / kLatent) + p.eps * up * up), grow = fmaxf(up, 1.f), back = fminf(up, 1.f);
  if (to.pos < 0) return;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    float f[8], w[8];
    load(k, f);
    bf16x8_unpack(load16(p, p.weight + 128 * k + 8 * l, p.weight, kLatent), w);
    scale8(f, grow);
    norm8_back(f, inv, w, back);
    put_row8(p, t, to.slot, 128 * k + 8 * l, f);
  }
}

// ---- the latents of two rows: lane l of a row's 16 holds columns 128 k + 8 l .. (k = 0..3).  t is past the
// last token for the half that has none. ----
__device__ __forceinline__ void append_latents(const KvAppendParams& p, int t, int lane) {
  const int l = lane & 15;
  Target to = {-1, -1};
  uint4 v[4];
  if (t < p.T) {
    const int pos = token_int(p, p.positions, t);
    const int64_t slot = token_int(p, p.slots, t);
    const __nv_bfloat16* src = p.c_kv + t * p.c_kv_stride + 8 * l;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = load16(p, src + 128 * k, p.c_kv, (p.T - 1) * p.c_kv_stride + kLatent);
    to = row_target(p, pos, slot, l == 0);
  }
  float inv = 1.f;
  if (p.weight) {
    float sum = 0.f;
    if (to.pos >= 0) {
      float part[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[8];
        bf16x8_unpack(v[k], f);
        part[k] = square_sum8(f);
      }
      sum = (part[0] + part[1]) + (part[2] + part[3]);
    }
    const float mean = row_sum16(sum) * (1.f / kLatent) + p.eps;
    const bool huge = mean > 5e35f, tiny = mean < 0x1p-100f && to.pos >= 0;
    if (__any_sync(~0u, huge || tiny)) return append_far_latents(p, t, to, lane, huge ? 0x1p-96f : tiny ? 0x1p96f : 1.f);
    inv = rsqrt_newton(mean);
  }
  if (to.pos < 0) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float f[8];
    bf16x8_unpack(v[k], f);
    if (p.weight) {
      float wf[8];
      bf16x8_unpack(load16(p, p.weight + 128 * k + 8 * l, p.weight, kLatent), wf);
      norm8(f, inv, wf);
    }
    put_row8(p, t, to.slot, 128 * k + 8 * l, f);
  }
}

// ---- 4-bit rows ----
// Sixteen columns, eight in each of two lanes: their scale and codes.
struct Fp4Part {
  uint32_t scale;    // e4m3
  uint32_t codes;    // this lane's eight, first in the lowest four bits
  bool unsure;       // a value near a border
};
constexpr float kBelow = 1.f - 0x1p-20f, kAbove = 1.f + 0x1p-20f;

__device__ __forceinline__ uint32_t e4m3_byte(float v) { return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3); }
__device__ __forceinline__ uint32_t e2m1_byte(float lo, float hi) {
  return (uint8_t)__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}
// the largest of sixteen columns' sizes: as bits a NaN is above all
__device__ __forceinline__ float largest16(const float (&y)[8], uint32_t pair) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(y[i]) & 0x7fffffffu);
  return __uint_as_float(max(a, __shfl_xor_sync(pair, a, 1)));
}
// max(a / 6, 2^-9) and a NaN where a is one
__device__ __forceinline__ float scale_of(float v) { return v < 0x1p-9f ? 0x1p-9f : v; }

// from values y of fp32 precision; inv6: 1 / (6 kv_scale)
__device__ __forceinline__ Fp4Part fp4_part(const float (&y)[8], float kv_scale, float inv6, uint32_t pair) {
  Fp4Part r;
  const float u = largest16(y, pair) * inv6;
  r.scale = e4m3_byte(scale_of(u * kBelow));
  r.unsure = r.scale != e4m3_byte(scale_of(u * kAbove));
  const float inv = 1.f / (e4m3_to_f32(r.scale) * kv_scale);
  uint32_t above = 0;
  r.codes = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float a = y[i] * inv, b = y[i + 1] * inv;
    r.codes |= e2m1_byte(a * kBelow, b * kBelow) << (4 * i);
    above |= e2m1_byte(a * kAbove, b * kAbove) << (4 * i);
  }
  r.unsure |= r.codes != above;
  return r;
}

// the size of a code in halves
__device__ __forceinline__ int e2m1_halves(uint32_t c) {
  c &= 7u;
  return c < 4 ? (int)c : (int)((2u + (c & 1u)) << ((c >> 1) - 1u));
}
// The same decided in fp64: y[i] = c[i] w[i] inv, and near a border the value against the border times scale and kv_scale.
__device__ __forceinline__ Fp4Part fp4_part_exact(const double (&y)[8], float kv_scale, uint32_t pair) {
  Fp4Part r;
  r.unsure = false;
  double top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!(fabs(y[i]) <= top)) top = fabs(y[i]);     // a NaN takes the place of any
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (y[i] != y[i]) top = y[i];                   // and keeps it
  const double other = __shfl_xor_sync(pair, top, 1);
  if (other != other || other > top) top = other;
  const float u = (float)(top / (6.0 * kv_scale));
  uint32_t lo = e4m3_byte(scale_of(u * kBelow));
  const uint32_t hi = e4m3_byte(scale_of(u * kAbove));
  if (lo != hi) {    // their midpoint has five bits
    const double mid = 3.0 * ((double)e4m3_to_f32(lo) + (double)e4m3_to_f32(hi)) * kv_scale;   // 6 times it
    if (top > mid || (top == mid && (hi & 1u) == 0)) lo = hi;
  }
  r.scale = lo;
  const double unit = (double)e4m3_to_f32(lo) * kv_scale;
  const float inv = (float)(1.0 / unit);
  r.codes = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const float t = (float)fmin(fmax(y[i], -0x1p126), 0x1p126) * inv;
    uint32_t a = e2m1_byte(t * kBelow, 0.f) & 15u;
    const uint32_t b = e2m1_byte(t * kAbove, 0.f) & 15u;
    if (a != b) {
      const double border = (e2m1_halves(a) + e2m1_halves(b)) * 0.25 * unit, v = fabs(y[i]);
      if (v > border || (v == border && (b & 1u) == 0)) a = b;
    }
    r.codes |= a << (4 * i);
  }
  return r;
}

__device__ __forceinline__ void store_part(const KvAppendParams& p, int64_t row, int k, int l, const Fp4Part& part) {
  uint8_t* dst = reinterpret_cast<uint8_t*>(p.cache) + row * kFp4Row;
  const uint64_t ext = (uint64_t)p.cache_rows * kFp4Row;
  if (guard_span(p.err, G_STEP_OUT, dst + 64 * k + 4 * l, 4, p.cache, ext)) *reinterpret_cast<uint32_t*>(dst + 64 * k + 4 * l) = part.codes;
  if ((l & 1) == 0 && guard_span(p.err, G_STEP_OUT, dst + kFp4Codes + 8 * k + l / 2, 1, p.cache, ext))
    dst[kFp4Codes + 8 * k + l / 2] = (uint8_t)part.scale;
}
__device__ __forceinline__ void put_latent8_fp4(const KvAppendParams& p, int t, int col, const float (&f)[8]) {
  if (p.kv_out) store16(p, p.kv_out + t * p.kv_out_stride + col, p.kv_out, (p.T - 1) * p.kv_out_stride + kDk, f);
}

// A row done again in fp64, by its sixteen lanes; rows of any size.  v: the row as it was read (kv_out may be c_kv's place).
__device__ __noinline__ void append_exact_latent_fp4(const KvAppendParams& p, int t, int64_t slot, int lane, const uint4 (&v)[4]) {
  const int l = lane & 15;
  const uint32_t row = 0xffffu << (lane & 16), pair = 3u << (lane & 30);
  double inv = 1;
  if (p.weight) {
    double sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[8];
      bf16x8_unpack(v[k], f);
      double s[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i & 1] = fma((double)f[i], (double)f[i], s[i & 1]);
      sum += s[0] + s[1];
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(row, sum, d);
    inv = 1.0 / sqrt(sum * (1.0 / kLatent) + (double)p.eps);
  }
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    float f[8], w[8];
    double y[8];
    bf16x8_unpack(k == 0 ? v[0] : k == 1 ? v[1] : k == 2 ? v[2] : v[3], f);
    if (p.weight) bf16x8_unpack(load16(p, p.weight + 128 * k + 8 * l, p.weight, kLatent), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = p.weight ? (double)f[i] * inv * (double)w[i] : (double)f[i];
      f[i] = (float)y[i];
    }
    if (slot >= 0) store_part(p, slot, k, l, fp4_part_exact(y, p.kv_scale, pair));
    put_latent8_fp4(p, t, 128 * k + 8 * l, f);
  }
}

// as append_latents; t is past the last token for the half that has none
__device__ __forceinline__ void append_latents_fp4(const KvAppendParams& p, int t, int lane) {
  const int l = lane & 15;
  const uint32_t pair = 3u << (lane & 30), row = 0xffffu << (lane & 16);
  Target to = {-1, -1};
  uint4 v[4];
  if (t < p.T) {
    const int pos = token_int(p, p.positions, t);
    const int64_t slot = token_int(p, p.slots, t);
    const __nv_bfloat16* src = p.c_kv + t * p.c_kv_stride + 8 * l;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = load16(p, src + 128 * k, p.c_kv, (p.T - 1) * p.c_kv_stride + kLatent);
    to = row_target(p, pos, slot, l == 0);
  }
  if (to.pos < 0) return;
  float inv = 1.f;
  bool unsure = false;
  if (p.weight) {
    float part[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[8];
      bf16x8_unpack(v[k], f);
      part[k] = square_sum8(f);
    }
    float sum = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(row, sum, d);
    const float mean = sum * (1.f / kLatent) + p.eps;
    unsure = mean > 5e35f || mean < 0x1p-100f;        // squares that leave fp32
    inv = rsqrt_newton(mean);
  }
  const float inv6 = 1.f / (6.f * p.kv_scale);
  if (!unsure) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[8];
      bf16x8_unpack(v[k], f);
      if (p.weight) {
        float wf[8];
        bf16x8_unpack(load16(p, p.weight + 128 * k + 8 * l, p.weight, kLatent), wf);
        norm8(f, inv, wf);
      }
      if (to.slot >= 0) {
        const Fp4Part part = fp4_part(f, p.kv_scale, inv6, pair);
        unsure |= part.unsure;
        store_part(p, to.slot, k, l, part);
      }
      put_latent8_fp4(p, t, 128 * k + 8 * l, f);
    }
  }
  if (__any_sync(row, unsure)) append_exact_latent_fp4(p, t, to.slot, lane, v);
}

// CTAs of four warps: of eight, 15.0 us for the 32768 rows above and 2.7 for the decode step.
// The first warps bring two latents each, the next the RoPE columns of eight rows, the others the heads.
template <bool kFp4>
__global__ void __launch_bounds__(128, 8) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  const int lane = threadIdx.x & 31;
  uint32_t w = blockIdx.x * 4 + (threadIdx.x >> 5);
  const uint32_t latents = ((uint32_t)p.T + 1) / 2, pes = ((uint32_t)p.T + 7) / 8;
  if (w < latents) {
    if constexpr (kFp4) append_latents_fp4(p, 2 * w + (lane >> 4), lane);
    else append_latents(p, 2 * w + (lane >> 4), lane);
    return;
  }
  w -= latents;
  if (w < pes) return append_pe<kFp4>(p, 8 * w + (lane >> 2), lane);
  w -= pes;
  const uint32_t parts = (p.H + kHeadsPerWarp - 1) / kHeadsPerWarp, t = parts ? w / parts : p.T;
  if (t < (uint32_t)p.T) turn_heads(p, t, (w - t * parts) * kHeadsPerWarp, lane);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
  const int64_t warps = ((int64_t)p.T + 1) / 2 + ((int64_t)p.T + 7) / 8 + (int64_t)p.T * ((p.H + kHeadsPerWarp - 1) / kHeadsPerWarp);
  const unsigned blocks = (unsigned)((warps + 3) / 4);
  if (p.e4m3 == kCacheFp4) kv_append_kernel<true><<<blocks, 128, 0, stream>>>(p);
  else kv_append_kernel<false><<<blocks, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
