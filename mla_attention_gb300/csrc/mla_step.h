// The serving step around the latent attention: parameters and launchers of the slot map, the RMS
// norm, the cache append by slots and the products with 4-bit weights.
#pragma once
#include "mla_cache.h"

namespace mla {

// block tables, positions and slots of one step's tokens, from request lengths
struct SlotMapParams {
  const int32_t* lens;        // [B] tokens held before the step
  const int32_t* new_tokens;  // [B] tokens appended (> 0) or dropped (< 0)
  int32_t* block_table;       // [B, max_pages]
  int32_t* pool;              // [num_pages] ring of free page ids
  const int32_t* pool_state;  // [2] ring head, free pages
  int32_t* cu_tokens;         // [B + 1]
  int32_t* positions;         // [N]
  int32_t* slots;             // [N]
  int32_t* lens_out;          // [B], may be lens
  int32_t* pool_state_out;    // [2], may be pool_state
  uint32_t* err;
  int64_t num_pages;
  int B, max_pages, page_size, N;
  int page_log2;              // of page_size, -1 if it is not a power of two
};
cudaError_t launch_slot_map(const SlotMapParams& p, cudaStream_t stream);

// y = h / sqrt(mean(h^2) + eps) * w with h = x (+ residual), out in bf16 or e4m3 with scales
struct RmsNormParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* residual;      // nullable
  const __nv_bfloat16* weight;        // [D]
  __nv_bfloat16* residual_out;        // with residual
  void* out;                          // bf16, or e4m3 with scales
  float* scales;                      // [T, groups] or null (bf16 out)
  uint32_t* err;                      // guarded build: guard_word(), else null
  int64_t x_stride, residual_stride, residual_out_stride, out_stride;  // elements
  float eps;
  int T, D;
  int group;                          // columns per scale (D: one a row)
};
constexpr int kNormMaxD = 32768;    // a row's values stay in one CTA's registers
cudaError_t launch_rms_norm(const RmsNormParams& p, cudaStream_t stream);

// cache rows [norm(c_kv) w | rotated k_pe] by slot, rotated q_pe into the fused query
struct KvAppendParams {
  const __nv_bfloat16* c_kv;       // [T, 512] rows
  const __nv_bfloat16* k_pe;       // [T, 64] rows
  const __nv_bfloat16* weight;     // [512] or null (no norm)
  const __nv_bfloat16* q_pe;       // [T, H, 64] or null
  __nv_bfloat16* q_out;            // [T, H, >= 576], columns 512..575 written
  __nv_bfloat16* kv_out;           // [T, 576] rows or null
  void* cache;                     // [num_pages * page_size, 576] bf16 or e4m3, or 4-bit rows of 416 bytes
  const int32_t* positions;        // [T]
  const int32_t* slots;            // [T]
  const float* cos_sin;            // [max_pos, 64]
  uint32_t* err;
  int64_t c_kv_stride, k_pe_stride, q_pe_stride_t, q_pe_stride_h, q_out_stride_t, q_out_stride_h, kv_out_stride;
  int64_t cache_rows;
  float eps, kv_scale, inv_kv_scale;
  int T, H, max_pos, is_neox;
  int e4m3;                        // a CacheFormat
};
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream);

// out[t, h, n] = sum_k x[t, h, k] (code[h, n, k] - 8) scale[h, n, k / group]
struct BmmW4Params {
  const __nv_bfloat16* x;
  const uint8_t* w4;            // [H, N, K / 2], even k in the low half of a byte
  const void* scales;           // [H, N, K / group] bf16 or fp32
  __nv_bfloat16* out;
  int64_t x_stride_t, x_stride_h, out_stride_t, out_stride_h;  // elements
  uint32_t* err;
  uint32_t spin_limit;
  int T, H, N, K, group, scales_f32;
};
struct W4Plan {
  int cluster;     // CTAs along k
  int rounds;      // of 128 columns a CTA does one after another
  int blocks_h;    // CTAs of a head's columns
  int vec_x;       // x rows on 16-byte boundaries
  int vec_out;     // out rows on 16-byte boundaries
  int vec_s;       // scales likewise (bf16 ones on 8-byte boundaries)
};
constexpr int kW4MaxT = 1 << 19, kW4MaxK = 1 << 30;
cudaError_t launch_bmm_w4(const BmmW4Params& p, cudaStream_t stream);

}  // namespace mla
