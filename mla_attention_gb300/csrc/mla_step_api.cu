// The C ABI of the serving step's operators: argument validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "mla_step.h"

using namespace mla;

namespace {

mla_status fail(mla_status s, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_last_error(s, msg);
}
mla_status finish(cudaError_t e, const char* name) {
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  return set_last_error(MLA_OK, "");
}
bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// rows of `width` elements at strides st, sh over T tokens and H heads do not overlap
bool rows_apart(int64_t st, int64_t sh, int T, int H, int width) {
  const bool token_major = (H == 1 || sh >= width) && (T == 1 || st >= (int64_t)(H - 1) * sh + width);
  const bool head_major = (T == 1 || st >= width) && (H == 1 || sh >= (int64_t)(T - 1) * st + width);
  return st >= 0 && sh >= 0 && (token_major || head_major);
}

#define MLA_REQUIRE(cond, ...)                            \
  do {                                                    \
    if (!(cond)) return fail(MLA_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

mla_status append_impl(const char* name, int format, const void* c_kv, int64_t c_kv_stride, const void* k_pe, int64_t k_pe_stride,
                       const void* norm_weight, float eps, const void* q_pe, int64_t q_pe_stride_t, int64_t q_pe_stride_h,
                       const int32_t* positions, const int32_t* slots, const float* cos_sin, int max_pos, int is_neox, int T, int H,
                       void* kv_cache, float kv_scale, int64_t num_pages, int page_size, void* q_out, int64_t q_out_stride_t,
                       int64_t q_out_stride_h, void* kv_out, int64_t kv_out_stride, void* workspace, size_t workspace_bytes,
                       void* stream) {
  MLA_REQUIRE(T >= 0 && H >= 0 && max_pos >= 1 && num_pages >= 0 && page_size >= 1,
              "%s: need T >= 0, H >= 0, max_pos >= 1, num_pages >= 0, page_size >= 1", name);
  MLA_REQUIRE(num_pages <= INT32_MAX / page_size, "%s: num_pages * page_size must be below 2^31", name);
  MLA_REQUIRE(is_neox == 0 || is_neox == 1, "%s: is_neox must be 0 or 1", name);
  MLA_REQUIRE(format != kCacheE4m3 || (kv_scale >= 0x1p-126f && kv_scale <= 0x1p126f),
              "%s: kv_scale must be positive and normal, as must its reciprocal", name);
  MLA_REQUIRE(format != kCacheFp4 || (kv_scale >= 0x1p-100f && kv_scale <= 0x1p100f), "%s: kv_scale must be between 2^-100 and 2^100", name);
  MLA_REQUIRE(!norm_weight || (std::isfinite(eps) && eps >= 0.f), "%s: eps must be finite and not negative", name);
  MLA_REQUIRE((int64_t)T * (1 + ((int64_t)H + 15) / 16) <= (int64_t)INT32_MAX - 8, "%s: too many (token, head) rows", name);
  if (!workspace || workspace_bytes < mla_kv_append_workspace_size(T))
    return fail(MLA_ERR_WORKSPACE, "%s: workspace must hold %zu bytes", name, mla_kv_append_workspace_size(T));
  if (T == 0) return finish(cudaSuccess, "");
  MLA_REQUIRE(c_kv && k_pe && positions && slots && cos_sin, "%s: c_kv, k_pe, positions, slots, cos_sin required", name);
  MLA_REQUIRE(num_pages == 0 || kv_cache, "%s: kv_cache required", name);
  MLA_REQUIRE(H == 0 || (q_pe && q_out), "%s: q_pe and q_out required where H > 0", name);
  MLA_REQUIRE(aligned(c_kv, 16) && aligned(k_pe, 16) && aligned(norm_weight, 16) && aligned(kv_cache, 16) &&
                  aligned(cos_sin, 16) && aligned(kv_out, 16) && aligned(positions, 4) && aligned(slots, 4) &&
                  aligned(workspace, 4) && (H == 0 || (aligned(q_pe, 16) && aligned(q_out, 16))),
              "%s: tensors must be 16-byte aligned (int32 ones 4-byte)", name);
  MLA_REQUIRE(c_kv_stride >= 0 && k_pe_stride >= 0 && c_kv_stride % 8 == 0 && k_pe_stride % 8 == 0,
              "%s: row strides of c_kv and k_pe must be multiples of 8 elements", name);
  MLA_REQUIRE(!kv_out || T == 1 || (kv_out_stride >= kDk && kv_out_stride % 8 == 0),
              "%s: kv_out rows need a stride of at least 576, a multiple of 8", name);
  if (H > 0) {
    MLA_REQUIRE(q_pe_stride_t >= 0 && q_pe_stride_h >= 0 && q_pe_stride_t % 8 == 0 && q_pe_stride_h % 8 == 0 &&
                    q_out_stride_t % 8 == 0 && q_out_stride_h % 8 == 0,
                "%s: strides of q_pe and q_out must be multiples of 8 elements", name);
    MLA_REQUIRE(rows_apart(q_out_stride_t, q_out_stride_h, T, H, kDk), "%s: q_out rows of 576 must not overlap", name);
  }
  KvAppendParams p;
  p.c_kv = reinterpret_cast<const __nv_bfloat16*>(c_kv);
  p.k_pe = reinterpret_cast<const __nv_bfloat16*>(k_pe);
  p.weight = reinterpret_cast<const __nv_bfloat16*>(norm_weight);
  p.q_pe = reinterpret_cast<const __nv_bfloat16*>(q_pe);
  p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  p.kv_out = reinterpret_cast<__nv_bfloat16*>(kv_out);
  p.cache = kv_cache;
  p.positions = positions;
  p.slots = slots;
  p.cos_sin = cos_sin;
  p.err = reinterpret_cast<uint32_t*>(workspace);
  p.c_kv_stride = c_kv_stride;
  p.k_pe_stride = k_pe_stride;
  p.q_pe_stride_t = q_pe_stride_t;
  p.q_pe_stride_h = q_pe_stride_h;
  p.q_out_stride_t = q_out_stride_t;
  p.q_out_stride_h = q_out_stride_h;
  p.kv_out_stride = kv_out_stride;
  p.cache_rows = num_pages * page_size;
  p.eps = eps;
  p.kv_scale = kv_scale;
  p.inv_kv_scale = 1.f / kv_scale;
  p.T = T;
  p.H = H;
  p.max_pos = max_pos;
  p.is_neox = is_neox;
  p.e4m3 = format;
  return finish(launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream)), name);
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
size_t mla_slot_map_workspace_size(int B) {
  (void)B;
  return kWsHeader;
}

mla_status mla_slot_map(const int32_t* lens, const int32_t* new_tokens, int B, int32_t* block_table, int max_pages,
                        int page_size, int64_t num_pages, int32_t* pool, const int32_t* pool_state, int N,
                        int32_t* cu_tokens, int32_t* positions, int32_t* slots, int32_t* lens_out,
                        int32_t* pool_state_out, void* workspace, size_t workspace_bytes, void* stream) {
  MLA_REQUIRE(B >= 0 && N >= 0 && max_pages >= 0 && page_size >= 1 && num_pages >= 0,
              "mla_slot_map: need B >= 0, N >= 0, max_pages >= 0, page_size >= 1, num_pages >= 0");
  MLA_REQUIRE(num_pages <= INT32_MAX / page_size, "mla_slot_map: num_pages * page_size must be below 2^31");
  if (!workspace || workspace_bytes < mla_slot_map_workspace_size(B))
    return fail(MLA_ERR_WORKSPACE, "mla_slot_map: workspace must hold %zu bytes", mla_slot_map_workspace_size(B));
  MLA_REQUIRE(pool_state && pool_state_out && cu_tokens, "mla_slot_map: pool_state, pool_state_out, cu_tokens required");
  MLA_REQUIRE(B == 0 || (lens && new_tokens && lens_out), "mla_slot_map: lens, new_tokens, lens_out required");
  MLA_REQUIRE(B == 0 || max_pages == 0 || block_table, "mla_slot_map: block_table required");
  MLA_REQUIRE(num_pages == 0 || pool, "mla_slot_map: pool required");
  MLA_REQUIRE(N == 0 || (positions && slots && positions != slots), "mla_slot_map: positions and slots required");
  for (const void* q : {(const void*)lens, (const void*)new_tokens, (const void*)block_table, (const void*)pool,
                        (const void*)pool_state, (const void*)cu_tokens, (const void*)positions, (const void*)slots,
                        (const void*)lens_out, (const void*)pool_state_out, (const void*)workspace})
    MLA_REQUIRE(aligned(q, 4), "mla_slot_map: buffers must be 4-byte aligned");
  SlotMapParams p;
  p.lens = lens;
  p.new_tokens = new_tokens;
  p.block_table = block_table;
  p.pool = pool;
  p.pool_state = pool_state;
  p.cu_tokens = cu_tokens;
  p.positions = positions;
  p.slots = slots;
  p.lens_out = lens_out;
  p.pool_state_out = pool_state_out;
  p.err = reinterpret_cast<uint32_t*>(workspace);
  p.num_pages = num_pages;
  p.B = B;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.N = N;
  p.page_log2 = -1;
  for (int i = 0; i < 31; ++i)
    if (page_size == 1 << i) p.page_log2 = i;
  return finish(launch_slot_map(p, reinterpret_cast<cudaStream_t>(stream)), "mla_slot_map");
}

// ---------------------------------------------------------------------------
mla_status mla_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                        const void* weight, float eps, int T, int D, void* residual_out, int64_t residual_out_stride,
                        int out_e4m3, int group, void* out, int64_t out_stride, float* scales, void* stream) {
  MLA_REQUIRE(T >= 0 && D >= 1, "mla_rms_norm: need T >= 0, D >= 1 (got %d, %d)", T, D);
  if (D > kNormMaxD) return fail(MLA_ERR_UNSUPPORTED, "mla_rms_norm: D <= %d (got %d)", kNormMaxD, D);
  MLA_REQUIRE(std::isfinite(eps) && eps >= 0.f, "mla_rms_norm: eps must be finite and not negative");
  MLA_REQUIRE(out_e4m3 == 0 || out_e4m3 == 1, "mla_rms_norm: out_e4m3 must be 0 or 1");
  MLA_REQUIRE((out_e4m3 == 1) == (scales != nullptr) || T == 0, "mla_rms_norm: scales go with an e4m3 output, and only with it");
  MLA_REQUIRE(group == 0 || (out_e4m3 && (group == 32 || group == 64 || group == 128) && D % group == 0),
              "mla_rms_norm: group is 0, or with e4m3 32, 64 or 128 dividing D (got %d, D = %d)", group, D);
  MLA_REQUIRE((residual == nullptr) == (residual_out == nullptr), "mla_rms_norm: residual and residual_out go together");
  if (T == 0) return finish(cudaSuccess, "");
  MLA_REQUIRE(x && weight && out, "mla_rms_norm: x, weight and out required");
  MLA_REQUIRE(aligned(x, 2) && aligned(weight, 2) && aligned(residual, 2) && aligned(residual_out, 2) &&
                  aligned(out, out_e4m3 ? 1 : 2) && aligned(scales, 4),
              "mla_rms_norm: tensors must be aligned to their elements");
  MLA_REQUIRE(x_stride >= 0 && residual_stride >= 0, "mla_rms_norm: negative row stride");
  MLA_REQUIRE(T == 1 || (out_stride >= D && (!residual || residual_out_stride >= D)),
              "mla_rms_norm: rows of out and residual_out must not overlap");
  RmsNormParams p;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.residual = reinterpret_cast<const __nv_bfloat16*>(residual);
  p.weight = reinterpret_cast<const __nv_bfloat16*>(weight);
  p.residual_out = reinterpret_cast<__nv_bfloat16*>(residual_out);
  p.out = out;
  p.scales = scales;
  p.x_stride = x_stride;
  p.residual_stride = residual_stride;
  p.residual_out_stride = residual_out_stride;
  p.out_stride = out_stride;
  p.eps = eps;
  p.T = T;
  p.D = D;
  p.group = group ? group : D;
  p.err = guard_word();
  return finish(launch_rms_norm(p, reinterpret_cast<cudaStream_t>(stream)), "mla_rms_norm");
}

// ---------------------------------------------------------------------------
size_t mla_kv_append_workspace_size(int T) {
  (void)T;
  return kWsHeader;
}

mla_status mla_kv_append(const void* c_kv, int64_t c_kv_stride, const void* k_pe, int64_t k_pe_stride,
                         const void* norm_weight, float eps, const void* q_pe, int64_t q_pe_stride_t,
                         int64_t q_pe_stride_h, const int32_t* positions, const int32_t* slots, const float* cos_sin,
                         int max_pos, int is_neox, int T, int H, void* kv_cache, int cache_e4m3, float kv_scale,
                         int64_t num_pages, int page_size, void* q_out, int64_t q_out_stride_t, int64_t q_out_stride_h,
                         void* kv_out, int64_t kv_out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  MLA_REQUIRE(cache_e4m3 == 0 || cache_e4m3 == 1, "mla_kv_append: cache_e4m3 must be 0 or 1");
  return append_impl("mla_kv_append", cache_e4m3, c_kv, c_kv_stride, k_pe, k_pe_stride, norm_weight, eps, q_pe, q_pe_stride_t,
                     q_pe_stride_h, positions, slots, cos_sin, max_pos, is_neox, T, H, kv_cache, kv_scale, num_pages, page_size,
                     q_out, q_out_stride_t, q_out_stride_h, kv_out, kv_out_stride, workspace, workspace_bytes, stream);
}

// its 4-bit rows (the cache's other calls are in mla_cache_api.cu)
size_t mla_kv_append_fp4_workspace_size(int T) { return mla_kv_append_workspace_size(T); }

mla_status mla_kv_append_fp4(const void* c_kv, int64_t c_kv_stride, const void* k_pe, int64_t k_pe_stride,
                             const void* norm_weight, float eps, const void* q_pe, int64_t q_pe_stride_t,
                             int64_t q_pe_stride_h, const int32_t* positions, const int32_t* slots,
                             const float* cos_sin, int max_pos, int is_neox, int T, int H, void* kv_cache_fp4,
                             float kv_scale, int64_t num_pages, int page_size, void* q_out, int64_t q_out_stride_t,
                             int64_t q_out_stride_h, void* kv_out, int64_t kv_out_stride, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return append_impl("mla_kv_append_fp4", kCacheFp4, c_kv, c_kv_stride, k_pe, k_pe_stride, norm_weight, eps, q_pe, q_pe_stride_t,
                     q_pe_stride_h, positions, slots, cos_sin, max_pos, is_neox, T, H, kv_cache_fp4, kv_scale, num_pages, page_size,
                     q_out, q_out_stride_t, q_out_stride_h, kv_out, kv_out_stride, workspace, workspace_bytes, stream);
}

// ---------------------------------------------------------------------------
mla_status mla_bmm_w4(const void* x, int64_t x_stride_t, int64_t x_stride_h, const void* w4, const void* scales,
                      int scales_f32, int group, int T, int H, int N, int K, void* out, int64_t out_stride_t,
                      int64_t out_stride_h, void* workspace, size_t workspace_bytes, void* stream) {
  MLA_REQUIRE(T >= 0 && H >= 1 && N >= 1 && K >= 1, "mla_bmm_w4: need T >= 0, H >= 1, N >= 1, K >= 1");
  MLA_REQUIRE(group == 32 || group == 64 || group == 128, "mla_bmm_w4: group must be 32, 64 or 128 (got %d)", group);
  MLA_REQUIRE(K % group == 0, "mla_bmm_w4: K must be a multiple of the group (got %d, %d)", K, group);
  MLA_REQUIRE(scales_f32 == 0 || scales_f32 == 1, "mla_bmm_w4: scales_f32 must be 0 or 1");
  MLA_REQUIRE((int64_t)H * N <= INT32_MAX && T <= kW4MaxT && H <= 65535 && K <= kW4MaxK,
              "mla_bmm_w4: H <= 65535, H * N below 2^31, T <= %d and K <= %d", kW4MaxT, kW4MaxK);
  if (!workspace || workspace_bytes < kWsHeader) return fail(MLA_ERR_WORKSPACE, "mla_bmm_w4: workspace must hold %zu bytes", (size_t)kWsHeader);
  if (T == 0) return finish(cudaSuccess, "");
  MLA_REQUIRE(x && w4 && scales && out, "mla_bmm_w4: every tensor is required");
  MLA_REQUIRE(aligned(x, 2) && aligned(out, 2) && aligned(scales, scales_f32 ? 4 : 2) && aligned(w4, 16) && aligned(workspace, 4),
              "mla_bmm_w4: w4 must be 16-byte aligned, the other tensors to their elements");
  MLA_REQUIRE(x_stride_t >= 0 && x_stride_h >= 0, "mla_bmm_w4: negative stride of x");
  MLA_REQUIRE(rows_apart(out_stride_t, out_stride_h, T, H, N), "mla_bmm_w4: rows of out must not overlap");
  BmmW4Params p;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.w4 = reinterpret_cast<const uint8_t*>(w4);
  p.scales = scales;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.x_stride_t = x_stride_t;
  p.x_stride_h = x_stride_h;
  p.out_stride_t = out_stride_t;
  p.out_stride_h = out_stride_h;
  p.T = T;
  p.H = H;
  p.N = N;
  p.K = K;
  p.group = group;
  p.scales_f32 = scales_f32;
  p.err = reinterpret_cast<uint32_t*>(workspace);
  p.spin_limit = spin_limit();
  return finish(launch_bmm_w4(p, reinterpret_cast<cudaStream_t>(stream)), "mla_bmm_w4");
}

}  // extern "C"
