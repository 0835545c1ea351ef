// The C ABI of the smaller cache: argument validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "mla_cache.h"

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
bool scale_ok(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }

#define MLA_REQUIRE(cond, ...)                            \
  do {                                                    \
    if (!(cond)) return fail(MLA_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

// what the paged calls share: sizes first, then (with requests) the pointers
mla_status check_paged(const char* name, const PagedRows& kv) {
  MLA_REQUIRE(kv.B >= 0 && kv.num_pages >= 0 && kv.max_pages >= 0 && kv.page_size >= 1,
              "%s: need B >= 0, num_pages >= 0, max_pages >= 0, page_size >= 1", name);
  MLA_REQUIRE(kv.num_pages <= INT32_MAX / kv.page_size, "%s: num_pages * page_size must be below 2^31", name);
  MLA_REQUIRE((int64_t)kv.max_pages * kv.page_size <= INT32_MAX - 65536, "%s: max_pages * page_size must be below 2^31 - 2^16", name);
  MLA_REQUIRE(kv.B == 0 || kv.max_pages == 0 || kv.block_table, "%s: block_table required", name);
  MLA_REQUIRE(kv.B == 0 || kv.num_pages == 0 || kv.cache, "%s: the cache is required", name);
  MLA_REQUIRE(aligned(kv.cache, 16) && aligned(kv.block_table, 4) && aligned(kv.lens, 4),
              "%s: the cache must be 16-byte aligned, block_table and lens 4-byte", name);
  return MLA_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
size_t mla_decode_fp4_workspace_size(int B, int q_per_req, int H, int num_splits) {
  if (B < 0 || q_per_req < 1 || H < 1 || num_splits < 0) return kWsHeader;
  const DecodeFp4Scratch w = decode_fp4_scratch(B, q_per_req, H, num_splits);
  return kWsHeader + w.before + w.part_stat + w.part_o;
}

mla_status mla_decode_fp4(const void* q, int q_per_req, const void* kv_cache_fp4, float kv_scale, int64_t num_pages,
                          int page_size, const int32_t* block_table, int max_pages, const int32_t* lens, int B, int H,
                          float scale, const float* sinks, int num_splits, void* out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const PagedRows kv = {reinterpret_cast<const uint8_t*>(kv_cache_fp4), block_table, lens, num_pages, max_pages, page_size, B, kFp4Row};
  if (mla_status s = check_paged("mla_decode_fp4", kv)) return s;
  MLA_REQUIRE(H >= 1 && q_per_req >= 1 && num_splits >= 0 && num_splits <= 65535,
              "mla_decode_fp4: need H >= 1, q_per_req >= 1, 0 <= num_splits <= 65535");
  MLA_REQUIRE((int64_t)B * q_per_req <= (int64_t)1 << 24, "mla_decode_fp4: B * q_per_req <= 2^24 (got %d, %d)", B, q_per_req);
  if (H > kRows) return fail(MLA_ERR_UNSUPPORTED, "mla_decode_fp4: H <= 128 (got %d)", H);
  MLA_REQUIRE(std::isfinite(scale) && scale_ok(kv_scale), "mla_decode_fp4: scale must be finite, kv_scale between 2^-100 and 2^100");
  const size_t need = mla_decode_fp4_workspace_size(B, q_per_req, H, num_splits);
  if (!workspace || workspace_bytes < need) return fail(MLA_ERR_WORKSPACE, "mla_decode_fp4: workspace must hold %zu bytes", need);
  if (B == 0) return finish(cudaSuccess, "");
  MLA_REQUIRE(q && lens && out, "mla_decode_fp4: q, lens and out required");
  MLA_REQUIRE(aligned(q, 16) && aligned(out, 16) && aligned(lse, 4) && aligned(sinks, 4) && aligned(workspace, 16),
              "mla_decode_fp4: q, out and the workspace must be 16-byte aligned, lse and sinks 4-byte");
  DecodeFp4Params p;
  p.kv = kv;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.sinks = sinks;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = reinterpret_cast<uint32_t*>(workspace);
  p.scale = scale * kv_scale;
  p.kv_scale = kv_scale;
  p.spin_limit = spin_limit();
  p.debug_stall = debug_stall();
  p.s = q_per_req;
  p.H = H;
  const DecodeFp4Scratch w = decode_fp4_scratch(B, q_per_req, H, num_splits);
  p.row_tiles = w.row_tiles;
  p.part_rows = w.part_rows;
  p.groups = w.groups;
  char* at = reinterpret_cast<char*>(workspace) + kWsHeader;
  p.before = reinterpret_cast<int64_t*>(at);
  p.part_stat = reinterpret_cast<float*>(at + w.before);
  p.part_o = reinterpret_cast<float*>(at + w.before + w.part_stat);
  p.part_stat_bytes = w.part_stat;
  p.part_o_bytes = w.part_o;
  return finish(launch_decode_fp4(p, w.pairs, reinterpret_cast<cudaStream_t>(stream)), "mla_decode_fp4");
}

// ---------------------------------------------------------------------------
size_t mla_key_weights_workspace_size(int B, int q_per_req, int H, int width) {
  size_t before;
  const size_t part = key_weights_scratch(B, (int64_t)q_per_req * H, width, &before);
  return kWsHeader + (before + 255) / 256 * 256 + part;
}

mla_status mla_key_weights(const void* q, int q_per_req, const float* lse, const void* kv_cache, int cache_format,
                           float kv_scale, int64_t num_pages, int page_size, const int32_t* block_table, int max_pages,
                           const int32_t* lens, int B, int H, float scale, float decay, float* weights,
                           int64_t weights_stride, int width, void* workspace, size_t workspace_bytes, void* stream) {
  MLA_REQUIRE(cache_format >= 0 && cache_format <= 2, "mla_key_weights: cache_format must be 0, 1 or 2 (got %d)", cache_format);
  const int row_bytes = cache_format == 0 ? 2 * kDk : cache_format == 1 ? kDk : kFp4Row;
  const PagedRows kv = {reinterpret_cast<const uint8_t*>(kv_cache), block_table, lens, num_pages, max_pages, page_size, B, row_bytes};
  if (mla_status s = check_paged("mla_key_weights", kv)) return s;
  MLA_REQUIRE(H >= 1 && q_per_req >= 1 && (int64_t)q_per_req * H <= 1 << 20,
              "mla_key_weights: need H >= 1, q_per_req >= 1, q_per_req * H <= 2^20 (got %d, %d)", H, q_per_req);
  MLA_REQUIRE(std::isfinite(scale) && scale_ok(kv_scale), "mla_key_weights: scale must be finite, kv_scale between 2^-100 and 2^100");
  MLA_REQUIRE(std::isfinite(decay) && decay >= 0.f, "mla_key_weights: decay must be finite and not negative");
  MLA_REQUIRE(width >= 0 && weights_stride >= 0, "mla_key_weights: need width >= 0 and weights_stride >= 0");
  MLA_REQUIRE(B <= 65535, "mla_key_weights: B <= 65535 (got %d)", B);
  const size_t need = mla_key_weights_workspace_size(B, q_per_req, H, width);
  if (!workspace || workspace_bytes < need) return fail(MLA_ERR_WORKSPACE, "mla_key_weights: workspace must hold %zu bytes", need);
  if (B == 0) return finish(cudaSuccess, "");
  MLA_REQUIRE(q && lse && lens && (weights || width == 0), "mla_key_weights: q, lse, lens and weights required");
  MLA_REQUIRE(aligned(q, 16) && aligned(lse, 4) && aligned(weights, 4) && aligned(workspace, 4),
              "mla_key_weights: q must be 16-byte aligned, lse and weights 4-byte");
  MLA_REQUIRE(B == 1 || weights_stride >= width, "mla_key_weights: rows of weights must not overlap");
  KeyWeightsParams p;
  p.kv = kv;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.lse = lse;
  p.weights = weights;
  p.stride = weights_stride;
  p.err = reinterpret_cast<uint32_t*>(workspace);
  p.scale = scale * kv_scale;
  p.decay = decay;
  p.spin_limit = spin_limit();
  p.debug_stall = debug_stall();
  p.format = cache_format;
  p.s = q_per_req;
  p.H = H;
  p.width = width;
  size_t before;
  p.part_bytes = key_weights_scratch(B, (int64_t)q_per_req * H, width, &before);
  p.before = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(workspace) + kWsHeader);
  p.part = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kWsHeader + (before + 255) / 256 * 256);
  return finish(launch_key_weights(p, reinterpret_cast<cudaStream_t>(stream)), "mla_key_weights");
}

// ---------------------------------------------------------------------------
size_t mla_select_keys_workspace_size(int B) {
  (void)B;
  return kWsHeader;
}

mla_status mla_select_keys(const float* weights, int64_t weights_stride, int width, const int32_t* lens,
                           const int32_t* keep, int first, int recent, int B, int K, int32_t* idx, int32_t* count,
                           int32_t* dropped, void* workspace, size_t workspace_bytes, void* stream) {
  MLA_REQUIRE(B >= 0 && K >= 0 && width >= 0 && first >= 0 && recent >= 0 && weights_stride >= 0,
              "mla_select_keys: need B, K, width, first, recent, weights_stride >= 0");
  MLA_REQUIRE(K <= INT32_MAX - 65536 && width <= INT32_MAX - 65536, "mla_select_keys: K and width must be below 2^31 - 2^16");
  if (!workspace || workspace_bytes < kWsHeader) return fail(MLA_ERR_WORKSPACE, "mla_select_keys: workspace must hold %zu bytes", (size_t)kWsHeader);
  if (B == 0) return finish(cudaSuccess, "");
  MLA_REQUIRE((weights || width == 0) && lens && keep && (idx || K == 0) && count && dropped,
              "mla_select_keys: weights, lens, keep, idx, count and dropped required");
  MLA_REQUIRE(aligned(weights, 4) && aligned(lens, 4) && aligned(keep, 4) && aligned(idx, 4) && aligned(count, 4) &&
                  aligned(dropped, 4) && aligned(workspace, 4), "mla_select_keys: tensors must be 4-byte aligned");
  SelectParams p;
  p.weights = weights;
  p.lens = lens;
  p.keep = keep;
  p.idx = idx;
  p.count = count;
  p.dropped = dropped;
  p.err = reinterpret_cast<uint32_t*>(workspace);
  p.stride = weights_stride;
  p.width = width;
  p.first = first;
  p.recent = recent;
  p.B = B;
  p.K = K;
  return finish(launch_select_keys(p, reinterpret_cast<cudaStream_t>(stream)), "mla_select_keys");
}

// ---------------------------------------------------------------------------
size_t mla_compact_rows_workspace_size(int B) {
  (void)B;
  return kWsHeader;
}

mla_status mla_compact_rows(void* kv_cache, int row_bytes, int64_t num_pages, int page_size, const int32_t* block_table,
                            int max_pages, const int32_t* idx, int K, const int32_t* count, int B, float* weights,
                            int64_t weights_stride, int width, void* workspace, size_t workspace_bytes, void* stream) {
  MLA_REQUIRE(row_bytes >= 16 && row_bytes <= 65536 && row_bytes % 16 == 0,
              "mla_compact_rows: row_bytes must be a multiple of 16 up to 65536 (got %d)", row_bytes);
  const PagedRows kv = {reinterpret_cast<const uint8_t*>(kv_cache), block_table, nullptr, num_pages, max_pages, page_size, B, row_bytes};
  if (mla_status s = check_paged("mla_compact_rows", kv)) return s;
  MLA_REQUIRE(K >= 0 && width >= 0 && weights_stride >= 0, "mla_compact_rows: need K, width, weights_stride >= 0");
  MLA_REQUIRE(B <= 65535, "mla_compact_rows: B <= 65535 (got %d)", B);
  if (!workspace || workspace_bytes < kWsHeader) return fail(MLA_ERR_WORKSPACE, "mla_compact_rows: workspace must hold %zu bytes", (size_t)kWsHeader);
  if (B == 0 || K == 0) return finish(cudaSuccess, "");
  MLA_REQUIRE(idx && count, "mla_compact_rows: idx and count required");
  MLA_REQUIRE(aligned(idx, 4) && aligned(count, 4) && aligned(weights, 4) && aligned(workspace, 4),
              "mla_compact_rows: idx, count and weights must be 4-byte aligned");
  MLA_REQUIRE(!weights || B == 1 || weights_stride >= width, "mla_compact_rows: rows of weights must not overlap");
  CompactParams p;
  p.kv = kv;
  p.idx = idx;
  p.count = count;
  p.weights = weights;
  p.err = reinterpret_cast<uint32_t*>(workspace);
  p.spin_limit = spin_limit();
  p.debug_stall = debug_stall();
  p.stride = weights_stride;
  p.K = K;
  p.width = width;
  return finish(launch_compact_rows(p, reinterpret_cast<cudaStream_t>(stream)), "mla_compact_rows");
}

}  // extern "C"
