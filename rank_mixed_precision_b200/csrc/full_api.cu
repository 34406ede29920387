// C entry points of full-width layers (include/starkv_full.h): argument checks and launches.
#include <algorithm>
#include <cstdint>

#include "full.cuh"

using namespace starkv;

namespace {

constexpr int kMaxGrid = 65535;         // grid.y and grid.z
constexpr int kMaxPages = 1 << 26;      // 16 tokens each: token indices stay in int32
constexpr int64_t kMaxBlocks = 0x7fffffff;

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

starkv_status check_ctx(const starkv_ctx* ctx) {
  if (!ctx) return fail(STARKV_ERR_INVALID_ARG, "ctx is NULL");
  int device = -1;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const int want = reinterpret_cast<const Ctx*>(ctx)->device;
  if (device != want)
    return fail(STARKV_ERR_INVALID_ARG, "the context is device %d's, the current device is %d", want, device);
  return STARKV_OK;
}

starkv_status check_cache(const starkv_kv4_cache* cache) {
  if (!cache) return fail(STARKV_ERR_INVALID_ARG, "cache is NULL");
  if (cache->n_pages < 0) return fail(STARKV_ERR_INVALID_ARG, "cache.n_pages < 0");
  if (cache->n_pages > 0 && !cache->pages) return fail(STARKV_ERR_INVALID_ARG, "cache.pages is NULL");
  if (!aligned(cache->pages, 16) || !aligned(cache->weights, 16))
    return fail(STARKV_ERR_INVALID_ARG, "cache.pages and cache.weights must be 16-byte aligned");
  return STARKV_OK;
}

starkv_status check_sizes(int32_t batch, int32_t max_pages) {
  if (batch < 0 || max_pages < 0) return fail(STARKV_ERR_INVALID_ARG, "negative size");
  if (batch > kMaxGrid) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "batch %d: at most %d", batch, kMaxGrid);
  if (max_pages > kMaxPages) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "max_pages %d: at most %d", max_pages, kMaxPages);
  return STARKV_OK;
}

starkv_status check_tables(int32_t batch, int32_t max_pages) {
  const starkv_status st = check_sizes(batch, max_pages);
  if (st) return st;
  if (batch > 0 && max_pages == 0) return fail(STARKV_ERR_INVALID_ARG, "max_pages must be >= 1");
  return STARKV_OK;
}

starkv_status check_rows(const void* p, int64_t stride, int64_t width, const char* name) {
  if (!p) return fail(STARKV_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 16)) return fail(STARKV_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  // a row's bytes stay below the 2^40 of a tensor map's stride
  if (stride < width || stride % 8 != 0 || stride >= (int64_t)1 << 38)
    return fail(STARKV_ERR_INVALID_ARG, "%s_stride %lld: need a multiple of 8, >= %lld", name, (long long)stride,
                (long long)width);
  return STARKV_OK;
}

starkv_status check_packed(const Ctx* c, const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                           const int32_t* cu_q, const int32_t* cu_k, int64_t total_q, int64_t total_k) {
  const starkv_config& f = c->cfg;
  if (!cu_q || !cu_k) return fail(STARKV_ERR_INVALID_ARG, "cu_q or cu_k is NULL");
  starkv_status st = STARKV_OK;
  if (total_q > 0) st = check_rows(q, q_stride, (int64_t)f.num_q_heads * f.head_dim, "q");
  if (!st && total_k > 0) st = check_rows(k, k_stride, (int64_t)f.num_kv_heads * f.head_dim, "k");
  return st;
}

}  // namespace

namespace starkv {
starkv_status full_workspace_bytes(const Ctx& c, int op, int batch, int max_pages, int64_t total_q, size_t* out) {
  if (op != STARKV_OP_KV4_DECODE) return fail(STARKV_ERR_INVALID_ARG, "unknown op %d", op);
  const starkv_status st = check_sizes(batch, max_pages);
  if (st) return st;
  *out = plan_kv4_decode(c, batch, max_pages, total_q != 0).ws_bytes;
  return ok();
}
}  // namespace starkv

extern "C" {

starkv_status starkv_kv4_layout(const starkv_config* cfg, int64_t n_pages, starkv_kv4_sizes* out) {
  starkv_status st = check_config(cfg, nullptr, nullptr);
  if (st) return st;
  if (!out) return fail(STARKV_ERR_INVALID_ARG, "out is NULL");
  if (n_pages < 0) return fail(STARKV_ERR_INVALID_ARG, "n_pages < 0");
  if (n_pages > INT64_MAX / cfg->num_kv_heads / kv4_page_bytes(cfg->head_dim))
    return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "n_pages %lld: 2^63 bytes or more", (long long)n_pages);
  out->head_page_bytes = kv4_page_bytes(cfg->head_dim);
  out->groups = cfg->head_dim / STARKV_KV4_GROUP;
  out->pages_bytes = n_pages * cfg->num_kv_heads * out->head_page_bytes;
  out->weights_bytes = n_pages * cfg->num_kv_heads * kPage * 4;
  return ok();
}

starkv_status starkv_kv4_append(starkv_ctx* ctx, const starkv_kv4_cache* cache, const void* k, const void* v,
                                int64_t k_stride, int64_t v_stride, const int64_t* slot_mapping, const float* weights,
                                int64_t n, starkv_stream_t stream) {
  starkv_status st = check_ctx(ctx);
  if (!st) st = check_cache(cache);
  if (st) return st;
  const Ctx* c = reinterpret_cast<const Ctx*>(ctx);
  if (n < 0) return fail(STARKV_ERR_INVALID_ARG, "n < 0");
  if (n == 0) return ok();
  const int64_t width = (int64_t)c->cfg.num_kv_heads * c->cfg.head_dim;
  st = check_rows(k, k_stride, width, "k");
  if (!st) st = check_rows(v, v_stride, width, "v");
  if (st) return st;
  if (!slot_mapping) return fail(STARKV_ERR_INVALID_ARG, "slot_mapping is NULL");
  if (cache->n_pages == 0) return fail(STARKV_ERR_INVALID_ARG, "cache has no pages");
  if (n > kMaxBlocks * 16 / width) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "n %lld: too many tokens", (long long)n);
  const cudaError_t e =
      launch_kv4_append(*c, *cache, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, k_stride, v_stride, slot_mapping,
                        weights, n, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv4 append launch");
  return ok();
}

starkv_status starkv_kv4_read(starkv_ctx* ctx, const starkv_kv4_cache* cache, const int32_t* block_table,
                              const int32_t* starts, const int32_t* cu, int32_t batch, int32_t max_pages,
                              int64_t total, void* k_out, void* v_out, starkv_stream_t stream) {
  starkv_status st = check_ctx(ctx);
  if (!st) st = check_cache(cache);
  if (!st) st = check_tables(batch, max_pages);
  if (st) return st;
  const Ctx* c = reinterpret_cast<const Ctx*>(ctx);
  if (total < 0) return fail(STARKV_ERR_INVALID_ARG, "total < 0");
  if (total == 0) return ok();
  if (batch == 0) return fail(STARKV_ERR_INVALID_ARG, "rows of no sequence");
  if (!block_table || !cu || !k_out || !v_out) return fail(STARKV_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(STARKV_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  if (total > kMaxBlocks) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "total %lld: too many tokens", (long long)total);
  const cudaError_t e = launch_kv4_read(*c, *cache, block_table, starts, cu, batch, max_pages, total,
                                        (__nv_bfloat16*)k_out, (__nv_bfloat16*)v_out, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv4 read launch");
  return ok();
}

starkv_status starkv_kv4_decode_attn(starkv_ctx* ctx, const starkv_kv4_cache* cache, const void* q,
                                     const int32_t* block_table, const int32_t* seq_lens, int32_t batch,
                                     int32_t max_pages, int32_t accumulate, void* out, void* workspace,
                                     size_t workspace_bytes, starkv_stream_t stream) {
  starkv_status st = check_ctx(ctx);
  if (!st) st = check_cache(cache);
  if (!st) st = check_tables(batch, max_pages);
  if (st) return st;
  const Ctx* c = reinterpret_cast<const Ctx*>(ctx);
  if (batch == 0) return ok();
  if (!q || !block_table || !seq_lens || !out) return fail(STARKV_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(STARKV_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (accumulate && !cache->weights && cache->n_pages > 0)
    return fail(STARKV_ERR_INVALID_ARG, "accumulate without cache.weights");
  const Kv4DecodePlan plan = plan_kv4_decode(*c, batch, max_pages, accumulate != 0);
  if (plan.ws_bytes > 0 && (!workspace || workspace_bytes < plan.ws_bytes))
    return fail(STARKV_ERR_WORKSPACE_TOO_SMALL, "decode needs %zu workspace bytes, got %zu", plan.ws_bytes,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned(workspace, 256)) return fail(STARKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const cudaError_t e =
      launch_kv4_decode(*c, *cache, (const __nv_bfloat16*)q, block_table, seq_lens, batch, max_pages, accumulate != 0,
                        (__nv_bfloat16*)out, workspace, plan, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv4 decode launch");
  return ok();
}

starkv_status starkv_kv4_evict(starkv_ctx* ctx, const starkv_kv4_cache* cache, const int32_t* block_table,
                               const int32_t* seq_lens, const int32_t* keep_lens, int32_t recent, int32_t batch,
                               int32_t max_pages, const int32_t* dst_block_table, int32_t dst_max_pages,
                               int32_t* new_lens, int32_t* kept, starkv_stream_t stream) {
  starkv_status st = check_ctx(ctx);
  if (!st) st = check_cache(cache);
  if (!st) st = check_tables(batch, max_pages);
  if (!st) st = check_tables(batch, dst_max_pages);
  if (st) return st;
  const Ctx* c = reinterpret_cast<const Ctx*>(ctx);
  if (recent < 0) return fail(STARKV_ERR_INVALID_ARG, "recent < 0");
  if (batch == 0) return ok();
  if (!block_table || !seq_lens || !keep_lens || !dst_block_table || !new_lens || !kept)
    return fail(STARKV_ERR_INVALID_ARG, "NULL argument");
  if (!cache->weights && cache->n_pages > 0) return fail(STARKV_ERR_INVALID_ARG, "the cache keeps no weights");
  const cudaError_t e = launch_kv4_evict(*c, *cache, block_table, seq_lens, keep_lens, recent, batch, max_pages,
                                         dst_block_table, dst_max_pages, new_lens, kept, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv4 eviction launch");
  return ok();
}

starkv_status starkv_prompt_attn(starkv_ctx* ctx, const void* q, const void* k, const void* v, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k,
                                 int32_t batch, int64_t total_q, int64_t total_k, int32_t max_q_len, void* out,
                                 float* lse, void* workspace, size_t workspace_bytes, starkv_stream_t stream) {
  starkv_status st = check_ctx(ctx);
  if (st) return st;
  const Ctx* c = reinterpret_cast<const Ctx*>(ctx);
  if (batch < 0 || total_q < 0 || total_k < 0 || max_q_len < 0) return fail(STARKV_ERR_INVALID_ARG, "negative size");
  if (batch > kMaxGrid) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "batch %d: at most %d", batch, kMaxGrid);
  if (total_q > 0x7fffffff || total_k > 0x7fffffff) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "2^31 rows or more");
  if (total_q == 0) return ok();
  if (batch == 0 || max_q_len == 0) return fail(STARKV_ERR_INVALID_ARG, "queries of no sequence");
  st = check_packed(c, q, k, q_stride, k_stride, cu_q, cu_k, total_q, total_k);
  if (!st && total_k > 0) st = check_rows(v, v_stride, (int64_t)c->cfg.num_kv_heads * c->cfg.head_dim, "v");
  if (st) return st;
  if (!out || !aligned(out, 16) || !aligned(lse, 4))
    return fail(STARKV_ERR_INVALID_ARG, "out must be given and 16-byte aligned, lse 4-byte");
  max_q_len = (int32_t)std::min<int64_t>(max_q_len, total_q);  // a loose bound launches no blocks of its own
  const PromptPlan plan = plan_prompt(*c, batch, total_q, total_k, max_q_len);
  if (plan.blocks > kMaxBlocks) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "too many blocks");
  if (plan.ws_bytes > 0 && (!workspace || workspace_bytes < plan.ws_bytes))
    return fail(STARKV_ERR_WORKSPACE_TOO_SMALL, "prompt attention needs %zu workspace bytes, got %zu", plan.ws_bytes,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned(workspace, 256)) return fail(STARKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  PromptArgs a{(const __nv_bfloat16*)q, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, q_stride, k_stride, v_stride,
               cu_q, cu_k, batch, total_q, total_k};
  const cudaError_t e = launch_prompt_attn(*c, a, max_q_len, (__nv_bfloat16*)out, lse, workspace, plan,
                                           (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "prompt attention launch");
  return ok();
}

starkv_status starkv_prompt_weights(starkv_ctx* ctx, const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                                    const float* lse, const int32_t* cu_q, const int32_t* cu_k, int32_t batch,
                                    int64_t total_q, int64_t total_k, int32_t max_k_len, int32_t window,
                                    float* weights, starkv_stream_t stream) {
  starkv_status st = check_ctx(ctx);
  if (st) return st;
  const Ctx* c = reinterpret_cast<const Ctx*>(ctx);
  if (batch < 0 || total_q < 0 || total_k < 0 || max_k_len < 0 || window < 0)
    return fail(STARKV_ERR_INVALID_ARG, "negative size");
  if (batch > kMaxGrid) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "batch %d: at most %d", batch, kMaxGrid);
  if (total_q > 0x7fffffff || total_k > 0x7fffffff) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "2^31 rows or more");
  if (total_k == 0) return ok();
  if (batch == 0 || max_k_len == 0) return fail(STARKV_ERR_INVALID_ARG, "keys of no sequence");
  st = check_packed(c, q, k, q_stride, k_stride, cu_q, cu_k, total_q, total_k);
  if (st) return st;
  if ((total_q > 0 && !lse) || !weights || !aligned(lse, 4) || !aligned(weights, 4))
    return fail(STARKV_ERR_INVALID_ARG, "lse and weights must be given and 4-byte aligned");
  max_k_len = (int32_t)std::min<int64_t>(max_k_len, total_k);
  if (weights_items(*c, batch, max_k_len) > kMaxBlocks) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "too many key tiles");
  PromptArgs a{(const __nv_bfloat16*)q, (const __nv_bfloat16*)k, nullptr, q_stride, k_stride, 0, cu_q, cu_k, batch,
               total_q, total_k};
  const cudaError_t e = launch_prompt_weights(*c, a, lse, max_k_len, window, weights, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "prompt weights launch");
  return ok();
}

starkv_status starkv_prompt_workspace_bytes(const starkv_ctx* ctx, int32_t batch, int64_t total_q, int64_t total_k,
                                            size_t* out) {
  if (!ctx || !out) return fail(STARKV_ERR_INVALID_ARG, "NULL argument");
  if (batch < 0 || total_q < 0 || total_k < 0) return fail(STARKV_ERR_INVALID_ARG, "negative size");
  if (batch > kMaxGrid) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "batch %d: at most %d", batch, kMaxGrid);
  if (total_q > 0x7fffffff || total_k > 0x7fffffff) return fail(STARKV_ERR_UNSUPPORTED_SHAPE, "2^31 rows or more");
  *out = batch == 0 || total_q == 0 ? 0 : plan_prompt(*reinterpret_cast<const Ctx*>(ctx), batch, total_q, total_k, 1).ws_bytes;
  return ok();
}

}  // extern "C"
