// Full-width layers: the 4-bit cache's page layout, argument blocks and launchers.
#pragma once

#include "../../include/starkv_full.h"
#include "internal.cuh"

namespace starkv {

// One KV head's part of a 4-bit page (include/starkv_full.h): four planes, each
// token by token, so that a token's codes are whole sectors (an append or an
// eviction touches no other token's) and a page of one head is one contiguous
// block for a bulk copy.  A K row keeps word (c, group) at c * NG + group: the
// thread that holds columns 2c, 2c+1, 2c+8, 2c+9 of every k-step of an
// m16n8k16 A operand then reads its codes of all groups with one load.
template <int D>
struct Kv4 {
  static constexpr int kGroups = D / STARKV_KV4_GROUP;
  static constexpr int kRow = D / 2;                // code bytes of a token, K or V
  static constexpr int kMetaRow = kGroups * 4;      // metadata bytes of a token, K or V
  static constexpr int kV = kPage * kRow;           // V codes
  static constexpr int kKMeta = 2 * kPage * kRow;   // K metadata
  static constexpr int kVMeta = kKMeta + kPage * kMetaRow;
  static constexpr int kBytes = kVMeta + kPage * kMetaRow;
};

inline int kv4_page_bytes(int d) { return kPage * d + 2 * kPage * 4 * (d / STARKV_KV4_GROUP); }

// 2^x on the special function unit (2^-22 relative; results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Work laid end to end and cut evenly: the position at which CTA c's stretch begins, and the CTA
// whose stretch holds position x < total.  Where there are fewer positions than CTAs, the last CTAs
// have none: no stretch between two others is empty.
__device__ __forceinline__ int64_t cut(int64_t c, int64_t total, int ctas) {
  return total <= ctas ? min(c, total) : c * total / ctas;
}
__device__ __forceinline__ int64_t cta_of(int64_t x, int64_t total, int ctas) {
  if (total <= ctas) return x;
  const int64_t y = (x + 1) * ctas - 1;
  // (a division in 64 bits is hundreds of cycles of a join's short life)
  return (y | total) >> 32 == 0 ? (int64_t)((uint32_t)y / (uint32_t)total) : y / total;
}

inline int sm_count(const Ctx& c) {
  int n = 148;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, c.device);
  return n;
}

struct Kv4Pool {
  uint8_t* pages;
  float* weights;
  int64_t n_pages;
  int h_kv;
};

// ---- kv4.cu
cudaError_t launch_kv4_append(const Ctx& c, const starkv_kv4_cache& cache, const __nv_bfloat16* k,
                              const __nv_bfloat16* v, int64_t k_stride, int64_t v_stride, const int64_t* slots,
                              const float* weights, int64_t n, cudaStream_t s);
cudaError_t launch_kv4_read(const Ctx& c, const starkv_kv4_cache& cache, const int32_t* block_table,
                            const int32_t* starts, const int32_t* cu, int batch, int max_pages, int64_t total,
                            __nv_bfloat16* k, __nv_bfloat16* v, cudaStream_t s);
cudaError_t launch_kv4_evict(const Ctx& c, const starkv_kv4_cache& cache, const int32_t* block_table,
                             const int32_t* seq_lens, const int32_t* keep_lens, int recent, int batch, int max_pages,
                             const int32_t* dst_table, int dst_max_pages, int32_t* new_lens, int32_t* kept,
                             cudaStream_t s);

// ---- kv4_decode.cu
struct Kv4DecodePlan {
  int ctas;             // CTAs that share the batch's pages (0: one per sequence and unit)
  int head_blocks;      // blocks of at most 8 query heads of a KV head
  int units;            // num_kv_heads * head_blocks
  int score_heads;      // floats of a token's scores in the workspace (0: not kept)
  size_t off_ml, off_unit, off_before, off_scores, ws_bytes;
};
Kv4DecodePlan plan_kv4_decode(const Ctx& c, int batch, int max_pages, bool accumulate);
cudaError_t launch_kv4_decode(const Ctx& c, const starkv_kv4_cache& cache, const __nv_bfloat16* q,
                              const int32_t* block_table, const int32_t* seq_lens, int batch, int max_pages,
                              bool accumulate, __nv_bfloat16* out, void* ws, const Kv4DecodePlan& plan,
                              cudaStream_t s);

// ---- prompt_tc.cu
struct PromptArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;       // NULL for the weights
  int64_t q_stride, k_stride, v_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int batch;
  int64_t total_q, total_k;
};
struct PromptPlan {
  int ctas;             // CTAs that share the key tiles (0: one per pair of query tiles)
  int64_t blocks;
  size_t off_ml, off_cuts, ws_bytes;
};
PromptPlan plan_prompt(const Ctx& c, int batch, int64_t total_q, int64_t total_k, int max_q_len);
int64_t weights_items(const Ctx& c, int batch, int max_k_len);
cudaError_t launch_prompt_attn(const Ctx& c, const PromptArgs& a, int max_q_len, __nv_bfloat16* out, float* lse,
                               void* ws, const PromptPlan& plan, cudaStream_t s);
cudaError_t launch_prompt_weights(const Ctx& c, const PromptArgs& a, const float* lse, int max_k_len, int window,
                                  float* weights, cudaStream_t s);

}  // namespace starkv
