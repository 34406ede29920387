// The 4-bit cache of full-width layers: append, read back, eviction.
#include "full.cuh"
#include "sm100.cuh"

namespace starkv {

using namespace sm100;

namespace {

// ---------------------------------------------------------------------------
// Append.  Eight channels (one 16-byte load, one code word) per thread; the four
// threads of a 32-channel group share its minimum and maximum by two shuffles.
// 2 D/8 threads hold one (token, KV head): K's channels, then V's.
// ---------------------------------------------------------------------------
struct AppendArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t k_stride, v_stride;
  const int64_t* slots;
  const float* weights;
  int64_t n;
  Kv4Pool pool;
  unsigned int* status;
};

constexpr int kAppendThreads = 256;

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const AppendArgs a) {
  using P = Kv4<D>;
  constexpr int kPer = 2 * D / 8;  // threads of one (token, head): 32 or 16
  pdl_wait();
  pdl_launch_dependents();
  const int64_t id = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
  const int64_t th = id / kPer;
  const int w2 = (int)(id % kPer);
  const bool is_v = w2 >= D / 8;
  const int w = is_v ? w2 - D / 8 : w2;
  const int64_t token = th / a.pool.h_kv;
  const int head = (int)(th % a.pool.h_kv);
  const bool live = token < a.n;
  int64_t slot = live ? a.slots[token] : -1;
  if (slot >= a.pool.n_pages * kPage) {
    if (w2 == 0) set_status(a.status, STARKV_DEV_BAD_SLOT);
    slot = -1;
  }
  float x[8];
  float mn = 0.f, mx = 0.f;
  bool finite = true;
  if (slot >= 0) {
    const __nv_bfloat16* src = (is_v ? a.v + token * a.v_stride : a.k + token * a.k_stride) + head * D + w * 8;
    const uint4 raw = *reinterpret_cast<const uint4*>(src);
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
    mn = mx = x[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mn = fminf(mn, x[i]);
      mx = fmaxf(mx, x[i]);
      finite = finite && isfinite(x[i]);
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    finite = __shfl_xor_sync(0xffffffffu, (int)finite, o) != 0 && finite;
  }
  if (slot < 0) return;
  __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.f));
  __half z16 = __float2half_rn(mn);
  const float sf = __half2float(s16), zf = __half2float(z16);
  // decode widens code * s + z in fp16, so the top code must stay inside it too
  const bool fits = finite && isfinite(sf) && isfinite(zf) && isfinite(__half2float(__float2half_rn(fmaf(15.f, sf, zf))));
  uint32_t word = 0;
  if (!fits) {
    s16 = z16 = __float2half_rn(0.f);
    if ((w & 3) == 0) set_status(a.status, STARKV_DEV_QUANT_OVERFLOW);
  } else if (sf != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], zf), sf)), 0.f), 15.f);
      word |= (uint32_t)c << (4 * i);
    }
  }
  const int64_t page = slot / kPage;
  const int t = (int)(slot % kPage);
  uint8_t* base = a.pool.pages + (page * a.pool.h_kv + head) * (int64_t)P::kBytes;
  const int at = is_v ? w : (w & 3) * P::kGroups + (w >> 2);
  *reinterpret_cast<uint32_t*>(base + (is_v ? P::kV : 0) + t * P::kRow + at * 4) = word;
  if ((w & 3) == 0)
    *reinterpret_cast<uint32_t*>(base + (is_v ? P::kVMeta : P::kKMeta) + t * P::kMetaRow + (w >> 2) * 4) =
        (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(z16) << 16);
  if (w2 == 0 && a.pool.weights)
    a.pool.weights[(page * a.pool.h_kv + head) * kPage + t] = a.weights ? a.weights[token * a.pool.h_kv + head] : 0.f;
}

// ---------------------------------------------------------------------------
// Read back.  One code word per thread: 4 bytes in, eight bf16 values (16 bytes)
// out; a row's slot is looked up once per block.
// ---------------------------------------------------------------------------
struct ReadArgs {
  const int32_t* block_table;
  const int32_t* starts;
  const int32_t* cu;
  int batch, max_pages;
  int64_t total;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  Kv4Pool pool;
  unsigned int* status;
};

constexpr int kReadThreads = 256;
constexpr int kReadRows = 4;

template <int D>
__global__ void __launch_bounds__(kReadThreads) kv4_read_kernel(const ReadArgs a) {
  using P = Kv4<D>;
  __shared__ int64_t slot_of[kReadRows];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row0 = (int64_t)blockIdx.x * kReadRows;
  if (threadIdx.x < kReadRows) {
    const int64_t row = row0 + threadIdx.x;
    int64_t slot = -1;
    if (row < a.total) {
      // the last sequence that starts at or before the row (empty ones share its start)
      int lo = 0, hi = a.batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu[mid] <= row) lo = mid;
        else hi = mid - 1;
      }
      const int64_t c0 = a.cu[lo], c1 = a.cu[lo + 1];
      if (a.cu[0] != 0 || a.cu[a.batch] != a.total || row < c0 || row >= c1) {
        set_status(a.status, STARKV_DEV_BAD_QUERY_SPAN);
      } else {
        const int64_t t = (a.starts ? a.starts[lo] : 0) + (row - c0);
        if (t < 0 || t >= (int64_t)a.max_pages * kPage) {
          set_status(a.status, STARKV_DEV_BAD_SEQ_LEN);
        } else {
          const int64_t page = a.block_table[(int64_t)lo * a.max_pages + t / kPage];
          if (page < 0 || page >= a.pool.n_pages) set_status(a.status, STARKV_DEV_BAD_PAGE);
          else slot = page * kPage + t % kPage;
        }
      }
    }
    slot_of[threadIdx.x] = slot;
  }
  __syncthreads();
  const int per_row = a.pool.h_kv * (2 * D / 8);
  const int rows = (int)min((int64_t)kReadRows, a.total - row0);
  for (int e = threadIdx.x; e < rows * per_row; e += kReadThreads) {
    const int r = e / per_row, f = e - r * per_row;
    const int head = f / (2 * D / 8), w2 = f % (2 * D / 8);
    const bool is_v = w2 >= D / 8;
    const int w = is_v ? w2 - D / 8 : w2;
    const int64_t slot = slot_of[r];
    uint4 o = make_uint4(0, 0, 0, 0);
    if (slot >= 0) {
      const int t = (int)(slot % kPage);
      const uint8_t* base = a.pool.pages + (slot / kPage * a.pool.h_kv + head) * (int64_t)P::kBytes;
      const int at = is_v ? w : (w & 3) * P::kGroups + (w >> 2);
      const uint32_t word = *reinterpret_cast<const uint32_t*>(base + (is_v ? P::kV : 0) + t * P::kRow + at * 4);
      const float2 sz = unpack_meta(
          *reinterpret_cast<const uint32_t*>(base + (is_v ? P::kVMeta : P::kKMeta) + t * P::kMetaRow + (w >> 2) * 4));
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // code * s is exact in fp32: one rounding for the sum, one to bf16
        const __nv_bfloat162 b =
            __floats2bfloat162_rn(fmaf((float)((word >> (8 * i)) & 15u), sz.x, sz.y),
                                  fmaf((float)((word >> (8 * i + 4)) & 15u), sz.x, sz.y));
        p[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      o = make_uint4(p[0], p[1], p[2], p[3]);
    }
    __nv_bfloat16* dst = (is_v ? a.v : a.k) + ((row0 + r) * a.pool.h_kv + head) * (int64_t)D + w * 8;
    *reinterpret_cast<uint4*>(dst) = o;
  }
}

// ---------------------------------------------------------------------------
// Eviction, step 1: the kept tokens of one (sequence, KV head).
//
// Each token gets a 32-bit key that orders like its weight (recent tokens above
// all, NaN below all); the value of the keep-th largest key is found digit by digit
// (11, 11 and 10 bits, counts in shared memory), then one ordered pass lists the
// tokens above it and the first of those equal to it.
// ---------------------------------------------------------------------------
struct EvictArgs {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* keep_lens;
  int recent, max_pages;
  const int32_t* dst_table;
  int dst_max_pages;
  int32_t* new_lens;
  int32_t* kept;
  Kv4Pool pool;
  unsigned int* status;
  int smem_keys;  // keys that shared memory holds (the rest is read again)
};

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kKeysInSmem = 48 * 1024;  // beside the bins within 227 KB

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  // order-preserving map of floats, moved up by one so that NaN stays below -inf
  return ((u & 0x80000000u) ? ~u : (u | 0x80000000u)) + 1u;
}

__global__ void __launch_bounds__(kSelThreads, 1) kv4_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t bins[kBins];
  __shared__ uint32_t wsum[2][32];
  __shared__ uint32_t found[2];
  __shared__ unsigned bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.x, b = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.seq_lens[b];
  const int want = a.keep_lens[b];
  const int cap = a.dst_max_pages * kPage;
  int32_t* kept = a.kept + ((int64_t)b * a.pool.h_kv + head) * cap;
  if (tid == 0) bad = 0;
  __syncthreads();
  const int keep = min(n, want);
  if (n < 0 || want < 0 || n > a.max_pages * kPage || keep > cap) {
    if (tid == 0) bad = STARKV_DEV_BAD_SEQ_LEN;
  } else {
    for (int i = tid; i < (n + kPage - 1) / kPage; i += kSelThreads) {
      const int64_t p = a.block_table[(int64_t)b * a.max_pages + i];
      if (p < 0 || p >= a.pool.n_pages) atomicOr(&bad, STARKV_DEV_BAD_PAGE);
    }
    for (int i = tid; i < (keep + kPage - 1) / kPage; i += kSelThreads) {
      const int64_t p = a.dst_table[(int64_t)b * a.dst_max_pages + i];
      if (p < 0 || p >= a.pool.n_pages) atomicOr(&bad, STARKV_DEV_BAD_PAGE);
    }
  }
  __syncthreads();
  if (bad || keep <= 0) {
    if (bad && tid == 0) set_status(a.status, bad);
    for (int i = tid; i < cap; i += kSelThreads) kept[i] = -1;
    return;
  }
  for (int i = keep + tid; i < cap; i += kSelThreads) kept[i] = -1;
  if (keep == n) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  const int first_recent = n - min(a.recent, keep);
  auto key_at = [&](int i) -> uint32_t {
    if (i >= first_recent) return 0xffffffffu;
    const int64_t p = a.block_table[(int64_t)b * a.max_pages + i / kPage];
    return weight_key(a.pool.weights[(p * a.pool.h_kv + head) * kPage + i % kPage]);
  };
  for (int i = tid; i < min(n, a.smem_keys); i += kSelThreads) keys[i] = key_at(i);
  auto key_of = [&](int i) -> uint32_t { return i < a.smem_keys ? keys[i] : key_at(i); };
  uint32_t prefix = 0, need = (uint32_t)keep;  // digits found so far; how many still to take among their equals
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1024u : 2048u;
    for (int i = tid; i < kBins; i += kSelThreads) bins[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = key_of(i);
      if (pass == 0 || (k >> (pass == 1 ? 21 : 10)) == prefix) atomicAdd(&bins[(k >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    // thread i owns the two bins 2i, 2i+1 counted from the top: find the one that holds the need-th key
    const uint32_t top = kBins - 1 - 2 * tid;
    const uint32_t c0 = bins[top], c1 = bins[top - 1];
    uint32_t inc = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[0][warp] = inc;
    __syncthreads();
    uint32_t before = inc - c0 - c1;
    for (int w = 0; w < warp; ++w) before += wsum[0][w];
    if (before < need && need <= before + c0 + c1) {
      const bool upper = need <= before + c0;
      found[0] = upper ? top : top - 1;
      found[1] = need - (upper ? before : before + c0);
    }
    __syncthreads();
    prefix = (prefix << (pass == 2 ? 10 : 11)) | found[0];
    need = found[1];
    __syncthreads();
  }
  // the tokens above the threshold, and the first `need` equal to it, in order: each
  // warp counts its own stretch, then writes behind the counts of the warps before it
  const int per = ((n + 31) / 32 + 31) / 32 * 32;
  const int lo = min(n, warp * per), hi = min(n, lo + per);
  uint32_t above = 0, equal = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? key_of(i) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i < hi && k > prefix));
    equal += __popc(__ballot_sync(0xffffffffu, i < hi && k == prefix));
  }
  if (lane == 0) {
    wsum[0][warp] = above;
    wsum[1][warp] = equal;
  }
  __syncthreads();
  above = equal = 0;
  for (int w = 0; w < warp; ++w) {
    above += wsum[0][w];
    equal += wsum[1][w];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? key_of(i) : 0u;
    const uint32_t ba = __ballot_sync(0xffffffffu, i < hi && k > prefix);
    const uint32_t be = __ballot_sync(0xffffffffu, i < hi && k == prefix);
    const uint32_t e = equal + __popc(be & below);
    if (i < hi && (k > prefix || (k == prefix && e < need)))
      kept[above + __popc(ba & below) + min(need, e)] = i;
    above += __popc(ba);
    equal += __popc(be);
  }
}

// ---------------------------------------------------------------------------
// Eviction, step 2: gather the kept tokens' rows.  One warp fills one (destination
// page, KV head): all its loads are issued before the first store.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) kv4_move_kernel(const EvictArgs a) {
  using P = Kv4<D>;
  constexpr int kChunks = P::kRow / 16;             // 16-byte pieces of a token's codes: 4 or 2
  constexpr int kPer = kPage * kChunks / 32;        // pieces a lane moves, K or V: 2 or 1
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.z, head = blockIdx.y;
  const int page = blockIdx.x * (kMoveThreads / 32) + warp;
  pdl_wait();
  pdl_launch_dependents();
  const int cap = a.dst_max_pages * kPage;
  const int32_t* kept = a.kept + ((int64_t)b * a.pool.h_kv + head) * cap;
  if (blockIdx.x == 0 && head == 0 && threadIdx.x == 0) {
    int lo = 0, hi = cap;  // the kept count: where the -1 begin
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (kept[mid] >= 0) lo = mid + 1;
      else hi = mid;
    }
    a.new_lens[b] = lo;
  }
  if (page >= a.dst_max_pages) return;
  const int mine = lane < kPage ? kept[page * kPage + lane] : -1;
  if (!__any_sync(0xffffffffu, mine >= 0)) return;
  int64_t from = -1;  // lane t: source of token t as page * 16 + offset
  if (mine >= 0) from = (int64_t)a.block_table[(int64_t)b * a.max_pages + mine / kPage] * kPage + mine % kPage;
  uint8_t* to = a.pool.pages +
                ((int64_t)a.dst_table[(int64_t)b * a.dst_max_pages + page] * a.pool.h_kv + head) * (int64_t)P::kBytes;
  uint4 codes[2][kPer];
  int64_t src[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int t = (i * 32 + lane) / kChunks;
    src[i] = __shfl_sync(0xffffffffu, from, t);
    if (src[i] < 0) continue;
    const uint8_t* base = a.pool.pages + (src[i] / kPage * a.pool.h_kv + head) * (int64_t)P::kBytes +
                          (src[i] % kPage) * P::kRow + (lane % kChunks) * 16;
    codes[0][i] = *reinterpret_cast<const uint4*>(base);
    codes[1][i] = *reinterpret_cast<const uint4*>(base + P::kV);
  }
  // lanes 0..15 move the K metadata, 16..31 the V metadata of token lane % 16
  const int64_t msrc = __shfl_sync(0xffffffffu, from, lane & 15);
  const int moff = lane < 16 ? P::kKMeta : P::kVMeta;
  uint32_t meta[P::kGroups];
  float w = 0.f;
  if (msrc >= 0) {
    const int64_t ph = msrc / kPage * a.pool.h_kv + head;
    const uint32_t* m = reinterpret_cast<const uint32_t*>(a.pool.pages + ph * (int64_t)P::kBytes + moff +
                                                          (msrc % kPage) * P::kMetaRow);
#pragma unroll
    for (int i = 0; i < P::kGroups; ++i) meta[i] = m[i];
    if (lane < 16) w = a.pool.weights[ph * kPage + msrc % kPage];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (src[i] < 0) continue;
    const int e = i * 32 + lane;
    uint8_t* base = to + (e / kChunks) * P::kRow + (lane % kChunks) * 16;
    *reinterpret_cast<uint4*>(base) = codes[0][i];
    *reinterpret_cast<uint4*>(base + P::kV) = codes[1][i];
  }
  if (msrc >= 0) {
    uint32_t* m = reinterpret_cast<uint32_t*>(to + moff + (lane & 15) * P::kMetaRow);
#pragma unroll
    for (int i = 0; i < P::kGroups; ++i) m[i] = meta[i];
    if (lane < 16)
      a.pool.weights[((int64_t)a.dst_table[(int64_t)b * a.dst_max_pages + page] * a.pool.h_kv + head) * kPage + lane] = w;
  }
}

Kv4Pool pool_of(const Ctx& c, const starkv_kv4_cache& cache) {
  return Kv4Pool{(uint8_t*)cache.pages, cache.weights, cache.n_pages, c.cfg.num_kv_heads};
}

}  // namespace

cudaError_t launch_kv4_append(const Ctx& c, const starkv_kv4_cache& cache, const __nv_bfloat16* k,
                              const __nv_bfloat16* v, int64_t k_stride, int64_t v_stride, const int64_t* slots,
                              const float* weights, int64_t n, cudaStream_t s) {
  AppendArgs a{k, v, k_stride, v_stride, slots, weights, n, pool_of(c, cache), c.status};
  const int d = c.cfg.head_dim;
  const int64_t threads = n * c.cfg.num_kv_heads * (2 * d / 8);
  const int64_t blocks = (threads + kAppendThreads - 1) / kAppendThreads;
  return launch_chained(d == 64 ? kv4_append_kernel<64> : kv4_append_kernel<128>, dim3((unsigned)blocks),
                        dim3(kAppendThreads), 0, s, 1u, a);
}

cudaError_t launch_kv4_read(const Ctx& c, const starkv_kv4_cache& cache, const int32_t* block_table,
                            const int32_t* starts, const int32_t* cu, int batch, int max_pages, int64_t total,
                            __nv_bfloat16* k, __nv_bfloat16* v, cudaStream_t s) {
  ReadArgs a{block_table, starts, cu, batch, max_pages, total, k, v, pool_of(c, cache), c.status};
  const int64_t blocks = (total + kReadRows - 1) / kReadRows;
  return launch_chained(c.cfg.head_dim == 64 ? kv4_read_kernel<64> : kv4_read_kernel<128>, dim3((unsigned)blocks),
                        dim3(kReadThreads), 0, s, 1u, a);
}

cudaError_t launch_kv4_evict(const Ctx& c, const starkv_kv4_cache& cache, const int32_t* block_table,
                             const int32_t* seq_lens, const int32_t* keep_lens, int recent, int batch, int max_pages,
                             const int32_t* dst_table, int dst_max_pages, int32_t* new_lens, int32_t* kept,
                             cudaStream_t s) {
  EvictArgs a{block_table, seq_lens, keep_lens, recent, max_pages, dst_table, dst_max_pages, new_lens, kept,
              pool_of(c, cache), c.status, 0};
  const int64_t most = (int64_t)max_pages * kPage;
  a.smem_keys = (int)(most < kKeysInSmem ? most : kKeysInSmem);
  const size_t smem = (size_t)a.smem_keys * 4;
  cudaError_t e = cudaFuncSetAttribute(kv4_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kKeysInSmem * 4);
  if (e != cudaSuccess) return e;
  e = launch_chained(kv4_select_kernel, dim3(c.cfg.num_kv_heads, batch), dim3(kSelThreads), smem, s, 1u, a);
  if (e != cudaSuccess) return e;
  const int per = kMoveThreads / 32;
  return launch_chained(c.cfg.head_dim == 64 ? kv4_move_kernel<64> : kv4_move_kernel<128>,
                        dim3((dst_max_pages + per - 1) / per, c.cfg.num_kv_heads, batch), dim3(kMoveThreads), 0, s, 1u,
                        a);
}

}  // namespace starkv
