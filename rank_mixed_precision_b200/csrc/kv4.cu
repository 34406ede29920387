// The 4-bit cache of full-width layers: append, read back, eviction.
// (Times in this file: a call's time on the GPU, calls back to back in a graph, unless a kernel's own.)
#include "full.cuh"
#include "sm100.cuh"

namespace starkv {

using namespace sm100;

namespace {

// ---------------------------------------------------------------------------
// Append.  A thread quantises one group of 32 channels (four 16-byte loads, four code words):
// the group's scale is worked out once and no thread waits for another.  The kernel is bound by
// its instructions, 127 a code word (with eight channels a thread, the group's ends by
// shuffles and the scale worked out four times, it took 222, and 70 us, the kernel alone, instead
// of 46 for 8098 tokens of 32 heads of 128: 3.8 TB/s).
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

constexpr int kRowThreads = 256;
constexpr int kReadTokens = 8;  // tokens a block of the read takes where there are many

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// fl16(fl32(d / 15)).  d * fl(1/15) is within 2^-23 of the quotient (relative), so where both ends
// of that interval round to the same fp16 number it is the one; else the quotient is taken.
__device__ __forceinline__ __half scale_of(float d) {
  const float q = d * 0.0666666666666666666667f;
  const __half lo = __float2half_rn(q * 0.9999997f), hi = __float2half_rn(q * 1.0000003f);
  return __half_as_ushort(lo) == __half_as_ushort(hi) ? lo : __float2half_rn(__fdiv_rn(d, 15.f));
}

// Eight codes clamp(rint(fl(fl(x - z) / s)), 0, 15) in a word, low nibble first; x: the channels
// in bf16 pairs, inv: 1 / (15 s).  A product with inv saturates to [0, 1]; 15 of it is within 5e-6
// of the clamped quotient and rounds to the same integer unless it lies that close to a half: then
// (a word in two hundred, mostly true halves) the quotient is taken.
__device__ __forceinline__ uint32_t codes_of(const uint4& x, float z, float s, float inv) {
  const uint32_t r[4] = {x.x, x.y, x.z, x.w};
  const f32x2 minus_z = pair(-z, -z), k15 = pair(15.f, 15.f), k_round = pair(12582912.f, 12582912.f);  // 1.5 2^23
  const f32x2 minus_1 = pair(-1.f, -1.f);
  uint32_t word = 0;
  float off = 0.f;  // largest distance from an integer
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 d = unpair(add2(pair(__uint_as_float(r[e] << 16), __uint_as_float(r[e] & 0xffff0000u)), minus_z));
    const f32x2 q = pair(__saturatef(d.x * inv), __saturatef(d.y * inv));
    const f32x2 n = fma2(q, k15, k_round);  // the sum's low bits are the integer
    const float2 rest = unpair(fma2(q, k15, fma2(n, minus_1, k_round))), bits = unpair(n);
    off = fmaxf(off, fmaxf(fabsf(rest.x), fabsf(rest.y)));
    word += (__float_as_uint(bits.x) << (8 * e)) + (__float_as_uint(bits.y) << (8 * e + 4));
  }
  word -= 0x4b400000u + 0xb4000000u + 0x40000000u;  // 2^23's pattern above the first three integers (the others' leaves the word)
  if (off > 0.49999f) {
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const uint32_t two = e < 2 ? x.x : e < 4 ? x.y : e < 6 ? x.z : x.w;
      const float d = __fsub_rn(__uint_as_float(e & 1 ? two & 0xffff0000u : two << 16), z);
      const float q = __saturatef(d * inv) * 15.f;
      if (fabsf(q - rintf(q)) > 0.49998f)
        word = (word & ~(15u << (4 * e))) | (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(d, s)), 0.f), 15.f) << (4 * e);
    }
  }
  return word;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const AppendArgs a) {
  using P = Kv4<D>;
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t half = (uint32_t)a.pool.h_kv * P::kGroups;  // groups of a token's K row, and of its V row
  const uint32_t id = blockIdx.x * (uint32_t)kRowThreads + threadIdx.x;
  const uint32_t token = id / (2 * half), unit = id - token * 2 * half;
  if (token >= a.n) return;
  const bool is_v = unit >= half;
  const uint32_t at_row = is_v ? unit - half : unit;
  const int head = (int)(at_row / P::kGroups), g = (int)(at_row % P::kGroups);
  const int64_t slot = a.slots[token];
  const uint4* src =
      reinterpret_cast<const uint4*>((is_v ? a.v + token * a.v_stride : a.k + token * a.k_stride) + at_row * 32);
  uint4 x[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) x[c] = src[c];
  if (slot >= a.pool.n_pages * kPage) {
    if (unit == 0) set_status(a.status, STARKV_DEV_BAD_SLOT);
    return;
  }
  if (slot < 0) return;
  // minimum and maximum in bf16 (exact); NaN passes through both, so a group whose ends are finite is finite
  const __nv_bfloat162* y = reinterpret_cast<const __nv_bfloat162*>(x);
  __nv_bfloat162 lo = y[0], hi = y[0];
#pragma unroll
  for (int e = 1; e < 16; ++e) {
    lo = __hmin2_nan(lo, y[e]);
    hi = __hmax2_nan(hi, y[e]);
  }
  const float mn = __bfloat162float(__hmin_nan(__low2bfloat16(lo), __high2bfloat16(lo)));
  const float mx = __bfloat162float(__hmax_nan(__low2bfloat16(hi), __high2bfloat16(hi)));
  __half s16 = scale_of(__fsub_rn(mx, mn));
  __half z16 = __float2half_rn(mn);
  const float sf = __half2float(s16), zf = __half2float(z16);
  // decode widens code * s + z in fp16, so the top code must stay inside it too
  const bool fits = isfinite(mn) && isfinite(mx) && isfinite(sf) && isfinite(zf) &&
                    isfinite(__half2float(__float2half_rn(fmaf(15.f, sf, zf))));
  uint32_t code[4] = {0, 0, 0, 0};
  if (!fits) {
    s16 = z16 = __float2half_rn(0.f);
    set_status(a.status, STARKV_DEV_QUANT_OVERFLOW);
  } else if (sf != 0.f) {
    const float inv = rcp_approx(sf) * 0.0666666666666666666667f;
#pragma unroll
    for (int c = 0; c < 4; ++c) code[c] = codes_of(x[c], zf, sf, inv);
  }
  const int64_t ph = (slot >> 4) * a.pool.h_kv + head;
  const int t = (int)(slot & 15);
  uint8_t* base = a.pool.pages + ph * P::kBytes;
  if (is_v) {
    *reinterpret_cast<uint4*>(base + P::kV + t * P::kRow + g * 16) = make_uint4(code[0], code[1], code[2], code[3]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint32_t*>(base + t * P::kRow + (c * P::kGroups + g) * 4) = code[c];
  }
  *reinterpret_cast<uint32_t*>(base + (is_v ? P::kVMeta : P::kKMeta) + t * P::kMetaRow + g * 4) =
      (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(z16) << 16);
  if (!is_v && g == 0 && a.pool.weights)
    a.pool.weights[ph * kPage + t] = a.weights ? a.weights[(int64_t)token * a.pool.h_kv + head] : 0.f;
}

// ---------------------------------------------------------------------------
// Read back.  One code word per thread and token: 4 bytes and the group's scale and
// zero in, eight bf16 values (16 bytes) out.  A block takes 256 code words of the rows of
// T tokens, whose slots it looks up once.
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

// The slot of row `row` of the output, -1 (and a status bit) where there is none.
__device__ int64_t slot_of_row(const ReadArgs& a, int64_t row) {
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
    return -1;
  }
  const int64_t t = (a.starts ? a.starts[lo] : 0) + (row - c0);
  if (t < 0 || t >= (int64_t)a.max_pages * kPage) {
    set_status(a.status, STARKV_DEV_BAD_SEQ_LEN);
    return -1;
  }
  const int64_t page = a.block_table[(int64_t)lo * a.max_pages + t / kPage];
  if (page < 0 || page >= a.pool.n_pages) {
    set_status(a.status, STARKV_DEV_BAD_PAGE);
    return -1;
  }
  return page * kPage + t % kPage;
}

template <int D, int T>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const ReadArgs a) {
  using P = Kv4<D>;
  __shared__ int64_t slot_of[T];
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0)  // a row's own sequence does not show that another's bounds fall
    for (int i = threadIdx.x; i < a.batch; i += kRowThreads)
      if (a.cu[i + 1] < a.cu[i]) set_status(a.status, STARKV_DEV_BAD_QUERY_SPAN);
  const int64_t row0 = (int64_t)blockIdx.x * T;
  if (threadIdx.x < T) slot_of[threadIdx.x] = row0 + threadIdx.x < a.total ? slot_of_row(a, row0 + threadIdx.x) : -1;
  __syncthreads();
  const int half = a.pool.h_kv * (D / 8);
  const int word = blockIdx.y * kRowThreads + threadIdx.x;
  if (word >= 2 * half) return;
  const bool is_v = word >= half;
  const int at_row = is_v ? word - half : word;
  const int head = at_row / (D / 8), w = at_row % (D / 8);
  const int code_at = (is_v ? P::kV : 0) + (is_v ? w : (w & 3) * P::kGroups + (w >> 2)) * 4;
  const int meta_at = (is_v ? P::kVMeta : P::kKMeta) + (w >> 2) * 4;
  uint32_t code[T], meta[T];
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int64_t slot = slot_of[i];
    code[i] = meta[i] = 0;  // a token that is not there reads as zeros
    if (slot < 0) continue;
    const int t = (int)(slot % kPage);
    const uint8_t* base = a.pool.pages + (slot / kPage * a.pool.h_kv + head) * (int64_t)P::kBytes;
    code[i] = *reinterpret_cast<const uint32_t*>(base + code_at + t * P::kRow);
    meta[i] = *reinterpret_cast<const uint32_t*>(base + meta_at + t * P::kMetaRow);
  }
  __nv_bfloat16* out = (is_v ? a.v : a.k) + at_row * 8;
#pragma unroll
  for (int i = 0; i < T; ++i) {
    if (row0 + i >= a.total) break;
    const float2 sz = unpack_meta(meta[i]);
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // 2^23 + code is a pattern; code * s is exact in fp32: one rounding for the sum, one to bf16
      const float c0 = __uint_as_float(0x4b000000u | ((code[i] >> (8 * e)) & 15u)) - 8388608.f;
      const float c1 = __uint_as_float(0x4b000000u | ((code[i] >> (8 * e + 4)) & 15u)) - 8388608.f;
      const __nv_bfloat162 b = __floats2bfloat162_rn(fmaf(c0, sz.x, sz.y), fmaf(c1, sz.x, sz.y));
      p[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(out + (row0 + i) * half * 8) = make_uint4(p[0], p[1], p[2], p[3]);
  }
}

// ---------------------------------------------------------------------------
// Eviction, step 1: the kept tokens of one (sequence, KV head).
//
// Each token that may go gets a 32-bit key that orders like its weight (NaN below all).
// A cluster of CTAs shares a long sequence out; the threads hold the keys in registers (eight
// tokens of each stretch of 4096 a thread, four stretches; keys beyond are read again each
// time).  The threshold, the need-th largest key, is found by counts in 2048 equal bins of the
// range that is left: all of [least, largest] first, then the bin that holds it, until a bin is
// one key or ends exactly at the need-th (three passes at most, two for most weights).  Bins of
// the range, not leading digits: weights share their exponents' digits, and counts of few bins
// queue up.  One ordered pass then lists the keys above the threshold and the first equal to it.
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
  int cluster;  // CTAs that share a (sequence, KV head) in the selection
};

// CTAs of a cluster at most: 32 lists of 32768 tokens take 69 us, the move among them, on one CTA each,
// 56 on two, 54 on four, 62 on eight.
constexpr int kMostCluster = 4;
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelEach = 8;                            // tokens of a thread in a stretch
constexpr int kBins = 2048;                            // four a thread
constexpr int kStretch = kSelThreads * kSelEach;
constexpr int kHeld = 4;                               // stretches whose keys stay in registers

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  // order-preserving map of floats, moved up by one so that NaN stays below -inf
  return ((u & 0x80000000u) ? ~u : (u | 0x80000000u)) + 1u;
}

// Sum (and the sum before) of a value over the block's warps' lanes; sum: scratch, free again behind the next barrier.
__device__ __forceinline__ uint32_t block_scan(uint32_t mine, uint32_t* sum, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sum[warp] = inc;
  __syncthreads();
  const uint32_t w = lane < kSelWarps ? sum[lane] : 0u;
  total = __reduce_add_sync(0xffffffffu, w);
  return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u) + inc - mine;
}

// grid (num_kv_heads * cluster, batch); two CTAs an SM at 64 registers a thread, of which 44 bytes spill
__global__ void __launch_bounds__(kSelThreads, 2) kv4_select_kernel(const EvictArgs a) {
  __shared__ __align__(16) uint32_t bins[kBins];
  __shared__ uint32_t scan[2][kSelWarps];
  __shared__ uint32_t ends[2][kSelWarps];
  __shared__ uint32_t shared[4];  // for the cluster: a bad length or page, least and largest key; the counts of the list
  __shared__ uint32_t found[3];   // bin of the threshold, keys above the bin, keys in it
  __shared__ unsigned bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = a.cluster, rank = C > 1 ? (int)cluster_rank() : 0;
  const int head = blockIdx.x / C, b = blockIdx.y;
  auto sync = [&]() {
    if (C > 1) cluster_sync();
    else __syncthreads();
  };
  auto of_rank = [&](const uint32_t* p, int r) -> uint32_t {
    return C > 1 ? __float_as_uint(dsmem_ld_f32(dsmem_addr(p, (uint32_t)r))) : *p;
  };
  if (tid == 0) bad = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.seq_lens[b];
  const int want = a.keep_lens[b];
  const int cap = a.dst_max_pages * kPage;
  int32_t* kept = a.kept + ((int64_t)b * a.pool.h_kv + head) * cap;
  const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
  const int keep = min(n, want);
  const bool sane = n >= 0 && want >= 0 && n <= a.max_pages * kPage && keep <= cap;
  const int recent = min(a.recent, keep);
  const int need = keep - recent;            // how many of the others stay
  // the CTA's tokens: t0 .. t1 - 1, of which those below old may go
  const int per = sane ? (int)(((int64_t)n + C * kPage - 1) / (C * kPage)) * kPage : 0;
  const int t0 = min((int64_t)n, (int64_t)rank * per), t1 = min((int64_t)n, (int64_t)t0 + per), old = min(t1, n - recent);
  auto check = [&](int64_t p) {
    if (p >= 0 && p < a.pool.n_pages) return true;
    atomicOr(&bad, STARKV_DEV_BAD_PAGE);
    return false;
  };
  // keys of tokens i0 .. i0 + 7 (one page's half: 32 contiguous bytes); the page is the caller's to check
  auto keys_of = [&](int64_t p, int i0, uint32_t (&k)[kSelEach]) {
    const float4* w = reinterpret_cast<const float4*>(a.pool.weights + (p * a.pool.h_kv + head) * kPage + i0 % kPage);
    const float4 x = w[0], y = w[1];
    const float v[kSelEach] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < kSelEach; ++e) k[e] = i0 + e < old ? weight_key(v[e]) : 0u;
  };
  uint32_t held[kHeld][kSelEach];
#pragma unroll
  for (int g = 0; g < kHeld; ++g) {
#pragma unroll
    for (int e = 0; e < kSelEach; ++e) held[g][e] = 0;
  }
  if (!sane) {
    if (tid == 0) bad = STARKV_DEV_BAD_SEQ_LEN;
  } else {
    for (int i = rank * kSelThreads + tid; i < (keep + kPage - 1) / kPage; i += C * kSelThreads)
      check(a.dst_table[(int64_t)b * a.dst_max_pages + i]);
#pragma unroll
    for (int g = 0; g < kHeld; ++g) {
      const int i0 = t0 + g * kStretch + tid * kSelEach;
      if (i0 >= t1) continue;
      const int64_t p = table[i0 / kPage];
      if (check(p) && need > 0 && keep < n && i0 < old) keys_of(p, i0, held[g]);
    }
    for (int i0 = t0 + kHeld * kStretch + tid * kSelEach; i0 < t1; i0 += kStretch) check(table[i0 / kPage]);
  }
  __syncthreads();
  // f(key) of every key of the CTA that may go
  auto each = [&](auto&& f) {
#pragma unroll
    for (int g = 0; g < kHeld; ++g)
      if (t0 + g * kStretch < old) {
#pragma unroll
        for (int e = 0; e < kSelEach; ++e)
          if (t0 + g * kStretch + tid * kSelEach + e < old) f(held[g][e]);
      }
    for (int i0 = t0 + kHeld * kStretch + tid * kSelEach; i0 < old; i0 += kStretch) {
      uint32_t k[kSelEach];
      keys_of(table[i0 / kPage], i0, k);
#pragma unroll
      for (int e = 0; e < kSelEach; ++e)
        if (i0 + e < old) f(k[e]);
    }
  };
  uint32_t lo = 0xffffffffu, hi = 0;
  if (!bad && need > 0 && keep < n)
    each([&](uint32_t k) {
      lo = min(lo, k);
      hi = max(hi, k);
    });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    ends[0][warp] = lo;
    ends[1][warp] = hi;
  }
  __syncthreads();
  if (warp == 0) {
    lo = __reduce_min_sync(0xffffffffu, lane < kSelWarps ? ends[0][lane] : 0xffffffffu);
    hi = __reduce_max_sync(0xffffffffu, lane < kSelWarps ? ends[1][lane] : 0u);
    if (lane == 0) {
      shared[0] = bad;
      shared[1] = lo;
      shared[2] = hi;
    }
  }
  sync();
  unsigned wrong = 0;
  lo = 0xffffffffu;
  hi = 0;
  for (int r = 0; r < C; ++r) {
    wrong |= of_rank(&shared[0], r);
    lo = min(lo, of_rank(&shared[1], r));
    hi = max(hi, of_rank(&shared[2], r));
  }
  // what needs no search; the CTAs share the writing out
  const int step = C * kSelThreads, at0 = rank * kSelThreads + tid;
  const int kept_now = wrong || keep < 0 ? 0 : keep;
  if (wrong && rank == 0 && tid == 0) set_status(a.status, wrong);
  for (int i = kept_now + at0; i < cap; i += step) kept[i] = -1;
  if (kept_now == n) {
    for (int i = at0; i < n; i += step) kept[i] = i;
  } else if (kept_now > 0) {
    for (int i = at0; i < recent; i += step) kept[need + i] = n - recent + i;
  }
  if (kept_now == 0 || kept_now == n || need == 0) {
    if (C > 1) cluster_sync();  // (its shared memory has been read)
    return;
  }
  // keys above the range [lo, hi] stay; `left` of the keys in it do
  uint32_t left = (uint32_t)need;
  uint32_t threshold;
  while (true) {
    const uint32_t width = hi - lo;
    const int shift = max(0, 32 - __clz(width) - 11);  // width >> shift < 2048
    uint4* mine = reinterpret_cast<uint4*>(bins) + (kBins / 4 - 1 - tid);  // thread i: the i-th four bins from the top
    *mine = make_uint4(0, 0, 0, 0);
    __syncthreads();
    each([&](uint32_t k) {
      if (k - lo <= width) atomicAdd(&bins[(k - lo) >> shift], 1u);
    });
    sync();
    uint32_t c[4] = {0, 0, 0, 0};  // from the top
    if (C == 1) {
      const uint4 x = *mine;
      c[0] = x.w, c[1] = x.z, c[2] = x.y, c[3] = x.x;
    } else {
      for (int r = 0; r < C; ++r) {
        const float4 x = dsmem_ld_f4(dsmem_addr(mine, (uint32_t)r));
        c[0] += __float_as_uint(x.w), c[1] += __float_as_uint(x.z), c[2] += __float_as_uint(x.y), c[3] += __float_as_uint(x.x);
      }
    }
    uint32_t all, before = block_scan(c[0] + c[1] + c[2] + c[3], scan[0], all);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (before < left && left <= before + c[e]) {
        found[0] = (kBins / 4 - 1 - tid) * 4 + 3 - e;
        found[1] = before;
        found[2] = c[e];
      }
      before += c[e];
    }
    sync();  // (and the bins have been read)
    left -= found[1];
    lo += found[0] << shift;
    const uint32_t in_bin = found[2];
    if (left == in_bin) {  // all of the bin's keys stay
      threshold = lo - 1;  // (lo > 0: fewer than all keys stay)
      left = 0;
      break;
    }
    if (shift == 0) {
      threshold = lo;
      break;
    }
    hi = lo + ((1u << shift) - 1);
  }
  const uint32_t equals = left;  // of the keys equal to the threshold, the first so many stay
  // the ordered list, behind the CTAs before this one: a stretch at a time, each thread behind the threads before it
  uint32_t base = 0, base_eq = 0;
  if (C > 1) {
    uint32_t up = 0, eq = 0;
    each([&](uint32_t k) {
      up += k > threshold;
      eq += k == threshold;
    });
    uint32_t total;
    block_scan(up, scan[0], total);
    if (tid == 0) shared[0] = total;
    block_scan(eq, scan[1], total);
    if (tid == 0) shared[3] = total;
    sync();
    for (int r = 0; r < rank; ++r) {
      base += of_rank(&shared[0], r);
      base_eq += of_rank(&shared[3], r);
    }
    sync();
  }
  int turn = 0;
  auto list = [&](int i0, const uint32_t (&k)[kSelEach]) {
    uint32_t mine = 0;  // above in the low half, equal in the high half: at most 4096 each in a stretch
#pragma unroll
    for (int e = 0; e < kSelEach; ++e)
      if (i0 + e < old) mine += k[e] > threshold ? 1u : k[e] == threshold ? 0x10000u : 0u;
    uint32_t total;
    const uint32_t before = block_scan(mine, scan[turn & 1], total);  // (two scratches: one barrier a stretch)
    ++turn;
    uint32_t up = base + (before & 0xffffu), eq = base_eq + (before >> 16);
#pragma unroll
    for (int e = 0; e < kSelEach; ++e)
      if (i0 + e < old) {
        if (k[e] > threshold) {
          kept[up + min(eq, equals)] = i0 + e;
          ++up;
        } else if (k[e] == threshold) {
          if (eq < equals) kept[up + eq] = i0 + e;
          ++eq;
        }
      }
    base += total & 0xffffu;
    base_eq += total >> 16;
  };
  __syncthreads();
#pragma unroll
  for (int g = 0; g < kHeld; ++g)
    if (t0 + g * kStretch < old) list(t0 + g * kStretch + tid * kSelEach, held[g]);
  for (int i = t0 + kHeld * kStretch; i < old; i += kStretch) {
    uint32_t k[kSelEach] = {};
    const int i0 = i + tid * kSelEach;
    if (i0 < old) keys_of(table[i0 / kPage], i0, k);
    list(i0, k);
  }
}

// ---------------------------------------------------------------------------
// Eviction, step 2: gather the kept tokens' rows.  A warp fills kMovePages (destination
// page, KV head)s: all their source slots are looked up first, and a page's rows are asked
// for before the page before it is stored, so that the chain of dependent loads (kept index,
// page, rows) is waited for once in four pages.  (At width 64 the compiler stays at 40 registers and spills 12 bytes.)
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 128;
constexpr int kMovePages = 4;

template <int D>
struct MoveRows {
  using P = Kv4<D>;
  static constexpr int kChunks = P::kRow / 16;       // 16-byte pieces of a token's codes: 4 or 2
  static constexpr int kPer = kPage * kChunks / 32;  // pieces a lane moves, K or V: 2 or 1
  uint4 codes[2][kPer];
  uint32_t meta[P::kGroups];
  float w;
  uint32_t have;  // tokens of the page that are there

  // from: lane t's source slot of token t (-1: none)
  __device__ __forceinline__ void load(const Kv4Pool& pool, int head, int64_t from, int lane) {
    have = __ballot_sync(0xffffffffu, from >= 0) & 0xffffu;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t src = __shfl_sync(0xffffffffu, from, (i * 32 + lane) / kChunks);
      if (src < 0) continue;
      const uint8_t* base = pool.pages + (src / kPage * pool.h_kv + head) * (int64_t)P::kBytes +
                            (src % kPage) * P::kRow + (lane % kChunks) * 16;
      codes[0][i] = *reinterpret_cast<const uint4*>(base);
      codes[1][i] = *reinterpret_cast<const uint4*>(base + P::kV);
    }
    // lanes 0..15 move the K metadata, 16..31 the V metadata of token lane % 16
    const int64_t src = __shfl_sync(0xffffffffu, from, lane & 15);
    if (src < 0) return;
    const int64_t ph = src / kPage * pool.h_kv + head;
    const uint8_t* m = pool.pages + ph * (int64_t)P::kBytes + (lane < 16 ? P::kKMeta : P::kVMeta) + (src % kPage) * P::kMetaRow;
    if constexpr (P::kGroups == 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(m);
      meta[0] = x.x, meta[1] = x.y, meta[2] = x.z, meta[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(m);
      meta[0] = x.x, meta[1] = x.y;
    }
    if (lane < 16) w = pool.weights[ph * kPage + src % kPage];
  }

  __device__ __forceinline__ void store(const Kv4Pool& pool, int head, int64_t page, int lane) const {
    uint8_t* to = pool.pages + (page * pool.h_kv + head) * (int64_t)P::kBytes;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = (i * 32 + lane) / kChunks;
      if (!(have >> t & 1)) continue;
      uint8_t* base = to + t * P::kRow + (lane % kChunks) * 16;
      *reinterpret_cast<uint4*>(base) = codes[0][i];
      *reinterpret_cast<uint4*>(base + P::kV) = codes[1][i];
    }
    if (!(have >> (lane & 15) & 1)) return;
    uint8_t* m = to + (lane < 16 ? P::kKMeta : P::kVMeta) + (lane & 15) * P::kMetaRow;
    if constexpr (P::kGroups == 4)
      *reinterpret_cast<uint4*>(m) = make_uint4(meta[0], meta[1], meta[2], meta[3]);
    else
      *reinterpret_cast<uint2*>(m) = make_uint2(meta[0], meta[1]);
    if (lane < 16) pool.weights[(page * pool.h_kv + head) * kPage + lane] = w;
  }
};

template <int D>
__global__ void __launch_bounds__(kMoveThreads) kv4_move_kernel(const EvictArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.z, head = blockIdx.y;
  const int page0 = (blockIdx.x * (kMoveThreads / 32) + warp) * kMovePages;
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
  // lane 16 h + t: source slots of tokens t of pages page0 + h and page0 + 2 + h
  int64_t from[kMovePages / 2];
#pragma unroll
  for (int i = 0; i < kMovePages / 2; ++i) {
    const int at = (page0 + 2 * i) * kPage + lane;
    const int mine = at < cap ? kept[at] : -1;
    from[i] = mine < 0 ? -1 : (int64_t)a.block_table[(int64_t)b * a.max_pages + mine / kPage] * kPage + mine % kPage;
  }
  int64_t to = -1;  // lane i: destination page page0 + i
  if (lane < kMovePages && page0 + lane < a.dst_max_pages && kept[(page0 + lane) * kPage] >= 0)
    to = a.dst_table[(int64_t)b * a.dst_max_pages + page0 + lane];
  MoveRows<D> rows[2];
  auto of_page = [&](int i) { return __shfl_sync(0xffffffffu, from[i >> 1], (i & 1) * 16 + (lane & 15)); };
  rows[0].load(a.pool, head, of_page(0), lane);
#pragma unroll
  for (int i = 0; i < kMovePages; ++i) {
    if (i + 1 < kMovePages) rows[(i + 1) & 1].load(a.pool, head, of_page(i + 1), lane);
    const int64_t page = __shfl_sync(0xffffffffu, to, i);
    if (page >= 0) rows[i & 1].store(a.pool, head, page, lane);
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
  const int64_t threads = n * c.cfg.num_kv_heads * (2 * d / STARKV_KV4_GROUP);
  return launch_chained(d == 64 ? kv4_append_kernel<64> : kv4_append_kernel<128>,
                        dim3((unsigned)((threads + kRowThreads - 1) / kRowThreads)), dim3(kRowThreads), 0, s, 1u, a);
}

cudaError_t launch_kv4_read(const Ctx& c, const starkv_kv4_cache& cache, const int32_t* block_table,
                            const int32_t* starts, const int32_t* cu, int batch, int max_pages, int64_t total,
                            __nv_bfloat16* k, __nv_bfloat16* v, cudaStream_t s) {
  ReadArgs a{block_table, starts, cu, batch, max_pages, total, k, v, pool_of(c, cache), c.status};
  const int d = c.cfg.head_dim;
  const unsigned gy = (unsigned)((c.cfg.num_kv_heads * (2 * d / 8) + kRowThreads - 1) / kRowThreads);
  const dim3 block(kRowThreads);
  // blocks of several tokens where they fill the GPU twice over, else of one, over more SMs (8 heads of 128,
  // with the append before: 32 tokens 5.8 us, 6.6 in blocks of eight; 1000 tokens 9.2 and
  // 8.3: the rule could switch a little earlier)
  if ((total + kReadTokens - 1) / kReadTokens * gy >= 2 * sm_count(c)) {
    const dim3 grid((unsigned)((total + kReadTokens - 1) / kReadTokens), gy);
    return launch_chained(d == 64 ? kv4_read_kernel<64, kReadTokens> : kv4_read_kernel<128, kReadTokens>, grid, block, 0,
                          s, 1u, a);
  }
  return launch_chained(d == 64 ? kv4_read_kernel<64, 1> : kv4_read_kernel<128, 1>, dim3((unsigned)total, gy), block, 0,
                        s, 1u, a);
}

cudaError_t launch_kv4_evict(const Ctx& c, const starkv_kv4_cache& cache, const int32_t* block_table,
                             const int32_t* seq_lens, const int32_t* keep_lens, int recent, int batch, int max_pages,
                             const int32_t* dst_table, int dst_max_pages, int32_t* new_lens, int32_t* kept,
                             cudaStream_t s) {
  EvictArgs a{block_table, seq_lens, keep_lens, recent, max_pages, dst_table, dst_max_pages, new_lens, kept,
              pool_of(c, cache), c.status, 1};
  // clusters where a list is long and there are few: two CTAs run on an SM
  const int sms = sm_count(c);
  const int64_t most = (int64_t)max_pages * kPage, lists = (int64_t)c.cfg.num_kv_heads * batch;
  while (a.cluster < kMostCluster && most / a.cluster > kStretch && lists * a.cluster * 2 <= 2 * sms) a.cluster *= 2;
  cudaError_t e = launch_chained(kv4_select_kernel, dim3(c.cfg.num_kv_heads * a.cluster, batch), dim3(kSelThreads), 0, s,
                                 (unsigned)a.cluster, a);
  if (e != cudaSuccess) return e;
  const int per = kMoveThreads / 32 * kMovePages;
  return launch_chained(c.cfg.head_dim == 64 ? kv4_move_kernel<64> : kv4_move_kernel<128>,
                        dim3((dst_max_pages + per - 1) / per, c.cfg.num_kv_heads, batch), dim3(kMoveThreads), 0, s, 1u,
                        a);
}

}  // namespace starkv
