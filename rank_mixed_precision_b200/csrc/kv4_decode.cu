// Decode attention over the 4-bit cache of full-width layers.
//
// One CTA takes a chunk of pages of one (sequence, KV head, block of at most eight
// query heads); its four warps take the chunk's pages in turn, each with its own
// ring of bulk copies (one 16-token page of one head is one contiguous copy), its
// own running maximum and sum, and its own output accumulators.  Scores and
// outputs run on mma.sync m16n8k16: the eight query heads are the N of both
// products, so a page's codes are read once for all of them.  With N = 8 the
// products are small (2 x 16 x 8 x D per page) and their operands come out of
// 4-bit codes in registers, which tcgen05 (operands in shared or tensor memory,
// N of a whole tile) could only take after a round trip through shared memory.
//
//   scores   s[t, h] = sum_g ( sc[t, g] * sum_{c in g} n[t, c] q[h, c] + z[t, g] * sum_{c in g} q[h, c] )
//     A = the codes n of the page's tokens, B = q.  A masked code (w & 0x000f000f) is
//     already two fp16 numbers, n 2^-24 (subnormal, exact), and (w & 0x00f000f0) is
//     16 n 2^-24, so widening costs one AND for two codes; q is bf16, scaled by a power
//     of two per head (and by 1/16 for the odd codes), so it too is exact in fp16.  The
//     products are exact and the sums fp32: the probabilities that are added to the
//     cache's weights keep fp32 accuracy.
//   output   o[c, h] = sum_t v[t, c] p[t, h]
//     A = V^T, widened to fp16 (code * s + z, one rounding), B = p in fp16 (at most 2^8
//     against the running maximum, which moves only when it grows by more than that).
#include "full.cuh"
#include "sm100.cuh"

namespace starkv {

using namespace sm100;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kHeads = 8;            // query heads of one CTA (the N of the products)
constexpr float kMoveMax = 8.f;      // the running maximum moves when a score passes it by this (log2)
constexpr float kNoMax = -1e30f;     // running maximum before the first score

struct DecodeArgs {
  const __nv_bfloat16* q;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int H, group, head_blocks, max_pages, chunk, splits, score_heads;
  float scale_log2;        // log2(e) / sqrt(D)
  Kv4Pool pool;
  __nv_bfloat16* out;
  float* part_o;           // [B][h_kv * head_blocks][splits][8][D], relative to the split's maximum
  float2* part_ml;         // [B][h_kv * head_blocks][splits][8] (maximum, sum)
  float* scores;           // [B][h_kv][max_pages * 16][score_heads], log2 units
  unsigned int* status;
};

template <int D>
struct DecodeSmem {
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kRing = kWarps * kStages * Kv4<D>::kBytes;
  static constexpr int kMerge = kWarps * kHeads * D * 4;  // shares the ring's bytes
  static constexpr int kBytes = (kRing > kMerge ? kRing : kMerge);
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 x 8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t movm_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Token of a page that row r (K's A operand) or k index r (V's) stands for, r = 2t + e + 8f: any
// bijection serves.  With this one the two rows of neighbouring lanes (e = 0, 1) lie in different
// halves of the 32 banks, and so do V's four rows of a load (t = 0..3).
__device__ __forceinline__ int token_of(int t, int e, int f) { return 8 * f + 4 * e + ((t + e) & 3); }

template <int D>
__global__ void __launch_bounds__(kThreads, 4) kv4_decode_kernel(const DecodeArgs a) {
  using P = Kv4<D>;
  using SM = DecodeSmem<D>;
  constexpr int NG = P::kGroups;
  constexpr int MT = D / 16;   // 16-channel tiles of the output
  constexpr int ST = SM::kStages;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(8) uint64_t full[kWarps * ST];
  __shared__ float2 ml[kWarps][kHeads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, b = blockIdx.z;
  const int kv = blockIdx.y / a.head_blocks, hb = blockIdx.y % a.head_blocks;
  const int heads = min(kHeads, a.group - hb * kHeads);
  const int h0 = kv * a.group + hb * kHeads;
  if (lane < ST) mbar_init(&full[warp * ST + lane], 1);
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  int len = a.seq_lens[b];
  if (len < 0 || len > a.max_pages * kPage) {
    if (tid == 0 && split == 0) set_status(a.status, STARKV_DEV_BAD_SEQ_LEN);
    len = 0;
  }
  const int pages = (len + kPage - 1) / kPage;
  const int p0 = split * a.chunk, p1 = min(pages, p0 + a.chunk);
  if (p0 >= p1) {
    // nothing here; an empty sequence's first split writes the zero row
    if (split == 0 && a.splits == 1)
      for (int i = tid; i < heads * D; i += kThreads)
        a.out[((int64_t)b * a.H + h0) * D + i] = __float2bfloat16_rn(0.f);
    return;
  }
  // ---- the warp's copies: pages p0 + warp + 4 i
  const int mine = (p1 - p0 - warp + kWarps - 1) / kWarps;  // pages of this warp (may be <= 0)
  const int32_t* table = a.block_table + (int64_t)b * a.max_pages + p0 + warp;
  uint8_t* ring = sm + warp * ST * P::kBytes;
  uint64_t* bar = full + warp * ST;
  int32_t ids = 0;      // lane i: page of iteration (base of 32) + i
  int32_t ids_next = 0;
  auto load_ids = [&](int base) -> int32_t {
    int32_t id = -1;
    if (base + lane < mine) {
      id = table[(base + lane) * kWarps];
      if (id < 0 || id >= a.pool.n_pages) {
        set_status(a.status, STARKV_DEV_BAD_PAGE);
        id = -1;
      }
    }
    return id;
  };
  ids = load_ids(0);
  ids_next = load_ids(32);
  // issue the copy of iteration i (its id is in `ids` or, past the current 32, in `ids_next`)
  auto issue = [&](int i, int base) {
    if (i >= mine) return;
    const int32_t id = __shfl_sync(0xffffffffu, i - base < 32 ? ids : ids_next, i & 31);
    if (lane == 0) {
      const int s = i % ST;
      if (id < 0) {
        mbar_arrive(&bar[s]);  // nothing to copy: the page is left out
      } else {
        mbar_arrive_expect_tx(&bar[s], P::kBytes);
        bulk_g2s(ring + s * P::kBytes, a.pool.pages + ((int64_t)id * a.pool.h_kv + kv) * P::kBytes, P::kBytes, &bar[s]);
      }
    }
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue(i, 0);

  // ---- q: B operands of the score products, and the sums that the zero-points take
  uint32_t qb[NG][4];
  float qsum[NG][2];
  float fq[2];
  {
    const __nv_bfloat16* qrow = a.q + ((int64_t)b * a.H + h0 + g) * D;
    float x[NG][8];  // channels 32 kp + 8 t + i of head g
    float top = 0.f;
#pragma unroll
    for (int kp = 0; kp < NG; ++kp) {
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (g < heads) raw = *reinterpret_cast<const uint4*>(qrow + 32 * kp + 8 * t);
      const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[kp][2 * i] = __uint_as_float(r[i] << 16);
        x[kp][2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        top = fmaxf(top, fmaxf(fabsf(x[kp][2 * i]), fabsf(x[kp][2 * i + 1])));
        sum += x[kp][2 * i] + x[kp][2 * i + 1];
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      // D's columns 2t, 2t+1 are heads 2t, 2t+1: their sums sit in lanes 4 h
      qsum[kp][0] = __shfl_sync(0xffffffffu, sum, 8 * t) * a.scale_log2;
      qsum[kp][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4) * a.scale_log2;
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the head's power of two: its largest |q| in [2^13, 2^14), so that q / 16 too is
    // exact down to 2^-24 of it; the exponent is kept so that the inverse stays normal
    int e = 0;
    if (top > 0.f && isfinite(top)) {
      frexpf(top, &e);
      e = max(-100, min(100, 14 - e));
    }
    const float up = ldexpf(1.f, e);
    const float back = ldexpf(a.scale_log2, 24 - e);
    fq[0] = __shfl_sync(0xffffffffu, back, 8 * t);
    fq[1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
    for (int kp = 0; kp < NG; ++kp) {
      // code i of a word sits at bits 4 i: the pairs are (0, 4), (1, 5), (2, 6), (3, 7)
      qb[kp][0] = pack_h2(x[kp][0] * up, x[kp][4] * up);
      qb[kp][1] = pack_h2(x[kp][1] * up * 0.0625f, x[kp][5] * up * 0.0625f);
      qb[kp][2] = pack_h2(x[kp][2] * up, x[kp][6] * up);
      qb[kp][3] = pack_h2(x[kp][3] * up * 0.0625f, x[kp][7] * up * 0.0625f);
    }
  }

  float o[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[m][i] = 0.f;
  float mx[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f};
  const int tok_a = token_of(g >> 1, g & 1, 0);
  float* srow = a.scores ? a.scores + ((int64_t)b * a.pool.h_kv + kv) * a.max_pages * kPage * a.score_heads : nullptr;
  bool ok = true;
  int done = 0;

#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    if ((i & 31) == 0 && i > 0) {
      ids = ids_next;
      ids_next = load_ids(i + 32);
    }
    issue(i + ST - 1, i & ~31);
    const int s = i % ST;
    if (!__all_sync(0xffffffffu, mbar_wait(&bar[s], (i / ST) & 1))) {
      ok = false;
      break;
    }
    done = i + 1;
    const int page = p0 + warp + i * kWarps;
    const int left = len - page * kPage;  // tokens of the page (16 or more: all)
    const bool there = __shfl_sync(0xffffffffu, ids, i & 31) >= 0;
    const uint8_t* pg = ring + s * P::kBytes;
    // ---- scores of tokens tok_a (row g) and tok_a + 8 (row g + 8)
    float sa[2] = {-INFINITY, -INFINITY}, sb[2] = {-INFINITY, -INFINITY};
    if (there) {
      uint32_t ka[NG], kb[NG], ma[NG], mb[NG];
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(pg + tok_a * P::kRow + t * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(pg + (tok_a + 8) * P::kRow + t * 16);
        const uint4 z = *reinterpret_cast<const uint4*>(pg + P::kKMeta + tok_a * P::kMetaRow);
        const uint4 w = *reinterpret_cast<const uint4*>(pg + P::kKMeta + (tok_a + 8) * P::kMetaRow);
        ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
        kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
        ma[0] = z.x, ma[1] = z.y, ma[2] = z.z, ma[3] = z.w;
        mb[0] = w.x, mb[1] = w.y, mb[2] = w.z, mb[3] = w.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(pg + tok_a * P::kRow + t * 8);
        const uint2 y = *reinterpret_cast<const uint2*>(pg + (tok_a + 8) * P::kRow + t * 8);
        const uint2 z = *reinterpret_cast<const uint2*>(pg + P::kKMeta + tok_a * P::kMetaRow);
        const uint2 w = *reinterpret_cast<const uint2*>(pg + P::kKMeta + (tok_a + 8) * P::kMetaRow);
        ka[0] = x.x, ka[1] = x.y;
        kb[0] = y.x, kb[1] = y.y;
        ma[0] = z.x, ma[1] = z.y;
        mb[0] = w.x, mb[1] = w.y;
      }
      float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, zer[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int kp = 0; kp < NG; ++kp) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t wa = ka[kp], wb = kb[kp], va = wa >> 8, vb = wb >> 8;
        mma16816(d, wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u, wb & 0x00f000f0u, qb[kp][0], qb[kp][1]);
        mma16816(d, va & 0x000f000fu, vb & 0x000f000fu, va & 0x00f000f0u, vb & 0x00f000f0u, qb[kp][2], qb[kp][3]);
        const float2 sza = unpack_meta(ma[kp]), szb = unpack_meta(mb[kp]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          acc[0][c] = fmaf(sza.x, d[c], acc[0][c]);
          acc[1][c] = fmaf(szb.x, d[2 + c], acc[1][c]);
          zer[0][c] = fmaf(sza.y, qsum[kp][c], zer[0][c]);
          zer[1][c] = fmaf(szb.y, qsum[kp][c], zer[1][c]);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sa[c] = tok_a < left ? fmaf(acc[0][c], fq[c], zer[0][c]) : -INFINITY;
        sb[c] = tok_a + 8 < left ? fmaf(acc[1][c], fq[c], zer[1][c]) : -INFINITY;
      }
    }
    if (srow && 2 * t < heads) {
      float* d = srow + ((int64_t)page * kPage + tok_a) * a.score_heads + hb * kHeads + 2 * t;
      if (a.score_heads == 1) {
        d[0] = sa[0];
        d[8] = sb[0];
      } else {
        *reinterpret_cast<float2*>(d) = make_float2(sa[0], sa[1]);
        *reinterpret_cast<float2*>(d + 8 * a.score_heads) = make_float2(sb[0], sb[1]);
      }
    }
    if (there) {
      // ---- running maximum (per head; the same in the eight lanes that share its columns)
      const float c0 = fmaxf(sa[0], sb[0]), c1 = fmaxf(sa[1], sb[1]);
      if (__any_sync(0xffffffffu, c0 > mx[0] + kMoveMax || c1 > mx[1] + kMoveMax)) {
        float n0 = fmaxf(mx[0], c0), n1 = fmaxf(mx[1], c1);
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, w));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, w));
        }
        const float r0 = ex2(mx[0] - n0), r1 = ex2(mx[1] - n1);
        mx[0] = n0;
        mx[1] = n1;
        l[0] *= r0;
        l[1] *= r1;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          o[m][0] *= r0;
          o[m][1] *= r1;
          o[m][2] *= r0;
          o[m][3] *= r1;
        }
      }
      const float pa0 = ex2(sa[0] - mx[0]), pa1 = ex2(sa[1] - mx[1]);
      const float pb0 = ex2(sb[0] - mx[0]), pb1 = ex2(sb[1] - mx[1]);
      l[0] += pa0 + pb0;
      l[1] += pa1 + pb1;
      const uint32_t b0 = movm_trans(pack_h2(pa0, pa1)), b1 = movm_trans(pack_h2(pb0, pb1));
      // ---- V: the thread's D/8 channels (from (D/8) g) of tokens (e, f) = j, all in one group
      uint32_t vm[4], vw[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int tok = token_of(t, j & 1, j >> 1);
        if constexpr (D == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(pg + P::kV + tok * P::kRow + g * 8);
          vw[j][0] = x.x;
          vw[j][1] = x.y;
          vm[j] = *reinterpret_cast<const uint32_t*>(pg + P::kVMeta + tok * P::kMetaRow + (g >> 1) * 4);
        } else {
          vw[j][0] = *reinterpret_cast<const uint32_t*>(pg + P::kV + tok * P::kRow + g * 4);
          vm[j] = *reinterpret_cast<const uint32_t*>(pg + P::kVMeta + tok * P::kMetaRow + (g >> 2) * 4);
        }
        if (tok >= left) vm[j] = 0;  // whatever a free slot holds counts as 0
      }
      uint32_t sc[2], ze[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        sc[f] = __byte_perm(vm[2 * f], vm[2 * f + 1], 0x5410);
        ze[f] = __byte_perm(vm[2 * f], vm[2 * f + 1], 0x7632);
      }
      const __half2 k1024 = __halves2half2(__ushort_as_half(0x6400), __ushort_as_half(0x6400));
      const __half2 k16th = __halves2half2(__ushort_as_half(0x2c00), __ushort_as_half(0x2c00));
      const __half2 km64 = __halves2half2(__ushort_as_half(0xd400), __ushort_as_half(0xd400));
      // codes at bits 0..3 (or 4..7) of both halves -> fp16 values code * s + z
      auto even = [&](uint32_t y, int f) -> uint32_t {
        const uint32_t x = (y & 0x000f000fu) | 0x64006400u;  // 1024 + n
        const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&x), k1024);
        const __half2 v = __hfma2(n, *reinterpret_cast<const __half2*>(&sc[f]), *reinterpret_cast<const __half2*>(&ze[f]));
        return *reinterpret_cast<const uint32_t*>(&v);
      };
      auto odd = [&](uint32_t y, int f) -> uint32_t {
        const uint32_t x = (y & 0x00f000f0u) | 0x64006400u;  // 1024 + 16 n
        const __half2 n = __hfma2(*reinterpret_cast<const __half2*>(&x), k16th, km64);
        const __half2 v = __hfma2(n, *reinterpret_cast<const __half2*>(&sc[f]), *reinterpret_cast<const __half2*>(&ze[f]));
        return *reinterpret_cast<const uint32_t*>(&v);
      };
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        // channels 0..3 (x) and 4..7 (y) of word w, tokens j = 0, 1 and j = 2, 3 in the halves
        const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), y0 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
        const uint32_t x1 = __byte_perm(vw[2][w], vw[3][w], 0x5410), y1 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
        mma16816(o[4 * w], even(x0, 0), even(y0, 0), even(x1, 1), even(y1, 1), b0, b1);
        mma16816(o[4 * w + 1], odd(x0, 0), odd(y0, 0), odd(x1, 1), odd(y1, 1), b0, b1);
        mma16816(o[4 * w + 2], even(x0 >> 8, 0), even(y0 >> 8, 0), even(x1 >> 8, 1), even(y1 >> 8, 1), b0, b1);
        mma16816(o[4 * w + 3], odd(x0 >> 8, 0), odd(y0 >> 8, 0), odd(x1 >> 8, 1), odd(y1 >> 8, 1), b0, b1);
      }
    }
    __syncwarp();  // every lane has read the stage before its next copy is issued
  }
  if (!ok) {
    // give up: wait (with a limit) for the copies in flight before the memory is left
    if (lane == 0) set_status(a.status, kDevWaitTimeout);
    for (int i = done; i < min(mine, done + ST); ++i) mbar_wait(&bar[i % ST], (i / ST) & 1, 100000000ull);
  }
  // ---- join the four warps
#pragma unroll
  for (int w = 4; w < 32; w <<= 1) {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], w);
    l[1] += __shfl_xor_sync(0xffffffffu, l[1], w);
  }
  if (g == 0) {
    ml[warp][2 * t] = make_float2(mx[0], l[0]);
    ml[warp][2 * t + 1] = make_float2(mx[1], l[1]);
  }
  __syncthreads();  // the rings are read out; their bytes now hold the warps' outputs [warp][head][D]
  float* mo = reinterpret_cast<float*>(sm) + warp * kHeads * D;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int c = g * (D / 8) + (m >> 2) * 8 + (m & 3);  // rows g, g + 8 of tile m: channels c, c + 4
    mo[(2 * t) * D + c] = o[m][0];
    mo[(2 * t + 1) * D + c] = o[m][1];
    mo[(2 * t) * D + c + 4] = o[m][2];
    mo[(2 * t + 1) * D + c + 4] = o[m][3];
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(sm);
  const int64_t unit = ((int64_t)b * gridDim.y + blockIdx.y) * a.splits + split;
  for (int e = tid; e < heads * (D / 4); e += kThreads) {
    const int h = e / (D / 4), c = (e % (D / 4)) * 4;
    float top = kNoMax, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][h].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float r = ex2(ml[w][h].x - top);
      sum = fmaf(ml[w][h].y, r, sum);
      const float4 x = *reinterpret_cast<const float4*>(all + (w * kHeads + h) * D + c);
      v.x = fmaf(x.x, r, v.x);
      v.y = fmaf(x.y, r, v.y);
      v.z = fmaf(x.z, r, v.z);
      v.w = fmaf(x.w, r, v.w);
    }
    if (a.part_ml && c == 0) a.part_ml[unit * kHeads + h] = make_float2(top, sum);
    if (a.splits > 1) {
      *reinterpret_cast<float4*>(a.part_o + (unit * kHeads + h) * D + c) = v;
    } else {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
      uint2 w2;
      w2.x = *reinterpret_cast<const uint32_t*>(&lo);
      w2.y = *reinterpret_cast<const uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.H + h0 + h) * D + c) = w2;
    }
  }
}

// ---------------------------------------------------------------------------
// Join of the splits, and the weights.  Block x = 0 of a (sequence, KV head) joins
// the outputs; blocks x >= 1 add the probabilities of 1024 tokens each.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kJoinTokens = 1024;
constexpr int kJoinHeads = 32;  // heads whose maximum and 1 / sum a pass holds

template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const DecodeArgs a) {
  __shared__ float2 norm[kJoinHeads];  // maximum, 1 / sum
  const int tid = threadIdx.x;
  const int kv = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  pdl_launch_dependents();
  const int len = a.seq_lens[b];
  const bool good = len > 0 && len <= a.max_pages * kPage;
  const int used = good ? ((len + kPage - 1) / kPage + a.chunk - 1) / a.chunk : 0;  // splits that wrote
  const int units = a.pool.h_kv * a.head_blocks;
  const int token0 = ((int)blockIdx.x - 1) * kJoinTokens;
  if (blockIdx.x > 0 && token0 >= (good ? len : 0)) return;
  float add[kJoinTokens / kJoinThreads];
#pragma unroll
  for (int i = 0; i < kJoinTokens / kJoinThreads; ++i) add[i] = 0.f;
  for (int h0 = 0; h0 < a.group; h0 += kJoinHeads) {
    const int heads = min(kJoinHeads, a.group - h0);
    __syncthreads();
    // eight threads a head: the sequence's maximum and sum over its splits
    {
      const int h = h0 + tid / 8;
      float top = kNoMax, sum = 0.f;
      const bool mine = tid / 8 < heads;
      const float2* ml = a.part_ml +
                         (((int64_t)b * units + kv * a.head_blocks + h / kHeads) * a.splits) * kHeads + h % kHeads;
      if (mine)
        for (int s = tid & 7; s < used; s += 8) top = fmaxf(top, ml[(int64_t)s * kHeads].x);
#pragma unroll
      for (int w = 1; w < 8; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      if (mine)
        for (int s = tid & 7; s < used; s += 8) {
          const float2 v = ml[(int64_t)s * kHeads];
          sum = fmaf(v.y, ex2(v.x - top), sum);
        }
#pragma unroll
      for (int w = 1; w < 8; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      if (mine && (tid & 7) == 0) norm[tid / 8] = make_float2(top, sum == 0.f ? 0.f : 1.f / sum);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
      if (a.splits > 1)
        for (int e = tid; e < heads * (D / 4); e += kJoinThreads) {
          const int hh = e / (D / 4), h = h0 + hh, c = (e % (D / 4)) * 4;
          const int64_t unit0 = ((int64_t)b * units + kv * a.head_blocks + h / kHeads) * a.splits;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int s = 0; s < used; ++s) {
            const int64_t row = (unit0 + s) * kHeads + h % kHeads;
            const float r = ex2(a.part_ml[row].x - norm[hh].x);
            const float4 x = *reinterpret_cast<const float4*>(a.part_o + row * D + c);
            v.x = fmaf(x.x, r, v.x);
            v.y = fmaf(x.y, r, v.y);
            v.z = fmaf(x.z, r, v.z);
            v.w = fmaf(x.w, r, v.w);
          }
          const float inv = norm[hh].y;
          const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv);
          const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
          uint2 w2;
          w2.x = *reinterpret_cast<const uint32_t*>(&lo);
          w2.y = *reinterpret_cast<const uint32_t*>(&hi);
          *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.H + kv * a.group + h) * D + c) = w2;
        }
    } else {
      const float* rows = a.scores + (((int64_t)b * a.pool.h_kv + kv) * a.max_pages * kPage) * a.score_heads + h0;
#pragma unroll
      for (int i = 0; i < kJoinTokens / kJoinThreads; ++i) {
        const int tok = token0 + i * kJoinThreads + tid;
        if (tok < len)
          for (int h = 0; h < heads; ++h)
            add[i] = fmaf(ex2(rows[(int64_t)tok * a.score_heads + h] - norm[h].x), norm[h].y, add[i]);
      }
    }
  }
  if (blockIdx.x == 0) return;
#pragma unroll
  for (int i = 0; i < kJoinTokens / kJoinThreads; ++i) {
    const int tok = token0 + i * kJoinThreads + tid;
    if (tok >= len) continue;
    const int64_t page = a.block_table[(int64_t)b * a.max_pages + tok / kPage];
    if (page < 0 || page >= a.pool.n_pages) continue;
    // one addition a token and call: atomic only for a page that two tables share
    atomicAdd(&a.pool.weights[(page * a.pool.h_kv + kv) * kPage + tok % kPage], add[i]);
  }
}

}  // namespace

Kv4DecodePlan plan_kv4_decode(const Ctx& c, int batch, int max_pages, bool accumulate) {
  Kv4DecodePlan p;
  const starkv_config& f = c.cfg;
  p.head_blocks = (c.group + kHeads - 1) / kHeads;
  int sms = 148;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c.device);
  // chunks of equal pages, so that a batch of ragged sequences makes equal work: about four
  // rounds of the 4 CTAs that an SM holds, but 8 pages (2 a warp) at least
  const int64_t units = (int64_t)(batch > 0 ? batch : 1) * f.num_kv_heads * p.head_blocks;
  const int64_t want = ((int64_t)sms * 16 + units - 1) / units;
  int64_t chunk = max_pages > 0 ? (max_pages + want - 1) / want : 1;
  chunk = (chunk + kWarps - 1) / kWarps * kWarps;
  if (chunk < 8) chunk = 8;
  p.chunk = (int)chunk;
  p.splits = max_pages > 0 ? (max_pages + p.chunk - 1) / p.chunk : 1;
  p.score_heads = !accumulate ? 0 : c.group == 1 ? 1 : (c.group + 1) / 2 * 2;
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)units * p.splits * kHeads;
  p.off_ml = p.splits > 1 ? al(rows * f.head_dim * 4) : 0;
  p.off_scores = p.off_ml + (p.splits > 1 || accumulate ? al(rows * 8) : 0);
  p.ws_bytes = p.off_scores + al((size_t)(batch > 0 ? batch : 1) * f.num_kv_heads * max_pages * kPage * p.score_heads * 4);
  return p;
}

template <int D>
static cudaError_t launch_decode_d(const Ctx& c, const DecodeArgs& a, int batch, const Kv4DecodePlan& plan,
                                   bool accumulate, cudaStream_t s) {
  const int smem = DecodeSmem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_chained(kv4_decode_kernel<D>, dim3(plan.splits, c.cfg.num_kv_heads * plan.head_blocks, batch),
                     dim3(kThreads), (size_t)smem, s, 1u, a);
  if (e != cudaSuccess || (plan.splits == 1 && !accumulate)) return e;
  const unsigned chunks = accumulate ? (unsigned)(((int64_t)a.max_pages * kPage + kJoinTokens - 1) / kJoinTokens) : 0;
  return launch_chained(kv4_join_kernel<D>, dim3(1 + chunks, c.cfg.num_kv_heads, batch), dim3(kJoinThreads), 0, s, 1u,
                        a);
}

cudaError_t launch_kv4_decode(const Ctx& c, const starkv_kv4_cache& cache, const __nv_bfloat16* q,
                              const int32_t* block_table, const int32_t* seq_lens, int batch, int max_pages,
                              bool accumulate, __nv_bfloat16* out, void* ws, const Kv4DecodePlan& plan,
                              cudaStream_t s) {
  DecodeArgs a;
  a.q = q;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.H = c.cfg.num_q_heads;
  a.group = c.group;
  a.head_blocks = plan.head_blocks;
  a.max_pages = max_pages;
  a.chunk = plan.chunk;
  a.splits = plan.splits;
  a.score_heads = plan.score_heads;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)c.cfg.head_dim));
  a.pool = Kv4Pool{(uint8_t*)cache.pages, cache.weights, cache.n_pages, c.cfg.num_kv_heads};
  a.out = out;
  a.part_o = plan.splits > 1 ? (float*)ws : nullptr;
  a.part_ml = plan.splits > 1 || accumulate ? (float2*)((char*)ws + plan.off_ml) : nullptr;
  a.scores = accumulate ? (float*)((char*)ws + plan.off_scores) : nullptr;
  a.status = c.status;
  return c.cfg.head_dim == 64 ? launch_decode_d<64>(c, a, batch, plan, accumulate, s)
                              : launch_decode_d<128>(c, a, batch, plan, accumulate, s);
}

}  // namespace starkv
