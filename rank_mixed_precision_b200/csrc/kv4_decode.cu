// Decode attention over the 4-bit cache of full-width layers.
//
// The batch's pages, laid end to end as (sequence, unit, page) with a unit = one KV head
// and a block of at most eight of its query heads, are cut into equal stretches, one per
// CTA (four CTAs an SM, one round): ragged lengths cost no idle SMs, and a CTA's
// start (its queries, its first copies) is paid once for about a hundred pages.  A unit
// that a cut goes through leaves partial results, which a second kernel joins; where the
// tables are short, a CTA takes a whole unit and there is no second kernel.
// A CTA's four warps take a stretch's pages two at a time in turn, each with its own ring of
// bulk copies (one 16-token page of one head is one contiguous copy), its own reference of p
// and sum, and its own output accumulators.  Scores and outputs run on mma.sync
// m16n8k16: the eight query heads are the N of both products, so a page's codes are read
// once for all of them.  With N = 8 the products are small (2 x 16 x 8 x D per page) and
// their operands come out of 4-bit codes in registers, which tcgen05 (operands in shared
// or tensor memory, N of a whole tile) could only take after a round trip through shared
// memory.
// (Times in this file: a call's time on the GPU, calls back to back in a graph.)
//
//   scores   s[t, h] = sum_g ( sc[t, g] * sum_{c in g} n[t, c] q[h, c] ) + sum_g z[t, g] * sum_{c in g} q[h, c]
//     A = the codes n of the page's tokens, B = q.  A masked code (w & 0x000f000f) is
//     already two fp16 numbers, n 2^-24 (subnormal, exact), and (w & 0x00f000f0) is
//     16 n 2^-24, so widening costs one AND for two codes; q is bf16, scaled by a power
//     of two per head (and by 1/16 for the odd codes), so it too is exact in fp16.  The
//     products are exact and the sums fp32: the probabilities that are added to the
//     cache's weights keep fp32 accuracy.
//   output   o[c, h] = sum_t v[t, c] p[t, h]
//     A = V^T, widened to fp16 (code * s + z, one rounding), B = p in fp16.  p is taken against a
//     reference 2^7 below the largest score when that last moved it, and the reference moves when p
//     would pass 2^15: fp16 then holds probabilities down to 2^-32 of the largest (half a step; with the
//     maximum itself as reference 2^-25, and the tail of a context of millions of tokens fell out of the
//     output while the sum, in fp32, still held it).
#include <algorithm>

#include "full.cuh"
#include "sm100.cuh"

namespace starkv {

using namespace sm100;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kHeads = 8;            // query heads of one CTA (the N of the products)
// CTAs of an SM: 128 registers a thread, of which 108 bytes spill at head width 128 (none at 64).  Five, with 102
// registers, were slower (one sequence of 32768 tokens: 68 us for 59 at the time).
constexpr int kCtas = 4;
// A CTA takes a whole unit where tables hold at most kWholePages pages, or kWholePagesMany where there
// are kManyUnits units or more; else the pages are cut evenly (a second segment's start in most CTAs,
// and the join).  Whole and cut in us: 4 heads of 64, 512 tokens 6.0 and 8.5, 2048 tokens 15.2 and 9.2;
// heads of 128, 64 units of 1024 tokens 12.5 and 12.3, 256 units of 2048 28.3 and 33.5, of 4096 51.7
// and 50.6 (equal lengths: ragged ones favour the cut).
constexpr int kWholePages = 32;
constexpr int kWholePagesMany = 128;
constexpr int kManyUnits = 64;
// CTAs of a unit at most: more parts cost the join more than they spare.  (At most 32, 74, 148 and any
// number, us: 8 heads of 128 over one, 100000 tokens 38, 25, 22, 46; 40 of 64 over one, 20000 tokens 14, 15, 19, 19.)
constexpr int kMostParts = 74;
constexpr float kBelow = 7.f;        // the reference of p, below the largest score (log2),
constexpr float kMoveMax = 15.f;     // and how far scores may pass it before it moves: p <= 2^15, fp16 ends at 2^16
constexpr float kNoMax = -3.402823466e38f;  // reference before the first score: finite, and below all scores

struct DecodeArgs {
  const __nv_bfloat16* q;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int H, group, head_blocks, units, batch, max_pages, ctas, score_heads;  // ctas 0: one per (sequence, unit)
  float scale_log2;        // log2(e) / sqrt(D)
  Kv4Pool pool;
  __nv_bfloat16* out;
  float* part_o;           // [ctas][2][8][D], relative to the part's reference: [0] of a unit that began before the
  float2* part_ml;         // [ctas][2][8] (reference, sum)                   CTA's stretch, [1] of one that goes on behind
  float2* unit_ml;         // [B][units][8], of units within one CTA (NULL: not asked for)
  int64_t* before;         // [B + 1] pages before each sequence, and of all (ctas > 0)
  float* scores;           // [B][h_kv][max_pages * 16][score_heads], log2 units (NULL: not asked for)
  unsigned int* status;
  int side, outs;          // the join: heads a block joins side by side, and its blocks of a (sequence, KV head) for that
};

template <int D>
struct DecodeSmem {
  static constexpr int kPair = 2 * Kv4<D>::kBytes;   // a stage: two pages
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kRing = kWarps * kStages * kPair;
  static constexpr int kMerge = kWarps * kHeads * D * 4;  // shares the ring's bytes
  static constexpr int kBytes = (kRing > kMerge ? kRing : kMerge);
};

// Pages of sequence b; 0 where its length is bad.
__device__ __forceinline__ int pages_of(const DecodeArgs& a, int b) {
  const int len = a.seq_lens[b];
  return len < 0 || len > a.max_pages * kPage ? 0 : (len + kPage - 1) / kPage;
}

// Sum of value over the block's threads (T of them; sum: scratch of T / 32).
template <int T>
__device__ __forceinline__ int64_t block_sum(int64_t value, int64_t* sum) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) value += __shfl_xor_sync(0xffffffffu, value, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = value;
  __syncthreads();
  value = 0;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) value += sum[w];
  return value;
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Adds to four floats, each atomically; p is 16-byte aligned.
__device__ __forceinline__ void red_add4(float* p, const float (&x)[4]) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3])
               : "memory");
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
__global__ void __launch_bounds__(kThreads, kCtas) kv4_decode_kernel(const DecodeArgs a) {
  using P = Kv4<D>;
  using SM = DecodeSmem<D>;
  constexpr int NG = P::kGroups;
  constexpr int MT = D / 16;   // 16-channel tiles of the output
  constexpr int ST = SM::kStages;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(8) uint64_t full[kWarps * ST];
  __shared__ float2 ml[kWarps][kHeads];
  __shared__ int64_t sums[kWarps];
  __shared__ int64_t begin[2];  // the stretch's first sequence, and the pages before it
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (lane < ST) mbar_init(&full[warp * ST + lane], 2);
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();

  // ---- the stretch: positions pos .. end - 1, in sequence b (whose first page is at units * before)
  int b;
  int64_t pos, end, before;
  if (a.ctas == 0) {
    b = blockIdx.x / a.units;
    before = 0;
    const int pages = pages_of(a, b);
    const int u = blockIdx.x % a.units;
    pos = (int64_t)u * pages;
    end = pos + pages;
    if (tid == 0 && u == 0 && pages == 0 && a.seq_lens[b] != 0) set_status(a.status, STARKV_DEV_BAD_SEQ_LEN);
    if (pages == 0) {
      const int heads = min(kHeads, a.group - u % a.head_blocks * kHeads);
      const int h0 = u / a.head_blocks * a.group + u % a.head_blocks * kHeads;
      for (int i = tid; i < heads * D; i += kThreads) a.out[((int64_t)b * a.H + h0) * D + i] = __float2bfloat16_rn(0.f);
      return;
    }
    __syncthreads();
  } else {
    int64_t mine = 0;
    for (int i = tid; i < a.batch; i += kThreads) {
      const int pages = pages_of(a, i);
      if (blockIdx.x == 0 && pages == 0 && a.seq_lens[i] != 0) set_status(a.status, STARKV_DEV_BAD_SEQ_LEN);
      mine += pages;
    }
    const int64_t total = block_sum<kThreads>(mine, sums) * a.units;
    pos = cut(blockIdx.x, total, a.ctas);
    end = cut(blockIdx.x + 1, total, a.ctas);
    if (blockIdx.x == 0 && tid == 0) a.before[a.batch] = total / a.units;
    if (pos == end) return;
    // the last sequence that starts at or before pos, among those that have pages
    int64_t carry = 0;
    for (int i0 = 0; i0 < a.batch; i0 += kThreads) {
      const int pages = i0 + tid < a.batch ? pages_of(a, i0 + tid) : 0;
      int64_t inc = pages;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncthreads();
      if (lane == 31) sums[warp] = inc;
      __syncthreads();
      int64_t first = carry + inc - pages;
      for (int w = 0; w < warp; ++w) first += sums[w];
      if (blockIdx.x == 0 && i0 + tid < a.batch) a.before[i0 + tid] = first;
      if (pages > 0 && first * a.units <= pos && pos < (first + pages) * a.units) {
        begin[0] = i0 + tid;
        begin[1] = first;
      }
      for (int w = 0; w < kWarps; ++w) carry += sums[w];
    }
    __syncthreads();
    b = (int)begin[0];
    before = begin[1];
  }

  uint8_t* ring = sm + warp * ST * SM::kPair;
  uint64_t* bar = full + warp * ST;
  int s = 0;           // the ring's next stage
  uint32_t ph = 0;     // and its phase
  const int tok_a = token_of(g >> 1, g & 1, 0);
  bool ok = true;

#pragma unroll 1
  while (pos < end) {
    const int pages = pages_of(a, b);
    const int64_t in_seq = pos - before * a.units;
    if (in_seq >= (int64_t)pages * a.units) {
      before += pages;
      ++b;
      continue;
    }
    const int len = a.seq_lens[b];
    const int u = (int)(in_seq / pages);
    const int p0 = (int)(in_seq - (int64_t)u * pages);
    const int p1 = (int)min((int64_t)pages, p0 + (end - pos));
    pos += p1 - p0;
    const int kv = u / a.head_blocks, hb = u % a.head_blocks;
    const int heads = min(kHeads, a.group - hb * kHeads);
    const int h0 = kv * a.group + hb * kHeads;
    // ---- the warp's copies: pairs of pages first + 8 i, first + 8 i + 1
    const int first = p0 + 2 * warp;
    const int mine = (p1 - first + 2 * kWarps - 1) / (2 * kWarps);  // pairs of this warp (may be <= 0; the last may lack its second page)
    const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
    const uint8_t* head_pages = a.pool.pages + (int64_t)kv * P::kBytes;
    int32_t ids = 0, ids_next = 0;  // lane 2 i + f: page f of iteration (base of 16) + i, and of 16 further
    auto load_ids = [&](int base) -> int32_t {
      const int page = first + (base + (lane >> 1)) * 2 * kWarps + (lane & 1);
      int32_t id = -1;
      if (page < p1) {
        id = table[page];
        if (id < 0 || id >= a.pool.n_pages) {
          set_status(a.status, STARKV_DEV_BAD_PAGE);
          id = -1;
        }
      }
      return id;
    };
    ids = load_ids(0);
    ids_next = load_ids(16);
    uint32_t there = __ballot_sync(0xffffffffu, ids >= 0);
    // issue the copies of iteration i to stage st: the lanes that hold the pages' ids do
    auto issue = [&](int i, int base, int st) {
      if ((lane >> 1) == (i & 15) && i < mine) {
        const int32_t id = i - base < 16 ? ids : ids_next;
        if (id < 0) {
          mbar_arrive(&bar[st]);  // nothing to copy: there is no page, or it is left out
        } else {
          mbar_arrive_expect_tx(&bar[st], P::kBytes);
          bulk_g2s(ring + st * SM::kPair + (lane & 1) * P::kBytes, head_pages + (int64_t)id * a.pool.h_kv * P::kBytes,
                   P::kBytes, &bar[st]);
        }
      }
    };
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) issue(i, 0, s + i < ST ? s + i : s + i - ST);

    // ---- q: B operands of the score products, and the sums that the zero-points take
    uint32_t qb[NG][4];
    uint32_t qz[2] = {0, 0};
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
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[kp][2 * i] = __uint_as_float(r[i] << 16);
          x[kp][2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
          top = fmaxf(top, fmaxf(fabsf(x[kp][2 * i]), fabsf(x[kp][2 * i + 1])));
        }
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
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[kp][i] *= up;
          sum += x[kp][i];
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        // the zero-points' operand: the head's sum in three fp16 pieces (33 bits, as good as fp32), piece e of
        // group kp at k = NG e + kp; scaled by 2^-5 the first is at most 2^14
        sum *= 0.03125f;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          const __half piece = __float2half_rn(sum);
          sum -= __half2float(piece);
          const int k = NG * e + kp;  // the lane holds k = 2 t, 2 t + 1 (and 8 further)
          if (t == (k & 7) >> 1) qz[k >> 3] |= (uint32_t)__half_as_ushort(piece) << (16 * (k & 1));
        }
        // code i of a word sits at bits 4 i: the pairs are (0, 4), (1, 5), (2, 6), (3, 7)
        qb[kp][0] = pack_h2(x[kp][0], x[kp][4]);
        qb[kp][1] = pack_h2(x[kp][1] * 0.0625f, x[kp][5] * 0.0625f);
        qb[kp][2] = pack_h2(x[kp][2], x[kp][6]);
        qb[kp][3] = pack_h2(x[kp][3] * 0.0625f, x[kp][7] * 0.0625f);
      }
    }

    float o[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[m][i] = 0.f;
    float mx[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f};
    float* srow = nullptr;  // scores of the warp's pair, from token tok_a and head 2 t on
    if (a.scores && 2 * t < heads)
      srow = a.scores + (((int64_t)b * a.pool.h_kv + kv) * a.max_pages * kPage + (int64_t)first * kPage + tok_a) * a.score_heads +
             hb * kHeads + 2 * t;
    int left = len - first * kPage;  // tokens of the pair's pages (32 or more: all)
    int done = 0;

#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      if ((i & 15) == 0 && i > 0) {
        ids = ids_next;
        ids_next = load_ids(i + 16);
        there = __ballot_sync(0xffffffffu, ids >= 0);
      }
      issue(i + ST - 1, i & ~15, s == 0 ? ST - 1 : s - 1);
      if (!__all_sync(0xffffffffu, mbar_test(&bar[s], ph)) && !__all_sync(0xffffffffu, mbar_wait(&bar[s], ph))) {
        ok = false;
        break;
      }
      done = i + 1;
      const uint8_t* pair_at = ring + s * SM::kPair;
      if (++s == ST) {
        s = 0;
        ph ^= 1;
      }
      const uint32_t in = there >> (2 * (i & 15));
      const int held[2] = {in & 1 ? left : 0, in & 2 ? left - kPage : 0};  // the pages' tokens that count
      // ---- scores of tokens tok_a (row g) and tok_a + 8 (row g + 8) of both pages, without fq
      float sa[2][2], sb[2][2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint8_t* pg = pair_at + f * P::kBytes;
        uint32_t ka[NG], kb[NG], ma[NG], mb[NG];
        uint32_t za, zb;  // A of the zero-points' product: the k-th column holds group k mod NG's
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(pg + tok_a * P::kRow + t * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(pg + (tok_a + 8) * P::kRow + t * 16);
          const uint4 z = *reinterpret_cast<const uint4*>(pg + P::kKMeta + tok_a * P::kMetaRow);
          const uint4 w = *reinterpret_cast<const uint4*>(pg + P::kKMeta + (tok_a + 8) * P::kMetaRow);
          ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
          kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
          ma[0] = z.x, ma[1] = z.y, ma[2] = z.z, ma[3] = z.w;
          mb[0] = w.x, mb[1] = w.y, mb[2] = w.z, mb[3] = w.w;
          za = t & 1 ? __byte_perm(z.z, z.w, 0x7632) : __byte_perm(z.x, z.y, 0x7632);
          zb = t & 1 ? __byte_perm(w.z, w.w, 0x7632) : __byte_perm(w.x, w.y, 0x7632);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(pg + tok_a * P::kRow + t * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(pg + (tok_a + 8) * P::kRow + t * 8);
          const uint2 z = *reinterpret_cast<const uint2*>(pg + P::kKMeta + tok_a * P::kMetaRow);
          const uint2 w = *reinterpret_cast<const uint2*>(pg + P::kKMeta + (tok_a + 8) * P::kMetaRow);
          ka[0] = x.x, ka[1] = x.y;
          kb[0] = y.x, kb[1] = y.y;
          ma[0] = z.x, ma[1] = z.y;
          mb[0] = w.x, mb[1] = w.y;
          za = __byte_perm(z.x, z.y, 0x7632);
          zb = __byte_perm(w.x, w.y, 0x7632);
        }
        float d[4];
        mma16816_zero(d, za, zb, za, zb, qz[0], qz[1]);
        // 2^5 (the pieces' scale) 2^-24 (the unit of the codes' products)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sa[f][c] = d[c] * 1.9073486328125e-6f;
          sb[f][c] = d[2 + c] * 1.9073486328125e-6f;
        }
#pragma unroll
        for (int kp = 0; kp < NG; ++kp) {
          const uint32_t wa = ka[kp], wb = kb[kp], va = wa >> 8, vb = wb >> 8;
          mma16816_zero(d, wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u, wb & 0x00f000f0u, qb[kp][0], qb[kp][1]);
          mma16816(d, va & 0x000f000fu, vb & 0x000f000fu, va & 0x00f000f0u, vb & 0x00f000f0u, qb[kp][2], qb[kp][3]);
          const float sca = __low2float(*reinterpret_cast<const __half2*>(&ma[kp]));
          const float scb = __low2float(*reinterpret_cast<const __half2*>(&mb[kp]));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            sa[f][c] = fmaf(sca, d[c], sa[f][c]);
            sb[f][c] = fmaf(scb, d[2 + c], sb[f][c]);
          }
        }
        if (held[f] < kPage) {  // a sequence's last page, or one that is left out: free slots may hold anything
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (tok_a >= held[f]) sa[f][c] = -INFINITY;
            if (tok_a + 8 >= held[f]) sb[f][c] = -INFINITY;
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sa[f][c] *= fq[c];
          sb[f][c] *= fq[c];
        }
        if (srow && (f == 0 || first + i * 2 * kWarps + 1 < p1)) {
          float* to = srow + f * kPage * a.score_heads;
          if (a.score_heads == 1) {
            to[0] = sa[f][0];
            to[8] = sb[f][0];
          } else {
            *reinterpret_cast<float2*>(to) = make_float2(sa[f][0], sa[f][1]);
            *reinterpret_cast<float2*>(to + 8 * a.score_heads) = make_float2(sb[f][0], sb[f][1]);
          }
        }
      }
      if (srow) srow += 2 * kWarps * kPage * a.score_heads;
      left -= 2 * kWarps * kPage;
      // ---- reference (per head; the same in the eight lanes that share its columns)
      const float c0 = fmaxf(fmaxf(sa[0][0], sb[0][0]), fmaxf(sa[1][0], sb[1][0]));
      const float c1 = fmaxf(fmaxf(sa[0][1], sb[0][1]), fmaxf(sa[1][1], sb[1][1]));
      // (the difference is exact where it matters; a sum with kMoveMax may round up past the score)
      if (__any_sync(0xffffffffu, c0 - mx[0] > kMoveMax || c1 - mx[1] > kMoveMax)) {
        float n0 = fmaxf(mx[0], c0 - kBelow), n1 = fmaxf(mx[1], c1 - kBelow);
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
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint8_t* pg = pair_at + f * P::kBytes;
        const float pa0 = ex2(sa[f][0] - mx[0]), pa1 = ex2(sa[f][1] - mx[1]);
        const float pb0 = ex2(sb[f][0] - mx[0]), pb1 = ex2(sb[f][1] - mx[1]);
        l[0] += pa0 + pb0;
        l[1] += pa1 + pb1;
        const uint32_t b0 = movm_trans(pack_h2(pa0, pa1)), b1 = movm_trans(pack_h2(pb0, pb1));
        // ---- V: the thread's D/8 channels (from (D/8) g) of tokens (e, h) = j, all in one group
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
        }
        if (held[f] < kPage) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (token_of(t, j & 1, j >> 1) >= held[f]) vm[j] = 0;
        }
        uint32_t sc[2], ze[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sc[h] = __byte_perm(vm[2 * h], vm[2 * h + 1], 0x5410);
          ze[h] = __byte_perm(vm[2 * h], vm[2 * h + 1], 0x7632);
        }
        const __half2 k1024 = __halves2half2(__ushort_as_half(0x6400), __ushort_as_half(0x6400));
        const __half2 k16th = __halves2half2(__ushort_as_half(0x2c00), __ushort_as_half(0x2c00));
        const __half2 km64 = __halves2half2(__ushort_as_half(0xd400), __ushort_as_half(0xd400));
        // codes at bits 0..3 (or 4..7) of both halves -> fp16 values code * s + z
        auto even = [&](uint32_t y, int h) -> uint32_t {
          const uint32_t x = (y & 0x000f000fu) | 0x64006400u;  // 1024 + n
          const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&x), k1024);
          const __half2 v = __hfma2(n, *reinterpret_cast<const __half2*>(&sc[h]), *reinterpret_cast<const __half2*>(&ze[h]));
          return *reinterpret_cast<const uint32_t*>(&v);
        };
        auto odd = [&](uint32_t y, int h) -> uint32_t {
          const uint32_t x = (y & 0x00f000f0u) | 0x64006400u;  // 1024 + 16 n
          const __half2 n = __hfma2(*reinterpret_cast<const __half2*>(&x), k16th, km64);
          const __half2 v = __hfma2(n, *reinterpret_cast<const __half2*>(&sc[h]), *reinterpret_cast<const __half2*>(&ze[h]));
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
      __syncwarp();  // every lane has read the stage before its next copies are issued
    }
    if (!ok) {
      // give up: wait (with a limit) for the copies in flight before the memory is left
      if (lane == 0) set_status(a.status, kDevWaitTimeout);
      for (int i = done; i < min(mine, done + ST); ++i) {
        mbar_wait(&bar[s], ph, 100000000ull);
        if (++s == ST) {
          s = 0;
          ph ^= 1;
        }
      }
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
    const bool stop = __syncthreads_or(!ok);  // the rings are read out; their bytes now hold the warps' outputs [warp][head][D]
    float* mo = reinterpret_cast<float*>(sm) + warp * kHeads * D;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int c = g * (D / 8) + (m >> 2) * 8 + (m & 3);  // rows g, g + 8 of tile m: channels c, c + 4
      if (2 * t < heads) {
        mo[(2 * t) * D + c] = o[m][0];
        mo[(2 * t) * D + c + 4] = o[m][2];
      }
      if (2 * t + 1 < heads) {
        mo[(2 * t + 1) * D + c] = o[m][1];
        mo[(2 * t + 1) * D + c + 4] = o[m][3];
      }
    }
    __syncthreads();
    const float* all = reinterpret_cast<const float*>(sm);
    const bool whole = p0 == 0 && p1 == pages;
    const int64_t part = ((int64_t)blockIdx.x * 2 + (p0 == 0)) * kHeads;
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
      if (!whole) {
        if (c == 0) a.part_ml[part + h] = make_float2(top, sum);
        *reinterpret_cast<float4*>(a.part_o + (part + h) * D + c) = v;
      } else {
        if (c == 0 && a.unit_ml) a.unit_ml[((int64_t)b * a.units + u) * kHeads + h] = make_float2(top, sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        uint2 w2;
        w2.x = *reinterpret_cast<const uint32_t*>(&lo);
        w2.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.H + h0 + h) * D + c) = w2;
      }
    }
    if (stop) return;
    fence_async_smem();  // the outputs' bytes become the ring again
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Join of the parts, and the weights.  Blocks x < outs of a (sequence, KV head) join the
// outputs of its units that a cut went through (and write an empty sequence's zero rows), `side`
// heads each: the more parts a unit has, the fewer heads a block, and the more threads share a
// head's parts out.  (Two sequences of 21648 tokens, 14 heads of 64 over 2, 74 parts a unit:
// 14 us; all seven heads in one block 22.)  The other blocks add the probabilities of 1024 tokens
// each: a warp reads the scores of 32 tokens at a time, and a transpose among four lanes gives
// each lane four neighbours of one page, which it adds at once: one page to look up and one
// addition of 16 bytes.  (Decode and
// join of 32 sequences of 4096 to 8192 tokens, 32 heads over 8: 84 us; with a token a lane at a
// time, and the norms read for each, 92 for 87 at the time; with six blocks an SM, not eight, 88.)
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kJoinTokens = 4 * kJoinThreads;
constexpr int kJoinHeads = 32;  // heads whose reference and 1 / sum a pass holds

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 8) kv4_join_kernel(const DecodeArgs a) {
  __shared__ float2 norm[kJoinHeads];  // reference, 1 / sum
  __shared__ float4 acc[kJoinThreads];
  const int tid = threadIdx.x;
  const int kv = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  pdl_launch_dependents();
  const int pages = pages_of(a, b);
  const int len = pages > 0 ? a.seq_lens[b] : 0;
  const bool joins = (int)blockIdx.x < a.outs;
  const int token0 = ((int)blockIdx.x - a.outs) * kJoinTokens;
  if (!joins && token0 >= len) return;
  const int first_head = joins ? (int)blockIdx.x * a.side : 0, last_head = joins ? min(first_head + a.side, a.group) : a.group;
  if (pages == 0) {
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + ((int64_t)b * a.H + kv * a.group) * D);
    if (a.ctas > 0)
      for (int i = first_head * (D / 2) + tid; i < last_head * (D / 2); i += kJoinThreads) out[i] = 0u;
    return;
  }
  const int64_t before = a.ctas > 0 ? a.before[b] * a.units : 0, total = a.ctas > 0 ? a.before[a.batch] * a.units : 0;
  // the lane's scores are those of tokens at + 32 i, its sums in the end those of tokens quad .. quad + 3
  const int lane = tid & 31, at = token0 + (tid >> 5) * 128 + lane, quad = at - lane + (lane & 3) * 32 + (lane >> 2) * 4;
  // (asked for before the sums are)
  const int64_t page = !joins && quad < len ? a.block_table[(int64_t)b * a.max_pages + quad / kPage] : -1;
  // the CTAs whose stretches hold unit u's first and last page
  auto ctas_of = [&](int u, int64_t& c0, int64_t& c1) {
    const int64_t first = before + (int64_t)u * pages;
    c0 = a.ctas > 0 ? cta_of(first, total, a.ctas) : 0;
    c1 = a.ctas > 0 ? cta_of(first + pages - 1, total, a.ctas) : 0;
  };
  float add[4] = {0.f, 0.f, 0.f, 0.f};
  for (int h0 = first_head; h0 < last_head; h0 += kJoinHeads) {
    const int heads = min(kJoinHeads, last_head - h0);
    __syncthreads();
    // a warp, or eight threads, a head: the sequence's reference and sum over its parts
    {
      const int per = heads <= kJoinThreads / 32 ? 32 : 8, one = tid & (per - 1), hh = tid / per;
      const int h = h0 + hh;
      const bool mine = hh < heads;
      float top = kNoMax, sum = 0.f;
      int64_t c0 = 0, c1 = 0;
      const int u = kv * a.head_blocks + h / kHeads;
      if (mine) ctas_of(u, c0, c1);
      const bool parts = mine && c0 < c1;
      auto ml = [&](int64_t c) { return a.part_ml[(c * 2 + (c == c0)) * kHeads + h % kHeads]; };
      if (parts)
        for (int64_t c = c0 + one; c <= c1; c += per) top = fmaxf(top, ml(c).x);
      for (int w = 1; w < per; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      if (parts)
        for (int64_t c = c0 + one; c <= c1; c += per) {
          const float2 v = ml(c);
          sum = fmaf(v.y, ex2(v.x - top), sum);
        }
      for (int w = 1; w < per; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      if (mine && !parts && a.unit_ml) {
        const float2 v = a.unit_ml[((int64_t)b * a.units + u) * kHeads + h % kHeads];
        top = v.x;
        sum = v.y;
      }
      if (mine && one == 0) norm[hh] = make_float2(top, sum == 0.f ? 0.f : 1.f / sum);
    }
    __syncthreads();
    if (joins) {
      // kRow threads hold a head's row; `side` heads go side by side, and what threads are left share a head's
      // parts out, then add up
      constexpr int kRow = D / 4;
      constexpr int kRows = kJoinThreads / kRow;
      const int side = a.side, ways = kRows / side;
      const int c4 = (tid % kRow) * 4, way = tid / kRow / side, hh = tid / kRow % side, h = h0 + hh;
      int64_t c0, c1;
      ctas_of(kv * a.head_blocks + h0 / kHeads, c0, c1);
      if (c0 == c1) return;  // (the same for the whole block: the heads side by side share a unit)
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (hh < heads)
#pragma unroll 2
        for (int64_t c = c0 + way; c <= c1; c += ways) {
          const int64_t row = (c * 2 + (c == c0)) * kHeads + h % kHeads;
          const float r = ex2(a.part_ml[row].x - norm[hh].x);
          const float4 x = *reinterpret_cast<const float4*>(a.part_o + row * D + c4);
          v.x = fmaf(x.x, r, v.x);
          v.y = fmaf(x.y, r, v.y);
          v.z = fmaf(x.z, r, v.z);
          v.w = fmaf(x.w, r, v.w);
        }
      if (ways > 1) {
        acc[tid] = v;
        __syncthreads();
      }
      if (way == 0 && hh < heads) {
        for (int w = 1; w < ways && w <= c1 - c0; ++w) {
          const float4 x = acc[w * side * kRow + tid];
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
        }
        const float inv = norm[hh].y;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        uint2 w2;
        w2.x = *reinterpret_cast<const uint32_t*>(&lo);
        w2.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.H + kv * a.group + h) * D + c4) = w2;
      }
      return;
    } else {
      const float* row = a.scores + (((int64_t)b * a.pool.h_kv + kv) * a.max_pages * kPage + at) * a.score_heads + h0;
      if (a.score_heads <= 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (at + i * 32 >= len) continue;
          const float* x = row + i * 32 * a.score_heads;
          add[i] = ex2(x[0] - norm[0].x) * norm[0].y;
          if (a.score_heads == 2) add[i] = fmaf(ex2(x[1] - norm[1].x), norm[1].y, add[i]);
        }
      } else {
#pragma unroll 1
        for (int h = 0; h < heads; h += 4) {
          float4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (at + i * 32 < len) x[i] = *reinterpret_cast<const float4*>(row + i * 32 * a.score_heads + h);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (h + e >= heads) break;
            const float2 n = norm[h + e];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              add[i] = fmaf(ex2((e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w) - n.x), n.y, add[i]);
          }
        }
      }
    }
  }
  // 4 x 4 transpose among the lanes 4 q .. 4 q + 3
#pragma unroll
  for (int w = 1; w < 4; w <<= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(i & w)) {
        const float got = __shfl_xor_sync(0xffffffffu, up ? add[i] : add[i | w], w);
        (up ? add[i] : add[i | w]) = got;
      }
  }
  if (page < 0 || page >= a.pool.n_pages) return;  // (-1 behind the last token)
  // one addition a token and call: atomic only for a page that two tables share
  float* to = &a.pool.weights[(page * a.pool.h_kv + kv) * kPage + quad % kPage];
  if (quad + 4 <= len) {
    red_add4(to, add);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (quad + e < len) atomicAdd(to + e, add[e]);
  }
}

}  // namespace

Kv4DecodePlan plan_kv4_decode(const Ctx& c, int batch, int max_pages, bool accumulate) {
  Kv4DecodePlan p;
  const starkv_config& f = c.cfg;
  p.head_blocks = (c.group + kHeads - 1) / kHeads;
  p.units = f.num_kv_heads * p.head_blocks;
  const int sms = sm_count(c);
  // one round of CTAs at most, with 8 pages (a pair a warp) at least where the tables are full
  const bool whole = max_pages <= ((int64_t)batch * p.units >= kManyUnits ? kWholePagesMany : kWholePages);
  const int64_t most = (int64_t)batch * p.units * max_pages;
  const int64_t round = std::min((int64_t)sms * kCtas, (int64_t)batch * p.units * kMostParts);
  p.ctas = whole ? 0 : (int)(most / 8 < round ? most / 8 : round);
  p.score_heads = !accumulate ? 0 : c.group <= 2 ? c.group : (c.group + 3) / 4 * 4;
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)p.ctas * 2 * kHeads;
  p.off_ml = al(rows * f.head_dim * 4);
  p.off_unit = p.off_ml + al(rows * 8);
  p.off_before = p.off_unit + (accumulate ? al((size_t)batch * p.units * kHeads * 8) : 0);
  p.off_scores = p.off_before + (p.ctas > 0 ? al(((size_t)batch + 1) * 8) : 0);
  p.ws_bytes = p.off_scores + al((size_t)batch * f.num_kv_heads * max_pages * kPage * p.score_heads * 4);
  return p;
}

template <int D>
static cudaError_t launch_decode_d(const Ctx& c, const DecodeArgs& a, cudaStream_t s) {
  const int smem = DecodeSmem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const unsigned blocks = a.ctas > 0 ? (unsigned)a.ctas : (unsigned)(a.batch * a.units);
  e = launch_chained(kv4_decode_kernel<D>, dim3(blocks), dim3(kThreads), (size_t)smem, s, 1u, a);
  if (e != cudaSuccess || (a.ctas == 0 && !a.scores)) return e;
  const unsigned chunks = a.scores ? (unsigned)(((int64_t)a.max_pages * kPage + kJoinTokens - 1) / kJoinTokens) : 0;
  return launch_chained(kv4_join_kernel<D>, dim3(a.outs + chunks, c.cfg.num_kv_heads, a.batch), dim3(kJoinThreads), 0, s, 1u,
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
  a.units = plan.units;
  a.batch = batch;
  a.max_pages = max_pages;
  a.ctas = plan.ctas;
  a.score_heads = plan.score_heads;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)c.cfg.head_dim));
  a.pool = Kv4Pool{(uint8_t*)cache.pages, cache.weights, cache.n_pages, c.cfg.num_kv_heads};
  a.out = out;
  a.part_o = (float*)ws;
  a.part_ml = (float2*)((char*)ws + plan.off_ml);
  a.unit_ml = accumulate ? (float2*)((char*)ws + plan.off_unit) : nullptr;
  a.before = (int64_t*)((char*)ws + plan.off_before);
  a.scores = accumulate ? (float*)((char*)ws + plan.off_scores) : nullptr;
  a.status = c.status;
  // heads side by side in the join: at most a unit's, fewer where a head's threads would take more than two parts each
  const int rows = kJoinThreads / (c.cfg.head_dim / 4), parts = plan.ctas / (batch * plan.units) + 1;
  a.side = 1;
  while (a.side < c.group && a.side < kHeads) a.side *= 2;
  while (a.side > 1 && rows / a.side * 2 < parts) a.side /= 2;
  a.outs = plan.ctas > 0 ? (c.group + a.side - 1) / a.side : 0;
  return c.cfg.head_dim == 64 ? launch_decode_d<64>(c, a, s) : launch_decode_d<128>(c, a, s);
}

}  // namespace starkv
