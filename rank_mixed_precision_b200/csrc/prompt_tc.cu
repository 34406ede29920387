// Full-width layers: causal attention of packed prompts, and the attention weights
// of a prompt, on tcgen05 / TMEM.
//
// Both kernels pack the query heads of a KV head into the rows of a tile: row r of a
// tile is query r / gb of the tile, head r % gb of the group (gb heads, R = 128 / gb
// queries), which one 3-D TMA box per 64 channels brings in.  A tile's K and V then
// serve every head of the group, and a causal tile wastes 128 / gb queries at most.
#include "full.cuh"
#include "sm100.cuh"

namespace starkv {

using namespace sm100;

namespace {

constexpr int kTile = 128;            // rows of a query tile, keys of a key tile
constexpr uint32_t kSub = 16384;      // one 64-channel sub-tile of 128 rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMoveMax = 8.f;       // the running maximum moves when a score passes it by this (log2)

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) { return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Pairs of fp32 in one 64-bit register: one instruction works on both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2^x for x <= 126 on the FMA pipe, for a part of the exponentials (the special function unit
// takes 16 a cycle and SM, half as long again as the products of the same tile): x = n + f with
// n = rint(x), 2^f by the polynomial of degree 5 of least relative error on [-1/2, 1/2] (Remez
// exchange; 7.5e-8, in fp32 2.2e-7, as much as ex2.approx is off), 2^n from the bits of the sum
// that rounds x.  Below -126.5 the bits of 2^n are those of
// 0; NaN passes through.
__device__ __forceinline__ f32x2 ex2_fma(f32x2 x) {
  float2 y = unpair(x);
  x = pair(max_nan(y.x, -127.f), max_nan(y.y, -127.f));
  const float kRound = 12582912.f + 127.f;  // 1.5 2^23, and the bias of an exponent
  const f32x2 r = add2(x, pair(kRound, kRound));
  const f32x2 f = add2(x, mul2(add2(r, pair(-kRound, -kRound)), pair(-1.f, -1.f)));
  f32x2 p = fma2(f, pair(0.001327647245f, 0.001327647245f), pair(0.009675540961f, 0.009675540961f));
  p = fma2(p, f, pair(0.05550713092f, 0.05550713092f));
  p = fma2(p, f, pair(0.2402212024f, 0.2402212024f));
  p = fma2(p, f, pair(0.693146944f, 0.693146944f));
  p = fma2(p, f, pair(1.000000119f, 1.000000119f));
  y = unpair(r);
  return mul2(p, pair(__uint_as_float(__float_as_uint(y.x) << 23), __uint_as_float(__float_as_uint(y.y) << 23)));
}

// 2^x of a pair on the special function unit.
__device__ __forceinline__ f32x2 ex2_sfu(f32x2 x) {
  const float2 y = unpair(x);
  return pair(ex2(y.x), ex2(y.y));
}

__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Instruction descriptor of kind::f16 with bf16 operands, fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return make_idesc_f16(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);
}

// The products are issued by a whole warp that stays together, behind elect.sync: the
// compiler then keeps descriptors in uniform registers.  (128 x 128 x 128 of products takes 512
// cycles; issued by a branch on the lane it took 690, from a loop that was not unrolled 1240.)
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// D[tmem] (+)= A[tmem] * B[smem]; issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A descriptor's start address moved by `bytes` (it stays within the field: shared memory is smaller).
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

// 3-D tiled TMA load (no multicast).
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(smem_dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

struct SeqSpan {
  int q0, n;        // first query row, queries
  int k0, keys;     // first key row, keys
  bool ok;
};

struct PromptKArgs {
  int H, h_kv, group, gb, head_blocks, R, batch, max_q, max_k, qtiles, ktiles, window, mode;
  int64_t total_q, total_k;
  const __nv_bfloat16* v;
  int64_t v_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  float scale, scale_log2;
  __nv_bfloat16* out;
  const float* lse_in;
  float* lse;
  float* weights;
  unsigned int* status;
};

__device__ __forceinline__ SeqSpan span_of(const PromptKArgs& a, int b) {
  SeqSpan s;
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  s.ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k && q1 - q0 <= a.max_q &&
         k1 - k0 <= a.max_k && (b > 0 || (q0 == 0 && k0 == 0)) &&
         (b < a.batch - 1 || (q1 == a.total_q && k1 == a.total_k));
  s.q0 = q0;
  s.n = q1 - q0;
  s.k0 = k0;
  s.keys = k1 - k0;
  return s;
}

// ===========================================================================
// Attention
// ===========================================================================
// A CTA takes two query tiles (2 R queries) of one (sequence, KV head, head block) and
// walks the keys once for both.  Warps 0..3 and 4..7 each hold one tile's softmax (one
// row per thread), warp 8 copies, warp 9 issues the products, warps 10 and 11 look the V
// tiles of masked keys over.
//   S_t = Q_t K_j^T into TMEM; the softmax warps replace it by P_t in bf16 (the same
//   columns, half as many), which is the A operand of O_t += P_t V_j from TMEM.  In issue
//   order P_0 V_j, S_0 (j + 1), P_1 V_j, S_1 (j + 1): one tile's products run while the
//   other tile's softmax does.  The running maximum moves when a score passes it by more
//   than 2^8 only, and then the row's O is rescaled in place; S_t (j) complete implies
//   that P_t V_(j-1) is, so no further barrier guards that.
constexpr int kAttnThreads = 384;
#ifndef FMA_PAIR
#define FMA_PAIR(u) ((u) % 8 == 7)
#endif

template <int D>
struct AttnSmem {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kRing = 2 * kTileBytes;  // behind the two Q tiles: K_0, V_0, K_1, V_1, ...
  static constexpr uint32_t kBar = kRing + kStages * kTileBytes;
  static constexpr uint32_t kBytes = kBar + 256 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const PromptKArgs a) {
  using SM = AttnSmem<D>;
  constexpr int NSUB = D / 64;
  constexpr int ST = SM::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::kBar);
  uint64_t* qfull = bar;              // both Q tiles landed
  uint64_t* sfull = bar + 1;          // [2] S_t ready
  uint64_t* pfull = bar + 3;          // [2][2] P_t written: its first 64 keys, the others
  uint64_t* look = bar + 7;           // one phase per masked V tile: it is there,
  uint64_t* clean = bar + 8;          // and it has been looked over
  uint64_t* odone = bar + 9;          // every product done
  uint64_t* full = bar + 10;          // [ST]
  uint64_t* empty = full + ST;        // [ST]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(empty + ST);
  int* dirty = reinterpret_cast<int*>(tslot + 1);  // a masked V tile held a value that is not finite
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int units = a.h_kv * a.head_blocks * a.batch;
  const int unit = blockIdx.x % units;
  const int qt = a.qtiles - 1 - (int)(blockIdx.x / units);  // the tiles with the most keys first
  const int hb = unit % a.head_blocks, kv = unit / a.head_blocks % a.h_kv, b = unit / a.head_blocks / a.h_kv;
  pdl_wait();
  pdl_launch_dependents();
  const SeqSpan q = span_of(a, b);
  if (!q.ok) {
    if (tid == 0) set_status(a.status, STARKV_DEV_BAD_QUERY_SPAN);
    return;
  }
  const int qbase = qt * 2 * a.R;
  if (qbase >= q.n) return;
  const int off = q.keys - q.n;  // query i sees keys 0 .. off + i
  const int heads = min(a.gb, a.group - hb * a.gb);
  const int h0 = kv * a.group + hb * a.gb;
  int ntile[2];  // key tiles of the two query tiles
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int rows = min(a.R, q.n - qbase - t * a.R);
    const int keys = rows > 0 ? off + qbase + t * a.R + rows : 0;  // keys that its last query sees
    ntile[t] = keys > 0 ? (keys + kTile - 1) / kTile : 0;
  }
  const int nt = max(ntile[0], ntile[1]);
  // the first key tile that some row does not see whole
  const int first_masked = max(0, off + qbase + 1) / kTile;

  if (warp == 9) tmem_alloc(tslot, 512);
  if (tid == 0) {
    mbar_init(qfull, 1);
    mbar_init(&sfull[0], 1);
    mbar_init(&sfull[1], 1);
    for (int s = 0; s < 4; ++s) mbar_init(&pfull[s], 4);
    mbar_init(look, 1);
    mbar_init(clean, 2);
    mbar_init(odone, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    *dirty = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  bool ok = true;

  if (warp == 8) {
    // ---------------- copies ----------------
    if (lane == 0 && nt > 0) {
      mbar_arrive_expect_tx(qfull, 2u * NSUB * a.R * a.gb * 128);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < NSUB; ++i)
          tma_load_3d(sm + t * SM::kTileBytes + i * kSub, &q_map, i * 64, h0, q.q0 + qbase + t * a.R, qfull);
      int issued = 0;
      for (; issued < 2 * nt; ++issued) {
        const int s = issued % ST, j = issued >> 1;
        if (!mbar_wait_short(&empty[s], ((issued / ST) & 1) ^ 1)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[s], SM::kTileBytes);
#pragma unroll
        for (int i = 0; i < NSUB; ++i)
          tma_load_2d(sm + SM::kRing + s * SM::kTileBytes + i * kSub, issued & 1 ? &v_map : &k_map, kv * D + i * 64,
                      q.k0 + j * kTile, &full[s]);
      }
      if (!ok) {  // wait (with a limit) for the copies in flight
        mbar_wait(qfull, 0, 100000000ull);
        for (int i = max(0, issued - ST); i < issued; ++i) mbar_wait(&full[i % ST], (i / ST) & 1, 100000000ull);
      }
    }
  } else if (warp == 9) {
    // ---------------- products ----------------
    if (nt > 0) {
      constexpr uint32_t idesc_s = idesc_bf16(128, kTile, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(128, D, false, true);
      const bool lead = elected();
      const uint64_t qd = make_sdesc(smem_u32(sm), 16, 1024, 2);
      const uint64_t kd = make_sdesc(smem_u32(sm + SM::kRing), 16, 1024, 2);
      const uint64_t vd = make_sdesc(smem_u32(sm + SM::kRing), kSub, 1024, 2);
      auto issue_s = [&](int t, int stage) {
        const uint64_t q0 = desc_at(qd, t * SM::kTileBytes), k0 = desc_at(kd, stage * SM::kTileBytes);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (ks >> 2) * kSub + (ks & 3) * 32;
          mma_f16(tmem + t * kTile, desc_at(q0, o), desc_at(k0, o), idesc_s, ks > 0);
        }
        mma_commit(&sfull[t]);
      };
      auto all = [&](bool got) { return __all_sync(0xffffffffu, got) != 0; };
      // the ring's positions: K_j at kst, V_j at vst, each with its phase
      int kst = 0, vst = 1;
      uint32_t kph = 0, vph = 0;
      auto on = [&](int& st, uint32_t& ph) {
        st += 2;
        if (st >= ST) {
          st -= ST;
          ph ^= 1;
        }
      };
      ok = all(mbar_wait_short(qfull, 0) && mbar_wait_short(&full[0], 0));
      if (ok) {
        tc_fence_after();
        if (lead) {
          if (ntile[0] > 0) issue_s(0, 0);
          if (ntile[1] > 0) issue_s(1, 0);
          mma_commit(&empty[0]);
        }
        __syncwarp();
      }
      uint32_t looked = 0;
      for (int j = 0; ok && j < nt; ++j) {
        on(kst, kph);
        bool got = mbar_wait_short(&full[vst], vph);
        if (got && j >= first_masked) {
          if (lane == 0) mbar_arrive(look);
          got = mbar_wait_short(clean, looked);
          looked ^= 1;
        }
        if (got && j + 1 < nt) got = mbar_wait_short(&full[kst], kph);
        ok = all(got);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || j >= ntile[t]) continue;
          const uint64_t v0 = desc_at(vd, vst * SM::kTileBytes);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!all(ok && mbar_wait_short(&pfull[t * 2 + h], j & 1))) {
              ok = false;
              continue;
            }
            tc_fence_after();
            if (lead) {
#pragma unroll
              for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
                mma_f16_ts(tmem + 256 + t * kTile, tmem + t * kTile + ks * 8, desc_at(v0, ks * 2048), idesc_o,
                           j > 0 || ks > 0);
            }
            __syncwarp();
          }
          if (!ok) continue;
          if (lead) {
            if (t == 1 || j >= ntile[1]) mma_commit(&empty[vst]);
            if (j + 1 < ntile[t]) issue_s(t, kst);
          }
          __syncwarp();
        }
        if (ok && j + 1 < nt && lead) mma_commit(&empty[kst]);
        on(vst, vph);
      }
      if (lead) mma_commit(odone);  // completes once every product issued above has
      __syncwarp();
      if (!ok) mbar_wait(odone, 0, 100000000ull);
    }
  } else if (warp >= 10) {
    // ---------------- V tiles with masked keys ----------------
    // A key that some row does not see has p = 0 there, but 0 * inf and 0 * NaN are not 0, and the
    // rows behind the sequence are another's.  So values that are not finite are cleared (rows
    // behind the sequence, whatever they hold) and, where a row does see them, added at the end.
    for (int j = first_masked; ok && j < nt; ++j) {
      const int i = 2 * j + 1;
      const bool got = mbar_wait_short(look, (j - first_masked) & 1) && mbar_wait_short(&full[i % ST], (i / ST) & 1);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      uint8_t* tile = sm + SM::kRing + (i % ST) * SM::kTileBytes;
      bool mine = false;
      for (int e = (warp - 10) * 32 + lane; e < kTile * D / 8; e += 64) {
        uint4* p = reinterpret_cast<uint4*>(tile) + e;
        uint4 x = *p;
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
        bool hit = false;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if ((w[u] & 0x7f80u) == 0x7f80u) {
            w[u] &= 0xffff0000u;
            hit = true;
          }
          if ((w[u] & 0x7f800000u) == 0x7f800000u) {
            w[u] &= 0x0000ffffu;
            hit = true;
          }
        }
        if (hit) {
          *p = x;
          mine = true;
        }
      }
      if (mine) *reinterpret_cast<volatile int*>(dirty) = 1;
      __threadfence_block();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(clean);
    }
  } else {
    // ---------------- softmax: one row per thread ----------------
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int qi = qbase + t * a.R + r / a.gb;  // query of the row
    const int hh = r % a.gb;
    const bool live = r < a.R * a.gb && qi < q.n && hh < heads;
    const int seen = live ? off + qi + 1 : 1 << 30;  // keys the row sees (may be <= 0); a row of nothing masks nothing
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = trow + t * kTile, to = trow + 256 + t * kTile;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < ntile[t]; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait_short(&sfull[t], j & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      float sv[kTile];
      {
        uint32_t(&raw)[kTile] = *reinterpret_cast<uint32_t(*)[kTile]>(sv);
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c) tmem_ld32(ts + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&raw[c * 32]));
        tmem_ld_wait();
      }
      const int lim = seen - j * kTile;
      if (__any_sync(0xffffffffu, lim < kTile)) {
#pragma unroll
        for (int c = 0; c < kTile; ++c) sv[c] = c < lim ? sv[c] : -INFINITY;
      }
      float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
      for (int c = 4; c < kTile - 4; c += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], sv[c + u], sv[c + 4 + u]);
      const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], sv[kTile - 4], sv[kTile - 3]),
                             fmaxf(sv[kTile - 2], sv[kTile - 1]));
      const bool move = live && (top - m) * a.scale_log2 > kMoveMax;  // m = -inf: true but for a row without scores
      if (__any_sync(0xffffffffu, move)) {
        if (j > 0) {
          const float f = move ? ex2((m - top) * a.scale_log2) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(to + c * 16, o);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
            tmem_st16(to + c * 16, o);
          }
          l *= f;
        }
        if (move) m = top;
      }
      const float base = m == -INFINITY ? 0.f : -m * a.scale_log2;
      const f32x2 scale2 = pair(a.scale_log2, a.scale_log2), base2 = pair(base, base);
      f32x2 sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
      // four quarters; the first half of P goes on its way while the third quarter is computed
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const f32x2 x = fma2(pair(sv[c * 32 + 2 * u], sv[c * 32 + 2 * u + 1]), scale2, base2);
          const f32x2 p = FMA_PAIR(u) ? ex2_fma(x) : ex2_sfu(x);
          sum[u & 1] = add2(sum[u & 1], p);
          const float2 y = unpair(p);
          w[u] = pack_bf2(y.x, y.y);
        }
        if (c == 2) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[t * 2]);
        }
        tmem_st16(ts + c * 16, w);
      }
      const float2 s0 = unpair(sum[0]), s1 = unpair(sum[1]);
      l += (s0.x + s0.y) + (s1.x + s1.y);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[t * 2 + 1]);
    }
    // ---- O / l, and lse
    if (ntile[t] > 0 && ok && !__all_sync(0xffffffffu, mbar_wait_short(odone, 0))) ok = false;
    if (ok) {
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t row = (int64_t)(q.q0 + qi) * a.H + h0 + hh;
      const bool fix = ntile[t] > 0 && *reinterpret_cast<volatile int*>(dirty) != 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (ntile[t] > 0) {
          tmem_ld32(to + c * 32, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) o[u] = 0u;
        }
        if (!live) continue;
        if (fix)
          for (int j = first_masked * kTile; j < seen; ++j) {
            const __nv_bfloat16* vr = a.v + (int64_t)(q.k0 + j) * a.v_stride + kv * D + c * 32;
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const float x = __bfloat162float(vr[u]);
              if (!isfinite(x)) o[u] = __float_as_uint(__uint_as_float(o[u]) + x);
            }
          }
        uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + c * 32);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = pack_bf2(__uint_as_float(o[8 * u + 2 * x]) * inv, __uint_as_float(o[8 * u + 2 * x + 1]) * inv);
          dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : fmaf(m, a.scale, logf(l));
    }
  }
  if (!ok && lane == 0) set_status(a.status, kDevWaitTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ===========================================================================
// Attention weights
// ===========================================================================
// An item is 128 keys of one (sequence, KV head); its steps are the tiles of queries that
// count and see any of them.  A step's product S^T = K Q^T (TMEM, four buffers) has one
// key per lane, so that the sum over queries and heads stays in a register of the thread
// that holds the key.  Warps 0..7 take the even steps, 8..15 the odd ones, half of the
// columns each (four warps a scheduler keep the exponentials going while others wait for
// their columns); warp 16 copies, warp 17 issues the products and notes for each what its sums go by, warps 18
// and 19 lay out each column's log-sum-exp and the last key it sees.  One CTA an SM walks over many items, three ways:
//   resident  the counting queries of a (sequence, KV head) fit the ring (a window): a CTA
//             takes an equal stretch of the items in (sequence, KV head, key) order and
//             loads them once per (sequence, KV head); only K tiles stream.
//   streamed  items in the order of their first key (those of the first keys have the most
//             steps), dealt forth and back, so that the CTAs' sums of steps come out alike.
//   split     where there are few items, a cluster shares one item's steps out and adds the
//             sums through distributed shared memory, in rank order.
constexpr int kWeightThreads = 640;
constexpr int kColNone = -(1 << 30);  // a column that sees no key
enum { kResident = 0, kStreamed = 1 };  // > 1: split over so many CTAs

template <int D>
struct WeightSmem {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 3 : 6;   // Q tiles
  static constexpr int kKeys = D == 128 ? 3 : 4;     // K tiles
  static constexpr uint32_t kRing = kKeys * kTileBytes;
  static constexpr uint32_t kCols = kRing + kStages * kTileBytes;  // [stage][128] -lse in log2 units, [stage][128] last key
  static constexpr uint32_t kSums = kCols + kStages * kTile * 8;   // [2][3][128] sums of warps 4 .. 15
  static constexpr uint32_t kNotes = kSums + 2 * 3 * kTile * 4;    // [4] what a product's sums go by
  static constexpr uint32_t kBar = kNotes + 4 * 32;
  static constexpr uint32_t kBytes = kBar + 512 + 1024;
};

// One product's note, beside its TMEM buffer.
struct __align__(16) Note {
  int flags;     // kWhole: no column is masked for any key; kLast: the item's last step; kLeave: its Q tile's last use; kStop
  int stage;     // the Q tile's
  int live;      // columns that hold queries
  int key0, keys;  // the item's first key, and the keys of its sequence
  int unused;
  int64_t row;   // the sequence's first row, times h_kv, plus the KV head
};
static_assert(sizeof(Note) == 32, "a note is two 16-byte words");
enum { kWhole = 1, kLast = 2, kLeave = 4, kStop = 8 };

// The items of a CTA, in order; every role walks its own copy.
struct Items {
  const PromptKArgs& a;
  int64_t at, end;   // resident: positions of the stretch; streamed: the turn
  int64_t before;    // resident: items of the sequences before b
  int b, kv, kt, tiles;
  SeqSpan q;
  int off, first, per, steps;
  bool fresh;        // another (sequence, KV head) than the item before
  bool started;

  __device__ Items(const PromptKArgs& args, int64_t pos, int64_t stop, int seq, int64_t items_before)
      : a(args), at(pos), end(stop), before(items_before), b(seq), kv(-1), kt(0), tiles(0), started(false) {}

  __device__ void steps_of() {
    off = q.keys - q.n;
    // queries first .. n - 1 count; the tile's first key is seen from query kt * 128 - off on
    // (resident: the sequence's Q tiles serve all its items)
    first = max(max(0, q.n - a.window), (a.mode == kResident ? 0 : kt * kTile) - off);
    per = first < q.n ? (q.n - first + a.R - 1) / a.R : 0;
    steps = per * a.head_blocks;
  }

  __device__ bool next() {
    if (a.mode == kResident) {
      if (at >= end) return false;
      fresh = true;
      if (!started) {
        started = true;
        q = span_of(a, b);
        tiles = (q.keys + kTile - 1) / kTile;
        kv = (int)((at - before) / tiles);
        kt = (int)((at - before) - (int64_t)kv * tiles);
      } else if (++kt < tiles) {
        fresh = false;
      } else {
        kt = 0;
        if (++kv == a.h_kv) {
          kv = 0;
          do {  // (a position behind this one is some sequence's)
            q = span_of(a, ++b);
            tiles = q.ok ? (q.keys + kTile - 1) / kTile : 0;
          } while (tiles == 0);
        }
      }
      ++at;
      if (fresh) steps_of();
      return true;
    }
    const uint32_t each = (uint32_t)a.h_kv * a.batch, items = each * a.ktiles;  // (below 2^32: checked)
    fresh = true;
    while (at < end) {
      // turn i takes item i C + c, or i C + C - 1 - c where i is odd
      const uint32_t ctas = a.mode > 1 ? items : gridDim.x, c = a.mode > 1 ? blockIdx.x / a.mode : blockIdx.x;
      const int64_t at_item = at * ctas + (at & 1 ? ctas - 1 - c : c);
      ++at;
      if (at_item >= items) continue;
      const uint32_t w = (uint32_t)at_item;
      kt = (int)(w / each);
      kv = (int)(w % each % a.h_kv);
      b = (int)(w % each / a.h_kv);
      q = span_of(a, b);
      if (!q.ok || kt * kTile >= q.keys) continue;
      steps_of();
      return true;
    }
    return false;
  }
};

template <int D>
__global__ void __launch_bounds__(kWeightThreads, 1)
    prompt_weights_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                          const PromptKArgs a) {
  using SM = WeightSmem<D>;
  constexpr int NSUB = D / 64;
  constexpr int ST = SM::kStages, KS = SM::kKeys;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t part[kWeightThreads / 32];
  __shared__ int64_t begin[2];
  uint8_t* sm = align1024(smem_raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::kBar);
  uint64_t* kfull = bar;           // [KS]
  uint64_t* kempty = kfull + KS;   // [KS]
  uint64_t* full = kempty + KS;    // [ST] Q tile landed
  uint64_t* empty = full + ST;     // [ST] Q tile read by its products, its columns by 8 warps
  uint64_t* sfull = empty + ST;    // [4] a product, its columns (2 warps) and its note are there,
  uint64_t* sempty = sfull + 4;    // [4] and have been read
  uint64_t* sums = sempty + 4;     // [2][4] three warps' sums are there
  uint64_t* taken = sums + 8;      // [2][4] and have been added
  uint64_t* done = taken + 8;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  float* lse2 = reinterpret_cast<float*>(sm + SM::kCols);
  int* last = reinterpret_cast<int*>(sm + SM::kCols + ST * kTile * 4);
  float* other = reinterpret_cast<float*>(sm + SM::kSums);
  Note* notes = reinterpret_cast<Note*>(sm + SM::kNotes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = a.mode > 1 ? a.mode : 1;
  const int rank = a.mode > 1 ? blockIdx.x % a.mode : 0;  // (clusters are consecutive blocks)

  // rows behind the box of a tile stay zero: they are columns of the products
  for (int s = 0; s < ST; ++s)
    for (int e = tid; e < (kTile - a.R * a.gb) * D / 8; e += kWeightThreads) {
      const int r = a.R * a.gb + e / (D / 8), c = e % (D / 8);
      *reinterpret_cast<uint4*>(sm + SM::kRing + s * SM::kTileBytes + (c >> 3) * kSub + r * 128 + (c & 7) * 16) =
          make_uint4(0, 0, 0, 0);
    }
  fence_async_smem();
  if (warp == 17) tmem_alloc(tslot, 512);
  if (tid == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 9);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sfull[s], 3);
      mbar_init(&sempty[s], 8);
    }
    for (int s = 0; s < 8; ++s) {
      mbar_init(&sums[s], 3);
      mbar_init(&taken[s], 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  // ---- the CTA's items
  int64_t pos = 0, end = 0, before = 0;
  int seq = 0;
  if (a.mode == kResident) {
    // as many items of each CTA: cut the sequences' items, laid end to end
    int64_t mine = 0;
    for (int i = tid; i < a.batch; i += kWeightThreads) {
      const SeqSpan q = span_of(a, i);
      if (!q.ok && blockIdx.x == 0) set_status(a.status, STARKV_DEV_BAD_QUERY_SPAN);
      if (q.ok) mine += (q.keys + kTile - 1) / kTile;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWeightThreads / 32; ++w) total += part[w];
    total *= a.h_kv;
    pos = total * blockIdx.x / gridDim.x;
    end = total * (blockIdx.x + 1) / gridDim.x;
    // the sequence that holds pos, warp 0 in steps of 32 sequences
    if (warp == 0) {
      int64_t carry = 0;
      for (int i0 = 0; i0 < a.batch; i0 += 32) {
        int tiles = 0;
        if (i0 + lane < a.batch) {
          const SeqSpan q = span_of(a, i0 + lane);
          if (q.ok) tiles = (q.keys + kTile - 1) / kTile;
        }
        int64_t inc = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const int64_t s0 = (carry + inc - tiles) * a.h_kv;
        if (s0 <= pos && pos < s0 + (int64_t)tiles * a.h_kv) {
          begin[0] = i0 + lane;
          begin[1] = s0;
        }
        carry += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  } else {
    const int64_t items = (int64_t)a.ktiles * a.h_kv * a.batch;
    end = a.mode > 1 ? 1 : (items + gridDim.x - 1) / gridDim.x;
    if (blockIdx.x == 0)
      for (int i = tid; i < a.batch; i += kWeightThreads)
        if (!span_of(a, i).ok) set_status(a.status, STARKV_DEV_BAD_QUERY_SPAN);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (a.mode == kResident && pos < end) {
    seq = (int)begin[0];
    before = begin[1];
  }
  const uint32_t tmem = *tslot;
  const bool resident = a.mode == kResident;
  bool ok = true;
  Items it(a, pos, end, seq, before);
  // Stage and phase of step v, the u-th of this CTA.  Resident: the stage is the step's number, and
  // `flips` holds the stages' phases (a stage turns when a (sequence, KV head) that used it is done).
  uint32_t flips = 0;
  auto stage_of = [&](int v, int u) { return resident ? v : u % ST; };
  auto phase_of = [&](int v, int u) { return resident ? (flips >> v) & 1u : (uint32_t)(u / ST) & 1u; };
  float acc = 0.f;

  if (warp == 16) {
    // ---------------- copies ----------------
    if (lane == 0) {
      int ki = 0, u = 0;  // K tiles and Q tiles so far
      while (ok && it.next()) {
        if (it.steps == 0) continue;
        const int ks = ki % KS;
        if (!mbar_wait_short(&kempty[ks], ((ki / KS) & 1) ^ 1)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&kfull[ks], SM::kTileBytes);
#pragma unroll
        for (int i = 0; i < NSUB; ++i)
          tma_load_2d(sm + ks * SM::kTileBytes + i * kSub, &k_map, it.kv * D + i * 64, it.q.k0 + it.kt * kTile,
                      &kfull[ks]);
        ++ki;
        if (resident && !it.fresh) continue;
        for (int v = rank; v < it.steps; v += split, ++u) {
          const int s = stage_of(v, u);
          const uint32_t ph = phase_of(v, u);
          if (!mbar_wait_short(&empty[s], ph ^ 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], NSUB * a.R * a.gb * 128);
          const int hb = v / it.per, i0 = it.first + (v % it.per) * a.R;
#pragma unroll
          for (int i = 0; i < NSUB; ++i)
            tma_load_3d(sm + SM::kRing + s * SM::kTileBytes + i * kSub, &q_map, i * 64, it.kv * a.group + hb * a.gb,
                        it.q.q0 + i0, &full[s]);
        }
        flips ^= (1u << min(it.steps, ST)) - 1;
      }
      if (!ok) {  // wait (with a limit) for the copies in flight
        for (int i = max(0, ki - KS); i < ki; ++i) mbar_wait(&kfull[i % KS], (i / KS) & 1, 100000000ull);
        if (resident)
          for (int s = 0; s < ST; ++s) mbar_wait(&full[s], ((flips >> s) & 1) ^ 1, 100000000ull);
        else
          for (int i = max(0, u - ST); i < u; ++i) mbar_wait(&full[i % ST], (i / ST) & 1, 100000000ull);
      }
    }
  } else if (warp == 17) {
    // ---------------- products ----------------
    constexpr uint32_t idesc = idesc_bf16(128, kTile, false, false);
    const bool lead = elected();
    const uint64_t kd = make_sdesc(smem_u32(sm), 16, 1024, 2), qd = make_sdesc(smem_u32(sm + SM::kRing), 16, 1024, 2);
    int u = 0, ks = 0, st = 0;  // steps so far, the K ring's next tile, the Q ring's (streamed)
    uint32_t kph = 0, sph = 0;
    bool more = it.next();
    while (ok && more) {
      const int steps = it.steps;
      more = it.next();
      if (steps == 0) continue;
      const bool free_q = !resident || !more || it.fresh;  // resident: the Q tiles' last use
      ok = __all_sync(0xffffffffu, mbar_wait_short(&kfull[ks], kph));
      const uint64_t k0 = desc_at(kd, ks * SM::kTileBytes);
      int v = rank;
      for (; ok && v < steps; v += split, ++u) {
        const int s = resident ? v : st, w = u & 3;
        const uint32_t ph = resident ? (flips >> v) & 1u : sph;
        ok = __all_sync(0xffffffffu, mbar_wait_short(&full[s], ph) && mbar_wait_short(&sempty[w], ((u >> 2) & 1) ^ 1));
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          const uint64_t q0 = desc_at(qd, s * SM::kTileBytes);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t o = (e >> 2) * kSub + (e & 3) * 32;
            mma_f16(tmem + w * kTile, desc_at(k0, o), desc_at(q0, o), idesc, e > 0);
          }
          mma_commit(&sfull[w]);
          if (free_q) mma_commit(&empty[s]);
        }
        __syncwarp();
        if (++st == ST) {
          st = 0;
          sph ^= 1;
        }
      }
      if (ok && v == rank + split) {  // one step: a note without a product ends the item for the other warps
        const int w = u & 3;
        ok = __all_sync(0xffffffffu, mbar_wait_short(&sempty[w], ((u >> 2) & 1) ^ 1));
        if (lane == 0) mbar_arrive(&sfull[w]);
        ++u;
      }
      if (lead) mma_commit(&kempty[ks]);
      __syncwarp();
      if (++ks == KS) {
        ks = 0;
        kph ^= 1;
      }
      if (!resident || free_q) flips ^= (1u << min(steps, ST)) - 1;
    }
    for (int e = 0; ok && e < 2; ++e, ++u) {  // nothing more: two notes without products
      const int w = u & 3;
      ok = __all_sync(0xffffffffu, mbar_wait_short(&sempty[w], ((u >> 2) & 1) ^ 1));
      if (lane == 0) mbar_arrive(&sfull[w]);
    }
    if (lead) mma_commit(done);
    __syncwarp();
    mbar_wait(done, 0, ok ? 2000000000ull : 100000000ull);
  } else if (warp >= 18) {
    // ---------------- columns and notes (and the zeros of keys that no counting query sees) ----------------
    int u = 0, st = 0;
    uint32_t sph = 0;
    int col_r[2], col_h[2];  // the lane's columns: query within the tile, head within the block
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = (warp - 18) * 64 + e * 32 + lane;
      col_r[e] = c / a.gb;
      col_h[e] = c % a.gb;
    }
    auto note = [&](const Note& n) {  // for the u-th product, whose buffer must be free
      const int w = u & 3;
      if (!__all_sync(0xffffffffu, mbar_wait_short(&sempty[w], ((u >> 2) & 1) ^ 1))) return false;
      if (lane == 0) {
        if (warp == 18) notes[w] = n;
        mbar_arrive(&sfull[w]);
      }
      ++u;
      return true;
    };
    bool more = it.next();
    while (ok && more) {
      const int steps = it.steps, per = it.per, first = it.first, off = it.off, n = it.q.n, keys = it.q.keys, kv = it.kv;
      const int q0 = it.q.q0, key0 = it.kt * kTile;
      const int64_t row = (int64_t)it.q.k0 * a.h_kv + kv;
      const bool fresh = it.fresh;
      more = it.next();
      if (steps == 0) {
        for (int r = key0 + tid - 18 * 32; r < min(key0 + kTile, keys); r += 64) a.weights[row + (int64_t)r * a.h_kv] = 0.f;
        continue;
      }
      const bool lay = !resident || fresh, leave = !resident || !more || it.fresh;
      // the next step's log-sum-exps are asked for before this step's stage is free
      float x[2], next_x[2];
      int k[2], next_k[2];
      int hb = rank / per, i0 = first + rank % per * a.R;  // the step's head block and first query
      auto fetch = [&](int v, int hb, int i0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = i0 + col_r[e], h = hb * a.gb + col_h[e];
          const bool live = v < steps && col_r[e] < a.R && i < n && h < a.group;
          next_x[e] = 0.f;
          next_k[e] = kColNone;
          if (live) {
            next_x[e] = a.lse_in[(int64_t)(q0 + i) * a.H + kv * a.group + h];
            next_k[e] = off + i;
          }
        }
      };
      if (lay) fetch(rank, hb, i0);
      for (int v = rank; v < steps; v += split) {
        const int s = resident ? v : st;
        const uint32_t ph = resident ? (flips >> v) & 1u : sph;
        if (++st == ST) {
          st = 0;
          sph ^= 1;
        }
        // a column is masked for some key of the tile in the first tiles only
        const bool whole = off + i0 >= key0 + kTile - 1 && (hb + 1) * a.gb <= a.group;
        const Note told{(whole ? kWhole : 0) | (v + 2 * split >= steps ? kLast : 0) | (leave ? kLeave : 0), s,
                        min(a.R, n - i0) * a.gb, key0, keys, 0, row};
        i0 += split * a.R;
        while (i0 >= first + per * a.R) {
          i0 -= per * a.R;
          ++hb;
        }
        if (lay) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[e] = next_x[e];
            k[e] = next_k[e];
          }
          fetch(v + split, hb, i0);
          if (!__all_sync(0xffffffffu, mbar_wait_short(&empty[s], ph ^ 1))) {
            ok = false;
            break;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = (warp - 18) * 64 + e * 32 + lane;
            lse2[s * kTile + c] = x[e] * -kLog2e;
            last[s * kTile + c] = k[e];
          }
          __syncwarp();
        }
        if (!note(told)) {
          ok = false;
          break;
        }
      }
      if (ok && rank < steps && rank + split >= steps) ok = note(Note{kLast, 0, 0, key0, keys, 0, row});
      if (lay) flips ^= (1u << min(steps, ST)) - 1;
    }
    for (int e = 0; ok && e < 2; ++e) ok = note(Note{kStop, 0, 0, 0, 0, 0, 0});
  } else {
    // ---------------- sums: one key per thread ----------------
    const int g = warp >> 2, half = g & 1, row = (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 64;
    int items = 0;
    for (int u = g >> 1;; u += 2) {
      const int w = u & 3;
      if (!__all_sync(0xffffffffu, mbar_wait_short(&sfull[w], (u >> 2) & 1))) {
        ok = false;
        break;
      }
      const Note note = notes[w];
      if (note.flags & kStop) break;
      tc_fence_after();
      const int s = note.stage, key = note.key0 + row;
      const int live = note.live - half * 64;  // of the warp's columns
      const float* x = lse2 + s * kTile + half * 64;
      const int* k = last + s * kTile + half * 64;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      if ((note.flags & kWhole) && live >= 64) {
        uint32_t y[64];
        tmem_ld32(trow + w * kTile, *reinterpret_cast<uint32_t(*)[32]>(&y[0]));
        tmem_ld32(trow + w * kTile + 32, *reinterpret_cast<uint32_t(*)[32]>(&y[32]));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[w]);
        f32x2 two[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
        const f32x2 scale = pair(a.scale_log2, a.scale_log2);
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float4 z = *reinterpret_cast<const float4*>(x + e);
          const f32x2 t0 = fma2(pair(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), scale, pair(z.x, z.y));
          const f32x2 t1 = fma2(pair(__uint_as_float(y[e + 2]), __uint_as_float(y[e + 3])), scale, pair(z.z, z.w));
          two[0] = add2(two[0], ex2_sfu(t0));
          two[1] = add2(two[1], ex2_sfu(t1));
        }
        const float2 a0 = unpair(two[0]), a1 = unpair(two[1]);
        sum[0] = a0.x, sum[1] = a0.y, sum[2] = a1.x, sum[3] = a1.y;
      } else {
#pragma unroll 1
        for (int c = 0; c < 64 && c < live; c += 32) {
          uint32_t y[32];
          tmem_ld32(trow + w * kTile + c, y);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p = ex2(fmaf(__uint_as_float(y[e]), a.scale_log2, x[c + e]));
            sum[e & 3] += key <= k[c + e] ? p : 0.f;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[w]);
      }
      acc += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (note.flags & kLeave) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
      }
      if (!(note.flags & kLast)) continue;
      // the four groups' sums: warps 4..15 hand theirs over, warps 0..3 add and store
      const int buf = items & 1, set = buf * 4 + (warp & 3);
      const uint32_t ph = (items >> 1) & 1;
      ++items;
      if (g > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait_short(&taken[set], ph ^ 1))) {
          ok = false;
          break;
        }
        other[(buf * 3 + g - 1) * kTile + row] = acc;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sums[set]);
        acc = 0.f;
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait_short(&sums[set], ph))) {
          ok = false;
          break;
        }
        const float* o = other + buf * 3 * kTile + row;
        acc = (acc + o[0]) + (o[kTile] + o[2 * kTile]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken[set]);
        if (split == 1) {
          if (key < note.keys) a.weights[note.row + (int64_t)key * a.h_kv] = acc;
          acc = 0.f;
        }
      }
    }
  }
  if (!ok && lane == 0) set_status(a.status, kDevWaitTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (split > 1) {
    // one item: the ranks' sums, in rank order (the columns' memory is free by now)
    if (warp < 4) lse2[tid] = acc;
    cluster_sync();
    Items one(a, 0, 1, 0, 0);
    if (rank == 0 && warp < 4 && one.next() && one.steps > 0 && one.kt * kTile + tid < one.q.keys) {
      float sum = 0.f;
      for (int r = 0; r < split; ++r) sum += dsmem_ld_f32(dsmem_addr(&lse2[tid], (uint32_t)r));
      a.weights[((int64_t)one.q.k0 + one.kt * kTile + tid) * a.h_kv + one.kv] = sum;
    }
    cluster_sync();
  }
}

PromptKArgs args_of(const Ctx& c, const PromptArgs& p) {
  PromptKArgs a = {};
  const starkv_config& f = c.cfg;
  a.H = f.num_q_heads;
  a.h_kv = f.num_kv_heads;
  a.group = c.group;
  a.head_blocks = (c.group + kTile - 1) / kTile;
  a.gb = (c.group + a.head_blocks - 1) / a.head_blocks;
  a.R = kTile / a.gb;
  a.batch = p.batch;
  a.total_q = p.total_q;
  a.total_k = p.total_k;
  a.v = p.v;
  a.v_stride = p.v_stride;
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.scale = (float)(1.0 / sqrt((double)f.head_dim));
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)f.head_dim));
  a.status = c.status;
  a.max_q = a.max_k = 0x7fffffff;
  return a;
}

// Maps of q (64 channels x gb heads x R queries) and of k or v (64 channels x 128 rows).
bool map_q(const Ctx& c, const PromptArgs& p, const PromptKArgs& a, CUtensorMap* m) {
  return encode_map_heads(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<__nv_bfloat16*>(p.q), c.cfg.head_dim,
                          c.cfg.num_q_heads, p.total_q, p.q_stride * 2, 64, a.gb, a.R, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_kv(const Ctx& c, const void* base, int64_t stride, int64_t rows, CUtensorMap* m) {
  return encode_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<void*>(base),
                       (uint64_t)c.cfg.num_kv_heads * c.cfg.head_dim, (uint64_t)rows, (uint64_t)stride * 2, 64, kTile,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D>
cudaError_t launch_attn_d(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const PromptKArgs& a,
                          cudaStream_t s) {
  const size_t smem = AttnSmem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(prompt_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const unsigned blocks = (unsigned)a.qtiles * a.h_kv * a.head_blocks * a.batch;
  return launch_chained(prompt_attn_kernel<D>, dim3(blocks), dim3(kAttnThreads), smem, s, 1u, qm, km, vm, a);
}

template <int D>
cudaError_t launch_weights_d(const CUtensorMap& qm, const CUtensorMap& km, PromptKArgs a, int sms, cudaStream_t s) {
  const size_t smem = WeightSmem<D>::kBytes;
  cudaError_t e =
      cudaFuncSetAttribute(prompt_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)a.ktiles * a.h_kv * a.batch;
  // steps of an item whose keys every counting query sees
  const int64_t most = ((int64_t)(a.window < a.max_k ? a.window : a.max_k) + a.R - 1) / a.R * a.head_blocks;
  a.mode = most <= WeightSmem<D>::kStages ? kResident : kStreamed;
  unsigned grid = (unsigned)(items < sms ? items : sms), cluster = 1;
  if (a.mode == kStreamed && items * 2 <= sms) {
    while (cluster < 8 && items * cluster * 2 <= sms && cluster * 2 <= most) cluster *= 2;
    if (cluster > 1) {
      a.mode = (int)cluster;
      grid = (unsigned)items * cluster;
    }
  }
  return launch_chained(prompt_weights_kernel<D>, dim3(grid), dim3(kWeightThreads), smem, s, cluster, qm, km, a);
}

}  // namespace

int64_t weights_items(const Ctx& c, int batch, int max_k_len) {
  return ((int64_t)max_k_len + kTile - 1) / kTile * c.cfg.num_kv_heads * batch;
}

int64_t prompt_blocks(const Ctx& c, int batch, int max_q_len) {
  PromptArgs p = {};
  const PromptKArgs a = args_of(c, p);
  return ((int64_t)max_q_len + 2 * a.R - 1) / (2 * a.R) * a.h_kv * a.head_blocks * batch;
}

cudaError_t launch_prompt_attn(const Ctx& c, const PromptArgs& p, int max_q_len, __nv_bfloat16* out, float* lse,
                               cudaStream_t s) {
  PromptKArgs a = args_of(c, p);
  a.max_q = max_q_len;
  a.qtiles = (max_q_len + 2 * a.R - 1) / (2 * a.R);
  a.out = out;
  a.lse = lse;
  CUtensorMap qm, km, vm;
  if (!map_q(c, p, a, &qm)) return cudaErrorInvalidValue;
  km = vm = qm;  // no keys at all: nothing is copied
  if (p.total_k > 0 && (!map_kv(c, p.k, p.k_stride, p.total_k, &km) || !map_kv(c, p.v, p.v_stride, p.total_k, &vm)))
    return cudaErrorInvalidValue;
  return c.cfg.head_dim == 64 ? launch_attn_d<64>(qm, km, vm, a, s) : launch_attn_d<128>(qm, km, vm, a, s);
}

cudaError_t launch_prompt_weights(const Ctx& c, const PromptArgs& p, const float* lse, int max_k_len, int window,
                                  float* weights, cudaStream_t s) {
  PromptKArgs a = args_of(c, p);
  a.max_k = max_k_len;
  a.window = window;
  a.lse_in = lse;
  a.weights = weights;
  CUtensorMap qm, km;
  if (!map_kv(c, p.k, p.k_stride, p.total_k, &km)) return cudaErrorInvalidValue;
  qm = km;  // no queries at all: nothing is copied
  if (p.total_q > 0 && !map_q(c, p, a, &qm)) return cudaErrorInvalidValue;
  a.ktiles = (max_k_len + kTile - 1) / kTile;
  int sms = 148;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c.device);
  return c.cfg.head_dim == 64 ? launch_weights_d<64>(qm, km, a, sms, s) : launch_weights_d<128>(qm, km, a, sms, s);
}

}  // namespace starkv
