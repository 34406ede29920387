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

__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Instruction descriptor of kind::f16 with bf16 operands, fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return make_idesc_f16(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);
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
  int H, h_kv, group, gb, head_blocks, R, batch, max_q, max_k, qtiles, window;
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
  uint64_t* pfull = bar + 3;          // [2] P_t written
  uint64_t* look = bar + 5;           // one phase per masked V tile: it is there,
  uint64_t* clean = bar + 6;          // and it has been looked over
  uint64_t* odone = bar + 7;          // every product done
  uint64_t* full = bar + 8;           // [ST]
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
    mbar_init(&pfull[0], 4);
    mbar_init(&pfull[1], 4);
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
        if (!mbar_wait(&empty[s], ((issued / ST) & 1) ^ 1)) {
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
    if (lane == 0 && nt > 0) {
      constexpr uint32_t idesc_s = idesc_bf16(128, kTile, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(128, D, false, true);
      const uint32_t ring = smem_u32(sm + SM::kRing), qa = smem_u32(sm);
      auto issue_s = [&](int t, int j) {
        const uint32_t ka = ring + (2 * j % ST) * SM::kTileBytes;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (ks >> 2) * kSub + (ks & 3) * 32;
          mma_f16(tmem + t * kTile, make_sdesc(qa + t * SM::kTileBytes + o, 16, 1024, 2),
                  make_sdesc(ka + o, 16, 1024, 2), idesc_s, ks > 0);
        }
        mma_commit(&sfull[t]);
      };
      auto wait_full = [&](int i) { return mbar_wait_poll(&full[i % ST], (i / ST) & 1); };
      ok = mbar_wait_poll(qfull, 0) && wait_full(0);
      if (ok) {
        tc_fence_after();
        if (ntile[0] > 0) issue_s(0, 0);
        if (ntile[1] > 0) issue_s(1, 0);
        mma_commit(&empty[0]);
      }
      int looked = 0;
      for (int j = 0; ok && j < nt; ++j) {
        ok = wait_full(2 * j + 1);
        if (ok && j >= first_masked) {
          mbar_arrive(look);
          ok = mbar_wait_poll(clean, looked++ & 1);
        }
        if (ok && j + 1 < nt) ok = wait_full(2 * j + 2);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || j >= ntile[t]) continue;
          if (!mbar_wait_poll(&pfull[t], j & 1)) {
            ok = false;
            continue;
          }
          tc_fence_after();
          const uint32_t va = ring + ((2 * j + 1) % ST) * SM::kTileBytes;
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            mma_f16_ts(tmem + 256 + t * kTile, tmem + t * kTile + ks * 8, make_sdesc(va + ks * 2048, kSub, 1024, 2),
                       idesc_o, (j > 0 || ks > 0) ? 1u : 0u);
          if (t == 1 || j >= ntile[1]) mma_commit(&empty[(2 * j + 1) % ST]);
          if (j + 1 < ntile[t]) issue_s(t, j + 1);
        }
        if (ok && j + 1 < nt) mma_commit(&empty[(2 * j + 2) % ST]);
      }
      mma_commit(odone);  // completes once every product issued above has
      if (!ok) mbar_wait(odone, 0, 100000000ull);
    }
  } else if (warp >= 10) {
    // ---------------- V tiles with masked keys ----------------
    // A key that some row does not see has p = 0 there, but 0 * inf and 0 * NaN are not 0, and the
    // rows behind the sequence are another's.  So values that are not finite are cleared (rows
    // behind the sequence, whatever they hold) and, where a row does see them, added at the end.
    for (int j = first_masked; ok && j < nt; ++j) {
      const int i = 2 * j + 1;
      const bool got = mbar_wait(look, (j - first_masked) & 1) && mbar_wait(&full[i % ST], (i / ST) & 1);
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
      if (!__all_sync(0xffffffffu, mbar_wait_poll(&sfull[t], j & 1))) {
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
      for (int c = 4; c < kTile; c += 4)
#pragma unroll
        for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], sv[c + u]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const bool move = live && (top - m) * a.scale_log2 > kMoveMax;  // m = -inf: true but for a row without scores
      if (__any_sync(0xffffffffu, move)) {
        if (j > 0) {
          const float f = move ? ex2((m - top) * a.scale_log2) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(to + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
            tmem_st32(to + c * 32, o);
          }
          l *= f;
        }
        if (move) m = top;
      }
      const float base = m == -INFINITY ? 0.f : m * a.scale_log2;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kTile / 64; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          const float p0 = ex2(fmaf(sv[c * 64 + 2 * u], a.scale_log2, -base));
          const float p1 = ex2(fmaf(sv[c * 64 + 2 * u + 1], a.scale_log2, -base));
          sum[(2 * u) & 3] += p0;
          sum[(2 * u + 1) & 3] += p1;
          w[u] = pack_bf2(p0, p1);
        }
        tmem_st32(ts + c * 32, w);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[t]);
    }
    // ---- O / l, and lse
    if (ntile[t] > 0 && ok && !__all_sync(0xffffffffu, mbar_wait(odone, 0))) ok = false;
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
// A CTA takes 128 keys of one (sequence, KV head), holds their K tile and walks the
// query tiles: S^T = K Q^T into TMEM (four buffers), one key per lane, so that the sum
// over queries and heads stays in a register.  Warps 0..3 take the even tiles, 4..7 the
// odd ones, warp 8 copies, warp 9 issues the products, warps 10 and 11 lay out each
// column's log-sum-exp and the last key it sees.
constexpr int kWeightThreads = 384;
constexpr int kColNone = -(1 << 30);  // a column that sees no key

template <int D>
struct WeightSmem {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr int kStages = 4;
  static constexpr uint32_t kRing = kTileBytes;  // behind the K tile
  static constexpr uint32_t kCols = kRing + kStages * kTileBytes;  // [stage][128] (lse in log2 units), [stage][128] last key
  static constexpr uint32_t kBar = kCols + kStages * kTile * 8;
  static constexpr uint32_t kBytes = kBar + 256 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kWeightThreads, 1)
    prompt_weights_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                          const PromptKArgs a) {
  using SM = WeightSmem<D>;
  constexpr int NSUB = D / 64;
  constexpr int ST = SM::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::kBar);
  uint64_t* kfull = bar;
  uint64_t* full = bar + 1;        // [ST] Q tile landed
  uint64_t* cols = full + ST;      // [ST] columns laid out (2 warps)
  uint64_t* empty = cols + ST;     // [ST] Q tile read by its products, columns by the 4 warps
  uint64_t* sfull = empty + ST;    // [4]
  uint64_t* sempty = sfull + 4;    // [4]
  uint64_t* done = sempty + 4;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  float* lse2 = reinterpret_cast<float*>(sm + SM::kCols);
  int* last = reinterpret_cast<int*>(sm + SM::kCols + ST * kTile * 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kt = blockIdx.x, kv = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  pdl_launch_dependents();
  const SeqSpan q = span_of(a, b);
  if (!q.ok) {
    if (tid == 0) set_status(a.status, STARKV_DEV_BAD_QUERY_SPAN);
    return;
  }
  if (kt * kTile >= q.keys) return;
  const int off = q.keys - q.n;
  // queries first .. n - 1 count; the tile's first key is seen from query kt * 128 - off on
  const int first = max(max(0, q.n - a.window), kt * kTile - off);
  const int per = first < q.n ? (q.n - first + a.R - 1) / a.R : 0;  // query tiles
  const int nt = per * a.head_blocks;

  // rows behind the box of a tile stay zero: they are columns of the products
  for (int s = 0; s < ST; ++s)
    for (int e = tid; e < (kTile - a.R * a.gb) * D / 8; e += kWeightThreads) {
      const int r = a.R * a.gb + e / (D / 8), c = e % (D / 8);
      *reinterpret_cast<uint4*>(sm + SM::kRing + s * SM::kTileBytes + (c >> 3) * kSub + r * 128 + (c & 7) * 16) =
          make_uint4(0, 0, 0, 0);
    }
  fence_async_smem();
  if (warp == 9) tmem_alloc(tslot, 512);
  if (tid == 0) {
    mbar_init(kfull, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&cols[s], 2);
      mbar_init(&empty[s], 5);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], 4);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  bool ok = true;
  float acc = 0.f;

  if (warp == 8) {
    // ---------------- copies ----------------
    if (lane == 0 && nt > 0) {
      mbar_arrive_expect_tx(kfull, SM::kTileBytes);
#pragma unroll
      for (int i = 0; i < NSUB; ++i)
        tma_load_2d(sm + i * kSub, &k_map, kv * D + i * 64, q.k0 + kt * kTile, kfull);
      int u = 0;
      for (; u < nt; ++u) {
        const int s = u % ST;
        if (!mbar_wait(&empty[s], ((u / ST) & 1) ^ 1)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[s], NSUB * a.R * a.gb * 128);
        const int hb = u / per, i0 = first + (u % per) * a.R;
#pragma unroll
        for (int i = 0; i < NSUB; ++i)
          tma_load_3d(sm + SM::kRing + s * SM::kTileBytes + i * kSub, &q_map, i * 64, kv * a.group + hb * a.gb,
                      q.q0 + i0, &full[s]);
      }
      if (!ok) {  // wait (with a limit) for the copies in flight
        mbar_wait(kfull, 0, 100000000ull);
        for (int i = max(0, u - ST); i < u; ++i) mbar_wait(&full[i % ST], (i / ST) & 1, 100000000ull);
      }
    }
  } else if (warp == 9) {
    // ---------------- products ----------------
    if (lane == 0 && nt > 0) {
      constexpr uint32_t idesc = idesc_bf16(128, kTile, false, false);
      const uint32_t ka = smem_u32(sm);
      ok = mbar_wait_poll(kfull, 0);
      for (int u = 0; ok && u < nt; ++u) {
        const int s = u % ST, w = u & 3;
        if (!mbar_wait_poll(&full[s], (u / ST) & 1) || !mbar_wait_poll(&sempty[w], ((u >> 2) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t qa = smem_u32(sm + SM::kRing + s * SM::kTileBytes);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (ks >> 2) * kSub + (ks & 3) * 32;
          mma_f16(tmem + w * kTile, make_sdesc(ka + o, 16, 1024, 2), make_sdesc(qa + o, 16, 1024, 2), idesc, ks > 0);
        }
        mma_commit(&sfull[w]);
        mma_commit(&empty[s]);
      }
      mma_commit(done);
      if (!ok) mbar_wait(done, 0, 100000000ull);
    }
  } else if (warp >= 10) {
    // ---------------- columns ----------------
    for (int u = 0; u < nt; ++u) {
      const int s = u % ST;
      const int hb = u / per, i0 = first + (u % per) * a.R;
      const int heads = min(a.gb, a.group - hb * a.gb);
      float x[2];
      int k[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = (warp - 10) * 64 + e * 32 + lane;
        const int i = i0 + c / a.gb, hh = c % a.gb;
        const bool live = c < a.R * a.gb && i < q.n && hh < heads;
        x[e] = 0.f;
        k[e] = kColNone;
        if (live) {
          x[e] = a.lse_in[(int64_t)(q.q0 + i) * a.H + kv * a.group + hb * a.gb + hh] * kLog2e;
          k[e] = off + i;
        }
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ((u / ST) & 1) ^ 1))) {
        ok = false;
        break;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = (warp - 10) * 64 + e * 32 + lane;
        lse2[s * kTile + c] = x[e];
        last[s * kTile + c] = k[e];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&cols[s]);
    }
  } else {
    // ---------------- sums: one key per thread ----------------
    const int g = warp >> 2;
    const int key = kt * kTile + (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    for (int u = g; u < nt; u += 2) {
      const int s = u % ST, w = u & 3;
      const bool got = mbar_wait_poll(&sfull[w], (u >> 2) & 1) && mbar_wait_poll(&cols[s], (u / ST) & 1);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // a column is masked for some key of the tile, or none of a query, in the first and the last tiles only
      const int i0 = first + (u % per) * a.R;
      const bool whole = off + i0 >= kt * kTile + kTile - 1 && i0 + a.R <= q.n && a.group % a.gb == 0;
      const float* x = lse2 + s * kTile;
      const int* k = last + s * kTile;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int c = 0; c < kTile; c += 32) {
        uint32_t v[32];
        tmem_ld32(trow + w * kTile + c, v);
        tmem_ld_wait();
        if (whole && c + 32 <= a.R * a.gb) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 y = *reinterpret_cast<const float4*>(x + c + e);
            sum[0] += ex2(fmaf(__uint_as_float(v[e]), a.scale_log2, -y.x));
            sum[1] += ex2(fmaf(__uint_as_float(v[e + 1]), a.scale_log2, -y.y));
            sum[2] += ex2(fmaf(__uint_as_float(v[e + 2]), a.scale_log2, -y.z));
            sum[3] += ex2(fmaf(__uint_as_float(v[e + 3]), a.scale_log2, -y.w));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p = ex2(fmaf(__uint_as_float(v[e]), a.scale_log2, -x[c + e]));
            sum[e & 3] += key <= k[c + e] ? p : 0.f;
          }
        }
      }
      acc += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sempty[w]);
        mbar_arrive(&empty[s]);
      }
    }
  }
  if (!ok && lane == 0) set_status(a.status, kDevWaitTimeout);
  if (warp == 9 && lane == 0 && nt > 0 && ok) mbar_wait(done, 0);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // the odd tiles' sums join the even ones' (the columns' memory is free by now)
  if (warp >= 4 && warp < 8) lse2[tid - 128] = acc;
  __syncthreads();
  if (warp < 4 && kt * kTile + tid < q.keys)
    a.weights[((int64_t)q.k0 + kt * kTile + tid) * a.h_kv + kv] = acc + lse2[tid];
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
cudaError_t launch_weights_d(const CUtensorMap& qm, const CUtensorMap& km, const PromptKArgs& a, int ktiles,
                             cudaStream_t s) {
  const size_t smem = WeightSmem<D>::kBytes;
  cudaError_t e =
      cudaFuncSetAttribute(prompt_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_chained(prompt_weights_kernel<D>, dim3(ktiles, a.h_kv, a.batch), dim3(kWeightThreads), smem, s, 1u, qm,
                        km, a);
}

}  // namespace

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
  const int ktiles = (max_k_len + kTile - 1) / kTile;
  return c.cfg.head_dim == 64 ? launch_weights_d<64>(qm, km, a, ktiles, s) : launch_weights_d<128>(qm, km, a, ktiles, s);
}

}  // namespace starkv
