// Full-width layers: causal attention of packed prompts, and the attention weights
// of a prompt, on tcgen05 / TMEM.
//
// Both kernels pack the query heads of a KV head into the rows of a tile: row r of a
// tile is query r / gb of the tile, head r % gb of the group (gb heads, R = 128 / gb
// queries), which one 3-D TMA box per 64 channels brings in.  A tile's K and V then
// serve every head of the group, and a causal tile wastes 128 / gb queries at most.
//
// Times in this file: of the large cases (sixteen packed prompts of 1 to 1999 tokens, 32 query
// over 8 KV heads; 2048 queries over 32768 keys, 32 heads; the weights of the last 64 queries of
// 4 x 32768 and of every query of 8001, 32 heads over 8) passes among others, a second and more of
// them, under the power cap; of the others a call's time on the GPU, calls back to back in a graph.
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
// exchange; with its coefficients in fp32 1.55e-7, evaluated in fp32 2.14e-7, within ex2.approx's
// 2^-22), 2^n from the bits of the sum that rounds x.  From -126.5 down those bits are 0's; NaN
// passes through.
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
// A value that is the same in every lane, said so that the compiler knows it: loops that
// issue products go by such values only, or their descriptors leave the uniform registers.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

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

struct Cut;

struct PromptKArgs {
  int ctas;             // CTAs that share the units' key tiles (0: one per unit)
  float* part_o;        // [ctas][2][256][D], relative to the part's maximum: [0] of a unit that began before the
  float2* part_ml;      // [ctas][2][256] (maximum, sum)                     CTA's stretch, [1] of one that goes on behind
  Cut* cuts;            // [ctas]
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
// A unit is two query tiles (2 R queries) of one (sequence, KV head, head block) with all the
// key tiles that they see.  One CTA an SM takes an equal stretch of the units' key tiles, laid
// end to end (each unit somewhat longer, for its start and its end), so that neither few
// long units nor many of unequal lengths leave SMs idle; a unit that a cut goes through leaves
// partial results, which a second kernel joins.  Where there are few keys, a CTA takes a whole
// unit and there is no second kernel.
//
// Warps 0..3 and 4..7 each hold one tile's softmax (one row per thread), warp 8 copies, warp 9
// issues the products, warps 10 and 11 look the V tiles of masked keys over.
//   S_t = Q_t K_j^T into TMEM; the softmax warps replace it by P_t in bf16 (the same
//   columns, half as many), which is the A operand of O_t += P_t V_j from TMEM.  In issue
//   order P_0 V_j, S_0 (j + 1), P_1 V_j, S_1 (j + 1): one tile's products run while the
//   other tile's softmax does.  The running maximum moves when a score passes it by more
//   than 2^8 only, and then the row's O is rescaled in place; S_t (j) complete implies
//   that P_t V_(j-1) is, so no further barrier guards that.  The next unit's Q and first
//   products run while the softmax warps write the last unit out.
constexpr int kAttnThreads = 384;  // 168 registers a thread, 12 bytes of which spill
// A CTA takes a whole unit where there are at most kFewKeys keys in all (32 query over 8 KV heads of 128,
// with the host's time: 256 tokens 23 us, 31 us cut and joined; 1000 tokens 25 and 42; one query of 1000
// keys 19 and 24), and where there are units for all SMs and the keys and values do not stay in L2: units
// that start together then read the same tiles together, stretches do not (32768 keys of 32 heads: 1046 us
// and 1116 us, for 65% and 26% of hits in L2; sixteen prompts that fit: 294 us and 275 us).
constexpr int kFewKeys = 1024;
constexpr int64_t kMostCached = (int64_t)96 << 20;  // bytes of keys and values
constexpr int kLeastTiles = 2;    // key tiles of a stretch, where there are few
// Positions that a unit counts for beside its key tiles: its start and its end cost as much as two
// (sixteen packed prompts: counted as 1, 2, 3, 4: 285, 275, 275, 280 us).
constexpr int kUnitCost = 2;
// Pairs of exponentials that go to the FMA pipe: one of eight.  (2048 queries over 32768 keys: none
// 1051 us, one of eight 1045, one of four 1053, half 1146: the softmax warps' issue slots bound them too.
// In short runs, below the power cap, 914, 894, 982 and 1070.)
__device__ constexpr bool on_fma_pipe(int pair) { return pair % 8 == 7; }

template <int D>
struct AttnSmem {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kRing = 2 * kTileBytes;  // behind the two Q tiles: K_0, V_0, K_1, V_1, ...
  static constexpr uint32_t kTold = kRing + kStages * kTileBytes;
  static constexpr uint32_t kBar = kTold + 2 * 64;
  static constexpr uint32_t kBytes = kBar + 384 + 1024;
};

// sum over i < n of floor((a i + b) / m), a, b >= 0, by the Euclidean steps of (a, m).
__device__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// Units of a sequence: pairs of query tiles, each with its key tiles.
struct Pairs {
  int n, off, M, count;  // queries; query i sees keys 0 .. off + i; queries of a pair
  __device__ Pairs() {}
  __device__ Pairs(const SeqSpan& q, int R) : n(q.ok ? q.n : 0), off(q.keys - q.n), M(2 * R) { count = (n + M - 1) / M; }
  // key tiles of pair i
  __device__ int tiles(int i) const {
    const int64_t seen = (int64_t)off + min((int64_t)n, (int64_t)(i + 1) * M);
    return seen > 0 ? (int)((seen + kTile - 1) / kTile) : 0;
  }
  // positions (key tiles, and kUnitCost a pair) of the pairs before pair x
  __device__ int64_t before(int x) const {
    const int64_t whole = min(x, count - 1);                               // pairs of M queries
    const int64_t first = off >= 0 ? 0 : ((int64_t)M - off) / M - 1;       // the first that sees a key
    int64_t sum = (int64_t)x * kUnitCost;
    if (whole > first) sum += floor_sum(whole - first, kTile, M, off + (first + 1) * M + kTile - 1);
    if (x == count && x > 0) sum += tiles(count - 1);
    return sum;
  }
};

// The pieces of a CTA, in order; every role walks its own copy.
struct Pieces {
  const PromptKArgs& a;
  int64_t pos, end;   // positions left
  int b, u, i, p;     // the next piece's sequence, KV head and head block, pair, and position in the unit
  SeqSpan q;
  Pairs pairs;
  // the present piece: key tiles j0 .. j1 - 1 of nt
  int j0, j1, nt, kv, hb, pair;
  bool fresh;         // the next piece is another unit's

  __device__ Pieces(const PromptKArgs& args, int64_t first, int64_t stop, int b_, const int (&start)[3], const SeqSpan& span)
      : a(args), pos(first), end(stop), b(b_), u(start[0]), i(start[1]), p(start[2]), fresh(false) {
    if (pos < end) {
      q = span;
      pairs = Pairs(q, a.R);
    }
  }
  __device__ bool next() {
    while (pos < end) {
      if (fresh) {
        fresh = false;
        p = 0;
        if (++i == pairs.count) {
          i = 0;
          if (++u == a.h_kv * a.head_blocks) {
            u = 0;
            do {  // (a position behind this one is some sequence's)
              q = span_of(a, ++b);
              pairs = Pairs(q, a.R);
            } while (pairs.count == 0);
          }
        }
      }
      nt = pairs.tiles(i);
      const int take = (int)min((int64_t)(nt + kUnitCost - p), end - pos);
      j0 = max(0, p - kUnitCost);
      j1 = max(0, p + take - kUnitCost);
      kv = u / a.head_blocks;
      hb = u % a.head_blocks;
      pair = i;
      pos += take;
      p += take;
      fresh = p == nt + kUnitCost;
      if (j1 > j0 || (nt == 0 && fresh)) return true;
    }
    return false;
  }
  __device__ bool whole() const { return j0 == 0 && j1 == nt; }
  __device__ int qbase() const { return pair * pairs.M; }
  // key tiles of query tile t
  __device__ int tiles_of(int t) const {
    const int rows = min(a.R, pairs.n - qbase() - t * a.R);
    const int keys = rows > 0 ? pairs.off + qbase() + t * a.R + rows : 0;
    return keys > 0 ? (keys + kTile - 1) / kTile : 0;
  }
  // the end of query tile t's key tiles in this piece (j0: none)
  __device__ int stop_of(int t) const { return max(j0, min(j1, tiles_of(t))); }
  // the first key tile that some row does not see whole
  __device__ int first_masked() const { return max(0, pairs.off + qbase() + 1) / kTile; }
};

// A piece as the softmax warps need it (warp 8 lays it out; two of them, in turn).
struct __align__(16) Told {
  int j0, stop[2];        // key tiles j0 .. stop[t] - 1 of query tile t
  int flags;              // kTold...
  int n, off, qbase;      // queries; query i sees keys 0 .. off + i; the pair's first query
  int heads;              // of the head block
  int first_masked;
  int k0, kv_at;          // the sequence's first key row, and the KV head's first channel
  int q_row;              // the pair's first query row
  int head0;              // the block's first head
  int pad[3];
};
static_assert(sizeof(Told) == 64, "");
enum { kToldWhole = 1, kToldLater = 2, kToldStop = 4 };  // all of the unit; not its first tiles; no more pieces

// What the join goes by: a unit that begins in this CTA and goes on behind its stretch.
struct Cut {
  int there, last;        // 0: none; the CTA that ends the unit
  int b, kv, hb, pair;
};

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const PromptKArgs a) {
  using SM = AttnSmem<D>;
  constexpr int NSUB = D / 64;
  constexpr int ST = SM::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t part[kAttnThreads / 32];
  __shared__ int64_t begin[2];        // the stretch's first sequence, and the positions before it
  __shared__ int start[3];            // and its unit: u, pair, position
  __shared__ SeqSpan first_span;
  uint8_t* sm = align1024(smem_raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::kBar);
  uint64_t* qfull = bar;              // both Q tiles landed
  uint64_t* qempty = bar + 1;         // and have been read
  uint64_t* sfull = bar + 2;          // [2] S_t ready
  uint64_t* pfull = bar + 4;          // [2][2] P_t written: its first 64 keys, the others
  uint64_t* odone = bar + 8;          // [2] a piece's products into O_t done
  uint64_t* oempty = bar + 10;        // [2] O_t read
  uint64_t* look = bar + 12;          // [4] masked V tiles, in turn: one has been asked for
  uint64_t* clean = bar + 16;         // [4] and it has been looked over
  uint64_t* told = bar + 20;          // [2] a piece is laid out,
  uint64_t* heard = bar + 22;         // [2] and done with
  uint64_t* full = bar + 24;          // [ST]
  uint64_t* empty = full + ST;        // [ST]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(empty + ST);
  Told* piece = reinterpret_cast<Told*>(sm + SM::kTold);
  int* dirty = reinterpret_cast<int*>(tslot + 1);  // a masked V tile held a value that is not finite
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  if (warp == 9) tmem_alloc(tslot, 512);
  if (tid == 0) {
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&odone[s], 1);
      mbar_init(&oempty[s], 4);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&pfull[s], 4);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&look[s], 1);
      mbar_init(&clean[s], 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&told[s], 1);
      mbar_init(&heard[s], 8);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    *dirty = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  // ---- the CTA's stretch
  const int units = a.h_kv * a.head_blocks;
  int64_t pos = 0, end = 0, total = 0;
  if (a.ctas == 0) {
    const int each = units * a.batch, unit = blockIdx.x % each;
    if (tid == 0) {
      const int i = a.qtiles - 1 - (int)(blockIdx.x / each);  // the pairs with the most keys first
      begin[0] = unit / units;
      start[0] = unit % units;
      start[1] = i;
      start[2] = 0;
      const SeqSpan q = span_of(a, unit / units);
      first_span = q;
      if (!q.ok) set_status(a.status, STARKV_DEV_BAD_QUERY_SPAN);
      const Pairs pairs(q, a.R);
      begin[1] = i < pairs.count ? pairs.tiles(i) + kUnitCost : 0;
    }
    tc_fence_before();
    __syncthreads();
    end = begin[1];
  } else {
    int64_t mine = 0;
    for (int i = tid; i < a.batch; i += kAttnThreads) {
      const SeqSpan q = span_of(a, i);
      if (!q.ok && blockIdx.x == 0) set_status(a.status, STARKV_DEV_BAD_QUERY_SPAN);
      const Pairs pairs(q, a.R);
      mine += pairs.before(pairs.count);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) part[warp] = mine;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAttnThreads / 32; ++w) total += part[w];
    total *= units;
    pos = cut(blockIdx.x, total, a.ctas);
    end = cut(blockIdx.x + 1, total, a.ctas);
    if (warp == 0 && pos < end) {
      // the sequence that holds pos, 32 at a time
      int64_t carry = 0;
      for (int i0 = 0; i0 < a.batch; i0 += 32) {
        int64_t w = 0;
        if (i0 + lane < a.batch) {
          const Pairs pairs(span_of(a, i0 + lane), a.R);
          w = pairs.before(pairs.count) * units;
        }
        int64_t inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        if (carry + inc - w <= pos && pos < carry + inc) {
          begin[0] = i0 + lane;
          begin[1] = carry + inc - w;
        }
        carry += __shfl_sync(0xffffffffu, inc, 31);
      }
      __syncwarp();
      // its unit: the last pair that begins at or before the position, in 32 parts at a time
      const SeqSpan span = span_of(a, (int)begin[0]);
      const Pairs pairs(span, a.R);
      if (lane == 0) first_span = span;
      const int64_t each = pairs.before(pairs.count), in = pos - begin[1], rest = in % each;
      int lo = 0, hi = pairs.count;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const uint32_t yes = __ballot_sync(0xffffffffu, at < hi && pairs.before(at) <= rest);
        lo += (31 - __clz(yes)) * step;  // (lane 0's is always one)
        hi = min(hi, lo + step);
      }
      if (lane == 0) {
        start[0] = (int)(in / each);
        start[1] = lo;
        start[2] = (int)(rest - pairs.before(lo));
      }
    }
    tc_fence_before();
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tslot);
  bool ok = true;
  Pieces it(a, pos, end, (int)begin[0], start, first_span);

  if (warp == 8) {
    // ---------------- copies ----------------
    if (lane == 0) {
      int r = 0, pieces = 0, all = 0, masked = 0;  // ring positions, pieces with keys, pieces, masked V tiles so far
      auto tell = [&](const Told& x) {
        if (!mbar_wait_short(&heard[all & 1], ((all >> 1) & 1) ^ 1)) return false;
        piece[all & 1] = x;
        mbar_arrive(&told[all & 1]);
        ++all;
        return true;
      };
      while (ok && it.next()) {
        ok = tell(Told{it.j0, {it.nt > 0 ? it.stop_of(0) : it.j0, it.nt > 0 ? it.stop_of(1) : it.j0},
                       (it.whole() ? kToldWhole : 0) | (it.j0 > 0 ? kToldLater : 0), it.pairs.n, it.pairs.off, it.qbase(),
                       min(a.gb, a.group - it.hb * a.gb), it.first_masked(), it.q.k0, it.kv * D, it.q.q0 + it.qbase(),
                       it.kv * a.group + it.hb * a.gb, {0, 0, 0}});
        if (!ok) break;
        if (it.nt == 0) continue;
        if (!mbar_wait_short(qempty, (pieces & 1) ^ 1)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(qfull, 2u * NSUB * a.R * a.gb * 128);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < NSUB; ++i)
            tma_load_3d(sm + t * SM::kTileBytes + i * kSub, &q_map, i * 64, it.kv * a.group + it.hb * a.gb,
                        it.q.q0 + it.qbase() + t * a.R, qfull);
        ++pieces;
        const int first_masked = it.first_masked();
        for (int e = 2 * it.j0; e < 2 * it.j1; ++e, ++r) {
          const int s = r % ST;
          if (!mbar_wait_short(&empty[s], ((r / ST) & 1) ^ 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], SM::kTileBytes);
#pragma unroll
          for (int i = 0; i < NSUB; ++i)
            tma_load_2d(sm + SM::kRing + s * SM::kTileBytes + i * kSub, e & 1 ? &v_map : &k_map, it.kv * D + i * 64,
                        it.q.k0 + (e >> 1) * kTile, &full[s]);
          // (the ring holds four V tiles at most, so none of the four barriers is two phases ahead)
          if ((e & 1) && (e >> 1) >= first_masked) mbar_arrive(&look[masked++ & 3]);
        }
      }
      if (ok) ok = tell(Told{0, {0, 0}, kToldStop, 0, 0, 0, 0, 0, 0, 0, 0, 0, {0, 0, 0}});
      if (!ok) {  // wait (with a limit) for the copies in flight
        if (pieces > 0) mbar_wait(qfull, (pieces - 1) & 1, 100000000ull);
        for (int i = max(0, r - ST); i < r; ++i) mbar_wait(&full[i % ST], (i / ST) & 1, 100000000ull);
      }
    }
  } else if (warp == 9) {
    // ---------------- products ----------------
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
    auto all = [&](bool got) { return uniform(__all_sync(0xffffffffu, got)) != 0; };
    // the ring's positions: a piece's next K and V tiles, each with its phase
    int kst = 0, vst = 1;
    uint32_t kph = 0, vph = 0;
    auto on = [&](int& st, uint32_t& ph) {
      st += 2;
      if (st >= ST) {
        st -= ST;
        ph ^= 1;
      }
    };
    int looked = 0;
    uint32_t qph = 0, pph[2] = {0, 0}, oph[2] = {0, 0};
    while (ok && uniform(it.next())) {
      if (uniform(it.nt) == 0) continue;
      const int j0 = uniform(it.j0), j1 = uniform(it.j1), first_masked = uniform(it.first_masked());
      const int stop[2] = {uniform(it.stop_of(0)), uniform(it.stop_of(1))};
      ok = all(mbar_wait_short(qfull, qph) && mbar_wait_short(&full[kst], kph));
      qph ^= 1;
      if (!ok) break;
      tc_fence_after();
      if (lead) {
        if (stop[0] > j0) issue_s(0, kst);
        if (stop[1] > j0) issue_s(1, kst);
        mma_commit(&empty[kst]);
        if (j1 - j0 == 1) mma_commit(qempty);
      }
      __syncwarp();
      on(kst, kph);
      for (int j = j0; ok && j < j1; ++j) {
        const bool more = j + 1 < j1;
        bool got = mbar_wait_short(&full[vst], vph);
        if (got && j >= first_masked) {
          got = mbar_wait_short(&clean[looked & 3], (looked >> 2) & 1);
          ++looked;
        }
        if (got && more) got = mbar_wait_short(&full[kst], kph);
        ok = all(got);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || j >= stop[t]) continue;
          if (j == j0) {  // the piece before has been read out of O_t
            ok = all(mbar_wait_short(&oempty[t], oph[t] ^ 1));
            oph[t] ^= 1;
          }
          const uint64_t v0 = desc_at(vd, vst * SM::kTileBytes);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!all(ok && mbar_wait_short(&pfull[t * 2 + h], pph[t]))) {
              ok = false;
              continue;
            }
            tc_fence_after();
            if (lead) {
#pragma unroll
              for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
                mma_f16_ts(tmem + 256 + t * kTile, tmem + t * kTile + ks * 8, desc_at(v0, ks * 2048), idesc_o,
                           j > j0 || ks > 0);
            }
            __syncwarp();
          }
          pph[t] ^= 1;
          if (!ok) continue;
          if (lead) {
            if (j + 1 < stop[t]) issue_s(t, kst);
            else mma_commit(&odone[t]);
          }
          __syncwarp();
        }
        if (ok && lead) {
          mma_commit(&empty[vst]);
          if (more) mma_commit(&empty[kst]);
          if (j + 2 == j1) mma_commit(qempty);
        }
        __syncwarp();
        on(vst, vph);
        if (more) on(kst, kph);
      }
      // (K_(j1) of the next piece follows V_(j1 - 1): kst already stands there)
    }
    if (!ok) {  // the products in flight still read shared memory and TMEM: wait (with a limit)
      if (lead) mma_commit(&odone[0]);
      __syncwarp();
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < 100000000ull) {
      }
    }
  } else if (warp >= 10) {
    // ---------------- V tiles with masked keys ----------------
    // A key that some row does not see has p = 0 there, but 0 * inf and 0 * NaN are not 0, and the
    // rows behind the sequence are another's.  So values that are not finite are cleared (rows
    // behind the sequence, whatever they hold) and, where a row does see them, added at the end.
    int r = 0, looked = 0;
    while (ok && it.next()) {
      if (it.nt == 0) continue;
      for (int j = max(it.j0, it.first_masked()); j < it.j1; ++j, ++looked) {
        const int i = r + 2 * (j - it.j0) + 1;
        const bool got =
            mbar_wait_short(&look[looked & 3], (looked >> 2) & 1) && mbar_wait_short(&full[i % ST], (i / ST) & 1);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        uint4* tile = reinterpret_cast<uint4*>(sm + SM::kRing + (i % ST) * SM::kTileBytes) + (warp - 10) * 32 + lane;
        __nv_bfloat162 top = __halves2bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));  // largest magnitude, NaN if any
#pragma unroll 8
        for (int e = 0; e < kTile * D / 8 / 64; ++e) {
          const uint4 x = tile[e * 64];
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[u])));
        }
        if (!isfinite(__low2float(top)) || !isfinite(__high2float(top))) {
          for (int e = 0; e < kTile * D / 8 / 64; ++e) {
            uint4 x = tile[e * 64];
            uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if ((w[u] & 0x7f80u) == 0x7f80u) w[u] &= 0xffff0000u;
              if ((w[u] & 0x7f800000u) == 0x7f800000u) w[u] &= 0x0000ffffu;
            }
            tile[e * 64] = x;
          }
          *reinterpret_cast<volatile int*>(dirty) = 1;
        }
        __threadfence_block();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&clean[looked & 3]);
      }
      r += 2 * (it.j1 - it.j0);
    }
  } else {
    // ---------------- softmax: one row per thread ----------------
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int row_q = t * a.R + r / a.gb, hh = r % a.gb;  // the row's query within the pair, and head within the block
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = trow + t * kTile, to = trow + 256 + t * kTile;
    uint32_t sph = 0, oph = 0;
    const bool in_tile = r < a.R * a.gb;
    for (int n = 0;; ++n) {
      if (!__all_sync(0xffffffffu, mbar_wait_short(&told[n & 1], (n >> 1) & 1))) {
        ok = false;
        break;
      }
      const Told& x = piece[n & 1];
      if (x.flags & kToldStop) break;
      const bool live = in_tile && x.qbase + row_q < x.n && hh < x.heads;
      // keys the row sees (may be <= 0); a row of nothing masks nothing
      const int seen = live ? x.off + x.qbase + row_q + 1 : 1 << 30;
      const int j0 = x.j0, stop = x.stop[t];
      float m = -INFINITY, l = 0.f;
      for (int j = j0; j < stop; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait_short(&sfull[t], sph))) {
          ok = false;
          break;
        }
        sph ^= 1;
        tc_fence_after();
        // masked keys (last tiles only): -inf takes their scores' place in TMEM, a quarter at a time in one
        // rolled loop, so that the code of the other tiles stays short (it is bound by its fetch, too)
        const int lim = seen - j * kTile;
        if (__any_sync(0xffffffffu, lim < kTile)) {
#pragma unroll 1
          for (int c = 0; c < kTile; c += 32) {
            if (!__any_sync(0xffffffffu, lim < c + 32)) continue;
            uint32_t y[32];
            tmem_ld32(ts + c, y);
            tmem_ld_wait32(y);
#pragma unroll
            for (int u = 0; u < 32; ++u) y[u] = u < lim - c ? y[u] : 0xff800000u;
            tmem_st32(ts + c, y);
          }
          tmem_st_wait();
        }
        // four quarters of the row's scores; the last is let go after the maximum and loaded again when the
        // first has been used up (all four beside P's words are more registers than a thread has)
        uint32_t sv[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, sv[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait32(sv[c]);
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          auto at = [&](int u) { return __uint_as_float(sv[c][u]); };
          float y[2] = {max3(at(0), at(1), at(2)), max3(at(3), at(4), at(5))};
#pragma unroll
          for (int u = 6; u < 30; u += 4) {
            y[0] = max3(y[0], at(u), at(u + 1));
            y[1] = max3(y[1], at(u + 2), at(u + 3));
          }
          mx[c] = max3(fmaxf(at(30), at(31)), y[0], y[1]);
        }
        const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        const bool move = live && (top - m) * a.scale_log2 > kMoveMax;  // m = -inf: true but for a row without scores
        if (__any_sync(0xffffffffu, move)) {
          if (j > j0) {
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
        // the first half of P goes on its way while the third quarter is computed
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
          if (c == 1) tmem_ld32(ts + 96, sv[3]);
          if (c == 3) tmem_ld_wait32(sv[3]);
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const f32x2 z = fma2(pair(__uint_as_float(sv[c][2 * u]), __uint_as_float(sv[c][2 * u + 1])), scale2, base2);
            const f32x2 p = on_fma_pipe(u) ? ex2_fma(z) : ex2_sfu(z);
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
      if (!ok) break;
      // ---- O / l and lse, or the part: O, m, l
      const bool any = stop > j0;
      if (any) {
        if (!__all_sync(0xffffffffu, mbar_wait_short(&odone[t], oph))) {
          ok = false;
          break;
        }
        oph ^= 1;
        tc_fence_after();
      }
      const bool whole = x.flags & kToldWhole;
      const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const int64_t row = (int64_t)(x.q_row + row_q) * a.H + x.head0 + hh;
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (x.flags & kToldLater ? 0 : 1)) * 2 * kTile + t * kTile + r;
      const bool fix = any && *reinterpret_cast<volatile int*>(dirty) != 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        __syncwarp();
        if (any) {
          tmem_ld32(to + c * 32, o);
          tmem_ld_wait();
          if (c == D / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&oempty[t]);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) o[u] = 0u;
        }
        if (!live) continue;
        if (fix)
          for (int j = max(x.first_masked, j0) * kTile; j < min(seen, stop * kTile); ++j) {
            const __nv_bfloat16* vr = a.v + (int64_t)(x.k0 + j) * a.v_stride + x.kv_at + c * 32;
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const float y = __bfloat162float(vr[u]);
              if (!isfinite(y)) o[u] = __float_as_uint(__uint_as_float(o[u]) + y);
            }
          }
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + c * 32);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf2(__uint_as_float(o[8 * u + 2 * e]) * inv, __uint_as_float(o[8 * u + 2 * e + 1]) * inv);
            dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(a.part_o + slot * D + c * 32);
#pragma unroll
          for (int u = 0; u < 8; ++u) dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
      }
      if (live && whole && a.lse) a.lse[row] = l == 0.f ? -INFINITY : fmaf(m, a.scale, logf(l));
      if (live && !whole) a.part_ml[slot] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&heard[n & 1]);
    }
  }
  if (!ok && lane == 0) set_status(a.status, kDevWaitTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (a.ctas > 0 && tid == 0) {
    // the unit that goes on behind the stretch, if its first key tiles are here: the last piece's
    Cut c = {0, 0, 0, 0, 0, 0};
    if (pos < end) {
      Pieces last(a, pos, end, (int)begin[0], start, first_span);
      bool any = false;
      int64_t unit_end = 0;
      while (last.next()) {
        any = last.j0 == 0 && last.j1 < last.nt;
        unit_end = last.pos + (last.nt - last.j1);
      }
      if (any) c = Cut{1, (int)cta_of(unit_end - 1, total, a.ctas), last.b, last.kv, last.hb, last.pair};
    }
    a.cuts[blockIdx.x] = c;
  }
}

// ---------------------------------------------------------------------------
// Join of the units that a cut went through: block (c, y) takes the y-th of the rows (as many as
// its threads hold at once) of the unit that begins in CTA c's stretch and goes on behind it.
// (16 queries of 32 heads over 8, 8000 keys: 25 us in all; with 32 rows a block, one after the other, 55.)
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) prompt_join_kernel(const PromptKArgs a) {
  constexpr int kRow = D / 4, kRows = kMergeThreads / kRow;  // threads of a row, rows of a block
  pdl_wait();
  pdl_launch_dependents();
  const int first = blockIdx.x;
  const Cut c = a.cuts[first];
  if (!c.there) return;
  const SeqSpan q = span_of(a, c.b);
  const int c4 = threadIdx.x % kRow * 4;
  // the thread's row of the unit, its tile, and its row there
  const int r2 = blockIdx.y * kRows + threadIdx.x / kRow, t = r2 / kTile, r = r2 % kTile;
  const int qi = c.pair * 2 * a.R + t * a.R + r / a.gb, hh = r % a.gb;
  if (r >= a.R * a.gb || qi >= q.n || hh >= min(a.gb, a.group - c.hb * a.gb)) return;
  auto slot = [&](int k) { return ((int64_t)k * 2 + (k == first)) * 2 * kTile + r2; };
  float m = -INFINITY;
  // (unrolled: a unit may have a part on every SM, and a part's loads take a round trip)
#pragma unroll 8
  for (int k = first; k <= c.last; ++k) m = fmaxf(m, a.part_ml[slot(k)].x);
  float l = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = first; k <= c.last; ++k) {
    const float2 ml = a.part_ml[slot(k)];
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + slot(k) * D + c4);
    const bool some = ml.y != 0.f;  // else no scores of the row there
    const float f = !some ? 0.f : m == -INFINITY ? 1.f : ex2((ml.x - m) * a.scale_log2);
    l = fmaf(ml.y, f, l);
    v.x = fmaf(some ? x.x : 0.f, f, v.x);
    v.y = fmaf(some ? x.y : 0.f, f, v.y);
    v.z = fmaf(some ? x.z : 0.f, f, v.z);
    v.w = fmaf(some ? x.w : 0.f, f, v.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t row = (int64_t)(q.q0 + qi) * a.H + c.kv * a.group + c.hb * a.gb + hh;
  *reinterpret_cast<uint2*>(a.out + row * D + c4) =
      make_uint2(pack_bf2(v.x * inv, v.y * inv), pack_bf2(v.z * inv, v.w * inv));
  if (c4 == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : fmaf(m, a.scale, logf(l));
}

// ===========================================================================
// Attention weights
// ===========================================================================
// An item is 128 keys of one (sequence, KV head); its steps are the tiles of queries that
// count and see any of them.  A step's product S^T = K Q^T (TMEM, four buffers) has one
// key per lane, so that the sum over queries and heads stays in a register of the thread
// that holds the key.  Warps 0..7 take the even steps, 8..15 the odd ones, half of the
// columns each (four warps a scheduler keep the exponentials going while others wait for
// their columns); warp 16 copies, warp 17 issues the products, warps 18 and 19 lay out each
// column's log-sum-exp and the last key it sees and note for each product what its sums go
// by.  A note without a product makes up an item's number where it has to be even.  One CTA an SM
// walks over many items, three ways:
//   resident  the counting queries of a (sequence, KV head) fit the ring (a window): a CTA
//             takes an equal stretch of the items in (sequence, KV head, key) order and
//             loads them once per (sequence, KV head); only K tiles stream.  (64 queries of
//             32 heads, 8 KV heads, 32768 keys: 27 us, streamed 44.)
//   streamed  items in the order of their first key (those of the first keys have the most
//             steps), dealt forth and back, so that the CTAs' sums of steps come out alike.
//   split     where there are few items, a cluster shares one item's steps out and adds the
//             sums through distributed shared memory, in rank order.  (2000 queries of 16
//             heads over one: 26 us, unsplit 160.)
constexpr int kWeightThreads = 640;
constexpr int kColNone = -(1 << 30);  // a column that sees no key
enum { kResident = 0, kStreamed = 1 };  // > 1: split over so many CTAs

template <int D>
struct WeightSmem {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 3 : 6;   // Q tiles
  static constexpr int kKeys = D == 128 ? 3 : 4;     // K tiles
  static constexpr uint32_t kRing = kKeys * kTileBytes;
  static constexpr int kSlots = 8;                   // steps' columns: they are read longer than the Q tile is
  static constexpr uint32_t kCols = kRing + kStages * kTileBytes;  // [slot][128] -lse in log2 units, [slot][128] last key
  static constexpr uint32_t kSums = kCols + kSlots * kTile * 8;    // [2][3][128] sums of warps 4 .. 15
  static constexpr uint32_t kNotes = kSums + 2 * 3 * kTile * 4;    // [4] what a product's sums go by
  static constexpr uint32_t kBar = kNotes + 4 * 32;
  static constexpr uint32_t kBytes = kBar + 512 + 1024;
};

// One product's note, beside its TMEM buffer.
struct __align__(16) Note {
  int flags;     // kWhole: no column is masked for any key; kLast: the item's last step; kLeave: its columns' last use; kStop
  int slot;      // the columns'
  int live;      // columns that hold queries
  int key0, keys;  // the item's first key, and the keys of its sequence
  int pad;
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
  uint64_t* empty = full + ST;     // [ST] and read by its products
  uint64_t* cfree = empty + ST;    // [kSlots] columns read by 8 warps
  uint64_t* sfull = cfree + SM::kSlots;  // [4] a product, and its columns and note are there,
  uint64_t* sempty = sfull + 4;    // [4] and have been read
  uint64_t* sums = sempty + 4;     // [2][4] three warps' sums are there
  uint64_t* taken = sums + 8;      // [2][4] and have been added
  uint64_t* done = taken + 8;
  uint64_t* both = done + 1;       // resident: warps 18 and 19 have laid a (sequence, KV head)'s columns out
  uint32_t* tslot = reinterpret_cast<uint32_t*>(both + 1);
  float* lse2 = reinterpret_cast<float*>(sm + SM::kCols);
  int* last = reinterpret_cast<int*>(sm + SM::kCols + SM::kSlots * kTile * 4);
  float* other = reinterpret_cast<float*>(sm + SM::kSums);
  Note* notes = reinterpret_cast<Note*>(sm + SM::kNotes);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
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
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < SM::kSlots; ++s) mbar_init(&cfree[s], 8);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sfull[s], 2);
      mbar_init(&sempty[s], 8);
    }
    for (int s = 0; s < 8; ++s) {
      mbar_init(&sums[s], 3);
      mbar_init(&taken[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(both, 2);
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
  const uint32_t tmem = (uint32_t)uniform((int)*tslot);
  const bool resident = a.mode == kResident;
  bool ok = true;
  Items it(a, pos, end, seq, before);
  // Stage and phase of step v, the u-th of this CTA.  Resident: the stage is the step's number, and
  // `flips` holds the stages' phases (a stage turns when a (sequence, KV head) that used it is done).
  uint32_t flips = 0;
  // A note without a product follows an item's steps where there is one alone (it ends the item for the
  // other warps), and where a resident item's number is odd: its columns stay over many items and only the
  // last item's readers say that they are done, so a step has to be read by the same eight warps in each.
  auto made_up = [&](int steps) { return (rank < steps && rank + split >= steps) || (resident && steps % 2 == 1); };
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
    bool more = uniform(it.next());
    while (ok && more) {
      const int steps = uniform(it.steps);
      more = uniform(it.next());
      if (steps == 0) continue;
      const bool free_q = uniform(!resident || !more || it.fresh);  // resident: the Q tiles' last use
      ok = uniform(__all_sync(0xffffffffu, mbar_wait_short(&kfull[ks], kph)));
      const uint64_t k0 = desc_at(kd, ks * SM::kTileBytes);
      for (int v = rank; ok && v < steps; v += split, ++u) {
        const int s = resident ? v : st, w = u & 3;
        const uint32_t ph = resident ? (flips >> v) & 1u : sph;
        ok = uniform(__all_sync(0xffffffffu, mbar_wait_short(&full[s], ph) && mbar_wait_short(&sempty[w], ((u >> 2) & 1) ^ 1)));
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
      if (ok && made_up(steps)) {
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
    // warp 18 does the even steps, warp 19 the odd ones: a step's work in one warp is longer than a step
    int u = 0, laid = 0, laid_units = 0;  // notes, (streamed) columns and (resident) (sequence, KV head)s so far
    auto my_turn = [&]() { return (u & 1) == warp - 18; };
    int col_r[4], col_h[4];  // the lane's columns: query within the tile, head within the block
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = e * 32 + lane;
      col_r[e] = c / a.gb;
      col_h[e] = c % a.gb;
    }
    auto note = [&](const Note& n) {  // for the u-th product, whose buffer must be free
      const int w = u & 3;
      if (!my_turn()) {
        ++u;
        return true;
      }
      if (!__all_sync(0xffffffffu, mbar_wait_short(&sempty[w], ((u >> 2) & 1) ^ 1))) return false;
      if (lane == 0) {
        notes[w] = n;
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
      // the log-sum-exps of the warp's next step are asked for before this step's slot is free
      float x[4], next_x[4];
      int hb = rank / per, i0 = first + rank % per * a.R;  // the step's head block and first query
      auto advance = [&](int& hb, int& i0) {
        i0 += split * a.R;
        while (i0 >= first + per * a.R) {
          i0 -= per * a.R;
          ++hb;
        }
      };
      auto live = [&](int e, int hb, int i0) {
        return col_r[e] < a.R && i0 + col_r[e] < n && hb * a.gb + col_h[e] < a.group;
      };
      auto fetch = [&](int v, int hb, int i0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          next_x[e] = 0.f;
          if (v < steps && live(e, hb, i0))
            next_x[e] = a.lse_in[(int64_t)(q0 + i0 + col_r[e]) * a.H + kv * a.group + hb * a.gb + col_h[e]];
        }
      };
      if (lay) {
        int h = hb, i = i0, v = rank;
        if (!my_turn()) {
          advance(h, i);
          v += split;
        }
        fetch(v, h, i);
      }
      for (int v = rank; v < steps; v += split) {
        const int s = resident ? v : laid % SM::kSlots;
        const uint32_t ph = resident ? (flips >> v) & 1u : (uint32_t)(laid / SM::kSlots) & 1u;
        ++laid;
        if (!my_turn()) {
          ++u;
          advance(hb, i0);
          continue;
        }
        if (lay) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = next_x[e];
          int h = hb, i = i0;
          advance(h, i);
          advance(h, i);
          fetch(v + 2 * split, h, i);
          if (!__all_sync(0xffffffffu, mbar_wait_short(&cfree[s], ph ^ 1))) {
            ok = false;
            break;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            lse2[s * kTile + e * 32 + lane] = x[e] * -kLog2e;
            last[s * kTile + e * 32 + lane] = live(e, hb, i0) ? off + i0 + col_r[e] : kColNone;
          }
          __syncwarp();
        }
        // a column is masked for some key of the tile in the first tiles only
        const bool whole = off + i0 >= key0 + kTile - 1 && (hb + 1) * a.gb <= a.group;
        if (!note(Note{(whole ? kWhole : 0) | (v + 2 * split >= steps ? kLast : 0) | (leave ? kLeave : 0), s,
                       min(a.R, n - i0) * a.gb, key0, keys, 0, row})) {
          ok = false;
          break;
        }
        advance(hb, i0);
      }
      if (ok && made_up(steps)) ok = note(Note{rank + split >= steps ? kLast : 0, 0, 0, key0, keys, 0, row});
      if (lay) flips ^= (1u << min(steps, ST)) - 1;
      // The two warps meet when a (sequence, KV head)'s columns are there.  (No order hangs on it; without it the
      // last 64 queries of 4 x 32768 take, in short runs in turn, 98 us for 89, 96 queries of each, three steps,
      // 136 for 124.)
      if (ok && resident && fresh) {
        if (lane == 0) mbar_arrive(both);
        ok = __all_sync(0xffffffffu, mbar_wait_short(both, laid_units & 1));
        ++laid_units;
      }
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
      const int s = note.slot, key = note.key0 + row;
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
          // one pair of eight on the FMA pipe (every query of 8001: 338 us, none 344, one of four 342; the last 64
          // of 4 x 32768: 100, 103 and 110)
          two[1] = add2(two[1], e % 16 == 0 ? ex2_fma(t1) : ex2_sfu(t1));
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
        if (lane == 0) mbar_arrive(&cfree[s]);
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
  const unsigned blocks = a.ctas > 0 ? (unsigned)a.ctas : (unsigned)a.qtiles * a.h_kv * a.head_blocks * a.batch;
  e = launch_chained(prompt_attn_kernel<D>, dim3(blocks), dim3(kAttnThreads), smem, s, 1u, qm, km, vm, a);
  if (e != cudaSuccess || a.ctas == 0) return e;
  return launch_chained(prompt_join_kernel<D>, dim3(a.ctas, 2 * kTile * (D / 4) / kMergeThreads), dim3(kMergeThreads), 0,
                        s, 1u, a);
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
  if (a.mode == kStreamed) {
    while (cluster < 8 && items * cluster * 2 <= sms && cluster * 2 <= most) cluster *= 2;
    // Pairs of CTAs where they come in two rounds, too, if all queries count: the items' steps then fall evenly
    // from `most` to none, and a pair that ends takes one of the short ones.  That spares most * sms / (4 items)
    // steps and costs a second round's start, 14 steps.  (Queries of 32 heads over 8: 1300 30 and 21 us, 2000 45
    // and 33, 256 of 2048 11 and, in pairs, 20; 4000 of 4 heads of 64 24 and 24.)
    if (items * 2 > sms && items <= sms && a.window >= a.max_k && most * sms > 56 * items) cluster = 2;
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

PromptPlan plan_prompt(const Ctx& c, int batch, int64_t total_q, int64_t total_k, int max_q_len) {
  PromptPlan p = {};
  const PromptKArgs a = args_of(c, PromptArgs{});
  const int64_t units = (int64_t)a.h_kv * a.head_blocks;
  p.blocks = ((int64_t)max_q_len + 2 * a.R - 1) / (2 * a.R) * units * batch;
  if (total_k <= kFewKeys) return p;
  const int sms = sm_count(c);
  // at most so many pairs of query tiles, and key tiles of one
  const int64_t pairs = total_q / (2 * a.R) + batch, tiles = (total_k + kTile - 1) / kTile;
  if (total_k * a.h_kv * c.cfg.head_dim * 4 > kMostCached && total_q / (2 * a.R) * units >= sms) return p;
  const int64_t most = pairs * units >= sms ? sms : pairs * units * ((tiles + kLeastTiles - 1) / kLeastTiles);
  p.ctas = (int)(most < sms ? most : sms);
  p.blocks = p.ctas;
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)p.ctas * 2 * 2 * kTile;
  p.off_ml = al(rows * c.cfg.head_dim * 4);
  p.off_cuts = p.off_ml + al(rows * 8);
  p.ws_bytes = p.off_cuts + al((size_t)p.ctas * sizeof(Cut));
  return p;
}

cudaError_t launch_prompt_attn(const Ctx& c, const PromptArgs& p, int max_q_len, __nv_bfloat16* out, float* lse,
                               void* ws, const PromptPlan& plan, cudaStream_t s) {
  PromptKArgs a = args_of(c, p);
  a.max_q = max_q_len;
  a.qtiles = (int)(((int64_t)max_q_len + 2 * a.R - 1) / (2 * a.R));
  a.out = out;
  a.lse = lse;
  a.ctas = plan.ctas;
  a.part_o = (float*)ws;
  a.part_ml = (float2*)((char*)ws + plan.off_ml);
  a.cuts = (Cut*)((char*)ws + plan.off_cuts);
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
  a.ktiles = (int)(((int64_t)max_k_len + kTile - 1) / kTile);
  const int sms = sm_count(c);
  return c.cfg.head_dim == 64 ? launch_weights_d<64>(qm, km, a, sms, s) : launch_weights_d<128>(qm, km, a, sms, s);
}

}  // namespace starkv
