// Attention over whole sequences, backward. With p_ij = e^(s_ij - lse_i) recomputed from q, k and the forward's lse:
//   dP = dO v^T,  D_i = sum_c dO_ic o_ic (= sum_j p_ij dP_ij),  dS = p (dP - D)
//   dv_j = sum_i p_ij dO_i,   dk_j = scale sum_i dS_ij q_i,   dq_i = scale sum_j dS_ij k_j
// summed over the query heads of a key head for dk and dv.
//
// Three kernels. k_attn_delta leaves D and lse log2(e) by head. k_attn_dq owns 128 queries and walks the key tiles they see;
// k_attn_dkv owns 128 keys of a key head and walks the query tiles (and the group's heads) that see them. Each output is
// summed in the accumulators of one CTA's tensor core in a fixed order, so nothing is added atomically and results do not depend on
// the order of blocks; the price is that both recompute s and dP: seven products of 128 x 128 x D a tile pair, where adding dq up in
// memory would need five.
//
// k_attn_dkv works on transposed scores, keys on the TMEM lanes, so that P^T and dS^T are TMEM-resident A operands:
//   S^T = K Q^T, dP^T = V dO^T  (shared-memory operands, K-major)
//   dV += P^T dO, dK += dS^T Q  (the same Q and dO tiles read MN-major)
// TMEM: S^T (P^T over it), dP^T (dS^T over it), dV, dK. The products run in the order dV(i), S(i+1), dK(i), dP(i+1): while a pair of
// them runs, the softmax warps turn the scores (or dP) of the other pair's into the next operand.
// k_attn_dq: S = Q K^T, dP = dO V^T, dQ += dS K (dS over S in TMEM; S double-buffered, a tile ahead).
// Both go through their output tiles in turn, one CTA an SM: an output leaves while the next tile's operands arrive and its first
// products run (2 x 4096 tokens x 16 heads: a CTA per tile spent 40 of 203 us, and 22 of 152, on starting and ending).
//
// Eight softmax warps, two to a quarter of the TMEM lanes, each on half of a tile's columns. The bf16 operand's halves lie over the
// columns that their own writers have read. 2 x 4096 causal tokens x 16 heads of 128: 18 us for D, 141 for dq, 181 for dk and dv, 1400 TFLOP/s
// of the seven products; the tensor core is busy 63 to 67% of it, the rest is the chain from a score to the operand made of it, for which
// TMEM (all 512 columns in use) leaves no second buffer. p and dS are rounded to bf16 (as the products' operands); all sums are fp32.
//
// D from o carries o's rounding to bf16, which a query of few keys feels (dP - D is small there, and 0 for a single key). So the
// query tiles that see one key tile, the first 128 queries of a causal sequence and all of a shorter one, have it from the scores
// themselves: sum_j p_ij dP_ij / sum_j p_ij. k_attn_dq, which has a query's whole row there, leaves it to k_attn_dkv, and a query
// of a single key has dS = 0 in both, at 1% of the time of the larger calls. (Sequences of 3 to 20 tokens: dq and dk off by 0.0027
// to 0.0033 of their size with o's D, 0.0024 so, what the operands' and outputs' roundings make.)
// The other queries keep o's D whatever their weights. Where one key has nearly all of the weight, dP - D is small at that key too, and so is the gradient:
// its error keeps the size of o's rounding (1024 causal tokens, heads of 128, every query leaning to one key: at a mean largest weight
// of 0.30 dq of the queries from the 128th on is off by 0.0038 of its size, at 0.95 by 0.034, at 0.999 by 0.37, where the
// gradient itself is a fortieth of evenly spread weights'; in no case was the error above 0.026 of the latter). A D
// as good as the first tile's would take the sum over p dP of all of a query's keys before the first of its dS: two products more of seven.
#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 384;                        // 8 softmax warps, the MMA warp, the TMA warp, two gate warps
constexpr int kMma = 8, kTma = 9, kGate = 10;        // the latter four
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;   // 8 x 208 + 4 x 88 = 12 x 168, the launch's
constexpr int kSoftmax = 256;
constexpr int kCols = 64;                            // columns of a tile to a softmax warp

template <int D>
struct Cfg {
  static constexpr int kTile = kAttnTile * D * 2;
  static constexpr int kSmem = 7 * kTile + 2 * 1024 + 512;  // 2 fixed tiles, rings of 3 and 2, two stages of vectors, barriers
};

// 64 columns of x, rounded to bf16, to 32 columns of TMEM.
__device__ __forceinline__ void store_operand(uint32_t t, const float* x) {
  float w[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) w[e] = __uint_as_float(pack_bf16(x[2 * e], x[2 * e + 1]));
  tmem_st32(t, w);
}

// kN columns of an accumulator row times f, as bf16.
template <int kN>
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, uint32_t t, float f, bool mine, bool wide) {
  float o[kN];
#pragma unroll
  for (int q = 0; q < kN / 32; ++q) tmem_ld32(t + q * 32, o + q * 32);
  tmem_wait_ld_regs(o);
  if (mine)
#pragma unroll
    for (int q = 0; q < kN / 32; ++q) store_bf16x32(dst + q * 32, o + q * 32, f, wide);
}

// Output tiles are handed out as CTAs get free, the ones with the most work first (a fixed assignment left some CTAs 20% more work
// on documents with grouped heads; a tile's result does not depend on who computes it). The producer warp takes the next one and
// passes it to the CTA's other threads through two places in shared memory.
struct Handout {
  long long* tile;             // [2]
  uint64_t *full, *empty;      // [2]
  unsigned* counter;           // tiles taken beyond every CTA's first, zeroed by k_attn_delta
  long long total;
  __device__ __forceinline__ void init(int readers) const {
    for (int i = 0; i < 2; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], readers);
  }
  // The producer warp's round: true with the tile, false at the end (`*ok`) or after an error.
  template <class W>
  __device__ __forceinline__ bool take(long long round, long long* i, bool* ok, W wait) const {
    const int at = int(round & 1);
    if (round >= 2) *ok = __all_sync(0xffffffffu, wait(&empty[at], (round >> 1) - 1 & 1, kDevTimeoutSync));
    if (!*ok) return false;
    long long mine = blockIdx.x;
    if ((threadIdx.x & 31) == 0) {
      if (round > 0) mine = (long long)gridDim.x + atomicAdd(counter, 1u);
      tile[at] = mine;
      mbar_arrive(&full[at]);
    }
    *i = __shfl_sync(0xffffffffu, mine, 0);
    return *i < total;
  }
  // Another thread's round, the same. kWarp: a warp's, known to be the same for its lanes (the MMA warp's control flow).
  template <bool kWarp, class W>
  __device__ __forceinline__ bool get(long long round, long long* i, bool* ok, W wait) const {
    const int at = int(round & 1);
    *ok = wait(&full[at], round >> 1 & 1, kDevTimeoutSync);
    if (kWarp) *ok = __all_sync(0xffffffffu, *ok);
    if (!*ok) return false;
    const unsigned got = unsigned(tile[at]);
    *i = kWarp ? __reduce_max_sync(0xffffffffu, got) : got;
    mbar_arrive(&empty[at]);
    return *i < total;
  }
};

}  // namespace

// -D_i and -lse_i log2(e) of 32 rows of a head a warp.
template <int D>
__global__ void __launch_bounds__(256) k_attn_delta(const __grid_constant__ AttnParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, which = lane / kLanes;
  const long long chunks = (p.rows + 31) / 32, item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  wait_for_previous();
  if (blockIdx.x == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0;
  if (item >= chunks * p.H) return;
  const int h = int(item % p.H);
  const long long row0 = item / p.H * 32;
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    const long long row = row0 + i * kRows + which;
    float x = 0.f;
    if (row < p.rows) {
      const long long at = (row * p.H + h) * D + sub * 8;
      const uint4 a = *reinterpret_cast<const uint4*>(p.dO + at), b = *reinterpret_cast<const uint4*>(p.o_in + at);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) x = fmaf(bf16_lo(u[e]), bf16_lo(v[e]), fmaf(bf16_hi(u[e]), bf16_hi(v[e]), x));
    }
#pragma unroll
    for (int d = kLanes / 2; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    // row i kRows + w of the 32 was summed by the lanes of part w
    const float got = __shfl_sync(0xffffffffu, x, (lane % kRows) * kLanes);
    if (lane / kRows == i) mine = got;
  }
  const long long row = row0 + lane;
  if (row < p.rows) {
    p.delta[h * p.rows + row] = -mine;
    p.lse2[h * p.rows + row] = p.lse_in[row * p.H + h] * -kLog2e;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_dkv(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
               const __grid_constant__ CUtensorMap mdo, const __grid_constant__ AttnParams p) {
  constexpr int kTile = Cfg<D>::kTile, kQ = 3, kO = 2;  // stages of Q and of dO (a Q tile is needed longer)
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t *sK = sm, *sV = sK + kTile, *sQ = sV + kTile, *sO = sQ + kQ * kTile;
  float* vec = reinterpret_cast<float*>(sO + kO * kTile);  // [2][lse2 | delta][128]
  uint64_t* bar = reinterpret_cast<uint64_t*>(vec + 2 * 256);
  uint64_t *kv_full = bar, *kv_empty = bar + 1, *q_full = bar + 2, *q_empty = bar + 5, *o_full = bar + 8, *o_empty = bar + 10, *ready = bar + 12, *vec_free = bar + 14,
           *s_full = bar + 16, *dp_full = bar + 17, *p_ready = bar + 18, *ds_ready = bar + 19, *done = bar + 20, *drained = bar + 21;
  const Handout hand{reinterpret_cast<long long*>(bar + 22), bar + 24, bar + 26, p.counters, (long long)p.tiles * p.Hk};
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 28);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + 29);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMma) tmem_alloc(tslot, 512);
  if (tid == 0) {
    *abort_flag = 0;
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    for (int i = 0; i < kQ; ++i) mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], 1);
    for (int i = 0; i < kO; ++i) mbar_init(&o_full[i], 1), mbar_init(&o_empty[i], 1), mbar_init(&ready[i], 32), mbar_init(&vec_free[i], kSoftmax);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, kSoftmax + 1);
    mbar_init(ds_ready, kSoftmax + 1);
    mbar_init(done, 1);
    mbar_init(drained, 1);
    hand.init(kSoftmax + 32 + 2);  // the softmax warps, the MMA warp and the gates
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_for_previous();
  constexpr uint32_t tS = 0, tP = 128, tV = 256, tK = 256 + D;  // all of TMEM, so it starts at column 0
  auto wait = [&](uint64_t* b, uint32_t ph, int code) { return attn_wait(b, ph, abort_flag, p.status, code); };
  // A warp's: its lanes come out of it together and of one mind, as the instructions on TMEM behind it need (tcgen05 `.sync.aligned`).
  auto warp_wait = [&](uint64_t* b, uint32_t ph, int code) { return bool(__all_sync(0xffffffffu, wait(b, ph, code))); };

  // A tile: its key head, keys, first query tile, query tiles a head, and all it walks.
  struct Item {
    int hk, i0, per, n;
    AttnTile tl;
    bool ragged;
  };
  auto describe = [&](long long i, Item* x) {
    x->hk = int(i % p.Hk);
    x->tl = attn_tile(p, int(i / p.Hk), kAttnTile, p.causal != 0);
    const int all = (x->tl.len + kAttnTile - 1) / kAttnTile;
    x->i0 = p.causal ? x->tl.first / kAttnTile : 0;
    x->per = all - x->i0;
    x->n = x->per * p.group;
    x->ragged = all * kAttnTile > x->tl.len;
  };
  Item x;
  // The round's tile, as the producer and the others learn of it; false at the end, and after an error (*ok false).
  auto take = [&](long long round, bool* ok) {
    long long i;
    if (!hand.take(round, &i, ok, wait)) return false;
    describe(i, &x);
    return true;
  };
  auto get = [&](long long round, bool* ok) {
    long long i;
    if (!hand.get<false>(round, &i, ok, wait)) return false;
    describe(i, &x);
    return true;
  };
  auto get_warp = [&](long long round, bool* ok) {
    long long i;
    if (!hand.get<true>(round, &i, ok, wait)) return false;
    describe(i, &x);
    return true;
  };

  if (warp >= kMma) {
    regs_dec<kOtherRegs>();
    if (warp == kTma) {
      // ---------------- producer ----------------
      Ring<kQ, 1> rq(0);
      Ring<kO, 1> ro(0);
      int use = 0;        // query tiles requested
      uint32_t tiles = 0;  // key tiles
      bool ok = true;
      for (long long rd = 0; ok && take(rd, &ok); ++rd) {
        if (tiles > 0) ok = __all_sync(0xffffffffu, wait(kv_empty, (tiles - 1) & 1, kDevTimeoutMma));
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(kv_full, 2 * kTile);
          load_attn_tile<D>(sK, &mk, x.hk * D, x.tl.row0 + x.tl.first, kv_full);
          load_attn_tile<D>(sV, &mv, x.hk * D, x.tl.row0 + x.tl.first, kv_full);
        }
        ++tiles;
        int h = x.hk * p.group, q0 = x.i0 * kAttnTile;
        for (int it = 0; it < x.n && ok; ++it) {
          const int y = x.tl.row0 + q0;
          ok = use < kQ || wait(&q_empty[rq.at], rq.phase ^ 1u, kDevTimeoutMma);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (lane == 0) {
            mbar_expect_tx(&q_full[rq.at], kTile);
            load_attn_tile<D>(sQ + rq.at * kTile, &mq, h * D, y, &q_full[rq.at]);
          }
          ok = use < kO || (wait(&o_empty[ro.at], ro.phase ^ 1u, kDevTimeoutMma) && wait(&vec_free[ro.at], ro.phase ^ 1u, kDevTimeoutSync));
          if (!(ok = __all_sync(0xffffffffu, ok))) {
            if (lane == 0) mbar_drain(&q_full[rq.at], rq.phase);
            break;
          }
          if (lane == 0) {
            mbar_expect_tx(&o_full[ro.at], kTile);
            load_attn_tile<D>(sO + ro.at * kTile, &mdo, h * D, y, &o_full[ro.at]);
          }
          float* v = vec + ro.at * 256;
          const long long at = (long long)h * p.rows + y;
#pragma unroll
          for (int e = lane; e < kAttnTile; e += 32) {
            const bool in = q0 + e < x.tl.len;
            v[e] = in ? p.lse2[at + e] : -INFINITY;
            v[128 + e] = in ? p.delta[at + e] : 0.f;
          }
          if (x.ragged && q0 + kAttnTile > x.tl.len) {
            ok = wait(&q_full[rq.at], rq.phase, kDevTimeoutTma) && wait(&o_full[ro.at], ro.phase, kDevTimeoutTma);
            if (!(ok = __all_sync(0xffffffffu, ok))) {
              if (lane == 0) mbar_drain(&q_full[rq.at], rq.phase), mbar_drain(&o_full[ro.at], ro.phase);
              break;
            }
            zero_attn_rows<D>(sQ + rq.at * kTile, x.tl.len - q0, lane);
            zero_attn_rows<D>(sO + ro.at * kTile, x.tl.len - q0, lane);
            fence_async_smem();
          }
          mbar_arrive(&ready[ro.at]);
          ++use;
          rq.next();
          ro.next();
          q0 += kAttnTile;
          if (q0 >= x.tl.len) {  // the next head of the group
            q0 = x.i0 * kAttnTile;
            ++h;
          }
        }
      }
      if (!ok && lane == 0) {  // the copies in flight land before their destination is given up
        if (tiles) mbar_drain(kv_full, (tiles - 1) & 1);
        for (int k = max(0, use - kQ); k < use; ++k) mbar_drain(&q_full[k % kQ], k / kQ & 1);
        for (int k = max(0, use - kO); k < use; ++k) mbar_drain(&o_full[k % kO], k / kO & 1);
      }
    } else if (warp == kMma) {
      // ---------------- MMA issuer ----------------
      const uint32_t lead = elect_lead();
      const uint32_t aK = desc_low_k(smem_u32(sK)), aV = desc_low_k(smem_u32(sV)), bQ = desc_low_k(smem_u32(sQ)), bO = desc_low_k(smem_u32(sO)),
                     nQ = desc_low_mn(smem_u32(sQ), kAttnPanel), nO = desc_low_mn(smem_u32(sO), kAttnPanel);
      Ring<kQ, 1> rq(0);   // the products' Q, S's one tile ahead of dK's
      uint32_t u = 0;      // query tiles so far
      auto scores = [&](int at) {
        product_ss<D>(lead, tS, aK, bQ + at * (kTile >> 4));
        commit(lead, s_full);
      };
      auto dprobs = [&](uint32_t os, bool last) {
        product_ss<D>(lead, tP, aV, bO + os * (kTile >> 4));
        commit(lead, dp_full);
        if (last) commit(lead, kv_empty);
      };
      bool ok = true;
      for (long long rd = 0; ok && get_warp(rd, &ok); ++rd) {
        // the first products overwrite operands that the products issued so far have read
        ok = warp_wait(kv_full, rd & 1, kDevTimeoutTma) && warp_wait(&q_full[rq.at], rq.phase, kDevTimeoutTma) && warp_wait(&ready[u & 1], u >> 1 & 1, kDevTimeoutSync);
        if (!ok) break;
        tc_fence_after();
        scores(rq.at);
        if (!(ok = warp_wait(&o_full[u & 1], u >> 1 & 1, kDevTimeoutTma))) break;
        dprobs(u & 1, x.n == 1);
        for (int it = 0; it < x.n; ++it, ++u) {
          // the gates answer for the tiles of the products that follow either operand
          if (!(ok = warp_wait(p_ready, u & 1, kDevTimeoutSync))) break;
          tc_fence_after();
          const int qs = rq.at;
          const uint32_t os = u & 1;
          rq.next();
          product_ts<D, kCols / 2>(lead, tV, tS, nO + os * (kTile >> 4), it > 0);
          commit(lead, &o_empty[os]);
          if (it + 1 < x.n) scores(rq.at);
          if (!(ok = warp_wait(ds_ready, u & 1, kDevTimeoutSync))) break;
          tc_fence_after();
          product_ts<D, kCols / 2>(lead, tK, tP, nQ + qs * (kTile >> 4), it > 0);
          commit(lead, &q_empty[qs]);
          if (it + 1 < x.n) dprobs(os ^ 1u, it + 2 == x.n);
        }
        if (ok) commit(lead, done);
      }
      if (!ok) {  // the products in flight end before their accumulators are given up
        commit(lead, drained);
        mbar_drain(drained, 0);
      }
    } else if (warp >= kGate && lane == 0) {
      // ---------------- gates: one warp for S(it + 1) behind dV(it), the other for dP(it + 1) behind dK(it) ----------------
      uint64_t* b = warp == kGate ? p_ready : ds_ready;
      Ring<kQ, 1> rq(0);
      uint32_t u = 0;
      bool ok = true;
      for (long long rd = 0; ok && get(rd, &ok); ++rd)
        for (int it = 0; it < x.n && ok; ++it, ++u) {
          rq.next();
          if (it + 1 < x.n) {
            const uint32_t os = (u + 1) & 1, ph = (u + 1) >> 1 & 1;
            ok = warp == kGate ? wait(&q_full[rq.at], rq.phase, kDevTimeoutTma) && wait(&ready[os], ph, kDevTimeoutSync) : wait(&o_full[os], ph, kDevTimeoutTma);
            if (!ok) break;
          }
          mbar_arrive(b);
          ok = wait(b, u & 1, kDevTimeoutSync);  // the next arrival belongs to the next phase
        }
    }
  } else {
    // ---------------- softmax: 32 key rows a warp, half of the queries ----------------
    // The rows' values come as the products' fragments (four rows and every fourth pair of columns a thread), so that a query's
    // lse and D, which differ by column, are read from shared memory once for four rows: with a row a thread those reads took 128
    // KB of shared memory's bandwidth an iteration, beside 192 KB of the products' and 64 KB of the copies'.
    regs_inc<kSoftmaxRegs>();
    const int half = warp >> 2, g = lane >> 2, col = (lane & 3) * 2, key0 = (warp & 3) * 32 + g;  // rows key0 + 8 r
    const uint32_t lane0 = tmem_lane_base(warp), lb = lane0 + uint32_t(half) * kCols;
    const F2 c2 = dup2(p.scale * kLog2e);
    const bool wide = (reinterpret_cast<uintptr_t>(half ? p.dk : p.dv) & 31) == 0;
    bool ok = true;
    uint32_t u = 0;
    for (long long rd = 0; ok && get_warp(rd, &ok); ++rd) {
      const AttnTile& tl = x.tl;
      int q0 = x.i0 * kAttnTile + half * kCols;
      for (int it = 0; it < x.n && ok; ++it, ++u) {
        const uint32_t os = u & 1;
        const float2 *lse = reinterpret_cast<const float2*>(vec + os * 256 + half * kCols + col), *delta = lse + 64;
        ok = warp_wait(&ready[os], u >> 1 & 1, kDevTimeoutSync) && warp_wait(s_full, u & 1, kDevTimeoutMma);
        if (!ok) break;
        tc_fence_after();
        // w[32 h + 4 b + 2 r + y]: row key0 + 16 h + 8 r, column 8 b + col + y
        float w[64];
        tmem_ld_16x64(tS + lb, w);
        tmem_ld_16x64(tS + lb + (16u << 16), w + 32);
        tmem_wait_ld_regs(w);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const float2 l = lse[4 * b];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float* x = w + (r >> 1) * 32 + 4 * b + (r & 1) * 2;
            unf2(fma2(f2(x[0], x[1]), c2, f2(l.x, l.y)), &x[0], &x[1]);
            x[0] = exp2_approx(x[0]);
            x[1] = exp2_approx(x[1]);
          }
        }
        const int to = tl.len - q0 - col;  // columns (from this thread's first) of queries that exist
        if (tl.len - q0 < kCols || (p.causal && tl.first + kAttnTile > q0)) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int from = p.causal ? tl.first + key0 + 8 * r - q0 - col : 0;  // and of those that see the row's key
#pragma unroll
            for (int b = 0; b < 8; ++b)
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if (8 * b + y < from || 8 * b + y >= to) w[(r >> 1) * 32 + 4 * b + (r & 1) * 2 + y] = 0.f;
          }
        }
        uint32_t out[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) out[e] = pack_bf16(w[2 * e], w[2 * e + 1]);
        tmem_st_16x32(tS + lb, out);
        tmem_st_16x32(tS + lb + (16u << 16), out + 16);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready);
        if (!(ok = warp_wait(dp_full, u & 1, kDevTimeoutMma))) break;
        tc_fence_after();
        float d[64];
        tmem_ld_16x64(tP + lb, d);
        tmem_ld_16x64(tP + lb + (16u << 16), d + 32);
        tmem_wait_ld_regs(d);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const float2 l = delta[4 * b];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int at = (r >> 1) * 32 + 4 * b + (r & 1) * 2;
            unf2(mul2(f2(w[at], w[at + 1]), add2(f2(d[at], d[at + 1]), f2(l.x, l.y))), &d[at], &d[at + 1]);
          }
        }
        mbar_arrive(&vec_free[os]);
        if (q0 + col == 0 && (p.causal || tl.len == 1))  // the sequence's first query sees a single key
#pragma unroll
          for (int r = 0; r < 4; ++r) d[(r >> 1) * 32 + (r & 1) * 2] = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) out[e] = pack_bf16(d[2 * e], d[2 * e + 1]);
        tmem_st_16x32(tP + lb, out);
        tmem_st_16x32(tP + lb + (16u << 16), out + 16);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(ds_ready);
        q0 += kAttnTile;
        if (q0 - half * kCols >= tl.len) q0 = x.i0 * kAttnTile + half * kCols;  // the next head of the group
      }
      if (!ok || !(ok = warp_wait(done, rd & 1, kDevTimeoutMma))) break;
      tc_fence_after();
      const int key = tl.first + (tid & 127);
      __nv_bfloat16* dst = (half ? p.dk : p.dv) + ((size_t(tl.row0) + key) * p.Hk + x.hk) * D;
      const uint32_t acc = (half ? tK : tV) + lane0;
      store_row<D>(dst, acc, half ? p.scale : 1.f, key < tl.len, wide);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(*tslot, 512);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_dq(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
              const __grid_constant__ CUtensorMap mdo, const __grid_constant__ AttnParams p) {
  constexpr int kTile = Cfg<D>::kTile, kK = 3, kV = 2;  // stages of K (needed longer) and V
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t *sQ = sm, *sO = sQ + kTile, *sK = sO + kTile, *sV = sK + kK * kTile;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sV + kV * kTile);
  uint64_t *q_full = bar, *q_empty = bar + 1, *k_full = bar + 2, *k_empty = bar + 5, *zeroed = bar + 8, *v_full = bar + 11, *v_empty = bar + 13, *s_full = bar + 15,
           *dp_full = bar + 17, *ds_ready = bar + 18, *done = bar + 19, *drained = bar + 20;
  const Handout hand{reinterpret_cast<long long*>(bar + 21), bar + 23, bar + 25, p.counters + 1, (long long)p.tiles * p.H};
  uint64_t* summed = bar + 27;  // [4]: both halves of 32 queries' rows
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 31);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + 32);
  float2* sums = reinterpret_cast<float2*>(bar + 64);  // [256]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMma) tmem_alloc(tslot, 512);
  if (tid == 0) {
    *abort_flag = 0;
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < kK; ++i) mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1), mbar_init(&zeroed[i], 32);
    for (int i = 0; i < kV; ++i) mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 1), mbar_init(&s_full[i], 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_ready, kSoftmax + 1);
    mbar_init(done, 1);
    mbar_init(drained, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&summed[i], 64);
    hand.init(kSoftmax + 32 + 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_for_previous();
  constexpr uint32_t tP = 256, tQ = 384;  // all of TMEM, so it starts at column 0
  auto tS = [&](uint32_t u) { return (u & 1) * 128; };
  auto wait = [&](uint64_t* b, uint32_t ph, int code) { return attn_wait(b, ph, abort_flag, p.status, code); };
  auto warp_wait = [&](uint64_t* b, uint32_t ph, int code) { return bool(__all_sync(0xffffffffu, wait(b, ph, code))); };

  // A tile: its head and key head, queries, key tiles, and whether the last of those reaches past the sequence.
  struct Item {
    int h, hk, n;
    bool tail;
    AttnTile tl;
  };
  auto describe = [&](long long i, Item* x) {
    x->h = int(i % p.H);
    x->hk = x->h / p.group;
    x->tl = attn_tile(p, int(i / p.H), kAttnTile, false);
    x->n = p.causal ? x->tl.first / kAttnTile + 1 : (x->tl.len + kAttnTile - 1) / kAttnTile;
    x->tail = x->n * kAttnTile > x->tl.len;
  };
  Item x;
  // The round's tile, as the producer and the others learn of it; false at the end, and after an error (*ok false).
  auto take = [&](long long round, bool* ok) {
    long long i;
    if (!hand.take(round, &i, ok, wait)) return false;
    describe(i, &x);
    return true;
  };
  auto get = [&](long long round, bool* ok) {
    long long i;
    if (!hand.get<false>(round, &i, ok, wait)) return false;
    describe(i, &x);
    return true;
  };
  auto get_warp = [&](long long round, bool* ok) {
    long long i;
    if (!hand.get<true>(round, &i, ok, wait)) return false;
    describe(i, &x);
    return true;
  };

  if (warp >= kMma) {
    regs_dec<kOtherRegs>();
    if (warp == kTma) {
      // ---------------- producer ----------------
      Ring<kK, 1> rk(0);
      Ring<kV, 1> rv(0);
      int use = 0;         // key tiles requested
      uint32_t tiles = 0;  // query tiles
      bool ok = true;
      for (long long rd = 0; ok && take(rd, &ok); ++rd) {
        if (tiles > 0) ok = __all_sync(0xffffffffu, wait(q_empty, (tiles - 1) & 1, kDevTimeoutMma));
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(q_full, 2 * kTile);
          load_attn_tile<D>(sQ, &mq, x.h * D, x.tl.row0 + x.tl.first, q_full);
          load_attn_tile<D>(sO, &mdo, x.h * D, x.tl.row0 + x.tl.first, q_full);
        }
        ++tiles;
        for (int i = 0; i < x.n && ok; ++i) {
          const int y = x.tl.row0 + i * kAttnTile;
          ok = use < kK || wait(&k_empty[rk.at], rk.phase ^ 1u, kDevTimeoutMma);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (lane == 0) {
            mbar_expect_tx(&k_full[rk.at], kTile);
            load_attn_tile<D>(sK + rk.at * kTile, &mk, x.hk * D, y, &k_full[rk.at]);
          }
          ok = use < kV || wait(&v_empty[rv.at], rv.phase ^ 1u, kDevTimeoutMma);
          if (!(ok = __all_sync(0xffffffffu, ok))) {
            if (lane == 0) mbar_drain(&k_full[rk.at], rk.phase);
            break;
          }
          if (lane == 0) {
            mbar_expect_tx(&v_full[rv.at], kTile);
            load_attn_tile<D>(sV + rv.at * kTile, &mv, x.hk * D, y, &v_full[rv.at]);
          }
          if (x.tail && i + 1 == x.n) {
            ok = __all_sync(0xffffffffu, wait(&k_full[rk.at], rk.phase, kDevTimeoutTma));
            if (!ok) {
              if (lane == 0) mbar_drain(&k_full[rk.at], rk.phase), mbar_drain(&v_full[rv.at], rv.phase);
              break;
            }
            zero_attn_rows<D>(sK + rk.at * kTile, x.tl.len - i * kAttnTile, lane);
            fence_async_smem();
            mbar_arrive(&zeroed[rk.at]);
          }
          ++use;
          rk.next();
          rv.next();
        }
      }
      if (!ok && lane == 0) {  // the copies in flight land before their destination is given up
        if (tiles) mbar_drain(q_full, (tiles - 1) & 1);
        for (int k = max(0, use - kK); k < use; ++k) mbar_drain(&k_full[k % kK], k / kK & 1);
        for (int k = max(0, use - kV); k < use; ++k) mbar_drain(&v_full[k % kV], k / kV & 1);
      }
    } else if (warp == kMma) {
      // ---------------- MMA issuer ----------------
      const uint32_t lead = elect_lead();
      const uint32_t aQ = desc_low_k(smem_u32(sQ)), aO = desc_low_k(smem_u32(sO)), bK = desc_low_k(smem_u32(sK)), bV = desc_low_k(smem_u32(sV)),
                     nK = desc_low_mn(smem_u32(sK), kAttnPanel);
      Ring<kK, 1> rs(0), rk(0);  // K of the scores, and of dq
      uint32_t u = 0, zeros = 0;  // key tiles so far; a bit per stage, the phase of its next zeroing
      auto scores = [&](uint32_t at, bool last) {  // S of key tile u = at, once its K has landed
        bool there = warp_wait(&k_full[rs.at], rs.phase, kDevTimeoutTma);
        if (there && last && x.tail) {
          there = warp_wait(&zeroed[rs.at], zeros >> rs.at & 1u, kDevTimeoutSync);
          zeros ^= 1u << rs.at;
        }
        if (!there) return false;
        tc_fence_after();
        product_ss<D>(lead, tS(at), aQ, bK + rs.at * (kTile >> 4));
        commit(lead, &s_full[at & 1]);
        rs.next();
        return true;
      };
      auto dprobs = [&](uint32_t at, bool last) {
        product_ss<D>(lead, tP, aO, bV + (at & 1) * (kTile >> 4));
        commit(lead, dp_full);
        commit(lead, &v_empty[at & 1]);
        if (last) commit(lead, q_empty);  // and the scores, issued before, have read Q
      };
      bool ok = true;
      for (long long rd = 0; ok && get_warp(rd, &ok); ++rd) {
        // the first products overwrite operands that the products issued so far have read
        if (!(ok = warp_wait(q_full, rd & 1, kDevTimeoutTma) && scores(u, x.n == 1) && warp_wait(&v_full[u & 1], u >> 1 & 1, kDevTimeoutTma))) break;
        if (x.n > 1) {
          dprobs(u, false);
          if (!(ok = scores(u + 1, x.n == 2))) break;
        } else {
          dprobs(u, true);
        }
        for (int i = 0; i < x.n; ++i, ++u) {
          // the gate answers for V of the next tile
          if (!(ok = warp_wait(ds_ready, u & 1, kDevTimeoutSync))) break;
          tc_fence_after();
          if (i + 1 < x.n) dprobs(u + 1, i + 2 == x.n);
          product_ts<D, kCols / 2>(lead, tQ, tS(u), nK + rk.at * (kTile >> 4), i > 0);
          commit(lead, &k_empty[rk.at]);
          rk.next();
          // K of the tile after next is requested when the product before this one has let go of its stage
          if (i + 2 < x.n && !(ok = scores(u + 2, i + 3 == x.n))) break;
        }
        if (ok) commit(lead, done);
      }
      if (!ok) {  // the products in flight end before their accumulators are given up
        commit(lead, drained);
        mbar_drain(drained, 0);
      }
    } else if (warp == kGate && lane == 0) {
      // ---------------- gate: V of the product that follows dS(i) has landed ----------------
      uint32_t u = 0;
      bool ok = true;
      for (long long rd = 0; ok && get(rd, &ok); ++rd)
        for (int i = 0; i < x.n && ok; ++i, ++u) {
          if (i + 1 < x.n && !(ok = wait(&v_full[(u + 1) & 1], (u + 1) >> 1 & 1, kDevTimeoutTma))) break;
          mbar_arrive(ds_ready);
          ok = wait(ds_ready, u & 1, kDevTimeoutSync);  // the next arrival belongs to the next phase
        }
    }
  } else {
    // ---------------- softmax: query row, half of the keys ----------------
    regs_inc<kSoftmaxRegs>();
    const int half = warp >> 2, row = tid & 127;
    const uint32_t lane0 = tmem_lane_base(warp), lb = lane0 + uint32_t(half) * kCols;
    const F2 c2 = dup2(p.scale * kLog2e);
    const bool wide = (reinterpret_cast<uintptr_t>(p.dq) & 31) == 0;
    bool ok = true;
    uint32_t u = 0, short_rows = 0;
    for (long long rd = 0; ok && get_warp(rd, &ok); ++rd) {
      const int qi = x.tl.first + row;
      const bool mine = qi < x.tl.len;
      const long long at = (long long)x.h * p.rows + x.tl.row0 + qi;
      const F2 lse = dup2(mine ? p.lse2[at] : 0.f);
      F2 delta = dup2(mine && x.n > 1 ? p.delta[at] : 0.f);
      for (int i = 0; i < x.n && ok; ++i, ++u) {
        if (!(ok = warp_wait(&s_full[u & 1], u >> 1 & 1, kDevTimeoutMma))) break;
        tc_fence_after();
        float w[kCols], d[kCols];
        tmem_ld64(tS(u) + lb, w);
        tmem_wait_ld_regs(w);
#pragma unroll
        for (int e = 0; e < kCols / 2; ++e) {
          float a, b;
          unf2(fma2(f2(w[2 * e], w[2 * e + 1]), c2, lse), &a, &b);
          w[2 * e] = exp2_approx(a);
          w[2 * e + 1] = exp2_approx(b);
        }
        if (!(ok = warp_wait(dp_full, u & 1, kDevTimeoutMma))) break;
        tc_fence_after();
        tmem_ld64(tP + lb, d);
        tmem_wait_ld_regs(d);
        const int seen = p.causal ? min(qi + 1, x.tl.len) : x.tl.len;
        const int left = seen - i * kAttnTile - half * kCols;
        if (x.n == 1) {
          // the row's D from its two halves' sums; a half's slot is written again only after the other's dS of this tile
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            if (e >= left) w[e] = d[e] = 0.f;
          F2 a = dup2(0.f), b = a;
#pragma unroll
          for (int e = 0; e < kCols / 2; ++e) {
            a = fma2(f2(w[2 * e], w[2 * e + 1]), f2(d[2 * e], d[2 * e + 1]), a);
            b = add2(b, f2(w[2 * e], w[2 * e + 1]));
          }
          float a0, a1, b0, b1;
          unf2(a, &a0, &a1);
          unf2(b, &b0, &b1);
          sums[tid] = make_float2(a0 + a1, b0 + b1);
          mbar_arrive(&summed[warp & 3]);
          if (!(ok = warp_wait(&summed[warp & 3], short_rows++ & 1, kDevTimeoutSync))) break;
          const float2 lo = sums[row], hi = sums[row + 128];
          const float own = -(lo.x + hi.x) / (lo.y + hi.y);
          delta = dup2(own);
          if (mine && half == 0) p.delta[at] = own;
        }
#pragma unroll
        for (int e = 0; e < kCols / 2; ++e) unf2(mul2(f2(w[2 * e], w[2 * e + 1]), add2(f2(d[2 * e], d[2 * e + 1]), delta)), &d[2 * e], &d[2 * e + 1]);
        if (i + 1 == x.n && (p.causal || x.tail)) {
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            if (e >= left) d[e] = 0.f;
        }
        if (seen == 1 && half == 0) d[0] = 0.f;
        store_operand(tS(u) + lb, d);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(ds_ready);
      }
      if (!ok || !(ok = warp_wait(done, rd & 1, kDevTimeoutMma))) break;
      tc_fence_after();
      __nv_bfloat16* dst = p.dq + ((size_t(x.tl.row0) + qi) * p.H + x.h) * D + half * (D / 2);
      store_row<D / 2>(dst, tQ + lane0 + half * (D / 2), p.scale, mine, wide);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(*tslot, 512);
}

template <int D>
static cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo, const AttnParams& p, const AttnParams& pk, cudaStream_t s) {
  constexpr int kSmem = Cfg<D>::kSmem;
  static std::atomic<unsigned long long> done_dkv{0}, done_dq{0};
  cudaError_t e = allow_smem(k_attn_dkv<D>, kSmem, &done_dkv);
  if (e == cudaSuccess) e = allow_smem(k_attn_dq<D>, kSmem, &done_dq);
  if (e != cudaSuccess) return e;
  const long long items = (p.rows + 31) / 32 * p.H;
  e = launch_after(k_attn_delta<D>, dim3(unsigned((items + 7) / 8)), dim3(256), 0, s, p);
  if (e != cudaSuccess) return e;
  const long long nk = (long long)p.tiles * p.Hk, nq = (long long)p.tiles * p.H;
  e = launch_after(k_attn_dq<D>, dim3(unsigned(nq < p.sms ? nq : p.sms)), dim3(kThreads), kSmem, s, mq, mk, mv, mdo, p);
  if (e != cudaSuccess) return e;
  return launch_after(k_attn_dkv<D>, dim3(unsigned(nk < p.sms ? nk : p.sms)), dim3(kThreads), kSmem, s, mq, mk, mv, mdo, pk);
}

cudaError_t launch_attn_bwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo, int D, const AttnParams& p, const AttnParams& pk,
                            cudaStream_t s) {
  return D == 128 ? launch<128>(mq, mk, mv, mdo, p, pk, s) : launch<64>(mq, mk, mv, mdo, p, pk, s);
}

}  // namespace gdn
