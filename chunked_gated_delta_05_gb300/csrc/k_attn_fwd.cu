// Attention over whole sequences, forward.
//
// For every query i of a head and the keys j it sees (all of its sequence, or those up to itself):
//   s_ij = scale q_i . k_j,  o_i = sum_j e^(s_ij) v_j / sum_j e^(s_ij),  lse_i = log sum_j e^(s_ij)
// in one pass over the keys: with a running reference m (log2 units below), weights p = 2^(c s - m), their sum l and the
// weighted sum of v are kept, and o = sum / l at the end.
//
// A CTA takes 256 queries of one head at a time, as two tiles of 128, and goes through such items in turn. A tile's row of scores
// belongs to two threads, one for either half of its keys (TMEM lane = row), so the softmax needs no shuffles. The two tiles
// alternate on the tensor core: while one tile's 256 threads turn scores into weights, the other's products run.
//   S_t = Q_t K_j^T        128 x 128 x D, operands in shared memory (128-byte swizzle, by TMA)
//   O_t += P_t V_j         128 x D x 128, P_t bf16 in TMEM over S_t's columns (the A operand), V_j read MN-major
// TMEM: S_0, S_1, O_0, O_1. Keys and values come through one ring of stages. Weights are rounded to bf16 (2^-8 relative at most, the
// type of v and o); scores, sums and the accumulators are fp32.
//
// What bounds it: with heads of 128 the tensor core. A tile's two products take 1312 cycles (its 128 x 128 x 16 steps 64, or 100 where both
// operands come from shared memory), so two tiles 2624 of the 2870 that an iteration takes: 16 heads x 8192 causal
// queries in 188 us, 1460 TFLOP/s. With heads of 64 it is the chain of a tile, softmax (1400 cycles), products and the signals between
// them (1200): 8 x 1001 queries x 16 heads, every key, 53 us. One thread a row, with 8 softmax warps for 16, took 193 and 57 us: a warp
// alone on its scheduler has 1060 cycles for a row's 128 weights, two with 64 each have 800.
// An instruction is taken only when the one before it is nearly done, and every wait, even for a phase long past, costs some 75 cycles
// in which the core may idle. So the issuing thread waits once per tile and iteration, on a barrier on which both the tile's
// 256 softmax threads and a gate thread arrive, the latter when the K and V tiles needed next have landed.
//
// The reference m is the row's maximum in its first tile and moves only when half of a later tile has weights that sum to more than
// 2^16 (then l and the accumulator are rescaled and the tile's weights taken again): weights up to that cost no precision in bf16 or
// fp32, almost no tile needs it, and no maximum is taken in the others. The two warps of a row agree on it at a barrier of their own,
// in every tile. It needs no wait: the commit that announces S_t(j) also covers the product O_t(j - 1) issued before it.
//
// Keys past the sequence's end are masked in the scores, and the last tile's values past it are zeroed in shared memory: they
// belong to the next sequence, and 0 x NaN would carry a neighbour's NaN over. Within a causal sequence nothing is zeroed: a value that is not
// finite reaches the queries before it in its own tile, as it does in the product that defines o.
//
// With heads of 128 the compiler spills 24 bytes a thread (an item's key tiles, indexed by the query tile).
#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 640;                      // 16 softmax warps, the MMA warp, the TMA warp and a gate warp for either tile
constexpr int kMma = 16, kTma = 17, kGate = 18;
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;  // 16 x 104 + 4 x 64 = 20 x 96, the launch's
constexpr int kCols = 64;                          // columns of a tile to a softmax warp
constexpr float kHigh = 65536.f;  // sum of half a tile's weights that moves the reference
// The reference of a row whose scores so far are all minus infinity: their weights come out as zero, and any other score moves it.
constexpr float kNone = -1e30f;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = kAttnTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kSmem = (2 + kStages) * kTileBytes + 512 + 2048;  // tiles, barriers, sums of the rows' halves
};

// Whether any of the two warps that share a tile's 32 rows says so. Both take part in every one, whatever befell either.
__device__ __forceinline__ bool pair_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(uint32_t(x))
      : "memory");
  return r != 0;
}

// The CTA's item of a round, most work first: every other round the other way round, so that the CTAs' sums of work come out
// alike. False where the last round has none for it.
struct Item {
  int h, hk, n[2], most;  // head and key head; key tiles of either query tile (the second sees no fewer, or has no rows)
  bool tail;              // the last key tile reaches past the sequence
  AttnTile tl;
};
__device__ __forceinline__ bool item_of(const AttnParams& p, long long round, long long total, Item* it) {
  const long long i = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  if (i >= total) return false;
  it->h = int(i % p.H);
  it->hk = it->h / p.group;
  it->tl = attn_tile(p, int(i / p.H), kAttnPair, false);
  const int all = (it->tl.len + kAttnTile - 1) / kAttnTile;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int q0 = it->tl.first + t * kAttnTile;
    it->n[t] = q0 >= it->tl.len ? 0 : p.causal ? q0 / kAttnTile + 1 : all;
  }
  it->most = max(it->n[0], it->n[1]);
  it->tail = it->most * kAttnTile > it->tl.len;
  return true;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_fwd(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnParams p) {
  using C = Cfg<D>;
  constexpr int kS = C::kStages, kTile = C::kTileBytes;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* sKV = sm + 2 * kTile;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sKV + kS * kTile);
  uint64_t *q_full = bar, *q_empty = bar + 2, *s_full = bar + 4, *p_full = bar + 6, *o_full = bar + 8, *kv_full = bar + 10, *kv_empty = kv_full + kS, *zeroed = kv_empty + kS,
           *drained = zeroed + kS;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(drained + 2);
  float* halves = reinterpret_cast<float*>(bar + 64);  // [2][2][128], by tile, half and row: the half's sum of weights
  static_assert(10 + 3 * kS + 3 <= 64, "barriers");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long total = (long long)p.tiles * p.H, rounds = (total + gridDim.x - 1) / gridDim.x;
  if (warp == kMma) tmem_alloc(tslot, 512);
  if (tid == 0) {
    *abort_flag = 0;
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 2 * kAttnTile + 1);
      mbar_init(&o_full[t], 1);
    }
    for (int i = 0; i < kS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
      mbar_init(&zeroed[i], 32);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_for_previous();
  // All of TMEM, so it starts at column 0: S_t at 128 t, O_t at 256 + D t.
  auto tS = [&](int t) { return uint32_t(t) * 128; };
  auto tO = [&](int t) { return 256 + uint32_t(t) * D; };
  auto wait = [&](uint64_t* b, uint32_t ph, int code) { return attn_wait(b, ph, abort_flag, p.status, code); };
  Item it;

  if (warp >= kMma) {
    regs_dec<kOtherRegs>();
    if (warp == kTma) {
      // ---------------- producer: Q, then K and V tile by tile through the ring ----------------
      Ring<kS, 1> r(0);
      int use = 0;                   // tiles requested through the ring
      uint32_t q_use[2] = {0, 0};    // items whose tile t has rows
      bool ok = true;
      for (long long rd = 0; rd < rounds && ok; ++rd) {
        if (!item_of(p, rd, total, &it)) break;
        for (int i = 0; i < 2 * it.most && ok; ++i, ++use, r.next()) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (i != t || !it.n[t]) continue;  // Q_0 ahead of the first K, Q_1 behind it
            ok = q_use[t] == 0 || wait(&q_empty[t], (q_use[t] - 1) & 1, kDevTimeoutMma);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) {
              mbar_expect_tx(&q_full[t], kTile);
              load_attn_tile<D>(sm + t * kTile, &mq, it.h * D, it.tl.row0 + it.tl.first + t * kAttnTile, &q_full[t]);
            }
            ++q_use[t];
          }
          ok = ok && (use < kS || wait(&kv_empty[r.at], r.phase ^ 1u, kDevTimeoutMma));
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          uint8_t* dst = sKV + r.at * kTile;
          if (lane == 0) {
            mbar_expect_tx(&kv_full[r.at], kTile);
            load_attn_tile<D>(dst, i & 1 ? &mv : &mk, it.hk * D, it.tl.row0 + (i >> 1) * kAttnTile, &kv_full[r.at]);
          }
          if (it.tail && i == 2 * it.most - 1) {
            ok = __all_sync(0xffffffffu, wait(&kv_full[r.at], r.phase, kDevTimeoutTma));
            if (!ok) break;
            zero_attn_rows<D>(dst, it.tl.len - (it.most - 1) * kAttnTile, lane);
            fence_async_smem();
            mbar_arrive(&zeroed[r.at]);
          }
        }
      }
      if (!ok && lane == 0) {  // the copies in flight land before their destination is given up
        for (int k = max(0, use - kS + 1); k < use; ++k) mbar_drain(&kv_full[k % kS], (k / kS) & 1);
        mbar_drain(&kv_full[r.at], r.phase, 1000000ull);  // this one if it was requested
        for (int t = 0; t < 2; ++t)
          if (q_use[t]) mbar_drain(&q_full[t], (q_use[t] - 1) & 1);
      }
    } else if (warp == kMma) {
      // ---------------- MMA issuer ----------------
      const uint32_t lead = elect_lead();
      const uint32_t q = desc_low_k(smem_u32(sm)), kk = desc_low_k(smem_u32(sKV)), vv = desc_low_mn(smem_u32(sKV), kAttnPanel);
      Ring<kS, 2> rk(0), rv(1);
      uint32_t cnt[2] = {0, 0}, q_use[2] = {0, 0};  // iterations and items of either tile so far
      bool ok = true, begun[2];
      auto all_wait = [&](uint64_t* b, uint32_t ph, int code) { return bool(__all_sync(0xffffffffu, wait(b, ph, code))); };
      auto scores = [&](int t, int at, bool last) {
        product_ss<D>(lead, uint32_t(t) * 128, q + t * (kTile >> 4), kk + at * (kTile >> 4));
        commit(lead, &s_full[t]);
        if (last) commit(lead, &q_empty[t]);
      };
      auto outputs = [&](int t, int j) {
        const uint32_t v = vv + rv.at * (kTile >> 4), d = 256 + uint32_t(t) * D;
        if (!all_wait(&p_full[t], cnt[t]++ & 1, kDevTimeoutSync)) return false;
        tc_fence_after();
        product_ts<D, kCols / 2>(lead, d, uint32_t(t) * 128, v, j > 0);
        return true;
      };
      // A tile's first scores of an item overwrite the weights of the item before it, which the products issued so far have read; its
      // first output product waits for weights from threads that have taken the former item's output out before.
      auto begin = [&](int t, const Item& x, int use) {  // use: of the item's first K tile
        begun[t] = true;
        if (!x.n[t]) return true;
        if (t == 0 && !all_wait(&kv_full[use % kS], use / kS & 1, kDevTimeoutTma)) return false;  // the first tile begins first
        if (!all_wait(&q_full[t], q_use[t]++ & 1, kDevTimeoutTma)) return false;
        scores(t, use % kS, x.n[t] == 1);
        return true;
      };
      Item next;
      int use = 0;
      bool more = item_of(p, 0, total, &it);
      if (more) ok = begin(0, it, 0) && begin(1, it, 0);
      for (long long rd = 0; more && ok; ++rd) {
        more = item_of(p, rd + 1, total, &next);
        use += 2 * it.most;
        begun[0] = begun[1] = false;
        for (int j = 0; j < it.most && ok; ++j) {
          rk.next();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok) continue;
            if (j >= it.n[t]) {  // ahead of the other tile: the next item's scores meanwhile
              if (t == 0 && more && !begun[0]) ok = begin(0, next, use);
              continue;
            }
            if (!(ok = outputs(t, j))) break;
            if (j + 1 < it.n[t]) scores(t, rk.at, j + 2 == it.n[t]);
            else commit(lead, &o_full[t]);
          }
          rv.next();
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && more && !begun[t]) ok = begin(t, next, use);
        it = next;
      }
      if (!ok) {  // the products in flight end before their accumulators are given up
        commit(lead, drained);
        mbar_drain(drained, 0);
      }
    } else if (warp >= kGate && lane == 0) {
      // ---------------- gate of a tile: the tiles that the products behind its weights read have landed ----------------
      const int t = warp - kGate;
      Ring<kS, 2> rk(0), rv(1);
      uint32_t cnt = 0, outs = 0, zeros = 0;  // iterations and items so far; a bit per stage, the phase of its next zeroing
      bool ok = true;
      for (long long rd = 0; rd < rounds && ok; ++rd) {
        if (!item_of(p, rd, total, &it)) break;
        const bool frees = t == 1 || !it.n[1];  // this tile's products are the last to read a stage
        for (int j = 0; j < it.most && ok; ++j) {
          const int k = rk.at, v = rv.at;
          const uint32_t v_phase = rv.phase;
          rk.next();
          rv.next();
          if (it.tail && j + 1 == it.most) zeros ^= 1u << v;
          if (j >= it.n[t]) continue;
          ok = wait(&kv_full[v], v_phase, kDevTimeoutTma) && (j + 1 == it.n[t] || wait(&kv_full[rk.at], rk.phase, kDevTimeoutTma)) &&
               (!it.tail || j + 1 < it.most || wait(&zeroed[v], ~zeros >> v & 1u, kDevTimeoutSync));
          if (!ok) break;
          mbar_arrive(&p_full[t]);
          // weights j are there: their scores are done, and the output product of the weights before them
          ok = wait(&p_full[t], cnt++ & 1, kDevTimeoutSync);
          if (!ok) break;
          if (frees) {
            mbar_arrive(&kv_empty[k]);
            if (j > 0) mbar_arrive(&kv_empty[v >= 2 ? v - 2 : v - 2 + kS]);
          }
          if (j + 1 == it.n[t]) {
            ok = wait(&o_full[t], outs++ & 1, kDevTimeoutMma);
            if (ok && frees) mbar_arrive(&kv_empty[v]);
          }
        }
      }
    }
  } else {
    // ---------------- softmax: a query row and half of its keys a thread ----------------
    regs_inc<kSoftmaxRegs>();
    const int t = warp >> 3, half = warp >> 2 & 1, row = tid & 127, pair = 1 + t * 4 + (warp & 3);
    const uint32_t lb = tmem_lane_base(warp), lS = tS(t) + lb + uint32_t(half) * kCols, lO = tO(t) + lb + uint32_t(half) * (D / 2);
    float *own = halves + (2 * t + half) * kAttnTile + row, *his = halves + (2 * t + (half ^ 1)) * kAttnTile + row;
    const float c = p.scale * kLog2e;
    const F2 c2 = dup2(c);
    const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
    uint32_t cnt = 0, outs = 0;
    bool ok = true;
    auto warp_wait = [&](uint64_t* b, uint32_t ph) { return bool(__all_sync(0xffffffffu, wait(b, ph, kDevTimeoutMma))); };
    for (long long rd = 0; rd < rounds && ok; ++rd) {
      if (!item_of(p, rd, total, &it)) break;
      const int mine = it.n[t], len = it.tl.len, qi = it.tl.first + t * kAttnTile + row;  // in the sequence
      if (mine == 0) continue;
      const float high = qi < len ? kHigh : INFINITY;  // rows behind the sequence hold its neighbour's queries: they move no reference
      float m = -INFINITY;
      F2 l2 = dup2(0.f);
      for (int j = 0; j < mine; ++j) {
        ok = warp_wait(&s_full[t], cnt++ & 1);
        tc_fence_after();
        const bool cut = j + 1 == mine && (p.causal || it.tail);
        const int seen = (p.causal ? min(qi + 1, len) : len) - j * kAttnTile - half * kCols;
        float w[kCols / 2];
        bool fresh = j == 0;  // the reference is taken from this tile
#pragma unroll 1
        while (true) {
          if (fresh) {
            // the maximum over both halves, before either is overwritten with its weights
            float next = m;
#pragma unroll 1
            for (int y = 0; y < 2; ++y) {
              float s[kCols];
              tmem_ld64(tS(t) + lb + y * kCols, s);
              tmem_wait_ld_regs(s);
              if (cut)
#pragma unroll
                for (int e = 0; e < kCols; ++e)
                  if (e + (y - half) * kCols >= seen) s[e] = -INFINITY;
              float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
              for (int e = 4; e < 60; e += 8)
#pragma unroll
                for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], s[e + u], s[e + 4 + u]);
              next = max3(next, max3(mx[0], mx[1], s[60]), max3(mx[2], mx[3], fmaxf(s[61], fmaxf(s[62], s[63]))));
            }
            if (pair_any(pair, !ok)) {
              ok = false;
              break;
            }
            const float f = next == m ? 1.f : exp2_approx((m - next) * c);
            m = next == -INFINITY ? kNone : next;
            l2 = mul2(l2, dup2(f));
            if (j > 0) {
#pragma unroll
              for (int q = 0; q < D / 64; ++q) {
                float o[32];
                tmem_ld32(lO + q * 32, o);
                tmem_wait_ld_regs(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tmem_st32(lO + q * 32, o);
              }
            }
          }
          const F2 mc = dup2(-m * c);
          F2 sum[2] = {dup2(0.f), dup2(0.f)};
          float s[kCols];
          tmem_ld64(lS, s);
          tmem_wait_ld_regs(s);
          if (cut)
#pragma unroll
            for (int e = 0; e < kCols; ++e)
              if (e >= seen) s[e] = -INFINITY;
#pragma unroll
          for (int e = 0; e < kCols / 2; ++e) {
            float a, b;
            unf2(fma2(f2(s[2 * e], s[2 * e + 1]), c2, mc), &a, &b);
            a = exp2_approx(a);
            b = exp2_approx(b);
            sum[e & 1] = add2(sum[e & 1], f2(a, b));
            w[e] = __uint_as_float(pack_bf16(a, b));
          }
          sum[0] = add2(sum[0], sum[1]);
          if (fresh || !pair_any(pair, !ok || sum2(sum[0]) > high)) {
            l2 = add2(l2, sum[0]);
            break;
          }
          if (pair_any(pair, !ok)) {
            ok = false;
            break;
          }
          fresh = true;
        }
        if (!ok) break;
        tmem_st32(lS, w);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      *own = sum2(l2);  // the other thread has read the last item's before this item's first barrier
      ok = warp_wait(&o_full[t], outs++ & 1);
      if (pair_any(pair, !ok)) break;
      tc_fence_after();
      const float l = *own + *his, r = 1.f / l;
      const size_t at = (size_t(it.tl.row0) + qi) * p.H + it.h;
      if (half == 0 && qi < len) p.lse[at] = m * p.scale + logf(l);
      float o[D / 2];
#pragma unroll
      for (int q = 0; q < D / 64; ++q) tmem_ld32(lO + q * 32, o + q * 32);
      tmem_wait_ld_regs(o);
      if (qi < len)
#pragma unroll
        for (int q = 0; q < D / 64; ++q) store_bf16x32(p.o + at * D + half * (D / 2) + q * 32, o + q * 32, r, wide);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(*tslot, 512);
}

template <int D>
static cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const AttnParams& p, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(k_attn_fwd<D>, Cfg<D>::kSmem, &done);
  if (e != cudaSuccess) return e;
  const long long items = (long long)p.tiles * p.H;
  return launch_after(k_attn_fwd<D>, dim3(unsigned(items < p.sms ? items : p.sms)), dim3(kThreads), Cfg<D>::kSmem, s, mq, mk, mv, p);
}

cudaError_t launch_attn_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int D, const AttnParams& p, cudaStream_t s) {
  return D == 128 ? launch<128>(mq, mk, mv, p, s) : launch<64>(mq, mk, mv, p, s);
}

}  // namespace gdn
