// Attention over whole sequences, backward. With p_ij = e^(s_ij - lse_i) recomputed from q, k and the forward's lse:
//   dP = dO v^T,  D_i = sum_c dO_ic o_ic (= sum_j p_ij dP_ij),  dS = p (dP - D)
//   dv_j = sum_i p_ij dO_i,   dk_j = scale sum_i dS_ij q_i,   dq_i = scale sum_j dS_ij k_j
// summed over the query heads of a key head for dk and dv.
//
// Three kernels. k_attn_delta leaves D and lse log2(e) by head. k_attn_dkv owns 128 keys of a key head and walks the query tiles
// (and the group's heads) that see them; k_attn_dq owns 128 queries and walks the key tiles they see. Each output is
// summed in registers of one CTA's tensor core in a fixed order, so nothing is added atomically and results do not depend on
// the order of blocks; the price is that both recompute s and dP: seven products of 128 x 128 x D a tile pair, where adding dq up in
// memory would need five.
//
// k_attn_dkv works on transposed scores, keys on the TMEM lanes, so that P^T and dS^T are TMEM-resident A operands:
//   S^T = K Q^T, dP^T = V dO^T  (shared-memory operands, K-major)
//   dV += P^T dO, dK += dS^T Q  (the same Q and dO tiles read MN-major)
// TMEM: S^T (P^T over it), dP^T (dS^T over it), dV, dK. The products run in the order dV(i), S(i+1), dK(i), dP(i+1): while a pair of
// them runs, the softmax warps turn the scores (or dP) of the other pair's into the next operand.
// k_attn_dq: S = Q K^T, dP = dO V^T, dQ += dS K (dS over S in TMEM; S double-buffered, a tile ahead).
//
// Eight softmax warps, two to a quarter of the TMEM lanes, each on half of a tile's columns. The bf16 operand's halves lie over the
// columns that their own writers have read. p and dS are rounded to bf16 (as the products' operands); all sums are fp32.
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

// 32 columns of an accumulator row times f, as bf16.
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, uint32_t t, float f, bool mine, bool wide) {
  float o[32];
  tmem_ld32(t, o);
  tmem_wait_ld_regs(o);
  if (mine) store_bf16x32(dst, o, f, wide);
}

// Ring position and phase of use i.
__device__ __forceinline__ int slot(int i, int n) { return i % n; }
__device__ __forceinline__ uint32_t phase(int i, int n) { return uint32_t(i / n) & 1u; }

}  // namespace

// -D_i and -lse_i log2(e) of 32 rows of a head a warp.
template <int D>
__global__ void __launch_bounds__(256) k_attn_delta(const AttnParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, which = lane / kLanes;
  const long long chunks = (p.rows + 31) / 32, item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  wait_for_previous();
  if (item >= chunks * p.H) return;
  const int h = int(item % p.H);
  const long long row0 = item / p.H * 32;
  float mine = 0.f;
#pragma unroll 4
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
               const __grid_constant__ CUtensorMap mdo, const AttnParams p) {
  constexpr int kTile = Cfg<D>::kTile, kQ = 3, kO = 2;  // stages of Q and of dO (a Q tile is needed longer)
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t *sK = sm, *sV = sK + kTile, *sQ = sV + kTile, *sO = sQ + kQ * kTile;
  float* vec = reinterpret_cast<float*>(sO + kO * kTile);  // [2][lse2 | delta][128]
  uint64_t* bar = reinterpret_cast<uint64_t*>(vec + 2 * 256);
  uint64_t *kv_full = bar, *q_full = bar + 1, *q_empty = bar + 4, *o_full = bar + 7, *o_empty = bar + 9, *ready = bar + 11, *vec_free = bar + 13, *s_full = bar + 15,
           *dp_full = bar + 16, *p_ready = bar + 17, *ds_ready = bar + 18, *done = bar + 19;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 20);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + 21);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x % p.Hk;
  wait_for_previous();
  const AttnTile tl = attn_tile(p, blockIdx.x / p.Hk, kAttnTile, p.causal != 0);
  const int all = (tl.len + kAttnTile - 1) / kAttnTile, i0 = p.causal ? tl.first / kAttnTile : 0, per = all - i0, n = per * p.group;
  const bool ragged = all * kAttnTile > tl.len;

  if (warp == kMma) tmem_alloc(tslot, 512);
  if (tid == 0) {
    *abort_flag = 0;
    mbar_init(kv_full, 1);
    for (int i = 0; i < kQ; ++i) mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], 1);
    for (int i = 0; i < kO; ++i) mbar_init(&o_full[i], 1), mbar_init(&o_empty[i], 1), mbar_init(&ready[i], 32), mbar_init(&vec_free[i], kSoftmax);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, kSoftmax + 1);
    mbar_init(ds_ready, kSoftmax + 1);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tS = 0, tP = 128, tV = 256, tK = 256 + D;  // all of TMEM, so it starts at column 0

  if (warp >= kMma) {
    regs_dec<kOtherRegs>();
    if (warp == kTma) {
      // ---------------- producer ----------------
      if (lane == 0) {
        mbar_expect_tx(kv_full, 2 * kTile);
        load_attn_tile<D>(sK, &mk, hk * D, tl.row0 + tl.first, kv_full);
        load_attn_tile<D>(sV, &mv, hk * D, tl.row0 + tl.first, kv_full);
      }
      int it = 0;
      bool ok = true;
      for (; it < n; ++it) {
        const int h = hk * p.group + it / per, q0 = (i0 + it % per) * kAttnTile, y = tl.row0 + q0, qs = slot(it, kQ), os = slot(it, kO);
        if (it >= kQ) ok = attn_wait(&q_empty[qs], phase(it - kQ, kQ), abort_flag, p.status, kDevTimeoutMma);
        if (ok && lane == 0) {
          mbar_expect_tx(&q_full[qs], kTile);
          load_attn_tile<D>(sQ + qs * kTile, &mq, h * D, y, &q_full[qs]);
        }
        if (ok && it >= kO)
          ok = attn_wait(&o_empty[os], phase(it - kO, kO), abort_flag, p.status, kDevTimeoutMma) &&
               attn_wait(&vec_free[os], phase(it - kO, kO), abort_flag, p.status, kDevTimeoutSync);
        if (ok && lane == 0) {
          mbar_expect_tx(&o_full[os], kTile);
          load_attn_tile<D>(sO + os * kTile, &mdo, h * D, y, &o_full[os]);
        }
        if (!__all_sync(0xffffffffu, ok)) break;
        float* v = vec + os * 256;
        const long long at = (long long)h * p.rows + y;
#pragma unroll
        for (int e = lane; e < kAttnTile; e += 32) {
          const bool in = q0 + e < tl.len;
          v[e] = in ? p.lse2[at + e] : -INFINITY;
          v[128 + e] = in ? p.delta[at + e] : 0.f;
        }
        if (ragged && q0 + kAttnTile > tl.len) {
          ok = attn_wait(&q_full[qs], phase(it, kQ), abort_flag, p.status, kDevTimeoutTma) &&
               attn_wait(&o_full[os], phase(it, kO), abort_flag, p.status, kDevTimeoutTma);
          if (!__all_sync(0xffffffffu, ok)) break;
          zero_attn_rows<D>(sQ + qs * kTile, tl.len - q0, lane);
          zero_attn_rows<D>(sO + os * kTile, tl.len - q0, lane);
          fence_async_smem();
        }
        mbar_arrive(&ready[os]);
      }
      if (it < n && lane == 0) {  // the copies in flight land before their destination is given up
        mbar_drain(kv_full, 0);
        for (int k = max(0, it - kQ + 1); k < it; ++k) mbar_drain(&q_full[slot(k, kQ)], phase(k, kQ));
        for (int k = max(0, it - kO + 1); k < it; ++k) mbar_drain(&o_full[slot(k, kO)], phase(k, kO));
        // the last ones, if they were requested
        mbar_drain(&q_full[slot(it, kQ)], phase(it, kQ), 1000000ull);
        mbar_drain(&o_full[slot(it, kO)], phase(it, kO), 1000000ull);
      }
    } else if (warp == kMma) {
      // ---------------- MMA issuer ----------------
      const uint32_t lead = elect_lead();
      const uint32_t aK = desc_low_k(smem_u32(sK)), aV = desc_low_k(smem_u32(sV)), bQ = desc_low_k(smem_u32(sQ)), bO = desc_low_k(smem_u32(sO)),
                     nQ = desc_low_mn(smem_u32(sQ), kAttnPanel), nO = desc_low_mn(smem_u32(sO), kAttnPanel);
      auto wait = [&](uint64_t* b, uint32_t ph, int code) { return bool(__all_sync(0xffffffffu, attn_wait(b, ph, abort_flag, p.status, code))); };
      auto scores = [&](int at) {
        product_ss<D>(lead, tS, aK, bQ + at * (kTile >> 4));
        commit(lead, s_full);
      };
      auto dprobs = [&](int at) {
        product_ss<D>(lead, tP, aV, bO + at * (kTile >> 4));
        commit(lead, dp_full);
      };
      Ring<kQ, 1> rq(0);
      bool ok = wait(kv_full, 0, kDevTimeoutTma) && wait(&q_full[0], 0, kDevTimeoutTma) && wait(&ready[0], 0, kDevTimeoutSync);
      if (ok) scores(0);
      ok = ok && wait(&o_full[0], 0, kDevTimeoutTma);
      if (ok) dprobs(0);
      for (int it = 0; it < n && ok; ++it) {
        // the gates answer for the tiles of the products that follow either operand
        if (!(ok = wait(p_ready, it & 1, kDevTimeoutSync))) break;
        tc_fence_after();
        const int qs = rq.at, os = it & 1;
        rq.next();
        product_ts<D, kCols / 2, 0, kAttnTile / 16>(lead, tV, tS, nO + os * (kTile >> 4), it > 0);
        commit(lead, &o_empty[os]);
        if (it + 1 < n) scores(rq.at);
        if (!(ok = wait(ds_ready, it & 1, kDevTimeoutSync))) break;
        tc_fence_after();
        product_ts<D, kCols / 2, 0, kAttnTile / 16>(lead, tK, tP, nQ + qs * (kTile >> 4), it > 0);
        commit(lead, &q_empty[qs]);
        if (it + 1 < n) dprobs(os ^ 1);
      }
      commit(lead, done);  // the softmax warps wait for it, or, after an error:
      if (!ok) mbar_drain(done, 0);
    } else if (warp >= kGate && lane == 0) {
      // ---------------- gates: one warp for S(it + 1) behind dV(it), the other for dP(it + 1) behind dK(it) ----------------
      uint64_t* bar = warp == kGate ? p_ready : ds_ready;
      Ring<kQ, 1> rq(0);
      bool ok = true;
      for (int it = 0; it < n && ok; ++it) {
        rq.next();
        if (it + 1 < n) {
          const int os = (it + 1) & 1;
          const uint32_t ph = phase(it + 1, kO);
          ok = warp == kGate ? attn_wait(&q_full[rq.at], rq.phase, abort_flag, p.status, kDevTimeoutTma) && attn_wait(&ready[os], ph, abort_flag, p.status, kDevTimeoutSync)
                          : attn_wait(&o_full[os], ph, abort_flag, p.status, kDevTimeoutTma);
          if (!ok) break;
        }
        mbar_arrive(bar);
        ok = attn_wait(bar, it & 1, abort_flag, p.status, kDevTimeoutSync);  // the next arrival belongs to the next phase
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
    bool ok = true;
    for (int it = 0; it < n && ok; ++it) {
      const int q0 = (i0 + it % per) * kAttnTile + half * kCols, os = it & 1;
      const float2 *lse = reinterpret_cast<const float2*>(vec + os * 256 + half * kCols + col), *delta = lse + 64;
      ok = attn_wait(&ready[os], phase(it, kO), abort_flag, p.status, kDevTimeoutSync) && attn_wait(s_full, it & 1, abort_flag, p.status, kDevTimeoutMma);
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
      ok = attn_wait(dp_full, it & 1, abort_flag, p.status, kDevTimeoutMma);
      if (!ok) break;
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
#pragma unroll
      for (int e = 0; e < 32; ++e) out[e] = pack_bf16(d[2 * e], d[2 * e + 1]);
      tmem_st_16x32(tP + lb, out);
      tmem_st_16x32(tP + lb + (16u << 16), out + 16);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(ds_ready);
    }
    if (ok && attn_wait(done, 0, abort_flag, p.status, kDevTimeoutMma)) {
      tc_fence_after();
      const int key = tl.first + (tid & 127);
      const bool wide = (reinterpret_cast<uintptr_t>(half ? p.dk : p.dv) & 31) == 0;
      __nv_bfloat16* dst = (half ? p.dk : p.dv) + ((size_t(tl.row0) + key) * p.Hk + hk) * D;
      const uint32_t acc = (half ? tK : tV) + lane0;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) store_row(dst + q * 32, acc + q * 32, half ? p.scale : 1.f, key < tl.len, wide);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(*tslot, 512);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_dq(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
              const __grid_constant__ CUtensorMap mdo, const AttnParams p) {
  constexpr int kTile = Cfg<D>::kTile, kK = 3, kV = 2;  // stages of K (needed longer) and V
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t *sQ = sm, *sO = sQ + kTile, *sK = sO + kTile, *sV = sK + kK * kTile;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sV + kV * kTile);
  uint64_t *q_full = bar, *k_full = bar + 1, *k_empty = bar + 4, *v_full = bar + 7, *v_empty = bar + 9, *s_full = bar + 11, *dp_full = bar + 13, *ds_ready = bar + 14,
           *tail_ready = bar + 15, *done = bar + 16;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 17);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + 18);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.H, hk = h / p.group;
  wait_for_previous();
  const AttnTile tl = attn_tile(p, blockIdx.x / p.H, kAttnTile, false);
  const int all = (tl.len + kAttnTile - 1) / kAttnTile, n = p.causal ? tl.first / kAttnTile + 1 : all;
  const bool tail = n * kAttnTile > tl.len;

  if (warp == kMma) tmem_alloc(tslot, 512);
  if (tid == 0) {
    *abort_flag = 0;
    mbar_init(q_full, 1);
    for (int i = 0; i < kK; ++i) mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
    for (int i = 0; i < kV; ++i) mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 1), mbar_init(&s_full[i], 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_ready, kSoftmax + 1);
    mbar_init(tail_ready, 32);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tP = 256, tQ = 384;  // all of TMEM, so it starts at column 0
  auto tS = [&](int i) { return uint32_t(i & 1) * 128; };

  if (warp >= kMma) {
    regs_dec<kOtherRegs>();
    if (warp == kTma) {
      // ---------------- producer ----------------
      int it = 0;
      if (lane == 0) {
        mbar_expect_tx(q_full, 2 * kTile);
        load_attn_tile<D>(sQ, &mq, h * D, tl.row0 + tl.first, q_full);
        load_attn_tile<D>(sO, &mdo, h * D, tl.row0 + tl.first, q_full);
        for (; it < n; ++it) {
          const int ks = slot(it, kK), vs = slot(it, kV), y = tl.row0 + it * kAttnTile;
          if (it >= kK && !attn_wait(&k_empty[ks], phase(it - kK, kK), abort_flag, p.status, kDevTimeoutMma)) break;
          mbar_expect_tx(&k_full[ks], kTile);
          load_attn_tile<D>(sK + ks * kTile, &mk, hk * D, y, &k_full[ks]);
          if (it >= kV && !attn_wait(&v_empty[vs], phase(it - kV, kV), abort_flag, p.status, kDevTimeoutMma)) {
            mbar_drain(&k_full[ks], phase(it, kK));
            break;
          }
          mbar_expect_tx(&v_full[vs], kTile);
          load_attn_tile<D>(sV + vs * kTile, &mv, hk * D, y, &v_full[vs]);
        }
        if (it < n) {  // the copies in flight land before their destination is given up
          mbar_drain(q_full, 0);
          for (int k = max(0, it - kK); k < it; ++k) mbar_drain(&k_full[slot(k, kK)], phase(k, kK));
          for (int k = max(0, it - kV); k < it; ++k) mbar_drain(&v_full[slot(k, kV)], phase(k, kV));
        }
      }
      it = __shfl_sync(0xffffffffu, it, 0);
      if (tail && it == n && attn_wait(&k_full[slot(n - 1, kK)], phase(n - 1, kK), abort_flag, p.status, kDevTimeoutTma)) {
        zero_attn_rows<D>(sK + slot(n - 1, kK) * kTile, tl.len - (n - 1) * kAttnTile, lane);
        fence_async_smem();
        mbar_arrive(tail_ready);
      }
    } else if (warp == kMma) {
      // ---------------- MMA issuer ----------------
      const uint32_t lead = elect_lead();
      const uint32_t aQ = desc_low_k(smem_u32(sQ)), aO = desc_low_k(smem_u32(sO)), bK = desc_low_k(smem_u32(sK)), bV = desc_low_k(smem_u32(sV)),
                     nK = desc_low_mn(smem_u32(sK), kAttnPanel);
      auto wait = [&](uint64_t* b, uint32_t ph, int code) { return bool(__all_sync(0xffffffffu, attn_wait(b, ph, abort_flag, p.status, code))); };
      Ring<kK, 1> rs(0), rk(0);  // K of the scores, and of dq
      auto scores = [&](int i) {
        product_ss<D>(lead, tS(i), aQ, bK + rs.at * (kTile >> 4));
        commit(lead, &s_full[i & 1]);
        rs.next();
      };
      auto dprobs = [&](int i) {
        product_ss<D>(lead, tP, aO, bV + (i & 1) * (kTile >> 4));
        commit(lead, dp_full);
        commit(lead, &v_empty[i & 1]);
      };
      auto k_there = [&](int i) {
        return wait(&k_full[slot(i, kK)], phase(i, kK), kDevTimeoutTma) && (!tail || i + 1 < n || wait(tail_ready, 0, kDevTimeoutSync));
      };
      bool ok = wait(q_full, 0, kDevTimeoutTma) && k_there(0);
      if (ok) scores(0);
      ok = ok && wait(&v_full[0], 0, kDevTimeoutTma);
      if (ok) dprobs(0);
      if (n > 1 && ok && (ok = k_there(1))) scores(1);
      for (int i = 0; i < n && ok; ++i) {
        // the gate answers for V of the next tile
        if (!(ok = wait(ds_ready, i & 1, kDevTimeoutSync))) break;
        tc_fence_after();
        if (i + 1 < n) dprobs(i + 1);
        product_ts<D, kCols / 2, 0, kAttnTile / 16>(lead, tQ, tS(i), nK + rk.at * (kTile >> 4), i > 0);
        commit(lead, &k_empty[rk.at]);
        rk.next();
        // K of the tile after next is requested when the product before this one has let go of its stage
        if (i + 2 < n && (ok = k_there(i + 2))) scores(i + 2);
      }
      commit(lead, done);  // the softmax warps wait for it, or, after an error:
      if (!ok) mbar_drain(done, 0);
    } else if (warp == kGate && lane == 0) {
      // ---------------- gate: V of the product that follows dS(i) has landed ----------------
      auto wait = [&](uint64_t* b, uint32_t ph, int code) { return attn_wait(b, ph, abort_flag, p.status, code); };
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        if (i + 1 < n && !(ok = wait(&v_full[(i + 1) & 1], phase(i + 1, kV), kDevTimeoutTma))) break;
        mbar_arrive(ds_ready);
        ok = wait(ds_ready, i & 1, kDevTimeoutSync);  // the next arrival belongs to the next phase
      }
    }
  } else {
    // ---------------- softmax: query row, half of the keys ----------------
    regs_inc<kSoftmaxRegs>();
    const int half = warp >> 2, row = tid & 127, qi = tl.first + row;
    const uint32_t lane0 = tmem_lane_base(warp), lb = lane0 + uint32_t(half) * kCols;
    const bool mine = qi < tl.len;
    const long long at = (long long)h * p.rows + tl.row0 + qi;
    const F2 c2 = dup2(p.scale * kLog2e), lse = dup2(mine ? p.lse2[at] : 0.f), delta = dup2(mine ? p.delta[at] : 0.f);
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      ok = attn_wait(&s_full[i & 1], (i >> 1) & 1, abort_flag, p.status, kDevTimeoutMma);
      if (!ok) break;
      tc_fence_after();
      float w[kCols], d[kCols];
      tmem_ld64(tS(i) + lb, w);
      tmem_wait_ld_regs(w);
#pragma unroll
      for (int e = 0; e < kCols / 2; ++e) {
        float a, b;
        unf2(fma2(f2(w[2 * e], w[2 * e + 1]), c2, lse), &a, &b);
        w[2 * e] = exp2_approx(a);
        w[2 * e + 1] = exp2_approx(b);
      }
      ok = attn_wait(dp_full, i & 1, abort_flag, p.status, kDevTimeoutMma);
      if (!ok) break;
      tc_fence_after();
      tmem_ld64(tP + lb, d);
      tmem_wait_ld_regs(d);
#pragma unroll
      for (int e = 0; e < kCols / 2; ++e) unf2(mul2(f2(w[2 * e], w[2 * e + 1]), add2(f2(d[2 * e], d[2 * e + 1]), delta)), &d[2 * e], &d[2 * e + 1]);
      if (i + 1 == n && (p.causal || tail)) {
        const int seen = (p.causal ? min(qi + 1, tl.len) : tl.len) - i * kAttnTile - half * kCols;
#pragma unroll
        for (int e = 0; e < kCols; ++e)
          if (e >= seen) d[e] = 0.f;
      }
      store_operand(tS(i) + lb, d);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(ds_ready);
    }
    if (ok && attn_wait(done, 0, abort_flag, p.status, kDevTimeoutMma)) {
      tc_fence_after();
      const bool wide = (reinterpret_cast<uintptr_t>(p.dq) & 31) == 0;
      __nv_bfloat16* dst = p.dq + ((size_t(tl.row0) + qi) * p.H + h) * D + half * (D / 2);
#pragma unroll
      for (int q = 0; q < D / 64; ++q) store_row(dst + q * 32, tQ + lane0 + half * (D / 2) + q * 32, p.scale, mine, wide);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(*tslot, 512);
}

template <int D>
static cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo, const AttnParams& p, const int* keys, cudaStream_t s) {
  constexpr int kSmem = Cfg<D>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(k_attn_dkv<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_attn_dq<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const long long items = (p.rows + 31) / 32 * p.H;
  e = launch_after(k_attn_delta<D>, dim3(unsigned((items + 7) / 8)), dim3(256), 0, s, p);
  if (e != cudaSuccess) return e;
  AttnParams pk = p;
  pk.table = keys;
  e = launch_after(k_attn_dkv<D>, dim3(unsigned(p.tiles * p.Hk)), dim3(kThreads), kSmem, s, mq, mk, mv, mdo, pk);
  if (e != cudaSuccess) return e;
  return launch_after(k_attn_dq<D>, dim3(unsigned(p.tiles * p.H)), dim3(kThreads), kSmem, s, mq, mk, mv, mdo, p);
}

cudaError_t launch_attn_bwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo, int D, const AttnParams& p, const int* keys,
                            cudaStream_t s) {
  return D == 128 ? launch<128>(mq, mk, mv, mdo, p, keys, s) : launch<64>(mq, mk, mv, mdo, p, keys, s);
}

}  // namespace gdn
