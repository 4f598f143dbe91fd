// Attention over whole sequences, forward.
//
// For every query i of a head and the keys j it sees (all of its sequence, or those up to itself):
//   s_ij = scale q_i . k_j,  o_i = sum_j e^(s_ij) v_j / sum_j e^(s_ij),  lse_i = log sum_j e^(s_ij)
// in one pass over the keys: with a running reference m (log2 units below), weights p = 2^(c s - m), their sum l and the
// weighted sum of v are kept, and o = sum / l at the end.
//
// One CTA takes 256 queries of one head as two tiles of 128. A tile's row of scores belongs to one thread (TMEM lane = row), so
// the softmax needs no shuffles. The two tiles alternate on the tensor core: while one tile's 128 threads turn scores into
// weights, the other's products run.
//   S_t = Q_t K_j^T        128 x 128 x D, operands in shared memory (128-byte swizzle, by TMA)
//   O_t += P_t V_j         128 x D x 128, P_t bf16 in TMEM over S_t's columns (the A operand), V_j read MN-major
// TMEM: S_0, S_1, O_0, O_1. Keys and values come through one ring of stages. Weights are rounded to bf16 (2^-9 relative, the
// type of v and o); scores, sums and the accumulators are fp32.
//
// The reference m is the first tile's row maximum and moves only when a later one lies more than 2^8 above it (then the
// accumulator and l are rescaled): weights up to 256 cost no precision in bf16 or fp32, and almost no tile needs the rescaling.
// It needs no wait: the commit that announces S_t(j) also covers the product O_t(j - 1) issued before it.
//
// Keys past the sequence's end are masked in the scores, and the last tile's values past it are zeroed in shared memory: they
// belong to the next sequence, and 0 x NaN would carry a neighbour's NaN over.
#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 384;  // 8 softmax warps, the MMA warp, the TMA warp and two that only give their registers
// The launch's 168 registers a thread (12 warps x 168 x 32 = 64512) are shared out anew: 208 for the softmax's rows of 128 scores,
// 88 for the rest (8 x 208 + 4 x 88 = 12 x 168).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr float kRescale = 8.f;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = kAttnTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes;
};

template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* m, int x, int y, uint64_t* bar) {
  mbar_expect_tx(bar, Cfg<D>::kTileBytes);
  load_attn_tile<D>(dst, m, x, y, bar);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_fwd(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const AttnParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = sm + 2 * C::kTileBytes;
  __shared__ uint64_t q_full[2], kv_full[C::kStages], kv_empty[C::kStages], s_full[2], p_full[2], o_full[2], tail_ready, drained;
  __shared__ uint32_t tslot;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.H, hk = h / p.group;
  wait_for_previous();
  const AttnTile tl = attn_tile(p, blockIdx.x / p.H, kAttnPair, false);
  const int all = (tl.len + kAttnTile - 1) / kAttnTile;
  int n[2];  // key tiles of either query tile; the second sees no fewer, or has no rows
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int q0 = tl.first + t * kAttnTile;
    n[t] = q0 >= tl.len ? 0 : p.causal ? q0 / kAttnTile + 1 : all;
  }
  const int most = max(n[0], n[1]), last_tile = n[1] > 0 ? 1 : 0;
  const bool tail = most * kAttnTile > tl.len;

  if (warp == 8) tmem_alloc(&tslot, 512);
  if (tid == 0) {
    abort_flag = 0;
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], kAttnTile);
      mbar_init(&o_full[t], 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&tail_ready, 32);
    mbar_init(&drained, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tslot;
  // S_t at 128 t, O_t at 256 + D t
  auto tS = [&](int t) { return tb + uint32_t(t) * 128; };
  auto tO = [&](int t) { return tb + 256 + uint32_t(t) * D; };

  if (warp >= 8) {
    regs_dec<kOtherRegs>();
    if (warp == 9) {
      // ---------------- producer: Q, then K and V tile by tile through the ring ----------------
      bool ok = true;
      if (lane == 0) {
        load_tile<D>(sm, &mq, h * D, tl.row0 + tl.first, &q_full[0]);
        if (n[1]) load_tile<D>(sm + C::kTileBytes, &mq, h * D, tl.row0 + tl.first + kAttnTile, &q_full[1]);
        for (int i = 0; i < 2 * most; ++i) {
          const int st = i % C::kStages, use = i / C::kStages;
          if (use > 0 && !mbar_wait(&kv_empty[st], (use - 1) & 1, &abort_flag, p.status, kDevTimeoutMma)) {
            // the copies in flight land before their destination is given up
            for (int k = max(0, i - C::kStages); k < i; ++k) mbar_drain(&kv_full[k % C::kStages], (k / C::kStages) & 1);
            for (int t = 0; t < 1 + last_tile; ++t) mbar_drain(&q_full[t], 0);
            ok = false;
            break;
          }
          load_tile<D>(sKV + st * C::kTileBytes, i & 1 ? &mv : &mk, hk * D, tl.row0 + (i >> 1) * kAttnTile, &kv_full[st]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (tail && ok) {
        const int i = 2 * most - 1, st = i % C::kStages;
        if (mbar_wait(&kv_full[st], (i / C::kStages) & 1, &abort_flag, p.status, kDevTimeoutTma)) {
          zero_attn_rows<D>(sKV + st * C::kTileBytes, tl.len - (most - 1) * kAttnTile, lane);
          fence_async_smem();
          mbar_arrive(&tail_ready);
        }
      }
    } else if (warp == 8) {
      // ---------------- MMA issuer ----------------
      if (lane == 0) {
        constexpr uint32_t idS = idesc_bf16(128, 128), idO = idesc_bf16(128, D, false, true);
        const uint32_t sQ = smem_u32(sm), kv = smem_u32(sKV);
        auto full = [&](int i) { return mbar_wait(&kv_full[i % C::kStages], (i / C::kStages) & 1, &abort_flag, p.status, kDevTimeoutTma); };
        auto tile = [&](int i) { return kv + uint32_t(i % C::kStages) * C::kTileBytes; };
        auto scores = [&](int t, int j) {
          const uint32_t a = sQ + t * C::kTileBytes, b = tile(2 * j);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) mma_bf16_ss(tS(t), desc_kmajor(a, kAttnPanel, s), desc_kmajor(b, kAttnPanel, s), idS, s > 0);
          mma_commit(&s_full[t]);
          if (t == last_tile) mma_commit(&kv_empty[(2 * j) % C::kStages]);
        };
        auto outputs = [&](int t, int j) {
          const uint32_t b = tile(2 * j + 1);
#pragma unroll
          for (int s = 0; s < kAttnTile / 16; ++s) mma_bf16_ts(tO(t), tS(t) + s * 8, desc_mnmajor_bf16(b, kAttnPanel, s), idO, j > 0 || s > 0);
          if (t == last_tile) mma_commit(&kv_empty[(2 * j + 1) % C::kStages]);
          if (j + 1 == n[t]) mma_commit(&o_full[t]);
        };
        bool ok = full(0);
        for (int t = 0; t < 2 && ok; ++t)
          if (n[t]) {
            ok = mbar_wait(&q_full[t], 0, &abort_flag, p.status, kDevTimeoutTma);
            if (ok) scores(t, 0);
          }
        for (int j = 0; j < most && ok; ++j) {
          ok = full(2 * j + 1);
          if (ok && tail && j + 1 == most) ok = mbar_wait(&tail_ready, 0, &abort_flag, p.status, kDevTimeoutSync);
          for (int t = 0; t < 2 && ok; ++t) {
            if (j >= n[t]) continue;
            if (!mbar_wait(&p_full[t], j & 1, &abort_flag, p.status, kDevTimeoutSync)) {
              ok = false;
              break;
            }
            tc_fence_after();
            outputs(t, j);
            if (j + 1 < n[t]) {
              if (!full(2 * j + 2)) {
                ok = false;
                break;
              }
              scores(t, j + 1);
            }
          }
        }
        if (!ok) {  // the products in flight end before their accumulators are given up
          mma_commit(&drained);
          mbar_drain(&drained, 0);
        }
      }
    }
  } else {
    // ---------------- softmax: one query row a thread ----------------
    regs_inc<kSoftmaxRegs>();
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lb = tmem_lane_base(warp);
    const int qi = tl.first + t * kAttnTile + row;  // in the sequence
    const float c = p.scale * kLog2e, far = kRescale / c;
    const F2 c2 = dup2(c);
    float m = -INFINITY;
    F2 l2 = dup2(0.f);
    bool ok = true;
    for (int j = 0; j < n[t]; ++j) {
      if (!mbar_wait(&s_full[t], j & 1, &abort_flag, p.status, kDevTimeoutMma)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[128];
      tmem_ld64(tS(t) + lb, s);
      tmem_ld64(tS(t) + lb + 64, s + 64);
      tmem_wait_ld_regs(s);
      const int k0 = j * kAttnTile;
      if (k0 + kAttnTile > tl.len || (p.causal && k0 + kAttnTile > tl.first + t * kAttnTile)) {
        const int seen = (p.causal ? min(qi + 1, tl.len) : tl.len) - k0;
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (e >= seen) s[e] = -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int e = 4; e < 128; e += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) mx[u] = e + 4 + u < 128 ? fmaxf(fmaxf(mx[u], s[e + u]), s[e + 4 + u]) : fmaxf(mx[u], s[e + u]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (j == 0) {
        m = top;
      } else if (__any_sync(0xffffffffu, top > m + far)) {
        const float next = fmaxf(m, top), f = next == -INFINITY ? 1.f : exp2_approx((m - next) * c);
        m = next;
        l2 = mul2(l2, dup2(f));
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          float o[32];
          tmem_ld32(tO(t) + lb + q * 32, o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          tmem_st32(tO(t) + lb + q * 32, o);
        }
      }
      const F2 mc = dup2(-m * c);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a, b;
          unf2(fma2(f2(s[q * 32 + 2 * e], s[q * 32 + 2 * e + 1]), c2, mc), &a, &b);
          a = exp2_approx(a);
          b = exp2_approx(b);
          l2 = add2(l2, f2(a, b));
          w[e] = __uint_as_float(pack_bf16(a, b));
        }
        tmem_st16(tS(t) + lb + q * 16, w);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[t]);
    }
    if (ok && n[t] && mbar_wait(&o_full[t], 0, &abort_flag, p.status, kDevTimeoutMma)) {
      tc_fence_after();
      const float l = sum2(l2), r = 1.f / l;
      const bool mine = qi < tl.len;
      const size_t at = (size_t(tl.row0) + qi) * p.H + h;
      if (mine) p.lse[at] = m * p.scale + logf(l);
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        tmem_ld32(tO(t) + lb + q * 32, o);
        tmem_wait_ld_regs(o);
        if (mine)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* x = o + 8 * e;
            *reinterpret_cast<uint4*>(p.o + at * D + q * 32 + 8 * e) =
                make_uint4(pack_bf16(x[0] * r, x[1] * r), pack_bf16(x[2] * r, x[3] * r), pack_bf16(x[4] * r, x[5] * r), pack_bf16(x[6] * r, x[7] * r));
          }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tb, 512);
}

template <int D>
static cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const AttnParams& p, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(k_attn_fwd<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(k_attn_fwd<D>, dim3(p.tiles * p.H), dim3(kThreads), Cfg<D>::kSmem, s, mq, mk, mv, p);
}

cudaError_t launch_attn_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int D, const AttnParams& p, cudaStream_t s) {
  return D == 128 ? launch<128>(mq, mk, mv, p, s) : launch<64>(mq, mk, mv, p, s);
}

}  // namespace gdn
