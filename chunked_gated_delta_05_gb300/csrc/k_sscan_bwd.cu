// Selective scan, backward. With dy0 = dy silu(z) and a_t = exp(dt_t A), over tokens in reverse,
//   dh_t = C_t dy0_t + a_{t+1} dh_{t+1},
//   dC_t = sum_d dy0 h_t,  dB_t = sum_d dh_t dt u,  du = dt (B . dh) + D dy0,
//   w = dh_t a_t h_{t-1},  dA = sum_t w dt,  ddt = u (B . dh) + A . w,  ddelta = ddt sigmoid(delta + bias),
//   dz = dy (C . h + D u) silu'(z),  dD = sum_t dy0 u,  dh0 = a_1 dh_1.
//
// Two lanes walk one channel. The states they need in reverse come from those a training forward keeps before every 8th
// token (8 bytes a token and channel): each tile of 8, last to first, is run forward again and then walked back. Keeping
// fewer costs another forward walk, which this kernel, bound by its instructions at 15% of HBM's rate, cannot hide as it
// does the reads. The adjoint chain is cut into segments like the forward's. The sums over channels in dB and dC begin as
// matrix products with ones: a lane's four states are its share of the A operand of m16n8k8, whose products add up four
// lanes' channels (each term as two tf32 operands, 22 bits of it), and three exchanges add up the groups of lanes. All sums are
// fp32; dB and dC are rounded to bf16 once.
//
// On GB300, 4093 tokens in 7 documents x 2048 channels x 16 states: 241 us (adjoint maps 37, composition 8, this walk
// 190, last sums 8 warm), of which the second operand of every term takes 29 (14% of the backward; without it dB and dC shrink by
// 3.5e-4, and by 5% of their value where channels cancel to 1%). 168 registers leave three warps a scheduler. Tried before that
// operand, when the backward took 212 us: exchanges between the two lanes in place of their sums' trip through shared memory, 226;
// adding up the lane groups at the tile's end in place of the exchanges, 222. The rest of the terms as bf16, two to a register
// (six products a token in place of eight): 241 as well; selectors of their own for dC and dB: 256.
#include <atomic>

#include "k_sscan.cuh"

namespace gdn {
namespace {

constexpr int kRGroup = 4;
constexpr int kRt = 16;  // tokens the adjoint map stages together, double-buffered

template <int NP>
struct RmapSmem {
  BcTile<NP, kRt> C[2];
  ChTile<kRt> delta[2], dy[2], z[2];
};

// The adjoint map of a segment: from a zero exit gradient to the gradient of the state before its first token. Two channels
// a thread, as in the forward.
template <int NP>
__global__ void __launch_bounds__(kSscanThreads, 7) k_sscan_rmap(SscanParams p, int blocks) {
  extern __shared__ __align__(16) char smem_raw[];
  RmapSmem<NP>& sm = *reinterpret_cast<RmapSmem<NP>*>(smem_raw);
  wait_for_previous();
  const int seg = blockIdx.x / blocks;
  const SscanSeg sg = sscan_seg(p, seg);
  if (sg.j == 0) return;
  const SscanChan ch = sscan_chan(p, blockIdx.x % blocks);
  F2 A2[2][NP / 2], g[2][NP / 2];
  const F2 bias = f2(param(p.bias, ch.d[0]), param(p.bias, ch.d[1]));
  F2 dt_sum = f2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    load_A2<NP>(A2[e], p, ch.d[e]);
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) g[e][i] = f2(0.f, 0.f);
  }
  const bool gate = p.z != nullptr, softplus_on = p.softplus;
  BcRegs<NP, kRt> rc;
  auto request = [&](int tb, int buf) {
    const long long row = sg.row0 + tb;
    const int len = sg.len - tb;
    sm.delta[buf].load(p.delta + row * p.dt_s + ch.d0, p.dt_s, len, ch.chans, p.vec);
    sm.dy[buf].load(p.dy + row * p.D + ch.d0, p.D, len, ch.chans, p.vec);
    if (gate) sm.z[buf].load(p.z + row * p.z_s + ch.d0, p.z_s, len, ch.chans, p.vec);
    copies_commit();
    rc.load(p.Cm + row * p.c_s + ch.g * p.N, p.c_s, len, p.N);
  };
  const int last = (sg.len - 1) / kRt * kRt;
  request(last, 0);
  rc.store(sm.C[0]);
  for (int tb = last, buf = 0; tb >= 0; tb -= kRt, buf ^= 1) {
    copies_wait();
    __syncthreads();
    if (tb > 0) request(tb - kRt, buf ^ 1);
    const int len = min(kRt, sg.len - tb);
    // as in the forward: tokens in groups, no branch in a token's work; past the segment's end dt and dy are 0
#pragma unroll 1
    for (int t0 = (len - 1) / kRGroup * kRGroup; t0 >= 0; t0 -= kRGroup) {
      float dt[kRGroup][2], dy0[kRGroup][2];
#pragma unroll
      for (int i = 0; i < kRGroup; ++i) {
        const F2 x = add2(sm.delta[buf].pair(t0 + i), bias), sp = softplus2(x), dy = sm.dy[buf].pair(t0 + i);
        const F2 gated = mul2(dy, silu2(sm.z[buf].pair(t0 + i)));
        const bool in = t0 + i < len;
        unf2(softplus_on ? sp : x, &dt[i][0], &dt[i][1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) dt[i][e] = in ? dt[i][e] : 0.f;
        dt_sum = add2(dt_sum, f2(dt[i][0], dt[i][1]));
        unf2(gate ? gated : dy, &dy0[i][0], &dy0[i][1]);
      }
#pragma unroll
      for (int i = kRGroup - 1; i >= 0; --i) {
        const F2 dt2[2] = {dup2(dt[i][0]), dup2(dt[i][1])}, dy2[2] = {dup2(dy0[i][0]), dup2(dy0[i][1])};
#pragma unroll
        for (int s = 0; s < NP / 2; s += 2) {
          F2 c[2];
          sm.C[buf].quad(c, t0 + i, s / 2);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) g[e][s + k] = mul2(decay2(dt2[e], A2[e][s + k]), fma2(c[k], dy2[e], g[e][s + k]));
        }
      }
    }
    if (tb > 0) rc.store(sm.C[buf ^ 1]);
  }
  store_rows<NP>(g, p.seg_state + (size_t)seg * p.N * p.D, p, ch);
  float dts[2];
  unf2(dt_sum, &dts[0], &dts[1]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (!ch.live[e]) continue;
    p.seg_dt[(size_t)seg * p.D + ch.d[e]] = dts[e];
  }
}

// One thread per (sequence, state, channel): from the sequence's end, each segment's exit gradient.
__global__ void __launch_bounds__(256) k_sscan_rcompose(SscanParams p) {
  const long long per = (long long)p.N * p.D, at = (long long)blockIdx.x * 256 + threadIdx.x;
  if (at >= per * p.seqs) return;
  const int seq = int(at / per), nd = int(at - seq * per), n = nd / p.D, d = nd - n * p.D;
  const int s0 = p.cu ? p.seg_base[seq] : seq * p.nseg_dense, s1 = p.cu ? p.seg_base[seq + 1] : s0 + p.nseg_dense;
  const float a2 = kLog2e * p.A[(size_t)d * p.N + n];
  wait_for_previous();
  float carry = p.dfinal ? p.dfinal[((size_t)seq * p.D + d) * p.N + n] : 0.f;
  constexpr int kAhead = 8;
  for (int s = s1 - 1; s >= s0; s -= kAhead) {
    float f[kAhead], t[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s - i > s0) {
        f[i] = p.seg_state[(size_t)(s - i) * per + nd];
        t[i] = p.seg_dt[(size_t)(s - i) * p.D + d];
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s - i >= s0) {
        p.seg_state[(size_t)(s - i) * per + nd] = carry;
        if (s - i > s0) carry = fmaf(decay(t[i], a2), carry, f[i]);
      }
  }
}

// D = A B + C for one m16n8k8 product: this lane holds A's rows lane / 4 and lane / 4 + 8 at k = lane % 4 (a0, a1) and
// k = lane % 4 + 4 (a2, a3), and B's column lane / 4 at the same two k.
__device__ __forceinline__ void mma_tf32(float* d, float a0, float a1, float a2, float a3, float b0, float b1, const float* c) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
        "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// The upper 11 significant bits of x, which tf32 holds exactly: the operands above are to be tf32 values.
__device__ __forceinline__ float tf32_part(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

// One value for two lanes: the lane with `up` keeps b, the other a, each plus the other lane's.
__device__ __forceinline__ float exchange(float a, float b, bool up, int mask) {
  return (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, mask);
}

// ------------------------------------------------------------------ two lanes a channel, states in pairs

constexpr int kBwdChans = kSscanBwdChans, kBwdThreads = 2 * kBwdChans, kWarps = kBwdThreads / 32;
constexpr int kTile = kSscanBlock, kHalf = kTile / 2;

// A tile of tokens of B or C as fp32, [token][NP], filled by kBwdChans threads.
template <int NP>
struct VecTile {
  static constexpr int kPer = (kTile * NP + kBwdChans - 1) / kBwdChans;
  struct Raw {
    uint16_t r[kPer];
  };
  float v[kTile][NP];
  __device__ __forceinline__ static Raw fetch(const __nv_bfloat16* src, long long row, int len, int N, int tid) {
    Raw x;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = tid + j * kBwdChans, t = e / NP, n = e % NP;
      x.r[j] = t < len && t < kTile && n < N ? __ldg(reinterpret_cast<const uint16_t*>(src + t * row + n)) : uint16_t(0);
    }
    return x;
  }
  __device__ __forceinline__ void put(const Raw& x, int tid) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (tid + j * kBwdChans < kTile * NP) (&v[0][0])[tid + j * kBwdChans] = __uint_as_float(uint32_t(x.r[j]) << 16);
  }
  // States n0 .. n0 + 2 PAIRS - 1 of token t.
  template <int PAIRS>
  __device__ __forceinline__ void pairs(F2* out, int t, int n0) const {
#pragma unroll
    for (int i = 0; i < PAIRS / 2; ++i) {
      const float4 q = reinterpret_cast<const float4*>(&v[t][n0])[i];
      out[2 * i] = f2(q.x, q.y);
      out[2 * i + 1] = f2(q.z, q.w);
    }
  }
};

template <int NP>
struct BwdSmem {
  VecTile<NP> B[2], C[2];
  ChTile<kTile, kBwdChans, kBwdChans, 8> u[2], delta[2], z[2], dy[2];  // du, ddelta and dz replace u, delta and z
  float ck[2][2][NP / 2 * kBwdChans + 16];               // states before the tile, each half's [state][channel] 16 banks from the other's
  float4 tok[kTile][kBwdChans];                          // a token's dt, dt u, dy silu(z), d dt / d delta
  float4 sums[2][kTile][kBwdChans];                      // each lane's share of C . h, B . dh and A . w
  float red[kWarps][kTile][2][NP];                         // the warps' sums over their channels: dC, dB
};

// Tile by tile, the last first: forward over the tile's tokens, whose states stay in registers, then back over them. A channel
// takes two lanes of a warp, 16 apart, each with half of the states: that leaves registers for a whole tile's states and for
// three warps a scheduler, and each lane does the scalar work (step size, gates, their gradients) of half of the tile's tokens.
template <int NP>
__global__ void __launch_bounds__(kBwdThreads, 3) k_sscan_bwd(SscanParams p, int blocks) {
  constexpr int SP = NP / 2, PR = SP / 2, NQ = SP / 4;  // states, state pairs and quads of a lane
  extern __shared__ __align__(16) char smem_raw[];
  BwdSmem<NP>& sm = *reinterpret_cast<BwdSmem<NP>*>(smem_raw);
  if (!p.seg_state) wait_for_previous();
  const int seg = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const SscanSeg sg = sscan_seg(p, seg);
  const SscanChan ch = sscan_chan<kBwdChans>(p, cb);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = lane >> 4, part = tid & (kBwdChans - 1);
  const int c = warp * 16 + (lane & 15), d = ch.d0 + min(c, ch.chans - 1), n0 = half * SP, ns = p.N - n0;
  const bool gate = p.z != nullptr, softplus_on = p.softplus, live = c < ch.chans, low = tid < kBwdChans;
  // The products below put quad j into columns 2 j and 2 j + 1, and once more into 4 + 2 j and 5 + 2 j.
  float sel[NQ][2];
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) sel[j][e] = (lane >> 2 & 3) == 2 * j + e ? 1.f : 0.f;
  F2 A2[PR], g[PR], dA[PR];
  load_states<SP>(A2, p.A + (size_t)d * p.N + n0, 1, ns);
#pragma unroll
  for (int i = 0; i < PR; ++i) {
    A2[i] = mul2(A2[i], dup2(kLog2e));
    g[i] = dA[i] = f2(0.f, 0.f);
  }
  const float bias = param(p.bias, d), skip = param(p.Dskip, d);
  F2 dD = f2(0.f, 0.f), dbias = f2(0.f, 0.f);
  typename VecTile<NP>::Raw raw;
  auto request = [&](int tb, int buf) {
    const long long row = sg.row0 + tb;
    const int len = sg.len - tb;
    if (low) {
      sm.u[buf].load(p.u + row * p.u_s + ch.d0, p.u_s, len, ch.chans, p.vec, part);
      sm.delta[buf].load(p.delta + row * p.dt_s + ch.d0, p.dt_s, len, ch.chans, p.vec, part);
      raw = VecTile<NP>::fetch(p.Bm + row * p.b_s + ch.g * p.N, p.b_s, len, p.N, part);
    } else {
      sm.dy[buf].load(p.dy + row * p.D + ch.d0, p.D, len, ch.chans, p.vec, part);
      if (gate) sm.z[buf].load(p.z + row * p.z_s + ch.d0, p.z_s, len, ch.chans, p.vec, part);
      raw = VecTile<NP>::fetch(p.Cm + row * p.c_s + ch.g * p.N, p.c_s, len, p.N, part);
    }
    const float* ck = p.ck + (size_t)(sg.ck0 + tb / kTile) * p.N * p.D;
    if (p.quad) {  // four channels a copy; channels and states that the group lacks read as 0
      constexpr int kRow = kBwdChans / 4, kStep = kBwdThreads / kRow;
      const int c4 = tid % kRow * 4, n = tid / kRow;
      const bool in = c4 < ch.chans;
      const float* from = ck + (in ? ch.d0 + c4 : 0);
#pragma unroll
      for (int j = 0; j < NP / kStep; ++j) {
        const int s = n + j * kStep;
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&sm.ck[buf][s / SP][s % SP * kBwdChans + c4]));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from + (size_t)min(s, p.N - 1) * p.D), "r"(in && s < p.N ? 16 : 0)
                     : "memory");
      }
    } else {
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&sm.ck[buf][half][c]));
#pragma unroll
      for (int n = 0; n < SP; ++n)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + n * kBwdChans * 4), "l"(ck + (size_t)min(n0 + n, p.N - 1) * p.D + d),
                     "r"(n < ns ? 4 : 0)
                     : "memory");
    }
    copies_commit();
  };
  auto arrive = [&](int buf) { (low ? sm.B[buf] : sm.C[buf]).put(raw, part); };
  const int last = (sg.len - 1) / kTile * kTile;
  request(last, 0);
  arrive(0);
  if (p.seg_state) wait_for_previous();  // the composed gradients; the rest above are the call's inputs
  if (live) {
    if (p.seg_state) load_states<SP>(g, p.seg_state + ((size_t)seg * p.N + n0) * p.D + d, p.D, ns);
    else if (p.dfinal) load_states<SP>(g, p.dfinal + ((size_t)sg.seq * p.D + d) * p.N + n0, 1, ns);
  }
  for (int tb = last, buf = 0; tb >= 0; tb -= kTile, buf ^= 1) {
    const int len = min(kTile, sg.len - tb);
    const long long row = sg.row0 + tb;
    copies_wait();
    __syncthreads();
    if (tb > 0) request(tb - kTile, buf ^ 1);
    // The lane's half of the tokens. Past the segment's end dt and d dt / d delta are 0, dy is 0, and the state stays.
#pragma unroll
    for (int i = 0; i < kHalf; i += 2) {
      const int t = half * kHalf + i;
      const F2 x = add2(sm.delta[buf].next(t, c), dup2(bias)), u = sm.u[buf].next(t, c), dy = sm.dy[buf].next(t, c);
      F2 slope;
      const F2 sp = softplus2(x, &slope), gated = mul2(dy, silu2(sm.z[buf].next(t, c)));
      float dt[2], dtu[2], dy0[2], dd[2];
      unf2(softplus_on ? sp : x, &dt[0], &dt[1]);
      unf2(softplus_on ? slope : dup2(1.f), &dd[0], &dd[1]);
      unf2(gate ? gated : dy, &dy0[0], &dy0[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        dt[e] = t + e < len ? dt[e] : 0.f;
        dd[e] = t + e < len ? dd[e] : 0.f;
      }
      unf2(mul2(f2(dt[0], dt[1]), u), &dtu[0], &dtu[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) sm.tok[t + e][c] = make_float4(dt[e], dtu[e], dy0[e], dd[e]);
    }
    __syncwarp();
    F2 H[kTile][PR] = {};
    auto before = [&](int t, int s) { return t ? H[t ? t - 1 : 0][s] : f2(sm.ck[buf][half][2 * s * kBwdChans + c], sm.ck[buf][half][(2 * s + 1) * kBwdChans + c]); };
#pragma unroll
    for (int t = 0; t < kTile; ++t) {
      const float2 q = *reinterpret_cast<const float2*>(&sm.tok[t][c]);
      const F2 dt2 = dup2(q.x), dtu2 = dup2(q.y);
      F2 v[PR];
      sm.B[buf].template pairs<PR>(v, t, n0);
#pragma unroll
      for (int s = 0; s < PR; ++s) H[t][s] = fma2(decay2(dt2, A2[s]), before(t, s), mul2(dtu2, v[s]));
    }
#pragma unroll
    for (int t = kTile - 1; t >= 0; --t) {
      const float4 q = sm.tok[t][c];
      const F2 dt2 = dup2(q.x), dtu2 = dup2(q.y), dy2 = dup2(q.z);
      F2 v[PR];
      sm.C[buf].template pairs<PR>(v, t, n0);
      F2 y2 = f2(0.f, 0.f), sB = f2(0.f, 0.f), sA = f2(0.f, 0.f);
      // Sums over the four channels of each four lanes: a lane's quad of states is its share of A, ones in B pick columns. A term
      // goes in as its upper 11 bits and the 11 bits after those (the rest of it is below 2^-21 of it), so the sums are as good as
      // fp32's; the upper part alone would take 2^-11 off every term. dC and dB have accumulators of their own: fewer selectors,
      // and what is not finite in one does not reach the other. (Within one, a term that is infinite or NaN makes NaN of the token's
      // sums over all states.)
      float acc[2][4] = {};
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        F2 w[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int s = 2 * j + i;
          y2 = fma2(H[t][s], v[s], y2);
          g[s] = fma2(v[s], dy2, g[s]);
          w[0][i] = mul2(H[t][s], dy2);
          w[1][i] = mul2(g[s], dtu2);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float high[4], low[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            unf2(w[k][i], &high[2 * i], &high[2 * i + 1]);
            high[2 * i] = tf32_part(high[2 * i]), high[2 * i + 1] = tf32_part(high[2 * i + 1]);
            unf2(fma2(f2(high[2 * i], high[2 * i + 1]), dup2(-1.f), w[k][i]), &low[2 * i], &low[2 * i + 1]);
            low[2 * i] = tf32_part(low[2 * i]), low[2 * i + 1] = tf32_part(low[2 * i + 1]);
          }
          mma_tf32(acc[k], high[0], high[1], high[2], high[3], sel[j][0], sel[j][1], acc[k]);
          mma_tf32(acc[k], low[0], low[1], low[2], low[3], sel[j][0], sel[j][1], acc[k]);
        }
      }
      sm.B[buf].template pairs<PR>(v, t, n0);
#pragma unroll
      for (int s = 0; s < PR; ++s) {
        sB = fma2(g[s], v[s], sB);
        g[s] = mul2(g[s], decay2(dt2, A2[s]));
        const F2 x = mul2(g[s], before(t, s));
        sA = fma2(x, A2[s], sA);
        dA[s] = fma2(x, dt2, dA[s]);
      }
      sm.sums[half][t][c] = make_float4(sum2(y2), sum2(sB), sum2(sA), 0.f);
      // Lane 4 r + i now holds quad i % 2 of both, of the four lanes r; it goes on with dC's (i < 2) or dB's states 0, 2, 1, 3 in
      // k[0 .. 3]: added up over the half's four r, each lane ends with one.
      const bool is_dB = lane & 2, r0 = lane & 4, r1 = lane & 8;
      float k[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = is_dB ? acc[1][e] : acc[0][e];
      const float k0 = exchange(k[0], k[1], r0, 4), k1 = exchange(k[2], k[3], r0, 4), r = exchange(k0, k1, r1, 8);
      if ((lane & 1) < NQ) sm.red[warp][t][(lane >> 1) & 1][n0 + (lane & 1) * 4 + (r0 ? 2 : 0) + (r1 ? 1 : 0)] = r;
    }
    __syncwarp();
    // Both lanes' shares together; each lane ends its half of the tokens.
#pragma unroll
    for (int i = 0; i < kHalf; i += 2) {
      const int t = half * kHalf + i;
      float y[2], dhB[2], w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 s0 = sm.sums[0][t + e][c], s1 = sm.sums[1][t + e][c];
        y[e] = s0.x + s1.x;
        dhB[e] = s0.y + s1.y;
        w[e] = s0.z + s1.z;
      }
      const float4 q0 = sm.tok[t][c], q1 = sm.tok[t + 1][c];
      const F2 u = sm.u[buf].next(t, c), z = sm.z[buf].next(t, c), dy0 = f2(q0.z, q1.z), B2 = f2(dhB[0], dhB[1]);
      const F2 dd = mul2(fma2(u, B2, mul2(dup2(0.6931471805599453f), f2(w[0], w[1]))), f2(q0.w, q1.w)), sig = sigmoid2(z);
      dD = fma2(dy0, u, dD);
      dbias = add2(dbias, dd);
      const F2 slope = mul2(sig, fma2(z, fma2(sig, dup2(-1.f), dup2(1.f)), dup2(1.f)));
      const F2 dz = mul2(mul2(sm.dy[buf].next(t, c), fma2(dup2(skip), u, f2(y[0], y[1]))), slope);
      sm.u[buf].set_next(t, c, fma2(f2(q0.x, q1.x), B2, mul2(dup2(skip), dy0)));
      sm.delta[buf].set_next(t, c, dd);
      sm.z[buf].set_next(t, c, dz);
    }
    if (tb > 0) arrive(buf ^ 1);
    __syncthreads();
    if (low) {
      sm.u[buf].store(p.du + row * p.D + ch.d0, p.D, len, ch.chans, p.vec_out, part);
      sm.delta[buf].store(p.ddelta + row * p.D + ch.d0, p.D, len, ch.chans, p.vec_out, part);
    } else if (gate) {
      sm.z[buf].store(p.dz + row * p.D + ch.d0, p.D, len, ch.chans, p.vec_out, part);
    }
    // partial dC and dB of the tile: [token][dC, dB][N]
#pragma unroll
    for (int e = tid; e < kTile * 32; e += kBwdThreads) {
      const int t = e / 32, which = e / 16 % 2, n = e % 16;
      float r = 0.f;
      if (n < NP)
#pragma unroll
        for (int k = 0; k < kWarps; ++k) r += sm.red[k][t][which][n];
      if (t < len && n < p.N) p.part_bc[((size_t)cb * p.rows + row + t) * 2 * p.N + which * p.N + n] = r;
    }
  }
  const float dD_half = sum2(dD), dbias_half = sum2(dbias);
  const float dD_sum = dD_half + __shfl_xor_sync(0xffffffffu, dD_half, 16), dbias_sum = dbias_half + __shfl_xor_sync(0xffffffffu, dbias_half, 16);
  if (!live) return;
  if (p.dh0 && sg.j == 0) store_states<SP>(g, p.dh0 + ((size_t)sg.seq * p.D + d) * p.N + n0, 1, ns);
  float* par = p.part_par + (size_t)seg * (p.N + 2) * p.D + d;
  store_states<SP>(dA, par + (size_t)n0 * p.D, p.D, ns);
  if (half == 0) {
    par[(size_t)p.N * p.D] = dD_sum;
    par[(size_t)(p.N + 1) * p.D] = dbias_sum;
  }
}

// The last sums, in one launch. Blocks below `bc`: dC and dB of one (row, group, state) a thread, over the group's channel
// blocks in order. The others: dA, dD and ddelta_bias of 32 channels x 8 segment lanes, over the segments in a fixed order.
__global__ void __launch_bounds__(256) k_sscan_sums(SscanParams p, int bpg, int bc) {
  __shared__ float s[8][33];
  wait_for_previous();
  if (int(blockIdx.x) < bc) {
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x, per = 2ll * p.N;
    if (at >= p.rows * p.G * per) return;
    const int w = int(at % per), which = w / p.N, n = w - which * p.N;
    const long long rg = at / per, row = rg / p.G;
    const int g = int(rg - row * p.G);
    float t = 0.f;
#pragma unroll 8
    for (int k = 0; k < bpg; ++k) t += p.part_bc[((size_t)(g * bpg + k) * p.rows + row) * per + w];
    (which ? p.dB : p.dC)[(row * p.G + g) * p.N + n] = __float2bfloat16_rn(t);
    return;
  }
  const int b = blockIdx.x - bc, k = b % (p.N + 2), x = threadIdx.x & 31, y = threadIdx.x >> 5, d = b / (p.N + 2) * 32 + x;
  float t = 0.f;
  if (d < p.D)
#pragma unroll 8
    for (int i = y; i < p.segs; i += 8) t += p.part_par[((size_t)i * (p.N + 2) + k) * p.D + d];
  s[y][x] = t;
  __syncthreads();
  if (y || d >= p.D) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += s[i][x];
  if (k < p.N) p.dA[(size_t)d * p.N + k] = t;
  else if (k == p.N && p.dD) p.dD[d] = t;
  else if (k == p.N + 1 && p.dbias) p.dbias[d] = t;
}

template <int NP>
cudaError_t run(const SscanParams& p, cudaStream_t s) {
  const int blocks = sscan_blocks(p.G, p.Dg), grid = blocks * p.segs;
  const int smem = int(sizeof(BwdSmem<NP>)), bblocks = sscan_blocks(p.G, p.Dg, kBwdChans), bc = int((p.rows * p.G * 2 * p.N + 255) / 256);
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (e == cudaSuccess && !(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_sscan_bwd<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  if (e == cudaSuccess && p.seg_state) {
    const long long n = (long long)p.seqs * p.N * p.D;
    e = launch_after(k_sscan_rmap<NP>, grid, kSscanThreads, sizeof(RmapSmem<NP>), s, p, blocks);
    if (e == cudaSuccess) e = launch_after(k_sscan_rcompose, int((n + 255) / 256), 256, 0, s, p);
  }
  if (e == cudaSuccess) e = launch_after(k_sscan_bwd<NP>, bblocks * p.segs, kBwdThreads, smem, s, p, bblocks);
  return e == cudaSuccess ? launch_after(k_sscan_sums, bc + (p.D + 31) / 32 * (p.N + 2), 256, 0, s, p, bblocks / p.G, bc) : e;
}

}  // namespace

cudaError_t launch_sscan_bwd(const SscanParams& p, cudaStream_t s) { return p.N <= 8 ? run<8>(p, s) : run<16>(p, s); }

}  // namespace gdn
