// Selective scan, backward. With dy0 = dy silu(z) and a_t = exp(dt_t A), over tokens in reverse,
//   dh_t = C_t dy0_t + a_{t+1} dh_{t+1},
//   dC_t = sum_d dy0 h_t,  dB_t = sum_d dh_t dt u,  du = dt (B . dh) + D dy0,
//   w = dh_t a_t h_{t-1},  dA = sum_t w dt,  ddt = u (B . dh) + A . w,  ddelta = ddt sigmoid(delta + bias),
//   dz = dy (C . h + D u) silu'(z),  dD = sum_t dy0 u,  dh0 = a_1 dh_1.
//
// One thread walks one channel. The states it needs in reverse come from those a training forward keeps before every 8th
// token (8 bytes a token and channel): each tile of 8, last to first, is run forward again and then walked back. Keeping
// fewer costs another forward walk, which this kernel, bound by its instructions at 7% of HBM's rate, cannot hide as it
// does the reads. The adjoint chain is cut into segments like the forward's. The sums over channels in dB and dC begin as matrix products with ones: a
// lane's four states are its share of the A operand of m16n8k8, whose products add up four lanes' channels (tf32 operands;
// the results are bf16), and seven exchanges add up the eight groups of lanes. All other sums are fp32.
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
  const int seg = blockIdx.x / blocks;
  const SscanSeg sg = sscan_seg(p, seg);
  if (sg.j == 0) return;
  const SscanChan ch = sscan_chan(p, blockIdx.x % blocks);
  F2 A2[2][NP / 2], g[2][NP / 2];
  float bias[2], dt_sum[2] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    load_A2<NP>(A2[e], p, ch.d[e]);
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) g[e][i] = f2(0.f, 0.f);
    bias[e] = param(p.bias, ch.d[e]);
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
    for (int t0 = kRt - kRGroup; t0 >= 0; t0 -= kRGroup) {
      float dt[kRGroup][2], dy0[kRGroup][2];
#pragma unroll
      for (int i = 0; i < kRGroup; ++i) {
        const float2 dr = sm.delta[buf].at(t0 + i), yr = sm.dy[buf].at(t0 + i), zr = sm.z[buf].at(t0 + i);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = (e ? dr.y : dr.x) + bias[e], dy = e ? yr.y : yr.x, z = e ? zr.y : zr.x;
          float slope;
          const float sp = softplus(x, &slope);
          dt[i][e] = t0 + i < len ? (softplus_on ? sp : x) : 0.f;
          dt_sum[e] += dt[i][e];
          dy0[i][e] = gate ? dy * (z * sigmoid_fast(z)) : dy;
        }
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
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (!ch.live[e]) continue;
    p.seg_dt[(size_t)seg * p.D + ch.d[e]] = dt_sum[e];
  }
}

// One thread per (sequence, state, channel): from the sequence's end, each segment's exit gradient.
__global__ void __launch_bounds__(256) k_sscan_rcompose(SscanParams p) {
  const long long per = (long long)p.N * p.D, at = (long long)blockIdx.x * 256 + threadIdx.x;
  if (at >= per * p.seqs) return;
  const int seq = int(at / per), nd = int(at - seq * per), n = nd / p.D, d = nd - n * p.D;
  const int s0 = p.cu ? p.seg_base[seq] : seq * p.nseg_dense, s1 = p.cu ? p.seg_base[seq + 1] : s0 + p.nseg_dense;
  const float a2 = kLog2e * p.A[(size_t)d * p.N + n];
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

// Sums over the four channels of lanes 4 r .. 4 r + 3 of NP values a lane (pairs over states): states 4 j .. 4 j + 3 enter
// product j as A, whose B has ones in column 2 j for k < 4 and in column 2 j + 1 for k >= 4 (sel). Lane 4 r + j then holds the
// sums of states 4 j + {0, 2, 1, 3} of the four lanes.
template <int NP>
__device__ __forceinline__ void channel_sum(float* c, const F2* v, const float (*sel)[2]) {
  const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NP / 4; ++j) {
    float a0, a1, a2, a3;
    unf2(v[2 * j], &a0, &a1);
    unf2(v[2 * j + 1], &a2, &a3);
    mma_tf32(c, a0, a1, a2, a3, sel[j][0], sel[j][1], j ? c : zero);
  }
}
// One value for two lanes: the lane with `up` keeps b, the other a, each plus the other lane's.
__device__ __forceinline__ float exchange(float a, float b, bool up, int mask) {
  return (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, mask);
}

// ------------------------------------------------------------------ one channel a thread, states in pairs

constexpr int kBwdThreads = kSscanChans;
constexpr int kWarps = kBwdThreads / 32;
constexpr int kTile = kSscanBlock, kHalf = kTile / 2;

// A tile of tokens of B or C as fp32, [token][NP]: one element a thread.
template <int NP>
struct VecTile {
  float v[kTile][NP];
  static_assert(kTile * NP <= kBwdThreads, "one element a thread");
  __device__ __forceinline__ static uint16_t fetch(const __nv_bfloat16* src, long long row, int len, int N) {
    const int t = threadIdx.x / NP, n = threadIdx.x % NP;
    return t < len && t < kTile && n < N ? __ldg(reinterpret_cast<const uint16_t*>(src + t * row + n)) : uint16_t(0);
  }
  __device__ __forceinline__ void put(uint16_t r) {
    if (threadIdx.x < kTile * NP) (&v[0][0])[threadIdx.x] = __uint_as_float(uint32_t(r) << 16);
  }
  __device__ __forceinline__ void pairs(F2* out, int t) const {
#pragma unroll
    for (int i = 0; i < NP / 4; ++i) {
      const float4 q = reinterpret_cast<const float4*>(v[t])[i];
      out[2 * i] = f2(q.x, q.y);
      out[2 * i + 1] = f2(q.z, q.w);
    }
  }
};

template <int NP>
struct BwdSmem {
  VecTile<NP> B[2], C[2];
  ChTile<kTile, kBwdThreads> u[2], delta[2], z[2], dy[2];  // du, ddelta and dz replace u, delta and z token by token
  float ck[2][NP][kBwdThreads];                            // states before the tile
  float4 H[kHalf][NP / 4][kBwdThreads];                    // states after the tokens of the tile's first half
  float2 dts[kTile][kBwdThreads];                          // dt and d dt / d delta
  float red[kWarps][kTile][2][16];                         // the warps' sums over their channels: dC, dB
};

// Tile by tile, the last first: forward over the tile's tokens, whose states stay in shared memory (first half) and
// registers (second half), then back over them.
template <int NP>
__global__ void __launch_bounds__(kBwdThreads, 2) k_sscan_bwd(SscanParams p, int blocks) {
  extern __shared__ __align__(16) char smem_raw[];
  BwdSmem<NP>& sm = *reinterpret_cast<BwdSmem<NP>*>(smem_raw);
  const int seg = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const SscanSeg sg = sscan_seg(p, seg);
  const SscanChan ch = sscan_chan(p, cb);
  const int tid = threadIdx.x, d = ch.d0 + min(tid, ch.chans - 1), lane = tid & 31, warp = tid >> 5;
  const bool gate = p.z != nullptr, softplus_on = p.softplus, live = tid < ch.chans;
  float sel[NP / 4][2];
#pragma unroll
  for (int j = 0; j < NP / 4; ++j) {
    sel[j][0] = (lane >> 2) == 2 * j ? 1.f : 0.f;
    sel[j][1] = (lane >> 2) == 2 * j + 1 ? 1.f : 0.f;
  }
  F2 A2[NP / 2], g[NP / 2], dA[NP / 2];
  load_A2<NP>(A2, p, d);
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) g[i] = dA[i] = f2(0.f, 0.f);
  if (live) {
    if (p.seg_state) load_states<NP>(g, p.seg_state + (size_t)seg * p.N * p.D + d, p.D, p.N);
    else if (p.dfinal) load_states<NP>(g, p.dfinal + ((size_t)sg.seq * p.D + d) * p.N, 1, p.N);
  }
  const float bias = param(p.bias, d), skip = param(p.Dskip, d);
  float dD = 0.f, dbias = 0.f;
  uint16_t rb, rc;
  auto request = [&](int tb, int buf) {
    const long long row = sg.row0 + tb;
    const int len = sg.len - tb;
    sm.u[buf].load(p.u + row * p.u_s + ch.d0, p.u_s, len, ch.chans, p.vec);
    sm.delta[buf].load(p.delta + row * p.dt_s + ch.d0, p.dt_s, len, ch.chans, p.vec);
    sm.dy[buf].load(p.dy + row * p.D + ch.d0, p.D, len, ch.chans, p.vec);
    if (gate) sm.z[buf].load(p.z + row * p.z_s + ch.d0, p.z_s, len, ch.chans, p.vec);
    const float* ck = p.ck + (size_t)(sg.ck0 + tb / kTile) * p.N * p.D + d;
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&sm.ck[buf][0][tid]));
#pragma unroll
    for (int n = 0; n < NP; ++n)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + n * kBwdThreads * 4), "l"(ck + (size_t)min(n, p.N - 1) * p.D),
                   "r"(n < p.N ? 4 : 0)
                   : "memory");
    copies_commit();
    rb = VecTile<NP>::fetch(p.Bm + row * p.b_s + ch.g * p.N, p.b_s, len, p.N);
    rc = VecTile<NP>::fetch(p.Cm + row * p.c_s + ch.g * p.N, p.c_s, len, p.N);
  };
  const int last = (sg.len - 1) / kTile * kTile;
  request(last, 0);
  sm.B[0].put(rb);
  sm.C[0].put(rc);
  for (int tb = last, buf = 0; tb >= 0; tb -= kTile, buf ^= 1) {
    const int len = min(kTile, sg.len - tb);
    const long long row = sg.row0 + tb;
    copies_wait();
    __syncthreads();
    if (tb > 0) request(tb - kTile, buf ^ 1);
    // No branch in a token's work: past the segment's end dt and d dt / d delta are 0, dy is 0, and the state stays.
    F2 h[NP / 2], H[kHalf][NP / 2];
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) h[i] = f2(sm.ck[buf][2 * i][tid], sm.ck[buf][2 * i + 1][tid]);
    auto forward = [&](int t, const F2* from, F2* to) {
      const float x = sm.delta[buf].one(t, tid) + bias, u = sm.u[buf].one(t, tid);
      float slope, dt = softplus(x, &slope);
      dt = t < len ? (softplus_on ? dt : x) : 0.f;
      slope = t < len ? (softplus_on ? slope : 1.f) : 0.f;
      sm.dts[t][tid] = make_float2(dt, slope);
      const F2 dt2 = dup2(dt), dtu2 = dup2(dt * u);
      F2 v[NP / 2];
      sm.B[buf].pairs(v, t);
#pragma unroll
      for (int s = 0; s < NP / 2; ++s) to[s] = fma2(decay2(dt2, A2[s]), from[s], mul2(dtu2, v[s]));
    };
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      forward(i, h, h);
#pragma unroll
      for (int s = 0; s < NP / 4; ++s) {
        float4 q;
        unf2(h[2 * s], &q.x, &q.y);
        unf2(h[2 * s + 1], &q.z, &q.w);
        sm.H[i][s][tid] = q;
      }
    }
#pragma unroll
    for (int i = 0; i < kHalf; ++i) forward(kHalf + i, i ? H[i ? i - 1 : 0] : h, H[i]);
#pragma unroll 1
    for (int half = 1; half >= 0; --half) {
      if (half == 0) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
#pragma unroll
          for (int s = 0; s < NP / 4; ++s) {
            const float4 q = sm.H[i][s][tid];
            H[i][2 * s] = f2(q.x, q.y);
            H[i][2 * s + 1] = f2(q.z, q.w);
          }
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) h[i] = f2(sm.ck[buf][2 * i][tid], sm.ck[buf][2 * i + 1][tid]);
      }
#pragma unroll
      for (int i = kHalf - 1; i >= 0; --i) {
        const int t = half * kHalf + i;
        const float u = sm.u[buf].one(t, tid), dy = sm.dy[buf].one(t, tid), z = sm.z[buf].one(t, tid);
        const float2 ds = sm.dts[t][tid];
        const float dt = ds.x, sig = sigmoid_fast(z), dy0 = gate ? dy * (z * sig) : dy;
        const F2 dt2 = dup2(dt), dtu2 = dup2(dt * u), dy2 = dup2(dy0);
        float cC[4], cB[4];
        F2 v[NP / 2], w[NP / 2];
        sm.C[buf].pairs(v, t);
        F2 y2 = f2(skip * u, 0.f), sB = f2(0.f, 0.f), sA = f2(0.f, 0.f);
#pragma unroll
        for (int s = 0; s < NP / 2; ++s) {
          y2 = fma2(H[i][s], v[s], y2);
          g[s] = fma2(v[s], dy2, g[s]);
          w[s] = mul2(H[i][s], dy2);
        }
        channel_sum<NP>(cC, w, sel);
#pragma unroll
        for (int s = 0; s < NP / 2; ++s) w[s] = mul2(g[s], dtu2);
        channel_sum<NP>(cB, w, sel);
        sm.B[buf].pairs(v, t);
#pragma unroll
        for (int s = 0; s < NP / 2; ++s) {
          sB = fma2(g[s], v[s], sB);
          g[s] = mul2(g[s], decay2(dt2, A2[s]));
          const F2 x = mul2(g[s], i ? H[i ? i - 1 : 0][s] : h[s]);
          sA = fma2(x, A2[s], sA);
          dA[s] = fma2(x, dt2, dA[s]);
        }
        const float dhB = sum2(sB);
        const float ddt = fmaf(u, dhB, 0.6931471805599453f * sum2(sA)), dd = ddt * ds.y;
        dD = fmaf(dy0, u, dD);
        dbias += dd;
        sm.u[buf].set_one(t, tid, fmaf(dt, dhB, skip * dy0));
        sm.delta[buf].set_one(t, tid, dd);
        sm.z[buf].set_one(t, tid, dy * sum2(y2) * (sig * fmaf(z, 1.f - sig, 1.f)));
        // the eight sums of lane 4 r + j over its four lanes, added up over r, of which each lane ends with one
        const bool r0 = lane & 4, r1 = lane & 8, r2 = lane & 16;
        const float k0 = exchange(cC[0], cB[0], r0, 4), k1 = exchange(cC[1], cB[1], r0, 4);
        const float k2 = exchange(cC[2], cB[2], r0, 4), k3 = exchange(cC[3], cB[3], r0, 4);
        const float l0 = exchange(k0, k1, r1, 8), l1 = exchange(k2, k3, r1, 8);
        // accumulator 0, 1, 2, 3 = states 4 j + 0, 2, 1, 3
        sm.red[warp][t][r0][(lane & 3) * 4 + (r1 ? 2 : 0) + (r2 ? 1 : 0)] = exchange(l0, l1, r2, 16);
      }
    }
    if (tb > 0) {
      sm.B[buf ^ 1].put(rb);
      sm.C[buf ^ 1].put(rc);
    }
    __syncthreads();
    sm.u[buf].store(p.du + row * p.D + ch.d0, p.D, len, ch.chans, p.vec_out);
    sm.delta[buf].store(p.ddelta + row * p.D + ch.d0, p.D, len, ch.chans, p.vec_out);
    if (gate) sm.z[buf].store(p.dz + row * p.D + ch.d0, p.D, len, ch.chans, p.vec_out);
    // partial dC and dB of the tile: [token][dC, dB][N]
    float* part = p.part_bc + ((size_t)cb * p.rows + row) * 2 * p.N;
#pragma unroll
    for (int j = 0; j < kTile * 32 / kBwdThreads; ++j) {
      const int e = tid + j * kBwdThreads, t = e / 32, which = e / 16 % 2, n = e % 16;
      float r = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) r += sm.red[k][t][which][n];
      if (t < len && n < p.N) part[(t * 2 + which) * p.N + n] = r;
    }
  }
  if (!live) return;
  if (p.dh0 && sg.j == 0) store_states<NP>(g, p.dh0 + ((size_t)sg.seq * p.D + d) * p.N, 1, p.N);
  float* par = p.part_par + (size_t)seg * (p.N + 2) * p.D + d;
  store_states<NP>(dA, par, p.D, p.N);
  par[(size_t)p.N * p.D] = dD;
  par[(size_t)(p.N + 1) * p.D] = dbias;
}

// dC and dB of one (row, group, state): the sum over the group's channel blocks, in order.
__global__ void __launch_bounds__(256) k_sscan_sum_bc(SscanParams p, int bpg) {
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x, per = 2ll * p.N;
  if (at >= p.rows * p.G * per) return;
  const int w = int(at % per), which = w / p.N, n = w - which * p.N;
  const long long rg = at / per, row = rg / p.G;
  const int g = int(rg - row * p.G);
  float s = 0.f;
  for (int k = 0; k < bpg; ++k) s += p.part_bc[((size_t)(g * bpg + k) * p.rows + row) * per + w];
  (which ? p.dB : p.dC)[(row * p.G + g) * p.N + n] = __float2bfloat16_rn(s);
}

// dA, dD and ddelta_bias of one channel: the sum over the segments, in a fixed order. 32 channels x 8 segment lanes.
__global__ void __launch_bounds__(256) k_sscan_sum_par(SscanParams p) {
  __shared__ float s[8][33];
  const int d = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
  float t = 0.f;
  if (d < p.D)
#pragma unroll 4
    for (int i = threadIdx.y; i < p.segs; i += 8) t += p.part_par[((size_t)i * (p.N + 2) + k) * p.D + d];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y || d >= p.D) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += s[i][threadIdx.x];
  if (k < p.N) p.dA[(size_t)d * p.N + k] = t;
  else if (k == p.N && p.dD) p.dD[d] = t;
  else if (k == p.N + 1 && p.dbias) p.dbias[d] = t;
}

template <int NP>
cudaError_t run(const SscanParams& p, cudaStream_t s) {
  const int blocks = sscan_blocks(p.G, p.Dg), grid = blocks * p.segs;
  if (p.seg_state) {
    k_sscan_rmap<NP><<<grid, kSscanThreads, sizeof(RmapSmem<NP>), s>>>(p, blocks);
    const long long n = (long long)p.seqs * p.N * p.D;
    k_sscan_rcompose<<<int((n + 255) / 256), 256, 0, s>>>(p);
  }
  const int smem = int(sizeof(BwdSmem<NP>));
  cudaError_t e = cudaFuncSetAttribute(k_sscan_bwd<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_sscan_bwd<NP><<<grid, kBwdThreads, smem, s>>>(p, blocks);
  const long long n = p.rows * p.G * 2 * p.N;
  k_sscan_sum_bc<<<int((n + 255) / 256), 256, 0, s>>>(p, blocks / p.G);
  k_sscan_sum_par<<<dim3((p.D + 31) / 32, p.N + 2), dim3(32, 8), 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sscan_bwd(const SscanParams& p, cudaStream_t s) { return p.N <= 8 ? run<8>(p, s) : run<16>(p, s); }

}  // namespace gdn
