// Selective scan, forward. For every channel d with N states and every token t of a sequence,
//   h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,   y_t = (C_t . h_t + D u_t) silu(z_t),   dt = softplus(delta + bias).
//
// One thread walks two channels with their N states in registers: the sums over states stay in the thread, B and C are
// broadcast from shared memory, and u, delta, z and y are read and written once. The work per state and token is one
// exponential and four multiply-adds (packed for both channels), which the exponential unit and the fp32 pipe bound
// alike: about 4 cycles per warp and state on each.
//
// Few channels leave the GPU empty, so the tokens are cut into segments of L. The map of a segment,
// h_out = exp(A sum dt) h_in + F, is diagonal: a first pass runs every segment but the last from zero for F and sum dt,
// a small kernel composes them into entry states, and a second pass runs every segment from its entry state.
// With enough channels and sequences there is one segment and one pass.
#include "k_sscan.cuh"

namespace gdn {
namespace {

constexpr int kTt = 16;  // tokens staged together, double-buffered; kSscanBlock is a multiple of it

template <int NP, bool MAP>
struct PassSmem {
  BcTile<NP, kTt> B[2], C[MAP ? 1 : 2];
  ChTile<kTt> delta[2], u[2], z[MAP ? 1 : 2];  // y replaces u token by token
};

template <int NP, bool MAP>
__global__ void __launch_bounds__(kSscanThreads, 8) k_sscan_pass(SscanParams p, int blocks) {
  extern __shared__ __align__(16) char smem_raw[];
  PassSmem<NP, MAP>& sm = *reinterpret_cast<PassSmem<NP, MAP>*>(smem_raw);
  const int seg = blockIdx.x / blocks;
  const SscanSeg sg = sscan_seg(p, seg);
  if (MAP && sg.j == sg.nseg - 1) return;
  const SscanChan ch = sscan_chan(p, blockIdx.x % blocks);

  F2 A2[NP], h[NP];
  load_A2<NP>(A2, p, ch);
#pragma unroll
  for (int n = 0; n < NP; ++n) h[n] = f2(0.f, 0.f);
  if (!MAP) {
    if (p.seg_state) load_state<NP>(h, p.seg_state + (size_t)seg * p.N * p.D, p, ch);
    else if (p.h0) load_user_state<NP>(h, p.h0 + (size_t)sg.seq * p.D * p.N, p, ch);
  }
  const F2 bias = load_param(p.bias, ch), skip = load_param(MAP ? nullptr : p.Dskip, ch);
  const bool out = !MAP && p.y, gate = out && p.z, softplus_on = p.softplus;
  F2 dt_sum = f2(0.f, 0.f);

  BcRegs<NP, kTt> rb, rc;
  auto request = [&](int tb, int buf) {
    const long long row = sg.row0 + tb;
    const int len = sg.len - tb;
    sm.delta[buf].load(p.delta + row * p.dt_s + ch.d0, p.dt_s, len, ch.chans, p.vec);
    sm.u[buf].load(p.u + row * p.u_s + ch.d0, p.u_s, len, ch.chans, p.vec);
    if (!MAP && gate) sm.z[buf].load(p.z + row * p.z_s + ch.d0, p.z_s, len, ch.chans, p.vec);
    copies_commit();
    rb.load(p.Bm + row * p.b_s + ch.g * p.N, p.b_s, len, p.N);
    if (!MAP) rc.load(p.Cm + row * p.c_s + ch.g * p.N, p.c_s, len, p.N);
  };
  auto arrive = [&](int buf) {
    rb.store(sm.B[buf]);
    if (!MAP) rc.store(sm.C[buf]);
  };
  request(0, 0);
  arrive(0);
  for (int tb = 0, buf = 0; tb < sg.len; tb += kTt, buf ^= 1) {
    copies_wait();
    __syncthreads();
    const bool more = tb + kTt < sg.len;
    if (more) request(tb + kTt, buf ^ 1);
    if (!MAP && p.ck && tb % kSscanBlock == 0) store_state<NP>(h, p.ck + (size_t)(sg.ck0 + tb / kSscanBlock) * p.N * p.D, p, ch);
    const int len = min(kTt, sg.len - tb);
    // no branch in a token's work, so that the compiler can overlap several tokens: past the segment's end dt = 0, which
    // leaves the state as it is, and without softplus or gate their results are not selected
#pragma unroll 2
    for (int t = 0; t < kTt; ++t) {
      const F2 x = add2(sm.delta[buf].at(t), bias), u = sm.u[buf].at(t);
      F2 dt = softplus2<false>(x, nullptr);
      dt = select2(t < len, select2(softplus_on, dt, x), f2(0.f, 0.f));
      const F2 dtu = mul2(dt, u);
      F2 y = mul2(skip, u);
#pragma unroll
      for (int n = 0; n < NP; n += 2) {
        F2 b[2], c[2];
        load_two(b, &sm.B[buf].v[t][n]);
        if (!MAP) load_two(c, &sm.C[buf].v[t][n]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          h[n + e] = fma2(exp2_approx2(mul2(dt, A2[n + e])), h[n + e], mul2(dtu, b[e]));
          if (!MAP) y = fma2(h[n + e], c[e], y);
        }
      }
      if (MAP) {
        dt_sum = add2(dt_sum, dt);
      } else {
        const F2 z = sm.z[MAP ? 0 : buf].at(t);
        sm.u[buf].set(t, select2(gate, mul2(y, mul2(z, sigmoid2(z))), y));
      }
    }
    if (more) arrive(buf ^ 1);
    if (out) {
      __syncthreads();
      sm.u[buf].store(p.y + (sg.row0 + tb) * p.D + ch.d0, p.D, len, ch.chans, p.vec_out);
    }
  }
  if (MAP) {
    store_state<NP>(h, p.seg_state + (size_t)seg * p.N * p.D, p, ch);
    store_pair(p.seg_dt + (size_t)seg * p.D, dt_sum, ch);
  } else if (p.final_state && sg.j == sg.nseg - 1) {
    store_user_state<NP>(h, p.final_state + (size_t)sg.seq * p.D * p.N, p, ch);
  }
}

// One thread per (sequence, state, channel): walks the sequence's segments, leaving each its entry state.
__global__ void __launch_bounds__(256) k_sscan_compose(SscanParams p) {
  const long long per = (long long)p.N * p.D, at = (long long)blockIdx.x * 256 + threadIdx.x;
  if (at >= per * p.seqs) return;
  const int seq = int(at / per), nd = int(at - seq * per), n = nd / p.D, d = nd - n * p.D;
  const int s0 = p.cu ? p.seg_base[seq] : seq * p.nseg_dense, s1 = p.cu ? p.seg_base[seq + 1] : s0 + p.nseg_dense;
  const float a2 = kLog2e * p.A[(size_t)d * p.N + n];
  float carry = p.h0 ? p.h0[((size_t)seq * p.D + d) * p.N + n] : 0.f;
  constexpr int kAhead = 8;
  for (int s = s0; s < s1; s += kAhead) {
    float f[kAhead], t[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s + i < s1 - 1) {
        f[i] = p.seg_state[(size_t)(s + i) * per + nd];
        t[i] = p.seg_dt[(size_t)(s + i) * p.D + d];
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s + i < s1) {
        p.seg_state[(size_t)(s + i) * per + nd] = carry;
        if (s + i < s1 - 1) carry = fmaf(exp2_approx(a2 * t[i]), carry, f[i]);
      }
  }
}

template <int NP>
cudaError_t run(const SscanParams& p, cudaStream_t s) {
  const int blocks = sscan_blocks(p.G, p.Dg), grid = blocks * p.segs;
  if (p.seg_state) {
    k_sscan_pass<NP, true><<<grid, kSscanThreads, sizeof(PassSmem<NP, true>), s>>>(p, blocks);
    const long long n = (long long)p.seqs * p.N * p.D;
    k_sscan_compose<<<int((n + 255) / 256), 256, 0, s>>>(p);
  }
  k_sscan_pass<NP, false><<<grid, kSscanThreads, sizeof(PassSmem<NP, false>), s>>>(p, blocks);
  return cudaGetLastError();
}

}  // namespace

static_assert(sizeof(PassSmem<kSscanMaxN, false>) <= 48 * 1024, "fits the default shared memory limit");

cudaError_t launch_sscan_fwd(const SscanParams& p, cudaStream_t s) { return p.N <= 8 ? run<8>(p, s) : run<16>(p, s); }

}  // namespace gdn
