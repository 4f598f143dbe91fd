// Selective scan, forward. For every channel d with N states and every token t of a sequence,
//   h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,   y_t = (C_t . h_t + D u_t) silu(z_t),   dt = softplus(delta + bias).
//
// One thread walks two channels with their N states in registers: the sums over states stay in the thread, B and C are
// broadcast from shared memory, and u, delta, z and y are read and written once. The work per state and token is one
// exponential and four multiply-adds (packed in state pairs), which the exponential unit and the fp32 pipe bound
// alike: about 4 cycles per warp and state on each.
//
// On GB300, 8192 tokens x 4096 channels x 16 states: 245 us (maps 98, composition 9, outputs 140; 2.2e12 state updates a
// second in two passes, 1.1 TB/s of algorithmic bytes), with both units 45 to 60% busy. In isolation a pass's
// loop takes 290 cycles per warp-token (64 channels) and scheduler, where either unit alone would take 130 to 150.
//
// Few channels leave the GPU empty, so the tokens are cut into segments of L. The map of a segment,
// h_out = exp(A sum dt) h_in + F, is diagonal: a first pass runs every segment but the last from zero for F and sum dt,
// a small kernel composes them into entry states, and a second pass runs every segment from its entry state.
// With enough channels and sequences there is one segment and one pass.
#include "k_sscan.cuh"

namespace gdn {
namespace {

constexpr int kGroup = 4;
constexpr int kTt = 16;  // tokens staged together, double-buffered; a multiple of kSscanBlock and kGroup

template <int NP, bool MAP>
struct PassSmem {
  static constexpr int kBc = MAP ? 2 : 1;      // the pass with outputs has a barrier between tiles anyway
  BcTile<NP, kTt> B[kBc], C[1];
  ChTile<kTt> delta[2], u[2], z[MAP ? 1 : 2];  // y replaces u token by token
};

template <int NP, bool MAP>
__global__ void __launch_bounds__(kSscanThreads, 8) k_sscan_pass(SscanParams p, int blocks) {
  extern __shared__ __align__(16) char smem_raw[];
  PassSmem<NP, MAP>& sm = *reinterpret_cast<PassSmem<NP, MAP>*>(smem_raw);
  if (MAP || !p.seg_state) wait_for_previous();
  const int seg = blockIdx.x / blocks;
  const SscanSeg sg = sscan_seg(p, seg);
  if (MAP && sg.j == sg.nseg - 1) return;
  const SscanChan ch = sscan_chan(p, blockIdx.x % blocks);

  F2 A2[2][NP / 2], h[2][NP / 2];
  const F2 bias = f2(param(p.bias, ch.d[0]), param(p.bias, ch.d[1]));
  const F2 skip = f2(param(MAP ? nullptr : p.Dskip, ch.d[0]), param(MAP ? nullptr : p.Dskip, ch.d[1]));
  F2 dt_sum = f2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 2; ++e) load_A2<NP>(A2[e], p, ch.d[e]);
  const bool out = !MAP && p.y, gate = out && p.z, softplus_on = p.softplus;

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
    rb.store(sm.B[MAP ? buf : 0]);
    if (!MAP) rc.store(sm.C[0]);
  };
  request(0, 0);
  arrive(0);
  if (!MAP && p.seg_state) wait_for_previous();  // the composed states; the rest above are the call's inputs
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int d = ch.d[e];
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) h[e][i] = f2(0.f, 0.f);
    if (!MAP) {
      if (p.seg_state) load_states<NP>(h[e], p.seg_state + (size_t)seg * p.N * p.D + d, p.D, p.N);
      else if (p.h0) load_states<NP>(h[e], p.h0 + ((size_t)sg.seq * p.D + d) * p.N, 1, p.N);
    }
  }
  for (int tb = 0, buf = 0; tb < sg.len; tb += kTt, buf ^= 1) {
    copies_wait();
    __syncthreads();
    const bool more = tb + kTt < sg.len;
    if (more) request(tb + kTt, buf ^ 1);
    const int len = min(kTt, sg.len - tb);
    // Tokens go in groups, whose step sizes and gates (long dependent chains) are computed side by side before and after the
    // states. No branch in a token's work: past the segment's end dt = 0, which leaves the state as it is, and without
    // softplus or gate their results are not selected.
#pragma unroll 1
    for (int t0 = 0; t0 < len; t0 += kGroup) {
      if (!MAP && p.ck && t0 % kSscanBlock == 0)
        store_rows<NP>(h, p.ck + (size_t)(sg.ck0 + (tb + t0) / kSscanBlock) * p.N * p.D, p, ch);
      float dt[kGroup][2], dtu[kGroup][2];
      F2 y[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const F2 u = sm.u[buf].pair(t0 + i), x = add2(sm.delta[buf].pair(t0 + i), bias), sp = softplus2(x);
        const bool in = t0 + i < len;
        unf2(softplus_on ? sp : x, &dt[i][0], &dt[i][1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) dt[i][e] = in ? dt[i][e] : 0.f;
        const F2 both = f2(dt[i][0], dt[i][1]);
        unf2(mul2(both, u), &dtu[i][0], &dtu[i][1]);
        if (MAP) dt_sum = add2(dt_sum, both);
        else y[i] = mul2(skip, u);
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        F2 y2[2];
        const F2 dt2[2] = {dup2(dt[i][0]), dup2(dt[i][1])}, dtu2[2] = {dup2(dtu[i][0]), dup2(dtu[i][1])};
#pragma unroll
        for (int s = 0; s < NP / 2; s += 2) {
          F2 b[2], c[2];
          sm.B[MAP ? buf : 0].quad(b, t0 + i, s / 2);
          if (!MAP) sm.C[0].quad(c, t0 + i, s / 2);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              h[e][s + k] = fma2(decay2(dt2[e], A2[e][s + k]), h[e][s + k], mul2(dtu2[e], b[k]));
              if (!MAP) y2[e] = s + k ? fma2(h[e][s + k], c[k], y2[e]) : mul2(h[e][0], c[0]);
            }
        }
        if (!MAP) y[i] = add2(y[i], f2(sum2(y2[0]), sum2(y2[1])));
      }
      if (!MAP) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const F2 a = mul2(y[i], silu2(sm.z[MAP ? 0 : buf].pair(t0 + i)));
          float lo, hi;
          unf2(gate ? a : y[i], &lo, &hi);
          sm.u[buf].set(t0 + i, lo, hi);
        }
      }
    }
    if (!MAP) __syncthreads();
    if (more) arrive(buf ^ 1);
    if (out) sm.u[buf].store(p.y + (sg.row0 + tb) * p.D + ch.d0, p.D, len, ch.chans, p.vec_out);
  }
  if (MAP) store_rows<NP>(h, p.seg_state + (size_t)seg * p.N * p.D, p, ch);
  float dts[2];
  unf2(dt_sum, &dts[0], &dts[1]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (!ch.live[e]) continue;
    const int d = ch.d[e];
    if (MAP) {
      p.seg_dt[(size_t)seg * p.D + d] = dts[e];
    } else if (p.final_state && sg.j == sg.nseg - 1) {
      store_states<NP>(h[e], p.final_state + ((size_t)sg.seq * p.D + d) * p.N, 1, p.N);
    }
  }
}

// One thread per (sequence, state, channel): walks the sequence's segments, leaving each its entry state.
__global__ void __launch_bounds__(256) k_sscan_compose(SscanParams p) {
  const long long per = (long long)p.N * p.D, at = (long long)blockIdx.x * 256 + threadIdx.x;
  if (at >= per * p.seqs) return;
  const int seq = int(at / per), nd = int(at - seq * per), n = nd / p.D, d = nd - n * p.D;
  const int s0 = p.cu ? p.seg_base[seq] : seq * p.nseg_dense, s1 = p.cu ? p.seg_base[seq + 1] : s0 + p.nseg_dense;
  const float a2 = kLog2e * p.A[(size_t)d * p.N + n];
  wait_for_previous();
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
        if (s + i < s1 - 1) carry = fmaf(decay(t[i], a2), carry, f[i]);
      }
  }
}

template <int NP>
cudaError_t run(const SscanParams& p, cudaStream_t s) {
  const int blocks = sscan_blocks(p.G, p.Dg), grid = blocks * p.segs;
  const dim3 block(kSscanThreads);
  cudaError_t e = cudaSuccess;
  if (p.seg_state) {
    const long long n = (long long)p.seqs * p.N * p.D;
    e = launch_after(k_sscan_pass<NP, true>, grid, block, sizeof(PassSmem<NP, true>), s, p, blocks);
    if (e == cudaSuccess) e = launch_after(k_sscan_compose, int((n + 255) / 256), 256, 0, s, p);
  }
  return e == cudaSuccess ? launch_after(k_sscan_pass<NP, false>, grid, block, sizeof(PassSmem<NP, false>), s, p, blocks) : e;
}

}  // namespace

static_assert(sizeof(PassSmem<kSscanMaxN, false>) <= 48 * 1024, "fits the default shared memory limit");

cudaError_t launch_sscan_fwd(const SscanParams& p, cudaStream_t s) { return p.N <= 8 ? run<8>(p, s) : run<16>(p, s); }

}  // namespace gdn
