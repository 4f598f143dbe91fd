// Selective scan, forward. For every channel d with N states and every token t of a sequence,
//   h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,   y_t = (C_t . h_t + D u_t) silu(z_t),   dt = softplus(delta + bias).
//
// One thread walks one channel with its N states in registers: the sums over states stay in the thread, B and C are
// broadcast from shared memory, and u, delta, z and y are read and written once. The work per state and token is one
// exponential and four multiply-adds (packed in pairs), which the exponential unit and the fp32 pipe bound alike:
// about 4 cycles per warp and state on each.
//
// Few channels leave the GPU empty, so the tokens are cut into segments of L. The map of a segment,
// h_out = exp(A sum dt) h_in + F, is diagonal: a first pass runs every segment but the last from zero for F and sum dt,
// a small kernel composes them into entry states, and a second pass runs every segment from its entry state.
// With enough channels and sequences there is one segment and one pass.
#include "k_sscan.cuh"

namespace gdn {
namespace {

constexpr int kGroup = 8;  // tokens whose inputs are loaded together, one group ahead

template <int NP, bool MAP>
__global__ void __launch_bounds__(kSscanThreads) k_sscan_pass(SscanParams p, int blocks) {
  __shared__ BcTile<NP> bc[2];
  const SscanSeg sg = sscan_seg(p, blockIdx.x / blocks);
  if (MAP && sg.j == sg.nseg - 1) return;
  const SscanChan ch = sscan_chan(p, blockIdx.x % blocks);
  const int d = ch.d, seg = blockIdx.x / blocks;

  F2 A2[NP / 2], h[NP / 2];
  load_A2<NP>(A2, p, d);
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) h[i] = f2(0.f, 0.f);
  if (!MAP) {
    if (p.seg_state) load_state<NP>(h, p.seg_state + (size_t)seg * p.N * p.D, p, d);
    else if (p.h0) load_user_state<NP>(h, p.h0 + (size_t)sg.seq * p.D * p.N, p, d);
  }
  const float bias = p.bias ? __ldg(p.bias + d) : 0.f, skip = !MAP && p.Dskip ? __ldg(p.Dskip + d) : 0.f;
  const bool gate = !MAP && p.z != nullptr;
  const __nv_bfloat16 *up = p.u + sg.row0 * p.u_s + d, *dp = p.delta + sg.row0 * p.dt_s + d;
  const __nv_bfloat16* zp = gate ? p.z + sg.row0 * p.z_s + d : nullptr;
  __nv_bfloat16* yp = p.y ? p.y + sg.row0 * p.D + d : nullptr;
  float dt_sum = 0.f;

  BcRegs<NP> raw;
  raw.load(p, ch.g, sg.row0, sg.len, true, !MAP);
  raw.store(bc[0]);
  float un[kGroup], dn[kGroup], zn[kGroup];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const bool in = t0 + i < sg.len;
      un[i] = in ? bf16_at(up + (t0 + i) * p.u_s) : 0.f;
      dn[i] = in ? bf16_at(dp + (t0 + i) * p.dt_s) : 0.f;
      zn[i] = in && gate ? bf16_at(zp + (t0 + i) * p.z_s) : 0.f;
    }
  };
  fetch(0);
  __syncthreads();
  for (int tb = 0, buf = 0; tb < sg.len; tb += kSscanBlock, buf ^= 1) {
    const bool more = tb + kSscanBlock < sg.len;
    if (more) raw.load(p, ch.g, sg.row0 + tb + kSscanBlock, sg.len - tb - kSscanBlock, true, !MAP);
    if (!MAP && p.ck && ch.live) store_state<NP>(h, p.ck + (size_t)(sg.ck0 + tb / kSscanBlock) * p.N * p.D, p, d);
    const int n = min(kSscanBlock, sg.len - tb);
    for (int q = 0; q < n; q += kGroup) {
      float uc[kGroup], dc[kGroup], zc[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) uc[i] = un[i], dc[i] = dn[i], zc[i] = zn[i];
      fetch(tb + q + kGroup);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        if (q + i < n) {
          float dt = dc[i] + bias, slope;
          if (p.softplus) dt = softplus(dt, &slope);
          const float dtu = dt * uc[i];
          const F2 dt2 = f2(dt, dt), dtu2 = f2(dtu, dtu);
          F2 v[NP / 2];
          load_pairs(v, bc[buf].B[q + i], NP);
#pragma unroll
          for (int s = 0; s < NP / 2; ++s) h[s] = fma2(exp2_approx2(mul2(dt2, A2[s])), h[s], mul2(dtu2, v[s]));
          if (MAP) {
            dt_sum += dt;
          } else if (yp) {
            load_pairs(v, bc[buf].C[q + i], NP);
            F2 y2 = f2(skip * uc[i], 0.f);
#pragma unroll
            for (int s = 0; s < NP / 2; ++s) y2 = fma2(h[s], v[s], y2);
            float y = sum2(y2);
            if (gate) y *= zc[i] * sigmoid_fast(zc[i]);
            if (ch.live) yp[(long long)(tb + q + i) * p.D] = __float2bfloat16_rn(y);
          }
        }
      }
    }
    if (more) raw.store(bc[buf ^ 1]);
    __syncthreads();
  }
  if (!ch.live) return;
  if (MAP) {
    store_state<NP>(h, p.seg_state + (size_t)seg * p.N * p.D, p, d);
    p.seg_dt[(size_t)seg * p.D + d] = dt_sum;
  } else if (p.final_state && sg.j == sg.nseg - 1) {
    store_user_state<NP>(h, p.final_state + (size_t)sg.seq * p.D * p.N, p, d);
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
    k_sscan_pass<NP, true><<<grid, kSscanThreads, 0, s>>>(p, blocks);
    const long long n = (long long)p.seqs * p.N * p.D;
    k_sscan_compose<<<int((n + 255) / 256), 256, 0, s>>>(p);
  }
  k_sscan_pass<NP, false><<<grid, kSscanThreads, 0, s>>>(p, blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sscan_fwd(const SscanParams& p, cudaStream_t s) { return p.N <= 8 ? run<8>(p, s) : run<16>(p, s); }

}  // namespace gdn
