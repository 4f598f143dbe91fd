// Selective scan, backward. With dy0 = dy silu(z) and a_t = exp(dt_t A), over tokens in reverse,
//   dh_t = C_t dy0_t + a_{t+1} dh_{t+1},
//   dC_t = sum_d dy0 h_t,  dB_t = sum_d dh_t dt u,  du = dt (B . dh) + D dy0,
//   w = dh_t a_t h_{t-1},  dA = sum_t w dt,  ddt = u (B . dh) + A . w,  ddelta = ddt sigmoid(delta + bias),
//   dz = dy (C . h + D u) silu'(z),  dD = sum_t dy0 u,  dh0 = a_1 dh_1.
//
// One thread walks one channel. The states it needs in reverse come from the states a training forward keeps before every
// 32nd token: a block of 32 is run forward once to leave the entry states of its 8-token tiles in shared memory, and each
// tile, last to first, is run forward again into registers and then walked back. The adjoint chain is cut into segments
// like the forward's. The sums over channels in dB and dC are matrix products with ones: a lane's pair of states is a
// column of the B operand of m16n8k8, selector rows of A put state n into row n of the accumulator, and four lanes' channels
// add up in each product (tf32 operands; the results are bf16). All other sums are fp32.
#include "k_sscan.cuh"

namespace gdn {
namespace {

constexpr int kTile = 8;
constexpr int kTiles = kSscanBlock / kTile;
constexpr int kWarps = kSscanThreads / 32;

// The adjoint map of a segment: from a zero exit gradient to the gradient of the state before its first token.
template <int NP>
__global__ void __launch_bounds__(kSscanThreads) k_sscan_rmap(SscanParams p, int blocks) {
  __shared__ BcTile<NP> bc[2];
  const SscanSeg sg = sscan_seg(p, blockIdx.x / blocks);
  if (sg.j == 0) return;
  const SscanChan ch = sscan_chan(p, blockIdx.x % blocks);
  const int d = ch.d, seg = blockIdx.x / blocks;
  F2 A2[NP / 2], g[NP / 2];
  load_A2<NP>(A2, p, d);
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) g[i] = f2(0.f, 0.f);
  const float bias = p.bias ? __ldg(p.bias + d) : 0.f;
  const bool gate = p.z != nullptr;
  const __nv_bfloat16 *dp = p.delta + sg.row0 * p.dt_s + d, *yp = p.dy + sg.row0 * p.D + d;
  const __nv_bfloat16* zp = gate ? p.z + sg.row0 * p.z_s + d : nullptr;
  float dt_sum = 0.f;
  const int nb = (sg.len + kSscanBlock - 1) / kSscanBlock;
  BcRegs<NP> raw;
  raw.load(p, ch.g, sg.row0 + (nb - 1) * kSscanBlock, sg.len - (nb - 1) * kSscanBlock, false, true);
  raw.store(bc[0]);
  float yn[kTile], dn[kTile], zn[kTile];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      const bool in = t0 >= 0 && t0 + i < sg.len;
      yn[i] = in ? bf16_at(yp + (long long)(t0 + i) * p.D) : 0.f;
      dn[i] = in ? bf16_at(dp + (t0 + i) * p.dt_s) : 0.f;
      zn[i] = in && gate ? bf16_at(zp + (t0 + i) * p.z_s) : 0.f;
    }
  };
  fetch((sg.len - 1) / kTile * kTile);
  __syncthreads();
  for (int b = nb - 1, buf = 0; b >= 0; --b, buf ^= 1) {
    const int tb = b * kSscanBlock, n = min(kSscanBlock, sg.len - tb);
    if (b > 0) raw.load(p, ch.g, sg.row0 + tb - kSscanBlock, kSscanBlock, false, true);
    for (int q = (n - 1) / kTile * kTile; q >= 0; q -= kTile) {
      float yc[kTile], dc[kTile], zc[kTile];
#pragma unroll
      for (int i = 0; i < kTile; ++i) yc[i] = yn[i], dc[i] = dn[i], zc[i] = zn[i];
      fetch(tb + q - kTile);
#pragma unroll
      for (int i = kTile - 1; i >= 0; --i) {
        if (q + i < n) {
          float dt = dc[i] + bias, slope;
          if (p.softplus) dt = softplus(dt, &slope);
          dt_sum += dt;
          const float dy0 = gate ? yc[i] * zc[i] * sigmoid_fast(zc[i]) : yc[i];
          const F2 dt2 = f2(dt, dt), dy2 = f2(dy0, dy0);
          F2 v[NP / 2];
          load_pairs(v, bc[buf].C[q + i], NP);
#pragma unroll
          for (int s = 0; s < NP / 2; ++s) g[s] = mul2(exp2_approx2(mul2(dt2, A2[s])), fma2(v[s], dy2, g[s]));
        }
      }
    }
    if (b > 0) raw.store(bc[buf ^ 1]);
    __syncthreads();
  }
  if (!ch.live) return;
  store_state<NP>(g, p.seg_state + (size_t)seg * p.N * p.D, p, d);
  p.seg_dt[(size_t)seg * p.D + d] = dt_sum;
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
        if (s - i > s0) carry = fmaf(exp2_approx(a2 * t[i]), carry, f[i]);
      }
  }
}

// C[r][c] += sum_k A[r][k] B[k][c] with this lane's b0 (k = lane % 4) and b1 (k = lane % 4 + 4) of column lane / 4.
__device__ __forceinline__ void mma_sel(float* c, float a0, float a1, float a2, float a3, float b0, float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
        "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// Adds this lane's NP values (pairs over states) into accumulator rows = states, columns = groups of four lanes.
template <int NP>
__device__ __forceinline__ void channel_sum(float* c, const F2* v, const float* even, const float* odd) {
#pragma unroll
  for (int j = 0; j < NP / 2; ++j) {
    float lo, hi;
    unf2(v[j], &lo, &hi);
    if (j < 4) mma_sel(c, even[j], 0.f, odd[j], 0.f, lo, hi);
    else mma_sel(c, 0.f, even[j - 4], 0.f, odd[j - 4], lo, hi);
  }
}

template <int NP>
struct BwdSmem {
  BcTile<NP> bc;
  float entry[kTiles][NP / 2][kSscanThreads][2];       // states before each tile
  float red[kWarps][kSscanBlock][2][16];               // the warps' sums over their channels: dC, dB
};

template <int NP>
__global__ void __launch_bounds__(kSscanThreads) k_sscan_bwd(SscanParams p, int blocks) {
  extern __shared__ __align__(16) char smem_raw[];
  BwdSmem<NP>& sm = *reinterpret_cast<BwdSmem<NP>*>(smem_raw);
  const int seg = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const SscanSeg sg = sscan_seg(p, seg);
  const SscanChan ch = sscan_chan(p, cb);
  const int d = ch.d, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool gate = p.z != nullptr;
  float even[4], odd[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    even[j] = (lane >> 2) == 2 * j ? 1.f : 0.f;
    odd[j] = (lane >> 2) == 2 * j + 1 ? 1.f : 0.f;
  }
  F2 A2[NP / 2], g[NP / 2], dA[NP / 2];
  load_A2<NP>(A2, p, d);
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) g[i] = dA[i] = f2(0.f, 0.f);
  if (ch.live) {
    if (p.seg_state) load_state<NP>(g, p.seg_state + (size_t)seg * p.N * p.D, p, d);
    else if (p.dfinal) load_user_state<NP>(g, p.dfinal + (size_t)sg.seq * p.D * p.N, p, d);
  }
  const float bias = p.bias ? __ldg(p.bias + d) : 0.f, skip = p.Dskip ? __ldg(p.Dskip + d) : 0.f;
  const __nv_bfloat16 *up = p.u + sg.row0 * p.u_s + d, *dp = p.delta + sg.row0 * p.dt_s + d, *yp = p.dy + sg.row0 * p.D + d;
  const __nv_bfloat16* zp = gate ? p.z + sg.row0 * p.z_s + d : nullptr;
  const long long out0 = sg.row0 * p.D + d;
  float dD = 0.f, dbias = 0.f;
  const int nb = (sg.len + kSscanBlock - 1) / kSscanBlock;
  for (int b = nb - 1; b >= 0; --b) {
    const int tb = b * kSscanBlock, n = min(kSscanBlock, sg.len - tb);
    {
      BcRegs<NP> raw;
      raw.load(p, ch.g, sg.row0 + tb, n, true, true);
      __syncthreads();  // the previous block's tile and sums have been read
      raw.store(sm.bc);
    }
    __syncthreads();
    F2 h[NP / 2];
    load_state<NP>(h, p.ck + (size_t)(sg.ck0 + b) * p.N * p.D, p, d);
    const int tiles = (n + kTile - 1) / kTile;
    for (int q = 0; q < tiles; ++q) {
#pragma unroll
      for (int s = 0; s < NP / 2; ++s) *reinterpret_cast<unsigned long long*>(sm.entry[q][s][tid]) = h[s].v;
      if (q == tiles - 1) break;
      float uc[kTile], dc[kTile];
#pragma unroll
      for (int i = 0; i < kTile; ++i) {
        uc[i] = bf16_at(up + (tb + q * kTile + i) * p.u_s);
        dc[i] = bf16_at(dp + (tb + q * kTile + i) * p.dt_s);
      }
#pragma unroll
      for (int i = 0; i < kTile; ++i) {
        float dt = dc[i] + bias, slope;
        if (p.softplus) dt = softplus(dt, &slope);
        const float dtu = dt * uc[i];
        const F2 dt2 = f2(dt, dt), dtu2 = f2(dtu, dtu);
        F2 v[NP / 2];
        load_pairs(v, sm.bc.B[q * kTile + i], NP);
#pragma unroll
        for (int s = 0; s < NP / 2; ++s) h[s] = fma2(exp2_approx2(mul2(dt2, A2[s])), h[s], mul2(dtu2, v[s]));
      }
    }
    for (int q = tiles - 1; q >= 0; --q) {
      const int t0 = tb + q * kTile, m = min(kTile, sg.len - t0);
      float uc[kTile], dt[kTile], slope[kTile], yc[kTile], zc[kTile];
#pragma unroll
      for (int i = 0; i < kTile; ++i) {
        const bool in = i < m && ch.live;
        uc[i] = in ? bf16_at(up + (t0 + i) * p.u_s) : 0.f;
        dt[i] = in ? bf16_at(dp + (t0 + i) * p.dt_s) : 0.f;
        yc[i] = in ? bf16_at(yp + (long long)(t0 + i) * p.D) : 0.f;
        zc[i] = in && gate ? bf16_at(zp + (t0 + i) * p.z_s) : 0.f;
      }
      F2 H[kTile][NP / 2];
#pragma unroll
      for (int s = 0; s < NP / 2; ++s) h[s].v = *reinterpret_cast<const unsigned long long*>(sm.entry[q][s][tid]);
#pragma unroll
      for (int i = 0; i < kTile; ++i) {
        dt[i] += bias;
        slope[i] = 1.f;
        if (p.softplus) dt[i] = softplus(dt[i], &slope[i]);
        const float dtu = dt[i] * uc[i];
        const F2 dt2 = f2(dt[i], dt[i]), dtu2 = f2(dtu, dtu);
        F2 v[NP / 2];
        load_pairs(v, sm.bc.B[q * kTile + i], NP);
#pragma unroll
        for (int s = 0; s < NP / 2; ++s) H[i][s] = fma2(exp2_approx2(mul2(dt2, A2[s])), i ? H[i ? i - 1 : 0][s] : h[s], mul2(dtu2, v[s]));
      }
#pragma unroll
      for (int i = kTile - 1; i >= 0; --i) {
        if (i < m) {
          float dy0 = yc[i], sig = 0.f;
          if (gate) {
            sig = sigmoid_fast(zc[i]);
            dy0 *= zc[i] * sig;
          }
          const float dtu = dt[i] * uc[i];
          const F2 dt2 = f2(dt[i], dt[i]), dtu2 = f2(dtu, dtu), dy2 = f2(dy0, dy0);
          float cC[4] = {0.f, 0.f, 0.f, 0.f}, cB[4] = {0.f, 0.f, 0.f, 0.f};
          F2 v[NP / 2], t[NP / 2];
          load_pairs(v, sm.bc.C[q * kTile + i], NP);
          F2 y2 = f2(skip * uc[i], 0.f), sB = f2(0.f, 0.f), sA = f2(0.f, 0.f);
#pragma unroll
          for (int s = 0; s < NP / 2; ++s) {
            y2 = fma2(H[i][s], v[s], y2);
            g[s] = fma2(v[s], dy2, g[s]);
            t[s] = mul2(H[i][s], dy2);
          }
          channel_sum<NP>(cC, t, even, odd);
#pragma unroll
          for (int s = 0; s < NP / 2; ++s) t[s] = mul2(g[s], dtu2);
          channel_sum<NP>(cB, t, even, odd);
          load_pairs(v, sm.bc.B[q * kTile + i], NP);
#pragma unroll
          for (int s = 0; s < NP / 2; ++s) {
            sB = fma2(g[s], v[s], sB);
            g[s] = mul2(g[s], exp2_approx2(mul2(dt2, A2[s])));
            const F2 w = mul2(g[s], i ? H[i ? i - 1 : 0][s] : h[s]);
            sA = fma2(w, A2[s], sA);
            dA[s] = fma2(w, dt2, dA[s]);
          }
          const float dhB = sum2(sB);
          const float ddt = fmaf(uc[i], dhB, 0.6931471805599453f * sum2(sA)), dd = ddt * slope[i];
          dD = fmaf(dy0, uc[i], dD);
          dbias += dd;
          if (ch.live) {
            const long long at = out0 + (long long)(t0 + i) * p.D;
            p.du[at] = __float2bfloat16_rn(fmaf(dt[i], dhB, skip * dy0));
            p.ddelta[at] = __float2bfloat16_rn(dd);
            if (gate) p.dz[at] = __float2bfloat16_rn(yc[i] * sum2(y2) * sig * (1.f + zc[i] * (1.f - sig)));
          }
          // rows of the accumulators = states, the four lanes of a row hold two column groups each: of the four sums
          // (dC, dB of states < 8 and >= 8) each lane ends with one
          const bool o1 = lane & 1, o2 = lane & 2;
          const float c0 = cC[0] + cC[1], c1 = cC[2] + cC[3], b0 = cB[0] + cB[1], b1 = cB[2] + cB[3];
          const float k0 = (o1 ? b0 : c0) + __shfl_xor_sync(0xffffffffu, o1 ? c0 : b0, 1);
          const float k1 = (o1 ? b1 : c1) + __shfl_xor_sync(0xffffffffu, o1 ? c1 : b1, 1);
          const float r = (o2 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, o2 ? k0 : k1, 2);
          sm.red[warp][q * kTile + i][o1][(lane >> 2) + (o2 ? 8 : 0)] = r;
        }
      }
    }
    __syncthreads();
    const int per = 2 * p.N;
    float* part = p.part_bc + ((size_t)cb * p.rows + sg.row0 + tb) * per;
    for (int e = tid; e < n * per; e += kSscanThreads) {
      const int t = e / per, w = e % per, which = w / p.N, st = w - which * p.N;
      float r = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) r += sm.red[k][t][which][st];
      part[e] = r;
    }
  }
  if (!ch.live) return;
  if (p.dh0 && sg.j == 0) store_user_state<NP>(g, p.dh0 + (size_t)sg.seq * p.D * p.N, p, d);
  float* par = p.part_par + (size_t)seg * (p.N + 2) * p.D;
  store_state<NP>(dA, par, p, d);
  par[(size_t)p.N * p.D + d] = dD;
  par[(size_t)(p.N + 1) * p.D + d] = dbias;
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
    k_sscan_rmap<NP><<<grid, kSscanThreads, 0, s>>>(p, blocks);
    const long long n = (long long)p.seqs * p.N * p.D;
    k_sscan_rcompose<<<int((n + 255) / 256), 256, 0, s>>>(p);
  }
  const int smem = int(sizeof(BwdSmem<NP>));
  cudaError_t e = cudaFuncSetAttribute(k_sscan_bwd<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_sscan_bwd<NP><<<grid, kSscanThreads, smem, s>>>(p, blocks);
  const long long n = p.rows * p.G * 2 * p.N;
  k_sscan_sum_bc<<<int((n + 255) / 256), 256, 0, s>>>(p, blocks / p.G);
  k_sscan_sum_par<<<dim3((p.D + 31) / 32, p.N + 2), dim3(32, 8), 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sscan_bwd(const SscanParams& p, cudaStream_t s) { return p.N <= 8 ? run<8>(p, s) : run<16>(p, s); }

}  // namespace gdn
