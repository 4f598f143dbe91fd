// Single-token forms: one new token per batch row, states updated in place. All of them read and write a state that
// is far larger than the token's vectors and do a few operations per value of it, so HBM bounds a large batch and the
// launch a small one; every state element is read once and written once, in 16-byte pieces where its layout allows.
//
//   convolution  z = b + sum_i w_i x[t - (W-1-i) d],  y = silu(z);  the state holds the last (W-1) d inputs.
//   delta rule   S' = exp(g) S,  d = b (v - S'^T k),  S = S' + k d^T,  o = scale S^T q = scale (S'^T q + (q.k) d):
//                both products with S' come out of one pass, so the state is read before one barrier and written after it.
//   scan         h = exp(dt A) h + dt u B,  y = (C.h + D u) silu(z).
#include <algorithm>

#include "block_ops.cuh"
#include "gdn.h"

namespace gdn {
namespace {

// State slot of batch row b, or -1 for a padding row (or an index outside the pool, which is recorded).
__device__ __forceinline__ int slot_of(const int* index, int b, int slots, int* status) {
  if (!index) return b;
  const int i = __ldg(index + b);
  if (i >= slots) {
    if (status && threadIdx.x == 0) atomicCAS(status, 0, GDN_ERANGE);
    return -1;
  }
  return i;
}

// ------------------------------------------------------------------ short convolution

// Four channels per thread: the weights stay in registers while the block walks its batch rows. Latency bounds it: the state
// of a serving batch (250 of 320 rows x 6144 channels x 3: 12 MB) stays in L2, and a thread has one row's loads in flight.
// 4.3 us for those 22 MB of reads and writes (5.1 TB/s), 1.4 us for one row.
template <int W>
__global__ void __launch_bounds__(128) k_conv_step(ConvStepParams p) {
  wait_for_previous();
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
  const bool live = c < p.C;
  float w[4][W], bias[4];
  if (live) {
    // 4 W consecutive floats, 16-byte aligned for an aligned weight
    if (p.vec_w) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(p.w + (size_t)c * W) + i);
        w[(4 * i) / W][(4 * i) % W] = q.x, w[(4 * i + 1) / W][(4 * i + 1) % W] = q.y;
        w[(4 * i + 2) / W][(4 * i + 2) % W] = q.z, w[(4 * i + 3) / W][(4 * i + 3) % W] = q.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < W; ++i) w[e][i] = __ldg(p.w + (size_t)(c + e) * W + i);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) bias[e] = p.bias ? __ldg(p.bias + c + e) : 0.f;
  }
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int slot = slot_of(p.index, b, p.slots, p.status);
    if (!live) continue;
    uint2* y = reinterpret_cast<uint2*>(p.y + (size_t)b * p.C + c);
    if (slot < 0) {
      *y = make_uint2(0, 0);
      continue;
    }
    const uint2 xu = __ldg(reinterpret_cast<const uint2*>(p.x + (size_t)b * p.x_stride + c));
    uint2* st = reinterpret_cast<uint2*>(p.state + (size_t)slot * p.HW * p.C + c);
    const size_t row = size_t(p.C) / 4;
    float z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = bias[e];
    auto tap = [&](const uint2& u, int i) {
      z[0] = fmaf(bf16_lo(u.x), w[0][i], z[0]);
      z[1] = fmaf(bf16_hi(u.x), w[1][i], z[1]);
      z[2] = fmaf(bf16_lo(u.y), w[2][i], z[2]);
      z[3] = fmaf(bf16_hi(u.y), w[3][i], z[3]);
    };
    if (p.dil == 1) {
      uint2 h[W];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) h[i] = st[i * row];
      h[W - 1] = xu;
#pragma unroll
      for (int i = 0; i < W; ++i) tap(h[i], i);
#pragma unroll
      for (int i = 0; i < W - 1; ++i) st[i * row] = h[i + 1];
    } else {
      // oldest row first: row j moves to j - 1; rows that are multiples of the dilation are taps
#pragma unroll
      for (int i = 0; i < W - 1; ++i) tap(st[(size_t)i * p.dil * row], i);
      tap(xu, W - 1);
      for (int j = 0; j + 1 < p.HW; ++j) st[j * row] = st[(j + 1) * row];
      if (p.HW > 0) st[(size_t)(p.HW - 1) * row] = xu;
    }
    if (p.silu)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] *= sigmoid_fast(z[e]);
    *y = make_uint2(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]));
  }
}

// The last HW inputs of every sequence (its halo's, or zeros, where it is shorter): what a prompt leaves for the step.
__global__ void __launch_bounds__(128) k_conv_state(ConvStateParams p) {
  const int cblocks = (p.C / 8 + 127) / 128;
  const int c = (blockIdx.x % cblocks * 128 + threadIdx.x) * 8;
  const int nj = blockIdx.x / cblocks, n = nj / p.HW, j = nj % p.HW;
  if (c >= p.C) return;
  const long long t0 = p.cu ? p.cu[n] : (long long)n * p.T, t1 = p.cu ? p.cu[n + 1] : t0 + p.T;
  const long long t = t1 - p.HW + j;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (t >= t0)
    v = __ldg(reinterpret_cast<const uint4*>(p.x + t * p.C + c));
  else if (p.halo)
    v = __ldg(reinterpret_cast<const uint4*>(p.halo + ((long long)n * p.HW + (p.HW + (t - t0))) * p.C + c));
  *reinterpret_cast<uint4*>(p.state + ((long long)n * p.HW + j) * p.C + c) = v;
}

// ------------------------------------------------------------------ delta rule

// One CTA per (row, head, 32 of the 128 value columns): a thread holds 4 columns of 4 key rows in registers from their load to
// their store; each load instruction of a warp covers four 128-byte lines. (64 and 128 columns a CTA: within 3% on large
// batches, fewer CTAs on small ones.) The state is stored with the streaming hint, so that a large pool passes through L2
// without pushing out what is still to be read: 42.0 -> 39.9 us for 105 rows x 16 heads, 220 MB. HBM bounds it: scalar gates,
// 105 rows x 16 heads (and 15 of padding), 37.3 us for 221 MB (5.9 TB/s, 87% of the copy rate); per-channel gate logits, 48
// rows x 32 heads, 31.5 us for 204 MB (6.5 TB/s, 95%); one row 2.2 us.
constexpr int kVSplit = 4;

__global__ void __launch_bounds__(256) k_delta_step(DeltaStepParams p) {
  constexpr int kCols = kD / kVSplit, kLanes = kCols / 4, kRows = 8 * (32 / kLanes), kPer = kD / kRows;  // lanes a row, rows of a pass, passes
  __shared__ float qs[kD], ks[kD], dec[kD], qk_s;
  __shared__ float4 red[2][8][kLanes];
  wait_for_previous();
  const int vt = blockIdx.x % kVSplit, h = (blockIdx.x / kVSplit) % p.H;
  const int b = blockIdx.x / (kVSplit * p.H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = slot_of(p.index, b, p.slots, p.status);
  __nv_bfloat16* o = p.o + ((size_t)b * p.H + h) * kD + vt * kCols;
  if (slot < 0) {
    if (tid < kCols / 2) reinterpret_cast<uint32_t*>(o)[tid] = 0;
    return;
  }
  const int cg = lane & (kLanes - 1), rg = warp * (32 / kLanes) + lane / kLanes;  // column group, key row modulo kRows
  float4* S = reinterpret_cast<float4*>(p.state + (((size_t)slot * p.H + h) * kD) * kD + vt * kCols) + cg;
  float4 st[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) st[i] = S[(size_t)(rg + kRows * i) * (kD / 4)];

  const int hk = h / p.group;
  if (warp == 0) {
    const uint2 qu = *reinterpret_cast<const uint2*>(p.q + (size_t)b * p.q_stride + hk * kD + lane * 4);
    const uint2 ku = *reinterpret_cast<const uint2*>(p.k + (size_t)b * p.k_stride + hk * kD + lane * 4);
    float q[4] = {bf16_lo(qu.x), bf16_hi(qu.x), bf16_lo(qu.y), bf16_hi(qu.y)};
    float k[4] = {bf16_lo(ku.x), bf16_hi(ku.x), bf16_lo(ku.y), bf16_hi(ku.y)};
    float qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      qq = fmaf(q[e], q[e], qq);
      kk = fmaf(k[e], k[e], kk);
      qk = fmaf(q[e], k[e], qk);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      qq += __shfl_xor_sync(0xffffffffu, qq, m);
      kk += __shfl_xor_sync(0xffffffffu, kk, m);
      qk += __shfl_xor_sync(0xffffffffu, qk, m);
    }
    const float rq = p.l2norm ? rsqrtf(qq + 1e-6f) : 1.f, rk = p.l2norm ? rsqrtf(kk + 1e-6f) : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      qs[lane * 4 + e] = q[e] * rq;
      ks[lane * 4 + e] = k[e] * rk;
    }
    if (lane == 0) qk_s = qk * rq * rk;
  } else if (warp >= 4) {
    const int i = tid - 128;
    float g;
    if (!p.kda) {
      g = __ldg(p.g + (size_t)b * p.H + h);
    } else {
      g = __ldg(p.g + ((size_t)b * p.H + h) * kD + i);
      if (p.gate_act) g = p.lower_bound * sigmoid_fast(expf(__ldg(p.A_log + h)) * (g + __ldg(p.dt_bias + h * kD + i)));
    }
    dec[i] = exp2_approx(g * kLog2e);
  }
  __syncthreads();
  float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = rg + kRows * i;
    const float d = dec[r], kr = ks[r], qr = qs[r];
    st[i].x *= d, st[i].y *= d, st[i].z *= d, st[i].w *= d;
    pk.x = fmaf(kr, st[i].x, pk.x), pk.y = fmaf(kr, st[i].y, pk.y), pk.z = fmaf(kr, st[i].z, pk.z), pk.w = fmaf(kr, st[i].w, pk.w);
    pq.x = fmaf(qr, st[i].x, pq.x), pq.y = fmaf(qr, st[i].y, pq.y), pq.z = fmaf(qr, st[i].z, pq.z), pq.w = fmaf(qr, st[i].w, pq.w);
  }
#pragma unroll
  for (int m = kLanes; m <= 16; m <<= 1) {
    pk.x += __shfl_xor_sync(0xffffffffu, pk.x, m), pk.y += __shfl_xor_sync(0xffffffffu, pk.y, m);
    pk.z += __shfl_xor_sync(0xffffffffu, pk.z, m), pk.w += __shfl_xor_sync(0xffffffffu, pk.w, m);
    pq.x += __shfl_xor_sync(0xffffffffu, pq.x, m), pq.y += __shfl_xor_sync(0xffffffffu, pq.y, m);
    pq.z += __shfl_xor_sync(0xffffffffu, pq.z, m), pq.w += __shfl_xor_sync(0xffffffffu, pq.w, m);
  }
  if (lane < kLanes) {
    red[0][warp][cg] = pk;
    red[1][warp][cg] = pq;
  }
  __syncthreads();
  float4 a = red[0][0][cg];
#pragma unroll
  for (int w = 1; w < 8; ++w) {
    const float4 t = red[0][w][cg];
    a.x += t.x, a.y += t.y, a.z += t.z, a.w += t.w;
  }
  float beta = __bfloat162float(p.beta[(size_t)b * p.H + h]);
  if (p.beta_sigmoid) beta = sigmoid_fast(beta);
  const uint2 vu = *reinterpret_cast<const uint2*>(p.v + (size_t)b * p.v_stride + h * kD + vt * kCols + cg * 4);
  const float4 dl = make_float4(beta * (bf16_lo(vu.x) - a.x), beta * (bf16_hi(vu.x) - a.y), beta * (bf16_lo(vu.y) - a.z), beta * (bf16_hi(vu.y) - a.w));
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float kr = ks[rg + kRows * i];
    st[i].x = fmaf(kr, dl.x, st[i].x), st[i].y = fmaf(kr, dl.y, st[i].y), st[i].z = fmaf(kr, dl.z, st[i].z), st[i].w = fmaf(kr, dl.w, st[i].w);
    __stcs(S + (size_t)(rg + kRows * i) * (kD / 4), st[i]);
  }
  if (tid < kLanes) {
    float4 c = red[1][0][cg];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float4 t = red[1][w][cg];
      c.x += t.x, c.y += t.y, c.z += t.z, c.w += t.w;
    }
    const float qk = qk_s, sc = p.scale;
    reinterpret_cast<uint2*>(o)[cg] = make_uint2(pack_bf16(sc * fmaf(qk, dl.x, c.x), sc * fmaf(qk, dl.y, c.y)),
                                                 pack_bf16(sc * fmaf(qk, dl.z, c.z), sc * fmaf(qk, dl.w, c.w)));
  }
}

// ------------------------------------------------------------------ selective scan

// Two lanes per channel, whose quads of states take turns: a load or store instruction of a warp covers whole sectors. A block
// walks its channels over several batch rows: A, D and the bias are read once, a row's loads are in flight while the one
// before it is computed, and its slot is known a row earlier still. VEC: the states, B and C in 16- and 8-byte pieces (N a
// multiple of 4 and these aligned; A, read once a block, comes by elements either way). 120 of 160 rows x 4096 channels x 16
// states: 12.4 us for 59 MB (4.7 TB/s). The states (42 MB) come from L2, whose latency bounds it: 80 registers leave six blocks
// of four warps an SM, each thread with one row in flight and one in hand. (Eight consecutive states a lane, and a grid of
// more blocks than fit: 14.9 us.)
template <int NQ, bool VEC>
struct SscanRow {
  int slot;
  float h[NQ][4];
  uint2 B[NQ], C[NQ];
  uint16_t u, dt, z;

  // half: the lane's turn; bc: the group's place in a row of B and C
  __device__ __forceinline__ void load(const SscanStepParams& p, int b, int slot_, int d, int half, int bc) {
    slot = slot_;
    if (slot < 0) return;
    const float* hp = p.state + ((size_t)slot * p.D + d) * p.N;
    const __nv_bfloat16 *bp = p.Bm + (size_t)b * p.b_s + bc, *cp = p.Cm + (size_t)b * p.c_s + bc;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const int n0 = (2 * j + half) * 4;
      if (VEC) {
        const bool in = n0 < p.N;
        const float4 q = in ? *reinterpret_cast<const float4*>(hp + n0) : make_float4(0.f, 0.f, 0.f, 0.f);
        h[j][0] = q.x, h[j][1] = q.y, h[j][2] = q.z, h[j][3] = q.w;
        B[j] = in ? __ldg(reinterpret_cast<const uint2*>(bp + n0)) : make_uint2(0, 0);
        C[j] = in ? __ldg(reinterpret_cast<const uint2*>(cp + n0)) : make_uint2(0, 0);
      } else {
        uint32_t v[2][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = n0 + e;
          h[j][e] = n < p.N ? hp[n] : 0.f;
          v[0][e] = n < p.N ? __ldg(reinterpret_cast<const uint16_t*>(bp) + n) : 0;
          v[1][e] = n < p.N ? __ldg(reinterpret_cast<const uint16_t*>(cp) + n) : 0;
        }
        B[j] = make_uint2(v[0][0] | v[0][1] << 16, v[0][2] | v[0][3] << 16);
        C[j] = make_uint2(v[1][0] | v[1][1] << 16, v[1][2] | v[1][3] << 16);
      }
    }
    u = __ldg(reinterpret_cast<const uint16_t*>(p.u + (size_t)b * p.u_s + d));
    dt = __ldg(reinterpret_cast<const uint16_t*>(p.delta + (size_t)b * p.dt_s + d));
    z = p.z ? __ldg(reinterpret_cast<const uint16_t*>(p.z + (size_t)b * p.z_s + d)) : uint16_t(0);
  }
};

template <int NQ, bool VEC>
__global__ void __launch_bounds__(128) k_sscan_step(SscanStepParams p) {
  wait_for_previous();
  const int i = blockIdx.x * 128 + threadIdx.x, d = i >> 1, half = i & 1;
  const bool live = d < p.D;
  const int dc = live ? d : p.D - 1;
  float a[NQ][4];
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = (2 * j + half) * 4 + e;
      a[j][e] = n < p.N ? kLog2e * __ldg(p.A + (size_t)dc * p.N + n) : 0.f;
    }
  const float bias = p.bias ? __ldg(p.bias + dc) : 0.f, skip = p.Dskip && half == 0 ? __ldg(p.Dskip + dc) : 0.f;
  const int bc = (dc / p.Dg) * p.N, stride = gridDim.y;
  auto slot_at = [&](int b) { return b < p.B ? slot_of(p.index, b, p.slots, p.status) : -1; };
  auto compute = [&](SscanRow<NQ, VEC>& row, int b) {
    float y = 0.f;
    if (row.slot >= 0) {
      const float u = bf16_lo(row.u), x = bf16_lo(row.dt) + bias, z = bf16_lo(row.z);
      const float dt = p.softplus ? softplus(x) : x, dtu = dt * u;
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t bw = e & 2 ? row.B[j].y : row.B[j].x, cw = e & 2 ? row.C[j].y : row.C[j].x;
          row.h[j][e] = fmaf(decay(dt, a[j][e]), row.h[j][e], dtu * (e & 1 ? bf16_hi(bw) : bf16_lo(bw)));
          y = fmaf(row.h[j][e], e & 1 ? bf16_hi(cw) : bf16_lo(cw), y);
        }
      y = fmaf(skip, u, y);
      if (live) {
        float* hp = p.state + ((size_t)row.slot * p.D + d) * p.N;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
          const int n0 = (2 * j + half) * 4;
          if (VEC) {
            if (n0 < p.N) *reinterpret_cast<float4*>(hp + n0) = make_float4(row.h[j][0], row.h[j][1], row.h[j][2], row.h[j][3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n0 + e < p.N) hp[n0 + e] = row.h[j][e];
          }
        }
      }
      y += __shfl_xor_sync(0xffffffffu, y, 1);
      if (p.z) y *= z * sigmoid_fast(z);
    }
    if (live && half == 0) p.y[(size_t)b * p.D + d] = __float2bfloat16_rn(y);
  };
  // two rows in turn, so that none is copied
  SscanRow<NQ, VEC> even, odd;
  int b = blockIdx.y;
  even.load(p, b, slot_at(b), dc, half, bc);
  int slot = slot_at(b + stride);
  for (; b < p.B; b += 2 * stride) {
    odd.load(p, b + stride, slot, dc, half, bc);
    slot = slot_at(b + 2 * stride);
    compute(even, b);
    if (b + stride >= p.B) break;
    even.load(p, b + 2 * stride, slot, dc, half, bc);
    slot = slot_at(b + 3 * stride);
    compute(odd, b + stride);
  }
}

}  // namespace

// How many blocks share the B rows of a step, where bx blocks cover a row and `resident` run at once: whole rounds of resident
// blocks, several rows a block. Of one to four rounds the one with the fewest rows in turn, a round's start counted as
// one. (120 rows of the scan step, bx = 64, resident = 912: 14 blocks 12.5 us; 15, a second round for a few, 16.6; 10 15.0.)
static int row_blocks(int B, int bx, int resident) {
  int best = 1;
  long long least = -1;
  for (int r = 1; r <= 4; ++r) {
    const int by = std::min({B, 65535, std::max(1, int((long long)r * resident / bx))});
    const long long rounds = ((long long)bx * by + resident - 1) / resident, cost = rounds * ((B + by - 1) / by + 1);
    if (least < 0 || cost < least) least = cost, best = by;
  }
  return best;
}

cudaError_t launch_conv_step(const ConvStepParams& p, cudaStream_t s) {
  const int bx = (p.C / 4 + 127) / 128;
  const dim3 grid(bx, row_blocks(p.B, bx, p.sms * 8));
  switch (p.W) {
    case 1: return launch_after(k_conv_step<1>, grid, 128, 0, s, p);
    case 2: return launch_after(k_conv_step<2>, grid, 128, 0, s, p);
    case 3: return launch_after(k_conv_step<3>, grid, 128, 0, s, p);
    case 4: return launch_after(k_conv_step<4>, grid, 128, 0, s, p);
    case 5: return launch_after(k_conv_step<5>, grid, 128, 0, s, p);
    case 6: return launch_after(k_conv_step<6>, grid, 128, 0, s, p);
    case 7: return launch_after(k_conv_step<7>, grid, 128, 0, s, p);
    default: return launch_after(k_conv_step<8>, grid, 128, 0, s, p);
  }
}

cudaError_t launch_conv_state(const ConvStateParams& p, cudaStream_t s) {
  k_conv_state<<<(p.C / 8 + 127) / 128 * p.N * p.HW, 128, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_delta_step(const DeltaStepParams& p, cudaStream_t s) {
  return launch_after(k_delta_step, p.B * p.H * kVSplit, 256, 0, s, p);
}

template <bool VEC>
static cudaError_t run_sscan_step(const SscanStepParams& p, cudaStream_t s) {
  const int bx = (2 * p.D + 127) / 128;
  const dim3 grid(bx, row_blocks(p.B, bx, p.sms * (p.N <= 8 ? 8 : 6)));
  return p.N <= 8 ? launch_after(k_sscan_step<1, VEC>, grid, 128, 0, s, p) : launch_after(k_sscan_step<2, VEC>, grid, 128, 0, s, p);
}

cudaError_t launch_sscan_step(const SscanStepParams& p, cudaStream_t s) { return p.vec ? run_sscan_step<true>(p, s) : run_sscan_step<false>(p, s); }

}  // namespace gdn
