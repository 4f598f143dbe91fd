// RMS norm and position rotation of query and key heads, in one pass, with its gradient; and the same with the rotated keys and
// the values written into a paged cache.
//
// Per token at position p and head: n = x rsqrt(mean(x^2) + eps) w, then the first `rotary` channels of n in pairs (a, b), the
// i-th turned by the angle p f_i: a' = a cos - b sin, b' = b cos + a sin. Pairs are (i, i + rotary/2), or (2i, 2i + 1).
// Backward: the turn undone on dy, then the norm's gradient (n's statistics are recomputed from x), dw summed over all tokens and
// heads: per lane over its rows, over the block's warps and then over the blocks in a fixed order.
//
// Angles: p f reaches thousands of turns, of which fp32 keeps too little. The turns per position f / 2 pi are held as a 64-bit
// fraction of a turn; its product with p modulo one turn is a few integer instructions and exact to 2^-31 turns wherever the text
// is, and the remainder, in half a turn to either side, is what the sine unit is exact for (its error, 2^-20.9, is far below
// a bf16 rounding). A token's angles serve all of its heads.
//
// Memory bound: a head's row is one 16-byte piece a lane (two heads of 128 channels a warp), four of them requested together.
// A warp takes a token; calls of few tokens share a token's heads among several warps.
#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8, kAhead = 4;

// f / 2 pi modulo 1, in units of 2^-64: the 24-bit significand times 2^66 / 2 pi, shifted to its place.
__device__ __forceinline__ unsigned long long turns_per_position(float f) {
  constexpr unsigned long long kInv = 11743562013128004906ull;  // round(2^66 / (2 pi))
  const uint32_t u = __float_as_uint(f);
  const int e = int((u >> 23) & 255);
  const unsigned long long m = e ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;
  // f = m 2^(max(e,1) - 150); the product m kInv is in units of 2^(max(e,1) - 150 - 66) turns
  const unsigned long long hi = __umul64hi(m, kInv), lo = m * kInv;
  const int right = 152 - max(e, 1);  // to units of 2^-64
  unsigned long long r;
  if (right >= 128 || e == 255)
    r = 0;
  else if (right >= 64)
    r = hi >> (right - 64);
  else if (right > 0)
    r = (lo >> right) | (hi << (64 - right));
  else
    r = -right < 64 ? lo << -right : 0;
  return u >> 31 ? 0ull - r : r;
}

// cos and sin of the angle of position p.
__device__ __forceinline__ void cos_sin(unsigned long long f, int p, float* c, float* s) {
  const uint32_t lo = uint32_t(f), hi = uint32_t(f >> 32), turn = uint32_t(p) * hi + __umulhi(uint32_t(p), lo) - (p < 0 ? lo : 0u);
  const float a = float(int(turn)) * (6.283185307179586f / 4294967296.f);
  *c = __cosf(a);
  *s = __sinf(a);
}

__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// A lane's share of a head: channels 8 sub .. 8 sub + 7.
template <int D, bool kPairs>
struct Turn {
  static constexpr int kN = kPairs ? 4 : 8;  // angles of a lane
  unsigned long long f[kN];
  float c[kN], s[kN];
  bool rot;
  int partner;  // lane that holds the other halves of the pairs
  __device__ __forceinline__ Turn(const RopeParams& p, int lane) {
    const int sub = lane % (D / 8), half = p.rotary / 2;
    rot = sub * 8 < p.rotary;
    const bool first = sub * 8 < half;
    partner = kPairs || !rot ? lane : lane + (first ? half / 8 : -half / 8);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = kPairs ? sub * 4 + i : sub * 8 + i - (first ? 0 : half);
      f[i] = rot ? turns_per_position(p.inv_freq[at]) : 0;
      if (!kPairs && first) f[i] = 0 - f[i];  // a' = a cos + b sin(-angle)
    }
  }
  __device__ __forceinline__ void at(int pos) {
#pragma unroll
    for (int i = 0; i < kN; ++i) cos_sin(f[i], pos, &c[i], &s[i]);
  }
  // In place; kBack: the inverse turn.
  template <bool kBack>
  __device__ __forceinline__ void apply(float* x) const {
    if (kPairs) {
      if (!rot) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1], sn = kBack ? -s[i] : s[i];
        x[2 * i] = a * c[i] - b * sn;
        x[2 * i + 1] = b * c[i] + a * sn;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_sync(0xffffffffu, x[i], partner), sn = kBack ? -s[i % kN] : s[i % kN];
        if (rot) x[i] = x[i] * c[i % kN] + other * sn;
      }
    }
  }
};

// Sum over the lanes of a head.
template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int d = D / 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

struct Token {
  int pos;
  long long cache_row;  // where its key and value go, or -1
  bool live;            // false: padding
};

// Sequence of `row`, then its position and place in the cache.
__device__ __forceinline__ Token token_of(const RopeParams& p, long long row, bool report) {
  int n, t, len;
  if (p.cu) {
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= row) lo = mid; else hi = mid;
    }
    n = lo;
    t = int(row) - p.cu[n];
    len = p.cu[n + 1] - p.cu[n];
  } else {
    n = int(row / p.T);
    t = int(row - (long long)n * p.T);
    len = p.T;
  }
  Token k{p.positions ? p.positions[row] : t, -1, true};
  if (!p.lengths) return k;
  const int total = p.lengths[n];
  if (total <= 0) return {0, -1, false};
  const int pos = total - len + t;
  bool ok = total >= len && pos / p.page < p.width;
  if (ok) {
    const int page = p.table[(long long)n * p.width + pos / p.page];
    ok = page >= 0 && page < p.pages;
    k.cache_row = (long long)page * p.page + pos % p.page;
  }
  k.pos = pos;
  if (!ok) {
    if (report && p.status) atomicCAS(p.status, 0, kDevGateRange);
    return {0, -1, false};
  }
  return k;
}

}  // namespace

// Items are (token, chunk of its passes): a pass is as many heads of q, then k, then (store) v as a warp holds.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32) k_rope_fwd(const RopeParams p, int chunks, int per) {
  wait_for_previous();
  constexpr int kHeads = 256 / D;
  const int lane = threadIdx.x & 31, sub = lane % (D / 8), which = lane / (D / 8);
  const bool norm = p.qw != nullptr;
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wq[i] = norm ? p.qw[sub * 8 + i] : 1.f;
    wk[i] = norm ? p.kw[sub * 8 + i] : 1.f;
  }
  Turn<D, kPairs> turn(p, lane);
  const int pq = (p.H + kHeads - 1) / kHeads, pk = (p.Hk + kHeads - 1) / kHeads, passes = pq + pk * (p.lengths ? 2 : 1);
  const long long items = p.rows * chunks, step = (long long)gridDim.x * kWarps;
  for (long long it = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items; it += step) {
    const long long row = it / chunks;
    const int from = int(it - row * chunks) * per, to = min(passes, from + per);
    const Token tk = token_of(p, row, lane == 0);
    turn.at(tk.pos);
    for (int p0 = from; p0 < to; p0 += kAhead) {
      uint4 in[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int ps = p0 + a;
        const int kind = ps < pq ? 0 : ps < pq + pk ? 1 : 2, hh = (ps - (kind == 0 ? 0 : kind == 1 ? pq : pq + pk)) * kHeads + which;
        const __nv_bfloat16* src = kind == 0 ? p.q + row * p.q_s : kind == 1 ? p.k + row * p.k_s : p.v + row * p.v_s;
        in[a] = make_uint4(0, 0, 0, 0);
        if (ps < to && hh < (kind ? p.Hk : p.H)) in[a] = *reinterpret_cast<const uint4*>(src + hh * D + sub * 8);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int ps = p0 + a;
        if (ps >= to) break;
        const int kind = ps < pq ? 0 : ps < pq + pk ? 1 : 2, hh = (ps - (kind == 0 ? 0 : kind == 1 ? pq : pq + pk)) * kHeads + which;
        const bool there = hh < (kind ? p.Hk : p.H);
        const long long cached = tk.cache_row < 0 ? -1 : (tk.cache_row * p.Hk + hh) * D + sub * 8;
        if (kind == 2) {
          if (there && cached >= 0) *reinterpret_cast<uint4*>(p.vc + cached) = in[a];
          continue;
        }
        float x[8];
        unpack8(in[a], x);
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
          const float rstd = rsqrtf(fmaf(head_sum<D>(ss), 1.f / D, p.eps));
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * rstd * (kind ? wk[i] : wq[i]);
        }
        turn.template apply<false>(x);
        const uint4 y = tk.live ? pack8(x) : make_uint4(0, 0, 0, 0);
        if (!there) continue;
        if (kind == 0) {
          *reinterpret_cast<uint4*>(p.qo + (row * p.H + hh) * D + sub * 8) = y;
        } else {
          *reinterpret_cast<uint4*>(p.ko + (row * p.Hk + hh) * D + sub * 8) = y;
          if (cached >= 0) *reinterpret_cast<uint4*>(p.kc + cached) = y;
        }
      }
    }
  }
}

template <int D, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32) k_rope_bwd(const RopeParams p) {
  wait_for_previous();
  constexpr int kHeads = 256 / D, kTwo = 2;
  __shared__ float part[kWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % (D / 8), which = lane / (D / 8);
  const bool norm = p.qw != nullptr;
  Turn<D, kPairs> turn(p, lane);
  float dw[2][8] = {};
  float w[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[0][i] = norm ? p.qw[sub * 8 + i] : 1.f;
    w[1][i] = norm ? p.kw[sub * 8 + i] : 1.f;
  }
  const long long step = (long long)gridDim.x * kWarps;
  for (long long row = (long long)blockIdx.x * kWarps + warp; row < p.rows; row += step) {
    turn.at(token_of(p, row, false).pos);
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int heads = kind ? p.Hk : p.H;
      const __nv_bfloat16 *x_ = (kind ? p.k + row * p.k_s : p.q + row * p.q_s) + sub * 8, *dy_ = (kind ? p.dko : p.dqo) + row * heads * D + sub * 8;
      __nv_bfloat16* dx_ = (kind ? p.dk : p.dq) + row * heads * D + sub * 8;
      for (int h0 = 0; h0 < heads; h0 += kHeads * kTwo) {
        uint4 xin[kTwo], din[kTwo];
#pragma unroll
        for (int a = 0; a < kTwo; ++a) {
          const int hh = h0 + a * kHeads + which;
          xin[a] = din[a] = make_uint4(0, 0, 0, 0);
          if (hh < heads) {
            din[a] = *reinterpret_cast<const uint4*>(dy_ + hh * D);
            if (norm) xin[a] = *reinterpret_cast<const uint4*>(x_ + hh * D);
          }
        }
#pragma unroll
        for (int a = 0; a < kTwo; ++a) {
          const int hh = h0 + a * kHeads + which;
          float x[8], d[8];
          unpack8(din[a], d);
          turn.template apply<true>(d);
          if (norm) {
            unpack8(xin[a], x);
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            const float rstd = rsqrtf(fmaf(head_sum<D>(ss), 1.f / D, p.eps));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] *= rstd;
              dw[kind][i] = fmaf(d[i], x[i], dw[kind][i]);  // zero where the head does not exist
              d[i] *= w[kind][i];
              dot = fmaf(d[i], x[i], dot);
            }
            const float mean = head_sum<D>(dot) * (1.f / D);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = rstd * (d[i] - x[i] * mean);
          }
          if (hh < heads) *reinterpret_cast<uint4*>(dx_ + hh * D) = pack8(d);
        }
      }
    }
  }
  if (!norm) return;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = dw[kind][i];
#pragma unroll
      for (int d = D / 8; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
      if (which == 0) part[warp][kind][sub * 8 + i] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) v += part[j][i / D][i % D];
    p.part[(long long)blockIdx.x * 2 * D + i] = v;
  }
}

// Weight gradients: the blocks' partial sums, 32 columns a block, rows strided over 32 warps and then added in order.
template <int D>
__global__ void __launch_bounds__(1024) k_rope_dw(const RopeParams p, int blocks) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  wait_for_previous();
  float v = 0.f;
  for (int r = warp; r < blocks; r += 32) v += p.part[(long long)r * 2 * D + col];
  acc[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += acc[i][lane];
    (col < D ? p.dqw : p.dkw - D)[col] = s;
  }
}

namespace {
constexpr int kBwdBlocks = 152 * 3;

template <int D, bool kPairs>
cudaError_t fwd(const RopeParams& p, cudaStream_t s) {
  constexpr int kHeads = 256 / D;
  const int passes = (p.H + kHeads - 1) / kHeads + (p.Hk + kHeads - 1) / kHeads * (p.lengths ? 2 : 1);
  // a token to a warp, its passes shared among more while there are fewer warps than the SMs hold
  const long long room = (long long)p.sms * 16;
  int chunks = 1;
  if (p.rows < room) chunks = int(room / p.rows < passes ? room / p.rows : passes);
  const int per = (passes + chunks - 1) / chunks;
  chunks = (passes + per - 1) / per;
  const long long want = (p.rows * chunks + kWarps - 1) / kWarps, most = (long long)p.sms * 8;
  return launch_after(k_rope_fwd<D, kPairs>, dim3(unsigned(want < most ? want : most)), dim3(kWarps * 32), 0, s, p, chunks, per);
}

template <int D, bool kPairs>
cudaError_t bwd(const RopeParams& p, cudaStream_t s) {
  const long long want = (p.rows + kWarps - 1) / kWarps;
  const int blocks = int(want < kBwdBlocks ? want : kBwdBlocks);
  cudaError_t e = launch_after(k_rope_bwd<D, kPairs>, dim3(blocks), dim3(kWarps * 32), 0, s, p);
  if (e == cudaSuccess && p.qw) e = launch_after(k_rope_dw<D>, dim3(2 * D / 32), dim3(1024), 0, s, p, blocks);
  return e;
}
}  // namespace

int rope_bwd_blocks() { return kBwdBlocks; }
cudaError_t launch_rope_fwd(const RopeParams& p, int D, cudaStream_t s) {
  if (D == 128) return p.interleaved ? fwd<128, true>(p, s) : fwd<128, false>(p, s);
  return p.interleaved ? fwd<64, true>(p, s) : fwd<64, false>(p, s);
}
cudaError_t launch_rope_bwd(const RopeParams& p, int D, cudaStream_t s) {
  if (D == 128) return p.interleaved ? bwd<128, true>(p, s) : bwd<128, false>(p, s);
  return p.interleaved ? bwd<64, true>(p, s) : bwd<64, false>(p, s);
}

}  // namespace gdn
