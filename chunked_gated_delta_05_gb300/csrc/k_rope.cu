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
// Memory bound: a head's row is 16 (or 8) lanes of eight channels, in two pieces of four whose channels are each other's partners, so
// that a turn needs no shuffles; a warp has two (or four) heads at a time, kAhead such rows of heads requested together.
// A warp takes a token; calls of few tokens share a token's heads among several warps. Arithmetic in packed pairs.
// 8192 tokens of 16 + 4 heads of 128 (84 MB): 19 us, 4.4 TB/s; the schedulers issue in 58% of the cycles. Shares of a token's heads that
// would even out the warps' walks cost more, by its angles, than they gave (21 us).
#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8, kAhead = 4, kFwdBlocks = 3, kBwdPerSm = 2;  // blocks an SM holds

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

// A lane's share of a head's row: four channels and their four partners (channel i of `a` turns with channel i of `b`), as packed
// pairs. Pieces of four channels lie at `ca` and `cb`.
struct Share {
  F2 a[2], b[2];
};

template <int D, bool kPairs>
struct Lane {
  int ca, cb;
  bool rot;                  // false: channels behind the turned ones, which stay
  unsigned long long f[4];   // turns per position
  F2 c[2], s[2];             // cosines and sines at the token's position
  __device__ __forceinline__ Lane(const RopeParams& p, int lane) {
    const int l = lane % (D / 8), half = p.rotary / 8;  // lanes that hold pairs, when those lie half the rotary width apart
    if (kPairs) {
      ca = 8 * l;
      cb = 8 * l + 4;
      rot = 8 * l < p.rotary;
    } else {
      rot = l < half;
      ca = rot ? 4 * l : p.rotary + 8 * (l - half);
      cb = rot ? 4 * (l + half) : ca + 4;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = rot ? turns_per_position(p.inv_freq[4 * l + i]) : 0;
  }
  __device__ __forceinline__ void at(int pos) {
    float x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) cos_sin(f[i], pos, &x[i], &y[i]);
    c[0] = f2(x[0], x[1]), c[1] = f2(x[2], x[3]);
    s[0] = f2(y[0], y[1]), s[1] = f2(y[2], y[3]);
  }
  // Eight channels as loaded (pieces at ca and cb) to a share and back.
  static __device__ __forceinline__ Share split(const float* x) {
    if (kPairs) return {{f2(x[0], x[2]), f2(x[4], x[6])}, {f2(x[1], x[3]), f2(x[5], x[7])}};
    return {{f2(x[0], x[1]), f2(x[2], x[3])}, {f2(x[4], x[5]), f2(x[6], x[7])}};
  }
  static __device__ __forceinline__ void join(const Share& v, float* x) {
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      unf2(v.a[i], &a[2 * i], &a[2 * i + 1]);
      unf2(v.b[i], &b[2 * i], &b[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[kPairs ? 2 * i : i] = a[i];
      x[kPairs ? 2 * i + 1 : 4 + i] = b[i];
    }
  }
  __device__ __forceinline__ Share weights(const float* w) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = w ? w[ca + i] : 1.f;
      x[4 + i] = w ? w[cb + i] : 1.f;
    }
    return split(x);
  }
  __device__ __forceinline__ void load(uint2* in, const __nv_bfloat16* row) const {
    in[0] = *reinterpret_cast<const uint2*>(row + ca);
    in[1] = *reinterpret_cast<const uint2*>(row + cb);
  }
  static __device__ __forceinline__ Share unpack(const uint2* in) {
    const uint32_t w[4] = {in[0].x, in[0].y, in[1].x, in[1].y};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
    return split(x);
  }
  static __device__ __forceinline__ void pack(const Share& v, uint2* out) {
    float x[8];
    join(v, x);
    out[0] = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    out[1] = make_uint2(pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
  __device__ __forceinline__ void store(const uint2* out, __nv_bfloat16* row) const {
    *reinterpret_cast<uint2*>(row + ca) = out[0];
    *reinterpret_cast<uint2*>(row + cb) = out[1];
  }
  // In place; kBack: the inverse turn.
  template <bool kBack>
  __device__ __forceinline__ void turn(Share* v) const {
    if (!rot) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const F2 a = v->a[i], b = v->b[i], minus = mul2(s[i], dup2(-1.f));
      v->a[i] = fma2(b, kBack ? s[i] : minus, mul2(a, c[i]));
      v->b[i] = fma2(a, kBack ? minus : s[i], mul2(b, c[i]));
    }
  }
};

// Sum over the lanes of a head of x y.
template <int D>
__device__ __forceinline__ float head_dot(const Share& x, const Share& y) {
  F2 t = mul2(x.a[0], y.a[0]);
  t = fma2(x.a[1], y.a[1], t);
  t = fma2(x.b[0], y.b[0], t);
  t = fma2(x.b[1], y.b[1], t);
  float v = sum2(t);
#pragma unroll
  for (int d = D / 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ void scale(Share* x, F2 f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) x->a[i] = mul2(x->a[i], f), x->b[i] = mul2(x->b[i], f);
}
__device__ __forceinline__ void times(Share* x, const Share& w) {
#pragma unroll
  for (int i = 0; i < 2; ++i) x->a[i] = mul2(x->a[i], w.a[i]), x->b[i] = mul2(x->b[i], w.b[i]);
}

struct Token {
  int pos;
  long long cache_row;  // where its key and value go, or -1
  bool live;            // false: padding
};

// Sequence of `row`, then its position and place in the cache.
__device__ __forceinline__ Token token_of(const RopeParams& p, int row, bool report) {
  int n, t, len;
  if (p.packed) {
    auto cu = [&](int i) { return p.cu ? p.cu[i] : p.few[i]; };
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu(mid) <= row) lo = mid; else hi = mid;
    }
    n = lo;
    t = row - cu(n);
    len = cu(n + 1) - cu(n);
  } else {
    n = int(unsigned(row) / unsigned(p.T));
    t = row - n * p.T;
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

// Heads of one kind (kKind 0: queries, 1: keys, 2: values, which are only copied) of a token, passes from .. to - 1 of as many heads
// as a warp holds.
template <int D, bool kPairs, int kKind>
__device__ __forceinline__ void rope_heads(const RopeParams& p, const Lane<D, kPairs>& ln, const Share& w, bool norm, const Token& tk, int row, int which, int from, int to) {
  constexpr int kHeads = 256 / D, kStep = kHeads * D;
  const int heads = kKind ? p.Hk : p.H;
  const __nv_bfloat16* src = (kKind == 0 ? p.q + row * p.q_s : kKind == 1 ? p.k + row * p.k_s : p.v + row * p.v_s) + which * D;
  __nv_bfloat16* dst = (kKind == 0 ? p.qo : p.ko) + (long long)row * heads * D + which * D;
  __nv_bfloat16* cache = kKind ? (kKind == 1 ? p.kc : p.vc) + tk.cache_row * heads * D + which * D : nullptr;
  const bool cached = kKind && tk.cache_row >= 0;
  for (int p0 = from; p0 < to; p0 += kAhead) {
    uint2 in[kAhead][2];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      in[a][0] = in[a][1] = make_uint2(0, 0);
      if (p0 + a < to && (p0 + a) * kHeads + which < heads) ln.load(in[a], src + (p0 + a) * kStep);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (p0 + a >= to) break;
      const int at = (p0 + a) * kStep;
      const bool there = (p0 + a) * kHeads + which < heads;
      if (kKind == 2) {
        if (there && cached) ln.store(in[a], cache + at);
        continue;
      }
      Share x = ln.unpack(in[a]);
      if (norm) {
        const float rstd = rsqrtf(fmaf(head_dot<D>(x, x), 1.f / D, p.eps));
        scale(&x, dup2(rstd));
        times(&x, w);
      }
      ln.template turn<false>(&x);
      uint2 y[2];
      ln.pack(x, y);
      if (!tk.live) y[0] = y[1] = make_uint2(0, 0);
      if (!there) continue;
      ln.store(y, dst + at);
      if (cached) ln.store(y, cache + at);
    }
  }
}

// blockIdx.y: the chunk of `per` of a token's passes (q's, then k's, then (store) v's).
template <int D, bool kPairs, bool kStore>
__global__ void __launch_bounds__(kWarps * 32, kFwdBlocks) k_rope_fwd(const __grid_constant__ RopeParams p, int per) {
  constexpr int kHeads = 256 / D;
  wait_for_previous();
  const int lane = threadIdx.x & 31, which = lane / (D / 8);
  const bool norm = p.qw != nullptr;
  Lane<D, kPairs> ln(p, lane);
  const Share wq = ln.weights(p.qw), wk = ln.weights(p.kw);
  const int pq = (p.H + kHeads - 1) / kHeads, pk = (p.Hk + kHeads - 1) / kHeads, from = blockIdx.y * per, to = from + per;
  const int step = gridDim.x * kWarps;
  for (int row = blockIdx.x * kWarps + (threadIdx.x >> 5); row < p.rows; row += step) {
    const Token tk = token_of(p, row, lane == 0);
    ln.at(tk.pos);
    rope_heads<D, kPairs, 0>(p, ln, wq, norm, tk, row, which, from, min(to, pq));
    rope_heads<D, kPairs, 1>(p, ln, wk, norm, tk, row, which, max(from - pq, 0), min(to - pq, pk));
    if (kStore) rope_heads<D, kPairs, 2>(p, ln, wk, norm, tk, row, which, max(from - pq - pk, 0), min(to - pq - pk, pk));
  }
}

// The first `q_blocks` blocks take the queries' heads, the others the keys': a token of one kind to a warp, the next group of heads
// requested before one is computed. (2 x 4096 tokens of 16 + 16 heads, forward and backward: 75 us with a warp for both kinds of
// a token, 73 without requests ahead, 69 so; 128 registers a thread, of which the compiler spills 8 to 24 bytes.)
template <int D, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32, kBwdPerSm) k_rope_bwd(const __grid_constant__ RopeParams p, int q_blocks) {
  constexpr int kHeads = 256 / D, kTogether = 4;
  __shared__ float part[kWarps][D];
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = lane / (D / 8);
  const bool keys = int(blockIdx.x) >= q_blocks;
  const int block = keys ? blockIdx.x - q_blocks : blockIdx.x, blocks = keys ? gridDim.x - q_blocks : q_blocks, heads = keys ? p.Hk : p.H;
  const __nv_bfloat16 *xs = (keys ? p.k : p.q) + which * D, *dys = (keys ? p.dko : p.dqo) + which * D;
  __nv_bfloat16* dxs = (keys ? p.dk : p.dq) + which * D;
  const long long x_s = keys ? p.k_s : p.q_s;
  const float* weight = keys ? p.kw : p.qw;
  const bool norm = weight != nullptr;
  Lane<D, kPairs> ln(p, lane);
  const Share w = ln.weights(weight);
  Share dw;
#pragma unroll
  for (int i = 0; i < 2; ++i) dw.a[i] = dw.b[i] = dup2(0.f);
  uint2 xin[kTogether][2], din[kTogether][2];
  auto fetch = [&](int row, int h0, uint2 (&xi)[kTogether][2], uint2 (&di)[kTogether][2]) {
    const __nv_bfloat16 *x_ = xs + row * x_s, *dy_ = dys + (long long)row * heads * D;
#pragma unroll
    for (int a = 0; a < kTogether; ++a) {
      const int hh = h0 + a * kHeads + which;
      xi[a][0] = xi[a][1] = di[a][0] = di[a][1] = make_uint2(0, 0);
      if (row < p.rows && hh < heads) {
        ln.load(di[a], dy_ + (h0 + a * kHeads) * D);
        if (norm) ln.load(xi[a], x_ + (h0 + a * kHeads) * D);
      }
    }
  };
  const int first = block * kWarps + warp;
  if (first < p.rows) fetch(first, 0, xin, din);
  for (int row = first; row < p.rows; row += blocks * kWarps) {
    ln.at(token_of(p, row, false).pos);
    __nv_bfloat16* dx_ = dxs + (long long)row * heads * D;
    for (int h0 = 0; h0 < heads; h0 += kHeads * kTogether) {
      uint2 xn[kTogether][2], dn[kTogether][2];
      const bool more = h0 + kHeads * kTogether < heads;
      fetch(more ? row : row + blocks * kWarps, more ? h0 + kHeads * kTogether : 0, xn, dn);
#pragma unroll
      for (int a = 0; a < kTogether; ++a) {
        const int hh = h0 + a * kHeads + which;
        if (h0 + a * kHeads >= heads) break;
        Share d = ln.unpack(din[a]);
        ln.template turn<true>(&d);
        if (norm) {
          Share x = ln.unpack(xin[a]);
          const float norm2 = fmaf(head_dot<D>(x, x), 1.f / D, p.eps), rstd = hh < heads ? rsqrtf(norm2) : 0.f;
          scale(&x, dup2(rstd));
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // zero where the head does not exist
            dw.a[i] = fma2(d.a[i], x.a[i], dw.a[i]);
            dw.b[i] = fma2(d.b[i], x.b[i], dw.b[i]);
          }
          times(&d, w);
          const F2 mean = dup2(head_dot<D>(d, x) * (-1.f / D));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            d.a[i] = fma2(x.a[i], mean, d.a[i]);
            d.b[i] = fma2(x.b[i], mean, d.b[i]);
          }
          scale(&d, dup2(rstd));
        }
        uint2 out[2];
        ln.pack(d, out);
        if (hh < heads) ln.store(out, dx_ + (h0 + a * kHeads) * D);
      }
#pragma unroll
      for (int a = 0; a < kTogether; ++a)
#pragma unroll
        for (int i = 0; i < 2; ++i) xin[a][i] = xn[a][i], din[a][i] = dn[a][i];
    }
  }
  if (!norm) return;
  float x[8];
  ln.join(dw, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int d = D / 8; d < 32; d <<= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
    if (which == 0) part[warp][(i < 4 ? ln.ca : ln.cb - 4) + i] = x[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) v += part[j][i];
    p.part[(long long)blockIdx.x * D + i] = v;
  }
}

// Weight gradients: the blocks' partial sums, 32 columns a block, rows strided over 32 warps and then added in order.
template <int D>
__global__ void __launch_bounds__(1024) k_rope_dw(const RopeParams p, int q_blocks, int blocks) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  const bool keys = col >= D;
  wait_for_previous();
  float v = 0.f;
  for (int r = (keys ? q_blocks : 0) + warp; r < (keys ? blocks : q_blocks); r += 32) v += p.part[(long long)r * D + col % D];
  acc[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += acc[i][lane];
    (keys ? p.dkw - D : p.dqw)[col] = s;
  }
}

namespace {
constexpr int kBwdBlocks = 152 * kBwdPerSm;

template <int D, bool kPairs>
cudaError_t fwd(const RopeParams& p, cudaStream_t s) {
  constexpr int kHeads = 256 / D;
  const int passes = (p.H + kHeads - 1) / kHeads + (p.Hk + kHeads - 1) / kHeads * (p.lengths ? 2 : 1);
  // a token to a warp, its passes shared among more while there are fewer warps than the SMs hold
  const long long room = (long long)p.sms * kWarps * kFwdBlocks;
  int chunks = 1;
  if (p.rows < room) chunks = int(room / p.rows < passes ? room / p.rows : passes);
  const int per = (passes + chunks - 1) / chunks;
  chunks = (passes + per - 1) / per;
  const long long want = (p.rows + kWarps - 1) / kWarps, most = (long long)p.sms * kFwdBlocks;
  const dim3 grid(unsigned(want < most ? want : most), chunks);
  return p.lengths ? launch_after(k_rope_fwd<D, kPairs, true>, grid, dim3(kWarps * 32), 0, s, p, per)
                   : launch_after(k_rope_fwd<D, kPairs, false>, grid, dim3(kWarps * 32), 0, s, p, per);
}

template <int D, bool kPairs>
cudaError_t bwd(const RopeParams& p, cudaStream_t s) {
  // blocks in proportion to the heads, at least one for either kind
  const long long want = (p.rows + kWarps - 1) / kWarps * 2;
  const int blocks = int(want < kBwdBlocks ? want : kBwdBlocks);
  int q_blocks = int((long long)blocks * p.H / (p.H + p.Hk));
  q_blocks = q_blocks < 1 ? 1 : q_blocks > blocks - 1 ? blocks - 1 : q_blocks;
  cudaError_t e = launch_after(k_rope_bwd<D, kPairs>, dim3(blocks), dim3(kWarps * 32), 0, s, p, q_blocks);
  if (e == cudaSuccess && p.qw) e = launch_after(k_rope_dw<D>, dim3(2 * D / 32), dim3(1024), 0, s, p, q_blocks, blocks);
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
