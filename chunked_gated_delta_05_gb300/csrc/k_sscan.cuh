// Device pieces shared by the selective scan's forward and backward kernels. A thread walks two neighbouring channels, each
// state pair packed in one 64-bit register pair: a token's B and C come out of shared memory once for both channels, four
// bytes a state, which matters because shared memory returns 128 bytes a cycle to an SM whether lanes share them or not.
#pragma once
#include "block_ops.cuh"

namespace gdn {

struct SscanSeg {
  int seq, j, nseg;     // sequence, segment within it, its segments
  int len;              // tokens of the segment
  long long row0;       // first row of the segment
  long long ck0;        // kept state of its first token
};

// Segment s of the call: computed for a dense batch, found in the offsets' tables for packed documents.
__device__ __forceinline__ SscanSeg sscan_seg(const SscanParams& p, int s) {
  SscanSeg r;
  if (!p.cu) {
    r.seq = s / p.nseg_dense;
    r.j = s - r.seq * p.nseg_dense;
    r.nseg = p.nseg_dense;
    r.row0 = (long long)r.seq * p.T + (long long)r.j * p.L;
    r.len = min(p.L, p.T - r.j * p.L);
    r.ck0 = (long long)r.seq * p.nck_dense + (long long)r.j * (p.L / kSscanBlock);
  } else {
    int lo = 0, hi = p.seqs;  // seg_base[lo] <= s < seg_base[hi]
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (__ldg(p.seg_base + m) <= s) lo = m;
      else hi = m;
    }
    const int b = __ldg(p.seg_base + lo), c0 = __ldg(p.cu + lo), c1 = __ldg(p.cu + lo + 1);
    r.seq = lo;
    r.j = s - b;
    r.nseg = __ldg(p.seg_base + lo + 1) - b;
    r.row0 = c0 + r.j * p.L;
    r.len = min(p.L, c1 - int(r.row0));
    r.ck0 = __ldg(p.ck_base + lo) + r.j * (p.L / kSscanBlock);
  }
  return r;
}

// Channel block of the call: its group, first channel and channels, and this thread's pair (channels the block lacks are
// clamped: they run along on zeros and store nothing).
struct SscanChan {
  int g, d0, chans;
  int d[2];
  bool live[2];
};
template <int CH = kSscanChans>
__device__ __forceinline__ SscanChan sscan_chan(const SscanParams& p, int cb) {
  const int bpg = (p.Dg + CH - 1) / CH;
  SscanChan c;
  c.g = cb / bpg;
  const int first = (cb - c.g * bpg) * CH;
  c.d0 = c.g * p.Dg + first;
  c.chans = min(CH, p.Dg - first);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * threadIdx.x + e;
    c.live[e] = i < c.chans;
    c.d[e] = c.d0 + min(i, c.chans - 1);
  }
  return c;
}

// TT tokens of B or C as fp32 in shared memory, [token][NP], zero past the segment's end and past N. Every thread of the CTA
// reads the same token's vector.
template <int NP, int TT>
struct BcTile {
  float v[TT][NP];
  // States 4 i .. 4 i + 3 of token t as two pairs.
  __device__ __forceinline__ void quad(F2* out, int t, int i) const {
    const float4 q = reinterpret_cast<const float4*>(v[t])[i];
    out[0] = f2(q.x, q.y);
    out[1] = f2(q.z, q.w);
  }
};
template <int NP, int TT>
struct BcRegs {
  static constexpr int kPer = TT * NP / kSscanThreads;
  uint16_t r[kPer];
  __device__ __forceinline__ void load(const __nv_bfloat16* src, long long row, int len, int N) {
    if (len >= TT && N == NP) {
      const uint16_t* from = reinterpret_cast<const uint16_t*>(src + (threadIdx.x / NP) * row + threadIdx.x % NP);
#pragma unroll
      for (int j = 0; j < kPer; ++j) r[j] = __ldg(from + j * (kSscanThreads / NP) * row);
      return;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = threadIdx.x + j * kSscanThreads, t = e / NP, n = e % NP;
      r[j] = t < len && n < N ? __ldg(reinterpret_cast<const uint16_t*>(src + t * row + n)) : uint16_t(0);
    }
  }
  __device__ __forceinline__ void store(BcTile<NP, TT>& s) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      (&s.v[0][0])[threadIdx.x + j * kSscanThreads] = __uint_as_float(uint32_t(r[j]) << 16);
    }
  }
};
// TT tokens x kSscanChans channels of a bf16 tensor in shared memory, as they are in memory, zero past the segment's
// end and the group's channels. Copied in 16-byte pieces where every piece is aligned (`vec`), else by elements.
template <int TT, int THREADS = kSscanThreads, int CH = kSscanChans, int PAD = 0>
struct ChTile {
  uint16_t v[TT][CH + PAD];
  static constexpr int kPieces = CH / 8;
  // Thread tid of THREADS. src: element (first token, first channel); row: elements between tokens; len tokens and chans channels exist.
  __device__ __forceinline__ void load(const __nv_bfloat16* src, long long row, int len, int chans, bool vec, int tid = threadIdx.x) {
    if (vec && len >= TT && chans == CH) {  // a whole tile
      const __nv_bfloat16* from = src + (tid / kPieces) * row + tid % kPieces * 8;
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&v[tid / kPieces][tid % kPieces * 8]));
#pragma unroll
      for (int j = 0; j < TT * kPieces / THREADS; ++j)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + j * (THREADS / kPieces) * (CH + PAD) * 2), "l"(from + j * (THREADS / kPieces) * row) : "memory");
    } else if (vec) {
#pragma unroll
      for (int j = 0; j < TT * kPieces / THREADS; ++j) {
        const int e = tid + j * THREADS, t = e / kPieces, c = e % kPieces * 8;
        const int bytes = t < len ? max(0, min(8, chans - c)) * 2 : 0;
        const __nv_bfloat16* from = bytes ? src + t * row + c : src;
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&v[t][c]));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
      }
    } else {
      for (int c = tid; c < CH; c += THREADS)
#pragma unroll 8
        for (int t = 0; t < TT; ++t)
          v[t][c] = t < len && c < chans ? __ldg(reinterpret_cast<const uint16_t*>(src + t * row + c)) : uint16_t(0);
    }
  }
  // Writes the tile's valid part to dst; every element must have been written to the tile before a barrier.
  __device__ __forceinline__ void store(__nv_bfloat16* dst, long long row, int len, int chans, bool vec, int tid = threadIdx.x) const {
    if (vec && len >= TT && chans == CH) {
      __nv_bfloat16* to = dst + (tid / kPieces) * row + tid % kPieces * 8;
#pragma unroll
      for (int j = 0; j < TT * kPieces / THREADS; ++j)
        *reinterpret_cast<uint4*>(to + j * (THREADS / kPieces) * row) = *reinterpret_cast<const uint4*>(&v[tid / kPieces + j * (THREADS / kPieces)][tid % kPieces * 8]);
    } else if (vec) {
#pragma unroll
      for (int j = 0; j < TT * kPieces / THREADS; ++j) {
        const int e = tid + j * THREADS, t = e / kPieces, c = e % kPieces * 8;
        if (t < len && c < chans) *reinterpret_cast<uint4*>(dst + t * row + c) = *reinterpret_cast<const uint4*>(&v[t][c]);
      }
    } else {
      for (int c = tid; c < CH; c += THREADS)
        for (int t = 0; t < TT; ++t)
          if (t < len && c < chans) reinterpret_cast<uint16_t*>(dst)[t * row + c] = v[t][c];
    }
  }
  // One channel of token t, and the thread's pair.
  __device__ __forceinline__ float one(int t, int c) const { return __uint_as_float(uint32_t(v[t][c]) << 16); }
  __device__ __forceinline__ F2 next(int t, int c) const { return f2(one(t, c), one(t + 1, c)); }  // and of the token after it
  __device__ __forceinline__ void set_next(int t, int c, F2 x) {
    float lo, hi;
    unf2(x, &lo, &hi);
    const uint32_t u = pack_bf16(lo, hi);
    v[t][c] = uint16_t(u);
    v[t + 1][c] = uint16_t(u >> 16);
  }
  __device__ __forceinline__ float2 at(int t) const {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&v[t][2 * threadIdx.x]);
    return make_float2(bf16_lo(u), bf16_hi(u));
  }
  __device__ __forceinline__ F2 pair(int t) const {
    const float2 x = at(t);
    return f2(x.x, x.y);
  }
  __device__ __forceinline__ void set(int t, float a, float b) { *reinterpret_cast<uint32_t*>(&v[t][2 * threadIdx.x]) = pack_bf16(a, b); }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// The state pairs of one channel, `apart` elements between states: the channels' own layout ([..][N][D], segment and kept
// states) or a caller's ([..][D][N]). Zero past N.
template <int NP>
__device__ __forceinline__ void load_states(F2* h, const float* s, size_t apart, int N) {
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) h[i] = f2(2 * i < N ? s[2 * i * apart] : 0.f, 2 * i + 1 < N ? s[(2 * i + 1) * apart] : 0.f);
}
template <int NP>
__device__ __forceinline__ void store_states(const F2* h, float* s, size_t apart, int N) {
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    float lo, hi;
    unf2(h[i], &lo, &hi);
    if (2 * i < N) s[2 * i * apart] = lo;
    if (2 * i + 1 < N) s[(2 * i + 1) * apart] = hi;
  }
}
// Both channels' states into a kept or segment state (`row`: its first channel's place), in 8-byte pieces where the pairs are
// aligned.
template <int NP>
__device__ __forceinline__ void store_rows(const F2 (*h)[NP / 2], float* row, const SscanParams& p, const SscanChan& c) {
  if (!p.pair) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (c.live[e]) store_states<NP>(h[e], row + c.d[e], p.D, p.N);
    return;
  }
  if (!c.live[0]) return;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    float a0, a1, b0, b1;
    unf2(h[0][i], &a0, &a1);
    unf2(h[1][i], &b0, &b1);
    if (2 * i < p.N) *reinterpret_cast<float2*>(row + (size_t)(2 * i) * p.D + c.d[0]) = make_float2(a0, b0);
    if (2 * i + 1 < p.N) *reinterpret_cast<float2*>(row + (size_t)(2 * i + 1) * p.D + c.d[0]) = make_float2(a1, b1);
  }
}

// log2(e) A of one channel (a padded state then stays 0).
template <int NP>
__device__ __forceinline__ void load_A2(F2* A2, const SscanParams& p, int d) {
  if (p.vec_A && p.N == NP) {
    const float4* a = reinterpret_cast<const float4*>(p.A + (size_t)d * NP);
#pragma unroll
    for (int i = 0; i < NP / 4; ++i) {
      const float4 q = __ldg(a + i);
      A2[2 * i] = f2(q.x, q.y);
      A2[2 * i + 1] = f2(q.z, q.w);
    }
  } else {
    load_states<NP>(A2, p.A + (size_t)d * p.N, 1, p.N);
  }
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) A2[i] = mul2(A2[i], dup2(kLog2e));
}
__device__ __forceinline__ float param(const float* v, int d) { return v ? __ldg(v + d) : 0.f; }

}  // namespace gdn
