// Device pieces shared by the selective scan's forward and backward kernels.
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

// Channel block of the call: group, channel and whether this thread has one (the others run along on zeros).
struct SscanChan {
  int g, d;
  int d0, chans;  // the block's first channel and how many it has
  bool live;
};
__device__ __forceinline__ SscanChan sscan_chan(const SscanParams& p, int cb) {
  const int bpg = (p.Dg + kSscanThreads - 1) / kSscanThreads;
  SscanChan c;
  c.g = cb / bpg;
  const int i = (cb - c.g * bpg) * kSscanThreads + threadIdx.x;
  c.d0 = c.g * p.Dg + (cb - c.g * bpg) * kSscanThreads;
  c.chans = min(kSscanThreads, p.Dg - (cb - c.g * bpg) * kSscanThreads);
  c.live = i < p.Dg;
  c.d = c.g * p.Dg + min(i, p.Dg - 1);
  return c;
}

// TT tokens of B and C as fp32 in shared memory, [token][NP], zero past the segment's end and past N: every thread of
// the CTA reads the same token's vectors (broadcasts).
template <int NP, int TT>
struct BcTile {
  float B[TT][NP], C[TT][NP];
};
template <int NP, int TT>
struct BcRegs {
  static constexpr int kPer = TT * NP / kSscanThreads;
  uint16_t b[kPer], c[kPer];
  __device__ __forceinline__ void load(const SscanParams& p, int g, long long row, int len, bool want_b, bool want_c) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = threadIdx.x + j * kSscanThreads, t = e / NP, n = e % NP;
      const bool in = t < len && n < p.N;
      b[j] = in && want_b ? __ldg(reinterpret_cast<const uint16_t*>(p.Bm + (row + t) * p.b_s + g * p.N + n)) : 0;
      c[j] = in && want_c ? __ldg(reinterpret_cast<const uint16_t*>(p.Cm + (row + t) * p.c_s + g * p.N + n)) : 0;
    }
  }
  __device__ __forceinline__ void store(BcTile<NP, TT>& s) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = threadIdx.x + j * kSscanThreads;
      (&s.B[0][0])[e] = __uint_as_float(uint32_t(b[j]) << 16);
      (&s.C[0][0])[e] = __uint_as_float(uint32_t(c[j]) << 16);
    }
  }
};

// TT tokens x kSscanThreads channels of a bf16 tensor in shared memory, as they are in memory, zero past the segment's
// end and the group's channels. Copied in 16-byte pieces where every piece is aligned (`vec`), else by elements.
template <int TT>
struct ChTile {
  uint16_t v[TT][kSscanThreads];
  // src: element (first token, first channel); row: elements between tokens; len tokens and chans channels exist.
  __device__ __forceinline__ void load(const __nv_bfloat16* src, long long row, int len, int chans, bool vec) {
    if (vec) {
      constexpr int kPieces = kSscanThreads / 8;
#pragma unroll
      for (int j = 0; j < TT * kPieces / kSscanThreads; ++j) {
        const int e = threadIdx.x + j * kSscanThreads, t = e / kPieces, c = e % kPieces * 8;
        const int bytes = t < len ? max(0, min(8, chans - c)) * 2 : 0;
        const __nv_bfloat16* from = bytes ? src + t * row + c : src;
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&v[t][c]));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
      }
    } else {
      const int c = threadIdx.x;
#pragma unroll 8
      for (int t = 0; t < TT; ++t)
        v[t][c] = t < len && c < chans ? __ldg(reinterpret_cast<const uint16_t*>(src + t * row + c)) : uint16_t(0);
    }
  }
  // Writes the tile's valid part to dst; every element must have been written to the tile before a barrier.
  __device__ __forceinline__ void store(__nv_bfloat16* dst, long long row, int len, int chans, bool vec) const {
    if (vec) {
      constexpr int kPieces = kSscanThreads / 8;
#pragma unroll
      for (int j = 0; j < TT * kPieces / kSscanThreads; ++j) {
        const int e = threadIdx.x + j * kSscanThreads, t = e / kPieces, c = e % kPieces * 8;
        if (t < len && c < chans) *reinterpret_cast<uint4*>(dst + t * row + c) = *reinterpret_cast<const uint4*>(&v[t][c]);
      }
    } else {
      const int c = threadIdx.x;
      for (int t = 0; t < TT; ++t)
        if (t < len && c < chans) reinterpret_cast<uint16_t*>(dst)[t * row + c] = v[t][c];
    }
  }
  __device__ __forceinline__ float at(int t) const { return __uint_as_float(uint32_t(v[t][threadIdx.x]) << 16); }
  __device__ __forceinline__ void set(int t, float x) { v[t][threadIdx.x] = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Pair j of a token's vector.
__device__ __forceinline__ void load_pairs(F2* out, const float* src, int np) {
#pragma unroll
  for (int i = 0; i < np / 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(src)[i];
    out[2 * i] = f2(v.x, v.y);
    out[2 * i + 1] = f2(v.z, v.w);
  }
}

// log2(e) A of the thread's channel, zero past N (a padded state then stays 0).
template <int NP>
__device__ __forceinline__ void load_A2(F2* A2, const SscanParams& p, int d) {
  const float* a = p.A + (size_t)d * p.N;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i)
    A2[i] = f2(2 * i < p.N ? kLog2e * __ldg(a + 2 * i) : 0.f, 2 * i + 1 < p.N ? kLog2e * __ldg(a + 2 * i + 1) : 0.f);
}

// A [..][N][D] fp32 state (segment states, kept states): consecutive channels are contiguous.
template <int NP>
__device__ __forceinline__ void load_state(F2* h, const float* s, const SscanParams& p, int d) {
#pragma unroll
  for (int i = 0; i < NP / 2; ++i)
    h[i] = f2(2 * i < p.N ? s[(size_t)(2 * i) * p.D + d] : 0.f, 2 * i + 1 < p.N ? s[(size_t)(2 * i + 1) * p.D + d] : 0.f);
}
template <int NP>
__device__ __forceinline__ void store_state(const F2* h, float* s, const SscanParams& p, int d) {
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    float lo, hi;
    unf2(h[i], &lo, &hi);
    if (2 * i < p.N) s[(size_t)(2 * i) * p.D + d] = lo;
    if (2 * i + 1 < p.N) s[(size_t)(2 * i + 1) * p.D + d] = hi;
  }
}
// A caller's [..][D][N] state.
template <int NP>
__device__ __forceinline__ void load_user_state(F2* h, const float* s, const SscanParams& p, int d) {
  const float* q = s + (size_t)d * p.N;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) h[i] = f2(2 * i < p.N ? q[2 * i] : 0.f, 2 * i + 1 < p.N ? q[2 * i + 1] : 0.f);
}
template <int NP>
__device__ __forceinline__ void store_user_state(const F2* h, float* s, const SscanParams& p, int d) {
  float* q = s + (size_t)d * p.N;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    float lo, hi;
    unf2(h[i], &lo, &hi);
    if (2 * i < p.N) q[2 * i] = lo;
    if (2 * i + 1 < p.N) q[2 * i + 1] = hi;
  }
}

}  // namespace gdn
