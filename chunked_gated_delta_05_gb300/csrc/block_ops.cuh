// Parameters and device helpers of the operators around the recurrence: the block norms (k_norm.cu),
// the single-token steps (k_step.cu) and the selective scan (k_sscan*.cu).
#pragma once
#include "common.cuh"

namespace gdn {

// ------------------------------------------------------------------ device arithmetic

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_approx(1.f + exp2_approx(-kLog2e * x)); }

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1]. log1p(e) / e is a polynomial of degree 9, fitted here by exchange
// (Remez): the coefficients as written give it within 1.2e-8, rounded to fp32 within 3e-8, and fp32 arithmetic within 1.5e-7. Unlike log(1 + e) this keeps its relative precision
// for the small step sizes that softplus gives here, and unlike 2 atanh(e / (2 + e)) it needs no reciprocal.
constexpr int kLog1p = 9;
__device__ constexpr float kLog1pTerm[kLog1p + 1] = {1.f,           -0.4999990242f, 0.3332996235f,   -0.2495413302f, 0.1967593617f,
                                                     -0.1530558414f, 0.1060364124f, -0.05695940459f, 0.01985139552f, -0.003244010752f};
__device__ __forceinline__ float softplus(float x) {
  const float e = exp2_approx(-kLog2e * fabsf(x));
  float p = kLog1pTerm[kLog1p];
#pragma unroll
  for (int i = kLog1p - 1; i >= 0; --i) p = fmaf(p, e, kLog1pTerm[i]);
  return fmaf(e, p, fmaxf(x, 0.f));
}

// Pairs of fp32 in one 64-bit register pair: one instruction per two multiply-adds.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unf2(F2 a, float* lo, float* hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(a.v)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Added to the exponent of a decay: the exponential unit's results lie below the exact ones on average (measured on GB300: by
// 0.6e-8 for exponents under 0.003, by 1 to 3e-8 from there to 1, by 5e-8 above), and a recurrence compounds that over its
// memory. A shift s moves them up by 0.69 s and costs nothing: the product becomes a multiply-add. 2.4e-8 centres what lies
// between: over 28 calls of 1 to 10565 tokens the final states' error fell from 2.6e-7 (s = 1e-8) to 1.7e-7 on long ones
// and from 1.2e-6 to 7e-7 where few tokens carry an initial state on; 3.5e-8 is too much again (9e-7). What hardly decays
// (exponents under 0.003) is left 1e-8 a token too high.
constexpr float kDecayShift = 2.4e-8f;
__device__ __forceinline__ float decay(float dt, float a2) { return exp2_approx(fmaf(dt, a2, kDecayShift)); }
__device__ __forceinline__ F2 decay2(F2 dt, F2 a2) {
  float lo, hi;
  unf2(fma2(dt, a2, f2(kDecayShift, kDecayShift)), &lo, &hi);
  return f2(exp2_approx(lo), exp2_approx(hi));
}
__device__ __forceinline__ F2 dup2(float x) { return f2(x, x); }
// 1 / x, sigmoid, silu and softplus (*slope = d softplus / dx = sigmoid(x)) of both.
__device__ __forceinline__ F2 rcp2(F2 x) {
  float lo, hi;
  unf2(x, &lo, &hi);
  return f2(rcp_approx(lo), rcp_approx(hi));
}
__device__ __forceinline__ F2 sigmoid2(F2 z) {
  float lo, hi;
  unf2(mul2(z, dup2(-kLog2e)), &lo, &hi);
  return rcp2(add2(f2(exp2_approx(lo), exp2_approx(hi)), dup2(1.f)));
}
__device__ __forceinline__ F2 silu2(F2 z) { return mul2(z, sigmoid2(z)); }
__device__ __forceinline__ F2 softplus2(F2 x, F2* slope = nullptr) {
  float lo, hi;
  unf2(x, &lo, &hi);
  const F2 e = f2(exp2_approx(-kLog2e * fabsf(lo)), exp2_approx(-kLog2e * fabsf(hi)));
  F2 p = dup2(kLog1pTerm[kLog1p]);
#pragma unroll
  for (int i = kLog1p - 1; i >= 0; --i) p = fma2(p, e, dup2(kLog1pTerm[i]));
  if (slope) {
    const F2 r = rcp2(add2(e, dup2(1.f)));
    float r0, r1, s0, s1;
    unf2(r, &r0, &r1);
    unf2(mul2(e, r), &s0, &s1);
    *slope = f2(lo >= 0.f ? r0 : s0, hi >= 0.f ? r1 : s1);
  }
  return fma2(e, p, f2(fmaxf(lo, 0.f), fmaxf(hi, 0.f)));
}
__device__ __forceinline__ float sum2(F2 a) {
  float lo, hi;
  unf2(a, &lo, &hi);
  return lo + hi;
}

// ------------------------------------------------------------------ kernels behind each other

// The kernels of these operators are launched so that their launch overlaps the end of the kernel before them in the stream
// (programmatic stream serialisation): a kernel may start when the last block of the one before it has ended, ahead of its
// memory being flushed, and waits for that before it reads what that one wrote, or writes anything. (A call's later kernels may
// read the call's inputs at once: its first kernel has waited for whatever wrote them.) No kernel lets the next one
// start earlier: blocks that wait beside running ones were then packed onto few SMs, and the scan's small calls, bound by one
// block's walk, took up to twice as long (2048 channels, 256 tokens: 59 against 32 us).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Kernel kinds of the per-launch timing hook, after the recurrence's (names in api.cu).
enum BlockKernelKind {
  kKNormFwd = kKinds, kKNormBwd, kKConvStep, kKDeltaStep, kKSscanFwd, kKSscanBwd, kKSscanStep, kKAllKinds
};

// ------------------------------------------------------------------ parameter blocks

// Residual add and RMS norm before a block; gated RMS norm after it (k_norm.cu). `stream` is the
// residual stream: 0 none (x itself is normalised), 1 bf16, 2 fp32.
struct NormParams {
  long long rows;
  int width;
  float eps, scale;
  int stream_kind;
  int act;                     // gated: 1 SiLU, 2 sigmoid
  const __nv_bfloat16* x;      // [rows,width]
  const void* residual;        // [rows,width] of the stream's type, or null
  const __nv_bfloat16* gate;   // gated: [rows,width]
  const float* weight;         // [width]
  __nv_bfloat16* y;
  void* stream;                // forward: written; backward: read (the forward's, or x without a residual)
  const __nv_bfloat16* dy;
  const void* dstream;         // gradient w.r.t. the stream, its type (bf16 without a residual), or null
  __nv_bfloat16 *dx, *dgate;
  void* dresidual;             // or null
  float* part;                 // [norm_partial_rows()][width] partial weight gradients
  float* dweight;
  int sms;
};
cudaError_t launch_add_norm_fwd(const NormParams& p, cudaStream_t s);
cudaError_t launch_add_norm_bwd(const NormParams& p, cudaStream_t s);
cudaError_t launch_gated_norm_fwd(const NormParams& p, cudaStream_t s);
cudaError_t launch_gated_norm_bwd(const NormParams& p, cudaStream_t s);
constexpr int kNormMaxWidth = 16384;
// The most rows of partial weight gradients a backward writes.
int norm_partial_rows();

// Single-token steps (k_step.cu). Row b of the batch uses state slot index[b] (or b): a negative index marks a
// padding row (zero output, no state touched), one >= slots is recorded in the status word as GDN_ERANGE
// and treated the same.
struct ConvStepParams {
  int B, C, W, dil, HW, slots, silu;
  bool vec_w;                  // weight 16-byte aligned
  long long x_stride;          // elements between batch rows
  const int* index;
  const __nv_bfloat16* x;
  const float *w, *bias;
  __nv_bfloat16 *state, *y;    // [slots,HW,C], [B,C]
  int* status;
  int sms;
};
cudaError_t launch_conv_step(const ConvStepParams& p, cudaStream_t s);

struct ConvStateParams {
  int N, T, C, HW;
  const int* cu;               // device offsets [N+1], or null (dense: N rows of T tokens)
  const __nv_bfloat16 *x, *halo;
  __nv_bfloat16* state;        // [N,HW,C]
};
cudaError_t launch_conv_state(const ConvStateParams& p, cudaStream_t s);

struct DeltaStepParams {
  int B, H, group, slots;      // group: value heads per q/k head
  int kda, l2norm, beta_sigmoid, gate_act;
  float scale, lower_bound;
  long long q_stride, k_stride, v_stride;
  const int* index;
  const __nv_bfloat16 *q, *k, *v, *beta;
  const float *g, *A_log, *dt_bias;
  float* state;                // [slots,H,128,128]
  __nv_bfloat16* o;            // [B,H,128]
  int* status;
};
cudaError_t launch_delta_step(const DeltaStepParams& p, cudaStream_t s);

// Selective scan (k_sscan_fwd.cu, k_sscan_bwd.cu, k_step.cu).
constexpr int kSscanMaxN = 16;     // states per channel
constexpr int kSscanBlock = 8;     // tokens between the states a training forward keeps
constexpr int kSscanCut = 32;      // segments are multiples of this
constexpr int kSscanChans = 128;   // channels per CTA
constexpr int kSscanThreads = kSscanChans / 2;
constexpr int kSscanBwdChans = 64; // channels per CTA of the backward's main kernel

struct SscanParams {
  int T, D, N, G, Dg, seqs;    // Dg = D / G channels per group
  int nseg_dense, nck_dense;   // segments and kept states per sequence of a dense batch
  int L;                       // tokens per segment
  int segs;                    // segments of all sequences
  const int *cu, *seg_base, *ck_base;  // packed: device arrays [seqs+1] (tokens, segments, kept states), else null
  int softplus;
  bool pair;                   // neighbouring channels of a state row 8-byte aligned
  bool quad;                   // and four of them 16-byte aligned
  bool vec_A;                  // A 16-byte aligned
  bool vec, vec_out;           // u, delta, z (dy): every 8 channels of a block 16-byte aligned; the same of the outputs
  long long u_s, dt_s, z_s, b_s, c_s;  // elements between tokens
  const __nv_bfloat16 *u, *delta, *z, *Bm, *Cm;
  const float *A, *Dskip, *bias, *h0;
  __nv_bfloat16* y;            // [rows,D]
  float* final_state;          // [seqs,D,N] or null
  float* ck;                   // [kept states][N][D]: state before every kSscanBlock-th token, or null
  float* seg_state;            // [segs][N][D]: the segments' end states, then their entry states
  float* seg_dt;               // [segs][D]: sum of the step sizes
  // backward
  const __nv_bfloat16* dy;
  const float* dfinal;
  __nv_bfloat16 *du, *ddelta, *dz, *dB, *dC;
  float *dA, *dD, *dbias, *dh0;
  float* part_bc;              // [channel blocks][rows][2][N] partial dB, dC
  float* part_par;             // [segs][N+2][D] partial dA, dD, ddelta_bias
  long long rows;
};
// Channel blocks of all groups.
inline int sscan_blocks(int G, int Dg, int chans = kSscanChans) { return G * ((Dg + chans - 1) / chans); }
cudaError_t launch_sscan_fwd(const SscanParams& p, cudaStream_t s);
cudaError_t launch_sscan_bwd(const SscanParams& p, cudaStream_t s);

struct SscanStepParams {
  int B, D, N, G, Dg, slots, softplus, sms;
  bool vec;                    // N % 4 == 0 and states, B and C aligned to four of their elements
  long long u_s, dt_s, z_s, b_s, c_s;  // elements between batch rows
  const int* index;
  const __nv_bfloat16 *u, *delta, *z, *Bm, *Cm;
  const float *A, *Dskip, *bias;
  float* state;                // [slots,D,N]
  __nv_bfloat16* y;            // [B,D]
  int* status;
};
cudaError_t launch_sscan_step(const SscanStepParams& p, cudaStream_t s);

}  // namespace gdn
