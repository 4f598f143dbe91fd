// RMS norms before and after a block.
//
// Before:  r = residual + scale x (kept in the stream's type),  y = r rstd(r) w,  rstd(r) = (mean(r^2) + eps)^(-1/2).
//   dr = dstream + rstd (dy w - xh mean(dy w xh)),  xh = r rstd;   dx = scale dr,  dresidual = dr,  dw = sum_rows dy xh.
// After:   y = x rstd(x) w act(gate), act = SiLU or sigmoid.
//   dn = dy act;  dx = rstd (dn w - xh mean(dn w xh));  dgate = dy xh w act';  dw = sum_rows dn xh.
// The backward kernels recompute rstd: sum r^2 and sum dy w r come out of the same pass over the row, so nothing but
// the stream is kept by the forward.
//
// A row is held in registers by G threads (a power of two; in the forward of wide rows, a multiple of 32) of NV vectors of VEC
// elements each: one read and one write of every tensor. All sums are fp32. Rows of widths that are no multiple of 8, or unaligned
// tensors, take the element path (VEC = 1).
//
// Bound: HBM, a few operations a byte. On GB300: residual norm of 8192 x 2048 with an fp32 stream, forward and backward, 78.5 us
// for 470 MB (6.0 TB/s, 88% of the copy rate: 31.3 + 47.2 us, the sums of the weight gradients included); gated norm of 262144 x
// 128, both, 91.8 us for 537 MB (5.9 TB/s); its forward alone at 131072 x 128, 15.7 us for 101 MB (6.4 TB/s).
#include <algorithm>
#include <initializer_list>

#include "block_ops.cuh"

namespace gdn {
namespace {

enum { kAdd = 0, kSilu = 1, kSigmoid = 2 };  // before a block, and after it by activation

// A vector of VEC elements as it is in memory: requested early, widened when it is used.
template <int VEC, typename T>
struct Raw;
template <>
struct Raw<8, __nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* src) { u = __ldg(reinterpret_cast<const uint4*>(src)); }
  __device__ __forceinline__ float operator[](int e) const {
    const uint32_t w = e < 2 ? u.x : e < 4 ? u.y : e < 6 ? u.z : u.w;
    return e & 1 ? bf16_hi(w) : bf16_lo(w);
  }
};
template <>
struct Raw<8, float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* src) {
    a = __ldg(reinterpret_cast<const float4*>(src));
    b = __ldg(reinterpret_cast<const float4*>(src) + 1);
  }
  __device__ __forceinline__ float operator[](int e) const {
    const float4 q = e < 4 ? a : b;
    return e % 4 == 0 ? q.x : e % 4 == 1 ? q.y : e % 4 == 2 ? q.z : q.w;
  }
};
template <typename T>
struct Raw<1, T> {
  T x;
  __device__ __forceinline__ void load(const T* src) { x = src[0]; }
  __device__ __forceinline__ float operator[](int) const { return float(x); }
};

// The arithmetic of the backward is written once for pairs of elements and for single ones.
template <int VEC>
struct Elems {  // 8: pairs
  using T = F2;
  static constexpr int kCount = VEC / 2;
  template <typename R>
  __device__ __forceinline__ static T of(const R& raw, int i) { return f2(raw[2 * i], raw[2 * i + 1]); }
  __device__ __forceinline__ static T dup(float x) { return dup2(x); }
  __device__ __forceinline__ static void put(float* v, int i, T x) { unf2(x, v + 2 * i, v + 2 * i + 1); }
};
template <>
struct Elems<1> {
  using T = float;
  static constexpr int kCount = 1;
  template <typename R>
  __device__ __forceinline__ static T of(const R& raw, int i) { return raw[i]; }
  __device__ __forceinline__ static T dup(float x) { return x; }
  __device__ __forceinline__ static void put(float* v, int i, T x) { v[i] = x; }
};
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sum2(float a) { return a; }
__device__ __forceinline__ float sigmoid2(float z) { return sigmoid_fast(z); }

template <int VEC>
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, const float* v) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    dst[0] = __float2bfloat16_rn(v[0]);
}
template <int VEC>
__device__ __forceinline__ void store_row(float* dst, const float* v) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    dst[0] = v[0];
  }
}
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) { return __bfloat162float(__float2bfloat16_rn(v)); }

// Sums of NS values over the G threads of a row; every thread of the block takes part. `red` (NS x 32 floats) is another
// one for every second call, so that one barrier a call is enough.
template <int NS>
__device__ __forceinline__ void row_sum(float* s, int G, float (*red)[32]) {
  const int lanes = min(G, 32);
  for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (G <= 32) return;
  const int warp = threadIdx.x >> 5, per = G >> 5, first = warp / per * per;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NS; ++i) red[i][warp] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    float t = 0.f;
    for (int w = 0; w < per; ++w) t += red[i][first + w];
    s[i] = t;
  }
}

// The activation of a gate whose sigmoid is sg.
template <int KIND>
__device__ __forceinline__ float act_of(float g, float sg) {
  return KIND == kSilu ? g * sg : sg;
}

// A row's vectors of one thread. The gated kernels hold two where a row takes one vector a thread: the next row's loads are in
// flight while this one is computed. (The residual norm, whose rows cross warps behind a barrier, was slower so: 34.7 ->
// 42.5 us forward at 8192 x 2048; a block per row hides the loads with more blocks.)
template <int KIND, int VEC, int NV, typename ST>
struct FwdRow {
  Raw<VEC, __nv_bfloat16> x[NV], gate[NV];
  Raw<VEC, ST> res[NV];
  __device__ __forceinline__ void load(const NormParams& p, long long r, int lane, int G, int units) {
    if (r >= p.rows) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = lane + j * G;
      if (u < units) {
        const long long at = r * p.width + (long long)u * VEC;
        x[j].load(p.x + at);
        if (KIND == kAdd && p.residual) res[j].load(static_cast<const ST*>(p.residual) + at);
        if (KIND != kAdd) gate[j].load(p.gate + at);
      }
    }
  }
};

template <int KIND, int VEC, int NV, int THREADS, typename ST>
__global__ void __launch_bounds__(THREADS) k_norm_fwd(NormParams p, int G) {
  constexpr bool kAhead = NV == 1 && KIND != kAdd;
  __shared__ float red[2][1][32];
  wait_for_previous();
  const bool whole = G == blockDim.x;  // else G is a power of two
  const int log = 31 - __clz(G), per_block = whole ? 1 : blockDim.x >> log, grp = whole ? 0 : threadIdx.x >> log, lane = threadIdx.x - (grp << log);
  const int units = p.width / VEC;
  const float inv = 1.f / float(p.width);
  const long long step = (long long)gridDim.x * per_block;
  int turn = 0;
  FwdRow<KIND, VEC, NV, ST> row, next;
  Raw<VEC, float> w[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (lane + j * G < units) w[j].load(p.weight + (lane + j * G) * VEC);
  if (kAhead) row.load(p, (long long)blockIdx.x * per_block + grp, lane, G, units);
  for (long long r0 = (long long)blockIdx.x * per_block; r0 < p.rows; r0 += step, turn ^= 1) {
    const long long r = r0 + grp;
    const bool live = r < p.rows;
    const long long base = r * p.width;
    if (kAhead) next.load(p, r + step, lane, G, units);
    else row.load(p, r, lane, G, units);
    float v[NV][VEC], ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = lane + j * G;
      if (live && u < units) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] = row.x[j][e];
        if (KIND == kAdd && p.residual) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[j][e] = round_to(fmaf(p.scale, v[j][e], row.res[j][e]), (const ST*)nullptr);
          store_row<VEC>(static_cast<ST*>(p.stream) + base + (long long)u * VEC, v[j]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[0] = fmaf(v[j][e], v[j][e], ss[0]);
      }
    }
    row_sum<1>(ss, G, red[turn]);
    const float rstd = rsqrtf(fmaf(ss[0], inv, p.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = lane + j * G;
      if (live && u < units) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] = v[j][e] * rstd * (KIND != kAdd ? w[j][e] * act_of<KIND>(row.gate[j][e], sigmoid_fast(row.gate[j][e])) : w[j][e]);
        store_row<VEC>(p.y + base + (long long)u * VEC, v[j]);
      }
    }
    if (kAhead) row = next;
  }
}

template <int KIND, int VEC, int NV, typename ST, bool DS>
struct BwdRow {
  Raw<VEC, __nv_bfloat16> dy[NV], gate[NV];
  Raw<VEC, ST> x[NV], ds[DS ? NV : 1];
  __device__ __forceinline__ void load(const NormParams& p, long long r, int lane, int G, int units) {
    if (r >= p.rows) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = lane + j * G;
      if (u < units) {
        const long long at = r * p.width + (long long)u * VEC;
        x[j].load(KIND == kAdd ? static_cast<const ST*>(p.stream) + at : reinterpret_cast<const ST*>(p.x) + at);
        dy[j].load(p.dy + at);
        if (KIND != kAdd) gate[j].load(p.gate + at);
        if (DS && KIND == kAdd && p.dstream) ds[j].load(static_cast<const ST*>(p.dstream) + at);
      }
    }
  }
};

// Rows of more than one vector a thread keep their weight gradients in shared memory instead of registers (and load dstream
// only when it is added), where that leaves room for another block: with an fp32 stream (8192 wide, 4096 wide: 71 -> 64, 58 ->
// 49 us for 268 MB) and with a gate (109 -> 76, 84 -> 79 us for 336 MB); with a bf16 stream it costs (8192 wide 48.8 -> 51.9).
template <int KIND, int VEC, int NV, int THREADS, typename ST>
constexpr bool kLean = VEC == 8 && NV > 1 && THREADS == 256 && (KIND != kAdd || sizeof(ST) == 4);
// Blocks an SM that the registers must allow, where the compiler's own choice was slower: four for one vector a thread (SiLU's
// gate then takes 64 instead of 79 registers: 87 -> 63 us at 262144 x 128, 107 -> 79 us at 16384 x 2048), and for gates
// four for two vectors (86 -> 79 us at 8192 x 4096) and two for four (107 -> 76 us at 4096 x 8192).
template <int KIND, int VEC, int NV, int THREADS>
constexpr int kBwdBlocks = VEC != 8 || THREADS != 256 ? 0 : NV == 1 ? 4 : KIND == kAdd ? 0 : NV == 2 ? 4 : 2;

// One pass per row; each thread keeps its columns' weight gradients (in registers, or kLean) over all rows of its group, the groups of
// the block add theirs in shared memory in a fixed order, and the block writes one row of partial sums.
template <int KIND, int VEC, int NV, int THREADS, typename ST>
__global__ void __launch_bounds__(THREADS, kBwdBlocks<KIND, VEC, NV, THREADS>) k_norm_bwd(NormParams p, int G) {
  constexpr bool kAhead = NV == 1 && KIND != kAdd, kShared = kLean<KIND, VEC, NV, THREADS, ST>;
  extern __shared__ __align__(16) float acc_s[];
  __shared__ float red[2][2][32];
  const int per_block = blockDim.x / G, lane = threadIdx.x & (G - 1), grp = threadIdx.x / G;
  const int units = p.width / VEC;
  const float inv = 1.f / float(p.width);
  const long long step = (long long)gridDim.x * per_block;
  wait_for_previous();
  using E = Elems<VEC>;
  using T = typename E::T;
  T dw[NV][E::kCount];
  // a unit's eight sums in shared memory, four and four
  auto lean = [&](int u, int half) { return reinterpret_cast<float4*>(acc_s) + half * units + u; };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int e = 0; e < E::kCount; ++e) dw[j][e] = E::dup(0.f);
    const int u = lane + j * G;
    if (kShared && u < units) *lean(u, 0) = *lean(u, 1) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  int turn = 0;
  BwdRow<KIND, VEC, NV, ST, !kShared> row, next;
  Raw<VEC, float> w[NV];
  if (kAhead && lane < units) w[0].load(p.weight + lane * VEC);
  if (kAhead) row.load(p, (long long)blockIdx.x * per_block + grp, lane, G, units);
  for (long long r0 = (long long)blockIdx.x * per_block; r0 < p.rows; r0 += step, turn ^= 1) {
    const long long r = r0 + grp;
    const bool live = r < p.rows;
    const long long base = r * p.width;
    if (kAhead) next.load(p, r + step, lane, G, units);
    else row.load(p, r, lane, G, units);
    T s2[2] = {E::dup(0.f), E::dup(0.f)}, sg[NV][E::kCount];  // sigmoid(gate), used again below
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = lane + j * G;
      if (live && u < units) {
        if (!kAhead) w[j].load(p.weight + u * VEC);
#pragma unroll
        for (int e = 0; e < E::kCount; ++e) {
          const T v = E::of(row.x[j], e);
          T dn = mul2(E::of(row.dy[j], e), E::of(w[j], e));
          if (KIND != kAdd) {
            const T g = E::of(row.gate[j], e);
            sg[j][e] = sigmoid2(g);
            dn = mul2(dn, KIND == kSilu ? mul2(g, sg[j][e]) : sg[j][e]);
          }
          s2[0] = fma2(v, v, s2[0]);
          s2[1] = fma2(dn, v, s2[1]);
        }
      }
    }
    float s[2] = {sum2(s2[0]), sum2(s2[1])};
    row_sum<2>(s, G, red[turn]);
    const float rstd = rsqrtf(fmaf(s[0], inv, p.eps));
    const float c = -s[1] * inv * rstd * rstd * rstd;  // xh mean(dn w xh) rstd = -x c
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = lane + j * G;
      if (live && u < units) {
        const long long at = base + (long long)u * VEC;
        if (!kAhead) w[j].load(p.weight + u * VEC);
        if (kShared && KIND == kAdd && p.dstream) row.ds[0].load(static_cast<const ST*>(p.dstream) + at);
        if (kShared) {
          const float4 a = *lean(u, 0), b = *lean(u, 1);
          const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < E::kCount; ++e) dw[j][e] = E::of(v, e);
        }
        float o[VEC], q[VEC];
#pragma unroll
        for (int e = 0; e < E::kCount; ++e) {
          const T one = E::dup(1.f), v = E::of(row.x[j], e), xh = mul2(v, E::dup(rstd)), dy = E::of(row.dy[j], e), dyw = mul2(dy, E::of(w[j], e));
          T dn = dy, dnw = dyw;
          if (KIND != kAdd) {
            const T a = sg[j][e], act = KIND == kSilu ? mul2(E::of(row.gate[j], e), a) : a, not_a = fma2(a, E::dup(-1.f), one);
            // act' = sg + act (1 - sg), or sg (1 - sg)
            E::put(q, e, mul2(mul2(dyw, xh), KIND == kSilu ? fma2(act, not_a, a) : mul2(a, not_a)));
            dn = mul2(dn, act);
            dnw = mul2(dnw, act);
          }
          E::put(o, e, fma2(dnw, E::dup(rstd), mul2(v, E::dup(c))));
          dw[j][e] = fma2(dn, xh, dw[j][e]);
        }
        if (kShared) {
          float v[8];
#pragma unroll
          for (int e = 0; e < E::kCount; ++e) E::put(v, e, dw[j][e]);
          *lean(u, 0) = make_float4(v[0], v[1], v[2], v[3]);
          *lean(u, 1) = make_float4(v[4], v[5], v[6], v[7]);
        }
        if (KIND == kAdd) {
          if (p.dstream) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] += row.ds[kShared ? 0 : j][e];
          }
          if (p.dresidual) store_row<VEC>(static_cast<ST*>(p.dresidual) + at, o);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o[e] *= p.scale;
        } else {
          store_row<VEC>(p.dgate + at, q);
        }
        store_row<VEC>(p.dx + at, o);
      }
    }
    if (kAhead) row = next;
  }
  if (kShared) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = lane + j * G;
      if (u < units)
#pragma unroll
        for (int half = 0; half < 2; ++half) *reinterpret_cast<float4*>(p.part + (long long)blockIdx.x * p.width + u * 8 + half * 4) = *lean(u, half);
    }
    return;
  }
  for (int g = 0; g < per_block; ++g) {
    if (grp == g) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float mine[VEC];
#pragma unroll
        for (int e = 0; e < E::kCount; ++e) E::put(mine, e, dw[j][e]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int u = lane + j * G;
          if (u >= units) continue;
          const int at = u * VEC + e;
          const float t = g == 0 ? mine[e] : acc_s[at] + mine[e];
          if (g == per_block - 1)
            p.part[(long long)blockIdx.x * p.width + at] = t;
          else
            acc_s[at] = t;
        }
      }
    }
    if (per_block > 1) __syncthreads();
  }
}

// dweight[c] = sum over the blocks' partial rows, in a fixed order: COLS columns x 1024 / COLS row lanes per block. 8 columns
// (a sector) give few columns more blocks and a thread fewer loads in turn: 1.2 us less at 128 and 2048 columns; 32 (a
// line) read wide rows faster: 5 us less at 8192.
template <int COLS>
__global__ void __launch_bounds__(1024) k_norm_reduce(const float* part, float* dw, int rows, int width) {
  constexpr int kLanes = 1024 / COLS;
  __shared__ float s[COLS][kLanes + 4];
  const int x = threadIdx.x % COLS, y = threadIdx.x / COLS, c = blockIdx.x * COLS + x;
  wait_for_previous();
  float t = 0.f;
  if (c < width)
#pragma unroll 10
    for (int r = y; r < rows; r += kLanes) t += part[(long long)r * width + c];
  s[x][y] = t;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cc = blockIdx.x * COLS + warp;
  if (warp >= COLS || cc >= width) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kLanes / 32; ++i) v += s[warp][lane + 32 * i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) dw[cc] = v;
}

struct Plan {
  int vec, nv, G, threads;
};

// Threads and vectors of a row: one vector a thread (8 elements; on the element path too) while 256 threads hold the row, so
// that the loads of many rows are in flight in few registers; more vectors, then 512 threads, beyond (the element path takes
// the threads first).
Plan plan_rows(int width, bool vec8) {
  Plan p;
  p.vec = vec8 ? 8 : 1;
  const int units = width / p.vec, few = vec8 ? 1 : 8, most = vec8 ? 4 : 32;
  int G = 8;
  while (G < (vec8 ? 256 : 512) && G * few < units) G *= 2;
  if (G * most < units) G = 512;
  const int nv = (units + G - 1) / G;
  p.nv = nv <= few ? few : vec8 && nv <= 2 ? 2 : most;
  p.G = G;
  p.threads = G > 256 ? G : 256;
  return p;
}

constexpr int kFwdBlocksPerSm = 5, kBwdBlocksPerSm = 4;
constexpr int kMaxPartialRows = 160 * kBwdBlocksPerSm;

// Calls f<VEC, NV, THREADS>() of the plan.
#define GDN_NORM_DISPATCH(q, CALL)                                   \
  if (q.vec == 8) {                                                  \
    if (q.threads == 512) { CALL(8, 4, 512); }                       \
    else if (q.nv == 1) { CALL(8, 1, 256); }                         \
    else if (q.nv == 2) { CALL(8, 2, 256); }                         \
    else { CALL(8, 4, 256); }                                        \
  } else {                                                           \
    if (q.threads == 256) { CALL(1, 8, 256); }                       \
    else if (q.nv == 8) { CALL(1, 8, 512); }                         \
    else { CALL(1, 32, 512); }                                       \
  }

template <int KIND, typename ST>
cudaError_t run_fwd(const NormParams& p, bool vec8, cudaStream_t s) {
  Plan q = plan_rows(p.width, vec8);
  int block = q.threads;
  // No warp of a wide row without work: 53 -> 36 us at 5120 columns. (The backward was slower so: 62 -> 67 us at 6144.)
  if (vec8 && q.nv > 1) block = q.G = ((p.width / 8 + q.nv - 1) / q.nv + 31) / 32 * 32;
  const int per_block = block / q.G;
  const long long blocks = (p.rows + per_block - 1) / per_block;
  // resident blocks that walk the rows a warp or less holds, one loaded ahead; else a block per row (or few rows)
  const int grid = int(std::min(blocks, KIND != kAdd && q.nv == 1 && q.G <= 32 ? (long long)p.sms * kFwdBlocksPerSm : 1ll << 30));
#define GDN_CALL(VEC, NV, T) return launch_after(k_norm_fwd<KIND, VEC, NV, T, ST>, grid, block, 0, s, p, q.G)
  GDN_NORM_DISPATCH(q, GDN_CALL)
#undef GDN_CALL
}

template <int KIND, typename ST>
cudaError_t run_bwd(const NormParams& p, bool vec8, cudaStream_t s) {
  const Plan q = plan_rows(p.width, vec8);
  const int per_block = q.threads / q.G;
  const long long blocks = (p.rows + per_block - 1) / per_block;
  const long long most = std::min((long long)p.sms * kBwdBlocksPerSm, (long long)kMaxPartialRows);
  const int grid = int(std::min(blocks, most));
  cudaError_t e = cudaSuccess;
#define GDN_CALL(VEC, NV, T) \
  e = launch_after(k_norm_bwd<KIND, VEC, NV, T, ST>, grid, T, per_block > 1 || kLean<KIND, VEC, NV, T, ST> ? size_t(p.width) * 4 : 0, s, p, q.G)
  GDN_NORM_DISPATCH(q, GDN_CALL)
#undef GDN_CALL
  if (e != cudaSuccess) return e;
  if (p.width <= 8 * 2 * p.sms)  // 8-column blocks, two of which fit an SM, are all resident
    return launch_after(k_norm_reduce<8>, (p.width + 7) / 8, 1024, 0, s, (const float*)p.part, p.dweight, grid, p.width);
  return launch_after(k_norm_reduce<32>, (p.width + 31) / 32, 1024, 0, s, (const float*)p.part, p.dweight, grid, p.width);
}

bool all16(std::initializer_list<const void*> ps) {
  uintptr_t m = 0;
  for (const void* q : ps) m |= reinterpret_cast<uintptr_t>(q);
  return (m & 15) == 0;
}

}  // namespace

int norm_partial_rows() { return kMaxPartialRows; }

cudaError_t launch_add_norm_fwd(const NormParams& p, cudaStream_t s) {
  const bool v = p.width % 8 == 0 && all16({p.x, p.residual, p.weight, p.y, p.stream});
  return p.stream_kind == 2 ? run_fwd<kAdd, float>(p, v, s) : run_fwd<kAdd, __nv_bfloat16>(p, v, s);
}
cudaError_t launch_add_norm_bwd(const NormParams& p, cudaStream_t s) {
  const bool v = p.width % 8 == 0 && all16({p.dy, p.dstream, p.stream, p.weight, p.dx, p.dresidual});
  return p.stream_kind == 2 ? run_bwd<kAdd, float>(p, v, s) : run_bwd<kAdd, __nv_bfloat16>(p, v, s);
}
cudaError_t launch_gated_norm_fwd(const NormParams& p, cudaStream_t s) {
  const bool v = p.width % 8 == 0 && all16({p.x, p.gate, p.weight, p.y});
  return p.act == 1 ? run_fwd<kSilu, __nv_bfloat16>(p, v, s) : run_fwd<kSigmoid, __nv_bfloat16>(p, v, s);
}
cudaError_t launch_gated_norm_bwd(const NormParams& p, cudaStream_t s) {
  const bool v = p.width % 8 == 0 && all16({p.x, p.gate, p.weight, p.dy, p.dx, p.dgate});
  return p.act == 1 ? run_bwd<kSilu, __nv_bfloat16>(p, v, s) : run_bwd<kSigmoid, __nv_bfloat16>(p, v, s);
}

}  // namespace gdn
