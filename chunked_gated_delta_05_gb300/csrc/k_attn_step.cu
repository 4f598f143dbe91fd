// Attention of one token per sequence over a paged cache: o = sum_j e^(scale q.k_j) v_j / sum_j e^(scale q.k_j) over the
// sequence's first `length` keys, which lie in the pages its row of the table names.
//
// Memory bound: every key and value is read once (4 D bytes a key and key head) for the group's query heads together, two
// products of 4 D group flops. A warp takes 16 keys at a time, K and V in 16-byte pieces by asynchronous copies two groups of keys
// ahead; each lane copies what it reads itself, so that no lane waits for another. The products run on the tensor core with the
// query heads as the 16 rows (m16n8k16: for so few rows the larger tcgen05 shapes would be idle rows).
//
// No shuffles between the products: in q k^T a lane's 16-byte piece of a key stands for whichever products' inner indices it falls
// on (the same channels are taken from q), so it needs no rearranging; the weights come out where the second product
// wants them; and a lane's pieces of four keys' values give, pair by pair of keys, that product's other operand, whose columns
// stand for channels 8 apart.
//
// A sequence's keys are cut into `splits` pieces of equal length, a block each, whose four warps take 16 keys in turn. Blocks leave
// a weighted sum, its reference and the sum of weights; a second kernel joins them. The reference moves only when a score
// lies 2^8 above it. Weights are rounded to bf16 for the product (the values' type), sums are fp32.
#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4, kKeys = 16, kStages = 3;
// A warp's stage of 16 keys: pieces of 16 bytes by lane.
template <int D>
struct Stage {
  static constexpr int kPieces = D / 32, kHalves = D / 64;  // of a key, of half a value row, to a lane
  static constexpr int kCount = 2 * kPieces + 4 * kHalves, kBytes = kCount * 512;
  static constexpr int kSmem = kWarps * kStages * kBytes;
};
constexpr float kRescale = 8.f;

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with rows 8 .. 15 empty.
__device__ __forceinline__ void mma16816_low(float* c, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  float x, y;
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%9,%9};"
               : "+f"(c[0]), "+f"(c[1]), "=f"(x), "=f"(y)
               : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}

// 16 bytes to shared memory, zeros where `there` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const __nv_bfloat16* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t part(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

}  // namespace

// kRows: 1 for up to 8 query heads of a key head in a block, 2 for up to 16.
template <int D, int kRows>
__global__ void __launch_bounds__(kWarps * 32) k_attn_step(const AttnStepParams p, int row_blocks) {
  using St = Stage<D>;
  constexpr int kPieces = St::kPieces, kHalves = St::kHalves;
  extern __shared__ __align__(16) uint8_t smem[];  // the warps' stages, then their sums
  __shared__ float ml_s[kWarps][8 * kRows][2];
  float(*acc_s)[8 * kRows][D] = reinterpret_cast<float(*)[8 * kRows][D]>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  int i = blockIdx.x;
  const int split = i % p.splits;
  i /= p.splits;
  const int rb = i % row_blocks;
  i /= row_blocks;
  const int hk = i % p.Hk, b = i / p.Hk;
  const int head0 = hk * p.group + rb * 8 * kRows, heads = min(8 * kRows, p.group - rb * 8 * kRows);
  wait_for_previous();
  int len = p.lengths[b];
  if (len > 0 && (len - 1) / p.page >= p.width) {  // longer than its row of the table
    if (threadIdx.x == 0 && p.status) atomicCAS(p.status, 0, kDevGateRange);
    len = 0;
  }
  if (len <= 0) {
    if (p.splits == 1)
      for (int x = threadIdx.x; x < heads * D; x += kWarps * 32) p.o[((long long)b * p.H + head0) * D + x] = __float2bfloat16(0.f);
    return;
  }
  const int piece = ((len + p.splits - 1) / p.splits + kKeys - 1) / kKeys * kKeys, from = split * piece, to = min(len, from + piece);
  if (from >= to) return;

  // queries: rows g and (kRows 2) g + 8
  uint4 q[kRows][kPieces];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      q[r][j] = make_uint4(0, 0, 0, 0);
      if (g + 8 * r < heads) q[r][j] = *reinterpret_cast<const uint4*>(p.q + b * p.q_stride + (head0 + g + 8 * r) * D + (c + 4 * j) * 8);
    }
  const float cs = p.scale * kLog2e, far = fminf(kRescale / cs, 3e38f);
  float m[kRows], l[kRows], o[kHalves][8][2 * kRows > 2 ? 4 : 2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
  for (int h2 = 0; h2 < kHalves; ++h2)
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int x = 0; x < 2 * kRows; ++x) o[h2][e][x] = 0.f;

  // Row of the cache (pages one after the other) of key k, -1 past the piece's end, and for a page that does not exist.
  const int* table = p.table + (long long)b * p.width;
  auto cache_row = [&](int k) -> long long {
    if (k >= to) return -1;
    const int page = table[k / p.page];
    if (page < 0 || page >= p.pages) {
      if (p.status) atomicCAS(p.status, 0, kDevGateRange);
      return -1;
    }
    return (long long)page * p.page + k % p.page;
  };
  const long long token = (long long)p.Hk * D;
  const __nv_bfloat16 *kc = p.kc + hk * D, *vc = p.vc + hk * D;
  const uint32_t mem = smem_u32(smem) + warp * (kStages * St::kBytes) + lane * 16;
  // Requests the pieces of 16 keys whose cache rows the lanes hold; bit x: this lane's x-th value row is there.
  auto request = [&](uint32_t at, long long mine) -> uint32_t {
#pragma unroll
    for (int u = 0; u < 2; ++u) {  // key g of either eight
      const long long r = __shfl_sync(0xffffffffu, mine, u * 8 + g);
      const __nv_bfloat16* src = kc + (r < 0 ? 0 : r) * token + c * 8;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) copy16(at + (u * kPieces + j) * 512, src + j * 32, r >= 0);
    }
    uint32_t bits = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {  // values of keys 2c, 2c + 1, 2c + 8, 2c + 9
      const long long r = __shfl_sync(0xffffffffu, mine, (x >> 1) * 8 + 2 * c + (x & 1));
      const __nv_bfloat16* src = vc + (r < 0 ? 0 : r) * token + g * 8;
      bits |= uint32_t(r >= 0) << x;
#pragma unroll
      for (int h2 = 0; h2 < kHalves; ++h2) copy16(at + (2 * kPieces + x * kHalves + h2) * 512, src + h2 * 64, r >= 0);
    }
    return bits;
  };
  constexpr int kStride = kWarps * kKeys;
  const int first = from + warp * kKeys;
  uint32_t bits[kStages] = {};
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    bits[i] = request(mem + i * St::kBytes, cache_row(first + i * kStride + (lane & 15)));
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  long long mine = cache_row(first + (kStages - 1) * kStride + (lane & 15));
  int stage = 0;
  for (int k0 = first; k0 < to; k0 += kStride) {
    bits[kStages - 1] = request(mem + (stage == 0 ? kStages - 1 : stage - 1) * St::kBytes, mine);
    asm volatile("cp.async.commit_group;" ::: "memory");
    mine = cache_row(k0 + kStages * kStride + (lane & 15));
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    const uint32_t at = mem + stage * St::kBytes;
    uint4 kk[2][kPieces], vv[4][kHalves];
    bool there[4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < kPieces; ++j) kk[u][j] = lds16(at + (u * kPieces + j) * 512);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      there[x] = bits[0] >> x & 1u;
#pragma unroll
      for (int h2 = 0; h2 < kHalves; ++h2) vv[x][h2] = lds16(at + (2 * kPieces + x * kHalves + h2) * 512);
    }
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) bits[i] = bits[i + 1];
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float s[2][4] = {};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t b0 = part(kk[u][j], 2 * hf), b1 = part(kk[u][j], 2 * hf + 1);
          if (kRows == 1) {
            mma16816_low(s[u], part(q[0][j], 2 * hf), part(q[0][j], 2 * hf + 1), b0, b1);
          } else {
            const uint32_t a[4] = {part(q[0][j], 2 * hf), part(q[kRows - 1][j], 2 * hf), part(q[0][j], 2 * hf + 1), part(q[kRows - 1][j], 2 * hf + 1)};
            mma16816(s[u], a, b0, b1);
          }
        }
    uint32_t w[4] = {};  // weights: rows g and g + 8, keys 2c, 2c + 1 of either eight
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float x[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) x[y] = there[y] ? s[y >> 1][2 * r + (y & 1)] : -INFINITY;
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (__any_sync(0xffffffffu, top > m[r] + far)) {  // the first keys too: their reference is -inf
        const float next = fmaxf(m[r], top), f = next == m[r] ? 1.f : exp2_approx((m[r] - next) * cs);
        m[r] = next;
        l[r] *= f;
#pragma unroll
        for (int h2 = 0; h2 < kHalves; ++h2)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            o[h2][e][2 * r] *= f;
            o[h2][e][2 * r + 1] *= f;
          }
      }
      const float ref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        x[y] = there[y] ? exp2_approx((x[y] - ref) * cs) : 0.f;
        l[r] += x[y];
      }
      w[r] = pack_bf16(x[0], x[1]);
      w[2 + r] = pack_bf16(x[2], x[3]);
    }
#pragma unroll
    for (int h2 = 0; h2 < kHalves; ++h2)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t pick = e & 1 ? 0x7632 : 0x5410;
        const uint32_t b0 = __byte_perm(part(vv[0][h2], e >> 1), part(vv[1][h2], e >> 1), pick);
        const uint32_t b1 = __byte_perm(part(vv[2][h2], e >> 1), part(vv[3][h2], e >> 1), pick);
        if (kRows == 1) mma16816_low(o[h2][e], w[0], w[2], b0, b1);
        else mma16816(o[h2][e], w, b0, b1);
      }
  }

  // the block's warps joined, their sums where the stages were
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (c == 0) {
      ml_s[warp][g + 8 * r][0] = m[r];
      ml_s[warp][g + 8 * r][1] = l[r];
    }
#pragma unroll
    for (int h2 = 0; h2 < kHalves; ++h2)
#pragma unroll
      for (int y = 0; y < 2; ++y) {  // channels h2 64 + (2c + y) 8 + e
        float* dst = &acc_s[warp][g + 8 * r][h2 * 64 + (2 * c + y) * 8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[e] = o[h2][e][2 * r + y];
      }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < heads * D; x += kWarps * 32) {
    const int r = x / D, d = x % D;
    float top = -INFINITY;
#pragma unroll
    for (int y = 0; y < kWarps; ++y) top = fmaxf(top, ml_s[y][r][0]);
    float sum = 0.f, total = 0.f;
#pragma unroll
    for (int y = 0; y < kWarps; ++y) {
      const float mw = ml_s[y][r][0], f = mw == top ? 1.f : exp2_approx((mw - top) * cs);
      sum = fmaf(acc_s[y][r][d], f, sum);
      total = fmaf(ml_s[y][r][1], f, total);
    }
    const long long at = (long long)b * p.H + head0 + r;
    if (p.splits == 1) {
      p.o[at * D + d] = __float2bfloat16(total == 0.f ? 0.f : sum / total);
    } else {
      const long long i = at * p.splits + split;
      p.part[i * D + d] = sum;
      if (d == 0) *reinterpret_cast<float2*>(p.part + (long long)p.B * p.H * p.splits * D + 2 * i) = make_float2(top, total);
    }
  }
}

// Joins the pieces of a (row, head): a block each, its kJoin warps taking pieces in turn, four requested together.
template <int D, int kJoin>
__global__ void __launch_bounds__(kJoin * 32) k_attn_join(const AttnStepParams p) {
  constexpr int kPer = D / 32;
  __shared__ float acc[kJoin][D], tot[kJoin];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long at = blockIdx.x;
  wait_for_previous();
  int len = p.lengths[at / p.H];
  if (len > 0 && (len - 1) / p.page >= p.width) len = 0;
  float sum[kPer] = {}, total = 0.f;
  if (len > 0) {
    const int piece = ((len + p.splits - 1) / p.splits + kKeys - 1) / kKeys * kKeys, n = (len + piece - 1) / piece;
    const float* src = p.part + at * p.splits * D + lane * kPer;
    const float2* ml = reinterpret_cast<const float2*>(p.part + (long long)p.B * p.H * p.splits * D) + at * p.splits;
    const float cs = p.scale * kLog2e;
    float top = -INFINITY;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, ml[i].x);
    for (int i0 = warp; i0 < n; i0 += 4 * kJoin) {
      float x[4][kPer];
      float2 y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kJoin;
        y[u] = i < n ? ml[i] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[u][e] = i < n ? src[(long long)i * D + e] : 0.f;
      }
      if (i0 == warp)
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = y[u].x == top ? 1.f : exp2_approx((y[u].x - top) * cs);
        total = fmaf(y[u].y, f, total);
#pragma unroll
        for (int e = 0; e < kPer; ++e) sum[e] = fmaf(x[u][e], f, sum[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[warp][lane * kPer + e] = sum[e];
  if (lane == 0) tot[warp] = total;
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kJoin * 32) {
    float v = 0.f, l = 0.f;
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      v += acc[i][d];
      l += tot[i];
    }
    p.o[at * D + d] = __float2bfloat16(l == 0.f ? 0.f : v / l);
  }
}

template <int D, int kRows>
static cudaError_t launch(const AttnStepParams& p, cudaStream_t s) {
  constexpr int kSmem = Stage<D>::kSmem;
  static_assert(kSmem >= kWarps * 8 * kRows * D * 4, "the warps' sums lie where the stages were");
  const int rb = (p.group + 8 * kRows - 1) / (8 * kRows);
  const dim3 grid(unsigned((long long)p.B * p.Hk * rb * p.splits)), block(kWarps * 32);
  cudaError_t e = cudaFuncSetAttribute(k_attn_step<D, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) e = launch_after(k_attn_step<D, kRows>, grid, block, kSmem, s, p, rb);
  if (e == cudaSuccess && p.splits > 1) e = p.splits > 16 ? launch_after(k_attn_join<D, 16>, dim3(unsigned((long long)p.B * p.H)), dim3(512), 0, s, p)
                                                      : launch_after(k_attn_join<D, 4>, dim3(unsigned((long long)p.B * p.H)), dim3(128), 0, s, p);
  return e;
}

cudaError_t launch_attn_step(const AttnStepParams& p, int D, cudaStream_t s) {
  if (D == 128) return p.group > 8 ? launch<128, 2>(p, s) : launch<128, 1>(p, s);
  return p.group > 8 ? launch<64, 2>(p, s) : launch<64, 1>(p, s);
}

}  // namespace gdn
