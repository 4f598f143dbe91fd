// Attention of one token per sequence over a paged cache: o = sum_j e^(scale q.k_j) v_j / sum_j e^(scale q.k_j) over the
// sequence's first `length` keys, which lie in the pages its row of the table names.
//
// Memory bound: every key and value is read once (4 D bytes a key and key head) for the group's query heads together, two
// products of 4 D group flops. A warp takes 16 keys at a time, whole K and V rows by asynchronous bulk copies (a lane each) a group
// of keys ahead: twelve warps an SM with two stages each read faster than eight with three (120 rows, 1.14 GB: 173 us, 6.6 TB/s,
// against 196). The products run on the tensor core, the keys (then the channels) as the 16 rows of m16n8k16 and the query heads
// as its 8 columns (for so few heads the larger tcgen05 shapes would be idle columns):
//   S^T [16 keys, 8 heads] = K q^T,   O^T [16 channels, 8 heads] += V^T P^T
// K comes by ldmatrix, V^T by its transposing form, and the weights' 8 x 8 blocks are transposed in registers between the two.
// A warp iteration is about 150 instructions for 8 KB; with the heads as rows it was over 500, which held the call to 5.0 TB/s.
//
// The rows' keys, in units of 64 one after the other, are cut into equal shares, as many as make the SMs' blocks with one for
// each key head (or 16 query heads of one): rows differ in length, and their lengths are known on the device only. The key
// heads' blocks of a share run side by side, so that a token's row of the cache is read at one time. A block's four warps take 16
// keys of a unit each. Where a row's units lie in several shares, the blocks leave a weighted sum, its reference and the sum of
// weights, which a second kernel joins. The reference moves only for a score whose weight would exceed 2^8, so no maximum is taken otherwise.
// Weights are rounded to bf16 for the product (the values' type), sums are fp32. (Heads of 64, up to 8 of a key head: 12 bytes a thread are spilled.)
#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4, kKeys = 16, kUnit = kWarps * kKeys, kStages = 2;
// A warp's stage of 16 keys: their K rows, then their V rows, 16 bytes further apart than they are long (ldmatrix's eight rows then
// lie in different banks).
template <int D>
struct Stage {
  static constexpr int kRow = D * 2, kPitch = kRow + 16, kBytes = 2 * kKeys * kPitch, kSmem = kWarps * kStages * kBytes;
};
constexpr float kRescale = 8.f;

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four 8 x 8 blocks whose rows the lanes name (block lane / 8, row lane % 8); `kT`: transposed.
template <bool kT>
__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t at) {
  if (kT)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
}  // namespace

// Units of row b: none of a padding row, nor of one longer than its row of the table.
__device__ __forceinline__ int units_of(const AttnStepParams& p, int b, bool report) {
  const int len = p.lengths[b];
  if (len <= 0) return 0;
  if ((len - 1) / p.page >= p.width) {
    if (report && p.status) atomicCAS(p.status, 0, kDevGateRange);
    return 0;
  }
  return (len + kUnit - 1) / kUnit;
}

// kRows: 1 for up to 8 query heads of a key head in a block, 2 for up to 16 (two blocks of eight columns).
template <int D, int kRows>
__global__ void __launch_bounds__(kWarps * 32) k_attn_step(const AttnStepParams p, int row_blocks) {
  using St = Stage<D>;
  extern __shared__ __align__(128) uint8_t smem[];  // the warps' stages, then their sums
  __shared__ float ml_s[kWarps][8 * kRows][2];
  float(*acc_s)[8 * kRows][D] = reinterpret_cast<float(*)[8 * kRows][D]>(smem);
  __shared__ long long warp_sum[kWarps];
  __shared__ int start_b, start_k, abort_flag;
  __shared__ uint64_t full[kWarps][kStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int parts = p.Hk * row_blocks;  // of a row: its key heads, in blocks of 8 kRows query heads
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&full[0][0] + i, 32);
    fence_mbar_init();
  }
  wait_for_previous();

  // The units before every thread's rows, then this block's share and where it starts: a row, and units into its segments.
  const int per = (p.B + kWarps * 32 - 1) / (kWarps * 32), row0 = min(p.B, int(threadIdx.x) * per), row1 = min(p.B, row0 + per);
  long long sum = 0;
  for (int r = row0; r < row1; ++r) sum += units_of(p, r, true);
  long long before = sum, all = 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long left = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += left;
  }
  if (lane == 31) warp_sum[warp] = before;
  __syncthreads();
  before -= sum;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += warp_sum[i];
    all += warp_sum[i];
  }
  const int part = blockIdx.x % parts, which = blockIdx.x / parts;  // blocks of all parts of a share side by side: they read the same tokens
  const long long share = (all + p.shares - 1) / p.shares, end = min(all, share * (which + 1));
  long long u = share * which;
  if (u >= end) return;
  if (before <= u && u < before + sum) {
    long long at = before;
    int r = row0;
    while (u >= at + units_of(p, r, false)) at += units_of(p, r++, false);
    start_b = r;
    start_k = int(u - at);
  }
  __syncthreads();
  int b = start_b, k_unit = start_k;
  const int hk = part / row_blocks, rb = part - hk * row_blocks, head0 = hk * p.group + rb * 8 * kRows, heads = min(8 * kRows, p.group - rb * 8 * kRows);

  const float cs = p.scale * kLog2e, far = fminf(kRescale / cs, 3e38f);
  int stage = 0;
  uint32_t phases = 0;  // a bit per stage
  bool ok = true;
  while (u < end) {  // a row, or what the share holds of it
    const int n_units = units_of(p, b, false);
    if (n_units == 0) {
      ++b;
      continue;
    }
    const int len = p.lengths[b], take = int(min(end - u, (long long)(n_units - k_unit)));
    const int from = k_unit * kUnit, to = min(len, from + take * kUnit);
    // queries as the products' columns: of head g (and g + 8), channels 16 j + 2 c, + 1 and + 8, + 9
    uint32_t q[kRows][D / 16][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          q[r][j][y] = g + 8 * r < heads ? *reinterpret_cast<const uint32_t*>(p.q + b * p.q_stride + (head0 + g + 8 * r) * D + 16 * j + 2 * c + 8 * y) : 0u;
    // reference and partial sum of weights of heads 2 c + y (+ 8 r); sums over values: o[r][j] channels 16 j + g, + 8 of those heads
    float m[kRows][2], l[kRows][2], o[kRows][D / 16][4];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int y = 0; y < 2; ++y) m[r][y] = -INFINITY, l[r][y] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[r][j][x] = 0.f;
    }

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
    uint8_t* mem = smem + warp * (kStages * St::kBytes);
    // Requests the rows of 16 keys into stage st: lanes 0 .. 15 hold the keys' cache rows and copy K, the others copy V.
    auto request = [&](int st, long long mine) {
      uint8_t* dst = mem + st * St::kBytes + lane * St::kPitch;
      if (mine >= 0) {
        mbar_expect_tx(&full[warp][st], St::kRow);
        bulk_load(dst, (lane < 16 ? kc : vc) + mine * token, St::kRow, &full[warp][st]);
      } else {
#pragma unroll
        for (int i = 0; i < St::kRow / 16; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
        fence_async_smem();  // before a copy to the same place
        mbar_arrive(&full[warp][st]);
      }
    };
    constexpr int kStride = kWarps * kKeys;
    const int first = from + warp * kKeys;
    uint32_t valid[kStages] = {};  // of the stages ahead, the keys that are there
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const long long row = cache_row(first + i * kStride + (lane & 15));
      valid[i] = __ballot_sync(0xffffffffu, row >= 0);
      request((stage + i) % kStages, row);
    }
    long long mine = cache_row(first + (kStages - 1) * kStride + (lane & 15));
    for (int k0 = first; k0 < to; k0 += kStride) {
      valid[kStages - 1] = __ballot_sync(0xffffffffu, mine >= 0);
      __syncwarp();  // every lane has read the stage before this one
      request(stage == 0 ? kStages - 1 : stage - 1, mine);
      mine = cache_row(k0 + kStages * kStride + (lane & 15));
      ok = __all_sync(0xffffffffu, attn_wait(&full[warp][stage], phases >> stage & 1u, &abort_flag, p.status, kDevTimeoutTma));
      if (!ok) break;
      phases ^= 1u << stage;
      const uint32_t at = smem_u32(mem + stage * St::kBytes);
      float sc[kRows][4] = {};
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t a[4];
        ldmatrix4<false>(a, at + (lane & 15) * St::kPitch + (2 * j + (lane >> 4)) * 16);
#pragma unroll
        for (int r = 0; r < kRows; ++r) mma16816(sc[r], a, q[r][j][0], q[r][j][1]);
      }
      const bool there[2] = {bool(valid[0] >> g & 1u), bool(valid[0] >> (g + 8) & 1u)};
      uint32_t w[kRows][2];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        bool high = false;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (!there[x >> 1]) sc[r][x] = -INFINITY;
          high |= sc[r][x] > m[r][x & 1] + far;
        }
        if (__any_sync(0xffffffffu, high)) {  // the first keys too: their reference is -inf
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float top = fmaxf(sc[r][y], sc[r][2 + y]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float next = fmaxf(m[r][y], top), f = next == m[r][y] ? 1.f : exp2_approx((m[r][y] - next) * cs);
            m[r][y] = next;
            l[r][y] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[r][j][y] *= f;
              o[r][j][2 + y] *= f;
            }
          }
        }
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[r][e & 1] == -INFINITY ? 0.f : m[r][e & 1];
          x[e] = there[e >> 1] ? exp2_approx((sc[r][e] - ref) * cs) : 0.f;
          l[r][e & 1] += x[e];
        }
        w[r][0] = transpose8(pack_bf16(x[0], x[1]));
        w[r][1] = transpose8(pack_bf16(x[2], x[3]));
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t a[4];
        ldmatrix4<true>(a, at + (kKeys + ((lane >> 4) << 3) + (lane & 7)) * St::kPitch + (2 * j + ((lane >> 3) & 1)) * 16);
#pragma unroll
        for (int r = 0; r < kRows; ++r) mma16816(o[r][j], a, w[r][0], w[r][1]);
      }
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) valid[i] = valid[i + 1];
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // Rows before this one and shares before this one together number the pieces of a part's rows.
    const bool whole = k_unit == 0 && take == n_units;
    const long long slot = (long long)(b + which) * parts + part;
    // the block's warps joined, their sums where the stages were
    for (int i = 0; i < (ok ? kStages - 1 : kStages); ++i) {  // the stages ahead, which hold no key of the row (after an error: what is in flight)
      const int st = stage + i >= kStages ? stage + i - kStages : stage + i;
      mbar_drain(&full[warp][st], phases >> st & 1u);
      phases ^= 1u << st;
    }
    __syncthreads();
    if (abort_flag) return;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[r][y] += __shfl_xor_sync(0xffffffffu, l[r][y], d);
        const int head = 8 * r + 2 * c + y;
        if (g == 0) {
          ml_s[warp][head][0] = m[r][y];
          ml_s[warp][head][1] = l[r][y];
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          acc_s[warp][head][16 * j + g] = o[r][j][y];
          acc_s[warp][head][16 * j + g + 8] = o[r][j][2 + y];
        }
      }
    __syncthreads();
    for (int x = threadIdx.x; x < heads * D; x += kWarps * 32) {
      const int r = x / D, d = x % D;
      float top = -INFINITY;
#pragma unroll
      for (int y = 0; y < kWarps; ++y) top = fmaxf(top, ml_s[y][r][0]);
      float sum = 0.f, total = 0.f;  // of the warps
#pragma unroll
      for (int y = 0; y < kWarps; ++y) {
        const float mw = ml_s[y][r][0], f = mw == top ? 1.f : exp2_approx((mw - top) * cs);
        sum = fmaf(acc_s[y][r][d], f, sum);
        total = fmaf(ml_s[y][r][1], f, total);
      }
      const long long at = (long long)b * p.H + head0 + r;
      if (whole) {
        p.o[at * D + d] = __float2bfloat16(total == 0.f ? 0.f : sum / total);
      } else {
        const long long i = (slot * 8 * kRows + r);
        p.part[i * D + d] = sum;
        if (d == 0) p.ml[i] = make_float2(top, total);
      }
    }
    if (threadIdx.x == 0 && k_unit == 0) p.span[(long long)b * parts + part] = make_int2(which, int((u + n_units - 1) / share));
    __syncthreads();  // the sums are read before the stages are written again
    fence_async_smem();
    u += take;
    k_unit = 0;
    ++b;
  }
}

// Joins the pieces of a row's head, where they are several, kJoin warps taking pieces in turn, four requested together. Rows
// without keys are zeroed.
template <int D, int kRows, int kJoin>
__global__ void __launch_bounds__(kJoin * 32) k_attn_join(const AttnStepParams p, int row_blocks) {
  constexpr int kPer = D / 32;
  __shared__ float acc[kJoin][D], tot[kJoin];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long at = blockIdx.x;
  const int b = int(at / p.H), h = int(at - (long long)b * p.H), hk = h / p.group, in = h - hk * p.group, rb = in / (8 * kRows), r = in - rb * 8 * kRows;
  wait_for_previous();
  if (units_of(p, b, false) == 0) {
    for (int d = threadIdx.x; d < D; d += kJoin * 32) p.o[at * D + d] = __float2bfloat16(0.f);
    return;
  }
  const int parts = p.Hk * row_blocks, part = hk * row_blocks + rb;
  const int2 span = p.span[(long long)b * parts + part];
  // Written by its only block; or by none, where a wait of the step ran out, and then what stands there names no pieces.
  if (span.x < 0 || span.x >= span.y || span.y >= p.shares) return;
  const int n = span.y - span.x + 1;
  const long long first = (long long)(b + span.x) * parts + part, step = (long long)parts * 8 * kRows;  // rows from one piece to the next
  const float* src = p.part + (first * 8 * kRows + r) * D + lane * kPer;
  const float2* ml = p.ml + first * 8 * kRows + r;
  const float cs = p.scale * kLog2e;
  float sum[kPer] = {}, total = 0.f, top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, ml[i * step].x);
  for (int i0 = warp; i0 < n; i0 += 4 * kJoin) {
    float x[4][kPer];
    float2 y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kJoin;
      y[u] = i < n ? ml[i * step] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[u][e] = i < n ? src[i * step * D + e] : 0.f;
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
  const dim3 block(kWarps * 32), rows(unsigned((long long)p.B * p.H));
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(k_attn_step<D, kRows>, kSmem, &done);
  if (e == cudaSuccess) e = launch_after(k_attn_step<D, kRows>, dim3(unsigned(p.shares * p.Hk * rb)), block, kSmem, s, p, rb);
  if (e != cudaSuccess) return e;
  // A row's pieces are about the shares over the rows: 16 warps take them where there are many, else 4. Both kernels, rows of 8192 keys with 4 and with
  // 16 warps: 16 heads of 128 over 4 (114 shares), 1 row 12.6 and 11.9 us, 6 rows 21.9 and 21.8, 8 rows 30.6 and 30.8, 48 rows 126 and 131;
  // 8 heads over one (456 shares), 4 rows 13.3 and 12.6, 16 rows 19.6 and 19.4, 24 rows 23.8 and 24.3.
  if (p.shares > 16 * p.B) return launch_after(k_attn_join<D, kRows, 16>, rows, dim3(512), 0, s, p, rb);
  return launch_after(k_attn_join<D, kRows, 4>, rows, dim3(128), 0, s, p, rb);
}

cudaError_t launch_attn_step(const AttnStepParams& p, int D, cudaStream_t s) {
  if (D == 128) return p.group > 8 ? launch<128, 2>(p, s) : launch<128, 1>(p, s);
  return p.group > 8 ? launch<64, 2>(p, s) : launch<64, 1>(p, s);
}

}  // namespace gdn
