// Parameters and device helpers of the attention block: norm and rotation of query and key heads (k_rope.cu), attention over
// whole sequences (k_attn_fwd.cu, k_attn_bwd.cu) and of single tokens over a paged cache (k_attn_step.cu).
#pragma once
#include <atomic>

#include "block_ops.cuh"
#include "umma.cuh"

namespace gdn {

// Kernel kinds of the per-launch timing hook, after the block operators' (names in api.cu).
enum AttnKernelKind { kKRopeFwd = kKAllKinds, kKRopeBwd, kKAttnFwd, kKAttnBwd, kKAttnStep, kKEveryKind };

// One thread issues the products, and what it takes to form an instruction's operands sets their pace: with the descriptors of
// umma.cuh built anew for every step it took 90 cycles an instruction, where the tensor core needs 64 (measured, products of
// 128 x 128 x 128). So the descriptors' low words are kept and a step is one addition; the high word is a constant.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart, version, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_low_k(uint32_t base) { return (base >> 4) | (1u << 16); }                                     // K-major
__device__ __forceinline__ uint32_t desc_low_mn(uint32_t base, uint32_t panel) { return (base >> 4) | ((panel >> 4) << 16); }          // MN-major
//
// The whole issuing warp walks the code, and `lead` (one lane) issues: control flow that the compiler knows to be the same for all
// lanes keeps descriptors and addresses in uniform registers, where the instruction wants them.
template <bool kAcc>
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 x, y;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "n"(int(kAcc)), "r"(lead)
      : "memory");
}
// A operand in TMEM, bf16: M lanes, two neighbouring K entries per 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 y;\n mov.b64 y, {%2, %4};\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "r"(uint32_t(acc)), "r"(lead)
      : "memory");
}
// Arrive on `bar` once every product that the leading lane has issued so far is complete.
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_lead() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}

// mbar_wait (bounded, umma.cuh) behind tries that let the hardware suspend the thread for up to a millisecond: it wakes with the
// phase, and neither spins nor reads a clock meanwhile.
__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, int code) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    if (ok) return true;
  }
  return mbar_wait(bar, parity, abort, status, code);
}

// 16 lanes x 64 columns: registers 4 i .. 4 i + 3 hold columns 8 i + 2 (t % 4), + 1 of lane t / 4, then of lane t / 4 + 8 (t: the thread).
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
        "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
        "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
// 16 lanes x 32 columns: registers 2 i, 2 i + 1 go to column 4 i + t % 4 of lanes t / 4 and t / 4 + 8.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
        "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A warpgroup's share of the block's registers.
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------ attention over whole sequences

constexpr int kAttnTile = 128;       // queries or keys of a tile (an MMA's M and N)
constexpr int kAttnPair = 2 * kAttnTile;  // queries of a forward CTA

// One tile of a sequence: the sequence's first row, its length, and the tile's first token in it.
struct AttnTile {
  int row0, len, first;
};

constexpr int kAttnInline = 170;     // tiles whose table goes along with the parameters (packed calls of up to some 20000 tokens)

struct AttnParams {
  int H, Hk, group;            // group = H / Hk query heads read one key head
  int T, N;                    // dense: tokens per sequence and sequences
  int tiles;                   // tiles of all sequences
  int sms;
  bool packed;                 // else the tiles are computed
  const int* table;            // packed: 3 ints per tile, most work first, or null: `few`
  int few[3 * kAttnInline];
  int causal;
  float scale;
  long long rows;
  __nv_bfloat16* o;            // [rows,H,D]
  float* lse;                  // [rows,H]
  // backward
  const __nv_bfloat16 *dO, *o_in;  // [rows,H,D]
  const float* lse_in;
  float *lse2, *delta;         // [H][rows]: -lse log2(e), and minus the rows' sums of dO o
  __nv_bfloat16 *dq, *dk, *dv;
  unsigned* counters;          // [2]: tiles handed out
  int* status;
};

// Tile `i` of `step` tokens. Of a dense batch's sequences the last tiles come first (causal: the longest rows), or the first ones
// (`ascending`: causal keys, which the most queries see).
__device__ __forceinline__ AttnTile attn_tile(const AttnParams& p, int i, int step, bool ascending) {
  if (p.packed) {
    if (p.table) return {p.table[3 * i], p.table[3 * i + 1], p.table[3 * i + 2]};
    return {p.few[3 * i], p.few[3 * i + 1], p.few[3 * i + 2]};
  }
  const int level = i / p.N, n = i - level * p.N, per = (p.T + step - 1) / step;
  return {n * p.T, p.T, (ascending ? level : per - 1 - level) * step};
}

// A tile of 128 rows x D columns in shared memory: panels of 64 columns, 128-byte rows, 128-byte swizzle.
constexpr int kAttnPanel = kAttnTile * 128;
template <int D>
__device__ __forceinline__ void load_attn_tile(uint8_t* dst, const CUtensorMap* m, int x, int y, uint64_t* bar) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) tma_load_2d(dst + i * kAttnPanel, m, x + i * 64, y, bar);
}
// d = A B^T of two such tiles (inner dimension D), from their descriptors' low words.
template <int D>
__device__ __forceinline__ void product_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t id = idesc_bf16(kAttnTile, kAttnTile);
  mma_ss<false>(lead, d, a, b, id);
#pragma unroll
  for (int s = 1; s < D / 16; ++s) {
    const uint32_t o = ((s >> 2) * kAttnPanel + (s & 3) * 32) >> 4;
    mma_ss<true>(lead, d, a + o, b + o, id);
  }
}
// d (+)= A B, A [128,128] in TMEM in parts of 2 kPart columns of which the first kPart hold it; B a tile read MN-major.
template <int D, int kPart>
__device__ __forceinline__ void product_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, bool acc) {
  constexpr uint32_t id = idesc_bf16(kAttnTile, D, false, true);
  constexpr int kPer = kPart / 8;  // steps of 16 inner entries in a part
#pragma unroll
  for (int s = 0; s < kAttnTile / 16; ++s) mma_ts(lead, d, a + (s / kPer) * 2 * kPart + (s % kPer) * 8, b + s * 128, id, acc || s > 0);
}
// 32 bf16 of a row times f from 32 fp32 columns, to 16-byte aligned memory (32-byte aligned: whole sectors a store).
__device__ __forceinline__ void store_bf16x32(__nv_bfloat16* dst, const float* x, float f, bool wide) {
  uint32_t u[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) u[e] = pack_bf16(x[2 * e] * f, x[2 * e + 1] * f);
  if (wide) {
#pragma unroll
    for (int e = 0; e < 16; e += 8)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 2 * e), "r"(u[e]), "r"(u[e + 1]), "r"(u[e + 2]), "r"(u[e + 3]), "r"(u[e + 4]), "r"(u[e + 5]),
                   "r"(u[e + 6]), "r"(u[e + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(u[e], u[e + 1], u[e + 2], u[e + 3]);
  }
}
// A ring of kN stages walked kStep uses at a time: this use's stage and phase.
template <int kN, int kStep>
struct Ring {
  int at;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int first) : at(first) {}
  __device__ __forceinline__ void next() {
    at += kStep;
    if (at >= kN) {
      at -= kN;
      phase ^= 1u;
    }
  }
};
// Rows `from` .. 127 of a tile zeroed by a warp. They belong to the next sequence, and 0 x NaN would carry its NaN over.
template <int D>
__device__ __forceinline__ void zero_attn_rows(uint8_t* tile, int from, int lane) {
  for (int r = from * 8 + lane; r < kAttnTile * 8; r += 32)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) *reinterpret_cast<uint4*>(tile + c * kAttnPanel + r * 16) = make_uint4(0, 0, 0, 0);
}

cudaError_t launch_attn_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int D, const AttnParams& p, cudaStream_t s);
// Backward: `p` holds the dq kernel's tiles (128 queries, most work first) and `pk` the dk / dv kernel's.
cudaError_t launch_attn_bwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo, int D, const AttnParams& p, const AttnParams& pk,
                            cudaStream_t s);
// Sets a kernel's shared memory limit, once per kernel (`done`: a bit per device) and device.
template <typename K>
cudaError_t allow_smem(K* kernel, int bytes, std::atomic<unsigned long long>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done->load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

// ------------------------------------------------------------------ norm and rotation of query and key heads

constexpr int kRopeInline = 64;      // offsets that go along with the parameters

struct RopeParams {
  long long rows;              // tokens of all sequences
  int T, N;                    // dense: tokens per sequence; sequences
  bool packed;
  const int* cu;               // packed: device offsets [N+1], or null: `few`
  int few[kRopeInline];
  int H, Hk, rotary, interleaved;
  float eps;
  long long q_s, k_s, v_s;     // elements between tokens
  const __nv_bfloat16 *q, *k, *v;
  const float *qw, *kw, *inv_freq;  // weights (both or neither); inv_freq [rotary/2]
  const int* positions;        // [rows] or null: counted from the sequence's first token
  __nv_bfloat16 *qo, *ko;      // [rows,H,D], [rows,Hk,D]
  // store
  const int *lengths, *table;  // [N], [N,width]; null without a cache
  int pages, page, width;
  __nv_bfloat16 *kc, *vc;      // [pages,page,Hk,D]
  int* status;
  // backward
  const __nv_bfloat16 *dqo, *dko;   // [rows,H,D], [rows,Hk,D]
  __nv_bfloat16 *dq, *dk;
  float *part, *dqw, *dkw;     // part: [rope_bwd_blocks()][D]
  int sms;
};
cudaError_t launch_rope_fwd(const RopeParams& p, int D, cudaStream_t s);
cudaError_t launch_rope_bwd(const RopeParams& p, int D, cudaStream_t s);
// The most blocks of a backward (rows of partial weight gradients).
int rope_bwd_blocks();

// ------------------------------------------------------------------ single tokens over a paged cache

struct AttnStepParams {
  int B, H, Hk, group;
  int pages, page, width;      // cache pages, keys in a page, entries of a row of the table
  int shares;                  // the rows' keys are cut into
  float scale;
  long long q_stride;
  const __nv_bfloat16 *q, *kc, *vc;
  const int *table, *lengths;
  __nv_bfloat16* o;            // [B,H,D]
  // pieces of rows that several shares hold, by row + share and part (key head, block of query heads): weighted sums [..][8 or 16][D]
  // and {reference, sum of weights}; and every row's and part's first and last share
  float* part;
  float2* ml;
  int2* span;
  int* status;
};
cudaError_t launch_attn_step(const AttnStepParams& p, int D, cudaStream_t s);
inline int attn_step_rows(int group) { return group > 8 ? 16 : 8; }  // query heads of a block
// Blocks that 152 SMs hold at once, by shared memory and registers: 3 each, or 6 (4 with 16 heads) of the narrower heads.
inline int attn_step_blocks(int D, int rows) { return 152 * (D == 128 ? 3 : rows == 8 ? 6 : 4); }

// Host: a 2-D bf16 tensor map (api.cu): rows of `cols` elements, `stride` elements apart, boxes of 64 x `box_rows`, 128-byte swizzle.
bool attn_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t stride, uint32_t box_rows);

}  // namespace gdn
