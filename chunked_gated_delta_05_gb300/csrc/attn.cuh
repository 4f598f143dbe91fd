// Parameters and device helpers of the attention block: norm and rotation of query and key heads (k_rope.cu), attention over
// whole sequences (k_attn_fwd.cu, k_attn_bwd.cu) and of single tokens over a paged cache (k_attn_step.cu).
#pragma once
#include "block_ops.cuh"
#include "umma.cuh"

namespace gdn {

// Kernel kinds of the per-launch timing hook, after the block operators' (names in api.cu).
enum AttnKernelKind { kKRopeFwd = kKAllKinds, kKRopeBwd, kKAttnFwd, kKAttnBwd, kKAttnStep, kKEveryKind };

// A operand read from TMEM, bf16: M lanes, two neighbouring K entries per 32-bit column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
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

struct AttnParams {
  int H, Hk, group;            // group = H / Hk query heads read one key head
  int T, N;                    // dense: tokens per sequence and sequences
  int tiles;                   // tiles of all sequences
  const int* table;            // packed: 3 ints per tile, most work first; else null (dense, computed)
  int causal;
  float scale;
  long long rows;
  __nv_bfloat16* o;            // [rows,H,D]
  float* lse;                  // [rows,H]
  // backward
  const __nv_bfloat16 *dO, *o_in;  // [rows,H,D]
  const float* lse_in;
  float *lse2, *delta;         // [H][rows]: lse log2(e), and the rows' sums of dO o
  __nv_bfloat16 *dq, *dk, *dv;
  int* status;
};

// Tile `i` of `step` tokens. Of a dense batch's sequences the last tiles come first (causal: the longest rows), or the first ones
// (`ascending`: causal keys, which the most queries see).
__device__ __forceinline__ AttnTile attn_tile(const AttnParams& p, int i, int step, bool ascending) {
  if (p.table) return {p.table[3 * i], p.table[3 * i + 1], p.table[3 * i + 2]};
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
// Rows `from` .. 127 of a tile zeroed by a warp. They belong to the next sequence, and 0 x NaN would carry its NaN over.
template <int D>
__device__ __forceinline__ void zero_attn_rows(uint8_t* tile, int from, int lane) {
  for (int r = from * 8 + lane; r < kAttnTile * 8; r += 32)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) *reinterpret_cast<uint4*>(tile + c * kAttnPanel + r * 16) = make_uint4(0, 0, 0, 0);
}

cudaError_t launch_attn_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int D, const AttnParams& p, cudaStream_t s);
// Backward: `order` holds the dq kernel's tiles (128 queries, most work first) and `keys` the dk / dv kernel's.
cudaError_t launch_attn_bwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo, int D, const AttnParams& p, const int* keys,
                            cudaStream_t s);

// ------------------------------------------------------------------ norm and rotation of query and key heads

struct RopeParams {
  long long rows;              // tokens of all sequences
  int T, N;                    // dense: tokens per sequence; sequences
  const int* cu;               // packed: device offsets [N+1], else null
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
  float *part, *dqw, *dkw;     // part: [rope_bwd_blocks()][2][D]
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
  int splits;                  // pieces a row's keys are cut into
  float scale;
  long long q_stride;
  const __nv_bfloat16 *q, *kc, *vc;
  const int *table, *lengths;
  __nv_bfloat16* o;            // [B,H,D]
  float* part;                 // splits > 1: [B,H,splits][D + 2]: weighted sum, reference, sum of weights
  int* status;
};
cudaError_t launch_attn_step(const AttnStepParams& p, int D, cudaStream_t s);

// Host: a 2-D bf16 tensor map (api.cu): rows of `cols` elements, `stride` elements apart, boxes of 64 x `box_rows`, 128-byte swizzle.
bool attn_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t stride, uint32_t box_rows);

}  // namespace gdn
