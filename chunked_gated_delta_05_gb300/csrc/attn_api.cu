// Host side of the attention blocks (declared in include/gdn.h): contract validation, workspace layout, the tiles of packed
// documents, tensor maps and the launches.
#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "attn.cuh"
#include "gdn.h"
#include "host.cuh"

namespace gdn {
namespace {

using bf = __nv_bfloat16;
using cbf = const __nv_bfloat16;

// Heads and sequences, which the descriptions share.
struct Shape {
  int B, T, H, Hk, D, N;
  long long rows;
  const int32_t* cu;  // the caller's host offsets, or null
};

int check_heads(int H, int Hk, int D, Shape* S) {
  if (H < 1 || Hk < 0) return bad("H must be positive");
  S->H = H;
  S->Hk = Hk ? Hk : H;
  if (H % S->Hk) return bad("num_k_heads must be 0 or divide H");
  if (D != 64 && D != 128) return bad("head_dim must be 64 or 128");
  if (H > (1 << 16)) return bad("too many heads");
  S->D = D;
  return GDN_OK;
}

template <class Desc>
int check_sequences(const Desc* d, Shape* S) {
  if (d->B < 1 || d->T < 1) return bad("B and T must be positive");
  S->B = d->B;
  S->T = d->T;
  S->rows = (long long)d->B * d->T;
  if (S->rows > (1ll << 30)) return bad("B*T too large");
  S->cu = d->cu_seqlens;
  S->N = d->B;
  if (S->cu) {
    if (d->B != 1) return bad("packed documents (cu_seqlens) require batch size 1");
    if (d->num_seqs < 1) return bad("num_seqs must be >= 1 with cu_seqlens");
    if (S->cu[0] != 0) return bad("cu_seqlens must start at 0");
    for (int i = 0; i < d->num_seqs; ++i)
      if (S->cu[i + 1] <= S->cu[i]) return bad("cu_seqlens must be strictly increasing (no empty documents)");
    if (S->cu[d->num_seqs] != d->T) return bad("cu_seqlens must end at T");
    S->N = d->num_seqs;
  }
  return GDN_OK;
}

// A token stride, 0 meaning contiguous; -1 when it is not usable.
long long stride_of(long long given, int heads, int D) {
  const long long s = given ? given : (long long)heads * D;
  return s < (long long)heads * D || s % 8 || s > (1ll << 32) ? -1 : s;
}
size_t extent(long long rows, long long stride, int heads, int D) { return (size_t(rows - 1) * stride + size_t(heads) * D) * 2; }

struct Span {
  const void* p;
  size_t n;
};
template <size_t NI, size_t NO>
bool alias(const Span (&in)[NI], const Span (&out)[NO]) {
  for (size_t o = 0; o < NO; ++o) {
    for (const Span& i : in)
      if (overlap(out[o].p, out[o].n, i.p, i.n)) return true;
    for (size_t k = 0; k < o; ++k)
      if (overlap(out[o].p, out[o].n, out[k].p, out[k].n)) return true;
  }
  return false;
}

// Makes the device's context current to this thread: the runtime does so at a thread's first call that needs it, but
// encoding a tensor map (a driver call) comes before that one in a thread that autograd has just started.
int bind_context() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaSetDevice(dev);
  return cuda_rc(e, "device context");
}

bool workspace_ok(const void* ws, size_t have, size_t need) { return ws && have >= need && aligned(ws, 256); }

// ------------------------------------------------------------------ norm and rotation

struct RopeProblem {
  Shape S;
  long long q_s, k_s, v_s;
};

int validate_rope(const gdn_rope_desc_t* d, RopeProblem* P, bool store) {
  if (!d) return bad("desc is NULL");
  int rc = check_heads(d->H, d->num_k_heads, d->head_dim, &P->S);
  if (!rc) rc = check_sequences(d, &P->S);
  if (rc) return rc;
  if (d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 16) return bad("rotary_dim must be a multiple of 16 up to head_dim");
  if (d->interleaved != 0 && d->interleaved != 1) return bad("interleaved must be 0 or 1");
  if (!(d->eps >= 0.f) || std::isinf(d->eps)) return bad("eps must be finite and not negative");
  P->q_s = stride_of(d->q_stride, P->S.H, P->S.D);
  P->k_s = stride_of(d->k_stride, P->S.Hk, P->S.D);
  P->v_s = stride_of(d->v_stride, P->S.Hk, P->S.D);
  if (P->q_s < 0 || P->k_s < 0 || P->v_s < 0) return bad("strides must be multiples of 8, at least a token's heads");
  if (store && (d->num_pages < 1 || d->page_size < 1 || d->table_width < 1)) return bad("num_pages, page_size and table_width must be positive");
  if (store && (long long)d->table_width * d->page_size > (1ll << 30)) return bad("the page table spans too many tokens");
  return GDN_OK;
}

struct RopeLayout {
  size_t cu, part, total;
};
RopeLayout layout_rope(const RopeProblem& P) {
  RopeLayout l{};
  l.part = align256(P.S.cu ? size_t(P.S.N + 1) * 4 : 4);
  l.total = l.part + align256(size_t(rope_bwd_blocks()) * P.S.D * 4);
  return l;
}

RopeParams rope_params(const gdn_rope_desc_t* d, const RopeProblem& P) {
  RopeParams p{};
  p.rows = P.S.rows;
  p.T = P.S.T;
  p.N = P.S.N;
  p.H = P.S.H;
  p.Hk = P.S.Hk;
  p.rotary = d->rotary_dim;
  p.interleaved = d->interleaved;
  p.eps = d->eps;
  p.q_s = P.q_s;
  p.k_s = P.k_s;
  p.v_s = P.v_s;
  return p;
}

// Packed offsets, which the kernels search for a token's document: few go along with the parameters, more to the device first.
int rope_offsets(const RopeProblem& P, const RopeLayout& l, void* ws, RopeParams* p, cudaStream_t s) {
  if (!P.S.cu) return GDN_OK;
  p->packed = true;
  if (P.S.N + 1 <= kRopeInline) {
    std::copy(P.S.cu, P.S.cu + P.S.N + 1, p->few);
    return GDN_OK;
  }
  int* cu = reinterpret_cast<int*>(static_cast<char*>(ws) + l.cu);
  p->cu = cu;
  return upload_offsets(P.S.cu, P.S.N + 1, cu, s);
}

int rope_fwd(const gdn_rope_desc_t* d, const gdn_rope_args_t* a, void* stream, bool store) {
  RopeProblem P{};
  int rc = validate_rope(d, &P, store);
  if (rc) return rc;
  if (!a || !a->q || !a->k || !a->q_out || !a->k_out) return bad("q, k, q_out and k_out must be non-NULL");
  if (!a->q_weight != !a->k_weight) return bad("q_weight and k_weight must both be given or both be NULL");
  if (d->rotary_dim && !a->inv_freq) return bad("inv_freq must be non-NULL with a rotation");
  if (store && (!a->v || !a->k_cache || !a->v_cache || !a->page_table || !a->lengths)) return bad("v, the caches, page_table and lengths must be non-NULL");
  if (store && a->positions) return bad("positions must be NULL with a store");
  for (const void* x : {a->q, a->k, store ? a->v : a->q, (const void*)a->q_out, (const void*)a->k_out, (const void*)a->k_cache, (const void*)a->v_cache})
    if (!aligned(x, 16)) return bad("q, k, v, the outputs and the caches must be 16-byte aligned");
  const size_t cache = store ? size_t(d->num_pages) * d->page_size * P.S.Hk * P.S.D * 2 : 0;
  const size_t qb = size_t(P.S.rows) * P.S.H * P.S.D * 2, kb = size_t(P.S.rows) * P.S.Hk * P.S.D * 2;
  const Span in[] = {{a->q, extent(P.S.rows, P.q_s, P.S.H, P.S.D)}, {a->k, extent(P.S.rows, P.k_s, P.S.Hk, P.S.D)},
                     {store ? a->v : nullptr, extent(P.S.rows, P.v_s, P.S.Hk, P.S.D)}};
  const Span out[] = {{a->q_out, qb}, {a->k_out, kb}, {store ? a->k_cache : nullptr, cache}, {store ? a->v_cache : nullptr, cache}};
  if (alias(in, out)) return bad("outputs and caches must not alias the inputs or each other");
  const RopeLayout l = layout_rope(P);
  if (P.S.cu && !workspace_ok(a->workspace, a->workspace_bytes, l.total)) return bad("workspace missing, too small or not 256-byte aligned");
  RopeParams p = rope_params(d, P);
  if ((rc = device_or_error(&p.sms))) return rc;
  p.q = static_cast<cbf*>(a->q);
  p.k = static_cast<cbf*>(a->k);
  p.qw = a->q_weight;
  p.kw = a->k_weight;
  p.inv_freq = a->inv_freq;
  p.positions = a->positions;
  p.qo = static_cast<bf*>(a->q_out);
  p.ko = static_cast<bf*>(a->k_out);
  if (store) {
    p.v = static_cast<cbf*>(a->v);
    p.lengths = a->lengths;
    p.table = a->page_table;
    p.pages = d->num_pages;
    p.page = d->page_size;
    p.width = d->table_width;
    p.kc = static_cast<bf*>(a->k_cache);
    p.vc = static_cast<bf*>(a->v_cache);
    p.status = a->status;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKRopeFwd, s);
  if ((rc = rope_offsets(P, l, a->workspace, &p, s))) return rc;
  return cuda_rc(launch_rope_fwd(p, P.S.D, s), "norm and rotation kernel");
}

// ------------------------------------------------------------------ attention over whole sequences

struct AttnProblem {
  Shape S;
  long long q_s, k_s, v_s;
  float scale;
  long long pairs, tiles;  // tiles of 256 and of 128 tokens of all sequences
};

int validate_attn(const gdn_attn_desc_t* d, AttnProblem* P) {
  if (!d) return bad("desc is NULL");
  int rc = check_heads(d->H, d->num_k_heads, d->head_dim, &P->S);
  if (!rc) rc = check_sequences(d, &P->S);
  if (rc) return rc;
  if (d->causal != 0 && d->causal != 1) return bad("causal must be 0 or 1");
  if (std::isnan(d->scale) || std::isinf(d->scale)) return bad("scale must be finite");
  P->scale = d->scale > 0.f ? d->scale : 1.f / std::sqrt(float(P->S.D));
  P->q_s = stride_of(d->q_stride, P->S.H, P->S.D);
  P->k_s = stride_of(d->k_stride, P->S.Hk, P->S.D);
  P->v_s = stride_of(d->v_stride, P->S.Hk, P->S.D);
  if (P->q_s < 0 || P->k_s < 0 || P->v_s < 0) return bad("strides must be multiples of 8, at least a token's heads");
  auto count = [&](long long step) {
    if (!P->S.cu) return (P->S.T + step - 1) / step * P->S.N;
    long long n = 0;
    for (int i = 0; i < P->S.N; ++i) n += (P->S.cu[i + 1] - P->S.cu[i] + step - 1) / step;
    return n;
  };
  P->pairs = count(kAttnPair);
  P->tiles = count(kAttnTile);
  if (P->tiles * P->S.H >= (1ll << 31)) return bad("problem too large");
  return GDN_OK;
}

size_t table_bytes(const AttnProblem& P, long long tiles) { return P.S.cu ? align256(size_t(tiles) * 12) : 0; }

// Packed documents: {first row, length, first token} of every tile of `step` tokens, a sequence's last tiles first (or its first
// ones, `ascending`), level by level through the sequences, longest first: the tiles with the most work start first. Few go along
// with the parameters, more to the device first.
int pack_tiles(const AttnProblem& P, int step, bool ascending, AttnParams* p, int* dst, cudaStream_t s) {
  const int32_t* cu = P.S.cu;
  std::vector<int> order(P.S.N);
  for (int i = 0; i < P.S.N; ++i) order[i] = i;
  std::stable_sort(order.begin(), order.end(), [cu](int a, int b) { return cu[a + 1] - cu[a] > cu[b + 1] - cu[b]; });
  std::vector<int32_t> table;
  table.reserve(size_t(3) * (step == kAttnPair ? P.pairs : P.tiles));
  auto tiles = [&](int i) { return (cu[order[i] + 1] - cu[order[i]] + step - 1) / step; };
  const int most = tiles(0);
  for (int k = 0; k < most; ++k) {
    // `left`: tiles that follow this one's level in work; a sequence takes part while it has that many
    const int left = most - k;
    for (int i = 0; i < P.S.N && tiles(i) >= left; ++i) {
      const int n = order[i], level = ascending ? tiles(i) - left : left - 1;
      table.push_back(cu[n]);
      table.push_back(cu[n + 1] - cu[n]);
      table.push_back(level * step);
    }
  }
  p->packed = true;
  if (table.size() <= 3 * kAttnInline) {
    std::copy(table.begin(), table.end(), p->few);
    return GDN_OK;
  }
  p->table = dst;
  return upload_offsets(table.data(), int(table.size()), dst, s);
}

AttnParams attn_params(const gdn_attn_desc_t* d, const AttnProblem& P) {
  AttnParams p{};
  p.H = P.S.H;
  p.Hk = P.S.Hk;
  p.group = P.S.H / P.S.Hk;
  p.T = P.S.T;
  p.N = P.S.N;
  p.causal = d->causal;
  p.scale = P.scale;
  p.rows = P.S.rows;
  return p;
}

bool input_maps(const AttnProblem& P, const void* q, const void* k, const void* v, CUtensorMap* mq, CUtensorMap* mk, CUtensorMap* mv) {
  const uint64_t D = P.S.D, R = P.S.rows;
  return attn_map(mq, q, P.S.H * D, R, P.q_s, kAttnTile) && attn_map(mk, k, P.S.Hk * D, R, P.k_s, kAttnTile) && attn_map(mv, v, P.S.Hk * D, R, P.v_s, kAttnTile);
}

size_t attn_fwd_ws(const AttnProblem& P) { return align256(std::max<size_t>(table_bytes(P, P.pairs), 1)); }

int attn_fwd(const gdn_attn_desc_t* d, const gdn_attn_fwd_args_t* a, void* stream) {
  AttnProblem P{};
  int rc = validate_attn(d, &P);
  if (rc) return rc;
  if (!a || !a->q || !a->k || !a->v || !a->o || !a->lse) return bad("q, k, v, o and lse must be non-NULL");
  for (const void* x : {a->q, a->k, a->v, (const void*)a->o})
    if (!aligned(x, 16)) return bad("q, k, v and o must be 16-byte aligned");
  const Span in[] = {{a->q, extent(P.S.rows, P.q_s, P.S.H, P.S.D)}, {a->k, extent(P.S.rows, P.k_s, P.S.Hk, P.S.D)}, {a->v, extent(P.S.rows, P.v_s, P.S.Hk, P.S.D)}};
  const Span out[] = {{a->o, size_t(P.S.rows) * P.S.H * P.S.D * 2}, {a->lse, size_t(P.S.rows) * P.S.H * 4}};
  if (alias(in, out)) return bad("o and lse must not alias the inputs or each other");
  if (P.S.cu && !workspace_ok(a->workspace, a->workspace_bytes, attn_fwd_ws(P))) return bad("workspace missing, too small or not 256-byte aligned");
  AttnParams p = attn_params(d, P);
  if ((rc = device_or_error(&p.sms)) || (rc = bind_context())) return rc;
  p.tiles = int(P.pairs);
  p.o = static_cast<bf*>(a->o);
  p.lse = a->lse;
  p.status = a->status;
  CUtensorMap mq, mk, mv;
  if (!input_maps(P, a->q, a->k, a->v, &mq, &mk, &mv)) return set_last_error(GDN_ECUDA, "cuTensorMapEncodeTiled failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKAttnFwd, s);
  if (P.S.cu && (rc = pack_tiles(P, kAttnPair, false, &p, static_cast<int*>(a->workspace), s))) return rc;
  return cuda_rc(launch_attn_fwd(mq, mk, mv, P.S.D, p, s), "attention kernel");
}

struct AttnBwdLayout {
  size_t order, keys, lse2, delta, counters, total;
};
AttnBwdLayout layout_attn_bwd(const AttnProblem& P) {
  AttnBwdLayout l{};
  l.keys = table_bytes(P, P.tiles);
  l.lse2 = 2 * l.keys;
  const size_t n = align256(size_t(P.S.rows) * P.S.H * 4);
  l.delta = l.lse2 + n;
  l.counters = l.delta + n;
  l.total = l.counters + 256;
  return l;
}

int attn_bwd(const gdn_attn_desc_t* d, const gdn_attn_bwd_args_t* a, void* stream) {
  AttnProblem P{};
  int rc = validate_attn(d, &P);
  if (rc) return rc;
  if (!a || !a->q || !a->k || !a->v || !a->o || !a->lse || !a->dO || !a->dq || !a->dk || !a->dv)
    return bad("q, k, v, o, lse, dO, dq, dk and dv must be non-NULL");
  for (const void* x : {a->q, a->k, a->v, a->o, a->dO, (const void*)a->dq, (const void*)a->dk, (const void*)a->dv})
    if (!aligned(x, 16)) return bad("q, k, v, o, dO and the gradients must be 16-byte aligned");
  const size_t qb = size_t(P.S.rows) * P.S.H * P.S.D * 2, kb = size_t(P.S.rows) * P.S.Hk * P.S.D * 2;
  const Span in[] = {{a->q, extent(P.S.rows, P.q_s, P.S.H, P.S.D)}, {a->k, extent(P.S.rows, P.k_s, P.S.Hk, P.S.D)}, {a->v, extent(P.S.rows, P.v_s, P.S.Hk, P.S.D)},
                     {a->o, qb}, {a->dO, qb}, {a->lse, size_t(P.S.rows) * P.S.H * 4}};
  const Span out[] = {{a->dq, qb}, {a->dk, kb}, {a->dv, kb}};
  if (alias(in, out)) return bad("the gradients must not alias the inputs or each other");
  const AttnBwdLayout l = layout_attn_bwd(P);
  if (!workspace_ok(a->workspace, a->workspace_bytes, l.total)) return bad("workspace missing, too small or not 256-byte aligned");
  AttnParams p = attn_params(d, P);
  if ((rc = device_or_error(&p.sms)) || (rc = bind_context())) return rc;
  char* ws = static_cast<char*>(a->workspace);
  p.tiles = int(P.tiles);
  p.dO = static_cast<cbf*>(a->dO);
  p.o_in = static_cast<cbf*>(a->o);
  p.lse_in = a->lse;
  p.lse2 = reinterpret_cast<float*>(ws + l.lse2);
  p.delta = reinterpret_cast<float*>(ws + l.delta);
  p.counters = reinterpret_cast<unsigned*>(ws + l.counters);
  p.dq = static_cast<bf*>(a->dq);
  p.dk = static_cast<bf*>(a->dk);
  p.dv = static_cast<bf*>(a->dv);
  p.status = a->status;
  CUtensorMap mq, mk, mv, mdo;
  if (!input_maps(P, a->q, a->k, a->v, &mq, &mk, &mv) || !attn_map(&mdo, a->dO, uint64_t(P.S.H) * P.S.D, P.S.rows, uint64_t(P.S.H) * P.S.D, kAttnTile))
    return set_last_error(GDN_ECUDA, "cuTensorMapEncodeTiled failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKAttnBwd, s);
  AttnParams pk = p;
  if (P.S.cu && ((rc = pack_tiles(P, kAttnTile, false, &p, reinterpret_cast<int*>(ws + l.order), s)) ||
                 (rc = pack_tiles(P, kAttnTile, true, &pk, reinterpret_cast<int*>(ws + l.keys), s))))
    return rc;
  return cuda_rc(launch_attn_bwd(mq, mk, mv, mdo, P.S.D, p, pk, s), "attention backward kernels");
}

// ------------------------------------------------------------------ single tokens

struct AttnStepProblem {
  Shape S;
  long long q_s;
  float scale;
  int parts, shares;
};

int validate_step(const gdn_attn_step_desc_t* d, AttnStepProblem* P) {
  if (!d) return bad("desc is NULL");
  const int rc = check_heads(d->H, d->num_k_heads, d->head_dim, &P->S);
  if (rc) return rc;
  if (d->B < 1) return bad("B must be positive");
  if (std::isnan(d->scale) || std::isinf(d->scale)) return bad("scale must be finite");
  if (d->num_pages < 1 || d->page_size < 1 || d->table_width < 1) return bad("num_pages, page_size and table_width must be positive");
  const long long room = (long long)d->table_width * d->page_size;
  if (room > (1ll << 30)) return bad("the page table spans too many tokens");
  P->S.B = d->B;
  P->scale = d->scale > 0.f ? d->scale : 1.f / std::sqrt(float(P->S.D));
  P->q_s = stride_of(d->q_stride, P->S.H, P->S.D);
  if (P->q_s < 0) return bad("q_stride must be a multiple of 8, at least a row");
  const int group = P->S.H / P->S.Hk, rows = attn_step_rows(group);
  P->parts = P->S.Hk * ((group + rows - 1) / rows);
  if ((long long)d->B * P->S.H >= (1ll << 31)) return bad("problem too large");
  P->shares = int(std::min((long long)std::max(1, attn_step_blocks(P->S.D, rows) / P->parts), d->B * ((room + 63) / 64)));
  return GDN_OK;
}

struct StepLayout {
  size_t ml, span, total;
};
StepLayout layout_step(const AttnStepProblem& P) {
  StepLayout l{};
  const size_t rows = (size_t(P.S.B) + P.shares) * P.parts * attn_step_rows(P.S.H / P.S.Hk);
  l.ml = align256(rows * P.S.D * 4);
  l.span = l.ml + align256(rows * 8);
  l.total = l.span + align256(size_t(P.S.B) * P.parts * 8);
  return l;
}

int attn_step(const gdn_attn_step_desc_t* d, const gdn_attn_step_args_t* a, void* stream) {
  AttnStepProblem P{};
  int rc = validate_step(d, &P);
  if (rc) return rc;
  if (!a || !a->q || !a->k_cache || !a->v_cache || !a->page_table || !a->lengths || !a->o) return bad("q, the caches, page_table, lengths and o must be non-NULL");
  for (const void* x : {a->q, a->k_cache, a->v_cache})
    if (!aligned(x, 16)) return bad("q and the caches must be 16-byte aligned");
  const size_t cache = size_t(d->num_pages) * d->page_size * P.S.Hk * P.S.D * 2;
  const Span in[] = {{a->q, extent(d->B, P.q_s, P.S.H, P.S.D)}, {a->k_cache, cache}, {a->v_cache, cache}}, out[] = {{a->o, size_t(d->B) * P.S.H * P.S.D * 2}};
  if (alias(in, out)) return bad("o must not alias the inputs");
  if (!workspace_ok(a->workspace, a->workspace_bytes, layout_step(P).total)) return bad("workspace missing, too small or not 256-byte aligned");
  if ((rc = device_or_error(nullptr))) return rc;
  AttnStepParams p{};
  p.B = d->B;
  p.H = P.S.H;
  p.Hk = P.S.Hk;
  p.group = P.S.H / P.S.Hk;
  p.pages = d->num_pages;
  p.page = d->page_size;
  p.width = d->table_width;
  p.shares = P.shares;
  p.scale = P.scale;
  p.q_stride = P.q_s;
  p.q = static_cast<cbf*>(a->q);
  p.kc = static_cast<cbf*>(a->k_cache);
  p.vc = static_cast<cbf*>(a->v_cache);
  p.table = a->page_table;
  p.lengths = a->lengths;
  p.o = static_cast<bf*>(a->o);
  const StepLayout l = layout_step(P);
  char* ws = static_cast<char*>(a->workspace);
  p.part = reinterpret_cast<float*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + l.ml);
  p.span = reinterpret_cast<int2*>(ws + l.span);
  p.status = a->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKAttnStep, s);
  return cuda_rc(launch_attn_step(p, P.S.D, s), "attention step kernel");
}

// The tile tables are built in host memory, which can run out: no exception leaves a C entry point.
template <class F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::exception&) {
    return set_last_error(GDN_ECUDA, "out of host memory");
  }
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_qk_norm_rope_workspace_size(const gdn_rope_desc_t* d) {
  RopeProblem P{};
  return validate_rope(d, &P, false) ? 0 : layout_rope(P).total;
}
int gdn_qk_norm_rope_fwd(const gdn_rope_desc_t* d, const gdn_rope_args_t* a, void* s) { return rope_fwd(d, a, s, false); }
int gdn_qk_norm_rope_store(const gdn_rope_desc_t* d, const gdn_rope_args_t* a, void* s) { return rope_fwd(d, a, s, true); }

int gdn_qk_norm_rope_bwd(const gdn_rope_desc_t* d, const gdn_rope_bwd_args_t* a, void* stream) {
  RopeProblem P{};
  int rc = validate_rope(d, &P, false);
  if (rc) return rc;
  if (!a || !a->q || !a->k || !a->dq_out || !a->dk_out || !a->dq || !a->dk) return bad("q, k, dq_out, dk_out, dq and dk must be non-NULL");
  if (!a->q_weight != !a->k_weight) return bad("q_weight and k_weight must both be given or both be NULL");
  if (!a->q_weight != !a->dq_weight || !a->k_weight != !a->dk_weight) return bad("dq_weight and dk_weight go with the weights");
  if (d->rotary_dim && !a->inv_freq) return bad("inv_freq must be non-NULL with a rotation");
  for (const void* x : {a->q, a->k, a->dq_out, a->dk_out, (const void*)a->dq, (const void*)a->dk})
    if (!aligned(x, 16)) return bad("q, k and the gradients must be 16-byte aligned");
  const size_t qb = size_t(P.S.rows) * P.S.H * P.S.D * 2, kb = size_t(P.S.rows) * P.S.Hk * P.S.D * 2;
  const Span in[] = {{a->q, extent(P.S.rows, P.q_s, P.S.H, P.S.D)}, {a->k, extent(P.S.rows, P.k_s, P.S.Hk, P.S.D)}, {a->dq_out, qb}, {a->dk_out, kb}};
  const Span out[] = {{a->dq, qb}, {a->dk, kb}, {a->dq_weight, size_t(P.S.D) * 4}, {a->dk_weight, size_t(P.S.D) * 4}};
  if (alias(in, out)) return bad("outputs must not alias the inputs or each other");
  const RopeLayout l = layout_rope(P);
  if (!workspace_ok(a->workspace, a->workspace_bytes, l.total)) return bad("workspace missing, too small or not 256-byte aligned");
  RopeParams p = rope_params(d, P);
  if ((rc = device_or_error(&p.sms))) return rc;
  p.q = static_cast<cbf*>(a->q);
  p.k = static_cast<cbf*>(a->k);
  p.qw = a->q_weight;
  p.kw = a->k_weight;
  p.inv_freq = a->inv_freq;
  p.positions = a->positions;
  p.dqo = static_cast<cbf*>(a->dq_out);
  p.dko = static_cast<cbf*>(a->dk_out);
  p.dq = static_cast<bf*>(a->dq);
  p.dk = static_cast<bf*>(a->dk);
  p.dqw = a->dq_weight;
  p.dkw = a->dk_weight;
  p.part = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + l.part);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKRopeBwd, s);
  if ((rc = rope_offsets(P, l, a->workspace, &p, s))) return rc;
  return cuda_rc(launch_rope_bwd(p, P.S.D, s), "norm and rotation backward kernels");
}

size_t gdn_attn_fwd_workspace_size(const gdn_attn_desc_t* d) {
  AttnProblem P{};
  return validate_attn(d, &P) ? 0 : attn_fwd_ws(P);
}
int gdn_attn_fwd(const gdn_attn_desc_t* d, const gdn_attn_fwd_args_t* a, void* s) {
  return guarded([&] { return attn_fwd(d, a, s); });
}

size_t gdn_attn_bwd_workspace_size(const gdn_attn_desc_t* d) {
  AttnProblem P{};
  return validate_attn(d, &P) ? 0 : layout_attn_bwd(P).total;
}
int gdn_attn_bwd(const gdn_attn_desc_t* d, const gdn_attn_bwd_args_t* a, void* s) {
  return guarded([&] { return attn_bwd(d, a, s); });
}

size_t gdn_attn_step_workspace_size(const gdn_attn_step_desc_t* d) {
  AttnStepProblem P{};
  return validate_step(d, &P) ? 0 : layout_step(P).total;
}
int gdn_attn_step(const gdn_attn_step_desc_t* d, const gdn_attn_step_args_t* a, void* s) { return attn_step(d, a, s); }

}  // extern "C"
