// Host side of the operators around the recurrence (declared in include/gdn.h): contract validation, workspace layout,
// the selective scan's segment plan, and the launches.
#include <algorithm>
#include <cmath>

#include "block_ops.cuh"
#include "conv.cuh"
#include "gdn.h"
#include "host.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------ norms

int validate_norm(const gdn_norm_desc_t* d, bool gated) {
  if (!d) return bad("desc is NULL");
  if (d->rows < 1 || d->width < 1 || d->width > kNormMaxWidth) return bad("rows >= 1 and width in 1..16384 required");
  if (d->rows > (1ll << 40) / d->width) return bad("problem too large");
  if (!(d->eps >= 0.f) || std::isinf(d->eps)) return bad("eps must be finite and not negative");
  if (gated) {
    if (d->activation != 1 && d->activation != 2) return bad("activation must be 1 (SiLU) or 2 (sigmoid)");
    return GDN_OK;
  }
  if (d->stream_kind < 0 || d->stream_kind > 2) return bad("stream_kind must be 0, 1 or 2");
  if (std::isnan(d->residual_scale) || std::isinf(d->residual_scale)) return bad("residual_scale must be finite");
  if (d->stream_kind == 0 && d->residual_scale != 1.f) return bad("residual_scale must be 1 without a residual");
  return GDN_OK;
}

NormParams norm_params(const gdn_norm_desc_t* d) {
  NormParams p{};
  p.rows = d->rows;
  p.width = d->width;
  p.eps = d->eps;
  p.scale = d->residual_scale;
  p.stream_kind = d->stream_kind;
  p.act = d->activation;
  return p;
}

int norm_fwd(const gdn_norm_desc_t* d, const gdn_norm_fwd_args_t* a, void* stream, bool gated) {
  int rc = validate_norm(d, gated);
  if (rc) return rc;
  const size_t n = size_t(d->rows) * d->width, sb = n * (d->stream_kind == 2 ? 4 : 2);
  if (!a || !a->x || !a->weight || !a->y) return bad("x, weight and y must be non-NULL");
  if (overlap(a->y, n * 2, a->x, n * 2)) return bad("y must not alias x");
  NormParams p = norm_params(d);
  p.x = static_cast<const __nv_bfloat16*>(a->x);
  p.weight = a->weight;
  p.y = static_cast<__nv_bfloat16*>(a->y);
  if (gated) {
    if (!a->residual) return bad("the gate must be non-NULL");
    if (overlap(a->y, n * 2, a->residual, n * 2)) return bad("y must not alias the gate");
    p.gate = static_cast<const __nv_bfloat16*>(a->residual);
  } else if (d->stream_kind) {
    if (!a->residual || !a->stream) return bad("residual and stream must be non-NULL with a residual");
    if (overlap(a->stream, sb, a->x, n * 2) || overlap(a->stream, sb, a->y, n * 2) || overlap(a->y, n * 2, a->residual, sb) ||
        (a->stream != a->residual && overlap(a->stream, sb, a->residual, sb)))
      return bad("stream must not alias x or y, nor residual except in place; y must not alias residual");
    p.residual = a->residual;
    p.stream = a->stream;
  } else if (a->residual || a->stream) {
    return bad("residual and stream must be NULL without a residual (stream_kind 0)");
  }
  if ((rc = device_or_error(&p.sms))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKNormFwd, s);
  return cuda_rc(gated ? launch_gated_norm_fwd(p, s) : launch_add_norm_fwd(p, s), "norm kernel");
}

size_t norm_ws(const gdn_norm_desc_t* d) { return align256(size_t(norm_partial_rows()) * d->width * 4); }

int norm_bwd(const gdn_norm_desc_t* d, const gdn_norm_bwd_args_t* a, void* stream, bool gated) {
  int rc = validate_norm(d, gated);
  if (rc) return rc;
  if (!a || !a->x || !a->weight || !a->dy || !a->dx || !a->dweight) return bad("x, weight, dy, dx and dweight must be non-NULL");
  if (gated && (!a->gate || !a->dgate)) return bad("gate and dgate must be non-NULL");
  if (!gated && a->dresidual && !d->stream_kind) return bad("dresidual needs a residual");
  const size_t n = size_t(d->rows) * d->width, sb = n * (!gated && d->stream_kind == 2 ? 4 : 2);
  const struct { const void* p; size_t n; } in[] = {{a->x, sb}, {a->dy, n * 2}, {gated ? a->gate : a->dstream, gated ? n * 2 : sb}};
  const struct { const void* p; size_t n; } out[] = {{a->dx, n * 2}, {gated ? a->dgate : a->dresidual, gated ? n * 2 : sb}};
  for (const auto& o : out)
    for (const auto& i : in)
      if (overlap(o.p, o.n, i.p, i.n)) return bad("an output must not alias an input");
  if (overlap(out[0].p, out[0].n, out[1].p, out[1].n)) return bad("the outputs must not alias each other");
  if (!a->workspace || a->workspace_bytes < norm_ws(d) || !aligned(a->workspace, 256))
    return bad("workspace missing, too small or not 256-byte aligned");
  NormParams p = norm_params(d);
  if ((rc = device_or_error(&p.sms))) return rc;
  p.weight = a->weight;
  p.dy = static_cast<const __nv_bfloat16*>(a->dy);
  p.dx = static_cast<__nv_bfloat16*>(a->dx);
  p.dweight = a->dweight;
  p.part = static_cast<float*>(a->workspace);
  if (gated) {
    p.x = static_cast<const __nv_bfloat16*>(a->x);
    p.gate = static_cast<const __nv_bfloat16*>(a->gate);
    p.dgate = static_cast<__nv_bfloat16*>(a->dgate);
  } else {
    p.stream = const_cast<void*>(a->x);
    p.dstream = a->dstream;
    p.dresidual = a->dresidual;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKNormBwd, s);
  return cuda_rc(gated ? launch_gated_norm_bwd(p, s) : launch_add_norm_bwd(p, s), "norm backward kernels");
}

// ------------------------------------------------------------------ selective scan

struct SscanProblem {
  int B, T, D, N, G, seqs;
  long long rows;
  const int32_t* cu;  // the caller's host offsets, or null
  long long u_s, dt_s, z_s, b_s, c_s;
};

int sequence_length(const SscanProblem& P, int i) { return P.cu ? P.cu[i + 1] - P.cu[i] : P.T; }

int validate_sscan(const gdn_sscan_desc_t* d, SscanProblem* P, bool step) {
  if (!d) return bad("desc is NULL");
  if (d->B < 1 || d->D < 1 || (!step && d->T < 1)) return bad("B, T and D must be positive");
  if (d->N < 1 || d->N > kSscanMaxN) return bad("N must be 1..16");
  if (d->G < 1 || d->D % d->G) return bad("G must divide D");
  if (d->D > (1 << 24)) return bad("D too large");
  P->B = d->B;
  P->T = step ? 1 : d->T;
  P->D = d->D;
  P->N = d->N;
  P->G = d->G;
  P->rows = (long long)d->B * P->T;
  if (P->rows > (1ll << 30)) return bad("B*T too large");
  const long long gn = (long long)d->G * d->N;
  P->u_s = d->u_stride ? d->u_stride : d->D;
  P->dt_s = d->delta_stride ? d->delta_stride : d->D;
  P->z_s = d->z_stride ? d->z_stride : d->D;
  P->b_s = d->B_stride ? d->B_stride : gn;
  P->c_s = d->C_stride ? d->C_stride : gn;
  if (P->u_s < d->D || P->dt_s < d->D || P->z_s < d->D || P->b_s < gn || P->c_s < gn) return bad("a token stride is shorter than a token");
  for (long long st : {P->u_s, P->dt_s, P->z_s, P->b_s, P->c_s})
    if (st > (1ll << 26)) return bad("a token stride is too large");
  P->cu = d->cu_seqlens;
  P->seqs = d->B;
  if (P->cu) {
    if (step) return bad("a step takes no cu_seqlens");
    if (d->B != 1) return bad("packed documents (cu_seqlens) require batch size 1");
    if (d->num_seqs < 1) return bad("num_seqs must be >= 1 with cu_seqlens");
    if (P->cu[0] != 0) return bad("cu_seqlens must start at 0");
    for (int i = 0; i < d->num_seqs; ++i)
      if (P->cu[i + 1] <= P->cu[i]) return bad("cu_seqlens must be strictly increasing (no empty documents)");
    if (P->cu[d->num_seqs] != d->T) return bad("cu_seqlens must end at T");
    P->seqs = d->num_seqs;
  }
  return GDN_OK;
}

// Segments. One CTA walks kSscanChans channels of one segment token by token, so a call needs CTAs enough for every SM;
// cutting the sequences costs the map pass, which walks all segments but the last ones again. The times compared are in
// steps of one CTA among others on its SM: whole sequences take the longest one's steps, at `alone` each while the SM has
// few CTAs, or one CTA after the other when there are more; cut ones take all steps and the map's, evenly spread but no fewer
// than a shortest segment's, and two more kernels. Of the lengths that fill one to `rounds` rounds of resident CTAs, the one whose rounds and fixed cost per CTA are least is taken.
struct SscanPlan {
  int L;                 // tokens per segment, a multiple of kSscanCut
  int most;              // most segments of a sequence
  long long segs, cks;   // segments and kept states of all sequences
};
constexpr int kSms = 152;
constexpr int kMinSegment = 32, kCtaTokens = 12;
struct SscanCost {
  int ctas, first, last; // resident CTAs per SM, and the rounds of them that are tried
  double alone, map;     // a step of a CTA alone on its SM, and of the map pass
  double launches;       // the map and compose kernels
};
constexpr SscanCost kFwdCost = {8, 1, 3, 2.4, 0.7, 120.0}, kBwdCost = {3, 4, 4, 2.0, 0.3, 60.0};

long long count_segments(const SscanProblem& P, long long L) {
  if (!P.cu) return (P.T + L - 1) / L * P.seqs;
  long long n = 0;
  for (int i = 0; i < P.seqs; ++i) n += (sequence_length(P, i) + L - 1) / L;
  return n;
}

SscanPlan plan_sscan(const SscanProblem& P, bool backward) {
  const SscanCost& c = backward ? kBwdCost : kFwdCost;
  const long long blocks = sscan_blocks(P.G, P.D / P.G), slots = (long long)kSms * c.ctas;
  int longest = P.T;
  if (P.cu) {
    longest = 0;
    for (int i = 0; i < P.seqs; ++i) longest = std::max(longest, sequence_length(P, i));
  }
  const double whole = longest * std::max(c.alone, double((P.seqs * blocks + kSms - 1) / kSms));
  const double cut = (1.0 + c.map) * std::max(double(P.rows) * blocks / kSms, c.alone * kMinSegment) + c.launches;
  const long long all = ((long long)longest + kSscanCut - 1) / kSscanCut * kSscanCut;
  long long best = all, least = 0;
  if (cut < whole) {
    for (int r = c.first; r <= c.last; ++r) {
      const long long unit = slots * r * kSscanCut;
      const long long L = std::min(all, std::max<long long>(kMinSegment, (P.rows * blocks + unit - 1) / unit * kSscanCut));
      const long long rounds = (count_segments(P, L) * blocks + slots - 1) / slots, cost = rounds * (L + kCtaTokens);
      if (!least || cost < least) least = cost, best = L;
    }
  }
  SscanPlan q{};
  q.L = int(best);
  q.segs = count_segments(P, best);
  q.most = int((longest + best - 1) / best);
  q.cks = count_segments(P, kSscanBlock);
  return q;
}

struct SscanLayout {
  size_t tables, seg_state, seg_dt, part_bc, part_par, ck, total;
};

size_t saved_bytes(const SscanProblem& P, const SscanPlan& q) { return align256(size_t(q.cks) * P.N * P.D * 4); }

SscanLayout layout_sscan(const SscanProblem& P, const SscanPlan& q, bool backward) {
  SscanLayout l{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  // a workspace is never empty: 0 bytes would read as an invalid description
  l.tables = take(P.cu ? size_t(P.seqs + 1) * 3 * 4 : 4);
  if (q.most > 1) {
    l.seg_state = take(size_t(q.segs) * P.N * P.D * 4);
    l.seg_dt = take(size_t(q.segs) * P.D * 4);
  }
  if (backward) {
    l.part_bc = take(size_t(sscan_blocks(P.G, P.D / P.G, kSscanBwdChans)) * P.rows * 2 * P.N * 4);
    l.part_par = take(size_t(q.segs) * (P.N + 2) * P.D * 4);
  }
  l.total = off;
  return l;
}

int check_sscan_size(const SscanProblem& P, const SscanPlan& q) {
  const long long blocks = sscan_blocks(P.G, P.D / P.G);
  if (2 * blocks * q.segs >= (1ll << 31) || P.rows * P.G * 2 * P.N >= (1ll << 38) || (long long)P.seqs * P.N * P.D >= (1ll << 38))
    return bad("problem too large");
  return GDN_OK;
}

// Offsets, then the running counts of segments, then of kept states (seqs + 1 each), uploaded through kernel parameters: as one
// array, so that a call with up to kMaxUploadInts / 3 documents takes one launch.
int upload_tables(const SscanProblem& P, const SscanPlan& q, int* dst, cudaStream_t s) {
  int32_t buf[kMaxUploadInts];
  const long long per = P.seqs + 1ll;
  int fill = 0;
  long long at = 0;
  for (int which = 0; which < 3; ++which) {
    long long run = 0;
    for (int i = 0; i <= P.seqs; ++i) {
      buf[fill++] = which == 0 ? P.cu[i] : int32_t(run);
      if (which && i < P.seqs) run += which == 1 ? (sequence_length(P, i) + q.L - 1) / q.L : (sequence_length(P, i) + kSscanBlock - 1) / kSscanBlock;
      if (fill == kMaxUploadInts || (which == 2 && i == P.seqs)) {
        const int rc = upload_offsets(buf, fill, dst + at, s);
        if (rc) return rc;
        at += fill;
        fill = 0;
      }
    }
  }
  return at == 3 * per ? GDN_OK : bad("internal: table upload");
}

void fill(const SscanProblem& P, const SscanPlan& q, const SscanLayout& l, char* ws, SscanParams* p) {
  p->T = P.T;
  p->D = P.D;
  p->N = P.N;
  p->G = P.G;
  p->Dg = P.D / P.G;
  p->seqs = P.seqs;
  p->rows = P.rows;
  p->L = q.L;
  p->segs = int(q.segs);
  p->u_s = P.u_s;
  p->dt_s = P.dt_s;
  p->z_s = P.z_s;
  p->b_s = P.b_s;
  p->c_s = P.c_s;
  if (P.cu) {
    int* t = reinterpret_cast<int*>(ws + l.tables);
    p->cu = t;
    p->seg_base = t + (P.seqs + 1);
    p->ck_base = t + 2 * size_t(P.seqs + 1);
  } else {
    p->nseg_dense = q.most;
    p->nck_dense = (P.T + kSscanBlock - 1) / kSscanBlock;
  }
  p->seg_state = nullptr;
  if (q.most > 1) {
    p->seg_state = reinterpret_cast<float*>(ws + l.seg_state);
    p->seg_dt = reinterpret_cast<float*>(ws + l.seg_dt);
  }
}

// Whether all channel blocks' rows start on 16-byte boundaries: the tensors, their strides and the groups.
void set_vectors(const SscanProblem& P, SscanParams* p) {
  p->vec_A = aligned(p->A, 16);
  p->pair = P.D % 2 == 0 && (P.D / P.G) % 2 == 0;
  p->quad = P.D % 4 == 0 && (P.D / P.G) % 4 == 0;
  const bool groups = P.G == 1 || (P.D / P.G) % 8 == 0;
  p->vec = groups && aligned(p->u, 16) && aligned(p->delta, 16) && aligned(p->z, 16) && aligned(p->dy, 16) && P.u_s % 8 == 0 &&
           P.dt_s % 8 == 0 && (!p->z || P.z_s % 8 == 0) && (!p->dy || P.D % 8 == 0);
  p->vec_out = groups && P.D % 8 == 0 && aligned(p->y, 16) && aligned(p->du, 16) && aligned(p->ddelta, 16) && aligned(p->dz, 16);
}

using bf = __nv_bfloat16;
using cbf = const __nv_bfloat16;

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_add_norm_fwd(const gdn_norm_desc_t* d, const gdn_norm_fwd_args_t* a, void* s) { return norm_fwd(d, a, s, false); }
int gdn_gated_norm_fwd(const gdn_norm_desc_t* d, const gdn_norm_fwd_args_t* a, void* s) { return norm_fwd(d, a, s, true); }
int gdn_add_norm_bwd(const gdn_norm_desc_t* d, const gdn_norm_bwd_args_t* a, void* s) { return norm_bwd(d, a, s, false); }
int gdn_gated_norm_bwd(const gdn_norm_desc_t* d, const gdn_norm_bwd_args_t* a, void* s) { return norm_bwd(d, a, s, true); }

size_t gdn_norm_bwd_workspace_size(const gdn_norm_desc_t* d) {
  if (!d || d->rows < 1 || d->width < 1 || d->width > kNormMaxWidth) {
    bad("rows >= 1 and width in 1..16384 required");
    return 0;
  }
  return norm_ws(d);
}

int gdn_conv_step(const gdn_conv_step_desc_t* d, const gdn_conv_step_args_t* a, void* stream) {
  if (!d) return bad("desc is NULL");
  if (d->B < 1 || d->C < 8 || d->C % 8) return bad("B >= 1 and C a positive multiple of 8 required");
  if (d->W < 1 || d->W > kConvMaxTaps) return bad("W must be 1..8");
  if (d->dilation < 1 || d->dilation > (1 << 20)) return bad("dilation must be >= 1");
  if (d->activation != 0 && d->activation != 1) return bad("activation must be 0 or 1");
  const long long xs = d->x_stride ? d->x_stride : d->C;
  if (xs < d->C || xs % 8) return bad("x_stride must be a multiple of 8, at least C");
  if (!a || !a->x || !a->weight || !a->y || (d->W > 1 && !a->state)) return bad("x, weight, state and y must be non-NULL");
  if (d->num_slots < 1 || (!a->state_indices && d->num_slots < d->B)) return bad("num_slots must cover the batch");
  if (!aligned(a->x, 16) || !aligned(a->y, 16) || !aligned(a->state, 16)) return bad("x, y and state must be 16-byte aligned");
  const size_t HW = size_t(d->W - 1) * d->dilation, xb = (size_t(d->B - 1) * xs + d->C) * 2, yb = size_t(d->B) * d->C * 2;
  const size_t sb = size_t(d->num_slots) * HW * d->C * 2;
  if (overlap(a->y, yb, a->x, xb) || overlap(a->state, sb, a->x, xb) || overlap(a->y, yb, a->state, sb))
    return bad("x, y and state must not alias");
  ConvStepParams p{};
  int rc = device_or_error(&p.sms);
  if (rc) return rc;
  p.B = d->B;
  p.C = d->C;
  p.W = d->W;
  p.dil = d->dilation;
  p.HW = int(HW);
  p.slots = d->num_slots;
  p.silu = d->activation;
  p.vec_w = aligned(a->weight, 16);
  p.x_stride = xs;
  p.index = a->state_indices;
  p.x = static_cast<cbf*>(a->x);
  p.w = a->weight;
  p.bias = a->bias;
  p.state = static_cast<bf*>(a->state);
  p.y = static_cast<bf*>(a->y);
  p.status = a->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKConvStep, s);
  return cuda_rc(launch_conv_step(p, s), "convolution step kernel");
}

int gdn_conv_state(const gdn_conv_desc_t* d, const gdn_conv_fwd_args_t* a, void* stream) {
  const size_t ws = gdn_conv_fwd_workspace_size(d);
  if (!ws) return GDN_EINVAL;  // the reason is recorded
  if (!a || !a->x || !a->y) return bad("x and y (the state) must be non-NULL");
  if (!aligned(a->x, 16) || !aligned(a->y, 16) || !aligned(a->halo, 16)) return bad("x, halo and y must be 16-byte aligned");
  if (!a->workspace || a->workspace_bytes < ws || !aligned(a->workspace, 256)) return bad("workspace missing, too small or not 256-byte aligned");
  ConvStateParams p{};
  p.N = d->cu_seqlens ? d->num_seqs : d->B;
  p.T = d->T;
  p.C = d->C;
  const long long HW = (long long)(d->W - 1) * d->dilation;
  if (HW == 0) return GDN_OK;  // one tap needs no past
  if (HW * p.N * ((d->C / 8 + 127) / 128) >= (1ll << 31)) return bad("problem too large");
  p.HW = int(HW);
  const size_t sb = size_t(p.N) * HW * d->C * 2;
  if (overlap(a->y, sb, a->x, size_t(d->B) * d->T * d->C * 2) || overlap(a->y, sb, a->halo, sb)) return bad("the state must not alias x or halo");
  int rc = device_or_error(nullptr);
  if (rc) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->cu_seqlens) {
    int* dcu = static_cast<int*>(a->workspace);
    if ((rc = upload_offsets(d->cu_seqlens, p.N + 1, dcu, s))) return rc;
    p.cu = dcu;
  }
  p.x = static_cast<cbf*>(a->x);
  p.halo = static_cast<cbf*>(a->halo);
  p.state = static_cast<bf*>(a->y);
  TimedScope t(kKConvStep, s);
  return cuda_rc(launch_conv_state(p, s), "convolution state kernel");
}

static int delta_step(const gdn_step_desc_t* d, const gdn_step_args_t* a, void* stream, bool kda) {
  if (!d) return bad("desc is NULL");
  if (d->B < 1 || d->H < 1) return bad("B and H must be positive");
  if (d->num_k_heads < 0 || (d->num_k_heads > 0 && d->H % d->num_k_heads)) return bad("num_k_heads must be 0 or divide H");
  if (std::isnan(d->scale) || std::isinf(d->scale)) return bad("scale must be finite");
  if (d->use_gate_in_kernel) {
    if (!kda) return bad("the in-kernel gate is a KDA option");
    if (!(d->lower_bound >= -5.f && d->lower_bound < 0.f)) return bad("lower_bound must lie in [-5, 0) with use_gate_in_kernel");
  }
  const long long Hk = d->num_k_heads > 0 ? d->num_k_heads : d->H;
  const long long qs = d->q_stride ? d->q_stride : Hk * kD, ks = d->k_stride ? d->k_stride : Hk * kD, vs = d->v_stride ? d->v_stride : (long long)d->H * kD;
  if (qs < Hk * kD || ks < Hk * kD || vs < (long long)d->H * kD || qs % 4 || ks % 4 || vs % 4)
    return bad("q, k and v strides must be multiples of 4 and cover a row");
  if ((long long)d->B * d->H >= (1ll << 28)) return bad("problem too large");
  if (!a || !a->q || !a->k || !a->v || !a->g || !a->beta || !a->state || !a->o) return bad("q, k, v, g, beta, state and o must be non-NULL");
  if (d->use_gate_in_kernel && (!a->A_log || !a->dt_bias)) return bad("A_log and dt_bias are required with use_gate_in_kernel");
  if (d->num_slots < 1 || (!a->state_indices && d->num_slots < d->B)) return bad("num_slots must cover the batch");
  if (!aligned(a->q, 8) || !aligned(a->k, 8) || !aligned(a->v, 8) || !aligned(a->o, 8)) return bad("q, k, v and o must be 8-byte aligned");
  if (!aligned(a->state, 16)) return bad("state must be 16-byte aligned");
  const size_t ob = size_t(d->B) * d->H * kD * 2, sb = size_t(d->num_slots) * d->H * kD * kD * 4;
  const size_t qb = (size_t(d->B - 1) * qs + Hk * kD) * 2, kb = (size_t(d->B - 1) * ks + Hk * kD) * 2, vb = (size_t(d->B - 1) * vs + d->H * kD) * 2;
  const struct { const void* p; size_t n; } in[] = {{a->q, qb}, {a->k, kb}, {a->v, vb}};
  for (const auto& i : in)
    if (overlap(a->o, ob, i.p, i.n) || overlap(a->state, sb, i.p, i.n)) return bad("o and state must not alias q, k or v");
  if (overlap(a->o, ob, a->state, sb)) return bad("o must not alias state");
  int rc = device_or_error(nullptr);
  if (rc) return rc;
  DeltaStepParams p{};
  p.B = d->B;
  p.H = d->H;
  p.group = int(d->H / Hk);
  p.slots = d->num_slots;
  p.kda = kda;
  p.l2norm = d->use_qk_l2norm != 0;
  p.beta_sigmoid = d->use_beta_sigmoid != 0;
  p.gate_act = d->use_gate_in_kernel != 0;
  p.scale = d->scale > 0.f ? d->scale : 1.0f / std::sqrt(float(kD));
  p.lower_bound = d->lower_bound;
  p.q_stride = qs;
  p.k_stride = ks;
  p.v_stride = vs;
  p.index = a->state_indices;
  p.q = static_cast<cbf*>(a->q);
  p.k = static_cast<cbf*>(a->k);
  p.v = static_cast<cbf*>(a->v);
  p.beta = static_cast<cbf*>(a->beta);
  p.g = a->g;
  p.A_log = a->A_log;
  p.dt_bias = a->dt_bias;
  p.state = a->state;
  p.o = static_cast<bf*>(a->o);
  p.status = a->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKDeltaStep, s);
  return cuda_rc(launch_delta_step(p, s), "delta rule step kernel");
}

int gdn_step(const gdn_step_desc_t* d, const gdn_step_args_t* a, void* s) { return delta_step(d, a, s, false); }
int kda_step(const gdn_step_desc_t* d, const gdn_step_args_t* a, void* s) { return delta_step(d, a, s, true); }

size_t gdn_sscan_fwd_workspace_size(const gdn_sscan_desc_t* d) {
  SscanProblem P{};
  if (validate_sscan(d, &P, false)) return 0;
  const SscanPlan q = plan_sscan(P, false);
  return check_sscan_size(P, q) ? 0 : layout_sscan(P, q, false).total;
}

size_t gdn_sscan_saved_size(const gdn_sscan_desc_t* d) {
  SscanProblem P{};
  if (validate_sscan(d, &P, false)) return 0;
  const SscanPlan q = plan_sscan(P, false);
  return check_sscan_size(P, q) ? 0 : saved_bytes(P, q);
}

// With the saved states in the caller's buffer the backward needs its own part only; without, a forward's workspace and
// the states come first.
size_t gdn_sscan_bwd_workspace_size(const gdn_sscan_desc_t* d) {
  SscanProblem P{};
  if (validate_sscan(d, &P, false)) return 0;
  const SscanPlan f = plan_sscan(P, false), q = plan_sscan(P, true);
  if (check_sscan_size(P, f) || check_sscan_size(P, q)) return 0;
  return std::max(layout_sscan(P, f, false).total, layout_sscan(P, q, true).total) + saved_bytes(P, f);
}

int gdn_sscan_fwd(const gdn_sscan_desc_t* d, const gdn_sscan_fwd_args_t* a, void* stream) {
  SscanProblem P{};
  int rc = validate_sscan(d, &P, false);
  if (rc) return rc;
  const SscanPlan q = plan_sscan(P, false);
  if ((rc = check_sscan_size(P, q))) return rc;
  if (!a || !a->u || !a->delta || !a->A || !a->Bm || !a->Cm || !a->y) return bad("u, delta, A, B, C and y must be non-NULL");
  const size_t yb = size_t(P.rows) * P.D * 2;
  auto span = [&](long long stride, long long width) { return (size_t(P.rows - 1) * stride + width) * 2; };
  if (overlap(a->y, yb, a->u, span(P.u_s, P.D)) || overlap(a->y, yb, a->delta, span(P.dt_s, P.D)) || overlap(a->y, yb, a->z, span(P.z_s, P.D)) ||
      overlap(a->y, yb, a->Bm, span(P.b_s, P.G * P.N)) || overlap(a->y, yb, a->Cm, span(P.c_s, P.G * P.N)))
    return bad("y must not alias an input");
  const SscanLayout l = layout_sscan(P, q, false);
  if (!a->workspace || a->workspace_bytes < l.total || !aligned(a->workspace, 256)) return bad("workspace missing, too small or not 256-byte aligned");
  if (a->saved && (a->saved_bytes < saved_bytes(P, q) || !aligned(a->saved, 256))) return bad("saved buffer too small or not 256-byte aligned");
  if ((rc = device_or_error(nullptr))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  SscanParams p{};
  fill(P, q, l, static_cast<char*>(a->workspace), &p);
  p.softplus = d->delta_softplus != 0;
  p.u = static_cast<cbf*>(a->u);
  p.delta = static_cast<cbf*>(a->delta);
  p.z = static_cast<cbf*>(a->z);
  p.Bm = static_cast<cbf*>(a->Bm);
  p.Cm = static_cast<cbf*>(a->Cm);
  p.A = a->A;
  p.Dskip = a->D;
  p.bias = a->delta_bias;
  p.h0 = a->initial_state;
  p.y = static_cast<bf*>(a->y);
  p.final_state = a->final_state;
  p.ck = static_cast<float*>(a->saved);
  if (P.cu && (rc = upload_tables(P, q, const_cast<int*>(p.cu), s))) return rc;
  set_vectors(P, &p);
  TimedScope t(kKSscanFwd, s);
  return cuda_rc(launch_sscan_fwd(p, s), "selective scan kernels");
}

int gdn_sscan_bwd(const gdn_sscan_desc_t* d, const gdn_sscan_bwd_args_t* a, void* stream) {
  SscanProblem P{};
  int rc = validate_sscan(d, &P, false);
  if (rc) return rc;
  const SscanPlan f = plan_sscan(P, false), q = plan_sscan(P, true);
  if ((rc = check_sscan_size(P, f)) || (rc = check_sscan_size(P, q))) return rc;
  if (!a || !a->u || !a->delta || !a->A || !a->Bm || !a->Cm || !a->dy) return bad("u, delta, A, B, C and dy must be non-NULL");
  if (!a->du || !a->ddelta || !a->dA || !a->dB || !a->dC) return bad("du, ddelta, dA, dB and dC must be non-NULL");
  if ((a->z != nullptr) != (a->dz != nullptr)) return bad("dz goes with z");
  if ((a->dD && !a->D) || (a->ddelta_bias && !a->delta_bias) || (a->dh0 && !a->initial_state)) return bad("a gradient's input is missing");
  const size_t yb = size_t(P.rows) * P.D * 2;
  auto span = [&](long long stride, long long width) { return (size_t(P.rows - 1) * stride + width) * 2; };
  const void* outs[] = {a->du, a->ddelta, a->dz};
  for (const void* o : outs)
    if (overlap(o, yb, a->u, span(P.u_s, P.D)) || overlap(o, yb, a->delta, span(P.dt_s, P.D)) || overlap(o, yb, a->z, span(P.z_s, P.D)) ||
        overlap(o, yb, a->dy, yb))
      return bad("du, ddelta and dz must not alias an input");
  if (overlap(a->du, yb, a->ddelta, yb) || overlap(a->du, yb, a->dz, yb) || overlap(a->ddelta, yb, a->dz, yb)) return bad("the outputs must not alias each other");
  const SscanLayout lf = layout_sscan(P, f, false), l = layout_sscan(P, q, true);
  const size_t sv = saved_bytes(P, f), own = std::max(lf.total, l.total);
  if (!a->workspace || a->workspace_bytes < own + (a->saved ? 0 : sv) || !aligned(a->workspace, 256))
    return bad("workspace missing, too small or not 256-byte aligned");
  if (a->saved && (a->saved_bytes < sv || !aligned(a->saved, 256))) return bad("saved buffer too small or not 256-byte aligned");
  if ((rc = device_or_error(nullptr))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(a->workspace);
  SscanParams p{};
  p.softplus = d->delta_softplus != 0;
  p.u = static_cast<cbf*>(a->u);
  p.delta = static_cast<cbf*>(a->delta);
  p.z = static_cast<cbf*>(a->z);
  p.Bm = static_cast<cbf*>(a->Bm);
  p.Cm = static_cast<cbf*>(a->Cm);
  p.A = a->A;
  p.Dskip = a->D;
  p.bias = a->delta_bias;
  p.h0 = a->initial_state;
  p.ck = a->saved ? static_cast<float*>(const_cast<void*>(a->saved)) : reinterpret_cast<float*>(ws + own);
  if (!a->saved) {  // the forward's states again, without its output
    fill(P, f, lf, ws, &p);
    if (P.cu && (rc = upload_tables(P, f, const_cast<int*>(p.cu), s))) return rc;
    set_vectors(P, &p);
    TimedScope t(kKSscanFwd, s);
    if ((rc = cuda_rc(launch_sscan_fwd(p, s), "selective scan kernels"))) return rc;
  }
  fill(P, q, l, ws, &p);
  p.dy = static_cast<cbf*>(a->dy);
  p.dfinal = a->dfinal;
  p.du = static_cast<bf*>(a->du);
  p.ddelta = static_cast<bf*>(a->ddelta);
  p.dz = static_cast<bf*>(a->dz);
  p.dB = static_cast<bf*>(a->dB);
  p.dC = static_cast<bf*>(a->dC);
  p.dA = a->dA;
  p.dD = a->dD;
  p.dbias = a->ddelta_bias;
  p.dh0 = a->dh0;
  p.part_bc = reinterpret_cast<float*>(ws + l.part_bc);
  p.part_par = reinterpret_cast<float*>(ws + l.part_par);
  if (P.cu && (rc = upload_tables(P, q, const_cast<int*>(p.cu), s))) return rc;
  set_vectors(P, &p);
  TimedScope t(kKSscanBwd, s);
  return cuda_rc(launch_sscan_bwd(p, s), "selective scan backward kernels");
}

int gdn_sscan_step(const gdn_sscan_desc_t* d, const gdn_sscan_step_args_t* a, void* stream) {
  SscanProblem P{};
  int rc = validate_sscan(d, &P, true);
  if (rc) return rc;
  if (!a || !a->u || !a->delta || !a->A || !a->Bm || !a->Cm || !a->state || !a->y) return bad("u, delta, A, B, C, state and y must be non-NULL");
  if (a->num_slots < 1 || (!a->state_indices && a->num_slots < P.B)) return bad("num_slots must cover the batch");
  if ((long long)P.B * ((P.D * 4ll + 255) / 256) >= (1ll << 31)) return bad("problem too large");
  auto span = [&](long long stride, long long width) { return (size_t(P.B - 1) * stride + width) * 2; };
  const size_t yb = size_t(P.B) * P.D * 2, sb = size_t(a->num_slots) * P.D * P.N * 4;
  const struct { const void* p; size_t n; } in[] = {{a->u, span(P.u_s, P.D)}, {a->delta, span(P.dt_s, P.D)}, {a->z, span(P.z_s, P.D)},
                                                    {a->Bm, span(P.b_s, P.G * P.N)}, {a->Cm, span(P.c_s, P.G * P.N)}};
  for (const auto& i : in)
    if (overlap(a->y, yb, i.p, i.n) || overlap(a->state, sb, i.p, i.n)) return bad("y and state must not alias an input");
  if (overlap(a->y, yb, a->state, sb)) return bad("y must not alias state");
  SscanStepParams p{};
  if ((rc = device_or_error(&p.sms))) return rc;
  p.vec = P.N % 4 == 0 && aligned(a->state, 16) && aligned(a->Bm, 8) && aligned(a->Cm, 8) && P.b_s % 4 == 0 && P.c_s % 4 == 0;
  p.B = P.B;
  p.D = P.D;
  p.N = P.N;
  p.G = P.G;
  p.Dg = P.D / P.G;
  p.slots = a->num_slots;
  p.softplus = d->delta_softplus != 0;
  p.u_s = P.u_s;
  p.dt_s = P.dt_s;
  p.z_s = P.z_s;
  p.b_s = P.b_s;
  p.c_s = P.c_s;
  p.index = a->state_indices;
  p.u = static_cast<cbf*>(a->u);
  p.delta = static_cast<cbf*>(a->delta);
  p.z = static_cast<cbf*>(a->z);
  p.Bm = static_cast<cbf*>(a->Bm);
  p.Cm = static_cast<cbf*>(a->Cm);
  p.A = a->A;
  p.Dskip = a->D;
  p.bias = a->delta_bias;
  p.state = a->state;
  p.y = static_cast<bf*>(a->y);
  p.status = a->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimedScope t(kKSscanStep, s);
  return cuda_rc(launch_sscan_step(p, s), "selective scan step kernel");
}

}  // extern "C"
