// C ABI of the operators around a recurrent layer's projections (declared in
// include/gdn.h): the short convolution, the selective state space scan and
// step, and the residual norm.  Host side only: every argument is validated
// before any HIP call, then the kernels are enqueued on the caller's stream.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

#include "gdn.h"
#include "gdn_api_check.h"
#include "gdn_api_common.h"
#include "gdn_layer.h"

using namespace gdn;

namespace {

constexpr int64_t kMaxThreads = (int64_t)1 << 32;  // of one launch
constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool head_dim(int64_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// A token stride the scan's 32-bit offsets inside a block can use; a single
// token's stride is never taken, and replaced by the row's own length.
constexpr int64_t kMaxTokenStride = (int64_t)1 << 24;

int token_stride(const char* name, int64_t row, Tokens* v) {
  if (v->T <= 1) v->st = row;
  if (v->st > kMaxTokenStride)
    return api_fail(GDN_ERR_LAYOUT, "%s: token stride must be at most 2^24 elements", name);
  return GDN_OK;
}

// The scan's sizes, layout and segments.
struct Ssm {
  bool bf16 = true;
  int64_t T = 0, H = 0, G = 0, N = 0, P = 0;
  Tokens x, dt, b, c, o;
  int64_t x_sh = 0, dt_sh = 0, b_sh = 0, c_sh = 0, o_sh = 0;
  Sequences seq;
  gdn_ssm_options opts;
  int64_t seg_len = 0, segs_per_seq = 1, max_segs = 1;
  bool cut = false;  // some sequence may have two or more segments
  int64_t max_cuts = 0, max_cut_segs = 0;  // such sequences, their segments
  size_t table = 0, seg_off = 0, cuts = 0, cut_table = 0, slots = 0, decay = 0, total = 0;
};

int ssm_options(const gdn_ssm_options* opts, gdn_ssm_options* o) {
  gdn_ssm_default_options(o);
  if (opts) *o = *opts;
  if (o->flags & ~GDN_SSM_SOFTPLUS) return api_fail(GDN_ERR_SHAPE, "unknown flag bits 0x%x", o->flags);
  if (o->segment_blocks < -1) return api_fail(GDN_ERR_SHAPE, "segment_blocks must be >= -1 (got %d)", o->segment_blocks);
  if ((uintptr_t)o->a_log % 4 || (uintptr_t)o->dt_bias % 4 || (uintptr_t)o->d_skip % 4)
    return api_fail(GDN_ERR_LAYOUT, "a_log, dt_bias and d_skip must be 4-byte aligned");
  return GDN_OK;
}

// The automatic choice makes no longer segments than this.
constexpr int64_t kMaxSegment = (int64_t)1 << 20;
int64_t ssm_groups_per_segment(const Ssm& P) {
  return P.H / gdn::ssm_group_heads(P.bf16, (int)P.P, (int)(P.H / P.G));
}

// Blocks per segment that spread the work over `groups` workgroups: of
// uniform sequences, as many equal segments as make at most that many
// workgroups; of packed ones, whose lengths the host does not know, an equal
// share of all blocks, less what the sequences' last segments, half full on
// average, take (at most half the groups, since sequences that fill the chip
// by themselves are best left whole).  Measured, 16 heads of 128 x 64 in two
// groups, so and in equal shares: 8 prompts of 200 to 16384 tokens 232 and 219
// us, 16 of 200 to 4096 138 and 138, 32 257 and 250, 64 325 and 427, 128 583
// and 582.  (The table's order came after this rule, and below 64 prompts has
// taken what the rule gained.)
int64_t ssm_spread(const Ssm& P, int64_t groups) {
  const int64_t block = gdn::kSsmBlock;
  const int64_t each = ssm_groups_per_segment(P);
  if (P.seq.packed) {
    const int64_t room = std::max(groups / 2, groups - P.seq.n * each / 2);
    return (((P.T + block - 1) / block) * each + room - 1) / room;
  }
  const int64_t all = (P.seq.len + block - 1) / block;
  const int64_t segs = std::max<int64_t>(1, groups / (each * P.seq.n));
  return (all + segs - 1) / segs;
}

// Tokens per segment.  The automatic choice spreads the tokens x heads over
// the two workgroups a compute unit holds, so that a few long sequences do
// not leave the chip idle; problems too small for segments of four blocks
// that way, over one workgroup a compute unit, in segments of two to four
// blocks.  Measured: 4096 tokens x 16 heads (128 x 128 states) take 44 us in
// segments of 4 blocks (the choice), 50 us in 2, 51 in 3, 47 in 5, 52 in 6, 70
// in 1; 16384 x 48 heads 291 us in 26 (the choice), 302 in 13, 386 in 43; five
// prompts of up to 1000 tokens x 8 heads of f32 34 us in 2 (the choice), 43 in
// 3, 51 in 4, 28 in 1.
int64_t ssm_segment_tokens(const Ssm& P) {
  const int64_t block = gdn::kSsmBlock;
  if (P.opts.segment_blocks != 0) {
    // as given, up to the whole of the longest sequence that there can be
    const int64_t longest = P.seq.packed ? P.T : P.seq.len;
    const int64_t all = std::max<int64_t>(1, (longest + block - 1) / block);
    return (P.opts.segment_blocks < 0 ? all : std::min<int64_t>(P.opts.segment_blocks, all)) * block;
  }
  const int64_t full = gdn::ssm_target_groups();
  int64_t blocks = ssm_spread(P, full);
  if (blocks < 4) blocks = std::min<int64_t>(4, std::max<int64_t>(2, ssm_spread(P, full / 2)));
  return std::min(blocks * block, kMaxSegment);
}

int ssm_sizes(const gdn_tensor* x, const gdn_tensor* b, const gdn_tensor* cu, const gdn_ssm_options* opts, Ssm* P) {
  int rc;
  if (!is_float(x->dtype)) return api_fail(GDN_ERR_DTYPE, "x must be bf16 or f32");
  if (b->dtype != x->dtype) return api_fail(GDN_ERR_DTYPE, "x, b, c and out must share one dtype");
  P->bf16 = x->dtype == GDN_DTYPE_BF16;
  if ((rc = ssm_options(opts, &P->opts))) return rc;
  if (x->ndim != 3 && x->ndim != 4) return api_fail(GDN_ERR_SHAPE, "x must be [T, H, P] or [B, L, H, P]");
  if (b->ndim != x->ndim) return api_fail(GDN_ERR_SHAPE, "x and b must have the same rank");
  for (int i = 0; i < x->ndim; ++i)
    if (x->shape[i] < 0 || b->shape[i] < 0 || x->shape[i] >= kMax32 || b->shape[i] >= kMax32)
      return api_fail(GDN_ERR_SHAPE, "size out of range");
  if ((rc = parse_tokens(x, "x", 2, &P->x)) || (rc = parse_tokens(b, "b", 2, &P->b))) return rc;
  const int r = x->ndim;
  P->T = P->x.T;
  P->H = x->shape[r - 2];
  P->P = x->shape[r - 1];
  P->G = b->shape[r - 2];
  P->N = b->shape[r - 1];
  if (P->b.T != P->T || P->b.B != P->x.B) return api_fail(GDN_ERR_SHAPE, "b token count differs from x");
  if (!head_dim(P->N) || !head_dim(P->P))
    return api_fail(GDN_ERR_UNSUPPORTED, "N and P must be 16, 32, 64 or 128 (got %lld, %lld)", (long long)P->N,
                    (long long)P->P);
  if (P->H < 1 || P->G < 1 || P->H % P->G)
    return api_fail(GDN_ERR_SHAPE, "heads (%lld) must be a positive multiple of groups (%lld)", (long long)P->H,
                    (long long)P->G);
  if (P->H > 65535) return api_fail(GDN_ERR_UNSUPPORTED, "at most 65535 heads");
  if ((rc = parse_sequences(cu, P->x.B, P->T, &P->seq))) return rc;

  P->seg_len = ssm_segment_tokens(*P);
  if (P->seq.packed) {
    P->cut = P->T > P->seg_len;
    P->max_segs = P->T / P->seg_len + P->seq.n;
    P->segs_per_seq = 0;
    // a cut sequence has at least seg_len + 1 tokens, and of its segments all
    // but one are full
    P->max_cuts = std::min<int64_t>(P->seq.n, P->T / (P->seg_len + 1));
    P->max_cut_segs = P->T / P->seg_len + P->max_cuts;
  } else {
    P->segs_per_seq = std::max<int64_t>(1, (P->seq.len + P->seg_len - 1) / P->seg_len);
    P->cut = P->segs_per_seq > 1;
    P->max_segs = P->segs_per_seq * P->seq.n;
    P->max_cuts = P->seq.n;
    P->max_cut_segs = P->max_segs;
  }
  // a launch has fewer than 2^32 threads (the scan's: 4 P per segment and
  // head, its segments rounded up by up to 7)
  if ((P->max_segs + 7) * P->H * 4 * P->P >= kMaxThreads || (P->cut && P->seq.n * P->H * 256 >= kMaxThreads))
    return api_fail(GDN_ERR_SHAPE, "too many (segment, head) pairs");
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  if (P->seq.packed) {
    P->table = take((size_t)P->max_segs * 16);
    P->seg_off = take((size_t)(P->seq.n + 1) * 4);
  }
  if (P->cut) {
    if (P->seq.packed) {
      P->cuts = take((size_t)(P->max_cuts + 1) * 16);
      P->cut_table = take((size_t)P->max_cut_segs * 16);
    }
    const size_t slots = (size_t)(P->max_cut_segs + P->max_cuts);
    P->decay = take(slots * P->H * 4);
    P->slots = take(slots * P->H * P->N * P->P * 4);
  }
  P->total = off;
  return GDN_OK;
}

int check_state(const gdn_tensor* s, const char* name, int64_t n, const Ssm& P) {
  if (s->dtype != GDN_DTYPE_F32) return api_fail(GDN_ERR_DTYPE, "%s must be f32", name);
  if (s->ndim != 4 || s->shape[0] != n || s->shape[1] != P.H || s->shape[2] != P.N || s->shape[3] != P.P)
    return api_fail(GDN_ERR_SHAPE, "%s must be [%lld, H=%lld, N=%lld, P=%lld]", name, (long long)n, (long long)P.H,
                    (long long)P.N, (long long)P.P);
  if (is_empty(s)) return GDN_OK;
  if (!contiguous(s)) return api_fail(GDN_ERR_LAYOUT, "%s must be contiguous", name);
  if (!s->data) return api_fail(GDN_ERR_NULL_ARG, "%s data is NULL", name);
  if (!aligned16(s->data)) return api_fail(GDN_ERR_LAYOUT, "%s must be 16-byte aligned", name);
  return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_short_conv(const gdn_tensor* x, const gdn_tensor* weight, const float* bias,
                   const gdn_tensor* cu_seqlens, const gdn_tensor* state_in, gdn_tensor* state_out,
                   gdn_tensor* out, uint32_t flags, void* stream) {
  if (!x || !weight || !out) return api_fail(GDN_ERR_NULL_ARG, "x, weight and out are required");
  if (!is_float(x->dtype)) return api_fail(GDN_ERR_DTYPE, "x must be bf16 or f32");
  if (out->dtype != x->dtype) return api_fail(GDN_ERR_DTYPE, "x and out must share one dtype");
  if (weight->dtype != GDN_DTYPE_F32) return api_fail(GDN_ERR_DTYPE, "weight must be f32");
  if (flags & ~GDN_CONV_SILU) return api_fail(GDN_ERR_SHAPE, "unknown flag bits 0x%x", flags);
  int rc;
  if ((rc = check_tensor(x, "x", 2, 3)) || (rc = check_tensor(out, "out", 2, 3)) ||
      (rc = check_tensor(weight, "weight", 2, 2)))
    return rc;
  if (out->ndim != x->ndim) return api_fail(GDN_ERR_SHAPE, "out must match x");
  for (int i = 0; i < x->ndim; ++i)
    if (out->shape[i] != x->shape[i]) return api_fail(GDN_ERR_SHAPE, "out must match x");
  Tokens tx, to;
  if ((rc = parse_tokens(x, "x", 1, &tx)) || (rc = parse_tokens(out, "out", 1, &to))) return rc;
  const int64_t D = x->shape[x->ndim - 1], W = weight->shape[1];
  if (weight->shape[0] != D) return api_fail(GDN_ERR_SHAPE, "weight must be [D, W]");
  if (W < 1 || W > 4) return api_fail(GDN_ERR_SHAPE, "W must be 1 .. 4 (got %lld)", (long long)W);
  if (D < 1 || D > kMaxCount) return api_fail(GDN_ERR_SHAPE, "D must be 1 .. 2^31 - 2^21");
  if (!contiguous(weight)) return api_fail(GDN_ERR_LAYOUT, "weight must be contiguous");
  if ((uintptr_t)bias % 4) return api_fail(GDN_ERR_LAYOUT, "bias must be 4-byte aligned");
  Sequences seq;
  if ((rc = parse_sequences(cu_seqlens, tx.B, tx.T, &seq))) return rc;
  const gdn_tensor* states[2] = {state_in, state_out};
  const char* names[2] = {"state_in", "state_out"};
  for (int i = 0; i < 2; ++i) {
    const gdn_tensor* t = states[i];
    if (!t) continue;
    if (t->dtype != x->dtype) return api_fail(GDN_ERR_DTYPE, "%s must have x's dtype", names[i]);
    if ((rc = check_tensor(t, names[i], 3, 3))) return rc;
    if (t->shape[0] != seq.n || t->shape[1] != W - 1 || t->shape[2] != D)
      return api_fail(GDN_ERR_SHAPE, "%s must be [N=%d, W - 1=%lld, D=%lld]", names[i], seq.n, (long long)(W - 1),
                      (long long)D);
    if (!is_empty(t) && !contiguous(t)) return api_fail(GDN_ERR_LAYOUT, "%s must be contiguous", names[i]);
  }
  if ((rc = check_rows("out", tx.T, to.st, 1, 0, D))) return rc;
  const Range outs[2] = {range_of(out, "out"), range_of(state_out, "state_out")};
  const Range ins[5] = {range_of(x, "x"), range_of(weight, "weight"), range_of(bias, 4 * D, "bias"),
                        range_of(cu_seqlens, "cu_seqlens"),
                        same_view(state_in, state_out) ? Range{} : range_of(state_in, "state_in")};
  if ((rc = check_overlaps(outs, 2, ins, 5))) return rc;
  if (same_view(state_in, state_out) && overlap(outs[0], range_of(state_in, "state_in")))
    return api_fail(GDN_ERR_LAYOUT, "out overlaps state_in");
  const hipStream_t s = (hipStream_t)stream;
  gdn::api_clear_error();
  if (seq.packed && (rc = gdn::api_debug_check_cu(cu_seqlens, seq.n, tx.T, s))) return rc;
  const int64_t epg = x->dtype == GDN_DTYPE_BF16 ? 8 : 4;
  const bool vec = D % epg == 0 && tx.st % epg == 0 && to.st % epg == 0 && aligned16(x->data) &&
                   aligned16(out->data) && (!state_in || aligned16(state_in->data)) &&
                   (!state_out || aligned16(state_out->data));
  gdn::ShortConvParams p{};
  p.x = x->data;
  p.out = out->data;
  p.w = (const float*)weight->data;
  p.bias = bias;
  // one tap keeps no history (and an empty array carries no data)
  p.state_in = state_in && W > 1 ? state_in->data : nullptr;
  p.state_out = state_out && W > 1 ? state_out->data : nullptr;
  p.cu = cu_seqlens ? cu_seqlens->data : nullptr;
  p.cu_i64 = cu_seqlens && cu_seqlens->dtype == GDN_DTYPE_I64;
  p.x_st = tx.st;
  p.o_st = to.st;
  p.n_seq = seq.n;
  p.seq_len = seq.len;
  p.t_total = (int32_t)tx.T;
  p.d = (int32_t)D;
  p.width = (int32_t)W;
  p.silu = (flags & GDN_CONV_SILU) ? 1 : 0;
  const hipError_t e = gdn::launch_short_conv(x->dtype == GDN_DTYPE_BF16, vec, p, s);
  if (e != hipSuccess) return api_fail(GDN_ERR_HIP, "short convolution launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

void gdn_ssm_default_options(gdn_ssm_options* opts) {
  if (!opts) return;
  opts->a_log = nullptr;
  opts->dt_bias = nullptr;
  opts->d_skip = nullptr;
  opts->flags = GDN_SSM_SOFTPLUS;
  opts->segment_blocks = 0;
}

int gdn_ssm_workspace_size(const gdn_tensor* x, const gdn_tensor* b, const gdn_tensor* cu_seqlens,
                           const gdn_ssm_options* opts, size_t* bytes) {
  if (!x || !b || !bytes) return api_fail(GDN_ERR_NULL_ARG, "x, b and bytes are required");
  Ssm P;
  const int rc = ssm_sizes(x, b, cu_seqlens, opts, &P);
  if (rc) return rc;
  *bytes = P.total;
  return GDN_OK;
}

int gdn_ssm_prefill(const gdn_tensor* x, const gdn_tensor* dt, const gdn_tensor* b, const gdn_tensor* c,
                    const gdn_tensor* cu_seqlens, const gdn_tensor* init_state, gdn_tensor* out,
                    gdn_tensor* final_state, const gdn_ssm_options* opts, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!x || !dt || !b || !c || !out) return api_fail(GDN_ERR_NULL_ARG, "x, dt, b, c and out are required");
  Ssm P;
  int rc;
  if ((rc = ssm_sizes(x, b, cu_seqlens, opts, &P))) return rc;
  if (c->dtype != x->dtype || out->dtype != x->dtype)
    return api_fail(GDN_ERR_DTYPE, "x, b, c and out must share one dtype");
  if (dt->dtype != GDN_DTYPE_F32) return api_fail(GDN_ERR_DTYPE, "dt must be f32");
  const int r = x->ndim;
  if ((rc = check_tensor(x, "x", 3, 4)) || (rc = check_tensor(b, "b", 3, 4)) || (rc = check_tensor(c, "c", 3, 4)) ||
      (rc = check_tensor(out, "out", 3, 4)) || (rc = check_tensor(dt, "dt", 2, 3, false)))
    return rc;
  if (c->ndim != r || out->ndim != r || dt->ndim != r - 1)
    return api_fail(GDN_ERR_SHAPE, "x, b, c and out must have one rank, dt one less");
  for (int i = 0; i < r; ++i) {
    if (c->shape[i] != b->shape[i]) return api_fail(GDN_ERR_SHAPE, "b and c shapes differ");
    if (out->shape[i] != x->shape[i]) return api_fail(GDN_ERR_SHAPE, "out must match x");
    if (i + 1 < r && dt->shape[i] != x->shape[i]) return api_fail(GDN_ERR_SHAPE, "dt must be [T, H]");
  }
  if ((rc = parse_tokens(c, "c", 2, &P.c)) || (rc = parse_tokens(out, "out", 2, &P.o)) ||
      (rc = parse_tokens(dt, "dt", 1, &P.dt)))
    return rc;
  const int64_t epg = P.bf16 ? 8 : 4;
  if ((rc = token_stride("x", P.P, &P.x)) || (rc = token_stride("b", P.N, &P.b)) ||
      (rc = token_stride("c", P.N, &P.c)) || (rc = token_stride("out", P.P, &P.o)) ||
      (rc = token_stride("dt", 1, &P.dt)))
    return rc;
  const struct { const gdn_tensor* t; const Tokens* v; const char* n; } vecs[] = {
      {x, &P.x, "x"}, {b, &P.b, "b"}, {c, &P.c, "c"}, {out, &P.o, "out"}};
  if (P.T > 0)
    for (const auto& v : vecs) {
      if (!aligned16(v.t->data)) return api_fail(GDN_ERR_LAYOUT, "%s must be 16-byte aligned", v.n);
      // (of a single head the stride is never taken either)
      if (v.v->st % epg || (v.t->shape[r - 2] > 1 && v.t->stride[r - 2] % epg))
        return api_fail(GDN_ERR_LAYOUT, "%s: token/head strides must be multiples of %lld elements", v.n,
                        (long long)epg);
    }
  if ((rc = check_rows("out", P.T, P.o.st, P.H, out->stride[r - 2], P.P))) return rc;
  if (init_state && (rc = check_state(init_state, "init_state", P.seq.n, P))) return rc;
  if (final_state && (rc = check_state(final_state, "final_state", P.seq.n, P))) return rc;
  if (P.total > 0 && (!workspace || workspace_bytes < P.total))
    return api_fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", P.total, workspace_bytes);
  if ((uintptr_t)workspace % kAlign) return api_fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const Range outs[3] = {range_of(out, "out"), range_of(final_state, "final_state"),
                         range_of(workspace, (int64_t)P.total, "workspace")};
  const bool in_place = same_view(init_state, final_state);
  const Range init = range_of(init_state, "init_state");
  const Range ins[9] = {range_of(x, "x"), range_of(dt, "dt"), range_of(b, "b"), range_of(c, "c"),
                        range_of(cu_seqlens, "cu_seqlens"), range_of(P.opts.a_log, 4 * P.H, "a_log"),
                        range_of(P.opts.dt_bias, 4 * P.H, "dt_bias"), range_of(P.opts.d_skip, 4 * P.H, "d_skip"),
                        in_place ? Range{} : init};
  if ((rc = check_overlaps(outs, 3, ins, 9))) return rc;

  const hipStream_t s = (hipStream_t)stream;
  gdn::api_clear_error();
  if (P.seq.packed && (rc = gdn::api_debug_check_cu(cu_seqlens, P.seq.n, P.T, s))) return rc;
  char* base = (char*)workspace;
  hipError_t e;
  gdn::SsmParams p{};
  p.x = x->data;
  p.dt = (const float*)dt->data;
  p.b = b->data;
  p.c = c->data;
  p.out = out->data;
  p.init = init_state ? (const float*)init_state->data : nullptr;
  p.final_state = final_state ? (float*)final_state->data : nullptr;
  p.a_log = P.opts.a_log;
  p.dt_bias = P.opts.dt_bias;
  p.d_skip = P.opts.d_skip;
  p.x_st = P.x.st; p.x_sh = x->stride[r - 2];
  p.dt_st = P.dt.st; p.dt_sh = dt->stride[r - 2];
  p.b_st = P.b.st; p.b_sh = b->stride[r - 2];
  p.c_st = P.c.st; p.c_sh = c->stride[r - 2];
  p.o_st = P.o.st; p.o_sh = out->stride[r - 2];
  p.heads = (int32_t)P.H;
  p.group = (int32_t)(P.H / P.G);
  p.softplus = (P.opts.flags & GDN_SSM_SOFTPLUS) ? 1 : 0;
  p.packed = P.seq.packed ? 1 : 0;
  p.n_seq = P.seq.n;
  p.seq_len = P.seq.len;
  p.seg_len = (int32_t)P.seg_len;
  p.segs_per_seq = (int32_t)P.segs_per_seq;
  p.max_segs = (int32_t)P.max_segs;
  p.max_cuts = (int32_t)P.max_cuts;
  p.max_cut_segs = (int32_t)P.max_cut_segs;
  if (P.seq.packed) {
    p.table = (const int32_t*)(base + P.table);
    p.seg_off = (const int32_t*)(base + P.seg_off);
    gdn::SsmTable tp{};
    tp.cu = cu_seqlens->data;
    tp.cu_i64 = cu_seqlens->dtype == GDN_DTYPE_I64 ? 1 : 0;
    tp.seg_off = (int32_t*)(base + P.seg_off);
    tp.table = (int32_t*)(base + P.table);
    tp.n_seq = P.seq.n;
    tp.t_total = (int32_t)P.T;
    tp.seg_len = (int32_t)P.seg_len;
    tp.max_segs = (int32_t)P.max_segs;
    if (P.cut) {
      tp.cuts = (int32_t*)(base + P.cuts);
      tp.cut_table = (int32_t*)(base + P.cut_table);
      tp.max_cuts = (int32_t)P.max_cuts;
      tp.max_cut_segs = (int32_t)P.max_cut_segs;
    }
    tp.round = (int32_t)(gdn::ssm_target_groups() / 2 / ssm_groups_per_segment(P));
    if ((e = gdn::launch_ssm_table(tp, s)) != hipSuccess)
      return api_fail(GDN_ERR_HIP, "segment table launch: %s", hipGetErrorString(e));
  }
  if (P.cut) {
    p.slots = (float*)(base + P.slots);
    p.seg_decay = (float*)(base + P.decay);
    p.cuts = (const int32_t*)(base + P.cuts);
    p.cut_table = (const int32_t*)(base + P.cut_table);
    if ((e = gdn::launch_ssm_states(P.bf16, (int)P.N, (int)P.P, p, s)) != hipSuccess)
      return api_fail(GDN_ERR_HIP, "segment states launch: %s", hipGetErrorString(e));
  }
  if ((e = gdn::launch_ssm_scan(P.bf16, (int)P.N, (int)P.P, p, s)) != hipSuccess)
    return api_fail(GDN_ERR_HIP, "scan launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

int gdn_ssm_decode(const gdn_tensor* x, const gdn_tensor* dt, const gdn_tensor* b, const gdn_tensor* c,
                   gdn_tensor* state, gdn_tensor* out, const gdn_ssm_options* opts, void* stream) {
  if (!x || !dt || !b || !c || !state || !out)
    return api_fail(GDN_ERR_NULL_ARG, "x, dt, b, c, state and out are required");
  if (!is_float(x->dtype)) return api_fail(GDN_ERR_DTYPE, "x must be bf16 or f32");
  if (b->dtype != x->dtype || c->dtype != x->dtype || out->dtype != x->dtype)
    return api_fail(GDN_ERR_DTYPE, "x, b, c and out must share one dtype");
  if (dt->dtype != GDN_DTYPE_F32) return api_fail(GDN_ERR_DTYPE, "dt must be f32");
  Ssm P;
  int rc;
  if ((rc = ssm_options(opts, &P.opts))) return rc;
  if ((rc = check_tensor(x, "x", 3, 3)) || (rc = check_tensor(b, "b", 3, 3)) || (rc = check_tensor(c, "c", 3, 3)) ||
      (rc = check_tensor(out, "out", 3, 3)) || (rc = check_tensor(dt, "dt", 2, 2, false)))
    return rc;
  const int64_t n = x->shape[0];
  P.H = x->shape[1];
  P.P = x->shape[2];
  P.G = b->shape[1];
  P.N = b->shape[2];
  for (int i = 0; i < 3; ++i) {
    if (c->shape[i] != b->shape[i]) return api_fail(GDN_ERR_SHAPE, "b and c shapes differ");
    if (out->shape[i] != x->shape[i]) return api_fail(GDN_ERR_SHAPE, "out must match x");
  }
  if (b->shape[0] != n) return api_fail(GDN_ERR_SHAPE, "b sequence count differs from x");
  if (dt->shape[0] != n || dt->shape[1] != P.H) return api_fail(GDN_ERR_SHAPE, "dt must be [N, H]");
  if (!head_dim(P.N) || !head_dim(P.P)) return api_fail(GDN_ERR_UNSUPPORTED, "N and P must be 16, 32, 64 or 128");
  if (P.H < 1 || P.G < 1 || P.H % P.G) return api_fail(GDN_ERR_SHAPE, "heads must be a positive multiple of groups");
  if (P.H > 65535) return api_fail(GDN_ERR_UNSUPPORTED, "at most 65535 heads");
  if (n > kMaxCount) return api_fail(GDN_ERR_SHAPE, "too many sequences");
  if ((rc = check_state(state, "state", n, P))) return rc;
  gdn::api_clear_error();
  if (n == 0) return GDN_OK;
  const int64_t es = element_size(x->dtype);
  const struct { const gdn_tensor* t; const char* name; } rows[] = {{x, "x"}, {out, "out"}};
  for (const auto& v : rows)
    if ((uintptr_t)v.t->data % (uintptr_t)(4 * es) || (n > 1 && v.t->stride[0] % 4) ||
        (P.H > 1 && v.t->stride[1] % 4))  // (of a single row or head the stride is never taken)
      return api_fail(GDN_ERR_LAYOUT, "%s rows must start on 4-element boundaries", v.name);
  if ((rc = check_rows("out", n, out->stride[0], P.H, out->stride[1], P.P))) return rc;
  const Range outs[2] = {range_of(out, "out"), range_of(state, "state")};
  const Range ins[7] = {range_of(x, "x"), range_of(dt, "dt"), range_of(b, "b"), range_of(c, "c"),
                        range_of(P.opts.a_log, 4 * P.H, "a_log"), range_of(P.opts.dt_bias, 4 * P.H, "dt_bias"),
                        range_of(P.opts.d_skip, 4 * P.H, "d_skip")};
  if ((rc = check_overlaps(outs, 2, ins, 7))) return rc;
  gdn::SsmStepParams p{};
  p.x = x->data;
  p.dt = (const float*)dt->data;
  p.b = b->data;
  p.c = c->data;
  p.state = (float*)state->data;
  p.out = out->data;
  p.a_log = P.opts.a_log;
  p.dt_bias = P.opts.dt_bias;
  p.d_skip = P.opts.d_skip;
  p.x_st = x->stride[0]; p.x_sh = x->stride[1];
  p.dt_st = dt->stride[0]; p.dt_sh = dt->stride[1];
  p.b_st = b->stride[0]; p.b_sh = b->stride[1];
  p.c_st = c->stride[0]; p.c_sh = c->stride[1];
  p.o_st = out->stride[0]; p.o_sh = out->stride[1];
  p.n = (int32_t)n;
  p.heads = (int32_t)P.H;
  p.group = (int32_t)(P.H / P.G);
  p.softplus = (P.opts.flags & GDN_SSM_SOFTPLUS) ? 1 : 0;
  const hipError_t e = gdn::launch_ssm_step(x->dtype == GDN_DTYPE_BF16, (int)P.N, (int)P.P, p, (hipStream_t)stream);
  if (e != hipSuccess) return api_fail(GDN_ERR_HIP, "step launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

int gdn_add_rms_norm(const gdn_tensor* x, const gdn_tensor* residual, const float* weight, float eps,
                     gdn_tensor* residual_out, gdn_tensor* out, gdn_tensor* out_q, gdn_tensor* scales,
                     void* stream) {
  if (!x) return api_fail(GDN_ERR_NULL_ARG, "x is required");
  if (!residual_out && !out && !out_q) return api_fail(GDN_ERR_NULL_ARG, "at least one output is required");
  if (!out_q != !scales) return api_fail(GDN_ERR_NULL_ARG, "out_q and scales go together");
  if (!is_float(x->dtype)) return api_fail(GDN_ERR_DTYPE, "x must be bf16 or f32");
  if ((residual && residual->dtype != x->dtype) || (residual_out && residual_out->dtype != x->dtype) ||
      (out && out->dtype != x->dtype))
    return api_fail(GDN_ERR_DTYPE, "x, residual, residual_out and out must share one dtype");
  if (out_q && out_q->dtype != GDN_E4M3) return api_fail(GDN_ERR_DTYPE, "out_q must be e4m3");
  if (scales && scales->dtype != GDN_DTYPE_F32) return api_fail(GDN_ERR_DTYPE, "scales must be f32");
  if (!(eps >= 0.f)) return api_fail(GDN_ERR_SHAPE, "eps must be >= 0");
  if ((uintptr_t)weight % 4) return api_fail(GDN_ERR_LAYOUT, "weight must be 4-byte aligned");
  int rc;
  const struct { const gdn_tensor* t; const char* name; } rows[] = {
      {x, "x"}, {residual, "residual"}, {residual_out, "residual_out"}, {out, "out"}, {out_q, "out_q"}};
  for (const auto& v : rows) {
    if (!v.t) continue;
    if ((rc = check_tensor(v.t, v.name, 2, 2))) return rc;
    if (v.t->shape[0] != x->shape[0] || v.t->shape[1] != x->shape[1])
      return api_fail(GDN_ERR_SHAPE, "%s must match x", v.name);
  }
  const int64_t R = x->shape[0], D = x->shape[1];
  if (D < 1 || D > 65536) return api_fail(GDN_ERR_UNSUPPORTED, "D must be 1 .. 65536 (got %lld)", (long long)D);
  int64_t groups = 0;
  if (scales) {
    if ((rc = check_tensor(scales, "scales", 1, 2))) return rc;
    const int64_t want = (D + 127) / 128;
    if (scales->shape[0] != R || (scales->ndim == 2 && scales->shape[1] != want))
      return api_fail(GDN_ERR_SHAPE, "scales must be [R=%lld] or [R, ceil(D/128)=%lld]", (long long)R, (long long)want);
    if (!is_empty(scales) && !contiguous(scales)) return api_fail(GDN_ERR_LAYOUT, "scales must be contiguous");
    groups = scales->ndim == 2 ? want : 0;
  }
  gdn::api_clear_error();
  if (R == 0) return GDN_OK;
  if (R >= kMax32) return api_fail(GDN_ERR_SHAPE, "too many rows");
  // residual_out may be x or residual in place, and out x or residual (each
  // element is written by the thread that read it)
  const Range outs[4] = {range_of(residual_out, "residual_out"), range_of(out, "out"), range_of(out_q, "out_q"),
                         range_of(scales, "scales")};
  const gdn_tensor* out_ts[4] = {residual_out, out, out_q, scales};
  const Range ins[3] = {range_of(x, "x"), range_of(residual, "residual"), range_of(weight, 4 * D, "weight")};
  const gdn_tensor* in_ts[3] = {x, residual, nullptr};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlap(outs[i], ins[j]) && !(i < 2 && same_view(out_ts[i], in_ts[j])))
        return api_fail(GDN_ERR_LAYOUT, "%s overlaps %s", outs[i].name, ins[j].name);
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return api_fail(GDN_ERR_LAYOUT, "%s overlaps %s", outs[i].name, outs[j].name);
    if (i < 3 && out_ts[i] && (rc = check_rows(outs[i].name, R, out_ts[i]->stride[0], 1, 0, D))) return rc;
  }
  const int64_t epg = x->dtype == GDN_DTYPE_BF16 ? 8 : 4;
  bool vec = D % 8 == 0 && aligned16(weight);
  for (const auto& v : rows) {
    if (!v.t) continue;
    if (v.t == out_q) vec = vec && (uintptr_t)v.t->data % 8 == 0 && v.t->stride[0] % 8 == 0;
    else vec = vec && aligned16(v.t->data) && v.t->stride[0] % epg == 0;
  }
  gdn::NormParams p{};
  p.x = x->data;
  p.res = residual ? residual->data : nullptr;
  p.w = weight;
  p.res_out = residual_out ? residual_out->data : nullptr;
  p.out = out ? out->data : nullptr;
  p.out_q = out_q ? (uint8_t*)out_q->data : nullptr;
  p.scales = scales ? (float*)scales->data : nullptr;
  p.rows = R;
  p.x_st = x->stride[0];
  p.r_st = residual ? residual->stride[0] : 0;
  p.ro_st = residual_out ? residual_out->stride[0] : 0;
  p.o_st = out ? out->stride[0] : 0;
  p.q_st = out_q ? out_q->stride[0] : 0;
  p.d = (int32_t)D;
  p.groups = (int32_t)groups;
  p.eps = eps;
  const hipError_t e = gdn::launch_add_rms_norm(x->dtype == GDN_DTYPE_BF16, vec, p, (hipStream_t)stream);
  if (e != hipSuccess) return api_fail(GDN_ERR_HIP, "residual norm launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

}  // extern "C"
