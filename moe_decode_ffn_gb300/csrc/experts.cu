// The routed experts of a batch in 16 bits and their gradients, as one call each: the
// pairs sorted by expert, the products of the sorted rows and SwiGLU (moe_matmul.cu), and
// the rows summed for their tokens (sort.cu). Host code only; the kernels' own files say
// what bounds them. One call instead of one for each step: the steps are many and, for a
// few tokens, shorter than what it takes to ask for them (a training step of 32 tokens
// 470 us of host time step by step, 297 in two calls, most of it autograd's).
#include "host.hpp"
#include "mxint8.cuh"
#include "sort.cuh"

namespace si {

// Places in the block that the forward pass keeps for the backward pass, and in the
// workspace of each.
struct ExpertsGeom {
  int64_t rows;
  size_t order, position, offsets, codes, scales, kept;       // of the kept block, its size
  size_t f_kept, f_sort, f_xs, f_h, f_ys, forward;            // f_kept: where nothing is kept
  size_t part_bytes, b_rows, b_ggu, b_wh, b_gx, backward;
};
static bool experts_ok(const si_experts *L, int n_tokens, int top_k) {
  auto width = [](int n) { return n >= 8 && n % 8 == 0 && n <= (1 << 20); };
  return L && width(L->hidden) && width(L->inter) && L->n_experts >= 1 && L->n_experts <= kSortMaxExperts &&
         n_tokens >= 1 && top_k >= 1 && top_k <= 8 && static_cast<int64_t>(n_tokens) * top_k <= 0x7FFFFFFF - 256;
}
static ExpertsGeom experts_geom(const si_experts &L, int n_tokens, int top_k) {
  ExpertsGeom g{};
  const int64_t R = static_cast<int64_t>(n_tokens) * top_k, H = L.hidden, I = L.inter;
  g.rows = R;
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t from = at;
    at = round_up(at + static_cast<size_t>(bytes), 256);
    return from;
  };
  g.order = take(R * 4);
  g.position = take(R * 4);
  g.offsets = take((L.n_experts + 1) * int64_t(4));
  const size_t lists = at;
  g.codes = take(R * 2 * I);
  g.scales = take(R * 2 * mi_blocks(I));
  g.kept = at;
  at = sizeof(WsHeader);
  g.f_kept = take(static_cast<int64_t>(lists));
  g.f_sort = take(static_cast<int64_t>(si_moe_sort_workspace_bytes(n_tokens, top_k, L.n_experts)));
  g.f_xs = take(R * H * 2);
  g.f_h = take(R * I * 2);
  g.f_ys = take(R * H * 4);
  g.forward = at;
  // the partial sums of si_moe_down_backward lie behind the header
  g.part_bytes = si_moe_down_backward_workspace_bytes(R, L.n_experts, I);
  at = round_up(g.part_bytes, 256);
  g.b_rows = take(R * H * 2);                    // the rows of gy, then of x
  g.b_ggu = take(R * 2 * I * 2);
  g.b_wh = take(R * I * 2);
  g.b_gx = take(R * H * 4);
  g.backward = at;
  return g;
}
template <typename T> static T *in(void *base, size_t at) { return reinterpret_cast<T *>(static_cast<uint8_t *>(base) + at); }

}  // namespace si

using namespace si;

extern "C" size_t si_moe_experts_workspace_bytes(const si_experts *L, int n_tokens, int top_k) {
  if (!experts_ok(L, n_tokens, top_k)) return 0;
  const ExpertsGeom g = experts_geom(*L, n_tokens, top_k);
  return g.forward > g.backward ? g.forward : g.backward;
}

extern "C" size_t si_moe_experts_kept_bytes(const si_experts *L, int n_tokens, int top_k) {
  return experts_ok(L, n_tokens, top_k) ? experts_geom(*L, n_tokens, top_k).kept : 0;
}

static si_status experts_check(const si_experts *L, int n_tokens, int top_k, const void *workspace, size_t bytes) {
  if (!experts_ok(L, n_tokens, top_k) || !L->gate_up || !L->down || !aligned16(L->gate_up) || !aligned16(L->down))
    return SI_ERR_INVALID_ARG;
  if (L->type != SI_BF16 && L->type != SI_F16) return SI_ERR_UNSUPPORTED;
  if (!workspace || !aligned256(workspace) || bytes < si_moe_experts_workspace_bytes(L, n_tokens, top_k))
    return SI_ERR_WORKSPACE;
  return SI_OK;
}

extern "C" si_status si_moe_experts(const si_experts *L, int n_tokens, int top_k, const void *x, const int32_t *topk_ids,
                                    const float *topk_w, void *y, void *kept, void *workspace, size_t workspace_bytes,
                                    void *stream) {
  si_status st = experts_check(L, n_tokens, top_k, workspace, workspace_bytes);
  if (st != SI_OK) return st;
  if (!x || !y || !aligned16(x) || !aligned16(y) || !topk_ids || !topk_w || (kept && !aligned256(kept)))
    return SI_ERR_INVALID_ARG;
  const ExpertsGeom g = experts_geom(*L, n_tokens, top_k);
  const int E = L->n_experts, H = L->hidden, I = L->inter;
  void *lists = kept ? kept : in<void>(workspace, g.f_kept);
  int32_t *order = in<int32_t>(lists, g.order), *position = in<int32_t>(lists, g.position);
  int32_t *offsets = in<int32_t>(lists, g.offsets);
  void *xs = in<void>(workspace, g.f_xs), *h = in<void>(workspace, g.f_h), *ys = in<void>(workspace, g.f_ys);
  const size_t sort_bytes = si_moe_sort_workspace_bytes(n_tokens, top_k, E);
  st = si_moe_sort(topk_ids, n_tokens, top_k, E, order, position, offsets, sort_bytes ? in<void>(workspace, g.f_sort) : nullptr,
                   sort_bytes, stream);
  if (st == SI_OK) st = si_moe_gather(x, L->type, n_tokens, top_k, H, position, offsets + E, xs, stream);
  if (st == SI_OK)
    st = si_moe_gateup(xs, L->type, g.rows, H, L->gate_up, E, I, H, offsets, h, kept ? in<void>(kept, g.codes) : nullptr,
                       kept ? in<void>(kept, g.scales) : nullptr, workspace, sizeof(WsHeader), stream);
  // h is an operand of the tensor cores and so of the matrices' type; the experts' rows stay fp32 until
  // the ranks are summed
  if (st == SI_OK)
    st = si_moe_matmul(h, L->type, g.rows, I, L->down, E, H, I, I, static_cast<int64_t>(H) * I, 0, offsets, ys, SI_F32,
                       H, workspace, sizeof(WsHeader), stream);
  if (st == SI_OK)
    st = si_moe_combine_f32(static_cast<const float *>(ys), n_tokens, top_k, H, position, topk_w, y, L->type, stream);
  return st;
}

extern "C" si_status si_moe_experts_backward(const si_experts *L, int n_tokens, int top_k, const void *gy, const void *x,
                                             const float *topk_w, const void *kept, void *gx, float *gw,
                                             void *ggate_up, void *gdown, void *workspace, size_t workspace_bytes,
                                             void *stream) {
  si_status st = experts_check(L, n_tokens, top_k, workspace, workspace_bytes);
  if (st != SI_OK) return st;
  if (!gy || !topk_w || !kept || !aligned16(gy) || !aligned256(kept) || (ggate_up && (!x || !aligned16(x))) ||
      !aligned16(gx) || !aligned16(ggate_up) || !aligned16(gdown) || (reinterpret_cast<uintptr_t>(gw) & 3u))
    return SI_ERR_INVALID_ARG;
  const ExpertsGeom g = experts_geom(*L, n_tokens, top_k);
  const int E = L->n_experts, H = L->hidden, I = L->inter;
  void *lists = const_cast<void *>(kept);
  const int32_t *order = in<int32_t>(lists, g.order), *position = in<int32_t>(lists, g.position);
  const int32_t *offsets = in<int32_t>(lists, g.offsets);
  void *rows = in<void>(workspace, g.b_rows), *ggu = in<void>(workspace, g.b_ggu), *wh = in<void>(workspace, g.b_wh);
  // nothing of the experts' outputs is kept: with gh = down^T gy, a weight's gradient is <gh, h>. ggu and
  // wh are operands, rounded to the matrices' type (gradients 0.0024 off in bf16; their own rounding alone 0.0017)
  st = si_moe_gather(gy, L->type, n_tokens, top_k, H, position, offsets + E, rows, stream);
  if (st == SI_OK)
    st = si_moe_down_backward(rows, L->type, g.rows, H, L->down, E, H, I, offsets, in<void>(lists, g.codes),
                              in<void>(lists, g.scales), topk_w, order, ggu, gdown ? wh : nullptr, gw, workspace,
                              g.part_bytes, stream);
  if (st == SI_OK && gdown)
    st = si_moe_matmul_grad_w(rows, H, wh, I, L->type, g.rows, E, H, I, offsets, gdown, L->type, workspace,
                              sizeof(WsHeader), stream);
  if (st == SI_OK && ggate_up) {
    st = si_moe_gather(x, L->type, n_tokens, top_k, H, position, offsets + E, rows, stream);
    if (st == SI_OK)
      st = si_moe_matmul_grad_w(ggu, 2 * int64_t(I), rows, H, L->type, g.rows, E, 2 * int64_t(I), H, offsets, ggate_up,
                                L->type, workspace, sizeof(WsHeader), stream);
  }
  if (st == SI_OK && gx) {
    void *gxs = in<void>(workspace, g.b_gx);
    st = si_moe_matmul(ggu, L->type, g.rows, 2 * int64_t(I), L->gate_up, E, H, 2 * int64_t(I), H,
                       2 * static_cast<int64_t>(I) * H, 1, offsets, gxs, SI_F32, H, workspace, sizeof(WsHeader), stream);
    if (st == SI_OK)
      st = si_moe_combine_f32(static_cast<const float *>(gxs), n_tokens, top_k, H, position, nullptr, gx, L->type, stream);
  }
  return st;
}
