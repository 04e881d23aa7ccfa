// Host side of the C ABI declared in include/lrm.h: argument validation, workspace layout and
// kernel launches.  No allocation, no synchronisation (except lrm_read_device_error).
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "lrm_forward.hpp"
#include "lrm_internal.hpp"

using lrm::WsLayout;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

static_assert(sizeof(lrm_router) == 24 && sizeof(lrm_tensor) == 32,
              "lrm_router and lrm_tensor layouts are part of the ABI");
static_assert(sizeof(lrm_admission) == 248 && offsetof(lrm_admission, mem_budget) == 208,
              "lrm_admission layout is part of the ABI");

lrm_status check_problem(const lrm_problem* p) {
  if (!p) return LRM_ERR_INVALID_ARGUMENT;
  if (p->T <= 0 || p->k <= 0 || p->E <= 0 || p->E_loc <= 0 || p->h <= 0 || p->d <= 0)
    return LRM_ERR_INVALID_ARGUMENT;
  if (p->k > p->E || p->e_lo < 0 || (int64_t)p->e_lo + p->E_loc > p->E)
    return LRM_ERR_INVALID_ARGUMENT;
  if (p->L_cap <= 0 || p->K_cap <= 0) return LRM_ERR_INVALID_ARGUMENT;
  if ((int64_t)p->T * p->k > INT32_MAX) return LRM_ERR_UNSUPPORTED;
  if (p->dtype != LRM_F32 && p->dtype != LRM_BF16) return LRM_ERR_UNSUPPORTED;
  if (p->h % 8 != 0 || p->d % 8 != 0) return LRM_ERR_UNSUPPORTED;
  if (p->h > (1 << 23) || p->d > (1 << 23)) return LRM_ERR_UNSUPPORTED;
  if (p->E > 4096 || p->E_loc > 1024) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

lrm_status check_ws(const lrm_problem* p, const void* ws, size_t ws_bytes, WsLayout* wl) {
  if (!ws) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(ws)) return LRM_ERR_UNSUPPORTED;
  *wl = lrm::ws_layout(*p);
  if (ws_bytes < wl->total) return LRM_ERR_WORKSPACE_TOO_SMALL;
  return LRM_OK;
}

lrm_status from_hip(hipError_t e) { return e == hipSuccess ? LRM_OK : LRM_ERR_HIP; }

// FC1's gradients are the grouped products of the FC2 calls with the widths exchanged: rows of
// width 2d (the activation's cotangent dH) against rows of width h (the token inputs x), and FC1
// weights [E_loc][2d][h].  The workspace layout of this problem differs from the original's only
// in the size of its last region (the split experts' partial slots).
lrm_problem fc1_problem(const lrm_problem& p) {
  lrm_problem q = p;
  q.h = 2 * p.d;
  q.d = p.h;
  return q;
}

lrm_status check_router(const lrm_router* r) {
  if (!r) return LRM_ERR_INVALID_ARGUMENT;
  if (r->T <= 0 || r->E <= 0 || r->k <= 0 || r->k > r->E) return LRM_ERR_INVALID_ARGUMENT;
  if (r->gate != LRM_GATE_TOPK && r->gate != LRM_GATE_ALL) return LRM_ERR_INVALID_ARGUMENT;
  if (!(r->balance_coef >= 0.0f) || r->balance_coef == INFINITY) return LRM_ERR_INVALID_ARGUMENT;
  if (r->dtype != LRM_F32 && r->dtype != LRM_BF16) return LRM_ERR_UNSUPPORTED;
  if (r->E > 4096 || (int64_t)r->T * r->k > INT32_MAX) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

// A problem of the forward calls and lrm_gate_dots, whose capacities may be 0: a share without rows.
lrm_status check_forward_problem(const lrm_problem* p) {
  if (!p) return LRM_ERR_INVALID_ARGUMENT;
  lrm_problem q = *p;
  q.L_cap += q.L_cap == 0;
  q.K_cap += q.K_cap == 0;
  return check_problem(&q);
}

lrm_status check_forward_ws(const lrm_problem* p, const void* ws, size_t ws_bytes) {
  if (!ws) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(ws)) return LRM_ERR_UNSUPPORTED;
  return ws_bytes < lrm::forward_ws_bytes(*p) ? LRM_ERR_WORKSPACE_TOO_SMALL : LRM_OK;
}

int64_t element_bytes(int32_t dtype) { return dtype == LRM_BF16 ? 2 : 4; }

// Largest operand the forward products address with 32-bit byte offsets.
constexpr int64_t kMaxOperand = (int64_t)1 << 31;

// Where an entry of a tensor list writes (id = 2 * its index) or reads (2 * index + 1).
struct Start {
  uintptr_t at;
  int64_t id;
};

bool before(const Start& a, const Start& b) { return a.at != b.at ? a.at < b.at : a.id < b.id; }

// Whether some element is written by one entry and read or written by another, or by an entry whose
// dst overlaps its src without being it.  The ranges are looked at in order of their starts: one
// overlaps an earlier one if it starts before that one's end.  The library allocates nothing, so each
// pass over the list takes the lowest starts that are left, kKeep to 2 kKeep of them, and sorts those: a
// list of 40 takes 2 us on the host, one of 1000 25 to 100 (one pass), one of 10000 0.5 to 3 ms (ten).
bool overlapping(const lrm_tensor* list, int32_t n) {
  constexpr int kKeep = 1024;
  Start batch[2 * kKeep], last{}, limit{};
  uintptr_t end = 0, written_end = 0;
  for (bool first = true, more = true; more; first = false) {
    int m = 0;
    more = false;   // starts beyond `limit`, the highest that is kept, are left for a later pass
    const auto take = [&](const void* p, int64_t id) {
      const Start r{(uintptr_t)p, id};
      if ((!first && !before(last, r)) || (more && before(limit, r))) return;
      if (m == 2 * kKeep) {
        std::nth_element(batch, batch + kKeep - 1, batch + m, before);
        limit = batch[kKeep - 1];
        m = kKeep;
        more = true;
        if (before(limit, r)) return;
      }
      batch[m++] = r;
    };
    for (int32_t i = 0; i < n; ++i) {
      if (list[i].count == 0) continue;
      take(list[i].dst, 2 * (int64_t)i);
      if (list[i].src != list[i].dst) take(list[i].src, 2 * (int64_t)i + 1);
    }
    std::sort(batch, batch + m, before);
    for (int i = 0; i < m; ++i) {
      const lrm_tensor& t = list[batch[i].id / 2];
      const uintptr_t lo = batch[i].at, hi = lo + (uintptr_t)(t.count * element_bytes(t.dtype));
      const bool written = batch[i].id % 2 == 0;
      if (lo < written_end || (written && lo < end)) return true;
      end = std::max(end, hi);
      if (written) written_end = std::max(written_end, hi);
    }
    if (m > 0) last = batch[m - 1];
  }
  return false;
}

// The list's entries are well formed; with `write`, also that they do not overlap.
lrm_status check_tensors(const lrm_tensor* list, int32_t n, bool write) {
  if (n < 0 || (n > 0 && !list)) return LRM_ERR_INVALID_ARGUMENT;
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const lrm_tensor& t = list[i];
    if (t.count < 0 || t.reserved != 0) return LRM_ERR_INVALID_ARGUMENT;
    if (t.dtype != LRM_F32 && t.dtype != LRM_BF16) return LRM_ERR_UNSUPPORTED;
    if (t.count >= ((int64_t)1 << 46) || (total += t.count) >= ((int64_t)1 << 46))
      return LRM_ERR_UNSUPPORTED;
    if (t.count == 0) continue;
    const uintptr_t e = (uintptr_t)element_bytes(t.dtype) - 1;
    if (!t.src || (write && !t.dst)) return LRM_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)t.src & e) || (write && ((uintptr_t)t.dst & e))) return LRM_ERR_UNSUPPORTED;
  }
  return write && overlapping(list, n) ? LRM_ERR_INVALID_ARGUMENT : LRM_OK;
}

lrm_status check_grad_ws(int32_t n, const void* ws, size_t ws_bytes) {
  if (!ws) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(ws)) return LRM_ERR_UNSUPPORTED;
  return ws_bytes < lrm::grad_ws_bytes(n) ? LRM_ERR_WORKSPACE_TOO_SMALL : LRM_OK;
}

}  // namespace

#define LRM_TRY(expr)                  \
  do {                                 \
    const lrm_status _s = (expr);      \
    if (_s != LRM_OK) return _s;       \
  } while (0)

namespace {

// lrm_grouped_fc2 and lrm_combine_tokens; `wide`: y in float32 whatever the layer's type.
lrm_status fc2(const lrm_problem* problem, const int32_t* fwd_off, const void* phi, const void* W,
               void* y, bool wide, void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_forward_problem(problem));
  if (!fwd_off || !W) return LRM_ERR_INVALID_ARGUMENT;
  if (problem->L_cap > 0 && (!phi || !y)) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(phi) || !aligned16(W) || !aligned16(y)) return LRM_ERR_UNSUPPORTED;
  // one expert's weights, and the 256 rows of phi of a tile
  const int64_t row = problem->d * element_bytes(problem->dtype);
  if (problem->h * row > kMaxOperand || 256 * row > kMaxOperand) return LRM_ERR_UNSUPPORTED;
  LRM_TRY(check_forward_ws(problem, ws, ws_bytes));
  return from_hip(lrm::launch_fc2(*problem, fwd_off, phi, W, y, wide, stream));
}

lrm_status combine(const lrm_problem* problem, const int32_t* row_pair, const int32_t* fwd_off,
                   const float* topk_w, const void* y, bool wide, const void* residual, void* out,
                   void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_forward_problem(problem));
  if (!fwd_off || !topk_w || !out) return LRM_ERR_INVALID_ARGUMENT;
  if (problem->L_cap > 0 && (!row_pair || !y)) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(y) || !aligned16(residual) || !aligned16(out)) return LRM_ERR_UNSUPPORTED;
  LRM_TRY(check_forward_ws(problem, ws, ws_bytes));
  return from_hip(lrm::launch_combine(*problem, row_pair, fwd_off, topk_w, y, wide, residual, out,
                                      (char*)ws, stream));
}

}  // namespace

extern "C" {

size_t lrm_workspace_bytes(const lrm_problem* problem) {
  if (check_problem(problem) != LRM_OK) return 0;
  const size_t a = lrm::ws_layout(*problem).total, b = lrm::ws_layout(fc1_problem(*problem)).total;
  return a > b ? a : b;
}

lrm_status lrm_plan_quotas(const lrm_problem* problem, const lrm_quota_policy* policy,
                           const int32_t* topk_idx, int32_t* counts, int32_t* fwd_off,
                           int32_t* row_pair, int32_t* quota, int32_t* cmp_off, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!policy || !topk_idx || !counts || !fwd_off || !row_pair || !quota || !cmp_off)
    return LRM_ERR_INVALID_ARGUMENT;
  if (!policy->full && (policy->rho_den <= 0 || policy->rho_num < 0))
    return LRM_ERR_INVALID_ARGUMENT;
  if (policy->kind < LRM_QUOTA_CAP || policy->kind > LRM_QUOTA_WATERFILL) return LRM_ERR_INVALID_ARGUMENT;
  if (policy->kind == LRM_QUOTA_PROPORTIONAL && policy->cap_abs >= 0) return LRM_ERR_INVALID_ARGUMENT;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_plan(*problem, *policy, topk_idx, counts, fwd_off, row_pair, quota,
                                   cmp_off, (char*)ws, wl, stream));
}

lrm_status lrm_admit_quotas(const lrm_problem* problem, const lrm_admission* admission,
                            const int32_t* fwd_off, int32_t* quota, int32_t* cmp_off,
                            int32_t* admitted, void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  const lrm_admission* a = admission;
  if (!a || !fwd_off || !quota || !cmp_off || !admitted) return LRM_ERR_INVALID_ARGUMENT;
  if (a->n_cand < 1 || a->n_cand > LRM_MAX_CANDIDATES) return LRM_ERR_INVALID_ARGUMENT;
  if (a->kind < LRM_QUOTA_CAP || a->kind > LRM_QUOTA_WATERFILL) return LRM_ERR_INVALID_ARGUMENT;
  if (a->kind == LRM_QUOTA_PROPORTIONAL && a->cap_abs >= 0) return LRM_ERR_INVALID_ARGUMENT;
  for (int c = 0; c < a->n_cand; ++c)
    if (!a->full[c] && (a->rho_den[c] <= 0 || a->rho_num[c] < 0)) return LRM_ERR_INVALID_ARGUMENT;
  const int64_t lim = (int64_t)1 << 32;
  if (a->mem_base < 0 || a->mem_per_row < 0 || a->mem_per_row > lim || a->comm_per_row < 0 ||
      a->comm_per_row > lim || a->mem_base > ((int64_t)1 << 62))
    return LRM_ERR_INVALID_ARGUMENT;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_admit(*problem, *a, fwd_off, quota, cmp_off, admitted, stream));
}

lrm_status lrm_score(const lrm_problem* problem, const float* topk_w, const void* g,
                     const void* phi, const int32_t* row_pair, const int32_t* fwd_off,
                     float* score, void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!topk_w || !g || !phi || !row_pair || !fwd_off || !score) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(g) || !aligned16(phi)) return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_score(*problem, topk_w, g, phi, row_pair, fwd_off, score, (char*)ws,
                                    wl, stream));
}

lrm_status lrm_score_norms(const lrm_problem* problem, const void* g, const void* phi, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!g || !phi) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(g) || !aligned16(phi)) return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_score_norms(*problem, g, phi, (char*)ws, wl, stream));
}

lrm_status lrm_score_combine(const lrm_problem* problem, const float* topk_w,
                             const int32_t* row_pair, const int32_t* fwd_off, float* score,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!topk_w || !row_pair || !fwd_off || !score) return LRM_ERR_INVALID_ARGUMENT;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_score_combine(*problem, topk_w, row_pair, fwd_off, score, (char*)ws,
                                            wl, stream));
}

lrm_status lrm_score_criterion(const lrm_problem* problem, int32_t criterion, const float* topk_w,
                               const void* g, const void* phi, const float* keys,
                               const int32_t* row_pair, const int32_t* fwd_off, float* score,
                               void* ws, size_t ws_bytes, hipStream_t stream) {
  if (criterion == LRM_CRIT_LRM)
    return lrm_score(problem, topk_w, g, phi, row_pair, fwd_off, score, ws, ws_bytes, stream);
  LRM_TRY(check_problem(problem));
  if (criterion != LRM_CRIT_GRAD_SQ && criterion != LRM_CRIT_GRAD_ABS && criterion != LRM_CRIT_RANDOM)
    return LRM_ERR_INVALID_ARGUMENT;
  if (!row_pair || !fwd_off || !score) return LRM_ERR_INVALID_ARGUMENT;
  if (criterion == LRM_CRIT_RANDOM ? !keys : !g) return LRM_ERR_INVALID_ARGUMENT;
  if (criterion != LRM_CRIT_RANDOM && !aligned16(g)) return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_score_criterion(*problem, criterion, g, keys, row_pair, fwd_off,
                                              score, (char*)ws, wl, stream));
}

lrm_status lrm_select(const lrm_problem* problem, const float* score, const int32_t* fwd_off,
                      const int32_t* quota, const int32_t* cmp_off, int32_t* sel_row, void* ws,
                      size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!score || !fwd_off || !quota || !cmp_off || !sel_row) return LRM_ERR_INVALID_ARGUMENT;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_select(*problem, score, fwd_off, quota, cmp_off, sel_row, (char*)ws,
                                     wl, stream));
}

lrm_status lrm_compact(const lrm_problem* problem, const int32_t* sel_row, const int32_t* row_pair,
                       const int32_t* cmp_off, const float* topk_w, const void* g,
                       const void* phi, void* Gc, void* Phic, int32_t* sel_pair, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!sel_row || !row_pair || !cmp_off || !topk_w || !g || !phi || !Gc || !Phic || !sel_pair)
    return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(g) || !aligned16(phi) || !aligned16(Gc) || !aligned16(Phic))
    return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_compact(*problem, sel_row, row_pair, cmp_off, topk_w, g, phi, Gc,
                                      Phic, sel_pair, (char*)ws, wl, stream));
}

lrm_status lrm_grouped_dw(const lrm_problem* problem, const void* Gc, const void* Phic,
                          const int32_t* cmp_off, float* dW, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!Gc || !Phic || !cmp_off || !dW) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(Gc) || !aligned16(Phic) || !aligned16(dW)) return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_dw(*problem, Gc, Phic, cmp_off, dW, (char*)ws, wl, stream));
}

lrm_status lrm_grouped_dx(const lrm_problem* problem, const void* Gc, const void* W,
                          const int32_t* cmp_off, float* dphi, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!Gc || !W || !cmp_off || !dphi) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(Gc) || !aligned16(W) || !aligned16(dphi)) return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_dx(*problem, Gc, W, cmp_off, dphi, (char*)ws, wl, stream));
}

lrm_status lrm_grouped_dw_dx(const lrm_problem* problem, const void* Gc, const void* Phic,
                             const void* W, const int32_t* cmp_off, float* dW, float* dphi,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!Gc || !Phic || !W || !cmp_off || !dW || !dphi) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(Gc) || !aligned16(Phic) || !aligned16(W) || !aligned16(dW) || !aligned16(dphi))
    return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_gemms(*problem, Gc, Phic, W, cmp_off, dW, dphi, (char*)ws, wl,
                                    stream, 2));
}

lrm_status lrm_grouped_dw_dx_noalloc(const lrm_problem* problem, const void* Gc,
                                     const void* Phic, const void* W, const int32_t* cmp_off,
                                     float* dW, float* dphi, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!Gc || !Phic || !W || !cmp_off || !dW || !dphi) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(Gc) || !aligned16(Phic) || !aligned16(W) || !aligned16(dW) || !aligned16(dphi))
    return LRM_ERR_UNSUPPORTED;
  if (lrm::noalloc_layout(*problem).total > lrm::kNoallocScratchBytes)
    return LRM_ERR_WORKSPACE_TOO_SMALL;
  return from_hip(lrm::launch_gemms_noalloc(*problem, Gc, Phic, W, cmp_off, dW, dphi, stream));
}

lrm_status lrm_swiglu_backward(const lrm_problem* problem, const int32_t* sel_row,
                                const int32_t* cmp_off, const float* dphi, const void* ac,
                                void* dH, void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!sel_row || !cmp_off || !dphi || !ac || !dH) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(dphi) || !aligned16(ac) || !aligned16(dH)) return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_swiglu_bwd(*problem, sel_row, cmp_off, dphi, ac, dH, (char*)ws, wl,
                                         stream));
}

lrm_status lrm_gather_tokens(const lrm_problem* problem, const int32_t* sel_pair,
                             const int32_t* cmp_off, const void* x, void* Xc, void* ws,
                             size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!sel_pair || !cmp_off || !x || !Xc) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(Xc)) return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_gather_tokens(*problem, sel_pair, cmp_off, x, Xc, (char*)ws, wl,
                                            stream));
}

lrm_status lrm_grouped_fc1_dw(const lrm_problem* problem, const void* dH, const void* Xc,
                              const int32_t* cmp_off, float* dW1, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!dH || !Xc || !cmp_off || !dW1) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(dH) || !aligned16(Xc) || !aligned16(dW1)) return LRM_ERR_UNSUPPORTED;
  const lrm_problem q = fc1_problem(*problem);
  WsLayout wl;
  LRM_TRY(check_ws(&q, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_dw(q, dH, Xc, cmp_off, dW1, (char*)ws, wl, stream));
}

lrm_status lrm_grouped_fc1_dx(const lrm_problem* problem, const void* dH, const void* W1,
                              const int32_t* cmp_off, float* dX, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!dH || !W1 || !cmp_off || !dX) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(dH) || !aligned16(W1) || !aligned16(dX)) return LRM_ERR_UNSUPPORTED;
  const lrm_problem q = fc1_problem(*problem);
  WsLayout wl;
  LRM_TRY(check_ws(&q, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_dx(q, dH, W1, cmp_off, dX, (char*)ws, wl, stream));
}

lrm_status lrm_grouped_fc1_dw_dx(const lrm_problem* problem, const void* dH, const void* Xc,
                                 const void* W1, const int32_t* cmp_off, float* dW1, float* dX,
                                 void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!dH || !Xc || !W1 || !cmp_off || !dW1 || !dX) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(dH) || !aligned16(Xc) || !aligned16(W1) || !aligned16(dW1) || !aligned16(dX))
    return LRM_ERR_UNSUPPORTED;
  const lrm_problem q = fc1_problem(*problem);
  WsLayout wl;
  LRM_TRY(check_ws(&q, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_gemms(q, dH, Xc, W1, cmp_off, dW1, dX, (char*)ws, wl, stream, 1));
}

lrm_status lrm_scatter_tokens(const lrm_problem* problem, const int32_t* sel_pair,
                              const int32_t* cmp_off, const float* dX, float* dx, void* ws,
                              size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_problem(problem));
  if (!sel_pair || !cmp_off || !dX || !dx) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(dX) || !aligned16(dx)) return LRM_ERR_UNSUPPORTED;
  WsLayout wl;
  LRM_TRY(check_ws(problem, ws, ws_bytes, &wl));
  return from_hip(lrm::launch_scatter_tokens(*problem, sel_pair, cmp_off, dX, dx, (char*)ws, wl,
                                             stream));
}

size_t lrm_router_workspace_bytes(const lrm_router* router) {
  return check_router(router) == LRM_OK ? lrm::route_ws(router->E).total : 0;
}

lrm_status lrm_route(const lrm_router* router, const void* logits, const uint8_t* mask,
                     int32_t* topk_idx, float* topk_w, float* lse, int32_t* counts, float* prob,
                     float* loss, void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_router(router));
  if (!logits || !topk_idx || !topk_w || !lse || !counts || !prob || !loss || !ws)
    return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(logits) || !aligned16(ws)) return LRM_ERR_UNSUPPORTED;
  if (ws_bytes < lrm::route_ws(router->E).total) return LRM_ERR_WORKSPACE_TOO_SMALL;
  return from_hip(lrm::launch_route(*router, logits, mask, topk_idx, topk_w, lse, counts, prob, loss,
                                    (char*)ws, stream));
}

lrm_status lrm_route_backward(const lrm_router* router, const void* logits,
                              const int32_t* topk_idx, const float* topk_w, const int32_t* counts,
                              const float* adot, float* dlogits, hipStream_t stream) {
  LRM_TRY(check_router(router));
  if (!logits || !topk_idx || !topk_w || !counts || !dlogits) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(logits) || !aligned16(dlogits)) return LRM_ERR_UNSUPPORTED;
  return from_hip(lrm::launch_route_backward(*router, logits, topk_idx, topk_w, counts, adot,
                                             dlogits, stream));
}

lrm_status lrm_gate_dots(const lrm_problem* problem, const int32_t* sel_pair,
                         const int32_t* cmp_off, const float* dphi, const void* Phic, float* adot,
                         void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_forward_problem(problem));
  if (!cmp_off || !adot) return LRM_ERR_INVALID_ARGUMENT;
  if (problem->K_cap > 0 && (!sel_pair || !dphi || !Phic)) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(dphi) || !aligned16(Phic)) return LRM_ERR_UNSUPPORTED;
  LRM_TRY(check_forward_ws(problem, ws, ws_bytes));
  return from_hip(lrm::launch_gate_dots(*problem, sel_pair, cmp_off, dphi, Phic, adot, (char*)ws,
                                        stream));
}

size_t lrm_forward_workspace_bytes(const lrm_problem* problem) {
  return check_forward_problem(problem) == LRM_OK ? lrm::forward_ws_bytes(*problem) : 0;
}

lrm_status lrm_grouped_fc1_swiglu(const lrm_problem* problem, const int32_t* row_pair,
                                  const int32_t* fwd_off, const void* x, const void* W1, void* ac,
                                  void* phi, void* ws, size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_forward_problem(problem));
  if (!fwd_off || !x || !W1) return LRM_ERR_INVALID_ARGUMENT;
  if (problem->L_cap > 0 && (!row_pair || !phi)) return LRM_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(W1) || !aligned16(ac) || !aligned16(phi)) return LRM_ERR_UNSUPPORTED;
  const int64_t row = problem->h * element_bytes(problem->dtype);
  if (problem->T * row > kMaxOperand || 2 * problem->d * row > kMaxOperand) return LRM_ERR_UNSUPPORTED;
  LRM_TRY(check_forward_ws(problem, ws, ws_bytes));
  return from_hip(lrm::launch_fc1_swiglu(*problem, row_pair, fwd_off, x, W1, ac, phi, (char*)ws,
                                         stream));
}

lrm_status lrm_grouped_fc2(const lrm_problem* problem, const int32_t* fwd_off, const void* phi,
                           const void* W, void* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  return fc2(problem, fwd_off, phi, W, y, false, ws, ws_bytes, stream);
}

lrm_status lrm_grouped_fc2_wide(const lrm_problem* problem, const int32_t* fwd_off, const void* phi,
                                const void* W, float* y, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  return fc2(problem, fwd_off, phi, W, y, true, ws, ws_bytes, stream);
}

lrm_status lrm_combine_tokens(const lrm_problem* problem, const int32_t* row_pair,
                              const int32_t* fwd_off, const float* topk_w, const void* y,
                              const void* residual, void* out, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  return combine(problem, row_pair, fwd_off, topk_w, y, false, residual, out, ws, ws_bytes, stream);
}

lrm_status lrm_combine_tokens_wide(const lrm_problem* problem, const int32_t* row_pair,
                                   const int32_t* fwd_off, const float* topk_w, const float* y,
                                   const void* residual, void* out, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
  return combine(problem, row_pair, fwd_off, topk_w, y, true, residual, out, ws, ws_bytes, stream);
}

size_t lrm_grad_workspace_bytes(const lrm_tensor* list, int32_t n) {
  return check_tensors(list, n, false) == LRM_OK ? lrm::grad_ws_bytes(n) : 0;
}

lrm_status lrm_grad_norm(const lrm_tensor* list, int32_t n, float* norm, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  LRM_TRY(check_tensors(list, n, false));
  if (!norm) return LRM_ERR_INVALID_ARGUMENT;
  LRM_TRY(check_grad_ws(n, ws, ws_bytes));
  return from_hip(lrm::launch_grad_norm(list, n, norm, (char*)ws, stream));
}

lrm_status lrm_clip_grads(const lrm_tensor* list, int32_t n, float max_norm, float* norm, void* ws,
                          size_t ws_bytes, hipStream_t stream) {
  LRM_TRY(check_tensors(list, n, true));
  if (!norm || !(max_norm > 0.0f) || max_norm == INFINITY) return LRM_ERR_INVALID_ARGUMENT;
  LRM_TRY(check_grad_ws(n, ws, ws_bytes));
  return from_hip(lrm::launch_clip(list, n, max_norm, norm, (char*)ws, stream));
}

lrm_status lrm_read_device_error(void* ws, int32_t* code, int32_t clear, hipStream_t stream) {
  if (!ws || !code) return LRM_ERR_INVALID_ARGUMENT;
  int32_t v = 0;
  if (hipMemcpyAsync(&v, ws, sizeof(v), hipMemcpyDeviceToHost, stream) != hipSuccess)
    return LRM_ERR_HIP;
  if (hipStreamSynchronize(stream) != hipSuccess) return LRM_ERR_HIP;
  *code = v;
  if (clear) {
    const int32_t z = 0;
    if (hipMemcpyAsync(ws, &z, sizeof(z), hipMemcpyHostToDevice, stream) != hipSuccess)
      return LRM_ERR_HIP;
    if (hipStreamSynchronize(stream) != hipSuccess) return LRM_ERR_HIP;
  }
  return LRM_OK;
}

const char* lrm_status_string(lrm_status status) {
  switch (status) {
    case LRM_OK: return "ok";
    case LRM_ERR_INVALID_ARGUMENT: return "invalid argument";
    case LRM_ERR_UNSUPPORTED: return "unsupported problem or alignment";
    case LRM_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case LRM_ERR_HIP: return "HIP launch or runtime error";
  }
  return "unknown status";
}

}  // extern "C"
