// C ABI of the operators around the recurrence: argument checks, workspace sizes
// and launches.  See include/gdr.h for the contract of every entry point.
#include "gdr_layer.h"

#include <cstdio>
#include <initializer_list>

#include "gdr_host.h"
#include "gdr_kernels.h"

namespace {

using gdr::host_status;

constexpr int64_t kAlign = 256;
int64_t round_up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

int32_t invalid(const char *msg) { return host_status(GDR_ERR_INVALID_ARG, msg); }
int32_t unsupported(const char *msg) { return host_status(GDR_ERR_UNSUPPORTED, msg); }

bool is_dtype(int32_t d) { return d == GDR_BF16 || d == GDR_F32; }
bool element_aligned(const void *p, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(p) % (dtype == GDR_BF16 ? 2 : 4) == 0;
}
// Stride of [T] rows `width` wide; rows of fewer than two tokens have none to check.
bool stride_ok(int64_t stride, int64_t width, int64_t T) { return T < 2 || stride >= width; }

// Whether one of a call's outputs is one of its inputs.  (Parts of one wider buffer,
// which rows may be, start at different addresses; other overlaps are the caller's.)
using Pointers = std::initializer_list<const void *>;
bool aliases(Pointers outs, Pointers ins) {
  for (const void *out : outs)
    for (const void *in : ins)
      if (out && out == in) return true;
  return false;
}

int32_t check_workspace(void *ws, int64_t have, int64_t need) {
  if (need > 0 && !ws) return host_status(GDR_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return host_status(GDR_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (have < need) {
    char msg[96];
    std::snprintf(msg, sizeof msg, "workspace too small: need %lld bytes, got %lld", (long long)need, (long long)have);
    return host_status(GDR_ERR_WORKSPACE, msg);
  }
  return GDR_OK;
}

// Device check, then the launches of one call; a failing one ends the call.
template <class F>
int32_t launch(int kernel, void *stream, const char *what, F f) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  return gdr::host_hip(gdr::timed_launch(kernel, st, [&] { return f(st); }), what);
}

// ---- convolution ----

int32_t check_conv(const gdr_conv *p, bool step) {
  if (!p) return invalid("problem is NULL");
  if (p->T < 0 || p->N < 0) return invalid("T and N must be >= 0");
  if (p->C < 1) return invalid("C must be positive");
  if (p->W < 2 || p->W > 8) return unsupported("W outside 2..8");
  if (!is_dtype(p->dtype) || !is_dtype(p->w_dtype)) return invalid("unknown dtype");
  if (p->activation != GDR_ACT_NONE && p->activation != GDR_ACT_SILU) return invalid("activation must be none or SiLU");
  // parameter sums index (W + 1) C columns with 32 bits
  if (p->C > (1 << 24)) return unsupported("C above 2^24");
  if (!stride_ok(p->x_stride, p->C, p->T)) return invalid("x_stride below C");
  if (p->T > 0 && (!p->x || !p->weight)) return invalid("x and weight must be non-NULL");
  if (!element_aligned(p->x, p->dtype) || !element_aligned(p->s0, p->dtype) || !element_aligned(p->weight, p->w_dtype) ||
      !element_aligned(p->bias, p->w_dtype))
    return invalid("x, weight, bias and s0 must be aligned to their elements");
  if (step) {
    if (p->N != p->T) return invalid("N must equal T");
    return GDR_OK;
  }
  const int64_t least = ((int64_t)p->T + 63) / 64;
  if (p->n_chunks < 0 || p->n_chunks > p->T || p->n_chunks < least || p->n_chunks > least + p->N)
    return invalid("n_chunks is inconsistent with T and N");
  if (p->n_chunks >= (1 << 28)) return unsupported("2^28 chunks or more");  // runs of 8 tokens are counted with 32 bits
  if (p->T > 0 && p->N == 0) return invalid("tokens without documents");
  if (p->N > 0 && !p->chunk_table) return invalid("chunk_table must be non-NULL");
  return GDR_OK;
}
const char *const kTooMany = "too many rows and channels for one launch";
// The parameter sums take a launch of their own over (W + 1) C columns.
bool conv_sum_fits(int32_t C, int32_t W) {
  return gdr::one_launch(gdr::sum_blocks((int64_t)(W + 1) * C), gdr::SUM_PARTS * gdr::SUM_COLS);
}
int64_t conv_bytes(int32_t n_chunks, int32_t C, int32_t W) {
  return round_up((int64_t)gdr::conv_bwd_plan(n_chunks, C).rows() * (W + 1) * C * 4);
}

int32_t conv_fwd(const gdr_conv *p, void *y, int64_t y_stride, void *st, void *stream) {
  int32_t rc = check_conv(p, false);
  if (rc) return rc;
  if (p->T > 0 && !y) return invalid("y is NULL");
  if (!stride_ok(y_stride, p->C, p->T)) return invalid("y_stride below C");
  const gdr::ConvFwdPlan plan = gdr::conv_fwd_plan(*p, st != nullptr);
  if (!gdr::one_launch(plan.rows(), plan.lanes)) return unsupported(kTooMany);
  if (!element_aligned(y, p->dtype) || !element_aligned(st, p->dtype)) return invalid("y and st must be aligned to their elements");
  if (aliases({y, st}, {p->x, p->weight, p->bias, p->s0, p->chunk_table})) return invalid("y or st is an input");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(gdr::TK_CONV_FWD, stream, "convolution launch",
                   [&](hipStream_t s) { return gdr::launch_conv_fwd(*p, y, y_stride, st, s); })))
    return rc;
  return host_status(GDR_OK, "");
}

int32_t conv_bwd(const gdr_conv *p, const void *dy, int64_t dy_stride, const void *dst, void *dx, int64_t dx_stride, float *dw,
                 float *dbias, void *ds0, void *ws, int64_t ws_bytes, void *stream) {
  int32_t rc = check_conv(p, false);
  if (rc) return rc;
  if (!dw) return invalid("dweight is NULL");
  if (p->T > 0 && (!dy || !dx)) return invalid("dy and dx must be non-NULL");
  // the kernel reads the weight wherever it is launched, for ds0 of empty documents too
  if (p->N > 0 && ds0 && !p->weight) return invalid("weight must be non-NULL with ds0");
  if (!stride_ok(dy_stride, p->C, p->T) || !stride_ok(dx_stride, p->C, p->T)) return invalid("dy_stride or dx_stride below C");
  const gdr::ConvBwdPlan plan = gdr::conv_bwd_plan(p->n_chunks, p->C);
  if (!conv_sum_fits(p->C, p->W) || !gdr::one_launch(plan.rows() + plan.docs(p->N, ds0 != nullptr), plan.lanes))
    return unsupported(kTooMany);
  if (!element_aligned(dy, p->dtype) || !element_aligned(dst, p->dtype) || !element_aligned(dx, p->dtype) ||
      !element_aligned(ds0, p->dtype) || !element_aligned(dw, GDR_F32) || !element_aligned(dbias, GDR_F32))
    return invalid("gradients must be aligned to their elements");
  const int64_t need = conv_bytes(p->n_chunks, p->C, p->W);
  if ((rc = check_workspace(ws, ws_bytes, need))) return rc;
  if (aliases({dx, dw, dbias, ds0}, {p->x, p->weight, p->bias, p->s0, p->chunk_table, dy, dst}))
    return invalid("dx, dweight, dbias or ds0 is an input");
  if ((rc = gdr::host_check_device())) return rc;
  const int rows = plan.rows();
  float *partial = static_cast<float *>(ws);
  if ((rc = launch(gdr::TK_CONV_BWD, stream, "convolution gradient launch", [&](hipStream_t s) {
         return gdr::launch_conv_bwd(*p, dy, dy_stride, dst, dx, dx_stride, ds0, partial, s);
       })))
    return rc;
  if ((rc = launch(gdr::TK_PARAM_SUM, stream, "parameter sum launch",
                   [&](hipStream_t s) { return gdr::launch_conv_sum(partial, rows, p->C, p->W, dw, dbias, s); })))
    return rc;
  return host_status(GDR_OK, "");
}

int32_t conv_step(const gdr_conv *p, void *y, int64_t y_stride, void *state, const int32_t *slots, int32_t n_slots, void *stream) {
  int32_t rc = check_conv(p, true);
  if (rc) return rc;
  if (n_slots < 0) return invalid("n_slots must be >= 0");
  if (!slots && p->N > n_slots) return invalid("fewer slots than sequences");
  if (p->T > 0 && (!y || (n_slots > 0 && !state))) return invalid("y and state must be non-NULL");
  if (!stride_ok(y_stride, p->C, p->T)) return invalid("y_stride below C");
  const gdr::ConvStepPlan plan = gdr::conv_step_plan(*p);
  if (!gdr::one_launch(plan.rows, plan.lanes)) return unsupported(kTooMany);
  if (!element_aligned(y, p->dtype) || !element_aligned(state, p->dtype) || !element_aligned(slots, GDR_F32))
    return invalid("y, state and slots must be aligned to their elements");
  if (aliases({y}, {p->x, p->weight, p->bias, slots, state}) || aliases({state}, {p->x, p->weight, p->bias, slots}))
    return invalid("y or state is an input");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(gdr::TK_CONV_STEP, stream, "convolution step launch",
                   [&](hipStream_t s) { return gdr::launch_conv_step(*p, y, y_stride, state, slots, n_slots, s); })))
    return rc;
  return host_status(GDR_OK, "");
}

// ---- gate ----

int32_t check_gate_sizes(int32_t T, int32_t H, int32_t D, int32_t dtype) {
  if (T < 0) return invalid("T must be >= 0");
  if (H < 1) return invalid("H must be positive");
  if (D != 1 && D != 128) return unsupported("D must be 1 or 128");
  if (H > 65536) return unsupported("H above 65536");
  if (!is_dtype(dtype)) return invalid("unknown dtype");
  return GDR_OK;
}
int32_t check_gate(const gdr_gate *p) {
  if (!p) return invalid("problem is NULL");
  const int32_t rc = check_gate_sizes(p->T, p->H, p->D, p->dtype);
  if (rc) return rc;
  if (p->kind != GDR_GATE_SOFTPLUS && p->kind != GDR_GATE_SIGMOID) return invalid("unknown gate kind");
  if (!(p->floor >= -8.f && p->floor < 0.f)) return invalid("floor outside [-8, 0)");
  if (!stride_ok(p->x_stride, (int64_t)p->H * p->D, p->T)) return invalid("x_stride below H * D");
  if (p->T > 0 && (!p->x || !p->a_log)) return invalid("x and a_log must be non-NULL");
  if (!element_aligned(p->x, p->dtype) || !element_aligned(p->a_log, GDR_F32) || !element_aligned(p->bias, GDR_F32))
    return invalid("x, a_log and bias must be aligned to their elements");
  return GDR_OK;
}
int64_t gate_bytes(int32_t T, int32_t C, int32_t D) {
  return round_up((int64_t)gdr::gate_rows(T, C) * gdr::gate_partial_row(C, D, gdr::gate_vec(C)) * 4);
}

int32_t gate_fwd(const gdr_gate *p, float *g, void *stream) {
  int32_t rc = check_gate(p);
  if (rc) return rc;
  if (p->T > 0 && !g) return invalid("g is NULL");
  if (!element_aligned(g, GDR_F32)) return invalid("g must be aligned to its elements");
  if (aliases({g}, {p->x, p->a_log, p->bias})) return invalid("g is an input");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(gdr::TK_GATE_FWD, stream, "gate launch", [&](hipStream_t s) { return gdr::launch_gate_fwd(*p, g, s); })))
    return rc;
  return host_status(GDR_OK, "");
}

int32_t gate_bwd(const gdr_gate *p, const float *dg, void *dx, int64_t dx_stride, float *da, float *dbias, void *ws,
                 int64_t ws_bytes, void *stream) {
  int32_t rc = check_gate(p);
  if (rc) return rc;
  if (!da) return invalid("da_log is NULL");
  if (p->T > 0 && (!dg || !dx)) return invalid("dg and dx must be non-NULL");
  const int32_t C = p->H * p->D;
  if (!stride_ok(dx_stride, C, p->T)) return invalid("dx_stride below H * D");
  if (!element_aligned(dg, GDR_F32) || !element_aligned(dx, p->dtype) || !element_aligned(da, GDR_F32) ||
      !element_aligned(dbias, GDR_F32))
    return invalid("gradients must be aligned to their elements");
  if ((rc = check_workspace(ws, ws_bytes, gate_bytes(p->T, C, p->D)))) return rc;
  if (aliases({dx, da, dbias}, {p->x, p->a_log, p->bias, dg})) return invalid("dx, da_log or dbias is an input");
  if ((rc = gdr::host_check_device())) return rc;
  float *partial = static_cast<float *>(ws);
  const int rows = gdr::gate_rows(p->T, C);
  if ((rc = launch(gdr::TK_GATE_BWD, stream, "gate gradient launch",
                   [&](hipStream_t s) { return gdr::launch_gate_bwd(*p, dg, dx, dx_stride, partial, s); })))
    return rc;
  if ((rc = launch(gdr::TK_PARAM_SUM, stream, "parameter sum launch",
                   [&](hipStream_t s) { return gdr::launch_gate_sum(partial, rows, p->H, p->D, da, dbias, s); })))
    return rc;
  return host_status(GDR_OK, "");
}

// ---- single-token recurrence ----

int32_t step(bool gdn, const gdr_step *p, uint16_t *o, void *stream) {
  if (!p) return invalid("problem is NULL");
  if (p->T < 0 || p->N < 0 || p->n_slots < 0) return invalid("T, N and n_slots must be >= 0");
  if (p->H_qk <= 0 || p->H_v <= 0) return invalid("head counts must be positive");
  if (p->K != 128 || p->V != 128) return unsupported("only K = V = 128 is implemented");
  if (!gdn && p->H_qk != p->H_v) return unsupported("KDA needs H_qk == H_v");
  if (gdn && p->H_v % p->H_qk != 0) return unsupported("GDN needs H_v to be a multiple of H_qk");
  if (p->H_v > 65536 || !gdr::one_launch((int64_t)p->N * p->H_v, 256)) return unsupported("problem too large");
  if (!(p->scale == p->scale)) return invalid("scale is NaN");
  if (p->input_flags & ~(GDR_IN_QK_L2NORM | GDR_IN_BETA_SIGMOID)) return invalid("unknown input flag");
  if (!p->cu_seqlens && p->N != p->T) return invalid("N must equal T without cu_seqlens");
  if (!p->slots && p->N > p->n_slots) return invalid("fewer slots than sequences");
  const int64_t wq = (int64_t)p->H_qk * 128, wv = (int64_t)p->H_v * 128;
  if (!stride_ok(p->q_stride, wq, p->T) || !stride_ok(p->k_stride, wq, p->T) || !stride_ok(p->v_stride, wv, p->T))
    return invalid("q_stride, k_stride or v_stride below the row's width");
  if (p->T > 0 && p->N > 0) {
    if (!p->q || !p->k || !p->v || !p->g || !p->beta || !o) return invalid("q, k, v, g, beta and o must be non-NULL");
    if (p->n_slots > 0 && !p->state) return invalid("state is NULL");
  }
  if (reinterpret_cast<uintptr_t>(p->state) % 16) return invalid("state is not 16-byte aligned");
  if (!element_aligned(p->q, GDR_BF16) || !element_aligned(p->k, GDR_BF16) || !element_aligned(p->v, GDR_BF16) ||
      !element_aligned(p->g, GDR_F32) || !element_aligned(p->beta, gdn ? GDR_F32 : GDR_BF16) ||
      !element_aligned(p->cu_seqlens, GDR_F32) || !element_aligned(p->slots, GDR_F32) || !element_aligned(o, GDR_BF16))
    return invalid("operands must be aligned to their elements");
  if (aliases({o}, {p->q, p->k, p->v, p->g, p->beta, p->cu_seqlens, p->slots, p->state}) ||
      aliases({p->state}, {p->q, p->k, p->v, p->g, p->beta, p->cu_seqlens, p->slots}))
    return invalid("o or state is an input");
  int32_t rc = gdr::host_check_device();
  if (rc) return rc;
  if ((rc = launch(gdr::TK_STEP, stream, "step launch", [&](hipStream_t s) { return gdr::launch_step(gdn, *p, o, s); }))) return rc;
  return host_status(GDR_OK, "");
}

// ---- norm ----

int32_t check_norm_sizes(int32_t T, int32_t H, int32_t D) {
  if (T < 0) return invalid("T must be >= 0");
  if (H < 1 || D < 1) return invalid("H and D must be positive");
  if (D > 16384) return unsupported("D above 16384");
  if ((int64_t)T * H > (int64_t(1) << 40)) return unsupported("more than 2^40 rows");
  return GDR_OK;
}
int32_t check_norm(const gdr_norm *p, bool fwd) {
  if (!p) return invalid("problem is NULL");
  const int32_t rc = check_norm_sizes(p->T, p->H, p->D);
  if (rc) return rc;
  if (!is_dtype(p->dtype) || !is_dtype(p->res_dtype) || !is_dtype(p->w_dtype)) return invalid("unknown dtype");
  if (p->placement < GDR_RES_NONE || p->placement > GDR_RES_AFTER) return invalid("unknown placement");
  if (p->placement != GDR_RES_NONE && p->dtype == GDR_F32 && p->res_dtype == GDR_BF16)
    return unsupported("a bf16 residual with fp32 rows");
  if (p->gate ? p->activation != GDR_ACT_SILU && p->activation != GDR_ACT_SIGMOID : p->activation != GDR_ACT_NONE)
    return invalid("activation must be SiLU or sigmoid with a gate, none without");
  if (!(p->eps >= 0.f)) return invalid("eps must be >= 0");
  if (!(p->scale == p->scale)) return invalid("scale is NaN");
  const bool before = p->placement == GDR_RES_BEFORE;
  const int64_t width = (int64_t)p->H * p->D;
  const bool reads_x = fwd || !before;
  if (p->T > 0) {
    if (reads_x && !p->x) return invalid("x is NULL");
    if (fwd && p->placement != GDR_RES_NONE && !p->residual) return invalid("residual is NULL");
    if (before && !p->s) return invalid("s is NULL");
  }
  if (reads_x && !stride_ok(p->x_stride, width, p->T)) return invalid("x_stride below H * D");
  if (p->gate && !stride_ok(p->gate_stride, width, p->T)) return invalid("gate_stride below H * D");
  if (!element_aligned(p->x, p->dtype) || !element_aligned(p->gate, p->dtype) || !element_aligned(p->weight, p->w_dtype) ||
      !element_aligned(p->residual, p->res_dtype) || !element_aligned(p->s, p->res_dtype))
    return invalid("operands must be aligned to their elements");
  return GDR_OK;
}

int32_t norm_fwd(const gdr_norm *p, void *y, void *stream) {
  int32_t rc = check_norm(p, true);
  if (rc) return rc;
  if (p->T > 0 && !y) return invalid("y is NULL");
  if (!element_aligned(y, p->placement == GDR_RES_AFTER ? p->res_dtype : p->dtype)) return invalid("y must be aligned to its elements");
  const void *s = p->placement == GDR_RES_BEFORE ? p->s : nullptr;
  if (aliases({y}, {p->x, p->weight, p->gate, p->residual, s}) || aliases({s}, {p->x, p->weight, p->gate, p->residual}))
    return invalid("y or s is an input");
  if ((rc = gdr::host_check_device())) return rc;
  if ((rc = launch(gdr::TK_NORM_FWD, stream, "norm launch", [&](hipStream_t s) { return gdr::launch_norm_fwd(*p, y, s); })))
    return rc;
  return host_status(GDR_OK, "");
}

int32_t norm_bwd(const gdr_norm *p, const void *dy, const void *ds, void *dx, int64_t dx_stride, void *dgate,
                 int64_t dgate_stride, void *dres, float *dw, void *ws, int64_t ws_bytes, void *stream) {
  int32_t rc = check_norm(p, false);
  if (rc) return rc;
  const bool before = p->placement == GDR_RES_BEFORE;
  const int64_t width = (int64_t)p->H * p->D;
  if (!before && (ds || dres)) return invalid("ds and dres belong to GDR_RES_BEFORE");
  if (!p->gate && dgate) return invalid("dgate without a gate");
  if (p->T > 0) {
    if (!dy) return invalid("dy is NULL");
    if (!before && !dx) return invalid("dx is NULL");
    if (before && !dres) return invalid("dres is NULL");
    if (p->gate && !dgate) return invalid("dgate is NULL");
  }
  if (dx && !stride_ok(dx_stride, width, p->T)) return invalid("dx_stride below H * D");
  if (dgate && !stride_ok(dgate_stride, width, p->T)) return invalid("dgate_stride below H * D");
  const int32_t ydt = p->placement == GDR_RES_AFTER ? p->res_dtype : p->dtype;
  if (!element_aligned(dy, ydt) || !element_aligned(ds, p->res_dtype) || !element_aligned(dx, p->dtype) ||
      !element_aligned(dgate, p->dtype) || !element_aligned(dres, p->res_dtype) || !element_aligned(dw, GDR_F32))
    return invalid("gradients must be aligned to their elements");
  const void *u = before ? p->s : p->x;  // the normed row
  const int most = gdr::norm_workers((int64_t)p->T * p->H, p->D);
  if (dw && (rc = check_workspace(ws, ws_bytes, round_up((int64_t)most * p->D * 4)))) return rc;
  if (aliases({dx, dgate, dres, dw}, {u, p->weight, p->gate, dy, ds})) return invalid("dx, dgate, dres or dweight is an input");
  if ((rc = gdr::host_check_device())) return rc;
  const int workers = gdr::norm_bwd_workers(*p);
  // one worker's partial row is the gradient itself
  const bool one = workers == 1;
  float *partial = !dw ? nullptr : one ? dw : static_cast<float *>(ws);
  if ((rc = launch(gdr::TK_NORM_BWD, stream, "norm gradient launch", [&](hipStream_t s) {
         return gdr::launch_norm_bwd(*p, dy, ds, dx, dx_stride, dgate, dgate_stride, dres, partial, workers, s);
       })))
    return rc;
  if (dw && !one && (rc = launch(gdr::TK_PARAM_SUM, stream, "parameter sum launch",
                         [&](hipStream_t s) { return gdr::launch_norm_sum(partial, workers, p->D, dw, s); })))
    return rc;
  return host_status(GDR_OK, "");
}

}  // namespace

extern "C" {

int32_t gdr_conv_fwd(const gdr_conv *p, void *y, int64_t y_stride, void *st, void *stream) {
  return conv_fwd(p, y, y_stride, st, stream);
}
int64_t gdr_conv_workspace_bytes(int32_t n_chunks, int32_t C, int32_t W, int32_t dtype) {
  if (n_chunks < 0 || C < 1 || !is_dtype(dtype)) return -(int64_t)invalid("n_chunks must be >= 0, C positive and dtype known");
  if (W < 2 || W > 8) return -(int64_t)unsupported("W outside 2..8");
  if (C > (1 << 24)) return -(int64_t)unsupported("C above 2^24");
  if (!conv_sum_fits(C, W)) return -(int64_t)unsupported(kTooMany);
  return conv_bytes(n_chunks, C, W);
}
int32_t gdr_conv_bwd(const gdr_conv *p, const void *dy, int64_t dy_stride, const void *dst, void *dx, int64_t dx_stride,
                     float *dweight, float *dbias, void *ds0, void *workspace, int64_t workspace_bytes, void *stream) {
  return conv_bwd(p, dy, dy_stride, dst, dx, dx_stride, dweight, dbias, ds0, workspace, workspace_bytes, stream);
}
int32_t gdr_conv_step(const gdr_conv *p, void *y, int64_t y_stride, void *state, const int32_t *slots, int32_t n_slots,
                      void *stream) {
  return conv_step(p, y, y_stride, state, slots, n_slots, stream);
}

int32_t gdr_gate_fwd(const gdr_gate *p, float *g, void *stream) { return gate_fwd(p, g, stream); }
int64_t gdr_gate_workspace_bytes(int32_t T, int32_t H, int32_t D, int32_t dtype) {
  const int32_t rc = check_gate_sizes(T, H, D, dtype);
  if (rc) return -(int64_t)rc;
  return gate_bytes(T, H * D, D);
}
int32_t gdr_gate_bwd(const gdr_gate *p, const float *dg, void *dx, int64_t dx_stride, float *da_log, float *dbias,
                     void *workspace, int64_t workspace_bytes, void *stream) {
  return gate_bwd(p, dg, dx, dx_stride, da_log, dbias, workspace, workspace_bytes, stream);
}

int32_t gdr_kda_step(const gdr_step *p, uint16_t *o, void *stream) { return step(false, p, o, stream); }
int32_t gdr_gdn_step(const gdr_step *p, uint16_t *o, void *stream) { return step(true, p, o, stream); }

int32_t gdr_norm_fwd(const gdr_norm *p, void *y, void *stream) { return norm_fwd(p, y, stream); }
int64_t gdr_norm_workspace_bytes(int32_t T, int32_t H, int32_t D) {
  const int32_t rc = check_norm_sizes(T, H, D);
  if (rc) return -(int64_t)rc;
  return round_up((int64_t)gdr::norm_workers((int64_t)T * H, D) * D * 4);
}
int32_t gdr_norm_bwd(const gdr_norm *p, const void *dy, const void *ds, void *dx, int64_t dx_stride, void *dgate,
                     int64_t dgate_stride, void *dres, float *dweight, void *workspace, int64_t workspace_bytes,
                     void *stream) {
  return norm_bwd(p, dy, ds, dx, dx_stride, dgate, dgate_stride, dres, dweight, workspace, workspace_bytes, stream);
}

}  // extern "C"
