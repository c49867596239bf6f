// C-ABI front end of the gated linear recurrence (include/ssm_scan.h). As in
// api.cpp, every check is host arithmetic on the parameter struct and precedes
// the first HIP call. The launches live in glr_fwd.hip, glr_chain.hip,
// glr_pieces.hip and glr_bwd.hip.
#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "kernels.h"
#include "kernels_glr.h"
#include "ssm_scan.h"

namespace {

using ssm::check_overlaps;
using ssm::check_pointers;
using ssm::dtype_size;
using ssm::fail;
using ssm::kLim;
using ssm::mul_ok;
using ssm::Need;
using ssm::ok;
using ssm::Range;
using ssm::range;
using ssm::span;
using ssm::valid_dtype;

constexpr int64_t kMaxLen = int64_t{1} << 27;
constexpr int64_t kMaxDim = int64_t{1} << 24;

struct GlrSizes {
  int64_t tokens, dense, state;  // B L, B L D, B D
  int64_t us, ds, is, zs;        // token strides
  int64_t u, d, i, z;            // elements spanned
  bool empty() const { return dense == 0; }
};

// Sizes, types and kinds common to the sequence and the decode window.
template <typename P>
ssm_status check_glr_sizes(const P* p, int64_t len, GlrSizes* s) {
  if (p->batch < 0 || len < 0 || p->dim < 0)
    return fail(SSM_ERR_BAD_SHAPE, "batch, length and dim must be >= 0 (got %lld, %lld, %lld)", (long long)p->batch,
                (long long)len, (long long)p->dim);
  if (len >= kMaxLen) return fail(SSM_ERR_BAD_SHAPE, "the length must be below 2^27 (got %lld)", (long long)len);
  if (p->dim > kMaxDim) return fail(SSM_ERR_BAD_SHAPE, "dim must be at most 2^24 (got %lld)", (long long)p->dim);
  if (!valid_dtype(p->in_dtype) || !valid_dtype(p->out_dtype))
    return fail(SSM_ERR_BAD_DTYPE, "in_dtype/out_dtype must be SSM_F32 or SSM_BF16");
  if (p->decay != SSM_GLR_SIGMOID && p->decay != SSM_GLR_SOFTPLUS)
    return fail(SSM_ERR_UNSUPPORTED, "unknown decay %d", p->decay);
  if (p->mix != SSM_GLR_UNIT && p->mix != SSM_GLR_REST && p->mix != SSM_GLR_ONE)
    return fail(SSM_ERR_UNSUPPORTED, "unknown mix %d", p->mix);
  const int64_t strides[] = {p->u_stride, p->dt_stride, p->in_stride, p->z_stride};
  int64_t* steps[] = {&s->us, &s->ds, &s->is, &s->zs};
  int64_t* spans[] = {&s->u, &s->d, &s->i, &s->z};
  if (!mul_ok(p->batch, len, &s->tokens) || !mul_ok(s->tokens, p->dim, &s->dense) ||
      !mul_ok(p->batch, p->dim, &s->state) || s->dense > kLim || s->state > kLim)
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows");
  for (int j = 0; j < 4; ++j) {
    if (strides[j] != 0 && strides[j] < p->dim)
      return fail(SSM_ERR_BAD_SHAPE, "a token stride is smaller than the token");
    if (strides[j] > ssm::kGlrMaxStride)
      return fail(SSM_ERR_BAD_SHAPE, "a token stride is above 2^24 (got %lld)", (long long)strides[j]);
    *steps[j] = strides[j] ? strides[j] : p->dim;
    if (!span(s->tokens, *steps[j], p->dim, spans[j]) || *spans[j] > kLim)
      return fail(SSM_ERR_BAD_SHAPE, "element count overflows");
  }
  return SSM_OK;
}

ssm_status no_grid() { return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows"); }

// How the forward runs: step by step (no pieces), as one walk or in pieces.
ssm_status plan_fwd(const ssm_glr_params* p, const GlrSizes& s, ssm::GlrPieces* pieces) {
  *pieces = ssm::GlrPieces{};
  if (s.empty()) return SSM_OK;
  if (ssm::glr_by_steps(p->seqlen)) return ssm::glr_steps_fit(p->batch, p->dim) ? SSM_OK : no_grid();
  *pieces = ssm::plan_glr(p->batch, p->seqlen, p->dim);
  return ssm::glr_grids_fit(p->batch, p->dim, *pieces) ? SSM_OK : no_grid();
}

ssm_status plan_bwd(const ssm_glr_params* p, GlrSizes* s, ssm::GlrPieces* pieces) {
  const ssm_status st = check_glr_sizes(p, p->seqlen, s);
  if (st != SSM_OK) return st;
  *pieces = ssm::GlrPieces{};
  if (s->empty()) return SSM_OK;
  *pieces = ssm::plan_glr_bwd(p->batch, p->seqlen, p->dim);
  return ssm::glr_grids_fit(p->batch, p->dim, *pieces) ? SSM_OK : no_grid();
}

template <typename P>
ssm::GlrPlan glr_plan(const P* p, int64_t len, const GlrSizes& s) {
  ssm::GlrPlan g{};
  g.B = p->batch;
  g.L = len;
  g.D = p->dim;
  g.in_bf16 = p->in_dtype == SSM_BF16;
  g.out_bf16 = p->out_dtype == SSM_BF16;
  g.decay = p->decay;
  g.mix = p->mix;
  g.u = p->u;
  g.dt = p->dt_raw;
  g.in = p->in_raw;
  g.z = p->z;
  g.us = s.us;
  g.ds = s.ds;
  g.is = s.is;
  g.zs = s.zs;
  g.A = p->A;
  g.dt_bias = p->dt_bias;
  g.in_bias = p->in_bias;
  return g;
}

// A bias without what it belongs to (an empty tensor's address may be NULL).
template <typename P>
ssm_status check_in_bias(const P* p, const GlrSizes& s) {
  if (p->in_bias && !p->in_raw && !s.empty()) return fail(SSM_ERR_NULL_POINTER, "in_raw is NULL, but in_bias is given");
  return SSM_OK;
}

// A gradient that has no input.
ssm_status check_gradients(const ssm_glr_params* p, const GlrSizes& s) {
  if (s.empty()) return SSM_OK;
  if (p->din_raw && !p->in_raw) return fail(SSM_ERR_NULL_POINTER, "in_raw is NULL, but din_raw is given");
  if (p->dz && !p->z) return fail(SSM_ERR_NULL_POINTER, "z is NULL, but dz is given");
  return SSM_OK;
}

ssm_status check_workspace(const void* workspace, size_t given, size_t needed) {
  if (needed > 0 && (!workspace || given < needed))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", needed,
                workspace ? given : static_cast<size_t>(0));
  return SSM_OK;
}

ssm_status enqueued(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

ssm_status ssm_glr_workspace_size(const ssm_glr_params* p, size_t* bytes) {
  if (!p || !bytes) return fail(SSM_ERR_NULL_POINTER, "params or bytes is NULL");
  GlrSizes s;
  ssm_status st = check_glr_sizes(p, p->seqlen, &s);
  ssm::GlrPieces pieces;
  if (st != SSM_OK || (st = plan_fwd(p, s, &pieces)) != SSM_OK) return st;
  *bytes = pieces.bytes;
  return ok();
}

ssm_status ssm_glr_fwd(const ssm_glr_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  GlrSizes s;
  ssm_status st = check_glr_sizes(p, p->seqlen, &s);
  ssm::GlrPieces pieces;
  if (st != SSM_OK || (st = plan_fwd(p, s, &pieces)) != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype);
  const Need needs[] = {
      {p->u, s.dense, si, "u", true},        {p->dt_raw, s.dense, si, "dt_raw", true},
      {p->A, s.dense, 4, "A", true},         {p->out, s.dense, so, "out", true},
      {p->in_raw, 0, si, "in_raw", false},   {p->z, 0, si, "z", false},
      {p->dt_bias, 0, 4, "dt_bias", false},  {p->in_bias, 0, 4, "in_bias", false},
      {p->h0, 0, 4, "h0", false},            {p->h_last, 0, 4, "h_last", false},
      {p->workspace, 0, 256, "workspace", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK || (st = check_in_bias(p, s)) != SSM_OK ||
      (st = check_workspace(p->workspace, p->workspace_bytes, pieces.bytes)) != SSM_OK)
    return st;
  const Range in[] = {
      range(p->u, s.u, si, "u"), range(p->dt_raw, s.d, si, "dt_raw"), range(p->in_raw, s.i, si, "in_raw"),
      range(p->z, s.z, si, "z"), range(p->A, p->dim, 4, "A"), range(p->dt_bias, p->dim, 4, "dt_bias"),
      range(p->in_bias, p->dim, 4, "in_bias"), range(p->reset, s.tokens, 1, "reset"), range(p->h0, s.state, 4, "h0"),
  };
  const Range out[] = {
      range(p->out, s.dense, so, "out"), range(p->h_last, s.state, 4, "h_last"),
      Range{pieces.bytes ? static_cast<const char*>(p->workspace) : nullptr, pieces.bytes, "workspace"},
  };
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_glr_fwd: B %lld L %lld D %lld, %s in, %s out, decay %d, mix %d, input gate %d, gate %d, resets %d; %lld "
          "pieces, workspace %zu bytes",
          (long long)p->batch, (long long)p->seqlen, (long long)p->dim, si == 2 ? "bf16" : "f32",
          so == 2 ? "bf16" : "f32", p->decay, p->mix, p->in_raw != nullptr, p->z != nullptr, p->reset != nullptr,
          (long long)pieces.pieces, pieces.bytes);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (s.empty())  // the state passes through an empty sequence
    return enqueued(ssm::launch_fill(p->h_last, p->h0, 0.0f, 0.0f, s.state, stream), "fill");
  ssm::GlrPlan plan = glr_plan(p, p->seqlen, s);
  plan.reset = p->reset;
  plan.h0 = p->h0;
  plan.out = p->out;
  plan.h_last = p->h_last;
  return enqueued(pieces.pieces > 0 ? ssm::launch_glr(plan, pieces, p->workspace, stream)
                                    : ssm::launch_glr_steps(plan, stream),
                  "gated recurrence");
}

ssm_status ssm_glr_update(const ssm_glr_update_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  GlrSizes s;
  ssm_status st = check_glr_sizes(p, p->tokens, &s);
  if (st != SSM_OK) return st;
  if (!s.empty() && !ssm::glr_steps_fit(p->batch, p->dim)) return no_grid();
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype);
  const Need needs[] = {
      {p->h, s.dense, 4, "h", true},         {p->u, s.dense, si, "u", true},
      {p->dt_raw, s.dense, si, "dt_raw", true}, {p->A, s.dense, 4, "A", true},
      {p->out, s.dense, so, "out", true},    {p->in_raw, 0, si, "in_raw", false},
      {p->z, 0, si, "z", false},             {p->dt_bias, 0, 4, "dt_bias", false},
      {p->in_bias, 0, 4, "in_bias", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK || (st = check_in_bias(p, s)) != SSM_OK) return st;
  const Range in[] = {
      range(p->u, s.u, si, "u"), range(p->dt_raw, s.d, si, "dt_raw"), range(p->in_raw, s.i, si, "in_raw"),
      range(p->z, s.z, si, "z"), range(p->A, p->dim, 4, "A"), range(p->dt_bias, p->dim, 4, "dt_bias"),
      range(p->in_bias, p->dim, 4, "in_bias"),
  };
  const Range out[] = {range(p->out, s.dense, so, "out"), range(p->h, s.state, 4, "h")};
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_glr_update: B %lld T %lld D %lld, %s in", (long long)p->batch, (long long)p->tokens, (long long)p->dim,
          si == 2 ? "bf16" : "f32");
  if (s.empty()) return ok();
  ssm::GlrPlan plan = glr_plan(p, p->tokens, s);
  plan.h0 = p->h;
  plan.h_last = p->h;
  plan.out = p->out;
  return enqueued(ssm::launch_glr_steps(plan, static_cast<hipStream_t>(hip_stream)), "gated recurrence window");
}

ssm_status ssm_glr_bwd_workspace_size(const ssm_glr_params* p, size_t* bytes) {
  if (!p || !bytes) return fail(SSM_ERR_NULL_POINTER, "params or bytes is NULL");
  GlrSizes s;
  ssm::GlrPieces pieces;
  const ssm_status st = plan_bwd(p, &s, &pieces);
  if (st != SSM_OK) return st;
  *bytes = pieces.bytes;
  return ok();
}

ssm_status ssm_glr_bwd(const ssm_glr_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  GlrSizes s;
  ssm::GlrPieces pieces;
  ssm_status st = plan_bwd(p, &s, &pieces);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype);
  const Need needs[] = {
      {p->u, s.dense, si, "u", true},          {p->dt_raw, s.dense, si, "dt_raw", true},
      {p->A, s.dense, 4, "A", true},           {p->dout, s.dense, si, "dout", true},
      {p->du, s.dense, so, "du", true},        {p->d_dt_raw, s.dense, so, "d_dt_raw", true},
      {p->din_raw, s.dense, so, "din_raw", p->in_raw != nullptr}, {p->dz, s.dense, so, "dz", p->z != nullptr},
      {p->dA, p->dim, 4, "dA", true},          {p->in_raw, 0, si, "in_raw", false},
      {p->z, 0, si, "z", false},               {p->dt_bias, 0, 4, "dt_bias", false},
      {p->in_bias, 0, 4, "in_bias", false},    {p->h0, 0, 4, "h0", false},
      {p->dh_last, 0, 4, "dh_last", false},    {p->d_dt_bias, 0, 4, "d_dt_bias", false},
      {p->din_bias, 0, 4, "din_bias", false},  {p->dh0, 0, 4, "dh0", false},
      {p->workspace, 0, 256, "workspace", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK || (st = check_in_bias(p, s)) != SSM_OK ||
      (st = check_gradients(p, s)) != SSM_OK ||
      (st = check_workspace(p->workspace, p->workspace_bytes, pieces.bytes)) != SSM_OK)
    return st;
  const Range in[] = {
      range(p->u, s.u, si, "u"), range(p->dt_raw, s.d, si, "dt_raw"), range(p->in_raw, s.i, si, "in_raw"),
      range(p->z, s.z, si, "z"), range(p->A, p->dim, 4, "A"), range(p->dt_bias, p->dim, 4, "dt_bias"),
      range(p->in_bias, p->dim, 4, "in_bias"), range(p->reset, s.tokens, 1, "reset"), range(p->h0, s.state, 4, "h0"),
      range(p->dout, s.dense, si, "dout"), range(p->dh_last, s.state, 4, "dh_last"),
  };
  const Range out[] = {
      range(p->du, s.dense, so, "du"), range(p->d_dt_raw, s.dense, so, "d_dt_raw"),
      range(p->din_raw, s.dense, so, "din_raw"), range(p->dz, s.dense, so, "dz"), range(p->dA, p->dim, 4, "dA"),
      range(p->d_dt_bias, p->dim, 4, "d_dt_bias"), range(p->din_bias, p->dim, 4, "din_bias"),
      range(p->dh0, s.state, 4, "dh0"),
      Range{pieces.bytes ? static_cast<const char*>(p->workspace) : nullptr, pieces.bytes, "workspace"},
  };
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_glr_bwd: B %lld L %lld D %lld, %s in, %s gradients; %lld pieces, workspace %zu bytes",
          (long long)p->batch, (long long)p->seqlen, (long long)p->dim, si == 2 ? "bf16" : "f32",
          so == 2 ? "bf16" : "f32", (long long)pieces.pieces, pieces.bytes);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (s.empty()) {  // no token: sums over nothing, and the adjoint passes through
    hipError_t e = ssm::launch_fill(p->dA, nullptr, 0.0f, 0.0f, p->dim, stream);
    if (e == hipSuccess) e = ssm::launch_fill(p->d_dt_bias, nullptr, 0.0f, 0.0f, p->dim, stream);
    if (e == hipSuccess) e = ssm::launch_fill(p->din_bias, nullptr, 0.0f, 0.0f, p->dim, stream);
    if (e == hipSuccess) e = ssm::launch_fill(p->dh0, p->dh_last, 0.0f, 0.0f, s.state, stream);
    return enqueued(e, "fill");
  }
  ssm::GlrPlan plan = glr_plan(p, p->seqlen, s);
  plan.reset = p->reset;
  plan.h0 = p->h0;
  plan.dout = p->dout;
  plan.dh_last = p->dh_last;
  plan.du = p->du;
  plan.d_dt = p->d_dt_raw;
  plan.d_in = p->din_raw;
  plan.dz = p->dz;
  plan.dA = p->dA;
  plan.d_dt_bias = p->d_dt_bias;
  plan.din_bias = p->din_bias;
  plan.dh0 = p->dh0;
  return enqueued(ssm::launch_glr_bwd(plan, pieces, p->workspace, stream), "gated recurrence backward");
}

}  // extern "C"
