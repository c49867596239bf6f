// C-ABI front end of the norms around a block (include/ssm_scan.h). As in
// api.cpp, every check is host arithmetic on the parameter struct and precedes
// the first HIP call. The launches live in gated_norm.hip, block_norm.hip and
// row_sums.hip.
#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "kernels.h"
#include "kernels_block.h"
#include "ssm_scan.h"

static_assert(SSM_MAX_NORM_DIM == ssm::kMaxRow, "the longest row is the kernels'");

namespace {

using ssm::check_overlaps;
using ssm::check_pointers;
using ssm::dtype_size;
using ssm::fail;
using ssm::fits_launch;
using ssm::kLim;
using ssm::mul_ok;
using ssm::Need;
using ssm::ok;
using ssm::Range;
using ssm::range;
using ssm::span;
using ssm::valid_dtype;

constexpr int64_t kMaxLen = int64_t{1} << 27;
constexpr int64_t kMaxHeads = 65536;

ssm_status check_flag(int32_t v, const char* name) {
  if (v != 0 && v != 1) return fail(SSM_ERR_UNSUPPORTED, "%s must be 0 or 1 (got %d)", name, v);
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

struct GatedSizes {
  int64_t tokens, dense, xs, zs, x, z, w;
  bool empty() const { return dense == 0; }
};

ssm_status check_gated(const ssm_gated_norm_params* p, GatedSizes* s) {
  if (p->batch < 0 || p->seqlen < 0 || p->heads < 0) return fail(SSM_ERR_BAD_SHAPE, "sizes must be >= 0");
  if (p->seqlen >= kMaxLen) return fail(SSM_ERR_BAD_SHAPE, "seqlen must be below 2^27 (got %lld)", (long long)p->seqlen);
  if (p->heads > kMaxHeads) return fail(SSM_ERR_BAD_SHAPE, "at most %lld heads", (long long)kMaxHeads);
  if (p->head_dim < 1 || p->head_dim > SSM_MAX_NORM_DIM)
    return fail(SSM_ERR_BAD_SHAPE, "head_dim must be in [1, %d] (got %lld)", SSM_MAX_NORM_DIM, (long long)p->head_dim);
  if (!valid_dtype(p->in_dtype) || !valid_dtype(p->out_dtype))
    return fail(SSM_ERR_BAD_DTYPE, "in_dtype/out_dtype must be SSM_F32 or SSM_BF16");
  ssm_status st = check_flag(p->gate_first, "gate_first");
  if (st != SSM_OK || (st = check_flag(p->w_per_head, "w_per_head")) != SSM_OK) return st;
  const int64_t token = p->heads * p->head_dim;
  if (p->x_stride < 0 || p->z_stride < 0 || (p->x_stride && p->x_stride < token) || (p->z_stride && p->z_stride < token))
    return fail(SSM_ERR_BAD_SHAPE, "a token stride is smaller than the token");
  s->xs = p->x_stride ? p->x_stride : token;
  s->zs = p->z_stride ? p->z_stride : token;
  s->w = p->w_per_head ? token : p->head_dim;
  if (!mul_ok(p->batch, p->seqlen, &s->tokens) || !mul_ok(s->tokens, token, &s->dense) || s->dense > kLim ||
      !span(s->tokens, s->xs, token, &s->x) || !span(s->tokens, s->zs, token, &s->z) || s->x > kLim || s->z > kLim)
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows");
  return SSM_OK;
}

ssm::GatedPlan gated_plan(const ssm_gated_norm_params* p, const GatedSizes& s) {
  ssm::GatedPlan g{};
  g.tokens = s.tokens;
  g.H = static_cast<int>(p->heads);
  g.d = static_cast<int>(p->head_dim);
  g.in_bf16 = p->in_dtype == SSM_BF16;
  g.out_bf16 = p->out_dtype == SSM_BF16;
  g.gate_first = p->gate_first;
  g.w_per_head = p->w_per_head;
  g.x = p->x;
  g.z = p->z;
  g.xs = s.xs;
  g.zs = s.zs;
  g.w = p->w;
  g.eps = p->eps;
  return g;
}

// The sums over the workgroups' rows: a workgroup of 1024 threads for 32 elements of each weight.
ssm_status check_gated_bwd(const ssm_gated_norm_params* p, GatedSizes* s) {
  const ssm_status st = check_gated(p, s);
  if (st != SSM_OK || !p->w_per_head || s->empty() || fits_launch(p->heads * ((p->head_dim + 31) / 32), 1024)) return st;
  return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
}

size_t gated_bytes(const ssm_gated_norm_params* p, const GatedSizes& s) {
  if (s.empty()) return 0;
  return static_cast<size_t>(ssm::gated_norm_bwd_blocks(s.tokens, static_cast<int>(p->heads),
                                                        static_cast<int>(p->head_dim), p->w_per_head)) *
         static_cast<size_t>(p->head_dim) * sizeof(float);
}

struct BlockSizes {
  int64_t tokens, dense, ys, y, gate;
  bool empty() const { return dense == 0; }
};

ssm_status check_block(const ssm_block_norm_params* p, BlockSizes* s) {
  if (p->batch < 0 || p->seqlen < 0) return fail(SSM_ERR_BAD_SHAPE, "sizes must be >= 0");
  if (p->seqlen >= kMaxLen) return fail(SSM_ERR_BAD_SHAPE, "seqlen must be below 2^27 (got %lld)", (long long)p->seqlen);
  if (p->dim < 1 || p->dim > SSM_MAX_NORM_DIM)
    return fail(SSM_ERR_BAD_SHAPE, "dim must be in [1, %d] (got %lld)", SSM_MAX_NORM_DIM, (long long)p->dim);
  if (!valid_dtype(p->in_dtype) || !valid_dtype(p->out_dtype) || !valid_dtype(p->res_dtype))
    return fail(SSM_ERR_BAD_DTYPE, "in_dtype/out_dtype/res_dtype must be SSM_F32 or SSM_BF16");
  ssm_status st = check_flag(p->post, "post");
  if (st != SSM_OK || (st = check_flag(p->gate_rows, "gate_rows")) != SSM_OK) return st;
  if (p->y_stride < 0 || (p->y_stride && p->y_stride < p->dim))
    return fail(SSM_ERR_BAD_SHAPE, "a token stride is smaller than the token");
  s->ys = p->y_stride ? p->y_stride : p->dim;
  if (!mul_ok(p->batch, p->seqlen, &s->tokens) || !mul_ok(s->tokens, p->dim, &s->dense) || s->dense > kLim ||
      !span(s->tokens, s->ys, p->dim, &s->y) || s->y > kLim || !mul_ok(p->batch, p->dim, &s->gate) || s->gate > kLim)
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows");
  if (!p->gate_rows) s->gate = p->dim;
  // a gate for each sequence: a workgroup of up to 1024 threads at least for each
  if (p->gate_rows && !s->empty() && !fits_launch(p->batch, 1024))
    return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
  return SSM_OK;
}

// dgate's sums over the workgroups' rows: a workgroup of 1024 threads for 32 of its elements.
ssm_status check_block_bwd(const ssm_block_norm_params* p, BlockSizes* s) {
  const ssm_status st = check_block(p, s);
  if (st != SSM_OK || !p->gate_rows || s->empty() || fits_launch(p->batch * ((p->dim + 31) / 32), 1024)) return st;
  return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
}

// Weights and gradients that belong to an option which is off.
ssm_status check_options(const ssm_block_norm_params* p, const BlockSizes& s) {
  if (p->w_post && !p->post) return fail(SSM_ERR_UNSUPPORTED, "w_post is given, but post is 0");
  if (p->dw_post && !p->post) return fail(SSM_ERR_UNSUPPORTED, "dw_post is given, but post is 0");
  if (s.empty()) return SSM_OK;  // (an empty tensor's address may be NULL)
  if (p->gate_rows && !p->gate) return fail(SSM_ERR_NULL_POINTER, "gate is NULL, but gate_rows is 1");
  if (p->dgate && !p->gate) return fail(SSM_ERR_NULL_POINTER, "gate is NULL, but dgate is given");
  if (p->dx && !p->x) return fail(SSM_ERR_NULL_POINTER, "x is NULL, but dx is given");
  return SSM_OK;
}

ssm::BlockPlan block_plan(const ssm_block_norm_params* p, const BlockSizes& s) {
  ssm::BlockPlan b{};
  b.B = p->batch;
  b.L = p->seqlen;
  b.D = static_cast<int>(p->dim);
  b.in_bf16 = p->in_dtype == SSM_BF16;
  b.out_bf16 = p->out_dtype == SSM_BF16;
  b.res_bf16 = p->res_dtype == SSM_BF16;
  b.post = p->post;
  b.gate_rows = p->gate_rows;
  b.y = p->y;
  b.ys = s.ys;
  b.x = p->x;
  b.w = p->w;
  b.w_post = p->w_post;
  b.gate = p->gate;
  b.eps = p->eps;
  b.scale = p->scale;
  return b;
}

size_t block_bytes(const ssm_block_norm_params* p, const BlockSizes& s) {
  if (s.empty()) return 0;
  return static_cast<size_t>(
             ssm::block_norm_bwd_blocks(p->batch, p->seqlen, static_cast<int>(p->dim), p->gate_rows)) *
         3 * static_cast<size_t>(p->dim) * sizeof(float);
}

}  // namespace

extern "C" {

ssm_status ssm_gated_norm_fwd(const ssm_gated_norm_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  GatedSizes s;
  ssm_status st = check_gated(p, &s);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype);
  const Need needs[] = {
      {p->x, s.dense, si, "x", true},     {p->z, s.dense, si, "z", true},
      {p->out, s.dense, so, "out", true}, {p->w, 0, 4, "w", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK) return st;
  const Range in[] = {range(p->x, s.x, si, "x"), range(p->z, s.z, si, "z"), range(p->w, s.w, 4, "w")};
  const Range out[] = {range(p->out, s.dense, so, "out")};
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_gated_norm_fwd: %lld tokens, %lld heads of %lld, gate first %d", (long long)s.tokens,
          (long long)p->heads, (long long)p->head_dim, p->gate_first);
  if (s.empty()) return ok();
  ssm::GatedPlan plan = gated_plan(p, s);
  plan.out = p->out;
  return enqueued(ssm::launch_gated_norm(plan, static_cast<hipStream_t>(hip_stream)), "gated norm");
}

ssm_status ssm_gated_norm_bwd_workspace_size(const ssm_gated_norm_params* p, size_t* bytes) {
  if (!p || !bytes) return fail(SSM_ERR_NULL_POINTER, "params or bytes is NULL");
  GatedSizes s;
  const ssm_status st = check_gated_bwd(p, &s);
  if (st != SSM_OK) return st;
  *bytes = gated_bytes(p, s);
  return ok();
}

ssm_status ssm_gated_norm_bwd(const ssm_gated_norm_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  GatedSizes s;
  ssm_status st = check_gated_bwd(p, &s);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype), ws = gated_bytes(p, s);
  const Need needs[] = {
      {p->x, s.dense, si, "x", true},   {p->z, s.dense, si, "z", true},   {p->dout, s.dense, si, "dout", true},
      {p->dx, s.dense, so, "dx", true}, {p->dz, s.dense, so, "dz", true}, {p->w, 0, 4, "w", false},
      {p->dw, 0, 4, "dw", false},       {p->workspace, 0, 16, "workspace", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK ||
      (st = check_workspace(p->workspace, p->workspace_bytes, ws)) != SSM_OK)
    return st;
  const Range in[] = {range(p->x, s.x, si, "x"), range(p->z, s.z, si, "z"), range(p->w, s.w, 4, "w"),
                      range(p->dout, s.dense, si, "dout")};
  const Range out[] = {
      range(p->dx, s.dense, so, "dx"), range(p->dz, s.dense, so, "dz"), range(p->dw, s.w, 4, "dw"),
      Range{ws ? static_cast<const char*>(p->workspace) : nullptr, ws, "workspace"},
  };
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_gated_norm_bwd: %lld tokens, %lld heads of %lld, gate first %d, workspace %zu bytes",
          (long long)s.tokens, (long long)p->heads, (long long)p->head_dim, p->gate_first, ws);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (s.empty()) return enqueued(ssm::launch_fill(p->dw, nullptr, 0.0f, 0.0f, s.w, stream), "fill");  // no row
  ssm::GatedPlan plan = gated_plan(p, s);
  plan.dout = p->dout;
  plan.dx = p->dx;
  plan.dz = p->dz;
  plan.dw = p->dw;
  return enqueued(ssm::launch_gated_norm_bwd(plan, static_cast<float*>(p->workspace), stream), "gated norm backward");
}

ssm_status ssm_block_norm_fwd(const ssm_block_norm_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  BlockSizes s;
  ssm_status st = check_block(p, &s);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype), sr = dtype_size(p->res_dtype);
  const Need needs[] = {
      {p->y, s.dense, si, "y", true},      {p->out, s.dense, so, "out", true}, {p->x, 0, sr, "x", false},
      {p->x_out, 0, sr, "x_out", false},   {p->w, 0, 4, "w", false},           {p->w_post, 0, 4, "w_post", false},
      {p->gate, 0, 4, "gate", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK || (st = check_options(p, s)) != SSM_OK) return st;
  const Range in[] = {range(p->y, s.y, si, "y"), range(p->x, s.dense, sr, "x"), range(p->w, p->dim, 4, "w"),
                      range(p->w_post, p->dim, 4, "w_post"), range(p->gate, s.gate, 4, "gate")};
  const Range out[] = {range(p->out, s.dense, so, "out"), range(p->x_out, s.dense, sr, "x_out")};
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_block_norm_fwd: %lld tokens of %lld, post %d, gate %d", (long long)s.tokens, (long long)p->dim, p->post,
          p->gate ? 1 + p->gate_rows : 0);
  if (s.empty()) return ok();
  ssm::BlockPlan plan = block_plan(p, s);
  plan.out = p->out;
  plan.x_out = p->x_out;
  return enqueued(ssm::launch_block_norm(plan, static_cast<hipStream_t>(hip_stream)), "block norm");
}

ssm_status ssm_block_norm_bwd_workspace_size(const ssm_block_norm_params* p, size_t* bytes) {
  if (!p || !bytes) return fail(SSM_ERR_NULL_POINTER, "params or bytes is NULL");
  BlockSizes s;
  const ssm_status st = check_block_bwd(p, &s);
  if (st != SSM_OK) return st;
  *bytes = block_bytes(p, s);
  return ok();
}

ssm_status ssm_block_norm_bwd(const ssm_block_norm_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  BlockSizes s;
  ssm_status st = check_block_bwd(p, &s);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype), sr = dtype_size(p->res_dtype);
  const size_t ws = block_bytes(p, s);
  const Need needs[] = {
      {p->y, s.dense, si, "y", true},        {p->dout, s.dense, si, "dout", true},
      {p->dy, s.dense, so, "dy", true},      {p->x, 0, sr, "x", false},
      {p->dx_out, 0, sr, "dx_out", false},   {p->dx, 0, sr, "dx", false},
      {p->w, 0, 4, "w", false},              {p->w_post, 0, 4, "w_post", false},
      {p->gate, 0, 4, "gate", false},        {p->dw, 0, 4, "dw", false},
      {p->dw_post, 0, 4, "dw_post", false},  {p->dgate, 0, 4, "dgate", false},
      {p->workspace, 0, 16, "workspace", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK || (st = check_options(p, s)) != SSM_OK ||
      (st = check_workspace(p->workspace, p->workspace_bytes, ws)) != SSM_OK)
    return st;
  const Range in[] = {range(p->y, s.y, si, "y"), range(p->x, s.dense, sr, "x"), range(p->w, p->dim, 4, "w"),
                      range(p->w_post, p->dim, 4, "w_post"), range(p->gate, s.gate, 4, "gate"),
                      range(p->dout, s.dense, si, "dout"), range(p->dx_out, s.dense, sr, "dx_out")};
  const Range out[] = {
      range(p->dy, s.dense, so, "dy"), range(p->dx, s.dense, sr, "dx"), range(p->dw, p->dim, 4, "dw"),
      range(p->dw_post, p->dim, 4, "dw_post"), range(p->dgate, s.gate, 4, "dgate"),
      Range{ws ? static_cast<const char*>(p->workspace) : nullptr, ws, "workspace"},
  };
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_block_norm_bwd: %lld tokens of %lld, post %d, gate %d, workspace %zu bytes", (long long)s.tokens,
          (long long)p->dim, p->post, p->gate ? 1 + p->gate_rows : 0, ws);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (s.empty()) {  // sums over no row
    hipError_t e = ssm::launch_fill(p->dw, nullptr, 0.0f, 0.0f, p->dim, stream);
    if (e == hipSuccess) e = ssm::launch_fill(p->dw_post, nullptr, 0.0f, 0.0f, p->dim, stream);
    if (e == hipSuccess) e = ssm::launch_fill(p->dgate, nullptr, 0.0f, 0.0f, s.gate, stream);
    return enqueued(e, "fill");
  }
  ssm::BlockPlan plan = block_plan(p, s);
  plan.dout = p->dout;
  plan.dx_out = p->dx_out;
  plan.dy = p->dy;
  plan.dx = p->dx;
  plan.dw = p->dw;
  plan.dw_post = p->dw_post;
  plan.dgate = p->dgate;
  return enqueued(ssm::launch_block_norm_bwd(plan, static_cast<float*>(p->workspace), stream), "block norm backward");
}

}  // extern "C"
