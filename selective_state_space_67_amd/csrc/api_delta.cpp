// C-ABI front end of the gated delta rule and of the head norms
// (include/ssm_scan.h). As in api.cpp, every check is host arithmetic on the
// parameter struct and precedes the first HIP call. The launches live in
// delta_step.hip, delta_chunk.hip, delta_chunk_bwd.hip and qk_norm.hip.
#include <hip/hip_runtime.h>

#include <limits>

#include "api_checks.h"
#include "kernels.h"
#include "kernels_delta.h"
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
using ssm::overlaps;
using ssm::Range;
using ssm::range;
using ssm::span;
using ssm::valid_dtype;

constexpr int64_t kMaxLen = int64_t{1} << 27;
constexpr int64_t kMaxHeads = 65536;
constexpr int64_t kMaxColumns = 65536;

struct DeltaSizes {
  int64_t tokens;              // B L
  int64_t q, k, v;             // elements spanned by q, k, v
  int64_t qs, ks, vs;          // token strides
  int64_t qk, vo, gate, state; // dense elements: (B,L,Hk,dk), (B,L,Hv,dv), (B,L,Hv), (B,Hv,dk,dv)
  bool empty() const { return vo == 0; }
};

// Sizes and types common to the forward, the backward and the decode window.
template <typename P>
ssm_status check_delta_sizes(const P* p, int64_t len, int32_t other_dtype, DeltaSizes* s) {
  if (p->batch < 0 || len < 0 || p->key_heads < 0 || p->value_heads < 0)
    return fail(SSM_ERR_BAD_SHAPE, "batch, length and heads must be >= 0 (got %lld, %lld, %lld, %lld)",
                (long long)p->batch, (long long)len, (long long)p->key_heads, (long long)p->value_heads);
  if (len >= kMaxLen) return fail(SSM_ERR_BAD_SHAPE, "the length must be below 2^27 (got %lld)", (long long)len);
  if (p->dk < 1 || p->dk > SSM_MAX_DSTATE)
    return fail(SSM_ERR_BAD_SHAPE, "dk must be in [1, %d] (got %lld)", SSM_MAX_DSTATE, (long long)p->dk);
  if (p->dv < 1 || p->dv > kMaxColumns)
    return fail(SSM_ERR_BAD_SHAPE, "dv must be in [1, %lld] (got %lld)", (long long)kMaxColumns, (long long)p->dv);
  if (p->value_heads > kMaxHeads || p->key_heads > kMaxHeads)
    return fail(SSM_ERR_BAD_SHAPE, "at most %lld heads", (long long)kMaxHeads);
  if (p->key_heads == 0 ? p->value_heads != 0 : p->value_heads == 0 || p->value_heads % p->key_heads != 0)
    return fail(SSM_ERR_BAD_SHAPE, "value_heads (%lld) must be a multiple of key_heads (%lld)",
                (long long)p->value_heads, (long long)p->key_heads);
  if (!valid_dtype(p->in_dtype) || !valid_dtype(other_dtype))
    return fail(SSM_ERR_BAD_DTYPE, "in_dtype and the output's dtype must be SSM_F32 or SSM_BF16");
  const int64_t kq = p->key_heads * p->dk, vv = p->value_heads * p->dv;
  if (p->q_stride < 0 || p->k_stride < 0 || p->v_stride < 0 || (p->q_stride && p->q_stride < kq) ||
      (p->k_stride && p->k_stride < kq) || (p->v_stride && p->v_stride < vv))
    return fail(SSM_ERR_BAD_SHAPE, "a token stride is smaller than the token");
  s->qs = p->q_stride ? p->q_stride : kq;
  s->ks = p->k_stride ? p->k_stride : kq;
  s->vs = p->v_stride ? p->v_stride : vv;
  int64_t bh;
  if (!mul_ok(p->batch, len, &s->tokens) || !span(s->tokens, s->qs, kq, &s->q) ||
      !span(s->tokens, s->ks, kq, &s->k) || !span(s->tokens, s->vs, vv, &s->v) || !mul_ok(s->tokens, kq, &s->qk) ||
      !mul_ok(s->tokens, vv, &s->vo) || !mul_ok(s->tokens, p->value_heads, &s->gate) ||
      !mul_ok(p->batch, p->value_heads, &bh) || !mul_ok(bh, p->dk * p->dv, &s->state) || s->qk > kLim ||
      s->vo > kLim || s->state > kLim)
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows");
  if (bh > std::numeric_limits<int32_t>::max())
    return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
  return SSM_OK;
}

// Step by step: a workgroup of 256 threads for every 64 columns of a head, and a launch has
// less than 2^32 threads.
ssm_status check_steps_grid(int64_t batch, int64_t heads, int64_t dv) {
  if (batch * heads > ((int64_t{1} << 24) - 1) / ((dv + 63) / 64))
    return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
  return SSM_OK;
}

template <typename P>
ssm::DeltaPlan delta_plan(const P* p, int64_t len, const DeltaSizes& s) {
  ssm::DeltaPlan d{};
  d.B = p->batch;
  d.L = len;
  d.Hk = static_cast<int>(p->key_heads);
  d.Hv = static_cast<int>(p->value_heads);
  d.dk = static_cast<int>(p->dk);
  d.dv = static_cast<int>(p->dv);
  d.in_bf16 = p->in_dtype == SSM_BF16;
  d.q = p->q;
  d.k = p->k;
  d.v = p->v;
  d.qs = s.qs;
  d.ks = s.ks;
  d.vs = s.vs;
  d.dt = p->dt_raw;
  d.br = p->beta_raw;
  d.dt_bias = p->dt_bias;
  d.A = p->A;
  d.scale = p->scale;
  d.beta_scale = p->beta_scale;
  return d;
}

// Sequences up to this long go step by step, unless pieces are asked for. The steps take
// the longer the more there are, a chunk about the same time however few of its 64 tokens
// are there. bfloat16, 128 x 128 states, 1 x 16 heads: 14.3, 18.0, 21.5 us at 12, 16, 20
// steps against 19.4 in chunks (8 x 12 heads: 15.1, 18.5, 22.3 against 20.4; 64 x 16: 62,
// 75, 90 against 107; 4 x 8 heads of 64 x 64: 11.6, 14.9, 17.8 against 16.3; 1 x 4 of 256 x
// 256: 18.5, 23.4, 28.2 against 31.8). float32, whose chunks take three times the products:
// 23.0, 29.7, 36.6 us at 24, 32, 40 steps against 29.5 (8 x 12: 25.1, 31.2, 37.7 against 30.5;
// 64 x 16: 102, 129, 158 against 185; 64 x 64: 18.6, 23.9, 28.4 against 22.6; 256 x 256:
// 33.5, 43.5, 53.4 against 71).
constexpr int64_t steps_max(int in_dtype) { return in_dtype == SSM_BF16 ? 16 : 32; }

// One workgroup for every chunk, and at most a workgroup for every 16 columns, in 31 bits: the
// plans can be made (and then say whether each launch fits).
ssm_status check_grid(int64_t batch, int64_t seqlen, int64_t heads, int64_t dv) {
  const int64_t chunks = (seqlen + 63) / 64;
  int64_t blocks;
  if (!mul_ok(batch * heads, chunks, &blocks) || !mul_ok(blocks, (dv + SSM_MAX_DSTATE) / 16 + 2, &blocks) ||
      blocks > std::numeric_limits<int32_t>::max())
    return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
  return SSM_OK;
}

// How the forward runs: step by step (no chunks, no workspace) or in chunks.
ssm_status plan_delta(const ssm_delta_params* p, const DeltaSizes& s, ssm::DeltaChunks* plan) {
  if (p->num_segments < 0) return fail(SSM_ERR_BAD_SHAPE, "num_segments must be >= 0");
  *plan = ssm::DeltaChunks{};
  if (s.empty()) return SSM_OK;
  if (p->seqlen <= steps_max(p->in_dtype) && p->num_segments <= 1)
    return check_steps_grid(p->batch, p->value_heads, p->dv);
  const ssm_status st = check_grid(p->batch, p->seqlen, p->value_heads, p->dv);
  if (st != SSM_OK) return st;
  *plan = ssm::plan_delta_chunks(p->batch, p->seqlen, static_cast<int>(p->value_heads), static_cast<int>(p->dk),
                                 static_cast<int>(p->dv), p->num_segments);
  if (!ssm::delta_grids_fit(p->batch * p->value_heads, static_cast<int>(p->dk), static_cast<int>(p->dv), *plan))
    return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
  return SSM_OK;
}

ssm_status plan_delta_bwd(const ssm_delta_bwd_params* p, DeltaSizes* s, ssm::DeltaBwdLayout* lay) {
  ssm_status st = check_delta_sizes(p, p->seqlen, p->grad_dtype, s);
  if (st != SSM_OK) return st;
  *lay = ssm::DeltaBwdLayout{};
  if (s->empty()) return SSM_OK;
  if ((st = check_grid(p->batch, p->seqlen, p->value_heads, p->dv)) != SSM_OK) return st;
  // per chunk and head: two states of up to (dk + 127) x (dv + 15), U and dR, the record, and
  // what a piece and a group of pieces need (at most one of each for two chunks)
  const int64_t chunks = (p->seqlen + 63) / 64;
  int64_t bytes;
  if (!mul_ok(p->batch * p->value_heads * chunks, 4 * (p->dk + 127) * (2 * p->dk + 4 * p->dv + 314) + 98304, &bytes) ||
      bytes > kLim)
    return fail(SSM_ERR_BAD_SHAPE, "backward workspace size overflows");
  *lay = ssm::plan_delta_bwd(p->batch, p->seqlen, static_cast<int>(p->value_heads), static_cast<int>(p->dk),
                             static_cast<int>(p->dv));
  if (!ssm::delta_bwd_grids_fit(p->batch * p->value_heads, p->batch * p->key_heads, static_cast<int>(p->dk),
                                static_cast<int>(p->dv), *lay))
    return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
  return SSM_OK;
}

struct NormSizes {
  int64_t tokens, q, k, qs, ks, q_dense, k_dense, table;
  bool empty() const { return q_dense == 0 && k_dense == 0; }
};

ssm_status check_norm_sizes(const ssm_qk_norm_params* p, NormSizes* s) {
  if (p->batch < 0 || p->seqlen < 0 || p->q_heads < 0 || p->k_heads < 0 || p->rot_positions < 0)
    return fail(SSM_ERR_BAD_SHAPE, "sizes must be >= 0");
  if (p->seqlen >= kMaxLen) return fail(SSM_ERR_BAD_SHAPE, "seqlen must be below 2^27 (got %lld)", (long long)p->seqlen);
  if (p->q_heads > kMaxHeads || p->k_heads > kMaxHeads)
    return fail(SSM_ERR_BAD_SHAPE, "at most %lld heads", (long long)kMaxHeads);
  if (p->head_dim < 1 || p->head_dim > SSM_MAX_HEAD_DIM)
    return fail(SSM_ERR_BAD_SHAPE, "head_dim must be in [1, %d] (got %lld)", SSM_MAX_HEAD_DIM, (long long)p->head_dim);
  if (p->rot_dim < 0 || p->rot_dim > p->head_dim || p->rot_dim % 2 != 0)
    return fail(SSM_ERR_BAD_SHAPE, "rot_dim must be even and in [0, head_dim] (got %lld)", (long long)p->rot_dim);
  if (p->norm_kind != SSM_NORM_RMS && p->norm_kind != SSM_NORM_L2)
    return fail(SSM_ERR_UNSUPPORTED, "unknown norm_kind %d", p->norm_kind);
  if (!valid_dtype(p->in_dtype) || !valid_dtype(p->out_dtype))
    return fail(SSM_ERR_BAD_DTYPE, "in_dtype/out_dtype must be SSM_F32 or SSM_BF16");
  const int64_t qt = p->q_heads * p->head_dim, kt = p->k_heads * p->head_dim;
  if (p->q_stride < 0 || p->k_stride < 0 || (p->q_stride && p->q_stride < qt) || (p->k_stride && p->k_stride < kt))
    return fail(SSM_ERR_BAD_SHAPE, "a token stride is smaller than the token");
  s->qs = p->q_stride ? p->q_stride : qt;
  s->ks = p->k_stride ? p->k_stride : kt;
  int64_t rows;
  if (!mul_ok(p->batch, p->seqlen, &s->tokens) || !span(s->tokens, s->qs, qt, &s->q) ||
      !span(s->tokens, s->ks, kt, &s->k) || !mul_ok(s->tokens, qt, &s->q_dense) ||
      !mul_ok(s->tokens, kt, &s->k_dense) || !mul_ok(p->rot_positions, p->rot_dim / 2, &s->table) ||
      !mul_ok(s->tokens, p->q_heads + p->k_heads, &rows) || s->q_dense > kLim || s->k_dense > kLim || s->table > kLim)
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows");
  // at most one workgroup for 4 rows (64 lanes a row)
  if (rows / 4 >= std::numeric_limits<int32_t>::max())
    return fail(SSM_ERR_BAD_SHAPE, "problem needs more workgroups than one launch allows");
  return SSM_OK;
}

ssm::NormPlan norm_plan(const ssm_qk_norm_params* p, const NormSizes& s) {
  ssm::NormPlan n{};
  n.B = p->batch;
  n.L = p->seqlen;
  n.P = p->rot_positions;
  n.Hq = static_cast<int>(p->q_heads);
  n.Hk = static_cast<int>(p->k_heads);
  n.d = static_cast<int>(p->head_dim);
  n.rot = static_cast<int>(p->rot_dim);
  n.in_bf16 = p->in_dtype == SSM_BF16;
  n.out_bf16 = p->out_dtype == SSM_BF16;
  n.q = p->q;
  n.k = p->k;
  n.qs = s.qs;
  n.ks = s.ks;
  n.wq = p->wq;
  n.wk = p->wk;
  n.cos = p->cos;
  n.sin = p->sin;
  n.positions = p->positions;
  n.eps = p->eps;
  n.l2 = p->norm_kind == SSM_NORM_L2;
  n.interleaved = p->interleaved != 0;
  return n;
}

size_t norm_bwd_bytes(const ssm_qk_norm_params* p, const NormSizes& s) {
  if (s.empty()) return 0;
  return static_cast<size_t>(ssm::norm_bwd_blocks(s.tokens, static_cast<int>(p->q_heads + p->k_heads),
                                                  static_cast<int>(p->head_dim))) *
         2 * static_cast<size_t>(p->head_dim) * sizeof(float);
}

}  // namespace

extern "C" {

ssm_status ssm_delta_workspace_size(const ssm_delta_params* p, size_t* bytes) {
  if (!p || !bytes) return fail(SSM_ERR_NULL_POINTER, "params or bytes is NULL");
  DeltaSizes s;
  ssm_status st = check_delta_sizes(p, p->seqlen, p->out_dtype, &s);
  if (st != SSM_OK) return st;
  ssm::DeltaChunks plan;
  if ((st = plan_delta(p, s, &plan)) != SSM_OK) return st;
  *bytes = plan.bytes;
  return ok();
}

ssm_status ssm_delta_fwd(const ssm_delta_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  DeltaSizes s;
  ssm_status st = check_delta_sizes(p, p->seqlen, p->out_dtype, &s);
  if (st != SSM_OK) return st;
  ssm::DeltaChunks chunks;
  if ((st = plan_delta(p, s, &chunks)) != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype);
  const Need needs[] = {
      {p->q, s.qk, si, "q", true},         {p->k, s.qk, si, "k", true},
      {p->v, s.vo, si, "v", true},         {p->dt_raw, s.gate, si, "dt_raw", true},
      {p->beta_raw, s.gate, si, "beta_raw", true}, {p->A, s.gate, 4, "A", true},
      {p->out, s.vo, so, "out", true},     {p->dt_bias, 0, 4, "dt_bias", false},
      {p->h0, 0, 4, "h0", false},          {p->h_last, 0, 4, "h_last", false},
      {p->workspace, 0, 256, "workspace", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK) return st;
  if (chunks.bytes > 0 && (!p->workspace || p->workspace_bytes < chunks.bytes))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", chunks.bytes,
                p->workspace ? p->workspace_bytes : static_cast<size_t>(0));
  const Range in[] = {
      range(p->q, s.q, si, "q"), range(p->k, s.k, si, "k"), range(p->v, s.v, si, "v"),
      range(p->dt_raw, s.gate, si, "dt_raw"), range(p->beta_raw, s.gate, si, "beta_raw"),
      range(p->A, p->value_heads, 4, "A"), range(p->dt_bias, p->value_heads, 4, "dt_bias"),
      range(p->reset, s.tokens, 1, "reset"), range(p->h0, s.state, 4, "h0"),
  };
  const Range out[] = {
      range(p->out, s.vo, so, "out"), range(p->h_last, s.state, 4, "h_last"),
      Range{chunks.bytes ? static_cast<const char*>(p->workspace) : nullptr, chunks.bytes, "workspace"},
  };
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_delta_fwd: B %lld L %lld heads %lld / %lld, dk %lld dv %lld, %s in, %s out, resets %d; %d chunks in %d "
          "pieces, workspace %zu bytes",
          (long long)p->batch, (long long)p->seqlen, (long long)p->key_heads, (long long)p->value_heads,
          (long long)p->dk, (long long)p->dv, si == 2 ? "bf16" : "f32", so == 2 ? "bf16" : "f32",
          p->reset != nullptr, chunks.chunks, chunks.pieces, chunks.bytes);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (s.empty()) {  // the state passes through an empty sequence
    const hipError_t e = ssm::launch_fill(p->h_last, p->h0, 0.0f, 0.0f, s.state, stream);
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "fill launch failed: %s", hipGetErrorString(e));
    return ok();
  }
  ssm::DeltaPlan plan = delta_plan(p, p->seqlen, s);
  plan.out_bf16 = p->out_dtype == SSM_BF16;
  plan.reset = p->reset;
  plan.h0 = p->h0;
  plan.out = p->out;
  plan.h_last = p->h_last;
  const hipError_t e = chunks.chunks > 0 ? ssm::launch_delta_chunks(plan, chunks, p->workspace, stream)
                                         : ssm::launch_delta_steps(plan, stream);
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "delta rule launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_delta_update(const ssm_delta_update_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  DeltaSizes s;
  ssm_status st = check_delta_sizes(p, p->tokens, p->out_dtype, &s);
  if (st == SSM_OK && !s.empty()) st = check_steps_grid(p->batch, p->value_heads, p->dv);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype);
  const Need needs[] = {
      {p->h, s.state, 4, "h", true},       {p->q, s.qk, si, "q", true},
      {p->k, s.qk, si, "k", true},         {p->v, s.vo, si, "v", true},
      {p->dt_raw, s.gate, si, "dt_raw", true}, {p->beta_raw, s.gate, si, "beta_raw", true},
      {p->A, s.gate, 4, "A", true},        {p->out, s.vo, so, "out", true},
      {p->dt_bias, 0, 4, "dt_bias", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK) return st;
  const Range in[] = {
      range(p->q, s.q, si, "q"), range(p->k, s.k, si, "k"), range(p->v, s.v, si, "v"),
      range(p->dt_raw, s.gate, si, "dt_raw"), range(p->beta_raw, s.gate, si, "beta_raw"),
      range(p->A, p->value_heads, 4, "A"), range(p->dt_bias, p->value_heads, 4, "dt_bias"),
  };
  const Range out[] = {range(p->out, s.vo, so, "out"), range(p->h, s.state, 4, "h")};
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_delta_update: B %lld T %lld heads %lld / %lld, dk %lld dv %lld, %s in", (long long)p->batch,
          (long long)p->tokens, (long long)p->key_heads, (long long)p->value_heads, (long long)p->dk,
          (long long)p->dv, si == 2 ? "bf16" : "f32");
  if (s.empty()) return ok();
  ssm::DeltaPlan plan = delta_plan(p, p->tokens, s);
  plan.out_bf16 = p->out_dtype == SSM_BF16;
  plan.h0 = p->h;
  plan.h_last = p->h;
  plan.out = p->out;
  const hipError_t e = ssm::launch_delta_steps(plan, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "delta window launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_delta_bwd_workspace_size(const ssm_delta_bwd_params* p, size_t* bytes) {
  if (!p || !bytes) return fail(SSM_ERR_NULL_POINTER, "params or bytes is NULL");
  DeltaSizes s;
  ssm::DeltaBwdLayout lay;
  const ssm_status st = plan_delta_bwd(p, &s, &lay);
  if (st != SSM_OK) return st;
  *bytes = lay.bytes;
  return ok();
}

ssm_status ssm_delta_bwd(const ssm_delta_bwd_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  DeltaSizes s;
  ssm::DeltaBwdLayout lay;
  ssm_status st = plan_delta_bwd(p, &s, &lay);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), sg = dtype_size(p->grad_dtype);
  const Need needs[] = {
      {p->q, s.qk, si, "q", true},          {p->k, s.qk, si, "k", true},
      {p->v, s.vo, si, "v", true},          {p->dt_raw, s.gate, si, "dt_raw", true},
      {p->beta_raw, s.gate, si, "beta_raw", true}, {p->A, s.gate, 4, "A", true},
      {p->dout, s.vo, si, "dout", true},    {p->dq, s.qk, sg, "dq", true},
      {p->dk_out, s.qk, sg, "dk_out", true}, {p->dv_out, s.vo, sg, "dv_out", true},
      {p->d_dt_raw, s.gate, sg, "d_dt_raw", true}, {p->dbeta_raw, s.gate, sg, "dbeta_raw", true},
      {p->dA, p->value_heads, 4, "dA", true}, {p->dt_bias, 0, 4, "dt_bias", false},
      {p->h0, 0, 4, "h0", false},           {p->dh_last, 0, 4, "dh_last", false},
      {p->d_dt_bias, 0, 4, "d_dt_bias", false}, {p->dh0, 0, 4, "dh0", false},
      {p->workspace, 0, 256, "workspace", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK) return st;
  if (lay.bytes > 0 && (!p->workspace || p->workspace_bytes < lay.bytes))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", lay.bytes,
                p->workspace ? p->workspace_bytes : static_cast<size_t>(0));
  const Range in[] = {
      range(p->q, s.q, si, "q"), range(p->k, s.k, si, "k"), range(p->v, s.v, si, "v"),
      range(p->dt_raw, s.gate, si, "dt_raw"), range(p->beta_raw, s.gate, si, "beta_raw"),
      range(p->A, p->value_heads, 4, "A"), range(p->dt_bias, p->value_heads, 4, "dt_bias"),
      range(p->reset, s.tokens, 1, "reset"), range(p->h0, s.state, 4, "h0"),
      range(p->dout, s.vo, si, "dout"), range(p->dh_last, s.state, 4, "dh_last"),
  };
  const Range out[] = {
      range(p->dq, s.qk, sg, "dq"), range(p->dk_out, s.qk, sg, "dk_out"), range(p->dv_out, s.vo, sg, "dv_out"),
      range(p->d_dt_raw, s.gate, sg, "d_dt_raw"), range(p->dbeta_raw, s.gate, sg, "dbeta_raw"),
      range(p->dA, p->value_heads, 4, "dA"), range(p->d_dt_bias, p->value_heads, 4, "d_dt_bias"),
      range(p->dh0, s.state, 4, "dh0"),
      Range{lay.bytes ? static_cast<const char*>(p->workspace) : nullptr, lay.bytes, "workspace"},
  };
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_delta_bwd: B %lld L %lld heads %lld / %lld, dk %lld dv %lld, %s in, %s gradients; %d chunks, workspace "
          "%zu bytes",
          (long long)p->batch, (long long)p->seqlen, (long long)p->key_heads, (long long)p->value_heads,
          (long long)p->dk, (long long)p->dv, si == 2 ? "bf16" : "f32", sg == 2 ? "bf16" : "f32", lay.chunks,
          lay.bytes);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (s.empty()) {  // no token: sums over nothing, and the adjoint passes through
    hipError_t e = ssm::launch_fill(p->dA, nullptr, 0.0f, 0.0f, p->value_heads, stream);
    if (e == hipSuccess) e = ssm::launch_fill(p->d_dt_bias, nullptr, 0.0f, 0.0f, p->value_heads, stream);
    if (e == hipSuccess) e = ssm::launch_fill(p->dh0, p->dh_last, 0.0f, 0.0f, s.state, stream);
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "fill launch failed: %s", hipGetErrorString(e));
    return ok();
  }
  ssm::DeltaPlan plan = delta_plan(p, p->seqlen, s);
  plan.reset = p->reset;
  plan.h0 = p->h0;
  ssm::DeltaBwdPlan g{};
  g.grad_bf16 = p->grad_dtype == SSM_BF16;
  g.dout = p->dout;
  g.dh_last = p->dh_last;
  g.dq = p->dq;
  g.dk = p->dk_out;
  g.dv = p->dv_out;
  g.ddt = p->d_dt_raw;
  g.dbr = p->dbeta_raw;
  g.dA = p->dA;
  g.dbias = p->d_dt_bias;
  g.dh0 = p->dh0;
  const hipError_t e = ssm::launch_delta_bwd(plan, g, lay, p->workspace, stream);
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "delta rule backward launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_qk_norm_fwd(const ssm_qk_norm_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  NormSizes s;
  ssm_status st = check_norm_sizes(p, &s);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype);
  const int64_t turned = p->rot_dim > 0 && !s.empty() ? s.table : 0;
  const Need needs[] = {
      {p->q, s.q_dense, si, "q", true},          {p->k, s.k_dense, si, "k", true},
      {p->q_out, s.q_dense, so, "q_out", true},  {p->k_out, s.k_dense, so, "k_out", true},
      {p->cos, turned, 4, "cos", true},          {p->sin, turned, 4, "sin", true},
      {p->wq, 0, 4, "wq", false},                {p->wk, 0, 4, "wk", false},
      {p->positions, 0, 4, "positions", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK) return st;
  const Range in[] = {
      range(p->q, s.q, si, "q"), range(p->k, s.k, si, "k"), range(p->wq, p->head_dim, 4, "wq"),
      range(p->wk, p->head_dim, 4, "wk"), range(p->cos, s.table, 4, "cos"), range(p->sin, s.table, 4, "sin"),
      range(p->positions, s.tokens, 4, "positions"),
  };
  const Range out[] = {range(p->q_out, s.q_dense, so, "q_out"), range(p->k_out, s.k_dense, so, "k_out")};
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_qk_norm_fwd: %lld tokens, heads %lld + %lld of %lld, %lld turned", (long long)s.tokens,
          (long long)p->q_heads, (long long)p->k_heads, (long long)p->head_dim, (long long)p->rot_dim);
  if (s.empty()) return ok();
  ssm::NormPlan plan = norm_plan(p, s);
  plan.q_out = p->q_out;
  plan.k_out = p->k_out;
  const hipError_t e = ssm::launch_qk_norm(plan, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "norm launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_qk_norm_bwd_workspace_size(const ssm_qk_norm_params* p, size_t* bytes) {
  if (!p || !bytes) return fail(SSM_ERR_NULL_POINTER, "params or bytes is NULL");
  NormSizes s;
  const ssm_status st = check_norm_sizes(p, &s);
  if (st != SSM_OK) return st;
  *bytes = norm_bwd_bytes(p, s);
  return ok();
}

ssm_status ssm_qk_norm_bwd(const ssm_qk_norm_params* p, void* hip_stream) {
  if (!p) return fail(SSM_ERR_NULL_POINTER, "params is NULL");
  NormSizes s;
  ssm_status st = check_norm_sizes(p, &s);
  if (st != SSM_OK) return st;
  const size_t si = dtype_size(p->in_dtype), so = dtype_size(p->out_dtype);
  const int64_t turned = p->rot_dim > 0 && !s.empty() ? s.table : 0;
  const Need needs[] = {
      {p->q, s.q_dense, si, "q", true},            {p->k, s.k_dense, si, "k", true},
      {p->dq_out, s.q_dense, si, "dq_out", true},  {p->dk_out, s.k_dense, si, "dk_out", true},
      {p->dq, s.q_dense, so, "dq", true},          {p->dk, s.k_dense, so, "dk", true},
      {p->cos, turned, 4, "cos", true},            {p->sin, turned, 4, "sin", true},
      {p->wq, 0, 4, "wq", false},                  {p->wk, 0, 4, "wk", false},
      {p->positions, 0, 4, "positions", false},    {p->dwq, 0, 4, "dwq", false},
      {p->dwk, 0, 4, "dwk", false},                {p->workspace, 0, 16, "workspace", false},
  };
  if ((st = check_pointers(needs)) != SSM_OK) return st;
  const size_t ws = norm_bwd_bytes(p, s);
  if (ws > 0 && (!p->workspace || p->workspace_bytes < ws))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", ws,
                p->workspace ? p->workspace_bytes : static_cast<size_t>(0));
  const Range in[] = {
      range(p->q, s.q, si, "q"), range(p->k, s.k, si, "k"), range(p->wq, p->head_dim, 4, "wq"),
      range(p->wk, p->head_dim, 4, "wk"), range(p->cos, s.table, 4, "cos"), range(p->sin, s.table, 4, "sin"),
      range(p->positions, s.tokens, 4, "positions"), range(p->dq_out, s.q_dense, si, "dq_out"),
      range(p->dk_out, s.k_dense, si, "dk_out"),
  };
  const Range out[] = {
      range(p->dq, s.q_dense, so, "dq"), range(p->dk, s.k_dense, so, "dk"), range(p->dwq, p->head_dim, 4, "dwq"),
      range(p->dwk, p->head_dim, 4, "dwk"),
      Range{ws ? static_cast<const char*>(p->workspace) : nullptr, ws, "workspace"},
  };
  if ((st = check_overlaps(in, out)) != SSM_OK) return st;
  SSM_LOG("ssm_qk_norm_bwd: %lld tokens, heads %lld + %lld of %lld, %lld turned, workspace %zu bytes",
          (long long)s.tokens, (long long)p->q_heads, (long long)p->k_heads, (long long)p->head_dim,
          (long long)p->rot_dim, ws);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (s.empty()) {  // sums over no row
    hipError_t e = ssm::launch_fill(p->dwq, nullptr, 0.0f, 0.0f, p->head_dim, stream);
    if (e == hipSuccess) e = ssm::launch_fill(p->dwk, nullptr, 0.0f, 0.0f, p->head_dim, stream);
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "fill launch failed: %s", hipGetErrorString(e));
    return ok();
  }
  ssm::NormPlan plan = norm_plan(p, s);
  plan.dq_out = p->dq_out;
  plan.dk_out = p->dk_out;
  plan.dq = p->dq;
  plan.dk = p->dk;
  plan.dwq = p->dwq;
  plan.dwk = p->dwk;
  plan.part = static_cast<float*>(p->workspace);
  const hipError_t e = ssm::launch_qk_norm_bwd(plan, stream);
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "norm backward launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
