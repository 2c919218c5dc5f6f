// C-ABI front end of linear attention with a decay for each head and of the
// norms at a block's end: argument validation and dispatch.  Plain C++, like
// kda_api.cpp: every argument error is reported before any launch.  The entry
// points and their contracts are declared in include/kda.h.
#include "kda.h"

#include <math.h>
#include <stdint.h>

#include "kda_block.h"
#include "kda_check.h"
#include "kda_launch.h"
#include "kda_linear.h"

// ---- linear attention --------------------------------------------------------
namespace {

struct LinearSizes {
  Tokens t;
  int bf16, decay;
  size_t esz, q_bytes, k_bytes, v_bytes, g_bytes;        // as strided inputs
  size_t dq_bytes, o_bytes, dg_bytes;                    // contiguous
  size_t state_floats, state_bytes;
  kda::LinearArgs a;
};

int check_linear(const kda_linear_desc_t* d, LinearSizes* s) {
  if (!d) return KDA_ERR_INVALID_ARGUMENT;
  const int dtype = as_int(d->dtype);
  s->decay = as_int(d->decay);
  const int st = check_tokens(d->B, d->T, d->n_seqs, dtype, &s->t);
  if (st == KDA_ERR_INVALID_ARGUMENT) return st;
  if (d->Hq < 1 || d->H < 1 || d->H % d->Hq != 0 || d->d_k < 1 || d->d_v < 1) return KDA_ERR_INVALID_ARGUMENT;
  if (s->decay != KDA_DECAY_NONE && s->decay != KDA_DECAY_HEAD && s->decay != KDA_DECAY_TOKEN)
    return KDA_ERR_INVALID_ARGUMENT;
  if (!isfinite(d->scale)) return KDA_ERR_INVALID_ARGUMENT;
  s->bf16 = dtype == KDA_DTYPE_BF16;
  s->esz = elem_size(dtype);
  const size_t n = s->t.n, H = (size_t)d->H;
  size_t qk_row, v_row;
  if (!mul((size_t)d->Hq, (size_t)d->d_k, &qk_row) || !mul(H, (size_t)d->d_v, &v_row)) return KDA_ERR_INVALID_ARGUMENT;
  kda::LinearArgs& a = s->a;
  a = kda::LinearArgs{};
  a.ld_q = d->ld_q;
  a.ld_k = d->ld_k;
  a.ld_v = d->ld_v;
  a.ld_g = d->ld_g;
  if (!strided(n, qk_row, &a.ld_q, s->esz, &s->q_bytes) || !strided(n, qk_row, &a.ld_k, s->esz, &s->k_bytes) ||
      !strided(n, v_row, &a.ld_v, s->esz, &s->v_bytes) || !strided(n, H, &a.ld_g, s->esz, &s->g_bytes))
    return KDA_ERR_INVALID_ARGUMENT;
  s->dg_bytes = 0;
  if (!bytes_of(n, qk_row, 1, s->esz, &s->dq_bytes) || !bytes_of(n, v_row, 1, s->esz, &s->o_bytes) ||
      !bytes_of(n, H, 1, s->esz, &s->dg_bytes) || !mul((size_t)d->d_k, (size_t)d->d_v, &s->state_floats) ||
      !bytes_of(s->t.seqs, H, s->state_floats, 4, &s->state_bytes))
    return KDA_ERR_INVALID_ARGUMENT;
  if (s->decay == KDA_DECAY_HEAD) s->g_bytes = H * 4;
  if (s->decay == KDA_DECAY_NONE) s->g_bytes = 0;
  if (st != KDA_OK) return st;
  if (d->d_k > kda::kLinearMaxDim || d->d_v > kda::kLinearMaxDim) return KDA_ERR_UNSUPPORTED;
  if (n > (size_t)INT32_MAX - 4096) return KDA_ERR_UNSUPPORTED;  // the kernels count tokens in 32 bits, a chunk ahead
  // a chunk's rows are one buffer of less than 2^31 bytes: 64 of 2 or 32 of 4 bytes an element, outputs in fp32
  const int64_t rows[] = {a.ld_q, a.ld_k, a.ld_v, a.ld_g, (int64_t)H * d->d_k, (int64_t)v_row};
  for (int64_t ld : rows)
    if (ld > (1 << 22)) return KDA_ERR_UNSUPPORTED;
  a.n_seqs = (int)s->t.seqs;
  a.T = d->T;
  a.tokens = (int64_t)n;
  a.Hq = d->Hq;
  a.H = d->H;
  a.dk = d->d_k;
  a.dv = d->d_v;
  a.scale = d->scale;
  return KDA_OK;
}

// False: a launch's grid would not fit.
bool linear_plan(const kda_linear_desc_t* d, const LinearSizes& s, bool backward, kda::LinearPlan* p) {
  *p = kda::plan_linear(s.a.tokens, (int)s.t.seqs, d->T, d->n_seqs > 0, d->H, kda::device_compute_units(),
                        d->d_k, d->d_v, backward);
  if (backward) kda::plan_linear_shared(p, s.a.tokens, d->H, d->Hq, d->d_k);
  return kda::linear_fits(*p, s.a.tokens, d->H, kda::linear_record(d->d_k, d->d_v), d->Hq, d->d_k);
}

// g and the offsets are there exactly where the descriptor says so
bool linear_given(const kda_linear_desc_t* d, const LinearSizes& s, const void* g, bool offsets, const int32_t* cu) {
  if ((s.decay != KDA_DECAY_NONE && (s.t.n > 0 || s.decay == KDA_DECAY_HEAD)) ? !g : s.decay == KDA_DECAY_NONE && g)
    return false;
  return !offsets || (d->n_seqs > 0) == (cu != nullptr);
}

void linear_args(LinearSizes* s, const kda::LinearPlan* p, const void* q, const void* k, const void* v, const void* g,
                 const float* h0, const int32_t* cu) {
  kda::LinearArgs& a = s->a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = s->decay == KDA_DECAY_TOKEN ? g : nullptr;
  a.decay = s->decay == KDA_DECAY_HEAD ? (const float*)g : nullptr;
  a.h0 = h0;
  a.cu = cu;
  if (p) {
    a.slot = p->slot;
    a.n_slots = (int)p->n_slots;
  }
}

void linear_inputs(Buffers* b, const LinearSizes& s, const void* q, const void* k, const void* v, const void* g) {
  b->input(q, s.q_bytes, s.esz);
  b->input(k, s.k_bytes, s.esz);
  b->input(v, s.v_bytes, s.esz);
  b->input(g, s.g_bytes, s.decay == KDA_DECAY_HEAD ? 4 : s.esz);
}

}  // namespace

extern "C" {

int kda_linear_attn_workspace_size(const kda_linear_desc_t* d, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  LinearSizes s;
  const int st = check_linear(d, &s);
  if (st != KDA_OK) return st;
  kda::LinearPlan p;
  if (!linear_plan(d, s, false, &p)) return KDA_ERR_UNSUPPORTED;
  *bytes = p.ws_bytes;
  return KDA_OK;
}

int kda_linear_attn_forward(const kda_linear_desc_t* d, const void* q, const void* k, const void* v, const void* g,
                            const float* h0, const int32_t* cu_seqlens, void* o, float* ht, void* workspace,
                            size_t workspace_bytes, void* stream) {
  LinearSizes s;
  int st = check_linear(d, &s);
  if (st != KDA_OK) return st;
  if (s.t.n > 0 && (!q || !k || !v || !o)) return KDA_ERR_INVALID_ARGUMENT;
  if (!linear_given(d, s, g, true, cu_seqlens)) return KDA_ERR_INVALID_ARGUMENT;
  kda::LinearPlan p;
  if (!linear_plan(d, s, false, &p)) return KDA_ERR_UNSUPPORTED;
  if ((st = check_workspace(workspace, workspace_bytes, p.ws_bytes)) != KDA_OK) return st;
  Buffers b;
  linear_inputs(&b, s, q, k, v, g);
  b.input(h0, s.state_bytes, 4);
  b.input(cu_seqlens, ((size_t)d->n_seqs + 1) * 4, 4);
  b.output(o, s.o_bytes, s.esz);
  b.output(ht, s.state_bytes, 4);
  b.output(p.ws_bytes ? workspace : nullptr, p.ws_bytes, 1);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (s.t.n == 0 && !ht) return KDA_OK;
  linear_args(&s, &p, q, k, v, g, h0, cu_seqlens);
  return hip_status(kda::launch_linear_forward(s.bf16, s.a, p, o, ht, workspace, stream));
}

int kda_linear_attn_step(const kda_linear_desc_t* d, const void* q, const void* k, const void* v, const void* g,
                         float* state, void* o, void* stream) {
  LinearSizes s;
  const int st = check_linear(d, &s);
  if (st != KDA_OK) return st;
  if (d->T != 1 || d->n_seqs != 0) return KDA_ERR_INVALID_ARGUMENT;
  if (!q || !k || !v || !state || !o || !linear_given(d, s, g, false, nullptr)) return KDA_ERR_INVALID_ARGUMENT;
  if (!kda::linear_step_fits(s.a)) return KDA_ERR_UNSUPPORTED;
  Buffers b;
  linear_inputs(&b, s, q, k, v, g);
  b.output(state, s.state_bytes, 4);
  b.output(o, s.o_bytes, s.esz);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  linear_args(&s, nullptr, q, k, v, g, nullptr, nullptr);
  return hip_status(kda::launch_linear_step(s.bf16, s.a, state, o, stream));
}

int kda_linear_attn_backward_workspace_size(const kda_linear_desc_t* d, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  LinearSizes s;
  const int st = check_linear(d, &s);
  if (st != KDA_OK) return st;
  kda::LinearPlan p;
  if (!linear_plan(d, s, true, &p)) return KDA_ERR_UNSUPPORTED;
  *bytes = p.ws_bytes;
  return KDA_OK;
}

int kda_linear_attn_backward(const kda_linear_desc_t* d, const void* q, const void* k, const void* v, const void* g,
                             const float* h0, const int32_t* cu_seqlens, const void* dout, const float* dht, void* dq,
                             void* dk, void* dv, void* dg, float* dh0, void* workspace, size_t workspace_bytes,
                             void* stream) {
  LinearSizes s;
  int st = check_linear(d, &s);
  if (st != KDA_OK) return st;
  if (s.t.n > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv)) return KDA_ERR_INVALID_ARGUMENT;
  if (!linear_given(d, s, g, true, cu_seqlens)) return KDA_ERR_INVALID_ARGUMENT;
  if (s.decay != KDA_DECAY_TOKEN && dg) return KDA_ERR_INVALID_ARGUMENT;
  kda::LinearPlan p;
  if (!linear_plan(d, s, true, &p)) return KDA_ERR_UNSUPPORTED;
  if ((st = check_workspace(workspace, workspace_bytes, p.ws_bytes)) != KDA_OK) return st;
  Buffers b;
  linear_inputs(&b, s, q, k, v, g);
  b.input(h0, s.state_bytes, 4);
  b.input(cu_seqlens, ((size_t)d->n_seqs + 1) * 4, 4);
  b.input(dout, s.o_bytes, s.esz);
  b.input(dht, s.state_bytes, 4);
  b.output(dq, s.dq_bytes, s.esz);
  b.output(dk, s.dq_bytes, s.esz);
  b.output(dv, s.o_bytes, s.esz);
  b.output(dg, s.dg_bytes, s.esz);
  b.output(dh0, s.state_bytes, 4);
  b.output(p.ws_bytes ? workspace : nullptr, p.ws_bytes, 1);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (s.t.n == 0 && !dh0) return KDA_OK;
  linear_args(&s, &p, q, k, v, g, h0, cu_seqlens);
  const kda::LinearGrads grads{dout, dht, dq, dk, dv, dg, dh0};
  return hip_status(kda::launch_linear_backward(s.bf16, s.a, p, grads, workspace, stream));
}

}  // extern "C"

// ---- the norms at a block's end ------------------------------------------------
namespace {

struct BlockSizes {
  int bf16;
  size_t esz, x_bytes, z_bytes, row_bytes, w_bytes;
  kda::BlockNormArgs a;
};

// n_tokens rows of H heads of D channels, x's and z's rows ld_x and ld_z apart.
int check_block(int n_tokens, int H, int D, int dtype, float eps, int64_t ld_x, int64_t ld_z, BlockSizes* s) {
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARGUMENT;
  if (n_tokens < 0 || H < 1 || D < 1) return KDA_ERR_INVALID_ARGUMENT;
  if (!(eps >= 0.0f) || isinf(eps)) return KDA_ERR_INVALID_ARGUMENT;
  s->bf16 = dtype == KDA_DTYPE_BF16;
  s->esz = elem_size(dtype);
  kda::BlockNormArgs& a = s->a;
  a = kda::BlockNormArgs{};
  a.ld_x = ld_x;
  a.ld_z = ld_z;
  const size_t n = (size_t)n_tokens, row = (size_t)H * (size_t)D;
  if (!strided(n, row, &a.ld_x, s->esz, &s->x_bytes) || !strided(n, row, &a.ld_z, s->esz, &s->z_bytes) ||
      !bytes_of(n, row, 1, s->esz, &s->row_bytes))
    return KDA_ERR_INVALID_ARGUMENT;
  s->w_bytes = (size_t)D * 4;
  if (D > kda::kBlockNormMaxDim || H > 65536) return KDA_ERR_UNSUPPORTED;
  a.rows = (int64_t)n * H;
  a.H = H;
  a.D = D;
  a.eps = eps;
  if (!kda::block_norm_fits(a.rows, D, (int)s->esz)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

int check_gated(const kda_gated_norm_desc_t* d, BlockSizes* s) {
  if (!d) return KDA_ERR_INVALID_ARGUMENT;
  const int act = as_int(d->activation);
  if (act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARGUMENT;
  const int st = check_block(d->n_tokens, d->H, d->d, as_int(d->dtype), d->eps, d->ld_x, d->ld_gate, s);
  s->a.act = act == KDA_ACT_SILU;
  return st;
}

int check_residual(const kda_residual_norm_desc_t* d, BlockSizes* s) {
  if (!d || !isfinite(d->scale)) return KDA_ERR_INVALID_ARGUMENT;
  const int st = check_block(d->n_tokens, 1, d->D, as_int(d->dtype), d->eps, d->ld_x, d->ld_residual, s);
  s->a.scale = d->scale;
  return st;
}

// rows of partial sums of `params` parameters
size_t block_ws_bytes(const BlockSizes& s, int params) {
  return (size_t)kda::block_norm_parts(s.a.rows, s.a.D, (int)s.esz) * (size_t)s.a.D * 4 * (size_t)params;
}

}  // namespace

extern "C" {

int kda_gated_norm_forward(const kda_gated_norm_desc_t* d, const void* x, const void* gate, const float* weight, void* y,
                           void* stream) {
  BlockSizes s;
  const int st = check_gated(d, &s);
  if (st != KDA_OK) return st;
  if (d->n_tokens > 0 && (!x || !gate || !y)) return KDA_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.input(x, s.x_bytes, s.esz);
  b.input(gate, s.z_bytes, s.esz);
  b.input(weight, s.w_bytes, 4);
  b.output(y, s.row_bytes, s.esz);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (d->n_tokens == 0) return KDA_OK;
  s.a.x = x;
  s.a.z = gate;
  s.a.w = weight;
  return hip_status(kda::launch_gated_norm_forward(s.bf16, s.a, y, stream));
}

int kda_gated_norm_backward_workspace_size(const kda_gated_norm_desc_t* d, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  BlockSizes s;
  const int st = check_gated(d, &s);
  if (st != KDA_OK) return st;
  *bytes = block_ws_bytes(s, 1);
  return KDA_OK;
}

int kda_gated_norm_backward(const kda_gated_norm_desc_t* d, const void* x, const void* gate, const float* weight,
                            const void* dy, void* dx, void* dgate, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream) {
  BlockSizes s;
  int st = check_gated(d, &s);
  if (st != KDA_OK) return st;
  if (d->n_tokens > 0 && (!x || !gate || !dy || !dx || !dgate)) return KDA_ERR_INVALID_ARGUMENT;
  const size_t need = block_ws_bytes(s, 1);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != KDA_OK) return st;
  Buffers b;
  b.input(x, s.x_bytes, s.esz);
  b.input(gate, s.z_bytes, s.esz);
  b.input(weight, s.w_bytes, 4);
  b.input(dy, s.row_bytes, s.esz);
  b.output(dx, s.row_bytes, s.esz);
  b.output(dgate, s.row_bytes, s.esz);
  b.output(dweight, s.w_bytes, 4);
  b.output(need ? workspace : nullptr, need, 1);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (d->n_tokens == 0 && !dweight) return KDA_OK;
  s.a.x = x;
  s.a.z = gate;
  s.a.w = weight;
  return hip_status(kda::launch_gated_norm_backward(s.bf16, s.a, dy, dx, dgate, dweight, (float*)workspace, stream));
}

int kda_residual_norm_forward(const kda_residual_norm_desc_t* d, const void* x, const void* residual,
                              const float* weight, const float* channel_scale, void* y, void* total, void* stream) {
  BlockSizes s;
  const int st = check_residual(d, &s);
  if (st != KDA_OK) return st;
  if (d->n_tokens > 0 && (!x || !residual || !y || !total)) return KDA_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.input(x, s.x_bytes, s.esz);
  b.input(residual, s.z_bytes, s.esz);
  b.input(weight, s.w_bytes, 4);
  b.input(channel_scale, s.w_bytes, 4);
  b.output(y, s.row_bytes, s.esz);
  b.output(total, s.row_bytes, s.esz);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (d->n_tokens == 0) return KDA_OK;
  s.a.x = x;
  s.a.z = residual;
  s.a.w = weight;
  s.a.channels = channel_scale;
  return hip_status(kda::launch_residual_norm_forward(s.bf16, s.a, y, total, stream));
}

int kda_residual_norm_backward_workspace_size(const kda_residual_norm_desc_t* d, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  BlockSizes s;
  const int st = check_residual(d, &s);
  if (st != KDA_OK) return st;
  *bytes = block_ws_bytes(s, 2);
  return KDA_OK;
}

int kda_residual_norm_backward(const kda_residual_norm_desc_t* d, const void* x, const void* total, const float* weight,
                               const float* channel_scale, const void* dy, const void* dtotal, void* dx,
                               void* dresidual, float* dweight, float* dchannel_scale, void* workspace,
                               size_t workspace_bytes, void* stream) {
  BlockSizes s;
  int st = check_residual(d, &s);
  if (st != KDA_OK) return st;
  if (d->n_tokens > 0 && (!total || !dy || !dresidual || (dchannel_scale && !x))) return KDA_ERR_INVALID_ARGUMENT;
  const size_t need = block_ws_bytes(s, 2);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != KDA_OK) return st;
  Buffers b;
  b.input(x, s.x_bytes, s.esz);
  b.input(total, s.z_bytes, s.esz);
  b.input(weight, s.w_bytes, 4);
  b.input(channel_scale, s.w_bytes, 4);
  b.input(dy, s.row_bytes, s.esz);
  b.input(dtotal, s.row_bytes, s.esz);
  b.output(dx, s.row_bytes, s.esz);
  b.output(dresidual, s.row_bytes, s.esz);
  b.output(dweight, s.w_bytes, 4);
  b.output(dchannel_scale, s.w_bytes, 4);
  b.output(need ? workspace : nullptr, need, 1);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (d->n_tokens == 0 && !dweight && !dchannel_scale) return KDA_OK;
  s.a.x = x;
  s.a.z = total;
  s.a.w = weight;
  s.a.channels = channel_scale;
  return hip_status(kda::launch_residual_norm_backward(s.bf16, s.a, dy, dtotal, dx, dresidual, dweight, dchannel_scale,
                                                       (float*)workspace, stream));
}

}  // extern "C"
