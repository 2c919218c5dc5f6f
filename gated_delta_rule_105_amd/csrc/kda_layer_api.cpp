// C-ABI front end of the operators around the recurrence: argument
// validation and dispatch for the short convolution, the selective scan and
// the norm of queries and keys.  Plain C++, like kda_api.cpp: every argument
// error is reported before any launch.  The entry points and their contracts
// are declared in include/kda.h.
#include "kda.h"

#include <math.h>
#include <stdint.h>

#include "kda_check.h"
#include "kda_launch.h"
#include "kda_layer.h"

namespace {

struct Tokens {
  size_t n;     // tokens of the whole batch
  size_t seqs;  // sequences
};

// The batch of B rows of T tokens, or n_seqs packed sequences.
int check_tokens(int B, int T, int n_seqs, int dtype, Tokens* t) {
  if (B < 1 || T < 0 || n_seqs < 0) return KDA_ERR_INVALID_ARGUMENT;
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARGUMENT;
  if (n_seqs > 0 && B != 1) return KDA_ERR_INVALID_ARGUMENT;
  t->n = (size_t)B * (size_t)T;
  t->seqs = n_seqs > 0 ? (size_t)n_seqs : (size_t)B;
  return t->n > (size_t)INT32_MAX ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// Bytes between the first and the last element of `rows` rows of `row`
// elements, `ld` elements apart; ld 0 means contiguous.  False: ld is shorter
// than a row, or the size overflows.
bool strided(size_t rows, size_t row, int64_t* ld, size_t esz, size_t* bytes) {
  if (*ld == 0) *ld = (int64_t)row;
  if (*ld < 0 || (size_t)*ld < row) return false;
  if (rows == 0) {
    *bytes = 0;
    return true;
  }
  size_t last;
  if (!mul(rows - 1, (size_t)*ld, &last) || last > SIZE_MAX - row || !mul(last + row, esz, bytes)) return false;
  return *bytes <= SIZE_MAX / 2;
}

bool bytes_of(size_t a, size_t b, size_t c, size_t esz, size_t* out) {
  size_t ab, abc;
  return mul(a, b, &ab) && mul(ab, c, &abc) && mul(abc, esz, out) && *out <= SIZE_MAX / 2;
}

// Ranges of a call's inputs and outputs; outputs overlap nothing.
struct Buffers {
  Range in[16], out[16];
  int n_in = 0, n_out = 0;
  bool fine = true;
  void input(const void* p, size_t bytes, size_t align) {
    fine = fine && aligned(p, align);
    in[n_in++] = range(p, p ? bytes : 0);
  }
  void output(const void* p, size_t bytes, size_t align) {
    fine = fine && aligned(p, align);
    out[n_out++] = range(p, p ? bytes : 0);
  }
  bool valid() const {
    if (!fine) return false;
    for (int i = 0; i < n_out; ++i) {
      for (int j = 0; j < n_in; ++j)
        if (overlap(out[i], in[j])) return false;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return false;
    }
    return true;
  }
};

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return KDA_OK;
  if (!ws || !aligned(ws, kWsAlign)) return KDA_ERR_INVALID_ARGUMENT;
  return have < need ? KDA_ERR_WORKSPACE_TOO_SMALL : KDA_OK;
}

int hip_status(int e) { return e == 0 ? KDA_OK : KDA_ERR_HIP; }

// ---- short convolution -----------------------------------------------------
struct ConvSizes {
  Tokens t;
  int bf16, silu;
  size_t esz, x_bytes, y_bytes, state_bytes, w_bytes, b_bytes;
  kda::ConvArgs a;
};

int check_conv(const kda_conv_desc_t* d, ConvSizes* s) {
  if (!d) return KDA_ERR_INVALID_ARGUMENT;
  const int dtype = as_int(d->dtype), act = as_int(d->activation);
  const int st = check_tokens(d->B, d->T, d->n_seqs, dtype, &s->t);
  if (st == KDA_ERR_INVALID_ARGUMENT) return st;
  if (d->D < 1 || d->width < 1) return KDA_ERR_INVALID_ARGUMENT;
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARGUMENT;
  s->bf16 = dtype == KDA_DTYPE_BF16;
  s->silu = act == KDA_ACT_SILU;
  s->esz = elem_size(dtype);
  const size_t D = (size_t)d->D, W = (size_t)d->width;
  kda::ConvArgs& a = s->a;
  a = kda::ConvArgs{};
  a.ld = d->ld_x;
  if (!strided(s->t.n, D, &a.ld, s->esz, &s->x_bytes)) return KDA_ERR_INVALID_ARGUMENT;
  if (!bytes_of(s->t.n, D, 1, s->esz, &s->y_bytes) || !bytes_of(s->t.seqs, W - 1, D, s->esz, &s->state_bytes) ||
      !bytes_of(D, W, 1, 4, &s->w_bytes))
    return KDA_ERR_INVALID_ARGUMENT;
  s->b_bytes = D * 4;
  if (st != KDA_OK) return st;
  if (d->width < 2 || d->width > 4) return KDA_ERR_UNSUPPORTED;
  if (d->D > (1 << 23)) return KDA_ERR_UNSUPPORTED;  // the grid's second dimension
  if (s->t.n > (size_t)INT32_MAX - 4096) return KDA_ERR_UNSUPPORTED;  // tokens are counted in 32 bits, with a batch ahead
  a.n_seqs = (int)s->t.seqs;
  a.T = d->T;
  a.tokens = (int64_t)s->t.n;
  a.D = d->D;
  return KDA_OK;
}

// The launch over `tile` tokens a wave, and a workgroup per kConvWaves rows of the states with `states`.
bool conv_fits(ConvSizes* s, int width, int tile, bool states) {
  s->a.tile = tile;
  s->a.n_part = kda::conv_parts(s->a.tokens, tile);
  const int64_t rows = states ? (int64_t)s->t.seqs * (width - 1) : 0;
  return kda::grid_fits(s->a.n_part + kda::ceil_div(rows, kda::kConvWaves), 64 * kda::kConvWaves);
}

}  // namespace

extern "C" {

int kda_short_conv_forward(const kda_conv_desc_t* d, const void* x, const float* weight, const float* bias,
                           const void* initial_state, const int32_t* cu_seqlens, void* y, void* final_state,
                           void* stream) {
  ConvSizes s;
  const int st = check_conv(d, &s);
  if (st != KDA_OK) return st;
  if (s.t.n > 0 && (!x || !weight || !y)) return KDA_ERR_INVALID_ARGUMENT;
  if ((d->n_seqs > 0) != (cu_seqlens != nullptr)) return KDA_ERR_INVALID_ARGUMENT;
  if (!conv_fits(&s, d->width, kda::conv_forward_tile(s.bf16, s.a.tokens, s.a.D), final_state != nullptr))
    return KDA_ERR_UNSUPPORTED;
  Buffers b;
  b.input(x, s.x_bytes, s.esz);
  b.input(weight, s.w_bytes, 4);
  b.input(bias, s.b_bytes, 4);
  b.input(initial_state, s.state_bytes, s.esz);
  b.input(cu_seqlens, ((size_t)d->n_seqs + 1) * 4, 4);
  b.output(y, s.y_bytes, s.esz);
  b.output(final_state, s.state_bytes, s.esz);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (s.t.n == 0 && !final_state) return KDA_OK;
  kda::ConvArgs& a = s.a;
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.init = initial_state;
  a.cu = cu_seqlens;
  return hip_status(kda::launch_conv_forward(s.bf16, d->width, s.silu, a, y, final_state, stream));
}

int kda_short_conv_step(const kda_conv_desc_t* d, const void* x, const float* weight, const float* bias, void* state,
                        void* y, void* stream) {
  ConvSizes s;
  const int st = check_conv(d, &s);
  if (st != KDA_OK) return st;
  if (d->T != 1 || d->n_seqs != 0) return KDA_ERR_INVALID_ARGUMENT;
  if (s.t.n * (size_t)d->D > (size_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;  // lanes are counted in 32 bits
  if (!x || !weight || !state || !y) return KDA_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.input(x, s.x_bytes, s.esz);
  b.input(weight, s.w_bytes, 4);
  b.input(bias, s.b_bytes, 4);
  b.output(state, s.state_bytes, s.esz);
  b.output(y, s.y_bytes, s.esz);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  kda::ConvArgs& a = s.a;
  a.x = x;
  a.w = weight;
  a.bias = bias;
  return hip_status(kda::launch_conv_step(s.bf16, d->width, s.silu, a, state, y, stream));
}

static size_t conv_ws_bytes(const kda_conv_desc_t* d, const ConvSizes& s) {
  const int tile = kda::conv_backward_tile(s.a.tokens, s.a.D);
  return (size_t)kda::conv_parts(s.a.tokens, tile) * ((size_t)d->width + 1) * (size_t)d->D * 4;
}

int kda_short_conv_backward_workspace_size(const kda_conv_desc_t* d, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  ConvSizes s;
  const int st = check_conv(d, &s);
  if (st != KDA_OK) return st;
  *bytes = conv_ws_bytes(d, s);
  return KDA_OK;
}

int kda_short_conv_backward(const kda_conv_desc_t* d, const void* x, const float* weight, const float* bias,
                            const void* initial_state, const int32_t* cu_seqlens, const void* dy, const void* dfinal,
                            void* dx, float* dweight, float* dbias, void* dinitial, void* workspace,
                            size_t workspace_bytes, void* stream) {
  ConvSizes s;
  int st = check_conv(d, &s);
  if (st != KDA_OK) return st;
  if (s.t.n > 0 && (!x || !dy || !dx)) return KDA_ERR_INVALID_ARGUMENT;
  if (!weight || !dweight) return KDA_ERR_INVALID_ARGUMENT;  // dinitial's workgroups read the taps of empty sequences too
  if ((d->n_seqs > 0) != (cu_seqlens != nullptr)) return KDA_ERR_INVALID_ARGUMENT;
  if (!conv_fits(&s, d->width, kda::conv_backward_tile(s.a.tokens, s.a.D), dinitial != nullptr))
    return KDA_ERR_UNSUPPORTED;
  const size_t need = conv_ws_bytes(d, s);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != KDA_OK) return st;
  Buffers b;
  b.input(x, s.x_bytes, s.esz);
  b.input(weight, s.w_bytes, 4);
  b.input(bias, s.b_bytes, 4);
  b.input(initial_state, s.state_bytes, s.esz);
  b.input(cu_seqlens, ((size_t)d->n_seqs + 1) * 4, 4);
  b.input(dy, s.y_bytes, s.esz);
  b.input(dfinal, s.state_bytes, s.esz);
  b.output(dx, s.y_bytes, s.esz);
  b.output(dweight, s.w_bytes, 4);
  b.output(dbias, s.b_bytes, 4);
  b.output(dinitial, s.state_bytes, s.esz);
  b.output(need ? workspace : nullptr, need, 1);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  kda::ConvArgs& a = s.a;
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.init = initial_state;
  a.cu = cu_seqlens;
  return hip_status(kda::launch_conv_backward(s.bf16, d->width, s.silu, a, dy, dfinal, dx, dweight, dbias, dinitial,
                                              (float*)workspace, stream));
}

}  // extern "C"

// ---- selective scan ----------------------------------------------------------
namespace {

struct ScanSizes {
  Tokens t;
  int bf16;
  size_t esz, x_bytes, dt_bytes, z_bytes, b_bytes, c_bytes;  // as strided inputs
  size_t row_bytes, bc_bytes;                                // contiguous [tokens, D] and [tokens, G, N]
  size_t a_bytes, d_bytes, state_bytes;
  kda::ScanArgs a;
};

int check_scan(const kda_scan_desc_t* d, ScanSizes* s) {
  if (!d) return KDA_ERR_INVALID_ARGUMENT;
  const int dtype = as_int(d->dtype);
  const int st = check_tokens(d->B, d->T, d->n_seqs, dtype, &s->t);
  if (st == KDA_ERR_INVALID_ARGUMENT) return st;
  if (d->D < 1 || d->N < 1 || d->G < 1 || d->D % d->G != 0) return KDA_ERR_INVALID_ARGUMENT;
  s->bf16 = dtype == KDA_DTYPE_BF16;
  s->esz = elem_size(dtype);
  const size_t n = s->t.n, D = (size_t)d->D, N = (size_t)d->N, GN = (size_t)d->G * N;
  kda::ScanArgs& a = s->a;
  a = kda::ScanArgs{};
  a.ld_x = d->ld_x;
  a.ld_dt = d->ld_dt;
  a.ld_z = d->ld_z;
  a.ld_b = d->ld_b;
  a.ld_c = d->ld_c;
  if (!strided(n, D, &a.ld_x, s->esz, &s->x_bytes) || !strided(n, D, &a.ld_dt, s->esz, &s->dt_bytes) ||
      !strided(n, D, &a.ld_z, s->esz, &s->z_bytes) || !strided(n, GN, &a.ld_b, s->esz, &s->b_bytes) ||
      !strided(n, GN, &a.ld_c, s->esz, &s->c_bytes))
    return KDA_ERR_INVALID_ARGUMENT;
  if (!bytes_of(n, D, 1, s->esz, &s->row_bytes) || !bytes_of(n, GN, 1, s->esz, &s->bc_bytes) ||
      !bytes_of(D, N, 1, 4, &s->a_bytes) || !bytes_of(s->t.seqs, D, N, 4, &s->state_bytes))
    return KDA_ERR_INVALID_ARGUMENT;
  s->d_bytes = D * 4;
  if (st != KDA_OK) return st;
  if (d->N > kda::kScanMaxStates) return KDA_ERR_UNSUPPORTED;
  // one workgroup per 16 channels and at least 64 tokens, in one grid dimension
  const double groups = (double)d->G * ceil((double)(d->D / d->G) / 16.0);
  if (groups * (ceil((double)n / 64.0) + (double)s->t.seqs + 8.0) > 2.0e9) return KDA_ERR_UNSUPPORTED;
  // the kernels count tokens in 32 bits and look a tile ahead; a lane's offset inside 16 rows has 32 bits
  if (n > (size_t)INT32_MAX - 4096) return KDA_ERR_UNSUPPORTED;
  const int64_t rows[] = {a.ld_x, a.ld_dt, a.ld_z, (int64_t)d->D};
  for (int64_t ld : rows)
    if (ld > (1 << 24)) return KDA_ERR_UNSUPPORTED;
  if ((int64_t)d->D * d->N > (1 << 28)) return KDA_ERR_UNSUPPORTED;  // likewise inside a row of states
  a.n_seqs = (int)s->t.seqs;
  a.T = d->T;
  a.tokens = (int64_t)n;
  a.D = d->D;
  a.N = d->N;
  a.G = d->G;
  a.softplus = d->softplus != 0;
  return KDA_OK;
}

kda::ScanPlan scan_plan(const kda_scan_desc_t* d, const ScanSizes& s) {
  return kda::plan_scan(s.a.tokens, (int)s.t.seqs, d->T, d->n_seqs > 0, d->D, d->N, d->G,
                        kda::device_compute_units());
}

void scan_inputs(Buffers* b, const ScanSizes& s, const void* x, const void* dt, const float* A, const void* Bm,
                 const void* Cm, const float* skip, const void* z, const float* dt_bias) {
  b->input(x, s.x_bytes, s.esz);
  b->input(dt, s.dt_bytes, s.esz);
  b->input(A, s.a_bytes, 4);
  b->input(Bm, s.b_bytes, s.esz);
  b->input(Cm, s.c_bytes, s.esz);
  b->input(skip, s.d_bytes, 4);
  b->input(z, s.z_bytes, s.esz);
  b->input(dt_bias, s.d_bytes, 4);
}

void scan_args(kda::ScanArgs* a, const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
               const float* skip, const void* z, const float* dt_bias, const float* h0, const int32_t* cu) {
  a->x = x;
  a->dt = dt;
  a->A = A;
  a->Bm = Bm;
  a->Cm = Cm;
  a->skip = skip;
  a->z = z ? z : x;
  a->has_z = z != nullptr;
  if (!z) a->ld_z = a->ld_x;
  a->bias = dt_bias;
  a->h0 = h0;
  a->cu = cu;
}

}  // namespace

extern "C" {

int kda_selective_scan_workspace_size(const kda_scan_desc_t* d, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  ScanSizes s;
  const int st = check_scan(d, &s);
  if (st != KDA_OK) return st;
  const kda::ScanPlan p = scan_plan(d, s);
  if (!kda::scan_fits(p, d->D, d->G)) return KDA_ERR_UNSUPPORTED;
  *bytes = p.ws_bytes;
  return KDA_OK;
}

int kda_selective_scan_forward(const kda_scan_desc_t* d, const void* x, const void* dt, const float* A,
                               const void* Bm, const void* Cm, const float* skip, const void* z,
                               const float* dt_bias, const float* h0, const int32_t* cu_seqlens, void* o, float* ht,
                               void* workspace, size_t workspace_bytes, void* stream) {
  ScanSizes s;
  int st = check_scan(d, &s);
  if (st != KDA_OK) return st;
  if (s.t.n > 0 && (!x || !dt || !Bm || !Cm || !o)) return KDA_ERR_INVALID_ARGUMENT;
  if (!A) return KDA_ERR_INVALID_ARGUMENT;  // read for the final states of empty sequences too
  if ((d->n_seqs > 0) != (cu_seqlens != nullptr)) return KDA_ERR_INVALID_ARGUMENT;
  const kda::ScanPlan p = scan_plan(d, s);
  if (!kda::scan_fits(p, d->D, d->G)) return KDA_ERR_UNSUPPORTED;
  if ((st = check_workspace(workspace, workspace_bytes, p.ws_bytes)) != KDA_OK) return st;
  Buffers b;
  scan_inputs(&b, s, x, dt, A, Bm, Cm, skip, z, dt_bias);
  b.input(h0, s.state_bytes, 4);
  b.input(cu_seqlens, ((size_t)d->n_seqs + 1) * 4, 4);
  b.output(o, s.row_bytes, s.esz);
  b.output(ht, s.state_bytes, 4);
  b.output(p.ws_bytes ? workspace : nullptr, p.ws_bytes, 1);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (s.t.n == 0 && !ht) return KDA_OK;
  scan_args(&s.a, x, dt, A, Bm, Cm, skip, z, dt_bias, h0, cu_seqlens);
  return hip_status(kda::launch_scan_forward(s.bf16, s.a, p, o, ht, workspace, stream));
}

int kda_selective_scan_step(const kda_scan_desc_t* d, const void* x, const void* dt, const float* A, const void* Bm,
                            const void* Cm, const float* skip, const void* z, const float* dt_bias, float* state,
                            void* o, void* stream) {
  ScanSizes s;
  const int st = check_scan(d, &s);
  if (st != KDA_OK) return st;
  if (d->T != 1 || d->n_seqs != 0) return KDA_ERR_INVALID_ARGUMENT;
  if (s.t.n * (size_t)d->D * 16 > (size_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;  // lanes are counted in 32 bits
  if (!x || !dt || !A || !Bm || !Cm || !state || !o) return KDA_ERR_INVALID_ARGUMENT;
  Buffers b;
  scan_inputs(&b, s, x, dt, A, Bm, Cm, skip, z, dt_bias);
  b.output(state, s.state_bytes, 4);
  b.output(o, s.row_bytes, s.esz);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  scan_args(&s.a, x, dt, A, Bm, Cm, skip, z, dt_bias, nullptr, nullptr);
  return hip_status(kda::launch_scan_step(s.bf16, s.a, state, o, stream));
}

int kda_selective_scan_backward_workspace_size(const kda_scan_desc_t* d, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  ScanSizes s;
  const int st = check_scan(d, &s);
  if (st != KDA_OK) return st;
  const kda::ScanBwdPlan p = kda::plan_scan_backward(s.a.tokens, s.a.n_seqs, d->D, d->N, d->G);
  if (!kda::scan_backward_fits(p, s.a.tokens, d->D, d->N, d->G)) return KDA_ERR_UNSUPPORTED;
  *bytes = p.ws_bytes;
  return KDA_OK;
}

int kda_selective_scan_backward(const kda_scan_desc_t* d, const void* x, const void* dt, const float* A,
                                const void* Bm, const void* Cm, const float* skip, const void* z,
                                const float* dt_bias, const float* h0, const int32_t* cu_seqlens, const void* dout,
                                const float* dht, void* dx, void* ddt, float* dA, void* dB, void* dC, float* dskip,
                                void* dz, float* ddt_bias, float* dh0, void* workspace, size_t workspace_bytes,
                                void* stream) {
  ScanSizes s;
  int st = check_scan(d, &s);
  if (st != KDA_OK) return st;
  if (!z) dz = nullptr;  // neither read nor written
  if (s.t.n > 0 && (!x || !dt || !A || !Bm || !Cm || !dout || !dx || !ddt || !dB || !dC || (z && !dz)))
    return KDA_ERR_INVALID_ARGUMENT;
  if (!A || !dA) return KDA_ERR_INVALID_ARGUMENT;
  if ((d->n_seqs > 0) != (cu_seqlens != nullptr)) return KDA_ERR_INVALID_ARGUMENT;
  const kda::ScanBwdPlan p = kda::plan_scan_backward(s.a.tokens, s.a.n_seqs, d->D, d->N, d->G);
  if (!kda::scan_backward_fits(p, s.a.tokens, d->D, d->N, d->G)) return KDA_ERR_UNSUPPORTED;
  if ((st = check_workspace(workspace, workspace_bytes, p.ws_bytes)) != KDA_OK) return st;
  Buffers b;
  scan_inputs(&b, s, x, dt, A, Bm, Cm, skip, z, dt_bias);
  b.input(h0, s.state_bytes, 4);
  b.input(cu_seqlens, ((size_t)d->n_seqs + 1) * 4, 4);
  b.input(dout, s.row_bytes, s.esz);
  b.input(dht, s.state_bytes, 4);
  b.output(dx, s.row_bytes, s.esz);
  b.output(ddt, s.row_bytes, s.esz);
  b.output(dA, s.a_bytes, 4);
  b.output(dB, s.bc_bytes, s.esz);
  b.output(dC, s.bc_bytes, s.esz);
  b.output(dskip, s.d_bytes, 4);
  b.output(dz, s.row_bytes, s.esz);
  b.output(ddt_bias, s.d_bytes, 4);
  b.output(dh0, s.state_bytes, 4);
  b.output(workspace, p.ws_bytes, 1);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  scan_args(&s.a, x, dt, A, Bm, Cm, skip, z, dt_bias, h0, cu_seqlens);
  const kda::ScanGrads g{dout, dht, dx, ddt, dz, dB, dC, dA, dskip, ddt_bias, dh0};
  return hip_status(kda::launch_scan_backward(s.bf16, s.a, p, g, workspace, stream));
}

}  // extern "C"

// ---- norm of queries and keys ------------------------------------------------
namespace {

struct NormSizes {
  int bf16;
  size_t esz, q_bytes, k_bytes, qo_bytes, ko_bytes, w_bytes, pos_bytes, freq_bytes;
  kda::NormArgs a;
};

int check_norm(const kda_qk_norm_desc_t* d, NormSizes* s) {
  if (!d) return KDA_ERR_INVALID_ARGUMENT;
  const int dtype = as_int(d->dtype), norm = as_int(d->norm);
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARGUMENT;
  if (norm != KDA_NORM_UNIT && norm != KDA_NORM_RMS) return KDA_ERR_INVALID_ARGUMENT;
  if (d->n_tokens < 0 || d->Hq < 1 || d->Hk < 1 || d->d < 1 || d->rot < 0 || d->rot > d->d || d->rot % 2 != 0)
    return KDA_ERR_INVALID_ARGUMENT;
  if (!(d->eps >= 0.0f) || isinf(d->eps) || !isfinite(d->q_scale)) return KDA_ERR_INVALID_ARGUMENT;
  s->bf16 = dtype == KDA_DTYPE_BF16;
  s->esz = elem_size(dtype);
  kda::NormArgs& a = s->a;
  a = kda::NormArgs{};
  a.ld_q = d->ld_q;
  a.ld_k = d->ld_k;
  const size_t n = (size_t)d->n_tokens, qr = (size_t)d->Hq * d->d, kr = (size_t)d->Hk * d->d;
  if (!strided(n, qr, &a.ld_q, s->esz, &s->q_bytes) || !strided(n, kr, &a.ld_k, s->esz, &s->k_bytes) ||
      !bytes_of(n, qr, 1, s->esz, &s->qo_bytes) || !bytes_of(n, kr, 1, s->esz, &s->ko_bytes))
    return KDA_ERR_INVALID_ARGUMENT;
  s->w_bytes = (size_t)d->d * 4;
  s->pos_bytes = n * 4;
  s->freq_bytes = (size_t)d->rot / 2 * 4;
  if (d->d % 2 != 0 || d->d > 512) return KDA_ERR_UNSUPPORTED;
  if (d->Hq > 65536 || d->Hk > 65536) return KDA_ERR_UNSUPPORTED;
  // a wave takes up to 16 heads of a token at least; the kernels count waves in 32 bits
  if ((double)d->n_tokens * (((double)d->Hq + d->Hk) / 16.0 + 3.0) > 2.0e9) return KDA_ERR_UNSUPPORTED;
  a.n_tokens = d->n_tokens;
  a.Hq = d->Hq;
  a.Hk = d->Hk;
  a.d = d->d;
  a.rot = d->rot;
  a.interleaved = d->interleaved != 0;
  a.sum_factor = norm == KDA_NORM_RMS ? 1.0f / (float)d->d : 1.0f;
  a.eps = d->eps;
  a.q_scale = d->q_scale;
  return KDA_OK;
}

void norm_inputs(Buffers* b, const NormSizes& s, const void* q, const void* k, const float* wq, const float* wk,
                 const int32_t* pos, const float* freq) {
  b->input(q, s.q_bytes, s.esz);
  b->input(k, s.k_bytes, s.esz);
  b->input(wq, s.w_bytes, 4);
  b->input(wk, s.w_bytes, 4);
  b->input(pos, s.pos_bytes, 4);
  b->input(freq, s.freq_bytes, 4);
}

void norm_args(kda::NormArgs* a, const void* q, const void* k, const float* wq, const float* wk, const int32_t* pos,
               const float* freq) {
  a->q = q;
  a->k = k;
  a->wq = wq;
  a->wk = wk;
  a->pos = pos;
  a->freq = freq;
}

// partial sums of dq_weight, then of dk_weight
size_t norm_ws_bytes(const kda_qk_norm_desc_t* d) { return (size_t)2 * kda::kNormParts * (size_t)d->d * 4; }

}  // namespace

extern "C" {

int kda_qk_norm_forward(const kda_qk_norm_desc_t* d, const void* q, const void* k, const float* q_weight,
                        const float* k_weight, const int32_t* positions, const float* inv_freq, void* q_out,
                        void* k_out, void* stream) {
  NormSizes s;
  const int st = check_norm(d, &s);
  if (st != KDA_OK) return st;
  if (d->n_tokens > 0 && (!q || !k || !q_out || !k_out || (d->rot > 0 && (!positions || !inv_freq))))
    return KDA_ERR_INVALID_ARGUMENT;
  if (d->rot == 0 && (positions || inv_freq)) return KDA_ERR_INVALID_ARGUMENT;
  Buffers b;
  norm_inputs(&b, s, q, k, q_weight, k_weight, positions, inv_freq);
  b.output(q_out, s.qo_bytes, s.esz);
  b.output(k_out, s.ko_bytes, s.esz);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (d->n_tokens == 0) return KDA_OK;
  if (!kda::norm_forward_fits(s.a)) return KDA_ERR_UNSUPPORTED;
  norm_args(&s.a, q, k, q_weight, k_weight, positions, inv_freq);
  return hip_status(kda::launch_norm_forward(s.bf16, s.a, q_out, k_out, stream));
}

int kda_qk_norm_backward_workspace_size(const kda_qk_norm_desc_t* d, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  NormSizes s;
  const int st = check_norm(d, &s);
  if (st != KDA_OK) return st;
  *bytes = norm_ws_bytes(d);
  return KDA_OK;
}

int kda_qk_norm_backward(const kda_qk_norm_desc_t* d, const void* q, const void* k, const float* q_weight,
                         const float* k_weight, const int32_t* positions, const float* inv_freq, const void* dq_out,
                         const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace,
                         size_t workspace_bytes, void* stream) {
  NormSizes s;
  int st = check_norm(d, &s);
  if (st != KDA_OK) return st;
  if (d->n_tokens > 0 &&
      (!q || !k || !dq_out || !dk_out || !dq || !dk || (d->rot > 0 && (!positions || !inv_freq))))
    return KDA_ERR_INVALID_ARGUMENT;
  if (d->rot == 0 && (positions || inv_freq)) return KDA_ERR_INVALID_ARGUMENT;
  const size_t need = norm_ws_bytes(d);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != KDA_OK) return st;
  Buffers b;
  norm_inputs(&b, s, q, k, q_weight, k_weight, positions, inv_freq);
  b.input(dq_out, s.qo_bytes, s.esz);
  b.input(dk_out, s.ko_bytes, s.esz);
  b.output(dq, s.qo_bytes, s.esz);
  b.output(dk, s.ko_bytes, s.esz);
  b.output(dq_weight, s.w_bytes, 4);
  b.output(dk_weight, s.w_bytes, 4);
  b.output(workspace, need, 1);
  if (!b.valid()) return KDA_ERR_INVALID_ARGUMENT;
  if (d->n_tokens == 0 && !dq_weight && !dk_weight) return KDA_OK;
  norm_args(&s.a, q, k, q_weight, k_weight, positions, inv_freq);
  return hip_status(kda::launch_norm_backward(s.bf16, s.a, dq_out, dk_out, dq, dk, dq_weight, dk_weight,
                                              (float*)workspace, stream));
}

}  // extern "C"
