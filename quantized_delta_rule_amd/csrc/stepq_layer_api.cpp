// stepq_layer_api.cpp -- host side of the convolution, the scan and the norm: argument checks and launches.  The
// ABI is declared (and each call documented) in stepq.h.
#include <hip/hip_runtime.h>

#include <climits>

#include "stepq.h"
#include "stepq_host.h"
#include "stepq_internal.h"
#include "stepq_layer.h"

using namespace stepq;

namespace {

int ok() {
  clear_error();
  return STEPQ_OK;
}

int launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(STEPQ_ERR_HIP, "%s failed: %s", what, hipGetErrorString(e));
  return ok();
}

bool row_type(int dt) { return dt == STEPQ_DTYPE_F32 || dt == STEPQ_DTYPE_BF16 || dt == STEPQ_DTYPE_F16; }

int sequences(int n_seqs, int n_tokens, const void* cu) {
  if (n_seqs < 0 || n_tokens < 0) return fail(STEPQ_ERR_INVALID_ARG, "n_seqs and n_tokens must be >= 0");
  if (n_seqs == 0 && n_tokens > 0 && !cu)
    return fail(STEPQ_ERR_INVALID_ARG, "n_tokens = %d without a sequence", n_tokens);
  if (!cu && n_seqs > 0 && n_tokens % n_seqs)
    return fail(STEPQ_ERR_INVALID_ARG, "without cu_seqlens n_tokens (%d) must be a multiple of n_seqs (%d)", n_tokens,
                n_seqs);
  return STEPQ_OK;
}

// A row stride: `given` or packed, in whole units of `unit` elements (16 bytes; 8 of 8-bit rows).
int stride(long long given, long long packed, long long unit, const char* what, long long* st) {
  *st = given ? given : packed;
  if (*st < packed || *st % unit || *st >= (1LL << 24))
    return fail(STEPQ_ERR_INVALID_ARG, "%s_stride %lld must be %lld .. 2^24 - 1 and a multiple of %lld elements", what,
                *st, packed, unit);
  return STEPQ_OK;
}

int pointers(bool needed, const void* const* p, const char* const* names, int n) {
  for (int i = 0; i < n; i++)
    if (needed && !p[i]) return fail(STEPQ_ERR_INVALID_ARG, "%s must be non-NULL", names[i]);
  return STEPQ_OK;
}

int all_aligned(const void* const* p, const char* const* names, int n, unsigned to) {
  for (int i = 0; i < n; i++)
    if (int rc = aligned(p[i], to, names[i])) return rc;
  return STEPQ_OK;
}

// Outputs that other workgroups would overwrite while an input at the same place is still read.
int apart(const void* out, const char* what, const void* const* in, const char* const* names, int n) {
  for (int i = 0; i < n; i++)
    if (out && out == in[i]) return fail(STEPQ_ERR_INVALID_ARG, "%s must not overlap %s", what, names[i]);
  return STEPQ_OK;
}

// An output's rows in the place of an input's: each row's own threads read it before they write it, which is right only
// where both have the same bytes for a row.
struct Rows {
  const void* p;
  const char* name;
  long long stride;
};
int rows_apart(const Rows& out, bool same_type, const Rows* in, int n) {
  for (int i = 0; i < n; i++)
    if (out.p && out.p == in[i].p && (!same_type || out.stride != in[i].stride))
      return fail(STEPQ_ERR_INVALID_ARG, "%s must not overlap %s, or have its type and row stride", out.name, in[i].name);
  return STEPQ_OK;
}

#define STEPQ_TRY(call) \
  if (int rc_ = (call)) return rc_

int conv_args(const stepq_conv_desc* d, ConvArgs* a) {
  if (!d) return fail(STEPQ_ERR_INVALID_ARG, "desc is NULL");
  if (!row_type(d->dtype)) return fail(STEPQ_ERR_INVALID_ARG, "dtype must be STEPQ_DTYPE_F32, _BF16 or _F16");
  if (!row_type(d->param_dtype))
    return fail(STEPQ_ERR_INVALID_ARG, "param_dtype must be STEPQ_DTYPE_F32, _BF16 or _F16");
  if (d->channels < 8 || d->channels % 8 || d->channels >= (1 << 24))
    return fail(STEPQ_ERR_INVALID_ARG, "channels (%d) must be a multiple of 8, 8 .. 2^24 - 8", d->channels);
  if (d->width < 2 || d->width > 4) return fail(STEPQ_ERR_UNSUPPORTED, "width must be 2, 3 or 4 (got %d)", d->width);
  if (d->activation != STEPQ_ACT_NONE && d->activation != STEPQ_ACT_SILU)
    return fail(STEPQ_ERR_INVALID_ARG, "activation must be STEPQ_ACT_NONE or STEPQ_ACT_SILU");
  STEPQ_TRY(sequences(d->n_seqs, d->n_tokens, d->cu_seqlens));
  // a wave for 16 tokens of 256 channels is more than any kernel launches
  const long long waves = (d->n_tokens / 16 + 2LL * d->n_seqs + 8) * (d->channels / 256 + 1);
  if (waves >= (1LL << 26))
    return fail(STEPQ_ERR_INVALID_ARG, "n_tokens (%d), n_seqs (%d) and channels (%d) exceed the launch grid", d->n_tokens,
                d->n_seqs, d->channels);
  const long long unit = d->dtype == STEPQ_DTYPE_F32 ? 4 : 8;
  *a = ConvArgs{};
  STEPQ_TRY(stride(d->x_stride, d->channels, unit, "x", &a->xs));
  STEPQ_TRY(stride(d->out_stride, d->channels, unit, "out", &a->os));
  a->dtype = d->dtype;
  a->pdtype = d->param_dtype;
  a->C = d->channels;
  a->W = d->width;
  a->act = d->activation;
  a->N = d->n_seqs;
  a->T = d->n_tokens;
  a->cu = d->cu_seqlens;
  a->status = d->status;
  return STEPQ_OK;
}

int scan_args(const stepq_scan_desc* d, ScanArgs* a) {
  if (!d) return fail(STEPQ_ERR_INVALID_ARG, "desc is NULL");
  if (!row_type(d->dtype)) return fail(STEPQ_ERR_INVALID_ARG, "dtype must be STEPQ_DTYPE_F32, _BF16 or _F16");
  if (d->n_groups < 1 || d->channels < 8 || d->channels >= (1 << 24) || d->channels % (8LL * d->n_groups))
    return fail(STEPQ_ERR_INVALID_ARG, "channels (%d) must be a multiple of 8 n_groups (%d), 8 .. 2^24 - 8", d->channels,
                d->n_groups);
  if (d->d_state != 8 && d->d_state != 16 && d->d_state != 32 && d->d_state != 64)
    return fail(STEPQ_ERR_UNSUPPORTED, "d_state must be 8, 16, 32 or 64 (got %d)", d->d_state);
  if (d->softplus != 0 && d->softplus != 1) return fail(STEPQ_ERR_INVALID_ARG, "softplus must be 0 or 1");
  STEPQ_TRY(sequences(d->n_seqs, d->n_tokens, d->cu_seqlens));
  // threads of a launch, below 2^32: 32 channels by 8 waves of every sequence and of segments, which are no more than
  // the sequences again where those are many; an element each of dB and dC
  const long long wide = ((d->channels / d->n_groups + 31LL) / 32) * d->n_groups;
  if (wide * d->n_seqs * 1024 > UINT_MAX || 2LL * d->n_groups * d->d_state * d->n_tokens + 256 > UINT_MAX)
    return fail(STEPQ_ERR_INVALID_ARG, "n_tokens (%d), n_seqs (%d) and channels (%d) exceed the launch grid", d->n_tokens,
                d->n_seqs, d->channels);
  const long long unit = d->dtype == STEPQ_DTYPE_F32 ? 4 : 8, gn = (long long)d->n_groups * d->d_state;
  *a = ScanArgs{};
  STEPQ_TRY(stride(d->x_stride, d->channels, unit, "x", &a->xs));
  STEPQ_TRY(stride(d->dt_stride, d->channels, unit, "dt", &a->dts));
  STEPQ_TRY(stride(d->z_stride, d->channels, unit, "z", &a->zs));
  STEPQ_TRY(stride(d->out_stride, d->channels, unit, "out", &a->os));
  STEPQ_TRY(stride(d->b_stride, gn, unit, "b", &a->bs));
  STEPQ_TRY(stride(d->c_stride, gn, unit, "c", &a->cs));
  a->dtype = d->dtype;
  a->C = d->channels;
  a->G = d->n_groups;
  a->Cg = d->channels / d->n_groups;
  a->n = d->d_state;
  a->softplus = d->softplus;
  a->N = d->n_seqs;
  a->T = d->n_tokens;
  a->cu = d->cu_seqlens;
  a->status = d->status;
  return STEPQ_OK;
}

int scan_grad_args(const stepq_scan_desc* d, ScanArgs* a) {
  STEPQ_TRY(scan_args(d, a));
  // the last sums: 16 threads a column of dA | dD | ddt_bias, in workgroups of 1,024
  if (((long long)a->C * (a->n + 2) + 63) / 64 * 1024 > UINT_MAX)
    return fail(STEPQ_ERR_INVALID_ARG, "channels (%d) x d_state (%d) exceed the gradient's launch grid", a->C, a->n);
  return STEPQ_OK;
}

int scan_inputs(ScanArgs* a, const void* x, const void* dt, const float* A, const void* B, const void* C,
                const float* D, const float* bias, const void* z, const float* S_in, const void* out) {
  const void* p[] = {x, dt, B, C, out, A, z, S_in};
  const char* names[] = {"x", "dt", "B", "C", "out (d_out)", "A", "z", "S_in"};
  STEPQ_TRY(pointers(a->T > 0 && a->N > 0, p, names, 5));
  STEPQ_TRY(pointers(a->N > 0, p + 5, names + 5, 1));
  STEPQ_TRY(all_aligned(p, names, 8, 16));
  STEPQ_TRY(aligned(D, 4, "D"));
  STEPQ_TRY(aligned(bias, 4, "dt_bias"));
  a->x = x;
  a->dt = dt;
  a->A = A;
  a->B = B;
  a->Cm = C;
  a->D = D;
  a->bias = bias;
  a->z = z;
  a->S_in = S_in;
  return STEPQ_OK;
}

int norm_args(const stepq_norm_desc* d, bool forward, NormArgs* a) {
  if (!d) return fail(STEPQ_ERR_INVALID_ARG, "desc is NULL");
  if (!row_type(d->dtype)) return fail(STEPQ_ERR_INVALID_ARG, "dtype must be STEPQ_DTYPE_F32, _BF16 or _F16");
  if (!row_type(d->param_dtype))
    return fail(STEPQ_ERR_INVALID_ARG, "param_dtype must be STEPQ_DTYPE_F32, _BF16 or _F16");
  const bool eight = d->out_dtype == STEPQ_DTYPE_E4M3 || d->out_dtype == STEPQ_DTYPE_I8;
  if (d->out_dtype != d->dtype && !eight)
    return fail(STEPQ_ERR_INVALID_ARG, "out_dtype must be dtype, STEPQ_DTYPE_E4M3 or STEPQ_DTYPE_I8");
  if (d->d < 8 || d->d % 8 || d->d > 32768)
    return fail(STEPQ_ERR_UNSUPPORTED, "d must be a multiple of 8, 8 .. 32768 (got %d)", d->d);
  if (d->n_rows < 0 || d->n_heads < 1 || (long long)d->n_rows * d->n_heads > INT_MAX)
    return fail(STEPQ_ERR_INVALID_ARG, "n_rows (%d) must be >= 0, n_heads (%d) >= 1, their product below 2^31", d->n_rows,
                d->n_heads);
  if (d->gate != STEPQ_ACT_SILU && d->gate != STEPQ_ACT_SIGMOID)
    return fail(STEPQ_ERR_INVALID_ARG, "gate must be STEPQ_ACT_SILU or STEPQ_ACT_SIGMOID");
  if (d->group && (!eight || (d->group != 64 && d->group != 128) || d->d % d->group))
    return fail(STEPQ_ERR_INVALID_ARG, "group must be 0, or with 8 bits 64 or 128 and divide d (got %d)", d->group);
  if (!(d->eps >= 0) || d->eps > 1e30f) return fail(STEPQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
  // the gradient's workgroups go over any number of rows, but rows above 512 columns have one limit both ways
  if ((forward || d->d > 512) && norm_threads((long long)d->n_rows * d->n_heads, d->d) > UINT_MAX)
    return fail(STEPQ_ERR_INVALID_ARG, "n_rows (%d) x n_heads (%d) exceeds the launch grid", d->n_rows, d->n_heads);
  const long long unit = d->dtype == STEPQ_DTYPE_F32 ? 4 : 8, all = (long long)d->n_heads * d->d;
  *a = NormArgs{};
  STEPQ_TRY(stride(d->x_stride, all, unit, "x", &a->xs));
  STEPQ_TRY(stride(d->residual_stride, all, unit, "residual", &a->rs));
  STEPQ_TRY(stride(d->z_stride, all, unit, "z", &a->zs));
  STEPQ_TRY(stride(d->out_stride, all, eight ? 8 : unit, "out", &a->os));
  a->dtype = d->dtype;
  a->pdtype = d->param_dtype;
  a->odtype = d->out_dtype;
  a->H = d->n_heads;
  a->D = d->d;
  a->gate = d->gate;
  a->group = d->group;
  a->R = (long long)d->n_rows * d->n_heads;
  a->eps = d->eps;
  return STEPQ_OK;
}

int norm_grad_args(const stepq_norm_desc* d, NormArgs* a) {
  STEPQ_TRY(norm_args(d, false, a));
  if (d->out_dtype != d->dtype) return fail(STEPQ_ERR_INVALID_ARG, "the gradient's out_dtype must be dtype");
  return STEPQ_OK;
}

template <class Desc, class Args>
int bytes_of(const Desc* desc, size_t* bytes, int (*check)(const Desc*, Args*), size_t (*need)(const Args&)) {
  Args a;
  STEPQ_TRY(check(desc, &a));
  if (!bytes) return fail(STEPQ_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = need(a);
  return ok();
}

}  // namespace

#define STEPQ_ON_DEVICE(dev)                                                     \
  if (int rc_ = seq_device(dev)) return rc_;                                     \
  DeviceGuard dg(dev);                                                           \
  if (!dg.ok_) return fail(STEPQ_ERR_HIP, "hipSetDevice(%d) failed", dev)

extern "C" {

int stepq_conv_forward(const stepq_conv_desc* desc, const void* x, const void* weight, const void* bias,
                       const void* S_in, void* S_out, int n_slots, const int32_t* slots, void* out, void* stream) {
  ConvArgs a;
  STEPQ_TRY(conv_args(desc, &a));
  const void* p[] = {x, out, weight, bias, S_in, S_out};
  const char* names[] = {"x", "out", "weight", "bias", "S_in", "S_out"};
  STEPQ_TRY(pointers(a.T > 0 && a.N > 0, p, names, 2));
  STEPQ_TRY(pointers(a.N > 0, p + 2, names + 2, 1));
  STEPQ_TRY(all_aligned(p, names, 6, 16));
  STEPQ_TRY(apart(a.T > 0 ? out : nullptr, "out", p, names, 1));
  if (slots && n_slots < 1) return fail(STEPQ_ERR_INVALID_ARG, "n_slots must be >= 1");
  STEPQ_ON_DEVICE(desc->device);
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.S_in = S_in;
  a.S_out = S_out;
  a.n_slots = n_slots;
  a.slots = slots;
  a.out = out;
  return launched(launch_conv(a, (hipStream_t)stream), "conv_forward");
}

int stepq_conv_backward_workspace(const stepq_conv_desc* desc, size_t* bytes) {
  return bytes_of(desc, bytes, conv_args, conv_backward_bytes);
}

int stepq_conv_backward(const stepq_conv_desc* desc, const void* x, const void* weight, const void* bias,
                        const void* S_in, const void* d_out, const void* dS_out, void* dx, float* dweight, float* dbias,
                        void* dS_in, void* workspace, size_t workspace_bytes, void* stream) {
  ConvArgs a;
  STEPQ_TRY(conv_args(desc, &a));
  const void* p[] = {x, d_out, dx, weight, dweight, bias, S_in, dS_out, dS_in};
  const char* names[] = {"x", "d_out", "dx", "weight", "dweight", "bias", "S_in", "dS_out", "dS_in"};
  STEPQ_TRY(pointers(a.T > 0 && a.N > 0, p, names, 3));
  STEPQ_TRY(pointers(a.N > 0, p + 3, names + 3, 1));
  STEPQ_TRY(pointers(true, p + 4, names + 4, 1));
  STEPQ_TRY(all_aligned(p, names, 9, 16));
  STEPQ_TRY(apart(a.T > 0 ? dx : nullptr, "dx", p, names, 2));
  STEPQ_TRY(apart(dS_in, "dS_in", p + 6, names + 6, 2));
  STEPQ_TRY(aligned(dbias, 4, "dbias"));
  STEPQ_TRY(seq_workspace(workspace, workspace_bytes, conv_backward_bytes(a)));
  STEPQ_ON_DEVICE(desc->device);
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.S_in = S_in;
  a.d_out = d_out;
  a.dS_out = dS_out;
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.dS_in = dS_in;
  a.ws = (float*)workspace;
  return launched(launch_conv_backward(a, (hipStream_t)stream), "conv_backward");
}

int stepq_scan_forward_workspace(const stepq_scan_desc* desc, size_t* bytes) {
  return bytes_of(desc, bytes, scan_args, scan_forward_bytes);
}

int stepq_scan_backward_workspace(const stepq_scan_desc* desc, size_t* bytes) {
  return bytes_of(desc, bytes, scan_grad_args, scan_backward_bytes);
}

int stepq_scan_forward(const stepq_scan_desc* desc, const void* x, const void* dt, const float* A, const void* B,
                       const void* C, const float* D, const float* dt_bias, const void* z, const float* S_in,
                       float* S_out, int n_slots, const int32_t* slots, void* out, void* workspace,
                       size_t workspace_bytes, void* stream) {
  ScanArgs a;
  STEPQ_TRY(scan_args(desc, &a));
  STEPQ_TRY(scan_inputs(&a, x, dt, A, B, C, D, dt_bias, z, S_in, out));
  STEPQ_TRY(aligned(S_out, 16, "S_out"));
  const void* in[] = {x, dt, z};
  const char* in_names[] = {"x", "dt", "z"};
  STEPQ_TRY(apart(a.T > 0 ? out : nullptr, "out", in, in_names, 3));
  if (slots && n_slots < 1) return fail(STEPQ_ERR_INVALID_ARG, "n_slots must be >= 1");
  STEPQ_TRY(seq_workspace(workspace, workspace_bytes, scan_forward_bytes(a)));
  STEPQ_ON_DEVICE(desc->device);
  a.S_out = S_out;
  a.n_slots = n_slots;
  a.slots = slots;
  a.out = out;
  a.ws = (char*)workspace;
  return launched(launch_scan(a, (hipStream_t)stream), "scan_forward");
}

int stepq_scan_backward(const stepq_scan_desc* desc, const void* x, const void* dt, const float* A, const void* B,
                        const void* C, const float* D, const float* dt_bias, const void* z, const float* S_in,
                        const void* d_out, const float* dS_out, void* dx, void* ddt, float* dA, void* dB, void* dC,
                        float* dD, float* ddt_bias, void* dz, float* dS_in, void* workspace, size_t workspace_bytes,
                        void* stream) {
  ScanArgs a;
  STEPQ_TRY(scan_grad_args(desc, &a));
  STEPQ_TRY(scan_inputs(&a, x, dt, A, B, C, D, dt_bias, z, S_in, d_out));
  const void* p[] = {dx, ddt, dB, dC, dA, dz, dS_out, dS_in};
  const char* names[] = {"dx", "ddt", "dB", "dC", "dA", "dz", "dS_out", "dS_in"};
  STEPQ_TRY(pointers(a.T > 0 && a.N > 0, p, names, 4));
  STEPQ_TRY(pointers(true, p + 4, names + 4, 1));
  STEPQ_TRY(pointers(z && a.T > 0 && a.N > 0, p + 5, names + 5, 1));
  STEPQ_TRY(all_aligned(p, names, 8, 16));
  const void* in[] = {x, dt, z, d_out};
  const char* in_names[] = {"x", "dt", "z", "d_out"};
  const void* out[] = {dx, ddt, dz};
  const char* out_names[] = {"dx", "ddt", "dz"};
  for (int i = 0; i < 3 && a.T > 0; i++) {
    STEPQ_TRY(apart(out[i], out_names[i], in, in_names, 4));
    STEPQ_TRY(apart(out[i], out_names[i], out, out_names, i));
  }
  const void* st[] = {dS_out, S_in};
  const char* st_names[] = {"dS_out", "S_in"};
  STEPQ_TRY(apart(dS_in, "dS_in", st, st_names, 2));
  STEPQ_TRY(aligned(dD, 4, "dD"));
  STEPQ_TRY(aligned(ddt_bias, 4, "ddt_bias"));
  STEPQ_TRY(seq_workspace(workspace, workspace_bytes, scan_backward_bytes(a)));
  STEPQ_ON_DEVICE(desc->device);
  a.ws = (char*)workspace;
  a.d_out = d_out;
  a.dS_out = dS_out;
  a.dx = dx;
  a.ddt = ddt;
  a.dz = dz;
  a.dB = dB;
  a.dC = dC;
  a.dA = dA;
  a.dD = dD;
  a.dbias = ddt_bias;
  a.dS_in = dS_in;
  return launched(launch_scan_backward(a, (hipStream_t)stream), "scan_backward");
}

int stepq_norm_forward(const stepq_norm_desc* desc, const void* x, const void* weight, const void* residual,
                       const void* z, void* out, float* scale, void* residual_out, void* stream) {
  NormArgs a;
  STEPQ_TRY(norm_args(desc, true, &a));
  const bool eight = a.odtype != a.dtype;
  const void* p[] = {x, weight, residual, z, residual_out, out};
  const char* names[] = {"x", "weight", "residual", "z", "residual_out", "out"};
  STEPQ_TRY(pointers(a.R > 0, p, names, 1));
  STEPQ_TRY(pointers(a.R > 0, p + 5, names + 5, 1));
  if (a.R > 0 && eight && !scale) return fail(STEPQ_ERR_INVALID_ARG, "scale must be non-NULL with 8 bits");
  STEPQ_TRY(all_aligned(p, names, 5, 16));
  STEPQ_TRY(aligned(out, eight ? 8 : 16, "out"));
  STEPQ_TRY(aligned(scale, 4, "scale"));
  const Rows in[] = {{x, "x", a.xs}, {residual, "residual", a.rs}, {z, "z", a.zs}};
  if (a.R > 0) {
    STEPQ_TRY(rows_apart({out, "out", a.os}, !eight, in, 3));
    STEPQ_TRY(rows_apart({residual_out, "residual_out", a.rs}, true, in, 3));
    STEPQ_TRY(apart(residual_out, "residual_out", p + 5, names + 5, 1));
  }
  STEPQ_ON_DEVICE(desc->device);
  a.x = x;
  a.w = weight;
  a.res = residual;
  a.z = z;
  a.out = out;
  a.scale = scale;
  a.res_out = residual_out;
  return launched(launch_norm(a, (hipStream_t)stream), "norm_forward");
}

int stepq_norm_backward_workspace(const stepq_norm_desc* desc, size_t* bytes) {
  return bytes_of(desc, bytes, norm_grad_args, norm_backward_bytes);
}

int stepq_norm_backward(const stepq_norm_desc* desc, const void* h, const void* weight, const void* z,
                        const void* d_out, const void* d_residual, void* dx, float* dweight, void* dz, void* workspace,
                        size_t workspace_bytes, void* stream) {
  NormArgs a;
  STEPQ_TRY(norm_grad_args(desc, &a));
  const void* p[] = {h, d_out, dx, dz, weight, z, d_residual};
  const char* names[] = {"h", "d_out", "dx", "dz", "weight", "z", "d_residual"};
  STEPQ_TRY(pointers(a.R > 0, p, names, 3));
  STEPQ_TRY(pointers(a.R > 0 && z, p + 3, names + 3, 1));
  STEPQ_TRY(all_aligned(p, names, 7, 16));
  STEPQ_TRY(aligned(dweight, 4, "dweight"));
  const Rows in[] = {{h, "h", a.xs}, {d_out, "d_out", a.os}, {z, "z", a.zs}, {d_residual, "d_residual", a.rs}};
  const long long packed = (long long)a.H * a.D;
  if (a.R > 0) {
    STEPQ_TRY(rows_apart({dx, "dx", packed}, true, in, 4));
    STEPQ_TRY(rows_apart({dz, "dz", packed}, true, in, 4));
    STEPQ_TRY(apart(dx, "dx", p + 3, names + 3, 1));
  }
  STEPQ_TRY(seq_workspace(workspace, workspace_bytes, dweight ? norm_backward_bytes(a) : 0));
  STEPQ_ON_DEVICE(desc->device);
  a.x = h;
  a.w = weight;
  a.z = z;
  a.d_out = d_out;
  a.res = d_residual;
  a.dx = dx;
  a.dw = dweight;
  a.dz = dz;
  a.ws = (float*)workspace;
  return launched(launch_norm_backward(a, (hipStream_t)stream), "norm_backward");
}

}  // extern "C"
