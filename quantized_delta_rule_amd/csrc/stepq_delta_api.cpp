// stepq_delta_api.cpp -- host side of the sequence calls: argument checks and launches.  The ABI is
// declared (and each call documented) in stepq.h.
#include <hip/hip_runtime.h>

#include <climits>

#include "stepq.h"
#include "stepq_delta.h"
#include "stepq_host.h"
#include "stepq_internal.h"

namespace stepq {

// Chunks pay from about 16 tokens a sequence on: a chunk pass costs two launches and the whole
// 64-row products whatever the length, a token by itself one step of the recurrence (us, d = 128 bf16,
// chunks against token by token at 8 / 16 / 32 tokens: 1 x 32 heads 16 / 16 / 16 against 12 / 21 / 39,
// 8 x 48 heads 42 / 42 / 43 against 20 / 29 / 51, 70 x 48 heads 179 / 182 / 190 against 103 / 165 / 304).
// Lengths are on the device.  Where they are shorter on average, but one may be long -- decoding requests
// and a prompt in one call --, both paths are launched and each takes its sequences (48 heads: 64 single tokens
// and 512 693 -> 122 us, 16 and 129 170 -> 51; where none is long the second path's empty launches cost
// 6 us: 64 of 4 tokens 76 -> 83).
constexpr int kShort = 16, kMaybeLong = 128;
enum Path { kTokens, kChunks, kBoth };
static Path forward_path(const SeqArgs& a) {
  if (a.kind != STEPQ_KIND_GDN || a.N <= 0) return kTokens;
  if ((long long)a.T >= (long long)kShort * a.N) return kChunks;
  return a.cu && a.T - a.N >= kMaybeLong ? kBoth : kTokens;
}

size_t forward_bytes(const SeqArgs& a) { return forward_path(a) == kTokens ? 0 : chunk_forward_bytes(a); }

hipError_t launch_forward(const SeqArgs& a, hipStream_t s) {
  const Path path = forward_path(a);
  if (path != kBoth) return path == kChunks ? launch_chunk_forward(a, s) : launch_recurrent(a, s);
  SeqArgs b = a;
  b.split = kShort;
  if (hipError_t e = launch_recurrent(b, s)) return e;
  return launch_chunk_forward(b, s);
}

int seq_args(const void* desc, SeqArgs* a) {
  const auto* d = (const stepq_delta_desc*)desc;
  if (!d) return fail(STEPQ_ERR_INVALID_ARG, "desc is NULL");
  if (d->kind != STEPQ_KIND_GDN && d->kind != STEPQ_KIND_KDA)
    return fail(STEPQ_ERR_INVALID_ARG, "kind must be STEPQ_KIND_GDN or STEPQ_KIND_KDA");
  if (d->order != STEPQ_ORDER_DELTA_FIRST && d->order != STEPQ_ORDER_DECAY_FIRST)
    return fail(STEPQ_ERR_INVALID_ARG, "order must be STEPQ_ORDER_DELTA_FIRST or STEPQ_ORDER_DECAY_FIRST");
  if (d->dtype != STEPQ_DTYPE_F32 && d->dtype != STEPQ_DTYPE_BF16 && d->dtype != STEPQ_DTYPE_F16)
    return fail(STEPQ_ERR_INVALID_ARG, "dtype must be STEPQ_DTYPE_F32, _BF16 or _F16");
  if (d->d != 64 && d->d != 128)
    return fail(STEPQ_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", d->d);
  if (d->n_qk_heads < 1 || d->n_heads < 1 || d->n_heads > 65535 || d->n_heads % d->n_qk_heads)
    return fail(STEPQ_ERR_INVALID_ARG, "n_heads (%d) must be a multiple of n_qk_heads (%d), 1 .. 65535",
                d->n_heads, d->n_qk_heads);
  if (d->n_seqs < 0 || d->n_tokens < 0)
    return fail(STEPQ_ERR_INVALID_ARG, "n_seqs and n_tokens must be >= 0");
  if (d->n_seqs == 0 && d->n_tokens > 0 && !d->cu_seqlens)
    return fail(STEPQ_ERR_INVALID_ARG, "n_tokens = %d without a sequence", d->n_tokens);
  if (!d->cu_seqlens && d->n_seqs > 0 && d->n_tokens % d->n_seqs)
    return fail(STEPQ_ERR_INVALID_ARG, "without cu_seqlens n_tokens (%d) must be a multiple of n_seqs (%d)",
                d->n_tokens, d->n_seqs);
  // 4 d threads and fewer a (sequence, head) and a chunk: below 2^32 in a grid's first dimension
  const long long pairs = (long long)d->n_seqs * d->n_heads;
  const long long chunks = d->n_tokens / 64 + (long long)d->n_seqs + 1;
  if ((pairs > chunks ? pairs : chunks) * 4 * d->d > UINT_MAX)
    return fail(STEPQ_ERR_INVALID_ARG, "n_seqs * n_heads = %lld or n_tokens = %d exceeds the launch grid",
                pairs, d->n_tokens);
  const long long unit = d->dtype == STEPQ_DTYPE_F32 ? 4 : 8;  // elements of 16 bytes
  const long long kd = (long long)d->n_qk_heads * d->d, vd = (long long)d->n_heads * d->d;
  const long long given[4] = {d->q_stride, d->k_stride, d->v_stride, d->out_stride};
  const long long packed[4] = {kd, kd, vd, vd};
  long long st[4];
  for (int i = 0; i < 4; i++) {
    st[i] = given[i] ? given[i] : packed[i];
    if (st[i] < packed[i] || st[i] % unit || st[i] >= (1LL << 23))  // 64 rows within 31 bits of bytes
      return fail(STEPQ_ERR_INVALID_ARG, "%s_stride %lld must be %lld .. 2^23 - 1 and a multiple of 16 bytes",
                  i == 0 ? "q" : i == 1 ? "k" : i == 2 ? "v" : "out", st[i], packed[i]);
  }
  *a = SeqArgs{};
  a->kind = d->kind;
  a->order = d->order;
  a->dtype = d->dtype;
  a->D = d->d;
  a->Hq = d->n_qk_heads;
  a->H = d->n_heads;
  a->grp = d->n_heads / d->n_qk_heads;
  a->N = d->n_seqs;
  a->T = d->n_tokens;
  a->cu = d->cu_seqlens;
  a->qs = st[0];
  a->ks = st[1];
  a->vs = st[2];
  a->os = st[3];
  a->status = d->status;
  return STEPQ_OK;
}

int seq_device(int device) {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) != hipSuccess || device < 0 || device >= ndev)
    return fail(STEPQ_ERR_INVALID_ARG, "device %d not available (%d devices)", device, ndev);
  return STEPQ_OK;
}

int aligned(const void* p, unsigned to, const char* what) {
  if (((uintptr_t)p & (to - 1)) != 0)
    return fail(STEPQ_ERR_INVALID_ARG, "%s must be %u-byte aligned", what, to);
  return STEPQ_OK;
}

int seq_inputs(SeqArgs* a, const void* q, const void* k, const void* v, const float* alpha,
               const float* beta, void* out) {
  if (a->T > 0 && a->N > 0 && (!q || !k || !v || !alpha || !beta || !out))
    return fail(STEPQ_ERR_INVALID_ARG, "q, k, v, alpha, beta and out (d_out) must be non-NULL");
  if (int rc = aligned(q, 16, "q")) return rc;
  if (int rc = aligned(k, 16, "k")) return rc;
  if (int rc = aligned(v, 16, "v")) return rc;
  if (int rc = aligned(out, 16, "out (d_out)")) return rc;
  if (int rc = aligned(alpha, a->kind == STEPQ_KIND_KDA ? 16 : 4, "alpha")) return rc;
  if (int rc = aligned(beta, 4, "beta")) return rc;
  a->q = q;
  a->k = k;
  a->v = v;
  a->alpha = alpha;
  a->beta = beta;
  a->out = out;
  return STEPQ_OK;
}

int seq_workspace(const void* ws, size_t have, size_t need) {
  if (have < need) return fail(STEPQ_ERR_INVALID_ARG, "workspace of %zu bytes, needs %zu", have, need);
  if (need && !ws) return fail(STEPQ_ERR_INVALID_ARG, "workspace is NULL");
  return aligned(ws, 256, "workspace");
}

}  // namespace stepq

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

int backward_args(const stepq_delta_desc* desc, SeqArgs* a) {
  if (int rc = seq_args(desc, a)) return rc;
  if (a->kind != STEPQ_KIND_GDN)
    return fail(STEPQ_ERR_UNSUPPORTED, "the gradient is built for STEPQ_KIND_GDN only");
  return STEPQ_OK;
}

}  // namespace

extern "C" {

int stepq_delta_forward_workspace(const stepq_delta_desc* desc, size_t* bytes) {
  SeqArgs a;
  if (int rc = seq_args(desc, &a)) return rc;
  if (!bytes) return fail(STEPQ_ERR_INVALID_ARG, "bytes is NULL");
  if (int rc = seq_device(desc->device)) return rc;
  *bytes = forward_bytes(a);
  return ok();
}

int stepq_delta_backward_workspace(const stepq_delta_desc* desc, size_t* bytes) {
  SeqArgs a;
  if (int rc = backward_args(desc, &a)) return rc;
  if (!bytes) return fail(STEPQ_ERR_INVALID_ARG, "bytes is NULL");
  if (int rc = seq_device(desc->device)) return rc;
  *bytes = chunk_backward_bytes(a);
  return ok();
}

int stepq_delta_forward(const stepq_delta_desc* desc, const void* q, const void* k, const void* v,
                        const float* alpha, const float* beta, const float* S_in, float* S_out,
                        int n_slots, const int32_t* slots, void* out, void* workspace,
                        size_t workspace_bytes, void* stream) {
  SeqArgs a;
  if (int rc = seq_args(desc, &a)) return rc;
  if (int rc = seq_inputs(&a, q, k, v, alpha, beta, out)) return rc;
  if (int rc = aligned(S_in, 16, "S_in")) return rc;
  if (int rc = aligned(S_out, 16, "S_out")) return rc;
  if (slots && n_slots < 1) return fail(STEPQ_ERR_INVALID_ARG, "n_slots must be >= 1");
  if (int rc = seq_workspace(workspace, workspace_bytes, forward_bytes(a))) return rc;
  if (int rc = seq_device(desc->device)) return rc;
  a.S_in = S_in;
  a.S_out = S_out;
  a.n_slots = n_slots;
  a.slots = slots;
  a.ws = (char*)workspace;
  if (a.N == 0) return ok();
  DeviceGuard dg(desc->device);
  if (!dg.ok_) return fail(STEPQ_ERR_HIP, "hipSetDevice(%d) failed", desc->device);
  hipStream_t s = (hipStream_t)stream;
  return launched(launch_forward(a, s), "delta_forward");
}

int stepq_delta_backward(const stepq_delta_desc* desc, const void* q, const void* k, const void* v,
                         const float* alpha, const float* beta, const float* S_in,
                         const void* d_out, const float* dS_out, void* dq, void* dk, void* dv,
                         float* dalpha, float* dbeta, float* dS_in, void* workspace,
                         size_t workspace_bytes, void* stream) {
  GradArgs g{};
  if (int rc = backward_args(desc, &g.f)) return rc;
  if (int rc = seq_inputs(&g.f, q, k, v, alpha, beta, (void*)d_out)) return rc;
  if (g.f.T > 0 && g.f.N > 0 && (!dq || !dk || !dv || !dalpha || !dbeta))
    return fail(STEPQ_ERR_INVALID_ARG, "dq, dk, dv, dalpha and dbeta must be non-NULL");
  const void* p[] = {S_in, dS_out, dq, dk, dv, dS_in};
  const char* names[] = {"S_in", "dS_out", "dq", "dk", "dv", "dS_in"};
  for (int i = 0; i < 6; i++)
    if (int rc = aligned(p[i], 16, names[i])) return rc;
  if (int rc = aligned(dalpha, 4, "dalpha")) return rc;
  if (int rc = aligned(dbeta, 4, "dbeta")) return rc;
  if (int rc = seq_workspace(workspace, workspace_bytes, chunk_backward_bytes(g.f))) return rc;
  if (int rc = seq_device(desc->device)) return rc;
  g.f.S_in = S_in;
  g.f.ws = (char*)workspace;
  g.f.out = nullptr;
  g.d_out = d_out;
  g.dS_out = dS_out;
  g.dq = dq;
  g.dk = dk;
  g.dv = dv;
  g.dalpha = dalpha;
  g.dbeta = dbeta;
  g.dS_in = dS_in;
  if (g.f.N == 0) return ok();
  DeviceGuard dg(desc->device);
  if (!dg.ok_) return fail(STEPQ_ERR_HIP, "hipSetDevice(%d) failed", desc->device);
  return launched(launch_chunk_backward(g, (hipStream_t)stream), "delta_backward");
}

}  // extern "C"
