// stepq_norm.hip -- root-mean-square norm of a head's row, with the residual's addition before it, a gate and eight
// bits behind it, and its gradient:
//   h = x + residual, r = 1 / sqrt(mean h^2 + eps), y = h r w act(z);  scale = max |y| / top, code = y / scale
//   p = dy w act(z):  dh = r (p - h r mean(p h r)) + d_residual;  dw = sum dy act(z) h r;  dz = dy h r w act'(z)
// A row stays in registers from its load to its store, eight neighbouring columns a lane: 8 to 64 lanes a row (to 512
// columns), or a workgroup of 256 (to 8,192) or 1,024 (to 32,768; 512 for the gradient to 16,384).  Bound by HBM, some ten
// operations an element: 16,381 x 48 rows of 128 with a gate, bf16, 120 us, 5.0 TB/s (a copy reaches 5.05); the gradient of
// 8,192 rows of 4,096 with the residual's 44 us for its 268 MB, some of them cached, and 5 for the last sums (without
// reading the next row ahead 69); 70 rows of 4,096 with the residual and e4m3 out 5.5 us.  16,384 rows with the residual,
// own type / e4m3 out, us: of 768 28 / 34, 1,024 30 / 36, 1,536 37 / 42, 2,048 47 / 49, 4,096 100 / 97: a workgroup of 256 holds one
// row, and one of 768 uses 96 of its threads.  The gradient of rows above 16,384 spills registers
// (1,024 of 32,768: 219 us, 0.9 TB/s).
#include "stepq_layer.h"

namespace stepq {
namespace {

using namespace lay;

// Sum (or maximum of values that are not negative) over the TPR threads of a row.  Where a row has several waves,
// `mem` holds one value of each; the next use of the same `mem` has to lie behind another barrier.
template <int TPR, bool MAX>
__device__ __forceinline__ float over_row(float v, float* mem) {
#pragma unroll
  for (int m = 1; m < (TPR < 64 ? TPR : 64); m *= 2) {
    const float o = __shfl_xor(v, m);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) mem[threadIdx.x >> 6] = v;
    __syncthreads();
    v = mem[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; i++) v = MAX ? fmaxf(v, mem[i]) : v + mem[i];
  }
  return v;
}

// Address of head row i where rows of H heads are `stride` elements apart.
__device__ __forceinline__ long long at_row(const NormArgs& A, long long i, long long stride) {
  if (A.H == 1) return i * stride;
  const long long t = i / A.H;
  return t * stride + (i - t * A.H) * A.D;
}

// y / scale, from inv = 1 / scale correctly rounded: the product is off by up to 1.5 units in the last place, a step with its
// exact remainder leaves m 2^-26 (1 + q m / 2) of one (m, q: mantissas), so the result is the rounded quotient but where that lies
// within two units of the numerator's last place of the middle between two values.  Of those, what lies beside a tie between two codes
// is 531 pairs of mantissas; all of them come out right (each was tried), so the codes are those of the rounded quotient.
// FAST needs a scale in (2^-90, inf): there the remainders of quotients of 2^-12 and more are exact, and smaller ones are
// codes of zero; other scales are divided by.  us with a product / this / a division: 16,384 rows of 768 29.0 / 29.9 / 32.0, of
// 1,536 33.6 / 33.4 / 37.0, of 4,096 96 / 96 / 97; 384,000 gated rows of 128 63.8 / 64.3 / 71.3.
template <bool FAST>
__device__ __forceinline__ float quotient(float y, float scale, float inv) {
  if constexpr (!FAST) return y / scale;
  const float q = y * inv;
  return fmaf(fmaf(-q, scale, y), inv, q);
}

// Codes of eight values y / scale.  A product with 1 / scale would put some of those that are near a tie between two codes on its
// other side.
template <bool FAST>
__device__ __forceinline__ void store_codes(int odt, void* out, long long i, const float* y, float scale, float inv) {
  int w[2];
  if (odt == kE4M3) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float u = copysignf(quotient<FAST>(y[j], scale, inv), y[j]);  // the step takes the sign of a zero
      v[j] = u == u ? fminf(fmaxf(u, -448.0f), 448.0f) : u;
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
      w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k], v[4 * k + 1], 0, false);
      w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k + 2], v[4 * k + 3], w[k], true);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; k++) {
      w[k] = 0;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float u = quotient<FAST>(y[4 * k + j], scale, inv), q = rintf(fminf(fmaxf(u, -127.0f), 127.0f));
        w[k] |= ((u == u ? (int)q : 0) & 255) << (8 * j);
      }
    }
  }
  *(int2*)((char*)out + i) = int2{w[0], w[1]};
}

template <int DT, int TPR, int K>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm(NormArgs A) {
  constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
  __shared__ float mem[2][THREADS / 64];
  const int r = threadIdx.x % TPR;
  const long long i = (long long)blockIdx.x * ROWS + threadIdx.x / TPR;
  const bool live = i < A.R;  // one row a workgroup where waves meet: there every row is live
  const long long row = live ? i : A.R - 1;
  const long long xo = at_row(A, row, A.xs), ro = at_row(A, row, A.rs), zo = at_row(A, row, A.zs);
  const long long oo = at_row(A, row, A.os);
  float h[K][8], z[K][8], sq = 0;
#pragma unroll
  for (int k = 0; k < K; k++) {
    const int c = (k * TPR + r) * 8;
    if (c < A.D) {
      load8<DT>(A.x, xo + c, h[k]);
      if (A.z) load8<DT>(A.z, zo + c, z[k]);
      if (A.res) {
        float more[8];
        load8<DT>(A.res, ro + c, more);
#pragma unroll
        for (int j = 0; j < 8; j++) h[k][j] += more[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) h[k][j] = 0, z[k][j] = 0;
    }
#pragma unroll
    for (int j = 0; j < 8; j++) sq = fmaf(h[k][j], h[k][j], sq);
  }
  const float rms = 1.0f / sqrtf(over_row<TPR, false>(sq, mem[0]) / (float)A.D + A.eps);
  float top = 0;
#pragma unroll
  for (int k = 0; k < K; k++) {
    const int c = (k * TPR + r) * 8;
    if (c >= A.D) continue;
    if (A.res_out && live) store8<DT>(A.res_out, ro + c, h[k]);
    float w[8];
    if (A.w) load8_any(A.pdtype, A.w, c, w);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      h[k][j] *= rms;
      if (A.w) h[k][j] *= w[j];
      if (A.z) h[k][j] *= act_of<DT>(A.gate, z[k][j]);
      top = fmaxf(top, fabsf(h[k][j]));
    }
    if (A.odtype == DT && live) store8<DT>(A.out, oo + c, h[k]);
  }
  if (A.odtype == DT) return;
  const float most = A.odtype == kE4M3 ? 448.0f : 127.0f;
  if (A.group == 0) top = over_row<TPR, true>(top, mem[1]);
#pragma unroll
  for (int k = 0; k < K; k++) {
    const int c = (k * TPR + r) * 8;
    if (A.group) {  // 8 or 16 neighbouring lanes
      top = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) top = fmaxf(top, fabsf(h[k][j]));
      for (int m = 1; m < A.group / 8; m *= 2) top = fmaxf(top, __shfl_xor(top, m));
    }
    const float scale = top > 0 ? fmaxf(top / most, 1.17549435e-38f) : 1.0f;
    if (c >= A.D || !live) continue;
    if (A.group == 0 ? c == 0 : c % A.group == 0) A.scale[A.group ? row * (A.D / A.group) + c / A.group : row] = scale;
    if (scale > 0x1p-90f && scale < __builtin_inff()) store_codes<true>(A.odtype, A.out, oo + c, h[k], scale, 1.0f / scale);
    else store_codes<false>(A.odtype, A.out, oo + c, h[k], scale, 0);
  }
}

// Each workgroup takes every gridDim.x'th set of rows and adds up its part of dw on the way; a set's rows are read while
// the set before it is worked on.
template <int DT, int TPR, int K>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm_grad(NormArgs A) {
  constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
  constexpr int size = DT == kF32 ? 4 : 2;
  // long rows: neither the next row nor the weights fit into registers beside a row
  constexpr bool AHEAD = K <= 2 && TPR <= 256;
  __shared__ float mem[2][THREADS / 64];
  __shared__ float part[TPR < 256 ? 4 : 1][TPR < 256 ? 512 : 1];
  const int r = threadIdx.x % TPR;
  float dw[K][8], kept[AHEAD ? K : 1][8];
  auto weight = [&](int k, float* w) {
    const int c = (k * TPR + r) * 8;
#pragma unroll
    for (int j = 0; j < 8; j++) w[j] = 1;
    if (A.w && c < A.D) load8_any(A.pdtype, A.w, c, w);
  };
#pragma unroll
  for (int k = 0; k < K; k++) {
#pragma unroll
    for (int j = 0; j < 8; j++) dw[k][j] = 0;
    if (AHEAD) weight(k, kept[k]);
  }
  Raw<DT, 8> nx[K], nu[K], nz[K], nr[K];  // without gate or residual their loads repeat x's
  const void *zp = A.z ? A.z : A.x, *rp = A.res ? A.res : A.x;
  const long long zs = A.z ? A.zs : A.xs, rs = A.res ? A.rs : A.xs, last = A.D - 8;
  auto fetch = [&](long long i) {
    const long long row = i < A.R ? i : A.R - 1;
    const long long xo = at_row(A, row, A.xs), uo = at_row(A, row, A.os), zo = at_row(A, row, zs), ro = at_row(A, row, rs);
#pragma unroll
    for (int k = 0; k < K; k++) {
      const long long c = (k * TPR + r) * 8, at = c < last ? c : last;
      nx[k].load(A.x, (xo + at) * size);
      nu[k].load(A.d_out, (uo + at) * size);
      nz[k].load(zp, (zo + at) * size);
      nr[k].load(rp, (ro + at) * size);
    }
  };
  const long long step = (long long)gridDim.x * ROWS;
  if (AHEAD) fetch((long long)blockIdx.x * ROWS + threadIdx.x / TPR);
  for (long long i0 = (long long)blockIdx.x * ROWS; i0 < A.R; i0 += step) {
    const long long row = i0 + threadIdx.x / TPR;
    const bool live = row < A.R;
    if (!AHEAD) fetch(row);
    float h[K][8], p[K][8], sq = 0;
    Raw<DT, 8> z[K], more[K];
#pragma unroll
    for (int k = 0; k < K; k++) {
      const bool in = (k * TPR + r) * 8 < A.D;
      z[k] = nz[k];
      more[k] = nr[k];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        h[k][j] = in ? nx[k][j] : 0;
        p[k][j] = in ? nu[k][j] : 0;
        sq = fmaf(h[k][j], h[k][j], sq);
      }
    }
    if (AHEAD && i0 + step < A.R) fetch(row + step);
    const float rms = 1.0f / sqrtf(over_row<TPR, false>(sq, mem[0]) / (float)A.D + A.eps);
    float dot = 0;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int c = (k * TPR + r) * 8;
      float dz[8], w[8];
      if (AHEAD) {
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] = kept[k][j];
      } else {
        weight(k, w);
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        h[k][j] *= rms;
        if (A.z) {
          const float v = z[k][j], s = sigmoid<DT>(v);
          const float slope = A.gate == kSilu ? fmaf(v * s, 1.0f - s, s) : s * (1.0f - s);
          dz[j] = p[k][j] * h[k][j] * w[j] * slope;
          p[k][j] *= A.gate == kSilu ? v * s : s;
        }
        if (live) dw[k][j] = fmaf(p[k][j], h[k][j], dw[k][j]);
        p[k][j] *= w[j];
        dot = fmaf(p[k][j], h[k][j], dot);
      }
      if (A.z && c < A.D && live) store8<DT>(A.dz, row * A.D + c, dz);
    }
    const float mean = over_row<TPR, false>(dot, mem[1]) / (float)A.D;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int c = (k * TPR + r) * 8;
      if (c >= A.D || !live) continue;
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        g[j] = rms * fmaf(-h[k][j], mean, p[k][j]);
        if (A.res) g[j] += more[k][j];
      }
      store8<DT>(A.dx, row * A.D + c, g);
    }
  }
  if (!A.dw) return;
  float* out = A.ws + (long long)blockIdx.x * A.D;
  if constexpr (TPR < 256) {  // rows of a wave, then its four waves
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int m = TPR; m < 64; m *= 2) {
#pragma unroll
      for (int j = 0; j < 8; j++) dw[0][j] += __shfl_xor(dw[0][j], m);
    }
    if (lane < TPR) {
#pragma unroll
      for (int j = 0; j < 8; j++) part[wave][lane * 8 + j] = dw[0][j];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < A.D; c += 256) out[c] = part[0][c] + part[1][c] + part[2][c] + part[3][c];
  } else {
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int c = (k * TPR + r) * 8;
      if (c < A.D) store8<kF32>(out, c, dw[k]);
    }
  }
}

// Workgroups of the gradient: four a CU where a workgroup's rows are short, two where they fill its registers and
// each adds a longer row of partial sums (us of 512 and 1,024 workgroups: 8,192 rows of 2,048 35 and 29, 262,144
// of 128 50 and 41; 8,192 of 4,096 45 and 49, 4,096 of 8,192 47 and 54).
long long grad_groups(const NormArgs& a) {
  const int rows = a.D <= 64 ? 32 : a.D <= 128 ? 16 : a.D <= 256 ? 8 : a.D <= 512 ? 4 : 1;  // of a workgroup, as by_size gives them
  const long long sets = (a.R + rows - 1) / rows, most = a.D <= 2048 ? 1024 : 512;
  return sets < most ? sets : most;
}

template <int DT, bool BACK, int TPR, int K>
hipError_t launch(const NormArgs& a, hipStream_t s) {
  constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
  if constexpr (BACK) {
    const long long groups = grad_groups(a);
    hipLaunchKernelGGL((k_norm_grad<DT, TPR, K>), dim3((unsigned)groups), dim3(THREADS), 0, s, a);
    if (hipError_t e = hipGetLastError()) return e;
    if (!a.dw) return hipSuccess;
    SumArgs m{a.ws, (int)groups, a.D, a.D, 0, a.dw, nullptr, nullptr};
    return launch_sum(m, s);
  } else {
    hipLaunchKernelGGL((k_norm<DT, TPR, K>), dim3((unsigned)((a.R + ROWS - 1) / ROWS)), dim3(THREADS), 0, s, a);
    return hipGetLastError();
  }
}

template <int DT, bool BACK>
hipError_t by_size(const NormArgs& a, hipStream_t s) {
  const int D = a.D;
  if (D <= 64) return launch<DT, BACK, 8, 1>(a, s);
  if (D <= 128) return launch<DT, BACK, 16, 1>(a, s);
  if (D <= 256) return launch<DT, BACK, 32, 1>(a, s);
  if (D <= 512) return launch<DT, BACK, 64, 1>(a, s);
  if (D <= 2048) return launch<DT, BACK, 256, 1>(a, s);
  if (D <= 4096) return launch<DT, BACK, 256, 2>(a, s);
  if (D <= 8192) return launch<DT, BACK, 256, 4>(a, s);
  if (D <= 16384) return launch<DT, BACK, BACK ? 512 : 1024, BACK ? 4 : 2>(a, s);
  return launch<DT, BACK, 1024, 4>(a, s);
}

template <bool BACK>
hipError_t by_type(const NormArgs& a, hipStream_t s) {
  return a.dtype == kF32 ? by_size<kF32, BACK>(a, s)
                         : a.dtype == kBF16 ? by_size<kBF16, BACK>(a, s) : by_size<kF16, BACK>(a, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) { return a.R <= 0 ? hipSuccess : by_type<false>(a, s); }

size_t norm_backward_bytes(const NormArgs& a) { return (size_t)grad_groups(a) * a.D * sizeof(float); }

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s) {
  if (a.R > 0) return by_type<true>(a, s);
  SumArgs m{nullptr, 0, a.D, a.D, 0, a.dw, nullptr, nullptr};
  return a.dw ? launch_sum(m, s) : hipSuccess;
}

}  // namespace stepq
