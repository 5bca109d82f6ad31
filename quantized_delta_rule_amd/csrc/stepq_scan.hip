// stepq_scan.hip -- selective state space scan, token by token:
//   h_t = exp(D_t A) h_{t-1} + D_t B_t x_t,  out_t = (C_t . h_t + D x_t) z sigmoid(z)
// A wave owns 256 / n channels of one group of a sequence: n / 4 neighbouring lanes a channel, four states a lane,
// so that states are read and written 16 bytes a lane side by side.
#include <type_traits>
#include <utility>

#include "stepq_scan.h"

namespace stepq {
namespace {

using namespace lay;

template <int DT, int LN>
__global__ __launch_bounds__(256) void k_scan_tokens(ScanArgs A, int tiles) {
  constexpr int GW = 64 / LN, n = 4 * LN;
  const int lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long per = (long long)tiles * A.G;
  if (unit >= per * A.N) return;
  const int s = (int)(unit / per), tg = (int)(unit - s * per), g = tg / tiles, tile = tg - g * tiles;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  const int slot = seq_slot(A, s, valid, tg == 0 && lane == 0);
  if (slot < 0) return;
  if (t0 == t1 && (!A.S_out || A.S_out == A.S_in)) return;
  const int cg = tile * GW + lane / LN, part = lane % LN;
  const bool live = cg < A.Cg;
  const int c = g * A.Cg + (live ? cg : A.Cg - 1);  // lanes past the group's end repeat its last channel
  const long long so = ((long long)slot * A.C + c) * n + 4 * part;
  f4 h = A.S_in ? *(const f4*)(A.S_in + so) : f4{0, 0, 0, 0};
  f4 a2 = *(const f4*)(A.A + (long long)c * n + 4 * part);
#pragma unroll
  for (int i = 0; i < 4; i++) a2[i] *= kLog2e;
  const float skip = A.D ? A.D[c] : 0.0f, bias = A.bias ? A.bias[c] : 0.0f;
  for (int t = t0; t < t1; t++) {
    float x, raw, z, slope;
    loadn<DT, 1>(A.x, t * A.xs + c, &x);
    loadn<DT, 1>(A.dt, t * A.dts + c, &raw);
    const f4 B = load4<DT>(A.B, t * A.bs + g * n + 4 * part), Cm = load4<DT>(A.Cm, t * A.cs + g * n + 4 * part);
    const float D = step_of(A.softplus, raw + bias, slope), dx = D * x;
    float y = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      h[i] = fmaf(decay(D, a2[i]), h[i], dx * B[i]);
      y = fmaf(Cm[i], h[i], y);
    }
#pragma unroll
    for (int m = 1; m < LN; m *= 2) y += __shfl_xor(y, m);
    if (A.D) y = fmaf(skip, x, y);
    if (A.z) {
      loadn<DT, 1>(A.z, t * A.zs + c, &z);
      y *= z * sigmoid(z);
    }
    if (live && part == 0) storen<DT, 1>(A.out, t * A.os + c, &y);
  }
  if (A.S_out && live) *(f4*)(A.S_out + so) = h;
}

// ---------------------------------------------------------------------------------------------
// Blocks of tokens: a workgroup takes CH channels of a sequence, or of one of its segments.  64 / CH
// parts of a wave and the NW waves share a channel's states out, NS each, so that 16 neighbouring lanes have the same B
// and C of a token: they hold the values of a token or two, and an instruction takes one of them for all lanes by itself (row broadcast of its
// operand).  For each block of 16 tokens the waves first turn raw steps into (D, D x) in LDS, a few channels
// each, then run all of them on their states, and add their parts of C . h up through LDS.
// ---------------------------------------------------------------------------------------------

constexpr int kBlock = 16;

// Long sequences run in segments of 2^sh tokens at once: first each segment's last state from the zero state and the
// sum of its steps, then, from what the segments before it leave, the segment itself.
struct Segments {
  int tiles;    // of 64 channels, in a group
  int sh;
  float* last;  // [segments, C, n]: the first of a sequence from its state, the others from zero
  float* steps; // [segments, C]
  float* first; // [N, C, n]: the sequences' first states (S_out may be S_in)
};

// E neighbouring elements as they lie in memory: kept until they are used, so that their load is not waited for before.
template <int DT, int E>
struct Raw {
  typedef typename std::conditional<DT == kF32, float, unsigned short>::type T;
  typedef T V __attribute__((ext_vector_type(E)));
  typename std::conditional<E == 1, T, V>::type v;
  __device__ __forceinline__ void load(const char* p, unsigned at) { v = *(const decltype(v)*)(p + at); }
  __device__ __forceinline__ float operator[](int i) const {
    T x;
    if constexpr (E == 1) x = v;
    else x = v[i];
    if constexpr (DT == kF32) return x;
    else return e_f<DT>(x);
  }
};

// Lane I of each 16 lanes' value, for all of them.
template <int I>
__device__ __forceinline__ float row_lane(float v) {
  const int x = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, x, 0x150 + I, 0xf, 0xf, true));
}

// sum_{i < 4} (lane I + i of each 16 lanes' value) h_i, added to y where MORE: the broadcast is part of the
// multiply-add, which the compiler does not do by itself.  The s_nop is the two wait states between a vector write
// and its read across lanes.
template <int I, bool MORE>
__device__ __forceinline__ float row_dot(float y, float v, const float* h) {
  if constexpr (MORE)
    asm("s_nop 1\n\tv_fmac_f32_dpp %0, %1, %2 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %4 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
        : "+&v"(y)
        : "v"(v), "v"(h[0]), "v"(h[1]), "v"(h[2]), "v"(h[3]), "n"(I), "n"(I + 1), "n"(I + 2), "n"(I + 3));
  else
    asm("s_nop 1\n\tv_mul_f32_dpp %0, %1, %2 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %4 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
        : "=&v"(y)
        : "v"(v), "v"(h[0]), "v"(h[1]), "v"(h[2]), "v"(h[3]), "n"(I), "n"(I + 1), "n"(I + 2), "n"(I + 3));
  return y;
}

template <int I>
__device__ __forceinline__ float row_dot2(float v, const float* h) {
  float y;
  asm("s_nop 1\n\tv_mul_f32_dpp %0, %1, %2 row_newbcast:%4 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%5 row_mask:0xf bank_mask:0xf"
      : "=&v"(y)
      : "v"(v), "v"(h[0]), "v"(h[1]), "n"(I), "n"(I + 1));
  return y;
}

// NS states at p, 16 or 8 bytes at a time.
template <int NS>
__device__ __forceinline__ void get_states(const float* p, float* h) {
  constexpr int W = NS < 4 ? NS : 4;
#pragma unroll
  for (int i = 0; i < NS; i += W) loadn<kF32, W>(p, i, h + i);
}
template <int NS>
__device__ __forceinline__ void put_states(float* p, const float* h) {
  constexpr int W = NS < 4 ? NS : 4;
#pragma unroll
  for (int i = 0; i < NS; i += W) storen<kF32, W>(p, i, h + i);
}

// PASS 0: a whole sequence.  1: a segment's last state and steps.  2: a segment.
template <int DT, int NS, int CH, int NW, int PASS>
__global__ __launch_bounds__(64 * NW) void k_scan_run(ScanArgs A, Segments Q) {
  constexpr int P = 64 / CH, n = NS * P * NW;  // parts of a channel's states in a wave
  constexpr int E = kBlock * CH / (64 * NW);  // neighbouring channels of a token that a thread prepares and finishes
  constexpr int V = 2 * NS, PT = 16 / V;       // values of a token, NS of B and of C; tokens in 16 lanes
  constexpr int R = kBlock / PT;
  __shared__ float2 steps[2][kBlock][CH];
  __shared__ float parts[PASS == 1 ? 1 : 2][PASS == 1 ? 1 : NW * P][kBlock][CH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = Q.tiles * A.G;
  // Neighbouring channels share cache lines: workgroups that share an L2, every eighth one, take neighbouring tiles.
  unsigned unit = blockIdx.x;
  if (unit < gridDim.x / (8 * P) * (8 * P)) unit = unit / (8 * P) * (8 * P) + unit % 8 * P + unit / 8 % P;
  const long long j = unit / per;
  const int tg = unit % per, g = tg / Q.tiles, tile = tg - g * Q.tiles;
  int s, a, b;
  long long idx = 0;
  if (PASS != 2 && tg == 0 && j < A.N) {  // one workgroup a sequence raises its flags
    const bool ok = seq_range(A, (int)j, a, b);
    seq_slot(A, (int)j, ok, threadIdx.x == 0);
  }
  if constexpr (PASS == 0) s = (int)j;
  else if (!piece(A, Q.sh, j, lane, s, idx)) return;
  const bool valid = seq_range(A, s, a, b);
  const int slot = seq_slot(A, s, valid, false);
  if (slot < 0) return;
  const int part = wave * P + lane / CH;  // which NS of a channel's states
  const long long len = b - a, p = PASS == 0 ? 0 : idx << Q.sh;
  if (PASS != 0 && p >= len && idx > 0) return;
  const bool ends = PASS == 0 || p + (1LL << Q.sh) >= len;
  const int count = (int)(ends ? len - p : 1LL << Q.sh);
  const int cl = lane % CH, cg = tile * CH + cl;
  const bool live = cg < A.Cg;
  const int c = g * A.Cg + (live ? cg : A.Cg - 1);  // lanes past the group's end repeat its last channel
  const long long so = ((long long)slot * A.C + c) * n + part * NS;
  float h[NS], a2[NS];
  get_states<NS>(A.A + (long long)c * n + part * NS, a2);
#pragma unroll
  for (int i = 0; i < NS; i++) a2[i] *= kLog2e, h[i] = 0;
  if (PASS == 2 && idx > 0) get_states<NS>(Q.last + ((j - idx) * A.C + c) * n + part * NS, h);
  else if (PASS == 2) get_states<NS>(Q.first + ((long long)s * A.C + c) * n + part * NS, h);
  else if (A.S_in && idx == 0) get_states<NS>(A.S_in + so, h);
  if constexpr (PASS == 1) {
    if (idx == 0 && live) put_states<NS>(Q.first + ((long long)s * A.C + c) * n + part * NS, h);
    if (ends) return;
  }
  if constexpr (PASS == 2) {
    for (long long k = 1; k < idx; k++) {
      const long long o = (j - idx + k) * A.C + c;
      const float D = Q.steps[o];
      float e[NS];
      get_states<NS>(Q.last + o * n + part * NS, e);
#pragma unroll
      for (int i = 0; i < NS; i++) h[i] = fmaf(decay(D, a2[i]), h[i], e[i]);
    }
  }
  // this thread's token of a block and its channels there
  const int tok = threadIdx.x / (CH / E), ch = threadIdx.x % (CH / E) * E, cgo = tile * CH + ch;
  const bool mine = cgo < A.Cg;  // a group is whole in eights: all E channels or none
  const int co = g * A.Cg + (mine ? cgo : A.Cg - 8);
  float skip[E], bias[E];
#pragma unroll
  for (int i = 0; i < E; i++) {
    skip[i] = A.D && PASS != 1 ? A.D[co + i] : 0.0f;
    bias[i] = A.bias ? A.bias[co + i] : 0.0f;
  }
  const long long row0 = a + p;
  // Raw values of the next block; x and z of the block before and of this one.  Without a gate z's loads repeat
  // x's, so that no branch stands between the loads.
  const void* zp = A.z ? A.z : A.x;
  constexpr int size = DT == kF32 ? 4 : 2;
  const unsigned ax = (unsigned)A.xs * size, ad = (unsigned)A.dts * size, az = (unsigned)(A.z ? A.zs : A.xs) * size;
  const unsigned ao = (unsigned)A.os * size;  // bytes of a row
  const char* xp = (const char*)A.x + row0 * ax;
  const char* dp = (const char*)A.dt + row0 * ad;
  const char* zq = (const char*)zp + row0 * az;
  char* op = (char*)A.out + row0 * ao;
  Raw<DT, E> rx, rd, rz, x0, z0, x1, z1;
  Raw<DT, 1> rv[R];
  float all[E];
#pragma unroll
  for (int i = 0; i < E; i++) all[i] = 0;
  const int sub = (lane & 15) / V, val = lane % V;  // this lane's token of PT, its value
  const unsigned vs = (unsigned)(val < NS ? A.bs : A.cs) * size;
  const char* vp = (const char*)(val < NS ? A.B : A.Cm) + row0 * vs + (long long)(g * n + part * NS + val % NS) * size;
  auto fetch = [&](int k) {  // blocks in order: the addresses move on
    const int most = count - k * kBlock - 1;  // the last token of the block, at most
    const unsigned t = tok < most ? tok : most;
    rx.load(xp, t * ax + co * size);
    rd.load(dp, t * ad + co * size);
    if (PASS != 1) rz.load(zq, t * az + co * size);
#pragma unroll
    for (int i = 0; i < R; i++) {
      const unsigned t = i * PT + sub < most ? i * PT + sub : most;
      rv[i].load(vp + (unsigned long long)t * vs, 0);
    }
    xp += (long long)ax * kBlock;
    dp += (long long)ad * kBlock;
    zq += (long long)az * kBlock;
    vp += (long long)vs * kBlock;
  };
  auto prepare = [&](int k) {
    float D[E], slope;
#pragma unroll
    for (int i = 0; i < E; i++) D[i] = rd[i] + bias[i];
    if (A.softplus) {
#pragma unroll
      for (int i = 0; i < E; i++) D[i] = step_of(1, D[i], slope);
    }
#pragma unroll
    for (int i = 0; i < E; i++) {
      steps[k & 1][tok][ch + i] = float2{D[i], D[i] * rx[i]};
      if (PASS == 1 && k * kBlock + tok < count) all[i] += D[i];
    }
    x1 = rx;
    z1 = rz;
  };
  auto finish = [&](int k) {
    float y[E];
    loadv<kF32, E>(&parts[k & 1][0][tok][ch], 0, y);
#pragma unroll
    for (int w = 1; w < NW * P; w++) {
      float m[E];
      loadv<kF32, E>(&parts[k & 1][w][tok][ch], 0, m);
#pragma unroll
      for (int i = 0; i < E; i++) y[i] += m[i];
    }
#pragma unroll
    for (int i = 0; i < E; i++) y[i] = fmaf(skip[i], x0[i], y[i]);
    if (A.z) {
#pragma unroll
      for (int i = 0; i < E; i++) y[i] *= z0[i] * sigmoid(z0[i]);
    }
    if (k * kBlock + tok < count && mine) storev<DT, E>(op + (unsigned)(tok * ao + co * size), 0, y);
    op += (long long)ao * kBlock;
  };
  auto one = [&]<int T>(int k, float bc) {  // token T of a block, whose values lie in lanes of `bc`
    const float2 d = steps[k & 1][T][cl];
    float y = 0;
    [&]<int... I>(std::integer_sequence<int, I...>) {
      ((h[I] = fmaf(decay(d.x, a2[I]), h[I], row_lane<T % PT * V + I>(bc) * d.y)), ...);
    }(std::make_integer_sequence<int, NS>{});
    if (PASS != 1) {
      if constexpr (NS == 2) y = row_dot2<T % PT * V + NS>(bc, h);
      else y = row_dot<T % PT * V + NS, false>(y, bc, h);
      if constexpr (NS == 8) y = row_dot<T % PT * V + NS + 4, true>(y, bc, h + 4);
      parts[k & 1][part][T][cl] = y;
    }
  };
  const int blocks = (count + kBlock - 1) / kBlock;
  if (blocks > 0) {
    fetch(0);
    prepare(0);
  }
  for (int k = 0; k < blocks; k++) {
    float bc[R];
#pragma unroll
    for (int i = 0; i < R; i++) bc[i] = rv[i][0];
    if (k + 1 < blocks) fetch(k + 1);
    __syncthreads();
    if (PASS != 1 && k > 0) finish(k - 1);
    x0 = x1;
    z0 = z1;
    const int left = count - k * kBlock;
    [&]<int... T>(std::integer_sequence<int, T...>) {
      if (left >= kBlock) (one.template operator()<T>(k, bc[T / PT]), ...);
      else ((T < left ? one.template operator()<T>(k, bc[T / PT]) : void()), ...);
    }(std::make_integer_sequence<int, kBlock>{});
    if (k + 1 < blocks) prepare(k + 1);
  }
  if (PASS != 1 && blocks > 0) {
    __syncthreads();
    finish(blocks - 1);
  }
  if constexpr (PASS == 1) {
    const long long o = j * A.C + c;
    float* sum = &parts[0][0][0][0];  // [kBlock][CH]
#pragma unroll
    for (int i = 0; i < E; i++) sum[tok * CH + ch + i] = all[i];
    __syncthreads();
    if (wave == 0 && live && lane < CH) {
      float D = sum[lane];
#pragma unroll
      for (int t = 1; t < kBlock; t++) D += sum[t * CH + lane];
      Q.steps[o] = D;
    }
    if (live) put_states<NS>(Q.last + o * n + part * NS, h);
  } else if (ends && A.S_out && live) {
    put_states<NS>(A.S_out + so, h);
  }
}

// Which path a call takes, and its segments (0: none).
struct Path {
  bool blocks;
  int sh;
};
Path path_of(const ScanArgs& a) {
  Path p{a.N > 0 && (long long)a.T >= 16LL * a.N, 0};
  const long long tiles = (a.Cg + 31) / 32 * a.G;
  if (p.blocks && tiles * a.N < 512) {
    int sh = 6;
    while (sh < 30 && ((long long)a.T >> sh) * tiles > 1024) sh++;
    if (a.T / a.N >= 2 << sh) p.sh = sh;
  }
  return p;
}
constexpr size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

template <int DT, int LN>
hipError_t tokens(const ScanArgs& a, hipStream_t s) {
  const int tiles = (a.Cg + 64 / LN - 1) / (64 / LN);
  const long long units = (long long)tiles * a.G * a.N;
  hipLaunchKernelGGL((k_scan_tokens<DT, LN>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, a, tiles);
  return hipGetLastError();
}

template <int DT, int NS, int CH, int NW>
hipError_t blocks(const ScanArgs& a, int sh, hipStream_t s) {
  Segments q{(a.Cg + CH - 1) / CH, sh, nullptr, nullptr, nullptr};
  const long long per = (long long)q.tiles * a.G;
  if (!sh) {
    hipLaunchKernelGGL((k_scan_run<DT, NS, CH, NW, 0>), dim3((unsigned)(per * a.N)), dim3(64 * NW), 0, s, a, q);
    return hipGetLastError();
  }
  const long long m = pieces(a, sh);
  q.last = (float*)a.ws;
  q.steps = (float*)(a.ws + up((size_t)m * a.C * a.n * 4));
  q.first = (float*)((char*)q.steps + up((size_t)m * a.C * 4));
  hipLaunchKernelGGL((k_scan_run<DT, NS, CH, NW, 1>), dim3((unsigned)(per * m)), dim3(64 * NW), 0, s, a, q);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL((k_scan_run<DT, NS, CH, NW, 2>), dim3((unsigned)(per * m)), dim3(64 * NW), 0, s, a, q);
  return hipGetLastError();
}

template <int DT>
hipError_t by_states(const ScanArgs& a, hipStream_t s) {
  const Path p = path_of(a);
  if (!p.blocks) {
    return a.n == 8 ? tokens<DT, 2>(a, s)
                    : a.n == 16 ? tokens<DT, 4>(a, s) : a.n == 32 ? tokens<DT, 8>(a, s) : tokens<DT, 16>(a, s);
  }
  return a.n == 8    ? blocks<DT, 2, 32, 2>(a, p.sh, s)
         : a.n == 16 ? blocks<DT, 2, 32, 4>(a, p.sh, s)
         : a.n == 32 ? blocks<DT, 4, 32, 4>(a, p.sh, s)
                     : blocks<DT, 8, 32, 4>(a, p.sh, s);
}

}  // namespace

size_t scan_forward_bytes(const ScanArgs& a) {
  const Path p = path_of(a);
  if (!p.sh) return 0;
  const size_t m = (size_t)pieces(a, p.sh);
  return up(m * a.C * a.n * 4) + up(m * a.C * 4) + up((size_t)a.N * a.C * a.n * 4);
}

hipError_t launch_scan(const ScanArgs& a, hipStream_t s) {
  if (a.N <= 0) return hipSuccess;
  return a.dtype == kF32 ? by_states<kF32>(a, s) : a.dtype == kBF16 ? by_states<kBF16>(a, s) : by_states<kF16>(a, s);
}

}  // namespace stepq
