// stepq_scan_grad.hip -- gradient of the selective scan.  With e_t = dout_t z sigmoid(z), a_t = exp(D_t A) and
// g_t the gradient of h_t:
//   g_t = C_t e_t + a_{t+1} g_{t+1} (behind the last token: the last state's gradient)
//   dC_t = sum_c e_t h_t;  dB_t = sum_c g_t D_t x_t;  dx_t = D_t sum_n g_t B_t + D e_t
//   dD_t = sum_n g_t (A a_t h_{t-1} + B_t x_t), ddt_t = dD_t sigmoid(dt + bias);  dA = sum_t D_t g_t a_t h_{t-1}
//   dz_t = dout_t (C_t . h_t + D x_t) (z sigmoid(z))';  dD = sum_t e_t x_t;  dS_in = a_1 g_1
// The forward pass keeps the states before every block of 16 tokens (k_scan_run, PASS 3); the reverse pass runs a
// block's tokens again from them, with the states and decays in registers, and then back.
//
// Bound by vector issue: five slots of 64 lanes a state and token to run it again, nine back, 1.5 for the sums over channels
// that dB and dC are, 1 for those over states; with the rest 25.8 (counted: 216 M for 8,192 tokens x 4,096 channels
// x 16 states).  There the states' pass takes 136-150 us, the way back 500-540 (78% of the issue while a CU is busy), the tiles'
// sums 23: 626 us in all.  That call has 512 workgroups, two a CU, so two waves a SIMD, where 16 states leave room for three of 16-bit
// rows (165 registers, 48 KB of LDS); 32 states leave room for two, of binary32 rows for one (256 registers and some accumulation
// registers: 3,001 tokens x 1,536 channels 306 us against 229 of 16-bit rows).  Sums over channels: two steps across
// lanes that also deal four values out to four lanes each (six instructions for four values, 16 a plain tree would
// take), the rest through LDS.  One block of instructions for what crosses lanes, ordered so that no wait states are needed
// inside: 683 -> 647 us.
#include "stepq_scan_block.h"

namespace stepq {
namespace {

// Workspace behind the segments': the kept states; partial dB and dC of every tile of channels; partial dA, dD and
// dbias of every segment; for segments, the gradients before them from zero behind them.
struct Space {
  Segments q;
  long long segs, row;  // segments, or sequences where there are none; floats of a row of dA | dD | dbias
  float* bc;
  float* par;
  float* back;
};
size_t space(const ScanArgs& a, char* ws, Space* w) {
  char* p;
  w->q = lay_segments(a, segments_of(a, kLeastBackward), ws, &p);
  const int sh = w->q.sh;
  w->segs = sh ? pieces(a, sh) : a.N;
  w->row = (long long)a.C * a.n + 2 * a.C;
  w->q.kept = (float*)p;
  p += up((size_t)pieces(a, 4) * w->q.tiles * a.G * 32 * a.n * 4);
  w->bc = (float*)p;
  p += up((size_t)w->q.tiles * a.T * a.G * a.n * 8);
  w->par = (float*)p;
  p += up((size_t)w->segs * w->row * 4);
  w->back = (float*)p;
  if (sh) p += up((size_t)w->segs * a.C * a.n * 4);
  return (size_t)(p - ws);
}

// What a token adds to NS states' gradients and takes from them across lanes.  With B and C in lanes I .. and I + NS ..
// of each 16 lanes' b:
//   g_i += C_i e;  y = sum_i C_i h_i, gB = sum_i B_i g_i, of which `both` is the sums of the wave's halves: y's in the
//   first 32 lanes, gB's in the others;
//   q: four values (g D x of two states, e h of the same) summed over every fourth of 16 lanes: the first four lanes
//   get the first value's sums (of lanes 0, 4, 8, 12; 1, 5, ..), the next four the second's, and so on.  Each step
//   adds a lane's value to that of the lane eight, then four, away, and writes only the lanes that go on with this value.
// One block of instructions, ordered so that none reads across lanes what one of the two before it wrote (two wait states; the
// s_nop is for b).
template <int I>
__device__ __forceinline__ void across2(float b, float e, float dx, const float* h, float* g, float& both, float* q) {
  float y, gB, u0, u1, u2, u3, r0, r1;
  asm("s_nop 1\n\t"
      "v_fmac_f32_dpp %0, %11, %12 row_newbcast:%18 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %11, %12 row_newbcast:%19 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %2, %11, %14 row_newbcast:%18 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %3, %11, %0 row_newbcast:%16 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32 %4, %0, %13\n\t"
      "v_fmac_f32_dpp %2, %11, %15 row_newbcast:%19 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32 %5, %1, %13\n\t"
      "v_fmac_f32_dpp %3, %11, %1 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32 %6, %12, %14\n\t"
      "v_mul_f32 %7, %12, %15\n\t"
      "v_add_f32_dpp %8, %4, %4 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %9, %5, %5 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_permlane32_swap_b32 %2, %3\n\t"
      "v_add_f32_dpp %8, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %9, %7, %7 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32 %2, %2, %3\n\t"
      "s_nop 0\n\t"
      "v_add_f32_dpp %10, %8, %8 row_ror:12 row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %10, %9, %9 row_ror:4 row_mask:0xf bank_mask:0xa"
      : "+&v"(g[0]), "+&v"(g[1]), "=&v"(y), "=&v"(gB), "=&v"(u0), "=&v"(u1), "=&v"(u2), "=&v"(u3), "=&v"(r0), "=&v"(r1),
        "=&v"(q[0])
      : "v"(b), "v"(e), "v"(dx), "v"(h[0]), "v"(h[1]), "n"(I), "n"(I + 1), "n"(I + 2), "n"(I + 3));
  both = y;
}

template <int I>
__device__ __forceinline__ void across4(float b, float e, float dx, const float* h, float* g, float& both, float* q) {
  float y, gB, u0, u1, u2, u3, r0, r1;
  asm("s_nop 1\n\t"
      "v_fmac_f32_dpp %0, %6, %7 row_newbcast:%16 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %6, %7 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %2, %6, %7 row_newbcast:%18 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %3, %6, %7 row_newbcast:%19 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %4, %6, %8 row_newbcast:%16 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %5, %6, %0 row_newbcast:%12 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %4, %6, %9 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %5, %6, %1 row_newbcast:%13 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %4, %6, %10 row_newbcast:%18 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %5, %6, %2 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %4, %6, %11 row_newbcast:%19 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %5, %6, %3 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1\n\t"
      "v_permlane32_swap_b32 %4, %5\n\t"
      "v_add_f32 %4, %4, %5"
      : "+&v"(g[0]), "+&v"(g[1]), "+&v"(g[2]), "+&v"(g[3]), "=&v"(y), "=&v"(gB)
      : "v"(b), "v"(e), "v"(h[0]), "v"(h[1]), "v"(h[2]), "v"(h[3]), "n"(I), "n"(I + 1), "n"(I + 2), "n"(I + 3), "n"(I + 4),
        "n"(I + 5), "n"(I + 6), "n"(I + 7));
  both = y;
#pragma unroll
  for (int k = 0; k < 2; k++)
    asm("v_mul_f32 %0, %7, %9\n\t"
        "v_mul_f32 %1, %8, %9\n\t"
        "v_mul_f32 %2, %10, %11\n\t"
        "v_mul_f32 %3, %10, %12\n\t"
        "v_add_f32_dpp %4, %0, %0 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %4, %2, %2 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %5, %1, %1 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %5, %3, %3 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %6, %4, %4 row_ror:12 row_mask:0xf bank_mask:0x5\n\t"
        "s_nop 0\n\t"
        "v_add_f32_dpp %6, %5, %5 row_ror:4 row_mask:0xf bank_mask:0xa"
        : "=&v"(u0), "=&v"(u1), "=&v"(u2), "=&v"(u3), "=&v"(r0), "=&v"(r1), "=&v"(q[k])
        : "v"(g[2 * k]), "v"(g[2 * k + 1]), "v"(dx), "v"(e), "v"(h[2 * k]), "v"(h[2 * k + 1]));
}

// v += (lane I of each 16 lanes' b) * e
template <int I>
__device__ __forceinline__ void row_fmac(float& v, float b, float e) {
  asm("s_nop 1\n\tv_fmac_f32_dpp %0, %1, %2 row_newbcast:%3 row_mask:0xf bank_mask:0xf" : "+v"(v) : "v"(b), "v"(e), "n"(I));
}

// Of two values the sums of a wave's halves: u's in the first 32 lanes, v's in the others.
__device__ __forceinline__ float half_sums(float u, float v) {
  float r;
  asm("s_nop 1\n\tv_permlane32_swap_b32 %1, %2\n\tv_add_f32 %0, %1, %2" : "=&v"(r), "+v"(u), "+v"(v));
  return r;
}

// PASS 0: whole sequences.  1: the gradient before a segment from zero behind it.  2: segments.
template <int DT, int NS, int NW, int PASS>
__global__ __launch_bounds__(64 * NW) void k_scan_back(ScanArgs A, Space S) {
  constexpr int CH = 32, P = 2, n = NS * P * NW;
  constexpr int E = kBlock * CH / (64 * NW);
  constexpr int V = 2 * NS, PT = 16 / V, R = kBlock / PT;
  constexpr bool OUT = PASS != 1;
  __shared__ f4 steps[kBlock][CH];                         // D, D x, e
  __shared__ float parts[OUT ? 3 : 1][NW][kBlock][CH];     // C . h, B . g, A . (g a h)
  __shared__ float quarters[OUT ? NS / 2 : 1][kBlock][NW][64];  // of g D x and e h, by state
  const Segments& Q = S.q;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = Q.tiles * A.G;
  const unsigned unit = neighbours(blockIdx.x, P);
  const long long j = unit / per;
  const int tg = unit % per, g = tg / Q.tiles, tile = tg - g * Q.tiles;
  const int sh = PASS == 0 ? 0 : Q.sh;
  Place W;
  const bool here = place(A, sh, Q.over, j, false, lane, W);
  const int part = wave * P + lane / CH;
  const int cl = lane % CH, cg = tile * CH + cl;
  const bool live = cg < A.Cg;
  const int c = g * A.Cg + (live ? cg : A.Cg - 1);
  float* par = S.par + j * S.row;
  if (!here) {  // nothing to add
    if (OUT && live) {
#pragma unroll
      for (int i = 0; i < NS; i++) par[(long long)c * n + part * NS + i] = 0;
      if (part < 2) par[(long long)A.C * n + (long long)part * A.C + c] = 0;
    }
    return;
  }
  if (PASS == 1 && W.idx == 0) return;
  const int count = W.count;
  const long long so = ((long long)W.s * A.C + c) * n + part * NS;
  float a1[NS], a2[NS], G[NS], dA[NS];
  get_states<NS>(A.A + (long long)c * n + part * NS, a1);
#pragma unroll
  for (int i = 0; i < NS; i++) a2[i] = a1[i] * kLog2e, G[i] = 0, dA[i] = 0;
  if (A.dS_out && (OUT || W.ends)) get_states<NS>(A.dS_out + so, G);
  if (PASS == 2 && !W.ends) {  // what the segments behind this one make of it, from the last one on
    const long long last = (W.len - 1) >> sh;
    const float* back = S.back + (long long)part * NS;
    // the last segment's already holds the last state's gradient
    get_states<NS>(back + ((W.more + last) * A.C + c) * n, G);
#pragma unroll 4
    for (long long k = last - 1; k > W.idx; k--) {
      const long long o = (W.more + k) * A.C + c;
      const float D = Q.steps[o];
      float e[NS];
      get_states<NS>(back + o * n, e);
#pragma unroll
      for (int i = 0; i < NS; i++) G[i] = fmaf(decay(D, a2[i]), G[i], e[i]);
    }
  }
  // this thread's token of a block and its channels there
  const int tok = threadIdx.x / (CH / E), ch = threadIdx.x % (CH / E) * E, cgo = tile * CH + ch;
  const bool mine = cgo < A.Cg;  // a group is whole in eights: all E channels or none
  const int co = g * A.Cg + (mine ? cgo : A.Cg - 8);
  float skip[E], bias[E], dD[E], dbias[E];
#pragma unroll
  for (int i = 0; i < E; i++) {
    skip[i] = A.D ? A.D[co + i] : 0.0f;
    bias[i] = A.bias ? A.bias[co + i] : 0.0f;
    dD[i] = dbias[i] = 0;
  }
  constexpr int size = DT == kF32 ? 4 : 2;
  const void* zp = A.z ? A.z : A.x;
  const unsigned ax = (unsigned)A.xs * size, ad = (unsigned)A.dts * size, az = (unsigned)(A.z ? A.zs : A.xs) * size;
  const unsigned au = (unsigned)A.os * size;
  // Read as one value of the wave: the compiler arranges the loop of PASS 2 as it does that of PASS 0 (4% faster than without).
  const int blocks = __builtin_amdgcn_readfirstlane((count + kBlock - 1) / kBlock);
  const long long kept0 = OUT ? first_block(A, W) : 0;
  Raw<DT, E> rx, rd, rz, ru;
  Raw<DT, 1> rv[R];
  float hk[NS];
  const int sub = (lane & 15) / V, val = lane % V;  // this lane's token of PT, its value
  const unsigned vs = (unsigned)(val < NS ? A.bs : A.cs) * size;
  const char* vp = (const char*)(val < NS ? A.B : A.Cm) + (long long)(g * n + part * NS + val % NS) * size;
  // offsets from a block's first row, as they are where the block is whole
  const unsigned ox = tok * ax + co * size, od = tok * ad + co * size, oz = tok * az + co * size, ou = tok * au + co * size;
  unsigned ov[R];
#pragma unroll
  for (int i = 0; i < R; i++) ov[i] = (i * PT + sub) * vs;
  auto fetch = [&](int k) {
    const int most = count - k * kBlock - 1;
    const long long row = W.row0 + (long long)k * kBlock;
    const char *xp = (const char*)A.x + row * ax, *dp = (const char*)A.dt + row * ad, *zq = (const char*)zp + row * az;
    const char *up = (const char*)A.d_out + row * au, *v = vp + row * vs;
    if (most >= kBlock - 1) {
      rx.load(xp + ox);
      rd.load(dp + od);
      rz.load(zq + oz);
      ru.load(up + ou);
#pragma unroll
      for (int i = 0; i < R; i++) rv[i].load(v + ov[i]);
    } else {
      const unsigned t = tok < most ? tok : most;
      rx.load(xp + (t * ax + co * size));
      rd.load(dp + (t * ad + co * size));
      rz.load(zq + (t * az + co * size));
      ru.load(up + (t * au + co * size));
#pragma unroll
      for (int i = 0; i < R; i++) {
        const unsigned t = i * PT + sub < most ? i * PT + sub : most;
        rv[i].load(v + t * vs);
      }
    }
    if (OUT) get_states<NS>(Q.kept + ((kept0 + k) * per + tg) * (64 * NW * NS) + threadIdx.x * NS, hk);
  };
  // of the block that runs: raw values, slopes of the steps, and z's part of the output
  Raw<DT, E> x0, z0, u0;
  float D0[E], slope0[E], e0[E], s0[E];
  auto prepare = [&](int k) {
    x0 = rx;
    z0 = rz;
    u0 = ru;
#pragma unroll
    for (int i = 0; i < E; i++) D0[i] = rd[i] + bias[i], slope0[i] = 1, e0[i] = ru[i];
    if (A.softplus) {
#pragma unroll
      for (int i = 0; i < E; i++) D0[i] = step_of<DT>(1, D0[i], slope0[i]);
    }
    if (A.z) {
#pragma unroll
      for (int i = 0; i < E; i++) {
        s0[i] = sigmoid<DT>(z0[i]);
        e0[i] *= z0[i] * s0[i];
      }
    }
    const bool in = k * kBlock + tok < count && mine;  // a token behind the last, a channel behind the group's: no step
#pragma unroll
    for (int i = 0; i < E; i++) {
      steps[tok][ch + i] = in ? f4{D0[i], D0[i] * x0[i], e0[i], 0} : f4{0, 0, 0, 0};
    }
  };
  const int b4 = threadIdx.x % 4, pt = threadIdx.x / 4 % (NW * P), tk = threadIdx.x / (4 * NW * P);
  float* bcp = S.bc + (((long long)tile * A.T + W.row0 + tk) * A.G + g) * (2 * n) + (b4 < 2 ? 0 : n) + pt * NS + b4 % 2;
  auto finish = [&](int k) {
    const int t = k * kBlock + tok;
    float y[E], gB[E], gA[E], dx[E], ddt[E], dz[E];
#pragma unroll
    for (int i = 0; i < E; i++) y[i] = gB[i] = gA[i] = 0;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      float m[E];
      loadv<kF32, E>(&parts[0][w][tok][ch], 0, m);
#pragma unroll
      for (int i = 0; i < E; i++) y[i] += m[i];
      loadv<kF32, E>(&parts[1][w][tok][ch], 0, m);
#pragma unroll
      for (int i = 0; i < E; i++) gB[i] += m[i];
      loadv<kF32, E>(&parts[2][w][tok][ch], 0, m);
#pragma unroll
      for (int i = 0; i < E; i++) gA[i] += m[i];
    }
    if (t < count && mine) {
      const long long base = (W.row0 + (long long)k * kBlock) * A.C * size;
      const unsigned o = (unsigned)(tok * A.C + co) * size;
#pragma unroll
      for (int i = 0; i < E; i++) {
        dx[i] = fmaf(D0[i], gB[i], skip[i] * e0[i]);
        ddt[i] = fmaf(x0[i], gB[i], gA[i]) * slope0[i];
        dD[i] = fmaf(e0[i], x0[i], dD[i]);
        dbias[i] += ddt[i];
      }
      storev<DT, E>((char*)A.dx + base + o, 0, dx);
      storev<DT, E>((char*)A.ddt + base + o, 0, ddt);
      if (A.z) {
#pragma unroll
        for (int i = 0; i < E; i++) {
          dz[i] = u0[i] * fmaf(skip[i], x0[i], y[i]) * fmaf(z0[i] * s0[i], 1.0f - s0[i], s0[i]);
        }
        storev<DT, E>((char*)A.dz + base + o, 0, dz);
      }
    }
    // dB and dC of this tile: a thread adds up one value of one part for every eighth token
    const int most = count - k * kBlock;
    float* to = bcp + (long long)k * kBlock * (2 * n * A.G);
#pragma unroll
    for (int r = 0; r < 2; r++) {
#pragma unroll
      for (int v = 0; v < NS / 2; v++) {
        const float* q = &quarters[v][tk + 8 * r][pt / P][pt % P * 32 + 4 * b4];
        float m0[4], m1[4];
        loadn<kF32, 4>(q, 0, m0);
        loadn<kF32, 4>(q, 16, m1);
        const float sum = ((m0[0] + m0[1]) + (m0[2] + m0[3])) + ((m1[0] + m1[1]) + (m1[2] + m1[3]));
        if (tk + 8 * r < most) to[8 * r * (2 * n * A.G) + 2 * v] = sum;
      }
    }
  };
  if (blocks > 0) {
    fetch(blocks - 1);
    prepare(blocks - 1);
  }
  for (int k = blocks - 1; k >= 0; k--) {
    float bc[R], h[NS], al[OUT ? kBlock : 1][NS], was[OUT ? kBlock : 1][NS], cA[NS];
    const int most = count - k * kBlock - 1;
#pragma unroll
    for (int i = 0; i < R; i++) bc[i] = i * PT + sub <= most ? rv[i][0] : 0.0f;
#pragma unroll
    for (int i = 0; i < NS; i++) h[i] = hk[i], cA[i] = 0;
    if (k > 0) fetch(k - 1);
    __syncthreads();
    if constexpr (OUT) {
      unrolled<kBlock>([&](auto t) {
        constexpr int T = t;
        const float2 d = *(const float2*)&steps[T][cl];
        unrolled<NS>([&](auto i) {
          al[T][i] = decay(d.x, a2[i]);
          was[T][i] = h[i];
          h[i] = fmaf(al[T][i], h[i], row_lane<T % PT * V + i>(bc[T / PT]) * d.y);
        });
      });
    }
    float gA_odd = 0;
    unrolled<kBlock>([&](auto t) {
      constexpr int T = kBlock - 1 - t, base = T % PT * V;
      const float b = bc[T / PT];
      const f4 d = steps[T][cl];
      if constexpr (OUT) {
        float both, q[NS / 2], gA = 0;
        if constexpr (NS == 2) across2<base>(b, d[2], d[1], h, G, both, q);
        else across4<base>(b, d[2], d[1], h, G, both, q);
        parts[lane / CH][wave][T][cl] = both;
#pragma unroll
        for (int v = 0; v < NS / 2; v++) quarters[v][T][wave][lane] = q[v];
#pragma unroll
        for (int i = 0; i < NS; i++) {
          G[i] *= al[T][i];
          const float w = G[i] * was[T][i];
          gA = fmaf(a1[i], w, gA);
          cA[i] = fmaf(d[0], w, cA[i]);
          h[i] = was[T][i];
        }
        if constexpr (T % 2) gA_odd = gA;
        else parts[2][wave][T + lane / CH][cl] = half_sums(gA, gA_odd);
      } else {
        unrolled<NS>([&](auto i) {
          row_fmac<base + NS + i>(G[i], b, d[2]);
          G[i] *= decay(d[0], a2[i]);
        });
      }
    });
#pragma unroll
    for (int i = 0; i < NS; i++) dA[i] += cA[i];
    __syncthreads();
    if (OUT) finish(k);
    if (k > 0) prepare(k - 1);
  }
  if constexpr (PASS == 1) {
    if (live) put_states<NS>(S.back + (j * A.C + c) * n + part * NS, G);
  } else {
    if (live) {
      if (W.idx == 0 && A.dS_in) put_states<NS>(A.dS_in + so, G);
      put_states<NS>(par + (long long)c * n + part * NS, dA);
    }
    float* sum = &parts[0][0][0][0];  // [2][kBlock][CH]; parts is large enough, its last reads are behind the next barrier
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; i++) {
      sum[tok * CH + ch + i] = dD[i];
      sum[(kBlock + tok) * CH + ch + i] = dbias[i];
    }
    __syncthreads();
    if (wave == 0 && live) {  // one half of the wave adds dD up, the other dbias
      float m = 0;
#pragma unroll
      for (int t = 0; t < kBlock; t++) m += sum[(lane / CH * kBlock + t) * CH + cl];
      par[(long long)A.C * n + (long long)(lane / CH) * A.C + c] = m;
    }
  }
}

// dB and dC of every token of a sequence: the tiles' partial sums in order.
template <int DT>
__global__ __launch_bounds__(256) void k_scan_bc(ScanArgs A, Space W) {
  const long long row = 2LL * A.G * A.n, i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= row * A.T) return;
  const int t = (int)(i / row), k = (int)(i % row), g = k / (2 * A.n), m = k % (2 * A.n);
  if (A.cu) {  // rows of no sequence are left alone: the last sequence that begins at or before t holds it, or none does
    int lo = 0, hi = A.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (A.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    int t0, t1;
    if (!seq_range(A, lo, t0, t1) || t < t0 || t >= t1) return;
  }
  const float* p = W.bc + i;
  float acc = 0;
#pragma unroll 8
  for (int q = 0; q < W.q.tiles; q++) acc += p[q * row * A.T];
  const long long o = ((long long)t * A.G + g) * A.n + (m < A.n ? m : m - A.n);
  storen<DT, 1>(m < A.n ? A.dB : A.dC, o, &acc);
}

template <int DT, int NS, int NW>
hipError_t launch(const ScanArgs& a, const Space& w, hipStream_t s) {
  const dim3 grid((unsigned)(w.segs * w.q.tiles * a.G)), block(64 * NW);
  if (w.q.sh) {
    hipLaunchKernelGGL((k_scan_run<DT, NS, 32, NW, 1>), grid, block, 0, s, a, w.q);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL((k_scan_back<DT, NS, NW, 1>), grid, block, 0, s, a, w);
    if (hipError_t e = hipGetLastError()) return e;
  }
  hipLaunchKernelGGL((k_scan_run<DT, NS, 32, NW, 3>), grid, block, 0, s, a, w.q);
  if (hipError_t e = hipGetLastError()) return e;
  if (w.q.sh) hipLaunchKernelGGL((k_scan_back<DT, NS, NW, 2>), grid, block, 0, s, a, w);
  else hipLaunchKernelGGL((k_scan_back<DT, NS, NW, 0>), grid, block, 0, s, a, w);
  if (hipError_t e = hipGetLastError()) return e;
  const long long all = 2LL * a.G * a.n * a.T;
  if (all) hipLaunchKernelGGL((k_scan_bc<DT>), dim3((unsigned)((all + 255) / 256)), dim3(256), 0, s, a, w);
  return hipGetLastError();
}

template <int DT>
hipError_t by_states(const ScanArgs& a, const Space& w, hipStream_t s) {
  return a.n == 8    ? launch<DT, 2, 2>(a, w, s)
         : a.n == 16 ? launch<DT, 2, 4>(a, w, s)
         : a.n == 32 ? launch<DT, 4, 4>(a, w, s)
                     : launch<DT, 4, 8>(a, w, s);
}

}  // namespace

size_t scan_backward_bytes(const ScanArgs& a) {
  Space w;
  return space(a, nullptr, &w);
}

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
  Space w;
  space(a, a.ws, &w);
  if (a.N > 0) {
    const hipError_t e = a.dtype == kF32    ? by_states<kF32>(a, w, s)
                         : a.dtype == kBF16 ? by_states<kBF16>(a, w, s)
                                            : by_states<kF16>(a, w, s);
    if (e) return e;
  }
  SumArgs m{w.par, (int)w.segs, w.row, (long long)a.C * a.n, a.C, a.dA, a.dD, a.dbias};
  return launch_sum(m, s);
}

}  // namespace stepq
