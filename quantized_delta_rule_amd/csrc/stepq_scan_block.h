// stepq_scan_block.h -- the scan in blocks of 16 tokens: the kernel of its forward pass, which the gradient runs for the
// states that it needs, and the pieces that the gradient's own kernel shares with it.
#pragma once
#include <utility>

#include "stepq_scan.h"

namespace stepq {
namespace {

using namespace lay;

// ---------------------------------------------------------------------------------------------
// Blocks of tokens: a workgroup takes CH channels of a sequence, or of one of its segments.  64 / CH parts of a wave and
// the NW waves share a channel's states out, NS each, so that 16 neighbouring lanes have the same B and C of a
// token: they hold the values of a token or more, and an instruction takes one of them for all 16 lanes by itself
// (row broadcast of its operand).  For each block of 16 tokens the waves first turn raw steps into (D, D x) in LDS,
// a few channels each, then run all of them on their states, and add their parts of C . h up through LDS.
//
// Bound by vector issue: a state and token take an exponential (two slots), the argument's product, two multiply-adds and a
// product, six slots; steps, gates and the parts' sums make it 9.7 (counted: 163 M slots of 64 lanes for 16,381 tokens x
// 4,096 channels x 16 states).  Eight ragged prompts of 16,381 x 4,096 take 337 us, 1.9 GHz of full issue on every SIMD
// (85% of the issue while a CU is busy); one sequence of 16,384 x 2,048 takes 254 us for its 142 M slots, 2.2 GHz of it (98%, the two
// passes 116 and 168 us under a tracer, where CUs run at 2.0 GHz): slots bind, not the prompts' unequal lengths.  What the
// layout was worth when it was chosen (us, 16,381 x 4,096 / 16,384 x 2,048): B and C through scalar loads 876 / 443 (their wait stops every LDS read too), row broadcasts 581 /
// 310; a thread's elements side by side, not 16 lanes apart, 510 / 281; 32 channels a workgroup, not 64, 355 / 293; two
// states a lane, not four, 329 / 272; 16 channels 457 / 337.
// ---------------------------------------------------------------------------------------------

constexpr int kBlock = 16;

// f of the constants 0 .. N - 1, one after the other.
template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
  (std::make_integer_sequence<int, N>{});
}

// Long sequences run in segments of 2^sh tokens at once: first each segment's last state from the zero state and the
// sum of its steps, then, from what the segments before it leave, the segment itself.
struct Segments {
  int tiles;    // of CH channels, in a group
  int sh;
  long long over;  // sequences longer than this are cut, the others run whole (in their first segment's place)
  float* last;  // [segments, C, n]: the first of a sequence from its state, the others from zero
  float* steps; // [segments, C]
  float* first; // [N, C, n]: the first states of sequences of several segments (S_out may be S_in)
  float* kept;  // states before every block of 16 tokens, as the kernel's lanes hold them (PASS 3)
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

// Segments are numbered by sequence first: segment 0 of sequence s is number s, so that the workgroups of sequences that are not
// cut lie side by side as they would without segments (the four sequences of 2,048 tokens x 2,048 channels that take 142 us whole
// take 238 where their workgroups lie apart: two meet on a CU, none on others).  The later ones follow: those of
// sequence s from number N + (cu[s] >> sh) on, which no two sequences share, since a sequence has (len - 1) >> sh of them.
// Sequence and segment of the later number e; false where no sequence begins before it.  The whole wave asks for one e.
__device__ __forceinline__ bool later(const ScanArgs& A, int sh, long long e, int lane, int& s, long long& idx) {
  if (!A.cu) {
    const long long more = (A.T / A.N - 1) >> sh;  // of each sequence; no call has e where it is zero
    s = (int)(e / more);
    idx = e - s * more + 1;
    return true;
  }
  long long lo = 0, n = A.N;
  do {  // 64 sequences at once, as `piece` does
    const long long step = (n + 63) >> 6, at = lo + lane * step;
    const int k = __popcll(__ballot(lane * step < n && A.cu[at] >> sh <= e));
    if (k == 0) return false;
    lo += (k - 1) * step;
    n = n - (k - 1) * step < step ? n - (k - 1) * step : step;
  } while (n > 1);
  s = __builtin_amdgcn_readfirstlane((int)lo);
  idx = e - (A.cu[s] >> sh) + 1;
  return true;
}

// Segment j, or sequence j where there are none: its sequence, place, rows and channels.  False: nothing to do.
struct Place {
  int s, slot, count;     // sequence, state index, tokens
  long long idx, len, p;  // segment of the sequence, the sequence's length, position in it
  long long row0;         // first row
  long long more;         // number of the sequence's segment k > 0, less k
  bool ends;              // the sequence's last segment
};
__device__ __forceinline__ bool place(const ScanArgs& A, int sh, long long over, long long j, bool report, int lane, Place& Q) {
  int a, b;
  if (report && j < A.N) {
    const bool ok = seq_range(A, (int)j, a, b);
    seq_slot(A, (int)j, ok, lane == 0);
  }
  Q.idx = 0;
  if (!sh || j < A.N) Q.s = (int)j;
  else if (!later(A, sh, j - A.N, lane, Q.s, Q.idx)) return false;
  const bool valid = seq_range(A, Q.s, a, b);
  Q.slot = seq_slot(A, Q.s, valid, false);
  Q.len = b - a;
  const bool cut = sh && Q.len > over;
  if (!cut && Q.idx > 0) return false;
  Q.p = cut ? Q.idx << sh : 0;
  Q.ends = !cut || Q.p + (1LL << sh) >= Q.len;
  Q.count = (int)(Q.ends ? Q.len - Q.p : 1LL << sh);
  Q.row0 = a + Q.p;
  Q.more = A.N - 1 + (A.cu ? (long long)a >> sh : Q.s * ((Q.len - 1) >> sh));
  return Q.slot >= 0 && (Q.p < Q.len || Q.idx == 0) && Q.len >= A.split;
}

// Number of a segment's first block of 16 tokens among all sequences' (pieces of 2^4 tokens).
__device__ __forceinline__ long long first_block(const ScanArgs& A, const Place& W) {
  const long long row = W.row0 - W.p;  // the sequence's first
  return (A.cu ? (row >> 4) + W.s : (long long)W.s * (W.len > 16 ? (W.len + 15) >> 4 : 1)) + (W.p >> 4);
}

// Neighbouring channels share cache lines: workgroups that share an L2, every eighth one, take P neighbouring tiles.
__device__ __forceinline__ unsigned neighbours(unsigned unit, unsigned P) {
  if (unit >= gridDim.x / (8 * P) * (8 * P)) return unit;
  return unit / (8 * P) * (8 * P) + unit % 8 * P + unit / 8 % P;
}

// PASS 0: a whole sequence.  1: a segment's last state and steps.  2: a segment.  3: either, for the states before
// its blocks alone.
template <int DT, int NS, int CH, int NW, int PASS>
__global__ __launch_bounds__(64 * NW) void k_scan_run(ScanArgs A, Segments Q) {
  constexpr int P = 64 / CH, n = NS * P * NW;  // parts of a channel's states in a wave
  constexpr int E = kBlock * CH / (64 * NW);  // neighbouring channels of a token that a thread prepares and finishes
  constexpr int V = 2 * NS, PT = 16 / V;       // values of a token, NS of B and of C; tokens in 16 lanes
  constexpr int R = kBlock / PT;
  constexpr bool OUT = PASS == 0 || PASS == 2;
  __shared__ float2 steps[2][kBlock][CH];
  __shared__ float parts[OUT ? 2 : 1][OUT ? NW * P : 1][kBlock][CH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = Q.tiles * A.G;
  const unsigned unit = neighbours(blockIdx.x, P);
  const long long j = unit / per;
  const int tg = unit % per, g = tg / Q.tiles, tile = tg - g * Q.tiles;
  const int sh = PASS == 0 ? 0 : Q.sh;
  Place W;
  if (!place(A, sh, Q.over, j, (PASS < 2 || (PASS == 3 && !sh)) && tg == 0 && threadIdx.x < 64, lane, W)) return;
  const int count = W.count, s = W.s;
  const long long idx = W.idx;
  const bool ends = W.ends;
  if (PASS == 1 && ends) return;  // nothing comes behind
  const int part = wave * P + lane / CH;  // which NS of a channel's states
  const int cl = lane % CH, cg = tile * CH + cl;
  const bool live = cg < A.Cg;
  const int c = g * A.Cg + (live ? cg : A.Cg - 1);  // lanes past the group's end repeat its last channel
  const long long so = ((long long)W.slot * A.C + c) * n + part * NS;
  float h[NS], a2[NS];
  get_states<NS>(A.A + (long long)c * n + part * NS, a2);
#pragma unroll
  for (int i = 0; i < NS; i++) a2[i] *= kLog2e, h[i] = 0;
  if (PASS < 2 || !sh || (idx == 0 && ends)) {  // a sequence of one segment is its own workgroup's alone
    if (A.S_in && idx == 0) get_states<NS>(A.S_in + so, h);
  } else if (idx > 0) {
    get_states<NS>(Q.last + ((long long)s * A.C + c) * n + part * NS, h);
  } else {
    get_states<NS>(Q.first + ((long long)s * A.C + c) * n + part * NS, h);
  }
  if constexpr (PASS == 1) {
    if (idx == 0 && live) put_states<NS>(Q.first + ((long long)s * A.C + c) * n + part * NS, h);
  }
  if (PASS >= 2) {
#pragma unroll 4
    for (long long k = 1; k < idx; k++) {
      const long long o = (W.more + k) * A.C + c;
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
    skip[i] = A.D && OUT ? A.D[co + i] : 0.0f;
    bias[i] = A.bias ? A.bias[co + i] : 0.0f;
  }
  const long long row0 = W.row0;
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
  // offsets from a block's first row, as they are where the block is whole
  const unsigned ox = tok * ax + co * size, od = tok * ad + co * size, oz = tok * az + co * size;
  unsigned ov[R];
#pragma unroll
  for (int i = 0; i < R; i++) ov[i] = (i * PT + sub) * vs;
  auto fetch = [&](int k) {  // blocks in order: the addresses move on
    const int most = count - k * kBlock - 1;  // the last token of the block, at most
    if (most >= kBlock - 1) {
      rx.load(xp + ox);
      rd.load(dp + od);
      if (OUT) rz.load(zq + oz);
#pragma unroll
      for (int i = 0; i < R; i++) rv[i].load(vp + ov[i]);
    } else {
      const unsigned t = tok < most ? tok : most;
      rx.load(xp + (t * ax + co * size));
      rd.load(dp + (t * ad + co * size));
      if (OUT) rz.load(zq + (t * az + co * size));
#pragma unroll
      for (int i = 0; i < R; i++) {
        const unsigned t = i * PT + sub < most ? i * PT + sub : most;
        rv[i].load(vp + t * vs);
      }
    }
    xp += (long long)ax * kBlock;
    dp += (long long)ad * kBlock;
    zq += (long long)az * kBlock;
    vp += (long long)vs * kBlock;
  };
  auto prepare = [&](int k) {
    float D[E];
#pragma unroll
    for (int i = 0; i < E; i++) D[i] = rd[i] + bias[i];
    if (A.softplus) {
#pragma unroll
      for (int i = 0; i < E; i++) D[i] = step_of<DT>(1, D[i]);
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
      for (int i = 0; i < E; i++) y[i] *= z0[i] * sigmoid<DT>(z0[i]);
    }
    if (k * kBlock + tok < count && mine) storev<DT, E>(op + (unsigned)(tok * ao + co * size), 0, y);
    op += (long long)ao * kBlock;
  };
  auto one = [&](auto t, int k, float bc) {  // a token of a block, whose values lie in lanes of `bc`
    constexpr int T = t, base = T % PT * V;
    const float2 d = steps[k & 1][T][cl];
    unrolled<NS>([&](auto i) { h[i] = fmaf(decay(d.x, a2[i]), h[i], row_lane<base + i>(bc) * d.y); });
    if constexpr (OUT) {
      float y = 0;
      if constexpr (NS == 2) y = row_dot2<base + NS>(bc, h);
      else y = row_dot<base + NS, false>(y, bc, h);
      if constexpr (NS == 8) y = row_dot<base + NS + 4, true>(y, bc, h + 4);
      parts[k & 1][part][T][cl] = y;
    }
  };
  const int blocks = __builtin_amdgcn_readfirstlane((count + kBlock - 1) / kBlock);  // (one value of the wave)
  const long long kept0 = PASS == 3 ? first_block(A, W) : 0;
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
    if (OUT && k > 0) finish(k - 1);
    x0 = x1;
    z0 = z1;
    if (PASS == 3) put_states<NS>(Q.kept + ((kept0 + k) * per + tg) * (64 * NW * NS) + threadIdx.x * NS, h);
    const int left = count - k * kBlock;
    if (left >= kBlock) {
      unrolled<kBlock>([&](auto t) { one(t, k, bc[t / PT]); });
    } else {
      unrolled<kBlock>([&](auto t) {
        if (t < left) one(t, k, bc[t / PT]);
      });
    }
    if (k + 1 < blocks) prepare(k + 1);
  }
  if (OUT && blocks > 0) {
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
  } else if (OUT && ends && A.S_out && live) {
    put_states<NS>(A.S_out + so, h);
  }
}

// Which sequences are cut, and how.  Where workgroups of 32 channels of whole sequences would be fewer than `least`, all of
// more than a segment: about ten workgroups of segments a CU, but no more than 64 segments of a sequence (each looks at all
// before it), of at least 64 tokens.  Otherwise those that would run long after the rest has ended.  Lengths are on the device; known
// here are their mean and what one of them may have (all tokens but one for each other sequence).  The rest ends after
// about `mean` tokens or, where CUs are full, what two workgroups a CU take for all tokens: longer by half and of more
// than 1,024 tokens is cut.  A call whose sequences turn out alike pays a pass that finds nothing to do.
struct Cut {
  int sh;          // segments of 2^sh tokens (0: none)
  long long over;  // of sequences longer than this
};
inline Cut segments_of(const ScanArgs& a, int least) {
  if (a.N <= 0) return Cut{0, 0};
  const long long tiles = (a.Cg + 31) / 32 * a.G, mean = a.T / a.N, longest = a.cu ? (long long)a.T - a.N + 1 : mean;
  auto length = [&](long long most, long long of) {
    int sh = 6;
    while (sh < 30 && (((long long)a.T >> sh) * tiles > most || of >> sh > 64)) sh++;
    return sh;
  };
  if (tiles * a.N < least) {
    const int sh = length(2560, mean);
    if (mean > 1LL << sh) return Cut{sh, 1LL << sh};
  }
  const int sh = length(tiles * a.N > 2560 ? tiles * a.N : 2560, longest);
  const long long full = a.T * tiles / 512, rest = mean > full ? mean : full;
  long long over = rest + rest / 2 > 1024 ? rest + rest / 2 : 1024;
  if (over < 1LL << sh) over = 1LL << sh;
  return longest > over ? Cut{sh, over} : Cut{0, 0};
}
// Both sides, us, 16 states, bf16 (whole or cut by an even rule on the mean, against this one).  One to three sequences of 2,048
// tokens x 4,096 channels, 128 workgroups each: whole 137 / 142 / 185, all cut 79 / 152 / 207; gradient 557 / 564 / 665 and 237 /
// 426 / 606.  Uneven: {1, 16,384} x 4,096 1,256 and 500; {7 of 1, 14,000} x 4,096 1,078 and 440, gradient 3,177 and 1,304; {3 of 1,
// 16,384} x 2,048 1,119 and 253; {60 of 1, 3,000} x 128 199 and 23, gradient 674 and 58; {200 of 1, 12,000} x 32 787 and 45, 2,643 and
// 124; {64 of 1, 2,048} x 4,096 140 and 114, 402 and 311.  Alike: 8 of 2,048 x 4,096 308 and 313, gradient 1,126 and 1,135; 70 of
// 128 181 and 177, 616 and 593; 4 of 2,048 x 2,048 143 and 148, 395 and 376; 4 of 350 x 2,048 28.5 and 32.5; 60 of 50 x 128 12 and
// 16, gradient 30 and 37: a pass that finds nothing to cut costs 4 to 8 us, so that calls of up to 1,024 tokens go without.
constexpr int kLeastForward = 256, kLeastBackward = 512;

constexpr size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace of the segments at `ws`, up to `end`.
inline Segments lay_segments(const ScanArgs& a, Cut cut, char* ws, char** end) {
  Segments q{(a.Cg + 31) / 32, cut.sh, cut.over, nullptr, nullptr, nullptr, nullptr};
  if (cut.sh) {
    const size_t m = (size_t)pieces(a, cut.sh);
    q.last = (float*)ws;
    q.steps = (float*)(ws += up(m * a.C * a.n * 4));
    q.first = (float*)(ws += up(m * a.C * 4));
    ws += up((size_t)a.N * a.C * a.n * 4);
  }
  *end = ws;
  return q;
}

}  // namespace
}  // namespace stepq
