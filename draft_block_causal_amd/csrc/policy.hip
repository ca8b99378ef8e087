// Log-probabilities of drafted tokens, and the clipped policy loss with its
// gradient with respect to the logits.
//
// For a row x of V logits with maximum M, in base-2 units t_v = c x_v - R,
// c = log2(e) / T, R an integer near c M:  s = sum 2^t_v,  u = sum 2^t_v t_v,
//     logp = ln 2 (c x_y - R) - ln s,   entropy = ln s - ln 2 u / s,
//     grad_v = coef (1[v = y] - 2^t_v / s),
// where coef is the loss's derivative with respect to logp times w / T.
// The token's own term e = 2^t_y is left out of the sums and added last: with r
// the sum of the others, s = e + r, logp = -ln(1 + r / e) and grad_y = coef r / s
// keep their digits where the token is nearly certain, and logp is never above 0.
// (With e among the sums grad_y was a difference of near equals: at 1 - p = 1e-6
// off by a fifth of itself.)
// R is an integer so that sums over different references are brought together
// by exact factors; t_v is two fused products, with the first 21 bits of c and
// with the rest.  Their roundings have no preferred direction: with all 24 bits of
// a float32 in the first part, the second product would be below half a step of
// most t_v and be lost (mean error of a log-probability over 151936 entries at
// T = 1.2: 1.6e-8, 1.4e-9 so).  While |c M| < 2^20, the second product is below 1,
// so t_v is off by (2 |t_v| + 1) 2^-24 at most, and the two roundings before R's
// own put R within 1/2 + 2^-3 of c M, so the largest terms of s have |t_v| < 1.
// (At 2^30 they were past what an exponential can hold.)  A row outside (a mask
// value in every entry, say) is taken again with t_v = c (x_v - M).
// What a row has one of (ln s, the ratio, the divergence, the loss) is in
// float64: a divergence is a small difference of numbers near 10.
//
// Launches on the caller's stream:
//   policy_held_kernel, a workgroup per row, where there are rows enough to fill
//     the device: the row is read once and held on chip (registers, and LDS for
//     the longest) between its sum and its gradient;
//   policy_stats_kernel, a workgroup per (row, vocabulary slice), for the other
//     rows, for calls without a gradient and for the log-probabilities;
//   policy_grad_kernel, a workgroup per (row, slice): brings its row's slices
//     together again (at most 32), forms coef and writes its slice of the
//     gradient; its first workgroups take the rows' logp, kl and loss terms and
//     the loss, so that neither needs a launch of its own;
//   logprobs_rows_kernel, 32 lanes per row: logp and entropy from the slices; or
//   logprobs_direct_kernel, a workgroup per row, alone: small calls, short rows.
// Bound by HBM: a row's logits once in and its gradient once out (held), or
// twice in and once out; a call of one block by its two launches (16 rows of
// 151936 entries: statistics 5.5 us, gradient 8.2 us, of which about 2 us each
// are the launch).
#include <math.h>
#include <string.h>

#include <algorithm>

#include "common.h"
#include "rollout.h"

namespace domino {

constexpr int kPolThreads = 256;
constexpr int kPolWaves = kPolThreads / 64;

// c = log2(e) / T, and c = hi + lo within 2^-45 of it, hi of 21 bits, 2^-22 hi <= lo <
// 2^-20 hi (so that x = -inf stays -inf)
struct Base2 {
  float hi, lo;
  double c;
};

// Maximum of some logits (the exact one), and sums relative to R(m); the drafted
// token's logit has no part in them.  The sums are in float64, added to by float32
// sums of 16 terms: one term near 1 would swallow the last bits of hundreds of
// small ones (2e-6 of a divergence).
struct SoftPart {
  float m;
  double s, u;
};

__device__ __forceinline__ float exp2_hw(float t) { return __builtin_amdgcn_exp2f(t); }

constexpr float kRefMax = 1048576.f;  // 2^20
// c m, in two roundings (it grows with m)
__device__ __forceinline__ float scaled(float m, Base2 c) { return fmaf(m, c.lo, m * c.hi); }
__device__ __forceinline__ float ref_of(float m, Base2 c) {
  return fminf(fmaxf(rintf(scaled(m, c)), -kRefMax), kRefMax);
}
// Whether a row's maximum lies where R(m) does not serve (not: no entry at all).
__device__ __forceinline__ bool far_out(float m, Base2 c) { return m != -INFINITY && !(fabsf(scaled(m, c)) < kRefMax); }

// What the sums of a part with maximum m are relative to: R(m), or c m where that
// does not serve.
__device__ __forceinline__ double base_of(float m, Base2 c) {
  return far_out(m, c) ? (double)m * ((double)c.hi + (double)c.lo) : (double)ref_of(m, c);
}

// t relative to R
__device__ __forceinline__ float base2(float x, float R, Base2 c) { return fmaf(x, c.lo, fmaf(x, c.hi, -R)); }

// p relative to R(m), m >= p.m
__device__ __forceinline__ SoftPart soft_to(SoftPart p, float m, Base2 c) {
  const float d = ref_of(p.m, c) - ref_of(m, c);
  const int e = (int)fmaxf(d, -4096.f);
  const double s = ldexp(p.s, e);
  return SoftPart{m, s, fma((double)e, s, ldexp(p.u, e))};
}

__device__ __forceinline__ SoftPart soft_merge(SoftPart a, SoftPart b, Base2 c) {
  const float m = fmaxf(a.m, b.m);
  a = soft_to(a, m, c);
  b = soft_to(b, m, c);
  return SoftPart{m, a.s + b.s, a.u + b.u};
}

// Over groups of WIDTH lanes: the maximum first, then every lane's sums brought
// to it once and added up.
template <int WIDTH>
__device__ __forceinline__ SoftPart lanes_soft(SoftPart p, Base2 c) {
  float m = p.m;
#pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  p = soft_to(p, m, c);
#pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) {
    p.s += __shfl_xor(p.s, o);
    p.u += __shfl_xor(p.u, o);
  }
  return p;
}

constexpr SoftPart kNone{-INFINITY, 0.0, 0.0};

// Folds N values into a running part whose reference R = R(p.m) is kept along.
// Values of -inf add nothing; a NaN makes s NaN.
template <int N, bool ENT>
__device__ __forceinline__ void soft_add(SoftPart& p, float& R, const float (&x)[N], Base2 c) {
  float top = x[0];
#pragma unroll
  for (int e = 1; e < N; ++e) top = fmaxf(top, x[e]);
  if (top > p.m) {
    p = soft_to(p, top, c);
    R = ref_of(top, c);
  }
  float f[N], g[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float t = base2(x[e], R, c);
    f[e] = exp2_hw(t);
    if (ENT) g[e] = f[e] * fmaxf(t, -200.f);
  }
#pragma unroll
  for (int h = N / 2; h > 0; h >>= 1)
#pragma unroll
    for (int e = 0; e < h; ++e) {
      f[e] += f[e + h];
      if (ENT) g[e] += g[e + h];
    }
  p.s += (double)f[0];
  if (ENT) p.u += (double)g[0];
}

__device__ __forceinline__ int clamp_id(int y, int V) { return min(max(y, 0), V - 1); }

// Entries [v0, v1) of slice s of S of a row of V at `row`: inner boundaries
// fall on 16-byte boundaries of the row's own memory.
__device__ __forceinline__ void row_slice(const float* row, int V, int s, int S, int& v0, int& v1) {
  const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) >> 2);
  const long n4 = (V - head) >> 2;
  v0 = s == 0 ? 0 : head + 4 * (int)(n4 * s / S);
  v1 = s == S - 1 ? V : head + 4 * (int)(n4 * (s + 1) / S);
}

// The whole 16-byte groups of entries v0 .. v1 - 1 (a4 .. b4 - 1), and the at
// most 6 entries outside them: outer entry e, e < outer.
struct Span {
  int v0, v1, a4, b4, n4, outer;
  __device__ __forceinline__ Span(const float* row, int v0_, int v1_) : v0(v0_), v1(v1_) {
    a4 = min(v1, v0 + ((int)((16 - (reinterpret_cast<uintptr_t>(row + v0) & 15)) & 15) >> 2));
    b4 = a4 + ((v1 - a4) & ~3);
    n4 = (b4 - a4) >> 2;
    outer = (a4 - v0) + (v1 - b4);
  }
  __device__ __forceinline__ int outer_at(int e) const { return e < a4 - v0 ? v0 + e : b4 + e - (a4 - v0); }
  // The layer of NT groups that entry v's group belongs to (-1: not in a whole group).
  __device__ __forceinline__ int layer(int v, int NT) const { return v >= a4 && v < b4 ? ((v - a4) >> 2) / NT : -1; }
  // The thread of NT that handles entry v (groups are dealt out in turn).
  __device__ __forceinline__ int owner(int v, int NT) const {
    return v < a4 ? v - v0 : v < b4 ? ((v - a4) >> 2) % NT : (a4 - v0) + v - b4;
  }
};

// The drafted token's place among the groups that a workgroup takes.
struct Token {
  int y, layer, thread, e;  // entry of the row; layer, thread and place in the group
  __device__ __forceinline__ Token(const Span& sp, int y_, int NT)
      : y(__builtin_amdgcn_readfirstlane(y_)), layer(sp.layer(y, NT)), thread(sp.owner(y, NT)), e((y - sp.a4) & 3) {}
  // Takes it out of a thread's groups of layers first, first + 1, ... (the branch on
  // the layer is the same for all threads).
  template <int G>
  __device__ __forceinline__ void leave_out(f32x4* v, int first) const {
    const unsigned at = (unsigned)(layer - first);
    if (at < (unsigned)G && (int)threadIdx.x == thread) {
#pragma unroll
      for (int i = 0; i < 4 * G; ++i)
        if (i == (int)(4 * at) + e) v[i >> 2][i & 3] = -INFINITY;
    }
  }
};

// A workgroup's part from its waves' parts; the result in every thread of wave
// 0 at least.  red: one entry per wave.
template <int WAVES>
__device__ __forceinline__ SoftPart block_soft(SoftPart p, SoftPart* red, Base2 c) {
  p = lanes_soft<64>(p, c);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = p;
  __syncthreads();
  p = red[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) p = soft_merge(p, red[w], c);
  return p;
}

// Sums of a far-out slice with maximum m, t = c (x - m), without entry y.  Every
// thread of the workgroup calls it (red: one entry per wave, not in use).
template <int WAVES>
__device__ SoftPart far_out_part(const float* x, int v0, int v1, int y, float m, Base2 c, SoftPart* red) {
  double s = 0.0, u = 0.0;
  for (int v = v0 + threadIdx.x; v < v1; v += WAVES * 64) {
    const float t = v == y ? -INFINITY : (x[v] - m) * (c.hi + c.lo), f = exp2_hw(t);
    s += (double)f;
    u += (double)(f * fmaxf(t, -200.f));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    u += __shfl_xor(u, o);
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = SoftPart{m, s, u};
  __syncthreads();
  SoftPart p = red[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) {
    p.s += red[w].s;
    p.u += red[w].u;
  }
  return p;
}

// The part of a span of a row without entry y (which may lie outside it), taken by
// a workgroup of NT threads (red: one entry per wave); the result in every thread.
template <int NT, bool ENT, bool ONCE>
__device__ __forceinline__ SoftPart span_soft(const float* x, const Span& sp, int y, Base2 c, SoftPart* red) {
  const Token tok(sp, y, NT);
  SoftPart p = kNone;
  float R = ref_of(p.m, c);
  const f32x4* x4 = reinterpret_cast<const f32x4*>(x + sp.a4);
  {
    // four groups a thread and step, the next step in flight while one is used;
    // the last step may be ragged
    constexpr int U = 4, kStep = U * NT;
    const int n = (sp.n4 + kStep - 1) / kStep;
    auto load = [&](f32x4 (&d)[U], int step) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const f32x4* at = x4 + min(step * kStep + i * NT + (int)threadIdx.x, sp.n4 - 1);
        d[i] = ONCE ? __builtin_nontemporal_load(at) : *at;
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto use = [&](f32x4 (&d)[U], int step) {
      if ((step + 1) * kStep > sp.n4) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (step * kStep + i * NT + (int)threadIdx.x >= sp.n4)
            d[i] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      }
      tok.leave_out<U>(d, step * U);
      float f[4 * U];
#pragma unroll
      for (int e = 0; e < 4 * U; ++e) f[e] = d[e >> 2][e & 3];
      soft_add<4 * U, ENT>(p, R, f, c);
      __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 b0[U], b1[U];
    if (n > 0) load(b0, 0);
    for (int i = 0; i < n; i += 2) {
      if (i + 1 < n) load(b1, i + 1);
      use(b0, i);
      if (i + 2 < n) load(b0, i + 2);
      if (i + 1 < n) use(b1, i + 1);
    }
  }
  if ((int)threadIdx.x < sp.outer) {
    const int v = sp.outer_at(threadIdx.x);
    const float f[1] = {v == tok.y ? -INFINITY : x[v]};
    soft_add<1, ENT>(p, R, f, c);
  }
  p = block_soft<NT / 64>(p, red, c);
  if (far_out(p.m, c)) p = far_out_part<NT / 64>(x, sp.v0, sp.v1, tok.y, p.m, c, red);
  return p;
}

// Row of workgroup b of n when a workgroup takes a row: groups of 8 consecutive
// rows are turned against the 8 XCDs that workgroups go round, each group by
// another step, so that positions of a block that are often masked (its last
// ones) do not all fall to the same XCD.
__device__ __forceinline__ int turned_row(int b, int n) {
  return (b | 7) < n ? (b & ~7) | ((b + (b >> 3) + (b >> 4)) & 7) : b;
}

// Workgroup b: slice b % S of row b / S, so that neighbouring slices go to
// different XCDs (64 blocks cut at their acceptance lengths: with all slices of
// a row on one XCD 70 us, the XCD of a block's first positions having 1.4 times
// the average work; 54 us).
// ONCE: the logits are not read again (non-temporal loads).
struct StatsDev {
  int row0, rows, V, S;
  Base2 c;
  const float* logits;
  const int32_t* tokens;
  const float* weights;
  SoftPart* stats;
  float* xy;
  unsigned int* ticket;  // cleared for policy_grad_kernel, if not null
};

template <bool ENT, bool ONCE>
__global__ void __launch_bounds__(kPolThreads) policy_stats_kernel(StatsDev a) {
  __shared__ SoftPart red[kPolWaves];
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.ticket) *a.ticket = 0;
  const int V = a.V, S = a.S;
  const int sl = (int)(blockIdx.x % (unsigned)S), row = a.row0 + turned_row((int)(blockIdx.x / (unsigned)S), a.rows - a.row0);
  if (a.weights && a.weights[row] == 0.f) return;
  const float* x = a.logits + (size_t)row * V;
  int v0, v1;
  row_slice(x, V, sl, S, v0, v1);
  const Span sp(x, v0, v1);
  // the token's logit, asked for first: at the end it would be two more waits
  const int y = clamp_id(a.tokens[row], V);
  const bool mine = y >= v0 && y < v1;
  const float x_y = mine ? x[y] : 0.f;
  const SoftPart p = span_soft<kPolThreads, ENT, ONCE>(x, sp, y, a.c, red);
  if (threadIdx.x == 0) {
    a.stats[(size_t)row * S + sl] = p;
    if (mine) a.xy[row] = x_y;
  }
}

// p brought to m >= p.m.  Where one of the two is far out the factor is no power of
// two: their bases are of different kinds.  (A part without entries has no base; its
// sums are 0, or NaN.)
__device__ __forceinline__ SoftPart part_to(SoftPart p, float m, Base2 c) {
  if (!far_out(m, c) && !far_out(p.m, c)) return soft_to(p, m, c);
  const double d = p.m == -INFINITY ? 0.0 : base_of(p.m, c) - base_of(m, c), e = exp2(d);
  return SoftPart{m, e * p.s, e == 0.0 ? 0.0 : e * fma(d, p.s, p.u)};
}

// The part of a row from its S <= 32 slices' parts, one a lane of a group of 32
// (kNone in the other lanes); the result in every lane of the group.
__device__ __forceinline__ SoftPart slices_soft(SoftPart p, Base2 c) {
  float m = p.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  p = part_to(p, m, c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    p.s += __shfl_xor(p.s, o);
    p.u += __shfl_xor(p.u, o);
  }
  return p;
}

__device__ __forceinline__ SoftPart row_part(const SoftPart* stats, int row, int S, Base2 c) {
  const int q = threadIdx.x & 31;
  return slices_soft(q < S ? stats[(size_t)row * S + q] : kNone, c);
}

// A row's sums: r of the entries but the token's, and the token's term e = 2^t.
// (The exponential, the quotient and the token's test among the groups cost a call of
// one block 0.5 us of 13.4, a large one nothing; asking for the first groups before
// the token's number, or taking e beforehand relative to a base of its own, gained
// nothing.)
struct RowSum {
  float m;
  double s, r, u, t, logp;
};

__device__ __forceinline__ RowSum row_sum(SoftPart p, float x_y, Base2 c) {
  const float m = fmaxf(p.m, x_y);
  p = part_to(p, m, c);
  const bool far = far_out(m, c);
  // t with the other terms' hi + lo, as R may be large; what c has besides counts
  // from the maximum on, where a token is far below it
  const double pair = (double)c.hi + (double)c.lo, d = fmax((double)x_y - (double)m, -1e300);
  const double t = far ? ((double)x_y - (double)m) * c.c : fma((double)x_y, pair, -(double)ref_of(m, c));
  const double tc = far ? t : fma(c.c - pair, d, t);
  const double e = exp2(t), s = p.s + e;
  // -ln(1 + q), q = r / e, with what 1 + q rounds off put back (over 1 + q, to
  // first order); or ln 2 t - ln s
  const bool most = p.s < e;
  const double q = p.s / e, a = most ? 1.0 + q : s, l = log(a);
  const double lp = most ? fma((a - 1.0) - q, 1.0 - q, -l) : fma(0.6931471805599453, tc, -l);
  return RowSum{m, s, p.s, p.u, t, lp};
}

struct LogpOut {
  float logp, entropy;
};

__device__ __forceinline__ LogpOut logp_out(const SoftPart& p, float x_y, Base2 c) {
  const RowSum q = row_sum(p, x_y, c);
  if (q.s == 0.0) return LogpOut{-INFINITY, 0.f};  // no distribution
  // ln s - ln 2 (u + e t) / s, in which what a token near 1 has of both cancels
  // beforehand; e counts for nothing below
  const double h = q.t > -64.0 ? fma(0.6931471805599453, fma(q.t, q.r, -q.u) / q.s, -q.logp)
                                 : log(q.s) - 0.6931471805599453 * (q.u / q.s);
  return LogpOut{(float)q.logp, h < 0.0 ? 0.f : (float)h};
}

// A workgroup a row, nothing to bring together.
template <int NT, bool ENT>
__global__ void __launch_bounds__(NT) logprobs_direct_kernel(StatsDev a, float* __restrict__ logp,
                                                             float* __restrict__ entropy) {
  __shared__ SoftPart red[NT / 64];
  const int row = turned_row(blockIdx.x, gridDim.x);
  LogpOut r{0.f, 0.f};
  if (!(a.weights && a.weights[row] == 0.f)) {
    const float* x = a.logits + (size_t)row * a.V;
    const float x_y = x[clamp_id(a.tokens[row], a.V)];
    const Span sp(x, 0, a.V);
    const SoftPart p = span_soft<NT, ENT, true>(x, sp, clamp_id(a.tokens[row], a.V), a.c, red);
    // (all waves at the same float64 chain hold each other up: 256 rows of 5003
    // entries 9.4 us, 8.0 so)
    if (threadIdx.x < 64) r = logp_out(p, x_y, a.c);
  }
  if (threadIdx.x == 0) {
    logp[row] = r.logp;
    if (ENT) entropy[row] = r.entropy;
  }
}

// 32 lanes a row
__global__ void __launch_bounds__(kPolThreads)
    logprobs_rows_kernel(int rows, int S, Base2 c, const SoftPart* __restrict__ stats,
                         const float* __restrict__ xy, const float* __restrict__ weights, float* __restrict__ logp,
                         float* __restrict__ entropy) {
  const int row = blockIdx.x * (kPolThreads / 32) + (threadIdx.x >> 5);
  if (row >= rows) return;
  const float x_y = xy[row], w = weights ? weights[row] : 1.f;
  const SoftPart p = row_part(stats, row, S, c);
  LogpOut r{0.f, 0.f};
  if (w != 0.f) r = logp_out(p, x_y, c);
  if ((threadIdx.x & 31) == 0) {
    logp[row] = r.logp;
    if (entropy) entropy[row] = r.entropy;
  }
}

struct PolicyDev {
  int rows, held, V;  // rows below `held` are the held kernel's
  int S, G;           // slices of a row's statistics, and of its gradient
  Base2 c;
  double inv_t, lo, hi, beta;  // clip range limits; KL coefficient
  const float *logits, *old_logp, *ref_logp, *advantages, *weights;
  const int32_t* tokens;
  const SoftPart* stats;
  const float* xy;
  double* terms;        // [held] weighted loss terms
  double* sums;         // [row_wgs] sums of the other rows' terms
  unsigned int* ticket;  // finished row workgroups (0 at the kernel's start)
  int row_wgs;
  float *loss, *logp, *kl, *grad;
};

struct RowTerms {
  float logp, kl;
  double term, coef;  // weighted loss term; its derivative with respect to logp, over T
  RowSum sum;
};

// What the loss reads of a row, loaded together.  (Rows of weight 0 are read
// too, and not used.)
struct RowIn {
  double w, adv, old, ref;
};

__device__ __forceinline__ RowIn row_in(const PolicyDev& a, int row) {
  return RowIn{a.weights ? (double)a.weights[row] : 1.0 / a.rows, a.advantages[row], a.old_logp[row],
               a.ref_logp ? a.ref_logp[row] : 0.0};
}

__device__ __forceinline__ RowTerms row_terms(const PolicyDev& a, const RowIn& in, float xy, const SoftPart& p) {
  RowTerms r{-INFINITY, 0.f, 0.0, 0.0, row_sum(p, xy, a.c)};
  if (r.sum.s == 0.0) return r;  // no distribution
  const double lp = r.sum.logp;
  const double w = in.w, adv = in.adv, ratio = exp(lp - in.old);
  const bool inside = adv >= 0.0 ? ratio <= a.hi : ratio >= a.lo;
  // (an advantage of 0 stays 0 whatever the ratio)
  double l = 0.0, g = 0.0;
  if (adv != 0.0) {
    l = inside ? -ratio * adv : -(adv >= 0.0 ? a.hi : a.lo) * adv;
    g = inside ? -ratio * adv : 0.0;
    if (ratio != ratio) l = g = ratio;
  }
  if (a.ref_logp) {
    const double d = in.ref - lp, e = expm1(d);
    const double kl = d == INFINITY ? INFINITY : e - d;
    r.kl = (float)kl;
    if (a.beta != 0.0) {
      l += a.beta * kl;
      g -= a.beta * e;
    }
  }
  r.logp = (float)lp;
  r.term = w * l;
  r.coef = w * g * a.inv_t;
  return r;
}

// The first `row_wgs` workgroups of policy_grad_kernel: logp, kl and the loss
// terms of the rows that are not held, 32 lanes a row and kRowsPerWg rows a
// workgroup, summed in order; the workgroup that finishes last adds up the
// workgroups' sums and the held rows' terms in a fixed order, so that the order
// of finishing does not show.
constexpr int kRowsPerWg = kPolThreads / 32;

__device__ void policy_rows(const PolicyDev& a) {
  __shared__ double part[kRowsPerWg];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int row = a.held + (int)blockIdx.x * kRowsPerWg + sub;
  double term = 0.0;
  if (row < a.rows) {
    const RowIn in = row_in(a, row);
    const float xy = a.xy[row];
    const SoftPart p = row_part(a.stats, row, a.S, a.c);
    RowTerms r{};
    if (in.w != 0.0) r = row_terms(a, in, xy, p);
    term = r.term;
    if (lane == 0) {
      if (a.logp) a.logp[row] = r.logp;
      if (a.kl) a.kl[row] = r.kl;
    }
  }
  if (lane == 0) part[sub] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = part[0];
    for (int q = 1; q < kRowsPerWg; ++q) sum += part[q];
    last = true;
    if (a.row_wgs > 1) {
      __hip_atomic_store(a.sums + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             (unsigned)a.row_wgs - 1u;
    } else {
      a.sums[0] = sum;
    }
  }
  __syncthreads();
  if (!last) return;
  double acc = 0.0;
  for (int q = threadIdx.x; q < a.row_wgs; q += kPolThreads)
    acc += __hip_atomic_load(a.sums + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int q = threadIdx.x; q < a.held; q += kPolThreads) acc += a.terms[q];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kPolWaves; ++w) acc += part[w];
    a.loss[0] = (float)acc;
  }
}

// What a row's gradient is made of: k 2^t, and `tok` at the token.
struct GradRow {
  float ref, k, tok;  // ref: R, or the maximum of a far-out row
  int far;
};

__device__ __forceinline__ GradRow grad_row(const RowTerms& r, Base2 c) {
  const bool far = far_out(r.sum.m, c);
  if (r.coef == 0.0) return GradRow{0.f, 0.f, 0.f, far};
  const double k = r.coef / r.sum.s;
  return GradRow{far ? r.sum.m : ref_of(r.sum.m, c), (float)-k, (float)(k * r.sum.r), far};
}

__device__ __forceinline__ float grad_of(float x, const GradRow& g, Base2 c) {
  const float t = g.far ? (x - g.ref) * (c.hi + c.lo) : base2(x, g.ref, c);
  return g.k * exp2_hw(t);
}

__device__ __forceinline__ f32x4 grad_of4(f32x4 x, const GradRow& g, Base2 c) {
  return f32x4{grad_of(x[0], g, c), grad_of(x[1], g, c), grad_of(x[2], g, c), grad_of(x[3], g, c)};
}

template <int NT>
__device__ __forceinline__ void zero_span(float* g, const Span& sp) {
  for (int q = threadIdx.x; q < sp.n4; q += NT) *reinterpret_cast<f32x4*>(g + sp.a4 + 4 * q) = f32x4{0.f, 0.f, 0.f, 0.f};
  if ((int)threadIdx.x < sp.outer) g[sp.outer_at(threadIdx.x)] = 0.f;
}

// (x and g may be the same buffer: every entry is read by the thread that
// writes it, before it does, and the token's logit comes from xy)
__global__ void __launch_bounds__(kPolThreads) policy_grad_kernel(PolicyDev a) {
  if ((int)blockIdx.x < a.row_wgs) {
    policy_rows(a);
    return;
  }
  __shared__ GradRow sh;
  const unsigned b = blockIdx.x - (unsigned)a.row_wgs;
  const int row = a.held + (int)(b / (unsigned)a.G), sl = (int)(b % (unsigned)a.G);
  const float* x = a.logits + (size_t)row * a.V;
  float* g = a.grad + (size_t)row * a.V;
  int v0, v1;
  row_slice(x, a.V, sl, a.G, v0, v1);
  const Span sp(g, v0, v1);
  const RowIn in = row_in(a, row);
  const float xy = a.xy[row];
  const int y = clamp_id(a.tokens[row], a.V);
  if (in.w == 0.0) {  // no logit is read
    zero_span<kPolThreads>(g, sp);
    return;
  }
  const bool alike = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(g)) & 15u) == 0;
  // the first groups are on their way while the row's sums are brought together
  constexpr int U = 4, kStep = U * kPolThreads;
  f32x4 d[U];
  auto load = [&](int at) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      d[i] = *reinterpret_cast<const f32x4*>(x + sp.a4 + 4 * min(at + i * kPolThreads + (int)threadIdx.x, sp.n4 - 1));
    __builtin_amdgcn_sched_barrier(0);
  };
  if (alike && sp.n4 > 0) load(0);
  if (threadIdx.x < 32) {
    const SoftPart p = row_part(a.stats, row, a.S, a.c);
    const RowTerms r = row_terms(a, in, xy, p);
    if (threadIdx.x == 0) sh = grad_row(r, a.c);
  }
  __syncthreads();
  const GradRow gr = sh;
  if (gr.k == 0.f && gr.tok == 0.f) {  // no gradient here
    zero_span<kPolThreads>(g, sp);
    return;
  }
  if (alike) {
    for (int at = 0; at < sp.n4; at += kStep) {
      if (at > 0) load(at);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int q = at + i * kPolThreads + (int)threadIdx.x;
        if (q < sp.n4) *reinterpret_cast<f32x4*>(g + sp.a4 + 4 * q) = grad_of4(d[i], gr, a.c);
      }
    }
    if ((int)threadIdx.x < sp.outer) {
      const int v = sp.outer_at(threadIdx.x);
      g[v] = grad_of(x[v], gr, a.c);
    }
    // (the owner's second store to the entry, in its program order)
    if (y >= v0 && y < v1 && (int)threadIdx.x == sp.owner(y, kPolThreads)) g[y] = gr.tok;
  } else {
    for (int v = v0 + threadIdx.x; v < v1; v += kPolThreads) {
      g[v] = v == y ? gr.tok : grad_of(x[v], gr, a.c);
    }
  }
}

// ---------------------------------------------------------------------------
// Held rows: NT threads; a layer is NT groups of 4 logits, one a thread.  H
// layers stay in registers, up to kHeldLds more in LDS (filled by loads that
// bypass the registers), and up to RM (the rest, the last one ragged) are read
// twice: before the registers fill up, and again into those freed by the first
// layers' gradients, so that no load is waited for alone.  What is beyond comes
// in a plain loop.  All other loads of a row are in flight at once, up to 500 KB
// a compute unit, and the row's terms are added up as they come in.
// Non-temporal both ways: nothing is read again from a cache but the RM layers
// (32 blocks of the Qwen3 vocabulary: 164 -> 137 us with RM layers read in a
// loop each time, 124 in this form with its two launches; a device copy of the
// same bytes takes 121).
// ---------------------------------------------------------------------------
constexpr int kHeldMost = 100;  // layers of 512
constexpr int kHeldLds = 19;  // 152 KB with 512 threads, 76 KB with 256
typedef __attribute__((address_space(1))) const void* held_gptr_t;
typedef __attribute__((address_space(3))) void* held_lptr_t;

template <int NT, int H, int RM>
__global__ void __launch_bounds__(NT) policy_held_kernel(PolicyDev a, int L) {
  static_assert(H % 4 == 0 && RM % 4 == 0 && H >= RM, "layers go in fours");
  constexpr int WAVES = NT / 64;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  f32x4* lds = reinterpret_cast<f32x4*>(smem);  // [L][NT]
  __shared__ SoftPart red[WAVES];
  __shared__ GradRow sh;
  const int row = turned_row(blockIdx.x, gridDim.x), tid = threadIdx.x;
  const float* x = a.logits + (size_t)row * a.V;
  float* g = a.grad + (size_t)row * a.V;
  const Span sp(x, 0, a.V);  // (g has the same alignment)
  const RowIn in = row_in(a, row);
  if (in.w == 0.0) {
    zero_span<NT>(g, sp);
    if (tid == 0) {
      if (a.logp) a.logp[row] = 0.f;
      if (a.kl) a.kl[row] = 0.f;
      a.terms[row] = 0.0;
    }
    return;
  }
  const int y = clamp_id(a.tokens[row], a.V);
  const float xy = x[y];
  const Token tok(sp, y, NT);
  const f32x4* x4 = reinterpret_cast<const f32x4*>(x + sp.a4);
  const int rest = (H + L) * NT;  // the first group that is not held
  SoftPart p = kNone;
  float R = ref_of(p.m, a.c);
  // (the token is taken out of the registers for good: its gradient comes last)
  auto add4 = [&](f32x4* v, int layer) {
    tok.leave_out<4>(v, layer);
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = v[e >> 2][e & 3];
    soft_add<16, false>(p, R, f, a.c);
  };
  auto load_rest = [&](f32x4 (&r)[RM]) {
#pragma unroll
    for (int i = 0; i < RM; ++i)
      if (rest + i * NT < sp.n4) r[i] = x4[min(rest + i * NT + tid, sp.n4 - 1)];
  };
  if (L > 0) {
    const int wave = wave_id();
    for (int l = 0; l < L; ++l)
      __builtin_amdgcn_global_load_lds((held_gptr_t)(x4 + (H + l) * NT + tid),
                                       (held_lptr_t)(smem + (l * WAVES + wave) * 1024), 16, 0, kLoadNonTemporal);
  }
  f32x4 h[H];
  {
    f32x4 r[RM];
    load_rest(r);
#pragma unroll
    for (int i = 0; i < H - RM; ++i) h[i] = __builtin_nontemporal_load(x4 + i * NT + tid);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < RM; ++i)
      if (rest + i * NT < sp.n4) {
        const bool in = rest + i * NT + tid < sp.n4;
        tok.leave_out<1>(r + i, H + L + i);
        const float f[4] = {in ? r[i][0] : -INFINITY, in ? r[i][1] : -INFINITY, in ? r[i][2] : -INFINITY,
                            in ? r[i][3] : -INFINITY};
        soft_add<4, false>(p, R, f, a.c);
      }
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = H - RM; i < H; ++i) h[i] = __builtin_nontemporal_load(x4 + i * NT + tid);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < H; i += 4) add4(h + i, i);
  if (L > 0) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's groups are in LDS, which only it reads
    __builtin_amdgcn_sched_barrier(0);
    int l = 0;
    for (; l + 4 <= L; l += 4) {
      f32x4 v[4] = {lds[l * NT + tid], lds[(l + 1) * NT + tid], lds[(l + 2) * NT + tid], lds[(l + 3) * NT + tid]};
      add4(v, H + l);
    }
    for (; l < L; ++l) {
      f32x4 v = lds[l * NT + tid];
      tok.leave_out<1>(&v, H + l);
      const float f[4] = {v[0], v[1], v[2], v[3]};
      soft_add<4, false>(p, R, f, a.c);
    }
  }
  for (int at = rest + RM * NT; at < sp.n4; at += 4 * NT) {
    f32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x4[min(at + i * NT + tid, sp.n4 - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * NT + tid >= sp.n4) v[i] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    add4(v, at / NT);
  }
  if (tid < sp.outer) {
    const int v = sp.outer_at(tid);
    const float f[1] = {v == y ? -INFINITY : x[v]};
    soft_add<1, false>(p, R, f, a.c);
  }
  p = block_soft<WAVES>(p, red, a.c);
  if (far_out(p.m, a.c)) p = far_out_part<WAVES>(x, 0, a.V, y, p.m, a.c, red);
  if (tid < 64) {
    const RowTerms r = row_terms(a, in, xy, p);
    if (tid == 0) {
      if (a.logp) a.logp[row] = r.logp;
      if (a.kl) a.kl[row] = r.kl;
      a.terms[row] = r.term;
      sh = grad_row(r, a.c);
    }
  }
  __syncthreads();
  const GradRow gr = sh;
  if (gr.k == 0.f && gr.tok == 0.f) {
    zero_span<NT>(g, sp);
    return;
  }
  f32x4* g4 = reinterpret_cast<f32x4*>(g + sp.a4);
  auto put = [&](int q, f32x4 v) { __builtin_nontemporal_store(grad_of4(v, gr, a.c), g4 + q); };
#pragma unroll
  for (int i = 0; i < RM; ++i) put(i * NT + tid, h[i]);
  __builtin_amdgcn_sched_barrier(0);
  {
    f32x4 r[RM];
    load_rest(r);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = RM; i < H; ++i) put(i * NT + tid, h[i]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < RM; ++i)
      if (rest + i * NT + tid < sp.n4) put(rest + i * NT + tid, r[i]);
  }
  for (int l = 0; l < L; ++l) put((H + l) * NT + tid, lds[l * NT + tid]);
  for (int at = rest + RM * NT; at < sp.n4; at += 4 * NT) {
    f32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x4[min(at + i * NT + tid, sp.n4 - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * NT + tid < sp.n4) put(at + i * NT + tid, v[i]);
  }
  if (tid < sp.outer) {
    const int v = sp.outer_at(tid);
    g[v] = grad_of(x[v], gr, a.c);
  }
  if (tid == tok.thread) g[y] = gr.tok;
}

template <int NT, int H, int RM>
static hipError_t launch_held(const PolicyDev& d, int L, hipStream_t s) {
  auto kern = policy_held_kernel<NT, H, RM>;
  if (L > 0) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kHeldLds * NT * 16);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)d.held), dim3(NT), L * NT * 16, s, d, L);
  return hipGetLastError();
}

// Whole layers of NT groups that every row has at least.
static int held_layers(int V, int NT) { return V < 8 ? 0 : ((V - 6) / 4) / NT; }

// Rows to hold on chip, and the threads a row: 256 as long as a row fits twice
// on a compute unit (which then reads one row while it writes another), else
// 512; 0 threads: rows too short or too long for it.
static int held_threads(int V) {
  if (held_layers(V, 256) < 4 || held_layers(V, 512) > kHeldMost) return 0;
  return held_layers(V, 256) < 48 + kHeldLds + 8 ? 256 : 512;
}
static int held_rows(int rows, int V, int num_cu) {
  const int nt = held_threads(V);
  // (20000 entries: 128 rows held 12.0 us, sliced 14.3; 10000 entries, 64 rows: 10 us both)
  if (nt == 256) return rows >= num_cu / 2 ? rows : 0;
  if (nt == 512) {
    // one row a compute unit: whole rounds, and a last one that is half full
    // (151936 entries: 128 rows held 40 us, sliced 46; 400 rows with the last 144 held
    // 99 us, sliced 115; 320 rows held 90 us, 85 with the last 64 sliced)
    const int rest = rows % num_cu;
    return 2 * rest >= num_cu ? rows : rows - rest;
  }
  return 0;
}

static hipError_t launch_held_rows(const PolicyDev& d, hipStream_t s) {
  if (held_threads(d.V) == 512) {  // (at least 37 layers)
    const int layers = held_layers(d.V, 512);
    return layers >= 48 ? launch_held<512, 48, 8>(d, std::min(layers - 48, kHeldLds), s)
                        : launch_held<512, 36, 12>(d, 0, s);
  }
  const int layers = held_layers(d.V, 256);
  if (layers >= 48) return launch_held<256, 48, 8>(d, std::min(layers - 48, kHeldLds), s);
  if (layers >= 36) return launch_held<256, 36, 12>(d, 0, s);
  if (layers >= 24) return launch_held<256, 24, 12>(d, 0, s);
  if (layers >= 16) return launch_held<256, 16, 8>(d, 0, s);
  if (layers >= 8) return launch_held<256, 8, 4>(d, std::min(layers - 8, 4), s);
  return launch_held<256, 4, 4>(d, 0, s);
}

static Base2 base2_factor(double temperature) {
  const double c = 1.4426950408889634 / temperature;
  const float f = (float)c;
  uint32_t bits;
  memcpy(&bits, &f, 4);
  bits &= ~7u;
  float hi;
  memcpy(&hi, &bits, 4);
  if (c - (double)hi < (double)hi * 0x1p-22) {  // leave something for lo
    bits -= 8u;
    memcpy(&hi, &bits, 4);
  }
  return Base2{hi, (float)(c - (double)hi), c};
}

template <bool ENT, bool ONCE>
static void launch_stats(const StatsDev& a, hipStream_t s) {
  hipLaunchKernelGGL((policy_stats_kernel<ENT, ONCE>), dim3((unsigned)(a.rows - a.row0) * (unsigned)a.S),
                     dim3(kPolThreads), 0, s, a);
}

template <int NT>
static void launch_direct(const StatsDev& a, float* logp, float* entropy, hipStream_t s) {
  if (entropy)
    hipLaunchKernelGGL((logprobs_direct_kernel<NT, true>), dim3((unsigned)a.rows), dim3(NT), 0, s, a, logp, entropy);
  else
    hipLaunchKernelGGL((logprobs_direct_kernel<NT, false>), dim3((unsigned)a.rows), dim3(NT), 0, s, a, logp, entropy);
}

hipError_t launch_token_logprobs(int B, int K, int V, const float* logits, const int32_t* tokens, const float* weights,
                                 double temperature, float* logp, float* entropy, const PolicyPlan& plan,
                                 void* workspace, int num_cu, hipStream_t s) {
  if (B <= 0) return hipSuccess;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const StatsDev a{0,      B * K,  V,       plan.S, base2_factor(temperature),
                   logits, tokens, weights, reinterpret_cast<SoftPart*>(ws + plan.stats),
                   reinterpret_cast<float*>(ws + plan.xy), nullptr};
  // Short rows, and longer ones of a small call, take a workgroup each and one
  // launch: what a small call from a program costs is its launches (16 x 20000: 8.0
  // us against 8.7 to 9.6 sliced, though 8.5 and 6.9 replayed from a graph; 16 x 60000:
  // 11 and 9 us; 512 x 32000: 20.5 and 16.5 us).  1024 threads while there are fewer rows
  // than fill the device, so that a row is in flight at once.
  if (V <= 8192 || (V <= 32768 && (long)a.rows * V <= 1l << 22) || plan.S == 1) {
    if (V > 4096 && a.rows < 4 * num_cu)
      launch_direct<1024>(a, logp, entropy, s);
    else
      launch_direct<kPolThreads>(a, logp, entropy, s);
    return hipGetLastError();
  }
  if (entropy)
    launch_stats<true, true>(a, s);
  else
    launch_stats<false, true>(a, s);
  hipLaunchKernelGGL(logprobs_rows_kernel, dim3((unsigned)((a.rows + kPolThreads / 32 - 1) / (kPolThreads / 32))),
                     dim3(kPolThreads), 0, s, a.rows, plan.S, a.c, a.stats, a.xy, weights, logp, entropy);
  return hipGetLastError();
}

hipError_t launch_policy_loss(const PolicyArgs& a, const PolicyPlan& plan, void* workspace, int num_cu,
                              hipStream_t s) {
  if (a.B <= 0) return hipSuccess;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  SoftPart* stats = reinterpret_cast<SoftPart*>(ws + plan.stats);
  float* xy = reinterpret_cast<float*>(ws + plan.xy);
  const int rows = a.B * a.K;
  PolicyDev d{rows,
              0,
              a.V,
              plan.S,
              1,
              base2_factor(a.temperature),
              1.0 / a.temperature,
              1.0 - a.clip_low,
              1.0 + a.clip_high,
              a.kl_coef,
              a.logits,
              a.old_logp,
              a.ref_logp,
              a.advantages,
              a.weights,
              a.tokens,
              stats,
              xy,
              reinterpret_cast<double*>(ws + plan.terms),
              reinterpret_cast<double*>(ws + plan.sums),
              reinterpret_cast<unsigned int*>(ws + plan.ticket),
              1,
              a.loss,
              a.logp,
              a.kl,
              a.grad};
  const bool alike = ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.grad)) & 15u) == 0;
  if (a.grad && alike) d.held = held_rows(rows, a.V, num_cu);
  if (d.held) {
    const hipError_t e = launch_held_rows(d, s);
    if (e != hipSuccess) return e;
  }
  if (d.held < rows)
    launch_stats<false, false>(
        StatsDev{d.held, rows, a.V, plan.S, d.c, a.logits, a.tokens, a.weights, stats, xy, d.ticket}, s);
  const int left = rows - d.held;
  d.row_wgs = std::max(1, (left + kRowsPerWg - 1) / kRowsPerWg);
  // a gradient workgroup brings its row's slices together before it can begin: at
  // least 4096 entries each, about 5 a compute unit at a time
  if (left > 0) d.G = std::max(1, std::min((5 * num_cu + left - 1) / left, a.V / 4096));
  const unsigned grid = (unsigned)d.row_wgs + (a.grad ? (unsigned)left * (unsigned)d.G : 0u);
  hipLaunchKernelGGL(policy_grad_kernel, dim3(grid), dim3(kPolThreads), 0, s, d);
  return hipGetLastError();
}

}  // namespace domino
