// Log-probabilities of drafted tokens, and the clipped policy loss with its
// gradient with respect to the logits.
//
// For a row x of V logits with maximum M, in base-2 units t_v = c (x_v - M),
// c = log2(e) / T:  s = sum 2^t_v,  u = sum 2^t_v t_v,
//     logp = (x_y - M) / T - ln s,   entropy = ln s - ln 2 u / s,
//     grad_v = coef (1[v = y] - 2^t_v / s),
// where coef is the loss's derivative with respect to logp times w / T.
//
// Launches on the caller's stream, grids over (row, vocabulary slice):
//   1. policy_stats_kernel: (M, s, u) of one slice, and the token's logit;
//   2. logprobs_rows_kernel: a thread per row merges the slices; or
//      policy_grad_kernel: each workgroup merges its row's slices again (at
//      most 32), forms coef and writes its slice of the gradient; workgroup 0
//      takes every row's logp, kl and loss term and the sum, so that neither
//      needs a launch of its own.
// Bound by HBM: V floats read in pass 1, V read and V written in pass 2.
//
// Everything a row has one of (ln s, the ratio, the divergence, the loss) is
// in float64: a divergence is a small difference of numbers near 10.  c is
// applied as a float32 pair, since its rounding would shift every term of s
// the same way (3e-8 |x - M| / T of s; the errors of the terms themselves
// average out).
#include <math.h>

#include "common.h"
#include "kernels.h"

namespace domino {

constexpr int kPolThreads = 256;
constexpr int kPolWaves = kPolThreads / 64;

// log2(e) / T as a float32 pair
struct Base2 {
  float hi, lo;
};

struct SoftPart {
  float m, s, u;
};

// 2^(c (x - m)): also for x = -inf (the low product is kept finite, which
// leaves a NaN to the high one).
__device__ __forceinline__ float base2(float x, float m, Base2 c) {
  const float d = x - m;
  return fmaf(d, c.hi, fmaxf(d, -3.0e38f) * c.lo);
}

__device__ __forceinline__ SoftPart soft_merge(SoftPart a, SoftPart b, Base2 c) {
  if (a.m == -INFINITY) return b;
  if (b.m == -INFINITY) return a;
  const float m = fmaxf(a.m, b.m);
  const float ta = base2(a.m, m, c), tb = base2(b.m, m, c);
  const float ea = __builtin_amdgcn_exp2f(ta), eb = __builtin_amdgcn_exp2f(tb);
  return SoftPart{m, ea * a.s + eb * b.s,
                  ea * (a.u + fmaxf(ta, -200.f) * a.s) + eb * (b.u + fmaxf(tb, -200.f) * b.s)};
}

__device__ __forceinline__ SoftPart wave_soft(SoftPart p, Base2 c) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const SoftPart q{__shfl_xor(p.m, o), __shfl_xor(p.s, o), __shfl_xor(p.u, o)};
    p = soft_merge(p, q, c);
  }
  return p;
}

// Folds n values into a running part; values of -inf add nothing, a NaN or
// +inf makes s NaN.
template <int N, bool ENT>
__device__ __forceinline__ void soft_add(SoftPart& p, const float (&x)[N], Base2 c) {
  float top = x[0];
#pragma unroll
  for (int e = 1; e < N; ++e) top = fmaxf(top, x[e]);
  if (top > p.m) {
    if (p.m != -INFINITY) {
      const float t = base2(p.m, top, c), f = __builtin_amdgcn_exp2f(t);
      if (ENT) p.u = f * (p.u + fmaxf(t, -200.f) * p.s);
      p.s *= f;
    }
    p.m = top;
  }
  const float m = p.m == -INFINITY ? 0.f : p.m;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float t = base2(x[e], m, c), f = __builtin_amdgcn_exp2f(t);
    p.s += f;
    if (ENT) p.u = fmaf(f, fmaxf(t, -200.f), p.u);
  }
}

// Entries [v0, v1) of slice s of S of a row of V at `row`: inner boundaries
// fall on 16-byte boundaries of the row's own memory.
__device__ __forceinline__ void row_slice(const float* row, int V, int s, int S, int& v0, int& v1) {
  const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) >> 2);
  const long n4 = (V - head) >> 2;
  v0 = s == 0 ? 0 : head + 4 * (int)(n4 * s / S);
  v1 = s == S - 1 ? V : head + 4 * (int)(n4 * (s + 1) / S);
}

__device__ __forceinline__ int clamp_id(int y, int V) { return min(max(y, 0), V - 1); }

// Entries v0 .. a4 - 1 and b4 .. v1 - 1 of a slice lie outside its whole
// 16-byte groups.
__device__ __forceinline__ void slice_vectors(const float* row, int v0, int v1, int& a4, int& b4) {
  a4 = min(v1, v0 + ((int)((16 - (reinterpret_cast<uintptr_t>(row + v0) & 15)) & 15) >> 2));
  b4 = a4 + ((v1 - a4) & ~3);
}

template <bool ENT>
__global__ void __launch_bounds__(kPolThreads)
    policy_stats_kernel(int V, int S, Base2 c, const float* __restrict__ logits, const int32_t* __restrict__ tokens,
                        const float* __restrict__ weights, float4* __restrict__ stats, float* __restrict__ xy) {
  __shared__ SoftPart red[kPolWaves];
  const int row = blockIdx.x, sl = blockIdx.y;
  if (weights && weights[row] == 0.f) return;
  const float* x = logits + (size_t)row * V;
  int v0, v1, a4, b4;
  row_slice(x, V, sl, S, v0, v1);
  slice_vectors(x, v0, v1, a4, b4);
  SoftPart p{-INFINITY, 0.f, 0.f};
  const float4* x4 = reinterpret_cast<const float4*>(x + a4);
  const int n4 = (b4 - a4) >> 2;
  int q = threadIdx.x;
  for (; q + 3 * kPolThreads < n4; q += 4 * kPolThreads) {
    const float4 f0 = x4[q], f1 = x4[q + kPolThreads], f2 = x4[q + 2 * kPolThreads], f3 = x4[q + 3 * kPolThreads];
    const float f[16] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w,
                         f2.x, f2.y, f2.z, f2.w, f3.x, f3.y, f3.z, f3.w};
    soft_add<16, ENT>(p, f, c);
  }
  for (; q < n4; q += kPolThreads) {
    const float4 f0 = x4[q];
    const float f[4] = {f0.x, f0.y, f0.z, f0.w};
    soft_add<4, ENT>(p, f, c);
  }
  const int outer = (a4 - v0) + (v1 - b4);  // at most 6
  if ((int)threadIdx.x < outer) {
    const int e = threadIdx.x, v = e < a4 - v0 ? v0 + e : b4 + e - (a4 - v0);
    const float f[1] = {x[v]};
    soft_add<1, ENT>(p, f, c);
  }
  p = wave_soft(p, c);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = p;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kPolWaves; ++w) p = soft_merge(p, red[w], c);
    stats[(size_t)row * S + sl] = float4{p.m, p.s, p.u, 0.f};
    const int y = clamp_id(tokens[row], V);
    if (y >= v0 && y < v1) xy[row] = x[y];
  }
}

// One row's statistics, its slices merged in order.
__device__ __forceinline__ SoftPart row_part(const float4* __restrict__ stats, int row, int S, Base2 c) {
  SoftPart p{-INFINITY, 0.f, 0.f};
  for (int q = 0; q < S; ++q) {
    const float4 f = stats[(size_t)row * S + q];
    p = soft_merge(p, SoftPart{f.x, f.y, f.z}, c);
  }
  return p;
}

__global__ void __launch_bounds__(kPolThreads)
    logprobs_rows_kernel(int rows, int S, Base2 c, double inv_t, const float4* __restrict__ stats,
                         const float* __restrict__ xy, const float* __restrict__ weights, float* __restrict__ logp,
                         float* __restrict__ entropy) {
  const int row = blockIdx.x * kPolThreads + threadIdx.x;
  if (row >= rows) return;
  float lp = 0.f, h = 0.f;
  if (!(weights && weights[row] == 0.f)) {
    const SoftPart p = row_part(stats, row, S, c);
    if (p.m == -INFINITY) {
      lp = -INFINITY;
    } else {
      const double ln_s = log((double)p.s);
      lp = (float)(((double)xy[row] - (double)p.m) * inv_t - ln_s);
      h = (float)(ln_s - 0.6931471805599453 * ((double)p.u / (double)p.s));
    }
  }
  logp[row] = lp;
  if (entropy) entropy[row] = h;
}

struct PolicyDev {
  int rows, V, S;
  Base2 c;
  double inv_t, lo, hi, beta;  // clip range limits; KL coefficient
  const float *logits, *old_logp, *ref_logp, *advantages, *weights;
  const int32_t* tokens;
  const float4* stats;
  const float* xy;
  float *loss, *logp, *kl, *grad;
};

struct RowTerms {
  float logp, kl;
  double term, coef;  // weighted loss term; derivative with respect to the row's logit of the token (1 - p_y aside)
};

__device__ __forceinline__ RowTerms row_terms(const PolicyDev& a, int row, SoftPart p) {
  RowTerms r{-INFINITY, 0.f, 0.0, 0.0};
  if (p.m == -INFINITY) return r;  // no distribution
  const double lp = ((double)a.xy[row] - (double)p.m) * a.inv_t - log((double)p.s);
  const double w = a.weights ? (double)a.weights[row] : 1.0 / a.rows;
  const double adv = a.advantages[row], ratio = exp(lp - (double)a.old_logp[row]);
  const bool inside = adv >= 0.0 ? ratio <= a.hi : ratio >= a.lo;
  // (an advantage of 0 stays 0 whatever the ratio)
  double l = 0.0, g = 0.0;
  if (adv != 0.0) {
    l = inside ? -ratio * adv : -(adv >= 0.0 ? a.hi : a.lo) * adv;
    g = inside ? -ratio * adv : 0.0;
    if (ratio != ratio) l = g = ratio;
  }
  if (a.ref_logp) {
    const double d = (double)a.ref_logp[row] - lp, e = expm1(d);
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

// Workgroup 0: every row's logp and kl, and the loss, each thread adding rows
// t, t + 256, ... in order and a fixed tree over the threads' sums.
__device__ void policy_rows(const PolicyDev& a) {
  __shared__ double part[kPolThreads];
  double acc = 0.0;
  for (int row = threadIdx.x; row < a.rows; row += kPolThreads) {
    RowTerms r{0.f, 0.f, 0.0, 0.0};
    if (!(a.weights && a.weights[row] == 0.f)) r = row_terms(a, row, row_part(a.stats, row, a.S, a.c));
    if (a.logp) a.logp[row] = r.logp;
    if (a.kl) a.kl[row] = r.kl;
    acc += r.term;
  }
  part[threadIdx.x] = acc;
  __syncthreads();
  for (int h = kPolThreads / 2; h > 0; h >>= 1) {
    if ((int)threadIdx.x < h) part[threadIdx.x] += part[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.loss[0] = (float)part[0];
}

__global__ void __launch_bounds__(kPolThreads) policy_grad_kernel(PolicyDev a) {
  if (blockIdx.x == 0) {
    policy_rows(a);
    return;
  }
  __shared__ float sh[3];
  const unsigned b = blockIdx.x - 1;
  const int row = (int)(b / (unsigned)a.S), sl = (int)(b % (unsigned)a.S);
  float m = 0.f, k = 0.f, coef = 0.f;
  if (!(a.weights && a.weights[row] == 0.f)) {
    if (threadIdx.x < 64) {
      // each lane takes one slice (S <= 32)
      const int q = threadIdx.x;
      SoftPart p{-INFINITY, 0.f, 0.f};
      if (q < a.S) {
        const float4 f = a.stats[(size_t)row * a.S + q];
        p = SoftPart{f.x, f.y, f.z};
      }
      p = wave_soft(p, a.c);
      if (q == 0) {
        const RowTerms r = row_terms(a, row, p);
        sh[0] = p.m;
        sh[1] = r.coef == 0.0 ? 0.f : (float)(-r.coef / (double)p.s);
        sh[2] = (float)r.coef;
      }
    }
    __syncthreads();
    m = sh[0];
    k = sh[1];
    coef = sh[2];
  }
  const float* x = a.logits + (size_t)row * a.V;
  float* g = a.grad + (size_t)row * a.V;
  int v0, v1, a4, b4;
  row_slice(x, a.V, sl, a.S, v0, v1);
  slice_vectors(g, v0, v1, a4, b4);
  const int y = clamp_id(a.tokens[row], a.V);
  const int n4 = (b4 - a4) >> 2;
  if (k == 0.f && coef == 0.f) {  // no gradient here: nothing is read
    for (int q = threadIdx.x; q < n4; q += kPolThreads)
      *reinterpret_cast<float4*>(g + a4 + 4 * q) = float4{0.f, 0.f, 0.f, 0.f};
    const int outer = (a4 - v0) + (v1 - b4);
    if ((int)threadIdx.x < outer) {
      const int e = threadIdx.x, v = e < a4 - v0 ? v0 + e : b4 + e - (a4 - v0);
      g[v] = 0.f;
    }
    return;
  }
  auto one = [&](float xv, int v) {
    const float e = k * __builtin_amdgcn_exp2f(base2(xv, m, a.c));
    return v == y ? e + coef : e;
  };
  if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(g)) & 15u) == 0) {
    for (int q = threadIdx.x; q < n4; q += kPolThreads) {
      const int v = a4 + 4 * q;
      const float4 f = *reinterpret_cast<const float4*>(x + v);
      *reinterpret_cast<float4*>(g + v) = float4{one(f.x, v), one(f.y, v + 1), one(f.z, v + 2), one(f.w, v + 3)};
    }
    const int outer = (a4 - v0) + (v1 - b4);
    if ((int)threadIdx.x < outer) {
      const int e = threadIdx.x, v = e < a4 - v0 ? v0 + e : b4 + e - (a4 - v0);
      g[v] = one(x[v], v);
    }
  } else {
    for (int v = v0 + threadIdx.x; v < v1; v += kPolThreads) g[v] = one(x[v], v);
  }
}

static Base2 base2_factor(float temperature) {
  const double c = 1.4426950408889634 / (double)temperature;
  const float hi = (float)c;
  return Base2{hi, (float)(c - (double)hi)};
}

template <bool ENT>
static void launch_stats(int rows, int V, int S, Base2 c, const float* logits, const int32_t* tokens,
                         const float* weights, float4* stats, float* xy, hipStream_t s) {
  hipLaunchKernelGGL((policy_stats_kernel<ENT>), dim3((unsigned)rows, (unsigned)S), dim3(kPolThreads), 0, s, V, S, c,
                     logits, tokens, weights, stats, xy);
}

hipError_t launch_token_logprobs(int B, int K, int V, const float* logits, const int32_t* tokens, const float* weights,
                                 float temperature, float* logp, float* entropy, const PolicyPlan& plan,
                                 void* workspace, hipStream_t s) {
  if (B <= 0) return hipSuccess;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  float4* stats = reinterpret_cast<float4*>(ws + plan.stats);
  float* xy = reinterpret_cast<float*>(ws + plan.xy);
  const int rows = B * K;
  const Base2 c = base2_factor(temperature);
  if (entropy)
    launch_stats<true>(rows, V, plan.S, c, logits, tokens, weights, stats, xy, s);
  else
    launch_stats<false>(rows, V, plan.S, c, logits, tokens, weights, stats, xy, s);
  hipLaunchKernelGGL(logprobs_rows_kernel, dim3((unsigned)((rows + kPolThreads - 1) / kPolThreads)), dim3(kPolThreads),
                     0, s, rows, plan.S, c, 1.0 / (double)temperature, stats, xy, weights, logp, entropy);
  return hipGetLastError();
}

hipError_t launch_policy_loss(const PolicyArgs& a, const PolicyPlan& plan, void* workspace, hipStream_t s) {
  if (a.B <= 0) return hipSuccess;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  float4* stats = reinterpret_cast<float4*>(ws + plan.stats);
  float* xy = reinterpret_cast<float*>(ws + plan.xy);
  const int rows = a.B * a.K;
  const PolicyDev d{rows,
                    a.V,
                    plan.S,
                    base2_factor(a.temperature),
                    1.0 / (double)a.temperature,
                    1.0 - (double)a.clip_low,
                    1.0 + (double)a.clip_high,
                    (double)a.kl_coef,
                    a.logits,
                    a.old_logp,
                    a.ref_logp,
                    a.advantages,
                    a.weights,
                    a.tokens,
                    stats,
                    xy,
                    a.loss,
                    a.logp,
                    a.kl,
                    a.grad};
  launch_stats<false>(rows, a.V, plan.S, d.c, a.logits, a.tokens, a.weights, stats, xy, s);
  const unsigned grid = a.grad ? 1u + (unsigned)rows * (unsigned)plan.S : 1u;
  hipLaunchKernelGGL(policy_grad_kernel, dim3(grid), dim3(kPolThreads), 0, s, d);
  return hipGetLastError();
}

}  // namespace domino
