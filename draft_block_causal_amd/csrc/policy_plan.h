// Arguments, launch shape and workspace layout of the drafted-token
// log-probabilities and the clipped policy loss (host-only arithmetic, shared
// by the launchers and the argument checks).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace domino {

constexpr int kMaxPolicyBlock = 1024;     // positions per block
constexpr int kMaxPolicyBatch = 1 << 20;  // blocks per call
// Positions per call: a launch counts its threads (256 a position and slice)
// in 32 bits.
constexpr int kMaxPolicyRows = 1 << 22;

struct PolicyArgs {
  int32_t B, K, V;
  const float* logits;      // [B K][V]
  const int32_t* tokens;    // [B K], as are the following
  const float *old_logp, *ref_logp, *advantages, *weights;
  double temperature, clip_low, clip_high, kl_coef;
  float *loss, *logp, *kl, *grad;  // [1], [B K], [B K], [B K][V]; all but loss may be null
};

constexpr size_t kPolicyPart = 24;  // float, double, double

struct PolicyPlan {
  int S;         // vocabulary slices per row
  size_t stats;  // byte offset of the [B K][S] partials (max, sum, sum of e t: kPolicyPart bytes)
  size_t xy;     // byte offset of the [B K] float logits of the tokens
  size_t terms;  // byte offset of the [B K] double loss terms of rows held on chip
  size_t sums;   // byte offset of the [B K] double sums of groups of rows
  size_t ticket;  // byte offset of a counter of finished workgroups
  size_t total;  // workspace bytes
};

// About 8192 workgroups (positions that are not read leave at once, so that the
// others must be many to spread evenly), each slice at least 2048 entries long, and at most 32
// slices per row (one wave merges a row's partials).
inline PolicyPlan policy_plan(int B, int K, int V) {
  auto align256 = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PolicyPlan p{};
  const long rows = (long)B * K;
  long S = (8192 + rows - 1) / rows;
  long smax = V / 2048 > 1 ? V / 2048 : 1;
  smax = smax > 32 ? 32 : smax;
  S = S < 1 ? 1 : S > smax ? smax : S;
  p.S = (int)S;
  p.stats = 0;
  p.xy = align256((size_t)rows * p.S * kPolicyPart);
  p.terms = align256(p.xy + (size_t)rows * 4);
  p.sums = align256(p.terms + (size_t)rows * 8);
  p.ticket = align256(p.sums + (size_t)rows * 8);
  p.total = p.ticket + 256;
  return p;
}

}  // namespace domino
