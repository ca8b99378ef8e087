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

// Slices of a row: enough for about 1024 workgroups as long as each has 2048
// entries, and, with 16384 entries each, for up to 8192 (positions that are not
// read leave at once, so that the others must be many to spread evenly); at
// most 32, since 32 lanes bring a row's slices together.
inline PolicyPlan policy_plan(int B, int K, int V) {
  auto align256 = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PolicyPlan p{};
  const long rows = (long)B * K;
  auto slices = [&](long workgroups, long entries) {
    const long want = (workgroups + rows - 1) / rows, most = V / entries;
    return want < most ? want : most;
  };
  const long few = slices(1024, 2048), many = slices(8192, 16384);
  long S = few > many ? few : many;
  S = S < 1 ? 1 : S > 32 ? 32 : S;
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
