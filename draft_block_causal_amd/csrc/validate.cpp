// Host-only argument validation and workspace layout of the Domino C ABI.
// Pure C++ (no HIP calls), so it can also be built and sanitised on a CPU.
#include "validate.h"
#include "kernels.h"

#include "psplit.h"

#include <cmath>
#include <initializer_list>

namespace domino {

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_size(int dtype) { return dtype == DOMINO_BF16 ? 2 : 4; }

int check_head(const domino_head* h) {
  if (!h) return DOMINO_ERR_NULL;
  if (h->dtype != DOMINO_F32 && h->dtype != DOMINO_BF16) return DOMINO_ERR_DTYPE;
  if (h->d <= 0 || h->vocab <= 0 || h->gru_hidden <= 0 || h->rank <= 0 || h->block <= 0) return DOMINO_ERR_SHAPE;
  if (h->d % 32 || h->gru_hidden % 32 || h->rank % 32) return DOMINO_ERR_SHAPE;
  if (h->block > kMaxBlock) return DOMINO_ERR_SHAPE;
  if (!h->lm_head || !h->embed || !h->w_ih || !h->w_hh || !h->w1 || !h->w2) return DOMINO_ERR_NULL;
  const void* mats[] = {h->lm_head, h->embed, h->w_ih, h->w_hh, h->w1, h->w2};
  for (const void* p : mats)
    if (!aligned16(p)) return DOMINO_ERR_ALIGN;
  if (h->gru_input_table && !aligned16(h->gru_input_table)) return DOMINO_ERR_ALIGN;
  const long es = elem_size(h->dtype);
  if ((long)h->d * es > kMaxRowBytes) return DOMINO_ERR_UNSUPPORTED;
  if (h->gru_hidden > kMaxGruHidden || h->rank > kMaxRank) return DOMINO_ERR_UNSUPPORTED;
  if (h->vocab > kMaxVocab) return DOMINO_ERR_UNSUPPORTED;
  return DOMINO_OK;
}

// ks: K-split of the W_ih e product, so that one 16-row tile of W_ih is shared
// by several waves; the slice must stay a multiple of 32 elements.
int gru_ksplit(int d) {
  for (int ks : {4, 2})
    if (d % (32 * ks) == 0) return ks;
  return 1;
}

static size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

WorkspaceLayout workspace_layout(const domino_head* h, int batch) {
  WorkspaceLayout w{};
  const size_t B = (size_t)batch, K = (size_t)h->block, H = (size_t)h->gru_hidden, r = (size_t)h->rank;
  const size_t ks = (size_t)gru_ksplit(h->d);
  size_t off = 0;
  w.keys = off;
  off += up256((K * B + 2) * sizeof(unsigned long long));  // keys + loop control words
  w.P = off;
  off += up256(B * K * r * sizeof(float));
  // K-slice partials of the hidden half of W1 h (bf16 heads): the single-block
  // loop and the per-position kernels add them up
  w.ppart = off;
  PSplit ps;
  if (h->dtype == DOMINO_BF16 && p_split_shape(h->d, h->rank, ps))
    off += up256((size_t)ps.S * B * K * r * sizeof(float));
  w.part_ih = off;
  off += up256(ks * B * 3 * H * sizeof(float));
  w.part_hh = off;
  off += up256(B * 3 * H * sizeof(float));
  w.u = off;
  off += up256(B * r * sizeof(float));
  w.states = off;
  off += up256(B * K * H * sizeof(float));
  // tagged exchange words of the persistent loop: partials, GRU state, u, keys,
  // each double-buffered by position parity
  const size_t multi = 2 * ((ks + 1) * B * 3 * H + B * H + B * r + (size_t)kMaxLoopWorkgroups * B);
  const size_t single = b1_exchange_words((int)H, (int)r, kMaxLoopWorkgroups);
  const size_t blocks = bn_exchange_words(batch, kMaxLoopWorkgroups, (int)H, (int)r);
  w.xwords = multi > single ? multi : single;
  if (blocks > w.xwords) w.xwords = blocks;
  w.xchg = off;
  off += up256(w.xwords * sizeof(unsigned long long));
  w.total = off;
  w.ks = (int)ks;
  return w;
}

bool forms_base_logits(const domino_head* h, int32_t batch) {
  return batch == 1 && h->dtype == DOMINO_BF16 && h->gru_input_table && h->block <= 16 &&
         (h->d == 2560 || h->d == 4096) && h->gru_hidden == 1024 && h->rank == 256;
}

int check_draft_io(const domino_head* h, int32_t batch, const void* hidden, const float* base_logits,
                   const int32_t* x_t, float temperature, int32_t* tokens, const float* logits,
                   const float* gru_states) {
  int st = check_head(h);
  if (st != DOMINO_OK) return st;
  if (batch < 0) return DOMINO_ERR_SHAPE;
  if (batch > kMaxBatch) return DOMINO_ERR_UNSUPPORTED;
  if (!std::isfinite(temperature) || temperature < 0.f) return DOMINO_ERR_ARG;
  if (batch == 0) return DOMINO_OK;
  if (!hidden || !x_t || !tokens) return DOMINO_ERR_NULL;
  if (!base_logits && !forms_base_logits(h, batch)) return DOMINO_ERR_UNSUPPORTED;
  if (!aligned16(hidden) || (base_logits && !aligned16(base_logits)) || !aligned16(tokens)) return DOMINO_ERR_ALIGN;
  if ((logits && !aligned16(logits)) || (gru_states && !aligned16(gru_states))) return DOMINO_ERR_ALIGN;
  return DOMINO_OK;
}

int check_draft_args(const domino_head* h, int32_t batch, const void* hidden, const float* base_logits,
                     const int32_t* x_t, float temperature, int32_t* tokens, const float* logits,
                     const float* gru_states, const void* workspace, size_t workspace_bytes) {
  int st = check_draft_io(h, batch, hidden, base_logits, x_t, temperature, tokens, logits, gru_states);
  if (st != DOMINO_OK || batch == 0) return st;
  const WorkspaceLayout w = workspace_layout(h, batch);
  if (!workspace) return DOMINO_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return DOMINO_ERR_WORKSPACE;
  if (workspace_bytes < w.total) return DOMINO_ERR_WORKSPACE;
  return DOMINO_OK;
}

int check_base_args(const domino_head* h, int32_t batch, const void* hidden, const float* base_logits) {
  int st = check_head(h);
  if (st != DOMINO_OK) return st;
  if (batch < 0) return DOMINO_ERR_SHAPE;
  if (batch > kMaxBatch) return DOMINO_ERR_UNSUPPORTED;
  if (batch == 0) return DOMINO_OK;
  if (!hidden || !base_logits) return DOMINO_ERR_NULL;
  if (!aligned16(hidden) || !aligned16(base_logits)) return DOMINO_ERR_ALIGN;
  return DOMINO_OK;
}

int check_accept_args(int32_t batch, int32_t block, const int32_t* draft, const int32_t* target,
                      const int32_t* accept) {
  if (batch < 0 || block <= 0 || block > 1024) return DOMINO_ERR_SHAPE;
  if (batch == 0) return DOMINO_OK;
  if (!draft || !target || !accept) return DOMINO_ERR_NULL;
  return DOMINO_OK;
}

size_t base_draft_workspace_bytes(int32_t batch, int32_t block) {
  if (batch < 1 || batch > kMaxVerifyBatch || block < 1 || block > 1024) return 0;
  return ((size_t)batch * block * 8 + 255) & ~(size_t)255;
}

int check_base_draft_args(int32_t batch, int32_t block, int32_t vocab, const float* base_logits, float temperature,
                          const int32_t* tokens, const void* workspace, size_t workspace_bytes) {
  if (batch < 0 || batch > kMaxVerifyBatch || block < 1 || block > 1024 || vocab < 1 || vocab > kMaxVocab)
    return DOMINO_ERR_SHAPE;
  if (!(temperature >= 0.f) || !std::isfinite(temperature)) return DOMINO_ERR_ARG;
  if (batch == 0) return DOMINO_OK;
  if (!base_logits || !tokens) return DOMINO_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(base_logits) & 3u) return DOMINO_ERR_ALIGN;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < base_draft_workspace_bytes(batch, block))
    return DOMINO_ERR_WORKSPACE;
  return DOMINO_OK;
}

int check_loss_args(int32_t batch, int32_t block, int32_t vocab, const float* base_logits, const float* final_logits,
                    const int32_t* targets, float lambda, float gamma, const float* loss, const float* ce_base,
                    const float* ce_final, const float* grad_base, const float* grad_final, const void* workspace,
                    size_t workspace_bytes) {
  if (batch < 0 || batch > kMaxLossBatch || block < 1 || block > kMaxLossBlock || vocab < 1 || vocab > kMaxVocab)
    return DOMINO_ERR_SHAPE;
  if (!std::isfinite(lambda) || lambda < 0.f || lambda > 1.f) return DOMINO_ERR_ARG;
  if (!std::isfinite(gamma) || !(gamma > 0.f) || gamma > 1.f) return DOMINO_ERR_ARG;
  if (batch == 0) return DOMINO_OK;
  if (!base_logits || !final_logits || !targets || !loss) return DOMINO_ERR_NULL;
  for (const void* q : {(const void*)base_logits, (const void*)final_logits, (const void*)loss, (const void*)ce_base,
                        (const void*)ce_final, (const void*)grad_base, (const void*)grad_final})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return DOMINO_ERR_ALIGN;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < loss_plan(batch, block, vocab).total)
    return DOMINO_ERR_WORKSPACE;
  return DOMINO_OK;
}

int check_backward_args(const domino_head* h, int32_t batch, const void* hidden, const float* gru_states,
                        const float* grad_final, const float* d_w2, const float* d_b2, const float* d_w1,
                        const float* d_b1, const float* d_states, const void* workspace, size_t workspace_bytes) {
  int st = check_head(h);
  if (st != DOMINO_OK) return st;
  if (batch < 0) return DOMINO_ERR_SHAPE;
  if (batch > kMaxBatch || h->rank > 512) return DOMINO_ERR_UNSUPPORTED;
  if (batch == 0) return DOMINO_OK;
  if (!hidden || !gru_states || !grad_final || !d_w2 || !d_w1) return DOMINO_ERR_NULL;
  if (!aligned16(hidden)) return DOMINO_ERR_ALIGN;
  for (const void* q : {(const void*)gru_states, (const void*)grad_final, (const void*)d_w2, (const void*)d_b2,
                        (const void*)d_w1, (const void*)d_b1, (const void*)d_states})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return DOMINO_ERR_ALIGN;
  const BackwardPlan pl = backward_plan(batch * h->block, h->rank, h->vocab, h->dtype, h->d + h->gru_hidden, h->gru_hidden);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < pl.total)
    return DOMINO_ERR_WORKSPACE;
  return DOMINO_OK;
}

int check_gru_backward_args(const domino_head* h, int32_t batch, const int32_t* x_t, const int32_t* teacher,
                            const float* gru_states, const float* d_states, const float* d_w_ih,
                            const float* d_w_hh, const float* d_b_ih, const float* d_b_hh, const void* workspace,
                            size_t workspace_bytes) {
  int st = check_head(h);
  if (st != DOMINO_OK) return st;
  if (batch < 0) return DOMINO_ERR_SHAPE;
  if (batch > kMaxBatch) return DOMINO_ERR_UNSUPPORTED;
  if (batch == 0) return DOMINO_OK;
  if (!x_t || !teacher || !gru_states || !d_states || !d_w_ih || !d_w_hh) return DOMINO_ERR_NULL;
  for (const void* q : {(const void*)x_t, (const void*)teacher, (const void*)gru_states, (const void*)d_states,
                        (const void*)d_w_ih, (const void*)d_w_hh, (const void*)d_b_ih, (const void*)d_b_hh})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return DOMINO_ERR_ALIGN;
  const GruBackwardPlan pl = gru_backward_plan(batch, h->block, h->d, h->gru_hidden, elem_size(h->dtype));
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < pl.total)
    return DOMINO_ERR_WORKSPACE;
  return DOMINO_OK;
}

int check_verify_args(int32_t batch, int32_t block, int32_t vocab, const float* target_logits,
                      const float* draft_logits, const int32_t* draft, float temperature, const int32_t* accept,
                      const int32_t* next_token, const void* workspace, size_t workspace_bytes) {
  if (batch < 0 || batch > kMaxVerifyBatch || block < 1 || block > kMaxVerifyBlock || vocab < 1 ||
      vocab > kMaxVocab)
    return DOMINO_ERR_SHAPE;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return DOMINO_ERR_ARG;
  if (batch == 0) return DOMINO_OK;
  if (!target_logits || !draft_logits || !draft || !accept || !next_token) return DOMINO_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(target_logits) & 3u) || (reinterpret_cast<uintptr_t>(draft_logits) & 3u))
    return DOMINO_ERR_ALIGN;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < verify_plan(batch, block, vocab).total)
    return DOMINO_ERR_WORKSPACE;
  return DOMINO_OK;
}

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte (a null
// pointer is no range).
static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < na : x - y < nb;
}

int check_quantize_args(int32_t rows, int32_t cols, int32_t dtype, const void* x, const int8_t* q,
                        const float* scale) {
  if (dtype != DOMINO_F32 && dtype != DOMINO_BF16) return DOMINO_ERR_DTYPE;
  if (rows < 0 || rows > kMaxVocab || cols < 32 || cols > kMaxI8Cols || cols % 32) return DOMINO_ERR_SHAPE;
  if (rows == 0) return DOMINO_OK;
  if (!x || !q || !scale) return DOMINO_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || (reinterpret_cast<uintptr_t>(scale) & 3u)) return DOMINO_ERR_ALIGN;
  const size_t n = (size_t)rows * cols, nx = n * elem_size(dtype), ns = (size_t)rows * 4;
  if (overlap(x, nx, q, n) || overlap(x, nx, scale, ns) || overlap(q, n, scale, ns)) return DOMINO_ERR_ARG;
  return DOMINO_OK;
}

int check_base_i8_args(int32_t batch, int32_t block, int32_t d, int32_t vocab, const int8_t* hidden_q,
                       const float* hidden_scale, const int8_t* lm_head_q, const float* lm_head_scale,
                       const float* base_logits) {
  if (batch < 0 || block < 1 || block > kMaxBlock || d < 32 || d > kMaxI8Cols || d % 32 || vocab < 1 ||
      vocab > kMaxVocab)
    return DOMINO_ERR_SHAPE;
  if (batch > kMaxBatch) return DOMINO_ERR_UNSUPPORTED;
  if (batch == 0) return DOMINO_OK;
  if (!hidden_q || !hidden_scale || !lm_head_q || !lm_head_scale || !base_logits) return DOMINO_ERR_NULL;
  if (!aligned16(hidden_q) || !aligned16(lm_head_q) || !aligned16(base_logits) ||
      (reinterpret_cast<uintptr_t>(hidden_scale) & 3u) || (reinterpret_cast<uintptr_t>(lm_head_scale) & 3u))
    return DOMINO_ERR_ALIGN;
  const size_t M = (size_t)batch * block, N = (size_t)vocab, D = (size_t)d;
  if (overlap(base_logits, M * N * 4, hidden_q, M * D) || overlap(base_logits, M * N * 4, hidden_scale, M * 4) ||
      overlap(base_logits, M * N * 4, lm_head_q, N * D) || overlap(base_logits, M * N * 4, lm_head_scale, N * 4))
    return DOMINO_ERR_ARG;
  return DOMINO_OK;
}

// (the kernels hold log2(e) / T as a pair of normal float32 numbers)
static bool bad_temperature(double t) { return !(t > 2e-38 && t < 1e20); }

static bool policy_shape(int32_t batch, int32_t block, int32_t vocab) {
  return batch >= 0 && batch <= kMaxPolicyBatch && block >= 1 && block <= kMaxPolicyBlock && vocab >= 1 &&
         vocab <= kMaxVocab;
}

struct Range {
  const void* p;
  size_t n;
};

// Whether an output overlaps an input or an output before it.
static bool any_overlap(std::initializer_list<Range> in, std::initializer_list<Range> out) {
  for (const Range* o = out.begin(); o != out.end(); ++o) {
    for (const Range& i : in)
      if (overlap(o->p, o->n, i.p, i.n)) return true;
    for (const Range* q = out.begin(); q != o; ++q)
      if (overlap(o->p, o->n, q->p, q->n)) return true;
  }
  return false;
}

static int check_policy_workspace(int32_t batch, int32_t block, int32_t vocab, const void* workspace, size_t bytes) {
  return !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                 bytes < policy_plan(batch, block, vocab).total
             ? DOMINO_ERR_WORKSPACE
             : DOMINO_OK;
}

int check_logprobs_args(int32_t batch, int32_t block, int32_t vocab, const float* logits, const int32_t* tokens,
                        const float* weights, double temperature, const float* logp, const float* entropy,
                        const void* workspace, size_t workspace_bytes) {
  if (!policy_shape(batch, block, vocab)) return DOMINO_ERR_SHAPE;
  if ((long)batch * block > kMaxPolicyRows) return DOMINO_ERR_UNSUPPORTED;
  if (bad_temperature(temperature)) return DOMINO_ERR_ARG;
  if (batch == 0) return DOMINO_OK;
  if (!logits || !tokens || !logp) return DOMINO_ERR_NULL;
  for (const void* q : {(const void*)logits, (const void*)tokens, (const void*)weights, (const void*)logp,
                        (const void*)entropy})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return DOMINO_ERR_ALIGN;
  const size_t r = (size_t)batch * block * 4;
  if (any_overlap({{logits, r * vocab}, {tokens, r}, {weights, r}},
                  {{logp, r}, {entropy, r}, {workspace, workspace_bytes}}))
    return DOMINO_ERR_ARG;
  return check_policy_workspace(batch, block, vocab, workspace, workspace_bytes);
}

int check_policy_args(const PolicyArgs& a, const void* workspace, size_t workspace_bytes) {
  if (!policy_shape(a.B, a.K, a.V)) return DOMINO_ERR_SHAPE;
  if ((long)a.B * a.K > kMaxPolicyRows) return DOMINO_ERR_UNSUPPORTED;
  if (bad_temperature(a.temperature)) return DOMINO_ERR_ARG;
  if (!std::isfinite(a.clip_low) || a.clip_low < 0.0 || a.clip_low > 1.0) return DOMINO_ERR_ARG;
  if (!std::isfinite(a.clip_high) || a.clip_high < 0.0) return DOMINO_ERR_ARG;
  if (!std::isfinite(a.kl_coef) || a.kl_coef < 0.0) return DOMINO_ERR_ARG;
  if (a.B == 0) return DOMINO_OK;
  if (!a.logits || !a.tokens || !a.old_logp || !a.advantages || !a.loss) return DOMINO_ERR_NULL;
  if (!a.ref_logp && a.kl_coef != 0.0) return DOMINO_ERR_NULL;
  for (const void* q : {(const void*)a.logits, (const void*)a.tokens, (const void*)a.old_logp,
                        (const void*)a.ref_logp, (const void*)a.advantages, (const void*)a.weights,
                        (const void*)a.loss, (const void*)a.logp, (const void*)a.kl, (const void*)a.grad})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return DOMINO_ERR_ALIGN;
  const size_t r = (size_t)a.B * a.K * 4, n = r * a.V;
  // (a gradient in the logits' own buffer is the one overlap allowed)
  const bool in_place = a.grad == a.logits;
  if (any_overlap({{in_place ? nullptr : a.logits, n}, {a.tokens, r}, {a.old_logp, r}, {a.ref_logp, r},
                   {a.advantages, r}, {a.weights, r}},
                  {{a.grad, n}, {a.loss, 4}, {a.logp, r}, {a.kl, r}, {workspace, workspace_bytes}}))
    return DOMINO_ERR_ARG;
  return check_policy_workspace(a.B, a.K, a.V, workspace, workspace_bytes);
}

}  // namespace domino

extern "C" const char* domino_status_string(int status) {
  switch (status) {
    case DOMINO_OK: return "ok";
    case DOMINO_ERR_NULL: return "a required pointer is NULL";
    case DOMINO_ERR_SHAPE: return "a size is out of range or not a multiple of 32";
    case DOMINO_ERR_DTYPE: return "unknown dtype code";
    case DOMINO_ERR_ALIGN: return "a pointer is not 16-byte aligned";
    case DOMINO_ERR_ARG: return "invalid scalar argument";
    case DOMINO_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
    case DOMINO_ERR_HIP: return "HIP runtime error";
    case DOMINO_ERR_UNSUPPORTED: return "request outside the library's limits";
    default: return "unknown status";
  }
}

extern "C" int domino_version(void) { return 100; }

extern "C" int domino_check_head(const domino_head* head) { return domino::check_head(head); }

extern "C" int domino_gru_table_size(const domino_head* head, size_t* bytes) {
  if (!bytes) return DOMINO_ERR_NULL;
  int st = domino::check_head(head);
  if (st != DOMINO_OK) return st;
  *bytes = (size_t)head->vocab * 3 * (size_t)head->gru_hidden * sizeof(float);
  return DOMINO_OK;
}

extern "C" int domino_workspace_size(const domino_head* head, int32_t batch, size_t* bytes) {
  if (!bytes) return DOMINO_ERR_NULL;
  int st = domino::check_head(head);
  if (st != DOMINO_OK) return st;
  if (batch < 0) return DOMINO_ERR_SHAPE;
  if (batch > domino::kMaxBatch) return DOMINO_ERR_UNSUPPORTED;
  *bytes = domino::workspace_layout(head, batch).total;
  return DOMINO_OK;
}
