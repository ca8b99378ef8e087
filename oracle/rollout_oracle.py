"""Plain float64 definitions of the 8-bit roll-out and policy-training calls.

TEST INFRASTRUCTURE, as domino_oracle: no code is shared with the HIP library.
Everything is written position by position from its formula.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

__all__ = ["quantize_row", "quantize_rows", "base_logits_i8", "token_logprobs", "policy_loss"]


def quantize_row(x):
    """One row in 8 bits in exact rational arithmetic: (q list, scale float64)."""
    if not np.all(np.isfinite(x)):
        return [0] * len(x), float("nan")
    fx = [Fraction(float(v)) for v in x]
    a = max(abs(v) for v in fx)
    if a == 0:
        return [0] * len(x), 0.0
    return [round(v * 127 / a) for v in fx], float(a / 127)  # round(): to nearest, ties to even


def quantize_rows(x):
    """Rows in 8 bits: q int8 and scale float64.  float64 decides every rounding of
    float32 values: 127 x is exact and a quotient differs from a half by 2^-32 or more,
    or by nothing."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x).all(-1)
    a = np.where(finite, np.abs(np.where(np.isfinite(x), x, 0)).max(-1), 0)
    safe = np.where(a > 0, a, 1)[..., None]
    q = np.where((finite & (a > 0))[..., None], np.rint(np.where(np.isfinite(x), x, 0) * 127 / safe), 0)
    return q.astype(np.int8), np.where(finite, a / 127, np.nan)


def base_logits_i8(hidden_q, hidden_scale, lm_head_q, lm_head_scale):
    s = np.asarray(hidden_q, dtype=np.float64) @ np.asarray(lm_head_q, dtype=np.float64).T
    return s * np.asarray(hidden_scale, np.float64)[..., None] * np.asarray(lm_head_scale, np.float64)


def _log_softmax(x, T):
    z = (x - x.max()) / T
    return z - np.log(np.exp(z).sum())


def token_logprobs(logits, tokens, T=1.0, weights=None):
    """(logp, entropy), each [B, K]."""
    B, K, V = logits.shape
    lp, h = np.zeros((B, K)), np.zeros((B, K))
    for b in range(B):
        for i in range(K):
            if weights is not None and weights[b, i] == 0:
                continue
            x = np.asarray(logits[b, i], dtype=np.float64)
            if np.all(x == -np.inf):
                lp[b, i] = -np.inf
                continue
            ls = _log_softmax(x, T)
            lp[b, i] = ls[min(max(int(tokens[b, i]), 0), V - 1)]
            p = np.exp(ls)
            h[b, i] = -np.sum(p[p > 0] * ls[p > 0])
    return lp, h


def policy_loss(logits, tokens, old, adv, clip_low=0.2, clip_high=0.2, beta=0.0, ref=None, weights=None, T=1.0):
    """dict(loss, logp, kl, grad, coef) of the clipped policy loss."""
    B, K, V = logits.shape
    w = np.full((B, K), 1.0 / (B * K)) if weights is None else np.asarray(weights, np.float64)
    lp, _ = token_logprobs(logits, tokens, T, weights)
    kl, grad, coef = np.zeros((B, K)), np.zeros((B, K, V)), np.zeros((B, K))
    loss = 0.0
    for b in range(B):
        for i in range(K):
            if w[b, i] == 0 or np.all(np.asarray(logits[b, i]) == -np.inf):
                continue
            y = min(max(int(tokens[b, i]), 0), V - 1)
            A, r = float(adv[b, i]), np.exp(lp[b, i] - float(old[b, i]))
            clipped = min(max(r, 1.0 - clip_low), 1.0 + clip_high)
            surrogate = min(r * A, clipped * A)
            # the slope of the smaller one; both are the same inside the range
            slope = -A * r if r * A <= clipped * A else 0.0
            value = -surrogate
            if ref is not None:
                d = float(ref[b, i]) - lp[b, i]
                kl[b, i] = np.expm1(d) - d
                value += beta * kl[b, i]
                slope += beta * (1.0 - np.exp(d))
            loss += w[b, i] * value
            coef[b, i] = w[b, i] * slope / T
            g = -np.exp(_log_softmax(np.asarray(logits[b, i], np.float64), T))
            g[y] += 1.0
            grad[b, i] = coef[b, i] * g
    return {"loss": loss, "logp": lp, "kl": kl, "grad": grad, "coef": coef}
