"""Cases of the 8-bit roll-out and policy-training operators of the draft head.

Four operators are measured: the row quantiser, the base logits of an 8-bit LM
head, the log-probabilities of drafted tokens, and the clipped policy loss
with its gradient.  `run` computes them in elementary torch operations, or
through the library where `own` is true; `exact` states them in 64 bits.
"""
import math

import torch

own = False

V = 151936  # the vocabulary of the Qwen3 heads


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the hidden states of one draft block before the 8-bit LM head: a latency-bound call in every draft step
        {"name": "quantize_one_block", "op": "quantize", "rows": 16, "cols": 4096, "type": "bf16"},
        # float32 hidden states of a batch of blocks at an odd row count
        {"name": "quantize_f32_batch", "op": "quantize", "rows": 645, "cols": 2560, "type": "f32"},
        # a whole bf16 LM head, each time its weights are loaded or refreshed
        {"name": "quantize_lm_head", "op": "quantize", "rows": V, "cols": 4096, "type": "bf16"},
        # one block of a Qwen3-8B head: the serving path of a single request
        {"name": "logits_one_block", "op": "logits", "batch": 1, "block": 16, "d": 4096, "vocab": V},
        # eight requests on a Qwen3-4B head
        {"name": "logits_8_blocks", "op": "logits", "batch": 8, "block": 16, "d": 2560, "vocab": V},
        # a roll-out batch of 32 blocks on a Qwen3-8B head
        {"name": "logits_32_blocks", "op": "logits", "batch": 32, "block": 16, "d": 4096, "vocab": V},
        # short blocks on a small head whose sizes fit no tile
        {"name": "logits_ragged", "op": "logits", "batch": 7, "block": 5, "d": 96, "vocab": 4099},
        # drafted tokens of one block, with the entropy that a roll-out logs
        {"name": "logprobs_one_block", "op": "logprobs", "batch": 1, "block": 16, "vocab": V, "cut": False, "temperature": 1.0},
        # a batch of drafts cut at their acceptance lengths, sampled at T = 0.7
        {"name": "logprobs_64_blocks_cut", "op": "logprobs", "batch": 64, "block": 16, "vocab": V, "cut": True, "temperature": 0.7},
        # a policy step on one block
        {"name": "policy_one_block", "op": "policy", "batch": 1, "block": 16, "vocab": V, "cut": False, "temperature": 1.0, "kl": 0.05},
        # the training batch: 32 blocks, every position live, with a KL term
        {"name": "policy_32_blocks", "op": "policy", "batch": 32, "block": 16, "vocab": V, "cut": False, "temperature": 1.0, "kl": 0.05},
        # a padded batch of short drafts over an odd vocabulary: rows of any alignment, blocks without a live row, no KL term
        {"name": "policy_odd_vocab_cut", "op": "policy", "batch": 48, "block": 7, "vocab": 49999, "cut": True, "temperature": 0.8, "kl": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "logits", "logprobs", "policy"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, V), "cols": 32 * _log_int(rng, 1, 128), "type": rng.choice(["bf16", "f32"])}
    batch, block = _log_int(rng, 1, 32), rng.choice([1, 3, 5, 8, 16, 16, 16])
    if op == "logits":
        return {"op": op, "batch": batch, "block": block, "d": 32 * _log_int(rng, 2, 128), "vocab": _log_int(rng, 700, V)}
    case = {"op": op, "batch": batch, "block": block, "vocab": _log_int(rng, 700, V), "cut": rng.random() < 0.4,
            "temperature": round(rng.uniform(0.6, 1.3), 2)}
    if op == "policy":
        case["kl"] = rng.choice([0.0, 0.05, 0.1])
    return case


def _lengths(case):
    """Live positions of each block: all of them, or a pattern of acceptance lengths with empty blocks in it."""
    B, K = case["batch"], case["block"]
    return [(5 * b + 3) % (K + 1) if case["cut"] else K for b in range(B)]


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 if case["type"] == "bf16" else 4) + n + 4 * case["rows"], "flops": 3 * n}
    if case["op"] == "logits":
        M, d, v = case["batch"] * case["block"], case["d"], case["vocab"]
        return {"bytes": M * d + v * d + 4 * (M + v) + 4 * M * v, "flops": 2 * M * d * v}
    rows, live, v = case["batch"] * case["block"], sum(_lengths(case)), case["vocab"]
    if case["op"] == "logprobs":
        return {"bytes": 4 * live * v + 16 * rows, "flops": 6 * live * v}
    return {"bytes": 4 * live * v + 4 * rows * v + 28 * rows, "flops": 8 * live * v}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _to_int8(x):
    """Weights or activations as a checkpoint holds them in 8 bits: symmetric, one scale a row."""
    scale = (x.abs().amax(-1) / 127).float()
    return (x / scale.unsqueeze(-1)).round().clamp(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "quantize":
        x = normal(case["rows"], case["cols"]) * (0.5 + normal(case["rows"], 1).abs())
        x = x.to(torch.bfloat16) if case["type"] == "bf16" else x
        return {"case": case, "x": x, "q": torch.empty(x.shape, dtype=torch.int8, device="cuda"),
                "scale": torch.empty(x.shape[0], device="cuda")}
    B, K, v = case["batch"], case["block"], case["vocab"]
    if case["op"] == "logits":
        hq, hs = _to_int8(normal(B, K, case["d"]))
        wq, ws = _to_int8(normal(v, case["d"]) * 0.02)
        return {"case": case, "hidden_q": hq, "hidden_scale": hs, "lm_head_q": wq, "lm_head_scale": ws,
                "out": torch.empty((B, K, v), device="cuda")}
    # logits of a draft head: a broad tail and a few likely tokens a position; the tokens are drawn from them
    T = case["temperature"]
    logits = normal(B, K, v) * 2
    likely = torch.randint(0, v, (B, K, 8), generator=g, device="cuda")
    logits.scatter_add_(2, likely, normal(B, K, 8) * 3 + 10)
    noise = -torch.empty((B, K, v), device="cuda").exponential_(generator=g).log_()
    tokens = noise.add_(logits / T).argmax(-1).to(torch.int32)
    del noise
    live = torch.arange(K, device="cuda") < torch.tensor(_lengths(case), device="cuda").unsqueeze(1)
    weights = live.float() / max(1, sum(_lengths(case)))
    state = {"case": case, "logits": logits, "tokens": tokens, "weights": weights if case["cut"] else None,
             "logp": torch.empty((B, K), device="cuda")}
    if case["op"] == "logprobs":
        return state | {"entropy": torch.empty((B, K), device="cuda")}
    # log-probabilities kept from the roll-out and the reference: the present ones with noise of a fine grid, off by
    # half a step so that no ratio lies on the border of the clip range
    now = torch.log_softmax(logits / T, -1).gather(2, tokens.long().unsqueeze(2)).squeeze(2)
    old = now - ((normal(B, K) * 0.15 * 64).floor() + 0.5) / 64
    ref = now + ((normal(B, K) * 0.3 * 64).floor() + 0.5) / 64
    adv = normal(B, 1).expand(B, K) + 0.1 * normal(B, K)
    return state | {"old_logp": old, "ref_logp": ref, "advantages": adv.contiguous(), "loss": torch.empty(1, device="cuda"),
                    "kl": torch.empty((B, K), device="cuda"), "grad": torch.empty_like(logits)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def _run_own(s):
    import draft_block_causal_amd as D

    c = s["case"]
    if c["op"] == "quantize":
        D.domino_quantize_rows(s["x"], q=s["q"], scale=s["scale"])
        return s["q"], s["scale"]
    if c["op"] == "logits":
        return D.domino_base_logits_i8(s["hidden_q"], s["hidden_scale"], s["lm_head_q"], s["lm_head_scale"], base_logits=s["out"])
    if "workspace" not in s:  # kept by a program from step to step
        size = D.domino_token_logprobs_workspace_size if c["op"] == "logprobs" else D.domino_policy_loss_workspace_size
        s["workspace"] = torch.empty(size(c["batch"], c["block"], c["vocab"]), dtype=torch.uint8, device="cuda")
    if c["op"] == "logprobs":
        D.domino_token_logprobs(s["logits"], s["tokens"], temperature=c["temperature"], weights=s["weights"], logp=s["logp"],
                                entropy=s["entropy"], workspace=s["workspace"])
        return s["logp"], s["entropy"]
    D.domino_policy_loss(s["logits"], s["tokens"], s["old_logp"], s["advantages"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                         kl_coef=c["kl"], ref_logp=s["ref_logp"], weights=s["weights"], temperature=c["temperature"],
                         loss=s["loss"], logp=s["logp"], kl=s["kl"], grad=s["grad"], workspace=s["workspace"])
    return s["loss"], s["logp"], s["kl"], s["grad"]


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "quantize":
        # bfloat16 values have exact products and correctly decided quotients in 32 bits, float32 ones need 64
        x = state["x"].float() if c["type"] == "bf16" else state["x"].double()
        top = x.abs().amax(-1, keepdim=True)
        q = torch.where(top > 0, x * 127 / top, 0).round().to(torch.int8)
        return q, (top.squeeze(-1) / 127).float()
    if c["op"] == "logits":
        h, w = state["hidden_q"].float(), state["lm_head_q"].float()
        y = h.view(-1, c["d"]) @ w.T
        return (y * state["hidden_scale"].view(-1, 1) * state["lm_head_scale"]).view(c["batch"], c["block"], c["vocab"])
    T, x, tokens = c["temperature"], state["logits"], state["tokens"].long().unsqueeze(2)
    if c["cut"]:
        live = state["weights"] != 0
    z = x - x.amax(2, keepdim=True)
    if T != 1.0:
        z = z / T
    e = z.exp()
    total = e.sum(2, keepdim=True, dtype=torch.float64)
    log_total = total.log().squeeze(2)
    # the log-probabilities stay in 64 bits until the ratios are formed: a KL term is a small difference of them
    lp = z.gather(2, tokens).squeeze(2).double() - log_total
    if c["op"] == "logprobs":
        ent = log_total - (e * z).sum(2, dtype=torch.float64) / total.squeeze(2)
        if c["cut"]:
            lp, ent = torch.where(live, lp, 0), torch.where(live, ent, 0)
        return lp.float(), ent.float()
    w = state["weights"].double() if c["cut"] else 1.0 / (c["batch"] * c["block"])
    A = state["advantages"].double()
    ratio = (lp - state["old_logp"].double()).exp()
    plain, clipped = ratio * A, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * A
    d = state["ref_logp"].double() - lp
    kl = d.exp() - d - 1
    loss = (w * (c["kl"] * kl - torch.minimum(plain, clipped))).sum()
    coef = w / T * (c["kl"] * (1 - d.exp()) - torch.where(plain <= clipped, plain, 0))
    grad = e * (-coef / total.squeeze(2)).float().unsqueeze(2)
    grad.scatter_add_(2, tokens, coef.float().unsqueeze(2))
    if c["cut"]:
        lp, kl = torch.where(live, lp, 0), torch.where(live, kl, 0)
    return loss.float().view(1), lp.float(), kl.float(), grad


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        q = torch.empty_like(s["q"])
        scale = torch.empty(case["rows"], dtype=torch.float64, device="cuda")
        step = 1 << 14
        for r in range(0, case["rows"], step):
            x = s["x"][r:r + step].double()
            scale[r:r + step] = torch.linalg.vector_norm(x, ord=math.inf, dim=1) / 127
            q[r:r + step] = torch.round(x * 127 / (127 * scale[r:r + step, None]).clamp_min(1e-300)).to(torch.int8)
        return None, scale
    if case["op"] == "logits":
        h = s["hidden_q"].double().flatten(0, 1) * s["hidden_scale"].double().reshape(-1, 1)
        out = torch.empty((h.shape[0], case["vocab"]), dtype=torch.float64, device="cuda")
        step = 1 << 14
        for v in range(0, case["vocab"], step):
            w = s["lm_head_q"][v:v + step].double() * s["lm_head_scale"][v:v + step].double().unsqueeze(1)
            out[:, v:v + step] = h @ w.T
        return out.view(case["batch"], case["block"], case["vocab"])
    B, K, v = case["batch"], case["block"], case["vocab"]
    T = case["temperature"]
    lengths = _lengths(case)
    lp, second = (torch.zeros((B, K), dtype=torch.float64, device="cuda") for _ in range(2))
    policy = case["op"] == "policy"
    if policy:
        loss = torch.zeros(1, dtype=torch.float64, device="cuda")
        grad = torch.zeros((B, K, v), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lengths[b]
        if n == 0:
            continue
        logp = torch.log_softmax(s["logits"][b, :n].double() / T, -1)
        y = s["tokens"][b, :n].long()
        at = torch.arange(n, device="cuda")
        p, a = logp.exp(), logp[at, y]
        lp[b, :n] = a
        if not policy:
            second[b, :n] = -(p * logp).sum(-1)
            continue
        A, r, d = s["advantages"][b, :n].double(), torch.exp(a - s["old_logp"][b, :n]), s["ref_logp"][b, :n] - a
        inside = torch.where(A >= 0, r <= 1 + CLIP_HIGH, r >= 1 - CLIP_LOW)
        border = torch.where(A >= 0, 1 + CLIP_HIGH, 1 - CLIP_LOW)
        second[b, :n] = torch.expm1(d) - d
        w = s["weights"][b, :n].double() if case["cut"] else torch.full_like(A, 1.0 / (B * K))
        loss += (w * (case["kl"] * second[b, :n] - torch.where(inside, r, border) * A)).sum()
        slope = w * (-case["kl"] * torch.expm1(d) - torch.where(inside, r * A, 0)) / T
        one = torch.zeros_like(p)
        one[at, y] = 1
        grad[b, :n] = slope.unsqueeze(1) * (one - p)
    return (loss, lp, second, grad) if policy else (lp, second)
