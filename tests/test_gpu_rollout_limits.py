"""The 8-bit roll-out and policy calls at the ends of their ranges: tensors of
more than 2^31 entries, the longest rows, the most rows, and calls that are
captured, replayed and run at the same time."""
import numpy as np
import pytest
import torch

import oracle as O
from _helpers import log

pytestmark = pytest.mark.gpu

E = 2.0**-24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_causal_amd as D

    D.load_library()
    torch.cuda.empty_cache()
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def test_quantize_more_than_2_31_values(dev):
    import draft_block_causal_amd as D

    rows, cols = 524288 + 37, 4096
    log("quantize past 2^31 values")
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev).normal_()
    q, scale = D.domino_quantize_rows(x)
    for r in (0, 262143, 262144, 524287, 524288, rows - 1):
        want_q, want_s = O.quantize_rows(x[r].float().cpu().numpy()[None])
        assert np.array_equal(q[r].cpu().numpy(), want_q[0]), r
        assert abs(scale[r].item() - want_s[0]) <= want_s[0] * E


def test_quantize_most_rows(dev):
    import draft_block_causal_amd as D

    rows = 2**24 - 1
    x = torch.arange(rows, dtype=torch.float32, device=dev)[:, None] * torch.linspace(-1, 1, 32, device=dev)
    q, scale = D.domino_quantize_rows(x)
    top = x.abs().amax(1)
    assert ((scale.double() - top.double() / 127).abs() <= scale.double() * 1.01 * E).all()
    assert (q[1:, 0] == -127).all() and (q[1:, 31] == 127).all() and not q[0].any()
    for r in (1, 5, 2**23, rows - 1):
        assert np.array_equal(q[r].cpu().numpy(), O.quantize_rows(x[r].cpu().numpy()[None])[0][0])


def test_logits_of_more_than_2_31_entries(dev):
    import draft_block_causal_amd as D

    B, K, d, V = 128, 64, 32, 262403
    log("base logits past 2^31 entries")
    gen = torch.Generator(device=dev).manual_seed(1)
    hq = torch.randint(-128, 128, (B, K, d), generator=gen, dtype=torch.int8, device=dev)
    wq = torch.randint(-128, 128, (V, d), generator=gen, dtype=torch.int8, device=dev)
    hs, ws = torch.rand((B, K), generator=gen, device=dev) + 0.01, torch.rand(V, generator=gen, device=dev) + 0.01
    out = D.domino_base_logits_i8(hq, hs, wq, ws)
    for b, i in ((0, 0), (63, 63), (64, 0), (127, 62), (127, 63)):
        want = O.base_logits_i8(*(t.cpu().numpy() for t in (hq[b:b + 1, i:i + 1], hs[b:b + 1, i:i + 1], wq, ws)))
        got = out[b, i].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - want[0, 0]) <= np.abs(want[0, 0]) * 3.001 * E), (b, i)


def _terms(x, y, T=1.0):
    """log-softmax of the rows and the bound rel(s) = (2.8 tbar + 8) e, tbar = sum p log2(e) (M - x) / T."""
    z = (x.double() - x.double().amax(-1, keepdim=True)) / T
    lp = z - z.exp().sum(-1, keepdim=True).log()
    return lp, lp.gather(-1, y.long()[..., None])[..., 0], (2.8 * 1.4427 * -(lp.exp() * z).sum(-1) + 8) * E


def test_policy_of_more_than_2_31_logits(dev):
    # held rows and, in the call without a gradient, rows in slices
    import draft_block_causal_amd as D

    B, K, V = 1024, 16, 131075
    log("policy past 2^31 logits")
    gen = torch.Generator(device=dev).manual_seed(2)
    x = torch.empty((B, K, V), device=dev).normal_(generator=gen)
    y = torch.randint(0, V, (B, K), generator=gen, device=dev, dtype=torch.int32)
    kept = [(0, 0), (511, 15), (512, 0), (1023, 14), (1023, 15)]
    rows = torch.stack([x[b, i] for b, i in kept])
    yk = torch.stack([y[b, i] for b, i in kept])
    all_lp, now, delta = _terms(rows, yk)
    h = torch.full((B, K), 99.0, device=dev)
    lp = D.domino_token_logprobs(x, y, entropy=h)
    at = lambda t: torch.stack([t[b, i] for b, i in kept])  # noqa: E731
    assert ((at(lp).double() - now).abs() <= delta + now.abs() * 1.01 * E).all()
    ent = -(all_lp.exp() * all_lp).sum(-1)
    assert ((at(h).double() - ent).abs() <= 40 * delta).all()  # (its own bound is tested where rows are few)
    adv, old = torch.ones((B, K), device=dev), lp - 0.1
    loss = D.domino_policy_loss(x, y, old, adv)
    lp2 = torch.empty_like(lp)
    loss2 = D.domino_policy_loss(x, y, old, adv, logp=lp2, grad=x)  # in place
    assert ((at(lp2).double() - now).abs() <= delta + now.abs() * 1.01 * E).all()
    ratio = (now - at(old).double()).exp()
    coef = -ratio / (B * K)
    want = -coef[:, None] * all_lp.exp()
    p_y = now.exp()
    want.scatter_(1, yk.long()[:, None], (coef * (1 - p_y))[:, None])
    # the ratio and s, a term (2.8 |t| + 2, |t| < 20 for normal logits), k and the product
    room = want.abs() * (2.02 * delta + 64 * E)[:, None]
    assert ((at(x).double() - want).abs() <= room + 1e-36).all()
    # the loss's log-probabilities and these are within rel(s) of the truth, 31 e where M < 6.7 and the weighted mean is 1;
    # these, of less than 24, are rounded, and so is the loss; every ratio is near e^0.1
    mean = -np.exp(0.1)
    lps = (lp.double() - old.double()).exp().mean().item()
    for value in (loss.item(), loss2.item()):
        assert abs(value + lps) <= lps * (2 * 31 * E + 24 * E + E) and abs(value - mean) < 1e-4


@pytest.mark.parametrize("B,K,V", [(1, 1, 2**24 - 1), (1, 3, 2**24 - 1), (131, 1, 2**22 + 1)])
def test_longest_rows(dev, B, K, V):
    import draft_block_causal_amd as D

    log(f"rows of {V}")
    gen = torch.Generator(device=dev).manual_seed(V + K)
    x = torch.empty((B, K, V), device=dev).normal_(generator=gen)
    y = torch.randint(0, V, (B, K), generator=gen, device=dev, dtype=torch.int32)
    y[-1, -1] = V - 1
    lp = D.domino_token_logprobs(x, y)
    g = torch.full_like(x, 99.0)
    lp2 = torch.empty_like(lp)
    D.domino_policy_loss(x, y, lp - 0.1, torch.ones_like(lp), logp=lp2, grad=g)
    for b, i in {(0, 0), (B - 1, K - 1), (B // 2, 0)}:
        all_lp, now, delta = _terms(x[b, i], y[b, i])
        for t in (lp, lp2):
            assert abs(t[b, i].item() - now.item()) <= delta.item() + abs(now.item()) * 1.01 * E
        coef = -(now - (lp[b, i] - 0.1).double()).exp().item() / (B * K)
        want = -coef * all_lp.exp()
        want[y[b, i].long()] += coef
        err = (g[b, i].double() - want).abs()
        assert (err <= want.abs() * (2.02 * delta.item() + 64 * E) + 1e-36).all()


def test_most_rows(dev):
    import draft_block_causal_amd as D

    B, K, V = 1 << 20, 4, 3
    log("2^22 rows")
    gen = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty((B, K, V), device=dev).normal_(generator=gen)
    y = torch.randint(0, V, (B, K), generator=gen, device=dev, dtype=torch.int32)
    w = (torch.rand((B, K), generator=gen, device=dev) < 0.7).float() / (B * K)
    adv = torch.empty((B, K), device=dev).normal_(generator=gen)
    all_lp, now, delta = _terms(x, y)
    h = torch.empty((B, K), device=dev)
    lp = D.domino_token_logprobs(x, y, weights=w, entropy=h)
    live = w != 0
    assert ((lp.double() - now).abs() <= delta + now.abs() * 1.01 * E)[live].all() and not lp[~live].any()
    assert ((h.double() + (all_lp.exp() * all_lp).sum(-1)).abs() <= 40 * delta)[live].all()
    old = (now - 0.1).float()
    g, kl, lp2 = torch.full_like(x, 99.0), torch.empty_like(lp), torch.empty_like(lp)
    loss = D.domino_policy_loss(x, y, old, adv, kl_coef=0.05, ref_logp=old, weights=w, logp=lp2, kl=kl, grad=g)
    ratio, d = (now - old.double()).exp(), old.double() - now
    value = 0.05 * (torch.expm1(d) - d) - ratio * adv.double()
    want = (w.double() * value).sum().item()
    room = (w.double() * (ratio * adv.double().abs() + 0.05) * 1.01 * delta).sum().item() + abs(want) * 1.01 * E
    assert abs(loss.item() - want) <= room
    coef = w.double() * (-ratio * adv.double() - 0.05 * torch.expm1(d))
    p = all_lp.exp()
    want = -coef[..., None] * p
    want.scatter_(2, y.long()[..., None], (coef * (1 - now.exp()))[..., None])
    parts = w.double() * (ratio * adv.double().abs() + 0.05 * d.exp())
    room = want.abs() * (2.02 * delta + 64 * E)[..., None] + p * parts[..., None] * 1.01 * delta[..., None]
    room.scatter_add_(2, y.long()[..., None], (parts * delta * 1.01)[..., None])
    assert ((g.double() - want).abs() <= room + 1e-36).all() and not g[~live].any() and not kl[~live].any()


def test_first_call_in_a_capture_and_two_graphs_at_once(dev):
    # kernels that need more LDS than the default, captured together, replayed on two streams at the same time, with eager
    # calls between the replays; each graph has its own workspace
    import draft_block_causal_amd as D

    B, K, V, d = 16, 16, 151936, 512
    gen = torch.Generator(device=dev).manual_seed(4)
    sets = []
    for _ in range(2):
        hidden = torch.empty((B, K, d), device=dev).normal_(generator=gen)
        wq, ws = D.domino_quantize_rows(torch.empty((V, d), device=dev).normal_(generator=gen) * 0.05)
        t = {"hq": torch.empty((B, K, d), dtype=torch.int8, device=dev), "hs": torch.empty((B, K), device=dev),
             "x": torch.empty((B, K, V), device=dev), "lp": torch.empty((B, K), device=dev),
             "h": torch.empty((B, K), device=dev), "loss": torch.zeros(1, device=dev), "g": torch.empty((B, K, V), device=dev)}
        y = torch.randint(0, V, (B, K), generator=gen, device=dev, dtype=torch.int32)
        adv = torch.empty((B, K), device=dev).normal_(generator=gen)
        old = torch.full((B, K), -12.0, device=dev)
        space = torch.empty(D.domino_policy_loss_workspace_size(B, K, V), dtype=torch.uint8, device=dev)

        def call(hidden=hidden, wq=wq, ws=ws, t=t, y=y, adv=adv, old=old, space=space):
            D.domino_quantize_rows(hidden, t["hq"], t["hs"])
            D.domino_base_logits_i8(t["hq"], t["hs"], wq, ws, t["x"])
            D.domino_token_logprobs(t["x"], y, 0.8, logp=t["lp"], entropy=t["h"], workspace=space)
            D.domino_policy_loss(t["x"], y, old, adv, temperature=0.8, loss=t["loss"], grad=t["g"], workspace=space)

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        sets.append((hidden, t, call, graph))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in range(3):
        for hidden, t, _, _ in sets:
            hidden.mul_(0.9)
            for o in t.values():
                o.fill_(-3)
        torch.cuda.synchronize()
        for s, (_, _, _, graph) in zip(streams, sets):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        got = [{k: v.clone() for k, v in t.items()} for _, t, _, _ in sets]
        for (_, t, call, _), g in zip(sets, got):
            call()
            torch.cuda.synchronize()
            for k in t:
                assert torch.equal(g[k], t[k]), (r, k)
