"""Drafted-token log-probabilities and the clipped policy loss on the GPU
against the float64 oracle.

Error bounds, in units e = 2^-24 (half a float32 step).  A term 2^t of the sum
s, t = log2(e) x / T - R with R within 1 of the row's largest, carries two
roundings of t, which move it by 2 ln 2 |t| e <= 2 (D + 1) e, D = |x - M| / T, and
one step (2 e) of the exponential.  A float32 sum of n terms in sequence adds n e
at most.  A workgroup's thread adds `chain` terms, then 6 lane merges, 7 wave
merges and at most 31 slice merges follow, an addition each (their factors are
powers of two).  So s is off by rel(s) <= (2 D + 4 + chain + 44) e, D over the
entries that matter (e^-D below 1e-9 of s does not; 160 stands for 46 below, as
before the factors were exact), and logp by that, plus its rounding to float32."""
import numpy as np
import pytest
import torch

import domino_synth as S
import oracle as O
from _helpers import device_head, log, workload_arrays

pytestmark = pytest.mark.gpu

E = 2.0**-24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_causal_amd as D

    D.load_library()
    return torch.device("cuda:0")


def _delta(V):
    # D = 40: e^-40 V < 1e-9; a thread's chain is at most V / 256 + 16 terms (slices only shorten it)
    return (2 * 40 + 2 + V / 256 + 16 + 160) * E


def _make(B, K, V, seed, T=1.0, cut=False):
    rng = np.random.default_rng(seed)
    x = (rng.normal(size=(B, K, V)) * 2).astype(np.float32)
    for b in range(B):
        for i in range(K):
            x[b, i, rng.integers(0, V, 4)] += np.float32(9)
    y = np.argmax(x / T + rng.gumbel(size=x.shape), axis=-1).astype(np.int32)
    lp, _ = O.token_logprobs(x, y, T)
    # ratios away from the borders of the clip range, where a rounding would decide
    off = rng.choice([-1.2, -0.5, -0.31, -0.1, 0.03, 0.12, 0.4, 1.1], size=(B, K))
    old = (lp - off).astype(np.float32)
    ref = (lp + rng.normal(size=(B, K)) * 0.4).astype(np.float32)
    adv = rng.normal(size=(B, K)).astype(np.float32)
    w = None
    if cut:
        n = rng.integers(0, K + 1, size=B)
        n[0] = K
        w = ((np.arange(K) < n[:, None]) * rng.uniform(0.5, 1.5, (B, K)) / max(1, n.sum())).astype(np.float32)
    return x, y, old, ref, adv, w


def _dev(dev, *arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in arrays]


def _check_logprobs(dev, x, y, T, w, logits=None):
    import draft_block_causal_amd as D

    tx, ty, tw = _dev(dev, x, y, w)
    tx = tx if logits is None else logits
    h = torch.full(y.shape, 99.0, device=dev)
    lp = D.domino_token_logprobs(tx, ty, T, tw, entropy=h)
    lp2 = D.domino_token_logprobs(tx, ty, T, tw)
    torch.cuda.synchronize()
    want, ent = O.token_logprobs(x, y, T, w)
    V, got = x.shape[-1], lp.cpu().numpy().astype(np.float64)
    same = got == want  # -inf and 0 of rows that take no part
    assert np.all(same | (np.abs(got - want) <= _delta(V) + np.abs(want) * E))
    assert np.allclose(lp2.cpu().numpy(), got, rtol=0, atol=2 * _delta(V), equal_nan=True)
    # sum p |t| e of u, and the same of s: entropy and its parts are below ln V + D
    np.testing.assert_allclose(h.cpu().numpy(), ent, rtol=0, atol=(np.log(V) + 42) * _delta(V) + 1e-7)


def _check_policy(dev, x, y, old, ref, adv, w, T=1.0, lo=0.2, hi=0.28, beta=0.05, logits=None, grad=None, want=None):
    import draft_block_causal_amd as D

    tx, ty, told, tref, tadv, tw = _dev(dev, x, y, old, ref, adv, w)
    tx = tx if logits is None else logits
    lp, kl = torch.full(y.shape, 99.0, device=dev), torch.full(y.shape, 99.0, device=dev)
    grad = torch.full_like(tx, 99.0) if grad is None else grad
    loss = D.domino_policy_loss(tx, ty, told, tadv, clip_low=lo, clip_high=hi, kl_coef=beta, ref_logp=tref, weights=tw,
                                temperature=T, logp=lp, kl=kl, grad=grad)
    torch.cuda.synchronize()
    want = O.policy_loss(x, y, old, adv, lo, hi, beta, ref, w, T) if want is None else want
    V, dl = x.shape[-1], _delta(x.shape[-1])
    got = lp.cpu().numpy().astype(np.float64)
    assert np.all((got == want["logp"]) | (np.abs(got - want["logp"]) <= dl + np.abs(want["logp"]) * E))
    ww = np.full(y.shape, 1.0 / y.size) if w is None else w.astype(np.float64)
    live = (ww != 0) & np.isfinite(want["logp"])
    ratio = np.where(live, np.exp(np.where(live, want["logp"] - old, 0)), 0)
    ed = np.where(live, np.exp(np.where(live, ref - want["logp"], 0)), 0) if ref is not None else np.zeros(y.shape)
    ra = ratio * np.where(live, np.abs(adv), 0)
    # logp off by dl moves a ratio by ratio dl, a divergence by |1 - e^d| dl
    np.testing.assert_array_less(np.abs(kl.cpu().numpy() - want["kl"]), np.abs(ed - 1) * 1.01 * dl + want["kl"] * 2 * E
                                 + dl * dl + 1e-30)
    dcoef = ww / T * (ra + beta * ed) * 1.01 * dl
    dloss = np.sum(np.where(live, ww * (ra + beta * np.abs(ed - 1)) * 1.01 * dl + ww * beta * dl * dl, 0))
    assert abs(loss.item() - want["loss"]) <= dloss + abs(want["loss"]) * 2 * E
    # p is off by its own term's and s's error, coef by dcoef; three float32 roundings at most
    coef = np.abs(want["coef"])[..., None]
    p = np.where(coef > 0, np.abs(want["grad"]) / np.where(coef > 0, coef, 1), 0)
    room = coef * p * 2 * dl + dcoef[..., None] * p + (coef + dcoef[..., None]) * 4 * E * np.maximum(p, 0)
    room += np.where(np.arange(V) == np.clip(y, 0, V - 1)[..., None], coef * (2 * dl + 4 * E), 0) + coef * 2.0**-120
    g = grad.cpu().numpy().astype(np.float64)
    bad = np.abs(g - want["grad"]) > room
    assert not bad.any(), (np.argwhere(bad)[:3], g[bad][:3], want["grad"][bad][:3], room[bad][:3])
    assert not g[~live].any()
    return loss


SIZES = [(1, 1, 1), (1, 1, 2), (1, 2, 5), (3, 5, 7), (2, 3, 63), (2, 3, 777), (4, 16, 4099), (1, 16, 49999), (5, 1, 2048),
         (3, 7, 8191), (2, 16, 4100), (40, 16, 1025)]


@pytest.mark.parametrize("B,K,V", SIZES)
@pytest.mark.parametrize("T,cut", [(1.0, False), (0.7, True)])
def test_logprobs_match_oracle(dev, B, K, V, T, cut):
    log(f"logprobs B={B} K={K} V={V} T={T} cut={cut}")
    x, y, _, _, _, w = _make(B, K, V, B + K + V, T, cut)
    _check_logprobs(dev, x, y, T, w)


@pytest.mark.parametrize("B,K,V", SIZES)
@pytest.mark.parametrize("T,cut,beta", [(1.0, False, 0.05), (0.7, True, 0.0), (1.4, True, 0.3)])
def test_policy_matches_oracle(dev, B, K, V, T, cut, beta):
    log(f"policy B={B} K={K} V={V} T={T} cut={cut} beta={beta}")
    x, y, old, ref, adv, w = _make(B, K, V, B + K + V, T, cut)
    _check_policy(dev, x, y, old, ref, adv, w, T=T, beta=beta)


def test_qwen_vocabulary(dev):
    x, y, old, ref, adv, w = _make(2, 3, 151936, 5)
    log("whole vocabulary")
    _check_logprobs(dev, x, y, 1.0, None)
    _check_policy(dev, x, y, old, ref, adv, None)


@pytest.mark.parametrize("V", [4103, 5003, 8197, 8200, 8300, 12001, 16390, 17000, 25001, 40003, 60001, 75000, 80003, 99001, 151936, 160001, 204802])
def test_rows_held_on_chip(dev, V):
    # as many rows as compute units and a few more: each held size, with and without rows left over
    import draft_block_causal_amd as D

    rows = torch.cuda.get_device_properties(dev).multi_processor_count + 13
    log(f"held rows V={V} rows={rows}")
    g = torch.Generator(device=dev).manual_seed(V)
    x = torch.randn((rows, 1, V), generator=g, device=dev) * 2
    y = torch.randint(0, V, (rows, 1), generator=g, device=dev, dtype=torch.int32)
    y[0, 0], y[1, 0], y[2, 0] = 0, V - 1, V - 2
    x.scatter_add_(2, y.long()[..., None], torch.full((rows, 1, 1), 9.0, device=dev))
    x[3] = -np.inf
    x[4] = -3.4e38
    x[5, 0, 0] = 1e30
    w = torch.full((rows, 1), 1.0 / rows, device=dev)
    w[6] = 0
    x[6] = np.nan
    lp = torch.log_softmax(x.double(), -1)
    now = lp.gather(2, y.long()[..., None])[..., 0]
    ok = torch.isfinite(now)
    off = torch.rand((rows, 1), generator=g, device=dev) * 0.1 + 0.03  # ratios inside the clip range: 1.03 .. 1.14
    old = torch.where(ok, now - off, 0).float()
    ref = torch.where(ok, now + 0.3, 0).float()
    adv = torch.randn((rows, 1), generator=g, device=dev)
    out = {k: torch.full((rows, 1), 99.0, device=dev) for k in ("logp", "kl")}
    kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.05, ref_logp=ref, weights=w, **out)
    grad = torch.full_like(x, 99.0)
    loss = D.domino_policy_loss(x, y, old, adv, grad=grad, **kw)
    first = [loss.clone(), out["logp"].clone(), out["kl"].clone()]
    # the terms in float64; row 5 has a token of probability 0, whose divergence is infinite: kept apart below
    r = torch.exp(now - old.double())
    d = ref.double() - now
    coef = w.double() * (-r * adv.double() - 0.05 * torch.expm1(d))
    take = ok & (w != 0) & (torch.arange(rows, device=dev)[:, None] != 5)
    dl = _delta(V)
    np.testing.assert_array_less((out["logp"].double() - now)[take].abs().cpu().numpy(),
                                 (dl + now[take].abs() * E).cpu().numpy())
    assert out["logp"][3].item() == -np.inf and out["logp"][6].item() == 0 and out["kl"][6].item() == 0
    p = lp.exp()
    p.scatter_add_(2, y.long()[..., None], torch.full((rows, 1, 1), -1.0, device=dev, dtype=torch.float64))
    for i in range(rows):
        if not take[i]:
            assert i in (3, 5, 6)
            continue
        want = -coef[i] * p[i, 0]
        room = coef[i].abs() * ((lp[i, 0].exp() + (torch.arange(V, device=dev) == y[i, 0])) * 8 * (dl + 4 * E)) + 1e-36
        bad = (grad[i, 0] - want).abs() > room
        assert not bad.any(), (i, torch.nonzero(bad)[:3])
    assert not grad[3].any() and not grad[6].any()
    ix = x.clone()
    again = D.domino_policy_loss(ix, y, old, adv, grad=ix, **kw)
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(ix), torch.nan_to_num(grad))
    for a, b in zip(first, (again, out["logp"], out["kl"])):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.parametrize("T", [1.0, 0.5])
@pytest.mark.parametrize("base", [1e4, -1e6, 3e7, -1e9, 8e8, -3e38])
def test_rows_far_from_zero(dev, base, T):
    # a large offset in every entry (a mask value in all of them, say): steps of the offset's own float32 grid apart
    V = 5003
    rng = np.random.default_rng(3)
    step = np.spacing(np.float32(abs(base)))
    x = (np.float32(base) - step * rng.integers(0, 40, size=(1, 4, V)).astype(np.float32)).astype(np.float32)
    x[0, 1] = np.float32(base)
    x[0, 2, ::2] = -np.inf
    x[0, 3, 1000:] -= np.float32(abs(base))
    y = np.argmax(x, -1).astype(np.int32)
    lp, _ = O.token_logprobs(x, y, T)
    _check_logprobs(dev, x, y, T, None)
    adv = np.ones((1, 4), np.float32)
    _check_policy(dev, x, y, (lp - 0.1).astype(np.float32), (lp + 0.3).astype(np.float32), adv, None, T=T)


def test_many_rows(dev):
    x, y, old, ref, adv, w = _make(300, 16, 33, 6, cut=True)
    _check_logprobs(dev, x, y, 1.0, w)
    _check_policy(dev, x, y, old, ref, adv, w)


def test_without_reference(dev):
    x, y, old, ref, adv, w = _make(3, 5, 333, 7, cut=True)
    _check_policy(dev, x, y, old, None, adv, w, beta=0.0)


@pytest.mark.parametrize("shift_x,shift_g", [(1, 1), (3, 3), (1, 2), (0, 1)])
@pytest.mark.parametrize("V", [4099, 256, 6])
def test_rows_of_any_alignment(dev, shift_x, shift_g, V):
    # 4-byte aligned buffers: rows start anywhere in a 16-byte group, logits and gradient not alike
    x, y, old, ref, adv, w = _make(2, 3, V, V)
    bx, bg = torch.zeros(x.size + 8, device=dev), torch.full((x.size + 8,), 5.5, device=dev)
    lx = bx[shift_x:shift_x + x.size].view(x.shape)
    lx.copy_(torch.from_numpy(x))
    lg = bg[shift_g:shift_g + x.size].view(x.shape)
    _check_policy(dev, x, y, old, ref, adv, w, logits=lx, grad=lg)
    _check_logprobs(dev, x, y, 1.0, None, logits=lx)
    assert torch.all(bg[:shift_g] == 5.5) and torch.all(bg[shift_g + x.size:] == 5.5)


def test_rows_that_take_no_part_may_hold_anything(dev):
    x, y, old, ref, adv, w = _make(4, 5, 777, 8, cut=True)
    w[2] = 0
    want = O.policy_loss(x, y, old, adv, 0.2, 0.28, 0.05, ref, w)
    dead = w == 0
    x[dead] = np.nan
    old[dead], ref[dead], adv[dead] = np.inf, np.nan, np.nan
    y[dead] = 1 << 30
    _check_logprobs(dev, x, y, 1.0, w)
    old_c, ref_c, adv_c = (np.where(dead, 0, a).astype(np.float32) for a in (old, ref, adv))
    tx, ty, told, tref, tadv, tw = _dev(dev, x, y, old, ref, adv, w)
    _check_policy(dev, np.where(dead[..., None], 0, x).astype(np.float32), np.where(dead, 0, y).astype(np.int32), old_c,
                  ref_c, adv_c, w, logits=tx, want=want)
    import draft_block_causal_amd as D

    g = torch.full_like(tx, 99.0)
    loss = D.domino_policy_loss(tx, ty, told, tadv, clip_high=0.28, kl_coef=0.05, ref_logp=tref, weights=tw, grad=g)
    torch.cuda.synchronize()
    assert np.isfinite(loss.item()) and loss.item() == pytest.approx(want["loss"], rel=1e-4)
    assert not g.cpu().numpy()[dead].any()
    zero = torch.zeros_like(tw)
    loss = D.domino_policy_loss(tx, ty, told, tadv, kl_coef=0.05, ref_logp=tref, weights=zero, grad=g)
    assert loss.item() == 0 and not g.any()


def test_excluded_entries_and_empty_rows(dev):
    x, y, old, ref, adv, w = _make(2, 6, 4099, 9)
    rng = np.random.default_rng(1)
    keep = rng.random(x.shape) < 0.3
    np.put_along_axis(keep, y[..., None].astype(np.int64), True, -1)
    x[0] = np.where(keep[0], x[0], -np.inf)                       # a vocabulary mask
    x[1, 0] = np.finfo(np.float32).min                            # lowest values alone: a uniform row
    x[1, 1] = np.where(keep[1, 1], x[1, 1], np.finfo(np.float32).min)
    x[1, 2] = -np.inf                                             # nothing left
    x[1, 3] = -np.inf
    x[1, 3, y[1, 3]] = -3.0e38                                    # one entry left
    for T in (1.0, 0.5):
        lp, _ = O.token_logprobs(x, y, T)
        lp = np.where(np.isfinite(lp), lp, 0)
        old = (lp - 0.1).astype(np.float32)
        ref = (lp + 0.3).astype(np.float32)
        _check_logprobs(dev, x, y, T, None)
        _check_policy(dev, x, y, old, ref, adv, None, T=T)


def test_bad_rows_leave_the_others_alone(dev):
    import draft_block_causal_amd as D

    x, y, old, ref, adv, w = _make(1, 6, 5003, 10)
    good, _ = O.token_logprobs(x, y)
    x[0, 1, 17], x[0, 3, 4000] = np.nan, np.inf
    tx, ty, told, tref, tadv = _dev(dev, x, y, old, ref, adv)
    h = torch.zeros((1, 6), device=dev)
    lp = D.domino_token_logprobs(tx, ty, entropy=h).cpu().numpy()[0]
    assert np.isnan(lp[[1, 3]]).all() and np.isnan(h.cpu().numpy()[0, [1, 3]]).all()
    ok = [0, 2, 4, 5]
    assert np.all(np.abs(lp[ok] - good[0, ok]) <= _delta(5003) + 20 * E)
    g = torch.zeros_like(tx)
    loss = D.domino_policy_loss(tx, ty, told, tadv, kl_coef=0.1, ref_logp=tref, grad=g)
    g = g.cpu().numpy()[0]
    assert np.isnan(loss.item()) and np.isnan(g[[1, 3]]).all() and np.isfinite(g[ok]).all()


def test_token_of_probability_zero(dev):
    import draft_block_causal_amd as D

    x, y, old, ref, adv, w = _make(1, 2, 300, 11)
    x[0, 0, y[0, 0]] = -np.inf
    adv[:] = [[1.0, 1.0]]
    tx, ty, told, tref, tadv = _dev(dev, x, y, old, ref, adv)
    kl, g = torch.zeros((1, 2), device=dev), torch.ones_like(tx)
    loss = D.domino_policy_loss(tx, ty, told, tadv, ref_logp=tref, kl=kl, grad=g)
    assert kl[0, 0].item() == np.inf and np.isfinite(loss.item()) and not g[0, 0].any()
    assert D.domino_policy_loss(tx, ty, told, tadv, kl_coef=0.1, ref_logp=tref).item() == np.inf


def test_extreme_ratios_and_zero_advantages(dev):
    import draft_block_causal_amd as D

    x, y, old, ref, adv, w = _make(1, 4, 100, 12)
    lp, _ = O.token_logprobs(x, y)
    old[0, :3] = lp[0, :3] - np.array([800.0, 800.0, -800.0])  # ratios beyond float64 and below it
    adv[0, :3] = [0.0, 1.0, -1.0]
    old[0, 3], adv[0, 3] = lp[0, 3] - 0.5, 0.0
    tx, ty, told, tadv = _dev(dev, x, y, old, adv)
    g = torch.ones_like(tx)
    loss = D.domino_policy_loss(tx, ty, told, tadv, grad=g)
    # 0, clipped at 1.2, clipped at 0.8 (A = -1), 0
    assert loss.item() == pytest.approx((-1.2 + 0.8) / 4, rel=1e-6) and not g.any()


def test_tokens_out_of_range_are_clamped(dev):
    x, y, old, ref, adv, w = _make(1, 4, 50, 13)
    y[0] = [-5, 50, 1 << 30, -(1 << 31)]
    lp, _ = O.token_logprobs(x, y)
    _check_policy(dev, x, y, (lp - 0.1).astype(np.float32), (lp + 0.2).astype(np.float32), adv, None)


@pytest.mark.parametrize("B,K,V", [(2, 16, 20011), (64, 4, 501)])
def test_in_place_repeatable_and_without_gradient(dev, B, K, V):
    import draft_block_causal_amd as D

    x, y, old, ref, adv, w = _make(B, K, V, 14, cut=True)
    tx, ty, told, tref, tadv, tw = _dev(dev, x, y, old, ref, adv, w)
    kw = dict(kl_coef=0.1, ref_logp=tref, weights=tw, temperature=0.9)
    g = torch.empty_like(tx)
    lp, kl = torch.empty((B, K), device=dev), torch.empty((B, K), device=dev)
    a = D.domino_policy_loss(tx, ty, told, tadv, grad=g, logp=lp, kl=kl, **kw)
    lp2, kl2 = torch.empty((B, K), device=dev), torch.empty((B, K), device=dev)
    b = D.domino_policy_loss(tx, ty, told, tadv, logp=lp2, kl=kl2, **kw)
    ix = tx.clone()
    c = D.domino_policy_loss(ix, ty, told, tadv, grad=ix, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(ix, g)
    assert torch.equal(lp, lp2) and torch.equal(kl, kl2)


def test_empty_batch_leaves_the_loss(dev):
    import draft_block_causal_amd as D

    z = torch.zeros((0, 16, 10), device=dev)
    zi, zf = torch.zeros((0, 16), dtype=torch.int32, device=dev), torch.zeros((0, 16), device=dev)
    loss = torch.full((1,), 7.0, device=dev)
    D.domino_policy_loss(z, zi, zf, zf, loss=loss)
    assert loss.item() == 7.0
    assert D.domino_token_logprobs(z, zi).shape == (0, 16)


def test_two_graphs_and_another_stream(dev):
    # captured calls with workspaces of their own, replayed in turn with eager calls and new inputs between them
    import draft_block_causal_amd as D

    cases = []
    for k, (B, K, V) in enumerate([(1, 16, 30011), (6, 5, 999), (40, 7, 5003)]):  # sliced, short, held on chip
        x, y, old, ref, adv, w = _make(B, K, V, 20 + k, cut=True)
        t = _dev(dev, x, y, old, ref, adv, w)
        ws = torch.empty(D.domino_policy_loss_workspace_size(B, K, V), dtype=torch.uint8, device=dev)
        out = dict(loss=torch.zeros(1, device=dev), logp=torch.zeros((B, K), device=dev), kl=torch.zeros((B, K), device=dev),
                   grad=torch.zeros_like(t[0]))

        def call(t=t, out=out, ws=ws, stream=None):
            D.domino_policy_loss(t[0], t[1], t[2], t[4], kl_coef=0.1, ref_logp=t[3], weights=t[5], workspace=ws,
                                 stream=stream, **out)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        cases.append((t, out, call, g))
    side = torch.cuda.Stream()
    for r in range(3):
        for t, out, call, g in cases:
            t[0].mul_(0.9)
            for o in out.values():
                o.fill_(-3)
            g.replay()
            torch.cuda.synchronize()
            got = {k: v.clone() for k, v in out.items()}
            side.wait_stream(torch.cuda.current_stream())
            call(stream=side)
            side.synchronize()
            for k in out:
                assert torch.equal(got[k], out[k]), (r, k)


@pytest.mark.parametrize("target_seed", [4, 6])  # 4: every draft is rejected at once (no advantage); 6: lengths differ
def test_roll_out_and_policy_step(dev, target_seed):
    """The calls in the order of a training program: the LM head in 8 bits, a sampled
    draft from its logits, its log-probabilities, the reward from the acceptance lengths,
    the bf16-policy forward on the drafted tokens, the policy loss and both backward passes."""
    import draft_block_causal_amd as D

    w = S.get_workload("tiny_stress_b4")
    head_np, inp = workload_arrays(w)
    head = device_head(w, dev)
    B, K, V = w.batch, w.block, w.vocab
    hidden, x_t = S.to_torch(inp["hidden"], dev), S.to_torch(inp["x_t"], dev)
    wq, ws = D.domino_quantize_rows(head.tensors["lm_head"])
    hq, hs = D.domino_quantize_rows(hidden)
    base8 = D.domino_base_logits_i8(hq, hs, wq, ws)
    roll = torch.empty_like(base8)
    tok = D.domino_draft_block(head, hidden, base8, x_t, temperature=1.0, seed=3, logits=roll)
    old = D.domino_token_logprobs(roll, tok)
    base = D.domino_base_logits(head, hidden)
    ref = D.domino_token_logprobs(base, tok)  # the head-off distribution as the reference
    target = S.to_torch(S.make_targets(tok.cpu().numpy(), V, p=0.7, seed=target_seed), dev)
    accept = D.domino_accept_len(tok, target)
    pos = torch.arange(K, device=dev)
    weights = (pos <= accept[:, None]).float()  # the accepted prefix and the first rejected token
    weights /= weights.sum()
    reward = accept.float()
    adv = ((reward - reward.mean()) / (reward.std() + 1e-3))[:, None].expand(B, K).contiguous()
    final, states = torch.empty_like(base), torch.empty((B, K, w.gru_hidden), device=dev)
    D.domino_draft_block(head, hidden, base, x_t, teacher=tok, logits=final, gru_states=states)
    logp, kl, grad = torch.empty_like(ref), torch.empty_like(ref), torch.empty_like(final)
    loss = D.domino_policy_loss(final, tok, old, adv, kl_coef=0.1, ref_logp=ref, weights=weights, logp=logp, kl=kl,
                                grad=grad)
    back = D.domino_correction_backward(head, hidden, states, grad)
    gru = D.domino_gru_backward(head, x_t, tok, states, back["d_states"])
    torch.cuda.synchronize()
    n = lambda t: t.cpu().numpy()  # noqa: E731
    want = O.policy_loss(n(final), n(tok), n(old), n(adv), 0.2, 0.2, 0.1, n(ref), n(weights))
    assert loss.item() == pytest.approx(want["loss"], abs=1e-5)
    f64 = {k: None if t is None else t.double().cpu().numpy() for k, t in head.tensors.items()}
    wb = O.correction_backward(f64, n(hidden).astype(np.float64), n(states).astype(np.float64), want["grad"])
    for k, o in (("d_w2", "dw2"), ("d_w1", "dw1"), ("d_states", "dg")):
        scale = np.abs(wb[o]).max()
        assert np.abs(n(back[k]) - wb[o]).max() <= 1e-3 * scale, k
    for k, t in gru.items():
        assert torch.isfinite(t).all(), k
    # the 8-bit roll-out and the policy give nearly the same probabilities to the drafted tokens: both read the same
    # tokens, so their logits differ by the base logits' rounding, at most sum |h| ws / 2 + hs sum |w| / 2 + d hs ws / 4,
    # and a log-probability by twice the largest such difference
    live = n(weights) != 0
    room = (hidden.abs().sum(-1).max() * ws.max() / 2 + hs.max() * head.tensors["lm_head"].abs().sum(-1).max() / 2
            + w.d * hs.max() * ws.max() / 4).item()
    assert np.isfinite(n(old)).all() and np.abs(n(logp) - n(old))[live].max() < 2 * room + 1e-4


def test_binding_refuses_wrong_tensors(dev):
    import draft_block_causal_amd as D

    def z(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device=dev)

    i8, i32 = torch.int8, torch.int32
    with pytest.raises(TypeError):
        D.domino_quantize_rows(z(2, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        D.domino_quantize_rows(z(64, 2).t())  # not contiguous
    with pytest.raises(ValueError):
        D.domino_quantize_rows(z(2, 64), q=z(2, 32, dtype=i8))
    with pytest.raises(D.DominoError):
        D.domino_quantize_rows(z(2, 40))
    with pytest.raises(TypeError):
        D.domino_base_logits_i8(z(1, 2, 64), z(1, 2), z(9, 64, dtype=i8), z(9))
    with pytest.raises(ValueError):
        D.domino_base_logits_i8(z(1, 2, 64, dtype=i8), z(1, 2), z(9, 32, dtype=i8), z(9))
    with pytest.raises(ValueError):
        D.domino_base_logits_i8(z(2, 64, dtype=i8), z(2), z(9, 64, dtype=i8), z(9))
    x, y = z(2, 3, 7), z(2, 3, dtype=i32)
    with pytest.raises(ValueError):
        D.domino_token_logprobs(x[0], y)
    with pytest.raises(TypeError):
        D.domino_token_logprobs(x, y.long())
    with pytest.raises(ValueError):
        D.domino_token_logprobs(x, y, weights=z(3))
    with pytest.raises(ValueError):
        D.domino_token_logprobs(x, y.cpu())
    with pytest.raises(D.DominoError):
        D.domino_token_logprobs(x, y, temperature=0.0)
    with pytest.raises(D.DominoError):
        D.domino_token_logprobs(x, y, workspace=z(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        D.domino_token_logprobs(x, y, workspace=z(1 << 16))
    with pytest.raises(TypeError):
        D.domino_policy_loss(x.bfloat16(), y, z(2, 3), z(2, 3))
    with pytest.raises(ValueError):
        D.domino_policy_loss(x, y, z(2, 3), z(2, 3), grad=z(2, 3, 8))
    with pytest.raises(D.DominoError):
        D.domino_policy_loss(x, y, z(2, 3), z(2, 3), kl_coef=0.1)  # no reference
    old = z(2, 3)
    with pytest.raises(D.DominoError):
        D.domino_policy_loss(x, y, old, z(2, 3), logp=old)  # an output over an input
