"""Values of the log-probability and policy kernels where a general sweep of
random rows does not reach: rows far from zero, rows held on chip, tokens of
probability near 1, against float64 with bounds from the kernels' arithmetic.

Bounds, in units e = 2^-24 (half a float32 step).  A term 2^t of a row's sum,
t = c x - R or c (x - M): t carries the rounding of x - M, of c to float32 and
of the product where the row is far from zero (1 + 2 + 1 e |t|), else two
roundings (2 e |t|, |t| within 1 of c |x - M|); a rounding of t moves the term
by ln 2 of it, and the exponential is off by a step (2 e).  Sixteen terms are
added in float32 (4 e), everything after in float64.  So the sum is off by
    rel(s) <= (2.8 tbar + 8) e,   tbar = sum p_v log2(e) (M - x_v) / T,
which moves a log-probability by as much; it is rounded to float32 once more."""
import numpy as np
import pytest
import torch

import oracle as O
from _helpers import log

pytestmark = pytest.mark.gpu

E = 2.0**-24
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_causal_amd as D

    D.load_library()
    return torch.device("cuda:0")


def _rel_s(x, T):
    """rel(s) of each row of x [..., V] (float64)."""
    z = (x - x.max(-1, keepdims=True)) / T
    p = np.exp(z)
    p /= p.sum(-1, keepdims=True)
    return (2.8 * LOG2E * (p * -np.where(p > 0, z, 0)).sum(-1) + 8) * E


def _neighbours(limit, T):
    """Float32 neighbours x1 < x2 with float32(log2(e) / T) x1 below the limit and x2 not."""
    hi = np.float32(LOG2E / T)
    if float(hi) >= LOG2E / T:
        hi = np.nextafter(hi, np.float32(0))
    x = np.float32(limit / float(hi))
    while not x * hi < np.float32(limit):
        x = np.nextafter(x, np.float32(0))
    while np.nextafter(x, np.float32(np.inf)) * hi < np.float32(limit):
        x = np.nextafter(x, np.float32(np.inf))
    return x, np.nextafter(x, np.float32(np.inf))


def _policy(dev, x, y, T, grad=True):
    """logp and gradient of a policy step with advantages 1 inside the clip range."""
    import draft_block_causal_amd as D

    lp, _ = O.token_logprobs(x, y, T)
    adv = np.ones(y.shape, np.float32)
    old = lp - 0.05
    t = [torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in (x, y, old.astype(np.float32), adv)]
    got, g = torch.full(y.shape, 99.0, device=dev), torch.full(x.shape, 99.0, device=dev)
    D.domino_policy_loss(*t, temperature=T, logp=got, grad=g)
    torch.cuda.synchronize()
    want = O.policy_loss(x, y, old.astype(np.float32), adv, T=T)
    return got.cpu().numpy().astype(np.float64), g.cpu().numpy().astype(np.float64), want


@pytest.mark.parametrize("limit,T", [(2.0**30, 1.39), (2.0**30, 0.7), (2.0**20, 1.39), (2.0**20, 1.0), (2.0**20, 0.7)])
@pytest.mark.parametrize("sign", [1, -1])
def test_slices_on_both_sides_of_a_limit(dev, limit, sign, T):
    # one slice's entries are the last below a magnitude, another's the first above it
    import draft_block_causal_amd as D

    V = 40003
    a, b = (np.float32(sign) * v for v in _neighbours(limit, T))
    x = np.full((1, 4, V), a, np.float32)
    x[0, 0, 20000:] = b
    x[0, 1, :30000] = b
    x[0, 2, 5:9] = b
    y = np.array([[30000, 30000, 6, 1]], np.int32)
    tx, ty = torch.from_numpy(x).to(dev), torch.from_numpy(y).to(dev)
    got = D.domino_token_logprobs(tx, ty, T).cpu().numpy().astype(np.float64)
    want, _ = O.token_logprobs(x, y, T)
    room = _rel_s(x.astype(np.float64), T) + np.abs(want) * E
    assert np.all(np.abs(got - want) <= room), (got, want)
    got, g, want = _policy(dev, x, y, T)
    assert np.all(np.abs(got - want["logp"]) <= room), (got, want["logp"])
    # tbar < 1/2: rel(s) < 10 e twice (probability, ratio), and at most 8 e of a term and the gradient's roundings
    scale = np.abs(want["coef"])[..., None]
    assert np.all(np.abs(g - want["grad"]) <= scale * 28 * E), np.abs(g - want["grad"]).max()


def _entropy_room(x, T, want):
    """ln s - ln 2 u / s with u = sum 2^t t: a term carries the error of 2^t and a product, sixteen are added in
    float32; t is within 1 of c (x - M)."""
    z = (x - x.max(-1, keepdims=True)) / T
    p = np.exp(z)
    p /= p.sum(-1, keepdims=True)
    t = 1 + LOG2E * -np.where(p > 0, z, 0)
    t1, t2 = (p * t).sum(-1), (p * t * t).sum(-1)
    rel = _rel_s(x, T)
    return rel + np.log(2) * (t1 * rel + (2.8 * t2 + 8 * t1) * E) + np.abs(want) * E


@pytest.mark.parametrize("T", [0.68, 0.7, 1.39])
@pytest.mark.parametrize("base", [928286528.0, 5e8, 1e8, 2e7, 1.5e6, 7e5, 1e5])
@pytest.mark.parametrize("sign", [1, -1])
def test_rows_far_from_zero_at_any_temperature(dev, sign, base, T):
    # a few steps of the base's own float32 grid apart: short rows, sliced ones, and as many as are held on chip
    import draft_block_causal_amd as D

    log(f"rows at {sign * base:g}, T={T}")
    rng = np.random.default_rng(11)
    step = np.spacing(np.float32(base))
    for B, V in ((1, 5003), (1, 40003), (34, 5003)):
        x = (np.float32(sign * base) - step * rng.integers(0, 40, size=(1, 4, V)).astype(np.float32)).astype(np.float32)
        x[0, 1] = np.float32(sign * base)
        x[0, 2, ::2] = -np.inf
        x[0, 3, 1000:] -= np.float32(base)
        y = np.argmax(x, -1).astype(np.int32)
        x64 = x.astype(np.float64)
        want, ent = O.token_logprobs(x, y, T)
        room = _rel_s(x64, T) + np.abs(want) * E
        xb, yb = np.repeat(x, B, 0), np.repeat(y, B, 0)
        tx, ty = torch.from_numpy(xb).to(dev), torch.from_numpy(yb).to(dev)
        h = torch.full((B, 4), 99.0, device=dev)
        got = D.domino_token_logprobs(tx, ty, T, entropy=h).cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - want) <= room), (B, V, got[0], want)
        bad = np.abs(h.cpu().numpy() - ent) > _entropy_room(x64, T, ent)
        assert not bad.any(), (B, V, h[0], ent)
        got, g, pol = _policy(dev, xb, yb, T)
        assert np.all(np.abs(got - want) <= room), (B, V, got[0], want)
        # as above with rel(s) of the row; a term that weighs anything has 2.8 |t| < 200
        scale = np.abs(pol["coef"])[..., None]
        assert np.all(np.abs(g - pol["grad"]) <= scale * (2.02 * _rel_s(x64, T)[..., None] + 208 * E)), (B, V)


@pytest.mark.parametrize("T", [1.0, 0.9, 1.2])
def test_mean_error_of_log_probabilities(dev, T):
    # Read from the divergence at d = 1 (e - 2 = 0.72): its rounding to float32, 3e-8 at most, stands for 1.7e-8 of a
    # log-probability, 1e-8 rms, 6e-10 in the mean of 256 rows; roundings of terms have no direction.  What is left is the
    # exponential's own mean error, a few hundredths of a step (1.2e-7).  A low part of log2(e) / T that gets lost in t
    # shows as 1.2e-8 or more.
    import draft_block_causal_amd as D

    V, rows = 151936, 256
    gen = torch.Generator(device=dev).manual_seed(V)
    x = torch.randn((rows, 1, V), generator=gen, device=dev) * 2
    y = torch.randint(0, V, (rows, 1), generator=gen, device=dev, dtype=torch.int32)
    now = torch.log_softmax(x.double() / T, -1).gather(2, y.long()[..., None])[..., 0]
    one = torch.ones((rows, 1), device=dev)
    ref = (now + 1).float()
    d = ref.double() - now
    for grad in (torch.empty_like(x), None):  # rows held on chip, rows in slices
        kl = torch.zeros((rows, 1), device=dev)
        D.domino_policy_loss(x, y, now.float(), one, ref_logp=ref, kl=kl, grad=grad, temperature=T)
        mean = ((kl.double() - (torch.expm1(d) - d)) / (1 - d.exp())).mean().item()
        log(f"mean error of logp at T={T}: {mean:.2e}")
        assert abs(mean) < 8e-9


@pytest.mark.parametrize("T", [1.0, 0.7])
@pytest.mark.parametrize("B,K,V,shift", [(1, 4, 5003, 0), (1, 4, 40003, 0), (3, 5, 99, 0), (3, 5, 4099, 1), (34, 4, 5003, 0),
                                         (34, 4, 20011, 0), (34, 4, 60001, 0), (34, 4, 151936, 0), (1, 3, 1, 0)])
def test_nearly_certain_tokens(dev, B, K, V, shift, T):
    # tokens of probability 1 - 1e-2 ... 1 - 1e-16 at any place of the row, in slices, short and held rows; shift: gradient
    # rows of another alignment than the logits'.  With r the sum of the other terms over the token's, logp = -ln(1 + r),
    # its gradient is coef r / (1 + r) and the entropy ln(1 + r) + sum p (z_y - z): all as exact as r is.
    import draft_block_causal_amd as D

    log(f"nearly certain tokens B={B} K={K} V={V} T={T}")
    rng = np.random.default_rng(V + B)
    x = (rng.normal(size=(B, K, V)) * 2).astype(np.float32)
    y = rng.integers(0, V, size=(B, K)).astype(np.int32)
    y.flat[0], y.flat[-1], y.flat[1] = 0, V - 1, max(0, V - 2)
    gap = np.float32(T) * (rng.uniform(4, 38, size=(B, K)) + np.log(V)).astype(np.float32) + x.max(-1)
    np.put_along_axis(x, y[..., None].astype(np.int64), gap[..., None], -1)
    adv = rng.choice([-1.0, 0.5, 2.0], size=(B, K)).astype(np.float32)
    z = (x.astype(np.float64) - gap[..., None]) / T
    q = np.exp(z)
    np.put_along_axis(q, y[..., None].astype(np.int64), 0.0, -1)
    r = q.sum(-1)
    lp, s = -np.log1p(r), 1 + r
    old = (lp - rng.uniform(-0.1, 0.1, size=lp.shape)).astype(np.float32)
    t = LOG2E * -z + 1
    mean_t = (q * t).sum(-1) / np.maximum(r, 1e-300)
    rel = (2.8 * mean_t + 8) * E  # of r
    tx, ty, told, tadv = [torch.from_numpy(a).to(dev) for a in (x, y, old, adv)]
    h = torch.full((B, K), 99.0, device=dev)
    got = D.domino_token_logprobs(tx, ty, T, entropy=h).cpu().numpy().astype(np.float64)
    room = np.abs(lp) * (rel + 1.01 * E) + 2.0**-149
    assert np.all(got <= 0) and np.all(np.abs(got - lp) <= room), np.abs(got / lp - 1).max()
    ent = np.log1p(r) - (q * z).sum(-1) / s
    spread = (q * t * (2.8 * t + 13)).sum(-1) * E  # a term's error, its product with t, sixteen added in float32
    got = h.cpu().numpy()
    assert np.all(got >= 0) and np.all(np.abs(got - ent) <= spread + np.abs(lp) * rel + ent * 1.01 * E + 2.0**-149)
    buf = torch.full((x.size + 8,), 5.5, device=dev)
    g = buf[shift:shift + x.size].view(x.shape)
    lpo = torch.full((B, K), 99.0, device=dev)
    D.domino_policy_loss(tx, ty, told, tadv, temperature=T, logp=lpo, grad=g)
    got = lpo.cpu().numpy().astype(np.float64)
    assert np.all(got <= 0) and np.all(np.abs(got - lp) <= room)
    ratio = np.exp(lp - old)  # inside the clip range
    coef = -ratio * adv / (B * K) / T
    want = coef[..., None] * (-q / s[..., None])
    np.put_along_axis(want, y[..., None].astype(np.int64), (coef * r / s)[..., None], -1)
    dcoef = np.abs(coef) * 1.01 * np.abs(lp) * rel
    # the others: the term (2.8 |t| + 2), k and the product; the token: r / s and one rounding
    term = np.abs(want) * ((2.8 * t + 8) * E + (r * rel / s + np.abs(lp) * rel * 1.01)[..., None])
    tok = np.abs(coef) * r / s * (rel + 1.01 * E) + dcoef * r / s
    np.put_along_axis(term, y[..., None].astype(np.int64), tok[..., None], -1)
    err = np.abs(g.cpu().numpy() - want)
    bad = err > term + 1e-36
    assert not bad.any(), (np.argwhere(bad)[:3], err[bad][:3], want[bad][:3])
    assert torch.all(buf[:shift] == 5.5) and torch.all(buf[shift + x.size:] == 5.5)


def test_no_log_probability_above_zero(dev):
    # rows in which nothing but the token's own term has weight: however that rounds, p is 1 and not more
    import draft_block_causal_amd as D

    rng = np.random.default_rng(5)
    for B, V in ((64, 33), (64, 5003), (1, 40003)):
        x = np.full((B, 16, V), -200, np.float32)
        y = rng.integers(0, V, size=(B, 16)).astype(np.int32)
        np.put_along_axis(x, y[..., None].astype(np.int64), rng.uniform(-30, 30, (B, 16, 1)).astype(np.float32), -1)
        tx, ty = torch.from_numpy(x).to(dev), torch.from_numpy(y).to(dev)
        h, lp = torch.full((B, 16), 99.0, device=dev), torch.full((B, 16), 99.0, device=dev)
        got = D.domino_token_logprobs(tx, ty, 0.9, entropy=h)
        assert not got.any() and not h.any(), (got.max(), h.min())
        g = torch.full_like(tx, 99.0)
        zero = torch.zeros((B, 16), device=dev)
        D.domino_policy_loss(tx, ty, zero, zero + 1, temperature=0.9, logp=lp, grad=g)
        assert not lp.any() and g.abs().max().item() < 1e-36
        other = (ty + 1) % V  # a token of no weight beside one of all
        D.domino_token_logprobs(tx, other, 0.9, entropy=h)
        assert (h >= 0).all() and h.max().item() < 1e-6


@pytest.mark.parametrize("T", [2.1e-38, 1e-30, 1e-6, 1e6, 9.9e19])
def test_extreme_temperatures(dev, T):
    import draft_block_causal_amd as D

    rng = np.random.default_rng(3)
    for V in (5003, 40003):
        x = rng.normal(size=(1, 4, V)).astype(np.float32) * 3
        x[0, 1] = np.round(x[0, 1])  # several largest entries
        x[0, 2, ::3] = -np.inf
        x[0, 3, 7] = np.finfo(np.float32).min
        y = np.argmax(x, -1).astype(np.int32)
        y[0, 3] = 8
        h = torch.full((1, 4), 99.0, device=dev)
        got = D.domino_token_logprobs(torch.from_numpy(x).to(dev), torch.from_numpy(y).to(dev), T, entropy=h)
        want, ent = O.token_logprobs(x, y, T)
        x64 = x.astype(np.float64)
        room = _rel_s(x64, T) + np.abs(want) * 1.01 * E
        got = got.cpu().numpy()
        with np.errstate(over="ignore"):  # a value past float32's largest, 3.4e38, rounds to -inf
            same = got == want.astype(np.float32)
        assert np.all(same | (np.abs(got - want) <= room)), (V, got, want)
        assert np.all(np.abs(h.cpu().numpy() - ent) <= _entropy_room(x64, T, ent)), (V, h, ent)


@pytest.mark.parametrize("V,extra", [(5003, 13), (20011, 0), (60001, 13), (99001, 13), (151936, 13), (151936, 0),
                                     (151936, 140)])
@pytest.mark.parametrize("kl_coef,T", [(0.05, 1.0), (0.0, 0.7)])
def test_loss_and_divergence_of_held_rows(dev, V, extra, kl_coef, T):
    # as many rows as compute units and `extra` (rows beyond a round of long ones go in slices; 140 are held again); ratios
    # on both sides of both limits, either sign of advantage, rows of weight 0.  A ratio and the loss move with rel(s) as
    # the log-probability does.
    import draft_block_causal_amd as D

    rows = torch.cuda.get_device_properties(dev).multi_processor_count + extra
    log(f"held rows: V={V} rows={rows} kl_coef={kl_coef} T={T}")
    gen = torch.Generator(device=dev).manual_seed(V + extra)
    x = torch.randn((rows, V), generator=gen, device=dev) * 2
    y = torch.randint(0, V, (rows, 1), generator=gen, device=dev)
    x.scatter_add_(1, y, torch.full((rows, 1), 7.0, device=dev))
    z = (x.double() - x.double().amax(1, keepdim=True)) / T
    lp = z - z.exp().sum(1, keepdim=True).log()
    p = lp.exp()
    delta = (2.8 * LOG2E * -(p * z).sum(1) + 8) * E
    now, p_y = lp.gather(1, y)[:, 0], p.gather(1, y)[:, 0]
    i = torch.arange(rows, device=dev)
    off = torch.tensor([-0.5, -0.1, 0.1, 0.22, 0.4], device=dev)[i % 5]  # ratios 0.61, 0.90, 1.11, 1.25, 1.49
    adv = torch.randn(rows, generator=gen, device=dev) * torch.where(i // 5 % 2 == 0, 1.0, -1.0)
    w = (torch.rand(rows, generator=gen, device=dev) + 0.5) / rows * (i % 7 != 6)
    old, ref = (now - off).float(), (now + torch.randn(rows, generator=gen, device=dev) * 0.4).float()
    v = lambda t: t.view(rows, 1)  # noqa: E731
    out = {k: torch.full((rows, 1), 99.0, device=dev) for k in ("logp", "kl")}
    grad = torch.full((rows, 1, V), 99.0, device=dev)
    loss = D.domino_policy_loss(x.view(rows, 1, V), v(y.int()), v(old), v(adv), clip_low=0.2, clip_high=0.28, kl_coef=kl_coef,
                                ref_logp=v(ref), weights=v(w), temperature=T, grad=grad, **out)
    live, A, W = w != 0, adv.double(), w.double()
    r, d = (now - old.double()).exp(), ref.double() - now
    kl = torch.expm1(d) - d
    plain, clipped = r * A, r.clamp(0.8, 1.28) * A
    inside = plain <= clipped
    assert inside[live].any() and (~inside)[live].any()
    want = (W * (kl_coef * kl - torch.minimum(plain, clipped))).sum()
    slope = torch.where(inside, plain.abs(), 0)
    room = (W * (slope + kl_coef * torch.expm1(d).abs()) * 1.01 * delta).sum() + want.abs() * 1.01 * E
    assert abs(loss.item() - want.item()) <= room.item(), (loss.item(), want.item(), room.item())
    got = out["logp"][:, 0].double()
    assert not got[~live].any() and ((got - now).abs() <= delta + now.abs() * 1.01 * E)[live].all()
    got = out["kl"][:, 0].double()
    room = torch.expm1(d).abs() * 1.01 * delta + delta**2 + kl * 1.01 * E
    assert not got[~live].any() and ((got - kl).abs() <= room)[live].all(), (got - kl).abs().max()
    coef = W / T * (-kl_coef * torch.expm1(d) - torch.where(inside, plain, 0))
    dcoef = W / T * (slope + kl_coef * d.exp()) * 1.01 * delta
    # others: the term, s, k and a product; the token: coef r / s, r of the other entries alone
    room = p * (coef.abs()[:, None] * ((5.6 + 2.8 * LOG2E * -z) * E + delta[:, None]) + dcoef[:, None])
    at_y = (1 - p_y) * (coef.abs() * (delta / (1 - p_y) + 1.01 * E) + dcoef)
    room.scatter_(1, y, at_y[:, None])
    want = -coef[:, None] * p
    want.scatter_(1, y, (coef * (1 - p_y))[:, None])
    bad = (grad[:, 0].double() - want).abs() > room + 1e-36
    assert not bad.any(), (torch.nonzero(bad)[:3], bad.sum())


def test_token_of_no_probability_in_held_rows(dev):
    # a token whose logit is -inf has an infinite divergence, which counts only with a coefficient; the other rows are as
    # they were
    import draft_block_causal_amd as D

    for V, extra in ((5003, 0), (99001, 13)):
        rows = torch.cuda.get_device_properties(dev).multi_processor_count + extra
        gen = torch.Generator(device=dev).manual_seed(V)
        x = torch.randn((rows, 1, V), generator=gen, device=dev)
        y = torch.randint(0, V, (rows, 1), generator=gen, device=dev, dtype=torch.int32)
        lp = D.domino_token_logprobs(x, y)
        one = torch.ones((rows, 1), device=dev)
        kl, g = torch.empty_like(one), torch.empty_like(x)
        a = D.domino_policy_loss(x, y, lp, one, ref_logp=lp, kl=kl, grad=g)
        kl0, g0, hit = kl.clone(), g.clone(), torch.zeros(rows, dtype=torch.bool, device=dev)
        for i in (2, rows - 1):
            x[i, 0, y[i, 0].item()] = -np.inf
            hit[i] = True
        b = D.domino_policy_loss(x, y, lp, one, ref_logp=lp, kl=kl, grad=g)
        assert (kl[hit] == np.inf).all() and not g[hit].any()  # ratio 0: neither loss nor gradient
        assert torch.equal(kl[~hit], kl0[~hit]) and torch.equal(g[~hit], g0[~hit])
        # each row gives -ratio / rows, ratio within rel(s) of 1; normal logits have M < 5.5 and a weighted mean of 1, so
        # tbar < 6.5 and rel(s) < 27 e; both losses, near -1, are rounded once
        assert abs((b - a).item() - 2 / rows) <= 2 / rows * 27 * E + 2 * E
        assert D.domino_policy_loss(x, y, lp, one, ref_logp=lp, kl_coef=0.1, grad=g).item() == np.inf


@pytest.mark.parametrize("T", [0.7, 1.3, 60.3])
@pytest.mark.parametrize("depth", [1e3, 1e5, 6e5, 1e7])
def test_tokens_far_below_their_rows_maximum(dev, depth, T):
    # log-probabilities of -1e3 ... -1e7: T counts with all its digits, so that a divergence from a reference near by is
    # right to the bound of the row's sum
    import draft_block_causal_amd as D

    rng = np.random.default_rng(8)
    for B, V in ((1, 300), (1, 40003), (34, 5003)):
        x = (rng.normal(size=(B, 4, V)) * 2 * T).astype(np.float32)
        y = rng.integers(0, V, size=(B, 4)).astype(np.int32)
        np.put_along_axis(x, y[..., None].astype(np.int64), (-depth * T * rng.uniform(1, 2, (B, 4, 1))).astype(np.float32), -1)
        x64 = x.astype(np.float64)
        want, _ = O.token_logprobs(x, y, T)
        ref = (want + rng.uniform(0.5, 1.5, want.shape)).astype(np.float32)
        d = ref.astype(np.float64) - want
        rel = _rel_s(x64, T) + 2.0**-50 * np.abs(want)  # (float64's own steps)
        t = [torch.from_numpy(a).to(dev) for a in (x, y, want.astype(np.float32), np.ones(y.shape, np.float32), ref)]
        kl, g = torch.full(y.shape, 99.0, device=dev), torch.empty_like(t[0])
        for grad in (g, None):
            D.domino_policy_loss(t[0], t[1], t[2], t[3], ref_logp=t[4], temperature=T, kl=kl, grad=grad)
            got = kl.cpu().numpy().astype(np.float64)
            value = np.expm1(d) - d
            room = np.abs(np.expm1(d)) * 1.01 * rel + rel**2 + value * 1.01 * E
            assert np.all(np.abs(got - value) <= room), (B, V, np.abs((got - value) / room).max())


@pytest.mark.parametrize("T", [1.0, 0.83, 1.17, 0.59])
@pytest.mark.parametrize("V", [2, 3])
def test_single_terms_far_from_zero(dev, V, T):
    # one or two terms besides the token's, so that no error averages out, up to and beyond the magnitude from which rows
    # are taken around their maximum; the divergence at d = 1 shows the log-probability to 2e-8
    import draft_block_causal_amd as D

    rng = np.random.default_rng(V)
    for log2 in (4, 10, 14, 16, 18, 19, 19.5, 19.9, 20.2, 22):
        base = np.float32(2.0**log2 / LOG2E * T)
        step = float(np.spacing(base)) if base > 2.0**17 else 2.0**-7
        for sign in (1, -1):
            x = (sign * base + step * np.round(rng.uniform(-6, 6, (64, 16, V)) / step)).astype(np.float32)
            y = rng.integers(0, V, size=(64, 16)).astype(np.int32)
            want, _ = O.token_logprobs(x, y, T)
            ref = (want + 1).astype(np.float32)
            d = ref.astype(np.float64) - want
            t = [torch.from_numpy(a).to(dev) for a in (x, y, want.astype(np.float32), np.ones(y.shape, np.float32), ref)]
            kl = torch.full(y.shape, 99.0, device=dev)
            D.domino_policy_loss(t[0], t[1], t[2], t[3], ref_logp=t[4], temperature=T, kl=kl)
            value = np.expm1(d) - d
            rel = _rel_s(x.astype(np.float64), T)
            err = np.abs(kl.cpu().numpy() - value) - value * 1.01 * E
            assert np.all(err <= np.expm1(d) * 1.01 * rel + rel**2), (log2, sign, (err / np.expm1(d) / rel).max())
