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


@pytest.mark.parametrize("limit,T", [(2.0**30, 1.39), (2.0**20, 1.39), (2.0**20, 1.0), (2.0**20, 0.7)])
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
    # R is a rounded float32 product without its low part: at 2^30 |t| is up to 32 + 128, whose rounding (2 e |t| ln 2)
    # moves every term
    steps = 1.4 * 160 * E if limit > 2.0**24 else 0.0
    room = _rel_s(x.astype(np.float64), T) + np.abs(want) * E + steps
    assert np.all(np.abs(got - want) <= room), (got, want)
    got, g, want = _policy(dev, x, y, T)
    assert np.all(np.abs(got - want["logp"]) <= room), (got, want["logp"])
    # tbar < 1/2: rel(s) < 10 e twice (probability, ratio), and at most 8 e of a term and the gradient's roundings
    scale = np.abs(want["coef"])[..., None]
    assert np.all(np.abs(g - want["grad"]) <= scale * (28 * E + 2 * steps)), np.abs(g - want["grad"]).max()
