"""Pins of the roll-out and policy oracle on the CPU: hand-worked values, exact
rational rounding, torch's own log-softmax, and the policy gradient against
central differences of the loss."""
import math

import numpy as np
import pytest
import torch

import domino_synth as S
import oracle as O


def test_quantize_by_hand():
    q, s = O.quantize_rows(np.array([[127.0, -127.0, 0.5, 1.5, -2.5, 0.0]], np.float32))
    assert q.tolist() == [[127, -127, 0, 2, -2, 0]] and s.tolist() == [1.0]  # ties go to the even integer
    q, s = O.quantize_rows(np.array([[0.0, 0.0], [np.inf, 1.0], [np.nan, 1.0]], np.float32))
    assert not q.any() and s[0] == 0 and np.isnan(s[1:]).all()


@pytest.mark.parametrize("bits", [False, True])
def test_quantize_against_rational_arithmetic(bits):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(40, 64)).astype(np.float32) * np.exp2(rng.integers(-120, 100, size=(40, 1))).astype(np.float32)
    if bits:
        x = S.bf16_bits_to_f32(S.f32_to_bf16_bits(x))
    q, s = O.quantize_rows(x)
    for r in range(len(x)):
        want, scale = O.quantize_row(x[r])
        assert q[r].tolist() == want
        assert s[r] == pytest.approx(scale, rel=1e-15)


def test_base_logits_i8_by_hand():
    out = O.base_logits_i8(np.array([[[1, -2]]], np.int8), np.array([[0.5]]), np.array([[3, 4], [-127, 127]], np.int8),
                           np.array([2.0, 0.1]))
    np.testing.assert_allclose(out, [[[-5.0, -19.05]]], rtol=1e-12)


def test_token_logprobs_against_torch():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(2, 3, 11)) * 3
    x[0, 1, 4] = -np.inf
    y = rng.integers(0, 11, size=(2, 3))
    lp, h = O.token_logprobs(x, y, 0.7)
    ls = torch.log_softmax(torch.from_numpy(x) / 0.7, -1)
    np.testing.assert_allclose(lp, ls.gather(-1, torch.from_numpy(y)[..., None])[..., 0].numpy(), rtol=1e-12)
    np.testing.assert_allclose(h, torch.distributions.Categorical(logits=ls).entropy().numpy(), rtol=1e-10)
    lp, h = O.token_logprobs(np.full((1, 2, 4), -np.inf), np.zeros((1, 2), int), weights=np.array([[1.0, 0.0]]))
    assert lp[0, 0] == -np.inf and lp[0, 1] == 0 and not h.any()


def test_policy_loss_by_hand():
    x = np.log(np.array([[[0.25, 0.75]]]))
    # ratio 0.25 / 0.2 = 1.25, A = 2: clipped at 1.2, no slope; reference 0.5: d = ln 2, kl = 2 - ln 2 - 1
    r = O.policy_loss(x, np.array([[0]]), np.log([[0.2]]), np.array([[2.0]]), beta=0.5, ref=np.log([[0.5]]))
    kl = 1 - math.log(2)
    assert r["loss"] == pytest.approx(-2.4 + 0.5 * kl)
    assert r["kl"][0, 0] == pytest.approx(kl)
    np.testing.assert_allclose(r["grad"][0, 0], -0.5 * np.array([0.75, -0.75]))
    # A = -2: not clipped from above
    r = O.policy_loss(x, np.array([[0]]), np.log([[0.2]]), np.array([[-2.0]]))
    assert r["loss"] == pytest.approx(2.5)
    np.testing.assert_allclose(r["grad"][0, 0], 2.5 * np.array([0.75, -0.75]))


@pytest.mark.parametrize("T,beta,ref", [(1.0, 0.0, False), (0.7, 0.3, True), (1.6, 0.0, True)])
def test_policy_gradient_against_differences(T, beta, ref):
    rng = np.random.default_rng(7)
    B, K, V = 2, 4, 6
    x = rng.normal(size=(B, K, V))
    y = rng.integers(0, V, size=(B, K))
    lp, _ = O.token_logprobs(x, y, T)
    old = lp - rng.choice([-0.5, -0.1, 0.1, 0.5], size=(B, K))  # ratios away from the borders 0.8 and 1.3
    A = rng.normal(size=(B, K))
    w = rng.uniform(0.5, 1.5, size=(B, K))
    w[1, 2] = 0
    rf = lp + rng.normal(size=(B, K)) * 0.3 if ref else None

    def loss(z):
        return O.policy_loss(z, y, old, A, 0.2, 0.3, beta, rf, w, T)["loss"]

    g = O.policy_loss(x, y, old, A, 0.2, 0.3, beta, rf, w, T)["grad"]
    h = 1e-6
    for idx in np.ndindex(B, K, V):
        up, dn = x.copy(), x.copy()
        up[idx] += h
        dn[idx] -= h
        assert (loss(up) - loss(dn)) / (2 * h) == pytest.approx(g[idx], abs=1e-7)
    assert not g[1, 2].any()
