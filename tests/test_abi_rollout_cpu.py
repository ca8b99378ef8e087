"""Host-side checks of the roll-out and policy calls: every refusal comes before
any GPU call, so it is tested on the CPU."""
import pytest
import torch

import draft_block_causal_amd as D

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_ARG, E_WS, E_HIP, E_UNSUP = 0, -1, -2, -3, -4, -5, -6, -7, -8


@pytest.fixture(scope="module")
def lib():
    return D.load_library()


def _quant(lib, rows=4, cols=64, dtype=1, x=0x10000, q=0x20000, scale=0x30000):
    return lib.domino_quantize_rows(rows, cols, dtype, x, q, scale, None)


def test_quantize_rows_refusals(lib):
    assert _quant(lib, rows=0, x=None, q=None, scale=None) == OK
    for cols in (0, 31, 33, 48, 8224, -32):
        assert _quant(lib, cols=cols) == E_SHAPE
    assert _quant(lib, rows=-1) == E_SHAPE
    assert _quant(lib, rows=1 << 24) == E_SHAPE
    assert _quant(lib, dtype=2) == E_DTYPE
    assert _quant(lib, x=None) == _quant(lib, q=None) == _quant(lib, scale=None) == E_NULL
    assert _quant(lib, x=0x10004) == _quant(lib, q=0x20008) == _quant(lib, scale=0x30002) == E_ALIGN
    assert _quant(lib, q=0x10000) == E_ARG          # in place
    assert _quant(lib, q=0x10000 + 4 * 64 * 2 - 16) == E_ARG
    assert _quant(lib, scale=0x20000 + 4 * 64 - 4) == E_ARG
    assert _quant(lib, scale=0x10010) == E_ARG


def _logits(lib, batch=2, block=3, d=64, vocab=100, hq=0x10000, hs=0x20000, wq=0x30000, ws=0x40000, out=0x50000):
    return lib.domino_base_logits_i8(batch, block, d, vocab, hq, hs, wq, ws, out, None)


def test_base_logits_i8_refusals(lib):
    assert _logits(lib, batch=0, hq=None, hs=None, wq=None, ws=None, out=None) == OK
    assert _logits(lib, batch=-1) == _logits(lib, block=0) == _logits(lib, block=65) == E_SHAPE
    for d in (0, 16, 48, 8224):
        assert _logits(lib, d=d) == E_SHAPE
    assert _logits(lib, vocab=0) == _logits(lib, vocab=1 << 24) == E_SHAPE
    assert _logits(lib, batch=129) == E_UNSUP
    for name in ("hq", "hs", "wq", "ws", "out"):
        assert _logits(lib, **{name: None}) == E_NULL
    assert _logits(lib, hq=0x10008) == _logits(lib, wq=0x30004) == _logits(lib, out=0x50008) == E_ALIGN
    assert _logits(lib, hs=0x20002) == _logits(lib, ws=0x40001) == E_ALIGN
    assert _logits(lib, out=0x10010) == _logits(lib, out=0x30000) == E_ARG
    assert _logits(lib, hs=0x50000) == _logits(lib, ws=0x50000 + 2 * 3 * 100 * 4 - 4) == E_ARG


NAN, INF = float("nan"), float("inf")


def _logp(lib, B=2, K=3, V=50, logits=0x100000, tokens=0x20000, w=None, T=1.0, logp=0x30000, ent=None, ws=0x40000,
          nb=None):
    nb = lib.domino_token_logprobs_workspace_size(max(B, 1), max(K, 1), max(V, 1)) if nb is None else nb
    return lib.domino_token_logprobs(B, K, V, logits, tokens, w, T, logp, ent, ws, nb, None)


def test_token_logprobs_refusals(lib):
    assert _logp(lib, B=0, logits=None, tokens=None, logp=None, ws=None) == OK
    assert _logp(lib, B=-1) == _logp(lib, B=(1 << 20) + 1) == _logp(lib, K=0) == _logp(lib, K=1025) == E_SHAPE
    assert _logp(lib, V=0) == _logp(lib, V=1 << 24) == E_SHAPE
    assert _logp(lib, B=1 << 20, K=5, nb=1 << 40) == E_UNSUP
    for T in (0.0, -1.0, NAN, INF, 1e-39, 1e21):
        assert _logp(lib, T=T) == E_ARG
    assert _logp(lib, logits=None) == _logp(lib, tokens=None) == _logp(lib, logp=None) == E_NULL
    assert _logp(lib, logits=0x100002) == _logp(lib, w=0x50001) == _logp(lib, ent=0x60002) == E_ALIGN
    assert _logp(lib, ent=0x30000) == _logp(lib, logp=0x20000) == _logp(lib, w=0x30014) == E_ARG
    assert _logp(lib, logp=0x100000 + 2 * 3 * 50 * 4 - 4) == E_ARG
    assert _logp(lib, logp=0x40000) == E_ARG  # inside the workspace
    assert _logp(lib, ws=None, nb=0) == _logp(lib, ws=0x40010) == E_WS
    assert _logp(lib, nb=lib.domino_token_logprobs_workspace_size(2, 3, 50) - 1) == E_WS


def test_workspace_sizes(lib):
    for f in (lib.domino_token_logprobs_workspace_size, lib.domino_policy_loss_workspace_size):
        assert f(0, 16, 100) == f(1, 0, 100) == f(1, 16, 0) == f((1 << 20) + 1, 1, 1) == f(1 << 20, 1024, 1) == 0
        assert f(1, 16, 151936) > 0 and f(1, 16, 151936) % 256 == 0
        assert f(32, 16, 151936) <= 1 << 20


def _policy(lib, B=2, K=3, V=50, logits=0x100000, tokens=0x20000, old=0x21000, ref=0x22000, adv=0x23000, w=0x24000,
            T=1.0, lo=0.2, hi=0.2, beta=0.1, loss=0x30000, logp=0x31000, kl=0x32000, grad=0x200000, ws=0x40000,
            nb=None):
    nb = lib.domino_policy_loss_workspace_size(max(B, 1), max(K, 1), max(V, 1)) if nb is None else nb
    return lib.domino_policy_loss(B, K, V, logits, tokens, old, ref, adv, w, T, lo, hi, beta, loss, logp, kl, grad, ws,
                                  nb, None)


def test_policy_loss_refusals(lib):
    assert _policy(lib, B=0, logits=None, loss=None, ws=None) == OK
    assert _policy(lib, B=-1) == _policy(lib, K=0) == _policy(lib, K=1025) == _policy(lib, V=0) == E_SHAPE
    assert _policy(lib, B=1 << 20, K=5, nb=1 << 40) == E_UNSUP
    for bad in ({"T": 0.0}, {"T": NAN}, {"lo": -0.1}, {"lo": 1.5}, {"lo": NAN}, {"hi": -0.1}, {"hi": INF},
                {"beta": -1.0}, {"beta": NAN}, {"beta": INF}):
        assert _policy(lib, **bad) == E_ARG, bad
    for name in ("logits", "tokens", "old", "adv", "loss"):
        assert _policy(lib, **{name: None}) == E_NULL, name
    assert _policy(lib, ref=None) == E_NULL  # a divergence term without a reference
    for name in ("logits", "tokens", "old", "ref", "adv", "w", "loss", "logp", "kl", "grad"):
        assert _policy(lib, **{name: 0x700002}) == E_ALIGN, name
    for bad in ({"logp": 0x21000}, {"kl": 0x22000}, {"loss": 0x23004}, {"logp": 0x32000}, {"loss": 0x31014},
                {"grad": 0x100004}, {"logp": 0x100000, "grad": 0x100000}, {"grad": 0x40000}, {"w": 0x200000}):
        assert _policy(lib, **bad) == E_ARG, bad
    assert _policy(lib, ws=None, nb=0) == _policy(lib, ws=0x40001) == E_WS
    assert _policy(lib, nb=lib.domino_policy_loss_workspace_size(2, 3, 50) - 1) == E_WS


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the behaviour without a GPU")
def test_valid_calls_without_gpu_report_hip_error(lib):
    assert _quant(lib) == E_HIP
    assert _logits(lib) == E_HIP
    assert _logp(lib) == E_HIP
    assert _policy(lib) == E_HIP
    assert _policy(lib, grad=0x100000) == E_HIP  # in place is allowed
    assert _policy(lib, ref=None, beta=0.0, w=None, logp=None, kl=None, grad=None) == E_HIP


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    z = torch.zeros
    with pytest.raises(ValueError, match="on a GPU"):
        D.domino_quantize_rows(z((2, 64)))
    with pytest.raises(ValueError, match="on a GPU"):
        D.domino_base_logits_i8(z((1, 2, 64), dtype=torch.int8), z((1, 2)), z((9, 64), dtype=torch.int8), z(9))
    x, y = z((2, 3, 7)), z((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        D.domino_token_logprobs(x, y)
    with pytest.raises(ValueError, match="on a GPU"):
        D.domino_policy_loss(x, y, z((2, 3)), z((2, 3)))
    with pytest.raises(TypeError):
        D.domino_quantize_rows([[1.0] * 32])


def test_workspace_over_an_input_is_refused(lib):
    """The workspace is written while the inputs are being read."""
    n, r = 2 * 3 * 50 * 4, 2 * 3 * 4
    for name, p, size in (("logits", 0x100000, n), ("tokens", 0x10000, r), ("w", 0x50000, r)):
        assert _logp(lib, **{name: p}, ws=p) == E_ARG, name
        assert _logp(lib, **{name: p - size}, ws=p) != E_ARG, name  # right before it
    for name, p, size in (("logits", 0x100000, n), ("tokens", 0x20000, r), ("old", 0x60000, r), ("ref", 0x70000, r),
                          ("adv", 0x80000, r), ("w", 0x90000, r)):
        assert _policy(lib, **{name: p}, ws=p) == E_ARG, name
        assert _policy(lib, **{name: p - size}, ws=p) != E_ARG, name
    assert _policy(lib, grad=0x100000, ws=0x100000) == E_ARG  # the logits' own buffer
