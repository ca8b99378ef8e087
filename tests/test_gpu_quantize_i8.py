"""Rows in 8 bits and the base logits of an 8-bit LM head on the GPU against
the oracle.  Quantised values are equal to the exactly rounded quotients; sums
are exact, so a logit is off by its three float32 roundings at most."""
import numpy as np
import pytest
import torch

import domino_synth as S
import oracle as O
from _helpers import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_causal_amd as D

    D.load_library()
    return torch.device("cuda:0")


def _rows(rows, cols, seed, bf16, spread=0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)).astype(np.float32)
    if spread:
        x *= np.exp2(rng.integers(-spread, spread, size=(rows, 1))).astype(np.float32)
    return S.bf16_bits_to_f32(S.f32_to_bf16_bits(x)) if bf16 else x


def _check_quantize(dev, x, bf16):
    import draft_block_causal_amd as D

    t = torch.from_numpy(x).to(dev)
    q, scale = D.domino_quantize_rows(t.bfloat16() if bf16 else t)
    torch.cuda.synchronize()
    want_q, want_s = O.quantize_rows(x)
    assert np.array_equal(q.cpu().numpy(), want_q)
    got = scale.cpu().numpy().astype(np.float64)
    # one rounding of the quotient; below 2^-126 steps are 2^-149
    fine = np.isfinite(want_s)
    assert np.array_equal(np.isnan(got), ~fine)
    assert np.all(np.abs(got - want_s)[fine] <= want_s[fine] * 2.0**-24 + 2.0**-150)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (16, 4096), (5, 512), (5, 544), (7, 1024), (9, 1056),
                                       (645, 2560), (2, 4128), (3, 8192), (1000, 64)])
def test_quantize_matches_exact_rounding(dev, rows, cols, bf16):
    log(f"quantize {rows} x {cols} {'bf16' if bf16 else 'f32'}")
    _check_quantize(dev, _rows(rows, cols, rows + cols, bf16), bf16)


@pytest.mark.parametrize("bf16", [True, False])
def test_quantize_range_of_magnitudes(dev, bf16):
    _check_quantize(dev, _rows(300, 128, 1, bf16, spread=120), bf16)


def test_quantize_ties_and_neighbours_of_ties(dev):
    # the row's largest value is 127, so quotients are the values: halves, and their float32 neighbours
    half = np.arange(-126.5, 127, 1.0, dtype=np.float32)
    x = np.concatenate([half, np.nextafter(half, np.float32(-200)), np.nextafter(half, np.float32(200)),
                        np.full(32 - 3 * 254 % 32, 127.0, np.float32)])[None]
    assert x.shape[1] % 32 == 0
    _check_quantize(dev, x, False)
    _check_quantize(dev, x * np.float32(2.0**-100), False)
    _check_quantize(dev, x * np.float32(2.0**-133), False)  # denormal values (the neighbours round onto the halves)
    scaled = (x * np.float32(0.3)).astype(np.float32)
    _check_quantize(dev, scaled, False)
    half = np.concatenate([np.arange(-126.5, 127, 1.0), [127.0, -127.0]]).astype(np.float32)[None]
    _check_quantize(dev, half, True)  # exact in bf16 up to 128


def test_quantize_rows_without_values(dev):
    x = _rows(6, 64, 2, True)
    x[1] = 0
    x[3, 5] = np.inf
    x[4, 63] = np.nan
    x[5, 0] = -np.inf
    _check_quantize(dev, x, True)
    x = _rows(4, 64, 2, False)
    x[2] = 0
    x[2, 7] = 1e-45
    x[3] = np.finfo(np.float32).max
    _check_quantize(dev, x, False)


def _i8(rng, *shape):
    return rng.integers(-128, 128, size=shape).astype(np.int8)


def _logits_case(dev, B, K, d, V, seed=0, full=None):
    import draft_block_causal_amd as D

    rng = np.random.default_rng(seed)
    hq, wq = (_i8(rng, B, K, d), _i8(rng, V, d)) if full is None else (
        np.full((B, K, d), full, np.int8), np.full((V, d), full, np.int8))
    hs = (rng.uniform(0.5, 2, size=(B, K)) * 0.03).astype(np.float32)
    ws = (rng.uniform(0.5, 2, size=V) * 0.0005).astype(np.float32)
    t = [torch.from_numpy(a).to(dev) for a in (hq, hs, wq, ws)]
    # the words after the output are watched: nothing may be written there
    buf = torch.full((B * K * V + 1024,), 7.25, device=dev)
    out = buf[:B * K * V].view(B, K, V)
    D.domino_base_logits_i8(*t, base_logits=out)
    torch.cuda.synchronize()
    want = O.base_logits_i8(hq, hs, wq, ws)
    got = out.cpu().numpy().astype(np.float64)
    assert torch.all(buf[B * K * V:] == 7.25)
    # conversion, two products: (1 + 2^-24)^3 - 1
    assert np.all(np.abs(got - want) <= np.abs(want) * 3.001 * 2.0**-24), np.abs(got - want).max()
    return t, out


# rows: 1 .. 64 (streamed), more (tiled); K with and without a half step of 64; ragged vocabularies
@pytest.mark.parametrize("B,K,d,V", [
    (1, 1, 32, 1), (1, 1, 4096, 777), (1, 16, 64, 15), (1, 16, 4096, 4099), (1, 17, 96, 16), (2, 16, 2560, 1000),
    (3, 5, 8192, 333), (7, 5, 96, 4099), (3, 16, 4064, 2049), (1, 33, 256, 300), (1, 49, 544, 515), (4, 16, 512, 8191),
    (1, 64, 1024, 17),
    (1, 5, 8160, 4097), (13, 5, 32, 257), (5, 13, 96, 4099), (8, 16, 2560, 3000), (9, 15, 160, 511), (2, 64, 64, 255),
    (16, 16, 224, 777), (17, 16, 4096, 1031), (32, 16, 256, 2047), (33, 16, 1056, 513), (128, 16, 128, 129),
    (65, 3, 8192, 260), (128, 64, 32, 33),
])
def test_base_logits_i8_matches_oracle(dev, B, K, d, V):
    log(f"base_logits_i8 B={B} K={K} d={d} V={V}")
    _logits_case(dev, B, K, d, V, seed=B + K + d + V)


@pytest.mark.parametrize("B,K", [(1, 16), (3, 32)])
def test_base_logits_i8_largest_sums(dev, B, K):
    # every product 128 * 128 over 8192 columns: 2^27, the largest magnitude a sum can have
    _logits_case(dev, B, K, 8192, 65, full=-128)


@pytest.mark.parametrize("B,d,V", [(1, 512, 151936), (4, 512, 151936), (8, 512, 151936), (20, 512, 151936),
                                   (5, 32, 151936), (8, 128, 151936), (7, 160, 220000), (8, 256, 300004), (8, 64, 65536),
                                   (12, 64, 151936), (16, 128, 220001), (3, 64, 500000), (1, 96, 999999)])
def test_base_logits_i8_over_a_whole_vocabulary(dev, B, d, V):
    # many tiles per workgroup, down to one step of K each; checked on every 37th column against the oracle, and two
    # calls agree
    import draft_block_causal_amd as D

    K = 16
    log(f"base_logits_i8 whole vocabulary B={B} d={d} V={V}")
    rng = np.random.default_rng(B)
    hq, wq = _i8(rng, B, K, d), _i8(rng, V, d)
    hs, ws = rng.uniform(0.01, 0.02, (B, K)).astype(np.float32), rng.uniform(0.01, 0.02, V).astype(np.float32)
    t = [torch.from_numpy(a).to(dev) for a in (hq, hs, wq, ws)]
    out = D.domino_base_logits_i8(*t)
    again = D.domino_base_logits_i8(*t)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    cols = np.unique(np.concatenate([np.arange(0, V, 37), np.arange(V - 600, V)]))
    want = O.base_logits_i8(hq, hs, wq[cols], ws[cols])
    got = out[:, :, torch.from_numpy(cols).to(dev)].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= np.abs(want) * 3.001 * 2.0**-24)


@pytest.mark.parametrize("B,d,V", [(8, 32, 128000), (5, 64, 128001), (8, 128, 128003), (8, 160, 128000),
                                   (8, 1024, 128000), (5, 32, 170001), (8, 128, 170001), (6, 192, 170000),
                                   (8, 416, 170002), (8, 96, 90000), (8, 3232, 70000), (6, 3264, 135001),
                                   (8, 32, 260000), (7, 224, 262145), (8, 32, 400001), (8, 288, 330000)])
def test_base_logits_i8_tiles_in_pairs(dev, B, d, V):
    # whole pairs, a single tile behind them and workgroups that differ by a tile, of 256 and of 320 columns; one step
    # of K, two and more; ragged tiles first or second in a pair
    test_base_logits_i8_over_a_whole_vocabulary(dev, B, d, V)


def test_scales_of_zero_nan_and_extremes(dev):
    import draft_block_causal_amd as D

    rng = np.random.default_rng(9)
    hq, wq = _i8(rng, 1, 4, 64), _i8(rng, 70, 64)
    hs = np.array([[0.0, np.nan, 1e-30, 1e30]], np.float32)
    ws = rng.uniform(0.5, 1, 70).astype(np.float32)
    ws[3], ws[5] = 0, np.nan
    out = D.domino_base_logits_i8(*[torch.from_numpy(a).to(dev) for a in (hq, hs, wq, ws)]).cpu().numpy()[0]
    assert np.isnan(out[1]).all() and np.isnan(out[:, 5]).all()
    keep = np.arange(70) != 5
    assert not out[0, keep].any() and not out[[0, 2, 3], 3].any()
    assert np.isfinite(out[2:, keep]).all()


def test_empty_batch_and_no_rows(dev):
    import draft_block_causal_amd as D

    w = torch.zeros((9, 64), dtype=torch.int8, device=dev)
    out = D.domino_base_logits_i8(torch.zeros((0, 16, 64), dtype=torch.int8, device=dev), torch.zeros((0, 16), device=dev),
                                  w, torch.zeros(9, device=dev))
    assert out.shape == (0, 16, 9)
    q, s = D.domino_quantize_rows(torch.zeros((0, 64), device=dev))
    assert q.shape == (0, 64) and s.shape == (0,)


def test_quantised_logits_are_near_the_unquantised(dev):
    # |x - q s| <= s / 2 on both sides: |error| <= sum |h| ws/2 + |w| hs/2 + hs ws / 4 per product
    import draft_block_causal_amd as D

    w = S.get_workload("tiny_stress_b4")
    head, inp = S.make_workload(w)
    h, lm = S.to_torch(inp["hidden"], dev), S.to_torch(head["lm_head"], dev)
    hq, hs = D.domino_quantize_rows(h)
    wq, ws = D.domino_quantize_rows(lm)
    out = D.domino_base_logits_i8(hq, hs, wq, ws).cpu().numpy().astype(np.float64)
    h, lm, hs, ws = (t.double().cpu().numpy() for t in (h, lm, hs, ws))
    want = h @ lm.T
    room = (np.abs(h).sum(-1)[..., None] * ws / 2 + hs[..., None] * np.abs(lm).sum(-1) / 2
            + w.d * hs[..., None] * ws / 4)
    assert np.all(np.abs(out - want) <= room * (1 + 1e-5))


def test_graph_replays_and_another_stream(dev):
    import draft_block_causal_amd as D

    x = torch.from_numpy(_rows(48, 2560, 4, True)).to(dev).bfloat16().view(3, 16, 2560)
    lm = torch.from_numpy(_rows(5000, 2560, 5, True)).to(dev).bfloat16()
    wq, ws = D.domino_quantize_rows(lm)
    out = torch.empty((3, 16, 5000), device=dev)
    q, s = torch.empty(x.shape, dtype=torch.int8, device=dev), torch.empty((3, 16), device=dev)

    def call(stream=None):
        D.domino_quantize_rows(x, q, s, stream=stream)
        D.domino_base_logits_i8(q, s, wq, ws, out, stream=stream)

    call()
    torch.cuda.synchronize()
    ref = out.clone()
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for r in range(3):
        x.copy_(torch.from_numpy(_rows(48, 2560, 10 + r, True)).view(3, 16, 2560))
        out.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, out), f"replay {r}"
