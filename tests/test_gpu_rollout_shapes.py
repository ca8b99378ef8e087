"""The kernels that the row quantiser and the base logits of an 8-bit LM head
choose by size: each of them against exact values.  Whole LM heads take one
wave a row; the product streams W for up to 64 rows in slices of K whose number
and width depend on K, and keeps finished tiles until its LDS is full."""
import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,cols", [(2049, 64), (4099, 512), (2050, 544), (2500, 1024), (2049, 1056), (3001, 2048),
                                       (2051, 2080), (2049, 2560), (2200, 4096), (2050, 4128), (2049, 8192), (2048, 4096)])
def test_quantize_many_rows(dev, rows, cols, bf16):
    # more than 2048 rows: one wave a row, 1, 2, 4, 8 and 16 groups a lane (2048: the last with four waves)
    import draft_block_causal_amd as D

    log(f"quantize {rows} x {cols} {'bf16' if bf16 else 'f32'}")
    rng = np.random.default_rng(rows + cols)
    x = torch.from_numpy(rng.normal(size=(rows, cols)).astype(np.float32) * np.exp2(rng.integers(-30, 30, (rows, 1))))
    x = x.bfloat16() if bf16 else x.float()
    x[5] = 0
    x[7, cols - 1] = np.inf
    x[9, 3] = np.nan
    x[11] = 1
    x[11, cols // 2] = 254  # ties: 1/2 everywhere else
    q = torch.full((rows + 1, cols), 55, dtype=torch.int8, device=dev)
    scale = torch.full((rows + 1,), 5.5, device=dev)
    D.domino_quantize_rows(x.to(dev), q[:rows], scale[:rows])
    torch.cuda.synchronize()
    want_q, want_s = O.quantize_rows(x.float().numpy())
    assert np.array_equal(q[:rows].cpu().numpy(), want_q)
    got, fine = scale[:rows].cpu().numpy().astype(np.float64), np.isfinite(want_s)
    assert np.array_equal(np.isnan(got), ~fine)
    assert np.all(np.abs(got - want_s)[fine] <= want_s[fine] * 2.0**-24)
    assert (q[rows] == 55).all() and scale[rows].item() == 5.5


def _check_logits(dev, M, d, V, seed, step=1):
    """`step`: every so many columns, the first and last hundred besides."""
    import draft_block_causal_amd as D

    gen = torch.Generator(device=dev).manual_seed(seed)
    hq = torch.randint(-128, 128, (1, M, d), generator=gen, dtype=torch.int8, device=dev)
    wq = torch.randint(-128, 128, (V, d), generator=gen, dtype=torch.int8, device=dev)
    hs = torch.rand((1, M), generator=gen, device=dev) * 0.03 + 0.01
    ws = torch.rand(V, generator=gen, device=dev) * 0.001 + 0.0001
    buf = torch.full((M * V + 1024,), 7.25, device=dev)
    out = buf[:M * V].view(1, M, V)
    D.domino_base_logits_i8(hq, hs, wq, ws, base_logits=out)
    torch.cuda.synchronize()
    assert torch.all(buf[M * V:] == 7.25)
    cols = np.unique(np.concatenate([np.arange(0, V, step), np.arange(min(V, 100)), np.arange(max(0, V - 100), V)]))
    at = torch.from_numpy(cols).to(dev)
    want = O.base_logits_i8(*(t.cpu().numpy() for t in (hq, hs, wq[at], ws[at])))
    got = out[:, :, at].cpu().numpy().astype(np.float64)
    # exact sums, their conversion and two products
    bad = np.abs(got - want) > np.abs(want) * 3.001 * 2.0**-24
    assert not bad.any(), np.argwhere(bad)[:5]


# every slice width and number of the streamed product, whole and cut short
@pytest.mark.parametrize("d", [32, 256, 288, 512, 576, 1024, 1056, 1536, 2048, 2080, 2560, 2592, 4096])
@pytest.mark.parametrize("M", [7, 16, 25, 32, 41, 48, 50, 64])
def test_streamed_logits(dev, M, d):
    log(f"streamed logits M={M} d={d}")
    _check_logits(dev, M, d, 4099, M + d)


@pytest.mark.parametrize("d,V", [(1024, 60000), (1536, 65537), (2048, 60003), (2560, 151936), (2560, 40002), (4096, 151936),
                                 (4096, 70001)])
@pytest.mark.parametrize("M", [16, 17, 48, 64])
def test_streamed_logits_in_several_flushes(dev, M, d, V):
    # more tiles a workgroup than its LDS holds, rows of C at any alignment
    log(f"streamed logits M={M} d={d} V={V}")
    _check_logits(dev, M, d, V, M + d, step=41)


@pytest.mark.parametrize("M", [1, 16])
@pytest.mark.parametrize("d,V", [(4128, 4099), (6144, 5000), (8192, 70001)])
def test_streamed_logits_of_long_rows(dev, M, d, V):
    log(f"streamed logits M={M} d={d} V={V}")
    _check_logits(dev, M, d, V, M + d, step=13)


@pytest.mark.parametrize("B,K,d,V", [(1, 17, 4128, 4099), (1, 64, 8192, 3001), (5, 13, 64, 999), (2, 64, 4096, 5001),
                                     (3, 43, 2560, 3333), (3, 64, 4096, 2050), (5, 51, 1056, 4099), (4, 64, 2560, 1031),
                                     (6, 43, 96, 777), (9, 57, 512, 1500)])
def test_tiled_logits(dev, B, K, d, V):
    # up to 64 rows of more than 4096 columns; more rows around the tiles' 128 and 256
    import draft_block_causal_amd as D

    log(f"tiled logits {B * K} rows d={d} V={V}")
    gen = torch.Generator(device=dev).manual_seed(B * K + d)
    hq = torch.randint(-128, 128, (B, K, d), generator=gen, dtype=torch.int8, device=dev)
    wq = torch.randint(-128, 128, (V, d), generator=gen, dtype=torch.int8, device=dev)
    hs, ws = torch.rand((B, K), generator=gen, device=dev) + 0.01, torch.rand(V, generator=gen, device=dev) + 0.01
    got = D.domino_base_logits_i8(hq, hs, wq, ws).cpu().numpy().astype(np.float64)
    want = O.base_logits_i8(*(t.cpu().numpy() for t in (hq, hs, wq, ws)))
    assert np.all(np.abs(got - want) <= np.abs(want) * 3.001 * 2.0**-24)
