"""The package imports where torch has no GPU support."""
import importlib.util
import sys

import pytest
import torch

import draft_block_causal_amd as D


def _import_again(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("binding_again", sys.modules[D.Head.__module__].__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_import_without_torch_gpu_support(monkeypatch):
    module = _import_again(monkeypatch)
    assert module.domino_version() == D.domino_version()
    with pytest.raises(ValueError, match="on a GPU"):
        module.domino_quantize_rows(torch.zeros((2, 64)))


@pytest.mark.gpu
def test_calls_without_the_short_way_to_the_stream(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    short = D._lib._raw_stream
    module = _import_again(monkeypatch)
    assert module._raw_stream is not short
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert module._raw_stream(0) == short(0) == side.cuda_stream
        x = torch.randn((5, 64), device="cuda")
        q, scale = module.domino_quantize_rows(x)
        want, want_scale = D.domino_quantize_rows(x)
    side.synchronize()
    assert torch.equal(q, want) and torch.equal(scale, want_scale)
