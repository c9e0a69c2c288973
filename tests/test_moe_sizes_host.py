"""Sizes outside what the expert layer's calls take reach the calls' own refusal: the
binding asks for no memory of such a size first."""
import pytest
import torch

from rmsnorm_linear_projection_gb300 import _experts as ex
from rmsnorm_linear_projection_gb300 import _native as nat


class Refuses:
    """A library that refuses every call, and notes with which arguments."""

    def __init__(self):
        self.args = []

    def __getattr__(self, name):
        if name == "rnl_workspace_size":
            return lambda *a: 0
        if name == "rnl_status_string":
            return lambda s: b"refused"

        def call(*a):
            self.args.append(a)
            return 4
        return call


@pytest.fixture
def lib(monkeypatch):
    r = Refuses()
    monkeypatch.setattr(nat, "load", lambda path=None: r)
    monkeypatch.setattr(nat, "_lib", None)
    monkeypatch.setattr(ex, "_workspace_size", nat.workspace_size)
    monkeypatch.setattr(nat, "_stream", lambda dev, stream: None)
    return r


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("block", [-64, -1, 0])
@pytest.mark.parametrize("call", [ex.rnl_add_rmsnorm_mxfp8, ex.rnl_quant_mxfp8])
def test_blocks(lib, call, block):
    with pytest.raises(nat.RnlError):
        call(z(4, 128), block=block)
    assert block in lib.args[-1]


@pytest.mark.parametrize("top_k", [-3, 0, 9, 1 << 40])
def test_top_k(lib, top_k):
    with pytest.raises(nat.RnlError):
        ex.rnl_moe_route(z(4, 8, dtype=torch.float32), top_k)
    assert top_k in lib.args[-1]
