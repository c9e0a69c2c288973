"""Finite rows whose sum of squares is past FP32's largest value, in the quantising
front ends: the rounding of the exact sum is infinity, so rstd is 0, the normed row
is zeros and its codes and scale are those of zeros, as the oracle has them.
rmsnorm_linear_mxfp8, rmsnorm_linear_w8a8 (streamed quantiser and row kernels) and
rnl_add_rmsnorm_mxfp8 agree bit for bit.

Rows: of size 1e20 (squares overflow), 3e18 (only their sum does; divided by K first
it does not), 1e16 (nothing does), 1, and 1 with a single element of 3e38.  (Zeros
keep their signs.)"""
import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu

rnl = pytest.importorskip("rmsnorm_linear_projection_gb300")


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rmsnorm_linear_projection_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    yield
    rnl.rnl_check_device_error()


def rows(T, K):
    g = torch.Generator().manual_seed(T + K)
    x = torch.randn(T, K, generator=g)
    size = [1.0, 1e20, 3e18, 1e16, 1.0, 1.0]
    x *= torch.tensor([size[t % 6] for t in range(T)])[:, None]
    x[5::6, K // 3] = 3e38
    gamma = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    return x.bfloat16(), gamma


def bits(t):
    return t.view(torch.uint16).numpy()


@pytest.mark.parametrize("T,K,block", [(6, 64, 32), (13, 1024, 64), (40, 4096, 32), (7, 8256, 64), (6, 36864, 64)])
@pytest.mark.parametrize("mode", [0, 1])
def test_mxfp8(orc, T, K, block, mode):
    x, gamma = rows(T, K)
    codes, scale = orc.mxfp8_quant_rows(bits(x), bits(gamma), 1e-6, mode, block)
    # the rows are what they are meant to be
    assert [bool(v.any()) for v in scale[:6]] == [True, False, mode == 1, True, True, False]
    got = rnl.rnl_add_rmsnorm_mxfp8(x.cuda(), gamma.cuda(), norm_mode=mode, block=block)
    w = torch.randint(0, 100, (32, K), dtype=torch.uint8, device="cuda")
    ws = torch.full((32, K // block), 120, dtype=torch.uint8, device="cuda")
    c, s = torch.empty((T, K), dtype=torch.uint8, device="cuda"), torch.empty((T, K // block), dtype=torch.uint8, device="cuda")
    out = rnl.rmsnorm_linear_mxfp8(x.cuda(), gamma.cuda(), w, ws, norm_mode=mode, block=block, x_codes_out=c, x_scale_out=s)
    rnl.rnl_check_device_error()
    for a, b in (got, (c, s)):
        assert np.array_equal(a.cpu().numpy(), codes) and np.array_equal(b.cpu().numpy(), scale)
    assert torch.isfinite(out).all() and (out[1] == 0).all()


@pytest.mark.parametrize("T,K", [(13, 1024), (40, 4096), (7, 8208)])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("stream", ["1", "0"])
def test_w8a8(orc, monkeypatch, T, K, mode, stream):
    monkeypatch.setenv("RNL_W8A8_STREAM", stream)
    x, gamma = rows(T, K)
    wq = np.random.default_rng(0).integers(-127, 128, (24, K)).astype(np.int8)
    w_scale = np.full(24, 0.01, np.float32)
    want = orc.rmsnorm_linear_w8a8(bits(x), bits(gamma), wq, w_scale, 1e-6, mode)
    assert want["x_scale"][1] == 0
    q, xs = torch.empty((T, K), dtype=torch.int8, device="cuda"), torch.empty((T,), dtype=torch.float32, device="cuda")
    out = rnl.rmsnorm_linear_w8a8(x.cuda(), gamma.cuda(), dev(wq), dev(w_scale), norm_mode=mode, q_out=q, x_scale_out=xs)
    rnl.rnl_check_device_error()
    assert np.array_equal(q.cpu().numpy(), want["q"]) and np.array_equal(xs.cpu().numpy(), want["x_scale"])
    assert torch.isfinite(out).all() and (out[1] == 0).all()
