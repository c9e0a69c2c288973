"""Rows into MXFP8 on the GPU (rnl_add_rmsnorm_mxfp8, rnl_quant_mxfp8).  Codes and
scales are exact functions of the inputs: they are compared bit for bit with
a plain implementation (the sum of squares exact in 64 bits, rounded to FP32
once, then one FP32 operation a step) and with the operands that
rmsnorm_linear_mxfp8 writes."""
import math

import pytest
import torch

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


def pow2(e):
    """2^e in FP32, -127 <= e <= 127."""
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e.double()).float()


def plain_quant(y, block):
    """FP32 rows -> (codes, scale bytes)."""
    b = y.unflatten(1, (-1, block))
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    X = torch.frexp(torch.where(bad, 1.0, amax)).exponent - 9
    X = torch.where(amax > 0, X, -127).clamp_min(-127)
    v = (b.double() * pow2(-X).double().unsqueeze(-1)).float().clamp(-448, 448)
    v = torch.where(bad.unsqueeze(-1), 0.0, v)
    codes = v.flatten(1).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.where(bad, 255, X + 127).to(torch.uint8)


def plain_norm(x, r, gamma, eps, mode):
    s = x.float()
    if r is not None:
        s = (s + r.float()).bfloat16().float()
    K = s.shape[1]
    inv = torch.tensor(1.0 / K, dtype=torch.float32, device=x.device)
    e = torch.tensor(eps, dtype=torch.float32, device=x.device)
    if mode == rnl.NORM_RSQRT:
        ms = s.double().square().sum(1, keepdim=True).float() * inv + e
    else:  # each FP32 square times 1 / K in FP32, then the sum
        ms = (s.square() * inv).double().sum(1, keepdim=True).float() + e
    y = s * (1.0 / torch.sqrt(ms))
    return s, y * gamma.float() if gamma is not None else y


ROWS = [(1, 32), (3, 64), (2, 320), (64, 4096), (700, 4096), (33, 1024), (5, 8192), (2000, 192), (3, 65536), (2, 36864),
        (700, 8256)]


@pytest.mark.parametrize("T,K,block", [(T, K, b) for T, K in ROWS for b in (32, 64) if K % b == 0])
@pytest.mark.parametrize("mode", [0, 1])
def test_norm(T, K, block, mode):
    g = torch.Generator(device="cuda").manual_seed(T * K + block)
    x = (torch.randn(T, K, generator=g, device="cuda") * torch.exp(torch.randn(K, generator=g, device="cuda"))).bfloat16()
    r = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    gamma = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).bfloat16()
    for res, gm in ((r, gamma), (None, gamma), (r, None), (None, None)):
        s, y = plain_norm(x, res, gm, 1e-5, mode)
        want = plain_quant(y, block)
        out = torch.empty_like(x) if res is not None else None
        got = rnl.rnl_add_rmsnorm_mxfp8(x, gm, residual=res, x_sum_out=out, eps=1e-5, norm_mode=mode, block=block)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        if out is not None:
            assert torch.equal(out, s.bfloat16())
    for target in (x, r):  # in place
        s, y = plain_norm(x, r, gamma, 1e-5, mode)
        a, b = x.clone(), r.clone()
        t = a if target is x else b
        got = rnl.rnl_add_rmsnorm_mxfp8(a, gamma, residual=b, x_sum_out=t, eps=1e-5, norm_mode=mode, block=block)
        assert torch.equal(t, s.bfloat16()) and torch.equal(got[0], plain_quant(y, block)[0])


@pytest.mark.parametrize("block", [32, 64])
def test_same_operand_as_the_projection(block):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(37, 1024, generator=g, device="cuda").bfloat16()
    gamma = torch.randn(1024, generator=g, device="cuda").bfloat16()
    w = torch.randint(0, 120, (128, 1024), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.full((128, 1024 // block), 120, device="cuda", dtype=torch.uint8)
    codes = torch.empty(37, 1024, device="cuda", dtype=torch.uint8)
    scale = torch.empty(37, 1024 // block, device="cuda", dtype=torch.uint8)
    out = rnl.rmsnorm_linear_mxfp8(x, gamma, w, ws, block=block, x_codes_out=codes, x_scale_out=scale)
    got = rnl.rnl_add_rmsnorm_mxfp8(x, gamma, block=block)
    assert torch.equal(got[0], codes) and torch.equal(got[1], scale)
    assert torch.equal(rnl.mxfp8_scaled_mm(*got, w, ws, block=block), out)


@pytest.mark.parametrize("T,K", [(1, 64), (130, 704), (1500, 2048), (3, 16384)])
@pytest.mark.parametrize("block", [32, 64])
def test_quant_of_rows_as_they_are(T, K, block):
    g = torch.Generator(device="cuda").manual_seed(T + K)
    # from far below the smallest scale up to bf16's largest values
    x = (torch.randn(T, K, generator=g, device="cuda").double()
         * torch.exp2(torch.randint(-130, 127, (T, K // block), generator=g, device="cuda").double())
         .repeat_interleave(block, 1)).float().bfloat16()
    x[0, :block] = 0
    if T > 1:
        x[1, 5] = math.inf
        x[T - 1, K - 1] = math.nan
    want = plain_quant(x.float(), block)
    got = rnl.rnl_quant_mxfp8(x, block=block)
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0], want[0])


def test_rows_that_are_not_finite_stay_among_themselves():
    x = torch.randn(6, 512, device="cuda").bfloat16()
    x[2, 100] = math.nan
    x[4, 7] = -math.inf
    codes, scale = rnl.rnl_add_rmsnorm_mxfp8(x, block=32)
    fine = rnl.rnl_add_rmsnorm_mxfp8(x[[0, 1, 3, 5]].contiguous(), block=32)
    assert torch.equal(codes[[0, 1, 3, 5]], fine[0]) and torch.equal(scale[[0, 1, 3, 5]], fine[1])
    assert (scale[2] == 255).all()   # the norm of a row with NaN
    assert scale[4, 0] == 255 and (scale[4, 1:] == 0).all()  # infinity times 0, and zeros
