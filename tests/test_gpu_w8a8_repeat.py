"""The streamed W8A8 quantiser, called again and again without a pause: every CTA
takes many rows through its ring of row slots, whose places are filled again
right behind the reads; the same codes, scales and outputs every time, and the
codes of an FP32 restatement but for rounding ties."""
import pytest
import torch

pytestmark = pytest.mark.gpu

rnl = pytest.importorskip("rmsnorm_linear_projection_gb300")


@pytest.mark.parametrize("T,K", [(6000, 2048), (9001, 1024), (3000, 4096), (5003, 7168)])
def test_calls_in_a_row(T, K):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rmsnorm_linear_projection_gb300 import build
    build.build()
    g = torch.Generator(device="cuda").manual_seed(K)
    N = 128
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).bfloat16()
    Wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    ws = torch.full((N,), 1e-3, device="cuda")
    work = torch.empty(rnl.workspace_size(rnl.OP_W8A8, T, K, N), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(20):
        q = torch.empty(T, K, dtype=torch.int8, device="cuda")
        s = torch.empty(T, device="cuda")
        outs.append((rnl.rmsnorm_linear_w8a8(x, gamma, Wq, ws, q_out=q, x_scale_out=s, workspace=work), q, s))
    torch.cuda.synchronize()
    rnl.rnl_check_device_error()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    xf = x.double()
    y = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6) * gamma.double()
    want = y * 127 / y.abs().amax(-1, keepdim=True)
    # half a code, and FP32 errors of a few 2^-24 of a value up to 127
    assert ((outs[0][1].double() - want).abs() <= 0.5 + 127 * 2.0 ** -20).all()
