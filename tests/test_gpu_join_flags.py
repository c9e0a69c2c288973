"""Joins of the grouped products leave no flag in the workspace: calls and replays of
a captured call, whose epoch is the same every time, on work that is cut between CTA
pairs.  (The flags stand in the workspace's last slot of 256 KB.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

rnl = pytest.importorskip("rmsnorm_linear_projection_gb300")
SLOT = 2 * 128 * 256 * 4


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rmsnorm_linear_projection_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    yield
    rnl.rnl_check_device_error()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,K,N", [(3, 4096, 512), (300, 2048, 1000), (5000, 1024, 2048)])
def test_no_flag_stays(mx, M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M)
    E = 3
    off = torch.tensor([0, M // 3, M // 3, M], dtype=torch.int32, device="cuda")
    ws = torch.zeros(rnl.workspace_size(rnl.OP_GROUPED, M, K, N, E), dtype=torch.uint8, device="cuda")
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    if mx:
        x, w = (torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8) for s in ((M, K), (E, N, K)))
        xs, wsc = (torch.full(s, 118, dtype=torch.uint8, device="cuda") for s in ((M, K // 64), (E, N, K // 64)))

        def call():
            rnl.rnl_grouped_linear_mxfp8(x, xs, w, wsc, off, out=out, workspace=ws)
    else:
        x, w = torch.randn(M, K, generator=g, device="cuda").bfloat16(), torch.randn(E, N, K, generator=g, device="cuda").bfloat16()

        def call():
            rnl.rnl_grouped_linear_bf16(x, w, off, out=out, workspace=ws)
    call()
    rnl.rnl_check_device_error()
    want = out.clone()
    assert ws[:-SLOT].any()  # partial sums were handed over
    assert not ws[-SLOT:].any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(5):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and not ws[-SLOT:].any()
    rnl.rnl_check_device_error()
