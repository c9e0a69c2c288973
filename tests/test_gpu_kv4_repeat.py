"""Attention over the 4-bit cache, called again and again without a pause: the
same bits every time, whatever stood in the workspace, and right ones.  Long
runs of prompts, in which the shared-memory places that hold a tile's codes are
filled again while the tile before is still being converted; pages of 128 tokens
and more come with a single copy, and fastest."""
import pytest
import torch

import kv4_plain as plain
from test_gpu_kv4 import filled, gen, i32, randn, wide

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


@pytest.mark.parametrize("D,block,page", [(64, 64, 128), (64, 64, 1024), (64, 64, 16), (64, 32, 128), (128, 64, 128),
                                          (128, 32, 128), (128, 64, 1024), (256, 64, 128)])
@pytest.mark.parametrize("lens,rows,G", [([6000, 17, 700], [300, 1, 70], 4), ([9000, 3000], [500, 1100], 1)])
def test_calls_in_a_row(D, block, page, lens, rows, G):
    g = gen(D + page + G)
    c, t = filled(g, lens, 2, page, D, block)
    t = wide(t, page)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    q = randn(g, cu[-1], 2 * G, D).bfloat16()
    lens_, cu_ = i32(lens), i32(cu)
    size = rnl.workspace_size(rnl.OP_KV4_ATTENTION, q.shape[0], D, 2 * G, 2)
    spaces = [torch.randint(0, 256, (size,), generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    ws = torch.empty_like(spaces[0])
    for causal in (True, False):
        outs = [(torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")) for _ in range(40 if D < 256 else 8)]
        torch.cuda.synchronize()
        for i, (out, lse) in enumerate(outs):
            ws.copy_(spaces[i & 1])
            rnl.rnl_kv4_attention(q, c, t, lens_, cu_, out=out, lse_out=lse, workspace=ws, causal=causal)
        torch.cuda.synchronize()
        rnl.rnl_check_device_error()
        o, z, tol, ltol = plain.attention(q, c, t, lens_, cu_, causal=causal)
        first = outs[0]
        assert ((first[0].double() - o).abs() <= tol).all() and ((first[1].double() - z).abs() <= ltol).all()
        assert all(torch.equal(a, first[0]) and torch.equal(b, first[1]) for a, b in outs[1:])


@pytest.mark.parametrize("D,block,page", [(64, 64, 128), (64, 32, 16), (128, 64, 1024), (128, 32, 64), (256, 64, 128),
                                          (256, 32, 16)])
@pytest.mark.parametrize("rows,G", [(1, 4), (1, 8), (2, 4), (4, 4), (1, 1)])
def test_few_rows_in_a_row(D, block, page, rows, G):
    """The few-row kernel's buffers are filled again as soon as they have been read."""
    g = gen(D + page + G + rows)
    lens = [20000, 300, 7000, 1, 12345, 64]
    c, t = filled(g, lens, 2, page, D, block)
    q = randn(g, rows * len(lens), 2 * G, D).bfloat16()
    lens_, cu_ = i32(lens), None if rows == 1 else i32([rows * b for b in range(len(lens) + 1)])
    ws = torch.empty(rnl.workspace_size(rnl.OP_KV4_ATTENTION, q.shape[0], D, 2 * G, 2), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")) for _ in range(100)]
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(outs):
        ws.fill_(i)
        rnl.rnl_kv4_attention(q, c, t, lens_, cu_, out=out, lse_out=lse, workspace=ws)
    torch.cuda.synchronize()
    rnl.rnl_check_device_error()
    o, z, tol, ltol = plain.attention(q, c, t, lens_, cu_)
    first = outs[0]
    assert ((first[0].double() - o).abs() <= tol).all()
    full = z > -float("inf")
    assert ((first[1].double() - z).abs() <= ltol)[full].all()
    assert all(torch.equal(a, first[0]) and torch.equal(b, first[1]) for a, b in outs[1:])
