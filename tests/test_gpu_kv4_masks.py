"""Attention over the 4-bit cache (rnl_kv4_attention): what the mask leaves out.
Pages in front of a window may have been freed."""
import pytest
import torch

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


@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 32), (128, 64), (256, 16), (256, 128)])
@pytest.mark.parametrize("rows", [1, 3, 60])
def test_pages_in_front_of_a_window_may_be_gone(D, page, rows):
    """Table entries of pages that no row reads any more are -1, or beyond the
    cache: the bits of the call with all pages there, and no device error."""
    g = gen(D + page + rows)
    lens = [300, 301, 316, 333, 347, 90]
    c, t = filled(g, lens, 2, page, D, 32)
    cu = i32([rows * b for b in range(len(lens) + 1)])
    q = randn(g, rows * len(lens), 8, D).bfloat16()
    for tt in (t, wide(t, page)):  # both kernels where there are many rows
        for window in (1, 17, 50, 130):
            want = rnl.rnl_kv4_attention(q, c, tt, i32(lens), cu, window=window)
            rnl.rnl_check_device_error()
            for gone in (-1, c.n_pages + 3):
                freed = tt.clone()
                for b, n in enumerate(lens):
                    freed[b, :max(0, n - rows + 1 - window) // page] = gone
                out = rnl.rnl_kv4_attention(q, c, freed, i32(lens), cu, window=window)
                rnl.rnl_check_device_error()
                assert torch.equal(out, want)
