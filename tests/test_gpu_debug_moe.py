"""The debug build on the expert layer: every call through the release library and
the debug library, the same bits and no check that fires."""
import pytest
import torch

from test_gpu_moe import gen, i32, layer, mx_case, randn, run_layer

pytestmark = pytest.mark.gpu

rnl = pytest.importorskip("rmsnorm_linear_projection_gb300")


@pytest.fixture(scope="module", autouse=True)
def debug_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rmsnorm_linear_projection_gb300 import build
    build.build()
    build.build(debug=True)
    torch.cuda.set_device(0)


def both(call):
    """The outputs of a call on either library, with no device error."""
    def run():
        out = call().clone().view(torch.int16)
        rnl.rnl_check_device_error()  # RNL_ERR_BOUNDS if a check fired
        return out
    release = run()
    with rnl.debug_library():
        assert rnl.rnl_debug_build()
        debug = run()
    assert torch.equal(release, debug)


@pytest.mark.parametrize("T,E,k,K,F", [(1, 8, 2, 512, 256), (300, 16, 4, 512, 352), (1500, 3, 2, 1088, 416)])
@pytest.mark.parametrize("mx", [False, True])
def test_layer(T, E, k, K, F, mx):
    g = gen(T)
    p = layer(g, T, E, k, K, F)
    x, res = randn(g, T, K).bfloat16(), randn(g, T, K).bfloat16()
    both(lambda: run_layer(p, x, res, k, mx)[0])


@pytest.mark.parametrize("counts", [[5, 0, 700, 1], [2000], [1] * 40])
@pytest.mark.parametrize("N", [513, 640])
def test_grouped(counts, N):
    x, xs, w, ws, offsets, rows, _ = mx_case(counts, 576, N, 64, True, 3)
    both(lambda: rnl.rnl_grouped_linear_mxfp8(x, xs, w, ws, i32(offsets), rows=rows))
    xb, wb = randn(gen(1), sum(counts), 200).bfloat16(), randn(gen(2), len(counts), N, 200).bfloat16()
    both(lambda: rnl.rnl_grouped_linear_bf16(xb, wb, i32(offsets)))
