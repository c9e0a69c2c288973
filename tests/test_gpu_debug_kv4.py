"""The debug build on the multi-axis rotary stage, the 4-bit cache and attention
over it: every kernel form through the release library and the debug library,
the same bits and no check that fires."""
import pytest
import torch

from test_gpu_kv4 import gen, i32, randn, tables, wide
from test_gpu_rope_axes import layouts, make

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
    """The outputs (bit patterns) of a call on either library, with no device error."""
    def run():
        out = [t.clone().view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8) for t in call()]
        rnl.rnl_check_device_error()  # RNL_ERR_BOUNDS if a check fired
        return out
    release = run()
    with rnl.debug_library():
        assert rnl.rnl_debug_build()
        debug = run()
    assert all(torch.equal(a, b) for a, b in zip(release, debug))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 3, 1), (77, 8, 2), (300, 33, 3)])
def test_rope_axes(D, T, Hq, Hkv):
    y, pos, gam, table = make(T, Hq, Hkv, D, 3)
    for name, m in layouts(D, 3).items():
        both(lambda: rnl.rnl_qkv_rope_axes(y, Hq, Hkv, D, gam[0] if name == "sections" else None, gam[1], pos, m, table))


@pytest.mark.parametrize("D,block,page,H", [(64, 64, 16, 1), (128, 32, 64, 8), (256, 32, 1024, 3)])
def test_cache(D, block, page, H):
    g = gen(D)
    lens, rows = [1, 40, 0, 1030], [1, 33, 0, 700]
    t, P = tables(g, lens, page)
    cu = i32([0, 1, 34, 34, 734])
    k, v = randn(g, 736, H, D).bfloat16(), randn(g, 736, H, D).bfloat16()

    def call():
        c = rnl.Kv4Cache.empty(P, H, page, D, block)
        for x in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
            x.zero_()
        rnl.rnl_kv4_append(k, v, c, t, i32(lens), cu)
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        rnl.rnl_kv4_gather(c, t, i32(lens), 736, cu, k_out=ko, v_out=vo)
        return c.k_codes, c.k_scales, c.v_codes, c.v_scales, ko, vo
    both(call)


@pytest.mark.parametrize("D,block,page", [(64, 32, 16), (64, 64, 128), (128, 32, 32), (128, 64, 64), (256, 32, 16),
                                          (256, 64, 64)])
@pytest.mark.parametrize("rows,G", [([1, 1, 1], 1), ([1, 1, 1], 4), ([2, 1, 2], 4), ([4, 3, 5], 4), ([300, 1, 70], 4),
                                    ([500, 260, 257], 1)])
def test_attention(D, block, page, rows, G):
    g = gen(D + sum(rows) + G)
    H, lens = 2, [6000, 17, 700]
    t, P = tables(g, lens, page)
    c = rnl.Kv4Cache.empty(P, H, page, D, block)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    rnl.rnl_kv4_append(randn(g, cu[-1], H, D).bfloat16(), randn(g, cu[-1], H, D).bfloat16(), c, t, i32(lens), i32(cu))
    # a token far above the others, so that rows are taken one at a time too
    c.k_scales[int(t[0, 5999 // page]), 0, 5999 % page] += 60
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    q = randn(g, cu[-1] + 1, G * H, D).bfloat16()
    cu = None if max(rows) == 1 else i32(cu)
    if cu is None:
        q = q[:-1]
    for tt in (t, wide(t, page)):
        for kw in (dict(), dict(window=100), dict(causal=False)):
            def call():
                out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
                rnl.rnl_kv4_attention(q, c, tt, i32(lens), cu, out=out, lse_out=lse, **kw)
                return out, lse
            both(call)
