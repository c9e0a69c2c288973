"""rnl_qkv_rope_axes (QKV split, optional head norm, rotary positions of several
axes) against a plain 64-bit implementation.  The normed values z are bf16 on
both sides and may fall on the other side of a rounding boundary (one ulp, at
most 2^-7 relative); the output mixes two of them and is rounded once more:
    |gpu - plain| <= 2^-7 (|z_i c_i| + |z_partner s_i|) + 2^-8 |out| + 2^-20.
Without the head norm z is the input itself: FP32 products and one rounding,
2^-8 |out| + 2^-22 (|z_i c_i| + |z_partner s_i|) (bf16's smallest steps aside)."""
import pytest
import torch

import kv4_plain as plain

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


def make(T, Hq, Hkv, D, axes, span=300, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    y = (2 * torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda")).bfloat16()
    pos = torch.randint(0, span, (axes, T), generator=g, device="cuda").int()
    gam = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    ang = torch.arange(span, dtype=torch.float64, device="cuda")[:, None] * 100.0 ** (
        -torch.arange(D // 2, dtype=torch.float64, device="cuda") * 2 / D)
    return y, pos, gam, torch.cat([ang.cos(), ang.sin()], 1).float()


def layouts(D, axes):
    half = D // 2
    return {"sections": [min(i * axes // half, axes - 1) for i in range(half)],
            "interleaved": [i % axes for i in range(half)],
            "uneven": [0 if i < half - 3 else axes - 1 for i in range(half)]}


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("layout", ["sections", "interleaved", "uneven"])
@pytest.mark.parametrize("norm", ["both", "none", "q", "k"])
def test_matches_plain(D, axes, layout, norm):
    Hq, Hkv, T = 5, 2, 37
    y, pos, gam, table = make(T, Hq, Hkv, D, axes)
    m = layouts(D, axes)[layout]
    qg = gam[0] if norm in ("both", "q") else None
    kg = gam[1] if norm in ("both", "k") else None
    q, k, v = rnl.rnl_qkv_rope_axes(y, Hq, Hkv, D, qg, kg, pos, m, table)
    wq, wk, wv, mq, mk = plain.rope_axes(y, Hq, Hkv, D, qg, kg, pos, m, table, 1e-6)
    assert torch.equal(v.double(), wv)
    for got, want, mag, gamma in ((q, wq, mq, qg), (k, wk, mk, kg)):
        f = 2.0 ** -7 if gamma is not None else 2.0 ** -22
        bound = f * mag + 2.0 ** -8 * want.abs() + (2.0 ** -20 if gamma is not None else 2.0 ** -100)
        assert ((got.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 32, 8, 128), (333, 7, 1, 64), (50, 4, 4, 256), (9, 0, 3, 128), (9, 3, 0, 128)])
def test_one_axis_is_the_single_position_stage(T, Hq, Hkv, D):
    y, pos, gam, table = make(T, Hq, Hkv, D, 1, seed=T)
    a = rnl.rnl_qkv_rope_axes(y, Hq, Hkv, D, gam[0], gam[1], pos, [0] * (D // 2), table)
    b = rnl.rnl_qkv_rope(y, Hq, Hkv, D, gam[0], gam[1], pos[0].contiguous(), table)
    assert all(torch.equal(x, z) for x, z in zip(a, b))


def test_bad_positions_leave_their_token_unwritten():
    Hq, Hkv, D, T = 4, 2, 128, 6
    y, pos, gam, table = make(T, Hq, Hkv, D, 3)
    pos[1, 2], pos[2, 4] = 300, -1
    m = layouts(D, 3)["sections"]
    q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    rnl.rnl_qkv_rope_axes(y, Hq, Hkv, D, gam[0], gam[1], pos, m, table, q_out=q, k_out=k)
    with pytest.raises(rnl.RnlError, match="RNL_ERR_ARG"):
        rnl.rnl_check_device_error()
    for t in range(T):
        assert bool((q[t] == 7).all()) == (t in (2, 4)) and bool((k[t] == 7).all()) == (t in (2, 4))
    # an axis that no pair uses is not read
    rnl.rnl_qkv_rope_axes(y, Hq, Hkv, D, None, None, pos, [0] * (D // 2), table)
    rnl.rnl_check_device_error()


def test_no_tokens():
    y, pos, gam, table = make(1, 4, 2, 64, 2)
    q, k, v = rnl.rnl_qkv_rope_axes(y[:0], 4, 2, 64, None, None, pos[:, :0].contiguous(), [0, 1] * 16, table)
    assert q.shape == (0, 4, 64) and v.shape == (0, 2, 64)
