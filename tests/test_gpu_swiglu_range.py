"""SwiGLU of the grouped products over the whole range of its gates, on the GPU:
sums that are exact (one product each), gates from -190 to 100 and ups from bf16's
smallest to its largest values, so that silu(g) u is a bf16 value though silu(g)
alone is below FP32's smallest; gates and ups that are infinite or NaN.

Tolerance, relative to |silu(g) u|: one rounding to bf16, 2^-8; an exponential of g
in FP32, its argument rounded twice, the function good to 2 units of 2^-23, as
exp(g / 4) four times: 8 + 1.2 |g| units with FP32's own exponential; the reciprocal
and six products, 1 unit each: 2^-8 + (16 + 1.2 |g|) 2^-23, times 1 + 2^-8 for the
product of the two.  Below bf16's normal range half its smallest step, 2^-134, and
FP32's, 2^-150, for the products there."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

rnl = pytest.importorskip("rmsnorm_linear_projection_gb300")
MAX = torch.finfo(torch.bfloat16).max


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rmsnorm_linear_projection_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    yield
    rnl.rnl_check_device_error()


def check(out, g, u):
    g, u = g.double(), u.double()
    # g / (1 + exp(-g)) without an overflow in front of the product
    ref = torch.where(g < 0, g * torch.exp(g / 2) * (torch.exp(g / 2) * u) / (1 + torch.exp(g)), g * u / (1 + torch.exp(-g)))
    assert not (ref[(g > -185) & (g != 0) & (u.abs() >= 2.0 ** 126)] == 0).any()
    bound = ref.abs() * (2.0 ** -8 + (16 + 1.2 * g.abs()) * 2.0 ** -23) * (1 + 2.0 ** -8) + 2.0 ** -134 + 2.0 ** -149
    got = out.double()
    big = ref.abs() > MAX * (1 - 2.0 ** -8)  # rounds to the largest value or to infinity
    assert ((got[big].abs() >= MAX * (1 - 2.0 ** -7)) & (got[big].sign() == ref[big].sign())).all()
    far = ((got - ref).abs() > bound) & ~big
    i = far.nonzero()[:4]
    assert not far.any(), [(g[tuple(j)].item(), u[tuple(j)].item(), ref[tuple(j)].item(), got[tuple(j)].item()) for j in i]


GATES = [-v for v in (190, 184, 180, 176, 160, 140, 120, 104, 103, 100, 96, 92, 90, 89, 88.5, 88, 87.5, 87, 86, 80, 64, 40,
                      20, 10, 5, 2, 1, 0.5, 0.01, 1e-6, 1e-30)] + [0.0, 1e-30, 0.01, 0.5, 1, 2, 5, 10, 20, 40, 87, 88, 89, 100]
UPS = [1.0, -3.0, 1e5, -1e20, 1e30, 3e38, -3e38, 1e-5, -1e-20, 1e-30, 1e-38, 1e-40]


@pytest.mark.parametrize("gather", [False, True])
def test_bf16(gather):
    """Features: the gates (rows of the weight); rows of x: the ups, an expert each with its sign."""
    F = 64
    g = torch.tensor(GATES + [-v * 0.37 for v in range(F - len(GATES))]).bfloat16()
    u = torch.tensor(UPS).bfloat16()
    R = len(UPS)
    x = torch.zeros(R, 64, dtype=torch.bfloat16)
    x[:, 0] = 1
    x[:, 1] = u
    w = torch.zeros(1, 2 * F, 64, dtype=torch.bfloat16)
    w[0, :F, 0] = g
    w[0, F:, 1] = 1
    rows = torch.arange(R, dtype=torch.int32, device="cuda").flip(0) if gather else None
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    out = rnl.rnl_grouped_linear_bf16(x.cuda(), w.cuda(), off, rows=rows, swiglu=True)
    rnl.rnl_check_device_error()
    out = out.cpu()
    if gather:
        out = out.flip(0)
    check(out, g[None].expand(R, F), u[:, None].expand(R, F))


@pytest.mark.parametrize("block", [32, 64])
def test_mxfp8(block):
    F = 64
    # E4M3 values times 2^6: -64 .. -112, and their halves, with either sign
    codes = torch.tensor([0xB8 + i for i in range(8)] + [0xB0 + i for i in range(8)] + [0x38 + i for i in range(4)] + [0x30, 0x28, 0x20, 0])
    codes = codes.repeat(3)[:F].to(torch.uint8)
    g = codes.view(torch.float8_e4m3fn).double() * 64
    x = torch.zeros(40, 2 * block, dtype=torch.uint8)
    x[:, 0] = 0x38             # 1
    x[:, block] = 0x38         # 1, with a scale of its own
    xs = torch.full((40, 2), 127, dtype=torch.uint8)
    xs[:, 1] = torch.arange(40) * 6 + 10   # ups 2^-117 .. 2^117
    w = torch.zeros(1, 2 * F, 2 * block, dtype=torch.uint8)
    w[0, :F, 0] = codes
    w[0, F:, block] = 0x38
    ws = torch.full((1, 2 * F, 2), 127, dtype=torch.uint8)
    ws[0, :F, 0] = 127 + 6
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    out = rnl.rnl_grouped_linear_mxfp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), off, swiglu=True, block=block)
    rnl.rnl_check_device_error()
    u = torch.exp2(xs[:, 1].double() - 127)
    check(out.cpu(), g[None].expand(40, F), u[:, None].expand(40, F))


def test_infinite_and_nan_gates_and_ups():
    """silu(g) u by its factors: silu(inf) = inf, silu(-inf) = -inf * 0 = NaN."""
    inf, nan = math.inf, math.nan
    pairs = [(inf, 2.0, inf), (inf, -2.0, -inf), (inf, 0.0, nan), (-inf, 1.0, nan), (nan, 1.0, nan), (1.0, nan, nan),
             (1.0, inf, inf), (-1.0, inf, -inf), (-100.0, inf, -inf), (0.0, inf, nan), (-2.0, -inf, inf), (inf, inf, inf)]
    F = 16
    w = torch.zeros(1, 2 * F, 64, dtype=torch.bfloat16)
    for i, (g, u, _) in enumerate(pairs):
        w[0, i, 0], w[0, F + i, 0] = g, u
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    x[:, 0] = 1
    out = rnl.rnl_grouped_linear_bf16(x.cuda(), w.cuda(), torch.tensor([0, 3], dtype=torch.int32, device="cuda"), swiglu=True)
    rnl.rnl_check_device_error()
    want = torch.tensor([p[2] for p in pairs], dtype=torch.float64)
    for row in out.cpu().double()[:, :len(pairs)]:
        assert torch.equal(torch.nan_to_num(row, nan=7.0), torch.nan_to_num(want, nan=7.0)), row.tolist()
    assert (out[:, len(pairs):] == 0).all()


def test_rows_with_such_gates_leave_the_others_alone():
    """A row's bits do not depend on the gates of the rows beside it."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(200, 256, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(1, 192, 256, generator=gen, device="cuda") / 8).bfloat16()
    off = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    want = rnl.rnl_grouped_linear_bf16(x, w, off, swiglu=True)
    far = x.clone()
    far[7::16] *= 200
    got = rnl.rnl_grouped_linear_bf16(far, w, off, swiglu=True)
    rnl.rnl_check_device_error()
    same = torch.ones(200, dtype=torch.bool, device="cuda")
    same[7::16] = False
    assert torch.equal(got[same], want[same]) and not torch.equal(got, want)
