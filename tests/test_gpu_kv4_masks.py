"""Attention over the 4-bit cache (rnl_kv4_attention): what the mask leaves out.
Pages in front of a window may have been freed, and tokens that a row does not
read, of whatever size, leave it alone."""
import math

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


def reference(q, c, t, lens, cu, window):
    """(out, lse, their bounds) in 64 bits.  The bounds are kv4_plain's (2^-8 of the
    output, 2^-11 + 2^-18 + 2 delta of sum p |v| / l, 2^-36 of the largest value),
    with delta and the largest value over the tokens that the row reads."""
    o, z, _, _ = plain.attention(q, c, t, i32(lens), i32(cu), window=window)
    tol, ltol = torch.full_like(o, math.nan), torch.full_like(z, math.nan)
    T, Hq, D = q.shape
    G, scale = Hq // c.n_kv_heads, D ** -0.5
    for b, n in enumerate(lens):
        r = cu[b + 1] - cu[b]
        rows = slice(cu[b], cu[b + 1])
        pos = torch.arange(n - r, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        see = (j <= pos) & ((j > pos - window) if window else True)
        for h in range(Hq):
            k, v = plain.sequence(c, t[b], n, h // G)
            k, v = k.nan_to_num(0, 0, 0), v.nan_to_num(0, 0, 0)  # (rows that read those are looked at apart)
            qd = q[rows, h].double()
            p = torch.softmax((qd @ k.t() * scale).masked_fill(~see, -math.inf), -1)
            delta = (D * 2.0 ** -23 * scale * (qd.abs() @ k.abs().t())).masked_fill(~see, 0).amax(-1, keepdim=True)
            top = torch.where(see, v.abs().amax(-1)[None], 0.0).amax(-1, keepdim=True)
            tol[rows, h] = (2.0 ** -8 * o[rows, h].abs() + (2.0 ** -11 + 2.0 ** -18 + 2 * delta) * (p @ v.abs()) +
                            2.0 ** -36 * top)
            ltol[rows, h] = delta[:, 0] + 2.0 ** -20 * z[rows, h].abs().clamp_min(1)
    return o, z, tol, ltol


def check(q, c, t, lens, cu, window, ref, skip=None):
    o, z, tol, ltol = ref
    for tt in (t, wide(t, c.page_size)):  # both kernels where there are many rows
        out, lse = torch.full_like(q, 320.0), torch.full(q.shape[:2], 123.0, device="cuda")
        rnl.rnl_kv4_attention(q, c, tt, i32(lens), i32(cu), out=out, lse_out=lse, window=window)
        rnl.rnl_check_device_error()
        ok = ((out.double() - o).abs() <= tol).all(-1) & ((lse.double() - z).abs() <= ltol)
        if skip is not None:
            assert out[skip].isnan().all() and lse[skip].isnan().all()
            ok = ok | skip
        assert ok.all(), f"{int((~ok).sum())} of {ok.numel()} rows, first {(~ok).nonzero()[0].tolist()}"


def louder(c, t, head, side, tok, up):
    """That token's keys or values times 2^up."""
    getattr(c, side + "_scales")[int(t[0, tok // c.page_size]), head, tok % c.page_size] += up


@pytest.mark.parametrize("D,block", [(64, 32), (128, 32), (128, 64), (256, 64)])
@pytest.mark.parametrize("rows,G", [(2, 1), (3, 4), (4, 4), (8, 2), (60, 1), (130, 2), (300, 1), (140, 8)])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("up", [60, 120])
def test_large_tokens_reach_only_the_rows_that_read_them(D, block, rows, G, window, up):
    """Keys and values 2^60 and 2^120 times the others, among the rows' own tokens
    and at the front of a window: a row that does not read one gets what it would
    get without it, to the bound of its own tokens."""
    g = gen(D + rows + window + up)
    n, H = 450, 2
    lens, cu = [n, 333], [0, rows, rows + 2]
    c, t = filled(g, lens, H, 32, D, block)
    marks = [(0, "k", n - 1), (0, "v", n - max(1, rows // 2)), (1, "v", n - 1)]
    if window:
        marks += [(0, "k", n - rows - window + 1), (1, "v", n - rows - window + 1), (1, "k", n - rows - window)]
    for h, side, tok in marks:
        louder(c, t, h, side, tok, up)
    q = randn(g, rows + 2, G * H, D).bfloat16()
    check(q, c, t, lens, cu, window, reference(q, c, t, lens, cu, window))


@pytest.mark.parametrize("D,rows,G,n", [(128, 4, 4, 9000), (64, 7, 1, 5000), (256, 30, 2, 3000), (128, 400, 4, 5000),
                                        (64, 90, 8, 7000)])
@pytest.mark.parametrize("window", [0, 1500])
@pytest.mark.parametrize("side", ["k", "v"])
def test_large_tokens_of_items_that_are_cut(D, rows, G, n, window, side):
    """One long sequence whose items several CTAs share: only some of the pieces
    hold a tile with such a token, and the pieces still join."""
    g = gen(n + rows + window)
    c, t = filled(g, [n], 1, 64, D, 32)
    louder(c, t, 0, side, n - 1, 80)
    louder(c, t, 0, side, n - rows - (window or rows) + 1, 50)
    q = randn(g, rows, G, D).bfloat16()
    check(q, c, t, [n], [0, rows], window, reference(q, c, t, [n], [0, rows], window))


@pytest.mark.parametrize("D,rows,G", [(64, 5, 2), (128, 5, 4), (256, 5, 1), (128, 200, 4), (64, 200, 1)])
def test_large_and_not_finite_tokens_together(D, rows, G):
    """A token that is far larger than the others and one that is not finite: rows
    that read the second get NaN, the others are right."""
    g = gen(D + rows)
    n = 400
    for side in ("k", "v"):
        c, t = filled(g, [n], 1, 16, D, 32)
        louder(c, t, 0, "k", n - 1, 70)
        louder(c, t, 0, "v", n - 2, 70)
        tok = n - 3
        bad = torch.zeros(rows, G, dtype=torch.bool, device="cuda")
        bad[rows - 3:] = True
        q = randn(g, rows, G, D).bfloat16()
        ref = reference(q, c, t, [n], [0, rows], 0)  # without the second
        getattr(c, side + "_scales")[int(t[0, tok // 16]), 0, tok % 16, 1] = 255
        check(q, c, t, [n], [0, rows], 0, ref, skip=bad)


@pytest.mark.parametrize("rows", [6, 150])
def test_small_early_values_under_large_later_ones(rows):
    """Values and keys that grow by 2^140 along the rows' own tokens: every row to
    the bound of what it reads."""
    g = gen(rows)
    n, D = 600, 128
    c, t = filled(g, [n], 1, 32, D, 32)
    for tok in range(n):
        up = 0 if tok < n - rows else 140 * (tok - (n - rows)) // rows
        for side in ("k", "v"):
            s = getattr(c, side + "_scales")
            at = (int(t[0, tok // 32]), 0, tok % 32)
            s[at] = (s[at].int() - 30 + up).clamp(1, 250).to(torch.uint8)
    q = (randn(g, rows, 4, D) * 2.0 ** -20).bfloat16()
    check(q, c, t, [n], [0, rows], 0, reference(q, c, t, [n], [0, rows], 0))


@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 4), (128, 2, 4), (128, 1, 16), (256, 1, 2)])
@pytest.mark.parametrize("rows", [1, 4, 150])
@pytest.mark.parametrize("scale", [1e5, -1e8, 1e14, 1e30])
def test_large_scores(D, Hkv, G, rows, scale):
    """Scores of 10^6 to 10^31: finite, and where one token's score is ahead of all
    others by more than the scores' own error (D 2^-23 scale sum |q k| each) and
    another 100, the output is that token's values and lse its score."""
    g = gen(D + rows)
    lens, cu = [700, 45], [0, rows, rows + 1]
    c, t = filled(g, lens, Hkv, 32, D, 32)
    q = randn(g, rows + 1, Hkv * G, D).bfloat16()
    for causal, tt in ((True, t), (False, t), (True, wide(t, 32)), (False, wide(t, 32))):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        rnl.rnl_kv4_attention(q, c, tt, i32(lens), i32(cu), scale=scale, causal=causal, out=out, lse_out=lse)
        rnl.rnl_check_device_error()
        assert out.isfinite().all() and lse.isfinite().all()
        clear = 0
        for b, n in enumerate(lens):
            r = cu[b + 1] - cu[b]
            pos = torch.arange(n - r, n, device="cuda")[:, None]
            see = (torch.arange(n, device="cuda")[None] <= pos) if causal else torch.ones(r, n, dtype=torch.bool, device="cuda")
            for h in range(Hkv * G):
                k, v = plain.sequence(c, t[b], n, h // G)
                qd = q[cu[b]:cu[b + 1], h].double()
                s = (qd @ k.t() * scale).masked_fill(~see, -math.inf)
                delta = (D * 2.0 ** -23 * abs(scale) * (qd.abs() @ k.abs().t())).amax(-1)
                top = s.topk(2, -1)
                ok = top.values[:, 0] - top.values[:, 1] > 2 * delta + 100
                clear += int(ok.sum())
                want = v[top.indices[:, 0]]
                assert ((out[cu[b]:cu[b + 1], h].double() - want).abs() <= 2.0 ** -8 * want.abs())[ok].all()
                off = (lse[cu[b]:cu[b + 1], h].double() - top.values[:, 0]).abs()
                assert (off <= delta + 2.0 ** -20 * top.values[:, 0].abs())[ok].all()
        assert clear > (rows + 1) * Hkv * G // 2


@pytest.mark.parametrize("rows,n", [(1, 300), (1, 9000), (4, 9000), (200, 3000)])
@pytest.mark.parametrize("scale", [1.0, 1e12, -1e25])
def test_equal_scores_of_any_size(rows, n, scale):
    """Equal keys: every token the same weight, the mean of the values, whatever the
    score is (the same sum for every token, in the same order)."""
    g = gen(rows + n)
    D = 128
    c, t = filled(g, [n], 1, 64, D, 32)
    for x in (c.k_codes, c.k_scales):
        x[:] = x[0, 0, 0].clone()
    c.k_scales.clamp_(100, 130)
    q = randn(g, rows, 4, D).bfloat16()
    v = plain.sequence(c, t[0], n, 0)[1]
    for tt in (t, wide(t, 64)):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        rnl.rnl_kv4_attention(q, c, tt, i32([n]), i32([0, rows]), scale=scale, causal=False, out=out, lse_out=lse)
        rnl.rnl_check_device_error()
        want, size = v.mean(0), v.abs().mean(0)
        # 2^-8 for the output, 2^-11 of sum p |v| for the weights, 2^-18 for the sums
        assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -18) * size).all()
        assert lse.isfinite().all()


@pytest.mark.parametrize("rows,G,D,copies", [(3, 2, 64, 800), (2, 4, 128, 800), (40, 1, 64, 300), (36, 2, 128, 300)])
def test_large_tokens_in_many_short_sequences(rows, G, D, copies):
    """A large token in every sequence of a batch, so that a CTA has more such items
    than it keeps apart (31): some twenty sequences, each many times over."""
    g = gen(rows + D)
    B = 23
    lens = [rows + (b * 7) % 40 for b in range(B)]
    c, t = filled(g, lens, 1, 16, D, 32)
    for side, up in (("k", 60), ("v", 90)):
        s = getattr(c, side + "_scales")
        last = torch.tensor([n - 1 - (side == "v") for n in lens], device="cuda")
        s[t[torch.arange(B, device="cuda"), last // 16].long(), :, last % 16] += up
    cu = [rows * b for b in range(B + 1)]
    q = randn(g, rows * B, G, D).bfloat16()
    o, z, tol, ltol = reference(q, c, t, lens, cu, 0)
    many = q.repeat(copies, 1, 1)
    out, lse = torch.empty_like(many), torch.empty(many.shape[:2], device="cuda")
    rnl.rnl_kv4_attention(many, c, t.repeat(copies, 1), i32(lens).repeat(copies),
                          i32([rows * b for b in range(B * copies + 1)]), out=out, lse_out=lse)
    rnl.rnl_check_device_error()
    assert ((out.view(copies, *q.shape).double() - o).abs() <= tol).all()
    assert ((lse.view(copies, *z.shape).double() - z).abs() <= ltol).all()


@pytest.mark.parametrize("D,rows,G", [(64, 1, 4), (128, 4, 4), (256, 3, 2), (128, 150, 2), (64, 300, 1)])
def test_queries_that_are_not_numbers_stay_to_themselves(D, rows, G):
    g = gen(D + rows)
    n = 500
    c, t = filled(g, [n, 77], 2, 32, D, 32)
    lens, cu = [n, 77], [0, rows, rows + 1]
    q = randn(g, rows + 1, 2 * G, D).bfloat16()
    ref = reference(q, c, t, lens, cu, 0)
    bad = torch.zeros(rows + 1, 2 * G, dtype=torch.bool, device="cuda")
    bad[rows // 2, 1] = bad[0, 0] = True
    q[rows // 2, 1, 5] = math.nan
    q[0, 0] = math.nan
    check(q, c, t, lens, cu, 0, ref, skip=bad)
