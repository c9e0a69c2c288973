"""The 4-bit paged KV cache (rnl_kv4_append, rnl_kv4_gather) and attention over
it (rnl_kv4_attention) on the GPU against plain 64-bit implementations
(kv4_plain.py, which also derives the tolerances).  Codes, scales and what is
read back are exact; attention is held to the derived bound."""
import math

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def garbage_cache(g, pages, H, page, D, block):
    """Every byte random (scale bytes too, 255 among them): what a recycled page holds."""
    c = rnl.Kv4Cache.empty(pages, H, page, D, block)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda").to(torch.uint8))
    return c


def tables(g, lens, page, extra=2):
    """Pages of all sequences in random order; unused table entries are out of range."""
    need = [-(-n // page) for n in lens]
    P = sum(need) + extra
    perm = torch.randperm(P, generator=g, device="cuda").int()
    t = torch.full((len(lens), max(need + [1])), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, P


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def filled(g, lens, H, page, D, block, spread=0.0, chan=0.5):
    """A cache that holds random keys and values of the given lengths, garbage elsewhere."""
    t, P = tables(g, lens, page)
    c = garbage_cache(g, P, H, page, D, block)
    T = sum(lens)
    if T:
        k = randn(g, T, H, D) * torch.exp(chan * randn(g, H, D))
        v = randn(g, T, H, D)
        if spread:  # tokens of very different magnitude
            k, v = k * torch.exp(0.3 * randn(g, T, 1, 1)), v * torch.exp2(spread * randn(g, T, 1, 1))
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        rnl.rnl_kv4_append(k.bfloat16(), v.bfloat16(), c, t, i32(lens), i32(cu))
    return c, t


def wide(t, page):
    """The tables with room for 2^19 tokens more: with many rows the call then expects
    enough work for the prompt kernel, which small tables keep from it."""
    more = torch.full((t.shape[0], 2 ** 19 // page), -9, dtype=torch.int32, device="cuda")
    return torch.cat([t, more], 1)


def check_attention(q, c, t, lens, cu=None, **kw):
    """Both kernels where many rows allow both; the narrow tables' outputs."""
    ref = plain.attention(q, c, t, i32(lens), None if cu is None else i32(cu), **kw)
    many = cu is not None and q.shape[0] * q.shape[1] // c.n_kv_heads > 32 and c.head_dim < 256
    if many:
        check_outputs(ref, q, c, wide(t, c.page_size), lens, cu, **kw)
    return check_outputs(ref, q, c, t, lens, cu, **kw)


def check_outputs(ref, q, c, t, lens, cu, **kw):
    T, Hq, D = q.shape
    lse = torch.full((T, Hq), 123.0, device="cuda")
    out = torch.full((T, Hq, D), 320.0, dtype=torch.bfloat16, device="cuda")
    rnl.rnl_kv4_attention(q, c, t, i32(lens), None if cu is None else i32(cu), out=out, lse_out=lse, **kw)
    rnl.rnl_check_device_error()
    o, z, tol, ltol = ref
    own = ~torch.isnan(z)
    assert (out[~own] == 320.0).all() and (lse[~own] == 123.0).all(), "rows of no sequence were written"
    off = (out.double() - o).abs()[own]
    bad = ~(off <= tol[own])
    worst = float((off / tol[own].clamp_min(1e-300)).nan_to_num(1e9).max()) if off.numel() else 0.0
    where = (~((out.double() - o).abs() <= tol) & own[..., None]).nonzero()[:4].tolist()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs out of bound, worst {worst:.3g} of it, at {where}"
    empty = z == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    full = own & ~empty
    zoff = (lse.double() - z).abs()[full]
    assert (zoff <= ltol[full]).all(), f"lse off by {float(zoff.max()):.3g}"
    return out, lse


# ------------------------------------------------------------------- cache
SPECIAL = [0.0, -0.0, 0.25, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 6.0, 7.0, -7.96875, 0.26, 0.24, 1e-3, 4.99, 1.0, -1.5]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("block", [32, 64])
@pytest.mark.parametrize("page,H", [(16, 3), (64, 8), (1024, 1)])
def test_append_and_gather_are_exact(D, block, page, H):
    g = gen(D + block + page)
    lens, rows = [1, 40, 0, 17, 130], [1, 33, 0, 17, 2]
    t, P = tables(g, lens, page)
    c = garbage_cache(g, P, H, page, D, block)
    before = [x.clone() for x in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    T, pad = sum(rows), 3
    # k and v as column ranges of one wider tensor, rows apart
    wide = randn(g, T + pad, 3 * H * D) * torch.exp2(20 * randn(g, T + pad, 1)).clamp(1e-30, 1e30)
    wide = wide.bfloat16()
    k, v = wide[:, H * D:2 * H * D].view(T + pad, H, D), wide[:, 2 * H * D:].view(T + pad, H, D)
    k[0, 0, :len(SPECIAL)] = torch.tensor(SPECIAL, dtype=torch.bfloat16)       # every tie and the saturated range
    k[0, 0, len(SPECIAL):] = 0
    k[1, 0] = 0                                                                # all-zero blocks
    v[1, 0] = 1e-39                                                            # subnormal bf16
    v[2, 0, 3] = 3.38e38                                                       # the top of the range
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    rnl.rnl_kv4_append(k, v, c, t, i32(lens), i32(cu))
    rnl.rnl_check_device_error()
    want = [x.clone() for x in before]
    for b, (n, r) in enumerate(zip(lens, rows)):
        for i in range(r):
            pos = n - r + i
            p, o = int(t[b, pos // page]), pos % page
            for x, cc, ss in ((k, 0, 1), (v, 2, 3)):
                want[cc][p, :, o], want[ss][p, :, o] = plain.quantise(x[cu[b] + i], block)
    for got, w in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), want):
        differ = got != w
        assert not differ.any(), differ.nonzero()[:5].tolist()  # the other tokens of every page too
    ko = torch.full((T + pad, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    rnl.rnl_kv4_gather(c, t, i32(lens), T + pad, i32(cu), k_out=ko, v_out=vo)
    rnl.rnl_check_device_error()
    assert (ko[T:] == 9).all() and (vo[T:] == 9).all()
    for b, (n, r) in enumerate(zip(lens, rows)):
        for h in range(H):
            kk, vv = plain.sequence(c, t[b], n, h)
            assert torch.equal(ko[cu[b]:cu[b + 1], h].double(), kk[n - r:])
            assert torch.equal(vo[cu[b]:cu[b + 1], h].double(), vv[n - r:])


def test_gather_reads_every_code_and_scale():
    c = rnl.Kv4Cache.empty(16, 1, 16, 64, 32)
    codes = torch.arange(256, device="cuda").to(torch.uint8)
    c.k_codes.copy_(codes.view(8, 32).repeat(32, 1).view(16, 1, 16, 32))
    c.v_codes.copy_(codes.flip(0).view(8, 32).repeat(32, 1).view(16, 1, 16, 32))
    s = torch.arange(512, device="cuda").remainder(256).to(torch.uint8).view(16, 1, 16, 2)
    c.k_scales.copy_(s)
    c.v_scales.copy_(s)
    t = torch.arange(16, device="cuda").int().view(1, 16)
    k, v = rnl.rnl_kv4_gather(c, t, i32([256]), 256, i32([0, 256]))
    for got, cc in ((k, c.k_codes), (v, c.v_codes)):
        want = plain.values(cc.view(256, 32), s.view(256, 2)).view(256, 1, 64).bfloat16()
        ok = (got == want) | (got.isnan() & want.isnan())
        assert ok.all()


def test_append_marks_blocks_that_are_not_finite():
    c = rnl.Kv4Cache.empty(1, 1, 16, 128, 32)
    k = torch.ones(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    q = k.clone()
    k[0, 0, 5], k[0, 0, 70] = math.inf, math.nan
    rnl.rnl_kv4_append(k, k, c, i32([[0]]), i32([1]))
    assert c.k_scales[0, 0, 0].tolist() == [255, 125, 255, 125]
    out = rnl.rnl_kv4_attention(q, c, i32([[0]]), i32([1]))
    assert not torch.isfinite(out).all()


def test_bad_sequences_are_reported_and_left_alone():
    g = gen(5)
    H, D, page = 2, 64, 16
    c = garbage_cache(g, 4, H, page, D, 32)
    before = [x.clone() for x in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    k = randn(g, 2, H, D).bfloat16()
    q = randn(g, 2, 2 * H, D).bfloat16()
    cases = [
        (i32([[4, 0], [9, 0]]), i32([3, 5]), None),       # page ids outside the cache
        (i32([[-1, 0], [-3, 0]]), i32([3, 5]), None),
        (i32([[0, 1], [2, 3]]), i32([33, -1]), None),      # lengths out of range
        (i32([[0, 1], [2, 3]]), i32([5, 5]), i32([0, 3, 2])),   # decreasing
        (i32([[0, 1], [2, 3]]), i32([5, 5]), i32([-1, 1, 9])),  # beyond the rows
        (i32([[0, 1], [2, 3]]), i32([0, 1]), i32([0, 1, 1])),   # a row without a position
    ]
    for n, (t, lens, cu) in enumerate(cases):
        ko = torch.full((2, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
        vo = ko.clone()
        calls = [lambda: rnl.rnl_kv4_append(k, k, c, t, lens, cu),
                 lambda: rnl.rnl_kv4_gather(c, t, lens, 2, cu, k_out=ko, v_out=vo)]
        if n < 5:
            calls.append(lambda: rnl.rnl_kv4_attention(q, c, t, lens, cu))
        for call in calls:
            call()
            with pytest.raises(rnl.RnlError, match="RNL_ERR_ARG"):
                rnl.rnl_check_device_error()
        assert (ko == 9).all() and (vo == 9).all()
        rnl.rnl_check_device_error()
    for x, y in zip(before, (c.k_codes, c.k_scales, c.v_codes, c.v_scales)):
        assert torch.equal(x, y)


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (64, 8, 1), (128, 8, 2), (128, 5, 1), (128, 32, 1), (256, 4, 2),
                                      (256, 16, 1)])
@pytest.mark.parametrize("block,page", [(32, 16), (64, 64), (32, 256)])
def test_single_tokens(D, Hq, Hkv, block, page):
    g = gen(D + Hq + page)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 0, 127, 129, 1000, 2049]
    c, t = filled(g, lens, Hkv, page, D, block)
    q = randn(g, len(lens), Hq, D).bfloat16()
    check_attention(q, c, t, lens)
    check_attention(q, c, t, lens, window=50)
    check_attention(q, c, t, lens, causal=False)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 2), (64, 8, 2), (128, 8, 2), (128, 3, 1), (128, 16, 1), (256, 4, 2)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (False, 0)])
def test_rows_of_ragged_sequences(D, Hq, Hkv, causal, window):
    g = gen(D + Hq + window)
    lens = [5, 70, 33, 0, 200, 131, 300, 1]
    rows = [5, 1, 33, 0, 7, 130, 129, 0]
    c, t = filled(g, lens, Hkv, 32, D, 32)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    pad = 4
    q = randn(g, sum(rows) + pad, Hq, D).bfloat16()
    check_attention(q, c, t, lens, cu, causal=causal, window=window)


@pytest.mark.parametrize("rows,n", [(1, 5000), (3, 700), (9, 4097), (128, 128), (257, 1025), (640, 3000)])
def test_lengths(rows, n):
    g = gen(rows)
    c, t = filled(g, [n, n // 2 + rows], 2, 64, 128, 64)
    q = randn(g, 2 * rows, 8, 128).bfloat16()
    check_attention(q, c, t, [n, n // 2 + rows], [0, rows, 2 * rows])


def test_rows_without_a_token():
    """Lengths of zero, causal rows before the first token, in single-token and
    in wide tiles."""
    g = gen(11)
    c, t = filled(g, [3, 0, 40, 100], 2, 16, 128, 32)
    q = randn(g, 1 + 4 + 60 + 300, 8, 128).bfloat16()
    check_attention(q, c, t, [3, 0, 40, 100], [0, 1, 5, 65, 365])
    check_attention(q, c, t, [3, 0, 40, 100], [0, 1, 5, 65, 365], causal=False)


@pytest.mark.parametrize("rows", [1, 6, 200])
def test_magnitudes(rows):
    """Values that differ by many powers of two between tokens, large and tiny
    keys and queries, one overwhelming score, and scores that are all equal."""
    g = gen(rows)
    n = 500
    c, t = filled(g, [n], 2, 16, 128, 32, spread=6.0)
    q = randn(g, rows, 8, 128)
    for f in (1.0, 1e-20, 1e3, 0.0):
        check_attention((q * f).bfloat16(), c, t, [n], [0, rows], causal=False)
    k = (randn(g, n, 2, 128) * 1e4).bfloat16()
    v = (randn(g, n, 2, 128) * 1e-6).bfloat16()
    v[7] = 1e6                     # a value far above the others, under a mask or a vanishing weight
    rnl.rnl_kv4_append(k, v, c, t, i32([n]), i32([0, n]))
    check_attention((q * 1e-4).bfloat16(), c, t, [n], [0, rows], causal=False)
    check_attention((q * 1e-4).bfloat16(), c, t, [n], [0, rows], window=100)
    check_attention(q.bfloat16(), c, t, [n], [0, rows], causal=False, scale=-0.001)


def test_sink_token():
    """Almost all weight on one token whose values are nearly nothing: what is
    left of the others decides the output."""
    g = gen(3)
    n, H, D = 900, 2, 128
    for rows in (1, 160):
        c, t = filled(g, [n], H, 64, D, 32)
        k, v = randn(g, 1, H, D), randn(g, 1, H, D) * 2.0 ** -20
        q = randn(g, rows, 8, D)
        k[0] = 0
        k[0, :, 0] = 30
        q[..., 0] = 4.6             # the sink's score is about 12 above the rest
        rnl.rnl_kv4_append(k.bfloat16(), v.bfloat16(), c, t, i32([1]), None)
        check_attention(q.bfloat16(), c, t, [n], [0, rows], causal=False)


def test_strided_queries_and_shared_pages():
    g = gen(21)
    Hq, Hkv, D = 8, 2, 128
    c, t = filled(g, [300], Hkv, 16, D, 32)
    t = t.repeat(3, 1)              # three sequences over one prefix
    lens = [300, 299, 17]
    wide = randn(g, 3, (Hq + 2 * Hkv) * D).bfloat16()
    check_attention(wide[:, :Hq * D].view(3, Hq, D), c, t, lens)


def test_offsets_beyond_32_bits():
    """Pages whose byte offsets pass 2^32."""
    g = gen(8)
    H, page, D = 8, 1024, 128
    P = 9000                        # 9000 * 8 * 1024 rows * 64 bytes = 4.7 GB each
    c = rnl.Kv4Cache.empty(P, H, page, D, 32)
    lens = [1500, 40]
    t = i32([[P - 1, P - 3], [P - 2, 0]])
    k, v = randn(g, 1540, H, D).bfloat16(), randn(g, 1540, H, D).bfloat16()
    rnl.rnl_kv4_append(k, v, c, t, i32(lens), i32([0, 1500, 1540]))
    ko, vo = rnl.rnl_kv4_gather(c, t, i32(lens), 1540, i32([0, 1500, 1540]))
    for x, o in ((k, ko), (v, vo)):
        cc, ss = plain.quantise(x, 32)
        assert torch.equal(o.double(), plain.values(cc, ss))
    check_attention(randn(g, 2, 32, D).bfloat16(), c, t, lens)
    check_attention(randn(g, 202, 32, D).bfloat16(), c, t, lens, [0, 200, 202])


def test_many_sequences():
    """More sequences than a CTA has threads, most of them short."""
    g = gen(77)
    lens = [2 + (i * 37) % 90 for i in range(1500)]
    c, t = filled(g, lens, 1, 16, 64, 32)
    q = randn(g, len(lens), 4, 64).bfloat16()
    check_attention(q, c, t, lens)
    rows = [(i * 7) % 3 for i in range(1500)]
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    check_attention(randn(g, cu[-1] + 2, 4, 64).bfloat16(), c, t, lens, cu)


def test_captured_call_follows_its_inputs():
    """One captured step: append, then attention, replayed while lengths, tables
    and tokens change in the same buffers; the same bits as eager calls.  The
    workspace is shared with a second captured graph."""
    g = gen(13)
    B, Hq, Hkv, D, page = 4, 8, 2, 128, 16
    full = [900, 33, 500, 64]
    c, t = filled(g, full, Hkv, page, D, 32)
    ws = torch.randint(0, 256, (rnl.workspace_size(rnl.OP_KV4_ATTENTION, B, D, Hq, Hkv) + 16,), device="cuda").to(torch.uint8)
    q, k, v = (randn(g, B, h, D).bfloat16() for h in (Hq, Hkv, Hkv))
    lens = i32([1, 1, 1, 1])
    out, out2 = torch.empty_like(q), torch.empty_like(q)

    def step(o, causal):
        rnl.rnl_kv4_append(k, v, c, t, lens)
        rnl.rnl_kv4_attention(q, c, t, lens, out=o, workspace=ws, causal=causal)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        step(out, True)
        side.synchronize()
        for o in (out, out2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                step(o, o is out)
            graphs.append(gr)
    torch.cuda.synchronize()
    for i, now in enumerate(([5, 33, 1, 64], [900, 2, 17, 1], [64, 16, 500, 3])):
        lens.copy_(i32(now))
        for x in (q, k, v):
            x.copy_(randn(gen(100 + i), *x.shape).bfloat16())
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        rnl.rnl_check_device_error()
        for o in (out, out2):
            want = rnl.rnl_kv4_attention(q, c, t, lens, causal=o is out)
            assert torch.equal(o, want)
        check_attention(q, c, t, now)


def test_repeated_calls_give_the_same_bits():
    g = gen(31)
    lens = [4000, 700, 2500]
    c, t = filled(g, lens, 4, 64, 128, 32)
    cu = [0, 1, 301, 321]
    q = randn(g, 321, 16, 128).bfloat16()
    first = rnl.rnl_kv4_attention(q, c, t, i32(lens), i32(cu))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):  # two streams at once, a workspace each
        with torch.cuda.stream(streams[i % 2]):
            outs.append(rnl.rnl_kv4_attention(q, c, t, i32(lens), i32(cu)))
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


def test_a_sequence_alone_or_in_a_batch():
    """Single-token, draft and prompt sequences in one call, and each on its own."""
    g = gen(41)
    lens, rows = [600, 3000, 90], [1, 200, 12]
    c, t = filled(g, lens, 2, 32, 128, 32)
    cu = [0, 1, 201, 213]
    q = randn(g, 213, 8, 128).bfloat16()
    check_attention(q, c, t, lens, cu)
    for b in range(3):
        check_attention(q[cu[b]:cu[b + 1]].contiguous(), c, t[b:b + 1].contiguous(), [lens[b]], [0, rows[b]])


# ------------------------------------------------------ the run as it is used
def test_prompt_then_steps_through_the_projection():
    """RMSNorm + projection, multi-axis RoPE, cache, attention: a prompt of two
    sequences, then single tokens; each attention call against the plain form on
    the same q and cache, and the cache against the plain quantiser."""
    g = gen(55)
    K, Hq, Hkv, D, page = 512, 8, 2, 128, 16
    N = (Hq + 2 * Hkv) * D
    W = (randn(g, N, K) / math.sqrt(K)).bfloat16()
    gamma = (1 + 0.1 * randn(g, K)).bfloat16()
    qg, kg = ((1 + 0.1 * randn(g, D)).bfloat16() for _ in range(2))
    ang = torch.arange(512, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(D // 2, dtype=torch.float64, device="cuda") * 2 / D)
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    axes = [0] * 16 + [1] * 24 + [2] * 24
    lens, rows = [70, 150], [70, 150]
    t, P = tables(g, [n + 4 for n in lens], page)
    c = garbage_cache(g, P, Hkv, page, D, 32)
    for step in range(4):
        T = sum(rows)
        cu = [0, rows[0], T]
        x = randn(g, T, K).bfloat16()
        y = rnl.rmsnorm_linear_bf16(x, gamma, W)
        pos = torch.randint(0, 512, (3, T), generator=g, device="cuda").int()
        q, k, v = rnl.rnl_qkv_rope_axes(y, Hq, Hkv, D, qg, kg, pos, axes, table)
        rnl.rnl_kv4_append(k, v, c, t, i32(lens), i32(cu))
        kk, vv = rnl.rnl_kv4_gather(c, t, i32(lens), T, i32(cu))
        assert torch.equal(kk.double(), plain.values(*plain.quantise(k, 32)))
        assert torch.equal(vv.double(), plain.values(*plain.quantise(v, 32)))
        check_attention(q, c, t, lens, cu if step == 0 else None)
        rows = [1, 1]
        lens = [n + 1 for n in lens]


@pytest.mark.parametrize("D,block", [(64, 64), (64, 32), (128, 32), (128, 64), (256, 32), (256, 64)])
@pytest.mark.parametrize("rows,G", [(1, 4), (2, 4), (4, 4), (1, 1), (200, 2), (140, 8)])
@pytest.mark.parametrize("window", [0, 90])
def test_blocks_that_are_not_finite_reach_only_the_rows_that_read_them(D, block, rows, G, window):
    """Keys and values that are not finite, in front of a window, among the rows'
    own tokens (which earlier rows do not read) and in the history: a row that
    reads one gets NaN and lse NaN, all others what they would get without it."""
    g = gen(D + rows + window)
    n, H = 450, 2
    c, t = filled(g, [n, 70], H, 32, D, block)
    lens, cu = [n, 70], [0, rows, rows + 1]
    # (head, side, token); with a window also old tokens that no row, or only the first rows, read
    marks = [(0, "k", n - 1), (0, "v", n - max(1, rows // 2)), (1, "v", n - 1)]
    if window:
        marks += [(0, "k", n - rows - window - 1), (0, "v", n - rows - window + 1), (1, "k", n - rows - window)]
    elif rows == 200:
        marks += [(1, "k", n - 130)]
    clean = rnl.Kv4Cache(*(x.clone() for x in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)))
    pos = torch.arange(n - rows, n)
    bad = torch.zeros(rows + 1, H, dtype=torch.bool)
    for h, side, tok in marks:
        page, off = int(t[0, tok // 32]), tok % 32
        part = tok % (D // block)
        getattr(c, side + "_scales")[page, h, off, part] = 255
        getattr(clean, side + "_scales")[page, h, off, part] = 0
        bad[:rows, h] |= (pos >= tok) & ((pos - tok < window) if window else True)
    q = randn(g, rows + 1, G * H, D).bfloat16()
    o, z, tol, ltol = plain.attention(q, clean, t, i32(lens), i32(cu), window=window)
    bad = bad.repeat_interleave(G, 1).cuda()
    for tt in (t, wide(t, 32)):
        out, lse = torch.empty_like(q), torch.empty(rows + 1, G * H, device="cuda")
        rnl.rnl_kv4_attention(q, c, tt, i32(lens), i32(cu), out=out, lse_out=lse, window=window)
        rnl.rnl_check_device_error()
        assert out[bad].isnan().all() and lse[bad].isnan().all()
        assert ((out.double() - o).abs() <= tol)[~bad].all()
        assert ((lse.double() - z).abs() <= ltol)[~bad].all()


@pytest.mark.parametrize("rows", [1, 4, 150])
def test_a_window_longer_than_any_sequence(rows):
    g = gen(rows)
    c, t = filled(g, [333], 2, 16, 128, 32)
    t = wide(t, 16)
    q = randn(g, rows, 8, 128).bfloat16()
    want = rnl.rnl_kv4_attention(q, c, t, i32([333]), i32([0, rows]))
    for window in (333, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1):
        assert torch.equal(rnl.rnl_kv4_attention(q, c, t, i32([333]), i32([0, rows]), window=window), want)
    # rows in front of the first token read nothing, whatever the window
    out, _ = check_attention(q, c, t, [0], [0, rows], window=2 ** 31 - 1)
    assert (out == 0).all()


def test_calls_on_two_streams_at_once():
    """Steps on one stream, a prompt on another, each with its own cache and
    workspace: the bits of the calls alone."""
    g = gen(77)
    jobs = []
    for lens, rows, D in (([5000] * 6, [1] * 6, 128), ([3000, 700], [900, 300], 128), ([2000] * 3, [4] * 3, 64)):
        c, t = filled(g, lens, 2, 64, D, 32)
        cu = [0]
        for r in rows:
            cu.append(cu[-1] + r)
        args = (randn(g, cu[-1], 8, D).bfloat16(), c, t, i32(lens), i32(cu))
        jobs.append((args, rnl.rnl_kv4_attention(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for args, _, s in jobs:
            with torch.cuda.stream(s):
                got.append(rnl.rnl_kv4_attention(*args))
    torch.cuda.synchronize()
    rnl.rnl_check_device_error()
    for i, out in enumerate(got):
        assert torch.equal(out, jobs[i % len(jobs)][1])


def test_bad_sequences_with_many_rows():
    """Page ids outside the cache, lengths and rows out of range, in the prompt
    kernel: reported, and the sequences beside them right."""
    g = gen(6)
    n, rows, page = 300, 90, 32
    c, t = filled(g, [n, n], 2, page, 128, 32)
    t = wide(t, page)
    q = randn(g, 2 * rows, 8, 128).bfloat16()
    bad_page, minus = t.clone(), t.clone()
    bad_page[0, 3], minus[0, 9] = c.n_pages, -1
    cu = i32([0, rows, 2 * rows])
    want = rnl.rnl_kv4_attention(q, c, t, i32([n, n]), cu)
    for tt, lens, rr in ((bad_page, i32([n, n]), cu), (minus, i32([n, n]), cu), (t, i32([-5, n]), cu),
                         (t, i32([2 ** 31 - 1, n]), cu), (t, i32([n, n]), i32([rows + 7, rows, 2 * rows]))):
        out = torch.full_like(q, 320.0)
        rnl.rnl_kv4_attention(q, c, tt, lens, rr, out=out)
        with pytest.raises(rnl.RnlError, match="RNL_ERR_ARG"):
            rnl.rnl_check_device_error()
        # (two bf16 roundings of sums whose weights differ by their own rounding)
        assert ((out[rows:].double() - want[rows:].double()).abs() <= 2.0 ** -7 * want[rows:].double().abs() + 1e-3).all()
        if tt is t:
            assert (out[:rows] == 320.0).all()
    rnl.rnl_check_device_error()


def test_captured_prompts_follow_their_inputs():
    """A captured call of many rows, replayed over other lengths, row counts and
    queries in the same buffers, with a workspace full of what was there before."""
    g = gen(14)
    T, Hq, Hkv, D, page = 400, 8, 2, 128, 64
    c, t = filled(g, [900, 640, 333], Hkv, page, D, 32)
    t = wide(t, page)
    q = randn(g, T, Hq, D).bfloat16()
    lens, cu = i32([900, 640, 333]), i32([0, 200, 380, 400])
    size = rnl.workspace_size(rnl.OP_KV4_ATTENTION, T, D, Hq, Hkv)
    ws = torch.randint(0, 256, (size,), device="cuda").to(torch.uint8)
    out, lse = torch.empty_like(q), torch.empty(T, Hq, device="cuda")

    def call():
        rnl.rnl_kv4_attention(q, c, t, lens, cu, out=out, lse_out=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            call()
    torch.cuda.synchronize()
    for i, (now, rows) in enumerate((([900, 640, 333], [0, 200, 380, 400]), ([300, 2, 1], [0, 300, 301, 302]),
                                     ([0, 640, 333], [0, 5, 10, 300]), ([900, 600, 330], [0, 0, 399, 400]))):
        lens.copy_(i32(now))
        cu.copy_(i32(rows))
        q.copy_(randn(gen(200 + i), *q.shape).bfloat16())
        out.fill_(320.0)
        gr.replay()
        torch.cuda.synchronize()
        rnl.rnl_check_device_error()
        n = rows[-1]
        want, _ = check_outputs(plain.attention(q, c, t, lens, cu), q, c, t, now, rows)
        assert torch.equal(out[:n], want[:n]) and (out[n:] == 320.0).all()
