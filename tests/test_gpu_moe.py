"""The expert layer on the GPU against plain 64-bit implementations: routing and
the sum back (rnl_moe_route, rnl_moe_combine), products grouped by expert
(rnl_grouped_linear_bf16) and rows into MXFP8 (rnl_add_rmsnorm_mxfp8,
rnl_quant_mxfp8).

Tolerances.  A product: the FP32 sum of K terms in the tensor core is off by at
most (K + pieces) roundings of 2^-23 relative to the sum of magnitudes (its
internal alignment keeps fewer bits than a rounded FP32 sum, so a step is
counted as 2^-23, twice FP32's half step); then one rounding to bf16, 2^-8
relative.  bound = 2^-8 |ref| + (K + 160) 2^-23 sum |terms|.  With swiglu the
derivative of silu(g) u carries the sums' errors on: |u| + |g| (silu' is at
most 1.1, silu at most |g|); the exponential and the division add a few units
of 2^-23 of the value, times |g| for the exponential's argument."""
import math

import pytest
import torch

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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ routing
def plain_route(logits, k, renorm):
    """Token by token on the host."""
    T, E = logits.shape
    l = logits.double().cpu()
    ids, weights = [], []
    groups = [[] for _ in range(E)]
    for t in range(T):
        v = [x if x == x else -math.inf for x in l[t].tolist()]
        order = [e for e in sorted(range(E), key=lambda e: -v[e]) if v[e] > -math.inf]  # stable: lower expert first
        m = v[order[0]] if order else 0.0
        p = [math.exp(x - m) if x != m else 1.0 for x in v]
        p = [0.0 if x == -math.inf else q for x, q in zip(v, p)]
        chosen = order[:k]
        total = sum(p[e] for e in chosen) if renorm else sum(p)
        ids.append(chosen + [-1] * (k - len(chosen)))
        weights.append([p[e] / total for e in chosen] + [0.0] * (k - len(chosen)))
        for j, e in enumerate(chosen):
            groups[e].append((t, j))
    slots = [[-1] * k for _ in range(T)]
    rows, offsets = [], [0]
    for g in groups:
        for t, j in g:
            slots[t][j] = len(rows)
            rows.append(t)
        offsets.append(len(rows))
    rows += [-1] * (T * k - len(rows))
    return ids, weights, offsets, rows, slots


def check_route(logits, k, renorm):
    got = rnl.rnl_moe_route(logits, k, renormalize=renorm)
    ids, weights, offsets, rows, slots = plain_route(logits, k, renorm)
    assert got.ids.tolist() == ids
    assert got.offsets.tolist() == offsets
    assert got.rows.tolist() == rows
    assert got.slots.tolist() == slots
    # exp of a difference of FP32 values (half a unit off, times its size up to 88)
    # and sums of up to 1024 terms by halves (10 + 32 steps): 2^-24 (88 + 42 + 4)
    w = torch.tensor(weights, dtype=torch.float64, device="cuda").view_as(got.weights)
    assert ((got.weights.double() - w).abs() <= 134 * 2.0 ** -24 * w + 1e-37).all()


@pytest.mark.parametrize("T,E,k,renorm", [(1, 1, 1, True), (1, 8, 2, False), (5, 33, 4, True), (64, 64, 8, True),
                                          (65, 64, 8, False), (300, 128, 8, True), (77, 300, 6, False),
                                          (130, 1024, 32, True), (1000, 5, 5, True), (333, 256, 1, False)])
def test_route(T, E, k, renorm):
    check_route(randn(gen(T + E), T, E) * 2, k, renorm)


@pytest.mark.parametrize("T", [3, 200])
def test_route_ties_masks_and_infinities(T):
    g = gen(T)
    l = torch.round(randn(g, T, 40) * 2) / 2  # many equal logits
    l[l == 0] = -0.0
    l[torch.rand(T, 40, generator=g, device="cuda") < 0.05] = 0.0
    l[:, 7] = -math.inf
    l[0] = -math.inf                # nothing to choose
    l[1, 3:] = -math.inf            # three to choose from
    l[1, 1] = math.nan
    l[2, 11] = math.inf
    l[2, 5] = math.inf              # two infinite ones
    check_route(l, 6, True)
    check_route(l, 6, False)


def test_route_all_tokens_one_expert():
    l = torch.zeros(500, 9, device="cuda")
    l[:, 4] = 5
    check_route(l, 1, True)
    check_route(l, 9, True)


def test_route_no_tokens():
    r = rnl.rnl_moe_route(torch.empty(0, 12, device="cuda"), 3)
    assert r.offsets.tolist() == [0] * 13 and r.rows.numel() == 0


def test_route_many_tokens_per_cta():
    """More tokens than 256 CTAs of 64: the group order is still that of a stable sort."""
    T, E, k = 40001, 16, 2
    l = torch.round(randn(gen(9), T, E) * 4) / 4
    r = rnl.rnl_moe_route(l, k)
    ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids.long(), ids)
    order = torch.sort(ids.flatten(), stable=True).indices
    assert torch.equal(r.rows.long(), order // k)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(r.slots.long().flatten(), place)
    assert torch.equal(r.offsets.long()[1:], torch.bincount(ids.flatten(), minlength=E).cumsum(0))


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("T,k,N,res", [(1, 1, 8, False), (1, 8, 4096, True), (37, 3, 520, True), (100, 5, 64, False),
                                       (9, 0, 16, True), (513, 32, 24, True)])
def test_combine(T, k, N, res):
    g = gen(T * 100 + k)
    M = max(T * k - 3, 1)
    y = randn(g, M, N).bfloat16()
    slots = torch.randint(-1, M, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    w[slots < 0] = math.nan  # weights of left-out places are not read as numbers
    r = randn(g, T, N).bfloat16() if res else None
    out = rnl.rnl_moe_combine(y, slots, w, residual=r)
    on = (slots >= 0)[..., None]
    terms = torch.where(on, w[..., None].double() * y[slots.long().clamp_min(0)].double(), 0.0)
    ref = terms.sum(1) + (r.double() if res else 0)
    mag = terms.abs().sum(1) + (r.double().abs() if res else 0)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (k + 1) * 2.0 ** -24 * mag).all()
    if res:  # in place
        rnl.rnl_moe_combine(y, slots, w, residual=r, out=r)
        assert torch.equal(r, out)


def test_combine_bad_slot_is_reported():
    y, w = torch.ones(4, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(2, 2, device="cuda")
    out = rnl.rnl_moe_combine(y, i32([[0, 4], [1, -2]]), w)
    with pytest.raises(rnl.RnlError) as e:
        rnl.rnl_check_device_error()
    assert e.value.status == 4
    assert (out == 1).all()


# ------------------------------------------------------- products by expert
def plain_grouped(x, W, offsets, rows, swiglu):
    """(ref, bound) of every grouped row, 64 bits."""
    refs, bounds = [], []
    K = x.shape[1]
    eps = (K + 160) * 2.0 ** -23
    for e in range(W.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        xe = (x[rows[a:b].long()] if rows is not None else x[a:b]).double()
        we = W[e].double()
        y, m = xe @ we.T, xe.abs() @ we.abs().T
        if swiglu:
            gt, up = y.chunk(2, dim=1)
            mg, mu = m.chunk(2, dim=1)
            y = gt * torch.sigmoid(gt) * up
            err = eps * (1.1 * mg * up.abs() + mu * gt.abs()) + (8 + gt.abs()) * 2.0 ** -22 * y.abs()
        else:
            err = eps * m
        refs.append(y)
        bounds.append(2.0 ** -8 * y.abs() + err)
    return torch.cat(refs), torch.cat(bounds)


def check_grouped(counts, K, N, swiglu, gather, seed=0, tail=0):
    g = gen(seed)
    E = len(counts)
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    M = offsets[-1] + tail
    R = max(M // 3, 1) if gather else M
    x = randn(g, R, K).bfloat16()
    W = (randn(g, E, N, K) / math.sqrt(K)).bfloat16()
    rows = torch.randint(0, R, (M,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    if tail and gather:
        rows[offsets[-1]:] = -1
    out = torch.full((M, N // 2 if swiglu else N), 7.0, dtype=torch.bfloat16, device="cuda")
    rnl.rnl_grouped_linear_bf16(x, W, i32(offsets), rows=rows, swiglu=swiglu, out=out)
    rnl.rnl_check_device_error()
    n = offsets[-1]
    ref, bound = plain_grouped(x, W, offsets, rows, swiglu)
    err = (out[:n].double() - ref).abs()
    assert (err <= bound).all(), f"{(err > bound).sum()} of {err.numel()}, worst {(err / bound).max():.2f}"
    assert (out[n:] == 7).all()


SHAPES = [
    ([1], 8, 1), ([1], 64, 128), ([3, 0, 0, 5], 72, 40), ([0, 16, 17, 1], 128, 256), ([255, 256, 257], 200, 130),
    ([300, 0, 31, 1, 600], 512, 513), ([0, 0, 0], 64, 64), ([1, 2, 3, 4, 5, 6, 7, 8], 1000, 520),
    ([4097], 64, 96), ([700, 20, 5000, 1], 256, 768), ([2] * 64, 2048, 256), ([128] * 8, 1024, 1024),
]


@pytest.mark.parametrize("counts,K,N", SHAPES)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(counts, K, N, gather):
    if sum(counts) == 0:
        check_grouped(counts, K, N, False, gather, tail=5)
    else:
        check_grouped(counts, K, N, False, gather)


@pytest.mark.parametrize("counts,K,N", [(c, K, max(32, N // 32 * 32)) for c, K, N in SHAPES])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_swiglu(counts, K, N, gather):
    check_grouped(counts, K, N, True, gather, tail=3)


def test_grouped_many_experts():
    """As many experts as the library takes, most without a row."""
    counts = [0] * 1024
    for e, c in ((0, 3), (1, 40), (500, 300), (501, 1), (1022, 7), (1023, 260)):
        counts[e] = c
    check_grouped(counts, 136, 96, False, True)
    check_grouped([1] * 1024, 64, 64, True, False)
    check_mx(counts, 192, 96, 32, False, True)
    check_mx([2] * 1024, 64, 64, 64, True, False)


def test_grouped_many_tiles_a_worker():
    """More tiles a CTA pair than are worked out at the start, whole and cut ones."""
    g = gen(12)
    counts = torch.randint(1, 230, (100,), generator=g, device="cuda").tolist()
    check_grouped(counts, 72, 8200, False, False)
    check_grouped(counts, 64, 8192, True, True)
    check_mx(counts, 64, 8200, 32, False, False)
    check_mx(counts, 192, 8192, 64, True, True)


# ------------------------------------------------- products by expert, MXFP8
def mx_values(codes, scales, block):
    v = codes.view(torch.float8_e4m3fn).double()
    return v * torch.exp2(scales.double() - 127).repeat_interleave(block, dim=-1)


def mx_codes(g, *shape):
    c = torch.randint(0, 252, shape, generator=g, device="cuda", dtype=torch.uint8)
    return torch.where(c < 126, c, c + 2)  # every value but NaN


def mx_case(counts, K, N, block, gather, seed, tail=0):
    g = gen(seed)
    E, M = len(counts), sum(counts) + tail
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    R = max(M // 3, 1) if gather else M
    x, w = mx_codes(g, R, K), mx_codes(g, E, N, K)
    xs = torch.randint(110, 130, (R, K // block), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(105, 118, (E, N, K // block), generator=g, device="cuda", dtype=torch.uint8)
    rows = torch.randint(0, R, (M,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    return x, xs, w, ws, offsets, rows, M


def check_mx(counts, K, N, block, swiglu, gather, seed=0, tail=0):
    x, xs, w, ws, offsets, rows, M = mx_case(counts, K, N, block, gather, seed, tail)
    if swiglu:
        ws = ws - 4  # gates of ordinary size
    out = torch.full((M, N // 2 if swiglu else N), 7.0, dtype=torch.bfloat16, device="cuda")
    rnl.rnl_grouped_linear_mxfp8(x, xs, w, ws, i32(offsets), rows=rows, swiglu=swiglu, block=block, out=out)
    rnl.rnl_check_device_error()
    n = offsets[-1]
    ref, bound = plain_grouped(mx_values(x, xs, block), mx_values(w, ws, block), offsets, rows, swiglu)
    err = (out[:n].double() - ref).abs()
    assert (err <= bound).all(), f"{(err > bound).sum()} of {err.numel()}, worst {(err / bound).max():.2f}"
    assert (out[n:] == 7).all()


MX_SHAPES = [
    ([1], 64, 1), ([1], 128, 128), ([3, 0, 0, 5], 192, 40), ([0, 16, 17, 1], 128, 256), ([223, 224, 225], 320, 130),
    ([300, 0, 31, 1, 600], 512, 513), ([1, 2, 3, 4, 5, 6, 7, 8], 1088, 520), ([4097], 64, 96),
    ([700, 20, 5000, 1], 256, 768), ([2] * 64, 2048, 256), ([128] * 8, 1024, 1024), ([500, 3], 4096, 640),
]


@pytest.mark.parametrize("counts,K,N", MX_SHAPES)
@pytest.mark.parametrize("block", [32, 64])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_mx(counts, K, N, block, gather):
    check_mx(counts, K, N, block, False, gather, tail=2)


@pytest.mark.parametrize("counts,K,N", [(c, K, max(32, N // 32 * 32)) for c, K, N in MX_SHAPES])
@pytest.mark.parametrize("block", [32, 64])
def test_grouped_mx_swiglu(counts, K, N, block):
    check_mx(counts, K, N, block, True, True)


@pytest.mark.parametrize("K", [32, 96, 160, 2080])
def test_grouped_mx_odd_blocks(K):
    """K / 32 odd: scale rows without any alignment."""
    check_mx([5, 40, 300], K, 200, 32, False, True)


def test_grouped_mx_agrees_with_scaled_mm():
    x, xs, w, ws, _, _, _ = mx_case([300], 1024, 384, 64, False, 4)
    a = rnl.rnl_grouped_linear_mxfp8(x, xs, w, ws, i32([0, 300]))
    b = rnl.mxfp8_scaled_mm(x, xs, w[0], ws[0])
    # each is within the bound of the exact value (the two add up in other orders, so
    # where terms cancel they are more than a bf16 step of the value apart):
    # |a - b| <= |a - ref| + |b - ref| <= 2 bound
    _, bound = plain_grouped(mx_values(x, xs, 64), mx_values(w, ws, 64), [0, 300], None, False)
    far = (a.double() - b.double()).abs() > 2 * bound
    assert not far.any(), int(far.sum())


def test_grouped_mx_nan_scales_stay_in_their_rows():
    x, xs, w, ws, offsets, _, _ = mx_case([40, 60], 512, 256, 32, False, 5)
    good = rnl.rnl_grouped_linear_mxfp8(x, xs, w, ws, i32(offsets), block=32)
    xs2, ws2 = xs.clone(), ws.clone()
    xs2[7, 3] = 255
    ws2[1, 100, 15] = 255
    out = rnl.rnl_grouped_linear_mxfp8(x, xs2, w, ws2, i32(offsets), block=32)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[7] = True
    bad[40:, 100] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], good[~bad])


# ------------------------------------------------------- how calls are made
def test_bad_offsets_and_rows_are_reported():
    g = gen(3)
    x, W = randn(g, 8, 64).bfloat16(), randn(g, 3, 32, 64).bfloat16()
    for off in ([0, 5, 3, 8], [0, 2, 4, 9], [-1, 2, 4, 8]):
        out = torch.full((8, 32), 7.0, dtype=torch.bfloat16, device="cuda")
        rnl.rnl_grouped_linear_bf16(x, W, i32(off), out=out)
        with pytest.raises(rnl.RnlError) as e:
            rnl.rnl_check_device_error()
        assert e.value.status == 4 and (out == 7).all()
    rows = i32([0, 1, 8, 3, -1, 5, 6, 7])
    good = i32([0, 1, 2, 3, 4, 5, 6, 7])
    off = i32([0, 3, 5, 8])
    out = rnl.rnl_grouped_linear_bf16(x, W, off, rows=rows)
    with pytest.raises(rnl.RnlError) as e:
        rnl.rnl_check_device_error()
    assert e.value.status == 4
    want = rnl.rnl_grouped_linear_bf16(x, W, off, rows=good)
    fine = [0, 1, 3, 5, 6, 7]
    assert torch.equal(out[fine], want[fine])


def test_rows_in_front_of_the_first_group_stay():
    g = gen(4)
    x, W = randn(g, 100, 128).bfloat16(), randn(g, 2, 64, 128).bfloat16()
    out = torch.full((100, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    rnl.rnl_grouped_linear_bf16(x, W, i32([30, 60, 90]), out=out)
    want = rnl.rnl_grouped_linear_bf16(x[30:90].contiguous(), W, i32([0, 30, 60]))
    assert (out[:30] == 7).all() and (out[90:] == 7).all() and torch.equal(out[30:90], want)


def layer(g, T, E, k, K, F):
    """A layer of experts: its weights, bf16 and MXFP8."""
    w1 = (randn(g, E, 2 * F, K) / math.sqrt(K)).bfloat16()
    w2 = (randn(g, E, K, F) / math.sqrt(F)).bfloat16()
    q1, s1 = rnl.rnl_quant_mxfp8(w1.view(-1, K), block=32)
    q2, s2 = rnl.rnl_quant_mxfp8(w2.view(-1, F), block=32)
    return dict(wr=(randn(g, E, K) / math.sqrt(K)).bfloat16(), gamma=(1 + 0.1 * randn(g, K)).bfloat16(), w1=w1, w2=w2,
                q1=q1.view(E, 2 * F, K), s1=s1.view(E, 2 * F, -1), q2=q2.view(E, K, F), s2=s2.view(E, K, -1))


def run_layer(p, x, res, k, mx, stream=None):
    """The calls as they are used: residual add and norm, router, experts, sum back."""
    st = dict(stream=stream)
    s = torch.empty_like(x)
    codes, scale = rnl.rnl_add_rmsnorm_mxfp8(x, p["gamma"], residual=res, x_sum_out=s, block=32, **st)
    logits = rnl.rmsnorm_linear_bf16(s, None, p["wr"], out_dtype=rnl.OUT_FP32, **st)
    r = rnl.rnl_moe_route(logits, k, **st)
    if mx:
        h = rnl.rnl_grouped_linear_mxfp8(codes, scale, p["q1"], p["s1"], r.offsets, rows=r.rows, swiglu=True, block=32, **st)
        hq, hs = rnl.rnl_quant_mxfp8(h, block=32, **st)
        y = rnl.rnl_grouped_linear_mxfp8(hq, hs, p["q2"], p["s2"], r.offsets, block=32, **st)
    else:
        h = rnl.rnl_grouped_linear_bf16(s, p["w1"], r.offsets, rows=r.rows, swiglu=True, **st)
        y = rnl.rnl_grouped_linear_bf16(h, p["w2"], r.offsets, **st)
    return rnl.rnl_moe_combine(y, r.slots, r.weights, residual=s, **st), s, logits, r, codes, scale, h


@pytest.mark.parametrize("T,E,k,K,F", [(1, 8, 2, 512, 256), (70, 16, 4, 512, 352), (600, 32, 4, 768, 384)])
@pytest.mark.parametrize("mx", [False, True])
def test_layer_of_experts(T, E, k, K, F, mx):
    """A run of the calls together, against 64 bits from the same routing.  The
    intermediate rows are the calls' own bf16 rows (their error is tested above);
    the last step is held to the sum of its rows' bounds."""
    g = gen(T + K)
    p = layer(g, T, E, k, K, F)
    x, res = randn(g, T, K).bfloat16(), randn(g, T, K).bfloat16()
    out, s, logits, r, codes, scale, h = run_layer(p, x, res, k, mx)
    rnl.rnl_check_device_error()
    assert torch.equal(s, (x.float() + res.float()).bfloat16())
    ids, weights, offsets, rows, slots = plain_route(logits, k, True)
    assert r.ids.tolist() == ids and r.rows.tolist() == rows
    if mx:
        a1, b1 = mx_values(codes, scale, 32), mx_values(p["q1"], p["s1"], 32)
        hq, hs = rnl.rnl_quant_mxfp8(h, block=32)
        a2, b2 = mx_values(hq, hs, 32), mx_values(p["q2"], p["s2"], 32)
    else:
        a1, b1, a2, b2 = s.double(), p["w1"].double(), h.double(), p["w2"].double()
    ref, bound = plain_grouped(a1, b1, offsets, r.rows, True)
    assert ((h.double() - ref).abs() <= bound).all()
    y, yb = plain_grouped(a2, b2, offsets, None, False)
    w = r.weights.double()[..., None]
    at = r.slots.long()
    want = s.double() + (w * y[at]).sum(1)
    tol = (w * yb[at]).sum(1) + 2.0 ** -8 * want.abs() + (k + 1) * 2.0 ** -24 * (s.double().abs() + (w * y[at].abs()).sum(1))
    assert ((out.double() - want).abs() <= tol * (1 + 2.0 ** -7)).all()  # (the sum rounds its bounds' rows too)


def test_layer_on_given_streams():
    """Layers in flight at once on streams of their own give the bits of the calls alone."""
    g = gen(8)
    jobs = []
    for T, E, k, K, F in ((200, 16, 4, 512, 256), (3, 16, 4, 512, 256), (1000, 8, 2, 768, 384)):
        p = layer(g, T, E, k, K, F)
        for mx in (False, True):
            jobs.append((p, randn(g, T, K).bfloat16(), randn(g, T, K).bfloat16(), k, mx))
    want = [run_layer(*j)[0] for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        got = [run_layer(*j, stream=s)[0] for j, s in zip(jobs, streams)]
        torch.full((1 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layer_captured_and_replayed():
    """A captured layer, replayed with other inputs and other routings in the same
    buffers, gives the bits of the calls made one by one."""
    g = gen(9)
    T, E, k, K, F = 300, 16, 4, 512, 256
    p = layer(g, T, E, k, K, F)
    x, res = randn(g, T, K).bfloat16(), randn(g, T, K).bfloat16()
    for mx in (False, True):
        run_layer(p, x, res, k, mx)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run_layer(p, x, res, k, mx)[0]
        for i in range(6):
            x.copy_(randn(g, T, K))
            if i % 2:
                p["wr"].copy_(randn(g, E, K) * (4 if i == 3 else 0.05))
            graph.replay()
            got = out.clone()
            assert torch.equal(got, run_layer(p, x, res, k, mx)[0]), i
        graph.replay()
        graph.replay()
        assert torch.equal(out, got)
    rnl.rnl_check_device_error()


def test_same_call_same_bits_whatever_the_workspace_holds():
    g = gen(10)
    x, W = randn(g, 900, 2048).bfloat16(), randn(g, 8, 640, 2048).bfloat16()
    off = i32([0, 100, 103, 103, 400, 401, 700, 800, 900])
    want = rnl.rnl_grouped_linear_bf16(x, W, off)
    n = rnl.workspace_size(rnl.OP_GROUPED, 900, 2048, 640, 8)
    for fill in (0, 255, 1):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(5):
            assert torch.equal(rnl.rnl_grouped_linear_bf16(x, W, off, workspace=ws), want)
    rnl.rnl_check_device_error()


def test_strided_and_wrong_device_arguments_are_refused():
    x, W, off = torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda"), i32([0, 4, 8])
    with pytest.raises(ValueError):
        rnl.rnl_grouped_linear_bf16(x[:, :64], W, off)
    with pytest.raises(ValueError):
        rnl.rnl_grouped_linear_bf16(x[:, :64].contiguous(), W, off.cpu())
    with pytest.raises(ValueError):
        rnl.rnl_grouped_linear_bf16(x[:, :64].contiguous(), W, off, workspace=torch.empty(1 << 26, dtype=torch.uint8))
    with pytest.raises(rnl.RnlError):
        rnl.rnl_grouped_linear_bf16(x[:, :64].contiguous(), W, off, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_offsets_past_32_bits():
    """Weights and outputs of more than 2^32 bytes (and elements, for the codes)."""
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("not enough memory")
    E, N, K = 9, 8192, 65536   # 4.8e9 codes
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    g = gen(11)
    w[0], w[8] = mx_codes(g, N, K), mx_codes(g, N, K)
    ws = torch.full((E, N, K // 64), 108, dtype=torch.uint8, device="cuda")
    x, xs = mx_codes(g, 9, K), torch.full((9, K // 64), 110, dtype=torch.uint8, device="cuda")
    out = rnl.rnl_grouped_linear_mxfp8(x, xs, w, ws, i32([0, 4] + [4] * 7 + [9]))
    for rows, e in ((slice(0, 4), 0), (slice(4, 9), 8)):
        ref, bound = plain_grouped(mx_values(x[rows], xs[rows], 64), mx_values(w[e:e + 1, ::64], ws[e:e + 1, ::64], 64),
                                   [0, rows.stop - rows.start], None, False)
        assert ((out[rows, ::64].double() - ref).abs() <= bound).all()
    del w
    # 2.2e9 outputs
    M, N, K = 270000, 8192, 64
    x, W = randn(g, M, K).bfloat16(), randn(g, 2, N, K).bfloat16()
    out = rnl.rnl_grouped_linear_bf16(x, W, i32([0, 5, M]))
    for rows in (slice(0, 5), slice(M - 300, M)):
        ref, bound = plain_grouped(x[rows], W[:1] if rows.start == 0 else W[1:], [0, rows.stop - rows.start], None, False)
        assert ((out[rows].double() - ref).abs() <= bound).all()
