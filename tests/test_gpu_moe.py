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
