"""Cases and plain forms of the operators between the qkv projection and the
attention output: rotary positions with several axes, the 4-bit paged KV cache
(write and read back), and attention over that cache.

    own = False   run() computes the plain forms with elementary torch operations
    own = True    run() makes the library's calls

Cache format (MX, E2M1 elements): codes uint8 [pages, Hkv, page, D / 2] (element
2j in the low nibble of byte j, 2j + 1 in the high one), scales uint8 [pages,
Hkv, page, D / block] (E8M0: 2^(byte - 127)); per block of a token's head row
X = floor(log2 max|x|) - 2 (at least -127), code = E2M1(x 2^-X), nearest even,
saturating at 6.
"""
import math
import random

import torch

own = False

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    heads = dict(Hq=32, Hkv=8, D=128)  # the grouped-query projection 4096 -> (32 + 2 * 8) * 128
    paged = dict(block=32, page=64, **heads)
    step = dict(kind="attn", rows_min=1, rows_max=1, causal=True, window=0, **paged)
    ahead = dict(kind="attn", causal=True, window=0, **paged)
    return [
        # positions: a prompt of 4096 tokens with an image and a video clip in it
        dict(name="rope_axes_prompt", kind="rope", T=4096, axes=3, layout="sections", norm=True, span=4096, **heads),
        # one decode step of four sequences
        dict(name="rope_axes_step", kind="rope", T=4, axes=3, layout="interleaved", norm=True, span=4096, **heads),
        # a video's patches through an encoder: two axes, no head norm, an odd count
        dict(name="rope_axes_patches", kind="rope", T=18433, axes=2, layout="sections", norm=False, span=512,
             Hq=16, Hkv=16, D=64),
        # cache: one new token for each of 64 running sequences
        dict(name="cache_step_64", kind="cache", B=64, rows_min=1, rows_max=1, len_min=1, len_max=8000, mix=1, **paged),
        # cache: five prompts of uneven length arrive together
        dict(name="cache_prompts", kind="cache", B=5, rows_min=300, rows_max=6000, len_min=300, len_max=12000, mix=2, **paged),
        # a cached prefix is fetched back as bf16
        dict(name="cache_fetch", kind="fetch", B=3, rows_min=9000, rows_max=20000, len_min=9000, len_max=20000, mix=3,
             block=64, page=16, **heads),
        # attention: one conversation, next token
        dict(name="step_1x4096", B=1, len_min=4097, len_max=4097, mix=4, **step),
        # a serving batch with ragged histories
        dict(name="step_64_ragged", B=64, len_min=1, len_max=16384, mix=5, **step),
        # long documents
        dict(name="step_8x131072", B=8, len_min=131000, len_max=131072, mix=6, **step),
        # drafted tokens checked four at a time
        dict(name="draft_32x4", B=32, rows_min=4, rows_max=4, len_min=2000, len_max=9000, mix=7, **ahead),
        # a chunk of a long prompt, its own tokens included, over what is cached already
        dict(name="prompt_chunk", B=2, rows_min=1000, rows_max=2048, len_min=6000, len_max=10240, mix=8, **ahead),
        # a decoder reading an encoder's states, every row sees all of them
        dict(name="cross_states", kind="attn", B=4, rows_min=200, rows_max=448, len_min=1500, len_max=1500, mix=9,
             causal=False, window=0, block=32, page=32, Hq=16, Hkv=16, D=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "cache", "fetch", "step", "step", "draft", "prompt", "cross"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    if kind == "rope":
        return dict(kind="rope", T=_log(rng, 1, 8000), axes=rng.choice([2, 3, 4]),
                    layout=rng.choice(["sections", "interleaved"]), norm=rng.random() < 0.5,
                    span=rng.choice([512, 4096]), Hq=Hq, Hkv=Hkv, D=D)
    c = dict(block=rng.choice([32, 64]), page=rng.choice([16, 32, 64, 128]), Hq=Hq, Hkv=Hkv, D=D,
             mix=rng.randrange(1 << 30))
    if kind in ("cache", "fetch"):
        hi = _log(rng, 1, 8000)
        lo = max(1, hi // 4)
        return dict(kind=kind, B=_log(rng, 1, 8 if hi > 100 else 100), rows_min=lo, rows_max=hi, len_min=lo,
                    len_max=hi + rng.randrange(500), **c)
    c.update(kind="attn", causal=True, window=rng.choice([0, 0, 0, 500]))
    if kind == "step":
        hi = _log(rng, 1, 40000)
        return dict(B=_log(rng, 1, max(2, min(100, 200000 // hi))), rows_min=1, rows_max=1,
                    len_min=max(1, hi // 8), len_max=hi, **c)
    if kind == "draft":
        hi = _log(rng, 20, 10000)
        return dict(B=_log(rng, 1, 20), rows_min=2, rows_max=9, len_min=max(9, hi // 4), len_max=hi, **c)
    if kind == "prompt":
        rows = _log(rng, 20, 2000)
        return dict(B=rng.choice([1, 2, 3]), rows_min=max(1, rows // 3), rows_max=rows, len_min=rows,
                    len_max=rows + _log(rng, 1, 4000), **c)
    c.update(causal=False, window=0)
    return dict(B=_log(rng, 1, 6), rows_min=1, rows_max=_log(rng, 1, 500), len_min=1, len_max=_log(rng, 1, 4000), **c)


def _plan(case):
    """(new rows, cached length) of each sequence; the length counts the new rows
    of a causal case."""
    rng = random.Random(case["mix"])
    out = []
    for _ in range(case["B"]):
        r = rng.randint(case["rows_min"], case["rows_max"])
        lo, hi = case["len_min"], case["len_max"]
        n = _log(rng, max(lo, 1), max(hi, 1)) if hi > 8 * max(lo, 1) else rng.randint(lo, hi)
        out.append((r, max(n, r) if case.get("causal", True) else n))
    return out


def _axis_of_pair(case):
    half, n = case["D"] // 2, case["axes"]
    if case["layout"] == "interleaved":
        return [i % n for i in range(half)]
    cuts = [half * (a + 1) // n for a in range(n)]
    return [sum(i >= c for c in cuts) for i in range(half)]


# ------------------------------------------------------------------ inputs
def _pow2(e):
    """2^e in float32 for integer tensors -126 <= e <= 127, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x, block):
    """bf16 [..., D] -> (codes [..., D / 2], scale bytes [..., D / block])."""
    b = x.float().unflatten(-1, (-1, block))
    amax = b.abs().amax(-1)
    e = torch.frexp(amax).exponent - 3
    X = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp_min(-127)
    y = b * _pow2(-X).unsqueeze(-1)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = (torch.round(a / step) * step).clamp_max(6.0)
    bounds = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    c = torch.bucketize(r, bounds).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), (X + 127).to(torch.uint8)


def _values(codes, scales, block, dtype):
    """The numbers that codes [..., D / 2] with scales [..., D / block] stand for."""
    lut = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=dtype, device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    v = lut[pair.int()].unflatten(-1, (-1, block))
    e = scales.int() - 127
    p = torch.where(e > -127, _pow2(e.clamp_min(-126)), torch.full_like(e, 2.0 ** -127, dtype=torch.float32))
    return (v * p.to(dtype).unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    st = dict(case)
    if case["kind"] == "rope":
        T, n, span = case["T"], case["axes"], case["span"]
        st["y"] = (randn(T, (Hq + 2 * Hkv) * D) * 1.5).bfloat16()
        st["positions"] = torch.randint(0, span, (n, T), generator=g, device="cuda", dtype=torch.int32)
        st["axis_of_pair"] = _axis_of_pair(case)
        inv = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") * 2 / D)
        ang = torch.arange(span, dtype=torch.float64, device="cuda")[:, None] * inv
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        st["q_gamma"] = (1 + 0.1 * randn(D)).bfloat16() if case["norm"] else None
        st["k_gamma"] = (1 + 0.1 * randn(D)).bfloat16() if case["norm"] else None
        return st
    plan = _plan(case)
    page, block, B = case["page"], case["block"], case["B"]
    need = [-(-n // page) for _, n in plan]
    T, P = sum(r for r, _ in plan), sum(need) + 1
    perm = torch.randperm(P, generator=g, device="cuda").int()
    table = torch.zeros(B, max(max(need), 1), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = [0]
    for r, _ in plan:
        cu.append(cu[-1] + r)
    st.update(T=T, plan=plan, cu=cu, block_table=table, longest=max(n for _, n in plan), most_rows=max(r for r, _ in plan),
              rows_of=torch.tensor([r for r, _ in plan], device="cuda"),
              seq_lens=torch.tensor([n for _, n in plan], dtype=torch.int32, device="cuda"),
              cu_rows=torch.tensor(cu, dtype=torch.int32, device="cuda") if case["rows_max"] > 1 else None)
    cache = []
    for which in range(2):
        codes = torch.empty(P, Hkv, page, D // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(P, Hkv, page, D // block, dtype=torch.uint8, device="cuda")
        chunk = max(1, (1 << 26) // (Hkv * page * D))
        # keys: a few channels of every head larger than the rest, as after a projection
        chan = torch.exp(0.5 * randn(Hkv, 1, D)) if which == 0 else torch.ones(Hkv, 1, D, device="cuda")
        for p in range(0, P, chunk):
            m = min(chunk, P - p)
            codes[p:p + m], scales[p:p + m] = _quantise((randn(m, Hkv, page, D) * chan).bfloat16(), block)
        cache += [codes, scales]
    st["cache"] = cache
    if case["kind"] == "cache":
        st["k"], st["v"] = randn(T, Hkv, D).bfloat16(), randn(T, Hkv, D).bfloat16()
    if case["kind"] == "attn":
        st["q"] = randn(T, Hq, D).bfloat16()
        st["scale"] = 1.0 / math.sqrt(D)
    return st


# ------------------------------------------------------------- plain forms
def _rope_plain(st):
    T, Hq, Hkv, D = st["y"].shape[0], st["Hq"], st["Hkv"], st["D"]
    y = st["y"].float().view(T, Hq + 2 * Hkv, D)
    axis = torch.tensor(st["axis_of_pair"], device=y.device)
    pos = st["positions"].long()[axis].t()                      # [T, D / 2]
    col = torch.arange(D // 2, device=y.device)
    c = st["cos_sin"][pos, col][:, None]
    s = st["cos_sin"][pos, col + D // 2][:, None]

    def turn(h, gamma):
        if gamma is not None:
            h = (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * gamma.float()).bfloat16().float()
        a, b = h[..., :D // 2], h[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], dim=-1).bfloat16()

    return (turn(y[:, :Hq], st["q_gamma"]), turn(y[:, Hq:Hq + Hkv], st["k_gamma"]),
            y[:, Hq + Hkv:].bfloat16())


def _slots(st):
    """Page and offset of every row's token (the last rows of each sequence)."""
    r, T = st["rows_of"], st["T"]
    seq = torch.repeat_interleave(torch.arange(st["B"], device="cuda"), r, output_size=T)
    pos = torch.arange(T, device="cuda") - (r.cumsum(0) - st["seq_lens"])[seq]
    return st["block_table"][seq, pos // st["page"]].long(), pos % st["page"]


def _fetch_plain(st):
    pg, off = _slots(st)
    kc, ks, vc, vs = st["cache"]
    return tuple(_values(c[pg, :, off], s[pg, :, off], st["block"], torch.float32).bfloat16()
                 for c, s in ((kc, ks), (vc, vs)))


def _cache_plain(st):
    pg, off = _slots(st)
    kc, ks, vc, vs = st["cache"]
    for x, c, s in ((st["k"], kc, ks), (st["v"], vc, vs)):
        c[pg, :, off], s[pg, :, off] = _quantise(x, st["block"])
    return _fetch_plain(st)


def _attn_plain(st):
    """Every sequence padded to the longest one, the padding masked."""
    B, Hq, Hkv, D = st["B"], st["Hq"], st["Hkv"], st["D"]
    rows, n = st["rows_of"][:, None], st["seq_lens"].long()[:, None]
    i = torch.arange(st["most_rows"], device="cuda")[None]
    at = (rows.cumsum(0) - rows + i).clamp_max(st["T"] - 1)                       # [B, R]
    q = st["q"][at].float().unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4)         # [B, Hkv, G, R, D]
    pages = st["block_table"][:, :-(-st["longest"] // st["page"])].long()
    kc, ks, vc, vs = (t[pages].transpose(1, 2).flatten(2, 3) for t in st["cache"])  # [B, Hkv, n, ...]
    s = q.flatten(2, 3) @ _values(kc, ks, st["block"], torch.float32).transpose(2, 3) * st["scale"]
    s = s.unflatten(2, (-1, st["most_rows"]))
    j = torch.arange(s.shape[-1], device="cuda")[None, None]
    seen = (j < n[..., None]) & torch.ones_like(i, dtype=torch.bool)[..., None]
    if st["causal"]:
        pos = (n - rows + i)[..., None]
        seen = (j <= pos) & (j < n[..., None])
        if st["window"]:
            seen &= j > pos - st["window"]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)                                  # a row that sees nothing: p = 0
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = p.flatten(2, 3) @ _values(vc, vs, st["block"], torch.float32)
    o = o.unflatten(2, (-1, st["most_rows"])) / torch.where(l > 0, l, torch.ones_like(l))
    live = (i < rows)
    out = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live].bfloat16()
    return out, (m + torch.log(l)).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[live]


def run(st):
    kind = st["kind"]
    if not own:
        return {"rope": _rope_plain, "cache": _cache_plain, "fetch": _fetch_plain, "attn": _attn_plain}[kind](st)
    import rmsnorm_linear_projection_gb300 as rnl
    if kind == "rope":
        return rnl.rnl_qkv_rope_axes(st["y"], st["Hq"], st["Hkv"], st["D"], st["q_gamma"], st["k_gamma"],
                                     st["positions"], st["axis_of_pair"], st["cos_sin"], eps=1e-6)
    cache = rnl.Kv4Cache(*st["cache"])
    if kind == "cache":
        rnl.rnl_kv4_append(st["k"], st["v"], cache, st["block_table"], st["seq_lens"], st["cu_rows"])
    if kind in ("cache", "fetch"):
        return rnl.rnl_kv4_gather(cache, st["block_table"], st["seq_lens"], st["T"], st["cu_rows"])
    lse = torch.empty(st["T"], st["Hq"], dtype=torch.float32, device="cuda")
    out = rnl.rnl_kv4_attention(st["q"], cache, st["block_table"], st["seq_lens"], st["cu_rows"],
                                scale=st["scale"], causal=st["causal"], window=st["window"], lse_out=lse)
    return out, lse


# ------------------------------------------------------------------- work
def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["kind"] == "rope":
        T, H = case["T"], Hq + 2 * Hkv
        table = min(T, case["span"]) * D * 4
        return {"bytes": 4 * T * H * D + 4 * T * case["axes"] + table, "flops": 8 * T * (Hq + Hkv) * D}
    plan = _plan(case)
    T = sum(r for r, _ in plan)
    token = 2 * Hkv * (D // 2 + D // case["block"])  # keys and values of one token in the cache
    table = sum(-(-n // case["page"]) for _, n in plan) * 4 + 8 * case["B"]
    if case["kind"] == "cache":
        return {"bytes": T * (8 * Hkv * D + token) + 8 * case["B"], "flops": 8 * T * Hkv * D}
    if case["kind"] == "fetch":
        return {"bytes": T * (4 * Hkv * D + token) + table, "flops": 4 * T * Hkv * D}
    pairs = tokens = 0
    for r, n in plan:
        if not case["causal"]:
            pairs, tokens = pairs + r * n, tokens + n
            continue
        w = case["window"] or n
        pairs += sum(min(p + 1, w) for p in range(n - r, n))
        tokens += min(n, w + r - 1)
    return {"bytes": tokens * token + T * Hq * (4 * D + 4) + table, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ exact
def _exact_decode(codes, scales, block):
    """Sign, exponent and fraction bits taken apart, in binary64."""
    c = torch.stack([codes % 16, codes // 16], dim=-1).flatten(-2).to(torch.float64)
    neg = (c >= 8).to(torch.float64)
    c = c - 8 * neg
    e = torch.floor(c / 2)
    f = c - 2 * e
    mag = torch.where(e == 0, f / 2, (1 + f / 2) * 2.0 ** (e - 1))
    x = ((scales.long() - 127 + 1023) << 52).view(torch.float64).repeat_interleave(block, dim=-1)
    return mag * (1 - 2 * neg) * x


def _exact_round(x, block):
    """Each element's nearest level of its block's grid (ties to the even code)."""
    shape = x.shape
    b = x.double().reshape(-1, block)
    top = b.abs().max(dim=1).values
    X = torch.frexp(top).exponent - 3
    X = torch.where(top > 0, X, torch.full_like(X, -127)).clamp(min=-127)
    unit = ((X.long() + 1023) << 52).view(torch.float64)[:, None]
    level = torch.tensor(_LEVELS, dtype=torch.float64, device=x.device)
    half = (level[1:] + level[:-1]) / 2
    a = (b.abs() / unit)[..., None]
    upper_even = torch.arange(1, 8, device=x.device) % 2 == 0
    code = ((a > half) | ((a == half) & upper_even)).sum(-1)
    return (torch.sign(b) * level[code] * unit).reshape(shape)


def exact(case, seed):
    st = prepare(case, seed)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["kind"] == "rope":
        T, half = case["T"], D // 2
        y = st["y"].double().reshape(T, Hq + 2 * Hkv, D)
        cos = torch.empty(T, half, dtype=torch.float64, device="cuda")
        sin = torch.empty_like(cos)
        for i, a in enumerate(st["axis_of_pair"]):
            p = st["positions"][a].long()
            cos[:, i] = st["cos_sin"].double()[p, i]
            sin[:, i] = st["cos_sin"].double()[p, half + i]
        res = []
        for lo, hi, gamma in ((0, Hq, st["q_gamma"]), (Hq, Hq + Hkv, st["k_gamma"])):
            z = y[:, lo:hi]
            if gamma is not None:
                # the normed head is a bf16 tensor by definition
                z = (z / torch.sqrt((z ** 2).sum(2, keepdim=True) / D + 1e-6) * gamma.double()).bfloat16().double()
            w = torch.complex(z[..., :half], z[..., half:]) * torch.complex(cos, sin)[:, None]
            res.append(torch.cat([w.real, w.imag], dim=2))
        return res[0], res[1], y[:, Hq + Hkv:]
    if case["kind"] in ("cache", "fetch"):
        if case["kind"] == "cache":
            return _exact_round(st["k"], case["block"]), _exact_round(st["v"], case["block"])
        res = ([], [])
        for b, (r, n) in enumerate(st["plan"]):
            pages = st["block_table"][b, :-(-n // case["page"])].long()
            for w in range(2):
                c, s = (t[pages].transpose(1, 2).flatten(0, 1)[n - r:n] for t in st["cache"][2 * w:2 * w + 2])
                res[w].append(_exact_decode(c, s, case["block"]))
        return torch.cat(res[0]), torch.cat(res[1])
    G = Hq // Hkv
    out = torch.zeros(st["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((st["T"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (r, n) in enumerate(st["plan"]):
        pages = st["block_table"][b, :-(-n // case["page"])].long()
        for h in range(Hq):
            if n == 0:
                continue
            if h % G == 0:
                c = [t[pages, h // G].flatten(0, 1)[:n] for t in st["cache"]]
                K, V = _exact_decode(c[0], c[1], case["block"]), _exact_decode(c[2], c[3], case["block"])
            for at in range(0, r, 512):
                m = min(512, r - at)
                lo = st["cu"][b] + at
                s = (st["q"][lo:lo + m, h].double() @ K.t()) * st["scale"]
                if case["causal"]:
                    back = torch.arange(n - r + at, n - r + at + m, device="cuda")[:, None] - torch.arange(n, device="cuda")
                    hide = back < 0
                    if case["window"]:
                        hide |= back >= case["window"]
                    s = s.masked_fill(hide, -math.inf)
                z = torch.logsumexp(s, dim=1, keepdim=True)
                out[lo:lo + m, h] = torch.exp(s - z) @ V
                lse[lo:lo + m, h] = z[:, 0]
    return out, lse
