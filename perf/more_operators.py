"""Cases and plain forms of the expert layer behind the projection: residual
add + RMSNorm into MXFP8, the routing of tokens to experts, the products
grouped by expert in bf16 and in MXFP8, and the weighted sum back.

    own = False   run() computes the plain forms with elementary torch operations
    own = True    run() makes the library's calls

Formats: E4M3 codes uint8 [rows, K] and E8M0 scale bytes uint8 [rows, K / block]
(2^(byte - 127)); per block of a row X = floor(log2 max|y|) - 8 (at least -127),
code = E4M3(y 2^-X), nearest even, saturating at 448.  Rows offsets[e] ..
offsets[e + 1] - 1 of a grouped product belong to expert e and read row
rows[i] of x (row i without rows).
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the norm behind the attention of one decode step of 64 sequences
        dict(name="norm_step", kind="norm", T=64, K=4096, block=32, residual=True, gamma=True),
        # the same for two prompts of 4096 tokens
        dict(name="norm_prompt", kind="norm", T=8192, K=4096, block=64, residual=True, gamma=True),
        # routing: a decode step, and a prompt over many experts
        dict(name="route_step", kind="route", T=16, E=64, k=4, renorm=True, ties=False, masked=0),
        dict(name="route_prompt", kind="route", T=8192, E=128, k=8, renorm=True, ties=True, masked=0),
        # bf16 experts: a decode step of 16 sequences (the weights of the chosen experts are what is read)
        dict(name="experts_step", kind="grouped", T=16, E=64, k=4, K=2048, N=2816, swiglu=True, gather=True, skew=0.5),
        # a prompt's gate and up products, experts unevenly liked
        dict(name="experts_prompt", kind="grouped", T=8192, E=32, k=4, K=2048, N=2816, swiglu=True, gather=True, skew=0.7),
        # the products back to the model's width, an odd number of rows
        dict(name="experts_down", kind="grouped", T=7001, E=32, k=4, K=1408, N=2048, swiglu=False, gather=False, skew=0.7),
        # MXFP8 experts: a decode step of 32 sequences
        dict(name="experts_mx_step", kind="grouped_mx", T=32, E=128, k=8, K=4096, N=1536, swiglu=True, gather=True,
             skew=0.5, block=32),
        # two prompts
        dict(name="experts_mx_prompt", kind="grouped_mx", T=8192, E=128, k=8, K=4096, N=1536, swiglu=True, gather=True,
             skew=0.5, block=64),
        # back to the model's width, one ragged prompt
        dict(name="experts_mx_down", kind="grouped_mx", T=3001, E=128, k=8, K=768, N=4096, swiglu=False, gather=False,
             skew=0.5, block=64),
        # the weighted sum of every token's expert rows, added to the residual
        dict(name="combine_step", kind="combine", T=16, k=4, N=2048, residual=True),
        dict(name="combine_prompt", kind="combine", T=8192, k=8, N=4096, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "route", "grouped", "grouped", "grouped_mx", "grouped_mx", "combine"])
    if kind == "norm":
        block = rng.choice([32, 64])
        K = block * _log(rng, 1, 8192 // block)
        return dict(kind=kind, T=min(_log(rng, 1, 16000), (8192 * 4096) // K), K=K, block=block,
                    residual=rng.random() < 0.7, gamma=rng.random() < 0.8)
    if kind == "combine":
        N = 8 * _log(rng, 8, 1000)
        k = rng.randint(1, 8)
        return dict(kind=kind, T=min(_log(rng, 1, 16000), (8192 * 8 * 4096) // (N * k)), k=k, N=N,
                    residual=rng.random() < 0.6)
    E = _log(rng, 4, 256)
    k = rng.randint(1, min(8, E // 2))
    if kind == "route":
        return dict(kind=kind, T=min(_log(rng, 1, 8192), (8192 * 128) // E), E=E, k=k, renorm=rng.random() < 0.6,
                    ties=rng.random() < 0.5, masked=rng.choice([0, 0, 1, E // 3]))
    swiglu = rng.random() < 0.5
    block = rng.choice([32, 64]) if kind == "grouped_mx" else 8
    K = block * _log(rng, max(1, 128 // block), 4096 // block)
    N = 32 * _log(rng, 4, 128) if swiglu else _log(rng, 64, 4096)
    E = max(4, min(E, 800_000_000 // (K * N)))
    k = min(k, E // 2)
    T = _log(rng, 1, 8000)
    T = max(1, min(T, int(3.7e11 / (2 * k * K * N))))
    c = dict(kind=kind, T=T, E=E, k=k, K=K, N=N, swiglu=swiglu, gather=rng.random() < 0.6, skew=rng.choice([0.0, 0.5, 1.0]))
    return dict(c, block=block) if kind == "grouped_mx" else c


# ------------------------------------------------------------------ inputs
def _route_plan(logits, k):
    """offsets [E + 1] and the tokens of the rows grouped by expert, for tokens that all have k experts."""
    T, E = logits.shape
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].flatten()
    order = torch.sort(ids, stable=True).indices
    counts = (torch.sort(ids).values[None] == torch.arange(E, device=ids.device)[:, None]).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    return offsets, (order // k).int(), int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    st, T, kind = dict(case), case["T"], case["kind"]
    if kind == "norm":
        K = case["K"]
        # a few channels larger than the rest, as in a residual stream
        chan = torch.exp(0.7 * randn(K))
        st["x"] = (randn(T, K) * chan).bfloat16()
        st["r"] = (randn(T, K) * chan * 2).bfloat16() if case["residual"] else None
        st["g"] = (1 + 0.2 * randn(K)).bfloat16() if case["gamma"] else None
        return st
    if kind == "combine":
        k, N = case["k"], case["N"]
        st["y"] = randn(T * k, N).bfloat16()
        st["slots"] = torch.randperm(T * k, generator=g, device="cuda").int().view(T, k)
        st["w"] = torch.softmax(randn(T, k), dim=1)
        st["r"] = randn(T, N).bfloat16() if case["residual"] else None
        return st
    E, k = case["E"], case["k"]
    if kind == "route":
        logits = randn(T, E) * 1.5 + 0.5 * randn(E)
        if case["ties"]:
            logits = torch.round(logits * 16) / 16
        if case["masked"]:
            logits[:, torch.randperm(E, generator=g, device="cuda")[:case["masked"]]] = -math.inf
        st["logits"] = logits
        return st
    K, N = case["K"], case["N"]
    st["offsets"], rows, st["most"] = _route_plan(randn(T, E) + case["skew"] * randn(E), k)
    M = T * k
    st["M"] = M
    st["rows"] = rows if case["gather"] else None
    R = T if case["gather"] else M
    if kind == "grouped":
        st["x"] = randn(R, K).bfloat16()
        st["w"] = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda").normal_(0, K ** -0.5, generator=g)
        return st
    nb = K // case["block"]

    def codes(*shape):  # any E4M3 value but NaN, small ones as often as large ones
        c = torch.randint(0, 252, shape, generator=g, device="cuda", dtype=torch.uint8)
        return torch.where(c < 126, c, c + 2)

    st["x"], st["xs"] = codes(R, K), torch.randint(116, 121, (R, nb), generator=g, device="cuda", dtype=torch.uint8)
    st["w"] = codes(E, N, K)
    st["ws"] = torch.randint(112, 116, (E, N, nb), generator=g, device="cuda", dtype=torch.uint8)
    return st


# ------------------------------------------------------------- plain forms
def _pow2(e):
    """2^e in float32 for integer tensors -126 <= e <= 127, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _norm_plain(st):
    x, block = st["x"].float(), st["block"]
    if st["r"] is not None:
        x = (x + st["r"].float()).bfloat16().float()
    # the row's sum in 64 bits: codes next to a rounding border go by it
    ss = x.double().square().sum(1, keepdim=True).float()
    y = x * (1.0 / torch.sqrt(ss * (1.0 / st["K"]) + EPS))
    if st["g"] is not None:
        y = y * st["g"].float()
    y = y.unflatten(1, (-1, block))
    amax = y.abs().amax(-1)
    e = torch.frexp(amax).exponent - 9
    X = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp_min(-127)
    c = (y * _pow2(-X).unsqueeze(-1)).clamp(-448.0, 448.0).flatten(1).to(torch.float8_e4m3fn)
    return {"codes": c, "scale": (X + 127).to(torch.uint8).view(torch.float8_e8m0fnu),
            "sum": x.bfloat16() if st["r"] is not None else None}


def _route_plain(st):
    l, k = st["logits"], st["k"]
    T, E = l.shape
    l = torch.where(torch.isnan(l), -math.inf, l)
    v, ids = torch.sort(l, dim=1, descending=True, stable=True)
    m = v[:, :1].clamp_min(-1e30)
    p = torch.exp(v - m)
    total = (p[:, :k] if st["renorm"] else p).sum(1, keepdim=True)
    w = p[:, :k] / torch.where(total > 0, total, torch.ones_like(total))
    v, ids = v[:, :k], ids[:, :k]
    live = v > -math.inf
    key = torch.where(live, ids, E).flatten()
    order = torch.sort(key, stable=True).indices
    counts = (key[None] == torch.arange(E, device=l.device)[:, None]).sum(1)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=l.device)
    used = torch.arange(T * k, device=l.device) < counts.sum()
    return {"ids": torch.where(live, ids, -1).int(), "weights": torch.where(live, w, 0.0),
            "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int(),
            "rows": torch.where(used, order // k, -1).int(),
            "slots": torch.where(live, place.view(T, k), -1).int()}


def _values(codes, scales, block):
    """The numbers that E4M3 codes with E8M0 scale bytes stand for, float32."""
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, block))
    return (v * _pow2(scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _grouped_plain(st):
    """Every group padded to the largest one."""
    M, off = st["M"], st["offsets"].long()
    if st["kind"] == "grouped":
        x, w = st["x"].float(), st["w"].float()
    else:
        x, w = _values(st["x"], st["xs"], st["block"]), _values(st["w"], st["ws"], st["block"])
    at = (off[:-1, None] + torch.arange(st["most"], device=x.device)).clamp_max(M - 1)
    y = x[st["rows"].long()[at] if st["rows"] is not None else at] @ w.transpose(1, 2)
    if st["swiglu"]:
        gate, up = y.chunk(2, dim=2)
        y = gate / (1 + torch.exp(-gate)) * up
    i = torch.arange(M, device=x.device)
    e = torch.searchsorted(off[1:].contiguous(), i, right=True)
    return y[e, i - off[e]].bfloat16()


def _combine_plain(st):
    y = st["y"][st["slots"].long()].float()
    out = (y * st["w"][..., None]).sum(1)
    if st["r"] is not None:
        out = out + st["r"].float()
    return out.bfloat16()


def run(st):
    kind = st["kind"]
    if not own:
        return {"norm": _norm_plain, "route": _route_plain, "grouped": _grouped_plain, "grouped_mx": _grouped_plain,
                "combine": _combine_plain}[kind](st)
    import rmsnorm_linear_projection_gb300 as rnl
    if kind == "norm":
        s = torch.empty_like(st["x"]) if st["r"] is not None else None
        codes, scale = rnl.rnl_add_rmsnorm_mxfp8(st["x"], st["g"], residual=st["r"], x_sum_out=s, eps=EPS, block=st["block"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scale": scale.view(torch.float8_e8m0fnu), "sum": s}
    if kind == "route":
        r = rnl.rnl_moe_route(st["logits"], st["k"], renormalize=st["renorm"])
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "slots": r.slots}
    if kind == "grouped":
        return rnl.rnl_grouped_linear_bf16(st["x"], st["w"], st["offsets"], rows=st["rows"], swiglu=st["swiglu"])
    if kind == "grouped_mx":
        return rnl.rnl_grouped_linear_mxfp8(st["x"], st["xs"], st["w"], st["ws"], st["offsets"], rows=st["rows"],
                                            swiglu=st["swiglu"], block=st["block"])
    return rnl.rnl_moe_combine(st["y"], st["slots"], st["w"], residual=st["r"])


# ------------------------------------------------------------------- work
def work(case):
    T, kind = case["T"], case["kind"]
    if kind == "norm":
        n = T * case["K"]
        return {"bytes": n * (7 if case["residual"] else 3) + n // case["block"] + 2 * case["K"], "flops": 8 * n}
    if kind == "combine":
        n = T * case["N"]
        return {"bytes": 2 * n * (case["k"] + 1 + bool(case["residual"])) + 8 * T * case["k"], "flops": 2 * n * case["k"]}
    E, k = case["E"], case["k"]
    if kind == "route":
        return {"bytes": 4 * T * E + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    K, N, M = case["K"], case["N"], T * k
    # experts that get a row when every token takes k of E
    used = min(E, max(1, round(E * (1 - (1 - k / E) ** T))))
    size = 2.0 if kind == "grouped" else 1.0 + 1.0 / case["block"]
    width = N // 2 if case["swiglu"] else N
    return {"bytes": int(size * K * (used * N + (T if case["gather"] else M))) + 2 * M * width + 4 * (E + 1)
            + (4 * M if case["gather"] else 0), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ exact
def _exact_values(codes, scales, block):
    """Sign, exponent and fraction bits taken apart, in binary64."""
    c = codes.to(torch.float64)
    neg = torch.where(c >= 128, -1.0, 1.0).to(torch.float64)
    c = torch.remainder(c, 128)
    e = torch.floor(c / 8)
    f = c - 8 * e
    v = torch.where(e > 0, (1 + f / 8) * torch.exp2(e - 7), f * 2.0 ** -9)
    s = torch.exp2(scales.to(torch.float64) - 127)
    return neg * v * s.repeat_interleave(block, dim=-1)


def _exact_norm(st):
    x = st["x"].double()
    if st["r"] is not None:
        x = (x + st["r"].double()).to(torch.bfloat16).double()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    if st["g"] is not None:
        y = y * st["g"].double()
    T, K = y.shape
    b = y.reshape(T, K // st["block"], st["block"])
    top = b.abs().max(2, keepdim=True).values
    X = torch.where(top > 0, torch.floor(torch.log2(top)) - 8, torch.full_like(top, -127.0)).clamp(min=-127.0)
    v = b / torch.exp2(X)
    # spacing of E4M3 at v: 2^(floor(log2 |v|) - 3), 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    c = (torch.round(v / step) * step).clamp(-448.0, 448.0)
    return {"codes": c.reshape(T, K), "scale": torch.exp2(X).squeeze(2), "sum": x if st["r"] is not None else None}


def _exact_grouped(st):
    off = st["offsets"].tolist()
    out = []
    for e in range(st["E"]):
        a, b = off[e], off[e + 1]
        i = st["rows"][a:b].long() if st["rows"] is not None else slice(a, b)
        if st["kind"] == "grouped":
            x, w = st["x"][i].double(), st["w"][e].double()
        else:
            x = _exact_values(st["x"][i], st["xs"][i], st["block"])
            w = _exact_values(st["w"][e], st["ws"][e], st["block"])
        y = torch.einsum("mk,nk->mn", x, w)
        if st["swiglu"]:
            h = y.shape[1] // 2
            y = y[:, :h] * torch.sigmoid(y[:, :h]) * y[:, h:]
        out.append(y)
    return torch.cat(out)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        return _exact_norm(st)
    if kind in ("grouped", "grouped_mx"):
        return _exact_grouped(st)
    if kind == "combine":
        out = st["r"].double() if st["r"] is not None else 0
        for j in range(st["k"]):
            out = out + st["w"][:, j:j + 1].double() * st["y"][st["slots"][:, j].long()].double()
        return out
    l = st["logits"].double()
    p = torch.softmax(l, dim=1)
    p = torch.sort(p, dim=1, descending=True).values
    w = p[:, :st["k"]]
    return {"ids": None, "weights": w / w.sum(1, keepdim=True) if st["renorm"] else w, "offsets": None, "rows": None,
            "slots": None}
