"""Plain 64-bit implementations of the multi-axis RoPE stage, the 4-bit paged KV
cache and attention over it, and the tolerances that follow from the kernels'
arithmetic.  Slow and direct: loops over sequences and heads, whole score
matrices.

Attention's bound, per output element (ref = sum p v / l exactly, A = sum p |v| / l):
  * the output is rounded to bf16 once: 2^-8 |ref|;
  * each weight is rounded to binary16: at most 2^-11 of it, so 2^-11 A;
  * each score is an FP32 sum of D exact products: an error of at most
    D 2^-23 scale sum_d |q_d k_d| (accumulation that truncates), which moves
    its weight and the normaliser by as much each: 2 delta A;
  * exp2 and the FP32 sums: a few 2^-22, counted as 2^-18 A;
  * operands below 2^-37 of the largest in the sequence may vanish:
    2^-36 max|v|.
lse: delta + 2^-20 max(1, |lse|).
"""
import math

import torch

LEVELS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def pow2(e):
    """2^e in float64 for integer tensors e, from its bits (pow and ldexp may be a unit off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantise(x, block):
    """x [..., D] (any finite values) -> codes uint8 [..., D / 2], scale bytes [..., D / block]."""
    b = x.double().unflatten(-1, (-1, block))
    amax = b.abs().amax(-1)
    _, e = torch.frexp(amax)
    X = torch.where(amax > 0, e - 3, torch.full_like(e, -127)).clamp_min(-127)
    y = b * pow2(-X).unsqueeze(-1)
    a = y.abs().unsqueeze(-1)
    L = LEVELS.to(x.device)
    mid = (L[1:] + L[:-1]) / 2
    even_above = torch.arange(1, 8, device=x.device) % 2 == 0     # a tie goes to the even code
    code = ((a > mid) | ((a == mid) & even_above)).sum(-1)
    code = (code + 8 * torch.signbit(y).long()).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (X + 127).to(torch.uint8)


def values(codes, scales):
    """float64 [..., D]; scale byte 255 reads as an infinite scale."""
    D = codes.shape[-1] * 2
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = LEVELS.to(codes.device)[c & 7] * torch.where(c >= 8, -1.0, 1.0).double()
    p = pow2(scales.long() - 127)
    p = torch.where(scales == 255, torch.full_like(p, math.inf), p)
    return v * p.repeat_interleave(D // scales.shape[-1], -1)


def rope_axes(y, Hq, Hkv, D, q_gamma, k_gamma, positions, axis_of_pair, cos_sin, eps):
    """(q, k, v) in float64 before the final rounding, and |z| terms for the bound."""
    T = y.shape[0]
    h = y.double().reshape(T, Hq + 2 * Hkv, D)
    half = D // 2
    i = torch.arange(half, device=y.device)
    pos = positions.long()[torch.tensor(list(axis_of_pair), device=y.device)].t()
    c, s = cos_sin.double()[pos, i][:, None], cos_sin.double()[pos, half + i][:, None]
    outs, mags = [], []
    for lo, hi, g in ((0, Hq, q_gamma), (Hq, Hq + Hkv, k_gamma)):
        z = h[:, lo:hi]
        if g is not None:
            z = (z * torch.rsqrt((z * z).mean(-1, keepdim=True) + eps) * g.double()).bfloat16().double()
        a, b = z[..., :half], z[..., half:]
        outs.append(torch.cat([a * c - b * s, b * c + a * s], -1))
        mags.append(torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1))
    return outs[0], outs[1], h[:, Hq + Hkv:], mags[0], mags[1]


def sequence(cache, table_row, n, head):
    """(k, v) float64 [n, D] of one head of one sequence."""
    pages = table_row.long()[torch.arange(n, device=table_row.device) // cache.page_size]
    off = torch.arange(n, device=table_row.device) % cache.page_size
    return tuple(values(c[pages, head, off], s[pages, head, off])
                 for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)))


def attention(q, cache, block_table, seq_lens, cu_rows=None, scale=None, causal=True, window=0):
    """(out, lse, bound of out, bound of lse) in float64; rows outside every
    sequence are NaN."""
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    lens = seq_lens.tolist()
    cu = list(range(len(lens) + 1)) if cu_rows is None else cu_rows.tolist()
    G = Hq // cache.n_kv_heads
    new = lambda *s: torch.full(s, math.nan, dtype=torch.float64, device=q.device)  # noqa: E731
    out, lse, tol, ltol = new(T, Hq, D), new(T, Hq), new(T, Hq, D), new(T, Hq)
    for b, n in enumerate(lens):
        r = cu[b + 1] - cu[b]
        if r == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        if n == 0:
            out[rows], lse[rows], tol[rows], ltol[rows] = 0, -math.inf, 0, 0
            continue
        pos = torch.arange(n - r, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        see = (j <= pos) if causal else torch.ones(r, n, dtype=torch.bool, device=q.device)
        if window:
            see = see & (j > pos - window)
        for h in range(Hq):
            if h % G == 0:
                k, v = sequence(cache, block_table[b], n, h // G)
            qd = q[rows, h].double()
            s = (qd @ k.t() * scale).masked_fill(~see, -math.inf)
            m = s.amax(-1, keepdim=True).clamp_min(-1e300)
            p = torch.exp(s - m)
            l = p.sum(-1, keepdim=True)
            ll = torch.where(l > 0, l, torch.ones_like(l))
            o = p @ v / ll
            out[rows, h] = o
            lse[rows, h] = torch.where(l > 0, m + torch.log(ll), torch.full_like(l, -math.inf))[:, 0]
            delta = D * 2.0 ** -23 * abs(scale) * (qd.abs() @ k.abs().t())
            delta = torch.where(see, delta, torch.zeros_like(delta)).amax(-1, keepdim=True)
            tol[rows, h] = (2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -18 + 2 * delta) * (p @ v.abs() / ll) +
                            2.0 ** -36 * v.abs().max())
            ltol[rows, h] = delta[:, 0] + 2.0 ** -20 * lse[rows, h].abs().clamp(1, 1e30)
    return out, lse, tol, ltol
