"""The multi-axis RoPE stage and the 4-bit cache calls on the host, without a
GPU: workspace sizes and every refusal of their arguments, from the C entry
points and from the Python binding.

The C calls run in a child process with CUDA_VISIBLE_DEVICES="", so that on
any machine a call that passes the checks ends at the missing device."""
import json
import os
import subprocess
import sys
import textwrap

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, ARG, WORKSPACE, UNSUPPORTED, DEVICE = 0, 1, 2, 3, 4, 5, 8, 9

CHILD = textwrap.dedent("""
    import ctypes, json, sys
    sys.path.insert(0, {root!r})
    from rmsnorm_linear_projection_gb300 import _native as nat
    lib = nat.load()
    A, B, C = 0x10000, 0x10008, 0x10002      # fake addresses, never dereferenced
    r = {{}}

    def rope(name, y=A, T=4, Hq=2, Hkv=1, D=64, qg=A, kg=A, eps=1e-6, pos=A, axes=2, pairs=None, cs=A, P=8,
             q=A, k=A, v=A):
        pairs = bytes([0, 1] * (max(D, 0) // 4)) if pairs is None else pairs
        r["rope_" + name] = lib.rnl_qkv_rope_axes(y, T, Hq, Hkv, D, qg, kg, eps, pos, axes, pairs or None, cs, P,
                                                  q, k, v, None)

    rope("no_device")
    rope("no_gammas", qg=None, kg=None)
    rope("no_tokens", y=None, T=0, pos=None, cs=None, q=None, k=None, v=None)
    rope("only_q", Hkv=0, k=None, v=None)
    rope("neg_T", T=-1)
    rope("no_heads", Hq=0, Hkv=0)
    rope("no_positions_in_table", P=0)
    rope("too_many_heads", Hq=1 << 40)
    rope("head_dim_96", D=96)
    rope("bad_eps", eps=-1.0)
    rope("no_axes", axes=0)
    rope("five_axes", axes=5)
    rope("axis_out_of_range", axes=1)
    rope("null_pairs", pairs=b"")
    rope("null_y", y=None)
    rope("null_k", k=None)
    rope("null_positions", pos=None)
    rope("misaligned_table", cs=B)
    rope("misaligned_positions", pos=C)
    rope("misaligned_gamma", kg=B)

    def cache(kc=A, ks=A, vc=A, vs=A, P=4, H=2, S=16, D=64, block=32):
        return nat._Kv4CacheC(kc, ks, vc, vs, P, H, S, D, block)

    def seqs(t=A, n=A, cu=A, B=2, M=4, T=5):
        return nat._Kv4SeqsC(t, n, cu, B, M, T)

    structs = dict(
        no_device=({{}}, {{}}), one_row_each=({{}}, dict(cu=None, T=2)),
        no_rows=(dict(kc=None, ks=None, vc=None, vs=None), dict(t=None, n=None, cu=None, B=0, T=0)),
        no_pages=(dict(P=0), {{}}), neg_heads=(dict(H=-1), {{}}), many_heads=(dict(H=1 << 17), {{}}),
        head_dim_80=(dict(D=80), {{}}), block_16=(dict(block=16), {{}}), page_24=(dict(S=24), {{}}),
        page_8=(dict(S=8), {{}}), page_2048=(dict(S=2048), {{}}), long_table=({{}}, dict(M=1 << 27)),
        neg_seqs=({{}}, dict(B=-1)), many_seqs=({{}}, dict(B=(1 << 30) + 1)), rows_are_not_sequences=({{}}, dict(cu=None)), huge_rows=({{}}, dict(T=1 << 40)),
        null_codes=(dict(vc=None), {{}}), null_scales=(dict(ks=None), {{}}), null_lens=({{}}, dict(n=None)),
        null_table=({{}}, dict(t=None)), misaligned_codes=(dict(kc=B), {{}}), misaligned_scales=(dict(vs=B), {{}}),
        misaligned_table=({{}}, dict(t=C)), misaligned_lens=({{}}, dict(n=C)), misaligned_rows=({{}}, dict(cu=C)))
    big = 1 << 30

    def append(name, c, s, k=A, ks=128, v=A, vs=128):
        r["append_" + name] = lib.rnl_kv4_append(k, ks, v, vs, c, s, None)

    def gather(name, c, s, k=A, v=A):
        r["gather_" + name] = lib.rnl_kv4_gather(c, s, k, v, None)

    def attention(name, c, s, q=A, stride=256, Hq=4, scale=0.1, causal=1, window=0, out=A, lse=A, ws=A, size=big):
        r["attention_" + name] = lib.rnl_kv4_attention(q, stride, Hq, c, s, scale, causal, window, out, lse, ws,
                                                       size, None)

    for name, (c, s) in structs.items():
        for call in (append, gather, attention):
            call(name, cache(**c), seqs(**s))
    for call in (append, gather, attention):
        call("null_cache", None, seqs())
        call("null_seqs", cache(), None)
    c, s = cache(), seqs()
    append("null_k", c, s, k=None)
    append("null_v", c, s, v=None)
    append("short_stride", c, s, ks=120)
    append("odd_stride", c, s, vs=132)
    append("misaligned_v", c, s, v=B)
    gather("null_out", c, s, v=None)
    gather("misaligned_out", c, s, k=B)
    attention("no_lse", c, s, lse=None)
    attention("null_q", c, s, q=None)
    attention("null_out", c, s, out=None)
    attention("heads_do_not_divide", c, s, Hq=5)
    attention("no_heads", c, s, Hq=0)
    attention("short_stride", c, s, stride=248)
    attention("odd_stride", c, s, stride=260)
    attention("neg_window", c, s, window=-1)
    attention("window_without_causal", c, s, causal=0, window=3)
    attention("bad_causal", c, s, causal=2)
    attention("nan_scale", c, s, scale=float("nan"))
    attention("inf_scale", c, s, scale=float("inf"))
    attention("misaligned_q", c, s, q=B)
    attention("misaligned_out", c, s, out=B)
    attention("misaligned_lse", c, s, lse=C)
    attention("misaligned_ws", c, s, ws=B)
    attention("no_ws", c, s, ws=None)
    need = lib.rnl_workspace_size(8, 5, 64, 4, 2)
    attention("small_ws", c, s, size=need - 1)
    attention("enough_ws", c, s, size=need)
    r["ws"] = [lib.rnl_workspace_size(8, T, D, 8, 2) for D in (64, 128, 256) for T in (0, 1, 8, 9, 100000)]
    r["ws_bad"] = [lib.rnl_workspace_size(8, 1, 96, 8, 2), lib.rnl_workspace_size(8, 1, 64, 8, 3),
                   lib.rnl_workspace_size(8, 1, 64, 8, 0), lib.rnl_workspace_size(8, 1, 64, 0, 2)]
    print(json.dumps(r))
""")


@pytest.fixture(scope="module")
def results():
    from rmsnorm_linear_projection_gb300 import build
    build.build()
    p = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], capture_output=True, text=True,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), cwd=ROOT, timeout=300)
    assert p.returncode == 0, p.stderr
    return json.loads(p.stdout.strip().splitlines()[-1])


WANT = {
    "rope_no_device": DEVICE, "rope_no_gammas": DEVICE, "rope_only_q": DEVICE, "rope_no_tokens": OK,
    "rope_neg_T": SHAPE, "rope_no_heads": SHAPE, "rope_no_positions_in_table": SHAPE, "rope_too_many_heads": SHAPE,
    "rope_head_dim_96": UNSUPPORTED, "rope_bad_eps": ARG, "rope_no_axes": ARG, "rope_five_axes": ARG,
    "rope_axis_out_of_range": ARG, "rope_null_pairs": NULL, "rope_null_y": NULL, "rope_null_k": NULL,
    "rope_null_positions": NULL, "rope_misaligned_table": ALIGN, "rope_misaligned_positions": ALIGN,
    "rope_misaligned_gamma": ALIGN,
    "append_null_k": NULL, "append_null_v": NULL, "append_short_stride": SHAPE, "append_odd_stride": ALIGN,
    "append_misaligned_v": ALIGN, "gather_null_out": NULL, "gather_misaligned_out": ALIGN,
    "attention_no_lse": DEVICE, "attention_enough_ws": DEVICE, "attention_null_q": NULL, "attention_null_out": NULL,
    "attention_heads_do_not_divide": SHAPE, "attention_no_heads": SHAPE, "attention_short_stride": SHAPE,
    "attention_odd_stride": ALIGN, "attention_neg_window": SHAPE, "attention_window_without_causal": ARG,
    "attention_bad_causal": ARG, "attention_nan_scale": ARG, "attention_inf_scale": ARG,
    "attention_misaligned_q": ALIGN, "attention_misaligned_out": ALIGN, "attention_misaligned_lse": ALIGN,
    "attention_misaligned_ws": ALIGN, "attention_no_ws": WORKSPACE, "attention_small_ws": WORKSPACE,
}
for _call in ("append", "gather", "attention"):
    WANT.update({f"{_call}_{_k}": _v for _k, _v in {
        "no_device": DEVICE, "one_row_each": DEVICE, "no_rows": OK, "no_pages": SHAPE, "neg_heads": SHAPE,
        "many_heads": SHAPE, "head_dim_80": UNSUPPORTED, "block_16": ARG, "page_24": UNSUPPORTED,
        "page_8": UNSUPPORTED, "page_2048": UNSUPPORTED, "long_table": SHAPE, "neg_seqs": SHAPE, "many_seqs": SHAPE,
        "rows_are_not_sequences": SHAPE, "huge_rows": SHAPE, "null_codes": NULL, "null_scales": NULL,
        "null_lens": NULL, "null_table": NULL, "misaligned_codes": ALIGN, "misaligned_scales": ALIGN,
        "misaligned_table": ALIGN, "misaligned_lens": ALIGN, "misaligned_rows": ALIGN, "null_cache": NULL,
        "null_seqs": NULL}.items()})


@pytest.mark.parametrize("key", sorted(WANT))
def test_argument_checks(results, key):
    assert results[key] == WANT[key]


def test_every_call_is_expected(results):
    assert sorted(k for k in results if not k.startswith("ws")) == sorted(WANT)


def test_workspace_sizes(results):
    ws = results["ws"]
    for i in range(0, 15, 5):
        none, one, eight, nine, many = ws[i:i + 5]
        assert 0 < none == one == eight and eight % 16 == 0
        assert nine == many and (nine > one if i < 10 else nine == one)  # many rows: another kernel up to D = 128
    assert all(x == 2 ** 64 - 1 for x in results["ws_bad"])


# ------------------------------------------------------------ the Python binding
def _cache(**kw):
    from rmsnorm_linear_projection_gb300 import Kv4Cache
    a = dict(P=4, H=2, S=16, D=64, block=32)
    a.update(kw)
    return Kv4Cache.empty(a["P"], a["H"], a["S"], a["D"], a["block"], device="cpu")


def test_cache_tensors_are_checked():
    from rmsnorm_linear_projection_gb300 import Kv4Cache
    c = _cache()
    assert (c.n_pages, c.n_kv_heads, c.page_size, c.head_dim, c.block) == (4, 2, 16, 64, 32)
    good = [c.k_codes, c.k_scales, c.v_codes, c.v_scales]
    for i in range(4):
        for wrong, err in ((good[i].to(torch.int8), TypeError), (good[i][:2], ValueError),
                           (good[i].transpose(0, 1), ValueError), (good[i].flatten(), ValueError)):
            with pytest.raises(err):
                Kv4Cache(*[wrong if j == i else x for j, x in enumerate(good)])


def test_binding_refuses_wrong_tensors():
    import rmsnorm_linear_projection_gb300 as rnl
    c = _cache()
    i32 = dict(dtype=torch.int32)
    table, lens, cu = torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(3, **i32)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    for f in (lambda x, *a: rnl.rnl_kv4_append(x, x, *a), lambda x, *a: rnl.rnl_kv4_append(k, x, *a)):
        with pytest.raises(TypeError):
            f(k.float(), c, table, lens, cu)
        with pytest.raises(ValueError):
            f(k[:, :1], c, table, lens, cu)
        with pytest.raises(ValueError):
            f(torch.zeros(5, 64, 2, dtype=torch.bfloat16).transpose(1, 2), c, table, lens, cu)
    calls = (lambda *a: rnl.rnl_kv4_append(k, k, c, *a), lambda *a: rnl.rnl_kv4_attention(q, c, *a),
             lambda t, n, u: rnl.rnl_kv4_gather(c, t, n, 5, u))
    for f in calls:
        for t, n, u, err in ((table.long(), lens, cu, TypeError), (table, lens.long(), cu, TypeError),
                             (table, lens, cu.long(), TypeError), (table[:1], lens, cu, ValueError),
                             (table, lens, cu[:2], ValueError), (table.t().contiguous().t(), lens, cu, ValueError),
                             (table, torch.zeros(4, **i32)[::2], cu, ValueError)):
            with pytest.raises(err):
                f(t, n, u)
        with pytest.raises(ValueError, match="CUDA device"):
            f(table, lens, cu)
    for kw, err in ((dict(out=q.float()), TypeError), (dict(out=q[:4]), ValueError),
                    (dict(lse_out=torch.zeros(5, 4, dtype=torch.bfloat16)), TypeError),
                    (dict(lse_out=torch.zeros(5, 3)), ValueError)):
        with pytest.raises(err):
            rnl.rnl_kv4_attention(q, c, table, lens, cu, **kw)
    with pytest.raises(ValueError):
        rnl.rnl_kv4_gather(c, table, lens, 5, cu, k_out=torch.zeros(4, 2, 64, dtype=torch.bfloat16))


def test_rope_binding_refuses_wrong_tensors():
    import rmsnorm_linear_projection_gb300 as rnl
    bf = dict(dtype=torch.bfloat16)
    a = dict(y=torch.zeros(3, 4 * 64, **bf), n_q_heads=2, n_kv_heads=1, head_dim=64, q_gamma=torch.ones(64, **bf),
             k_gamma=None, positions=torch.zeros(2, 3, dtype=torch.int32), axis_of_pair=[0] * 32,
             cos_sin=torch.zeros(8, 64))
    for kw, err in ((dict(y=a["y"].half()), TypeError), (dict(y=a["y"][:2]), ValueError),
                    (dict(y=torch.zeros(4 * 64, 3, **bf).t()), ValueError), (dict(q_gamma=torch.ones(64)), TypeError),
                    (dict(positions=torch.zeros(2, 3)), TypeError), (dict(positions=a["positions"][:, :2]), ValueError),
                    (dict(axis_of_pair=[0] * 31), ValueError), (dict(axis_of_pair=32), TypeError),
                    (dict(axis_of_pair=[0] * 31 + [256]), ValueError), (dict(axis_of_pair=[0] * 31 + [-1]), ValueError),
                    (dict(cos_sin=torch.zeros(8, 32)), ValueError), (dict(cos_sin=torch.zeros(8, 64, **bf)), TypeError),
                    (dict(q_out=torch.zeros(3, 1, 64, **bf)), ValueError)):
        with pytest.raises(err):
            rnl.rnl_qkv_rope_axes(**dict(a, **kw))
    with pytest.raises(ValueError, match="CUDA device"):
        rnl.rnl_qkv_rope_axes(**a)
