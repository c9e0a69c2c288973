"""The expert layer's calls on the host, without a GPU: workspace sizes, every
refusal of the C entry points and of the binding, and that what a call with an
explicit stream allocates belongs to that stream.

The C calls run in a child process with CUDA_VISIBLE_DEVICES="", so that on any
machine a call that passes the checks ends at the missing device."""
import contextlib
import inspect
import json
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from rmsnorm_linear_projection_gb300 import _experts as ex
from rmsnorm_linear_projection_gb300 import _native as nat

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, ARG, WORKSPACE, UNSUPPORTED, DEVICE = 0, 1, 2, 3, 4, 5, 8, 9

CHILD = textwrap.dedent("""
    import json, sys
    sys.path.insert(0, {root!r})
    from rmsnorm_linear_projection_gb300 import _native as nat
    lib = nat.load()
    A, B, C = 0x100000, 0x100008, 0x100002      # fake addresses, never dereferenced
    far = 1 << 40
    r = {{}}

    def norm(name, x=A, res=None, s=None, g=A, T=4, K=128, eps=1e-6, mode=0, block=64, codes=A, scale=C):
        r["norm_" + name] = lib.rnl_add_rmsnorm_mxfp8(x, res, s, g, T, K, eps, mode, block, codes, scale, None)
    norm("no_device")
    norm("no_rows", x=None, T=0, codes=None, scale=None)
    norm("no_gamma", g=None)
    norm("in_place", res=far, s=far)
    norm("sum_disjoint", res=far, s=2 * far)
    norm("sum_overlaps", res=far, s=far + 16)
    norm("sum_overlaps_x", res=far, s=A + 128)
    norm("sum_without_residual", s=far)
    norm("neg_T", T=-1)
    norm("no_K", K=0)
    norm("K_not_blocks", K=96)
    norm("K_blocks_of_32", K=96, block=32)
    norm("long_K", K=65536 + 64)
    norm("block_16", block=16)
    norm("bad_mode", mode=2)
    norm("bad_eps", eps=float("nan"))
    norm("null_x", x=None)
    norm("null_scale", scale=None)
    norm("misaligned_x", x=B)
    norm("misaligned_codes", codes=B)
    norm("misaligned_residual", res=B)

    def quant(name, x=A, T=4, K=128, block=64, codes=A, scale=C):
        r["quant_" + name] = lib.rnl_quant_mxfp8(x, T, K, block, codes, scale, None)
    quant("no_device")
    quant("no_rows", x=None, T=0)
    quant("block_0", block=0)
    quant("K_not_blocks", K=160)
    quant("long_K", K=1 << 17)
    quant("null_codes", codes=None)
    quant("misaligned_x", x=B)

    def route(name, l=A, T=4, E=8, k=2, renorm=1, ids=A, w=A, off=A, rows=A, slots=A, ws=None, size=0):
        r["route_" + name] = lib.rnl_moe_route(l, T, E, k, renorm, ids, w, off, rows, slots, ws, size, None)
    route("no_device")
    route("no_tokens", l=None, T=0, ids=None, w=None, rows=None, slots=None)
    route("no_tokens_no_offsets", T=0, off=None)
    route("no_experts", E=0)
    route("k_0", k=0)
    route("k_over_E", k=9)
    route("k_33", E=64, k=33)
    route("E_1025", E=1025)
    route("many_rows", T=1 << 30, k=4)
    route("bad_flag", renorm=2)
    route("null_logits", l=None)
    route("null_slots", slots=None)
    route("misaligned_ids", ids=C)
    route("many_tokens_no_workspace", T=65)
    route("many_tokens_small_workspace", T=65, ws=A, size=63)
    route("many_tokens", T=65, ws=A, size=64)

    def combine(name, y=A, M=8, N=64, slots=A, w=A, T=4, k=2, res=None, out=far, ):
        r["combine_" + name] = lib.rnl_moe_combine(y, M, N, slots, w, T, k, res, out, None)
    combine("no_device")
    combine("no_tokens", T=0, out=None)
    combine("nothing_to_add", M=0, y=None, k=0, slots=None, w=None)
    combine("N_60", N=60)
    combine("no_N", N=0)
    combine("neg_M", M=-1)
    combine("null_y", y=None)
    combine("null_slots", slots=None)
    combine("null_out", out=None)
    combine("in_place", res=far)
    combine("overlaps_residual", res=far + 16)
    combine("overlaps_y", out=A + 128)
    combine("misaligned_out", out=far + 8)
    combine("misaligned_weights", w=C)
    combine("huge", T=1 << 30, k=1, N=1 << 20)

    big = 1 << 30
    def g(name, x=A, R=8, W=A, E=4, N=64, K=64, off=A, rows=None, M=8, sw=0, out=A, ws=A, size=big):
        r["g_" + name] = lib.rnl_grouped_linear_bf16(x, R, W, E, N, K, off, rows, M, sw, out, ws, size, None)
        r["mx_" + name] = lib.rnl_grouped_linear_mxfp8(x, C, R, W, C, E, N, K, 32, off, rows, M, sw, out, ws, size, None)
    g("no_device")
    g("gathered", R=3, rows=A)
    g("no_rows", x=None, W=None, R=0, M=0, off=None, out=None, ws=None, size=0)
    g("rows_of_nothing", R=0, rows=A)
    g("M_is_not_R", M=7)
    g("neg_R", R=-1, rows=A)
    g("no_experts", E=0)
    g("E_1025", E=1025)
    g("no_N", N=0)
    g("no_K", K=0)
    g("huge_EN", E=1024, N=1 << 22)
    g("huge_K", K=(1 << 24) + 32)
    g("huge_M", R=(1 << 30) + 1, M=(1 << 30) + 1)
    g("huge_tiles", R=1 << 29, M=1 << 29, N=1 << 18)
    g("N_48_swiglu", N=48, sw=1)
    g("swiglu", sw=1)
    g("bad_flag", sw=2)
    g("null_x", x=None)
    g("null_W", W=None)
    g("null_offsets", off=None)
    g("null_out", out=None)
    g("null_workspace", ws=None)
    g("small_workspace", size=1000)
    g("misaligned_x", x=B)
    g("misaligned_W", W=B)
    g("misaligned_out", out=B)
    g("misaligned_offsets", off=C)
    g("misaligned_rows", rows=C)
    g("K_not_multiple", K=36)
    def mx(name, xs=C, ws=C, K=64, block=64):
        r["mx_" + name] = lib.rnl_grouped_linear_mxfp8(A, xs, 8, A, ws, 4, 64, K, block, A, None, 8, 0, A, A, big, None)
    mx("null_x_scale", xs=None)
    mx("null_w_scale", ws=None)
    mx("block_48", block=48)
    mx("K_96_block_64", K=96)
    for name, a in dict(grouped=(10, 8, 64, 64, 4), route=(11, 1000, 2, 128, 0), route_few=(11, 64, 8, 128, 0),
                        nine=(9, 1, 8, 8, 0)).items():
        r["ws_" + name] = lib.rnl_workspace_size(*a)
    print(json.dumps(r))
""")

REFUSALS = {
    "norm": dict(no_device=DEVICE, no_rows=OK, no_gamma=DEVICE, in_place=DEVICE, sum_disjoint=DEVICE, sum_overlaps=ARG,
                 sum_overlaps_x=ARG, sum_without_residual=ARG, neg_T=SHAPE, no_K=SHAPE, K_not_blocks=SHAPE,
                 K_blocks_of_32=DEVICE, long_K=UNSUPPORTED, block_16=ARG, bad_mode=ARG, bad_eps=ARG, null_x=NULL,
                 null_scale=NULL, misaligned_x=ALIGN, misaligned_codes=ALIGN, misaligned_residual=ALIGN),
    "quant": dict(no_device=DEVICE, no_rows=OK, block_0=ARG, K_not_blocks=SHAPE, long_K=UNSUPPORTED, null_codes=NULL,
                  misaligned_x=ALIGN),
    "route": dict(no_device=DEVICE, no_tokens=DEVICE, no_tokens_no_offsets=NULL, no_experts=SHAPE, k_0=SHAPE,
                  k_over_E=SHAPE, k_33=UNSUPPORTED, E_1025=UNSUPPORTED, many_rows=SHAPE, bad_flag=ARG, null_logits=NULL,
                  null_slots=NULL, misaligned_ids=ALIGN, many_tokens_no_workspace=WORKSPACE,
                  many_tokens_small_workspace=WORKSPACE, many_tokens=DEVICE),
    "combine": dict(no_device=DEVICE, no_tokens=OK, nothing_to_add=DEVICE, N_60=ALIGN, no_N=SHAPE, neg_M=SHAPE,
                    null_y=NULL, null_slots=NULL, null_out=NULL, in_place=DEVICE, overlaps_residual=ARG,
                    overlaps_y=ARG, misaligned_out=ALIGN, misaligned_weights=ALIGN, huge=SHAPE),
    "g": dict(no_device=DEVICE, gathered=DEVICE, no_rows=OK, rows_of_nothing=SHAPE, M_is_not_R=SHAPE, neg_R=SHAPE,
              no_experts=SHAPE, E_1025=UNSUPPORTED, no_N=SHAPE, no_K=SHAPE, huge_EN=SHAPE, huge_K=SHAPE, huge_M=SHAPE, huge_tiles=SHAPE,
              N_48_swiglu=UNSUPPORTED, swiglu=DEVICE, bad_flag=ARG, null_x=NULL, null_W=NULL, null_offsets=NULL,
              null_out=NULL, null_workspace=WORKSPACE, small_workspace=WORKSPACE, misaligned_x=ALIGN,
              misaligned_W=ALIGN, misaligned_out=ALIGN, misaligned_offsets=ALIGN, misaligned_rows=ALIGN,
              K_not_multiple=ALIGN),
}
REFUSALS["mx"] = dict(REFUSALS["g"], K_not_multiple=SHAPE, null_x_scale=NULL, null_w_scale=NULL, block_48=ARG,
                      K_96_block_64=SHAPE)


@pytest.fixture(scope="module")
def results():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    p = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], capture_output=True, text=True, cwd=ROOT,
                       env=env, timeout=300)
    assert p.returncode == 0, p.stderr
    return json.loads(p.stdout.splitlines()[-1])


@pytest.mark.parametrize("key,want", [(f"{c}_{n}", v) for c, d in REFUSALS.items() for n, v in d.items()])
def test_status(results, key, want):
    assert results[key] == want


def test_every_status_is_expected(results):
    assert {k for k in results if not k.startswith("ws_")} == {f"{c}_{n}" for c, d in REFUSALS.items() for n in d}


def test_workspace_sizes(results):
    assert results["ws_grouped"] == 128 * 2 * 128 * 256 * 4          # partial sums of the CTA pairs and their flags
    assert results["ws_route"] == 16 * 128 * 4                       # the experts' counts of 16 CTAs of 64 tokens
    assert results["ws_route_few"] == 0
    assert results["ws_nine"] == (1 << 64) - 1                       # 9 is no operation


# ------------------------------------------------------------------ binding
BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


CALLS = {
    "rnl_add_rmsnorm_mxfp8": lambda s: ex.rnl_add_rmsnorm_mxfp8(z(4, 64), stream=s),
    "rnl_quant_mxfp8": lambda s: ex.rnl_quant_mxfp8(z(4, 64), stream=s),
    "rnl_moe_route": lambda s: ex.rnl_moe_route(z(4, 8, dtype=F32), 2, stream=s),
    "rnl_grouped_linear_bf16": lambda s: ex.rnl_grouped_linear_bf16(z(4, 8), z(2, 6, 8), z(3, dtype=I32), stream=s),
    "rnl_grouped_linear_mxfp8": lambda s: ex.rnl_grouped_linear_mxfp8(
        z(4, 64, dtype=U8), z(4, 1, dtype=U8), z(2, 6, 64, dtype=U8), z(2, 6, 1, dtype=U8), z(3, dtype=I32), stream=s),
    "rnl_moe_combine": lambda s: ex.rnl_moe_combine(z(8, 16), z(4, 2, dtype=I32), z(4, 2, dtype=F32), stream=s),
}


class FakeStream:
    cuda_stream = 1234


class FakeLib:
    def __getattr__(self, name):
        return (lambda *a: 4096) if name == "rnl_workspace_size" else (lambda *a: 0)


@pytest.fixture
def seen(monkeypatch):
    """(where the allocations of a call were made, on which stream it was launched)."""
    now, allocated, launched = ["current"], [], []

    @contextlib.contextmanager
    def use(stream):
        now.append(stream)
        try:
            yield
        finally:
            now.pop()

    empty = torch.empty

    def counting(*a, **k):
        allocated.append(now[-1])
        return empty(*a, **k)

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(nat, "load", lambda path=None: FakeLib())
    monkeypatch.setattr(nat, "_lib", None)
    monkeypatch.setattr(ex, "_workspace_size", nat.workspace_size)  # not remembered
    monkeypatch.setattr(nat, "_stream", lambda dev, stream: launched.append(stream))

    def call(f, stream):
        monkeypatch.setattr(torch, "empty", counting)
        f(stream)
        return allocated, launched
    return call


@pytest.mark.parametrize("name", sorted(CALLS))
def test_what_a_call_allocates_belongs_to_its_stream(seen, name):
    s = FakeStream()
    allocated, launched = seen(CALLS[name], s)
    assert launched == [s]
    assert allocated and all(a in (s, s.cuda_stream) for a in allocated), allocated


@pytest.mark.parametrize("name", sorted(CALLS))
def test_without_a_stream_the_current_one_is_used(seen, name):
    allocated, launched = seen(CALLS[name], None)
    assert launched == [None]
    assert allocated and all(a == "current" for a in allocated)


def test_every_wrapper_is_covered_and_public():
    import rmsnorm_linear_projection_gb300 as rnl
    wrappers = {n for n, f in vars(ex).items() if inspect.isfunction(f) and not n.startswith("_")}
    assert wrappers == set(CALLS)
    assert all(getattr(rnl, n) is getattr(ex, n) for n in wrappers)
    assert wrappers <= set(rnl.EXPORTS)


def test_outputs_of_small_calls(monkeypatch):
    monkeypatch.setattr(nat, "load", lambda path=None: FakeLib())
    monkeypatch.setattr(nat, "_lib", None)
    monkeypatch.setattr(ex, "_workspace_size", nat.workspace_size)
    monkeypatch.setattr(nat, "_stream", lambda dev, stream: None)
    r = ex.rnl_moe_route(z(5, 7, dtype=F32), 3)
    for i, t in enumerate(r):
        t.fill_(i + 1)
    assert [t.shape for t in r] == [(5, 3), (5, 3), (8,), (15,), (5, 3)]
    assert all((t == i + 1).all() and t.is_contiguous() for i, t in enumerate(r))
    c, s = ex.rnl_quant_mxfp8(z(3, 128), block=32)
    c.fill_(1)
    s.fill_(2)
    assert (c == 1).all() and (s == 2).all() and c.shape == (3, 128) and s.shape == (3, 4)


@pytest.mark.parametrize("call,error", [
    (lambda: ex.rnl_add_rmsnorm_mxfp8(z(4, 64, dtype=F32)), TypeError),
    (lambda: ex.rnl_add_rmsnorm_mxfp8(z(4, 128)[:, :64]), ValueError),
    (lambda: ex.rnl_add_rmsnorm_mxfp8(z(4, 64), residual=z(3, 64)), ValueError),
    (lambda: ex.rnl_add_rmsnorm_mxfp8(z(4, 64), gamma=z(32)), ValueError),
    (lambda: ex.rnl_quant_mxfp8(z(4, 64), codes_out=z(4, 64, dtype=torch.int8)), TypeError),
    (lambda: ex.rnl_quant_mxfp8(z(4, 64), block=32, scale_out=z(4, 1, dtype=U8)), ValueError),
    (lambda: ex.rnl_moe_route(z(4, 8), 2), TypeError),
    (lambda: ex.rnl_moe_route(z(4, 8, dtype=F32), 2, ids_out=z(4, 3, dtype=I32)), ValueError),
    (lambda: ex.rnl_grouped_linear_bf16(z(4, 8), z(2, 6, 16), z(3, dtype=I32)), ValueError),
    (lambda: ex.rnl_grouped_linear_bf16(z(4, 8), z(2, 6, 8), z(2, dtype=I32)), ValueError),
    (lambda: ex.rnl_grouped_linear_bf16(z(4, 8), z(2, 6, 8), z(3, dtype=torch.int64)), TypeError),
    (lambda: ex.rnl_grouped_linear_bf16(z(4, 8), z(2, 6, 8), z(3, dtype=I32), rows=z(9)), TypeError),
    (lambda: ex.rnl_grouped_linear_bf16(z(4, 8), z(2, 6, 8), z(3, dtype=I32), swiglu=True, out=z(4, 6)), ValueError),
    (lambda: ex.rnl_grouped_linear_mxfp8(z(4, 64, dtype=U8), z(4, 2, dtype=U8), z(2, 6, 64, dtype=U8),
                                         z(2, 6, 1, dtype=U8), z(3, dtype=I32)), ValueError),
    (lambda: ex.rnl_moe_combine(z(8, 16), z(4, 2, dtype=I32), z(4, 3, dtype=F32)), ValueError),
    (lambda: ex.rnl_moe_combine(z(8, 16), z(4, 2, dtype=I32), z(4, 2)), TypeError),
])
def test_binding_refuses(call, error):
    with pytest.raises(error):
        call()
