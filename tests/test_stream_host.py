"""Calls with an explicit stream, on the host: everything that the binding
allocates for such a call (workspace and outputs) has to come from that
stream's memory.  A block of the current stream's pool goes back to that pool
when the call returns, and the next call or tensor gets it while the kernels on
the other stream still use it.

The library, the device check and torch.cuda.stream are replaced by recorders,
so that the allocations of every wrapper are seen without a GPU."""
import contextlib

import pytest
import torch

from rmsnorm_linear_projection_gb300 import _native as nat

BF, I8, U8, I32, F32 = torch.bfloat16, torch.int8, torch.uint8, torch.int32, torch.float32


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def kv4():
    return nat.Kv4Cache.empty(2, 1, 16, 64, 32, device="cpu"), z(3, 1, dtype=I32), z(3, dtype=I32)


def qkv():
    return (z(64), z(64), z(4, dtype=I32), z(8, 64, dtype=F32))


CALLS = {
    "rmsnorm_linear_bf16": lambda s: nat.rmsnorm_linear_bf16(z(4, 8), z(8), z(6, 8), stream=s),
    "rmsnorm_linear_bf16_ex": lambda s: nat.rmsnorm_linear_bf16_ex(z(4, 8), z(8), z(6, 8), stream=s),
    "rnl_qkv_rope": lambda s: nat.rnl_qkv_rope(z(4, 256), 2, 1, 64, *qkv(), stream=s),
    "rnl_qkv_rope_axes": lambda s: nat.rnl_qkv_rope_axes(z(4, 256), 2, 1, 64, None, None, z(1, 4, dtype=I32),
                                                         [0] * 32, z(8, 64, dtype=F32), stream=s),
    "rmsnorm_linear_qkv_rope": lambda s: nat.rmsnorm_linear_qkv_rope(z(4, 8), z(8), z(256, 8), 2, 1, 64, *qkv(),
                                                                    stream=s),
    "rnl_kv4_gather": lambda s: nat.rnl_kv4_gather(*kv4(), 3, stream=s),
    "rnl_kv4_attention": lambda s: nat.rnl_kv4_attention(z(3, 2, 64), *kv4(), stream=s),
    "quant_matmul_reduce_sum": lambda s: nat.quant_matmul_reduce_sum(z(2, 4, 8, dtype=I8), z(2, 8, 6, dtype=I8),
                                                                     z(2, 4, dtype=F32), z(6), stream=s),
    "rmsnorm_linear_w8a8": lambda s: nat.rmsnorm_linear_w8a8(z(4, 8), z(8), z(6, 8, dtype=I8), z(6, dtype=F32),
                                                             stream=s),
    "rnl_w8a8_prepare_weight": lambda s: nat.rnl_w8a8_prepare_weight(z(6, 8, dtype=I8), stream=s),
    "rmsnorm_linear_w8a8_prepared": lambda s: nat.rmsnorm_linear_w8a8_prepared(z(4, 8), z(8), z(6, 8),
                                                                              z(6, dtype=F32), stream=s),
    "rmsnorm_linear_mxfp8": lambda s: nat.rmsnorm_linear_mxfp8(z(4, 64), z(64), z(6, 64, dtype=U8),
                                                               z(6, 1, dtype=U8), stream=s),
    "mxfp8_scaled_mm": lambda s: nat.mxfp8_scaled_mm(z(4, 64, dtype=U8), z(4, 1, dtype=U8), z(6, 64, dtype=U8),
                                                     z(6, 1, dtype=U8), stream=s),
    "rnl_head_rmsnorm": lambda s: nat.rnl_head_rmsnorm(z(4, 128), 2, 64, stream=s),
    "mla_q_chain": lambda s: nat.mla_q_chain(z(4, 8), z(16, 8), z(16), z(6, 16), stream=s),
    "mla_q_chain_head_norm": lambda s: nat.mla_q_chain_head_norm(z(4, 8), z(16, 8), z(16), z(64, 16), 64, stream=s),
    "rmsnorm_linear_skinny_noalloc": lambda s: nat.rmsnorm_linear_skinny_noalloc(z(4, 8), z(6, 8), stream=s),
    "rnl_gemm_s8s8s32": lambda s: nat.rnl_gemm_s8s8s32(z(4, 16, dtype=I8), z(6, 16, dtype=I8), stream=s),
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

    def counting(f):
        def g(*a, **k):
            allocated.append(now[-1])
            return f(*a, **k)
        return g

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(nat, "load", lambda path=None: FakeLib())
    monkeypatch.setattr(nat, "_stream", lambda dev, stream: launched.append(stream))

    def call(f, stream):
        monkeypatch.setattr(torch, "empty", counting(torch.empty))
        monkeypatch.setattr(torch, "empty_like", counting(torch.empty_like))
        allocated.clear()
        f(stream)
        return list(allocated), list(launched)
    return call


@pytest.mark.parametrize("name", sorted(CALLS))
def test_what_a_call_allocates_belongs_to_its_stream(seen, name):
    kv4_cache = ("rnl_kv4_gather", "rnl_kv4_attention")
    s = FakeStream()
    allocated, launched = seen(CALLS[name], s)
    if name in kv4_cache:
        allocated = allocated[4:]  # the cache's own four tensors, made before the call
    assert launched == [s]
    assert allocated and all(a in (s, s.cuda_stream) for a in allocated), allocated


@pytest.mark.parametrize("name", sorted(CALLS))
def test_without_a_stream_the_current_one_is_used(seen, name):
    allocated, launched = seen(CALLS[name], None)
    assert launched == [None]
    assert allocated and all(a == "current" for a in allocated)


def test_every_wrapper_with_a_stream_is_covered():
    import inspect
    with_stream = {n for n, f in vars(nat).items() if inspect.isfunction(f) and not n.startswith("_") and
                   "stream" in inspect.signature(f).parameters}
    # these allocate nothing: the self-tests, the error word, a write into the caller's cache
    none = {"rnl_selftest_wait_timeout", "rnl_selftest_bounds_check", "rnl_check_device_error", "rnl_kv4_append"}
    assert with_stream == set(CALLS) | none
