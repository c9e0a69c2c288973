"""Calls with an explicit stream (stream=s) on the GPU: several of them in flight
at once from one current stream, each with the workspace and the outputs that
the binding allocates for it, give the bits of the calls alone."""
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


def attention_jobs(g):
    """Steps, drafts and prompts over a cache of random blocks (scale bytes of ordinary values)."""
    jobs = []
    for lens, rows, D in (([5000] * 6, [1] * 6, 128), ([2500, 40, 3000], [1, 1, 1], 64),
                          ([3000, 700], [900, 300], 128), ([2000] * 3, [4] * 3, 64)):
        H, page = 2, 64
        need = [-(-n // page) for n in lens]
        c = rnl.Kv4Cache.empty(sum(need), H, page, D, 32)
        for t, lo, hi in ((c.k_codes, 0, 256), (c.v_codes, 0, 256), (c.k_scales, 122, 127), (c.v_scales, 122, 127)):
            t.copy_(torch.randint(lo, hi, t.shape, generator=g, device="cuda"))
        table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.arange(at, at + n, device="cuda")
            at += n
        cu = [0]
        for r in rows:
            cu.append(cu[-1] + r)
        q = torch.randn(cu[-1], 8, D, generator=g, device="cuda").bfloat16()
        i32 = dict(dtype=torch.int32, device="cuda")
        jobs.append((q, c, table, torch.tensor(lens, **i32), torch.tensor(cu, **i32)))
    return jobs


def test_attention_on_given_streams():
    jobs = attention_jobs(torch.Generator(device="cuda").manual_seed(4))
    want = [rnl.rnl_kv4_attention(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        got = []
        for _ in range(6):
            got += [rnl.rnl_kv4_attention(*j, stream=s) for j, s in zip(jobs, streams)]
            # tensors of the current stream in between: they must not share a call's memory
            torch.full((1 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        rnl.rnl_check_device_error()
        for i, o in enumerate(got):
            assert torch.equal(o, want[i % len(jobs)])


def test_projections_on_given_streams():
    g = torch.Generator(device="cuda").manual_seed(5)
    jobs = []
    for T, K, N in ((700, 1024, 1536), (300, 2048, 520), (4, 4096, 2048)):
        x, W = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((T, K), (N, K)))
        gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
        Wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda").to(torch.int8)
        scale = torch.full((N,), 1 / (127 * math.sqrt(K)), device="cuda")
        jobs.append(lambda s, a=(x, gamma, W): rnl.rmsnorm_linear_bf16(*a, stream=s))
        jobs.append(lambda s, a=(x, gamma, Wq, scale): rnl.rmsnorm_linear_w8a8(*a, stream=s))
    want = [f(None) for f in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        got = []
        for _ in range(4):
            got += [f(s) for f, s in zip(jobs, streams)]
            torch.full((1 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        rnl.rnl_check_device_error()
        for i, o in enumerate(got):
            assert torch.equal(o, want[i % len(jobs)])


def test_an_output_does_not_take_memory_that_is_still_in_use():
    """A block that the current stream has freed but not finished with goes to no
    call on another stream."""
    jobs = attention_jobs(torch.Generator(device="cuda").manual_seed(6))
    q = jobs[0]
    want = rnl.rnl_kv4_attention(*q)
    s = torch.cuda.Stream()
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        old = torch.empty_like(want)
        for _ in range(6):
            big.add_(1)  # about 2 GB of traffic each: the fill below runs well after the call
        old.fill_(320.0)
        del old
        out = rnl.rnl_kv4_attention(*q, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_a_handle_of_another_library_is_a_stream_too():
    """Any object with a cuda_stream attribute, as before."""
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    job = attention_jobs(torch.Generator(device="cuda").manual_seed(7))[1]
    want = rnl.rnl_kv4_attention(*job)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = rnl.rnl_kv4_attention(*job, stream=Handle(s))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_captured_calls_on_given_streams():
    """Calls on the capturing stream and on one forked from it, inside one graph."""
    jobs = attention_jobs(torch.Generator(device="cuda").manual_seed(8))
    want = [rnl.rnl_kv4_attention(*j) for j in jobs]
    torch.cuda.synchronize()
    side, fork = torch.cuda.Stream(), torch.cuda.Stream()
    graph, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph, stream=side):
        fork.wait_stream(side)
        for i, j in enumerate(jobs):
            outs.append(rnl.rnl_kv4_attention(*j, stream=side if i % 2 else fork))
        side.wait_stream(fork)
    for _ in range(3):
        for o in outs:
            o.fill_(320.0)
        graph.replay()
        torch.cuda.synchronize()
        rnl.rnl_check_device_error()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
