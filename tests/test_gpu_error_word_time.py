"""rnl_check_device_error (and rnl_pipeline_wait, which ends the same way) reads
the error words of the modules in use only: a program that makes none of the
cache, attention and multi-axis rotary calls does not pay for their four words.

In a process of its own: the median time of the check before the first such
call against that of the check after one of each, 10 words against 14."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = textwrap.dedent("""
    import sys, time
    sys.path.insert(0, {root!r})
    import torch
    import rmsnorm_linear_projection_gb300 as rnl
    dev = dict(device="cuda")
    x = torch.ones(64, 512, dtype=torch.bfloat16, **dev)

    def check_us():
        rnl.rmsnorm_linear_bf16(x, None, x)
        rnl.rnl_check_device_error()
        times = []
        for _ in range(300):
            t = time.perf_counter()
            rnl.rnl_check_device_error()
            times.append(time.perf_counter() - t)
        return sorted(times)[150] * 1e6

    before = check_us()
    cache = rnl.Kv4Cache.empty(20, 1, 64, 64, 32)
    i32 = dict(dtype=torch.int32, **dev)
    table, lens, cu = torch.arange(20, **i32).repeat(1, 500), torch.tensor([640], **i32), torch.tensor([0, 640], **i32)
    y = torch.zeros(640, 192, dtype=torch.bfloat16, **dev)
    cs = torch.zeros(4, 64, **dev)
    q, k, v = rnl.rnl_qkv_rope_axes(y, 1, 1, 64, None, None, torch.zeros(1, 640, **i32), [0] * 32, cs)
    rnl.rnl_kv4_append(k, v, cache, table, lens, cu)
    out = rnl.rnl_kv4_attention(q, cache, table, lens, cu)
    assert (out == 0).all()
    after = check_us()
    print(before, after)
""")


def test_words_of_modules_that_are_not_in_use_are_not_read():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rmsnorm_linear_projection_gb300 import build
    build.build()
    p = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    assert p.returncode == 0, p.stderr
    before, after = map(float, p.stdout.split()[-2:])
    assert before < 0.87 * after, f"{before:.1f} us before, {after:.1f} us after"  # 10 / 14 words: 0.71 to 0.75
