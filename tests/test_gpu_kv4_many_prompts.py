"""Attention over the 4-bit cache with more sequences than the prompt kernel has
threads (640): prompts of more than 32 rows x heads among single tokens, drafts
and sequences without rows, in every part of the batch."""
import pytest
import torch

from test_gpu_kv4 import check_outputs, filled, gen, i32, randn, wide

import kv4_plain as plain

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


@pytest.mark.parametrize("prompts,D,G", [("all over", 64, 4), ("only late", 64, 2), ("one at the end", 64, 1),
                                         ("most", 128, 1), ("all over", 128, 1)])
def test_prompts_beyond_the_first_sequences(prompts, D, G):
    g = gen(D + len(prompts))
    B = 1500
    many = {"all over": lambda b: b % 97 == 5, "only late": lambda b: b in (641, 700, 1279, 1280, 1281, 1400),
            "one at the end": lambda b: b == B - 1, "most": lambda b: b % 5 != 0}[prompts]
    rows = [(33 + (b * 13) % 60) if many(b) else b % 4 for b in range(B)]
    lens = [r + (b * 37) % 90 for b, r in enumerate(rows)]
    c, t = filled(g, lens, 1, 32, D, 32)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    q = randn(g, cu[-1] + 3, G, D).bfloat16()
    window = 40 if D == 64 else 0
    ref = plain.attention(q, c, t, i32(lens), i32(cu), window=window)
    for tt in (t, wide(t, 32)):  # the first too small for the prompt kernel, but for most of them prompts
        check_outputs(ref, q, c, tt, lens, cu, window=window)
