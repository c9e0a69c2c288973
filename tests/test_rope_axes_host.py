"""The multi-axis rotary call's host argument, without a GPU."""
import array

import numpy as np
import pytest
import torch

from rmsnorm_linear_projection_gb300 import _native as nat


@pytest.mark.parametrize("kind", ["list", "tuple", "bytes", "array", "int64", "int32", "uint8", "tensor"])
def test_axis_numbers_of_any_sequence(monkeypatch, kind):
    """The library gets the axis numbers, whatever holds them (an array's memory
    is not its values)."""
    m = [i % 3 for i in range(32)]
    make = {"list": list, "tuple": tuple, "bytes": bytes, "array": lambda v: array.array("i", v), "int64": np.array,
            "int32": lambda v: np.array(v, np.int32), "uint8": lambda v: np.array(v, np.uint8), "tensor": torch.tensor}
    got = []

    class Lib:
        def rnl_qkv_rope_axes(self, *a):
            got.append(a[10])
            return 0

    monkeypatch.setattr(nat, "load", lambda path=None: Lib())
    monkeypatch.setattr(nat, "_stream", lambda dev, stream: None)
    nat.rnl_qkv_rope_axes(torch.zeros(3, 4 * 64, dtype=torch.bfloat16), 2, 1, 64, None, None,
                          torch.zeros(3, 3, dtype=torch.int32), make[kind](m), torch.zeros(8, 64))
    assert list(got[0][:32]) == m
