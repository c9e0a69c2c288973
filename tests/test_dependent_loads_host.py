"""Kernels that start as programmatic dependents are on the GPU while the kernel
before them still writes their inputs, so they read them by plain loads: the
read-only path is for data that does not change in a kernel's lifetime, and its
loads need not stay behind the wait.  Read from the sources, without a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rmsnorm_linear_projection_gb300", "csrc")


@pytest.mark.parametrize("name", ["grouped.cu", "grouped.cuh", "moe.cu", "mxquant.cu"])
def test_inputs_are_read_by_plain_loads(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert not re.findall(r"__ldg\s*\(|ld\.global\.nc|ld\.global\.[\w.]*nc\b", text)


@pytest.mark.parametrize("name", ["grouped.cu", "moe.cu", "mxquant.cu"])
def test_every_kernel_waits(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    kernels = text.split("__global__")[1:]
    assert kernels and all("grid_dependency_wait();" in k for k in kernels)
