"""What the early-launched kernels of the operators around the layer must keep to, read from their sources (CPU).

Such a kernel is resident while the one before it still writes.  Its memory may therefore not be called unchanging
for its lifetime (`__restrict__`, const or not, and the read-only loads allow the compiler to read it ahead of the
wait, or from a cache that does not see the writes), and the wait comes before it lets the next kernel come up.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dropless_mixture_experts_warp_gb300", "csrc")


def code(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)


@pytest.mark.parametrize("name", ["norm.cu", "balance.cu", "adamw.cu", "around.cuh"])
def test_memory_may_change_while_an_early_kernel_waits(name):
    for word in ("__restrict__", "__ldg", ".nc."):
        assert word not in code(name), f"{name}: {word}"


@pytest.mark.parametrize("name", ["norm.cu", "balance.cu", "adamw.cu"])
def test_each_kernel_waits_once_and_before_it_lets_the_next_come_up(name):
    kernels = re.split(r"__global__", code(name))[1:]
    assert kernels
    for k in kernels:
        assert k.count("wait_for_previous()") == 1, k[:100]
        if "launch_dependents()" in k:
            assert k.count("launch_dependents()") == 1 and k.index("wait_for_previous()") < k.index("launch_dependents()")
