"""Helpers of the tests of the operators around the layer: inputs on the device, and bounds."""
import numpy as np
import torch

from oracle import around as oa

DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def dev(a, kind):
    """A float64 array rounded to `kind` on the device, and the same rounded values in float64."""
    if a is None:
        return None, None
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DTYPE[kind])
    return t.cuda(), t.double().numpy()


def check(name, got, ref, kind, terms):
    """|got - ref| within the one rounding to `kind` and fp32 arithmetic: `terms` roundings of 2^-24 on the
    majorant (a sum of n terms rounds at most n times)."""
    value, majorant = ref
    got = got.double().cpu().numpy()
    assert got.shape == value.shape, name
    bound = oa.HALF_STEP[kind] * abs(value) + (1 + oa.HALF_STEP[kind]) * terms * oa.U32 * majorant + 1e-37
    off = abs(got - value)
    assert np.all(off <= bound), f"{name}: {np.max(off - bound)} over the bound, largest value {abs(value).max()}"
