"""The learners' inner step on the GPU where single rules meet.  Against the fp64 oracle (oracle/inner.py) or
against the same call in other parts.

Tolerances: theta within |theta| 2^-23 + |step| 2^-20 + 2^-149 (two roundings of values that
differ by the change's 2^-20, and the smallest subnormal); moments, codes and scale bytes equal;
norms of n terms within (n + 8) 2^-53 of themselves (n fp64 additions a side, halved by the root).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import diloco_outer_step_amd as dlc
from oracle import inner
from tests import test_gpu_inner as base

pytestmark = pytest.mark.gpu

DEV = "cuda"


def moments_of(coded):
    return ("mc", "ms", "vc", "vs") if coded else ("m", "v")


def step(b, tensors, coded, group, **kw):
    if coded:
        dlc.dlc_adamw_coded_step(b["theta"], b["grads"], b["mc"].view(torch.float8_e4m3fn), b["ms"],
                                 b["vc"].view(torch.float8_e5m2), b["vs"], b["steps"], tensors, group, seed=11, **kw)
    else:
        dlc.dlc_adamw_step(b["theta"], b["grads"], b["m"], b["v"], b["steps"], tensors, group, **kw)


def oracle_step(r, grads, tensors, coded, groups, clip=None, lr_scale=None):
    if coded:
        return inner.adamw_coded(r["theta"], grads, r["mc"], r["ms"], r["vc"], r["vs"], r["steps"], tensors, groups,
                                 None, 11, clip, lr_scale)
    return inner.adamw(r["theta"], grads, r["m"], r["v"], r["steps"], tensors, groups, None, clip, lr_scale)


def state(k, stride, tensors, grads="fp32", seed=0):
    b = base.draw(k, stride, tensors, [1] * k, grads, seed)
    base.coded_start(b, k, stride, seed + 1)
    return b


def clone(b):
    return {n: x if n == "mask" else x.clone() for n, x in b.items()}


# --- buffers side by side ------------------------------------------------------------------

def c_step(theta, grads, m, v, steps, stride, k, tensors, present=None, gs=None, lrs=None):
    """dlc_adamw_step on addresses (fp32 gradients, no working copy)."""
    arr, n = dlc._tensors(tensors)
    group = (ctypes.c_double * 5)(1e-3, 0.9, 0.999, 1e-8, 0.1)
    on = None if present is None else ctypes.cast((ctypes.c_uint8 * k)(*present), ctypes.c_void_p)
    dlc._check(dlc._lib.dlc_adamw_step(theta, grads, 0, m, v, steps, stride, k, on, arr, n, None,
                                       ctypes.cast(group, ctypes.c_void_p), 1, gs, lrs, None, 0, dlc._stream(None)))


def test_rows_of_several_buffers_may_take_turns_in_one():
    """theta, m, v and the gradients as columns of one [K][4 S] array: no element is shared."""
    tensors, s = base.layout(base.LISTS["ragged"])
    k = 3
    b = state(k, s, tensors)
    names = ("theta", "m", "v", "grads")
    one = torch.cat([b[n] for n in names], 1).contiguous()
    steps = b["steps"].clone()
    at = [one.data_ptr() + 4 * s * j for j in range(4)]
    c_step(at[0], at[3], at[1], at[2], steps.data_ptr(), 4 * s, k, tensors)
    step(b, tensors, False, dlc.AdamWGroup(1e-3, 0.9, 0.999, 1e-8, 0.1))
    torch.cuda.synchronize()
    assert torch.equal(one, torch.cat([b[n] for n in names], 1)) and torch.equal(steps, b["steps"])


def test_absent_learners_rows_may_hold_another_buffer():
    """Only learner 0 takes part: the moments lie where the absent learners' rows of theta would."""
    tensors, s = base.layout([100, 4097])
    b = state(1, s, tensors)
    one = torch.cat([b["theta"], b["m"], b["v"]]).contiguous()
    steps = b["steps"].clone()
    row = 4 * s
    c_step(one.data_ptr(), b["grads"].data_ptr(), one.data_ptr() + row, one.data_ptr() + 2 * row, steps.data_ptr(), s, 3,
           tensors, present=[1, 0, 0])
    step(b, tensors, False, dlc.AdamWGroup(1e-3, 0.9, 0.999, 1e-8, 0.1))
    torch.cuda.synchronize()
    assert torch.equal(one, torch.cat([b["theta"], b["m"], b["v"]]))


def test_what_is_only_read_may_be_shared_and_small_arrays_may_touch():
    tensors, s = base.layout([100, 4097])
    a, b = state(3, s, tensors), state(3, s, tensors)
    small = torch.zeros(9, dtype=torch.float64, device=DEV)  # norm, scale, factor end to end
    norm, scale, factor = small[:3], small[3:6], small[6:]
    ws = dlc.alloc_grad_norm_workspace(3, tensors)
    dlc.dlc_grad_norm(a["grads"], tensors, norm, scale, ws, max_norm=1e-2)
    factor.copy_(scale)
    step(a, tensors, False, dlc.AdamWGroup(), grad_scale=scale, lr_scale=scale)  # one array for both factors
    step(b, tensors, False, dlc.AdamWGroup(), grad_scale=scale.clone(), lr_scale=factor)
    torch.cuda.synchronize()
    for n in ("theta", "m", "v", "steps"):
        assert torch.equal(a[n], b[n]), n
