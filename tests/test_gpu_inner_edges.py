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
# Neighbours without padding, so that a call of the whole list has one range (and a last one apart), whose
# tiles of 256 and of 1024 elements end inside of tensors; one by one most of them end in a partial tile.
JOINED = [64 * 3, 64 * 5, 64 * 16, 64, 64 * 37, 64 * 64, 64 * 2, 64 * 15, 100]


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


# --- how the tensors are split -----------------------------------------------------------

def split_three_ways(b, tensors, coded, group):
    """The step of the whole list, of the tensors one by one, of the list in another order: bit for bit alike."""
    start = clone(b)
    step(b, tensors, coded, group)
    for parts in ([[t] for t in tensors[::-1]], [tensors[1::2] + tensors[::2]]):
        c = clone(start)
        for part in parts:
            c["steps"].copy_(start["steps"])
            step(c, part, coded, group)
        torch.cuda.synchronize()
        for n in ("theta", "steps") + moments_of(coded):
            same = torch.equal(b[n].view(torch.uint8), c[n].view(torch.uint8))
            assert same, (n, len(parts), int((b[n] != c[n]).sum()))
    return start


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("grads", ["fp32", "bf16"])
def test_results_do_not_depend_on_how_joined_tensors_are_split(coded, grads):
    tensors, stride = base.layout(JOINED)
    split_three_ways(state(2, stride, tensors, grads), tensors, coded, dlc.AdamWGroup(1e-3, 0.9, 0.999, 1e-8, 0.1))


# root = 1 / sqrt(1 - beta2^t) is 31.6 at the first step and 1 at a late one: eps on both sides of 2^-40 root and
# of 2^-36 root, the default, and the smallest
@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("eps", [1e-8, 4.7e-10, 4.5e-10, 3e-11, 1.5e-11, 1.4e-11, 1e-12, 9e-13, 1e-18, 1.2e-38])
@pytest.mark.parametrize("steps", [0, 1_000_000])
def test_tiny_second_moments_whatever_the_split(coded, eps, steps):
    tensors, stride = base.layout(JOINED)
    b = state(2, stride, tensors)
    b["steps"].fill_(steps)
    gen = torch.Generator().manual_seed(5)
    b["grads"] = (torch.randn(b["grads"].shape, generator=gen) * 3e-18).to(DEV)  # v is about 1e-38
    if coded:
        for n in moments_of(True):
            b[n].zero_()
    else:
        b["v"] = (torch.rand(b["v"].shape, generator=gen) * 2e-38).to(DEV)
        b["m"] = (torch.randn(b["m"].shape, generator=gen) * min(1.0, eps)).to(DEV)
    b["theta"].mul_(1e-6)  # the step's last bits show in theta
    group = dlc.AdamWGroup(1e-6, 0.9, 0.999, eps, 0.1)
    start = split_three_ways(b, tensors, coded, group)
    r = {n: base.host(start[n]).copy() for n in ("theta", "steps") + moments_of(coded)}
    size = oracle_step(r, base.host(start["grads"]), tensors, coded, [group])
    base.near_theta(base.host(b["theta"]), r["theta"], size, b["mask"], "theta")
    for n in moments_of(coded):
        base.same(np.where(b["mask"], base.host(b[n]), 0) if b[n].shape == b["theta"].shape else base.host(b[n]),
                  np.where(b["mask"], r[n], 0) if b[n].shape == b["theta"].shape else r[n], n)


# --- eps at the upper end ------------------------------------------------------------------

@pytest.mark.parametrize("eps", [2.0 ** 126, 2.0 ** 126 * (1 - 2.0 ** -24), 1e30])
def test_the_largest_eps(eps):
    tensors, stride = base.layout([1, 65, 4099, 256])
    b = state(2, stride, tensors)
    b["m"].mul_(2.0 ** 120)
    group = dlc.AdamWGroup(1.0, 0.9, 0.999, eps, 0.0)
    r = {n: base.host(b[n]).copy() for n in ("theta", "steps", "m", "v")}
    step(b, tensors, False, group)
    torch.cuda.synchronize()
    size = oracle_step(r, base.host(b["grads"]), tensors, False, [group])
    assert size[b["mask"]].max() > 1e-6
    base.near_theta(base.host(b["theta"]), r["theta"], size, b["mask"], "theta")


# --- what lies behind a tensor -------------------------------------------------------------

@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("grads", ["fp32", "bf16", "fp16"])
def test_padding_that_is_not_finite_has_no_influence_and_stays(coded, grads):
    tensors, stride = base.layout(base.LISTS["ragged"])
    clean = state(2, stride, tensors, grads)
    clean["work"] = torch.zeros((2, stride), dtype=torch.bfloat16, device=DEV)
    b = clone(clean)
    outside = torch.from_numpy(~clean["mask"]).to(DEV)
    for n in ("theta", "grads", "m", "v", "work"):
        b[n][outside] = math.nan
        b[n][outside & (torch.arange(stride, device=DEV) % 3 == 1)] = math.inf
    b["mc"][outside], b["vc"][outside] = 0x7F, 0x7C
    before = clone(b)
    for x in (clean, b):
        for _ in range(2):
            step(x, tensors, coded, dlc.AdamWGroup(), working=x["work"])
    torch.cuda.synchronize()
    whole = torch.from_numpy(clean["mask"]).to(DEV)
    for n in ("theta", "work") + (("mc", "vc") if coded else ("m", "v")):
        assert torch.equal(b[n][whole], clean[n][whole]), n
        raw = torch.uint8 if b[n].element_size() == 1 else torch.int16 if b[n].element_size() == 2 else torch.int32
        assert torch.equal(b[n].view(raw)[outside], before[n].view(raw)[outside]), n
    if coded:
        assert torch.equal(b["ms"], clean["ms"]) and torch.equal(b["vs"], clean["vs"])


# --- learners left out, their factors -------------------------------------------------------

@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("scale", [0.0, -1.0, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("name", ["around_a_block", "ragged"])  # the step counted by the blocks, by a kernel of its own
def test_a_learner_whose_step_is_left_out_keeps_every_bit(coded, scale, name):
    tensors, stride = base.layout(base.LISTS[name])
    b = state(3, stride, tensors, "bf16")
    b["work"] = torch.full((3, stride), 7.0, dtype=torch.bfloat16, device=DEV)
    clip = [1.0, scale, 0.25]
    start = clone(b)
    step(b, tensors, coded, base.GROUPS[0], working=b["work"],
         grad_scale=torch.tensor(clip, dtype=torch.float64, device=DEV))
    torch.cuda.synchronize()
    r = {n: base.host(start[n]).copy() for n in ("theta", "steps") + moments_of(coded)}
    size = oracle_step(r, base.host(start["grads"]), tensors, coded, [base.GROUPS[0]], clip)
    base.near_theta(base.host(b["theta"]), r["theta"], size, b["mask"], "theta")
    assert b["steps"].tolist() == r["steps"].tolist() == [1, 40, 81]
    for n in ("theta", "work") + moments_of(coded):
        assert torch.equal(b[n][1].view(torch.uint8), start[n][1].view(torch.uint8)), n
        if n in r and n != "theta":
            base.same(base.host(b[n]), r[n], n)
    assert not torch.equal(b["theta"][0], start["theta"][0]) and not torch.equal(b["theta"][2], start["theta"][2])


# --- the norm's one-block form --------------------------------------------------------------

@pytest.mark.parametrize("grads", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("sizes", [[65] * 8, [65] * 9, [1] * 8, [1 << 16], [(1 << 16) - 64, 64], [(1 << 16) + 1],
                                   [(1 << 13) - 3] * 8, [(1 << 13) + 1] * 8])
def test_norm_on_both_sides_of_the_one_block_forms_limits(grads, sizes):
    base.check_norm(sizes, grads, [1, 1, 0], 0.5, 1e-2)


# --- codes -------------------------------------------------------------------------------------

# exponents of the largest gradient of a block: m is the gradient itself (beta1 = 0), v its square (beta2 = 0)
WINDOWS = [(-148, -121), (-121, -64), (-64, -50), (-50, 0), (0, 63), (63, 127)]


@pytest.mark.parametrize("low,high", WINDOWS)
def test_every_range_of_exponents_is_coded_as_defined(low, high):
    """2^21 values of each window, each up to 2^26 below its block's largest: normal and subnormal codes, scale bytes
    from 0 to the end, values below the code's grid, subnormal fp32 moments, second moments past fp32's end."""
    n = 1 << 21
    rng = np.random.default_rng(200 + high)
    top = rng.integers(low, high, n // 64, endpoint=True).astype(np.float64)
    e = np.repeat(top, 64) - np.where(np.arange(n) % 64 == 0, 0, rng.integers(0, 26, n, endpoint=True))
    g = (np.exp2(np.minimum(e, 126)) * rng.uniform(1, 2, n) * rng.choice([-1, 1], n)).astype(np.float32)[None]
    tensors = [(0, 0, n)]
    group = (0.0, 0.0, 0.0, 1e-8, 0.0)
    r = dict(theta=np.zeros((1, n), np.float32), mc=np.zeros((1, n), np.uint8), ms=np.zeros((1, n // 64), np.uint8),
             vc=np.zeros((1, n), np.uint8), vs=np.zeros((1, n // 64), np.uint8), steps=np.full(1, high + 200, np.int64))
    b = {name: torch.from_numpy(x.copy()).to(DEV) for name, x in r.items()}
    b["grads"] = torch.from_numpy(g).to(DEV)
    step(b, tensors, True, dlc.AdamWGroup(*group))
    torch.cuda.synchronize()
    oracle_step(r, g, tensors, True, [group])
    for name in moments_of(True):
        base.same(base.host(b[name]), r[name], name)
