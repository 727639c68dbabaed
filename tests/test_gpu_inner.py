"""The learners' inner step on the GPU against the fp64 CPU oracle (oracle/inner.py).

Every buffer is filled with a sentinel outside the elements the call may touch, and the
sentinels are compared afterwards: padding between tensors, absent learners, the ends
of rows.  Tolerances, from the definitions in include/dlc.h:

  * moments: the same fp64 sums, a few 2^-53 apart, rounded to fp32 once: equal but where
    one straddles a rounding boundary, once in some 2^28 elements: equal on these inputs
    (and so are the codes);
  * theta: two roundings to fp32 of values that differ by the change's 2^-20:
    |theta| 2^-23 + |step| 2^-20, and the smallest subnormal;
  * the working copy: torch's rounding of the call's own theta, bit for bit;
  * norms: fp64 sums of at most 2^26 terms in some order: relative 2^-25 and less is seen as
    equal to n * 2^-53.
"""
import math

import numpy as np
import pytest
import torch

import diloco_outer_step_amd as dlc
import oracle
from oracle import inner

pytestmark = pytest.mark.gpu

DEV = "cuda"
SENT = 1234.5
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
GROUPS = [dlc.AdamWGroup(1e-3, 0.9, 0.999, 1e-8, 0.1), dlc.AdamWGroup(3e-3, 0.8, 0.95, 1e-6, 0.0),
          dlc.AdamWGroup(0.0, 0.0, 0.5, 1.0, 0.3)]

# sizes of the tensors, in row order; a gap of None leaves a whole 64-element group between two
LISTS = {
    "one_element": [1],
    "one_block": [64],
    "around_a_block": [63, 64, 65, 127, 128, 129],
    "joined": [64 * 7, 64, 4096, 64 * 70],                     # no padding: one range where the group is one
    "around_a_tile": [4095, 4096, 4097, 8191, 8192, 8193],
    "ragged": [1, 100003, 2, 65, 64 * 300 + 9, 4096 * 5 + 17, None, 31, 77777],
    "few_blocks": [64 * 256],                                  # the most that a call's blocks count themselves ...
    "more_blocks": [64 * 256 + 1],                             # ... and one more
    "few_coded_blocks": [64 * 1024],
    "more_coded_blocks": [64 * 1024 - 5, 6],
    "many": [(7 * i) % 200 + 1 for i in range(600)],           # more ranges than one launch takes
}


def layout(sizes, shuffle=0):
    """(tensors, row length): rows start with a group of no tensor; the list's order is shuffled."""
    at, out = 64, []
    for n in sizes:
        if n is None:
            at += 64
            continue
        out.append((len(out) * 64, at, n))
        at += -(-n // 64) * 64
    rng = np.random.default_rng(shuffle)
    offsets = np.cumsum([0] + [-(-n // 64) * 64 for _, _, n in out])
    out = [(int(offsets[i]), lo, n) for i, (_, lo, n) in enumerate(out)]
    if shuffle:
        out = [out[i] for i in rng.permutation(len(out))]
    return out, at + 128


def inside(shape, tensors, present):
    mask = np.zeros(shape, bool)
    for i in range(shape[0]):
        for _, lo, n in tensors:
            mask[i, lo:lo + n] = present[i]
    return mask


def host(t):
    return t.float().cpu().numpy() if t.dtype in (torch.bfloat16, torch.float16) else t.cpu().numpy()


def draw(k, stride, tensors, present, grads="fp32", seed=0):
    """Inputs of an inner step; sentinels outside the tensors and in absent learners' rows."""
    gen = torch.Generator().manual_seed(seed)
    mask = torch.from_numpy(inside((k, stride), tensors, present))
    spread = torch.exp(torch.randn((k, stride), generator=gen) * 2 - 6)

    def fill(x):
        return torch.where(mask, x, torch.full_like(x, SENT)).to(DEV)

    g = torch.randn((k, stride), generator=gen) * spread
    g[:, ::7] = 0
    return dict(theta=fill(torch.randn((k, stride), generator=gen) * 0.02), grads=fill(g.to(TYPES[grads])),
                m=fill(torch.randn((k, stride), generator=gen) * spread), v=fill(spread ** 2),
                steps=torch.arange(k, dtype=torch.int64, device=DEV) * 40, mask=mask.numpy())


def near_theta(got, want, size, mask, what):
    bound = np.abs(want.astype(np.float64)) * 2.0 ** -23 + size * 2.0 ** -20 + 2.0 ** -149
    bad = mask & ~(np.abs(got.astype(np.float64) - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], want[bad][:3])


def same(got, want, what):
    assert got.dtype == want.dtype and got.shape == want.shape
    bad = got.view(np.uint8 if got.itemsize == 1 else np.uint32) != want.view(np.uint8 if want.itemsize == 1 else np.uint32)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], want[bad][:3])


def check_adamw(case, groups, group_of, grads, working, present, clip=None, lr_scale=None, shuffle=0, k=3, seed=0,
                change=None):
    tensors, stride = layout(case, shuffle)
    b = draw(k, stride, tensors, present, grads, seed)
    if change:
        change(b, tensors)
    ids = None if group_of is None else [group_of(j) for j in range(len(tensors))]
    ref = {n: host(b[n]).copy() for n in ("theta", "m", "v", "steps")}
    size = inner.adamw(ref["theta"], host(b["grads"]), ref["m"], ref["v"], ref["steps"], tensors, groups, ids, clip,
                       lr_scale, present)
    work = torch.full((k, stride), SENT, dtype=TYPES[working], device=DEV) if working else None
    before = {n: b[n].clone() for n in ("theta", "grads")}

    def per(x):
        return None if x is None else torch.tensor(x, dtype=torch.float64, device=DEV)

    dlc.dlc_adamw_step(b["theta"], b["grads"], b["m"], b["v"], b["steps"], tensors, groups, group_of=ids,
                       grad_scale=per(clip), lr_scale=per(lr_scale), working=work, present=present)
    torch.cuda.synchronize()
    same(host(b["m"]), ref["m"], "m")
    same(host(b["v"]), ref["v"], "v")
    assert np.array_equal(host(b["steps"]), ref["steps"])
    near_theta(host(b["theta"]), ref["theta"], size, b["mask"], "theta")
    same(np.where(b["mask"], 0, host(b["theta"])), np.where(b["mask"], 0, host(before["theta"])), "theta's sentinels")
    assert torch.equal(b["grads"], before["grads"])
    if work is not None:
        took = b["mask"].copy()
        for i in range(k):
            took[i] &= clip is None or inner.takes_step(clip[i])
        want = torch.where(torch.from_numpy(took).to(DEV), b["theta"].to(work.dtype), torch.full_like(work, SENT))
        assert torch.equal(work, want)
    return b


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("grads,working", [("fp32", ""), ("bf16", "bf16"), ("fp16", "fp16")])
def test_adamw(name, grads, working):
    print(f"[adamw] {name} {grads}", flush=True)
    check_adamw(LISTS[name], GROUPS, lambda j: (j // 2) % 3, grads, working, [1, 1, 1])


@pytest.mark.parametrize("grads,working", [("fp32", "bf16"), ("fp32", "fp16"), ("bf16", ""), ("bf16", "fp16"),
                                           ("fp16", ""), ("fp16", "bf16")])
def test_adamw_other_type_pairs(grads, working):
    check_adamw(LISTS["ragged"], GROUPS[:1], None, grads, working, [1, 0, 1], clip=[0.5, 1.0, 0.125],
                lr_scale=[1.0, 0.0, 0.3], shuffle=4)


@pytest.mark.parametrize("present", [[1, 1, 0], [0, 0, 1], [0, 1, 0]])
def test_adamw_absent_learners_and_list_order(present):
    check_adamw(LISTS["ragged"], GROUPS, lambda j: j % 3, "bf16", "bf16", present, shuffle=3)
    check_adamw(LISTS["many"], GROUPS, lambda j: j % 2, "fp32", "", present, shuffle=5)


def test_adamw_64_learners():
    check_adamw([100, 4097], GROUPS[:2], lambda j: j, "fp32", "", [int(i % 5 != 0) for i in range(64)], k=64)


def test_adamw_tiny_second_moments_under_a_tiny_eps():
    """v among the subnormals, where its root still outweighs eps: neither is lost."""
    def change(b, tensors):
        for _, lo, n in tensors:
            b["v"][:, lo:lo + n].mul_(1e-36), b["m"][:, lo:lo + n].mul_(1e-18), b["grads"][:, lo:lo + n].mul_(1e-18)

    for eps in (1.2e-38, 1e-25, 1e-21, 1e-18, 1e-11):
        groups = [dlc.AdamWGroup(1e-3, 0.9, 0.999, eps, 0.1), dlc.AdamWGroup(1e-3, 0.9, 0.5, eps, 0.0)]
        for start in (0, 500):
            def both(b, tensors):
                change(b, tensors)
                b["steps"].fill_(start)

            check_adamw([1, 65, 4099, 256], groups, lambda j: j % 2, "fp32", "", [1, 1], k=2, change=both)


@pytest.mark.parametrize("scale", [0.0, -1.0, math.inf, -math.inf, math.nan])
def test_a_learner_without_a_usable_scale_is_left_out(scale):
    check_adamw(LISTS["ragged"], GROUPS, lambda j: j % 3, "fp32", "bf16", [1, 1, 1], clip=[1.0, scale, 0.25])


@pytest.mark.parametrize("kind", ["zeros", "tiny", "subnormal", "huge", "nan", "inf"])
@pytest.mark.parametrize("t", [0, 1, 1000, (1 << 31) + 5])
def test_adamw_values_at_the_ends(kind, t):
    def change(b, tensors):
        b["steps"].fill_(t)
        for _, lo, n in tensors:
            x = b["grads"][:, lo:lo + n]
            if kind == "zeros":
                x.zero_(), b["m"][:, lo:lo + n].zero_(), b["v"][:, lo:lo + n].zero_()
            elif kind == "tiny":
                x.mul_(1e-25), b["m"][:, lo:lo + n].zero_(), b["v"][:, lo:lo + n].zero_()
            elif kind == "subnormal":
                b["theta"][:, lo:lo + n].mul_(1e-37), b["m"][:, lo:lo + n].mul_(1e-38), b["v"][:, lo:lo + n].mul_(1e-38)
            elif kind == "huge":
                x.mul_(1e18), b["v"][:, lo:lo + n].mul_(1e30)
            else:
                x[:, ::5] = float(kind)

    def run():
        check_adamw([1, 65, 4099], GROUPS[:2], lambda j: j % 2, "fp32", "", [1, 1], k=2, change=change)

    if kind not in ("nan", "inf"):
        run()
        return
    # a NaN or an infinity spoils its own element and no other
    tensors, stride = layout([1, 65, 4099])
    b = draw(2, stride, tensors, [1, 1])
    clean = {n: b[n].clone() for n in ("theta", "m", "v", "steps")}
    change(b, tensors)
    bad = ~torch.isfinite(b["grads"])
    g = torch.where(bad, torch.zeros_like(b["grads"]), b["grads"])
    clean["steps"].fill_(t)
    dlc.dlc_adamw_step(clean["theta"], g, clean["m"], clean["v"], clean["steps"], tensors, GROUPS[0])
    dlc.dlc_adamw_step(b["theta"], b["grads"], b["m"], b["v"], b["steps"], tensors, GROUPS[0])
    torch.cuda.synchronize()
    for n in ("theta", "m", "v"):
        assert torch.equal(b[n][~bad], clean[n][~bad])
        assert not torch.isfinite(b["m"][bad]).any()


# --- the norm ------------------------------------------------------------------------

def check_norm(case, grads, present, unscale, max_norm, shuffle=0, k=3):
    tensors, stride = layout(case, shuffle)
    b = draw(k, stride, tensors, present, grads)
    norm = torch.full((k,), SENT, dtype=torch.float64, device=DEV)
    scale = torch.full((k,), SENT, dtype=torch.float64, device=DEV)
    ws = dlc.alloc_grad_norm_workspace(k, tensors)
    dlc.dlc_grad_norm(b["grads"], tensors, norm, scale, ws, max_norm=max_norm, unscale=unscale, present=present)
    torch.cuda.synchronize()
    got = (norm.clone(), scale.clone())
    g = host(b["grads"])
    terms = sum(n for _, _, n in tensors)
    for i in range(k):
        if not present[i]:
            assert norm[i] == SENT and scale[i] == SENT
            continue
        n, s = inner.grad_norm(g[i], tensors, unscale, max_norm)
        tol = (terms + 8) * 2.0 ** -53  # each side's relative error of the sum, halved by the root
        assert abs(float(norm[i]) - n) <= tol * n and abs(float(scale[i]) - s) <= tol * s, (i, float(norm[i]), n)
    dlc.dlc_grad_norm(b["grads"], tensors, norm, scale, ws.fill_(0xFF), max_norm=max_norm, unscale=unscale, present=present)
    torch.cuda.synchronize()
    assert torch.equal(got[0], norm) and torch.equal(got[1], scale)


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("grads", sorted(TYPES))
def test_norm(name, grads):
    print(f"[norm] {name} {grads}", flush=True)
    check_norm(LISTS[name], grads, [1, 1, 1], 1.0, math.inf)
    check_norm(LISTS[name], grads, [1, 0, 1], 0.125, 1e-3, shuffle=2)


def test_norm_of_64_learners_and_of_a_large_row():
    check_norm([4097, 64], "bf16", [int(i % 3 > 0) for i in range(64)], 2.0, 1.0, k=64)
    check_norm([1 << 24, 12345677], "fp32", [1], 1.0, 1.0, k=1)


def test_norm_of_nothing_and_of_what_is_not_finite():
    tensors, stride = layout([100, 4097])
    g = torch.zeros((4, stride), device=DEV)
    g[1, 64] = math.inf
    g[2, 200] = math.nan
    g[3, 64 + 100:128 + 64] = math.nan  # padding of the first tensor: not part of any
    g[3, 64] = 3e38
    g[3, 65] = 3e38
    norm, scale = (torch.zeros(4, dtype=torch.float64, device=DEV) for _ in range(2))
    dlc.dlc_grad_norm(g, tensors, norm, scale, dlc.alloc_grad_norm_workspace(4, tensors), max_norm=1.0, unscale=0.5)
    torch.cuda.synchronize()
    assert float(norm[0]) == 0.0 and float(scale[0]) == 0.5
    assert float(norm[1]) == math.inf and float(scale[1]) == 0.0
    assert math.isnan(float(norm[2])) and float(scale[2]) == 0.0
    want = 0.5 * math.sqrt(2) * float(np.float32(3e38))
    assert math.isclose(float(norm[3]), want, rel_tol=1e-15) and math.isclose(float(scale[3]), 0.5 / want, rel_tol=1e-15)


# --- coded moments -------------------------------------------------------------------

def coded_start(b, k, stride, seed=1):
    gen = torch.Generator().manual_seed(seed)
    mc = torch.randint(0, 0x77, (k, stride), generator=gen) | (torch.randint(0, 2, (k, stride), generator=gen) << 7)
    vc = torch.randint(0, 0x77, (k, stride), generator=gen)
    ms = torch.randint(90, 120, (k, stride // 64), generator=gen)
    vs = torch.randint(60, 110, (k, stride // 64), generator=gen)
    b.update(mc=mc.to(torch.uint8).to(DEV), vc=vc.to(torch.uint8).to(DEV), ms=ms.to(torch.uint8).to(DEV),
             vs=vs.to(torch.uint8).to(DEV))


def coded_call(b, tensors, groups, ids, seed, clip, lr_scale, work, present, stream=None):
    def per(x):
        return None if x is None else torch.tensor(x, dtype=torch.float64, device=DEV)

    dlc.dlc_adamw_coded_step(b["theta"], b["grads"], b["mc"].view(torch.float8_e4m3fn), b["ms"],
                             b["vc"].view(torch.float8_e5m2), b["vs"], b["steps"], tensors, groups, group_of=ids,
                             seed=seed, grad_scale=per(clip), lr_scale=per(lr_scale), working=work, present=present,
                             stream=stream)


CODED = ("theta", "mc", "ms", "vc", "vs", "steps")


def test_coded_tiny_moments_under_a_tiny_eps():
    def change(b, tensors):
        for n in ("mc", "ms", "vc", "vs"):
            b[n].zero_()
        b["grads"].mul_(1e-16)

    for eps in (1.2e-38, 1e-24, 1e-19):
        check_coded([1, 65, 4099, 1024], [dlc.AdamWGroup(1e-3, 0.9, 0.999, eps, 0.1)], None, "fp32", "", [1, 1], k=2,
                    change=change, times=3)


def check_coded(case, groups, group_of, grads, working, present, clip=None, lr_scale=None, shuffle=0, k=3, seed=9,
                change=None, times=2):
    tensors, stride = layout(case, shuffle)
    b = draw(k, stride, tensors, present, grads)
    coded_start(b, k, stride)
    if change:
        change(b, tensors)
    ids = None if group_of is None else [group_of(j) for j in range(len(tensors))]
    ref = {n: host(b[n]).copy() for n in CODED}
    work = torch.full((k, stride), SENT, dtype=TYPES[working], device=DEV) if working else None
    for _ in range(times):
        start = host(b["theta"]).copy()
        ref["theta"][:] = start
        size = inner.adamw_coded(ref["theta"], host(b["grads"]), ref["mc"], ref["ms"], ref["vc"], ref["vs"],
                                 ref["steps"], tensors, groups, ids, seed, clip, lr_scale, present)
        coded_call(b, tensors, groups, ids, seed, clip, lr_scale, work, present)
        torch.cuda.synchronize()
        for n in ("mc", "ms", "vc", "vs"):
            same(host(b[n]), ref[n], n)  # whole buffers: what is outside the tensors is as it was
        assert np.array_equal(host(b["steps"]), ref["steps"])
        near_theta(host(b["theta"]), ref["theta"], size, b["mask"], "theta")
        same(np.where(b["mask"], 0, host(b["theta"])), np.where(b["mask"], 0, start), "theta's sentinels")
        if work is not None:
            want = torch.where(torch.from_numpy(b["mask"]).to(DEV), b["theta"].to(work.dtype), torch.full_like(work, SENT))
            assert torch.equal(work, want)


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("grads,working", [("fp32", ""), ("bf16", "bf16"), ("fp16", "fp16")])
def test_coded(name, grads, working):
    print(f"[coded] {name} {grads}", flush=True)
    check_coded(LISTS[name], GROUPS, lambda j: (j // 2) % 3, grads, working, [1, 1, 1])


@pytest.mark.parametrize("grads,working", [("fp32", "bf16"), ("fp32", "fp16"), ("bf16", ""), ("bf16", "fp16"),
                                           ("fp16", ""), ("fp16", "bf16")])
def test_coded_other_type_pairs(grads, working):
    check_coded(LISTS["ragged"], GROUPS[:1], None, grads, working, [1, 0, 1], clip=[0.5, 1.0, 0.125],
                lr_scale=[1.0, 0.0, 0.3], shuffle=4, seed=(1 << 64) - 1)


def test_coded_64_learners():
    check_coded([100, 4097], GROUPS[:2], lambda j: j, "fp32", "", [int(i % 5 != 0) for i in range(64)], k=64)


@pytest.mark.parametrize("kind", ["zeros", "start", "tiny", "huge", "wide", "long"])
def test_coded_values_at_the_ends(kind):
    def change(b, tensors):
        if kind == "long":
            b["steps"].fill_((1 << 32) - 1)  # the step's low word wraps in the hash, the powers are far below the grid
            return
        for n in ("mc", "ms", "vc", "vs"):
            b[n].zero_()
        if kind == "zeros":
            b["grads"].zero_()
        elif kind == "tiny":
            b["grads"].mul_(1e-30)  # m below the scales' end, v below fp32
        elif kind == "huge":
            b["grads"].mul_(1e19)
        elif kind == "wide":  # 2^-40 .. 2^40 within a block: grids below the smallest normal code
            b["grads"].mul_(torch.exp2(torch.arange(b["grads"].shape[1], device=DEV) % 81 - 40.0))

    check_coded([1, 65, 4099, 64], GROUPS[:2], lambda j: j % 2, "fp32", "", [1, 1], k=2, change=change, times=3)


def test_coded_a_value_that_is_not_finite_spoils_its_own_element():
    tensors, stride = layout([300])
    b = draw(1, stride, tensors, [1])
    coded_start(b, 1, stride)
    c = {n: b[n].clone() for n in b if n != "mask"}
    bad = torch.zeros((1, stride), dtype=torch.bool, device=DEV)
    bad[:, 70:360:50] = True
    b["grads"][bad] = math.nan
    b["grads"][0, 120] = -math.inf
    # the same blocks with those elements' values too small to matter for a scale
    for x, zero in (("grads", 0.0), ("mc", 0), ("vc", 0)):
        c[x][bad] = zero
    for x in (b, c):
        coded_call(x, tensors, GROUPS[0], None, 3, None, None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(b["ms"], c["ms"]) and torch.equal(b["vs"], c["vs"])
    for n in ("mc", "vc", "theta"):
        assert torch.equal(b[n][~bad], c[n][~bad])
    assert torch.all(b["mc"][bad] & 0x7F == 0x7F) and torch.all(b["vc"][bad] == 0x7F)
    coded_call(b, tensors, GROUPS[0], None, 3, None, None, None, None)  # NaN stays NaN, the others go on
    torch.cuda.synchronize()
    assert torch.all(b["vc"][bad] == 0x7F) and not torch.any(b["vc"][:, 64:364][~bad[:, 64:364]] == 0x7F)


def test_coded_results_do_not_depend_on_how_the_tensors_are_split():
    tensors, stride = layout(LISTS["ragged"])
    b = draw(2, stride, tensors, [1, 1])
    coded_start(b, 2, stride)
    c = {n: b[n].clone() for n in b if n != "mask"}
    coded_call(b, tensors, GROUPS[0], None, 5, None, None, None, None)
    for t in tensors[::-1]:
        c["steps"].copy_(torch.arange(2, device=DEV) * 40)
        coded_call(c, [t], GROUPS[0], None, 5, None, None, None, None)
    torch.cuda.synchronize()
    for n in CODED:
        assert torch.equal(b[n], c[n]), n


# --- far rows, graphs, streams, the whole round ----------------------------------------

@pytest.mark.parametrize("coded", [False, True])
def test_elements_beyond_2_to_the_32(coded):
    """Tensors around element 2^32 of learner 1's row (offsets past 32 bits, and past 2^34 bytes)."""
    lo = (1 << 32) - 128
    sizes = [(lo, 128), (lo + 128, 4097), (lo + 128 + 4160, 65)]
    tensors = [(0 if i == 0 else 64 * 100 * i, a, n) for i, (a, n) in enumerate(sizes)]
    stride = lo + 8192
    small, short = [(o, a - lo, n) for (o, a, n) in tensors], 8192
    s = draw(2, short, small, [1, 1], "bf16")
    coded_start(s, 2, short)
    names = ("theta", "grads", "mc", "vc") if coded else ("theta", "grads", "m", "v")
    big = {n: torch.empty((2, stride), dtype=s[n].dtype, device=DEV) for n in names}
    for n in names:
        big[n][:, lo:] = s[n]
    if coded:
        for n in ("ms", "vs"):
            big[n] = torch.empty((2, stride // 64), dtype=torch.uint8, device=DEV)
            big[n][:, lo // 64:] = s[n]
    big["steps"] = s["steps"].clone()
    start = host(s["theta"])
    ref = {n: host(s[n]).copy() for n in ("theta", "m", "v", "steps", "mc", "ms", "vc", "vs")}
    norm, scale = (torch.zeros(2, dtype=torch.float64, device=DEV) for _ in range(2))
    dlc.dlc_grad_norm(big["grads"], tensors, norm, scale, dlc.alloc_grad_norm_workspace(2, tensors), max_norm=1.0)
    torch.cuda.synchronize()
    clip = scale.tolist()
    for i in range(2):
        assert math.isclose(float(norm[i]), inner.grad_norm(host(s["grads"])[i], small)[0], rel_tol=1e-12)
    if coded:
        dlc.dlc_adamw_coded_step(big["theta"], big["grads"], big["mc"].view(torch.float8_e4m3fn), big["ms"],
                                 big["vc"].view(torch.float8_e5m2), big["vs"], big["steps"], tensors, GROUPS[0], seed=4,
                                 grad_scale=scale)
        torch.cuda.synchronize()
        far = Far(ref, lo)
        size = far.step(host(s["grads"]), small, clip)
        for n in ("mc", "vc"):
            same(host(big[n][:, lo:]), ref[n], n)
        for n in ("ms", "vs"):
            same(host(big[n][:, lo // 64:]), ref[n], n)
    else:
        dlc.dlc_adamw_step(big["theta"], big["grads"], big["m"], big["v"], big["steps"], tensors, GROUPS[0],
                           grad_scale=scale)
        torch.cuda.synchronize()
        size = inner.adamw(ref["theta"], host(s["grads"]), ref["m"], ref["v"], ref["steps"], small, GROUPS, None, clip)
        for n in ("m", "v"):
            same(host(big[n][:, lo:]), ref[n], n)
    near_theta(host(big["theta"][:, lo:]), ref["theta"], size, s["mask"], "theta")
    same(np.where(s["mask"], 0, host(big["theta"][:, lo:])), np.where(s["mask"], 0, start), "theta's sentinels")


@pytest.mark.parametrize("coded", [False, True])
def test_the_largest_tensor(coded):
    """2^32 - 1 elements and a short tensor behind them, in two launches: windows at the start, around the middle
    and at the end against the oracle, every element against a fill that the step cannot leave."""
    big = (1 << 32) - 1
    tensors = [(0, 0, big), (1 << 32, 1 << 32, 5000)]
    stride = (1 << 32) + 8192
    windows = [(0, 4096), ((1 << 31) - 2048, 4096), (big - 4095, 4095), (1 << 32, 5000)]
    gen = torch.Generator().manual_seed(1)
    theta = torch.full((1, stride), 1.0, device=DEV)
    grads = torch.full((1, stride), 0.25, dtype=torch.bfloat16, device=DEV)
    for lo, n in windows:
        theta[0, lo:lo + n] = (torch.randn(n, generator=gen) * 0.02).to(DEV)
        grads[0, lo:lo + n] = torch.randn(n, generator=gen).to(torch.bfloat16).to(DEV)
    steps = torch.zeros(1, dtype=torch.int64, device=DEV)
    start = [host(theta[:, lo:lo + n]).copy() for lo, n in windows]
    gr = [host(grads[:, lo:lo + n]) for lo, n in windows]
    if coded:
        mc, ms, vc, vs = dlc.coded_moments(1, stride)
        dlc.dlc_adamw_coded_step(theta, grads, mc, ms, vc, vs, steps, tensors, GROUPS[0], seed=2)
    else:
        m, v = torch.zeros_like(theta), torch.zeros_like(theta)
        dlc.dlc_adamw_step(theta, grads, m, v, steps, tensors, GROUPS[0])
    torch.cuda.synchronize()
    assert int(steps[0]) == 1
    assert bool((theta[0, big + 1 + 5000:] == 1.0).all())
    for at in range(0, big, 1 << 28):
        assert not bool((theta[0, at:min(big, at + (1 << 28))] == 1.0).any()), at
    for (lo, n), th, g in zip(windows, start, gr):
        zero = [np.zeros((1, n), np.float32) for _ in range(2)]
        count = np.zeros(1, np.int64)
        if coded:
            blocks = -(-n // 64)
            r = dict(theta=th, mc=np.zeros((1, n), np.uint8), ms=np.zeros((1, blocks), np.uint8),
                     vc=np.zeros((1, n), np.uint8), vs=np.zeros((1, blocks), np.uint8), steps=count)
            whole = n if lo + n != big else n - n % 64  # a window that ends inside a block: its whole blocks
            size = Far(r, lo).step(g, [(0, 0, n)], None, seed=2)
            same(host(mc.view(torch.uint8)[:, lo:lo + n]), r["mc"], "m")
            same(host(vc.view(torch.uint8)[:, lo:lo + n]), r["vc"], "v")
            same(host(ms[:, lo // 64:(lo + whole) // 64]), r["ms"][:, :whole // 64], "m scales")
        else:
            size = inner.adamw(th, g, zero[0], zero[1], count, [(0, 0, n)], GROUPS)
            same(host(m[:, lo:lo + n]), zero[0], "m")
            same(host(v[:, lo:lo + n]), zero[1], "v")
        near_theta(host(theta[:, lo:lo + n]), th, size, np.ones((1, n), bool), "theta")


class Far:
    """The oracle's coded step on a short row whose element 0 is element `lo` of the real one."""

    def __init__(self, ref, lo):
        self.ref, self.lo = ref, lo

    def step(self, grads, tensors, clip, seed=4):
        words, r = inner.random_words, self.ref
        inner.random_words = lambda seed, t, i, lo, n: words(seed, t, i, lo + self.lo, n)
        try:
            return inner.adamw_coded(r["theta"], grads, r["mc"], r["ms"], r["vc"], r["vs"], r["steps"], tensors, GROUPS,
                                     None, seed, clip)
        finally:
            inner.random_words = words


@pytest.mark.parametrize("name", ["ragged", "around_a_block"])  # the step counted by a kernel of its own, by the blocks
@pytest.mark.parametrize("coded", [False, True])
def test_captured_steps_replay_the_eager_ones(coded, name):
    """Norm and step captured once: every replay counts its own step, reads the schedule's
    factor and the gradients of the moment, and equals the eager calls; two graphs with
    buffers of their own run one after the other."""
    tensors, stride = layout(LISTS[name])
    plan = dlc.TensorList(tensors)
    k = 3

    def state():
        b = draw(k, stride, tensors, [1, 1, 1], "bf16")
        coded_start(b, k, stride)
        b["lr_scale"] = torch.ones(k, dtype=torch.float64, device=DEV)
        b["norm"], b["scale"] = (torch.zeros(k, dtype=torch.float64, device=DEV) for _ in range(2))
        b["ws"] = dlc.alloc_grad_norm_workspace(k, plan)
        b["work"] = torch.zeros((k, stride), dtype=torch.bfloat16, device=DEV)
        return b

    def step(b):
        dlc.dlc_grad_norm(b["grads"], plan, b["norm"], b["scale"], b["ws"], max_norm=0.5)
        if coded:
            dlc.dlc_adamw_coded_step(b["theta"], b["grads"], b["mc"].view(torch.float8_e4m3fn), b["ms"],
                                     b["vc"].view(torch.float8_e5m2), b["vs"], b["steps"], plan, GROUPS[0], seed=8,
                                     grad_scale=b["scale"], lr_scale=b["lr_scale"], working=b["work"])
        else:
            dlc.dlc_adamw_step(b["theta"], b["grads"], b["m"], b["v"], b["steps"], plan, GROUPS[0],
                               grad_scale=b["scale"], lr_scale=b["lr_scale"], working=b["work"])

    e, c, d = state(), state(), state()
    graphs = []
    for b in (c, d):  # capture runs nothing
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                step(b)
        graphs.append(graph)
    torch.cuda.synchronize()
    for rep in range(4):
        g = torch.randn((k, stride), device=DEV, generator=torch.Generator(DEV).manual_seed(rep)).to(torch.bfloat16) * 0.01
        if rep == 2:
            g[1, 64] = math.inf  # learner 1's step is left out, and its count stays
        for b in (e, c, d):
            b["grads"].copy_(g)
            b["lr_scale"].fill_(1.0 / (rep + 1))
        step(e)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
            torch.randn(1 << 20, device=DEV).sum()
        torch.cuda.synchronize()
        for b in (c, d):
            for n in e:
                if n not in ("mask", "ws"):
                    assert torch.equal(torch.nan_to_num(b[n].float()), torch.nan_to_num(e[n].float())), (rep, n)
    assert e["steps"].tolist() == [4, 40 + 3, 80 + 4]


def test_calls_on_another_stream_follow_that_stream():
    tensors, stride = layout([1 << 20, 12345])
    a, b = draw(2, stride, tensors, [1, 1]), draw(2, stride, tensors, [1, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        dlc.dlc_adamw_step(a["theta"], a["grads"], a["m"], a["v"], a["steps"], tensors)
    for _ in range(3):
        dlc.dlc_adamw_step(b["theta"], b["grads"], b["m"], b["v"], b["steps"], tensors, stream=s)
    torch.cuda.synchronize()
    for n in ("theta", "m", "v", "steps"):
        assert torch.equal(a[n], b[n])


def test_two_streams_at_once_with_buffers_of_their_own():
    """Norm and step of two models, four passes each, side by side on two streams: as one after the other."""
    tensors, stride = layout([1 << 21, 12345, 64 * 1000])
    plan = dlc.TensorList(tensors)

    def state(seed):
        b = draw(2, stride, tensors, [1, 1], "bf16", seed)
        coded_start(b, 2, stride, seed)
        b["norm"], b["scale"] = (torch.zeros(2, dtype=torch.float64, device=DEV) for _ in range(2))
        b["ws"] = dlc.alloc_grad_norm_workspace(2, plan)
        return b

    def steps(b, coded, stream):
        for _ in range(4):
            dlc.dlc_grad_norm(b["grads"], plan, b["norm"], b["scale"], b["ws"], max_norm=0.5, stream=stream)
            if coded:
                dlc.dlc_adamw_coded_step(b["theta"], b["grads"], b["mc"].view(torch.float8_e4m3fn), b["ms"],
                                         b["vc"].view(torch.float8_e5m2), b["vs"], b["steps"], plan, seed=3,
                                         grad_scale=b["scale"], stream=stream)
            else:
                dlc.dlc_adamw_step(b["theta"], b["grads"], b["m"], b["v"], b["steps"], plan, grad_scale=b["scale"],
                                   stream=stream)

    alone, beside = [state(1), state(2)], [state(1), state(2)]
    for k, b in enumerate(alone):
        steps(b, k == 1, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k, b in enumerate(beside):
        steps(b, k == 1, streams[k])
    torch.cuda.synchronize()
    for a, b in zip(alone, beside):
        for n in a:
            if n not in ("mask", "ws"):
                assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("coded", [False, True])
def test_two_whole_rounds_of_inner_and_outer_steps(coded):
    """What the calls are for: H inner steps of every learner (norm, clipping, AdamW), then the
    outer step (quantize, merge) and the update sent back; twice, against the oracles."""
    sizes, k, rounds, h = [64 * 30, 1000, 4097, 64], 3, 2, 3
    tensors, stride = layout(sizes)
    plan = dlc.TensorList(tensors)
    gen = torch.Generator().manual_seed(3)
    glen = max(o + n for o, _, n in tensors)
    theta_g = (torch.randn(glen, generator=gen) * 0.02).to(DEV)
    mom = torch.zeros(glen, device=DEV)
    b = draw(k, stride, tensors, [1] * k)
    coded_start(b, k, stride)
    b["steps"].zero_()
    for n in ("m", "v", "mc", "ms", "vc", "vs"):
        b[n].zero_()
    codes, cb, rng = dlc.outputs_for(k, stride, len(plan))
    ws, nws = dlc.alloc_workspace(k, plan), dlc.alloc_grad_norm_workspace(k, plan)
    norm, scale = (torch.zeros(k, dtype=torch.float64, device=DEV) for _ in range(2))
    dlc.dlc_broadcast(theta_g, b["theta"], plan)
    for rnd in range(rounds):
        for _ in range(h):
            g = (torch.randn((k, stride), generator=gen) * 0.01).to(torch.bfloat16)
            b["grads"] = g.to(DEV)
            ref = {n: host(b[n]).copy() for n in ("theta", "m", "v", "steps", "mc", "ms", "vc", "vs")}
            dlc.dlc_grad_norm(b["grads"], plan, norm, scale, nws, max_norm=0.6)
            if coded:
                coded_call(b, plan, GROUPS[0], None, 1, scale.tolist(), None, None, None)
                size = inner.adamw_coded(ref["theta"], host(g), ref["mc"], ref["ms"], ref["vc"], ref["vs"], ref["steps"],
                                         tensors, GROUPS, None, 1, scale.tolist())
            else:
                dlc.dlc_adamw_step(b["theta"], b["grads"], b["m"], b["v"], b["steps"], plan, GROUPS[0], grad_scale=scale)
                size = inner.adamw(ref["theta"], host(g), ref["m"], ref["v"], ref["steps"], tensors, GROUPS, None,
                                   scale.tolist())
            torch.cuda.synchronize()
            assert all(0 < x < 1 for x in scale.tolist())
            near_theta(host(b["theta"]), ref["theta"], size, b["mask"], "theta")
        want = oracle.outer_step(host(theta_g), host(mom), host(b["theta"]), stride, tensors, [1.0] * k, [1] * k, 0.7, 0.9)
        dlc.dlc_quantize(theta_g, b["theta"], plan, codes, cb, rng, ws)
        dlc.dlc_merge_outer_step(theta_g, mom, codes, cb, [1.0] * k, plan)
        dlc.dlc_broadcast(theta_g, b["theta"], plan)
        torch.cuda.synchronize()
        for o, lo, n in tensors:
            th, wt = host(theta_g)[o:o + n], want["theta"][o:o + n]
            assert np.all(np.abs(th - wt) <= 1e-9 + 1e-5 * np.abs(wt))
            assert torch.equal(b["theta"][:, lo:lo + n], theta_g[o:o + n].expand(k, n))
    assert b["steps"].tolist() == [rounds * h] * k
