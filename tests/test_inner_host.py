"""The inner step's calls refuse what they cannot run, before anything reaches the device: the
C ABI's argument errors (nothing is launched, the addresses are never dereferenced) and the
binding's buffer checks on host tensors.  The same tests run once more against the library
with its host code under the sanitizers."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import diloco_outer_step_amd as dlc
from tests.test_host_sanitizers import CLANG, ROOT, asan_runtime, hostsan_library

F = [(i + 1) << 20 for i in range(16)]  # aligned addresses that are never dereferenced
L = dlc._lib
GOOD = (1e-3, 0.9, 0.999, 1e-8, 0.01)


def tens(spec):
    arr = (dlc._Tensor * max(1, len(spec)))()
    for i, (o, lo, n) in enumerate(spec):
        arr[i].offset, arr[i].loffset, arr[i].numel = o, lo, n
    return arr, len(spec)


def bytes_of(values):
    return None if values is None else ctypes.cast((ctypes.c_uint8 * len(values))(*values), ctypes.c_void_p)


def norm(k=2, spec=((0, 0, 4096),), stride=4096, grads=F[0], gt=0, present=None, unscale=1.0, max_norm=1.0, out=F[1],
         scale=F[2], ws=F[3], ws_bytes=1 << 20):
    arr, n = tens(spec)
    return L.dlc_grad_norm(grads, gt, stride, k, bytes_of(present), arr, n, unscale, max_norm, out, scale, ws, ws_bytes,
                           None)


def step(coded, k=2, spec=((0, 0, 4096),), stride=4096, theta=F[0], grads=F[1], gt=0, m=F[2], v=F[3], ms=F[4], vs=F[5],
         steps=F[6], present=None, groups=(GOOD,), n_groups=None, group_of=None, gs=None, lrs=None, work=None, wt=1):
    arr, n = tens(spec)
    flat = [x for g in groups or () for x in g]
    g = None if groups is None else ctypes.cast((ctypes.c_double * max(1, len(flat)))(*flat), ctypes.c_void_p)
    ids = None if group_of is None else ctypes.cast((ctypes.c_int32 * len(group_of))(*group_of), ctypes.c_void_p)
    ng = (0 if groups is None else len(groups)) if n_groups is None else n_groups
    if coded:
        return L.dlc_adamw_coded_step(theta, grads, gt, m, ms, v, vs, steps, stride, k, bytes_of(present), arr, n, ids, g,
                                      ng, 0, gs, lrs, work, wt, None)
    return L.dlc_adamw_step(theta, grads, gt, m, v, steps, stride, k, bytes_of(present), arr, n, ids, g, ng, gs, lrs, work,
                            wt, None)


INVALID, ALIGN, QUORUM, WORKSPACE = (dlc.DLC_ERR_INVALID_ARGUMENT, dlc.DLC_ERR_ALIGNMENT, dlc.DLC_ERR_NO_QUORUM,
                                     dlc.DLC_ERR_WORKSPACE)
SHARED = [
    (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(grads=None), INVALID), (dict(grads=F[0] + 64), ALIGN),
    (dict(gt=3), INVALID), (dict(gt=-1), INVALID), (dict(present=[0, 0]), QUORUM), (dict(spec=()), INVALID),
    (dict(spec=((0, 0, 4097),)), INVALID), (dict(spec=((0, 0, 0),)), INVALID), (dict(spec=((0, 32, 64),)), ALIGN),
    (dict(spec=((0, -64, 64),)), INVALID), (dict(stride=4000), ALIGN), (dict(stride=0), ALIGN),
    (dict(spec=((0, 0, 100), (128, 64, 100))), INVALID),
]


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(out=None), INVALID), (dict(scale=None), INVALID), (dict(out=F[1] + 4), ALIGN), (dict(scale=F[1]), INVALID),
    (dict(unscale=0.0), INVALID), (dict(unscale=float("inf")), INVALID), (dict(unscale=float("nan")), INVALID),
    (dict(max_norm=0.0), INVALID), (dict(max_norm=float("nan")), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=8), WORKSPACE), (dict(ws=F[3] + 8), ALIGN),
])
def test_grad_norm_argument_errors(bad, code):
    assert norm(**bad) == code and dlc.dlc_last_error() != ""


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(theta=None), INVALID), (dict(m=None), INVALID), (dict(v=None), INVALID), (dict(steps=None), INVALID),
    (dict(theta=F[0] + 128), ALIGN), (dict(v=F[3] + 16), ALIGN), (dict(steps=F[6] + 4), ALIGN), (dict(gs=F[7] + 4), ALIGN),
    (dict(lrs=F[7] + 2), ALIGN), (dict(work=F[8], wt=0), INVALID), (dict(work=F[8], wt=5), INVALID),
    (dict(work=F[8] + 32), ALIGN), (dict(m=F[3]), INVALID), (dict(grads=F[0]), INVALID), (dict(work=F[1]), INVALID),
    (dict(groups=None), INVALID), (dict(n_groups=0), INVALID), (dict(groups=(GOOD,) * 17), INVALID),
    (dict(group_of=[1]), INVALID), (dict(group_of=[-1]), INVALID),
    (dict(groups=((-1e-3,) + GOOD[1:],)), INVALID), (dict(groups=((float("inf"),) + GOOD[1:],)), INVALID),
    (dict(groups=((1e-3, 1.0, 0.999, 1e-8, 0.0),)), INVALID), (dict(groups=((1e-3, 0.9, -0.1, 1e-8, 0.0),)), INVALID),
    (dict(groups=((1e-3, 0.9, 0.999, 0.0, 0.0),)), INVALID), (dict(groups=((1e-3, 0.9, 0.999, 1e-40, 0.0),)), INVALID),
    (dict(groups=((1e-3, 0.9, 0.999, 1e-8, -0.1),)), INVALID), (dict(groups=((1e-3, float("nan"), 0.9, 1e-8, 0.1),)), INVALID),
])
def test_adamw_argument_errors(coded, bad, code):
    assert step(coded, **bad) == code and dlc.dlc_last_error() != ""


@pytest.mark.parametrize("bad", [dict(ms=None), dict(vs=None), dict(ms=F[5]), dict(vs=F[2])])
def test_coded_moments_need_their_own_scales(bad):
    assert step(True, **bad) == INVALID


def test_the_norm_workspace_grows_with_learners_and_covers_many_tensors():
    a = dlc.dlc_grad_norm_workspace_bytes(1, [(0, 0, 1 << 24)])
    b = dlc.dlc_grad_norm_workspace_bytes(16, [(0, 0, 1 << 24)])
    assert 0 < a < b and a % 256 == 0
    many = [(128 * i, 128 * i, 65) for i in range(3000)]
    assert dlc.dlc_grad_norm_workspace_bytes(2, many) >= 2 * 3000 * 8
    big = [(0, 0, (1 << 32) - 1), (1 << 32, 1 << 32, (1 << 32) - 64), (1 << 33, 1 << 33, 64)]
    assert dlc.dlc_grad_norm_workspace_bytes(64, big) > 0
    with pytest.raises(dlc.DlcError):
        dlc.dlc_grad_norm_workspace_bytes(0, [(0, 0, 64)])


# --- the binding -------------------------------------------------------------------

K, STRIDE = 3, 256
TENSORS = [(0, 0, 100), (128, 128, 70)]


def good():
    mc, ms, vc, vs = dlc.coded_moments(K, STRIDE, "cpu")
    z = torch.zeros
    return dict(theta_L=z((K, STRIDE)), grads=z((K, STRIDE), dtype=torch.bfloat16), exp_avg=z((K, STRIDE)),
                exp_avg_sq=z((K, STRIDE)), steps=z(K, dtype=torch.int64), m_codes=mc, m_scales=ms, v_codes=vc, v_scales=vs,
                grad_scale=z(K, dtype=torch.float64), lr_scale=z(K, dtype=torch.float64),
                working=z((K, STRIDE), dtype=torch.float16), norm=z(K, dtype=torch.float64),
                workspace=z(4096, dtype=torch.uint8))


def call(name, b, tensors=TENSORS, **kw):
    if name == "norm":
        dlc.dlc_grad_norm(b["grads"], tensors, b["norm"], b["grad_scale"], b["workspace"], **kw)
        return
    kw = dict(grad_scale=b["grad_scale"], lr_scale=b["lr_scale"], working=b["working"], **kw)
    if name == "adamw":
        dlc.dlc_adamw_step(b["theta_L"], b["grads"], b["exp_avg"], b["exp_avg_sq"], b["steps"], tensors, **kw)
    else:
        dlc.dlc_adamw_coded_step(b["theta_L"], b["grads"], b["m_codes"], b["m_scales"], b["v_codes"], b["v_scales"],
                                 b["steps"], tensors, **kw)


USES = {"norm": ("grads", "norm", "grad_scale", "workspace"),
        "adamw": ("theta_L", "grads", "exp_avg", "exp_avg_sq", "steps", "grad_scale", "lr_scale", "working"),
        "coded": ("theta_L", "grads", "m_codes", "m_scales", "v_codes", "v_scales", "steps", "grad_scale", "lr_scale",
                  "working")}


@pytest.mark.parametrize("name", sorted(USES))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="device tensor"):
        call(name, good())
    with pytest.raises(ValueError, match="device tensor"):
        call(name, good(), tensors=dlc.TensorList(TENSORS))


@pytest.mark.parametrize("name,buf", [(n, b) for n in sorted(USES) for b in USES[n]])
def test_wrong_dtype_layout_or_size_is_refused_before_the_device_check(name, buf):
    t = good()[buf]
    bad = [None if buf in ("grad_scale", "lr_scale", "working") and name != "norm" else 7, t.to(torch.complex64)]
    if t.dim() == 2:
        bad += [t.t().contiguous().t(), t[:, : t.shape[1] // 2].contiguous(), t[:2].contiguous(), t[0].contiguous()]
    elif buf != "workspace":
        bad += [t[:2].contiguous(), t.repeat(2)[::2]]
    for x in bad:
        if x is None:
            continue
        b = good()
        b[buf] = x
        with pytest.raises((ValueError, TypeError)) as e:
            call(name, b)
        assert "device tensor" not in str(e.value), (name, buf, str(e.value))


@pytest.mark.parametrize("name", sorted(USES))
def test_lists_must_match_the_call(name):
    with pytest.raises(ValueError, match="present holds 2 values"):
        call(name, good(), present=[1, 1])
    with pytest.raises(ValueError, match="reaches past"):
        call(name, good(), tensors=[(0, 192, 65)])
    if name != "norm":
        with pytest.raises(ValueError, match="group_of holds 3 values for 2 tensors"):
            call(name, good(), group_of=[0, 0, 0])
        with pytest.raises(ValueError, match="AdamWGroup"):
            call(name, good(), groups=[(1e-3, 0.9)])
    if name == "coded":
        for seed in (-1, 1 << 64):
            with pytest.raises(ValueError, match="seed"):
                call(name, good(), seed=seed)


def test_a_tensor_list_is_the_list_it_was_made_from():
    t = dlc.TensorList(TENSORS)
    assert list(t) == TENSORS and t == tuple(TENSORS)
    assert dlc.dlc_workspace_bytes(4, t) == dlc.dlc_workspace_bytes(4, TENSORS)
    assert dlc._extents(t) == dlc._extents(TENSORS)
    arr, n = dlc._tensors(t)
    assert n == 2 and (arr[1].offset, arr[1].loffset, arr[1].numel) == TENSORS[1]
    assert dlc._tensors(dlc.TensorList([]))[1] == 0
    ids = dlc.group_ids(np.array([0, 1]))
    assert list(ids) == [0, 1] and ids.itemsize == 4 and dlc.group_ids(ids) is ids


def test_a_call_runs_on_its_buffers_device_and_stream(monkeypatch):
    """Buffers on another device than the current one: that device is current during the call and its
    own current stream is used; a stream of another device is refused."""
    seen = []

    class Guard:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            seen.append(("enter", self.index))

        def __exit__(self, *exc):
            seen.append(("exit", self.index))

    class Stream:
        def __init__(self, index):
            self.device, self.cuda_stream = torch.device("cuda", index), 777

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)

    def fn(*args):
        seen.append(args)
        return 0

    dlc._on_device(0, None, fn, 5)
    dlc._on_device(1, None, fn, 6)
    assert seen == [(5, 1000), ("enter", 1), (6, 1001), ("exit", 1)]
    dlc._on_device(1, Stream(1), fn, 7)
    assert seen[-2][1].value == 777
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        dlc._on_device(1, Stream(0), fn, 8)


@pytest.mark.skipif(not os.path.exists(CLANG) or asan_runtime() is None,
                    reason="ROCm clang with the sanitizer runtimes is not installed")
@pytest.mark.skipif("DLC_LIBRARY" in os.environ, reason="already under the sanitizers")
def test_these_tests_under_the_sanitizers():
    env = dict(os.environ, LD_PRELOAD=asan_runtime(), DLC_LIBRARY=hostsan_library(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu", __file__],
                       capture_output=True, text=True, timeout=900, env=env, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-3000:]
