"""The mixture-of-experts calls refuse what they cannot run, before anything reaches the device: the C ABI's
argument errors (nothing is launched, the addresses are never dereferenced) and the binding's checks on host
tensors.  The same tests run once more against the library with its host code under the sanitizers.  The oracle's
definitions are pinned here too."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import diloco_outer_step_amd as dlc
from oracle import core, experts
from tests.test_host_sanitizers import CLANG, ROOT, asan_runtime, hostsan_library
from tests.test_inner_host import ALIGN, F, INVALID, QUORUM, WORKSPACE, bytes_of, tens

L = dlc._lib
NAN, INF = float("nan"), float("inf")


def doubles(v):
    return None if v is None else ctypes.cast((ctypes.c_double * max(1, len(v)))(*v), ctypes.c_void_p)


def ints(v):
    return None if v is None else ctypes.cast((ctypes.c_int32 * max(1, len(v)))(*v), ctypes.c_void_p)


def balance(x=F[0], xt=0, xl=800, xs=8, c=F[1], ct=1, cl=200, cs=2, mask=F[2], ml=100, k=2, present=None, t=100, e=8,
            top=2, coef=1.0, loss=F[3], counts=F[4], ns=8, means=F[5], totals=F[6], ts=8, g=F[7], gl=800, gs=8, up=F[8],
            flags=0, ws=F[9], ws_bytes=1 << 20):
    return L.dlc_expert_balance(x, xt, xl, xs, c, ct, cl, cs, mask, ml, k, bytes_of(present), t, e, top, coef, loss, counts,
                                ns, means, totals, ts, g, gl, gs, up, flags, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(t=-1), INVALID), (dict(t=(1 << 24) + 1), INVALID),
    (dict(e=0), INVALID), (dict(e=1025), INVALID), (dict(top=0), INVALID), (dict(top=9), INVALID),
    (dict(e=100, top=65), INVALID), (dict(xt=3), INVALID), (dict(xt=-1), INVALID), (dict(ct=2), INVALID),
    (dict(flags=1), INVALID), (dict(flags=17), INVALID), (dict(coef=NAN), INVALID), (dict(coef=INF), INVALID),
    (dict(x=None), INVALID), (dict(c=None), INVALID), (dict(loss=None), INVALID), (dict(counts=None), INVALID),
    (dict(present=[0, 0]), QUORUM), (dict(xl=-8), INVALID), (dict(xs=-1), INVALID), (dict(cl=-1), INVALID),
    (dict(cs=(1 << 48) + 1), INVALID), (dict(xs=1 << 47), INVALID), (dict(gl=1 << 62), INVALID), (dict(ns=1 << 62), INVALID),
    (dict(ts=-8), INVALID), (dict(ml=1 << 60), INVALID), (dict(ml=-1), INVALID), (dict(gl=-800), INVALID),
    (dict(x=F[0] + 2), ALIGN), (dict(x=F[0] + 1, xt=1), ALIGN), (dict(c=F[1] + 4), ALIGN), (dict(c=F[1] + 2, ct=0), ALIGN),
    (dict(g=F[7] + 1), ALIGN), (dict(loss=F[3] + 2), ALIGN), (dict(means=F[5] + 1), ALIGN), (dict(counts=F[4] + 4), ALIGN),
    (dict(totals=F[6] + 4), ALIGN), (dict(up=F[8] + 4), ALIGN), (dict(ws=F[9] + 8), ALIGN),
    (dict(gs=7), INVALID), (dict(gl=0), INVALID), (dict(gl=799), INVALID), (dict(ns=7), INVALID), (dict(ts=7), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=64, t=9000, xl=72000, gl=72000, cl=18000, ml=9000), WORKSPACE),
])
def test_the_balance_loss_refuses(bad, code):
    assert balance(**bad) == code and dlc.dlc_last_error()


@pytest.mark.parametrize("bad", [
    dict(g=F[0]), dict(g=F[0] + 2 * 3200 - 4), dict(g=F[1] + 8), dict(loss=F[0] + 4), dict(loss=F[4] + 4),
    dict(means=F[3] + 4), dict(counts=F[6]), dict(totals=F[4] + 64), dict(up=F[3]), dict(counts=F[1] + 80),
    dict(mask=F[7] + 5), dict(means=F[7] + 32), dict(loss=F[2] + 8), dict(up=F[6] + 8),
    dict(g=F[0], present=[0, 1]),
])
def test_the_balance_loss_refuses_buffers_that_overlap(bad):
    assert balance(**bad) == INVALID and "overlap" in dlc.dlc_last_error()


def test_the_workspace_serves_every_type_presence_and_number_of_choices():
    sizes = []
    for k, t, e in ((1, 0, 1), (1, 1, 1), (8, 32768, 256), (64, 1 << 24, 1024), (3, 5003, 60), (64, 100, 1024)):
        out = ctypes.c_size_t(0)
        assert L.dlc_expert_balance_workspace_bytes(k, t, e, ctypes.byref(out)) == 0
        sizes.append(out.value)
        wide = dict(t=t, e=e, k=k, xs=e, xl=t * e, cs=64, cl=64 * t, ml=t, gs=e, gl=t * e, ns=e, ts=e)
        far = dict(x=1 << 45, g=1 << 46, c=1 << 47, mask=1 << 44, ws=1 << 43)
        if t < 1000:
            continue
        # every need is met: the call fails for its workspace one byte below some need, never at the whole
        for xt in (0, 1):
            for top in (1, min(e, 64)):
                assert balance(**wide, **far, xt=xt, top=top, ws_bytes=0) == WORKSPACE
                need = int(dlc.dlc_last_error().split("need ")[1].split()[0])
                assert need <= out.value
    assert sizes[3] < 1 << 31 and sizes[2] < 1 << 24
    for bad in ((0, 1, 1), (65, 1, 1), (1, -1, 1), (1, 1 << 25, 1), (1, 1, 0), (1, 1, 1025)):
        assert L.dlc_expert_balance_workspace_bytes(*bad, ctypes.byref(out)) == INVALID
    assert L.dlc_expert_balance_workspace_bytes(1, 1, 1, None) == INVALID


def weights(counts=F[0], stride=4, k=2, e=4, w=(1.0, 2.0), q=None, of=(-1, 0, 3), n=None, out=F[1]):
    return L.dlc_expert_weights(counts, stride, k, e, doubles(w), doubles(q), ints(of), len(of or ()) if n is None else n,
                                out, None)


@pytest.mark.parametrize("bad,code", [
    (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(counts=None), INVALID), (dict(w=None), INVALID),
    (dict(of=None), INVALID), (dict(out=None), INVALID), (dict(e=0), INVALID), (dict(e=32768, stride=40000), INVALID),
    (dict(n=0), INVALID), (dict(counts=F[0] + 4), ALIGN), (dict(out=F[1] + 4), ALIGN), (dict(stride=3), INVALID),
    (dict(stride=-4), INVALID), (dict(stride=1 << 60), INVALID), (dict(w=(-1.0, 2.0)), INVALID), (dict(w=(NAN, 2.0)), INVALID), (dict(w=(INF, 2.0)), INVALID),
    (dict(w=(0.0, 0.0)), QUORUM), (dict(q=(-1.0, 1.0)), INVALID), (dict(q=(1.0, NAN)), INVALID), (dict(of=(4,)), INVALID),
    (dict(q=(1.0, 1e300)), INVALID), (dict(w=(1.5e308, 1.5e308)), INVALID),
    (dict(of=(-2,)), INVALID), (dict(out=F[0] + 8), INVALID), (dict(out=F[0] + 56), INVALID),
])
def test_the_merge_weights_refuse(bad, code):
    assert weights(**bad) == code and dlc.dlc_last_error()


def outer_norm(codes=F[0], stride=4096, k=2, cb=F[1], w=(1.0, 1.0), tw=None, spec=((0, 0, 4096),), max_norm=1.0, norm=F[2],
               scale=F[3], ws=F[4], ws_bytes=1 << 16):
    arr, n = tens(spec)
    return L.dlc_outer_grad_norm(codes, stride, k, cb, doubles(w), tw, arr, n, max_norm, norm, scale, ws, ws_bytes, None)


SHARED = [
    (dict(k=0), INVALID), (dict(k=65, w=[1.0] * 65), INVALID), (dict(codes=None), INVALID), (dict(cb=None), INVALID),
    (dict(w=None), INVALID), (dict(codes=F[0] + 64), ALIGN), (dict(cb=F[1] + 4), ALIGN), (dict(tw=F[5] + 4), ALIGN),
    (dict(w=(0.0, 0.0)), QUORUM), (dict(w=(NAN, 1.0)), INVALID), (dict(w=(-1.0, 1.0)), INVALID), (dict(spec=()), INVALID),
    (dict(spec=((0, 0, 4097),)), INVALID), (dict(spec=((0, 32, 64),)), ALIGN), (dict(stride=100), ALIGN),
    (dict(spec=((0, 0, 100), (64, 128, 100))), INVALID),
]


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(norm=None), INVALID), (dict(scale=None), INVALID), (dict(norm=F[2] + 4), ALIGN), (dict(scale=F[3] + 4), ALIGN),
    (dict(max_norm=0.0), INVALID), (dict(max_norm=-1.0), INVALID), (dict(max_norm=NAN), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=0), WORKSPACE), (dict(ws=F[4] + 8), ALIGN), (dict(scale=F[2]), INVALID), (dict(norm=F[4]), INVALID),
    (dict(norm=F[0] + 4096), INVALID), (dict(scale=F[1] + 2048 - 8), INVALID), (dict(ws=F[0]), INVALID),
    (dict(tw=F[2]), INVALID), (dict(tw=F[3] - 8), INVALID),
])
def test_the_outer_norm_refuses(bad, code):
    assert outer_norm(**bad) == code and dlc.dlc_last_error()


def step(theta=F[2], mom=F[3], codes=F[0], stride=4096, k=2, cb=F[1], w=(1.0, 1.0), tw=None, scale=None,
         spec=((0, 0, 4096),), lr=0.7, beta=0.9):
    arr, n = tens(spec)
    return L.dlc_merge_clipped_step(theta, mom, codes, stride, k, cb, doubles(w), tw, scale, arr, n, lr, beta, None)


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(theta=None), INVALID), (dict(mom=None), INVALID), (dict(theta=F[2] + 64), ALIGN), (dict(mom=F[3] + 4), ALIGN),
    (dict(scale=F[5] + 4), ALIGN), (dict(lr=NAN), INVALID), (dict(beta=INF), INVALID), (dict(mom=F[2]), INVALID),
    (dict(mom=F[2] + 4 * 4096 - 256), INVALID), (dict(theta=F[0] + 4096), INVALID), (dict(mom=F[1] + 1024), INVALID),
    (dict(scale=F[2] + 8), INVALID), (dict(tw=F[3] + 4 * 4096 - 8), INVALID),
])
def test_the_clipped_step_refuses(bad, code):
    assert step(**bad) == code and dlc.dlc_last_error()


# --- the binding -------------------------------------------------------------------------------

K, T, E, TOP = 2, 10, 6, 2


def good():
    return dict(logits=torch.zeros((K, T, E)), choices=torch.zeros((K, T, TOP), dtype=torch.int64), loss=torch.zeros(K),
                counts=torch.zeros((K, E), dtype=torch.int64), workspace=torch.zeros(4096, dtype=torch.uint8),
                mask=torch.ones((K, T), dtype=torch.bool), mean_probs=torch.zeros((K, E)),
                grad_logits=torch.zeros((K, T, E)), grad_scale=torch.ones(K, dtype=torch.float64),
                totals=torch.zeros((K, E), dtype=torch.int64))


def call(**change):
    b = {**good(), **change}
    first = [b.pop(n) for n in ("logits", "choices", "loss", "counts", "workspace")]
    dlc.dlc_expert_balance(*first, **b)


@pytest.mark.parametrize("change", [
    dict(logits=torch.zeros((K, T))), dict(logits=torch.zeros((K, T, E), dtype=torch.float64)),
    dict(logits=torch.zeros((K, T, 2 * E))[:, :, ::2]), dict(choices=torch.zeros((K, T, TOP))),
    dict(choices=torch.zeros((K, T + 1, TOP), dtype=torch.int64)), dict(choices=torch.zeros((K, T), dtype=torch.int64)),
    dict(choices=torch.zeros((K, TOP, T), dtype=torch.int64).transpose(1, 2)), dict(loss=torch.zeros(K + 1)),
    dict(loss=torch.zeros(K, dtype=torch.float64)), dict(loss=torch.zeros(2 * K)[::2]),
    dict(counts=torch.zeros((K, E), dtype=torch.int32)), dict(counts=torch.zeros((K, E + 1), dtype=torch.int64)),
    dict(counts=torch.zeros((E, K), dtype=torch.int64).T), dict(workspace=torch.zeros(4096)),
    dict(mask=torch.ones((K, T + 1), dtype=torch.bool)), dict(mask=torch.ones((K, T))),
    dict(mask=torch.ones((T, K), dtype=torch.bool).T), dict(mean_probs=torch.zeros((K, E + 1))),
    dict(mean_probs=torch.zeros((K, 2 * E))[:, :E]), dict(grad_logits=torch.zeros((K, T, E), dtype=torch.bfloat16)),
    dict(grad_logits=torch.zeros((K, T, E + 1))), dict(grad_logits=torch.zeros((K, E, T)).transpose(1, 2)),
    dict(grad_scale=torch.ones(K)), dict(grad_scale=torch.ones(K + 1, dtype=torch.float64)),
    dict(totals=torch.zeros((K, E))), dict(present=[1]), {},
])
def test_the_binding_refuses_before_the_library(change):
    with pytest.raises(ValueError):  # the last one: host tensors
        call(**change)


@pytest.mark.parametrize("name", ["choices", "counts", "mask", "totals", "grad_logits", "loss", "workspace", "mean_probs"])
def test_the_binding_wants_tensors(name):
    with pytest.raises((TypeError, ValueError)):
        call(**{name: [0]})


def test_the_binding_of_the_outer_calls_refuses():
    codes = torch.zeros((2, 256), dtype=torch.uint8)
    cb, th = torch.zeros((2, 1, 256)), torch.zeros(256)
    one = torch.zeros(1, dtype=torch.float64)
    ws = torch.zeros(256, dtype=torch.uint8)
    tensors = [(0, 0, 100)]
    for bad in (dict(tensors=[(0, 0, 300)]), dict(w=[1.0]), dict(cb=torch.zeros((1, 1, 256))), dict(cb=cb.double()),
                dict(one=torch.zeros(2, dtype=torch.float64)), dict(one=torch.zeros(1)), dict(codes=codes.int()),
                dict(tw=torch.zeros((2, 2), dtype=torch.float64)), dict(tw=torch.zeros((1, 2))), {}):
        a = {**dict(tensors=tensors, w=[1.0, 1.0], cb=cb, one=one, codes=codes, tw=None), **bad}
        with pytest.raises(ValueError):
            dlc.dlc_outer_grad_norm(a["codes"], a["cb"], a["w"], a["tensors"], a["one"], a["one"], ws,
                                    tensor_weights=a["tw"])
        with pytest.raises(ValueError):
            dlc.dlc_merge_clipped_step(th, th, a["codes"], a["cb"], a["w"], a["tensors"], grad_scale=a["one"],
                                       tensor_weights=a["tw"])
    for bad in (torch.zeros(99), torch.zeros(256, dtype=torch.float64), torch.zeros(512)[::2]):
        with pytest.raises(ValueError):
            dlc.dlc_merge_clipped_step(bad, th, codes, cb, [1.0, 1.0], tensors)
        with pytest.raises(ValueError):
            dlc.dlc_merge_clipped_step(th, bad, codes, cb, [1.0, 1.0], tensors)
    counts = torch.zeros((2, 3), dtype=torch.int64)
    out = torch.zeros((2, 2), dtype=torch.float64)
    for bad in (dict(counts=counts.int()), dict(counts=counts[0]), dict(w=[1.0]), dict(of=[0]), dict(q=[1.0]),
                dict(out=out.float()), {}):
        a = {**dict(counts=counts, w=[1.0, 1.0], of=[0, 1], q=None, out=out), **bad}
        with pytest.raises(ValueError):
            dlc.dlc_expert_weights(a["counts"], a["w"], a["of"], a["out"], token_weight=a["q"])


# --- the oracle ----------------------------------------------------------------------------------

def test_the_balance_loss_by_hand():
    x = np.log(np.array([[1.0, 3.0], [2.0, 2.0]]))
    loss, counts, means, grad = experts.balance(x, np.array([[1], [1]]), coef=2.0)
    assert counts.tolist() == [0, 2] and means == pytest.approx([0.375, 0.625])
    assert loss == pytest.approx(2 * 2 * 0.625)
    # d loss / d x = 4 * (1 / 2) p0 p1 on the chosen side
    assert grad[:, 1] == pytest.approx([2 * 0.25 * 0.75, 2 * 0.25]) and grad[:, 0] == pytest.approx(-grad[:, 1])


def test_the_oracles_gradient_against_differences_and_against_autograd():
    rng = np.random.default_rng(0)
    x, ids = rng.normal(size=(9, 5)), rng.integers(-1, 6, (9, 3))
    mask = rng.random(9) < 0.7
    loss, counts, means, grad = experts.balance(x, ids, mask, 0.3, 2.0)
    t = torch.tensor(x, requires_grad=True)
    p = torch.softmax(t, -1) * torch.tensor(mask)[:, None]
    n = mask.sum()
    f = torch.tensor([sum(int(v == e) for row, m in zip(ids, mask) if m for v in row) for e in range(5)], dtype=torch.float64) / (n * 3.0)
    want = 0.3 * 5 * (f * p.sum(0) / n).sum()
    want.backward()
    assert loss == pytest.approx(want.item()) and np.allclose(grad, 2 * t.grad.numpy(), atol=1e-15)
    h = 1e-6
    for i in range(9):
        for j in range(5):
            up, down = x.copy(), x.copy()
            up[i, j] += h
            down[i, j] -= h
            d = (experts.balance(up, ids, mask, 0.3)[0] - experts.balance(down, ids, mask, 0.3)[0]) / (2 * h)
            assert abs(2 * d - grad[i, j]) < 1e-8


def test_the_merge_weights_by_hand():
    counts = [[10, 0, 7], [30, 0, 7], [99, 0, 7]]
    got = experts.tensor_weights(counts, [1.0, 3.0, 0.0], [-1, 0, 1, 2], [1.0, 2.0, 1.0])
    assert got.tolist() == [[0.25, 0.75, 0], [10 / 70, 60 / 70, 0], [0.25, 0.75, 0], [7 / 21, 14 / 21, 0]]


def test_the_clipped_step_is_the_outer_step_of_a_shorter_gradient():
    rng = np.random.default_rng(1)
    codes, cb = rng.integers(0, 256, (2, 128), dtype=np.uint8), rng.normal(size=(2, 2, 256)).astype(np.float32)
    tensors, w = [(0, 64, 60), (64, 0, 50)], [1.0, 3.0]
    norm, scale = experts.outer_grad_norm(codes, cb, w, tensors, max_norm=0.5)
    g = [core.merge([codes[i, lo:lo + n] for i in range(2)], [cb[i, t] for i in range(2)], [0.25, 0.75])
         for t, (_, lo, n) in enumerate(tensors)]
    assert norm == pytest.approx(float(np.linalg.norm(np.concatenate(g)))) and scale * norm == pytest.approx(0.5)
    th, mo = rng.normal(size=128).astype(np.float32), rng.normal(size=128).astype(np.float32)
    a, b = th.copy(), mo.copy()
    experts.clipped_step(a, b, codes, cb, w, tensors, scale=scale)
    for t, (off, _, n) in enumerate(tensors):
        want = core.nesterov(th[off:off + n], mo[off:off + n], scale * g[t])
        assert np.allclose(a[off:off + n], want[0], rtol=1e-6) and np.allclose(b[off:off + n], want[1], rtol=1e-6)
    assert np.array_equal(a[60:64], th[60:64]) and np.array_equal(a[114:], th[114:])
    c = th.copy()
    experts.clipped_step(c, mo.copy(), codes, cb, w, tensors, scale=0.0)
    assert np.array_equal(c, th)


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
