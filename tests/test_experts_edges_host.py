"""More refusals of the mixture-of-experts calls, on host tensors and made-up addresses: nothing is launched."""
import ctypes
import os
import random
import subprocess
import sys

import pytest
import torch

import diloco_outer_step_amd as dlc
from tests.test_experts_host import L, balance, outer_norm, step
from tests.test_host_sanitizers import CLANG, ROOT, asan_runtime, hostsan_library
from tests.test_inner_host import F, INVALID, WORKSPACE


# --- merge weights that are a view ----------------------------------------------------------------

def outer_args():
    return dict(codes=torch.zeros((2, 256), dtype=torch.uint8), cb=torch.zeros((2, 3, 256)),
                tensors=[(0, 0, 60), (64, 64, 60), (128, 128, 60)], one=torch.zeros(1, dtype=torch.float64))


@pytest.mark.parametrize("view,match", [
    (torch.zeros((2, 3), dtype=torch.float64).T, "device tensor"),       # only for being on the host
    (torch.zeros((1, 2), dtype=torch.float64).expand(3, 2), "device tensor"),
    (torch.zeros((3, 4), dtype=torch.float64)[:, ::2], "device tensor"),
    (torch.zeros((2, 3)).T, "float64"),
    (torch.zeros((3, 2), dtype=torch.float64).T, "shape"),
    (torch.zeros((3, 2, 1), dtype=torch.float64).transpose(0, 1), "shape"),
])
def test_merge_weights_may_be_a_view_of_the_right_shape_and_type(view, match):
    a = outer_args()
    assert not view.is_contiguous()
    with pytest.raises(ValueError, match=f"(codes|tensor_weights).*{match}"):
        dlc.dlc_outer_grad_norm(a["codes"], a["cb"], [1.0, 1.0], a["tensors"], a["one"], a["one"],
                                torch.zeros(256, dtype=torch.uint8), tensor_weights=view)
    th = torch.zeros(256)
    with pytest.raises(ValueError, match=f"(codes|tensor_weights).*{match}"):
        dlc.dlc_merge_clipped_step(th, th, a["codes"], a["cb"], [1.0, 1.0], a["tensors"], tensor_weights=view)


@pytest.mark.parametrize("tw", [None, F[5]])
def test_weights_whose_sum_is_not_finite_are_refused(tw):
    """Each divided by it would be 0: every learner left out, without a word."""
    for call in (outer_norm, step):
        assert call(w=(1.5e308, 1.5e308), tw=tw) == INVALID and "sum" in dlc.dlc_last_error()


# --- the workspace of the balance loss ---------------------------------------------------------------

def size(k, t, e):
    out = ctypes.c_size_t(0)
    assert L.dlc_expert_balance_workspace_bytes(k, t, e, ctypes.byref(out)) == 0
    return out.value


def need(k, t, e, top, xt, gradient, present=None):
    """What a call asks for; one byte less is refused (a call that needs none takes any address)."""
    wide = dict(t=t, e=e, k=k, xt=xt, top=top, xs=e, xl=t * e, cs=64, cl=64 * t, ml=t, gs=e, gl=t * e, ns=e, ts=e, present=present,
                x=1 << 45, g=1 << 46 if gradient else None, c=1 << 47, mask=1 << 44)
    assert balance(**wide, ws=None, ws_bytes=1 << 62) == WORKSPACE
    n = int(dlc.dlc_last_error().split("need ")[1].split()[0])
    if n:
        assert balance(**wide, ws=1 << 43, ws_bytes=n - 1) == WORKSPACE
    return n


@pytest.mark.parametrize("k,e,longest,short", [(2, 1024, 4211, 3927), (2, 512, 4551, 4096), (3, 128, 6216, 5042)])
def test_the_workspace_of_the_longest_batch_serves_a_shorter_one(k, e, longest, short):
    for xt in (0, 1, 2):
        for gradient in (False, True):
            assert need(k, short, e, 8, xt, gradient) <= size(k, longest, e)


def test_the_workspace_serves_every_smaller_call():
    """Of every type, presence, number of choices, with and without a gradient, up to its tokens, experts and learners."""
    r = random.Random(5)
    for _ in range(400):
        k, e, t = r.randint(1, 64), r.randint(1, 1024), round(2 ** r.uniform(0, 24))
        whole = size(k, t, e)
        for _ in range(10):
            t1 = r.choice((t, r.randint(0, t), max(0, t - r.randint(0, 1000))))
            e1, k1 = r.choice((e, r.randint(1, e))), r.choice((k, r.randint(1, k)))
            present = None if r.random() < 0.3 else [int(i == 0 or r.random() < 0.5) for i in range(k1)]
            top = r.randint(1, min(e1, 64))
            assert need(k1, t1, e1, top, r.randint(0, 2), r.random() < 0.5, present) <= whole, (k, e, t, k1, e1, t1, top)
    for t in range(1, 9000, 7):  # every length below a longest one
        assert need(4, t, 256, 8, 1, False) <= size(4, 9000, 256) and size(4, t, 256) <= size(4, t + 7, 256)


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
