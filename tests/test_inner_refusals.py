"""Calls of the learners' inner step that look right argument by argument and are not: refused before
anything reaches the device.  Addresses of the C calls are never dereferenced.  The same tests run
once more against the library with its host code under the sanitizers."""
import ctypes
import copy
import os
import pickle
import subprocess
import sys

import pytest
import torch

import diloco_outer_step_amd as dlc
from tests.test_host_sanitizers import CLANG, ROOT, asan_runtime, hostsan_library
from tests.test_inner_host import F, INVALID, norm, step

ROW = 4096  # elements of a row in the calls below; two learners


# --- buffers that overlap ----------------------------------------------------------------

@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("bad", [
    dict(m=F[0] + 4 * ROW),                          # the moments' first row is theta's second
    dict(theta=F[2] + 256),
    dict(m=F[3] - 256),                              # the end of one row, the start of another buffer
    dict(grads=F[0] + 2 * 4 * ROW - 256),            # the last elements of the last row
    dict(grads=F[2] + 512, gt=1),                    # 16-bit rows within wider ones
    dict(work=F[0] + 256), dict(work=F[1] + 4 * ROW + 2 * ROW), dict(work=F[3] + 256, wt=2),
    dict(steps=F[0] + 8), dict(steps=F[1] + 2 * 4 * ROW - 8),
    dict(gs=F[6]), dict(gs=F[6] + 8), dict(gs=F[6] - 8), dict(lrs=F[6]), dict(lrs=F[6] - 8),
    dict(gs=F[0] + 4 * ROW), dict(lrs=F[3] + 64),
    dict(present=[0, 1], k=2, grads=F[0] + 256),
])
def test_adamw_refuses_buffers_that_overlap_by_an_offset(coded, bad):
    assert step(coded, **bad) == INVALID and "overlap" in dlc.dlc_last_error()


@pytest.mark.parametrize("bad", [
    dict(ms=F[2] + 256), dict(vs=F[2] + 2 * ROW - 256), dict(vs=F[4] - 0), dict(ms=F[0] + 1024), dict(vs=F[5], ms=F[5]),
    dict(steps=F[4] + 64), dict(gs=F[5] + 8), dict(m=F[4] - 256),
])
def test_the_coded_step_refuses_scale_bytes_that_overlap(bad):
    assert step(True, **bad) == INVALID and "overlap" in dlc.dlc_last_error()


@pytest.mark.parametrize("bad", [
    dict(scale=F[1] + 8), dict(out=F[2] + 8), dict(ws=F[0]), dict(ws=F[0] + 4 * ROW), dict(out=F[3] + 8),
    dict(scale=F[3]), dict(out=F[0] + 800), dict(scale=F[0] + 2 * 4 * ROW - 8), dict(ws=F[1]), dict(ws=F[2]),
])
def test_the_norm_refuses_buffers_that_overlap(bad):
    assert norm(**bad) == INVALID and "overlap" in dlc.dlc_last_error()


# --- eps -----------------------------------------------------------------------------------

@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("eps", [2.0 ** 126 * (1 + 2.0 ** -52), 2.0 ** 127, 3.4e38, 1e300, float("inf"), float("nan"),
                                 2.0 ** -126 * (1 - 2.0 ** -53)])
def test_adamw_refuses_an_eps_whose_reciprocal_is_not_a_normal_number(coded, eps):
    assert step(coded, groups=((1e-3, 0.9, 0.999, eps, 0.0),)) == INVALID and "eps" in dlc.dlc_last_error()


# --- the binding -----------------------------------------------------------------------------

def arguments(monkeypatch, during=lambda args: None):
    """An AdamW call on host tensors that stops before the library: what reaches it. `during` runs in its place."""
    seen = []

    def library(*args):
        during(args)
        seen.append(args)
        return 0

    monkeypatch.setattr(dlc, "_check_buffers", lambda bufs: None)
    monkeypatch.setattr(dlc, "_on_device", lambda index, stream, fn, *args: library(*args))

    def call(tensors, **kw):
        z = [torch.zeros((2, 256)) for _ in range(4)]
        dlc.dlc_adamw_step(*z, torch.zeros(2, dtype=torch.int64), tensors, **kw)
        return seen[-1]

    return call


def test_the_library_reads_group_ids_that_no_other_thread_can_change(monkeypatch):
    ids = dlc.group_ids([0, 1])
    own = ids.buffer_info()[0]

    def another_thread():  # ctypes has released the interpreter's lock by then
        ids[1] = 7
        ids.extend([7] * 100_000)  # moves the array's items

    read = []
    call = arguments(monkeypatch, lambda args: (another_thread(), read.extend((ctypes.c_int32 * 2).from_address(args[11]))))
    q = dlc.AdamWGroup()
    args = call([(0, 0, 64), (64, 64, 64)], groups=[q, q], group_of=ids)
    assert read == [0, 1] and args[11] != own
    assert len(ids) == 100_002


@pytest.mark.parametrize("groups", [
    [(1e-3, 0.9, 0.999, 1e-8), (0.1, 1e-3, 0.9, 0.999, 1e-8, 0.1)],  # ten values, in two entries of the wrong lengths
    [(1e-3, 0.9, 0.999, 1e-8, 0.1, 0.0)] * 5, [(1e-3,)] * 5, [()],
])
def test_every_group_holds_its_five_values(monkeypatch, groups):
    with pytest.raises(ValueError, match="AdamWGroup"):
        arguments(monkeypatch)([(0, 0, 64)], groups=groups)


def test_groups_as_a_single_one_as_a_list_and_as_plain_tuples(monkeypatch):
    call, q = arguments(monkeypatch), dlc.AdamWGroup(0.5, 0.25, 0.125, 1e-8, 2.0)
    for groups, n in ((q, 1), ([q], 1), ((tuple(q), list(q)), 2), ([q] * 16, 16)):
        assert call([(0, 0, 64)], groups=groups)[13] == n


@pytest.mark.parametrize("tensors", [
    [(0, 0, 64, 7), (64, 64, 64, 7), (128, 128, 64, 7)], [(0, 0), (64, 64, 64, 64)], [(0, 0)], [()], [0, 0, 64],
])
def test_every_entry_of_a_tensor_list_holds_three_values(tensors):
    with pytest.raises((ValueError, TypeError)):
        dlc.TensorList(tensors)


def test_a_tensor_list_does_not_follow_its_source():
    rows = [[0, 0, 64], [64, 64, 64]]
    t = dlc.TensorList(rows)
    rows[1][2] = 1 << 20
    assert list(t) == [(0, 0, 64), (64, 64, 64)] and dlc._extents(t) == (128, 128)
    assert dlc._tensors(t)[0][1].numel == 64


@pytest.mark.parametrize("tensors", [[], [(0, 0, 100), (128, 192, 70)]])
def test_a_tensor_list_can_be_pickled_and_copied(tensors):
    t = dlc.TensorList(tensors)
    for again in (pickle.loads(pickle.dumps(t)), copy.copy(t), copy.deepcopy(t)):
        assert type(again) is dlc.TensorList and again == t and dlc._extents(again) == dlc._extents(t)
        (arr, n), (want, _) = dlc._tensors(again), dlc._tensors(t)
        assert n == len(tensors) and bytes(arr) == bytes(want)


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
