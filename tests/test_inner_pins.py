"""The CPU oracle of the learners' inner step (oracle/inner.py), pinned to what fixes it:
hand-computed steps, closed forms under a constant gradient, the 8-bit formats'
values as torch holds them, and the stochastic rounding's mean and independence."""
import math

import numpy as np
import pytest
import torch

from oracle import inner


def rows(*values):
    return np.array(values, np.float32)


def test_the_first_step_moves_every_parameter_by_the_learning_rate():
    # t = 1: m / (1 - b1) = g, v / (1 - b2) = g^2, so the step is lr * g / (|g| + eps)
    theta, g = rows([1.0, 1.0, 1.0]), rows([0.5, -2.0, 0.0])
    m, v, steps = np.zeros_like(theta), np.zeros_like(theta), np.zeros(1, np.int64)
    inner.adamw(theta, g, m, v, steps, [(0, 0, 3)], ((0.1, 0.9, 0.999, 1e-8, 0.0),))
    assert np.allclose(theta, [[0.9, 1.1, 1.0]], rtol=1e-6) and steps[0] == 1
    assert np.allclose(m, [[0.05, -0.2, 0.0]]) and np.allclose(v, [[0.00025, 0.004, 0.0]])


def test_constant_gradients_follow_the_closed_form():
    lr, b1, b2, eps, wd = q = (0.01, 0.9, 0.99, 1e-12, 0.1)
    theta, m, v = np.full((1, 1), 2.0), np.zeros((1, 1)), np.zeros((1, 1))
    steps = np.zeros(1, np.int64)
    want = 2.0
    for t in range(1, 60):
        inner.adamw(theta, np.full((1, 1), 0.3), m, v, steps, [(0, 0, 1)], (q,))
        want = (1 - lr * wd) * want - lr  # m-hat / sqrt(v-hat) = 1
        assert math.isclose(theta[0, 0], want, rel_tol=1e-9)
        assert math.isclose(m[0, 0], 0.3 * (1 - b1 ** t), rel_tol=1e-12)
        assert math.isclose(v[0, 0], 0.09 * (1 - b2 ** t), rel_tol=1e-12)


def test_agrees_with_torch_adamw_in_fp64():
    gen = torch.Generator().manual_seed(0)
    p = torch.randn(50, dtype=torch.float64, generator=gen)
    opt = torch.optim.AdamW([torch.nn.Parameter(p.clone())], lr=0.02, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.3)
    theta, m, v = p.numpy()[None].copy(), np.zeros((1, 50)), np.zeros((1, 50))
    steps = np.zeros(1, np.int64)
    for _ in range(20):
        g = torch.randn(50, dtype=torch.float64, generator=gen)
        opt.param_groups[0]["params"][0].grad = g.clone()
        opt.step()
        inner.adamw(theta, g.numpy()[None], m, v, steps, [(0, 0, 50)], ((0.02, 0.8, 0.95, 1e-6, 0.3),))
    got = opt.param_groups[0]["params"][0].detach().numpy()
    assert np.allclose(theta[0], got, rtol=1e-12, atol=1e-14)


def test_norm_and_scale():
    g = np.array([3.0, 9e9, 4.0], np.float32)  # the middle element belongs to no tensor
    t = [(0, 0, 1), (0, 2, 1)]
    assert inner.grad_norm(g, t) == (5.0, 1.0)
    assert inner.grad_norm(g, t, 0.5, 1.0) == (2.5, 0.2)
    g[2] = np.inf
    assert inner.grad_norm(g, t)[1] == 0.0


@pytest.mark.parametrize("fmt,dtype", [(inner.E4M3, torch.float8_e4m3fn), (inner.E5M2, torch.float8_e5m2)])
def test_formats_decode_as_torch_does(fmt, dtype):
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(dtype).double().numpy()
    assert np.array_equal(fmt.decode(codes), want, equal_nan=True)


@pytest.mark.parametrize("fmt", [inner.E4M3, inner.E5M2])
def test_values_on_the_grid_are_coded_as_themselves_whatever_the_bits(fmt):
    top = int(np.searchsorted(fmt.value[:124], 2.0 ** fmt.top))
    codes = np.arange(top + 1, dtype=np.uint8)
    codes = np.concatenate([codes, codes[::-1], np.full(-2 * len(codes) % 64, top, np.uint8)])
    codes[::64] = top  # every block holds the largest value, so its scale is one
    x = fmt.decode(codes).astype(np.float32)
    for r in (0, 1, 32768, 65535):
        got, byte = inner.encode_blocks(fmt, x, np.full(len(x), r, np.uint64))
        assert np.array_equal(got, codes) and np.all(byte == 127)


@pytest.mark.parametrize("fmt", [inner.E4M3, inner.E5M2])
def test_rounding_is_to_a_neighbour_and_right_on_average(fmt):
    rng = np.random.default_rng(1)
    x = np.exp(rng.uniform(-9, 0, 64)).astype(np.float32) * rng.choice([-1, 1], 64).astype(np.float32)
    total, n = np.zeros(64), 4000
    for t in range(1, n + 1):
        r = inner.random_words(77, t, 0, 0, 64) & np.uint64(0xFFFF)
        codes, byte = inner.encode_blocks(fmt, x, r)
        y = inner.decode_blocks(fmt, codes, byte)
        total += y
        mag = np.abs(x.astype(np.float64)) / inner.scale_of(byte)[0]
        u = 2.0 ** (np.maximum(np.floor(np.log2(mag)), fmt.least) - fmt.mantissa) * inner.scale_of(byte)[0]
        assert np.all(np.abs(y - x) < u)
    # one draw has a deviation of at most u / 2: the mean of n is within 5 u / (2 sqrt(n)) but for one case in a million
    assert np.all(np.abs(total / n - x) <= 5 * u / (2 * math.sqrt(n)))


def test_random_words_are_uniform_and_their_halves_and_neighbours_independent():
    n = 1 << 16
    a = inner.random_words(5, 10, 0, 0, n)
    lo, hi = (a & np.uint64(0xFFFF)).astype(float) / 65536, (a >> np.uint64(16)).astype(float) / 65536
    others = [inner.random_words(5, 11, 0, 0, n), inner.random_words(5, 10, 1, 0, n), inner.random_words(6, 10, 0, 0, n),
              inner.random_words(5 + (1 << 40), 10, 0, 0, n), inner.random_words(5, 10, 0, 1 << 32, n)]
    tail = 5 / math.sqrt(n)
    for h in (lo, hi):
        counts = np.bincount((h * 64).astype(int), minlength=64)
        assert np.sum((counts - n / 64) ** 2 / (n / 64)) < 63 + 5 * math.sqrt(2 * 63)
    pairs = [(lo, hi), (lo[1:], lo[:-1]), (hi[1:], hi[:-1]), (lo[64:], lo[:-64])]
    pairs += [(lo, (o & np.uint64(0xFFFF)).astype(float)) for o in others]
    for x, y in pairs:
        assert abs(np.corrcoef(x, y)[0, 1]) < tail


def test_a_second_moment_decays_on_average_though_each_step_is_below_the_grid():
    # g = 0: v shrinks by 1 - b2 = 1/1000 a step, a hundredth of the format's step
    theta, g = np.zeros((1, 4096), np.float32), np.zeros((1, 4096), np.float32)
    mc, ms = np.zeros((1, 4096), np.uint8), np.zeros((1, 64), np.uint8)
    vc, vs = np.full((1, 4096), 0x70, np.uint8), np.full((1, 64), 100, np.uint8)
    start = inner.decode_blocks(inner.E5M2, vc[0], vs[0]).mean()
    steps = np.zeros(1, np.int64)
    for _ in range(200):
        inner.adamw_coded(theta, g, mc, ms, vc, vs, steps, [(0, 0, 4096)])
    now = inner.decode_blocks(inner.E5M2, vc[0], vs[0]).mean()
    # per element, 200 roundings of deviation at most u sqrt(f (1 - f)), f ~ 0.008, u <= v / 4: under 0.35 v in all;
    # the mean of 4096 within 5 * 0.35 / 64 = 0.028
    assert abs(now / start / 0.999 ** 200 - 1) < 0.03


def test_a_positive_second_moment_is_never_coded_as_zero():
    v32 = np.full(64, 1e-30, np.float32)
    v32[0] = 1.0
    theta, g = np.zeros((1, 64), np.float32), np.full((1, 64), 1e-12, np.float32)
    g[0, 0] = 1.0
    mc, ms = np.zeros((1, 64), np.uint8), np.zeros((1, 1), np.uint8)
    vc, vs = np.zeros((1, 64), np.uint8), np.zeros((1, 1), np.uint8)
    inner.adamw_coded(theta, g, mc, ms, vc, vs, np.zeros(1, np.int64), [(0, 0, 64)])
    assert np.all(vc[0, 1:] == 1) and vc[0, 0] > 1
